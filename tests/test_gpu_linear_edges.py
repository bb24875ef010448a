"""harts_linear_fwd / _bwd where calls differ in what they share and in how many tiles a block goes through."""
import pytest

torch = pytest.importorskip("torch")
pytest.importorskip("scipy")

from prefix_shared_chunkwise_gb300.api import linear_fwd
from tests.test_gpu_linear import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from prefix_shared_chunkwise_gb300 import build
    build.build()


@pytest.mark.parametrize("kind", ["none", "silu", "gelu"])
@pytest.mark.parametrize("C,K,N", [(1, 520, 264), (2, 520, 264), (3, 520, 264), (100, 2048, 72), (2000, 520, 264)])
def test_z_over_the_residual(C, K, N, kind):
    """A residual is read before either output is written, whichever kernel the number of rows leads to."""
    c = Case(C, K, N, True, True)
    y, z = linear_fwd(c.x, c.w, c.b, c.res, activation=kind, keep_z=True)
    res = c.res.clone()
    y2, z2 = linear_fwd(c.x, c.w, c.b, res, activation=kind, z=res)
    assert z2 is res and torch.equal(z2, z) and torch.equal(y2, y)
