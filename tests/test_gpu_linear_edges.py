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


# More tiles than workers, so that a pair of blocks goes on to a third tile and its accumulators are used again
# (152 SMs, tiles of 256 x 256: 4.5 - 4.75 a pair forward; backward 4 and a half of dweight's and then dx's; the last one has
# pairs that take one of dx's ahead of the others), with more than sixteen tiles along the side that is walked first, not
# a multiple of it (19 of 19, 18 of 19; 18 of 19 for dweight).
@pytest.mark.parametrize("C,K,N", [(4700, 64, 4616), (4360, 40, 4616), (9000, 64, 2312)])
@pytest.mark.parametrize("kind,bias,res,keep", [("gelu", True, True, True), ("none", False, False, False), ("silu", True, False, True)])
def test_forward_of_many_tiles(C, K, N, kind, bias, res, keep):
    c = Case(C, K, N, bias, res)
    y, z = c.check_forward(kind, keep)
    other = Case(C, K, N, bias, res, seed=1)
    linear_fwd(other.x, other.w, other.b, other.res, activation=kind, keep_z=keep, y=torch.empty_like(y))
    y2, z2 = linear_fwd(c.x, c.w, c.b, c.res, activation=kind, keep_z=keep)
    assert torch.equal(y, y2) and (z is None or torch.equal(z, z2))


@pytest.mark.parametrize("C,K,N,kind,bias", [(700, 4616, 4360, "gelu", True), (700, 4616, 4360, "none", False), (3000, 4616, 2600, "silu", True)])
def test_backward_of_many_tiles(C, K, N, kind, bias):
    c = Case(C, K, N, bias, False)
    _, z = linear_fwd(c.x, c.w, c.b, activation=kind, keep_z=kind != "none")
    c.check_backward(kind, z, bias)
