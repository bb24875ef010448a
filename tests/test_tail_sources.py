"""What the sources of the update-tail kernels must not do, checked on their text: faults of this
kind show only once in a while, so that no run of a kernel is a test for them."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "prefix_shared_chunkwise_gb300", "csrc")


def _source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def _arguments(text, call):
    """The first argument of every call of a function, with the parentheses inside it."""
    for m in re.finditer(re.escape(call) + r"\(", text):
        depth, i = 1, m.end()
        while depth:
            depth += {"(": 1, ")": -1}.get(text[i], 0)
            i += 1
        yield text[m.end():i - 1]


# What a caller hands in and no kernel of the call writes.  (px, pw: rows of x and weight; q: a
# gradient's values; w: the norm's weight.)
INPUTS = {"rmsnorm.cu": {"w", "p.rstd"}, "grad_clip.cu": {"q"},
          "linear_logprob.cu": {"px", "pw", "p.x", "p.row_ptr", "p.row_sem", "p.target", "p.dlogp"}}


@pytest.mark.parametrize("name", sorted(INPUTS))
def test_read_only_loads_read_only_inputs(name):
    """ld.global.nc wants memory that nothing writes while the kernel runs.  Kernels that overlap
    with the one before them read that one's results, which are therefore loaded plainly."""
    seen = set()
    for a in _arguments(_source(name), "__ldg"):
        a = re.sub(r"^reinterpret_cast<[^>]*>\(", "", a)
        seen.add(re.match(r"[\w.]+", a).group(0))
    assert seen and seen <= INPUTS[name], seen - INPUTS[name]
