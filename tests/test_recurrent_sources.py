"""What the sources of the kernels around a recurrent layer must not do, checked on their text (as
tests/test_tail_sources.py does for the update tail's)."""
import re

import pytest

from tests.test_tail_sources import _arguments, _source

# What a caller hands in and no kernel of the call writes.  (w0, w1: rows of the weight; bias + col: the
# bias; w + col: a norm's weight, through rows.cuh.)
INPUTS = {"block_norm.cu": {"p.r1", "p.r2", "w"}, "rows.cuh": {"w"},
          "linear.cu": {"bias", "w0", "w1", "p.x", "p.ep.bias", "p.dy", "p.z"}}


@pytest.mark.parametrize("name", sorted(INPUTS))
def test_read_only_loads_read_only_inputs(name):
    """ld.global.nc wants memory that nothing writes while the kernel runs: dz, pieces of sums and partial
    sums, which an earlier kernel of the call leaves, and a residual that is written over in place are loaded plainly."""
    seen = set()
    for a in _arguments(_source(name), "__ldg"):
        a = re.sub(r"^reinterpret_cast<[^>]*>\(", "", a)
        seen.add(re.match(r"[\w.]+", a).group(0))
    assert seen and seen <= INPUTS[name], seen - INPUTS[name]


def test_published_values_go_around_the_first_level_cache():
    """What the scan's blocks leave for one another is written and read with relaxed accesses of the whole
    GPU, never by plain loads, which may be served from a block's own cache."""
    text = _source("scan.cu")
    for name in ("p.inc", "p.agg"):
        assert name in text
        plain = [line for line in text.splitlines() if name in line and not re.search(
            r"look\(|publish\(|float2 \*agg =|p\.inc = |p\.agg = ", line)]
        assert plain == []
    assert text.count("ld.relaxed.gpu") == 2 and text.count("st.relaxed.gpu") == 2
