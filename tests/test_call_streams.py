"""Buffers that a call of the binding makes belong to the stream that it is given: one made on the
current stream is handed out again, as soon as the call returns, to work that does not wait for
the given stream's kernels."""
import inspect

import pytest

torch = pytest.importorskip("torch")

from prefix_shared_chunkwise_gb300 import api


class Entered(Exception):
    pass


CALLS = [n for n in api.__all__ if inspect.isfunction(getattr(api, n)) and n != "device_error"
         and "stream" in inspect.signature(getattr(api, n)).parameters]


@pytest.mark.parametrize("name", CALLS)
def test_a_call_enters_its_stream_first(name, monkeypatch):
    def enter(stream):
        assert stream == "given"
        raise Entered
    monkeypatch.setattr(torch.cuda, "stream", enter)
    call = getattr(api, name)
    kinds = [p for p in inspect.signature(call).parameters.values() if p.default is p.empty]
    positional = [None for p in kinds if p.kind is p.POSITIONAL_OR_KEYWORD]
    named = {p.name: None for p in kinds if p.kind is p.KEYWORD_ONLY}
    with pytest.raises(Entered):
        call(*positional, **named, stream="given")


def test_every_call_is_looked_at():
    assert {"kda_fwd", "kda_bwd", "conv_bwd", "attn_bwd", "logprob_bwd", "rmsnorm_bwd", "linear_logprob_bwd"} <= set(CALLS)


@pytest.mark.gpu
def test_workspaces_of_busy_streams_are_not_handed_out():
    """Backward passes on a second stream that is still busy, their workspaces dropped at once: what
    the current stream then allocates and fills must not reach them.  The same kernels in the same
    order of sums: equal to the bit."""
    import numpy as np
    from prefix_shared_chunkwise_gb300 import build
    from prefix_shared_chunkwise_gb300.synth import make_inputs
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    build.build()
    pl = api.Plan(np.array([-1, 0, 0], np.int32), np.array([150, 90, 70], np.int64), 64).upload()
    C = pl.info["C"]
    gen = torch.Generator().manual_seed(3)
    q, k, v, d = (torch.randn(C, 1, 128, generator=gen).bfloat16().cuda() for _ in range(4))
    cw, cb = torch.randn(128, 4, generator=gen).cuda(), torch.randn(128, generator=gen).cuda()
    kx = make_inputs(C, 1, 128, 128, "bf16", 0, device="cuda")
    cs = torch.empty(pl.chunk_state_bytes(1, 128, 128, 1) // 2, dtype=torch.bfloat16, device="cuda")

    def calls(stream):
        torch.cuda.synchronize()
        if stream is not None:
            with torch.cuda.stream(stream):
                torch.cuda._sleep(20_000_000)
        o, lse = api.attn_fwd(pl, q, k, v, stream=stream)
        out = [o, lse, *api.attn_bwd(pl, q, k, v, o, lse, d, stream=stream)]
        out += api.conv_bwd(pl, q, cw, cb, d, stream=stream)
        x = [kx[n] for n in ("q", "k", "v", "g", "beta")]
        ko, states, _, _ = api.kda_fwd(pl, *x, chunk_states=cs, stream=stream)
        out += [ko, *api.kda_bwd(pl, *x, kx["W"], states=states, chunk_states=cs, stream=stream).values()]
        junk = [torch.full((n,), 0x7f, dtype=torch.uint8, device="cuda")
                for n in (256, 4096, 1 << 16, 1 << 18, 1 << 20, 1 << 22) for _ in range(8)]
        torch.cuda.synchronize()
        del junk
        return out

    here, there = calls(None), calls(torch.cuda.Stream())
    assert pl.device_error() == 0
    for a, b in zip(here, there):
        assert torch.equal(a, b)
