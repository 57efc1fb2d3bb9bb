"""Calls on a given stream while the current one is busy: outputs and scratch
belong to the call's stream, inputs are ready before it."""
import pytest
import torch

from gated_deltanet_linear_04_gb300 import workloads as wl
from tests.test_gpu_attn import DEV, I32, attn, gen, make_cache, normal, status, tables, to_dev, weights  # noqa: F401

pytestmark = pytest.mark.gpu

BUSY = 100_000_000      # clocks that the current stream is kept busy: some 50 ms


def calls(attn):  # noqa: F811
    """name -> f(stream) -> dict of outputs."""
    B, P = 4, 16
    d = wl.AttnDims(B, 1, 16, 2, 256, 64)
    dt = d.with_(T=600)
    g = gen(31)
    cache = make_cache(attn, d, 200, P, True, g)
    table = tables(g, B, 50, 200).to(DEV)
    pos = torch.tensor([700, 30, 411, 90], dtype=I32, device=DEV)
    q1 = normal(g, B, 1, 16, 256).to(DEV)
    q, k, v = (normal(g, B, 600, h, 256).to(DEV) for h in (16, 2, 2))
    wq, wk = to_dev(*weights(g, d))
    fr = attn.rope_freqs(attn.rope_inv_freq(64), DEV)
    at = torch.arange(600, dtype=I32, device=DEV).expand(B, 600).contiguous()
    zero = torch.zeros(B, dtype=I32, device=DEV)
    spare = make_cache(attn, d, 200, P, True)
    return {
        "norm_rope": lambda s: dict(zip("qk", attn.qk_norm_rope(dt, q, k, wq, wk, fr, at, stream=s))),
        "norm_rope_backward": lambda s: attn.qk_norm_rope_backward(dt, q, k, wq, wk, fr, at, q, k, stream=s),
        "append": lambda s: {"q": attn.kv_append(dt, q, k, v, wq, wk, fr, spare, table, zero, stream=s)},
        "read": lambda s: dict(zip("kv", attn.kv_read(dt, cache, table, zero, stream=s))),
        "decode": lambda s: dict(zip(("out", "lse"), attn.attn_decode(d, q1, cache, table, pos, return_lse=True,
                                                                      stream=s))),
    }


@pytest.mark.parametrize("given", ["Stream", "handle"])
@pytest.mark.parametrize("name", ["norm_rope", "norm_rope_backward", "append", "read", "decode"])
def test_outputs_are_not_taken_from_work_on_the_current_stream(attn, name, given):  # noqa: F811
    call = calls(attn)[name]
    want = call(None)
    side = torch.cuda.Stream()
    stream = side if given == "Stream" else side.cuda_stream
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    # blocks of the outputs' sizes, given back while a fill and a copy of them are still queued behind a long wait
    blocks = [torch.empty_like(t) for t in want.values()]
    copies = [torch.empty_like(t) for t in want.values()]
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    for b, c in zip(blocks, copies):
        b.fill_(3.0)
        c.copy_(b)
    taken = {b.data_ptr() for b in blocks}
    del blocks, b
    got = call(stream)
    assert not taken & {t.data_ptr() for t in got.values()}
    torch.cuda.synchronize()
    for n in want:
        assert torch.equal(got[n], want[n]), n
    assert all(torch.all(c == 3.0) for c in copies)
    assert status() == 0


def test_outputs_outlive_their_use_on_the_current_stream(attn):  # noqa: F811
    """An output of a side stream that the current stream reads late and the
    caller lets go of: the next call on the side stream does not write it."""
    call = calls(attn)["norm_rope"]
    want = call(None)["q"]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    out = call(side)["q"]
    side.synchronize()
    out.fill_(5.0)
    late = torch.empty_like(out)
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    late.copy_(out)
    del out
    again = call(side)["q"]
    torch.cuda.synchronize()
    assert torch.equal(again, want) and torch.all(late == 5.0)


def test_a_given_stream_inside_a_capture(attn):  # noqa: F811
    """A side stream forked into a capture and joined again."""
    every = calls(attn)
    want = {n: f(None) for n, f in every.items()}
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        got = {n: f(side) for n, f in every.items()}
        torch.cuda.current_stream().wait_stream(side)
    graph.replay()
    torch.cuda.synchronize()
    for n in want:
        for x in want[n]:
            assert torch.equal(got[n][x], want[n][x]), (n, x)
