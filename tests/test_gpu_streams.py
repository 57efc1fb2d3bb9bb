"""The delta-rule calls on a given stream while the current one is busy: outputs
and scratch belong to the call's stream, inputs are ready before it."""
import pytest
import torch

from gated_deltanet_linear_04_gb300 import workloads as wl

pytestmark = pytest.mark.gpu

BUSY = 100_000_000      # clocks that the current stream is kept busy: some 50 ms
DEV = "cuda:0"


@pytest.fixture(scope="module")
def gdn():
    from gated_deltanet_linear_04_gb300.build import build_library
    build_library()
    from gated_deltanet_linear_04_gb300 import gdn as g
    assert torch.cuda.is_available(), "these tests need a GPU"
    torch.cuda.set_device(0)
    g.gdn_device_status()
    yield g
    assert g.gdn_device_status() == g.GDN_OK


def calls(gdn):
    """name -> f(stream) -> outputs."""
    d = wl.Dims(B=2, T=300, Hk=2, Hv=4, Dk=128, Dv=128, K=4)
    w = {k: v.to(DEV) for k, v in wl.workload_inputs(wl.WORKLOADS["tiny"], d).items() if isinstance(v, torch.Tensor)}
    one, few = d.with_(T=1), d.with_(T=4)
    cut = {n: {k: w[k][:, :n].contiguous() for k in ("qkv", "a", "b")} for n in (1, 4)}
    q, k, v = gdn.conv_update(d, w["qkv"], w["conv_w"])
    g, beta = gdn.gating(d, w["a"], w["b"], w["A_log"], w["dt_bias"])
    norm, z1 = torch.ones(d.Dv, device=DEV), v[:, :1].contiguous()
    gvec = g[..., None].expand(*g.shape, d.Dk).contiguous()

    def decode(f, dims, n, s, *rest, **kw):
        c = cut[n]
        return [f(dims, c["qkv"], w["conv_w"], fresh["conv_state"], c["a"], c["b"], w["A_log"], w["dt_bias"],
                  fresh["state"], *rest, stream=s, **kw)]

    # (the caches that a step advances are copied before the current stream gets busy)
    fresh = {}

    def renew():
        fresh.update(conv_state=w["conv_state"].clone(), state=w["state"].clone())

    table = {
        "conv_update": lambda s: gdn.conv_update(d, w["qkv"], w["conv_w"], stream=s),
        "gating": lambda s: gdn.gating(d, w["a"], w["b"], w["A_log"], w["dt_bias"], stream=s),
        "recurrent_decode": lambda s: decode(gdn.recurrent_decode, one, 1, s),
        "recurrent_decode_gated": lambda s: decode(gdn.recurrent_decode_gated, one, 1, s, z1, norm),
        "decode_window": lambda s: decode(gdn.decode_window, few, 4, s),
        "prefill": lambda s: gdn.prefill(d, q, k, v, g, beta, stream=s),
        "prefill_chunked": lambda s: gdn.prefill(d, q, k, v, g, beta, chunk=64, stream=s),
        "prefill_gated": lambda s: gdn.prefill_gated(d, q, k, v, g, beta, v, norm, stream=s),
        "prefill_vec": lambda s: gdn.prefill_vec(d, q, k, v, gvec, beta, stream=s),
        "prefill_backward": lambda s: list(gdn.prefill_backward(d, q, k, v, g, beta, v, stream=s).values()),
        "prefill_backward_chunked":
            lambda s: list(gdn.prefill_backward(d, q, k, v, g, beta, v, chunk=64, stream=s).values()),
        "rmsnorm_gated": lambda s: [gdn.rmsnorm_gated(d, v, v, norm, stream=s)],
    }
    return table, renew


NAMES = ["conv_update", "gating", "recurrent_decode", "recurrent_decode_gated", "decode_window", "prefill",
         "prefill_chunked", "prefill_gated", "prefill_vec", "prefill_backward", "prefill_backward_chunked",
         "rmsnorm_gated"]


def alike(name, got, want):
    """Equal bits; of the backward pass, whose f32 sums come in any order
    (atomics), a few thousand terms within 2^-24 each."""
    if "backward" not in name:
        return torch.equal(got, want)
    return bool(torch.all((got - want).abs() <= 2.0 ** -12 * want.abs().max()))


@pytest.mark.parametrize("given", ["Stream", "handle"])
@pytest.mark.parametrize("name", NAMES)
def test_outputs_are_not_taken_from_work_on_the_current_stream(gdn, name, given):
    table, renew = calls(gdn)
    renew()
    want = table[name](None)
    renew()
    side = torch.cuda.Stream()
    stream = side if given == "Stream" else side.cuda_stream
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    # blocks of the outputs' sizes, given back while a fill and a copy of them are still queued behind a long wait
    blocks = [torch.empty_like(t) for t in want]
    copies = [torch.empty_like(t) for t in want]
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    for b, c in zip(blocks, copies):
        b.fill_(3.0)
        c.copy_(b)
    taken = {b.data_ptr() for b in blocks}
    del blocks, b
    got = table[name](stream)
    assert not taken & {t.data_ptr() for t in got}
    torch.cuda.synchronize()
    assert all(alike(name, x, y) for x, y in zip(got, want))
    assert all(torch.all(c == 3.0) for c in copies)
