"""The device of a cache, without launches: tensors of several devices are
refused, and so is a cache on another device than a call's tensors."""
import ctypes

import pytest
import torch

from gated_deltanet_linear_04_gb300 import workloads as wl

BF16, I32 = torch.bfloat16, torch.int32
E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu


@pytest.fixture(scope="module")
def attn():
    from gated_deltanet_linear_04_gb300.build import build_library
    build_library()
    from gated_deltanet_linear_04_gb300 import attn as a
    return a


def test_tensors_of_two_devices(attn):
    k = torch.zeros((4, 2, 16, 64), dtype=BF16)
    with pytest.raises(ValueError, match="v is on meta, k on cpu"):
        attn.KVCache(k, k.to("meta"))
    # (also without pages, where no address is looked at)
    none = torch.zeros((0, 2, 16, 64), dtype=E4M3)
    scale = torch.zeros((0, 2, 16), dtype=torch.uint8).view(E8M0)
    for i in range(3):
        rest = [none, scale, scale]
        rest[i] = torch.empty(rest[i].shape, dtype=rest[i].dtype, device="meta")
        with pytest.raises(ValueError, match="is on meta"):
            attn.KVCache(none, *rest)
    assert attn.KVCache(none, none, scale, scale)._c.device == -1


def test_record_holds_the_device(attn):
    """The layout that the binding reads: the ABI's struct, then three i32."""
    r = attn._CacheRecord
    base = ctypes.sizeof(attn.GdnKvCache)
    assert [(n, getattr(r, n).offset) for n in ("Hkv", "D", "device")] == [("Hkv", base), ("D", base + 4), ("device", base + 8)]


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True])
def test_cache_on_another_device(attn, fp8):
    """A record that says another device (there is one GPU here): every call is
    refused before anything is queued."""
    d = wl.AttnDims(1, 1, 2, 1, 64, 0)
    cache = attn.KVCache.empty(d, 2, 16, E4M3 if fp8 else BF16, "cuda:0")
    assert cache._c.device == 0
    cache._c.device = 1
    q = torch.zeros((1, 1, 2, 64), dtype=BF16, device="cuda:0")
    k = q[:, :, :1].contiguous()
    table, pos = torch.zeros((1, 1), dtype=I32, device="cuda:0"), torch.zeros(1, dtype=I32, device="cuda:0")
    before = cache.k.view(torch.uint8).clone()
    with pytest.raises(ValueError, match="another device"):
        attn.kv_append(d, q, k + 1, k + 1, None, None, None, cache, table, pos)
    with pytest.raises(ValueError, match="another device"):
        attn.kv_read(d, cache, table, pos)
    with pytest.raises(ValueError, match="another device"):
        attn.attn_decode(d, q, cache, table, pos)
    assert torch.equal(cache.k.view(torch.uint8), before)
