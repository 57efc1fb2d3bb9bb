"""attn_decode where scores, keys, queries or gates are not finite: what a
token sees goes into its output and log-sum-exp, NaN included; zeros and -inf
are for tokens that see no key."""
import math

import pytest
import torch

from gated_deltanet_linear_04_gb300 import workloads as wl
from tests import _attn_ref as R
from tests.test_gpu_attn import BF16, DEV, I32, attn, check_decode, gen, make_cache, normal, status, tables  # noqa: F401

pytestmark = pytest.mark.gpu


def raw(t):
    return t.view(torch.uint8) if t.element_size() == 1 else t.view(torch.int16)


def nan_bits(t):
    return 0x7f if t.element_size() == 1 else 0x7fc0


def put(t, table, b, positions, value):
    """The bits `value` into every channel of the positions' rows."""
    P = t.shape[2]
    at = torch.as_tensor(list(positions))
    page = table[b, at // P].long()
    raw(t)[page.to(DEV), :, (at % P).to(DEV)] = value


def call(attn, d, q, cache, table, pos, **kw):  # noqa: F811
    out, lse = attn.attn_decode(d, q.to(DEV), cache, table.to(DEV), torch.tensor(pos, dtype=I32, device=DEV),
                                return_lse=True, **kw)
    return out.cpu(), lse.cpu()


def is_nan(t):
    return bool(torch.all(torch.isnan(t.float())))


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("Hq,Hkv,D,pos", [(8, 2, 64, [40, 0, 200]), (16, 2, 256, [3, 90, 0]), (4, 1, 128, [50000, 7, 9])])
def test_nan_query(attn, Hq, Hkv, D, pos, fp8, bad):  # noqa: F811
    """One channel of one query row that is not finite: that row's result is
    NaN, the others keep their bits."""
    B, T, P = 3, 2, 16
    d = wl.AttnDims(B, T, Hq, Hkv, D)
    g = gen(D + Hq)
    width = -(-(max(pos) + T) // P)
    cache = make_cache(attn, d, B * width + 1, P, fp8, g)
    table = tables(g, B, width, B * width + 1)
    q = normal(g, B, T, Hq, D)
    want, want_lse = call(attn, d, q, cache, table, pos)
    check_decode(want, want_lse, q, cache, table, pos, None, D ** -0.5)
    for b, t, h in ((0, 0, 1), (1, 1, Hq - 1), (2, 0, 0)):
        q2 = q.clone()
        q2[b, t, h, 5] = bad
        out, lse = call(attn, d, q2, cache, table, pos)
        assert is_nan(out[b, t, h])
        if math.isnan(bad):
            assert is_nan(lse[b, t, h])
        out[b, t, h], lse[b, t, h] = want[b, t, h], want_lse[b, t, h]
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
    assert status() == 0


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_nan_in_the_only_key(attn, D, fp8):  # noqa: F811
    B, P = 3, 16
    d = wl.AttnDims(B, 1, 8, 2, D)
    g = gen(D)
    cache = make_cache(attn, d, 4, P, fp8, g)
    table = tables(g, B, 1, 4)
    q, pos = normal(g, B, 1, 8, D), [0, 0, 4]
    want, want_lse = call(attn, d, q, cache, table, pos)
    put(cache.k, table, 1, [0], nan_bits(cache.k))
    out, lse = call(attn, d, q, cache, table, pos)
    assert is_nan(out[1]) and is_nan(lse[1])
    for b in (0, 2):
        assert torch.equal(out[b], want[b]) and torch.equal(lse[b], want_lse[b])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("first,last", [(0, 20000), (20000, 45000), (40000, 60001)])
def test_nan_keys_of_whole_shares(attn, first, last, fp8):  # noqa: F811
    """A stretch of NaN keys longer than what one CTA takes of the row: parts
    that are NaN throughout are joined with finite ones."""
    P, pos = 64, [60000, 30000]
    d = wl.AttnDims(2, 1, 8, 1, 64)
    g = gen(first + 1)
    width = -(-(max(pos) + 1) // P)
    cache = make_cache(attn, d, 2 * width, P, fp8, g)
    table = tables(g, 2, width, 2 * width)
    q = normal(g, 2, 1, 8, 64)
    want, want_lse = call(attn, d, q, cache, table, pos)
    put(cache.k, table, 0, range(first, last), nan_bits(cache.k))
    out, lse = call(attn, d, q, cache, table, pos)
    assert is_nan(out[0]) and is_nan(lse[0])
    assert torch.equal(out[1], want[1]) and torch.equal(lse[1], want_lse[1])


@pytest.mark.parametrize("fp8", [False, True])
def test_nan_keys_on_the_borders_of_shares(attn, fp8):  # noqa: F811
    """A row of two tiles (256 keys of 64 channels) for each SM, the list's two
    blank slots counted: the stretch of NaN ends where shares end, so that no
    part holds NaN and finite scores."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    P, n = 64, (2 * sms - 2) * 256
    d = wl.AttnDims(1, 1, 8, 1, 64)
    g = gen(21)
    cache = make_cache(attn, d, n // P, P, fp8, g)
    table = tables(g, 1, n // P, n // P)
    q = normal(g, 1, 1, 8, 64)
    clean = attn.KVCache(*(None if t is None else t.clone() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale)))
    out, lse = call(attn, d, q, cache, table, [n - 1])
    check_decode(out, lse, q, clean, table, [n - 1], None, 0.125)
    put(cache.k, table, 0, range(18 * 256, 118 * 256), nan_bits(cache.k))
    out, lse = call(attn, d, q, cache, table, [n - 1])
    assert is_nan(out) and is_nan(lse)


@pytest.mark.parametrize("first,last", [(0, 20000), (20000, 45000), (0, 60001)])
def test_scores_of_minus_infinity(attn, first, last):  # noqa: F811
    """Keys whose score is -inf weigh nothing; a row with no others is 0 / 0."""
    P, pos = 16, [60000]
    d = wl.AttnDims(1, 1, 8, 1, 64)
    g = gen(first + 2)
    first, last = first // P * P, -(-last // P) * P
    width = -(-(max(pos) + 1) // P)
    cache = make_cache(attn, d, width, P, False, g)
    table = tables(g, 1, width, width)
    q = normal(g, 1, 1, 8, 64)
    q[..., 0] = 1.0
    none = table.clone()
    none[0, first // P:last // P] = -1
    cpu = attn.KVCache(cache.k.clone(), cache.v.clone())
    stretch = torch.arange(first, min(last, pos[0] + 1))
    raw(cache.k)[table[0, stretch // P].long().to(DEV), :, (stretch % P).to(DEV), 0] = -128          # 0xff80
    out, lse = call(attn, d, q, cache, table, pos)
    if last > pos[0]:
        assert is_nan(out) and torch.all(lse == -math.inf)
    else:
        check_decode(out, lse, q, cpu, none, pos, None, 0.125)      # as if these keys were not there
    assert status() == 0


@pytest.mark.parametrize("fp8", [False, True])
def test_rows_of_bad_pages_see_nothing(attn, fp8):  # noqa: F811
    """Stretches without pages, over whole shares and over whole rows."""
    from gated_deltanet_linear_04_gb300 import gdn
    P, pos = 16, [40000, 30000, 60]
    d = wl.AttnDims(3, 1, 8, 1, 64)
    g = gen(3)
    width = -(-(max(pos) + 1) // P)
    cache = make_cache(attn, d, 3 * width, P, fp8, g)
    table = tables(g, 3, width, 3 * width)
    table[0, 300:1800] = -1
    table[1:] = -1
    q = normal(g, 3, 1, 8, 64)
    gate = torch.full_like(q, math.nan).to(DEV)
    out, lse = call(attn, d, q, cache, table, pos)
    assert status() == gdn.GDN_ERR_BAD_PAGE
    check_decode(out, lse, q, cache, table, pos, None, 0.125)
    assert torch.all(out[1:] == 0) and torch.all(lse[1:] == -math.inf)
    assert status() == 0
