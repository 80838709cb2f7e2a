"""Values that the 8-bit cache meets at its edges, on a B200: pages blanked by their
scale, elements that are not finite, rows of NaN in attention, and long walks of the
tensor-memory tiles.

Codes and scales are decisions of exact arithmetic and have to be equal; the
attention's tolerance is that of test_cache8_gpu.
"""

import math

import numpy as np
import pytest

import token_ref as ref
from test_cache8_gpu import TYPES, check_attend, f64, filled_cache, ints, tables

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from io_aware_exact_30_b200 import attn  # noqa: E402


def page_after(rows, held, old):
    """(codes of the held slots, codes of the rows, scale) of one page and head after
    rows (n, d) came behind the held codes: the definition, an element that is not
    finite left out of the scale and stored as NaN."""
    fine = np.isfinite(rows)
    s = max(ref.page_scale(float(np.abs(np.where(fine, rows, 0)).max())), old if len(held) else 0.0)
    new = np.where(fine, ref.e4m3_round(np.where(fine, rows, 0) / s) if s else 0.0, np.nan)
    return (ref.e4m3_round(held * (old / s)) if s > old else held), new, s


def append_and_compare(k, v, cache, page_id, fill):
    """Appends k, v (1, Hkv, T, d) behind the first `fill` slots of a page; compares
    codes (where the scale is 0 and stays 0, the values) and scales with page_after."""
    before = [f64(x) for x in cache]
    T = k.shape[2]
    attn.cache_append(k, v, cache, ints([[page_id]]), ints([fill]))
    assert attn.attn_last_device_status() == 0
    for i, x in ((0, k), (1, v)):
        codes, scale = f64(cache[i])[page_id], f64(cache[i + 2])[page_id]
        for h in range(k.shape[1]):
            held, new, s = page_after(f64(x)[0, h], before[i][page_id, h, :fill], before[i + 2][page_id, h])
            assert scale[h] == s
            assert np.array_equal(codes[h, :fill], held, equal_nan=True), cache._fields[i]
            assert np.array_equal(codes[h, fill:fill + T], new, equal_nan=True), cache._fields[i]
            assert np.array_equal(codes[h, fill + T:], before[i][page_id, h, fill + T:])


@pytest.mark.parametrize("page,d,dtype,fill,T", [(16, 64, "bf16", 2, 1), (32, 128, "fp16", 31, 1),
                                                 (64, 128, "bf16", 7, 40), (128, 64, "fp16", 100, 28)])
def test_append_behind_tokens_of_a_zero_scale(page, d, dtype, fill, T):
    """Tokens whose page has scale 0 stand for zeros, whatever their codes; they still
    do when a new token brings the page a scale."""
    cache = filled_cache(3, 2, page, d, 50)
    cache.k_scale[1, 0] = 0.0
    cache.v_scale[1, 1] = 0.0
    g = torch.Generator().manual_seed(51)
    k, v = (torch.randn(1, 2, T, d, generator=g).to(TYPES[dtype]).cuda() for _ in range(2))
    append_and_compare(k, v, cache, 1, fill)
    for codes, h in ((cache.k, 0), (cache.v, 1)):
        assert (codes[1, h, :fill].float() == 0).all()


def test_append_of_zeros_behind_tokens_of_a_zero_scale():
    """The scale stays 0: the held tokens' values do too."""
    cache = filled_cache(2, 1, 16, 64, 52)
    cache.k_scale.zero_(), cache.v_scale.zero_()
    x = torch.zeros(1, 1, 2, 64, device="cuda").bfloat16()
    append_and_compare(x, x, cache, 0, 3)
    x = x + 1
    append_and_compare(x, x, cache, 0, 5)
    assert (cache.k[0, 0, :5].float() == 0).all()


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("where", [(4,), (7,), (4, 7), tuple(range(64))])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("fill", [0, 5])
def test_append_of_elements_that_are_not_finite(bad, where, dtype, fill):
    """They become NaN codes and cost the page's other elements nothing: neither those
    of the same token, nor its neighbours, nor the tokens held before.  The largest
    finite value stands in an even and in an odd feature."""
    page, d = 32, 64
    g = torch.Generator().manual_seed(53)
    for top in (6, 11):
        cache = filled_cache(2, 2, page, d, 54)
        k, v = (torch.randn(1, 2, 6, d, generator=g) * 0.1 for _ in range(2))
        k[0, 0, 3, top], v[0, 1, 0, top] = 30.0, -50.0
        k[0, 0, 2, list(where)] = bad
        v[0, 1, 5, list(where)] = bad
        k, v = (x.to(TYPES[dtype]).cuda() for x in (k, v))
        append_and_compare(k, v, cache, 1, fill)
        assert torch.isnan(cache.k[1, 0, fill + 2].float()).sum() == len(where)


def test_drafts_in_front_of_a_token_of_nan_read_on_after_it_is_taken_back():
    """Five drafted tokens, the fourth NaN; with the length set back to the first three,
    attention is exact over what they hold."""
    page, d = 32, 128
    cache = filled_cache(4, 2, page, d, 55)
    g = torch.Generator().manual_seed(56)
    k, v = (torch.randn(1, 2, 5, d, generator=g).bfloat16().cuda() for _ in range(2))
    k[:, :, 3], v[:, :, 3] = math.nan, math.nan
    table = ints([[2, 0, 3, 1]])
    attn.cache_append(k, v, cache, table, ints([40]))
    for Hq in (2, 24):
        q = torch.randn(1, Hq, 3, d, generator=g).bfloat16().cuda()
        check_attend(q, cache, table, [43])


@pytest.mark.parametrize("Hq,T,lens", [(2, 2, [30, 600]),         # fragments of 8 rows, one split and several
                                       (12, 1, [30, 600]),        # of 16
                                       (40, 1, [30, 2000]),       # tiles
                                       (1, 1, [1, 9000])])
def test_attention_of_a_query_of_nan_is_nan(Hq, T, lens):
    """O and the log-sum-exp of a row that holds a NaN or sees a NaN key are NaN: a
    caller who joins parts by their log-sum-exp must not take it for a row that sees
    nothing (-inf).  The other rows stay right."""
    page, d, B = 16, 128, 2
    P, table = tables(B, -(-max(lens) // page), 57)
    cache = filled_cache(P, 1, page, d, 58)
    q = torch.randn(B, Hq, T, d, generator=torch.Generator().manual_seed(59)).bfloat16().cuda()
    first = [x[0].clone() for x in attn.cache_attend(q, cache, table, ints(lens))]
    bad = q.clone()
    bad[1, 0, T - 1, 17] = math.nan
    o, lse = attn.cache_attend(bad, cache, table, ints(lens))
    assert torch.isnan(o[1, 0, T - 1]).all() and torch.isnan(lse[1, 0, T - 1])
    # (which row moves the reference of a warp's rows may change their last bits)
    want, lse_w, weight, mag = ref.attend(f64(q), *(f64(x) for x in cache), table.cpu().numpy(), lens, [T] * B,
                                          True, 1 / math.sqrt(d))
    delta = 2.0 ** -16 * mag
    tol = torch.finfo(q.dtype).eps / 2 * np.abs(want) + (2.0 ** -11 + 2 * delta[..., None]) * weight
    same = np.ones((B, Hq, T), bool)
    same[1, 0, T - 1] = False
    assert np.all((np.abs(f64(o) - want) <= tol)[same])
    with np.errstate(invalid="ignore"):
        assert np.all(((np.abs(f64(lse) - lse_w) <= delta + 2.0 ** -20) | (f64(lse) == lse_w))[same])
    # a key of NaN in the first page of the longer sequence, seen by all its rows
    cache.k.view(torch.uint8)[table[1, 0].long(), 0, 0, 5] = 0x7F
    o, lse = attn.cache_attend(q, cache, table, ints(lens))
    assert torch.isnan(o[1]).all() and torch.isnan(lse[1]).all()
    assert torch.equal(o[0], first[0]) and torch.equal(lse[0], first[1])
    assert attn.attn_last_device_status() == 0


@pytest.mark.parametrize("d,Hq,dtype", [(64, 40, "bf16"), (128, 40, "fp16")])
def test_attend_tiles_over_thousands_of_keys_a_cta(d, Hq, dtype):
    """A bound of the lengths that is far too low leaves the last split of the
    tensor-memory tiles more than 64 tiles: pages and scales looked up in batches of 32
    tiles, each page with a scale of its own, a bad page right behind a batch's end."""
    page, n = 16, 9100
    P, table = tables(1, -(-n // page), 60)
    cache = filled_cache(P, 1, page, d, 61, spread=6)
    q = torch.randn(1, Hq, 1, d, generator=torch.Generator().manual_seed(62)).to(TYPES[dtype]).cuda()
    whole = check_attend(q, cache, table, [n])
    check_attend(q, cache, table, [n], max_len=600)
    check_attend(q, cache, table, [n - 13], max_len=1)  # one split
    for entry in (512 // 16 + 32 * 8, 512 // 16 + 32 * 8 - 1, 32 * 8, 64 * 8 + 3):
        table[0, entry] = P + 5
    check_attend(q, cache, table, [n], max_len=600, bad=True)
    check_attend(q, cache, table, [n], max_len=1, bad=True)
    again = attn.cache_attend(q, cache, table.clamp(max=P - 1), ints([n]))  # the same sizes still run
    assert attn.attn_last_device_status() == 0 and again[0].shape == whole[0].shape


@pytest.mark.parametrize("Hq,Hkv,T,n", [(16, 16, 1, 4096), (32, 8, 1, 3000), (16, 2, 5, 5001), (8, 1, 1, 700)])
def test_calls_repeat_themselves_bit_for_bit(Hq, Hkv, T, n):
    page, d, B = 64, 128, 4
    P, table = tables(B, -(-n // page), 63)
    cache = filled_cache(P, Hkv, page, d, 64)
    q = torch.randn(B, Hq, T, d, generator=torch.Generator().manual_seed(65)).bfloat16().cuda()
    lens = ints([n, n // 2, n // 3, T])
    want = [x.clone() for x in attn.cache_attend(q, cache, table, lens)]
    for _ in range(20):
        for a, b in zip(attn.cache_attend(q, cache, table, lens), want):
            assert torch.equal(a, b)
