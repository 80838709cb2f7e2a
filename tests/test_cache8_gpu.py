"""The 8-bit paged cache on a B200 against its 64-bit reference.

Codes and scales are decisions of exact arithmetic (a power-of-two scale, one
rounding): they have to be equal.  The attention's tolerance, per element:
  o    half a step of its type of |o|, plus (2^-11 + 2 delta) sum_j p_j |v_j|: the
       probabilities reach the product rounded to 16 bits (half a step of fp16,
       2^-11), and an error delta of the scores moves each by up to its share
  lse  delta + 2^-20
  delta = 2^-16 max_j scale sum |q k_j|: fp32 sums of up to 128 products (128 2^-24
       of their magnitude) and as much again for the exponent's own arithmetic.
"""

import math

import numpy as np
import pytest

import token_ref as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from io_aware_exact_30_b200 import attn  # noqa: E402

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def f64(t):
    return t.double().cpu().numpy()


def filled_cache(P, Hkv, page, d, seed, spread=3):
    """A cache of random codes, scales some binades apart."""
    g = torch.Generator().manual_seed(seed)
    c = attn.cache_alloc(P, Hkv, page, d)
    for codes, scale in ((c.k, c.k_scale), (c.v, c.v_scale)):
        codes.copy_((torch.randn(P, Hkv, page, d, generator=g) * 60).to(torch.float8_e4m3fn))
        scale.copy_(torch.exp2(-torch.randint(5, 5 + spread, (P, Hkv), generator=g).float()))
    return c


def tables(B, width, seed, spare=3):
    g = torch.Generator().manual_seed(seed)
    P = B * width + spare
    return P, torch.randperm(P, generator=g)[:B * width].to(torch.int32).view(B, width).cuda()


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def check_append(k, v, cache, table, lens, n_new, bad=False):
    want = [f64(x) for x in cache]
    ns = [k.shape[2]] * k.shape[0] if n_new is None else n_new
    got_bad = [ref.append(f64(x), want[i], want[i + 2], table.cpu().numpy(), lens, ns, cache.k.shape[0])
               for i, x in ((0, k), (1, v))]
    assert got_bad == [bad, bad]
    attn.cache_append(k, v, cache, table, ints(lens), None if n_new is None else ints(n_new))
    assert attn.attn_last_device_status() == (-11 if bad else 0)
    for name, g, w in zip(cache._fields, cache, want):
        assert np.array_equal(f64(g), w), name


@pytest.mark.parametrize("page,d,dtype,Hkv,T", [
    (16, 64, "bf16", 1, 1), (16, 128, "fp16", 3, 5), (32, 64, "fp16", 2, 33), (32, 128, "bf16", 2, 31),
    (64, 64, "bf16", 2, 65), (64, 128, "fp16", 1, 130), (128, 64, "fp16", 2, 129), (128, 128, "bf16", 2, 200)])
def test_append_codes_and_scales(page, d, dtype, Hkv, T):
    B, width = 5, -(-(2 * page + T) // page)
    P, table = tables(B, width, 1)
    cache = filled_cache(P, Hkv, page, d, 2)
    g = torch.Generator().manual_seed(3)
    # rows a few binades apart, so that pages outgrow what they held
    k, v = ((torch.randn(B, Hkv, T, d, generator=g) * torch.exp2(torch.randint(-4, 5, (B, Hkv, T, 1), generator=g).float()))
            .to(TYPES[dtype]).cuda() for _ in range(2))
    lens = [0, 1, page - 1, page, 2 * page - 3]
    check_append(k, v, cache, table, lens, None)
    check_append(k, v, cache, table, lens, [T, 0, min(1, T), T - 1, T])


def test_append_values_of_the_types_ends():
    page, d = 16, 64
    P, table = tables(4, 2, 1)
    for name, dt in TYPES.items():
        cache = attn.cache_alloc(P, 1, page, d)
        top = torch.finfo(dt).max
        rows = torch.zeros(4, 1, 3, d)
        rows[0, 0, 1] = torch.linspace(-1, 1, d) * top
        rows[1, 0, 2, 5] = torch.finfo(dt).tiny
        rows[2, 0, 0, 7] = -torch.finfo(dt).smallest_normal / 8
        x = rows.to(dt).cuda()
        check_append(x, -x, cache, table, [0, 3, 15, 16], None)  # sequence 3 stores zeros


def test_append_token_by_token_outgrows_its_page():
    page, d = 32, 128
    P, table = tables(1, 2, 4)
    cache = attn.cache_alloc(P, 2, page, d)
    g = torch.Generator().manual_seed(5)
    for t in range(40):
        x = (torch.randn(1, 2, 1, d, generator=g) * 1.3 ** t).bfloat16().cuda()
        check_append(x, (x.float() * 1.1 ** -t).bfloat16(), cache, table, [t], None)


def test_append_bad_pages_and_lengths_are_not_followed():
    page, d, B, T = 16, 64, 6, 20
    P, table = tables(B, 3, 6)
    table[1, 1] = P          # past the cache
    table[2, 0] = -1
    table[3, 2] = 2 ** 30
    cache = filled_cache(P, 2, page, d, 7)
    x = torch.randn(B, 2, T, d, device="cuda").bfloat16()
    # sequence 4 runs past its table, sequence 5 has a length below 0
    check_append(x, x + 1, cache, table, [3, 9, 0, 20, 40, -1], None, bad=True)
    check_append(x, x + 1, cache, table, [3, 0, 17, 0, 0, 0], [1, 1, 1, 1, T + 1, -1], bad=True)
    assert attn.attn_last_device_status() == 0  # cleared on read


def check_attend(q, cache, table, lens, causal=True, q_lens=None, scale=None, bad=False, **kw):
    B, Hq, T, d = q.shape
    sc = 1 / math.sqrt(d) if scale is None else scale
    qf, nq = f64(q), [T] * B if q_lens is None else q_lens
    want, lse_w, weight, mag = ref.attend(qf, *(f64(x) for x in cache), table.cpu().numpy(), lens, nq,
                                          causal, sc)
    o = torch.full_like(q, 7.0)
    lse = torch.full((B, Hq, T), 7.0, device="cuda")
    cap = kw.get("max_len") or table.shape[1] * cache.k.shape[2]
    need = attn.attn_cache_attend_workspace_bytes(B, Hq, cache.k.shape[1], T, d, cap)
    ws = torch.full((max(need, 16),), 255, dtype=torch.uint8, device="cuda")  # NaN in every word
    attn.attn_cache_attend(q, cache, table, ints(lens), o, lse, ws, causal, scale,
                           None if q_lens is None else ints(q_lens), **kw)
    assert attn.attn_last_device_status() == (-11 if bad else 0)
    got, lse_g = f64(o), f64(lse)
    skip = np.isnan(want)
    assert np.all(got[skip] == 7.0) and np.all(lse_g[np.isnan(lse_w)] == 7.0)  # left as they were
    delta = 2.0 ** -16 * mag
    tol = torch.finfo(q.dtype).eps / 2 * np.abs(want) + (2.0 ** -11 + 2 * delta[..., None]) * weight
    off = np.where(skip, 0, np.abs(np.where(skip, 0, got - want)) - tol)
    assert np.all(np.isfinite(got)) and off.max() <= 1e-30, off.max()
    seen = np.isfinite(lse_w)
    assert np.all(np.abs(lse_g[seen] - lse_w[seen]) <= delta[seen] + 2.0 ** -20)
    assert np.all(lse_g[np.isneginf(lse_w)] == -np.inf) and np.all(got[np.isneginf(lse_w)] == 0)
    return o, lse


@pytest.mark.parametrize("page,d,dtype,Hq,Hkv,T,lens", [
    (16, 64, "bf16", 1, 1, 1, [1]),
    (16, 64, "fp16", 6, 2, 1, [17, 16, 15, 0, 300]),
    (32, 128, "bf16", 8, 1, 1, [64, 33, 31, 1, 200]),
    (64, 128, "fp16", 4, 4, 1, [64, 65, 63, 2, 129]),
    (128, 64, "bf16", 32, 2, 1, [127, 128, 129, 255, 1000]),
    (64, 128, "bf16", 10, 2, 4, [4, 3, 70, 500, 1]),       # rows that see nothing
    (32, 64, "fp16", 6, 2, 7, [7, 40, 33, 900, 0]),
    (128, 128, "fp16", 3, 1, 17, [17, 128, 400, 16, 18]),
    (16, 128, "bf16", 40, 1, 2, [77, 16, 2, 1, 48]),
    (64, 64, "fp16", 2, 1, 70, [70, 300, 64, 1, 130]),
])
@pytest.mark.parametrize("causal", [True, False])
def test_attend(page, d, dtype, Hq, Hkv, T, lens, causal):
    B = len(lens)
    P, table = tables(B, -(-max(lens) // page) + 1, 8)
    cache = filled_cache(P, Hkv, page, d, 9)
    g = torch.Generator().manual_seed(10)
    q = torch.randn(B, Hq, T, d, generator=g).to(TYPES[dtype]).cuda()
    check_attend(q, cache, table, lens, causal)
    check_attend(q, cache, table, lens, causal, q_lens=[min(i, T) for i in range(B)], scale=0.3)


@pytest.mark.parametrize("Hq,Hkv,T,d,page", [(1, 1, 1, 128, 16), (8, 1, 1, 64, 128), (8, 2, 3, 128, 64),
                                             (2, 2, 1, 64, 16)])
def test_attend_long_sequences_are_split(Hq, Hkv, T, d, page):
    lens = [5000, 129, 12345]
    P, table = tables(3, -(-max(lens) // page) + 2, 11)
    cache = filled_cache(P, Hkv, page, d, 12)
    q = torch.randn(3, Hq, T, d, generator=torch.Generator().manual_seed(13)).bfloat16().cuda()
    a = check_attend(q, cache, table, lens)
    # a bound that is too low or far too high changes the split, never the keys seen
    for m in (12345, 100, 1 << 20):
        check_attend(q, cache, table, lens, max_len=m)
    b = check_attend(q, cache, table, lens)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])  # no order of arrival in it


def test_attend_scales_far_apart_and_masked_garbage():
    """Pages whose scales lie 2^60 apart, zero pages, a huge page that no weight
    falls on, and NaN codes in slots past the last token and in pages that no
    sequence names."""
    page, d, Hq = 16, 128, 4
    P, table = tables(2, 5, 14)
    cache = filled_cache(P, 1, page, d, 15)
    lens = [70, 33]
    t = table.cpu().long()
    cache.v_scale[t[0, 1]] = 2.0 ** -40
    cache.v_scale[t[0, 2]] = 2.0 ** 20
    cache.v_scale[t[1, 0]] = 0.0
    cache.k_scale[t[0, 3]] = 0.0
    cache.k_scale[t[0, 2]] = 2.0 ** -30
    free = torch.ones(P, dtype=torch.bool)
    free[t.flatten()] = False
    for c in (cache.k.view(torch.uint8), cache.v.view(torch.uint8)):
        c[free.cuda()] = 0x7F
        c[t[0, 4], :, lens[0] - 64:] = 0x7F
        c[t[1, 2], :, lens[1] - 32:] = 0x7F
        c[t[1, 3]] = 0xFF
    q = torch.randn(2, Hq, 3, d, generator=torch.Generator().manual_seed(16)).bfloat16().cuda()
    check_attend(q, cache, table, lens)
    check_attend(q * 1e-3, cache, table, lens, causal=False)
    cache.k_scale.mul_(2.0 ** 6)  # one key takes all the weight
    check_attend(q, cache, table, lens)


@pytest.mark.parametrize("d,dtype,Hq,T", [(128, "bf16", 12, 3), (64, "bf16", 40, 2), (128, "fp16", 6, 13)])
def test_attend_many_rows(d, dtype, Hq, T):
    """More than 16 rows of a key/value head (tensor-memory tiles): long sequences in
    several splits, sequences shorter than their queries, pages that end inside a
    tile, scales 2^60 apart, zero and bad pages, garbage past the last token."""
    lens = [1500, T - 1, 129, 0, 3000, 640]
    page, B = 16, len(lens)
    P, table = tables(B, 190, 40)
    cache = filled_cache(P, 1, page, d, 41)
    t = table.cpu().long()
    if dtype == "bf16":
        cache.v_scale[t[0, 3]] = 2.0 ** -40
        cache.v_scale[t[0, 60]] = 2.0 ** 20
    cache.v_scale[t[4, :9]] = 0.0
    cache.k_scale[t[4, 20:40]] = 0.0
    for c in (cache.k.view(torch.uint8), cache.v.view(torch.uint8)):
        c[t[2, 8], :, lens[2] - 128:] = 0x7F
        c[t[5, 40:]] = 0xFF
    q = torch.randn(B, Hq, T, d, generator=torch.Generator().manual_seed(42)).to(TYPES[dtype]).cuda()
    for causal in (True, False):
        check_attend(q, cache, table, lens, causal)
        check_attend(q, cache, table, lens, causal, q_lens=[T, 1, 0, T, 2, T - 1], max_len=700)
    table[4, 100], table[0, 0] = -7, P
    check_attend(q, cache, table, lens, bad=True)


def test_attend_scores_that_climb_past_every_reference():
    """Keys whose scores grow by hundreds of log2 units from tile to tile, first far
    below, then far above where a row began: the weight ends on the last ones."""
    for Hq in (4, 20):
        page, d, n = 64, 128, 640
        P, table = tables(1, n // page, 43)
        cache = filled_cache(P, 1, page, d, 44)
        order = table.cpu().long()[0]
        for i, pg in enumerate(order):
            cache.k_scale[pg] = 2.0 ** (-6 + i)
        q = torch.randn(1, Hq, 1, d, generator=torch.Generator().manual_seed(45)).bfloat16().cuda()
        check_attend(q, cache, table, [n])
        for i, pg in enumerate(order):
            cache.k_scale[pg] = 2.0 ** (3 - i)
        check_attend(q, cache, table, [n])
        cache.k.copy_(cache.k.float().abs().to(torch.float8_e4m3fn))
        for sign in (-1, 1):
            check_attend(sign * q.abs(), cache, table, [n - 13])


def test_attend_of_values_of_two_to_the_64():
    """The largest values the sums are sized for, under scores that climb from tile to
    tile by just less than moves a reference."""
    page, d, n = 64, 128, 640
    for Hq in (4, 40):
        P, table = tables(1, n // page, 46)
        cache = filled_cache(P, 1, page, d, 47)
        cache.k.copy_(cache.k.float().abs().to(torch.float8_e4m3fn))
        for i, pg in enumerate(table.cpu().long()[0]):
            cache.k_scale[pg] = 2.0 ** (-9 + i / 2 // 1)
            cache.v_scale[pg] = 2.0 ** 55  # codes to 448: 2^64
        q = torch.randn(1, Hq, 1, d, generator=torch.Generator().manual_seed(48)).bfloat16().cuda()
        check_attend(q.abs(), cache, table, [n])


def test_attend_bad_pages_are_not_seen():
    page, d = 32, 64
    P, table = tables(4, 4, 17)
    table[0, 1], table[1, 0], table[2, 3] = P, -5, 2 ** 31 - 1
    cache = filled_cache(P, 2, page, d, 18)
    q = torch.randn(4, 4, 2, d, generator=torch.Generator().manual_seed(19)).bfloat16().cuda()
    check_attend(q, cache, table, [100, 20, 128, 50], bad=True)
    good = torch.arange(16, dtype=torch.int32, device="cuda").view(4, 4)
    check_attend(q, cache, good, [100, 129, -3, 128], bad=True)  # lengths are clamped
    check_attend(q, cache, good, [100, 20, 3, 50], q_lens=[2, 3, 1, -1], bad=True)


def test_decoding_token_by_token_is_attention_of_the_whole():
    """A prompt and then single tokens through append and attend give, at every
    step, exact attention over the values the cache stands for."""
    B, Hq, Hkv, d, page, N = 3, 6, 2, 128, 32, 45
    prompt = [20, 1, 33]
    P, table = tables(B, 4, 20)
    cache = attn.cache_alloc(P, Hkv, page, d)
    g = torch.Generator().manual_seed(21)
    k, v = (torch.randn(B, Hkv, N + 20, d, generator=g).bfloat16().cuda() for _ in range(2))
    q = torch.randn(B, Hq, N + 20, d, generator=g).bfloat16().cuda()
    lens = ints(prompt)
    top = max(prompt)
    attn.cache_append(k[:, :, :top].contiguous(), v[:, :, :top].contiguous(), cache, table,
                      torch.zeros_like(lens), lens)
    now = list(prompt)
    for step in range(6):
        pick = lambda x: torch.stack([x[b, :, now[b]] for b in range(B)])[:, :, None].contiguous()  # noqa: E731
        check_append(pick(k), pick(v), cache, table, now, None)
        now = [n + 1 for n in now]
        check_attend(pick(q), cache, table, now)


def test_captured_and_on_another_stream():
    """Append and attend captured in one graph, replayed for the next tokens, and
    the same calls on a side stream."""
    B, Hq, Hkv, d, page = 2, 4, 2, 64, 16
    P, table = tables(B, 90, 22)
    g = torch.Generator().manual_seed(23)
    xs = [[torch.randn(B, h, 1, d, generator=g).half().cuda() for h in (Hq, Hkv, Hkv)] for _ in range(4)]
    lens0 = ints([900, 14])

    def fresh():
        return filled_cache(P, Hkv, page, d, 24)

    def eager(cache):
        lens, got = lens0.clone(), []
        for q, k, v in xs:
            attn.cache_append(k, v, cache, table, lens)
            lens += 1
            got.append([t.clone() for t in attn.cache_attend(q, cache, table, lens)])
        return got

    want = eager(fresh())
    side = torch.cuda.Stream()
    cache = fresh()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = eager(cache)
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(want, got):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])

    cache, lens = fresh(), lens0.clone()
    q, k, v = (x.clone() for x in xs[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        attn.cache_append(k, v, cache, table, lens)
        lens += 1
        o, lse = attn.cache_attend(q, cache, table, lens)
    for a, x in zip(want, xs):
        for dst, src in zip((q, k, v), x):
            dst.copy_(src)
        graph.replay()
        assert torch.equal(a[0], o) and torch.equal(a[1], lse)
    assert attn.attn_last_device_status() == 0


def test_two_attends_at_once_do_not_share_anything():
    d, page = 128, 64
    P, table = tables(2, 60, 25)
    cache = filled_cache(P, 2, page, d, 26)
    q = torch.randn(2, 2, 8, 1, d, generator=torch.Generator().manual_seed(27)).bfloat16().cuda()
    lens = ints([3800, 2222])
    want = [[t.clone() for t in attn.cache_attend(x, cache, table, lens)] for x in q]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        got = []
        for x, s in zip(q, streams):
            with torch.cuda.stream(s):
                got.append(attn.cache_attend(x, cache, table, lens))
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_a_cache_past_two_to_the_31_codes():
    """Pages at the far end of a cache of more than 2^31 codes."""
    page, d, Hkv = 128, 128, 16
    P = (1 << 31) // (page * d * Hkv) + 4
    cache = attn.cache_alloc(P, Hkv, page, d)
    B = 2
    table = torch.tensor([[P - 1, 0], [P - 2, P - 3]], dtype=torch.int32, device="cuda")
    g = torch.Generator().manual_seed(28)
    k, v = (torch.randn(B, Hkv, 140, d, generator=g).bfloat16().cuda() for _ in range(2))
    lens = ints([0, 3])
    attn.cache_append(k, v, cache, table, lens)
    small = attn.Cache8(*(t[[0, P - 3, P - 2, P - 1]].contiguous() for t in cache))
    to = torch.tensor([[3, 0], [2, 1]], dtype=torch.int32, device="cuda")
    again = attn.cache_alloc(4, Hkv, page, d)
    attn.cache_append(k, v, again, to, lens)
    for a, b in zip(small, again):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    q = torch.randn(B, Hkv, 1, d, generator=g).bfloat16().cuda()
    full = ints([140, 143])
    a, b = attn.cache_attend(q, cache, table, full), attn.cache_attend(q, again, to, full)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
