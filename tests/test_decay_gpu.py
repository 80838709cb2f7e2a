"""Linear attention with a decay for each head on a B200 against its 64-bit
reference.

Tolerances, relative L2 per head.  A 16-bit result passes three roundings to its
type (the in-chunk weights, the state's copy for the tensor cores, the result),
each uniform within half a step eps/2 and so eps/2/sqrt(3) in L2; three independent
ones make eps/2.  A head of few tokens has too few roundings to average: the weight of
a single token is one number, its rounding, up to eps/2, is the whole row's, and the
result's own comes on top, so there each of the three counts in full, 3 eps/2.  States
are fp32; their terms reach the tensor cores in 16-bit pieces (2^-16 of a term at most),
and fp32 sums of n terms add about sqrt(n) 2^-24: 2e-5.  A step rounds its result once and its state by a few 2^-24.
"""

import math

import numpy as np
import pytest

import token_ref as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from io_aware_exact_30_b200 import attn  # noqa: E402

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
STATE_TOL = 2e-5


def f64(t):
    return t.double().cpu().numpy()


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


FEW = 16


def close(got, want, tol, label, chunked=True):
    """Every head's relative L2; NaN in `want` marks rows that hold 7 still."""
    top = tol
    for b in range(want.shape[0]):
        for h in range(want.shape[1]):
            g, w = got[b, h], want[b, h]
            gone = np.isnan(w)
            tol = 3 * top if chunked and (~gone[:, 0]).sum() < FEW else top
            assert np.all(g[gone] == 7.0), f"{label} {(b, h)}: a row past the end was written"
            g, w = g[~gone], w[~gone]
            assert np.all(np.isfinite(g)), f"{label} {(b, h)}"
            norm = np.linalg.norm(w)
            assert np.linalg.norm(g - w) <= tol * norm, \
                f"{label} {(b, h)}: {np.linalg.norm(g - w) / max(norm, 1e-300)} > {tol}"


def inputs(B, H, N, d, dtype, seed, n=4):
    g = torch.Generator().manual_seed(seed)
    x = [torch.randn(B, H, N, d, generator=g).to(TYPES[dtype]).cuda() for _ in range(n)]
    s = [torch.randn(B, H, d, d, generator=g).cuda() for _ in range(2)]
    return x, s


def decays(H):
    """Memories from none to all."""
    some = [-0.004, 0.0, -1.0, -math.inf, -0.05, -1e-7, -20.0]
    return torch.tensor([some[h % 7] for h in range(H)], dtype=torch.float32, device="cuda")


def half(dtype):
    return torch.finfo(TYPES[dtype]).eps / 2


SHAPES = [(1, 1, 1, 64, "bf16"), (1, 2, 1, 128, "fp16"), (2, 3, 127, 64, "fp16"), (1, 3, 128, 128, "bf16"),
          (2, 2, 129, 128, "fp16"), (1, 7, 300, 64, "bf16"), (1, 2, 700, 128, "bf16"),
          (1, 3, 1100, 64, "fp16"), (2, 20, 200, 128, "bf16"), (1, 1, 2000, 128, "fp16"),
          (4, 40, 130, 64, "bf16")]


def pick(B, H):
    """Heads that the reference computes."""
    return slice(0, min(B, 2)), slice(0, 7)


@pytest.mark.parametrize("B,H,N,d,dtype", SHAPES)
@pytest.mark.parametrize("with_state", [True, False])
def test_forward(B, H, N, d, dtype, with_state):
    (q, k, v, _), (s0, _) = inputs(B, H, N, d, dtype, N)
    ld = decays(H)
    o, s1 = attn.decay_forward(q, k, v, ld, state=s0 if with_state else None)
    assert attn.attn_last_device_status() == 0
    bs, hs = pick(B, H)
    a = [f64(x[bs, hs]) for x in (q, k, v)]
    st = f64(s0[bs, hs]) * (1 if with_state else 0)
    want, s_want = ref.decay_forward(*a, f64(ld)[hs], st, [N] * a[0].shape[0], 1 / math.sqrt(d))
    close(f64(o[bs, hs]), want, half(dtype), "o")
    close(f64(s1[bs, hs]), s_want, STATE_TOL, "state")
    # the heads that were not compared follow the same arithmetic
    assert torch.isfinite(o.float()).all() and torch.isfinite(s1).all()


@pytest.mark.parametrize("B,H,N,d,dtype", SHAPES)
@pytest.mark.parametrize("with_state", [True, False])
def test_backward(B, H, N, d, dtype, with_state):
    (q, k, v, do), (s0, ds) = inputs(B, H, N, d, dtype, N + 1)
    ld = decays(H)
    got = attn.decay_backward(q, k, v, ld, do, state=s0 if with_state else None,
                              dstate=ds if with_state else None)
    assert attn.attn_last_device_status() == 0
    bs, hs = pick(B, H)
    a = [f64(x[bs, hs]) for x in (q, k, v)]
    on = 1 if with_state else 0
    want = ref.decay_backward(*a, f64(ld)[hs], f64(do[bs, hs]), f64(s0[bs, hs]) * on, f64(ds[bs, hs]) * on,
                              [N] * a[0].shape[0], 1 / math.sqrt(d))
    for name, g, w in zip(("dq", "dk", "dv"), got, want):
        close(f64(g[bs, hs]), w, half(dtype), name)
    close(f64(got[3][bs, hs]), want[3], STATE_TOL, "dstate")


@pytest.mark.parametrize("d,dtype,H", [(64, "fp16", 2), (128, "bf16", 3), (128, "fp16", 20)])
def test_padded_batch(d, dtype, H):
    """Lengths of every kind; the rows past them hold NaN and stay as they were."""
    lens = [0, 1, 127, 128, 129, 400, 385]
    B, N = len(lens), 400
    (q, k, v, do), (s0, ds) = inputs(B, H, N, d, dtype, 30)
    for x in (q, k, v, do):
        for b, n in enumerate(lens):
            x[b, :, n:] = math.nan
    ld = decays(H)
    hs = slice(0, 2)
    a = [np.nan_to_num(f64(x[:, hs])) for x in (q, k, v)]
    ws = [torch.full((max(16, attn.attn_decay_workspace_bytes(B, H, N, d, back)),), 255, dtype=torch.uint8,
                     device="cuda") for back in (False, True)]
    o, s1 = torch.full_like(q, 7.0), torch.empty_like(s0)
    attn.attn_decay_fwd(q, k, v, ld, o, s0, s1, ints(lens), ws[0])
    assert attn.attn_last_device_status() == 0
    want, s_want = ref.decay_forward(*a, f64(ld)[hs], f64(s0[:, hs]), lens, 1 / math.sqrt(d))
    close(f64(o[:, hs]), want, half(dtype), "o")
    close(f64(s1[:, hs]), s_want, STATE_TOL, "state")
    assert torch.equal(s1[0], s0[0])  # no token: the state passes unchanged
    assert attn.decay_forward(q, k, v, ld, state=s0, lens=ints(lens))[0][1, :, 1:].abs().sum() == 0

    got = [torch.full_like(q, 7.0) for _ in range(3)] + [torch.empty_like(s0)]
    attn.attn_decay_bwd(q, k, v, ld, do, *got[:3], s0, ds, got[3], ints(lens), ws[1])
    assert attn.attn_last_device_status() == 0
    want = ref.decay_backward(*a, f64(ld)[hs], np.nan_to_num(f64(do[:, hs])), f64(s0[:, hs]), f64(ds[:, hs]),
                              lens, 1 / math.sqrt(d))
    for name, g, w in zip(("dq", "dk", "dv"), got, want):
        close(f64(g[:, hs]), w, half(dtype), name)
    close(f64(got[3][:, hs]), want[3], STATE_TOL, "dstate")
    assert torch.equal(got[3][0], ds[0])


def test_lengths_are_clamped():
    (q, k, v, _), (s0, _) = inputs(3, 1, 50, 64, "bf16", 31)
    ld = decays(1)
    a = attn.decay_forward(q, k, v, ld, state=s0, lens=ints([99, -4, 50]))
    b = attn.decay_forward(q, k, v, ld, state=s0, lens=ints([50, 0, 50]))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("B,H,d,dtype", [(1, 1, 64, "bf16"), (3, 2, 128, "fp16"), (1, 16, 128, "bf16"),
                                         (64, 5, 64, "fp16"), (40, 16, 128, "bf16")])
def test_step(B, H, d, dtype):
    (q, k, v, _), (s0, _) = inputs(B, H, 1, d, dtype, 32)
    ld = decays(H)
    want, s_want = ref.decay_forward(f64(q), f64(k), f64(v), f64(ld), f64(s0), [1] * B, 0.3)
    o, s1 = attn.decay_step(q, k, v, ld, s0, 0.3)
    close(f64(o), want, half(dtype), "o", chunked=False)
    close(f64(s1), s_want, 2.0 ** -22, "state")
    keep = s0.clone()
    o2, s2 = attn.decay_step(q, k, v, ld, keep, 0.3, state_out=keep)  # in place
    assert s2 is keep and torch.equal(o, o2) and torch.equal(s1, keep)


@pytest.mark.parametrize("d,dtype", [(64, "fp16"), (128, "bf16")])
def test_prompt_then_tokens_is_the_whole_sequence(d, dtype):
    """Prefill of a padded batch of prompts, then single tokens, against one
    prefill of everything; and a prefill in two parts, the state updated in place."""
    B, H, N, lens = 3, 4, 260, [250, 129, 3]
    (q, k, v, _), (s0, _) = inputs(B, H, N, d, dtype, 33)
    ld = decays(H)
    want, s_want = ref.decay_forward(f64(q), f64(k), f64(v), f64(ld), f64(s0), [n + 6 for n in lens],
                                     1 / math.sqrt(d))
    state = s0.clone()
    attn.attn_decay_fwd(q, k, v, ld, torch.empty_like(q), state, state, ints(lens),
                        torch.empty(max(16, attn.attn_decay_workspace_bytes(B, H, N, d)), dtype=torch.uint8,
                                    device="cuda"))
    for i in range(6):
        cut = lambda x: torch.stack([x[b, :, n + i] for b, n in enumerate(lens)])[:, :, None].contiguous()  # noqa: E731
        o, _ = attn.decay_step(cut(q), cut(k), cut(v), ld, state, state_out=state)
        now = np.stack([want[b, :, n + i] for b, n in enumerate(lens)])[:, :, None]
        close(f64(o), now, half(dtype), f"token {i}", chunked=False)
    close(f64(state), s_want, STATE_TOL, "state")


def test_hybrid_decoder_layers_run_together():
    """A softmax layer over the 8-bit cache and a decayed linear layer decode the
    same tokens in one captured graph, each after its own prompt form."""
    B, H, d, page, n0 = 2, 4, 128, 16, 40
    (q, k, v, _), (s0, _) = inputs(B, H, n0 + 8, d, "bf16", 34)
    ld = decays(H)
    table = torch.arange(2 * 4, dtype=torch.int32, device="cuda").view(2, 4)
    cache = attn.cache_alloc(8, H, page, d)
    head = [x[:, :, :n0].contiguous() for x in (q, k, v)]
    attn.forward(*head, causal=True)
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    attn.cache_append(head[1], head[2], cache, table, lens)
    lens += n0
    o_lin, state = attn.decay_forward(*head, ld)
    now = [x[:, :, n0:n0 + 1].clone() for x in (q, k, v)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        attn.cache_append(now[1], now[2], cache, table, lens)
        lens += 1
        a, _ = attn.cache_attend(now[0], cache, table, lens)
        b, _ = attn.decay_step(*now, ld, state, state_out=state)
    f = [f64(x) for x in (q, k, v)]
    lin, _ = ref.decay_forward(*f, f64(ld), np.zeros((B, H, d, d)), [n0 + 8] * B, 1 / math.sqrt(d))
    close(f64(o_lin), lin[:, :, :n0], half("bf16"), "prompt")
    for t in range(n0, n0 + 8):
        for dst, src in zip(now, (q, k, v)):
            dst.copy_(src[:, :, t:t + 1])
        graph.replay()
        close(f64(b), lin[:, :, t:t + 1], half("bf16"), f"token {t}", chunked=False)
        c = [f64(x) for x in cache]
        want, _, w, mag = ref.attend(f64(now[0]), *c, table.cpu().numpy(), [t + 1] * B, [1] * B, True,
                                     1 / math.sqrt(d))
        tol = half("bf16") * np.abs(want) + (2.0 ** -11 + 2.0 ** -15 * mag[..., None]) * w
        assert np.all(np.abs(f64(a) - want) <= tol)
    assert attn.attn_last_device_status() == 0


def test_backward_captured_and_replayed():
    (q, k, v, do), (s0, ds) = inputs(2, 3, 150, 64, "bf16", 35)
    ld = decays(3)
    want = attn.decay_backward(q, k, v, ld, do, state=s0, dstate=ds)
    args = [x.clone() for x in (q, k, v, do)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = attn.decay_backward(*args[:3], ld, args[3], state=s0, dstate=ds)
    for x in args:
        x.zero_()
    graph.replay()
    for dst, src in zip(args, (q, k, v, do)):
        dst.copy_(src)
    graph.replay()
    for a, b in zip(want, got):
        assert torch.equal(a, b)


def test_large_heads_shape_and_repeatability():
    """The large-head shape: two runs agree bit for bit, and three of its heads
    agree with the same call on them alone."""
    (q, k, v, do), (s0, ds) = inputs(4, 16, 4096, 128, "bf16", 36)
    ld = torch.tensor([-(2.0 ** (-(h + 1) / 2)) for h in range(16)], device="cuda")
    a, b = (attn.decay_forward(q, k, v, ld, state=s0) for _ in range(2))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    ga, gb = (attn.decay_backward(q, k, v, ld, do, state=s0, dstate=ds) for _ in range(2))
    assert all(torch.equal(x, y) for x, y in zip(ga, gb))
    assert attn.attn_last_device_status() == 0
    for bi, h in ((0, 0), (1, 7), (3, 15)):
        one = [x[bi:bi + 1, h:h + 1].contiguous() for x in (q, k, v, do, s0, ds)]
        o, s1 = attn.decay_forward(*one[:3], ld[h:h + 1].clone(), state=one[4])
        close(f64(o), f64(a[0][bi:bi + 1, h:h + 1]), 2 * half("bf16"), "o")
        close(f64(s1), f64(a[1][bi:bi + 1, h:h + 1]), 2 * STATE_TOL, "state")
        g = attn.decay_backward(*one[:3], ld[h:h + 1].clone(), one[3], state=one[4], dstate=one[5])
        for x, y in zip(g[:3], ga):
            close(f64(x), f64(y[bi:bi + 1, h:h + 1]), 2 * half("bf16"), "grad")
        close(f64(g[3]), f64(ga[3][bi:bi + 1, h:h + 1]), 2 * STATE_TOL, "dstate")


@pytest.mark.parametrize("d", [64, 128])
def test_states_of_small_fp16_values(d):
    """Values and gradients of about 1e-4, near fp16's smallest normal number: the
    states, which are fp32, keep their precision."""
    (q, k, v, do), _ = inputs(1, 3, 333, d, "fp16", 37)
    v, do = v * 1e-4, do * 1e-4
    ld = decays(3)
    _, s1 = attn.decay_forward(q, k, v, ld)
    ds = attn.decay_backward(q, k, v, ld, do)[3]
    f = [f64(x) for x in (q, k, v, do)]
    zero = np.zeros((1, 3, d, d))
    _, want = ref.decay_forward(*f[:3], f64(ld), zero, [333], 1 / math.sqrt(d))
    close(f64(s1), want, STATE_TOL, "state")
    want = ref.decay_backward(*f[:3], f64(ld), f[3], zero, zero, [333], 1 / math.sqrt(d))[3]
    close(f64(ds), want, STATE_TOL, "dstate")


def test_a_decay_of_nan_is_not_hidden():
    (q, k, v, do), (s0, ds) = inputs(1, 3, 140, 64, "bf16", 38)
    ld = torch.tensor([-0.1, math.nan, -0.2], device="cuda")
    o, s1 = attn.decay_forward(q, k, v, ld, state=s0)
    grads = attn.decay_backward(q, k, v, ld, do, state=s0, dstate=ds)
    step = attn.decay_step(*(x[:, :, :1].contiguous() for x in (q, k, v)), ld, s0)
    assert attn.attn_last_device_status() == 0
    for x in (o, s1, *grads, *step):
        assert torch.isnan(x[:, 1]).all() and torch.isfinite(x[:, ::2]).all()


@pytest.mark.parametrize("B,H,N,d,lens", [(3, 2, 300, 64, [0, 129, 256]), (2, 1, 2000, 128, [1, 700]),
                                          (2, 20, 130, 128, [128, 37])])
def test_rows_past_the_end_of_padded_batches(B, H, N, d, lens):
    """The conveniences return zeros there (one and several segments), whatever the
    memory held; the rest is what the call that leaves them alone writes."""
    (q, k, v, do), (s0, ds) = inputs(B, H, N, d, "bf16", 39)
    ld = decays(H)
    junk = [torch.full_like(q, 7.0) for _ in range(6)]
    o = torch.full_like(q, 7.0)
    g = [torch.full_like(q, 7.0) for _ in range(3)]
    ws = [torch.empty(max(attn.attn_decay_workspace_bytes(B, H, N, d, bw), 16), dtype=torch.uint8, device="cuda")
          for bw in (False, True)]
    attn.attn_decay_fwd(q, k, v, ld, o, s0, None, ints(lens), ws[0])
    attn.attn_decay_bwd(q, k, v, ld, do, *g, s0, ds, None, ints(lens), ws[1])
    del junk
    got = [attn.decay_forward(q, k, v, ld, state=s0, lens=ints(lens))[0],
           *attn.decay_backward(q, k, v, ld, do, state=s0, dstate=ds, lens=ints(lens))[:3]]
    assert attn.attn_last_device_status() == 0
    for a, b in zip(got, (o, *g)):
        for i, n in enumerate(lens):
            assert torch.equal(a[i, :, :n], b[i, :, :n])
            assert (a[i, :, n:] == 0).all() and (b[i, :, n:] == 7).all()


def test_segmented_calls_back_to_back_in_a_graph():
    """Calls of several segments, whose launches overlap, one after another on the same
    workspace and the same state, eager and as a replayed graph."""
    B, H, N, d = 1, 2, 1600, 64
    ld = decays(H)
    xs = [inputs(B, H, N, d, "bf16", 40 + i)[0][:3] for i in range(3)]
    need = attn.attn_decay_workspace_bytes(B, H, N, d)
    assert need > 0
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    want, state = [], torch.zeros(B, H, d, d, device="cuda")
    for x in xs:
        o, state = attn.decay_forward(*x, ld, state=state)
        want.append(o)
        torch.cuda.synchronize()
    out, s = [torch.empty_like(x[0]) for x in xs], torch.zeros(B, H, d, d, device="cuda")

    def chain():
        s.zero_()
        for x, o in zip(xs, out):
            attn.attn_decay_fwd(*x, ld, o, s, s, None, ws)

    chain()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chain()
    for again in range(3):
        if again:
            for o in out:
                o.fill_(7.0)
            graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(out, want)) and torch.equal(s, state)
    assert attn.attn_last_device_status() == 0
