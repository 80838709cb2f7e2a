"""Decayed linear attention on a B200 over the range of its types and over long
memories: thousands of recurrent steps, small and large fp16 values, long sequences
against a 64-bit form.

Tolerances, relative L2 per head.
  States are fp32.  Their terms reach the tensor cores in 16-bit pieces that hold 22
bits of them (fp16, 2^-22 of a term at most, where it is above 2^-17 of its chunk's
largest) or 24 (bf16); the fp32 sums over a chunk's 128 tokens round 128 times,
independently, sqrt(128) 2^-24 = 2^-20.5 of them; each chunk adds two roundings and the
powers of the decay a few units of 2^-24.  Squares added: below STATE_TOL = 2^-20 for a few
dozen chunks that count (a rounding ages with its chunk).
  16-bit results pass three roundings of half a step in L2, eps / 2 together (as in
test_decay_gpu): the power-of-two factors that keep fp16 operands in its normal range
round nothing, so the same holds for small and large operands, while the results are
normal numbers of fp16 themselves; a subnormal result is off by up to half its step,
2^-25, on top.
  A recurrent step rounds the state twice, by at most 2^-24 and 2^-24 / sqrt(3) in L2.
Roundings of different tokens are independent, those of the same token met again need
not be: where nothing is forgotten (g = 1) a sum S + x drops x mod ulp(S), the same bits
each time while S stays in a binade.  n tokens met r times: r sqrt(2 n) 2^-24 / sqrt(3).
"""

import math

import numpy as np
import pytest

from test_decay_gpu import FEW, TYPES, f64, half, inputs, ints

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from io_aware_exact_30_b200 import attn  # noqa: E402

STATE_TOL = 2.0 ** -20


def rel(got, want):
    """The largest relative L2 of a head."""
    got, want = (x.double().reshape(-1, x.shape[-2] * x.shape[-1]) for x in (got, want))
    return float(((got - want).norm(dim=1) / want.norm(dim=1)).max())


def chunked(q, k, v, ld, s0, lens, scale):
    """The operator in 64 bits on the device, chunk by chunk (elementary operations)."""
    B, H, N, d = q.shape
    C = 128
    t = torch.arange(N, device=q.device)
    live = (t[None] < lens[:, None])[:, None, :, None]
    g = ld.view(1, H, 1, 1)
    k, v = torch.where(live, k, 0.0), torch.where(live, v, 0.0)
    S, out = s0, []
    for c in range(0, N, C):
        n = min(C, N - c)
        i = torch.arange(n, device=q.device, dtype=torch.float64)
        x, y, z = (a[:, :, c:c + n] for a in (q, k, v))
        gap = i[:, None] - i[None]
        w = torch.where(gap >= 0, torch.exp(g * gap.clamp(min=0)), 0.0)
        out.append(scale * (((x @ y.transpose(2, 3)) * w) @ z + torch.exp(g * (i + 1).view(1, 1, n, 1)) * (x @ S)))
        m = (lens - c).clamp(0, n).double().view(B, 1, 1, 1)  # tokens of the chunk
        S = torch.exp(g * m) * S + (y * torch.exp(g * (m - 1 - i.view(1, 1, n, 1)).clamp(min=0))).transpose(2, 3) @ z
    return torch.where(live, torch.cat(out, 2), 0.0), S


# (the first one's power over a chunk lies nearly half a step off fp32)
SLOW = [-0.0001446875, -0.002, 0.0]


@pytest.mark.parametrize("d,dtype", [(64, "fp16"), (128, "bf16")])
def test_thousands_of_steps_keep_the_decay(d, dtype):
    """20000 captured in-place steps against the 64-bit recurrence, and against one
    prompt of the same tokens.  A decay rounded to fp32 once is off in the same direction
    at every step, by 1.9e-4 after these.  (In fp32 arithmetic without that error they
    come to 3.4e-5, at a log decay of -3e-9.)"""
    lds = [SLOW[0], -1e-4, -1e-7, -3e-9, -0.01, -2.5, 0.0]
    B, H, n, again = 1, len(lds), 100, 200
    (q, k, v, _), (s0, _) = inputs(B, H, n, d, dtype, 70)
    s0 = s0 * 100
    ld = torch.tensor(lds, device="cuda")
    tokens = [[x[:, :, t:t + 1].contiguous() for x in (q, k, v)] for t in range(n)]
    state = s0.clone()
    attn.decay_step(*tokens[0], ld, state.clone())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for x in tokens:
            o, _ = attn.decay_step(*x, ld, state, state_out=state)
    for _ in range(again):
        graph.replay()
    many = [x.repeat(1, 1, again, 1) for x in (q, k, v)]
    want_o, want = chunked(*(x.double() for x in many), ld.double(), s0.double(), ints([n * again]).long(),
                           1 / math.sqrt(d))
    assert rel(state, want) <= again * math.sqrt(2 * n / 3) * 2.0 ** -24
    assert rel(o, want_o[:, :, -1:]) <= half(dtype)
    _, prompt = attn.decay_forward(*many, ld, state=s0)
    assert rel(prompt, want) <= STATE_TOL
    assert attn.attn_last_device_status() == 0


def scaled(seed, N, d, dtype, by, B=1, H=3):
    """q, k, v, do with standard deviations `by`."""
    x, s = inputs(B, H, N, d, "bf16", seed)
    return [(a.float() * f).to(TYPES[dtype]) for a, f in zip(x, by)], s


def near(got, want, dtype, label):
    """Half a step in L2 (three times that in heads of few tokens), and half a step of
    fp16's subnormal numbers."""
    got, want = f64(got), f64(want)
    for b in range(want.shape[0]):
        for h in range(want.shape[1]):
            assert np.all(np.isfinite(got[b, h])), f"{label} {(b, h)}"
            off, norm = np.linalg.norm(got[b, h] - want[b, h]), np.linalg.norm(want[b, h])
            few = np.any(want[b, h], axis=1).sum() < FEW
            tol = (3 if few else 1) * half(dtype) * norm + (2.0 ** -25 * math.sqrt(want[b, h].size) if dtype == "fp16" else 0.0)
            assert norm > 0 and off <= tol, f"{label} {(b, h)}: {off / norm} > {tol / norm}"


def gradients(q, k, v, ld, do, s0, ds, lens, scale):
    """64-bit gradients by automatic differentiation of `chunked`."""
    leaves = [x.double().requires_grad_() for x in (q, k, v, s0)]
    o, S = chunked(leaves[0], leaves[1], leaves[2], ld.double(), leaves[3], lens, scale)
    loss = (o * torch.nan_to_num(do.double())).sum() + (S * ds.double()).sum()
    return o.detach(), S.detach(), torch.autograd.grad(loss, leaves)


def check_all(xs, s0, ds, ld, dtype, lens=None, state_tol=STATE_TOL, heads=slice(None)):
    """Forward and backward against the 64-bit form; `heads` of them are compared."""
    q, k, v, do = xs
    B, H, N, d = q.shape
    n = None if lens is None else ints(lens)
    o, s1 = attn.decay_forward(q, k, v, ld, state=s0, lens=n)
    got = attn.decay_backward(q, k, v, ld, do, state=s0, dstate=ds, lens=n)
    assert attn.attn_last_device_status() == 0
    cut = [x[:, heads] for x in (q, k, v)]
    want_o, want_s, want = gradients(*cut, ld[heads], do[:, heads], s0[:, heads], ds[:, heads],
                                     ints([N] * B if lens is None else lens).long(), 1 / math.sqrt(d))
    near(o[:, heads], want_o, dtype, "o")
    for name, a, w in zip(("dq", "dk", "dv"), got, want):
        near(a[:, heads], w, dtype, name)
    assert rel(s1[:, heads], want_s) <= state_tol, ("state", rel(s1[:, heads], want_s))
    assert rel(got[3][:, heads], want[3]) <= state_tol, ("dstate", rel(got[3][:, heads], want[3]))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("size", [1.0, 1e-4, 1e-5, 1e-6])
def test_states_of_fp16_values_of_every_size(d, size):
    """States are fp32: terms of values far below fp16's smallest normal number (6e-5)
    keep their bits on the way through 16-bit pieces."""
    N = 333
    (q, k, v, do), _ = scaled(71, N, d, "fp16", (1, 1, size, size))
    ld = torch.tensor(SLOW, device="cuda")
    zero = torch.zeros(1, 3, d, d, device="cuda")
    _, s1 = attn.decay_forward(q, k, v, ld)
    ds = attn.decay_backward(q, k, v, ld, do)[3]
    _, want, grads = gradients(q, k, v, ld, do, zero, zero, ints([N]).long(), 1 / math.sqrt(d))
    assert rel(s1, want) <= STATE_TOL and rel(ds, grads[3]) <= STATE_TOL
    # few heads and a long sequence: the segments' own sums
    (q, k, v, do), _ = scaled(72, 2000, d, "fp16", (size, size, 1, 1))
    ds = attn.decay_backward(q, k, v, ld, do)[3]
    _, want, grads = gradients(q, k, v, ld, do, zero, zero, ints([2000]).long(), 1 / math.sqrt(d))
    assert rel(attn.decay_forward(q, k, v, ld)[1], want) <= STATE_TOL and rel(ds, grads[3]) <= STATE_TOL


# standard deviations of q, k, v and dout, and of the states; every result is within fp16's
# normal range, what is rounded to 16 bits on the way to it would not be
SIZES = {
    "small weights": ((3e-3, 3e-3, 30, 30), 3e-4, 3e-4),
    "smaller weights": ((1e-3, 1e-3, 300, 300), 1e-3, 1e-3),
    "weights past 65504": ((300, 300, 1e-3, 1e-3), 30, 0.1),
    "states past 65504": ((1e-3, 1, 1, 1e-3), 1e6, 1e-3),
    "gradients of states past 65504": ((60, 1e-3, 1e-3, 1500), 1e-3, 1e6),
    "a small state": ((300, 1e-3, 1e-3, 300), 1e-6, 1e-3),
}


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("sizes", SIZES.values(), ids=SIZES.keys())
def test_fp16_results_of_small_and_large_operands(sizes, d):
    by, state, dstate = sizes
    for N, seed in ((200, 73), (1300, 74)):
        xs, (s0, ds) = scaled(seed, N, d, "fp16", by)
        check_all(xs, s0 * state, ds * dstate, torch.tensor([-0.05, -0.6, -0.004], device="cuda"), "fp16")


@pytest.mark.parametrize("d", [64, 128])
def test_fp16_rows_of_many_sizes(d):
    """Tokens whose q, k and v differ by up to 2^12 each (results reach 5e4): every row of
    the result is right by itself.  Its error is that of the result's own rounding, of its
    weights P_ij, each up to eps / 2 of itself and so eps / 2 sqrt(sum_j P_ij^2 |v_j|^2) in
    L2, and of the state's copy, eps / 2 of each entry, scale L^t sqrt(sum_a q_a^2 |S_a|^2);
    few terms may make up a row, so three times the L2 of the three, and half a step of
    fp16's subnormal numbers.  (Relative to the row itself there is no bound: q S may
    cancel.)  Weights and entries far below the chunk's largest possible ones are off by
    2^-39 of those, d scale max|q| max|k| and the largest possible state, instead."""
    B, H, N = 1, 3, 700
    (q, k, v, do), (s0, ds) = inputs(B, H, N, d, "bf16", 80)
    g = torch.Generator().manual_seed(81)
    q, k, v, do = ((x.float() * torch.exp2(torch.randint(-6, 7, (B, H, N, 1), generator=g).float().cuda())).half()
                   for x in (q, k, v, do))
    v, do = v * 2.0 ** -6, do * 2.0 ** -6
    ld = torch.tensor([-0.05, -1.5, -0.0004], device="cuda")
    check_all((q, k, v, do), s0, ds, ld, "fp16")
    o, _ = attn.decay_forward(q, k, v, ld, state=s0)
    x, y, z, g = q.double(), k.double(), v.double(), ld.double().view(1, H, 1, 1)
    S, scale = s0.double(), 1 / math.sqrt(d)
    most = S.abs().amax((2, 3))
    for c in range(0, N, 128):
        cut = slice(c, min(N, c + 128))
        want, after = chunked(x[:, :, cut], y[:, :, cut], z[:, :, cut], ld.double(), S,
                              ints([cut.stop - c]).long(), scale)
        i = torch.arange(cut.stop - c, device="cuda", dtype=torch.float64)
        gap = i[:, None] - i[None]
        P = x[:, :, cut] @ y[:, :, cut].transpose(2, 3) * torch.where(gap >= 0, torch.exp(g * gap.clamp(min=0)), 0.0)
        size = (P ** 2) @ (z[:, :, cut] ** 2).sum(-1, keepdim=True) + \
            torch.exp(g * (i + 1).view(1, 1, -1, 1)) ** 2 * ((x[:, :, cut] ** 2) @ (S ** 2).sum(-1, keepdim=True))
        big = [a[:, :, cut].abs().amax((2, 3)) for a in (x, y, z)]
        least = 2.0 ** -39 * scale * (d * big[0] * big[1] * z[:, :, cut].norm(dim=(2, 3)) +
                                      x[:, :, cut].norm(dim=3).amax(2) * math.sqrt(d) * most)
        tol = 3 * half("fp16") * torch.sqrt((want ** 2).sum(-1) + scale ** 2 * size[..., 0]) + least[..., None] + \
            2.0 ** -25 * math.sqrt(d)
        off = (o[:, :, cut].double() - want).norm(dim=-1)
        assert (off <= tol).all(), (c, float((off / tol).max()))
        S, most = after, most + 128 * big[1] * big[2]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128])
def test_rows_past_the_end_have_no_say(dtype, d):
    """The largest finite numbers in the rows behind a sequence's last change nothing."""
    B, H, N, lens = 3, 2, 300, [130, 299, 7]
    xs, (s0, ds) = inputs(B, H, N, d, dtype, 75)
    xs = [x * 1e-3 for x in xs]
    ld = torch.tensor([-0.01, -0.3], device="cuda")
    calls = []
    for junk in (0.0, torch.finfo(xs[0].dtype).max, math.inf):
        for x in xs:
            for b, n in enumerate(lens):
                x[b, :, n:] = junk
        q, k, v, do = xs
        calls.append([*attn.decay_forward(q, k, v, ld, state=s0, lens=ints(lens)),
                      *attn.decay_backward(q, k, v, ld, do, state=s0, dstate=ds, lens=ints(lens))])
    for other in calls[1:]:
        assert all(torch.equal(a, b) for a, b in zip(calls[0], other))
    assert all(torch.isfinite(x.float()).all() for x in calls[0])


@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_an_element_that_is_not_finite_stays_where_it_belongs(bad, dtype):
    """In a query it spoils that row; in a value its feature of the state, and of the
    rows from its chunk on; nothing else."""
    d, N = 128, 400
    (q, k, v, _), (s0, _) = inputs(1, 2, N, d, dtype, 76)
    ld = torch.tensor([-0.01, -0.3], device="cuda")
    n = ints([N]).long()
    args = [x.double() for x in (q, k, v)]
    want_o, want_s = chunked(*args, ld.double(), s0.double(), n, 1 / math.sqrt(d))
    broken = q.clone()
    broken[0, 0, 150, 3] = bad
    o, s1 = attn.decay_forward(broken, k, v, ld, state=s0)
    assert not torch.isfinite(o[0, 0, 150].float()).any()
    rows = torch.arange(N, device="cuda") != 150
    near(o[:, :, rows], want_o[:, :, rows], dtype, "o")
    assert rel(s1, want_s) <= STATE_TOL
    broken = v.clone()
    broken[0, 1, 200, 70] = bad
    o, s1 = attn.decay_forward(q, k, broken, ld, state=s0)
    cols = torch.arange(d, device="cuda") != 70
    assert not torch.isfinite(s1[0, 1, :, 70]).any() and not torch.isfinite(o[0, 1, 256:, 70].float()).any()
    assert torch.isfinite(s1[..., cols]).all() and torch.isfinite(o[0, 0].float()).all()
    near(o[..., cols], want_o[..., cols], dtype, "o")
    assert rel(s1[..., cols], want_s[..., cols]) <= STATE_TOL
    near(o[:, 1:, :128], want_o[:, 1:, :128], dtype, "o")  # the chunks in front of it


@pytest.mark.parametrize("B,H,N,d,dtype,lens", [
    (1, 3, 9000, 64, "bf16", None), (1, 3, 9000, 128, "fp16", None), (2, 3, 5000, 128, "bf16", [4999, 2049]),
    (2, 3, 5000, 64, "fp16", [1, 4100])])
def test_long_sequences_and_slow_decays(B, H, N, d, dtype, lens):
    """Dozens of chunks in one segment or several, memories of thousands of tokens: the
    states would lose their precision with one 32-bit decay a chunk."""
    xs, (s0, ds) = inputs(B, H, N, d, dtype, 77)
    for x in xs:
        for b, n in enumerate(lens or []):
            x[b, :, n:] = 0
    check_all(xs, s0, ds, torch.tensor(SLOW, device="cuda"), dtype, lens)


def test_large_heads_against_the_64_bit_form():
    """The large-head shape, a walk of 32 chunks for each of 64 heads."""
    B, H, N, d = 4, 16, 4096, 128
    xs, (s0, ds) = inputs(B, H, N, d, "bf16", 78)
    ld = torch.tensor([SLOW[h % 3] * (1 + h) for h in range(H)], device="cuda")
    check_all(xs, s0, ds, ld, "bf16", heads=slice(0, 16, 5))


@pytest.mark.parametrize("N", [300, 4000])
def test_calls_repeat_themselves_bit_for_bit(N):
    xs, (s0, ds) = inputs(2, 4, N, 64, "fp16", 79)
    q, k, v, do = xs
    ld = torch.tensor([*SLOW, -1.0], device="cuda")
    step = [x[:, :, :1].contiguous() for x in (q, k, v)]

    def run():
        return [*attn.decay_forward(q, k, v, ld, state=s0), *attn.decay_step(*step, ld, s0),
                *attn.decay_backward(q, k, v, ld, do, state=s0, dstate=ds)]
    want = run()
    for _ in range(10):
        assert all(torch.equal(a, b) for a, b in zip(run(), want))


@pytest.mark.parametrize("N", [140, 1700])
def test_fp16_decays_at_their_ends(N):
    """A NaN decay makes its head NaN, no memory at all and a steep one stay right, in one
    segment and several."""
    xs, (s0, ds) = inputs(1, 4, N, 64, "fp16", 82)
    q, k, v, do = xs
    ld = torch.tensor([-0.1, math.nan, -math.inf, -1.7], device="cuda")
    o, s1 = attn.decay_forward(q, k, v, ld, state=s0)
    grads = attn.decay_backward(q, k, v, ld, do, state=s0, dstate=ds)
    assert attn.attn_last_device_status() == 0
    for x in (o, s1, *grads):
        assert torch.isnan(x[:, 1]).all()
    keep = [0, 2, 3]
    want_o, want_s, want = gradients(*(x[:, keep] for x in (q, k, v)), torch.nan_to_num(ld[keep], neginf=-1e4),
                                     do[:, keep], s0[:, keep], ds[:, keep], ints([N]).long(), 1 / math.sqrt(64))
    near(o[:, keep], want_o, "fp16", "o")
    for name, a, w in zip(("dq", "dk", "dv"), grads, want):
        near(a[:, keep], w, "fp16", name)
    assert rel(s1[:, keep], want_s) <= STATE_TOL
    dead = want[3].abs().amax((2, 3)) == 0  # (nothing of the first state is left)
    assert (grads[3][:, keep][dead] == 0).all()
    left = [h for i, h in enumerate(keep) if not dead[0, i]]
    if left:
        assert rel(grads[3][:, left], want[3][:, [i for i in range(3) if not dead[0, i]]]) <= STATE_TOL


def test_two_calls_at_once_do_not_share_anything():
    ld = torch.tensor([*SLOW, -1.0], device="cuda")
    sets = [inputs(1, 4, N, 128, "fp16", 83 + N) for N in (1500, 900)]
    run = lambda xs, st: [*attn.decay_forward(*xs[:3], ld, state=st[0]),  # noqa: E731
                          *attn.decay_backward(*xs[:3], ld, xs[3], state=st[0], dstate=st[1])]
    want = [[x.clone() for x in run(*s)] for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        got = []
        for s, side in zip(sets, streams):
            with torch.cuda.stream(side):
                got.append(run(*s))
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert attn.attn_last_device_status() == 0
