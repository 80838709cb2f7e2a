"""Decayed linear attention on a B200 over the range of its types and over long
memories: thousands of recurrent steps, small and large fp16 values, long sequences
against a 64-bit form.

Tolerances, relative L2 per head.
  States are fp32.  Their terms reach the tensor cores in 16-bit pieces that hold 22
bits of them (fp16) or 24 (bf16), 2^-23 at most; the fp32 sums over a chunk's 128 tokens
round 128 times, independently, sqrt(128) 2^-24 = 2^-20.5 of them; each chunk adds two
roundings and the powers of the decay a few units of 2^-24.  Squares added: below
STATE_TOL = 2^-20 for a few dozen chunks that count (a rounding ages with its chunk).
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
