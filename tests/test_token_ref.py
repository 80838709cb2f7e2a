"""The 64-bit references of the token-by-token operators against other routes:
torch's e4m3 cast, brute force, autograd and central differences (CPU)."""

import math

import numpy as np
import pytest

import token_ref as ref

torch = pytest.importorskip("torch")


def test_e4m3_rounding_is_torchs_cast():
    x = np.concatenate([np.linspace(-448, 448, 20011), np.ldexp(np.linspace(-2, 2, 4001), -7),
                        ref.E4M3, -ref.E4M3, (ref.E4M3[1:] + ref.E4M3[:-1]) / 2])
    want = torch.from_numpy(x.astype(np.float32)).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(ref.e4m3_round(x.astype(np.float32).astype(np.float64)), want)


def test_page_scale_is_the_least_power_of_two():
    for a in (1e-30, 1e-5, 0.4375, 0.43750003, 1.0, 448.0, 448.0001, 449.0, 3e38):
        s = ref.page_scale(a)
        assert math.frexp(s)[0] == 0.5 and a <= 448 * s and a > 448 * s / 2
    assert ref.page_scale(0.0) == 0.0


def test_growing_a_page_token_by_token_keeps_normal_codes():
    """Appending one by one ends at the scale of appending at once, and at the same
    codes but for values below the final scale's normal range (2^-6)."""
    rng = np.random.default_rng(0)
    x = rng.standard_normal((1, 1, 16, 64)) * np.exp2(rng.integers(-3, 6, (1, 1, 16, 1)))
    table, one, two = np.zeros((1, 1), np.int32), {}, {}
    for d, step in ((one, 16), (two, 1)):
        d["c"], d["s"] = np.zeros((1, 1, 16, 64)), np.zeros((1, 1))
        for t in range(0, 16, step):
            assert not ref.append(x[:, :, t:t + step], d["c"], d["s"], table, [t], [step], 1)
    assert one["s"] == two["s"]
    normal = np.abs(one["c"]) >= 2.0 ** -6
    assert normal.mean() > 0.9 and np.array_equal(one["c"][normal], two["c"][normal])
    assert np.abs(one["c"] - two["c"]).max() <= 2.0 ** -9


def test_attend_is_a_masked_softmax():
    rng = np.random.default_rng(1)
    B, Hq, Hkv, T, d, page = 2, 4, 2, 3, 8, 16
    k8, v8 = (ref.e4m3_round(rng.standard_normal((5, Hkv, page, d)) * 30) for _ in range(2))
    ks, vs = (np.exp2(rng.integers(-4, 0, (5, Hkv)).astype(float)) for _ in range(2))
    table = np.array([[3, 1], [0, 4]], np.int32)
    q, lens, q_lens = rng.standard_normal((B, Hq, T, d)), [20, 2], [3, 3]
    o, lse, _, _ = ref.attend(q, k8, v8, ks, vs, table, lens, q_lens, True, 0.3)
    for b in range(B):
        K, V = ((c[table[b]] * s[table[b]][..., None, None]).transpose(1, 0, 2, 3).reshape(Hkv, -1, d)
                for c, s in ((k8, ks), (v8, vs)))
        for h in range(Hq):
            for t in range(T):
                n = lens[b] - (T - 1 - t)
                if n <= 0:
                    assert np.all(o[b, h, t] == 0) and lse[b, h, t] == -np.inf
                    continue
                x = torch.from_numpy(K[h // 2, :n] @ q[b, h, t] * 0.3)
                assert abs(lse[b, h, t] - float(torch.logsumexp(x, 0))) < 1e-12
                assert np.allclose(o[b, h, t], torch.softmax(x, 0).numpy() @ V[h // 2, :n], atol=1e-12)


def _case(B=2, H=2, N=9, d=4, seed=2):
    rng = np.random.default_rng(seed)
    x = [rng.standard_normal((B, H, N, d)) for _ in range(4)]
    s = [rng.standard_normal((B, H, d, d)) for _ in range(2)]
    return x, s, np.array([-0.3, 0.0]), np.array([N, 5])


def test_decay_forward_is_the_weighted_sum():
    (q, k, v, _), (s0, _), ld, lens = _case()
    o, s1 = ref.decay_forward(q, k, v, ld, s0, lens, 0.5)
    for b in range(2):
        for h in range(2):
            for i in range(lens[b]):
                want = math.exp(ld[h] * (i + 1)) * (q[b, h, i] @ s0[b, h])
                for j in range(i + 1):
                    want = want + math.exp(ld[h] * (i - j)) * (q[b, h, i] @ k[b, h, j]) * v[b, h, j]
                assert np.allclose(o[b, h, i], 0.5 * want, atol=1e-12)
            assert np.isnan(o[b, h, lens[b]:]).all()


def test_decay_backward_against_autograd_and_differences():
    (q, k, v, do), (s0, ds), ld, lens = _case()
    got = ref.decay_backward(q, k, v, ld, do, s0, ds, lens, 0.5)

    def loss(q, k, v, s0):
        o, s1 = ref.decay_forward(q, k, v, ld, s0, lens, 0.5)
        return float(np.nansum(o * do) + (s1 * ds).sum())

    args = [q, k, v, s0]
    rng = np.random.default_rng(3)
    for i, g in enumerate(got):
        step = rng.standard_normal(args[i].shape)
        up, down = ([a + sign * 1e-5 * step if j == i else a for j, a in enumerate(args)]
                    for sign in (1, -1))
        want = (loss(*up) - loss(*down)) / 2e-5
        assert abs(np.nansum(g * step) - want) < 1e-6 * max(1, abs(want))

    t = [torch.from_numpy(a).requires_grad_() for a in args]
    total = torch.zeros((), dtype=torch.float64)
    for b in range(2):
        for h in range(2):
            S = t[3][b, h]
            for i in range(lens[b]):
                S = math.exp(ld[h]) * S + torch.outer(t[1][b, h, i], t[2][b, h, i])
                total = total + 0.5 * (t[0][b, h, i] @ S) @ torch.from_numpy(do[b, h, i])
            total = total + (S * torch.from_numpy(ds[b, h])).sum()
    total.backward()
    for a, g in zip(t, got):
        assert np.allclose(a.grad.numpy(), np.nan_to_num(g), atol=1e-11)
