"""Refusals of the token-by-token operators, before any device work (CPU)."""

import ctypes
import math

import pytest

torch = pytest.importorskip("torch")

from io_aware_exact_30_b200 import attn  # noqa: E402

P = ctypes.c_void_p(256)


def append(p=P, B=2, Hkv=2, T=3, d=64, num_pages=8, page=16, width=4, dt=0, v8=ctypes.c_void_p(512),
           vs=ctypes.c_void_p(512), k=None, n_new=None):
    return attn.lib().attn_cache_append(k or p, p, p, v8, p, vs, p, p, n_new, B, Hkv, T, d, num_pages, page,
                                        width, dt, None)


def attend(p=P, B=2, Hq=4, Hkv=2, T=3, d=64, num_pages=8, page=16, width=4, max_len=64, scale=0.1, dt=0,
           q=None, ws=None):
    return attn.lib().attn_cache_attend(q or p, p, p, p, p, p, p, None, p, p, ws or p, B, Hq, Hkv, T, d,
                                        num_pages, page, width, max_len, 1, scale, dt, None)


def at(i):
    return ctypes.c_void_p(4096 * i)


def fwd(p=P, B=2, H=2, N=5, d=64, scale=0.1, dt=0, q=None, ld=P, st=P, o=at(1)):
    return attn.lib().attn_decay_fwd(q or p, p, p, ld, st, None, p and o, st, p, B, H, N, d, 0, scale, dt, None)


def bwd(p=P, B=2, H=2, N=5, d=64, scale=0.1, dt=0, q=None, ld=P, ds=ctypes.c_void_p(512), g=(at(1), at(2), at(3))):
    return attn.lib().attn_decay_bwd(q or p, p, p, ld, p, p, p, None, *(p and x for x in g), ds, p, B, H, N, d,
                                     0, scale, dt, None)


def step(p=P, B=2, H=2, d=64, scale=0.1, dt=0, q=None, ld=P, o=at(1)):
    return attn.lib().attn_decay_step(q or p, p, p, ld, p, p and o, p, B, H, d, scale, dt, None)


ALL = (append, attend, fwd, bwd, step)


@pytest.mark.parametrize("call", ALL)
def test_common_refusals(call):
    assert call(p=None) == -1
    assert call(d=80) == -3 and call(d=0) == -3
    assert call(B=0) == -2 and call(B=-1) == -2
    assert call(B=1 << 26) in (-2,)
    assert call(dt=3) == -5
    odd = ctypes.c_void_p(264)
    assert (call(k=odd) if call is append else call(q=odd)) == -4
    if call is not append:
        for bad in (0.0, -1.0, math.nan, math.inf):
            assert call(scale=bad) == -9


def test_cache_refusals():
    for call in (append, attend):
        assert call(page=8) == -9 and call(page=48) == -9 and call(page=256) == -9
        assert call(num_pages=0) == -2 and call(width=0) == -2 and call(T=0) == -2
        assert call(width=1 << 27) == -2  # positions past 2^31
        assert call(Hkv=0) == -2
    assert append(v8=P) == -9 and append(vs=P) == -9
    assert append(n_new=ctypes.c_void_p(258)) == -4
    assert attend(Hkv=3) == -2 and attend(max_len=0) == -9
    assert attend(ws=ctypes.c_void_p(264)) == -4


def test_decay_refusals():
    for call in (fwd, bwd, step):
        assert call(ld=None) == -1 and call(ld=ctypes.c_void_p(258)) == -4
        assert call(H=0) == -2
    assert fwd(N=0) == -2 and bwd(N=0) == -2
    assert bwd(ds=P) == -9  # the gradient over an array that is read
    assert fwd(o=P) == -9 and step(o=P) == -9  # a result over an input
    assert bwd(g=(P, at(2), at(3))) == -9 and bwd(g=(at(1), at(2), at(1))) == -9
    assert attn.strerror(-11) and attn.strerror(-11) != attn.strerror(-99)


def test_cache_capacity_of_a_sequence():
    """Positions, rounded up to a tile, stay 32-bit: at most 2^30 tokens a sequence."""
    for call in (append, attend):
        assert call(page=128, width=(1 << 23) + 1) == -2 and call(page=16, width=(1 << 26) + 1) == -2


def test_workspace_sizes_of_invalid_calls_are_zero():
    assert attn.attn_cache_attend_workspace_bytes(1, 4, 3, 1, 64, 100) == 0
    assert attn.attn_cache_attend_workspace_bytes(1, 4, 2, 1, 96, 100) == 0
    assert attn.attn_cache_attend_workspace_bytes(1, 4, 2, 1, 64, 0) == 0
    assert attn.attn_decay_workspace_bytes(1, 4, 100, 96) == 0
    assert attn.attn_decay_workspace_bytes(1, 0, 100, 64, True) == 0


def _cache(P=4, H=2, page=16, d=64):
    c = torch.zeros(P, H, page, d, dtype=torch.uint8).view(torch.float8_e4m3fn)
    return attn.Cache8(c, c.clone(), torch.zeros(P, H), torch.zeros(P, H))


def test_binding_refuses_what_does_not_fit():
    x = torch.zeros(1, 2, 1, 64, dtype=torch.bfloat16)
    table, lens = torch.zeros(1, 4, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    c = _cache()
    for bad in (dict(cache=_cache(d=128)), dict(cache=_cache(H=1)), dict(table=table.long()),
                dict(table=table[:, ::2]), dict(lens=lens.long()), dict(lens=torch.zeros(2, dtype=torch.int32)),
                dict(cache=c._replace(k=c.k.float())), dict(cache=c._replace(v_scale=torch.zeros(4, 1))),
                dict(cache=c._replace(k=c.k.transpose(1, 2))), dict(n_new=torch.zeros(1)),
                dict(k=torch.zeros(1, 2, 2, 64, dtype=torch.bfloat16)[:, :, ::2].expand(1, 2, 1, 64)),
                dict(k=torch.zeros(1, 2, 1, 128, dtype=torch.bfloat16)[..., ::2])):
        a = dict(dict(k=x, cache=c, table=table, lens=lens, n_new=None), **bad)
        with pytest.raises(ValueError):
            attn.cache_append(a["k"], a["k"], a["cache"], a["table"], a["lens"], a["n_new"])
    with pytest.raises(TypeError):
        attn.cache_append(x.float(), x.float(), c, table, lens)
    with pytest.raises(ValueError):
        attn.cache_alloc(4, 2, 24, 64, device="cpu")
    o, lse = torch.zeros_like(x), torch.zeros(1, 2, 1)
    with pytest.raises(ValueError):
        attn.attn_cache_attend(x, c, table, lens, o.float(), lse)
    with pytest.raises(ValueError):
        attn.attn_cache_attend(x, c, table, lens, o, lse.double())

    ld, st = torch.zeros(2), torch.zeros(1, 2, 64, 64)
    with pytest.raises(ValueError):
        attn.decay_step(torch.zeros(1, 2, 2, 64).bfloat16(), x, x, ld, st)
    with pytest.raises(ValueError):
        attn.decay_forward(x, x, x, ld[:1], state=st)
    with pytest.raises(ValueError):
        attn.decay_forward(x, x, x, ld.double(), state=st)
    with pytest.raises(ValueError):
        attn.decay_forward(x, x, x, ld, state=st.half())
    with pytest.raises(ValueError):
        attn.decay_forward(x, x.half(), x, ld, state=st)
    with pytest.raises(ValueError):
        attn.decay_backward(x, x, x, ld, x, state=st, dstate=st[:, :1])
    with pytest.raises(ValueError):
        attn.decay_forward(x, x, x, ld, lens=torch.zeros(1))
    with pytest.raises(TypeError):
        attn.decay_forward(*[x.float()] * 3, ld)
