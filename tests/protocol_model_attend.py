"""A model of the mbarrier protocol of the cache attention's tile kernel
(cache_attend_tile_kernel in io_aware_exact_30_b200/csrc/cache8_tile.cuh), checked
on the CPU under random schedules with the rules of protocol_model.py.  Test
infrastructure only.

Roles: the MMA issuer, the conversion warps (two agents), the softmax warps (two
agents a half of the keys).  Per tile j (buffer j % 2 of K, V and S; P over S) the
issuer does S_{j+1} = Q K^T, then O_h += P_h V_h for both halves.  K's scales live in
four slots.
"""

from protocol_model import AsyncWork, ProtocolError, World, run_roles  # noqa: F401

NCONV, NHALF, NPER = 2, 2, 2  # conversion agents; halves; softmax agents a half

W = None


class Variant:
    def __init__(self, skip=(), one_pf=False, two_ks=False, raises=()):
        self.skip = set(skip)
        # mistake (seen in the kernel): one barrier for a written P, not one per buffer;
        # a half one tile ahead completes the other's phase
        self.one_pf = one_pf
        self.two_ks = two_ks        # mistake: K's scales in two slots
        self.raises = set(raises)   # tiles whose softmax moves the reference


def waits(v, *named):
    w = [(b, k) for name, b, k, on in named if on and name not in v.skip]
    if w:
        yield ("wait", w)


def pf(j, v):
    return ("PF0", j) if v.one_pf else (f"PF{j & 1}", j >> 1)


def ks(j, v):
    return ("KS", j % (2 if v.two_ks else 4))


def issue_s(j, v):
    s, u = j & 1, j >> 1
    yield from waits(v, ("kf", f"KF{s}", u, True), ("s_free", f"OD{s}", u - 1, j >= 2),
                     ("qf", "QF", 0, j == 0))

    def s_mma(j=j, s=s):
        W.read("Q", 0)
        for a in range(NCONV):
            W.read(("K", s, a), j)
        for h in range(NHALF):
            for a in range(NPER):
                W.write(("S", s, h, a), ("S", j))
    yield ("async", "mma", s_mma, f"S{s}")
    yield ("async", "mma", lambda s=s, u=u: W.bar(f"SF{s}").arrive(u))


def issuer(nt, v):
    if nt:
        yield from issue_s(0, v)
    for j in range(nt):
        s, u = j & 1, j >> 1
        if j + 1 < nt:
            yield from issue_s(j + 1, v)
        yield from waits(v, ("pf", *pf(j, v), True), ("vf", f"VF{s}", u, True))

        def pv_mma(j=j, s=s):
            for a in range(NCONV):
                W.read(("V", s, a), j)
            for h in range(NHALF):
                for a in range(NPER):
                    W.read(("S", s, h, a), ("P", j))
                    if j:
                        W.read(("O", h, a), ("scaled", j) if j in v.raises else j - 1)
                    W.write(("O", h, a), j)
        yield ("async", "mma", pv_mma, "O")
        yield ("async", "mma", lambda s=s, u=u: W.bar(f"OD{s}").arrive(u))


def conversion(a, nt, v):
    for j in range(nt):
        s, u = j & 1, j >> 1
        yield from waits(v, ("k_free", f"SF{s}", u - 1, j >= 2))
        yield ("write", (*ks(j, v), a), j)
        yield ("write", ("K", s, a), j)
        yield ("arrive", f"KF{s}", u)
        yield from waits(v, ("v_free", f"OD{s}", u - 1, j >= 2))
        yield ("write", ("V", s, a), j)
        yield ("arrive", f"VF{s}", u)


def softmax(h, a, nt, v):
    if h == 0 and a == 0:
        yield ("write", "Q", 0)
    if h == 0:
        yield ("arrive", "QF", 0)
    for j in range(nt):
        s, u = j & 1, j >> 1
        yield from waits(v, ("sf", f"SF{s}", u, True))
        for c in range(NCONV):
            yield ("read", (*ks(j, v), c), j)
        yield ("read", ("S", s, h, a), ("S", j))
        if j in v.raises and j:
            yield from waits(v, ("raise_od", f"OD{s ^ 1}", (j - 1) >> 1, True))
            yield ("read", ("O", h, a), j - 1)
            yield ("write", ("O", h, a), ("scaled", j))
        yield ("write", ("S", s, h, a), ("P", j))
        yield ("arrive", *pf(j, v))
    if nt:
        yield from waits(v, ("last_od", f"OD{(nt - 1) & 1}", (nt - 1) >> 1, True))
        yield ("read", ("O", h, a), nt - 1)


def run_schedule(nt, seed, variant=None, in_order=False, max_steps=200000):
    global W
    v = variant or Variant()
    W = World()
    for s in range(2):
        W.bar(f"KF{s}", NCONV)
        W.bar(f"VF{s}", NCONV)
        W.bar(f"PF{s}", NHALF * NPER)
    W.bar("QF", NPER)
    roles = {"mma": issuer(nt, v)}
    for a in range(NCONV):
        roles[f"conv{a}"] = conversion(a, nt, v)
    for h in range(NHALF):
        for a in range(NPER):
            roles[f"soft{h}{a}"] = softmax(h, a, nt, v)
    run_roles(W, roles, seed, in_order, max_steps)
