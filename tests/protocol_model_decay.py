"""A model of the mbarrier protocol of the decayed linear-attention kernel
(decay_chunk_kernel in io_aware_exact_30_b200/csrc/decay_sm100.cuh), checked on
the CPU under random schedules with the rules of protocol_model.py (barrier tests
in the phase they are for or the next, arrivals in their phase, reads of the
versions they need, no deadlock).  Test infrastructure only.

Roles: the TMA producer, the MMA issuer, the store thread, the row warps (P and the
output; two agents), the state warps (two agents) and the warps that make Zh (two
agents).  Per step i (stage i % 2 of X, Y, Z; A and P in buffer i % 2 of tensor
memory; one buffer each of KV, O, Zh and the state's copy) the issuer does, after
A_0, KV_i = Y^T Zh_i, OX_i = X S_i, A_{i+1} = X Y^T, O_i = P Z (over OX_i).  The
output is staged in the step's Z (own_o False) or in a buffer of its own.  The step
`partial` (the last one forwards, the first one backwards) is not full: the Zh
warps clear rows of its Y and Z, and its output is not stored by TMA.
"""

from protocol_model import AsyncWork, ProtocolError, World, run_roles  # noqa: F401

NROW = NSTATE = NZH = 2

W = None


class Variant:
    def __init__(self, skip=(), state_only=False, own_o=False, partial=None, one_kvf=False,
                 one_ow=False):
        self.skip = set(skip)          # waits left out, by name
        self.state_only = state_only
        self.own_o = own_o
        self.partial = partial         # index of the step that is not full
        self.one_kvf = one_kvf         # mistake: one completion barrier for KV, not one per stage
        # mistake (this model found it): one barrier for a written output, not one per
        # stage; rows two steps ahead of the store thread left it waiting for good
        self.one_ow = one_ow


def kvf(i, v):
    return ("KVF", i) if v.one_kvf else (f"KVF{i & 1}", i >> 1)


def ow(i, v):
    return ("OW0", i) if v.one_ow else (f"OW{i & 1}", i >> 1)


def waits(v, *named):
    """A wait for the named phases that are not left out."""
    w = [(b, k) for name, b, k, on in named if on and name not in v.skip]
    if w:
        yield ("wait", w)


def producer(nc, v):
    for i in range(nc):
        s, u = i & 1, i >> 1

        def land(x, bar, i=i, s=s, u=u):
            def f():
                W.write((x, s), (x, i))
                W.bar(f"{bar}{s}").arrive(u)
            return f
        yield from waits(v, ("y_free", *kvf(i - 2, v), i >= 2))
        yield ("async", "tma", land("Y", "YF"), "tma")
        if not v.state_only:
            yield from waits(v, ("x_free", f"QSD{s}", u - 1, i >= 2))
            yield ("async", "tma", land("X", "XF"), "tma")
            free = f"OD{s}" if v.own_o else f"OR{s}"
            yield from waits(v, ("z_free", free, u - 1, i >= 2))
        yield ("async", "tma", land("Z", "ZF"), "tma")


def y_version(i, v):
    """What a product reads in Y (and Z) of step i."""
    return lambda x: (x, i, "cleared") if v.partial == i else (x, i)


def issue_a(i, v):
    s, u = i & 1, i >> 1
    yield from waits(v, ("xf", f"XF{s}", u, True), ("yf", f"YF{s}", u, True),
                     ("a_free", f"OD{s}", u - 1, i >= 2))
    if v.partial == i:
        yield from waits(v, ("a_cleared", "ZH", i, True))

    def a_mma(i=i, s=s):
        W.read(("X", s), ("X", i))
        W.read(("Y", s), y_version(i, v)("Y"))
        for r in range(NROW):
            W.write(("A", s, r), ("A", i))
    yield ("async", "mma", a_mma, f"A{s}")
    yield ("async", "mma", lambda s=s, u=u: W.bar(f"AF{s}").arrive(u))


def issuer(nc, v):
    if not v.state_only and nc:
        yield from issue_a(0, v)
    for i in range(nc):
        s, u = i & 1, i >> 1
        yield from waits(v, ("zh", "ZH", i, True), ("kve", "KVE", i - 1, i >= 1),
                         ("yf", f"YF{s}", u, v.state_only))

        def kv_mma(i=i, s=s):
            W.read(("Y", s), y_version(i, v)("Y"))
            for a in range(NZH):
                W.read(("ZH", a), i)
            for a in range(NSTATE):
                W.write(("KV", a), i)
        yield ("async", "mma", kv_mma, "KV")
        bar, k = kvf(i, v)
        yield ("async", "mma", lambda bar=bar, k=k: W.bar(bar).arrive(k))
        if v.state_only:
            continue
        yield from waits(v, ("ssf", "SSF", i, True), ("oe", "OE", i - 1, i >= 1))

        def qs_mma(i=i, s=s):
            W.read(("X", s), ("X", i))
            for a in range(NSTATE):
                W.read(("S", a), i)
            for r in range(NROW):
                W.write(("O", r), ("OX", i))
        yield ("async", "mma", qs_mma, "O")
        yield ("async", "mma", lambda s=s, u=u: W.bar(f"QSD{s}").arrive(u))
        if i + 1 < nc:
            yield from issue_a(i + 1, v)
        yield from waits(v, ("pf", "PF", i, True))

        def pz_mma(i=i, s=s):
            W.read(("Z", s), y_version(i, v)("Z"))
            for r in range(NROW):
                W.read(("A", s, r), ("P", i))
                W.write(("O", r), ("O", i))
        yield ("async", "mma", pz_mma, "O")
        yield ("async", "mma", lambda s=s, u=u: W.bar(f"OD{s}").arrive(u))


def staging(i, v, r):
    return ("STG", r) if v.own_o else ("Z", i & 1)


def store(nc, v):
    for i in range(nc):
        s, u = i & 1, i >> 1
        yield from waits(v, ("ow", *ow(i, v), True))

        def read(i=i, s=s, u=u):
            if v.partial != i:
                for r in range(NROW):
                    if v.own_o:
                        W.read(("STG", r), i)
                    else:
                        W.read(("ZO", s, r), i)
            W.bar(f"OR{s}").arrive(u)
        yield ("async", "store", read)


def rows(r, nc, v):
    def stage(i):
        s = i & 1
        if v.own_o:
            yield from waits(v, ("stage_free", f"OR{s ^ 1}", (i - 1) >> 1, i >= 1))
        if v.partial != i:
            if v.own_o:
                yield ("write", ("STG", r), i)
            else:
                # this agent's part of the stage of Z; a product or a warp that still
                # read Z there would miss its version
                yield ("write", ("ZO", s, r), i)
                yield ("write", ("Z", s), ("staged", i))
        yield ("arrive", *ow(i, v))

    for i in range(nc):
        s, u = i & 1, i >> 1
        yield from waits(v, ("af", f"AF{s}", u, True))
        yield ("read", ("A", s, r), ("A", i))
        yield ("write", ("A", s, r), ("P", i))
        yield from waits(v, ("qsd", f"QSD{s}", u, True))
        yield ("read", ("O", r), ("OX", i))
        yield ("arrive", "PF", i)
        if v.own_o and i >= 1:
            yield from stage(i - 1)
        yield from waits(v, ("od", f"OD{s}", u, True))
        yield ("read", ("O", r), ("O", i))
        yield ("arrive", "OE", i)
        if not v.own_o:
            yield from stage(i)
    if v.own_o and nc:
        yield from stage(nc - 1)


def state(a, nc, v):
    if not v.state_only and nc:
        yield ("write", ("S", a), 0)
        yield ("arrive", "SSF", 0)
    for i in range(nc):
        yield from waits(v, ("state_kvf", *kvf(i, v), True))
        yield ("read", ("KV", a), i)
        yield ("arrive", "KVE", i)
        if not v.state_only and i + 1 < nc:
            yield from waits(v, ("s_free", f"QSD{i & 1}", i >> 1, True))
            yield ("write", ("S", a), i + 1)
            yield ("arrive", "SSF", i + 1)


def make_zh(a, nc, v):
    for i in range(nc):
        s, u = i & 1, i >> 1
        yield from waits(v, ("zf", f"ZF{s}", u, True))
        yield from waits(v, ("zh_free", *kvf(i - 1, v), i >= 1))
        if v.partial == i:
            yield from waits(v, ("zh_yf", f"YF{s}", u, True))
        if v.partial == i and a == 1:
            yield ("read", ("Z", s), ("Z", i, "cleared"))
        else:
            yield ("read", ("Z", s), ("Z", i))
        if v.partial == i and a == 0:
            # (agent 0 clears for both; agent 1 follows it)
            yield ("write", ("Y", s), ("Y", i, "cleared"))
            yield ("write", ("Z", s), ("Z", i, "cleared"))
            yield ("arrive", "CLR", 0)
        yield ("write", ("ZH", a), i)
        yield ("arrive", "ZH", i)


def zh_follower(a, nc, v):
    """Agent 1 of make_zh, which in the partial step reads what agent 0 left."""
    for op in make_zh(a, nc, v):
        if op[0] == "read" and op[2][-1] == "cleared":
            yield ("wait", [("CLR", 0)])
        yield op


def run_schedule(nc, seed, variant=None, in_order=False, max_steps=200000):
    """One random schedule of one CTA working through nc chunks; raises
    ProtocolError on a violation or a deadlock."""
    global W
    v = variant or Variant()
    W = World()
    for b, n in (("PF", NROW), ("OE", NROW), ("OW0", NROW), ("OW1", NROW), ("KVE", NSTATE), ("SSF", NSTATE), ("ZH", NZH)):
        W.bar(b, n)
    roles = {"prod": producer(nc, v), "mma": issuer(nc, v)}
    for a in range(NSTATE):
        roles[f"state{a}"] = state(a, nc, v)
    roles["zh0"], roles["zh1"] = make_zh(0, nc, v), zh_follower(1, nc, v)
    if not v.state_only:
        roles["store"] = store(nc, v)
        for r in range(NROW):
            roles[f"rows{r}"] = rows(r, nc, v)
    run_roles(W, roles, seed, in_order, max_steps)
