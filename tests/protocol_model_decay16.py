"""The mbarrier protocol of the decayed linear-attention kernel's fp16 form, which adds to
protocol_model_decay.py's roles the powers of two of its 16-bit operands:

  * Zh warps survey X and Y of a step before its Z lands, for bounds of A and of the state's
    growth (SV, a barrier for either step parity): in four slots each, X's maxima by warp (SX)
    and Y's, which meet in one word (SY), cleared by one warp two steps ahead.  The issuer waits for the survey in
    front of A, the row warps read it in front of P, the state warps in front of KVE;
  * state warps meet once, over the state that they begin with (SM), and write what takes
    the power out of each copy of the state (SD, two slots), which the row warps read with
    X S;
  * Zh warps read Z before they wait for the previous product, and write what takes
    their power out (ZD, four slots), which the state warps read with the sums.

Two agents of each role stand for its warps.  Test infrastructure only.
"""

import protocol_model_decay as pd
from protocol_model_decay import NROW, NSTATE, NZH, ProtocolError, Variant, World, run_roles, waits  # noqa: F401


def issuer(nc, v):
    """The base model's; A of a step behind its survey (which AF then implies for the rows)."""
    step = 0
    for op in pd.issuer(nc, v):
        if op[0] == "async" and len(op) == 4 and op[3] in ("A0", "A1"):
            yield from waits(v, ("sv", f"SV{step & 1}", step >> 1, True))
            step += 1
        yield op


def read_survey(i):  # (Y's part)
    for a in range(NZH):
        yield ("read", ("SY", i & 3, a), i)


def rows(r, nc, v):
    def stage(i):
        yield from waits(v, ("stage_free", f"OR{(i & 1) ^ 1}", (i - 1) >> 1, i >= 1))
        if v.partial != i:
            yield ("write", ("STG", r), i)
        yield ("arrive", *pd.ow(i, v))

    for i in range(nc):
        s, u = i & 1, i >> 1
        yield from waits(v, ("af", f"AF{s}", u, True))
        yield from read_survey(i)
        yield ("read", ("SX", i % v.sx_slots, r), i)
        yield ("read", ("A", s, r), ("A", i))
        yield ("write", ("A", s, r), ("P", i))
        yield from waits(v, ("qsd", f"QSD{s}", u, True))
        yield ("read", ("O", r), ("OX", i))
        yield ("read", ("SD", i % v.sd_slots), i)
        yield ("arrive", "PF", i)
        if i >= 1:
            yield from stage(i - 1)
        yield from waits(v, ("od", f"OD{s}", u, True))
        yield ("read", ("O", r), ("O", i))
        yield ("arrive", "OE", i)
    if nc:
        yield from stage(nc - 1)


def state(a, nc, v):
    def copy(i):
        if a == 0:
            yield ("write", ("SD", i % v.sd_slots), i)
        yield ("write", ("S", a), i)
        yield ("arrive", "SSF", i)

    if not v.state_only:
        yield ("write", ("SM", a), 0)
        yield ("arrive", "SM", 0)
        yield from waits(v, ("sm", "SM", 0, True))
        for b in range(NSTATE):
            yield ("read", ("SM", b), 0)
        yield from copy(0)
    for i in range(nc):
        s, u = i & 1, i >> 1
        yield from waits(v, ("state_kvf", *pd.kvf(i, v), True))
        for b in range(NZH):
            yield ("read", ("ZD", i % v.zd_slots, b), i)
        yield ("read", ("KV", a), i)
        if not v.state_only:
            yield from read_survey(i)
        yield ("arrive", "KVE", i)
        if not v.state_only and i + 1 < nc:
            yield from waits(v, ("s_free", f"QSD{s}", u, True))
            yield from copy(i + 1)


def make_zh(a, nc, v):
    for i in range(nc):
        s, u = i & 1, i >> 1
        if not v.state_only:
            yield from waits(v, ("sv_xf", f"XF{s}", u, True), ("sv_yf", f"YF{s}", u, True))
            yield ("read", ("X", s), ("X", i))
            # (rows of Y past the end may be cleared meanwhile; they are not looked at)
            yield ("live", ("Y", s), i)
            yield ("write", ("SX", i % v.sx_slots, a), i)
            yield ("read", ("SY", i & 3, a), "clear")
            yield ("write", ("SY", i & 3, a), i)
            yield ("arrive", f"SV{s}", u)
        yield from waits(v, ("zf", f"ZF{s}", u, True))
        # Z goes to registers here; its dead rows are cleared later, by the thread that read
        # them (the version the products need carries the clearing)
        yield ("read", ("Z", s, a), ("Z", i))
        yield ("write", ("ZD", i % v.zd_slots, a), i)
        yield from waits(v, ("zh_free", *pd.kvf(i - 1, v), i >= 1))
        if a == 0 and not v.state_only:
            for b in range(NZH):
                yield ("write", ("SY", (i + v.clear_ahead) & 3, b), "clear")
        if v.partial == i:
            yield from waits(v, ("zh_yf", f"YF{s}", u, True))
            yield ("write", ("Z", s, a), ("Z", i, "cleared"))
            yield ("write", ("Y", s, a), ("Y", i, "cleared"))
        yield ("write", ("ZH", a), i)
        yield ("arrive", "ZH", i)


class Variant16(Variant):
    def __init__(self, zd_slots=4, sx_slots=4, sd_slots=2, clear_ahead=2, **kw):
        super().__init__(own_o=True, **kw)
        self.clear_ahead = clear_ahead  # steps from a survey to the slot that it clears
        self.zd_slots, self.sx_slots, self.sd_slots = zd_slots, sx_slots, sd_slots


class Parts(World):
    """Y and Z as the parts that each Zh agent reads and clears."""

    def write(self, key, value):
        if key[0] in ("Y", "Z") and len(key) == 2:
            for a in range(NZH):
                super().write((*key, a), value)
        else:
            super().write(key, value)

    def read(self, key, want):
        if key[0] in ("Y", "Z") and len(key) == 2:
            for a in range(NZH):
                super().read((*key, a), want)
        else:
            super().read(key, want)


def live_rows(role):
    """("live", key, i): a read of the live rows of step i, cleared or not."""
    for op in role:
        if op[0] == "live":
            for a in range(NZH):
                have = pd.W.buf.get((*op[1], a))
                if have is None or have[1] != op[2]:
                    raise ProtocolError(f"read of {op[1]}: wants step {op[2]}, holds {have}")
        else:
            yield op


def run_schedule(nc, seed, variant=None, in_order=False, max_steps=200000):
    v = variant or Variant16()
    pd.W = W = Parts()
    for b, n in (("PF", NROW), ("OE", NROW), ("OW0", NROW), ("OW1", NROW), ("KVE", NSTATE), ("SSF", NSTATE),
                 ("ZH", NZH), ("SM", NSTATE), ("SV0", NZH), ("SV1", NZH)):
        W.bar(b, n)
    for i in range(4):
        for a in range(NZH):
            W.write(("SY", i, a), "clear")
    roles = {"prod": pd.producer(nc, v), "mma": issuer(nc, v)}
    for a in range(NSTATE):
        roles[f"state{a}"] = state(a, nc, v)
    for a in range(NZH):
        roles[f"zh{a}"] = live_rows(make_zh(a, nc, v))
    if not v.state_only:
        roles["store"] = pd.store(nc, v)
        for r in range(NROW):
            roles[f"rows{r}"] = rows(r, nc, v)
    run_roles(W, roles, seed, in_order, max_steps)
