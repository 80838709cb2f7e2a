"""The token-by-token operators of the attention library, as a user's program calls them.

Two ways to go on from a prompt, one for each kind of attention the library has:

  append    new tokens' K and V quantised into a paged e4m3 cache, one power-of-two scale
            for each page and head
  attend    softmax attention of the last few queries of each sequence over that cache
  prefill   causal linear attention with a decay for each head, chunk by chunk, from a
            state to a state
  step      its recurrent form for one token
  grad      the gradients of the chunked form

``own`` chooses between the plain form of each (elementary torch operations in 32 bits,
rounded once at the end) and the library's calls.
"""

import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------ cases --
def listed():
    return [
        # one new token for each of 64 sequences of a serving batch, at odd fill levels
        dict(name="append token", op="append", B=64, Hkv=8, T=1, d=128, page=64, cap=4096, dtype="bf16"),
        # four prompts of the large-head length enter the cache, padded to the longest
        dict(name="append prompts", op="append", B=4, Hkv=16, T=4096, d=128, page=128, cap=4096, dtype="bf16"),
        # one user: 16 heads over a 4096-token context, the latency of a single answer
        dict(name="attend single", op="attend", B=1, Hq=16, Hkv=16, T=1, d=128, page=64, cap=4096, dtype="bf16"),
        # a full serving batch with shared heads and uneven lengths
        dict(name="attend batch", op="attend", B=64, Hq=32, Hkv=8, T=1, d=128, page=64, cap=8192, dtype="bf16"),
        # the long trading day: every tick of the day in the cache, small heads, small pages
        dict(name="attend long day", op="attend", B=1, Hq=12, Hkv=12, T=1, d=64, page=16, cap=23400, dtype="fp16"),
        # five drafted tokens checked at once, few shared heads, long odd lengths
        dict(name="attend drafts", op="attend", B=16, Hq=16, Hkv=2, T=5, d=128, page=32, cap=16001, dtype="fp16"),
        # prompts of the large-head shape
        dict(name="prefill large head", op="prefill", B=4, H=16, N=4096, d=128, ragged=False, dtype="bf16"),
        # one long sequence with few small heads
        dict(name="prefill long day", op="prefill", B=1, H=12, N=23400, d=64, ragged=False, dtype="fp16"),
        # one token of one sequence
        dict(name="step single", op="step", B=1, H=16, d=128, dtype="bf16"),
        # one token for each sequence of a large batch
        dict(name="step batch", op="step", B=128, H=16, d=128, dtype="bf16"),
        # training at the GPT-2 shape, a padded batch
        dict(name="grad gpt2", op="grad", B=8, H=12, N=1024, d=64, ragged=True, dtype="fp16"),
        # training at the large-head shape
        dict(name="grad large head", op="grad", B=4, H=16, N=4096, d=128, ragged=False, dtype="bf16"),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["append", "attend", "attend", "prefill", "step", "grad"])
    d, dtype = rng.choice([64, 128]), rng.choice(["bf16", "fp16"])
    if op == "append":
        T = rng.choice([1, log(1, 4096)])
        Hkv, B = rng.choice([1, 2, 4, 8, 12, 16]), 0
        B = max(1, min(log(1, 64), (4 * 16 * 4096) // (Hkv * T)))
        return dict(op=op, B=B, Hkv=Hkv, T=T, d=d, page=rng.choice([16, 32, 64, 128]),
                    cap=max(T, log(100, 4096)), dtype=dtype)
    if op == "attend":
        Hkv, G = rng.choice([1, 2, 4, 8, 12, 16]), rng.choice([1, 2, 3, 4, 8])
        cap = log(64, 23400)
        B = max(1, min(log(1, 64), (64 * 8 * 8192) // (Hkv * cap)))
        return dict(op=op, B=B, Hq=Hkv * G, Hkv=Hkv, T=rng.choice([1, 1, rng.randint(2, 8)]), d=d,
                    page=rng.choice([16, 32, 64, 128]), cap=cap, dtype=dtype)
    if op == "step":
        return dict(op=op, B=log(1, 128), H=rng.choice([2, 4, 8, 12, 16]), d=d, dtype=dtype)
    H = rng.choice([2, 4, 8, 12, 16])
    N = log(64, 23400 if op == "prefill" else 4096)
    B = max(1, min(log(1, 8), (4 * 16 * 4096) // (H * N)))
    return dict(op=op, B=B, H=H, N=N, d=d, ragged=rng.random() < 0.5, dtype=dtype)


def spread(B, top):
    """Lengths of a batch between a third of `top` and `top`, the same for every seed but
    for their order; the longest is there."""
    return [max(1, top - int(top * 2 / 3 * ((b * 0.6180339887) % 1.0))) for b in range(B)]


def lengths(case):
    op = case["op"]
    if op == "append":  # (tokens held before, tokens that come)
        B, T, room = case["B"], case["T"], max(0, case["cap"] - case["T"])
        new = [T] * B if T == 1 else spread(B, T)
        return [x - 1 if x > 1 else 0 for x in spread(B, room + 1)], new
    if op == "attend":
        return [max(case["T"], n) for n in spread(case["B"], case["cap"])]
    return spread(case["B"], case["N"]) if case["ragged"] else [case["N"]] * case["B"]


def work(case):
    op, d = case["op"], case["d"]
    if op == "append":
        _, new = lengths(case)
        n = sum(new) * case["Hkv"] * d * 2
        return {"bytes": n * 3, "flops": 0}
    if op == "attend":
        n = sum(lengths(case))
        q = case["B"] * case["Hq"] * case["T"]
        scales = 2 * 4 * n * case["Hkv"] // case["page"]
        return {"bytes": 2 * n * case["Hkv"] * d + scales + q * (4 * d + 4),
                "flops": 4 * d * n * case["Hq"] * case["T"]}
    if op == "step":
        bh = case["B"] * case["H"]
        return {"bytes": bh * (8 * d * d + 8 * d), "flops": bh * 5 * d * d}
    rows = sum(lengths(case)) * case["H"]
    states = 2 * 4 * d * d * case["B"] * case["H"]
    # the recurrence's own arithmetic: a rank-one update and a product with the state a token
    if op == "prefill":
        return {"bytes": rows * d * 8 + states, "flops": rows * 4 * d * d}
    return {"bytes": rows * d * 14 + 2 * states, "flops": rows * 12 * d * d}


# ----------------------------------------------------------------- inputs --
def slopes(H):
    """ln of the decay of head h: -2^(-8 (h + 1) / H), memories of a token to hundreds."""
    return torch.tensor([-(2.0 ** (-8.0 * (h + 1) / H)) for h in range(H)], dtype=torch.float32, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt, d, B = DTYPES[case["dtype"]], case["d"], case["B"]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    s = dict(case)
    order = list(range(B))
    random.Random(seed).shuffle(order)
    if case["op"] in ("append", "attend"):
        Hkv, page = case["Hkv"], case["page"]
        if case["op"] == "append":
            before, new = lengths(case)
            total = [before[b] + new[b] for b in order]
            s["lens"], s["n_new"] = ints([before[b] for b in order]), ints([new[b] for b in order])
        else:
            total = [lengths(case)[b] for b in order]
            s["lens"] = ints(total)
        width = -(-max(total) // page)
        pages = B * width
        s["table"] = torch.randperm(pages, generator=g, device="cuda").to(torch.int32).view(B, width)
        # what earlier tokens left: e4m3 values over the range that normal data takes under
        # a power-of-two scale, the scales a binade or two apart
        codes, scales = [], []
        for _ in range(2):
            codes.append((normal(pages, Hkv, page, d) * 64).to(torch.float8_e4m3fn))
            scales.append(torch.exp2(-torch.randint(5, 8, (pages, Hkv), generator=g, device="cuda").float()))
        s["k8"], s["v8"], s["ks"], s["vs"] = codes[0], codes[1], scales[0], scales[1]
        if case["op"] == "append":
            s["k"], s["v"] = normal(B, Hkv, case["T"], d).to(dt), normal(B, Hkv, case["T"], d).to(dt)
        else:
            s["q"] = normal(B, case["Hq"], case["T"], d).to(dt)
        return s
    H = case["H"]
    s["decay"] = slopes(H)
    N = 1 if case["op"] == "step" else case["N"]
    for n in ("q", "k", "v"):
        s[n] = normal(B, H, N, d).to(dt)
    s["state"] = normal(B, H, d, d)
    if case["op"] == "step":
        s["next"] = torch.empty_like(s["state"])
        return s
    s["lens"] = ints([lengths(case)[b] for b in order]) if case["ragged"] else None
    if case["op"] == "grad":
        s["dout"], s["dstate"] = normal(B, H, N, d).to(dt), normal(B, H, d, d)
    return s


# ------------------------------------------------------------ plain forms --
def pow2_scale(amax):
    """The least power of two s with amax <= 448 s; 0 for amax 0."""
    m, e = torch.frexp(amax)  # amax = m 2^e, 1/2 <= m < 1;  448 = 0.875 2^9
    e = torch.where(m <= 0.875, e - 9, e - 8).clamp(min=-126)
    return torch.where(amax > 0, torch.ldexp(torch.ones_like(amax), e), torch.zeros_like(amax))


def plain_append(x, codes, scale, table, lens, n_new):
    """The new rows of x (B, Hkv, T, d) at positions lens .. lens + n_new - 1."""
    B, Hkv, T, d = x.shape
    page, width = codes.shape[2], table.shape[1]
    W = (T + page - 2) // page + 1  # pages that T tokens can touch
    fill = (lens % page).long()
    at = torch.arange(W * page, device=x.device)
    t = at[None] - fill[:, None]  # the token at each slot of the touched pages
    is_new = (t >= 0) & (t < n_new[:, None])
    rows = x.float().gather(2, t.clamp(0, T - 1)[:, None, :, None].expand(B, Hkv, W * page, d))
    rows = torch.where(is_new[:, None, :, None], rows, torch.zeros((), device=x.device))
    rows = rows.view(B, Hkv, W, page, d).transpose(1, 2)  # (B, W, Hkv, page, d)
    is_new = is_new.view(B, W, 1, page, 1)
    slot = (lens // page).long()[:, None] + torch.arange(W, device=x.device)[None]
    ids = table.long().gather(1, slot.clamp(max=width - 1))
    held = (t < 0).view(B, W, 1, page, 1)
    old = torch.where(held[:, :, :, 0, 0], scale[ids], torch.zeros((), device=x.device))
    new = torch.maximum(pow2_scale(rows.abs().amax(dim=(3, 4))), old)
    inv = torch.where(new > 0, 1 / new, torch.zeros_like(new))[..., None, None]
    was = codes[ids].float()
    out = torch.where(is_new, rows * inv, torch.where(held, was * (old[..., None, None] * inv), was))
    touched = is_new.any(dim=3).view(B, W)
    codes[ids[touched]] = out.to(torch.float8_e4m3fn)[touched]
    scale[ids[touched]] = new[touched]


def plain_attend(q, k8, v8, ks, vs, table, lens):
    B, Hq, T, d = q.shape
    Hkv, page = k8.shape[1], k8.shape[2]
    L, G = table.shape[1] * page, Hq // Hkv
    ids = table.long()

    def values(codes, scale):  # (B, Hkv, L, d)
        x = codes[ids].float() * scale[ids][..., None, None]
        return x.transpose(1, 2).reshape(B, Hkv, L, d)

    k, v = values(k8, ks), values(v8, vs)
    rows = q.float().view(B, Hkv, G * T, d)
    s = rows @ k.transpose(2, 3) * (1.0 / math.sqrt(d))
    end = lens[:, None] - (T - 1 - torch.arange(T, device=q.device))[None]  # keys query t sees
    hide = torch.arange(L, device=q.device)[None, None] >= end[:, :, None]  # (B, T, L)
    s = s.view(B, Hkv, G, T, L).masked_fill(hide[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True).clamp(min=-3e38)
    p = torch.exp(s - m)
    total = p.sum(-1, keepdim=True)
    o = (p.view(B, Hkv, G * T, L) @ v).view(B, Hkv, G, T, d) / total
    lse = (m + torch.log(total)).squeeze(-1)
    return o.view(B, Hq, T, d).to(q.dtype), lse.view(B, Hq, T)


def powers(decay, n):
    """exp(decay n) for whole numbers n (broadcast against (H,) in front)."""
    return torch.exp(decay.double() * n).float()


def plain_prefill(q, k, v, decay, state, lens, scale):
    B, H, N, d = q.shape
    C = 128
    nc = -(-N // C)
    dev = q.device
    n = torch.full((B,), N, device=dev) if lens is None else lens
    live = (torch.arange(N, device=dev)[None] < n[:, None])[:, None, :, None]
    zero = torch.zeros((), device=dev)

    def chunks(x):
        x = torch.where(live, x.float(), zero)
        return torch.nn.functional.pad(x, (0, 0, 0, nc * C - N)).view(B, H, nc, C, d)

    qc, kc, vc = chunks(q), chunks(k), chunks(v)
    i = torch.arange(C, device=dev)
    gap = i[:, None] - i[None]
    w = torch.where(gap >= 0, powers(decay[:, None, None], gap.clamp(min=0)), zero)  # (H, C, C)
    o = ((qc @ kc.transpose(3, 4)) * w[None, :, None]) @ vc
    # the state in front of each chunk
    kv = (kc * powers(decay[:, None], C - 1 - i)[None, :, None, :, None]).transpose(3, 4) @ vc
    c = torch.arange(nc, device=dev)
    apart = c[:, None] - 1 - c[None]
    wc = torch.where(apart >= 0, powers(decay[:, None, None], C * apart.clamp(min=0)), zero)
    before = torch.einsum("hce,bhexy->bhcxy", wc, kv)
    before = before + powers(decay[:, None], C * c)[None, :, :, None, None] * state[:, :, None]
    o = o + powers(decay[:, None], i + 1)[None, :, None, :, None] * (qc @ before)
    o = (o.reshape(B, H, nc * C, d)[:, :, :N] * scale).to(q.dtype)
    return torch.where(live, o, torch.zeros_like(o)), after(k, v, decay, state, n, live)


def after(k, v, decay, state, n, live):
    """The state after n tokens."""
    N = k.shape[2]
    left = (n[:, None] - 1 - torch.arange(N, device=k.device)[None]).clamp(min=0)[:, None]  # (B, 1, N)
    zero = torch.zeros((), device=k.device)
    kw = torch.where(live, k.float(), zero) * powers(decay[None, :, None], left)[..., None]
    end = powers(decay[None], n[:, None])[..., None, None] * state
    return end + kw.transpose(2, 3) @ torch.where(live, v.float(), zero)


def plain_step(q, k, v, decay, state, scale):
    new = powers(decay, 1)[None, :, None, None] * state + k.float().transpose(2, 3) * v.float()
    return ((q.float() @ new) * scale).to(q.dtype), new


def plain_grad(q, k, v, decay, dout, state, dstate, lens, scale):
    B, H, N, d = q.shape
    dev = q.device
    n = torch.full((B,), N, device=dev) if lens is None else lens
    i = torch.arange(N, device=dev)
    live = (i[None] < n[:, None])[:, None, :, None]
    zero = torch.zeros((), device=dev)
    qf, kf, vf, gf = (torch.where(live, x.float(), zero) for x in (q, k, v, dout))
    gap = i[:, None] - i[None]
    w = torch.where(gap >= 0, powers(decay[:, None, None], gap.clamp(min=0)), zero)[None] * scale
    p = (qf @ kf.transpose(2, 3)) * w
    dp = (gf @ vf.transpose(2, 3)) * w
    first = powers(decay[:, None], i + 1)[None, :, :, None] * scale
    left = powers(decay[None, :, None], (n[:, None] - 1 - i[None]).clamp(min=0)[:, None])[..., None]
    dq = dp @ kf + first * (gf @ state.transpose(2, 3))
    dk = dp.transpose(2, 3) @ qf + left * (vf @ dstate.transpose(2, 3))
    dv = p.transpose(2, 3) @ gf + left * (kf @ dstate)
    ds = powers(decay[None], n[:, None])[..., None, None] * dstate + (first * qf).transpose(2, 3) @ gf
    return [torch.where(live, x, zero).to(q.dtype) for x in (dq, dk, dv)] + [ds]


def run(s):
    if own:
        return run_own(s)
    op = s["op"]
    if op == "append":
        plain_append(s["k"], s["k8"], s["ks"], s["table"], s["lens"], s["n_new"])
        plain_append(s["v"], s["v8"], s["vs"], s["table"], s["lens"], s["n_new"])
        return {n: s[n] for n in ("k8", "v8", "ks", "vs")}
    if op == "attend":
        o, lse = plain_attend(s["q"], s["k8"], s["v8"], s["ks"], s["vs"], s["table"], s["lens"])
        return {"o": o, "lse": lse}
    scale = 1.0 / math.sqrt(s["d"])
    if op == "step":
        o, state = plain_step(s["q"], s["k"], s["v"], s["decay"], s["state"], scale)
        return {"o": o, "state": state}
    if op == "prefill":
        o, state = plain_prefill(s["q"], s["k"], s["v"], s["decay"], s["state"], s["lens"], scale)
        return {"o": o, "state": state}
    got = plain_grad(s["q"], s["k"], s["v"], s["decay"], s["dout"], s["state"], s["dstate"], s["lens"], scale)
    return dict(zip(("dq", "dk", "dv", "dstate"), got))


def run_own(s):
    from io_aware_exact_30_b200 import attn
    op = s["op"]
    if op == "append":
        cache = attn.Cache8(s["k8"], s["v8"], s["ks"], s["vs"])
        attn.cache_append(s["k"], s["v"], cache, s["table"], s["lens"], n_new=s["n_new"])
        return {n: s[n] for n in ("k8", "v8", "ks", "vs")}
    if op == "attend":
        cache = attn.Cache8(s["k8"], s["v8"], s["ks"], s["vs"])
        o, lse = attn.cache_attend(s["q"], cache, s["table"], s["lens"], causal=True)
        return {"o": o, "lse": lse}
    if op == "step":
        o, state = attn.decay_step(s["q"], s["k"], s["v"], s["decay"], s["state"], state_out=s["next"])
        return {"o": o, "state": state}
    if op == "prefill":
        o, state = attn.decay_forward(s["q"], s["k"], s["v"], s["decay"], state=s["state"], lens=s["lens"])
        return {"o": o, "state": state}
    got = attn.decay_backward(s["q"], s["k"], s["v"], s["decay"], s["dout"], state=s["state"],
                              dstate=s["dstate"], lens=s["lens"])
    return dict(zip(("dq", "dk", "dv", "dstate"), got))


# ------------------------------------------------------------------ exact --
def e4m3_values(device):
    """The 127 magnitudes of e4m3, ascending."""
    code = torch.arange(127, device=device)
    e, m = code >> 3, (code & 7).double()
    return torch.where(e > 0, (1 + m / 8) * torch.exp2(e.double() - 7), m / 8 * 2.0 ** -6)


def e4m3_nearest(x):
    """x in 64 bits to the nearest e4m3 value, ties to the even code."""
    grid = e4m3_values(x.device)
    a = x.abs()
    lo = (torch.searchsorted(grid, a.contiguous(), right=True) - 1).clamp(0, 125)
    up = grid[lo + 1] - a
    down = a - grid[lo]
    take = (up < down) | ((up == down) & (lo % 2 == 1))
    return torch.where(take, grid[lo + 1], grid[lo]) * torch.sign(x)


def exact_append(x, codes, scale, table, lens, n_new):
    codes, scale = codes.double(), scale.double()
    page = codes.shape[2]
    for b in range(x.shape[0]):
        at, end = int(lens[b]), int(lens[b]) + int(n_new[b])
        while at < end:  # page by page
            first = at % page
            upto = min(end, at - first + page)
            p = int(table[b, at // page])
            rows = x[b, :, at - int(lens[b]):upto - int(lens[b])].double()
            top = rows.abs().amax(dim=(1, 2))
            s = torch.where(top > 0, torch.exp2(torch.ceil(torch.log2(top / 448))), torch.zeros_like(top))
            if first:
                s = torch.maximum(s, scale[p])
                codes[p, :, :first] = e4m3_nearest(codes[p, :, :first] * (scale[p] / s)[:, None, None])
            codes[p, :, first:first + upto - at] = e4m3_nearest(rows / s[:, None, None])
            scale[p] = s
            at = upto
    return codes, scale


def exact_attend(s):
    q, table = s["q"].double(), s["table"].long()
    B, Hq, T, d = q.shape
    Hkv, page = s["k8"].shape[1], s["k8"].shape[2]
    o, lse = torch.empty_like(q), torch.empty(B, Hq, T, dtype=torch.float64, device=q.device)
    for b in range(B):
        n = int(s["lens"][b])
        ids = table[b, :-(-n // page)]
        k, v = ((s[c][ids].double() * s[f][ids].double()[..., None, None]).transpose(0, 1).reshape(Hkv, -1, d)[:, :n]
                for c, f in (("k8", "ks"), ("v8", "vs")))
        for t in range(T):
            end = n - (T - 1 - t)
            x = torch.einsum("hgd,hnd->hgn", q[b, :, t].view(Hkv, -1, d), k[:, :end]) / math.sqrt(d)
            lse[b, :, t] = torch.logsumexp(x, -1).view(-1)
            o[b, :, t] = torch.einsum("hgn,hnd->hgd", torch.softmax(x, -1), v[:, :end]).reshape(Hq, d)
    return {"o": o, "lse": lse}


def exact_recurrence(s):
    """The definition, token by token: S <- decay S + k v^T, o = scale q S; and back."""
    B, H, N, d = s["q"].shape
    q, k, v = (s[n].double() for n in ("q", "k", "v"))
    lam = torch.exp(s["decay"].double())[None, :, None, None]
    scale = 1.0 / math.sqrt(d)
    n = s.get("lens")
    n = torch.full((B,), N, device=q.device) if n is None else n
    S = s["state"].double()
    grad = s["op"] == "grad"
    g = s["dout"].double() if grad else None
    o, dq, dk, dv = torch.zeros_like(q), torch.zeros_like(q), torch.zeros_like(q), torch.zeros_like(q)
    last = int(n.max())
    least = int(n.min())
    for t in range(last):
        new = lam * S + k[:, :, t, :, None] * v[:, :, t, None, :]
        if t >= least:
            new = torch.where((t < n)[:, None, None, None], new, S)
        S = new
        if grad:
            dq[:, :, t] = (S @ g[:, :, t, :, None]).squeeze(-1) * scale
        else:
            o[:, :, t] = (q[:, :, t, None] @ S).squeeze(2) * scale
    if not grad:
        if s.get("lens") is not None:
            o *= (torch.arange(N, device=q.device)[None] < n[:, None])[:, None, :, None]
        return {"o": o, "state": S}
    G = s["dstate"].double()  # the gradient of the state after token t
    for t in range(last - 1, -1, -1):
        new = G + scale * q[:, :, t, :, None] * g[:, :, t, None, :]
        on = (t < n)[:, None, None, None]
        new = torch.where(on, new, G) if t >= least else new
        dv[:, :, t] = (k[:, :, t, None] @ new).squeeze(2)
        dk[:, :, t] = (new @ v[:, :, t, :, None]).squeeze(-1)
        G = torch.where(on, lam * new, new) if t >= least else lam * new
    live = (torch.arange(N, device=q.device)[None] < n[:, None])[:, None, :, None]
    return {"dq": dq * live, "dk": dk * live, "dv": dv * live, "dstate": G}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append":
        k8, ks = exact_append(s["k"], s["k8"], s["ks"], s["table"], s["lens"], s["n_new"])
        v8, vs = exact_append(s["v"], s["v8"], s["vs"], s["table"], s["lens"], s["n_new"])
        return {"k8": k8, "v8": v8, "ks": ks, "vs": vs}
    if case["op"] == "attend":
        return exact_attend(s)
    return exact_recurrence(s)
