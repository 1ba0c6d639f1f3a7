"""What stands around attention in a layer, as workloads: the rotation of queries and keys by their positions, alone or with
their norms in the same pass, forward and backward; the same on the way into the paged cache; attention with a sliding
window and a few first tokens that stay visible, forward and backward, and over the paged cache; a decoding step of the three.

A case says the sizes; the lengths of its sequences and requests follow from the case alone, the contents from the seed.
``run`` computes a case in elementary torch operations, or (``own``) by the calls a user makes of this package; ``exact``
computes it from the definitions in 64 bits.
"""
import math
import random

import torch

own = False

DEV = "cuda"
EPS = 1e-6


def listed():
    return [
        # one new token of a short-headed layer far into a text, a quarter of the head rotated in neighbouring pairs: a call's least work
        dict(name="rope one token", op="rope", B=1, N=1, Hq=12, Hk=12, d=64, rot=16, inter=True, norm=False, grad=False, scaled="none",
             start=1000000, rows=False, fused=True),
        # a long prompt's queries and keys out of one projection, rotated by frequencies stretched for long texts
        dict(name="rope long prompt", op="rope", B=1, N=16384, Hq=32, Hk=8, d=128, rot=128, inter=False, norm=False, grad=False,
             scaled="ramp", start=0, rows=False, fused=True),
        # a training step's pass of it with the norms: forward, then the gradients of inputs and weights
        dict(name="norm rope train", op="rope", B=4, N=4096, Hq=32, Hk=8, d=128, rot=128, inter=False, norm=True, grad=True,
             scaled="none", start=0, rows=False, fused=True),
        # the same for the short heads, an odd length, positions of its own for each sequence
        dict(name="norm rope train d64", op="rope", B=8, N=1001, Hq=12, Hk=12, d=64, rot=64, inter=True, norm=True, grad=True,
             scaled="linear", start=77, rows=True, fused=False),
        # the new tokens of a decoding batch on their way into the cache: norm, rotation and store
        dict(name="rope store decode", op="store", R=64, ctx=4096, new=1, chunks=0, ps=16, pad=0, lens=1, Hq=32, Hk=8, d=128, rot=128,
             inter=False, norm=True, scaled="none", fp8=False),
        # the tokens of long prompts into an 8-bit cache, half of each head rotated
        dict(name="rope store prompts e4m3", op="store", R=5, ctx=1, new=4095, chunks=5, ps=64, pad=1, lens=2, Hq=32, Hk=8, d=128,
             rot=64, inter=False, norm=False, scaled="base", fp8=True),
        # a long prompt through a layer with a wide window, grouped heads: the forward alone
        dict(name="window prompt", op="window", B=1, N=16384, ctx=0, Hq=32, Hk=8, d=128, W=4096, S=4, pad=False, grad=False, lens=3),
        # a training step's attention with a narrow window, grouped heads
        dict(name="window train", op="window", B=4, N=4096, ctx=0, Hq=32, Hk=8, d=128, W=512, S=4, pad=False, grad=True, lens=4),
        # short heads, a padded batch of ragged lengths, no first tokens kept
        dict(name="window train d64 padded", op="window", B=8, N=1001, ctx=0, Hq=12, Hk=12, d=64, W=200, S=0, pad=True, grad=True,
             lens=5),
        # a decoding batch of long texts of which the window sees a part
        dict(name="window decode", op="attn", R=64, ctx=8192, new=1, chunks=0, ps=16, pad=0, lens=6, Hq=32, Hk=8, d=128, W=1024, S=4,
             fp8=False),
        # chunks of long prompts over an 8-bit cache, more first tokens than one tile holds
        dict(name="window chunks e4m3", op="attn", R=3, ctx=8192, new=1024, chunks=3, ps=64, pad=2, lens=7, Hq=32, Hk=8, d=128, W=2000,
             S=130, fp8=True),
        # a decoding step of one layer: positions, norm with rotation and store, attention in the window
        dict(name="window step", op="step", R=128, ctx=4096, new=1, chunks=0, ps=16, pad=0, lens=8, Hq=16, Hk=8, d=64, rot=64,
             inter=False, norm=True, scaled="none", W=500, S=4, fp8=False),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi) + 0.49)))))

    op = rng.choice(["rope", "rope", "store", "window", "window", "attn", "attn", "step"])
    d = rng.choice([64, 128])
    Hk, G = rng.choice([1, 2, 4, 8, 12]), rng.choice([1, 2, 3, 4, 5, 8])
    if Hk * G > 40:
        G = 2
    c = dict(op=op, Hq=Hk * G, Hk=Hk, d=d)
    if op in ("rope", "store", "step"):
        c.update(rot=rng.choice([d, d, d // 2, 16, 48]), inter=rng.random() < 0.5, norm=rng.random() < 0.6,
                 scaled=rng.choice(["none", "linear", "base", "ramp"]))
    if op == "rope":
        B = rng.choice([1, 1, 2, 3, 8])
        c.update(B=B, N=log(1, 16384 // B), grad=rng.random() < 0.5, start=rng.choice([0, 0, log(1, 1 << 20)]),
                 rows=rng.random() < 0.3, fused=rng.random() < 0.6)
        return c
    if op == "window":
        B, W, S = rng.choice([1, 1, 2, 3, 5]), log(1, 4096), rng.choice([0, 0, 1, 4, 64, 130, 300])
        ctx = rng.choice([0, 0, 0, log(1, 4096)])
        N = log(1, max(1, min(16384 // B, int(1.2e11 / (B * c["Hq"] * d * (W + S))))))
        c.update(B=B, N=N, ctx=ctx, W=W, S=S, pad=rng.random() < 0.3, grad=rng.random() < 0.6, lens=rng.randrange(1 << 20))
        return c
    ps, lens, pad = rng.choice([16, 32, 64, 128]), rng.randrange(1 << 20), rng.choice([0, 0, 1, rng.randrange(2, 400)])
    c.update(ps=ps, lens=lens, pad=pad, fp8=rng.random() < 0.5)
    if op == "store":
        R = log(1, 200)
        c.update(R=R, ctx=log(1, 2000), new=log(1, 16000 // R), chunks=rng.choice([0, R]))
        return c
    c.update(W=log(1, 4096), S=rng.choice([0, 1, 4, 64, 130, 300]))
    if op == "step" or rng.random() < 0.5:  # decoding: one to a few new tokens for every request
        R, new = log(1, 96), rng.choice([1, 1, 2, 5])
        c.update(R=R, new=new, ctx=log(1, min(32768, 1600000 // (R * Hk * new))), chunks=R if new > 1 else 0)
        return c
    R, new = rng.choice([1, 2, 3, 5, 9]), log(2, 1500)  # chunks of prompts, alone or with decoding requests
    c.update(R=R, new=new, ctx=log(1, max(64, min(16384, 400000000 // (R * new * c["Hq"])))), chunks=rng.choice([1, R]))
    return c


def lengths(case):
    """Tokens in the cache and new tokens of each request: the first request has the most of both, ``chunks`` of the requests
    bring up to ``new`` tokens, the others one."""
    r = random.Random(case["lens"])
    R, most = case["R"], case["ctx"]
    c = [most] + [r.randint(0, most) for _ in range(R - 1)]
    n = [case["new"]] + [r.randint(1 + case["new"] // 2, max(1 + case["new"] // 2, case["new"])) for _ in range(R - 1)]
    return c, [x if i < max(1, case["chunks"]) else 1 for i, x in enumerate(n)]


def sizes(case):
    """Query rows and keys of each sequence of a padded batch."""
    r = random.Random(case["lens"])
    B, N, ctx = case["B"], case["N"], case["ctx"]
    q = [N] + [r.randint(1, N) for _ in range(B - 1)] if case["pad"] else [N] * B
    return q, [x + ctx for x in q]


def pages(n, ps):
    return -(-n // ps)


def angles(case):
    """The pairs' angles a position, and the factor of cosine and sine."""
    r = case["rot"]
    base = 10000.0 * (8.0 ** (r / (r - 2)) if case["scaled"] == "base" else 1.0)
    f = [base ** (-2.0 * i / r) for i in range(r // 2)]
    if case["scaled"] == "linear":
        f = [x / 8 for x in f]
    if case["scaled"] == "ramp":  # high frequencies as they are, low ones stretched, a ramp between them
        turns = [4096 * x / (2 * math.pi) for x in f]
        keep = [min(1.0, max(0.0, (t - 1) / 31)) for t in turns]
        f = [x * k + x / 8 * (1 - k) for x, k in zip(f, keep)]
    return f, 1.0 + 0.1 * math.log(8) if case["scaled"] == "ramp" else 1.0


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    op, Hq, Hk, d = case["op"], case["Hq"], case["Hk"], case["d"]
    s = dict(case)

    def normal(*shape):
        return torch.randn(shape, generator=g, device=DEV).to(torch.bfloat16)

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device=DEV)

    if "rot" in case:
        f, s["factor"] = angles(case)
        s["freqs"] = torch.tensor(f, dtype=torch.float64, device=DEV)
        s["wq"], s["wk"] = ((1 + 0.2 * torch.randn(d, generator=g, device=DEV)).to(torch.bfloat16) if case["norm"] else None for _ in range(2))
    if op == "rope":
        B, N = case["B"], case["N"]
        if case["fused"]:  # slices of one projection's output
            x = normal(B, N, Hq + 2 * Hk, d)
            s["q"], s["k"] = x[:, :, :Hq].transpose(1, 2), x[:, :, Hq:Hq + Hk].transpose(1, 2)
        else:
            s["q"], s["k"] = normal(B, N, Hq, d).transpose(1, 2), normal(B, N, Hk, d).transpose(1, 2)
        at = torch.arange(N, dtype=torch.int32, device=DEV) + case["start"]
        s["pos"] = (at + 13 * torch.arange(B, dtype=torch.int32, device=DEV)[:, None]).contiguous() if case["rows"] else at
        if case["grad"]:
            s["dyq"], s["dyk"] = normal(B, Hq, N, d), normal(B, Hk, N, d)
        return s
    s["scale"] = 1.0 / math.sqrt(d)
    if op == "window":
        B, N, Nk = case["B"], case["N"], case["N"] + case["ctx"]
        s["q"], s["k"], s["v"] = normal(B, Hq, N, d), normal(B, Hk, Nk, d), normal(B, Hk, Nk, d)
        if case["grad"]:
            s["dO"] = normal(B, Hq, N, d)
        a, b = sizes(case)
        s["lens_q"], s["lens_k"] = (ints(a), ints(b)) if case["pad"] else (None, None)
        return s
    c, n = lengths(case)
    R, ps, T = case["R"], case["ps"], sum(n) + case["pad"]
    have = [pages(a + b, ps) for a, b in zip(c, n)]
    width, P = max(have), sum(have) + 7
    perm = torch.randperm(P, generator=g, device=DEV).to(torch.int32)  # pages in no order
    held = torch.tensor(have, device=DEV)
    col = torch.arange(width, device=DEV)
    at = held.cumsum(0) - held
    s["table"] = torch.where(col < held[:, None], perm[(at[:, None] + col).clamp(max=P - 1)], -1).to(torch.int32).contiguous()
    start = [0]
    for x in n:
        start.append(start[-1] + x)
    s.update(T=T, P=P, total=start[-1], max_new=max(n), query_start=ints(start), seq_lens=ints([a + b for a, b in zip(c, n)]))
    where = [p for a, b in zip(c, n) for p in range(a, a + b)]
    s["pos"] = ints(where + [0] * case["pad"])
    of = torch.tensor([r for r, b in enumerate(n) for _ in range(b)], device=DEV)
    here = s["pos"][:start[-1]].long()
    s["slots"] = torch.full((T,), -1, dtype=torch.int32, device=DEV)
    s["slots"][:start[-1]] = s["table"][of, here // ps] * ps + (here % ps).int()
    x = normal(T, Hq + 2 * Hk, d)  # slices of one projection's output
    s["q"], s["k"], s["v"] = x[:, :Hq], x[:, Hq:Hq + Hk], x[:, Hq + Hk:]
    s["fk"], s["fv"] = (0.0123, 0.0171) if case["fp8"] else (1.0, 1.0)
    for name, f in (("k_cache", s["fk"]), ("v_cache", s["fv"])):
        x = torch.randn((P, Hk, ps, d), generator=g, device=DEV)
        s[name] = (x / f).clamp_(-448, 448).to(torch.float8_e4m3fn) if case["fp8"] else x.to(torch.bfloat16)
        del x
    s["q_out"] = torch.zeros((T, Hq, d), dtype=torch.bfloat16, device=DEV)
    s["positions"] = torch.zeros(T, dtype=torch.int32, device=DEV)
    if op != "store":
        s["o"] = torch.zeros((T, Hq, d), dtype=torch.bfloat16, device=DEV)
        s["lse"] = torch.zeros((T, Hq), dtype=torch.float32, device=DEV)
        # where each request's rows lie in a rectangle of R by the most new tokens, and back
        t = torch.arange(s["max_new"], device=DEV)
        s["row_of"] = (s["query_start"][:-1, None] + t).clamp(max=T - 1).long()
        s["rows"] = torch.tensor([r * s["max_new"] + i for r, b in enumerate(n) for i in range(b)], device=DEV)
    return s


# ---------------------------------------------------------------- the plain forms
def turn(x, c, sn, inter):
    """The pairs (a, b) of the last axis as (a c - b s, b c + a s)."""
    if inter:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack((a * c - b * sn, b * c + a * sn), -1).flatten(-2)
    a, b = x.chunk(2, -1)
    return torch.cat((a * c - b * sn, b * c + a * sn), -1)


def cos_sin(s, pos, dtype):
    a = pos.double()[..., None] * s["freqs"]  # far positions: angles in 64 bits
    return (a.cos() * s["factor"]).to(dtype), (a.sin() * s["factor"]).to(dtype)


def normed(x, w):
    r = (x.square().mean(-1, keepdim=True) + EPS).rsqrt()
    return x * r * w.to(x.dtype), r


def plain_rope(s, x, w, c, sn, dtype=torch.float32):
    x = x.to(dtype)
    if w is not None:
        x = normed(x, w)[0]
    r = s["rot"]
    return torch.cat((turn(x[..., :r], c, sn, s["inter"]), x[..., r:]), -1)


def plain_rope_grad(s, x, w, dy, c, sn):
    r, dy = s["rot"], dy.float()
    dz = torch.cat((turn(dy[..., :r], c, -sn, s["inter"]), dy[..., r:]), -1)
    if w is None:
        return dz.to(torch.bfloat16), None
    x = x.float()
    rstd = (x.square().mean(-1, keepdim=True) + EPS).rsqrt()
    xh, g = x * rstd, dz * w.float()
    dx = rstd * (g - xh * (g * xh).mean(-1, keepdim=True))
    return dx.to(torch.bfloat16), (dz * xh).sum((0, 1, 2))


def to_e4m3(y):
    """y rounded once to the E4M3 grid."""
    y = y.double().clamp(-448.0, 448.0)
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(y / step) * step).float().to(torch.float8_e4m3fn)


def plain_store(s, pos):
    ps, n = s["ps"], s["total"]  # the rows behind the last request go nowhere
    dtype = torch.float64 if s["fp8"] else torch.float32
    c, sn = (x[:, None] for x in cos_sin(s, pos[:n], dtype))
    s["q_out"][:n] = plain_rope(s, s["q"][:n], s["wq"], c, sn, dtype).to(torch.bfloat16)
    at = s["slots"][:n].long()
    k = plain_rope(s, s["k"][:n], s["wk"], c, sn, dtype)
    for name, x, f in (("k_cache", k, s["fk"]), ("v_cache", s["v"][:n], s["fv"])):
        if s["fp8"]:
            s[name].view(torch.uint8)[at // ps, :, at % ps] = to_e4m3(x.double() / f).view(torch.uint8)
        else:
            s[name][at // ps, :, at % ps] = x.to(torch.bfloat16)


def plain_positions(s):
    t = torch.arange(s["T"], device=DEV, dtype=torch.int32)
    r = torch.searchsorted(s["query_start"][1:].contiguous(), t, right=True).clamp(max=s["R"] - 1)
    at = s["seq_lens"][r] - s["query_start"][r + 1] + t
    s["positions"].copy_(torch.where(t < s["query_start"][-1], at, torch.full_like(at, -1)))
    return s["positions"]


def softmax_av(x, v):
    """Softmax of scores along the last axis times values, and the logsumexp; rows that see nothing: zeros, -inf."""
    m = x.amax(-1, keepdim=True)
    p = x.sub_(m.clamp(min=-3e38)).exp_()
    z = p.sum(-1, keepdim=True)
    p /= z.clamp(min=1e-38)
    return p, torch.matmul(p, v), (m + z.log()).squeeze(-1)


def plain_window(s):
    """Blocks of rows against the band of keys that they see and, before it, the first keys."""
    B, Hq, N, d = s["q"].shape
    Hk, Nk = s["k"].shape[1:3]
    G, W, S = Hq // Hk, min(s["W"], Nk), min(s["S"], Nk)
    bs = min(N, 128 if W <= 1024 else 512)
    nb = pages(N, bs)
    q_len = s["lens_q"].long() if s["pad"] else torch.full((B,), N, device=DEV)
    k_len = s["lens_k"].long() if s["pad"] else torch.full((B,), Nk, device=DEV)
    t = torch.arange(nb, device=DEV)[:, None]
    first = (k_len - q_len)[:, None, None] + t * bs  # the position of a block's first row
    j = torch.cat((torch.arange(S, device=DEV).expand(B, nb, S), first + torch.arange(W - 1 + bs, device=DEV) - (W - 1)), -1)
    row = t * bs + torch.arange(bs, device=DEV)
    p = (k_len - q_len)[:, None, None] + row
    band = torch.arange(j.shape[-1], device=DEV) >= S
    jj, pp = j[:, :, None], p[..., None]
    see = (jj <= pp) & (row < q_len[:, None, None])[..., None] & torch.where(band, (jj > pp - W) & (jj >= S), jj >= 0)
    hidden = ~see[:, None, :, None]  # [B, 1, nb, 1, bs, keys]
    at = j.clamp(0, Nk - 1)
    b_, h_ = torch.arange(B, device=DEV)[:, None, None, None], torch.arange(Hk, device=DEV)[None, :, None, None]
    k, v = (s[x][b_, h_, at[:, None]].float() for x in ("k", "v"))  # [B, Hk, nb, keys, d]

    def blocks(x):  # [B, Hq, N, d] to [B, Hk, nb, G bs, d]
        x = torch.nn.functional.pad(x.float(), (0, 0, 0, nb * bs - N))
        return x.view(B, Hk, G, nb, bs, d).transpose(2, 3).reshape(B, Hk, nb, G * bs, d)

    def rows(x):  # and back
        x = x.view(B, Hk, nb, G, bs, -1).transpose(2, 3).reshape(B, Hq, nb * bs, -1)
        return x[:, :, :N]

    q = blocks(s["q"])
    x = torch.matmul(q, k.transpose(-1, -2)).mul_(s["scale"])
    x.view(B, Hk, nb, G, bs, -1).masked_fill_(hidden, -math.inf)
    P, o, lse = softmax_av(x, v)
    out = [rows(o).to(torch.bfloat16), rows(lse[..., None]).squeeze(-1).contiguous()]
    if not s["grad"]:
        return out
    dO = blocks(s["dO"])
    dP = torch.matmul(dO, v.transpose(-1, -2))
    dS = dP.sub_((P * dP).sum(-1, keepdim=True)).mul_(P).mul_(s["scale"])
    out.append(rows(torch.matmul(dS, k)).to(torch.bfloat16))
    place = ((b_ * Hk + h_) * Nk + at[:, None]).reshape(-1)
    for w, x in ((dS, q), (P, dO)):
        dx = torch.zeros((B * Hk * Nk, d), device=DEV)
        dx.index_add_(0, place, torch.matmul(w.transpose(-1, -2), x).reshape(-1, d))
        out.append(dx.view(B, Hk, Nk, d).to(torch.bfloat16))
    return out


def plain_attn(s, q):
    R, N, Hk, d, ps = s["R"], s["max_new"], s["Hk"], s["d"], s["ps"]
    most = s["table"].shape[1] * ps
    G, W, S = s["Hq"] // Hk, min(s["W"], most), min(s["S"], most)
    lens, n = s["seq_lens"].long(), (s["query_start"][1:] - s["query_start"][:-1]).long()
    p = (lens - n)[:, None] + torch.arange(N, device=DEV)  # [R, N] positions
    j = torch.cat((torch.arange(S, device=DEV).expand(R, S), (lens - n)[:, None] + torch.arange(W - 1 + N, device=DEV) - (W - 1)), -1)
    band = torch.arange(j.shape[-1], device=DEV) >= S
    jj, pp = j[:, None], p[..., None]
    see = (jj <= pp) & (pp < lens[:, None, None]) & torch.where(band, (jj > pp - W) & (jj >= S), jj >= 0)
    at = j.clamp(min=0).minimum(lens[:, None] - 1)
    page = s["table"].gather(1, at // ps).long()
    k, v = (s[x].view(torch.uint8 if s["fp8"] else torch.bfloat16)[page, :, at % ps].view(s[x].dtype).float().transpose(1, 2)
            for x in ("k_cache", "v_cache"))
    q = q[s["row_of"]].float().reshape(R, N, Hk, G, d).permute(0, 2, 3, 1, 4).reshape(R, Hk, G * N, d)
    x = torch.matmul(q, k.transpose(2, 3)).mul_(s["fk"] * s["scale"])
    x.view(R, Hk, G, N, -1).masked_fill_(~see[:, None, None], -math.inf)
    _, o, lse = softmax_av(x, v)
    o = (o * s["fv"]).reshape(R, Hk, G, N, d).permute(0, 3, 1, 2, 4).reshape(R * N, Hk * G, d)
    lse = lse.reshape(R, Hk, G, N).permute(0, 3, 1, 2).reshape(R * N, Hk * G)
    s["o"][:s["total"]] = o[s["rows"]].to(torch.bfloat16)
    s["lse"][:s["total"]] = lse[s["rows"]]
    return s["o"], s["lse"]


def run(s):
    op = s["op"]
    if own:
        from exact_io_aware_32_gb300 import fa
        if op in ("rope", "store", "step"):
            kw = dict(interleaved=s["inter"], factor=s["factor"], q_weight=s["wq"], k_weight=s["wk"], eps=EPS)
        if op == "rope":
            out = fa.forward_rope(s["q"], s["k"], s["freqs"], s["pos"], **kw)
            if s["grad"]:
                out = (*out, *fa.backward_rope(s["dyq"], s["dyk"], s["freqs"], s["pos"], q=s["q"], k=s["k"], **kw))
            return out
        if op == "window":
            kw = dict(scale=s["scale"], seqlens_q=s["lens_q"], seqlens_k=s["lens_k"])
            o, lse = fa.forward_window(s["q"], s["k"], s["v"], s["W"], s["S"], **kw)
            if not s["grad"]:
                return o, lse
            return (o, lse, *fa.backward_window(s["q"], s["k"], s["v"], o, lse, s["dO"], s["W"], s["S"], **kw))
        q, pos = s["q"], s["pos"]
        if op == "step":
            pos = fa.paged_positions(s["query_start"], s["seq_lens"], s["T"], out=s["positions"])
        if op != "attn":
            q = fa.paged_rope_store(s["q"], s["k"], s["v"], s["slots"], pos, s["freqs"], s["k_cache"], s["v_cache"], out=s["q_out"],
                                    descale_k=s["fk"], descale_v=s["fv"], **kw)
            if op == "store":
                return q, s["k_cache"], s["v_cache"]
        o, lse = fa.forward_paged(q, s["k_cache"], s["v_cache"], s["table"], s["query_start"], s["seq_lens"], max_new=s["max_new"],
                                  scale=s["scale"], descale_k=s["fk"], descale_v=s["fv"], window=s["W"], sinks=s["S"], out=s["o"],
                                  lse=s["lse"])
        return (o, lse) if op == "attn" else (o, lse, pos, q, s["k_cache"], s["v_cache"])
    if op == "rope":
        c, sn = cos_sin(s, s["pos"], torch.float32)
        c, sn = (x[:, None] if s["rows"] else x for x in (c, sn))
        out = tuple(plain_rope(s, s[x], s["w" + x], c, sn).to(torch.bfloat16).contiguous() for x in ("q", "k"))
        if s["grad"]:
            a, b = (plain_rope_grad(s, s[x], s["w" + x], s["dy" + x], c, sn) for x in ("q", "k"))
            out = (*out, a[0], b[0], a[1], b[1])
        return out
    if op == "window":
        return plain_window(s)
    if op == "attn":
        return plain_attn(s, s["q"])
    pos = plain_positions(s) if op == "step" else s["pos"]
    plain_store(s, pos)
    if op == "store":
        return s["q_out"], s["k_cache"], s["v_cache"]
    return (*plain_attn(s, s["q_out"]), pos, s["q_out"], s["k_cache"], s["v_cache"])


def seen(p, W, S):
    """Keys that a row at position p sees."""
    return min(p + 1, W) + min(S, max(0, p + 1 - W))


def touched(first, n, W, S):
    """Keys that some row at positions first .. first + n - 1 sees."""
    lo = max(0, first - W + 1)
    return first + n - lo + min(S, lo)


def work(case):
    op, Hq, Hk, d = case["op"], case["Hq"], case["Hk"], case["d"]
    if op == "rope":
        rows = case["B"] * case["N"] * (Hq + Hk)
        flops = rows * (3 * case["rot"] + (4 * d if case["norm"] else 0))
        b = 4 * d * rows + 4 * case["N"] * (case["B"] if case["rows"] else 1)
        if case["grad"]:  # the gradients read and written; the inputs are read once for both directions
            b += 4 * d * rows + (12 * d if case["norm"] else 0)
            flops += rows * (3 * case["rot"] + (9 * d if case["norm"] else 0))
        return {"bytes": b, "flops": flops}
    if op == "window":
        W, S = case["W"], case["S"]
        q, k = sizes(case)
        pairs = sum(sum(seen(b - a + i, W, S) for i in range(a)) for a, b in zip(q, k))
        qb, kb = sum(q) * Hq, sum(touched(b - a, a, W, S) for a, b in zip(q, k)) * Hk
        b = 4 * d * qb + 4 * qb + 4 * d * kb
        if case["grad"]:
            b += 4 * d * qb + 4 * d * kb
        return {"bytes": b, "flops": pairs * Hq * d * (14 if case["grad"] else 4)}
    c, n = lengths(case)
    b, f, T = 0, 0, sum(n)
    if op in ("store", "step"):
        b += T * d * (4 * Hq + 2 * Hk * (2 + (1 if case["fp8"] else 2))) + 8 * T
        f += T * (Hq + Hk) * (3 * case["rot"] + (4 * d if case["norm"] else 0))
    if op in ("attn", "step"):
        W, S = case["W"], case["S"]
        b += T * Hq * (4 * d + 4) + 2 * Hk * d * (1 if case["fp8"] else 2) * sum(touched(x, y, W, S) for x, y in zip(c, n))
        b += 4 * sum(pages(touched(x, y, W, S), case["ps"]) for x, y in zip(c, n)) + 8 * case["R"]
        f += 4 * Hq * d * sum(seen(x + i, W, S) for x, y in zip(c, n) for i in range(y))
    return {"bytes": b, "flops": f}


# ---------------------------------------------------------------- the definition in 64 bits
def exact_rope(case, x, w, pos):
    """x [..., tokens, d] with pos [..., tokens]: the rotated rows, the norm's inverse deviation and the rotation's matrix entries."""
    f, factor = angles(case)
    r, x = case["rot"], x.double()
    rstd = 1 / torch.sqrt(torch.sum(x * x, -1, keepdim=True) / case["d"] + EPS) if w is not None else None
    z = x * rstd * w.double() if w is not None else x
    return exact_turn(case, z, pos, f, factor, 1.0), rstd


def exact_turn(case, z, pos, f, factor, sign):
    y = z.clone()
    r = case["rot"]
    for i in range(r // 2):
        a, b = (2 * i, 2 * i + 1) if case["inter"] else (i, i + r // 2)
        t = pos.double() * f[i]
        y[..., a] = factor * (z[..., a] * torch.cos(t) - sign * z[..., b] * torch.sin(t))
        y[..., b] = factor * (z[..., b] * torch.cos(t) + sign * z[..., a] * torch.sin(t))
    return y


def exact_rows(q, k, v, first, W, S, scale):
    """One head's rows at positions first, first + 1, ..: scores, weights and results over the keys from the first one seen on."""
    n = q.shape[0]
    lo = 0 if S > 0 else max(0, first - W + 1)
    p = torch.arange(first, first + n, device=DEV)[:, None]
    j = torch.arange(lo, first + n, device=DEV)[None, :]
    x = q @ k[lo:first + n].T * scale
    x = torch.where((j <= p) & ((p - j < W) | (j < S)), x, torch.full_like(x, -math.inf))
    z = torch.logsumexp(x, 1)
    P = torch.exp(x - z[:, None])
    return lo, P, P @ v[lo:first + n], z


def exact(case, seed):
    s = prepare(case, seed)
    op, Hq, Hk, d = case["op"], case["Hq"], case["Hk"], case["d"]
    G = Hq // Hk
    if op == "rope":
        pos = s["pos"][:, None] if case["rows"] else s["pos"]
        f, factor = angles(case)
        outs, grads, dws = [], [], []
        for x in ("q", "k"):
            w = s["w" + x]
            y, rstd = exact_rope(case, s[x], w, pos)
            outs.append(y)
            if case["grad"]:
                g = exact_turn(case, s["dy" + x].double(), pos, f, factor, -1.0)
                if w is None:
                    grads.append(g)
                    dws.append(None)
                    continue
                xs = s[x].double()
                dws.append(torch.einsum("bhnd,bhnd->d", g, xs * rstd))
                g = g * w.double()
                grads.append(rstd * g - xs * rstd ** 3 * torch.einsum("bhnd,bhnd->bhn", g, xs)[..., None] / d)
        return [*outs, *grads, *dws]
    W, S, step = case.get("W"), case.get("S"), 2048
    if op == "window":
        B, N, Nk = case["B"], case["N"], case["N"] + case["ctx"]
        a, b = sizes(case)
        o, dq = (torch.zeros((B, Hq, N, d), dtype=torch.float64, device=DEV) for _ in range(2))
        lse = torch.full((B, Hq, N), -math.inf, dtype=torch.float64, device=DEV)
        dk, dv = (torch.zeros((B, Hk, Nk, d), dtype=torch.float64, device=DEV) for _ in range(2))
        for i in range(B):
            for h in range(Hq):
                k, v = s["k"][i, h // G].double(), s["v"][i, h // G].double()
                for r0 in range(0, a[i], step):
                    r1 = min(a[i], r0 + step)
                    first = b[i] - a[i] + r0
                    q = s["q"][i, h, r0:r1].double()
                    lo, P, o[i, h, r0:r1], lse[i, h, r0:r1] = exact_rows(q, k, v, first, W, S, s["scale"])
                    if case["grad"]:
                        hi = first + r1 - r0
                        dO = s["dO"][i, h, r0:r1].double()
                        dv[i, h // G, lo:hi] += P.T @ dO
                        dP = dO @ v[lo:hi].T
                        dS = P * (dP - torch.sum(P * dP, 1, keepdim=True)) * s["scale"]
                        dq[i, h, r0:r1] = dS @ k[lo:hi]
                        dk[i, h // G, lo:hi] += dS.T @ q
        return [o, lse, dq, dk, dv] if case["grad"] else [o, lse]
    c, n = lengths(case)
    ps, total = case["ps"], sum(n)
    kc, vc, q = s["k_cache"].double(), s["v_cache"].double(), s["q"].double()
    if op != "attn":
        where = s["pos"][None, :total]
        q = s["q_out"].double()
        q[:total] = exact_rope(case, s["q"][:total].transpose(0, 1), s["wq"], where)[0].transpose(0, 1)
        k = exact_rope(case, s["k"][:total].transpose(0, 1), s["wk"], where)[0].transpose(0, 1)
        for t, slot in enumerate(s["slots"][:total].tolist()):
            kc[slot // ps, :, slot % ps] = k[t] / s["fk"]
            vc[slot // ps, :, slot % ps] = s["v"][t].double() / s["fv"]
        if op == "store":
            return [q, *(x.clamp(-448, 448) if case["fp8"] else x for x in (kc, vc))]
        # what the attention reads has been rounded to the types of the queries and the cache
        kr, vr = ((to_e4m3(x).double() if case["fp8"] else x.to(torch.bfloat16).double()) for x in (kc, vc))
        qr = q.to(torch.bfloat16).double()
    else:
        kr, vr, qr = kc, vc, q
    o, lse = s["o"].double(), s["lse"].double()
    table, row = s["table"].tolist(), 0
    for r in range(case["R"]):
        L = c[r] + n[r]
        idx = torch.tensor(table[r][:pages(L, ps)], device=DEV)
        key, val = (x[idx].permute(1, 0, 2, 3).reshape(Hk, -1, d)[:, :L] for x in (kr, vr))
        for h in range(Hq):
            _, _, x, z = exact_rows(qr[row:row + n[r], h], key[h // G], val[h // G], c[r], W, S, s["scale"] * s["fk"])
            o[row:row + n[r], h], lse[row:row + n[r], h] = x * s["fv"], z
        row += n[r]
    caches = [x.clamp(-448, 448) if case["fp8"] else x for x in (kc, vc)]
    return [o, lse] if op == "attn" else [o, lse, None, q, *caches]
