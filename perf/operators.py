"""The paged key/value cache's operators as workloads: building block tables and slot maps from request lengths, storing
new keys and values into the cache, attention of new tokens over the cache, and a whole serving step of the three.

A case says the sizes; the lengths of its requests follow from the case alone, the contents from the seed. ``run`` computes
a case in elementary torch operations, or (``own``) by the calls a user makes of this package; ``exact`` computes it from the
definitions in 64 bits.
"""
import math
import random

import torch

own = False

DEV = "cuda"


def listed():
    return [
        # every request of a decoding batch grows by one token: a step's bookkeeping, all latency
        dict(name="plan decode", op="plan", R=256, ctx=8192, new=1, chunks=0, ps=16, pad=0, lens=1),
        # prompts of many requests arrive together; the token rows are padded to a captured graph's size
        dict(name="plan prompts", op="plan", R=97, ctx=2000, new=700, chunks=97, ps=64, pad=511, lens=2),
        # the new tokens of a decoding batch go into the cache
        dict(name="store decode", op="store", R=64, ctx=4096, new=1, chunks=0, ps=16, pad=0, lens=3, Hq=32, Hkv=8, d=128,
             fp8=False, fused=True),
        # the tokens of long prompts go into an 8-bit cache, an odd number of them
        dict(name="store prompts e4m3", op="store", R=5, ctx=1, new=4095, chunks=5, ps=64, pad=1, lens=4, Hq=32, Hkv=8,
             d=128, fp8=True, fused=True),
        # one user, a short text, the head layout of the small d = 64 workload: the least work a call has
        dict(name="attn one short", op="attn", R=1, ctx=1000, new=1, chunks=0, ps=16, pad=0, lens=5, Hq=12, Hkv=12, d=64,
             fp8=False, fused=False),
        # one user, a long text: few rows, so the keys have to be spread over the card
        dict(name="attn one long", op="attn", R=1, ctx=131070, new=1, chunks=0, ps=128, pad=0, lens=6, Hq=16, Hkv=2, d=128,
             fp8=False, fused=False),
        # a decoding batch of unequal lengths, grouped heads
        dict(name="attn decode", op="attn", R=64, ctx=8192, new=1, chunks=0, ps=16, pad=0, lens=7, Hq=32, Hkv=8, d=128,
             fp8=False, fused=True),
        # the same with an 8-bit cache and longer texts; three rows behind the last request
        dict(name="attn decode e4m3", op="attn", R=48, ctx=16384, new=1, chunks=0, ps=64, pad=3, lens=8, Hq=32, Hkv=8, d=128,
             fp8=True, fused=False),
        # chunks of long prompts on top of what is cached
        dict(name="attn chunks", op="attn", R=3, ctx=8192, new=1024, chunks=3, ps=128, pad=0, lens=9, Hq=32, Hkv=8, d=128,
             fp8=False, fused=False),
        # whole prompts of the d = 64 workloads' length and heads, one query head per key head
        dict(name="attn prompts d64", op="attn", R=8, ctx=0, new=1024, chunks=8, ps=32, pad=0, lens=10, Hq=12, Hkv=12, d=64,
             fp8=False, fused=True),
        # one prompt's chunk rides along with a decoding batch, 8-bit cache
        dict(name="attn mixed e4m3", op="attn", R=33, ctx=4096, new=777, chunks=1, ps=16, pad=0, lens=11, Hq=16, Hkv=4,
             d=128, fp8=True, fused=False),
        # a whole decoding step of one layer: tables and slots, store, attention
        dict(name="step decode", op="step", R=128, ctx=4096, new=1, chunks=0, ps=16, pad=0, lens=12, Hq=32, Hkv=8, d=128,
             fp8=False, fused=True),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))

    op = rng.choice(["plan", "store", "attn", "attn", "attn", "step"])
    ps = rng.choice([16, 32, 64, 128])
    lens, pad = rng.randrange(1 << 20), rng.choice([0, 0, 1, rng.randrange(2, 400)])
    if op == "plan":
        R = log(1, 1024)
        chunks = rng.choice([0, R, R // 3])
        return dict(op=op, R=R, ctx=log(1, 8192), new=log(1, max(1, min(4000, 60000 // R))), chunks=chunks, ps=ps, pad=pad,
                    lens=lens)
    Hkv, G = rng.choice([1, 2, 4, 8, 12]), rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
    if Hkv * G > 40:
        G = 2
    heads = dict(Hq=Hkv * G, Hkv=Hkv, d=rng.choice([64, 128]), fp8=rng.random() < 0.5, fused=rng.random() < 0.5)
    if op == "store":
        R = log(1, 200)
        return dict(op=op, R=R, ctx=log(1, 2000), new=log(1, 16000 // R), chunks=R, ps=ps, pad=pad, lens=lens, **heads)
    if op == "step" or rng.random() < 0.5:  # decoding: one to a few new tokens for every request
        R, new = log(1, 96), rng.choice([1, 1, 2, 5])
        ctx = log(1, min(32768, 1600000 // (R * Hkv * new)))
        return dict(op=op, R=R, ctx=ctx, new=new, chunks=R if new > 1 else 0, ps=ps, pad=pad, lens=lens, **heads)
    R = rng.choice([1, 2, 3, 5, 9])  # chunks of prompts, alone or with decoding requests
    new = log(2, 1500)
    ctx = log(1, max(64, min(16384, 400000000 // (R * new * heads["Hq"]))))
    return dict(op=op, R=R, ctx=ctx, new=new, chunks=rng.choice([1, R]), ps=ps, pad=pad, lens=lens, **heads)


def lengths(case):
    """Tokens in the cache and new tokens of each request: the first request has the most of both, ``chunks`` of the requests
    bring up to ``new`` tokens, the others one."""
    r = random.Random(case["lens"])
    R, most = case["R"], case["ctx"]
    c = [most] + [r.randint(0, most) for _ in range(R - 1)]
    n = [case["new"]] + [r.randint(1 + case["new"] // 2, case["new"]) for _ in range(R - 1)]
    n = [x if i < max(1, case["chunks"]) else 1 for i, x in enumerate(n)]
    return c, n


def pages(n, ps):
    return -(-n // ps)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    c, n = lengths(case)
    R, ps, op = case["R"], case["ps"], case["op"]
    total = sum(n)
    T = total + case["pad"]
    width = max(pages(a + b, ps) for a, b in zip(c, n))
    held = [pages(a, ps) for a in c]
    after = [pages(a + b, ps) for a, b in zip(c, n)]
    P = sum(after) + 7

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device=DEV)

    s = dict(case, T=T, P=P, width=width, max_new=max(n), most=max(a + b for a, b in zip(c, n)))
    s["ctx_lens"], s["new_lens"] = ints(c), ints(n)
    # pages in no order: those held before the step, then the list of free ones
    perm = torch.randperm(P, generator=g, device=DEV).to(torch.int32)
    done = op in ("attn", "store")  # the plan has been made: the tables are those after it
    have = torch.tensor(after if done else held, device=DEV)
    col = torch.arange(width, device=DEV)
    at = have.cumsum(0) - have
    mask = col[None, :] < have[:, None]
    s["table"] = torch.where(mask, perm[(at[:, None] + col[None, :]).clamp(max=P - 1)], torch.full((), -1, device=DEV, dtype=torch.int32)).contiguous()
    if not done:
        s["free"] = perm[sum(held):].contiguous()
    start = [0]
    for x in n:
        start.append(start[-1] + x)
    s["query_start"], s["seq_lens"] = ints(start), ints([a + b for a, b in zip(c, n)])
    s["slots"] = torch.empty(T, dtype=torch.int32, device=DEV)
    if done:
        s["slots"].copy_(plain_slots(s["ctx_lens"], s["query_start"], s["table"], T, ps))
    if op in ("plan", "step"):
        s["taken"] = torch.empty(1, dtype=torch.int32, device=DEV)
        s["plan_start"], s["plan_lens"] = torch.empty_like(s["query_start"]), torch.empty_like(s["seq_lens"])
    if op == "plan":
        return s
    Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
    if case["fused"]:  # the three are slices of one projection's output
        qkv = torch.randn((T, (Hq + 2 * Hkv) * d), generator=g, device=DEV).to(torch.bfloat16)
        q, k, v = (x.unflatten(1, (-1, d)) for x in qkv.split([Hq * d, Hkv * d, Hkv * d], 1))
    else:
        q, k, v = (torch.randn((T, h, d), generator=g, device=DEV).to(torch.bfloat16) for h in (Hq, Hkv, Hkv))
    s["q"], s["k"], s["v"] = q, k, v
    s["fk"], s["fv"] = (0.0123, 0.0171) if case["fp8"] else (1.0, 1.0)
    for name, f in (("k_cache", s["fk"]), ("v_cache", s["fv"])):
        x = torch.randn((P, Hkv, ps, d), generator=g, device=DEV)
        s[name] = (x / f).clamp_(-448, 448).to(torch.float8_e4m3fn) if case["fp8"] else x.to(torch.bfloat16)
        del x
    if op != "store":
        s["o"] = torch.zeros((T, Hq, d), dtype=torch.bfloat16, device=DEV)
        s["lse"] = torch.zeros((T, Hq), dtype=torch.float32, device=DEV)
        # where each request's rows lie in a rectangle of R by the most new tokens, and back
        t = torch.arange(s["max_new"], device=DEV)
        s["row_of"] = (s["query_start"][:-1, None] + t[None, :]).clamp(max=T - 1).long()
        s["rows"] = torch.tensor([r * s["max_new"] + i for r, x in enumerate(n) for i in range(x)], device=DEV)
    s["total"] = total
    return s


# ---------------------------------------------------------------- the plain forms
def plain_slots(ctx, start, table, T, ps):
    t = torch.arange(T, device=DEV, dtype=torch.int32)
    r = torch.searchsorted(start[1:].contiguous(), t, right=True).clamp(max=ctx.numel() - 1)
    pos = ctx[r] + t - start[r]
    page = table[r, (pos // ps).clamp(0, table.shape[1] - 1).long()]
    return torch.where(t < start[-1], page * ps + pos % ps, torch.full_like(page, -1))


def plain_plan(s):
    c, n, ps = s["ctx_lens"], s["new_lens"], s["ps"]
    start = torch.nn.functional.pad(n.cumsum(0), (1, 0)).to(torch.int32)
    lens = c + n
    held, after = (c + ps - 1) // ps, (lens + ps - 1) // ps
    need = after - held
    first = need.cumsum(0) - need
    col = torch.arange(s["width"], device=DEV)
    fresh = (col >= held[:, None]) & (col < after[:, None])
    page = s["free"][(first[:, None] + col - held[:, None]).clamp(0, s["free"].numel() - 1)]
    table = torch.where(fresh, page, s["table"])
    s["table"].copy_(table)
    return start, lens, plain_slots(c, start, table, s["T"], ps), need.sum().to(torch.int32).reshape(1)


def to_e4m3(x, f):
    """x / f rounded once to the E4M3 grid: in 64 bits, so that quotients next to the middle of two codes fall right."""
    y = (x.double() / f).clamp(-448.0, 448.0)
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(y / step) * step).float().to(torch.float8_e4m3fn)


def plain_store(s, slots):
    ps, total = s["ps"], s["total"]  # the rows behind the last request go nowhere
    at = slots[:total].long()
    page, row = at // ps, at % ps
    for name, x, f in (("k_cache", s["k"], s["fk"]), ("v_cache", s["v"], s["fv"])):
        if s["fp8"]:
            s[name].view(torch.uint8)[page, :, row] = to_e4m3(x[:total], f).view(torch.uint8)
        else:
            s[name][page, :, row] = x[:total]
    return s["k_cache"], s["v_cache"]


def plain_attn(s, start, lens):
    R, N, Hkv, d, ps = s["R"], s["max_new"], s["Hkv"], s["d"], s["ps"]
    G, L = s["Hq"] // Hkv, s["width"] * ps
    table = s["table"].clamp(min=0).long()
    k, v = (s[x][table].float().transpose(1, 2).reshape(R, Hkv, L, d) for x in ("k_cache", "v_cache"))
    q = s["q"][s["row_of"]].float().reshape(R, N, Hkv, G, d).permute(0, 2, 3, 1, 4).reshape(R, Hkv, G * N, d)
    x = torch.matmul(q, k.transpose(2, 3)).mul_(s["fk"] / math.sqrt(d))
    n = start[1:] - start[:-1]
    last = (lens - n)[:, None] + torch.arange(N, device=DEV)  # the last key that each row sees
    hidden = torch.arange(L, device=DEV) > torch.minimum(last, lens[:, None] - 1)[:, :, None]
    hidden = hidden[:, None, None].expand(R, 1, G, N, L).reshape(R, 1, G * N, L)
    x.masked_fill_(hidden, -math.inf)
    v = v.masked_fill((torch.arange(L, device=DEV) >= lens[:, None])[:, None, :, None], 0.0)
    m = x.amax(-1, keepdim=True)
    p = x.sub_(m.clamp(min=-3e38)).exp_()
    z = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / z.clamp(min=1e-38) * s["fv"]
    lse = (m + z.log()).squeeze(-1)
    o = o.reshape(R, Hkv, G, N, d).permute(0, 3, 1, 2, 4).reshape(R * N, Hkv * G, d)
    lse = lse.reshape(R, Hkv, G, N).permute(0, 3, 1, 2).reshape(R * N, Hkv * G)
    s["o"][:s["total"]] = o[s["rows"]].to(torch.bfloat16)
    s["lse"][:s["total"]] = lse[s["rows"]]
    return s["o"], s["lse"]


def run(s):
    op = s["op"]
    if own:
        from exact_io_aware_32_gb300 import fa
        plan = None
        if op in ("plan", "step"):
            plan = fa.paged_plan(s["ctx_lens"], s["new_lens"], s["table"], s["free"], s["ps"], s["T"],
                                 out=(s["plan_start"], s["plan_lens"], s["slots"], s["taken"]))
            if op == "plan":
                return (*plan, s["table"])
        if op in ("store", "step"):
            fa.paged_store(s["k"], s["v"], s["slots"], s["k_cache"], s["v_cache"], descale_k=s["fk"], descale_v=s["fv"])
            if op == "store":
                return s["k_cache"], s["v_cache"]
        start, lens = (plan[0], plan[1]) if plan else (s["query_start"], s["seq_lens"])
        o, lse = fa.forward_paged(s["q"], s["k_cache"], s["v_cache"], s["table"], start, lens, max_new=s["max_new"],
                                  descale_k=s["fk"], descale_v=s["fv"], out=s["o"], lse=s["lse"])
        return (o, lse) if op == "attn" else (o, lse, *plan, s["table"], s["k_cache"], s["v_cache"])
    if op == "plan":
        return (*plain_plan(s), s["table"])
    if op == "store":
        return plain_store(s, s["slots"])
    if op == "attn":
        return plain_attn(s, s["query_start"], s["seq_lens"])
    plan = plain_plan(s)
    caches = plain_store(s, plan[2])
    return (*plain_attn(s, plan[0], plan[1]), *plan, s["table"], *caches)


def work(case):
    c, n = lengths(case)
    R, ps = case["R"], case["ps"]
    T = sum(n) + case["pad"]
    need = sum(pages(a + b, ps) - pages(a, ps) for a, b in zip(c, n))
    b, f = 0, 0
    if case["op"] in ("plan", "step"):
        b += 8 * R + 4 * R + 8 * R + 4 * T + 8 * need
    if case["op"] in ("store", "step"):
        row = 2 * case["Hkv"] * case["d"]
        b += sum(n) * row * (2 + (1 if case["fp8"] else 2)) + 4 * T
    if case["op"] in ("attn", "step"):
        Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
        b += sum(n) * Hq * (4 * d + 4) + 2 * sum(x + y for x, y in zip(c, n)) * Hkv * d * (1 if case["fp8"] else 2)
        b += 4 * sum(pages(x + y, ps) for x, y in zip(c, n)) + 8 * R
        f += 4 * Hq * d * sum(x * y + y * (y + 1) // 2 for x, y in zip(c, n))
    return {"bytes": b, "flops": f}


# ---------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    op, ps = case["op"], case["ps"]
    if op == "plan":
        return None
    c, n = lengths(case)
    if op == "store":
        out = []
        for name, x, f in (("k_cache", s["k"], s["fk"]), ("v_cache", s["v"], s["fv"])):
            cache = s[name].double()
            for t, slot in enumerate(s["slots"].tolist()):
                if slot >= 0:
                    cache[slot // ps, :, slot % ps] = (x[t].double() / f).clamp(-448, 448) if case["fp8"] else x[t].double()
            out.append(cache)
        return out
    Hkv, d, G = case["Hkv"], case["d"], case["Hq"] // case["Hkv"]
    o, lse = s["o"].double(), s["lse"].double()
    table, free, at = s["table"].tolist(), s["free"].tolist() if op == "step" else None, 0
    row = 0
    for r in range(case["R"]):
        L = c[r] + n[r]
        mine = table[r][:pages(L if op == "attn" else c[r], ps)]
        fresh = pages(L, ps) - len(mine)
        mine = mine + (free[at:at + fresh] if fresh else [])
        at += fresh
        idx = torch.tensor(mine, device=DEV)
        key, val = (s[x][idx].double().permute(1, 0, 2, 3).reshape(Hkv, -1, d)[:, :L] for x in ("k_cache", "v_cache"))
        if op == "step":  # the new tokens' rows are in the cache once they have been stored
            for cache, x, f in ((key, s["k"], s["fk"]), (val, s["v"], s["fv"])):
                new = x[row:row + n[r]]
                cache[:, c[r]:] = (to_e4m3(new, f).double() if case["fp8"] else new.double()).transpose(0, 1)
        last = torch.arange(n[r], device=DEV) + c[r]
        see = torch.arange(L, device=DEV)[None, :] <= last[:, None]
        for h in range(Hkv):
            q = s["q"][row:row + n[r], h * G:(h + 1) * G].double()
            for i in range(G):
                x = (q[:, i] @ key[h].T) * (s["fk"] / math.sqrt(d))
                x = torch.where(see, x, torch.full_like(x, -math.inf))
                z = torch.logsumexp(x, 1)
                lse[row:row + n[r], h * G + i] = z
                o[row:row + n[r], h * G + i] = torch.exp(x - z[:, None]) @ val[h] * s["fv"]
        row += n[r]
    return [o, lse] if op == "attn" else [o, lse, None, None, None, None, None, None, None]
