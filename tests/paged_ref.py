"""Plain 64-bit forms of the paged cache's operators, and seeded cases for their tests (CPU tensors)."""
import math

import torch


def plan(ctx, new, table, free, head, ps, T):
    """(query_start, seq_lens, slots, taken, table) from the definition; lists in, lists out."""
    table = [list(row) for row in table]
    start, lens, slots = [0], [], []
    at = head
    for r, (c, n) in enumerate(zip(ctx, new)):
        held, after = -(-c // ps), -(-(c + n) // ps)
        for i in range(held, after):
            table[r][i] = free[at]
            at += 1
        slots += [table[r][p // ps] * ps + p % ps for p in range(c, c + n)]
        start.append(start[-1] + n)
        lens.append(c + n)
    return start, lens, slots + [-1] * (T - len(slots)), at - head, table


def attention(q, k_cache, v_cache, table, start, lens, scale, causal, fk=1.0, fv=1.0):
    """o, lse and sum_j p_j |v_j| (what a relative error of the weights can move o by), fp64. Rows of no request: 0."""
    T, Hq, d = q.shape
    P, Hkv, ps, _ = k_cache.shape
    G = Hq // Hkv
    o = torch.zeros((T, Hq, d), dtype=torch.float64)
    spread = torch.zeros_like(o)
    lse = torch.zeros((T, Hq), dtype=torch.float64)
    for r in range(len(lens)):
        t0, t1, L = start[r], start[r + 1], lens[r]
        n = t1 - t0
        if n == 0:
            continue
        pages = table[r][:-(-L // ps)]
        k, v = (f * torch.cat([c[p].double() for p in pages] or [torch.zeros((Hkv, 0, d)).double()], 1)[:, :L]
                for c, f in ((k_cache, fk), (v_cache, fv)))
        see = torch.ones(n, L, dtype=torch.bool)
        if causal:
            see = torch.arange(L)[None, :] <= L - n + torch.arange(n)[:, None]
        qr = q[t0:t1].double().reshape(n, Hkv, G, d)
        s = torch.einsum("nhgd,hld->hgnl", qr, k) * scale
        s = s.masked_fill(~see, -math.inf)
        z = torch.logsumexp(s, -1) if L else torch.full((Hkv, G, n), -math.inf, dtype=torch.float64)
        p = torch.where(torch.isfinite(z)[..., None], torch.exp(s - z[..., None]), torch.zeros(()).double())
        o[t0:t1] = torch.einsum("hgnl,hld->nhgd", p, v).reshape(n, Hq, d)
        spread[t0:t1] = torch.einsum("hgnl,hld->nhgd", p, v.abs()).reshape(n, Hq, d)
        lse[t0:t1] = z.permute(2, 0, 1).reshape(n, Hq)
    return o, lse, spread


def e4m3(x):
    """x (fp64) rounded once to the E4M3 grid, saturating, as fp64."""
    y = x.clamp(-448.0, 448.0)
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(y / step) * step


def case(lens, Hq, Hkv, d, ps, fp8=False, pad=0, seed=0, fused=False, spare=3, width=0, gain=1.0):
    """A batch of requests [(cached, new), ...] whose caches are full, unwritten slots holding NaN. ``gain`` multiplies
    q (a sharper softmax)."""
    g = torch.Generator().manual_seed(seed)
    R = len(lens)
    n_pages = [-(-(c + n) // ps) for c, n in lens]
    P = sum(n_pages) + spare
    perm = torch.randperm(P, generator=g).tolist()
    width = max(max(n_pages), 1, width)
    table, at = [], 0
    for x in n_pages:
        table.append(perm[at:at + x] + [-7] * (width - x))
        at += x
    T = max(1, sum(n for _, n in lens) + pad)
    start = [0]
    for _, n in lens:
        start.append(start[-1] + n)
    if fused:
        qkv = torch.randn((T, (Hq + 2 * Hkv) * d), generator=g).to(torch.bfloat16)
        q, k, v = (x.unflatten(1, (-1, d)) for x in qkv.split([Hq * d, Hkv * d, Hkv * d], 1))
    else:
        q, k, v = (torch.randn((T, h, d), generator=g).to(torch.bfloat16) for h in (Hq, Hkv, Hkv))
    if gain != 1.0:
        q = (q * gain)
    fk, fv = (0.0131, 0.0097) if fp8 else (1.0, 1.0)
    caches = []
    for f in (fk, fv):
        x = torch.randn((P, Hkv, ps, d), generator=g)
        x = (x / f).clamp(-448, 448).to(torch.float8_e4m3fn) if fp8 else x.to(torch.bfloat16)
        used = torch.zeros((P, ps), dtype=torch.bool)
        for r, (c, n) in enumerate(lens):
            for i in range(n_pages[r]):
                used[table[r][i], :max(0, min(ps, c + n - i * ps))] = True
        x = x.view(torch.uint8) if fp8 else x
        x.masked_fill_(~used[:, None, :, None], 0x7F if fp8 else math.nan)
        caches.append(x.view(torch.float8_e4m3fn) if fp8 else x)
    return dict(q=q, k=k, v=v, k_cache=caches[0], v_cache=caches[1], table=table, start=start,
                lens=[c + n for c, n in lens], ctx=[c for c, _ in lens], new=[n for _, n in lens], fk=fk, fv=fv, T=T,
                free=perm[at:], R=R, Hq=Hq, Hkv=Hkv, d=d, ps=ps, fp8=fp8)


def rms_errors(o, ro, start):
    """Relative RMS error of o [T, Hq, d] against ro, by request and query head: [(request, head, error)]."""
    out = []
    for r in range(len(start) - 1):
        a, b = o[start[r]:start[r + 1]].double(), ro[start[r]:start[r + 1]].double()
        if a.numel():
            e = ((a - b) ** 2).sum((0, 2)) / (b ** 2).sum((0, 2)).clamp(min=1e-300)
            out += [(r, h, math.sqrt(float(x))) for h, x in enumerate(e)]
    return out


def rms_bound(fp8):
    """What relative RMS error the roundings leave: those of independent weights in P and of o are each at most half a step
    of 2^-7 relative and spread evenly over it, 2^-8 / sqrt(3) (P over E4M3 caches, in f16: 2^-11 / sqrt(3)); added as
    squares 0.0032 (0.0023), and a quarter more because a head of one token is 64 or 128 of them."""
    return 1.25 * math.sqrt((4.0 ** -11 if fp8 else 4.0 ** -8) + 4.0 ** -8) / math.sqrt(3)
