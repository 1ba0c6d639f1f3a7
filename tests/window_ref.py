"""Plain 64-bit forms of the attention in a window and of the rotation, and bounds of their kernels' roundings element by
element (tensors on any device)."""
import math

import torch

HALF = 2.0 ** -8  # half a step of bf16, relative


def sees(p, j, window, sinks):
    """Whether the row at position p sees key j."""
    return (j <= p) & ((p - j < window) | (j < sinks))


def attention(q, k, v, window, sinks, scale, sq=None, sk=None, dO=None):
    """One head's [Nq, d] rows against [Nk, d] keys (its first sq rows and sk keys), fp64: dict of o, lse and, with dO, dq, dk,
    dv; and of what the kernels' roundings can move each by.

    The scores are fp32 sums of d products: off by at most d 2^-23 sum |q_i k_i| scale, below e = 2^-10 for the normal inputs
    here (|s| below 16), which moves every weight by that much relatively and the logsumexp absolutely. P enters both
    products with V (forward) and dO (dV) as bf16, half a step; o, dq, dk and dv are rounded to bf16 once. The backward's D
    is the row sum of dO times the rounded o; dS is made of the fp32 P and of dP - D, and rounded to bf16."""
    Nq, Nk = q.shape[0], k.shape[0]
    sq, sk = sq or Nq, sk or Nk
    q, k, v = q.double(), k.double(), v.double()
    i = torch.arange(Nq, device=q.device)[:, None]
    j = torch.arange(Nk, device=q.device)[None, :]
    see = sees(i + sk - sq, j, window, sinks) & (i < sq) & (j < sk)
    s = torch.where(see, q @ k.T * scale, torch.full((), -math.inf, dtype=torch.float64, device=q.device))
    lse = torch.logsumexp(s, 1)
    P = torch.where(see, torch.exp(s - torch.where(lse.isfinite(), lse, torch.zeros_like(lse))[:, None]), torch.zeros_like(s))
    e, tiny = 2.0 ** -10, 1e-12
    o = P @ v
    bo = HALF * o.abs() + (HALF + e) * (P @ v.abs()) + tiny
    r = dict(o=o, lse=lse, bound_o=bo, bound_lse=torch.full_like(lse, e))
    if dO is not None:
        g = dO.double()
        g = torch.where(i < sq, g, torch.zeros_like(g))
        dP = g @ v.T
        D = (g * o).sum(1, keepdim=True)
        dS = P * (dP - D)
        off = P * (bo * g.abs()).sum(1, keepdim=True) + (HALF + 2 * e) * dS.abs() + e * P * (g.abs() @ v.abs().T)
        r.update(dq=scale * dS @ k, dk=scale * dS.T @ q, dv=P.T @ g)
        r.update(bound_dq=HALF * r["dq"].abs() + scale * off @ k.abs() + tiny, bound_dk=HALF * r["dk"].abs() + scale * off.T @ q.abs() + tiny,
                 bound_dv=HALF * r["dv"].abs() + (HALF + e) * (P.T @ g.abs()) + tiny)
    return r


def batch(q, k, v, window, sinks, scale, lens_q=None, lens_k=None, dO=None):
    """[B, Hq, Nq, d] over [B, Hkv, Nk, d]: the heads' dicts as one; a key head's gradients are sums over its query heads
    (rounded once, which the sum of the heads' bounds covers)."""
    B, Hq, Hkv = q.shape[0], q.shape[1], k.shape[1]
    G = Hq // Hkv
    out = {}
    for b in range(B):
        for h in range(Hq):
            r = attention(q[b, h], k[b, h // G], v[b, h // G], window, sinks, scale, lens_q and lens_q[b], lens_k and lens_k[b],
                          None if dO is None else dO[b, h])
            for name, x in r.items():
                out.setdefault(name, {})[b, h] = x
    full = {}
    for name, x in out.items():
        shared = name.removeprefix("bound_") in ("dk", "dv")
        rows = [[sum(x[b, h * G + g] for g in range(G)) for h in range(Hkv)] if shared else [x[b, h] for h in range(Hq)] for b in range(B)]
        full[name] = torch.stack([torch.stack(r) for r in rows])
    return full


def rms(x, ref):
    """Relative RMS error; where the reference vanishes (the gradients of a row that sees one key) against 1e-3 a value."""
    x, ref = x.double(), ref.double()
    return float((x - ref).norm() / max(float(ref.norm()), 1e-3 * math.sqrt(ref.numel())))


# ---------------------------------------------------------------- over the paged cache
def paged(q, k_cache, v_cache, table, start, lens, scale, window, sinks, fk=1.0, fv=1.0):
    """o, lse and sum_j p_j |v_j| as paged_ref.attention, in a window; only keys that a row sees are looked at."""
    T, Hq, d = q.shape
    Hkv, ps = k_cache.shape[1:3]
    G = Hq // Hkv
    o, spread = (torch.zeros((T, Hq, d), dtype=torch.float64) for _ in range(2))
    lse = torch.zeros((T, Hq), dtype=torch.float64)
    for r in range(len(lens)):
        t0, n, L = start[r], start[r + 1] - start[r], lens[r]
        for i in range(n):
            p = L - n + i
            j = torch.arange(max(p + 1, 0))
            j = j[sees(p, j, window, sinks)]
            lse[t0 + i] = -math.inf
            if not len(j):
                continue
            page = torch.tensor([table[r][x // ps] for x in j.tolist()])
            keys, vals = (f * c.double()[page, :, j % ps] for c, f in ((k_cache, fk), (v_cache, fv)))  # [keys, Hkv, d]
            s = torch.einsum("hgd,lhd->hgl", q[t0 + i].double().reshape(Hkv, G, d), keys) * scale
            z = torch.logsumexp(s, -1)
            w = torch.exp(s - z[..., None])
            o[t0 + i] = torch.einsum("hgl,lhd->hgd", w, vals).reshape(Hq, d)
            spread[t0 + i] = torch.einsum("hgl,lhd->hgd", w, vals.abs()).reshape(Hq, d)
            lse[t0 + i] = z.reshape(Hq)
    return o, lse, spread


# ---------------------------------------------------------------- rotation
def turned(z, pos, freqs, inter, factor, sign=1.0):
    """z [..., N, d] fp64 with pos [..., N]: each pair (a, b) as factor (a cos - b sin, b cos + a sin)."""
    half = len(freqs)
    t = pos.double()[..., None] * freqs.double()
    c, s = factor * torch.cos(t), sign * factor * torch.sin(t)
    y = z.clone()
    at = (2 * torch.arange(half), 2 * torch.arange(half) + 1) if inter else (torch.arange(half), half + torch.arange(half))
    a, b = z[..., at[0]], z[..., at[1]]
    y[..., at[0]], y[..., at[1]] = a * c - b * s, b * c + a * s
    return y


def rope(x, w, pos, freqs, inter, factor, eps):
    """The rows, normed (w not None) and rotated, fp64, and the size that fp32 errors go by: the pair's."""
    x = x.double()
    z = x if w is None else x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w.double()
    y = turned(z, pos, freqs, inter, factor)
    size = turned(z.abs(), pos * 0, freqs * 0, inter, 1.0)
    half = len(freqs)
    a, b = (z[..., 0:2 * half:2], z[..., 1:2 * half:2]) if inter else (z[..., :half], z[..., half:2 * half])
    pair = abs(factor) * (a.abs() + b.abs())
    if inter:
        size[..., :2 * half] = pair.repeat_interleave(2, -1)
    else:
        size[..., :2 * half] = torch.cat((pair, pair), -1)
    return y, size


def rope_backward(dy, x, w, pos, freqs, inter, factor, eps):
    """dx and dw (None without norms), fp64."""
    g = turned(dy.double(), pos, freqs, inter, factor, -1.0)
    if w is None:
        return g, None
    x = x.double()
    r = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    xh, u = x * r, g * w.double()
    return r * (u - xh * (u * xh).mean(-1, keepdim=True)), (g * xh).reshape(-1, x.shape[-1]).sum(0)
