"""Rotation by position at the edges of its values and factors, on the GPU."""
import math
from fractions import Fraction

import pytest
import torch

from exact_io_aware_32_gb300 import fa
import window_ref
from test_rope_gpu import check, randn

pytestmark = pytest.mark.gpu


def spoil(x, rotary, far):
    """x with infinities and NaN in elements from 'rotary' on, three kinds of them in turn (heads and tokens)."""
    x = x.clone()
    for i, bad in enumerate((math.inf, -math.inf, math.nan)):
        x[..., i::3, min(rotary + far + i, x.shape[-1] - 1)] = bad
    return x


def same(a, b):
    """Equal values, NaN for NaN."""
    assert torch.equal(a.isnan(), b.isnan()) and torch.equal(a.nan_to_num(0.0), b.nan_to_num(0.0))


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("d,rotary", [(64, 16), (64, 32), (64, 48), (128, 16), (128, 64), (128, 112), (64, 0), (128, 0)])
@pytest.mark.parametrize("far", [0, 3, 8, 24])
def test_what_is_not_rotated_stays_by_itself(d, rotary, far, inter):
    """Elements from 'rotary' on come out as they went in, whatever they hold, and the rotated ones do not meet them: forward,
    backward and on the way into a cache (bf16 and E4M3)."""
    T, Hq, Hk = 7, 5, 2
    freqs = fa.rope_frequencies(rotary) if rotary else torch.empty(0, dtype=torch.float64, device="cuda")
    clean = randn((1, Hq + Hk, T, d), rotary + far)
    x = spoil(clean, rotary, far)
    pos = torch.arange(1000, 1000 + T, dtype=torch.int32, device="cuda")
    kw = dict(interleaved=inter, factor=1.5)
    for back in (False, True):
        call = fa.backward_rope if back else fa.forward_rope
        ys = call(x[:, :Hq], x[:, Hq:], freqs, pos, **kw)[:2]
        refs = call(clean[:, :Hq], clean[:, Hq:], freqs, pos, **kw)[:2]
        for y, r, given in zip(ys, refs, (x[:, :Hq], x[:, Hq:])):
            assert torch.equal(y[..., :rotary], r[..., :rotary])
            same(y[..., rotary:], given[..., rotary:])
    q, k = (z[0].transpose(0, 1).contiguous() for z in (x[:, :Hq], x[:, Hq:]))
    cq, ck = (z[0].transpose(0, 1).contiguous() for z in (clean[:, :Hq], clean[:, Hq:]))
    slots = torch.arange(T, dtype=torch.int32, device="cuda")
    for kind in (torch.bfloat16, torch.float8_e4m3fn):
        caches = [torch.zeros((1, Hk, 16, d), dtype=torch.bfloat16, device="cuda").to(kind) for _ in range(4)]
        y = fa.paged_rope_store(q, k, k, slots, pos, freqs, *caches[:2], **kw)
        r = fa.paged_rope_store(cq, ck, ck, slots, pos, freqs, *caches[2:], **kw)
        assert torch.equal(y[..., :rotary], r[..., :rotary])
        same(y[..., rotary:], q[..., rotary:])
        got, ref = (c.float()[0, :, :T] for c in (caches[0], caches[2]))
        assert torch.equal(got[..., :rotary], ref[..., :rotary])
        rest = k.transpose(0, 1)[..., rotary:].float()
        same(got[..., rotary:], rest if kind == torch.bfloat16 else rest.clamp(-448, 448).to(kind).float())
    torch.cuda.synchronize()
    assert fa.fa_device_status(True) == fa.FA_OK


@pytest.mark.parametrize("inter", [False, True])
def test_a_rotated_infinity_stays_in_its_pair(inter):
    """Of the rotated elements a pair's two are the only ones that an infinity or a NaN in it reaches."""
    d, rotary = 128, 96
    freqs = fa.rope_frequencies(rotary)
    clean = randn((1, 3, 4, d), 5)
    x = clean.clone()
    x[0, 0, 1, 10], x[0, 1, 2, 95], x[0, 2, 3, 47] = math.inf, math.nan, -math.inf
    y, _ = fa.forward_rope(x, None, freqs, interleaved=inter)
    r, _ = fa.forward_rope(clean, None, freqs, interleaved=inter)
    pair = {10: (10, 11) if inter else (10, 58), 95: (94, 95) if inter else (47, 95), 47: (46, 47) if inter else (47, 95)}
    hit = torch.zeros_like(x, dtype=torch.bool)
    for h, n, e in ((0, 1, 10), (1, 2, 95), (2, 3, 47)):
        hit[0, h, n, list(pair[e])] = True
    assert torch.equal(~y.isfinite(), hit) and torch.equal(y[~hit], r[~hit])


@pytest.mark.parametrize("rotary", [0, 32])
@pytest.mark.parametrize("factor", [1e-45, 1e-40, 2.0 ** -128, 2.0 ** -126, 2.0 ** -101, 2.0 ** -100, 2.0 ** -99, 0.37, 2.0 ** 99, 2.0 ** 100,
                                    2.0 ** 120, 1.1 * 2.0 ** 126, 3e38])
def test_key_factors_far_from_one(factor, rotary):
    """Codes of keys for every factor that is taken, zeros among the keys: the nearest one, half a step of E4M3 (2^-4 of the
    value, 2^-10 below the normal codes), with room for the key's and the quotient's fp32 roundings: 2^-23 of the value for the
    quotient, and where the key is rotated 2^-19 of its pair's size; 2^-18 of both here."""
    f = float(torch.tensor(factor, dtype=torch.float32))
    T, Hk, d = 40, 3, 64
    g = torch.Generator().manual_seed(3)
    want = torch.randn((T, Hk, d), generator=g, dtype=torch.float64) * torch.tensor([0.01, 1.0, 200.0])[:, None]
    want[:, :, ::7] = 0.0
    want[5] = 0.0
    k = (want * f).clamp(-3e38, 3e38).to(torch.bfloat16).cuda()
    q = randn((T, 2, d), 1)
    freqs = fa.rope_frequencies(32)[:rotary // 2].contiguous()
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    caches = [torch.full((3, Hk, 16, d), 1.0, device="cuda").to(torch.float8_e4m3fn) for _ in range(2)]
    y = fa.paged_rope_store(q, k, k, pos, pos, freqs, *caches, descale_k=f, descale_v=f)
    torch.cuda.synchronize()
    assert fa.fa_device_status(True) == fa.FA_OK and y.isfinite().all()
    ref = window_ref.rope(k.transpose(0, 1), None, pos, freqs, False, 1.0, 1e-6)[0].transpose(0, 1) / f if rotary else k.double() / f
    for cache, r in zip(caches, (ref, k.double() / f)):
        got = cache.double().transpose(1, 2).reshape(48, Hk, d)[:T]
        r = r.clamp(-448, 448)
        # (the pair's size: at most twice the row's largest element)
        size = r.abs() + (2 * r.abs().amax(-1, keepdim=True) if cache is caches[0] and rotary else 0)
        step = torch.exp2(torch.floor(torch.log2(r.abs().clamp_min(2.0 ** -6))) - 4)
        assert got.isfinite().all()
        over = (got - r).abs() - step - 2.0 ** -18 * size
        assert float(over.max()) <= 0, (float(over.max()), factor)
        zero = r == 0
        assert not got[zero].any()


def inverse_turn():
    """1 / (2 pi) to 400 bits, by Machin's formula."""
    one = 1 << 420

    def atan_inverse(x):
        term = total = one // x
        n = 1
        while term:
            term //= -x * x
            n += 2
            total += term // n
        return total
    return Fraction(one, 2 * 4 * (4 * atan_inverse(5) - atan_inverse(239)))


def test_angles_are_those_of_the_given_frequencies():
    """Frequencies of 2^-60 to 2^32 radians a position, of both signs, at the farthest positions, against angles in whole numbers:
    2^-24 of a turn, so the bounds of test_rope_gpu.py."""
    d = 128
    g = torch.Generator().manual_seed(4)
    f = torch.exp2(torch.linspace(-60, 31, d // 2, dtype=torch.float64) + torch.rand(d // 2, generator=g, dtype=torch.float64))
    f[1::2] *= -1
    places = [2 ** 31 - 1, 2 ** 31 - 2, -2 ** 31, 1234567890, 2 ** 20 + 1, 1, 0, -7]
    inverse = inverse_turn()
    at = [[Fraction(w) * p * inverse % 1 for w in f.tolist()] for p in places]
    angle = 2 * math.pi * torch.tensor([[float(x if x < Fraction(1, 2) else x - 1) for x in row] for row in at], dtype=torch.float64)
    q = randn((1, 3, len(places), d), 9)
    y, _ = fa.forward_rope(q, None, f.cuda(), torch.tensor(places, dtype=torch.int64).to(torch.int32).cuda())
    a, b = q.double()[..., :64], q.double()[..., 64:]
    c, s = angle.cos().cuda(), angle.sin().cuda()
    size = a.abs() + b.abs()
    check(y, torch.cat((a * c - b * s, b * c + a * s), -1), torch.cat((size, size), -1))


@pytest.mark.parametrize("inter", [False, True])
def test_products_depend_on_the_distance_alone(inter):
    """q . k of rows that stand 'apart' positions from one another is the same wherever they stand, and that of the 64-bit form at
    this distance. Each side's elements are off by 2^-8 of themselves (their rounding) and 2^-17 of their pairs' sizes."""
    d = 128
    q, k = (randn((1, 1, 1, d), s).expand(1, 1, 6, d) for s in (11, 12))
    freqs = fa.rope_frequencies(d)
    starts = torch.tensor([0, 1, 77, 4096, 1 << 20, (1 << 31) - 2000], dtype=torch.int64)
    sums = {}
    for apart in (0, 1, 5, 300, 1999):
        yq, _ = fa.forward_rope(q, None, freqs, (starts + apart).to(torch.int32).cuda(), interleaved=inter)
        yk, _ = fa.forward_rope(k, None, freqs, starts.to(torch.int32).cuda(), interleaved=inter)
        got = (yq.double() * yk.double()).sum(-1).flatten()
        (rq, sq), (rk, sk) = (window_ref.rope(x[:, :, :1], None, torch.tensor([p], device="cuda"), freqs, inter, 1.0, 1e-6)
                              for x, p in ((q, apart), (k, 0)))
        ref = float((rq * rk).sum())
        # (an element is at most its pair's size, which the rotation keeps)
        bound = float((sq * sk).sum()) * (2 * 2.0 ** -8 + 2 * 2.0 ** -17 + 2.0 ** -15)
        assert float((got - ref).abs().max()) <= bound, (apart, float((got - ref).abs().max()), bound)
        sums[apart] = (ref, bound)
    assert abs(sums[0][0] - sums[300][0]) > sums[0][1] + sums[300][1]  # distances differ by more than that
