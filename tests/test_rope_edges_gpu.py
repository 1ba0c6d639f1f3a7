"""Rotation by position at the edges of its values and factors, on the GPU."""
import math

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
