"""Refusals of the rotation and of attention in a window, at the C ABI and in the helpers, before anything touches a device."""
import math

import pytest

from exact_io_aware_32_gb300 import build, fa

A = 1 << 32  # fake addresses, aligned and far apart; never dereferenced because validation fails first
INVALID, UNSUPPORTED, MISALIGNED, WORKSPACE = (fa.FA_ERR_INVALID_ARG, fa.FA_ERR_UNSUPPORTED, fa.FA_ERR_MISALIGNED,
                                               fa.FA_ERR_WORKSPACE)


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return fa.load()


def accepted(status):
    """What passes every check: without a GPU the call then stops at the device. (Not called where there is one, since the
    addresses are not real.)"""
    return status == fa.FA_ERR_LAUNCH


def no_gpu():
    import torch

    if torch.cuda.is_available():
        pytest.skip("would launch on addresses that are not real")


def rows(i, H, N=6, d=64, data=None, sb=None, sh=None, sn=None):
    return fa.Heads(i * A if data is None else data, H * N * d if sb is None else sb, N * d if sh is None else sh,
                    d if sn is None else sn)


def rope(back=False, q=None, k=None, qo=None, ko=None, **args):
    kw = dict(q_weight=5 * A, k_weight=6 * A, weights_fp32=False, eps=1e-6, freqs=7 * A, rotary=64, interleaved=False, factor=1.0,
              positions=8 * A, positions_stride=0, B=2, Hq=4, Hk=2, N=6, d=64)
    if back:
        kw.update(dq_weight=9 * A, dk_weight=10 * A, workspace=11 * A, workspace_bytes=1 << 30)
    kw.update(args)
    q, k, qo, ko = (x if x is not None else rows(i, H, kw["N"], kw["d"])
                    for x, i, H in ((q, 1, kw["Hq"]), (k, 2, kw["Hk"]), (qo, 3, kw["Hq"]), (ko, 4, kw["Hk"])))
    if back:
        return fa.fa_rope_bwd(dq_out=q, dk_out=k, q=rows(12, kw["Hq"], kw["N"], kw["d"]), k=rows(13, kw["Hk"], kw["N"], kw["d"]),
                              dq=qo, dk=ko, stream=0, **kw)
    return fa.fa_rope_fwd(q, k, qo, ko, stream=0, **kw)


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("args,status", [
    (dict(B=0), INVALID), (dict(N=0), INVALID), (dict(Hq=0), INVALID), (dict(Hk=-1), INVALID),
    (dict(B=1 << 30, N=1 << 10), INVALID), (dict(Hq=2 ** 31 - 1), INVALID),
    (dict(d=96), UNSUPPORTED), (dict(d=256), UNSUPPORTED), (dict(rotary=24), UNSUPPORTED), (dict(rotary=80), INVALID),
    (dict(rotary=-16), INVALID), (dict(freqs=None), INVALID), (dict(freqs=7 * A + 4), MISALIGNED),
    (dict(factor=math.inf), INVALID), (dict(factor=math.nan), INVALID),
    (dict(positions=8 * A + 2), MISALIGNED), (dict(positions_stride=-1), INVALID),
    (dict(q_weight=None), INVALID), (dict(k_weight=None), INVALID), (dict(eps=-1e-6), INVALID), (dict(eps=math.nan), INVALID),
    (dict(eps=math.inf), INVALID), (dict(q_weight=5 * A + 8), MISALIGNED), (dict(k_weight=6 * A + 2), MISALIGNED),
    (dict(Hk=0), INVALID),  # a weight for keys that are not there
    (dict(q=rows(0, 4)), INVALID), (dict(ko=rows(0, 2)), INVALID), (dict(q=rows(1, 4, data=A + 8)), MISALIGNED),
    (dict(qo=rows(3, 4, data=3 * A + 2)), MISALIGNED),
    (dict(q=rows(1, 4, sn=68)), MISALIGNED), (dict(k=rows(2, 2, sh=6 * 64 + 4)), MISALIGNED), (dict(q=rows(1, 4, sb=-64)), INVALID),
    (dict(q=rows(1, 4, sh=1 << 39)), INVALID),
    (dict(qo=rows(3, 4, sh=0)), INVALID),       # rows written twice
    (dict(qo=rows(3, 4, sn=56)), INVALID), (dict(ko=rows(4, 2, sb=64, sh=64, sn=128)), INVALID),
    (dict(ko=rows(4, 2, sb=2 * 6 * 64 - 8)), INVALID),
])
def test_rope(args, status, back):
    assert rope(back, **args) == status


@pytest.mark.parametrize("args,status", [
    (dict(dq_weight=None), INVALID), (dict(dk_weight=None), INVALID), (dict(dq_weight=9 * A + 2), MISALIGNED),
    (dict(workspace=None), WORKSPACE), (dict(workspace=11 * A + 8), WORKSPACE), (dict(workspace_bytes=0), WORKSPACE),
])
def test_rope_backward(args, status):
    assert rope(True, **args) == status


def test_rope_backward_workspace():
    need = fa.fa_rope_bwd_workspace_bytes(4, 2, 64)
    assert need > 0 and rope(True, workspace_bytes=need - 1) == WORKSPACE
    for args in ((0, 1, 64), (1, -1, 64), (1, 1, 96)):
        assert fa.fa_rope_bwd_workspace_bytes(*args) == 0


def test_rope_takes():
    """Queries alone, no norms, inputs broadcast by strides of 0, strides of dimensions of one: not refused."""
    no_gpu()
    for back in (False, True):
        for args in (dict(), dict(Hk=0, k_weight=None), dict(q_weight=None, k_weight=None), dict(rotary=0, freqs=None),
                     dict(positions=None), dict(positions_stride=6), dict(k=rows(2, 2, sh=0)), dict(q=rows(1, 4, sb=0, sn=0)),
                     dict(B=1, qo=rows(3, 4, sb=3)), dict(qo=rows(3, 4, sh=64, sn=4 * 64))):
            assert accepted(rope(back, **args)), (back, args)
    assert accepted(rope(True, q_weight=None, k_weight=None, dq_weight=None, dk_weight=None, workspace=None, workspace_bytes=0))


@pytest.mark.parametrize("args,status", [
    (dict(query_start=None), INVALID), (dict(seq_lens=None), INVALID), (dict(positions=None), INVALID), (dict(R=0), INVALID),
    (dict(T=0), INVALID), (dict(positions=3 * A + 2), MISALIGNED), (dict(query_start=A + 1), MISALIGNED),
    (dict(seq_lens=2 * A + 3), MISALIGNED),
])
def test_positions(args, status):
    kw = dict(query_start=A, seq_lens=2 * A, R=4, positions=3 * A, T=9)
    kw.update(args)
    assert fa.fa_paged_positions(**kw, stream=0) == status


def rope_store(**args):
    kw = dict(q=A, k=2 * A, v=3 * A, q_stride=8 * 64, k_stride=8 * 64, v_stride=8 * 64, slots=4 * A, positions=5 * A, freqs=6 * A,
              rotary=64, interleaved=False, factor=1.0, q_weight=7 * A, k_weight=8 * A, weights_fp32=False, eps=1e-6, q_out=9 * A,
              q_out_stride=4 * 64, T=5, Hq=4, Hkv=2, d=64, k_cache=10 * A, v_cache=11 * A, num_pages=9, page_size=16, fp8=True,
              descale_k=1.0, descale_v=1.0)
    kw.update(args)
    return fa.fa_paged_rope_store(**kw, stream=0)


@pytest.mark.parametrize("args,status", [
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(slots=None), INVALID),
    (dict(positions=None), INVALID), (dict(q_out=None), INVALID), (dict(k_cache=None), INVALID), (dict(v_cache=None), INVALID),
    (dict(T=0), INVALID), (dict(Hq=0), INVALID), (dict(Hkv=0), INVALID), (dict(num_pages=0), INVALID), (dict(page_size=0), INVALID),
    (dict(page_size=24), UNSUPPORTED), (dict(page_size=8), UNSUPPORTED), (dict(page_size=512), UNSUPPORTED),
    (dict(num_pages=2 ** 28, page_size=16), INVALID), (dict(d=80), UNSUPPORTED), (dict(rotary=40), UNSUPPORTED),
    (dict(rotary=128), INVALID), (dict(freqs=None), INVALID), (dict(factor=math.nan), INVALID),
    (dict(q_stride=4 * 64 - 8), INVALID), (dict(k_stride=64), INVALID), (dict(v_stride=0), INVALID), (dict(q_out_stride=64), INVALID),
    (dict(q_stride=4 * 64 + 4), MISALIGNED), (dict(v_stride=8 * 64 + 2), MISALIGNED),
    (dict(q=A + 8), MISALIGNED), (dict(v=3 * A + 4), MISALIGNED), (dict(q_out=9 * A + 8), MISALIGNED),
    (dict(k_cache=10 * A + 8), MISALIGNED), (dict(slots=4 * A + 2), MISALIGNED), (dict(positions=5 * A + 2), MISALIGNED),
    (dict(k_weight=None), INVALID), (dict(q_weight=None), INVALID), (dict(eps=-1.0), INVALID),
    (dict(descale_k=0.0), INVALID), (dict(descale_v=-1.0), INVALID), (dict(descale_k=math.inf), INVALID),
    (dict(descale_v=math.nan), INVALID),
])
def test_rope_store(args, status):
    assert rope_store(**args) == status


def test_rope_store_takes():
    no_gpu()
    for args in (dict(), dict(q_out=A, q_out_stride=8 * 64), dict(fp8=False, descale_k=0.0), dict(q_weight=None, k_weight=None),
                 dict(rotary=0, freqs=None), dict(T=1, q_stride=4 * 64)):
        assert accepted(rope_store(**args)), args


def window(back=False, **args):
    kw = dict(q=A, k=2 * A, v=3 * A, o=4 * A, lse=5 * A, B=2, Hq=4, Hkv=2, Nq=100, Nk=200, d=64, scale=0.125, window=50, sinks=4,
              seqlens_q=None, seqlens_k=None)
    if back:
        kw.update(dO=6 * A, dq=7 * A, dk=8 * A, dv=9 * A, workspace=10 * A, workspace_bytes=1 << 30)
    kw.update(args)
    return (fa.fa_bwd_window if back else fa.fa_fwd_window)(**kw, stream=0)


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("args,status", [
    (dict(window=0), INVALID), (dict(window=-1), INVALID), (dict(sinks=-1), INVALID), (dict(Hkv=3), INVALID), (dict(Hkv=0), INVALID),
    (dict(Hkv=8), INVALID), (dict(Nq=201), INVALID), (dict(Nq=0), INVALID), (dict(B=0), INVALID), (dict(Hq=0), INVALID),
    (dict(d=96), UNSUPPORTED), (dict(scale=math.nan), INVALID), (dict(scale=math.inf), INVALID),
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(o=None), INVALID), (dict(lse=None), INVALID),
    (dict(B=1 << 12, Nq=1 << 13, Nk=1 << 13), INVALID),  # 2^31 elements
    (dict(q=A + 8), MISALIGNED), (dict(lse=5 * A + 4), MISALIGNED), (dict(seqlens_k=11 * A + 2), MISALIGNED),
    (dict(seqlens_q=11 * A + 1), MISALIGNED),
])
def test_window(args, status, back):
    assert window(back, **args) == status


@pytest.mark.parametrize("args,status", [
    (dict(dO=None), INVALID), (dict(dq=None), INVALID), (dict(dk=None), INVALID), (dict(dv=None), INVALID),
    (dict(dk=8 * A + 8), MISALIGNED), (dict(workspace=None), WORKSPACE), (dict(workspace_bytes=16), WORKSPACE),
])
def test_window_backward(args, status):
    assert window(True, **args) == status


def test_window_backward_workspace():
    need = fa.fa_bwd_window_workspace_bytes(2, 4, 2, 100, 200, 64, 50, 4)
    assert need > 0 and window(True, workspace_bytes=need - 1) == WORKSPACE
    for bad in ((2, 4, 3, 100, 200, 64, 50, 4), (2, 4, 2, 100, 99, 64, 50, 4), (2, 4, 2, 100, 200, 64, 0, 4),
                (2, 4, 2, 100, 200, 64, 50, -1), (2, 4, 2, 100, 200, 80, 50, 4)):
        assert fa.fa_bwd_window_workspace_bytes(*bad) == 0


def test_window_takes():
    no_gpu()
    for back in (False, True):
        for args in (dict(), dict(window=2 ** 31 - 1, sinks=2 ** 31 - 1), dict(Nq=1, Nk=1, window=1, sinks=0), dict(Hkv=4), dict(Hkv=1)):
            assert accepted(window(back, **args)), (back, args)


def paged_window(**args):
    kw = dict(q=A, q_stride=256, k_cache=2 * A, v_cache=3 * A, fp8=False, descale_k=1.0, descale_v=1.0, block_table=4 * A, max_pages=8,
              query_start=5 * A, seq_lens=6 * A, o=7 * A, lse=8 * A, T=4, R=4, Hq=4, Hkv=2, d=64, num_pages=9, page_size=16, max_new=1,
              scale=0.125, window=50, sinks=4, workspace=9 * A, workspace_bytes=1 << 30)
    kw.update(args)
    return fa.fa_fwd_paged_window(**kw, stream=0)


@pytest.mark.parametrize("args,status", [
    (dict(window=0), INVALID), (dict(window=-3), INVALID), (dict(sinks=-1), INVALID), (dict(Hkv=3), INVALID), (dict(q=None), INVALID),
    (dict(block_table=None), INVALID), (dict(d=96), UNSUPPORTED), (dict(page_size=48), UNSUPPORTED), (dict(q=A + 8), MISALIGNED),
    (dict(scale=math.nan), INVALID), (dict(fp8=True, descale_v=0.0), INVALID), (dict(workspace=None), WORKSPACE),
    (dict(workspace_bytes=0), WORKSPACE),
])
def test_paged_window(args, status):
    assert paged_window(**args) == status


def test_paged_window_takes():
    no_gpu()
    for args in (dict(), dict(window=2 ** 31 - 1, sinks=2 ** 31 - 1), dict(window=1, sinks=0)):
        assert accepted(paged_window(**args)), args


def test_frequencies():
    for args in (dict(rotary=0), dict(rotary=7), dict(rotary=64, base=0.0), dict(rotary=64, linear=-1.0),
                 dict(rotary=2, base_stretch=2.0), dict(rotary=64, base_stretch=0.0), dict(rotary=64, ramp=(0.0, 100, 1, 32)),
                 dict(rotary=64, ramp=(4.0, 100, 32, 32))):
        with pytest.raises(ValueError):
            fa.rope_frequencies(**args, device="cpu")


def test_helpers_want_tensors_on_a_gpu():
    import torch

    x = torch.zeros(1, 2, 3, 64, dtype=torch.bfloat16)
    f = fa.rope_frequencies(64, device="cpu")
    ints = torch.zeros(3, dtype=torch.int32)
    cache = torch.zeros(2, 2, 16, 64, dtype=torch.bfloat16)
    for call in (lambda: fa.forward_rope(x, x, f), lambda: fa.rope(x, x, f), lambda: fa.backward_rope(x, x, f),
                 lambda: fa.forward_window(x, x, x, 2), lambda: fa.attention_window(x, x, x, 2),
                 lambda: fa.backward_window(x, x, x, x, x, x, 2), lambda: fa.paged_positions(ints, ints, 3),
                 lambda: fa.paged_rope_store(x[0], x[0], x[0], ints, ints, f, cache, cache),
                 lambda: fa.forward_paged(x[0], cache, cache, ints[None], ints, ints, window=2),
                 lambda: fa.forward_rope(None, x, f), lambda: fa.forward_window(x, x, None, 2)):
        with pytest.raises(ValueError):
            call()
