"""Refusals of the paged cache's entry points, before anything touches a device; the plain forms the GPU tests compare
with, against closed forms."""
import math

import pytest
import torch

from exact_io_aware_32_gb300 import build, fa
import paged_ref

A = 1 << 20  # a 16-byte aligned fake address; never dereferenced because validation fails first


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return fa.load()


@pytest.mark.parametrize("args,status", [
    (dict(ctx_lens=0), fa.FA_ERR_INVALID_ARG),
    (dict(slots=0), fa.FA_ERR_INVALID_ARG),
    (dict(pages_taken=0), fa.FA_ERR_INVALID_ARG),
    (dict(R=0), fa.FA_ERR_INVALID_ARG),
    (dict(T=0), fa.FA_ERR_INVALID_ARG),
    (dict(n_free=-1), fa.FA_ERR_INVALID_ARG),
    (dict(max_pages=0), fa.FA_ERR_INVALID_ARG),
    (dict(max_pages=1 << 27), fa.FA_ERR_INVALID_ARG),  # 2^31 tokens
    (dict(page_size=0), fa.FA_ERR_INVALID_ARG),
    (dict(page_size=24), fa.FA_ERR_UNSUPPORTED),
    (dict(page_size=8), fa.FA_ERR_UNSUPPORTED),
    (dict(page_size=512), fa.FA_ERR_UNSUPPORTED),
    (dict(block_table=A + 2), fa.FA_ERR_MISALIGNED),
    (dict(free_head=A + 1), fa.FA_ERR_MISALIGNED),
])
def test_plan_rejects_bad_args(args, status):
    kw = dict(ctx_lens=A, new_lens=A, R=4, page_size=16, free_pages=A, n_free=8, free_head=None, block_table=A,
              max_pages=9, query_start=A, seq_lens=A, slots=A, T=4, pages_taken=A)
    kw.update(args)
    assert fa.fa_paged_plan(**kw, stream=0) == status


@pytest.mark.parametrize("args,status", [
    (dict(k=0), fa.FA_ERR_INVALID_ARG),
    (dict(v_cache=0), fa.FA_ERR_INVALID_ARG),
    (dict(T=0), fa.FA_ERR_INVALID_ARG),
    (dict(Hkv=0), fa.FA_ERR_INVALID_ARG),
    (dict(num_pages=0), fa.FA_ERR_INVALID_ARG),
    (dict(num_pages=1 << 27), fa.FA_ERR_INVALID_ARG),  # 2^31 slots
    (dict(k_stride=255), fa.FA_ERR_INVALID_ARG),       # tokens would overlap
    (dict(v_stride=1 << 40), fa.FA_ERR_INVALID_ARG),
    (dict(k_stride=260), fa.FA_ERR_MISALIGNED),
    (dict(d=96, k_stride=512, v_stride=512), fa.FA_ERR_UNSUPPORTED),
    (dict(page_size=48), fa.FA_ERR_UNSUPPORTED),
    (dict(fp8=True, descale_k=0.0), fa.FA_ERR_INVALID_ARG),
    (dict(fp8=True, descale_v=math.inf), fa.FA_ERR_INVALID_ARG),
    (dict(v=A + 8), fa.FA_ERR_MISALIGNED),
    (dict(k_cache=A + 4), fa.FA_ERR_MISALIGNED),
    (dict(slots=A + 2), fa.FA_ERR_MISALIGNED),
])
def test_store_rejects_bad_args(args, status):
    kw = dict(k=A, v=A, k_stride=256, v_stride=256, slots=A, T=3, Hkv=4, d=64, k_cache=A, v_cache=A, num_pages=9,
              page_size=16, fp8=False, descale_k=1.0, descale_v=1.0)
    kw.update(args)
    assert fa.fa_paged_store(**kw, stream=0) == status


@pytest.mark.parametrize("args,status", [
    (dict(q=0), fa.FA_ERR_INVALID_ARG),
    (dict(lse=0), fa.FA_ERR_INVALID_ARG),
    (dict(R=0), fa.FA_ERR_INVALID_ARG),
    (dict(T=0), fa.FA_ERR_INVALID_ARG),
    (dict(max_new=0), fa.FA_ERR_INVALID_ARG),
    (dict(max_pages=0), fa.FA_ERR_INVALID_ARG),
    (dict(Hkv=3), fa.FA_ERR_INVALID_ARG),          # 8 query heads over 3
    (dict(q_stride=1000), fa.FA_ERR_INVALID_ARG),  # tokens would overlap
    (dict(q_stride=1028), fa.FA_ERR_MISALIGNED),
    (dict(scale=0.0), fa.FA_ERR_INVALID_ARG),
    (dict(scale=math.nan), fa.FA_ERR_INVALID_ARG),
    (dict(fp8=True, descale_k=-1.0), fa.FA_ERR_INVALID_ARG),
    (dict(fp8=True, descale_k=1e-30, scale=1e-30), fa.FA_ERR_INVALID_ARG),  # their product underflows
    (dict(T=1 << 29), fa.FA_ERR_INVALID_ARG),
    (dict(Hq=256, Hkv=1, q_stride=256 * 128), fa.FA_ERR_UNSUPPORTED),
    (dict(d=32), fa.FA_ERR_UNSUPPORTED),
    (dict(page_size=17), fa.FA_ERR_UNSUPPORTED),
    (dict(o=A + 8), fa.FA_ERR_MISALIGNED),
    (dict(query_start=A + 2), fa.FA_ERR_MISALIGNED),
    (dict(workspace=0), fa.FA_ERR_WORKSPACE),
    (dict(workspace=A + 128), fa.FA_ERR_WORKSPACE),
    (dict(workspace_bytes=0), fa.FA_ERR_WORKSPACE),
])
def test_fwd_paged_rejects_bad_args(args, status):
    kw = dict(q=A, q_stride=1024, k_cache=A, v_cache=A, fp8=False, descale_k=1.0, descale_v=1.0, block_table=A,
              max_pages=4, query_start=A, seq_lens=A, o=A, lse=A, T=5, R=2, Hq=8, Hkv=2, d=128, num_pages=11,
              page_size=32, max_new=4, scale=0.1, causal=True, workspace=A, workspace_bytes=1 << 40)
    kw.update(args)
    assert fa.fa_fwd_paged(**kw, stream=0) == status


def test_fwd_paged_rejects_more_work_than_it_counts():
    """Places in the row of tiles are 32-bit numbers of key blocks: 600 requests x 2 key heads x 2^31 / 128 blocks."""
    kw = dict(q=A, q_stride=1024, k_cache=A, v_cache=A, fp8=False, descale_k=1.0, descale_v=1.0, block_table=A,
              max_pages=(1 << 26) - 1, query_start=A, seq_lens=A, o=A, lse=A, T=600, R=600, Hq=8, Hkv=2, d=128,
              num_pages=11, page_size=32, max_new=1, scale=0.1, causal=True, workspace=A, workspace_bytes=1 << 40)
    assert fa.fa_fwd_paged(**kw, stream=0) == fa.FA_ERR_INVALID_ARG


@pytest.mark.parametrize("page_size", [16, 32, 64, 128, 256])
def test_fwd_paged_rejects_tables_whose_keys_it_cannot_count(page_size):
    """A place among the keys plus a few blocks must fit 32 bits: a table that ends within 512 tokens of 2^31 is refused,
    one page less is not (there the missing workspace is what stops the call)."""
    kw = dict(q=A, q_stride=64, k_cache=A, v_cache=A, fp8=True, descale_k=1.0, descale_v=1.0, block_table=A,
              query_start=A, seq_lens=A, o=A, lse=A, T=1, R=1, Hq=1, Hkv=1, d=64, num_pages=11, page_size=page_size,
              max_new=1, scale=0.1, causal=True, workspace=0, workspace_bytes=0)
    most = (2 ** 31 - 512) // page_size
    assert fa.fa_fwd_paged(max_pages=most + 1, **kw, stream=0) == fa.FA_ERR_INVALID_ARG
    assert fa.fa_fwd_paged(max_pages=most, **kw, stream=0) == fa.FA_ERR_WORKSPACE


def test_helpers_reject_bad_tensors():
    c = paged_ref.case([(5, 2)], 4, 2, 64, 16)
    ints = lambda x: torch.tensor(x, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError):  # CPU tensors
        fa.forward_paged(c["q"], c["k_cache"], c["v_cache"], ints(c["table"]), ints(c["start"]), ints(c["lens"]))
    with pytest.raises(ValueError):
        fa.paged_store(c["k"], c["v"], ints([0, 1]), c["k_cache"], c["v_cache"])
    with pytest.raises(ValueError):
        fa.paged_plan(ints(c["ctx"]), ints(c["new"]), ints(c["table"]), ints(c["free"]), 16, 2)


def test_status_name():
    assert fa.status_string(fa.FA_ERR_NO_PAGES) not in ("unknown status", fa.status_string(fa.FA_ERR_TIMEOUT))


def test_workspace_bytes_of_bad_shapes():
    assert fa.fa_fwd_paged_workspace_bytes(0, 1, 8, 2, 128, 1) == 0
    assert fa.fa_fwd_paged_workspace_bytes(4, 1, 8, 3, 128, 1) == 0
    assert fa.fa_fwd_paged_workspace_bytes(4, 1, 8, 2, 96, 1) == 0


def test_plain_attention_closed_forms():
    """q = 0: the mean of the visible values and the logarithm of their number; the last row equals the unmasked one."""
    c = paged_ref.case([(30, 3), (0, 2)], 4, 2, 64, 16, seed=4)
    q = torch.zeros_like(c["q"])
    o, lse, _ = paged_ref.attention(q, c["k_cache"], c["v_cache"], c["table"], c["start"], c["lens"], 0.5, True)
    v = torch.cat([c["v_cache"][p] for p in c["table"][0][:3]], 1).double()  # [Hkv, 48, d]
    for t in range(3):
        assert torch.allclose(o[t, 3], v[1, :31 + t].mean(0), atol=1e-12)
        assert abs(float(lse[t, 0]) - math.log(31 + t)) < 1e-12
    full = paged_ref.attention(c["q"], c["k_cache"], c["v_cache"], c["table"], c["start"], c["lens"], 0.5, False)
    mask = paged_ref.attention(c["q"], c["k_cache"], c["v_cache"], c["table"], c["start"], c["lens"], 0.5, True)
    assert torch.equal(full[0][2], mask[0][2]) and not torch.equal(full[0][1], mask[0][1])


def test_plain_e4m3_is_torchs_off_the_midpoints():
    g = torch.Generator().manual_seed(3)
    x = torch.randn(20000, generator=g) * 50
    assert torch.equal(paged_ref.e4m3(x.double()).float(), x.clamp(-448, 448).to(torch.float8_e4m3fn).float())


def test_plain_plan_by_hand():
    got = paged_ref.plan([3, 0], [14, 2], [[5, -1], [-1, -1]], [9, 8, 7], 0, 16, 20)
    assert got == ([0, 14, 16], [17, 2], [5 * 16 + p for p in range(3, 16)] + [9 * 16] + [128, 129] + [-1] * 4, 2,
                   [[5, 9], [8, -1]])


def test_kernels_launched_ahead_use_ordinary_loads():
    """A kernel launched as a programmatic dependent is there while the one ahead still writes what it will read, so
    its loads must not be those for data that nobody writes."""
    import os
    import re

    files = [f for f in os.listdir(build.CSRC) if f.endswith((".cu", ".cuh"))]
    text = {f: re.sub(r"//.*", "", open(os.path.join(build.CSRC, f)).read()) for f in files}
    ahead = {f for f in files if re.search(r"launch_dependent|grid_wait", text[f])}
    for _ in files:  # and what these include
        ahead |= {g for f in ahead for g in re.findall(r'#include "([^"/]+\.cuh)"', text[f])}
    assert {"paged_cache.cu", "paged_few.cu", "paged_chunk.cu", "paged_fwd.cu", "paged_pipe.cuh", "paged_work.cuh"} <= ahead
    for f in sorted(ahead):
        assert not re.search(r"__ldg|\.nc\b|__restrict__", text[f]), f
