"""The paged cache's operators on the GPU against their plain 64-bit forms.

Tolerances of the attention, element by element, from its roundings: the weights
enter the second product as bf16 (half a step is 2^-8 of each, so at most 2^-8
sum_j p_j |v_j| in o), o is rounded to bf16 (2^-8 |o|), and the scores are fp32
sums of at most 128 products (|s| stays below 16 here, their error below 128
2^-24 sum |q_i k_i| scale < 2^-13, which moves each weight by that much
relatively, and the logsumexp by it absolutely). With a gain on q the last part
grows with it.
"""
import math

import pytest
import torch

from exact_io_aware_32_gb300 import fa
import paged_ref
import parity

pytestmark = pytest.mark.gpu


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def on_gpu(c):
    if c["q"].stride(0) != c["q"].shape[1] * c["q"].shape[2]:  # slices of one tensor stay so
        base = c["q"]._base.cuda()
        q, k, v = (x.unflatten(1, (-1, c["d"])) for x in base.split([c["Hq"] * c["d"]] + 2 * [c["Hkv"] * c["d"]], 1))
    else:
        q, k, v = (c[x].cuda() for x in "qkv")
    return dict(q=q, k=k, v=v, k_cache=c["k_cache"].cuda(), v_cache=c["v_cache"].cuda(), table=ints(c["table"]),
                start=ints(c["start"]), lens=ints(c["lens"]))


def attend(c, g, causal=True, scale=None, **kw):
    return fa.forward_paged(g["q"], g["k_cache"], g["v_cache"], g["table"], g["start"], g["lens"], causal=causal,
                            scale=scale, descale_k=c["fk"], descale_v=c["fv"], **kw)


def check(c, o, lse, causal=True, scale=None, gain=1.0, start=None, lens=None):
    scale = 1.0 / math.sqrt(c["d"]) if scale is None else scale
    ro, rl, spread = paged_ref.attention(c["q"], c["k_cache"], c["v_cache"], c["table"], start or c["start"],
                                         lens or c["lens"], scale, causal, c["fk"], c["fv"])
    n = (start or c["start"])[-1]
    o, lse = o[:n].double().cpu(), lse[:n].double().cpu()
    ro, rl, spread = ro[:n], rl[:n], spread[:n]
    fin = torch.isfinite(rl)
    assert torch.equal(fin, torch.isfinite(lse)) and not torch.isnan(lse).any()
    score = 2.0 ** -12 * max(1.0, gain)
    err = (o - ro).abs() / (2.0 ** -8 * ro.abs() + (2.0 ** -8 + score) * spread + 1e-30)
    assert float(err.max() if err.numel() else 0.0) <= 1.0, float(err.max())
    assert float((o[~fin]).abs().sum()) == 0.0
    el = (lse[fin] - rl[fin]).abs()
    assert not el.numel() or float(el.max()) <= score + 2.0 ** -22 * float(rl[fin].abs().max()), float(el.max())


EDGE = [(0, 1), (1, 1), (14, 1), (15, 1), (16, 1), (30, 1), (126, 1), (127, 1), (128, 1), (300, 1), (1999, 1)]
CHUNKS = [(0, 129), (5, 127), (1000, 300), (0, 3), (130, 2), (127, 1), (250, 33)]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("ps", [16, 32, 64, 128, 256])
def test_decoding_lengths(ps, d, fp8):
    c = paged_ref.case(EDGE, 8, 2, d, ps, fp8=fp8, seed=ps + d, fused=ps == 32)
    g = on_gpu(c)
    o, lse = attend(c, g, max_new=1)
    parity.check_status()
    check(c, o, lse)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("ps", [16, 32, 64, 128, 256])
def test_chunk_lengths(ps, d, fp8):
    c = paged_ref.case(CHUNKS, 4, 2, d, ps, fp8=fp8, seed=2 * ps + d, fused=ps == 64)
    g = on_gpu(c)
    o, lse = attend(c, g, max_new=300)
    parity.check_status()
    check(c, o, lse)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (5, 5), (6, 2), (7, 1), (20, 4), (32, 2), (33, 1), (64, 1), (100, 1), (128, 1)])
def test_head_groups(Hq, Hkv, d, fp8):
    for lens, most in (([(200, 1), (70, 1), (0, 1)], 1), ([(200, 40), (3, 1), (0, 150)], 150), ([(90, 3), (1, 2)], 3)):
        c = paged_ref.case(lens, Hq, Hkv, d, 16, fp8=fp8, seed=Hq + d)
        g = on_gpu(c)
        o, lse = attend(c, g, max_new=most)
        parity.check_status()
        check(c, o, lse)


@pytest.mark.parametrize("most", [1, 2, 40, 5000])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_every_hint_is_right(d, causal, most):
    """max_new only chooses the layout: too small and too large hints give the same values."""
    c = paged_ref.case([(700, 5), (0, 1), (33, 0), (260, 150), (12, 1)], 8, 2, d, 32, pad=2, seed=d)
    g = on_gpu(c)
    o, lse = attend(c, g, causal=causal, max_new=most)
    parity.check_status()
    check(c, o, lse, causal=causal)


@pytest.mark.parametrize("most", [1, 64])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_rows_without_keys(d, fp8, most):
    """Requests without new tokens, without keys, and with fewer keys than new tokens (the first rows see none)."""
    c = paged_ref.case([(0, 0), (40, 20), (0, 9), (17, 0), (0, 64), (60, 4), (0, 0)], 4, 1, d, 16, fp8=fp8, seed=1)
    lens = list(c["lens"])
    lens[1], lens[2], lens[4] = 7, 0, 30  # rows 0 .. 12 of request 1, all of 2, the first 34 of 4 see no key
    g = on_gpu(c)
    g["lens"] = ints(lens)
    for causal in (True, False):
        o, lse = attend(c, g, causal=causal, max_new=most)
        parity.check_status()
        check(c, o, lse, causal=causal, lens=lens)


@pytest.mark.parametrize("most", [1, 5, 60])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_long_runs_of_requests_without_keys(d, fp8, most):
    """Dozens of tiles in a row that stream nothing (eight key heads each), between, before and behind ones that do."""
    for start in (0, 1):
        lens, keys = [], []
        for i in range(60):
            n = 1 + i % most
            lens.append((30 + 70 * (i % 3), n))
            keys.append(0 if (i // 7 + start) % 2 else lens[-1][0] + n)
        c = paged_ref.case(lens, 16, 8, d, 16, fp8=fp8, seed=d + most, width=100)
        g = on_gpu(c)
        g["lens"] = ints(keys)
        for causal in (True, False):
            o, lse = attend(c, g, causal=causal, max_new=most)
            parity.check_status()
            check(c, o, lse, causal=causal, lens=keys)


@pytest.mark.parametrize("most", [1, 200])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_nan_in_what_a_row_sees_is_not_hidden(d, fp8, most):
    """A NaN in a query, a key or a value reaches the rows that see it, no others (those keep their bits), also where
    the keys are split over the GPU."""
    c = paged_ref.case([(20000, 1), (70, 1), (500, 1 if most == 1 else 150)], 8, 2, d, 32, fp8=fp8, seed=d + most)
    g = on_gpu(c)
    o, lse = attend(c, g, max_new=most)
    check(c, o, lse)

    def planted(name, at):
        x = g[name].clone()
        (x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x)[at] = 0x7F if name != "q" and fp8 else math.nan
        return attend(c, dict(g, **{name: x}), max_new=most)

    def expect(got, rows, heads, cols, lse_too):
        nan = torch.zeros_like(o, dtype=torch.bool)
        nan[rows, heads, cols] = True
        assert torch.equal(torch.isnan(got[0]), nan)
        assert torch.equal(torch.isnan(got[1]), nan.any(-1) if lse_too else torch.zeros_like(lse, dtype=torch.bool))
        assert torch.equal(got[0][~nan], o[~nan])
        keep = ~nan.any(-1) if lse_too else slice(None)
        assert torch.equal(got[1][keep], lse[keep])

    every = slice(None)
    expect(planted("q", (0, 3, 17)), slice(0, 1), slice(3, 4), every, True)
    expect(planted("q", (2, 6, 1)), slice(2, 3), slice(6, 7), every, True)
    for r, key in ((0, 12345), (0, 20000), (1, 3), (2, 7)):  # keys that all tokens of the request see
        rows = slice(c["start"][r], c["start"][r + 1])
        page, slot = c["table"][r][key // 32], key % 32
        expect(planted("k_cache", (page, 1, slot, d - 1)), rows, slice(4, 8), every, True)
        expect(planted("v_cache", (page, 0, slot, 9)), rows, slice(0, 4), slice(9, 10), False)
    parity.check_status()


@pytest.mark.parametrize("most", [1, 200])
def test_rows_behind_the_last_request_stay(most):
    c = paged_ref.case([(100, 1), (5, 130), (0, 1)], 6, 2, 128, 16, pad=37, seed=8)
    g = on_gpu(c)
    n = c["start"][-1]
    o, bo = parity.guarded_empty((c["T"], 6, 128), torch.bfloat16, fill=2.5)
    lse, bl = parity.guarded_empty((c["T"], 6), torch.float32, fill=-3.5)
    need = fa.fa_fwd_paged_workspace_bytes(c["T"], c["R"], 6, 2, 128, most)
    ws, bw = parity.guarded_empty((need,), torch.uint8)
    attend(c, g, max_new=most, out=o, lse=lse, workspace=ws)
    parity.check_status()
    assert all(parity.guards_intact(b) for b in (bo, bl, bw))
    assert bool((o[n:] == 2.5).all()) and bool((lse[n:] == -3.5).all())
    check(c, o, lse)


@pytest.mark.parametrize("most", [1, 200])
def test_output_aligned_to_16_bytes_only(most):
    c = paged_ref.case([(100, 1), (5, 130), (0, 1)], 4, 2, 64, 16, seed=18)
    g = on_gpu(c)
    n = c["T"] * 4 * 64
    o = torch.zeros(n + 8, dtype=torch.bfloat16, device="cuda")[8:].view(c["T"], 4, 64)
    assert o.data_ptr() % 32 == 16
    o, lse = attend(c, g, max_new=most, out=o)
    parity.check_status()
    check(c, o, lse)


@pytest.mark.parametrize("fp8", [False, True])
def test_sharp_softmax(fp8):
    """Scores of hundreds: the running maximum moves far, and most weights vanish."""
    c = paged_ref.case([(900, 1), (300, 70), (2500, 1)], 8, 2, 128, 64, fp8=fp8, seed=5, gain=16.0)
    g = on_gpu(c)
    for most in (1, 70):
        o, lse = attend(c, g, max_new=most)
        parity.check_status()
        check(c, o, lse, gain=16.0)


@pytest.mark.parametrize("d,fp8,ps", [(128, False, 16), (64, True, 128), (128, True, 256), (64, False, 64)])
def test_long_request(d, fp8, ps):
    """One long request with one new token and with several: the keys are spread over the GPU and joined."""
    for lens, most in (([(70001, 1)], 1), ([(30011, 3), (20, 1)], 3)):
        c = paged_ref.case(lens, 4, 2, d, ps, fp8=fp8, seed=ps)
        g = on_gpu(c)
        o, lse = attend(c, g, max_new=most)
        parity.check_status()
        check(c, o, lse)
        again = attend(c, g, max_new=most)
        assert torch.equal(o, again[0]) and torch.equal(lse, again[1])


def test_long_chunk_with_decoding_requests():
    c = paged_ref.case([(9000, 1), (1500, 700), (31, 1), (0, 520)], 8, 4, 128, 32, pad=5, seed=77)
    g = on_gpu(c)
    o, lse = attend(c, g, max_new=700)
    parity.check_status()
    check(c, o, lse)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_mixed_batch_with_a_wide_table(d, fp8):
    """A table wide enough for many keys: decoding requests and chunks go to kernels of their own."""
    lens = [((i * 531) % 900, 1 + i % 3) for i in range(150)]
    lens[7], lens[70], lens[71], lens[149] = (300, 290), (0, 9), (40, 0), (10, 200)
    c = paged_ref.case(lens, 8, 2, d, 16, fp8=fp8, seed=31, width=2048, pad=3)
    g = on_gpu(c)
    lens = list(c["lens"])
    lens[70], lens[3], lens[149] = 4, 0, 100  # rows that see no key in each
    g["lens"] = ints(lens)
    for causal in (True, False):
        o, lse = attend(c, g, causal=causal, max_new=290)
        parity.check_status()
        check(c, o, lse, causal=causal, lens=lens)


@pytest.mark.parametrize("d", [64, 128])
def test_tiles_around_the_shortest_cut(d):
    """Tiles of 7 to 20 key blocks, few of them, so that every CTA's range ends somewhere inside one."""
    for blocks in (7, 8, 9, 11, 12, 13, 16, 20):
        c = paged_ref.case([(128 * blocks - 40, 36), (0, 1), (128 * blocks - 1, 1)], 2, 1, d, 128, seed=blocks)
        g = on_gpu(c)
        o, lse = attend(c, g, max_new=40)
        parity.check_status()
        check(c, o, lse)


@pytest.mark.parametrize("width", [64, 65])
@pytest.mark.parametrize("most", [1, 40])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_tables_of_eight_blocks_and_one_page_more(d, fp8, most, width):
    """Tables for 1024 keys: no tile is cut and no second kernel joins; for 1040: cuts again."""
    lens = [(16 * width - most, most), (1000, 1), (0, 1), (16 * width - 1, 1), (500, most)] * 7
    c = paged_ref.case(lens, 8, 2, d, 16, fp8=fp8, seed=width)
    g = on_gpu(c)
    o, lse = attend(c, g, max_new=most)
    parity.check_status()
    check(c, o, lse)


def test_many_requests():
    """More requests than threads of a block, most of them short, some empty."""
    lens = [((i * 37) % 90, (i * 7) % 3) for i in range(1500)]
    for most in (2, 40):
        c = paged_ref.case(lens, 2, 1, 64, 16, seed=9)
        g = on_gpu(c)
        o, lse = attend(c, g, max_new=most)
        parity.check_status()
        check(c, o, lse)


def test_pages_past_four_gigabytes():
    """The pages in use lie behind 2^32 bytes and 2^31 elements of the cache."""
    P, Hkv, ps, d = 40000, 4, 128, 128
    c = paged_ref.case([(300, 1), (129, 2)], 8, Hkv, d, ps, seed=13)
    g = on_gpu(c)
    big = [torch.empty((P, Hkv, ps, d), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    used = sorted({p for row in c["table"] for p in row if p >= 0})
    far = {p: P - 1 - i for i, p in enumerate(used)}
    for b, name in zip(big, ("k_cache", "v_cache")):
        for p in used:
            b[far[p]] = g[name][p]
    g["k_cache"], g["v_cache"] = big
    g["table"] = ints([[far.get(p, -1) for p in row] for row in c["table"]])
    o, lse = attend(c, g, max_new=2)
    parity.check_status()
    check(c, o, lse)
    k = torch.randn((1, Hkv, d), device="cuda").to(torch.bfloat16)
    fa.paged_store(k, k, ints([(P - 9) * ps + 77]), *big)
    parity.check_status()
    assert torch.equal(big[0][P - 9, :, 77], k[0]) and torch.equal(big[1][P - 9, :, 77], k[0])


def test_shared_pages():
    """Two requests whose first pages are the same ones."""
    c = paged_ref.case([(64, 1), (80, 1)], 4, 2, 64, 32, seed=3)
    c["table"][1][:2] = c["table"][0][:2]
    g = on_gpu(c)
    o, lse = attend(c, g, max_new=1)
    parity.check_status()
    check(c, o, lse)


def test_bad_pages_and_lengths_are_reported():
    """Nothing out of range is followed: the call reports it, the other requests' rows are right."""
    c = paged_ref.case([(200, 1), (90, 1), (40, 1), (300, 2)], 4, 2, 64, 16, seed=6)
    want = [torch.cat([x[:1], x[3:]]) for x in attend(c, on_gpu(c))]
    bad = [list(r) for r in c["table"]]
    bad[1][2], bad[2][0] = 1 << 30, -1
    g = on_gpu(c)
    g["table"] = ints(bad)
    for most in (1, 2, 100):
        o, lse = attend(c, g, max_new=most)
        torch.cuda.synchronize()
        assert fa.fa_device_status(True) == fa.FA_ERR_INVALID_ARG
        got = [torch.cat([x[:1], x[3:]]) for x in (o, lse)]
        assert (got[0].float() - want[0].float()).abs().max() < 0.05 and (got[1] - want[1]).abs().max() < 1e-3
        g2 = on_gpu(c)
        width = len(c["table"][0])
        for name, x in (("lens", [201, 91, 41, 10 ** 9]), ("lens", [201, 91, 41, -5]), ("start", [0, 1, 2, 3, 10 ** 9]),
                        ("start", [0, 1, -4, 3, 5]), ("start", [0, 3, 2, 3, 5])):
            g2 = on_gpu(c)
            g2[name] = ints(x)
            if name == "lens" and x[3] > 0:
                g2["table"] = ints([(row + [row[0]] * width)[:width] if i < 3 else
                                    [p if p >= 0 else row[0] for p in row] for i, row in enumerate(c["table"])])
            o, lse = attend(c, g2, max_new=most)
            torch.cuda.synchronize()
            assert fa.fa_device_status(True) == fa.FA_ERR_INVALID_ARG, (name, x)
            if name == "lens":
                assert (o[0].float() - want[0][0].float()).abs().max() < 0.05


# ---------------------------------------------------------------- plan
def run_plan(ctx, new, ps, pad=0, head=0, width=None, spare=5, seed=0):
    g = torch.Generator().manual_seed(seed)
    held = [-(-c // ps) for c in ctx]
    after = [-(-(c + n) // ps) for c, n in zip(ctx, new)]
    width = width or max(max(after), 1) + 2
    perm = torch.randperm(sum(after) + spare + head, generator=g).tolist()
    table, at = [], 0
    for x in held:
        table.append(perm[at:at + x] + [-1] * (width - x))
        at += x
    free, T = perm[at:], max(1, sum(new) + pad)
    tab = ints(table)
    got = fa.paged_plan(ints(ctx), ints(new), tab, ints(free), ps, T, free_head=ints([head]) if head else None)
    return got, tab, paged_ref.plan(ctx, new, table, free, head, ps, T)


@pytest.mark.parametrize("ps", [16, 128, 256])
@pytest.mark.parametrize("R", [1, 7, 8, 9, 256, 257, 3000, 9001])
def test_plan(R, ps):
    for ctx, new, kw in (([(i * 53) % 400 for i in range(R)], [1] * R, {}),
                         ([(i * 53) % 400 for i in range(R)], [(i * 31) % 140 for i in range(R)], dict(pad=300, head=3)),
                         ([0] * R, [0] * R, dict(pad=1)),
                         ([0] * R, [5000 if i == R // 2 else 0 for i in range(R)], {})):
        got, tab, want = run_plan(ctx, new, ps, seed=R, **kw)
        parity.check_status()
        start, lens, slots, taken, table = want
        assert got[0].tolist() == start and got[1].tolist() == lens and got[2].tolist() == slots
        assert got[3].tolist() == [taken] and tab.tolist() == table


def test_plan_reports_what_does_not_fit():
    ps = 16
    tab = ints([[3, -1], [-1, -1]])
    args = dict(block_table=tab, page_size=ps)
    # three pages needed, two free: the last request lacks one
    q, lens, slots, taken = fa.paged_plan(ints([10, 0]), ints([10, 20]), free_pages=ints([8, 9]), num_tokens=30, **args)
    torch.cuda.synchronize()
    assert fa.fa_device_status(True) == fa.FA_ERR_NO_PAGES
    assert tab.tolist() == [[3, 8], [9, -1]] and taken.tolist() == [2]
    assert slots.tolist() == [3 * 16 + p for p in range(10, 16)] + [128 + p for p in range(4)] + [144 + p for p in range(16)] + [-1] * 4
    assert q.tolist() == [0, 10, 30] and lens.tolist() == [20, 20]
    # an empty list, and a head past the list's end
    for kw in (dict(free_pages=ints([])), dict(free_pages=ints([8, 9]), free_head=ints([5]))):
        tab.copy_(ints([[3, -1], [-1, -1]]))
        slots, taken = fa.paged_plan(ints([15, 0]), ints([2, 0]), num_tokens=2, **kw, **args)[2:]
        torch.cuda.synchronize()
        assert fa.fa_device_status(True) == fa.FA_ERR_NO_PAGES
        assert slots.tolist() == [63, -1] and taken.tolist() == [0]
    # negative lengths, a table too narrow, more rows than T: reported, and nothing is written past an end
    many = ints(list(range(20, 30)))
    for ctx, new, T in (([-3, 0], [1, 1], 2), ([0, 0], [-1, 1], 2), ([0, 0], [40, 1], 41), ([0, 0], [3, 4], 5)):
        tab, bt = parity.guarded_empty((2, 2), torch.int32, fill=-1)
        slots, bs = parity.guarded_empty((T,), torch.int32, fill=-9)
        start, bq = parity.guarded_empty((3,), torch.int32, fill=-9)
        lens, bl = parity.guarded_empty((2,), torch.int32, fill=-9)
        fa.paged_plan(ints(ctx), ints(new), tab, many, ps, T, out=(start, lens, slots, ints([0])))
        torch.cuda.synchronize()
        assert fa.fa_device_status(True) == fa.FA_ERR_INVALID_ARG
        assert all(parity.guards_intact(b) for b in (bt, bs, bq, bl))
        assert max(start.tolist()) <= T and max(lens.tolist()) <= 32 and -9 not in slots.tolist()


# ---------------------------------------------------------------- store
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T,Hkv,d,ps,fused", [(1, 1, 64, 16, False), (3, 5, 128, 32, True), (130, 8, 64, 256, True),
                                              (1031, 2, 128, 64, False), (517, 12, 64, 128, False)])
def test_store(T, Hkv, d, ps, fused, fp8):
    gen = torch.Generator().manual_seed(T)
    P = T // ps + 4
    c = paged_ref.case([(0, T)], 2 * Hkv, Hkv, d, ps, seed=T, fused=fused)
    g = on_gpu(c)
    slots = torch.randperm(P * ps, generator=gen)[:T].tolist()
    for i in range(0, T, 7):
        slots[i] = -1 - i % 3
    fk, fv = (0.0131, 0.37) if fp8 else (1.0, 1.0)
    caches = []
    for _ in range(2):
        t, b = parity.guarded_empty((P, Hkv, ps, d), torch.uint8 if fp8 else torch.bfloat16)
        t.copy_(torch.randint(0, 120, t.shape, generator=gen).cuda())
        caches.append((t, b))
    want = [t.cpu() for t, _ in caches]
    fa.paged_store(g["k"], g["v"], ints(slots), caches[0][0], caches[1][0], fk, fv)
    parity.check_status()
    for w, x, f in zip(want, (c["k"], c["v"]), (fk, fv)):
        for t, s in enumerate(slots):
            if s >= 0:
                w[s // ps, :, s % ps] = paged_ref.e4m3(x[t].double() / f32(f)).float().to(torch.float8_e4m3fn).view(torch.uint8) \
                    if fp8 else x[t]
    for (t, b), w in zip(caches, want):
        assert parity.guards_intact(b) and torch.equal(t.cpu(), w)


@pytest.mark.parametrize("T,Hkv,d,ps,fused", [(12007, 8, 128, 64, True), (31001, 5, 64, 16, False), (16411, 3, 128, 256, False)])
def test_store_of_many_tokens(T, Hkv, d, ps, fused):
    """More E4M3 pieces than threads: each thread takes several, and pieces of the last pass end inside a block."""
    gen = torch.Generator().manual_seed(T)
    P = T // ps + 2
    base = torch.randn((T, 3 * Hkv * d), generator=gen).to(torch.bfloat16)
    k, v = (base[:, i * Hkv * d:(i + 1) * Hkv * d].unflatten(1, (Hkv, d)) for i in (1, 2))
    on = base.cuda()
    gk, gv = (on[:, i * Hkv * d:(i + 1) * Hkv * d].unflatten(1, (Hkv, d)) for i in (1, 2))
    if not fused:
        gk, gv = gk.contiguous(), gv.contiguous()
    slots = torch.randperm(P * ps, generator=gen)[:T].to(torch.int32)
    slots[::7] = -2
    caches = [parity.guarded_empty((P, Hkv, ps, d), torch.uint8) for _ in range(2)]
    for t, _ in caches:
        t.fill_(77)
    fa.paged_store(gk, gv, slots.cuda(), caches[0][0], caches[1][0], 0.0131, 0.37)
    parity.check_status()
    put = slots >= 0
    s = slots[put].long()
    for x, f, (t, b) in zip((k, v), (0.0131, 0.37), caches):
        want = torch.full((P, ps, Hkv, d), 77, dtype=torch.uint8)
        codes = paged_ref.e4m3(x[put].double() / f32(f)).float().to(torch.float8_e4m3fn).view(torch.uint8)
        want.view(P * ps, Hkv, d)[s] = codes
        assert parity.guards_intact(b) and torch.equal(t.cpu(), want.transpose(1, 2))


def f32(x):
    return float(torch.tensor(x, dtype=torch.float32))


def test_store_rounds_once():
    """Every bf16 value over factors chosen so that many quotients fall on or next to the middle of two codes; then
    what has no code: infinities saturate, NaN stays NaN."""
    bits = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    x = bits[torch.isfinite(bits.float())]
    x = torch.cat([x, torch.zeros((-x.numel()) % 64)]).to(torch.bfloat16).reshape(-1, 1, 64)
    T = x.shape[0]
    for f in (1.0, 0.0625, 3.0, f32(1 / 3), f32(0.1), f32(17 / 16), f32(1.0 + 2.0 ** -23), f32(1 - 2.0 ** -24), 1e-30, 1e30):
        k8, v8 = (torch.zeros((T // 16 + 1, 1, 16, 64), dtype=torch.uint8, device="cuda") for _ in range(2))
        fa.paged_store(x.cuda(), x.cuda(), ints(list(range(T))), k8, v8, f, f)
        parity.check_status()
        want = paged_ref.e4m3(x.double() / f).float().to(torch.float8_e4m3fn).float()
        got = k8.cpu().view(torch.float8_e4m3fn).float().reshape(-1, 1, 64)[:T]
        assert torch.equal(got, want), f
        assert torch.equal(k8, v8)
    odd = torch.zeros(1, 1, 64)
    odd[0, 0, :3] = torch.tensor([math.inf, -math.inf, math.nan])
    k8 = torch.zeros((1, 1, 16, 64), dtype=torch.float8_e4m3fn, device="cuda")
    fa.paged_store(odd.to(torch.bfloat16).cuda(), odd.to(torch.bfloat16).cuda(), ints([3]), k8, k8.clone(), 0.5, 0.5)
    got = k8[0, 0, 3, :4].float().tolist()
    assert got[:2] == [448.0, -448.0] and math.isnan(got[2]) and got[3] == 0.0


def test_store_reports_slots_past_the_cache():
    k = torch.randn((3, 2, 64), device="cuda").to(torch.bfloat16)
    kc, bk = parity.guarded_empty((2, 2, 16, 64), torch.bfloat16, fill=1.0)
    vc, bv = parity.guarded_empty((2, 2, 16, 64), torch.bfloat16, fill=1.0)
    fa.paged_store(k, k, ints([32, 5, 2 ** 31 - 1]), kc, vc)
    torch.cuda.synchronize()
    assert fa.fa_device_status(True) == fa.FA_ERR_INVALID_ARG
    assert parity.guards_intact(bk) and parity.guards_intact(bv)
    assert torch.equal(kc[0, :, 5], k[1]) and int((kc != 1.0).any(-1).sum()) <= 2


# ---------------------------------------------------------------- together
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_serving_equals_attention_over_the_whole_text(d, fp8):
    """Three requests, their prompts in chunks, then single tokens, through plan, store and attention: every row equals
    the row of plain causal attention over its request's whole text."""
    Hq, Hkv, ps, P = 6, 2, 32, 40
    steps = [(150, 0, 33), (70, 9, 0), (1, 200, 1), (1, 1, 1), (1, 1, 60), (1, 1, 1)]
    total = [sum(s[r] for s in steps) for r in range(3)]
    c = [paged_ref.case([(0, n)], Hq, Hkv, d, ps, fp8=fp8, seed=20 + r) for r, n in enumerate(total)]
    g = [on_gpu(x) for x in c]
    dt = torch.float8_e4m3fn if fp8 else torch.bfloat16
    cache = [torch.full((P, Hkv, ps, d), math.nan, device="cuda").to(dt) for _ in range(2)]
    table = torch.full((3, 16), -1, dtype=torch.int32, device="cuda")
    free, head = ints(torch.randperm(P).tolist()), ints([0])
    ctx, done = ints([0, 0, 0]), [0, 0, 0]
    got = [[], [], []]
    fk, fv = c[0]["fk"], c[0]["fv"]
    for s in steps:
        T = sum(s) + 2
        rows = {n: torch.cat([g[r][n][done[r]:done[r] + s[r]] for r in range(3)] + [g[0][n][:2]]) for n in "qkv"}
        start, lens, slots, taken = fa.paged_plan(ctx, ints(list(s)), table, free, ps, T, free_head=head)
        fa.paged_store(rows["k"], rows["v"], slots, *cache, descale_k=fk, descale_v=fv)
        o, lse = fa.forward_paged(rows["q"], *cache, table, start, lens, max_new=max(s), descale_k=fk, descale_v=fv)
        head = head + taken
        ctx = lens
        at = 0
        for r in range(3):
            got[r].append((o[at:at + s[r]], lse[at:at + s[r]]))
            at += s[r]
            done[r] += s[r]
    parity.check_status()
    for r in range(3):
        n, x = total[r], c[r]
        pages = -(-n // ps)
        for name, src, f in (("k_cache", "k", fk), ("v_cache", "v", fv)):
            rows = x[src].double()
            rows = paged_ref.e4m3(rows / f32(f)) if fp8 else rows
            full = torch.zeros((pages * ps, Hkv, d), dtype=torch.float64)
            full[:n] = rows
            x[name] = full.reshape(pages, ps, Hkv, d).permute(0, 2, 1, 3)
        x["table"] = [list(range(pages))]
        check(x, torch.cat([y[0] for y in got[r]]), torch.cat([y[1] for y in got[r]]))


@pytest.mark.parametrize("most", [1, 6])
def test_captured_step_replays_with_other_lengths(most):
    """Plan, store and attention captured once and replayed with other lengths, tables and rows."""
    Hq, Hkv, d, ps = 8, 2, 128, 16
    A = paged_ref.case([(40, 1), (300, most), (0, 1)], Hq, Hkv, d, ps, pad=4, seed=1, width=40, spare=40)
    B = paged_ref.case([(500, 1), (2, 1), (77, most)], Hq, Hkv, d, ps, pad=4, seed=2, width=40, spare=23)
    P = max(A["k_cache"].shape[0], B["k_cache"].shape[0])
    static = dict(q=torch.empty_like(A["q"], device="cuda"), ctx=ints(A["ctx"]), new=ints(A["new"]),
                  table=ints(A["table"]), lens=ints(A["lens"]), start=ints(A["start"]),
                  k_cache=torch.zeros((P, Hkv, ps, d), dtype=torch.bfloat16, device="cuda"),
                  v_cache=torch.zeros((P, Hkv, ps, d), dtype=torch.bfloat16, device="cuda"), free=ints(A["free"][:20]))
    out = [torch.empty(n, dtype=torch.int32, device="cuda") for n in (4, 3, A["T"], 1)]
    o = torch.zeros((A["T"], Hq, d), dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros((A["T"], Hq), dtype=torch.float32, device="cuda")
    k = torch.empty((A["T"], Hkv, d), dtype=torch.bfloat16, device="cuda")

    def load(c):
        static["q"].copy_(c["q"])
        static["ctx"].copy_(ints(c["ctx"]))
        static["new"].copy_(ints(c["new"]))
        # the tables before the step: only the pages held
        held = [[p if i < -(-n // ps) else -1 for i, p in enumerate(r)] for r, n in zip(c["table"], c["ctx"])]
        static["table"].copy_(ints(held))
        fresh = [p for r, n, t in zip(c["table"], c["ctx"], c["lens"]) for p in r[-(-n // ps):-(-t // ps)]]
        static["free"].copy_(ints((fresh + c["free"])[:20]))
        for name in ("k_cache", "v_cache"):
            static[name][:c[name].shape[0]] = c[name].cuda()
        k.copy_(new_rows(c))

    def new_rows(c):  # the new tokens' keys as the case's cache holds them
        x = torch.zeros((c["T"], Hkv, d), dtype=torch.bfloat16)
        for r in range(3):
            for i in range(c["new"][r]):
                p = c["ctx"][r] + i
                x[c["start"][r] + i] = c["k_cache"][c["table"][r][p // ps], :, p % ps]
        return x

    def step():
        start, lens, slots, _ = fa.paged_plan(static["ctx"], static["new"], static["table"], static["free"], ps,
                                              A["T"], out=out)
        fa.paged_store(k, k, slots, static["k_cache"], static["v_cache"])
        fa.forward_paged(static["q"], static["k_cache"], static["v_cache"], static["table"], start, lens, max_new=most,
                         out=o, lse=lse)

    load(A)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for c in (B, A, B):
        load(c)
        graph.replay()
        parity.check_status()
        same = dict(c)
        same["v_cache"] = c["v_cache"].clone()
        for r in range(3):  # the values of the new tokens are their keys here
            for i in range(c["new"][r]):
                p = c["ctx"][r] + i
                same["v_cache"][c["table"][r][p // ps], :, p % ps] = c["k_cache"][c["table"][r][p // ps], :, p % ps]
        check(same, o, lse)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("most", [1, 64])
def test_wait_that_runs_out_is_reported(most, fp8):
    """The failure path: the first query tile is withheld, every CTA gives up after a second, and the next call is right."""
    c = paged_ref.case([(100, 1), (600, 20)], 4, 2, 128, 16, fp8=fp8, seed=2)
    g = on_gpu(c)
    assert fa.fa_test_arm_fault(1) == fa.FA_OK
    attend(c, g, max_new=most)
    torch.cuda.synchronize()
    assert fa.fa_device_status(True) == fa.FA_ERR_TIMEOUT
    o, lse = attend(c, g, max_new=most)
    parity.check_status()
    check(c, o, lse)


def test_two_streams_at_once():
    """Two batches on two streams at the same time, each with its own workspace."""
    cs = [paged_ref.case(lens, 8, 2, 128, 16, seed=i) for i, lens in enumerate(([(4000, 1), (77, 1)], [(900, 200), (5, 1)]))]
    gs = [on_gpu(c) for c in cs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    res = []
    for _ in range(5):
        res = [attend(c, g, max_new=m, stream=s) for c, g, m, s in zip(cs, gs, (1, 200), streams)]
    parity.check_status()
    for c, (o, lse) in zip(cs, res):
        check(c, o, lse)


def test_helpers_refuse():
    c = paged_ref.case([(20, 2)], 4, 2, 64, 16, seed=1)
    g = on_gpu(c)
    with pytest.raises(ValueError):
        fa.forward_paged(g["q"].float(), g["k_cache"], g["v_cache"], g["table"], g["start"], g["lens"])
    with pytest.raises(ValueError):
        fa.forward_paged(g["q"].transpose(0, 1), g["k_cache"], g["v_cache"], g["table"], g["start"], g["lens"])
    with pytest.raises(ValueError):
        fa.forward_paged(g["q"], g["k_cache"], g["v_cache"].float(), g["table"], g["start"], g["lens"])
    with pytest.raises(ValueError):
        fa.forward_paged(g["q"], g["k_cache"], g["v_cache"], g["table"].long(), g["start"], g["lens"])
    with pytest.raises(ValueError):
        fa.forward_paged(g["q"], g["k_cache"], g["v_cache"], g["table"], g["start"][:-1], g["lens"])
    with pytest.raises(ValueError):
        attend(c, g, out=torch.empty((2, 4, 64), device="cuda"))
    with pytest.raises(fa.FAError):
        attend(c, g, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        fa.paged_store(g["k"][:, :1], g["v"], ints([0, 1]), g["k_cache"], g["v_cache"])
    with pytest.raises(ValueError):
        fa.paged_store(g["k"], g["v"], ints([0]), g["k_cache"], g["v_cache"])
    with pytest.raises(fa.FAError):
        fa.paged_plan(ints([3]), ints([1]), ints([[0]]), ints([1]), 20, 1)
