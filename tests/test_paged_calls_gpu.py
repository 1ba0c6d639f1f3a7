"""Calls of the paged cache's operators that their documentation allows and that are easy to get wrong: stream handles,
steps back to back, lengths and tables at the limits of what is counted."""
import math

import pytest
import torch

from exact_io_aware_32_gb300 import fa
import paged_ref
import parity
from test_paged_gpu import attend, check, f32, ints, on_gpu

pytestmark = pytest.mark.gpu


def test_stream_handles():
    """A raw handle names that very stream, 0 the default one: the work of a call stands behind what that stream holds."""
    c = paged_ref.case([(300, 1), (20, 3)], 4, 2, 64, 16, seed=40)
    g = on_gpu(c)
    want = attend(c, g, max_new=3)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for current, handle in ((side, 0), (side, torch.cuda.default_stream().cuda_stream),
                            (torch.cuda.default_stream(), side.cuda_stream)):
        with torch.cuda.stream(current), fa._on(handle, g["q"]):
            assert torch.cuda.current_stream().cuda_stream == handle
        # the queries arrive late on the handle's stream, which need not be the current one
        late = dict(g, q=torch.zeros_like(g["q"]))
        o, lse = torch.zeros_like(want[0]), torch.zeros_like(want[1])
        torch.cuda.synchronize()
        with torch.cuda.stream(torch.cuda.default_stream() if handle == 0 else side):
            torch.cuda._sleep(20000000)
            late["q"].copy_(g["q"])
        with torch.cuda.stream(current):
            attend(c, late, max_new=3, out=o, lse=lse, stream=handle)
        parity.check_status()
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_steps_back_to_back(d, fp8, captured):
    """Twelve steps of plan, store and attention with no other kernel between them, each step's lengths, table and rows
    written by the kernels just ahead, in place: every row as in plain attention over its request's whole text."""
    Hq, Hkv, ps, steps = 6, 2, 16, 12
    per = [(150, 1, 33) if i % 3 == 0 else (1, 1, 1) if i % 3 == 1 else (2, 70, 1) for i in range(steps)]
    total = [sum(s[r] for s in per) for r in range(3)]
    c = [paged_ref.case([(0, n)], Hq, Hkv, d, ps, fp8=fp8, seed=50 + r) for r, n in enumerate(total)]
    g = [on_gpu(x) for x in c]
    fk, fv = c[0]["fk"], c[0]["fv"]
    need = sum(-(-n // ps) for n in total)
    perm = torch.randperm(need + 3, generator=torch.Generator().manual_seed(d)).tolist()
    free = ints(perm)
    cache = [torch.zeros((need + 3, Hkv, ps, d), device="cuda").to(torch.float8_e4m3fn if fp8 else torch.bfloat16) for _ in "kv"]
    table = torch.full((3, max(-(-n // ps) for n in total)), -1, dtype=torch.int32, device="cuda")
    state, done, at = [], [0, 0, 0], 0
    ctx = zero = torch.zeros(3, dtype=torch.int32, device="cuda")
    for s in per:
        T = sum(s)
        rows = {n: torch.cat([g[r][n][done[r]:done[r] + s[r]] for r in range(3)]) for n in "qkv"}
        out = [torch.zeros(n, dtype=torch.int32, device="cuda") for n in (4, 3, T, 1)]
        state.append(dict(rows, new=ints(list(s)), T=T, ctx=ctx, free=free[at:], out=out, most=max(s),
                          o=torch.zeros((T, Hq, d), dtype=torch.bfloat16, device="cuda"),
                          lse=torch.zeros((T, Hq), dtype=torch.float32, device="cuda")))
        ctx = out[1]
        at += sum(-(-(done[r] + s[r]) // ps) - -(-done[r] // ps) for r in range(3))
        done = [a + b for a, b in zip(done, s)]
    ws = torch.empty(max(fa.fa_fwd_paged_workspace_bytes(x["T"], 3, Hq, Hkv, d, x["most"]) for x in state),
                     dtype=torch.uint8, device="cuda")

    def run():
        for x in state:
            start, lens, slots, _ = fa.paged_plan(x["ctx"], x["new"], table, x["free"], ps, x["T"], out=x["out"])
            fa.paged_store(x["k"], x["v"], slots, *cache, descale_k=fk, descale_v=fv)
            fa.forward_paged(x["q"], *cache, table, start, lens, max_new=x["most"], descale_k=fk, descale_v=fv,
                             out=x["o"], lse=x["lse"], workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run()
    for again in range(3):
        for x in state:
            x["o"].fill_(7.0)
            x["lse"].fill_(7.0)
            for t in x["out"]:
                t.fill_(-9)
        table.fill_(-1)
        for t in cache:
            t.view(torch.uint8).fill_(0)
        free.copy_(ints(perm if again != 1 else perm[::-1]))
        zero.zero_()
        graph.replay() if captured else run()
        parity.check_status()
        for r, n in enumerate(total):
            x = dict(c[r])
            pages = -(-n // ps)
            for name, src, f in (("k_cache", "k", fk), ("v_cache", "v", fv)):
                full = torch.zeros((pages * ps, Hkv, d), dtype=torch.float64)
                full[:n] = paged_ref.e4m3(x[src].double() / f32(f)) if fp8 else x[src].double()
                x[name] = full.reshape(pages, ps, Hkv, d).permute(0, 2, 1, 3)
            x["table"] = [list(range(pages))]
            at = [sum(s[:r]) for s in per]
            check(x, *(torch.cat([y[name][a:a + s[r]] for y, a, s in zip(state, at, per)]) for name in ("o", "lse")))


@pytest.mark.parametrize("most", [32, 1 << 21])
def test_two_million_tokens_of_which_few_see_a_key(most):
    """A request of 2^21 new tokens and 128 keys: the last 128 rows are right, the others saw no key. (Counted as if the
    tokens without keys had some, its tiles of 32 rows were more blocks than 32 bits hold.)"""
    T, n = 1 << 21, 128
    c = paged_ref.case([(0, n)], 8, 8, 64, 128, seed=60)
    g = on_gpu(c)
    q = torch.randn((T, 8, 64), device="cuda", dtype=torch.bfloat16)
    q[T - n:] = g["q"]
    o, lse = fa.forward_paged(q, g["k_cache"], g["v_cache"], g["table"], ints([0, T]), ints([n]), max_new=most)
    parity.check_status()
    check(c, o[T - n:], lse[T - n:])
    assert not bool(o[:T - n].any()) and bool((lse[:T - n] == -float("inf")).all())


@pytest.mark.parametrize("R", [64, 512])
@pytest.mark.parametrize("most", [1, 64, 1 << 16])
def test_requests_that_share_rows_are_not_counted_past_the_call(R, most):
    """Every other request claims all 2^16 rows: far more blocks than the call of so many rows that the host admitted
    (with 512 requests than 32 bits hold). Reported, and nothing out of range is walked."""
    T, Hq, Hkv, d, ps, keys = 1 << 16, 32, 8, 64, 256, 131072
    q = torch.ones((T, Hq, d), dtype=torch.bfloat16, device="cuda")
    kc, vc = (torch.ones((3, Hkv, ps, d), dtype=torch.bfloat16, device="cuda") for _ in "kv")
    table = torch.zeros((R, keys // ps), dtype=torch.int32, device="cuda")
    out, bo = parity.guarded_empty((T, Hq, d), torch.bfloat16, fill=2.5)
    lse, bl = parity.guarded_empty((T, Hq), torch.float32, fill=-3.5)
    fa.forward_paged(q, kc, vc, table, ints([0, T] * (R // 2) + [0]), ints([keys] * R), max_new=most, causal=False, out=out,
                     lse=lse)
    torch.cuda.synchronize()
    assert fa.fa_device_status(True) == fa.FA_ERR_INVALID_ARG
    assert parity.guards_intact(bo) and parity.guards_intact(bl)
    assert bool((out == 2.5).all()) and bool((lse == -3.5).all())


@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("d,fp8", [(64, False), (128, True)])
def test_the_widest_table(d, fp8, n):
    """2^31 - 612 keys, all but the last page's the same page of zero keys; the last page's keys stand out so far (a score
    of 40) that a row is the mean of its visible values there. Equal weights are powers of two, so o is off by its own
    rounding (2^-8) and fp32 sums of at most 156 terms (below 2^-12 of their mean magnitude); the 2^31 other keys weigh
    2^31 e^-39 < 2^-25."""
    ps, width = 256, (2 ** 31 - 512) // 256
    L = width * ps - 100
    dt = torch.float8_e4m3fn if fp8 else torch.bfloat16
    gen = torch.Generator().manual_seed(d)
    c = 5.0 if d == 64 else 3.5
    kc = torch.zeros((2, 1, ps, d))
    kc[1, 0, :156] = c
    vc = torch.randn((2, 1, ps, d), generator=gen)
    kc[1, 0, 156:], vc[1, 0, 156:] = float("nan"), float("nan")
    kc, vc = kc.to(dt), vc.to(dt)
    table = torch.zeros((1, width), dtype=torch.int32, device="cuda")
    table[0, -1] = 1
    q = torch.ones((n, 2, d), dtype=torch.bfloat16, device="cuda")
    o, lse = fa.forward_paged(q, kc.cuda(), vc.cuda(), table, ints([0, n]), ints([L]), max_new=n)
    parity.check_status()
    for t in range(n):
        seen = vc[1, 0, :156 - n + t + 1].double()
        want, mag = seen.mean(0), seen.abs().mean(0)
        assert bool(((o[t].double().cpu() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -12 * mag).all()), t
        s = math.sqrt(d) * c + math.log(seen.shape[0])
        assert bool(((lse[t].double().cpu() - s).abs() <= 2.0 ** -12).all()), t


def test_plan_reports_a_bad_free_list():
    """A negative page in the free list and a negative head are reported like any other entry out of range; what does
    not depend on them is right."""
    tab = ints([[3, -1], [-1, -1]])
    start, lens, slots, taken = fa.paged_plan(ints([10, 0]), ints([10, 4]), tab, ints([-5, 7]), 16, 14)
    torch.cuda.synchronize()
    assert fa.fa_device_status(True) == fa.FA_ERR_INVALID_ARG
    assert start.tolist() == [0, 10, 14] and lens.tolist() == [20, 4] and taken.tolist() == [2]
    assert slots.tolist() == [3 * 16 + p for p in range(10, 16)] + [-1] * 4 + [7 * 16 + p for p in range(4)]
    assert tab.tolist()[1] == [7, -1] and tab.tolist()[0][0] == 3
    tab = ints([[3, -1], [-1, -1]])
    start, lens, slots, taken = fa.paged_plan(ints([10, 0]), ints([2, 4]), tab, ints([5, 7]), 16, 6, free_head=ints([-2]))
    torch.cuda.synchronize()
    assert fa.fa_device_status(True) == fa.FA_ERR_INVALID_ARG
    assert tab.tolist() == [[3, -1], [5, -1]] and taken.tolist() == [1]
    assert slots.tolist() == [58, 59, 80, 81, 82, 83]
    # a negative page that nobody takes is nobody's fault
    fa.paged_plan(ints([10, 0]), ints([2, 4]), tab, ints([5, -7]), 16, 6)
    parity.check_status()


# Factors past 2^-100 and 2^100 and subnormal ones; then f = floor(2^20 X / 17) 2^-149 for 8-bit X, where x = X 2^-133 lies so
# little above f times 17 / 16, the middle of two codes, that x - 17 / 16 f is less than half the smallest subnormal.
FAR = [1.1 * 2.0 ** -101, 1.1 * 2.0 ** 101, 2.0 ** -100, 2.0 ** 100, 1e-37, 1e37, 1e-38, 3e-39, 1e-40, 7 * 2.0 ** -149, 2.0 ** -149,
       2.0 ** -126 * 1.37, 2.0 ** -127 * 1.9, 3.4e38] + [(2 ** 20 * X // 17) * 2.0 ** -149 for X in range(136, 256)]


def test_store_rounds_once_with_factors_far_from_one():
    """Every finite bf16 value over each factor, as the exact quotient rounds."""
    bits = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    x = bits[torch.isfinite(bits.float())]
    x = torch.cat([x, torch.zeros((-x.numel()) % 64)]).to(torch.bfloat16).reshape(-1, 1, 64)
    T = x.shape[0]
    gx, slots = x.cuda(), ints(list(range(T)))
    near = 0
    for f in map(f32, FAR):
        k8, v8 = (torch.zeros((T // 16 + 1, 1, 16, 64), dtype=torch.uint8, device="cuda") for _ in range(2))
        fa.paged_store(gx, gx, slots, k8, v8, f, f)
        parity.check_status()
        # in 64 bits the quotient of 8 and 24 bits is never rounded onto the middle of two codes
        want = paged_ref.e4m3(x.double() / f).float().to(torch.float8_e4m3fn).float()
        got = k8.cpu().view(torch.float8_e4m3fn).float().reshape(-1, 1, 64)[:T]
        assert torch.equal(got, want), (f, x[got != want])
        assert torch.equal(k8, v8)
        near += int(((x.double() / f - 17 / 16).abs() < 2.0 ** -24).sum())
    assert near >= 50  # the factors do what they are there for


@pytest.mark.parametrize("most", [1, 60])
@pytest.mark.parametrize("times", [1, 30, 300])
@pytest.mark.parametrize("d", [64, 128])
def test_a_dominating_channel_over_e4m3_keys(d, times, most):
    """One channel of q far above the others, its keys small, so that what the two E4M3 parts of q lose of the others is
    what shows. An element of q is off by less than 2^-16 of its row's largest, a score by D = scale f_k 2^-16 max |q| sum
    |code| at most, a weight by a factor within e^+-2D, the logsumexp by D; with that the roundings of P to f16 (2^-11),
    of o (2^-8), and of fp32 scores (|s| < 40: 128 2^-24 sum |q k| scale < 2^-10)."""
    c = paged_ref.case([(500, 1), (2000, most), (60, 1)], 8, 2, d, 16, fp8=True, seed=70 + d)
    c["q"][..., 5] = (c["q"][..., 5].float().sign() * times).to(torch.bfloat16)
    codes = c["k_cache"].float()
    codes[..., 5] = (codes[..., 5] / times).clamp(-20, 20)  # (NaN where nothing was written stays)
    c["k_cache"] = codes.to(torch.float8_e4m3fn)
    g = on_gpu(c)
    o, lse = attend(c, g, max_new=most)
    parity.check_status()
    scale = 1.0 / math.sqrt(d)
    ro, rl, spread = paged_ref.attention(c["q"], c["k_cache"], c["v_cache"], c["table"], c["start"], c["lens"], scale, True,
                                         c["fk"], c["fv"])
    worst = float(torch.nan_to_num(c["k_cache"].float()).abs().sum(-1).max())
    D = 2.0 ** -16 * c["q"].double().abs().amax(-1) * scale * c["fk"] * worst
    n = c["start"][-1]
    o, lse = o[:n].double().cpu(), lse[:n].double().cpu()
    assert bool(((lse - rl[:n]).abs() <= D[:n] + 2.0 ** -10).all())
    part = torch.expm1(2 * D)[:n, :, None] + 2.0 ** -10 + 2.0 ** -11
    assert bool(((o - ro[:n]).abs() <= 2.0 ** -8 * ro[:n].abs() + part * spread[:n]).all())
    print(times, float(D.max()), float((lse - rl[:n]).abs().max()))


def test_plan_with_more_tokens_than_rows_keeps_the_rest_right():
    """Ten new tokens for six rows: reported; the request that is cut has the keys of the tokens that got a row, the one
    after it none of its own, so that the step's attention reads nothing that was never stored."""
    Hq, Hkv, d, ps = 4, 2, 64, 16
    c = paged_ref.case([(20, 4), (33, 3), (18, 3)], Hq, Hkv, d, ps, seed=90)
    g = on_gpu(c)
    start, lens, slots, _ = fa.paged_plan(ints(c["ctx"]), ints(c["new"]), g["table"], ints([0]), ps, 6)
    torch.cuda.synchronize()
    assert fa.fa_device_status(True) == fa.FA_ERR_INVALID_ARG
    assert start.tolist() == [0, 4, 6, 6] and lens.tolist() == [24, 35, 18]
    place = lambda r, p: c["table"][r][p // ps] * ps + p % ps  # noqa: E731
    assert slots.tolist() == [place(0, p) for p in range(20, 24)] + [place(1, p) for p in range(33, 35)]
    o, lse = fa.forward_paged(g["q"][:6], g["k_cache"], g["v_cache"], g["table"], start, lens, max_new=4)
    parity.check_status()
    check(c, o, lse, start=start.tolist(), lens=lens.tolist())
