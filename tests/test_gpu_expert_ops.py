"""The expert operators on the GPU, against plain products in 64 bits.

Tolerances, fixed before any run.  A product's fp32 sum of D exact products
may be off by one unit (2^-23) per addition of the sum of the magnitudes, D + 2
additions; its one rounding to the result's type by half a step
(finfo.eps / 2 of the value, and half the smallest subnormal for fp16).  int8:
the integer sum is exact, then one conversion and two products in fp32.
SwiGLU: e^-g by the fast exponential is off by 2 + 1.173 |g| units in the last
place (CUDA's bound), the fast quotient by 2, every other operation by half;
one unit is 2^-23 of the value.
"""
import numpy as np
import pytest
import torch

import expert_ffn_layer_route_b200 as moe
import moe_inputs as mi

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
U = 2.0 ** -23


def half_step(t):
    return torch.finfo(t).eps / 2


def tiny(t):
    return {BF16: 2.0 ** -134, FP16: 2.0 ** -25, FP32: 2.0 ** -150}[t]


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def pitched(shape, dtype, extra=0):
    """Zeros whose rows start on 16-byte boundaries, `extra` pieces of 16 bytes longer than they have to be."""
    per = 16 // torch.empty(0, dtype=dtype).element_size()
    return torch.zeros(*shape[:-1], (-(-shape[-1] // per) + extra) * per, dtype=dtype, device=DEV)[..., : shape[-1]]


def normal(shape, dtype, g, std=1.0, extra=0):
    t = pitched(shape, dtype, extra)
    t.copy_(torch.randn(shape, generator=g, device=DEV) * std)
    return t


def codes(shape, g, extra=0):
    t = pitched(shape, torch.int8, extra)
    t.copy_(torch.randint(-127, 128, shape, generator=g, device=DEV))
    return t


def offsets_of(counts, first=0):
    return torch.tensor(np.concatenate([[first], first + np.cumsum(counts)]), dtype=torch.int32, device=DEV)


def ok():
    torch.cuda.synchronize()
    assert moe.moe_get_last_error() == 0


def check(got, ref, bound, t=None):
    t = t or got.dtype
    got = got.double()
    assert torch.equal(torch.isfinite(got), torch.isfinite(ref))
    allowed = ref.abs() * half_step(t) + tiny(t) + bound * (1 + half_step(t))
    worst = ((got - ref).abs() - allowed).max().item()
    assert worst <= 0, f"off by {worst:.3e} more than the bound"


def ref_forward(x, w, off):
    """(out, sum of magnitudes) in 64 bits; rows in no group are zero."""
    o = off.tolist()
    out = torch.zeros(x.shape[0], w.shape[1], dtype=torch.float64, device=DEV)
    mag = torch.zeros_like(out)
    for e in range(len(o) - 1):
        r = slice(o[e], o[e + 1])
        out[r] = x[r].double() @ w[e].double().t()
        mag[r] = x[r].double().abs() @ w[e].double().abs().t()
    return out, mag


def ref_grad_w(dy, x, off):
    o = off.tolist()
    E = len(o) - 1
    dw = torch.zeros(E, dy.shape[1], x.shape[1], dtype=torch.float64, device=DEV)
    mag = torch.zeros_like(dw)
    for e in range(E):
        r = slice(o[e], o[e + 1])
        dw[e] = dy[r].double().t() @ x[r].double()
        mag[e] = dy[r].double().abs().t() @ x[r].double().abs()
    return dw, mag


# name, rows of each expert, N, K
GROUPS = [
    ("one_row", [0, 1, 0], 40, 24),
    ("one_value", [1], 1, 1),
    ("few", [3, 0, 0, 7, 1], 130, 70),
    ("dense", [200], 257, 129),
    ("all_to_last", [0, 0, 0, 0, 65], 128, 64),
    ("all_to_first", [31, 0, 0], 64, 192),
    ("sixteens", [16, 32, 48, 64], 256, 128),
    ("off_by_one", [15, 17, 33, 63, 65, 127, 129], 136, 328),
    ("wide_tiles", [513, 255, 257, 1], 264, 200),
    ("many", [i % 5 for i in range(384)], 72, 88),
    ("limit_E", [(i * 7) % 3 for i in range(1024)], 16, 40),
    ("deep", [5, 9], 24, 5000),
    ("long", [1500, 700], 33, 31),
    ("gptoss_like", [2, 0, 1, 5, 0, 3], 2880, 2880),
]
IDS = [g[0] for g in GROUPS]


@pytest.mark.parametrize("name,counts,N,K", GROUPS, ids=IDS)
@pytest.mark.parametrize("t,ot", [(BF16, BF16), (FP16, FP16), (BF16, FP32), (FP16, BF16)], ids=str)
def test_forward(name, counts, N, K, t, ot):
    g = gen(1)
    R, E = sum(counts), len(counts)
    x, w, off = normal((R, K), t, g), normal((E, N, K), t, g, 0.1), offsets_of(counts)
    out = torch.full((R, N), 7.0, dtype=ot, device=DEV)
    moe.moe_grouped_gemm(x, w, off, out)
    ok()
    ref, mag = ref_forward(x, w, off)
    check(out, ref, mag * (K + 2) * U)


@pytest.mark.parametrize("name,counts,N,K", GROUPS, ids=IDS)
@pytest.mark.parametrize("t,ot", [(BF16, BF16), (FP16, FP16), (BF16, FP32), (FP16, BF16)], ids=str)
def test_grad_x(name, counts, N, K, t, ot):
    g = gen(2)
    R, E = sum(counts), len(counts)
    dy, w, off = normal((R, N), t, g), normal((E, N, K), t, g, 0.1), offsets_of(counts)
    dx = torch.full((R, K), 7.0, dtype=ot, device=DEV)
    moe.moe_grouped_gemm_grad_x(dy, w, off, dx)
    ok()
    ref, mag = ref_forward(dy, w.transpose(1, 2), off)
    check(dx, ref, mag * (N + 2) * U)


@pytest.mark.parametrize("name,counts,N,K", GROUPS, ids=IDS)
@pytest.mark.parametrize("t,ot", [(BF16, BF16), (FP16, FP16), (BF16, FP32), (FP16, BF16)], ids=str)
def test_grad_w(name, counts, N, K, t, ot):
    g = gen(3)
    R, E = sum(counts), len(counts)
    dy, x, off = normal((R, N), t, g), normal((R, K), t, g), offsets_of(counts)
    dw = torch.full((E, N, K), 7.0, dtype=ot, device=DEV)
    moe.moe_grouped_gemm_grad_w(dy, x, off, dw)
    ok()
    ref, mag = ref_grad_w(dy, x, off)
    check(dw, ref, mag * (max(counts) + 2) * U)


@pytest.mark.parametrize("name,counts,N,K", GROUPS, ids=IDS)
@pytest.mark.parametrize("ot", [BF16, FP16, FP32], ids=str)
def test_int8(name, counts, N, K, ot):
    g = gen(4)
    R, E = sum(counts), len(counts)
    x, w, off = codes((R, K), g), codes((E, N, K), g), offsets_of(counts)
    sx = torch.rand(R, generator=g, device=DEV) * 0.01
    sw = torch.rand(E, N, generator=g, device=DEV) * 0.01
    out = torch.full((R, N), 7.0, dtype=ot, device=DEV)
    moe.moe_grouped_gemm_i8(x, sx, w, sw, off, out)
    ok()
    acc, _ = ref_forward(x, w, off)
    e = torch.repeat_interleave(torch.arange(E, device=DEV), torch.tensor(counts, device=DEV))
    ref = acc * sx.double()[:, None] * sw.double()[e]
    check(out, ref, ref.abs() * 4 * 2.0 ** -24)


def test_int8_extreme_codes_sum_exactly():
    """-128 and 127 over the longest rows: the int32 sums reach 2^31 - 16384 and are exact."""
    K, N = 131056, 40
    x = torch.full((3, K), -128, dtype=torch.int8, device=DEV)
    w = torch.full((1, N, K), -128, dtype=torch.int8, device=DEV)
    x[1] = 127
    x[2, ::2] = 127
    out = torch.empty(3, N, dtype=FP32, device=DEV)
    moe.moe_grouped_gemm_i8(x, torch.ones(3, device=DEV), w, torch.ones(1, N, device=DEV), offsets_of([3]), out)
    ok()
    want = torch.tensor([128 * 128 * K, -127 * 128 * K, 64 * K], dtype=torch.float64).float()  # the one conversion
    assert torch.equal(out.cpu(), want[:, None].expand(3, N))


PITCHES = [(0, 0, 0, 0), (1, 0, 2, 0), (3, 8, 1, 5), (0, 3, 0, 1)]


@pytest.mark.parametrize("px,po,pw,ps", PITCHES)
def test_pitches_and_unaligned_results(px, po, pw, ps):
    """Operands with longer rows and matrices apart, results with odd pitches on odd addresses; what lies
    between the rows stays as it was."""
    g = gen(5)
    counts, N, K = [4, 0, 37, 2], 77, 53
    R, E = sum(counts), len(counts)
    off = offsets_of(counts)
    x, dy = normal((R, K), BF16, g, 1, px), normal((R, N), BF16, g, 1, px)
    w = normal((E, N + ps, K), BF16, g, 0.1, pw)[:, :N]
    for name, rows, cols in (("fwd", R, N), ("gx", R, K), ("gw", E * N, K)):
        for ot in (BF16, FP32):
            store = torch.full((rows * (cols + po) + 1,), 7.0, dtype=ot, device=DEV)
            view = store[1:].view(rows, cols + po)  # an address that is aligned to its type only
            if name == "fwd":
                moe.moe_grouped_gemm(x, w, off, view[:, :cols])
                ref, mag = ref_forward(x, w, off)
                b = mag * (K + 2) * U
            elif name == "gx":
                moe.moe_grouped_gemm_grad_x(dy, w, off, view[:, :cols])
                ref, mag = ref_forward(dy, w.transpose(1, 2), off)
                b = mag * (N + 2) * U
            else:
                moe.moe_grouped_gemm_grad_w(dy, x, off, view[:, :cols].unflatten(0, (E, N)))
                ref, mag = (t.flatten(0, 1) for t in ref_grad_w(dy, x, off))
                b = mag * (max(counts) + 2) * U
            ok()
            check(view[:, :cols], ref, b)
            assert store[0] == 7.0 and bool((view[:, cols:] == 7.0).all())


def _poison(t, rows):
    t[rows] = float("nan")
    t[rows, ::3] = float("inf")


@pytest.mark.parametrize("first,behind", [(0, 9), (5, 0), (3, 70)])
def test_rows_outside_the_groups(first, behind):
    """NaN and infinities in rows of no group reach nothing, and their results stay as they were."""
    g = gen(6)
    counts, N, K = [7, 0, 18, 1, 40], 96, 72
    R = first + sum(counts) + behind
    off = offsets_of(counts, first)
    last = first + sum(counts)
    rows = torch.cat([torch.arange(0, first), torch.arange(last, R)]).to(DEV)
    x, dy, w = normal((R, K), BF16, g), normal((R, N), BF16, g), normal((5, N, K), BF16, g, 0.1)
    _poison(x, rows)
    _poison(dy, rows)
    out, dx = (torch.full((R, n), 7.0, dtype=BF16, device=DEV) for n in (N, K))
    dw = torch.full((5, N, K), 7.0, device=DEV)
    moe.moe_grouped_gemm(x, w, off, out)
    moe.moe_grouped_gemm_grad_x(dy, w, off, dx)
    moe.moe_grouped_gemm_grad_w(dy, x, off, dw)
    ok()
    inside = slice(first, last)
    ref, mag = ref_forward(x, w, off)
    check(out[inside], ref[inside], mag[inside] * (K + 2) * U)
    ref, mag = ref_forward(dy, w.transpose(1, 2), off)
    check(dx[inside], ref[inside], mag[inside] * (N + 2) * U)
    ref, mag = ref_grad_w(dy, x, off)
    check(dw, ref, mag * 42 * U)
    assert bool((out[rows] == 7.0).all()) and bool((dx[rows] == 7.0).all())
    q, sx = codes((R, K), g), torch.rand(R, device=DEV)
    sx[rows] = float("nan")
    wq, sw = codes((5, N, K), g), torch.rand(5, N, device=DEV)
    out.fill_(7.0)
    moe.moe_grouped_gemm_i8(q, sx, wq, sw, off, out)
    ok()
    assert bool((out[rows] == 7.0).all()) and bool(torch.isfinite(out).all())


@pytest.mark.parametrize("counts", [[5, 3, 20], [17, 1, 1], [64, 65, 63], [1, 1, 1, 1]])
def test_a_row_with_nan_stays_in_its_row_and_its_expert(counts):
    g = gen(7)
    N, K = 80, 48
    R, E = sum(counts), len(counts)
    off = offsets_of(counts)
    x, dy, w = normal((R, K), FP16, g), normal((R, N), FP16, g), normal((E, N, K), FP16, g, 0.1)
    bad = counts[0]  # the first row of expert 1
    x[bad, 3] = float("nan")
    dy[bad, 5] = float("inf")
    out, dx = torch.empty(R, N, dtype=FP16, device=DEV), torch.empty(R, K, dtype=FP16, device=DEV)
    dw = torch.empty(E, N, K, device=DEV)
    moe.moe_grouped_gemm(x, w, off, out)
    moe.moe_grouped_gemm_grad_x(dy, w, off, dx)
    moe.moe_grouped_gemm_grad_w(dy, x, off, dw)
    ok()
    others = [r for r in range(R) if r != bad]
    assert bool(torch.isfinite(out[others]).all()) and bool(torch.isnan(out[bad]).all())
    assert bool(torch.isfinite(dx[others]).all()) and not bool(torch.isfinite(dx[bad]).any())
    assert bool(torch.isfinite(dw[[e for e in range(E) if e != 1]]).all())
    assert not bool(torch.isfinite(dw[1, 5]).any()) and not bool(torch.isfinite(dw[1, :, 3]).any())


def test_slot_map():
    """Matrices anywhere, twice, or not resident; a slot out of range is reported and skipped."""
    g = gen(8)
    counts, N, K = [6, 2, 0, 33, 1], 144, 96
    R = sum(counts)
    off = offsets_of(counts)
    x, dy, w = normal((R, K), BF16, g), normal((R, N), BF16, g), normal((3, N, K), BF16, g, 0.1)
    q, wq = codes((R, K), g), codes((3, N, K), g)
    sx, sw = torch.rand(R, device=DEV), torch.rand(3, N, device=DEV)
    for slots, status in (([2, 0, 1, 2, 1], 0), ([2, -1, -1, 0, 1], 0), ([2, 3, 1, 0, -7], 9), ([1, 1, 99, 1, 1], 0)):
        m = torch.tensor(slots, dtype=torch.int32, device=DEV)
        live = torch.tensor([r for e in range(5) for r in range(int(off[e]), int(off[e + 1])) if 0 <= slots[e] < 3])
        gone = torch.tensor([r for r in range(R) if r not in set(live.tolist())], dtype=torch.long)
        full = w[[s if 0 <= s < 3 else 0 for s in slots]]
        out, dx = torch.full((R, N), 7.0, dtype=BF16, device=DEV), torch.full((R, K), 7.0, dtype=BF16, device=DEV)
        o8 = torch.full((R, N), 7.0, dtype=FP32, device=DEV)
        for call in (lambda: moe.moe_grouped_gemm(x, w, off, out, slot_map=m),
                     lambda: moe.moe_grouped_gemm_grad_x(dy, w, off, dx, slot_map=m),
                     lambda: moe.moe_grouped_gemm_i8(q, sx, wq, sw, off, o8, slot_map=m)):
            call()
            assert moe.moe_get_last_error() == status  # (a bad slot of an empty group is not looked at)
        ref, mag = ref_forward(x, full, off)
        check(out[live], ref[live], mag[live] * (K + 2) * U)
        ref, mag = ref_forward(dy, full.transpose(1, 2), off)
        check(dx[live], ref[live], mag[live] * (N + 2) * U)
        e = torch.repeat_interleave(torch.arange(5, device=DEV), torch.tensor(counts, device=DEV))
        at = torch.tensor([s if 0 <= s < 3 else 0 for s in slots], device=DEV)[e]
        ref = ref_forward(q, wq[[s if 0 <= s < 3 else 0 for s in slots]], off)[0] * sx.double()[:, None] * sw.double()[at]
        check(o8[live], ref[live], ref[live].abs() * 2.0 ** -22)
        for t in (out, dx, o8):
            assert bool((t[gone] == 7.0).all())


def test_bad_offsets_are_reported_and_skipped():
    g = gen(9)
    N, K, R = 64, 64, 20
    x, dy, w = normal((R, K), BF16, g), normal((R, N), BF16, g), normal((3, N, K), BF16, g, 0.1)
    for o in ([0, 5, 3, 8], [-4, 2, 6, 9], [0, 4, 8, 21], [0, 4, 2 ** 31 - 1, 2 ** 31 - 1]):
        off = torch.tensor(o, dtype=torch.int32, device=DEV)
        good = [e for e in range(3) if 0 <= o[e] <= o[e + 1] <= R]
        out, dw = torch.full((R, N), 7.0, dtype=BF16, device=DEV), torch.full((3, N, K), 7.0, device=DEV)
        moe.moe_grouped_gemm(x, w, off, out)
        assert moe.moe_get_last_error() == 9
        moe.moe_grouped_gemm_grad_w(dy, x, off, dw)
        assert moe.moe_get_last_error() == 9
        for e in range(3):
            if e in good:
                r = slice(o[e], o[e + 1])
                ref = dy[r].double().t() @ x[r].double()
                check(dw[e], ref, (dy[r].double().abs().t() @ x[r].double().abs()) * 10 * U)
            else:
                assert bool((dw[e] == 0).all())
    out = torch.empty(R, N, dtype=BF16, device=DEV)
    moe.moe_grouped_gemm(x, w, offsets_of([5, 5, 10]), out)  # the library still works
    ok()


@pytest.mark.parametrize("R", [10, 300])
def test_offsets_that_go_back_and_forth(R):
    """Groups that claim the same rows: reported; every row gets the product of one of the experts, whole."""
    g = gen(26)
    E, N, K = 64, 96, 72
    off = torch.tensor([0, R - 3] * (E // 2) + [0], dtype=torch.int32, device=DEV)
    x = normal((R, K), BF16, g)
    w = normal((1, N, K), BF16, g, 0.1).expand(E, N, K).contiguous()
    out = torch.full((R, N), 7.0, dtype=BF16, device=DEV)
    moe.moe_grouped_gemm(x, w, off, out)
    assert moe.moe_get_last_error() == 9
    ref, mag = ref_forward(x, w, offsets_of([R - 3] + [0] * (E - 1)))
    check(out[: R - 3], ref[: R - 3], mag[: R - 3] * (K + 2) * U)
    assert bool((out[R - 3:] == 7.0).all())


@pytest.mark.parametrize("K", [40, 41])
def test_grad_w_accumulates(K):
    g = gen(10)
    counts, N = [30, 0, 3, 80], 100
    off = offsets_of(counts)
    dy, x = normal((113, N), BF16, g), normal((113, K), BF16, g)
    before = torch.randn(4, N, K, generator=g, device=DEV)
    dw = before.clone()
    moe.moe_grouped_gemm_grad_w(dy, x, off, dw, accumulate=True)
    ok()
    ref, mag = ref_grad_w(dy, x, off)
    check(dw, before.double() + ref, mag * 82 * U)
    assert torch.equal(dw[1], before[1])


def test_grad_w_without_rows_writes_zeros():
    for rows in (0, 5):
        dw = torch.full((3, 40, 24), 7.0, dtype=BF16, device=DEV)
        off = torch.zeros(4, dtype=torch.int32, device=DEV)
        moe.moe_grouped_gemm_grad_w(torch.zeros(rows, 40, dtype=BF16, device=DEV),
                                    torch.zeros(rows, 24, dtype=BF16, device=DEV), off, dw)
        ok()
        assert bool((dw == 0).all())


def test_fp16_overflow_becomes_infinity_and_fp32_keeps_it():
    x = torch.full((2, 64), 60000.0, dtype=FP16, device=DEV)
    w = torch.full((1, 16, 64), 100.0, dtype=FP16, device=DEV)
    out, out32 = torch.empty(2, 16, dtype=FP16, device=DEV), torch.empty(2, 16, dtype=FP32, device=DEV)
    moe.moe_grouped_gemm(x, w, offsets_of([2]), out)
    moe.moe_grouped_gemm(x, w, offsets_of([2]), out32)
    ok()
    assert bool(torch.isinf(out).all()) and bool((out32 == 64 * 60000.0 * 100.0).all())


def test_results_past_32_bit_offsets():
    """Elements beyond 2^31 of x, of the result and of the matrices."""
    K, N = 64, 4096
    R = (1 << 31) // N + 40
    x = torch.zeros(R, K, dtype=BF16, device=DEV)
    x[-24:] = torch.randn(24, K, device=DEV)
    w = torch.randn(2, N, K, device=DEV).to(BF16)
    out = torch.empty(R, N, dtype=BF16, device=DEV)
    off = torch.tensor([0, R - 16, R], dtype=torch.int32, device=DEV)
    moe.moe_grouped_gemm(x, w, off, out)
    ok()
    tail = slice(R - 24, R)
    ref, mag = ref_forward(x[tail], w, torch.tensor([0, 8, 24]))
    check(out[tail], ref, mag * (K + 2) * U)
    del out
    big = torch.zeros((1 << 31) // (2048 * 2048) + 2, 2048, 2048, dtype=BF16, device=DEV)
    E = big.shape[0]
    big[-1] = torch.randn(2048, 2048, device=DEV).to(BF16)
    xs = torch.randn(5, 2048, device=DEV).to(BF16)
    off = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    off[-1] = 5
    out = torch.empty(5, 2048, dtype=FP32, device=DEV)
    moe.moe_grouped_gemm(xs, big, off, out)
    ok()
    ref = xs.double() @ big[-1].double().t()
    check(out, ref, (xs.double().abs() @ big[-1].double().abs().t()) * 2050 * U)
    moe.moe_grouped_gemm_grad_w(out.to(BF16), xs, off, big)
    ok()
    ref = out.to(BF16).double().t() @ xs.double()
    check(big[-1], ref, (out.to(BF16).double().abs().t() @ xs.double().abs()) * 7 * U)
    assert bool((big[-2] == 0).all())


# rows of each expert, N, K: a handful of rows, where a kernel of its own runs, and just past it
FEW = [([1] * 4, 130, 264), ([0, 1, 0, 2, 0, 0, 1], 33, 17), ([2, 0, 1], 257, 1), ([1] * 12, 64, 2880),
       ([1] * 13, 64, 2880), ([1] * 16, 40, 5000), ([1] * 17, 40, 5000), ([5, 1, 1, 1, 0, 0, 0, 0], 96, 520),
       ([2], 100, 300), ([3], 100, 300), ([0] * 1023 + [1], 35, 1031), ([6], 70, 4099), ([7], 70, 4099),
       ([1, 5, 4], 129, 2600), ([2, 3], 5, 9), ([4], 2, 130), ([6, 6], 300, 8200)]


@pytest.mark.parametrize("counts,N,K", FEW, ids=[f"{sum(c)}of{len(c)}" for c, _, _ in FEW])
@pytest.mark.parametrize("first,behind", [(0, 0), (2, 3)])
def test_few_rows(counts, N, K, first, behind):
    """Pads and rows outside the groups hold NaN and garbage; slots are permuted."""
    g = gen(21)
    E, R = len(counts), first + sum(counts) + behind
    off = offsets_of(counts, first)
    inside = slice(first, first + sum(counts))
    slots = torch.randperm(E, generator=torch.Generator().manual_seed(2)).to(torch.int32)
    for t in (BF16, FP16):
        x, w = normal((R, K), t, g), normal((E, N, K), t, g, 0.1)
        for m in (x, w):  # behind the rows' ends
            if m._base is not None and m._base.shape[-1] > K:
                m._base[..., K:] = float("nan")
        x[:first], x[first + sum(counts):] = float("nan"), float("inf")
        for ot in (t, FP32):
            out = torch.full((R, N), 7.0, dtype=ot, device=DEV)
            moe.moe_grouped_gemm(x, w, off, out, slot_map=slots.to(DEV))
            ok()
            ref, mag = ref_forward(x, w[slots.long()], off)
            check(out[inside], ref[inside], mag[inside] * (K + 2) * U)
            assert bool((out[:first] == 7.0).all()) and bool((out[first + sum(counts):] == 7.0).all())
    x, w = codes((R, K), g), codes((E, N, K), g)
    for m in (x, w):
        if m._base is not None and m._base.shape[-1] > K:
            m._base[..., K:] = 99
    sx, sw = torch.rand(R, device=DEV), torch.rand(E, N, device=DEV)
    out = torch.full((R, N), 7.0, device=DEV)
    moe.moe_grouped_gemm_i8(x, sx, w, sw, off, out, slot_map=slots.to(DEV))
    ok()
    e = torch.repeat_interleave(torch.arange(E), torch.tensor(counts))
    ref = ref_forward(x, w[slots.long()], off)[0][inside]
    ref = ref * sx[inside].double()[:, None] * sw[slots.long()][e.to(DEV)].double()
    check(out[inside], ref, ref.abs() * 2.0 ** -22)


def test_pads_of_every_operand_are_not_read():
    """NaN behind the rows' ends and between the matrices reaches nothing, in every kernel."""
    g = gen(22)
    for counts, N, K in (([3, 40, 0, 9], 77, 53), ([300, 5], 150, 70)):
        R, E = sum(counts), len(counts)
        off = offsets_of(counts)
        x, dy = normal((R, K), BF16, g, 1, 1), normal((R, N), BF16, g, 1, 1)
        wide = normal((E, N + 3, K), BF16, g, 0.1, 1)
        w = wide[:, :N]
        for m, n in ((x, K), (dy, N), (wide, K)):
            m._base[..., n:] = float("nan")
        wide[:, N:] = float("inf")
        out, dx = torch.empty(R, N, dtype=BF16, device=DEV), torch.empty(R, K, dtype=BF16, device=DEV)
        dw = torch.empty(E, N, K, device=DEV)
        moe.moe_grouped_gemm(x, w, off, out)
        moe.moe_grouped_gemm_grad_x(dy, w, off, dx)
        moe.moe_grouped_gemm_grad_w(dy, x, off, dw)
        ok()
        ref, mag = ref_forward(x, w, off)
        check(out, ref, mag * (K + 2) * U)
        ref, mag = ref_forward(dy, w.transpose(1, 2), off)
        check(dx, ref, mag * (N + 2) * U)
        ref, mag = ref_grad_w(dy, x, off)
        check(dw, ref, mag * (max(counts) + 2) * U)


@pytest.mark.parametrize("R", [3, 40])
def test_no_group_at_all(R):
    """Every group empty, or every expert away: nothing is written but grad_w's zeros."""
    g = gen(23)
    x, dy, w = normal((R, 64), BF16, g), normal((R, 96), BF16, g), normal((5, 96, 64), BF16, g)
    q, wq, sx, sw = codes((R, 64), g), codes((5, 96, 64), g), torch.rand(R, device=DEV), torch.rand(5, 96, device=DEV)
    away = torch.full((5,), -1, dtype=torch.int32, device=DEV)
    for off, m in ((torch.zeros(6, dtype=torch.int32, device=DEV), None),
                   (torch.full((6,), R, dtype=torch.int32, device=DEV), None), (offsets_of([R, 0, 0, 0, 0]), away)):
        out, dx = torch.full((R, 96), 7.0, dtype=BF16, device=DEV), torch.full((R, 64), 7.0, dtype=BF16, device=DEV)
        moe.moe_grouped_gemm(x, w, off, out, slot_map=m)
        moe.moe_grouped_gemm_grad_x(dy, w, off, dx, slot_map=m)
        moe.moe_grouped_gemm_i8(q, sx, wq, sw, off, out, slot_map=m)
        ok()
        assert bool((out == 7.0).all()) and bool((dx == 7.0).all())
    dw = torch.full((5, 96, 64), 7.0, device=DEV)
    moe.moe_grouped_gemm_grad_w(dy, x, torch.zeros(6, dtype=torch.int32, device=DEV), dw)
    ok()
    assert bool((dw == 0).all())
    dw.fill_(7.0)
    moe.moe_grouped_gemm_grad_w(dy, x, torch.zeros(6, dtype=torch.int32, device=DEV), dw, accumulate=True)
    ok()
    assert bool((dw == 7.0).all())


@pytest.mark.parametrize("N,K", [(24, 40), (300, 264), (130, 67)])
def test_many_small_tiles_and_wide_offsets_of_one_call(N, K):
    """1024 experts, most of one to three rows, two with many."""
    g = gen(24)
    counts = [(i * 5) % 4 for i in range(1024)]
    counts[3], counts[700] = 600, 259
    off, R = offsets_of(counts), sum(counts)
    x, w = normal((R, K), FP16, g), normal((1024, N, K), FP16, g, 0.1)
    out = torch.empty(R, N, dtype=FP16, device=DEV)
    moe.moe_grouped_gemm(x, w, off, out)
    ok()
    ref, mag = ref_forward(x, w, off)
    check(out, ref, mag * (K + 2) * U)
    dy, dw = normal((R, N), FP16, g), torch.empty(1024, N, K, dtype=FP16, device=DEV)
    moe.moe_grouped_gemm_grad_w(dy, x, off, dw)
    ok()
    ref, mag = ref_grad_w(dy, x, off)
    check(dw, ref, mag * 602 * U)


def test_gradients_against_differences():
    """One number of x and of w moved a little either way: the slope of sum(out * dy) is the gradient."""
    g = gen(25)
    counts, N, K = [5, 0, 33], 40, 24
    off = offsets_of(counts)
    x, dy, w = normal((38, K), BF16, g), normal((38, N), BF16, g), normal((3, N, K), BF16, g, 0.1)
    dx, dw = torch.empty(38, K, device=DEV), torch.empty(3, N, K, device=DEV)
    moe.moe_grouped_gemm_grad_x(dy, w, off, dx)
    moe.moe_grouped_gemm_grad_w(dy, x, off, dw)
    ok()

    def loss(a, b):
        return (ref_forward(a, b, off)[0] * dy.double()).sum().item()

    xd, wd, step = x.double(), w.double(), 0.5  # the loss is linear in either: any step will do
    for r, k in ((0, 0), (4, 23), (5, 7), (37, 11)):
        e = torch.zeros_like(xd)
        e[r, k] = step
        assert abs((loss(xd + e, wd) - loss(xd - e, wd)) / (2 * step) - dx[r, k].item()) <= 1e-4
    for n, i, k in ((0, 0, 0), (0, 39, 23), (2, 17, 5), (1, 3, 3)):
        e = torch.zeros_like(wd)
        e[n, i, k] = step
        assert abs((loss(xd, wd + e) - loss(xd, wd - e)) / (2 * step) - dw[n, i, k].item()) <= 1e-3


@pytest.mark.parametrize("counts,N,K", [([40, 0, 33], 130, 14336), ([300, 45], 264, 5000), ([90, 20], 37, 641),
                                        ([3, 70], 64, 1281), ([20, 31], 33, 640)])
@pytest.mark.parametrize("odd", [0, 1])
def test_long_fp32_sums_keep_their_digits(counts, N, K, odd):
    """fp32 results of long sums: off by at most 2^-23 a product within a piece of 640 of them (its additions are
    cut short), and by a rounding for each piece: in the norm, where such errors are of random size and the partial
    sums smaller, well below 2e-6 of the result."""
    g = gen(28)
    R, E = sum(counts), len(counts)
    off = offsets_of(counts)

    def result(*shape):
        return torch.full((*shape[:-1], shape[-1] + odd), 7.0, device=DEV)[..., : shape[-1]]

    x, w, dy = normal((R, K), BF16, g), normal((E, N, K), BF16, g, 0.1), normal((R, N), BF16, g)
    out = result(R, N)
    moe.moe_grouped_gemm(x, w, off, out)
    ok()
    ref, mag = ref_forward(x, w, off)
    check(out, ref, mag * (640 + 2 + K / 640) * U)
    assert (out.double() - ref).norm() <= 2e-6 * ref.norm()
    wt = normal((E, K, N), BF16, g, 0.1)  # the other way round: the sums of dx run over K
    dyk, dx = normal((R, K), BF16, g), result(R, N)
    moe.moe_grouped_gemm_grad_x(dyk, wt, off, dx)
    ok()
    ref, mag = ref_forward(dyk, wt.transpose(1, 2), off)
    check(dx, ref, mag * (640 + 2 + K / 640) * U)
    assert (dx.double() - ref).norm() <= 2e-6 * ref.norm()
    long = [K, 3, 0]
    offl = offsets_of(long)
    xl, dyl = normal((K + 3, 40), BF16, g), normal((K + 3, 72), BF16, g)
    for accumulate in (False, True):
        dw = result(3, 72, 40)
        before = dw.double() if accumulate else 0
        moe.moe_grouped_gemm_grad_w(dyl, xl, offl, dw, accumulate=accumulate)
        ok()
        ref, mag = ref_grad_w(dyl, xl, offl)
        check(dw, ref + before, (mag + 7) * (640 + 2 + K / 640) * U)
        assert (dw.double() - ref - before).norm() <= 2e-6 * (ref + before).norm()


# ------------------------------------------------------------- row operators

def ref_codes(v):
    """The codes' rule, step by step in fp32 (numpy)."""
    amax = np.abs(v).max(axis=1)
    fin = np.isfinite(v).all(axis=1)
    live = fin & (amax >= np.float32(2.0 ** -120))
    safe = np.where(live, amax, np.float32(1))
    inv = (np.float32(127) / safe).astype(np.float32)
    q = np.rint((np.where(fin[:, None], v, 0) * inv[:, None]).astype(np.float32)).clip(-127, 127)
    scale = np.where(fin, np.where(live, (safe / np.float32(127)).astype(np.float32), np.float32(0)), np.float32("nan"))
    return (q * live[:, None]).astype(np.int8), scale.astype(np.float32)


@pytest.mark.parametrize("R,K,extra", [(1, 1, 0), (3, 8, 0), (5, 17, 1), (33, 2880, 0), (7, 2047, 0), (4, 2048, 2),
                                       (9, 4096, 0), (6, 8200, 0), (3, 14336, 0), (2, 20000, 0), (300, 96, 0)])
@pytest.mark.parametrize("t", [BF16, FP16], ids=str)
def test_quant_rows_bit_for_bit(R, K, extra, t):
    g = gen(11)
    x = normal((R, K), t, g, 3.0, extra)
    if R > 2:
        x[1] = 0
        x[2] *= 2.0 ** -12
    q = torch.full((R, K + 3), 99, dtype=torch.int8, device=DEV)[:, :K] if K % 8 else pitched((R, K), torch.int8, extra)
    s = torch.empty(R, device=DEV)
    moe.moe_quant_rows_i8(x, q, s)
    ok()
    rq, rs = ref_codes(x.float().cpu().numpy())
    assert np.array_equal(s.cpu().numpy(), rs) and np.array_equal(q.cpu().numpy(), rq)


LENGTHS = [1, 2, 30, 78, 250, 256, 257, 510, 1000, 1023, 1026, 2050, 4098, 5001, 8194, 15360, 15362]


def laid_out(shape, dtype, how):
    """A buffer whose rows start on 16-byte boundaries, side by side, or 2 values apart on an odd address."""
    if how == "pitched":
        return pitched(shape, dtype)
    gap = {"side_by_side": 0, "apart": 2}[how]
    flat = torch.zeros(shape[0] * (shape[1] + gap) + 1, dtype=dtype, device=DEV)
    return (flat[:-1] if gap == 0 else flat[1:]).view(shape[0], shape[1] + gap)[:, : shape[1]]


@pytest.mark.parametrize("K", LENGTHS)
@pytest.mark.parametrize("hx,hq", [("pitched", "pitched"), ("side_by_side", "side_by_side"), ("apart", "pitched"),
                                   ("pitched", "apart")])
def test_row_operators_over_lengths_and_layouts(K, hx, hq):
    g = gen(27)
    R = 11
    x = laid_out((R, K), BF16, hx).copy_(torch.randn(R, K, generator=g, device=DEV))
    q, s = laid_out((R, K), torch.int8, hq), torch.empty(R, device=DEV)
    base = q._base if q._base is not None else q
    base.fill_(99)
    moe.moe_quant_rows_i8(x, q, s)
    ok()
    rq, rs = ref_codes(x.float().cpu().numpy())
    assert np.array_equal(s.cpu().numpy(), rs) and np.array_equal(q.cpu().numpy(), rq)
    assert int((base != 99).sum()) <= R * K  # nothing between the rows
    gu = laid_out((R, 2 * K), BF16, hx).copy_(torch.randn(R, 2 * K, generator=g, device=DEV) * 2)
    dh = laid_out((R, K), BF16, hq).copy_(torch.randn(R, K, generator=g, device=DEV))
    h, d = laid_out((R, K), BF16, hq), laid_out((R, 2 * K), BF16, hq)
    moe.moe_swiglu(gu, h)
    moe.moe_swiglu_grad(gu, dh, d)
    moe.moe_swiglu_quant_i8(gu, q, s)
    ok()
    a = gu.double().requires_grad_()
    ga, ua = a[:, :K], a[:, K:]
    ref = ga * torch.sigmoid(ga) * ua
    ref.backward(dh.double())
    ga, v = ga.detach(), ref.detach()
    n = swiglu_ulps(ga)
    check(h, v, v.abs() * n * U)
    sg = torch.sigmoid(ga)
    m = (dh.double() * ua.detach() * sg).abs() * (1 + ga.abs() * (1 - sg + n * U))
    check(d[:, :K], a.grad[:, :K], m * 2 * n * U)
    check(d[:, K:], a.grad[:, K:], a.grad[:, K:].abs() * n * U)
    rel, amax = n.max() * U, v.abs().amax(1)
    assert bool(((s.double() - amax / 127).abs() <= amax / 127 * (rel + U)).all())
    assert bool(((v / (amax / 127)[:, None] - q.double()).abs() <= 0.5 + 127 * (2 * rel + 2 * U)).all())


@pytest.mark.parametrize("K", [264, 1500])
def test_quant_rows_gather_and_odd_rows(K):
    """Rows by token, one token for several rows, dropped pairs; NaN, infinities, the smallest and largest values."""
    g = gen(12)
    x = normal((6, K), BF16, g)
    x[1, 7] = float("nan")
    x[2, 9] = -float("inf")
    x[3] = torch.finfo(BF16).max
    x[4] = 2.0 ** -121
    x[5] = 0
    x[5, 263] = -(2.0 ** -120)
    tok = torch.tensor([5, 0, 0, 2, 3, -1, 6, 4, 1, 0, 2 ** 31 - 1], dtype=torch.int32, device=DEV)
    q = torch.full((11, K), 99, dtype=torch.int8, device=DEV)
    s = torch.full((11,), 99.0, device=DEV)
    moe.moe_quant_rows_i8(x, q, s, row_token=tok)
    ok()
    v = x.float().cpu().numpy()
    rq, rs = ref_codes(v)
    for i, t in enumerate(tok.tolist()):
        if 0 <= t < 6:
            assert np.array_equal(q[i].cpu().numpy(), rq[t]) and np.array_equal(s[i].cpu().numpy(), rs[t], equal_nan=True)
        else:
            assert not bool(q[i].any()) and s[i] == 0


def swiglu_ulps(g):
    return 9 + 1.2 * g.abs()


@pytest.mark.parametrize("R,F,extra", [(1, 1, 0), (3, 8, 0), (5, 17, 1), (33, 2880, 0), (7, 2047, 0), (2, 14336, 1),
                                       (300, 96, 0)])
@pytest.mark.parametrize("t", [BF16, FP16], ids=str)
def test_swiglu_and_its_gradient(R, F, extra, t):
    g = gen(13)
    gu, dh = normal((R, 2 * F), t, g, 3.0, extra), normal((R, F), t, g, 1.0, extra)
    h, d = torch.empty(R, F, dtype=t, device=DEV), pitched((R, 2 * F), t, extra)
    moe.moe_swiglu(gu, h)
    moe.moe_swiglu_grad(gu, dh, d)
    ok()
    a = gu.double().requires_grad_()
    ga, ua = a[:, :F], a[:, F:]
    ref = ga * torch.sigmoid(ga) * ua
    ref.backward(dh.double())
    n = swiglu_ulps(ga.detach())
    check(h, ref.detach(), ref.detach().abs() * n * U)
    s = torch.sigmoid(ga.detach())
    # dg cancels where 1 + g (1 - s) is near 0: bounded by its terms
    m = (dh.double() * ua.detach() * s).abs() * (1 + ga.detach().abs() * (1 - s + n * U))
    check(d[:, :F], a.grad[:, :F], m * 2 * n * U)
    check(d[:, F:], a.grad[:, F:], a.grad[:, F:].abs() * n * U)
    d2 = gu.clone() if not extra else gu
    moe.moe_swiglu_grad(d2, dh, d2)  # in place
    ok()
    assert torch.equal(d2, d)


def test_swiglu_gradient_against_differences():
    g = gen(14)
    gu, dh = normal((4, 64), BF16, g), normal((4, 32), BF16, g)
    d = torch.empty(4, 64, dtype=BF16, device=DEV)
    moe.moe_swiglu_grad(gu, dh, d)
    ok()

    def loss(v):
        return (v[:, :32] * torch.sigmoid(v[:, :32]) * v[:, 32:] * dh.double()).sum()

    step = 1e-5
    for i, j in ((0, 0), (1, 17), (3, 31), (0, 32), (2, 50), (3, 63)):
        v = gu.double()
        e = torch.zeros_like(v)
        e[i, j] = step
        slope = ((loss(v + e) - loss(v - e)) / (2 * step)).item()
        assert abs(slope - d[i, j].item()) <= abs(slope) * half_step(BF16) + 1e-6


@pytest.mark.parametrize("R,F,extra", [(1, 1, 0), (5, 17, 1), (33, 2880, 0), (3, 4100, 0), (2, 14336, 0), (2, 16008, 0)])
@pytest.mark.parametrize("t", [BF16, FP16], ids=str)
def test_swiglu_quant(R, F, extra, t):
    g = gen(15)
    gu = normal((R, 2 * F), t, g, 2.0, extra)
    q, s = pitched((R, F), torch.int8, extra), torch.empty(R, device=DEV)
    moe.moe_swiglu_quant_i8(gu, q, s)
    ok()
    ga, ua = gu.double()[:, :F], gu.double()[:, F:]
    v = ga * torch.sigmoid(ga) * ua
    rel = swiglu_ulps(ga).max() * U
    amax = v.abs().amax(1)
    assert bool(((s.double() - amax / 127).abs() <= amax / 127 * (rel + U)).all())
    # a code lies within half a step of its value, and a little for the value's own error
    assert bool(((v / (amax / 127)[:, None] - q.double()).abs() <= 0.5 + 127 * (2 * rel + 2 * U)).all())
    assert bool((q.abs().amax(1) == 127).all())
    # expf is off by 2 units of its last place, 4 U, at most; with the sum, the quotient and the product a value by
    # 7 U; with as much again for the row's largest and two roundings a code's argument by 16 U
    assert bool(((v / (amax / 127)[:, None] - q.double()).abs() <= 0.5 + 127 * 16 * U).all())


# ------------------------------------------------------------- used together

def _layer(T, shape, seed):
    hl = mi.draw_layer(shape, T, seed)
    return {k: v.to(DEV) for k, v in hl["experts"].items()}, hl["x"].to(DEV), hl["router"].to(DEV)


def _route(desc, shape, x, router):
    T, k, E = x.shape[0], shape.top_k, shape.n_experts
    ws = torch.empty(moe.moe_workspace_size(desc), dtype=torch.uint8, device=DEV)
    idx, gw = torch.empty(T, k, dtype=torch.int32, device=DEV), torch.empty(T, k, device=DEV)
    off, tok = torch.empty(E + 1, dtype=torch.int32, device=DEV), torch.empty(T * k, dtype=torch.int32, device=DEV)
    inv, xp = torch.empty_like(tok), torch.empty(T * k, x.shape[1], dtype=BF16, device=DEV)
    moe.moe_route_topk(desc, x, router, None, idx, gw, ws)
    moe.moe_permute(desc, idx, off, tok, inv, x=x, x_perm=xp)
    return idx, gw, off, tok, inv, xp


@pytest.mark.parametrize("T", [1, 5, 70])
def test_layer_from_the_operators_matches_the_fused_layer_and_trains(T):
    """Route, permute, product, SwiGLU, product, combine: the layer's own output; then the gradients of both
    expert matrices and of the rows, against 64-bit autograd of the same chain."""
    shape = mi.TINY.replace(d_model=320, d_ff=96, n_experts=7, top_k=3)
    ex, x, router = _layer(T, shape, 3)
    desc = moe.make_desc(shape, T)
    idx, gw, off, tok, inv, xp = _route(desc, shape, x, router)
    R, D, F = T * 3, 320, 96
    w13, w2 = ex["w13"].view(7, 2 * F, D), ex["w2"].view(7, D, F)
    gu, h = torch.empty(R, 2 * F, dtype=BF16, device=DEV), torch.empty(R, F, dtype=BF16, device=DEV)
    y, out = torch.empty(R, D, dtype=BF16, device=DEV), torch.empty(T, D, dtype=BF16, device=DEV)
    moe.moe_grouped_gemm(xp, w13, off, gu)
    moe.moe_swiglu(gu, h)
    moe.moe_grouped_gemm(h, w2, off, y)
    moe.moe_combine(desc, y, inv, gw, None, out)
    ws, fused = torch.empty(moe.moe_workspace_size(desc), dtype=torch.uint8, device=DEV), torch.empty_like(out)
    moe.moe_layer_forward(desc, x, router, None, moe.make_weights(ex), None, fused, ws)
    ok()
    assert (out.float() - fused.float()).abs().max() <= 2e-2 * fused.float().abs().max()
    g = gen(16)
    dy = torch.randn(R, D, generator=g, device=DEV).to(BF16)
    dh, dgu = torch.empty_like(h), torch.empty_like(gu)
    dx, dw13, dw2 = torch.empty_like(xp), torch.empty(7, 2 * F, D, device=DEV), torch.empty(7, D, F, device=DEV)
    moe.moe_grouped_gemm_grad_w(dy, h, off, dw2)
    moe.moe_grouped_gemm_grad_x(dy, w2, off, dh)
    moe.moe_swiglu_grad(gu, dh, dgu)
    moe.moe_grouped_gemm_grad_w(dgu, xp, off, dw13)
    moe.moe_grouped_gemm_grad_x(dgu, w13, off, dx)
    ok()
    leaves = [t.double().requires_grad_() for t in (xp, w13, w2)]
    xa, a13, a2 = leaves
    e = torch.repeat_interleave(torch.arange(7, device=DEV), (off[1:] - off[:-1]).long())
    ga = torch.bmm(a13[e], xa[:, :, None])[:, :, 0]
    ha = ga[:, :F] * torch.sigmoid(ga[:, :F]) * ga[:, F:]
    ya = torch.bmm(a2[e], ha[:, :, None])[:, :, 0]
    ya.backward(dy.double())
    # bf16 roundings on the way (gu, h, dh, dgu: half a step each, 2^-8) of values of the result's own size:
    # four of them, and a factor of two for the sums they pass through
    for got, want in ((dx, xa.grad), (dw13, a13.grad), (dw2, a2.grad)):
        assert (got.double() - want).norm() <= 8 * 2.0 ** -8 * want.norm()


@pytest.mark.parametrize("T", [1, 40])
def test_int8_layer(T):
    """Tokens -> int8 rows -> product -> SwiGLU to int8 rows -> product -> combine, against 64 bits of the same codes."""
    shape = mi.TINY.replace(d_model=320, d_ff=96, n_experts=7, top_k=3)
    ex, x, router = _layer(T, shape, 4)
    desc = moe.make_desc(shape, T)
    idx, gw, off, tok, inv, xp = _route(desc, shape, x, router)
    R, D, F = T * 3, 320, 96

    def weight_codes(w):  # a channel's codes by the row rule: quantise the channels as rows
        q, s = torch.empty(w.shape, dtype=torch.int8, device=DEV), torch.empty(w.shape[:2], device=DEV)
        moe.moe_quant_rows_i8(w.flatten(0, 1), q.flatten(0, 1), s.flatten())
        return q, s

    (q13, s13), (q2, s2) = weight_codes(ex["w13"].view(7, 2 * F, D)), weight_codes(ex["w2"].view(7, D, F))
    xq, xs = torch.empty(R, D, dtype=torch.int8, device=DEV), torch.empty(R, device=DEV)
    hq, hs = torch.empty(R, F, dtype=torch.int8, device=DEV), torch.empty(R, device=DEV)
    gu, y, out = (torch.empty(n, m, dtype=BF16, device=DEV) for n, m in ((R, 2 * F), (R, D), (T, D)))
    moe.moe_quant_rows_i8(x, xq, xs, row_token=tok)
    moe.moe_grouped_gemm_i8(xq, xs, q13, s13, off, gu)
    moe.moe_swiglu_quant_i8(gu, hq, hs)
    moe.moe_grouped_gemm_i8(hq, hs, q2, s2, off, y)
    moe.moe_combine(desc, y, inv, gw, None, out)
    ok()
    e = torch.repeat_interleave(torch.arange(7, device=DEV), (off[1:] - off[:-1]).long())
    ref = ref_forward(xq, q13, off)[0] * xs.double()[:, None] * s13.double()[e]
    check(gu, ref, ref.abs() * 2.0 ** -22)
    ref = ref_forward(hq, q2, off)[0] * hs.double()[:, None] * s2.double()[e]
    check(y, ref, ref.abs() * 2.0 ** -22)
    ws, fused = torch.empty(moe.moe_workspace_size(desc), dtype=torch.uint8, device=DEV), torch.empty_like(out)
    moe.moe_layer_forward(desc, x, router, None, moe.make_weights(ex), None, fused, ws)
    ok()
    # four int8 roundings of half a step in 127 of the row's largest value (a few times the rms): some per cent
    assert (out.float() - fused.float()).norm() <= 0.05 * fused.float().norm()


def _all_calls(seed, counts=(40, 0, 3, 150, 1), N=200, K=136):
    g = gen(seed)
    R, E = sum(counts), len(counts)
    x, dy, w = normal((R, K), BF16, g), normal((R, N), BF16, g), normal((E, N, K), BF16, g, 0.1)
    off = offsets_of(counts)
    q, wq = codes((R, K), g), codes((E, N, K), g)
    sx, sw = torch.rand(R, generator=g, device=DEV), torch.rand(E, N, generator=g, device=DEV)
    outs = [torch.zeros(R, N, dtype=BF16, device=DEV), torch.zeros(R, K, dtype=BF16, device=DEV),
            torch.zeros(E, N, K, device=DEV), torch.zeros(R, N, device=DEV), torch.zeros(R, N // 2, dtype=BF16, device=DEV),
            torch.zeros(R, N, dtype=BF16, device=DEV), torch.zeros(R, N // 2, dtype=torch.int8, device=DEV),
            torch.zeros(R, device=DEV)]

    def run(stream=None):
        moe.moe_grouped_gemm(x, w, off, outs[0], stream=stream)
        moe.moe_grouped_gemm_grad_x(dy, w, off, outs[1], stream=stream)
        moe.moe_grouped_gemm_grad_w(dy, x, off, outs[2], stream=stream)
        moe.moe_grouped_gemm_i8(q, sx, wq, sw, off, outs[3], stream=stream)
        moe.moe_swiglu(outs[0], outs[4], stream=stream)
        moe.moe_swiglu_grad(outs[0], outs[4], outs[5], stream=stream)
        moe.moe_swiglu_quant_i8(outs[0], outs[6], outs[7], stream=stream)

    return run, outs


def test_same_bits_again_captured_and_on_two_streams():
    run, outs = _all_calls(17)
    run()
    ok()
    first = [t.clone() for t in outs]

    def same():
        ok()
        assert all(torch.equal(a, b) for a, b in zip(first, outs))
        for t in outs:
            t.zero_()

    same()
    run()
    same()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    run(stream=s)
    same()
    run2, outs2 = _all_calls(18)
    torch.cuda.synchronize()
    s2 = torch.cuda.Stream()
    for _ in range(5):  # two users at once
        run(stream=s)
        run2(stream=s2)
    ok()
    second = [t.clone() for t in outs2]
    same()
    run2()
    ok()
    assert all(torch.equal(a, b) for a, b in zip(second, outs2))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    torch.cuda.synchronize()
    for _ in range(3):
        for t in outs:
            t.zero_()
        graph.replay()
        ok()
        assert all(torch.equal(a, b) for a, b in zip(first, outs))


def test_a_captured_product_follows_new_offsets():
    """The groups are read on the device: one captured call serves every routing of its rows."""
    g = gen(19)
    x, w = normal((64, 80), BF16, g), normal((4, 96, 80), BF16, g, 0.1)
    off, out = offsets_of([16, 16, 16, 16]), torch.zeros(64, 96, dtype=BF16, device=DEV)
    moe.moe_grouped_gemm(x, w, off, out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_grouped_gemm(x, w, off, out)
    for counts in ([64, 0, 0, 0], [1, 2, 3, 58], [0, 0, 64, 0], [20, 20, 24, 0]):
        off.copy_(offsets_of(counts))
        graph.replay()
        ok()
        ref, mag = ref_forward(x, w, off)
        check(out, ref, mag * 82 * U)


def test_profile_names_the_kernels():
    run, _ = _all_calls(20)
    moe.moe_profile_enable(True)
    try:
        run()
        torch.cuda.synchronize()
        names = moe.moe_profile_collect()
    finally:
        moe.moe_profile_enable(False)
    assert set(names) == {"grouped_gemm", "grouped_gemm_grad_x", "grouped_gemm_grad_w", "grouped_gemm_i8", "swiglu",
                          "swiglu_grad", "swiglu_quant_i8"}


# ------------------------------------------------- long sums of 16-bit results

@pytest.mark.parametrize("t", [BF16, FP16], ids=str)
@pytest.mark.parametrize("D", [4500, 28672])
@pytest.mark.parametrize("counts,N", [([40, 0, 33], 130), ([300, 45], 264)])
def test_16_bit_results_of_long_sums_are_those_of_the_rounded_sum(t, D, counts, N):
    """A sum that is off by d of its size turns a rounding over where it lies within d of a border between two
    steps: a share of 2 d / step of the values, each by one step, so sqrt(2 d step) in the norm; step is
    finfo.eps at most, and d 2e-6, as for fp32 results."""
    g = gen(29)
    bound = (2 * 2e-6 * torch.finfo(t).eps) ** 0.5
    R, E = sum(counts), len(counts)
    off = offsets_of(counts)

    def near(got, ref):
        want = ref.to(t).double()
        assert (got.double() - want).norm() <= bound * want.norm()

    x, w, out = normal((R, D), t, g), normal((E, N, D), t, g, 0.1), torch.empty(R, N, dtype=t, device=DEV)
    moe.moe_grouped_gemm(x, w, off, out)
    ok()
    near(out, ref_forward(x, w, off)[0])
    dy, wt, dx = normal((R, D), t, g), normal((E, D, N), t, g, 0.1), torch.empty(R, N, dtype=t, device=DEV)
    moe.moe_grouped_gemm_grad_x(dy, wt, off, dx)
    ok()
    near(dx, ref_forward(dy, wt.transpose(1, 2), off)[0])
    offl = offsets_of([D - 7, 0, 100])
    dyl, xl = normal((D + 93, N), t, g, 0.1), normal((D + 93, 72), t, g)
    dw = torch.empty(3, N, 72, dtype=t, device=DEV)
    moe.moe_grouped_gemm_grad_w(dyl, xl, offl, dw)
    ok()
    near(dw, ref_grad_w(dyl, xl, offl)[0])


@pytest.mark.parametrize("ot", [FP16, BF16, FP32], ids=str)
def test_grad_w_of_a_very_long_group(ot):
    """2^21 rows of one sign: off by at most 2^-23 a product within a piece of 640, and by a rounding for each piece;
    fp32 sums of 3300 pieces stay within 4e-6 (a random walk of roundings of 2^-25 each, twice over)."""
    g = gen(30)
    R = 1 << 21
    dy, x = (torch.empty(R, 32, dtype=FP16, device=DEV) for _ in range(2))
    for m in (dy, x):
        m.copy_((torch.rand(R, 32, generator=g, device=DEV) + 1) * 2.0 ** -7)
    dw = torch.empty(1, 32, 32, dtype=ot, device=DEV)
    moe.moe_grouped_gemm_grad_w(dy, x, offsets_of([R]), dw)
    ok()
    ref, mag = ref_grad_w(dy, x, offsets_of([R]))
    check(dw, ref, mag * (640 + 2 + R / 640) * U)
    if ot == FP32:
        assert (dw.double() - ref).norm() <= 4e-6 * ref.norm()


# ------------------------------------- rows that several pairs of offsets claim

@pytest.mark.parametrize("R,away", [(10, ()), (10, (0,)), (10, (0, 2, 4)), (300, ()), (300, (0, 6))])
def test_rows_claimed_by_several_experts_get_one_of_their_products(R, away):
    """Offsets that go back and forth, a matrix of its own for each expert, some of them not resident.  Few rows: the
    lowest resident expert's product, whole, and the same again; many: element by element one of the claimants'."""
    g = gen(31)
    E, N, K = 16, 96, 72
    off = torch.tensor([0, R - 3] * (E // 2) + [0], dtype=torch.int32, device=DEV)
    slots = torch.tensor([-1 if e in away else E - 1 - e for e in range(E)], dtype=torch.int32, device=DEV)
    x, w = normal((R, K), BF16, g), normal((E, N, K), BF16, g, 0.1)
    claim = [e for e in range(0, E, 2) if e not in away]
    refs = torch.stack([x[: R - 3].double() @ w[E - 1 - e].double().t() for e in claim])
    mags = torch.stack([x[: R - 3].double().abs() @ w[E - 1 - e].double().abs().t() for e in claim])
    for _ in range(20):
        out = torch.full((R, N), 7.0, dtype=BF16, device=DEV)
        moe.moe_grouped_gemm(x, w, off, out, slot_map=slots)
        assert moe.moe_get_last_error() == 9
        got = out[: R - 3].double()
        if R == 10:
            check(out[: R - 3], refs[0], mags[0] * (K + 2) * U)
        else:
            allowed = refs.abs() * half_step(BF16) + tiny(BF16) + mags * (K + 2) * U * (1 + half_step(BF16))
            assert bool(((got - refs).abs() <= allowed).any(0).all())
        assert bool((out[R - 3:] == 7.0).all())
    q, wq = codes((R, K), g), codes((E, N, K), g)
    sx, sw = torch.rand(R, generator=g, device=DEV), torch.rand(E, N, generator=g, device=DEV)
    out = torch.full((R, N), 7.0, device=DEV)
    moe.moe_grouped_gemm_i8(q, sx, wq, sw, off, out, slot_map=slots)
    assert moe.moe_get_last_error() == 9
    refs = torch.stack([(q[: R - 3].double() @ wq[E - 1 - e].double().t()) * sx[: R - 3].double()[:, None]
                        * sw[E - 1 - e].double() for e in claim])
    near = (out[: R - 3].double() - refs).abs() <= refs.abs() * 2.0 ** -22
    assert bool((near[0] if R == 10 else near.any(0)).all())


# ------------------------------------------------- a wait that spans many tiles

def test_a_wait_goes_on_while_the_pipeline_moves():
    """grad_w's clearing warp waits for a group's ragged end, before which any number of whole tiles may come: its
    limit starts anew with each; when nothing moves any more it gives up."""
    import time

    limit, flag = 50_000_000, torch.zeros(1, dtype=torch.int32, device=DEV)
    moe.moe_get_last_error()
    for moves, complete, finished, status in ((0, True, 2, 0), (6, True, 2, 0), (0, False, 1, 6), (4, False, 1, 6)):
        t0 = time.perf_counter()
        moe.moe_diag_wait_moving(limit, moves, complete, flag)
        assert moe.moe_get_last_error() == status and flag.item() == finished
        assert time.perf_counter() - t0 >= 0.6e-9 * limit * moves


def test_grad_w_ragged_groups_behind_whole_ones():
    """Many tiles of groups that are multiples of 16 rows before, between and after those of ragged ones, on every CTA."""
    g = gen(32)
    counts = [640, 0, 1280, 16, 7, 64, 64, 128, 48, 100, 0, 640, 1]
    N, K = 520, 2100
    off, R = offsets_of(counts), sum(counts)
    dy, x = normal((R, N), BF16, g), normal((R, K), BF16, g)
    for ot in (BF16, FP32):
        dw = torch.full((len(counts), N, K), 7.0, dtype=ot, device=DEV)
        moe.moe_grouped_gemm_grad_w(dy, x, off, dw)
        ok()
        ref, mag = ref_grad_w(dy, x, off)
        check(dw, ref, mag * (640 + 2 + 2) * U)


@pytest.mark.parametrize("K", [8, 300, 5000])
def test_rows_of_no_token_at_all(K):
    """No tokens, and rows whose pairs were all dropped: zeros with scale 0, nothing is read."""
    tok = torch.tensor([-1, 0, 5], dtype=torch.int32, device=DEV)
    q, s = torch.full((3, K), 99, dtype=torch.int8, device=DEV), torch.full((3,), 99.0, device=DEV)
    moe.moe_quant_rows_i8(torch.empty(0, K, dtype=BF16, device=DEV), q, s, row_token=tok)
    ok()
    assert not bool(q.any()) and not bool(s.any())
