"""Refusals of the expert operators, answered on the host before anything is
enqueued: no GPU needed, and no pointer is followed."""
import ctypes

import pytest
import torch

import expert_ffn_layer_route_b200 as moe

INVALID, UNSUPPORTED = 1, 2
P = 4096  # a 16-byte aligned address that nothing follows


def _desc(**kw):
    d = dict(rows=4, n_experts=2, N=32, K=48, dtype=0, out_dtype=0, n_physical=0, ld_x=0, ld_y=0, ld_w=0, stride_w=0)
    d.update(kw)
    return moe.GemmDesc(*[d[f] for f, _ in moe.GemmDesc._fields_])


def _forward(d, x=P, w=P, off=P, out=P):
    return moe.lib().moe_grouped_gemm(ctypes.byref(d), x, w, None, off, out, None)


def _grad_x(d, dy=P, w=P, off=P, dx=P):
    return moe.lib().moe_grouped_gemm_grad_x(ctypes.byref(d), dy, w, None, off, dx, None)


def _grad_w(d, dy=P, x=P, off=P, dw=P, acc=0):
    return moe.lib().moe_grouped_gemm_grad_w(ctypes.byref(d), dy, x, off, dw, acc, None)


def _int8(d, x=P, sx=P, w=P, sw=P, off=P, out=P):
    return moe.lib().moe_grouped_gemm_i8(ctypes.byref(d), x, sx, w, sw, None, off, out, None)


BAD = [
    (dict(rows=-1), INVALID), (dict(n_experts=0), INVALID), (dict(N=0), INVALID), (dict(K=0), INVALID),
    (dict(n_physical=-1), INVALID), (dict(out_dtype=3), INVALID), (dict(out_dtype=-1), INVALID),
    (dict(ld_x=47), INVALID), (dict(ld_y=31), INVALID), (dict(ld_w=47), INVALID), (dict(stride_w=31 * 48 + 47), INVALID),
    (dict(n_experts=1025), UNSUPPORTED), (dict(N=(1 << 20) + 1), UNSUPPORTED), (dict(K=(1 << 20) + 1), UNSUPPORTED),
    (dict(rows=(1 << 30) + 1), UNSUPPORTED), (dict(ld_w=1 << 31), UNSUPPORTED),
]


@pytest.mark.parametrize("kw,status", BAD, ids=[str(b[0]) for b in BAD])
def test_bad_descriptions(kw, status):
    assert _forward(_desc(**kw)) == status
    assert _grad_x(_desc(**kw)) == status
    assert _grad_w(_desc(**kw)) == status
    assert _int8(_desc(dtype=3, **kw)) == status


def test_types():
    for dtype in (2, 3, 4, -1):
        assert _forward(_desc(dtype=dtype)) == INVALID
        assert _grad_x(_desc(dtype=dtype)) == INVALID
        assert _grad_w(_desc(dtype=dtype)) == INVALID
    for dtype in (0, 1, 2):
        assert _int8(_desc(dtype=dtype)) == INVALID
    assert _int8(_desc(dtype=3, K=131072)) == UNSUPPORTED  # the int32 sum could overflow
    for out in (0, 1):
        assert _grad_w(_desc(out_dtype=out), acc=1) == INVALID  # sums are accumulated in fp32 only


def test_grad_w_rows_are_limited():
    assert _grad_w(_desc(rows=(1 << 26) + 1)) == UNSUPPORTED


def test_null_and_misaligned():
    d, q = _desc(), _desc(dtype=3)
    L = moe.lib()
    assert L.moe_grouped_gemm(None, P, P, None, P, P, None) == INVALID
    for bad in (None, P + 8):  # matrices that are read lie on 16 bytes
        assert _forward(d, x=bad) == _forward(d, w=bad) == INVALID
        assert _grad_x(d, dy=bad) == _grad_x(d, w=bad) == INVALID
        assert _grad_w(d, dy=bad) == _grad_w(d, x=bad) == INVALID
        assert _int8(q, x=bad) == _int8(q, w=bad) == INVALID
    for bad in (None, P + 1):  # results on their type
        assert _forward(d, out=bad) == _grad_x(d, dx=bad) == _grad_w(d, dw=bad) == _int8(q, out=bad) == INVALID
    assert _forward(_desc(out_dtype=2), out=P + 2) == INVALID
    assert _int8(q, sx=None) == _int8(q, sw=None) == _int8(q, sx=P + 2) == INVALID
    assert _forward(d, off=None) == _grad_x(d, off=None) == _grad_w(d, off=None) == _int8(q, off=None) == INVALID
    # row pitches of what is read: whole 16 bytes
    assert _forward(_desc(ld_x=52)) == _forward(_desc(ld_w=52)) == _forward(_desc(K=50)) == INVALID
    assert _grad_x(_desc(ld_y=36)) == _grad_x(_desc(ld_w=52)) == INVALID
    assert _grad_w(_desc(ld_y=36)) == _grad_w(_desc(ld_x=52)) == INVALID
    assert _int8(_desc(dtype=3, ld_x=56)) == _int8(_desc(dtype=3, ld_w=56)) == INVALID
    assert _forward(_desc(stride_w=32 * 48 + 4)) == INVALID


def test_no_rows_is_a_no_op():
    z = _desc(rows=0)
    assert _forward(z, None, None, None, None) == 0
    assert _grad_x(z, None, None, None, None) == 0
    assert _int8(_desc(rows=0, dtype=3), None, None, None, None, None, None) == 0
    assert _grad_w(z, None, None, None, None) == INVALID  # it has zeros to write
    L = moe.lib()
    assert L.moe_quant_rows_i8(0, 8, 0, None, 0, None, 0, None, 0, None, None) == 0
    assert L.moe_swiglu(0, 8, 0, None, 0, None, 0, None) == 0
    assert L.moe_swiglu_quant_i8(0, 8, 0, None, 0, None, 0, None, None) == 0
    assert L.moe_swiglu_grad(0, 8, 0, None, 0, None, 0, None, 0, None) == 0


def test_row_operators():
    L = moe.lib()

    def quant(rows=4, K=8, t=0, x=P, ldx=0, tok=None, n=4, q=P, ldq=0, s=P):
        return L.moe_quant_rows_i8(rows, K, t, x, ldx, tok, n, q, ldq, s, None)

    def swiglu(rows=4, F=8, t=0, gu=P, ldg=0, h=P, ldh=0):
        return L.moe_swiglu(rows, F, t, gu, ldg, h, ldh, None)

    def swiglu_q(rows=4, F=8, t=0, gu=P, ldg=0, q=P, ldq=0, s=P):
        return L.moe_swiglu_quant_i8(rows, F, t, gu, ldg, q, ldq, s, None)

    def grad(rows=4, F=8, t=0, gu=P, ldg=0, dh=P, ldh=0, d=2 * P, ldd=0):
        return L.moe_swiglu_grad(rows, F, t, gu, ldg, dh, ldh, d, ldd, None)

    for f, width in ((quant, "K"), (swiglu, "F"), (swiglu_q, "F"), (grad, "F")):
        assert f(rows=-1) == f(**{width: 0}) == f(t=2) == f(t=3) == f(t=-1) == INVALID
        assert f(**{width: (1 << 20) + 1}) == f(rows=(1 << 30) + 1) == UNSUPPORTED
        assert f(rows=1 << 30, **{width: 1 << 20}) == UNSUPPORTED
    assert quant(x=None) == quant(x=P + 1) == quant(q=None) == quant(s=None) == quant(s=P + 2) == INVALID
    assert quant(ldx=7) == quant(ldq=7) == quant(tok=P, n=-1) == quant(tok=P + 2) == INVALID
    assert swiglu(gu=None) == swiglu(gu=P + 1) == swiglu(h=None) == swiglu(ldg=15) == swiglu(ldh=7) == INVALID
    assert swiglu_q(gu=None) == swiglu_q(q=None) == swiglu_q(s=None) == swiglu_q(ldg=15) == swiglu_q(ldq=7) == INVALID
    assert grad(gu=None) == grad(dh=None) == grad(d=None) == grad(ldg=15) == grad(ldh=7) == grad(ldd=15) == INVALID
    assert grad(d=P, ldd=24) == INVALID  # in place with another pitch


# ---- the Python calls check the tensors they are given

def _t(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


def _refused(f, *a, **k):
    with pytest.raises(moe.MoeError) as e:
        f(*a, **k)
    assert e.value.status == INVALID
    return str(e.value)


def test_python_calls_check_shapes_types_and_places():
    x, w, off, out = _t(4, 16), _t(2, 8, 16), torch.zeros(3, dtype=torch.int32), _t(4, 8)
    f = moe.moe_grouped_gemm
    assert "CUDA" in _refused(f, x, w, off, out)  # host tensors
    assert "shape" in _refused(f, x, w, off, _t(4, 9))
    assert "shape" in _refused(f, _t(4, 15), w, off, out)
    assert "shape" in _refused(f, x, w, off, _t(5, 8))
    assert "types" in _refused(f, x.half(), w, off, out)
    assert "types" in _refused(f, x.float(), w.float(), off, out)
    assert "types" in _refused(f, x, w, off, out.double())
    assert "offsets" in _refused(f, x, w, off.long(), out)
    assert "offsets" in _refused(f, x, w, off[:1], out)
    assert "matrices" in _refused(f, x, w, torch.zeros(4, dtype=torch.int32), out)
    assert "slot_map" in _refused(f, x, w, torch.zeros(4, dtype=torch.int32), out, slot_map=off[:2])
    assert "contiguous" in _refused(f, _t(16, 4).t(), w, off, out)
    assert "contiguous" in _refused(f, x, _t(2, 16, 8).transpose(1, 2), off, out)
    assert "CUDA" in _refused(moe.moe_grouped_gemm_grad_x, out, w, off, x)
    assert "shape" in _refused(moe.moe_grouped_gemm_grad_x, out, w, off, _t(4, 8))
    assert "CUDA" in _refused(moe.moe_grouped_gemm_grad_w, out, x, off, w)
    assert "shape" in _refused(moe.moe_grouped_gemm_grad_w, out, _t(5, 16), off, w)
    assert "matrices" in _refused(moe.moe_grouped_gemm_grad_w, out, x, off, _t(3, 8, 16))
    xq, wq = _t(4, 16, dtype=torch.int8), _t(2, 8, 16, dtype=torch.int8)
    sx, sw = torch.zeros(4), torch.zeros(2, 8)
    g = moe.moe_grouped_gemm_i8
    assert "CUDA" in _refused(g, xq, sx, wq, sw, off, out)
    assert "types" in _refused(g, x, sx, wq, sw, off, out)
    assert "x_scale" in _refused(g, xq, sx[:3], wq, sw, off, out)
    assert "x_scale" in _refused(g, xq, sx.double(), wq, sw, off, out)
    assert "w_scale" in _refused(g, xq, sx, wq, sw[:, :7], off, out)
    q = moe.moe_quant_rows_i8
    assert "CUDA" in _refused(q, x, xq, sx)
    assert "rows" in _refused(q, _t(3, 16), xq, sx)
    assert "row_token" in _refused(q, _t(3, 16), xq, sx, row_token=off)
    assert "types" in _refused(q, x.float(), xq, sx)
    gu = _t(4, 32)
    assert "CUDA" in _refused(moe.moe_swiglu, gu, x)
    assert "types" in _refused(moe.moe_swiglu, gu, x.half())
    assert "gate_up" in _refused(moe.moe_swiglu, _t(4, 31), x)
    assert "CUDA" in _refused(moe.moe_swiglu_quant_i8, gu, xq, sx)
    assert "scale" in _refused(moe.moe_swiglu_quant_i8, gu, xq, sx[:2])
    assert "CUDA" in _refused(moe.moe_swiglu_grad, gu, x, gu)
    assert "shape" in _refused(moe.moe_swiglu_grad, gu, x, _t(4, 30))


def _rows_expanded(t):
    return t[:1].expand_as(t)


def test_expanded_tensors_are_refused():
    """A tensor expanded along its rows, or along the experts, has a pitch of 0, which the C calls read as "not
    given": every matrix argument of every call."""
    x, w, off, out = _t(4, 16), _t(2, 8, 16), torch.zeros(3, dtype=torch.int32), _t(4, 8)
    w_rows = w[:, :1].expand(2, 8, 16)
    w_experts = w[:1].expand(2, 8, 16)
    slots = torch.zeros(2, dtype=torch.int32)
    xq, wq = _t(4, 16, dtype=torch.int8), _t(2, 8, 16, dtype=torch.int8)
    sx, sw, gu = torch.zeros(4), torch.zeros(2, 8), _t(4, 32)
    e = _rows_expanded
    fwd, gx, gw, i8 = (moe.moe_grouped_gemm, moe.moe_grouped_gemm_grad_x, moe.moe_grouped_gemm_grad_w,
                       moe.moe_grouped_gemm_i8)
    for f, args in (
        (fwd, (e(x), w, off, out)), (fwd, (x, w_rows, off, out)), (fwd, (x, w_experts, off, out)),
        (fwd, (x, w, off, e(out))), (fwd, (x, w_experts, off, out, slots)),
        (gx, (e(out), w, off, x)), (gx, (out, w_rows, off, x)), (gx, (out, w_experts, off, x)), (gx, (out, w, off, e(x))),
        (gw, (e(out), x, off, w)), (gw, (out, e(x), off, w)), (gw, (out, x, off, w_rows)), (gw, (out, x, off, w_experts)),
        (i8, (e(xq), sx, wq, sw, off, out)), (i8, (xq, sx, wq[:, :1].expand(2, 8, 16), sw, off, out)),
        (i8, (xq, sx, wq[:1].expand(2, 8, 16), sw, off, out)), (i8, (xq, sx, wq, sw, off, e(out))),
        (moe.moe_quant_rows_i8, (e(x), xq, sx)), (moe.moe_quant_rows_i8, (x, e(xq), sx)),
        (moe.moe_quant_rows_i8, (e(x), xq, sx, torch.zeros(4, dtype=torch.int32))),
        (moe.moe_swiglu, (e(gu), x)), (moe.moe_swiglu, (gu, e(x))),
        (moe.moe_swiglu_quant_i8, (e(gu), xq, sx)), (moe.moe_swiglu_quant_i8, (gu, e(xq), sx)),
        (moe.moe_swiglu_grad, (e(gu), x, gu)), (moe.moe_swiglu_grad, (gu, e(x), gu)), (moe.moe_swiglu_grad, (gu, x, e(gu))),
    ):
        assert "overlap" in _refused(f, *args)
    # the gradient behind a sum over rows
    row = torch.ones(4, 8, requires_grad=True)
    row.sum(0).backward(torch.ones(8))
    assert "overlap" in _refused(gx, torch.ones(8).bfloat16().expand(4, 8), w, off, x)
    # pitches that are too small, and matrices that lie over one another
    assert "overlap" in _refused(fwd, torch.zeros(100).bfloat16().as_strided((4, 16), (8, 1)), w, off, out)
    assert "overlap" in _refused(fwd, x, torch.zeros(400).bfloat16().as_strided((2, 8, 16), (64, 16, 1)), off, out)
    # one row, one matrix, one column: their strides mean nothing
    one = _t(1, 16)
    assert "CUDA" in _refused(fwd, one.as_strided((1, 16), (0, 1)), w, off, _t(1, 8).as_strided((1, 8), (0, 1)))
    assert "CUDA" in _refused(fwd, x, w[:1].as_strided((1, 8, 16), (0, 16, 1)), off[:2], out)


def test_a_description_lives_until_c_has_read_it(monkeypatch):
    """Two threads that ask for the description of the same sizes at once: only one of the two is kept by the cache,
    and the other has to live through its own call all the same."""
    import gc
    import threading

    n = moe._native
    if n._torch is None:
        n._setup()
    both, live, calls = threading.Barrier(2), set(), []
    pitch = n._pitch

    class Desc(moe.GemmDesc):
        def __init__(self, *a):
            super().__init__(*a)
            live.add(ctypes.addressof(self))

        def __del__(self):
            live.discard(ctypes.addressof(self))

    def slow_pitch(*a):  # (inside the function that the cache holds the answers of: both threads miss)
        if a[-1] == "x":
            both.wait(60)
        return pitch(*a)

    def c_call(d, *a):
        both.wait(60)
        gc.collect()
        calls.append(d in live)
        both.wait(60)
        return 0

    class Lib:
        moe_grouped_gemm = moe_grouped_gemm_grad_x = moe_grouped_gemm_grad_w = moe_grouped_gemm_i8 = staticmethod(c_call)

    for name, value in (("GemmDesc", Desc), ("_pitch", slow_pitch), ("_LIB", Lib), ("_one_gpu", lambda *a: 0),
                        ("_raw_stream", lambda i: 0), ("_current", lambda: 0)):
        monkeypatch.setattr(n, name, value)
    x, w, off, out = _t(4, 72), _t(2, 56, 72), torch.zeros(3, dtype=torch.int32), _t(4, 56)
    q, wq = _t(4, 72, dtype=torch.int8), _t(2, 56, 72, dtype=torch.int8)
    for f, args in ((moe.moe_grouped_gemm, (x, w, off, out)), (moe.moe_grouped_gemm_grad_x, (out, w, off, x)),
                    (moe.moe_grouped_gemm_grad_w, (out, x, off, w)),
                    (moe.moe_grouped_gemm_i8, (q, torch.zeros(4), wq, torch.zeros(2, 56), off, out))):
        n._gemm_desc.cache_clear()
        calls.clear()
        threads = [threading.Thread(target=f, args=args) for _ in range(2)]
        for t in threads:
            t.start()
        for t in threads:
            t.join(120)
        assert calls == [True, True], f.__name__
    n._gemm_desc.cache_clear()


def test_fewer_matrices_than_experts_need_a_slot_map():
    """Without one expert e's matrix is matrix e, which has to exist."""
    L, off = moe.lib(), P
    for d in (_desc(n_experts=4, n_physical=3), _desc(n_experts=4, n_physical=1)):
        assert _forward(d) == _grad_x(d) == INVALID
    assert _int8(_desc(dtype=3, n_experts=4, n_physical=3)) == INVALID
    assert _forward(_desc(rows=0, n_experts=4, n_physical=3)) == INVALID
    # (with one: nothing to do, and no complaint)
    assert L.moe_grouped_gemm(ctypes.byref(_desc(rows=0, n_experts=4, n_physical=3)), P, P, P, off, P, None) == 0


def test_the_end_of_a_row_is_read_no_further(tmp_path):
    """The few-row kernel's reads of a row's last bytes, as the host sees them: inside the row, on their alignment,
    every byte once, zeros behind."""
    import os
    import subprocess

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src = tmp_path / "tail.cpp"
    src.write_text(r"""
#include "%s/expert_ffn_layer_route_b200/csrc/row_tail.cuh"
#include <cstring>
#include <cstdio>
alignas(16) static uint8_t buf[32];
static int n, seen[32], bad;
struct Load {
  template <typename T> T get(const uint8_t* p) const {
    const int at = (int)(p - buf);
    if (at %% (int)sizeof(T) || at < 0 || at + (int)sizeof(T) > n) ++bad;
    for (unsigned i = 0; i < sizeof(T); ++i) ++seen[at + i];
    T v;
    std::memcpy(&v, p, sizeof(T));
    return v;
  }
  uint32_t u32(const uint8_t* p, bool on) const { return on ? get<uint32_t>(p) : 0; }
  uint32_t u16(const uint8_t* p, bool on) const { return on ? get<uint16_t>(p) : 0; }
  uint32_t u8(const uint8_t* p, bool on) const { return on ? get<uint8_t>(p) : 0; }
};
int main() {
  for (int i = 0; i < 32; ++i) buf[i] = (uint8_t)(200 + i);
  for (n = 0; n <= 16; ++n) {
    std::memset(seen, 0, sizeof(seen));
    uint8_t got[16];
    for (int i = 0; i < 4; ++i) {
      const uint32_t w = moe::tail_word(buf + 4 * i, n - 4 * i, Load());
      std::memcpy(got + 4 * i, &w, 4);
    }
    for (int i = 0; i < 16; ++i)
      if (got[i] != (i < n ? buf[i] : 0) || seen[i] != (i < n)) ++bad;
  }
  std::printf("%%d\n", bad);
}
""" % root)
    exe = str(tmp_path / "tail")
    subprocess.run(["g++", "-O1", "-std=c++17", "-Wall", "-Werror", str(src), "-o", exe], check=True)
    assert subprocess.run([exe], capture_output=True, text=True, check=True).stdout == "0\n"
    # the kernel reads the last row of a buffer that way
    assert "tail_word" in open(os.path.join(root, "expert_ffn_layer_route_b200", "csrc", "grouped_gemv.cu")).read()
