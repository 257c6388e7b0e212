"""Pins of the block-scaled FP8 and head-norm oracle functions, and the
refusals of the calls beside them (no GPU)."""
import ctypes as C
from fractions import Fraction

import numpy as np
import pytest

import oracle.fp8 as of
import oracle.layer as ol
import oracle.plan as op
import workloads as wl
from chunked_prefill_hybrid_tau_gb300 import _lib as L
from chunked_prefill_hybrid_tau_gb300 import binding as B


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("rows,cols", [(1, 16), (3, 128), (5, 144), (130, 300), (257, 128)])
def test_quantize_blocks_group_by_group(rows, cols, block_rows):
    """Each group alone, by the rule: its maximum lands on 448, its scale is
    amax / 448, and the codes are torch's conversion of x * (448 / amax)."""
    torch = pytest.importorskip("torch")
    rng = np.random.default_rng(rows * 7 + cols)
    x = wl.bf16_round((rng.standard_normal((rows, cols)) * np.exp2(rng.integers(-30, 30, (rows, 1)))).astype(np.float32))
    q, s = of.quantize_blocks(x, block_rows)
    assert q.shape == x.shape and s.shape == (-(-rows // block_rows), -(-cols // 128))
    for i in range(s.shape[0]):
        for j in range(s.shape[1]):
            at = np.s_[i * block_rows:(i + 1) * block_rows, j * 128:(j + 1) * 128]
            g = x[at]
            amax = np.float32(np.abs(g).max())
            assert s[i, j] == amax / np.float32(448)
            y = torch.from_numpy(g * (np.float32(448) / amax)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
            assert np.array_equal(q[at], y) and np.abs(of.e4m3_decode(q[at])).max() == 448


def test_quantize_blocks_zero_and_tiny_groups():
    x = np.zeros((2, 384), np.float32)
    x[0, 130], x[0, 131] = 2.0 ** -120, -2.0 ** -121
    x[1, 5] = -1.0
    q, s = of.quantize_blocks(x, 1)
    assert s[0, 0] == 0 and s[0, 2] == 0 and not q[0, :128].any() and not q[0, 256:].any()
    assert s[0, 1] == np.float32(2.0 ** -112) / np.float32(448)      # the floor, finite
    d = of.dequantize_blocks(q, s, 1)
    assert abs(d[0, 130] - x[0, 130]) <= 2.0 ** -4 * abs(x[0, 130])
    assert d[1, 5] == pytest.approx(-1.0, rel=2.0 ** -23)
    # a power-of-two factor moves the scales alone
    y = wl.bf16_round(np.random.default_rng(1).standard_normal((3, 256)).astype(np.float32))
    (qa, sa), (qb, sb) = of.quantize_blocks(y, 1), of.quantize_blocks(y * np.float32(2.0 ** 9), 1)
    assert np.array_equal(qa, qb) and np.array_equal(sa * np.float32(2.0 ** 9), sb)


def test_gemm_blocks_equals_exact_sum():
    rng = np.random.default_rng(5)
    m, n, k = 3, 130, 272
    qa, sa = of.quantize_blocks(wl.bf16_round(rng.standard_normal((m, k)).astype(np.float32)), 1)
    qb, sb = of.quantize_blocks(wl.bf16_round(rng.standard_normal((n, k)).astype(np.float32)), 128)
    got = of.gemm_blocks(qa, sa, qb, sb)
    va, vb = of.e4m3_decode(qa), of.e4m3_decode(qb)
    for i, j in [(0, 0), (1, 127), (2, 128), (0, 129)]:
        exact = Fraction(0)
        for kk in range(k):
            exact += (Fraction(float(sa[i, kk // 128])) * Fraction(float(sb[j // 128, kk // 128])) *
                      Fraction(float(va[i, kk])) * Fraction(float(vb[j, kk])))
        size = sum(abs(float(va[i, kk] * vb[j, kk]) * float(sa[i, kk // 128]) * float(sb[j // 128, kk // 128]))
                   for kk in range(k))
        assert abs(got[i, j] - float(exact)) <= (k + 4) * 2.0 ** -53 * size


def test_head_norm_closed_forms():
    x = np.array([[[3.0, 4.0, 0.0, 0.0], [0.0, 0.0, 0.0, 0.0]]])
    g = np.array([1.0, 2.0, 5.0, -1.0])
    y = ol.head_norm(x, g, 0.25, np.float64)
    r = 1 / np.sqrt(25 / 4 + 0.25)
    assert np.allclose(y[0, 0], [3 * r, 8 * r, 0, 0], rtol=1e-15) and not y[0, 1].any()
    z = np.random.default_rng(0).standard_normal((5, 3, 64))
    n = ol.head_norm(z, np.ones(64), 0.0, np.float64)
    assert np.allclose((n * n).mean(-1), 1, rtol=1e-13)
    assert np.allclose(ol.head_norm(z * 37.0, np.ones(64), 0.0, np.float64), n, rtol=1e-13)


def qk_norm_layer(seed=0):
    w = wl.tiny_layer(seed=seed)
    rng = np.random.default_rng(seed + 100)
    gains = {k: wl.bf16_round((1 + 0.2 * rng.standard_normal(w.dims.d_head)).astype(np.float32)) for k in ("g_q", "g_k")}
    return w, {**w.weights[0], **gains}


def run(fn, w, weights, plan, **kw):
    cos, sin = ol.rope_tables(512, w.dims.d_head, w.dims.theta)
    return fn(weights, w.dims, plan, w.x, w.state.k_pool.copy(), w.state.v_pool.copy(), cos, sin, **kw)


def tiny_plan(w):
    st = w.state
    return op.plan_batch([r.done for r in st.decodes], [r.pages for r in st.decodes],
                         [r.prompt_len for r in st.prefills], [0], [[]], st.free_pool, 68, 64, 16, max_pages=32)


def test_layer_with_head_norms():
    """Normed heads ignore the size of the q and k projections and change the
    layer; the block-scaled layer is within E4M3's error of the bf16 one."""
    w, weights = qk_norm_layer()
    plan = tiny_plan(w)
    out = run(ol.layer_forward, w, weights, plan)
    plain = run(ol.layer_forward, w, w.weights[0], plan)
    assert np.linalg.norm(out - plain) > 1e-3 * np.linalg.norm(plain)
    dims = w.dims
    bigger = {**weights, "w_qkv": weights["w_qkv"].copy()}
    bigger["w_qkv"][:(dims.n_q + dims.n_kv) * dims.d_head] *= 64
    # epsilon is 1e-6 beside mean squares of order 0.1
    assert np.allclose(run(ol.layer_forward, w, bigger, plan), out, rtol=0, atol=1e-4)
    blocked = run(of.layer_forward, w, of.prepare_weights(weights, block=True), plan, block=True)
    rel = np.linalg.norm(blocked - out) / np.linalg.norm(out)
    assert 1e-3 < rel < 0.08


def test_planted_block_mistakes_are_caught():
    rng = np.random.default_rng(9)
    qa, sa = of.quantize_blocks(wl.bf16_round(rng.standard_normal((4, 256)).astype(np.float32) *
                                              np.repeat([[1.0, 30.0]], 128, 1).reshape(1, 256).astype(np.float32)), 1)
    qb, sb = of.quantize_blocks(wl.bf16_round(rng.standard_normal((200, 256)).astype(np.float32)), 128)
    ref = of.gemm_blocks(qa, sa, qb, sb)

    def off(c):
        return np.linalg.norm(c - ref) / np.linalg.norm(ref)

    assert off(of.gemm_blocks(qa, sa[:, ::-1], qb, sb)) > 0.1          # scales of the other K block
    assert off(of.gemm(qa, sa[:, 0], qb, np.repeat(sb[:, 0], 128)[:200])) > 0.1  # one scale a row
    assert off(of.gemm_blocks(qa, sa, qb, sb[::-1])) > 1e-3            # scales of the other row block


# ---------------------------------------------------------------- refusals
P16 = C.c_void_p(4096)  # an aligned address, never used


def refused(lib, st, text):
    assert st == L.HB_ERR_INVALID_ARG
    assert text in lib.hb_last_error().decode(), lib.hb_last_error()


def test_quantize_block_refusals(lib):
    f = lib.hb_quantize_e4m3_block
    refused(lib, f(None, P16, P16, 4, 128, 1, None), "null")
    refused(lib, f(P16, P16, None, 4, 128, 1, None), "null")
    refused(lib, f(P16, P16, P16, -1, 128, 1, None), "rows >= 0")
    refused(lib, f(P16, P16, P16, 4, 120, 1, None), "cols % 16")
    refused(lib, f(P16, P16, P16, 4, 0, 1, None), "cols % 16")
    refused(lib, f(P16, P16, P16, 4, 128, 64, None), "block_rows")
    refused(lib, f(P16, P16, P16, 4, 128, 0, None), "block_rows")
    refused(lib, f(P16, P16, P16, 2 ** 31 - 1, 128, 128, None), "at most")
    refused(lib, f(P16, P16, P16, 1, 2 ** 24 + 16, 1, None), "at most")
    refused(lib, f(C.c_void_p(4104), P16, P16, 4, 128, 1, None), "alignment")
    refused(lib, f(P16, P16, C.c_void_p(4098), 4, 128, 1, None), "alignment")
    n = lib.hb_kernel_launches()
    assert f(None, None, None, 0, 128, 1, None) == L.HB_OK and lib.hb_kernel_launches() == n  # nothing to do


def test_gemm_block_refusals(lib):
    def f(a=P16, sa=P16, b=P16, sb=P16, c=P16, r=None, m=4, n=128, k=128, epi=0):
        return lib.hb_gemm_e4m3_block(a, sa, b, sb, c, r, m, n, k, epi, None)

    for missing in ("a", "sa", "b", "sb", "c"):
        refused(lib, f(**{missing: None}), "null")
    refused(lib, f(m=0), "bad shape")
    refused(lib, f(k=24), "K % 16")
    for size in ("m", "n", "k"):
        refused(lib, f(**{size: 2 ** 31 - 128}), "2^30")
    refused(lib, f(n=100), "N % 8")
    refused(lib, f(epi=4), "epilogue")
    refused(lib, f(epi=-1), "epilogue")
    refused(lib, f(epi=L.HB_EPI_SWIGLU, n=192), "SWIGLU")
    refused(lib, f(epi=L.HB_EPI_RESIDUAL), "RESIDUAL")
    refused(lib, f(epi=L.HB_EPI_RESIDUAL, r=C.c_void_p(4104)), "aligned")
    refused(lib, f(a=C.c_void_p(4097)), "aligned")
    refused(lib, f(sb=C.c_void_p(4098)), "4-byte")


def test_kv_append_norm_refusals(lib):
    ds = B.dims_struct(wl.TINY)

    def f(T=3, max_pos=64, pages=4, dims=ds, g_q=P16, g_k=P16, q=P16):
        return lib.hb_kv_append_norm(P16, T, P16, P16, P16, max_pos, C.byref(dims), g_q, g_k, q, P16, P16, pages, None)

    refused(lib, f(T=-1), "sizes")
    refused(lib, f(max_pos=0), "sizes")
    refused(lib, f(g_q=None), "null")
    refused(lib, f(g_k=None), "null")
    refused(lib, f(q=C.c_void_p(4104)), "alignment")
    refused(lib, f(g_k=C.c_void_p(4104)), "alignment")
    refused(lib, f(dims=L.hb_layer_dims(256, 4, 3, 64, 688, 16, 1e-6, 1e4)), "n_q")
    refused(lib, f(dims=L.hb_layer_dims(256, 4, 2, 96, 688, 16, 1e-6, 1e4)), "d_head")
    assert lib.hb_kv_append_norm(None, 0, None, None, None, 64, C.byref(ds), None, None, None, None, None, 4,
                                 None) == L.HB_OK  # nothing to do


def test_layer_weight_refusals_and_counts(lib):
    ds = B.dims_struct(wl.TINY)
    plan = L.hb_device_plan(0, 0, 1, None, None, None, None, None, 0, 0, 0)

    def f(fmt, scales=P16, g_q=None, g_k=None, dims=ds):
        w = L.hb_layer_weights(P16, P16, P16, P16, scales, scales, scales, scales, fmt, g_q, g_k)
        return lib.hb_layer_forward(C.byref(w), C.byref(dims), C.byref(plan), P16, 64, P16, P16, P16, P16, 8, 64,
                                    None, 0, None, None)

    block = L.HB_WEIGHTS_E4M3_BLOCK
    assert f(block) == L.HB_OK and f(block, g_q=P16, g_k=P16) == L.HB_OK and f(0, g_q=P16, g_k=P16) == L.HB_OK
    refused(lib, f(block, scales=None), "scales")
    refused(lib, f(3), "unknown format")
    refused(lib, f(0, g_q=P16), "together")
    refused(lib, f(block, g_k=P16), "together")
    refused(lib, f(0, g_q=C.c_void_p(4104), g_k=P16), "aligned")
    refused(lib, f(block, dims=L.hb_layer_dims(256, 4, 2, 64, 680, 16, 1e-6, 1e4)), "d_ff")
    refused(lib, f(block, dims=L.hb_layer_dims(16448, 4, 2, 64, 688, 16, 1e-6, 1e4)), "16384")
    n = C.c_int32()
    for fmt, want in ((0, 8), (1, 10), (block, 11), (L.HB_LAYER_QK_NORM, 8), (1 | L.HB_LAYER_QK_NORM, 11),
                      (block | L.HB_LAYER_QK_NORM, 11)):
        assert lib.hb_layer_kernel_count(C.byref(ds), 68, fmt, C.byref(n)) == L.HB_OK and n.value == want, fmt
    refused(lib, lib.hb_layer_kernel_count(C.byref(ds), 68, 3, C.byref(n)), "unknown format")


def test_binding_refuses_operands_that_do_not_fit():
    """A tensor too small, of another element size, strided or on the host is
    refused before any device work."""
    torch = pytest.importorskip("torch")
    x = torch.zeros((4, 128), dtype=torch.bfloat16)
    with pytest.raises(B.HBError, match="contiguous device tensor"):
        B.hb_quantize_e4m3_block(x, torch.zeros((4, 128), dtype=torch.uint8), torch.zeros((4, 1)))
    a, s = torch.zeros((4, 128), dtype=torch.uint8), torch.zeros((4, 1))
    with pytest.raises(B.HBError, match="A must be"):
        B.hb_gemm_e4m3_block(a, s, a, s, torch.zeros((4, 4), dtype=torch.bfloat16))
