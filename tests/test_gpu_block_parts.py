"""The layers with block-scaled weights and with normed heads rebuilt from
their public parts, output and all, bit for bit, and the quantization that
carries a row's 1/rms against its definition in 64 bits (GPU).

The one step without a public call is that quantization: its codes are
hb_quantize_e4m3_block's, its scales those times 1/rms.  The sum of squares
behind 1/rms is formed here in the order that the kernel states (a thread has
every 256th 16-byte piece of the row; then the lanes of a warp, halving; then
the eight warps), each step rounded to fp32 from an exact 64-bit value, so
that equality can be asked for.
"""
import numpy as np
import pytest

import oracle.fp8 as of
import workloads as wl
from workloads import device as wd

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import chunked_prefill_hybrid_tau_gb300 as hb  # noqa: E402
from chunked_prefill_hybrid_tau_gb300 import _lib as L  # noqa: E402

THREADS = 256


def inv_rms(x, eps):
    """fp32 1/rms of the rows of x (bf16 values, float32 array), in the kernel's order."""
    rows, d = x.shape
    nv = -(-d // (8 * THREADS))
    full = np.zeros((rows, nv * THREADS * 8), np.float64)
    full[:, :d] = x
    full = full.reshape(rows, nv, THREADS, 8)
    ss = np.zeros((rows, THREADS), np.float32)
    for k in range(nv):
        for j in range(8):
            v = full[:, k, :, j]
            ss = (ss.astype(np.float64) + v * v).astype(np.float32)
    ss = ss.reshape(rows, 8, 32)
    for o in (16, 8, 4, 2, 1):
        ss = ss + ss[:, :, np.arange(32) ^ o]
    total = ss[:, 0, 0]
    for w in range(1, 8):
        total = total + ss[:, w, 0]
    assert total.dtype == np.float32
    mean = (total.astype(np.float64) * np.float64(np.float32(1) / np.float32(d)) +
            np.float64(np.float32(eps))).astype(np.float32)
    return torch.rsqrt(torch.from_numpy(mean).cuda())


def norm_quantize(x, eps):
    q, s = hb.hb_quantize_e4m3_block(x)
    return q, s * inv_rms(wd.to_numpy(x), eps)[:, None]


def setup(dims, T, spare=4):
    n_pages = -(-T // 16) + spare
    hp = hb.hb_plan_batch([], [], [T], [0], [[]], list(range(n_pages))[::-1], T, T)
    pools = [torch.zeros((n_pages, dims.n_kv, 16, dims.d_head), dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    ws = wd.workspace(hb.hb_layer_workspace_bytes(dims, T, 1, T))
    aws = wd.workspace(hb.hb_attention_workspace_bytes(dims, T, 1, T))
    return hb.DevicePlan(hp), wd.rope_table_device(T + 3, dims), pools, ws, aws


def bf16(*shape):
    return torch.empty(shape, dtype=torch.bfloat16, device="cuda")


# d_model up to 2048, 4096, 8192 and 16384: the four sizes of the norm
# quantization's kernel, with rows that fill its last pieces and rows that do
# not, and a last block of 64 columns
DIMS = [
    wl.TINY,
    wl.Dims(d_model=1984, n_q=3, n_kv=1, d_head=64, d_ff=208),
    wl.MISTRAL,
    wl.Dims(d_model=4160, n_q=4, n_kv=2, d_head=64, d_ff=304),
    wl.Dims(d_model=7168, n_q=8, n_kv=2, d_head=128, d_ff=1040),
    wl.Dims(d_model=8256, n_q=2, n_kv=2, d_head=64, d_ff=160),
    wl.Dims(d_model=16384, n_q=4, n_kv=1, d_head=128, d_ff=320),
]


@pytest.mark.parametrize("norms", [False, True])
@pytest.mark.parametrize("T", [1, 37, 150, 300])
@pytest.mark.parametrize("dims", DIMS, ids=lambda d: str(d.d_model))
def test_block_layer_rebuilt_bitwise(dims, T, norms):
    gen = wd.device_generator(dims.d_model + T)
    lw = wd.layer_weights_random(dims, dims.d_model, fmt="e4m3_block")
    if norms:
        lw.g_q, lw.g_k = ((1 + 0.2 * torch.randn(dims.d_head, generator=gen, device="cuda")).to(torch.bfloat16)
                          for _ in range(2))
    dp, rope, (k, v, k2, v2), ws, aws = setup(dims, T)
    x = wd.randn_bf16((T, dims.d_model), gen)
    out = torch.empty_like(x)
    hb.hb_layer_forward(lw, dims, dp, rope, T + 3, x, out, k, v, T, ws)
    hb.hb_check_status()

    hd, fp = dims.n_q * dims.d_head, -(-dims.d_ff // 64) * 64
    xq, sx = norm_quantize(x, dims.eps)
    qkv, q, o = bf16(T, dims.qkv_cols), bf16(T, dims.n_q, dims.d_head), bf16(T, hd)
    hb.hb_gemm_e4m3_block(xq, sx, lw.w_qkv, lw.s_qkv, qkv)
    args = (qkv, dp.field("row_pos"), dp.field("slot_mapping"), rope, T + 3, dims)
    if norms:
        hb.hb_kv_append_norm(*args, lw.g_q, lw.g_k, q, k2, v2)
    else:
        hb.hb_kv_append(*args, q, k2, v2)
    assert torch.equal(k, k2) and torch.equal(v, v2)
    hb.hb_attention(q, k2, v2, dp, dims, T, o, aws)
    h = torch.empty_like(x)
    hb.hb_gemm_e4m3_block(*hb.hb_quantize_e4m3_block(o), lw.w_o, lw.s_o, h, x, L.HB_EPI_RESIDUAL)
    a = bf16(T, fp)
    hb.hb_gemm_e4m3_block(*norm_quantize(h, dims.eps), lw.w_gu, lw.s_gu, a, epilogue=L.HB_EPI_SWIGLU)
    aq, sa = hb.hb_quantize_e4m3_block(a)
    again = torch.empty_like(x)
    hb.hb_gemm_e4m3_block(aq[:, :dims.d_ff].contiguous(), sa, lw.w_d, lw.s_d, again, h, L.HB_EPI_RESIDUAL)
    hb.hb_check_status()
    assert torch.equal(out, again)
    assert torch.isfinite(out.float()).all() and not torch.equal(out, h)


@pytest.mark.parametrize("dims", DIMS, ids=lambda d: str(d.d_model))
def test_norm_quantization_against_its_definition(dims):
    """V rows that pick one column of x each: V = code * scale / rms, seen in
    the cache.  In fp32 the sum of squares takes at most 8 NV + 5 + 8 <= 77
    adds (half a step each, halved by the root), the mean's fma, rsqrt (2
    steps), the scale, its product with 1/rms, the product with the weight's
    scale and the fma of the block 8 half steps more: under 47 * 2^-24 of the
    value, then bf16's half step."""
    T, n = 24, dims.n_kv * dims.d_head
    rng = np.random.default_rng(dims.d_model)
    cols = rng.permutation(dims.d_model)[:n]
    cols[:4] = [dims.d_model - 1, 0, min(2047, dims.d_model - 2), dims.d_model // 2]
    w = wl.layer_weights(rng, dims)
    w["w_qkv"][:] = 0.0
    w["w_qkv"][dims.qkv_cols - n + np.arange(n), cols] = 1.0
    lw = wd.layer_weights_device(w, dims, fmt="e4m3_block")
    blocks = -(-dims.d_model // 128)
    x = rng.standard_normal((T, dims.d_model)) * np.exp2(rng.uniform(-12, 12, (T, 1)))
    x *= np.repeat(np.exp2(rng.uniform(-6, 6, (T, blocks))), 128, 1)[:, :dims.d_model]
    x = wl.bf16_round(x.astype(np.float32))
    x[3] = 0.0
    x[4] *= np.float32(2.0 ** -40)          # far below the epsilon
    x[5, :128] = 0.0
    dp, rope, (k, v, _, _), ws, _ = setup(dims, T)
    out = bf16(T, dims.d_model)
    hb.hb_layer_forward(lw, dims, dp, rope, T + 3, wd.bf16_tensor(x), out, k, v, T, ws)
    hb.hb_check_status()
    slots = dp.field("slot_mapping").cpu().numpy()
    got = wd.to_numpy(v)[slots // 16, :, slots % 16].reshape(T, n).astype(np.float64)
    q, s = of.quantize_blocks(x, 1)
    r = 1.0 / np.sqrt(np.mean(np.square(x.astype(np.float64)), -1) + np.float64(np.float32(dims.eps)))
    ws448 = np.float64(np.float32(1) / np.float32(448)) * 448.0   # the picking weight as its block stores it
    ref = (of.dequantize_blocks(q, s, 1) * r[:, None])[:, cols] * ws448
    bound = 47 * 2.0 ** -24 * np.abs(ref)
    bound = bound + 2.0 ** -8 * (np.abs(ref) + bound) + 2.0 ** -133
    assert np.all(np.abs(got - ref) <= bound)
    assert not got[3].any() and got[0].any()


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_normed_queries_of_the_other_formats(fmt):
    """q of a layer with head norms, seen in its output: projections that pick
    columns of rows of +-1 make q, k and v +-1 exactly, W_o is the identity and
    gate and up are zero, so the output is x + attention(normed, rotated q, k;
    v), with o quantized per row for E4M3."""
    dims, T = wl.TINY, 45
    rng = np.random.default_rng(3)
    w = wl.layer_weights(rng, dims)
    w["w_qkv"][:] = 0.0
    w["w_qkv"][np.arange(dims.qkv_cols), rng.permutation(np.resize(np.arange(dims.d_model), dims.qkv_cols))] = 1.0
    w["w_o"] = np.eye(dims.d_model, dtype=np.float32)
    w["w_g"], w["w_u"] = np.zeros_like(w["w_g"]), np.zeros_like(w["w_u"])
    w.update({n: wl.bf16_round((1 + 0.3 * rng.standard_normal(64)).astype(np.float32)) for n in ("g_q", "g_k")})
    lw = wd.layer_weights_device(w, dims, fmt=fmt)
    signs = np.sign(rng.standard_normal((T, dims.d_model))).astype(np.float32)
    x = wd.bf16_tensor(signs)
    dp, rope, (k, v, k2, v2), ws, aws = setup(dims, T)
    out = torch.empty_like(x)
    hb.hb_layer_forward(lw, dims, dp, rope, T + 3, x, out, k, v, T, ws)
    hb.hb_check_status()
    qkv = wd.bf16_tensor(signs @ w["w_qkv"].T)
    q, o = bf16(T, dims.n_q, dims.d_head), bf16(T, dims.d_model)
    hb.hb_kv_append_norm(qkv, dp.field("row_pos"), dp.field("slot_mapping"), rope, T + 3, dims, lw.g_q, lw.g_k, q, k2,
                         v2)
    assert torch.equal(k, k2) and torch.equal(v, v2)
    hb.hb_attention(q, k2, v2, dp, dims, T, o, aws)
    if fmt == "bf16":
        ref = (x.float() + o.float()).to(torch.bfloat16)
    else:
        ref = torch.empty_like(x)
        hb.hb_gemm_e4m3(*hb.hb_quantize_e4m3(o), lw.w_o, lw.s_o, ref, x, L.HB_EPI_RESIDUAL)
    hb.hb_check_status()
    assert torch.equal(out, ref)
    # the attention does see the queries: those of the next head give another output
    o2 = torch.empty_like(o)
    hb.hb_attention(q.roll(1, 1).contiguous(), k2, v2, dp, dims, T, o2, aws)
    assert not torch.equal(o, o2)
