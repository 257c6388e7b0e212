"""The layer with normed q/k heads and with block-scaled E4M3 weights (GPU):
against the oracle, against its own parts, and its invariances.

Tolerances: a bf16 layer with head norms as every layer (gpu_harness).  With
E4M3 weights the two sides quantize activations they computed independently,
so a bf16 value within an ulp of a code boundary takes the neighbouring code
on one side (one step, 2^-3 relative); tests/test_gpu_fp8.py measures and
bounds that noise, and its bounds are used here.  Which of the layer's parts
is right does not hang on them: the same layer is also rebuilt from its parts
and compared bit for bit."""
import numpy as np
import pytest

import oracle.fp8 as of
import oracle.layer as ol
import workloads as wl
from workloads import device as wd
from tests.gpu_harness import GpuLayer, assert_close, assert_layer, oracle_layer_both, plan_both, rel_l2

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import chunked_prefill_hybrid_tau_gb300 as hb  # noqa: E402
from chunked_prefill_hybrid_tau_gb300 import _lib as L  # noqa: E402

FORMATS = {"bf16": L.HB_WEIGHTS_BF16, "e4m3": L.HB_WEIGHTS_E4M3, "e4m3_block": L.HB_WEIGHTS_E4M3_BLOCK}
E4M3_FLIP_ATOL = 5e-2


def gains(dims, seed):
    rng = np.random.default_rng(seed)
    return {k: wl.bf16_round((1 + 0.2 * rng.standard_normal(dims.d_head)).astype(np.float32)) for k in ("g_q", "g_k")}


def two_iterations(weights, fmt, check):
    """The tiny workload's prefix iteration, then the hybrid one."""
    w = wl.tiny_layer(seed=0)
    st, dims = w.state, w.dims
    gl = GpuLayer(weights, dims, st.k_pool, st.v_pool, 512, fmt=fmt)
    decodes, st.decodes = st.decodes, []
    hp, o = plan_both(st, 128, 128)
    check(gl, gl.forward(hp, w.x_prompt[:128], 512), o, w.x_prompt[:128], "prefix")
    for i, r in enumerate(st.prefills):
        r.pages = list(hp.pf_pages[i])
        r.done += int(hp.pf_take[i])
    st.free_pool = list(hp.free_pool)
    st.decodes = decodes
    hp, o = plan_both(st, 68, 64)
    check(gl, gl.forward(hp, w.x, 512), o, w.x, "hybrid")


def test_tiny_bf16_layer_with_head_norms():
    w = wl.tiny_layer(seed=0)
    dims = w.dims
    weights = {**w.weights[0], **gains(dims, 3)}
    p32 = [w.state.k_pool.copy(), w.state.v_pool.copy()]
    p16 = [w.state.k_pool.copy(), w.state.v_pool.copy()]

    def check(gl, got, o, x, what):
        ref, emu, h = oracle_layer_both(weights, dims, o, x, p32, p16, 512)
        assert_layer(got, ref, emu, h, what)
        assert_close(wd.to_numpy(gl.k), p16[0], what + " K")

    two_iterations(weights, "bf16", check)


@pytest.mark.parametrize("norms", [False, True])
def test_tiny_block_layer(norms):
    w = wl.tiny_layer(seed=0)
    dims = w.dims
    weights = {**w.weights[0], **(gains(dims, 4) if norms else {})}
    wq = of.prepare_weights(weights, block=True)
    cos, sin = ol.rope_tables(512, dims.d_head, dims.theta)
    pools = [w.state.k_pool.copy(), w.state.v_pool.copy()]

    def check(gl, got, o, x, what):
        ref = of.layer_forward(wq, dims, o, x, *pools, cos, sin, storage="bf16", block=True)
        assert_close(got, ref, what, atol=E4M3_FLIP_ATOL * float(np.sqrt(np.mean(ref * ref))))
        assert_close(wd.to_numpy(gl.k), pools[0], what + " K")

    two_iterations(weights, "e4m3_block", check)


def test_block_weight_preparation_bit_exact():
    """Gains folded in bf16, then block codes; gate and up each on its own."""
    w = wl.tiny_layer(seed=2).weights[0]
    F, d = w["w_g"].shape
    Fp = (F + 63) // 64 * 64
    lw = wd.layer_weights_device(w, wl.TINY, fmt="e4m3_block")
    ref = of.prepare_weights(w, block=True)
    for name in ("qkv", "o", "d"):
        assert np.array_equal(getattr(lw, "w_" + name).cpu().numpy(), ref[name][0]), name
        assert np.array_equal(getattr(lw, "s_" + name).cpu().numpy(), ref[name][1]), name
    assert np.array_equal(lw.s_gu.cpu().numpy(), np.concatenate([ref["g"][1], ref["u"][1]]))
    pad = [np.concatenate([ref[k][0], np.zeros((Fp - F, d), np.uint8)]).reshape(Fp // 64, 64, d) for k in "gu"]
    assert np.array_equal(lw.w_gu.cpu().numpy(), np.stack(pad, 1).reshape(2 * Fp, d))


@pytest.mark.parametrize("norms", [False, True])
def test_mistral_block_layer_tau512(norms):
    """The Mistral-7B-shaped layer at tau = 512: within the flip noise of the
    block-scaled oracle, and much closer to it than to the bf16 one."""
    w = wl.mistral_layer(seed=0)
    st, dims = w.state, w.dims
    weights = {**w.weights[0], **(gains(dims, 5) if norms else {})}
    hp, o = plan_both(st, 512, 512)
    gl = GpuLayer(weights, dims, st.k_pool, st.v_pool, 4096, fmt="e4m3_block")
    got = gl.forward(hp, w.x, int(hp.seq_kv_len.max()))
    cos, sin = ol.rope_tables(4096, dims.d_head, dims.theta)
    ref8 = of.layer_forward(of.prepare_weights(weights, block=True), dims, o, w.x, st.k_pool.copy(),
                            st.v_pool.copy(), cos, sin, storage="bf16", block=True)
    ref16 = ol.layer_forward(weights, dims, o, w.x, st.k_pool.copy(), st.v_pool.copy(), cos, sin)
    assert_close(got, ref8, "mistral block layer", atol=0.3 * float(np.sqrt(np.mean(ref8 ** 2))), rel_l2=0.05)
    d8, d16 = rel_l2(got, ref8), rel_l2(got, ref16)
    print(f"relL2 to the block-scaled oracle {d8:.4g}, to the bf16 one {d16:.4g}")
    assert d8 < 0.6 * d16


@pytest.mark.parametrize("fmt,norms,dims", [("e4m3_block", True, wl.TINY), ("e4m3_block", False, wl.MISTRAL),
                                            ("bf16", True, wl.TINY), ("e4m3", True, wl.TINY)])
def test_layer_equals_its_parts_bitwise(fmt, norms, dims):
    """hb_layer_forward against the same steps called one by one: where the
    parts are public they are called, the 1/rms in the scales is formed here
    as the definition has it (and compared within the order of a sum)."""
    from workloads import bf16_round
    rng = np.random.default_rng(7)
    w = wl.layer_weights(rng, dims)
    if norms:
        w.update(gains(dims, 6))
    lw = wd.layer_weights_device(w, dims, fmt=fmt)
    T, n_pages = 37, 8
    hp = hb.hb_plan_batch([], [], [T], [0], [[]], list(range(n_pages)), T, T)
    dp = hb.DevicePlan(hp)
    rope = wd.rope_table_device(64, dims)
    # rows of one value +-1: mean(x^2) = 1 whatever the order of the sum, and
    # 1/rms = rsqrt(1 + eps) for all of them
    x = wd.bf16_tensor(bf16_round(np.sign(rng.standard_normal((T, dims.d_model))).astype(np.float32)))
    k, v = (torch.zeros((n_pages, dims.n_kv, 16, dims.d_head), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    out = torch.empty_like(x)
    ws = wd.workspace(hb.hb_layer_workspace_bytes(dims, T, 1, T))
    n0 = hb.hb_kernel_launches()
    hb.hb_layer_forward(lw, dims, dp, rope, 64, x, out, k, v, T, ws)
    count = hb.hb_layer_kernel_count(dims, T, FORMATS[fmt] | (L.HB_LAYER_QK_NORM if norms else 0))
    assert hb.hb_kernel_launches() - n0 == count
    hb.hb_check_status()
    if fmt != "e4m3_block":
        # K of the layer: the plain layer's projection, normed and rotated
        plain = wd.layer_weights_device({a: b for a, b in w.items() if a not in ("g_q", "g_k")}, dims, fmt=fmt)
        k2, v2 = torch.zeros_like(k), torch.zeros_like(v)
        hb.hb_layer_forward(plain, dims, dp, rope, 64, x, torch.empty_like(x), k2, v2, T, ws)
        assert torch.equal(v, v2) and not torch.equal(k, k2)
        ident = torch.zeros((64, dims.d_head // 2, 2), device="cuda")
        ident[..., 0] = 1
        k3, v3 = torch.zeros_like(k), torch.zeros_like(v)
        # the unrotated K of the plain layer is qkv's: positions 0 rotate by nothing
        hb.hb_layer_forward(plain, dims, dp, ident, 64, x, torch.empty_like(x), k3, v3, T, ws)
        rows = k3.transpose(1, 2).reshape(-1, dims.n_kv, dims.d_head)[:, :, :]
        slots = dp.field("slot_mapping").long()
        qkv = torch.zeros((T, dims.n_q + 2 * dims.n_kv, dims.d_head), dtype=torch.bfloat16, device="cuda")
        qkv[:, dims.n_q:dims.n_q + dims.n_kv] = rows[slots]
        k4, v4 = torch.zeros_like(k), torch.zeros_like(v)
        q4 = torch.empty((T, dims.n_q, dims.d_head), dtype=torch.bfloat16, device="cuda")
        hb.hb_kv_append_norm(qkv.view(T, -1), dp.field("row_pos"), dp.field("slot_mapping"), rope, 64, dims, lw.g_q,
                             lw.g_k, q4, k4, v4)
        hb.hb_check_status()
        assert torch.equal(k4, k)
        return
    xq, sx = hb.hb_quantize_e4m3_block(x)
    r = float(np.float32(1) / np.sqrt(np.float32(1) + np.float32(dims.eps)))
    qkv = torch.empty((T, dims.qkv_cols), dtype=torch.bfloat16, device="cuda")
    hb.hb_gemm_e4m3_block(xq, sx * r, lw.w_qkv, lw.s_qkv, qkv)
    q = torch.empty((T, dims.n_q, dims.d_head), dtype=torch.bfloat16, device="cuda")
    k2, v2 = torch.zeros_like(k), torch.zeros_like(v)
    args = (qkv, dp.field("row_pos"), dp.field("slot_mapping"), rope, 64, dims)
    if norms:
        hb.hb_kv_append_norm(*args, lw.g_q, lw.g_k, q, k2, v2)
    else:
        hb.hb_kv_append(*args, q, k2, v2)
    # rsqrt is off by up to two steps: K and V agree to an ulp of bf16 where it
    # falls beside a rounding border, and almost everywhere bit for bit
    for a, b in ((k, k2), (v, v2)):
        assert float((a != b).float().mean()) < 1e-2
        assert bool(((a.float() - b.float()).abs() <= 2.0 ** -7 * b.float().abs() + 1e-30).all())
    assert torch.isfinite(out.float()).all()


@pytest.mark.parametrize("fmt", ["e4m3_block", "bf16"])
def test_chunked_equals_unchunked_bitwise(fmt):
    """A prompt prefilled in chunks, through every projection kernel, gives
    the unchunked outputs and KV bit for bit, normed heads included."""
    from tests.test_gpu_sweep import prefill_in_chunks
    dims = wl.MISTRAL
    P = 1536
    gen = wd.device_generator(47)
    lw = wd.layer_weights_random(dims, 4700, fmt=fmt)
    lw.g_q, lw.g_k = ((1 + 0.2 * torch.randn(128, generator=gen, device="cuda")).to(torch.bfloat16) for _ in range(2))
    x = wd.randn_bf16((P, dims.d_model), gen)
    rope = wd.rope_table_device(P + 1, dims)
    ref, kr, vr, _ = prefill_in_chunks(lw, dims, x, P, rope, P + 1, P // 16 + 8, seed=5)
    for c in [16, 48, 80, 512]:
        out, k, v, _ = prefill_in_chunks(lw, dims, x, c, rope, P + 1, P // 16 + 8, seed=5)
        assert torch.equal(out, ref), c
        assert torch.equal(k, kr) and torch.equal(v, vr), c
    assert torch.isfinite(ref.float()).all()


def test_stack_of_all_formats():
    """hb_layers_forward over bf16, E4M3 and block-scaled layers, with and
    without head norms, against one call per layer, out of place and in place:
    the same bits, and the launches the library's rule gives."""
    dims = wl.MISTRAL
    T, n_pages = 96, 16
    fmts = [("e4m3_block", True), ("bf16", False), ("bf16", True), ("e4m3", True), ("e4m3_block", False),
            ("e4m3_block", True), ("bf16", True)]
    gen = wd.device_generator(48)
    layers = []
    for i, (fmt, norm) in enumerate(fmts):
        lw = wd.layer_weights_random(dims, 4800 + i, fmt=fmt)
        if norm:
            lw.g_q, lw.g_k = ((1 + 0.2 * torch.randn(128, generator=gen, device="cuda")).to(torch.bfloat16)
                              for _ in range(2))
        layers.append(lw)
    hp = hb.hb_plan_batch([], [], [T], [0], [[]], list(range(n_pages)), T, T)
    dp = hb.DevicePlan(hp)
    rope = wd.rope_table_device(T + 1, dims)
    ws = wd.workspace(hb.hb_layer_workspace_bytes(dims, T, 1, T))
    x = wd.randn_bf16((T, dims.d_model), gen)
    shape = (n_pages, dims.n_kv, 16, dims.d_head)

    def pools():
        return [[torch.zeros(shape, dtype=torch.bfloat16, device="cuda") for _ in fmts] for _ in range(2)]

    one, (k1, v1), total = x.clone(), pools(), 0
    for i, lw in enumerate(layers):
        hb.hb_layer_forward(lw, dims, dp, rope, T + 1, one, one, k1[i], v1[i], T, ws)
        total += hb.hb_layer_kernel_count(dims, T, FORMATS[fmts[i][0]] | (L.HB_LAYER_QK_NORM if fmts[i][1] else 0))
    carried = sum(1 for i, (f, _) in enumerate(fmts) if i and f == "bf16" and fmts[i - 1][0] != "e4m3_block")
    for in_place in (False, True):
        x2 = x.clone()
        out = x2 if in_place else torch.empty_like(x)
        k2, v2 = pools()
        n0 = hb.hb_kernel_launches()
        hb.hb_layers_forward(layers, dims, dp, rope, T + 1, x2, out, k2, v2, T, ws)
        assert hb.hb_kernel_launches() - n0 == total - carried
        hb.hb_check_status()
        assert torch.equal(out, one)
        assert all(torch.equal(a, b) for a, b in zip(k1 + v1, k2 + v2))
    assert torch.isfinite(one.float()).all()


def test_block_layer_in_a_graph():
    """Captured and replayed with new inputs: the eager bits."""
    dims = wl.TINY
    w = wl.layer_weights(np.random.default_rng(3), dims)
    w.update(gains(dims, 8))
    lw = wd.layer_weights_device(w, dims, fmt="e4m3_block")
    T = 21
    hp = hb.hb_plan_batch([], [], [T], [0], [[]], list(range(4)), T, T)
    dp = hb.DevicePlan(hp)
    rope = wd.rope_table_device(64, dims)
    gen = wd.device_generator(9)
    k, v = (torch.zeros((4, dims.n_kv, 16, dims.d_head), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ws = wd.workspace(hb.hb_layer_workspace_bytes(dims, T, 1, T))
    x, out = wd.randn_bf16((T, dims.d_model), gen), torch.empty((T, dims.d_model), dtype=torch.bfloat16, device="cuda")

    def call():
        hb.hb_layer_forward(lw, dims, dp, rope, 64, x, out, k, v, T, ws)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    x.copy_(wd.randn_bf16((T, dims.d_model), gen))
    call()
    ref = out.clone()
    out.zero_()
    graph.replay()
    hb.hb_check_status()
    assert torch.equal(out, ref)
