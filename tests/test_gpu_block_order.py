"""Order of the block-scaled calls and what feeds them, on the GPU: weights
prepared on a stream of their own, and operands written by the call right
ahead of the one that reads them."""
import numpy as np
import pytest

import workloads as wl
from workloads import device as wd

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import chunked_prefill_hybrid_tau_gb300 as hb  # noqa: E402


@pytest.mark.parametrize("as_handle", [False, True])
@pytest.mark.parametrize("fmt", ["e4m3_block", "e4m3", "bf16"])
def test_prepare_on_a_side_stream(fmt, as_handle):
    """The weights that the current stream would have prepared, with work on
    the current stream that takes and gives back memory meanwhile."""
    dims = wl.Dims(d_model=1024, n_q=16, n_kv=4, d_head=64, d_ff=2112)
    gen = wd.device_generator(5)
    raw = [wd.randn_bf16(s, gen, 0.05) for s in ((dims.qkv_cols, 1024), (1024, 1024), (2112, 1024), (2112, 1024),
                                                 (1024, 2112), (1024,), (1024,))]
    names = ("w_qkv", "w_o", "w_gu", "w_d") + (() if fmt == "bf16" else ("s_qkv", "s_o", "s_gu", "s_d"))
    ref = hb.prepare_layer_weights(*[t.clone() for t in raw], fmt=fmt)
    side = torch.cuda.Stream()
    handle = side.cuda_stream if as_handle else side
    for _ in range(5):
        churn = [torch.full((3 << 20,), 7.0, device="cuda") for _ in range(4)]
        del churn
        copies = [t.clone() for t in raw]
        side.wait_stream(torch.cuda.current_stream())  # the caller's tensors are the caller's to order
        lw = hb.prepare_layer_weights(*copies, stream=handle, fmt=fmt)
        churn = [torch.full((3 << 20,), 9.0, device="cuda") for _ in range(4)]
        del churn
        side.synchronize()
        for k in names:
            assert torch.equal(getattr(lw, k).view(torch.uint8), getattr(ref, k).view(torch.uint8)), k
        torch.cuda.synchronize()
    hb.hb_check_status()


# one shape for each kernel that hb_gemm_e4m3_block may choose: few tokens, one
# CTA's 128 x 128 tiles, a pair's 256 x 128 and 256 x 256
SHAPES = [(4, 8192, 4096), (100, 20096, 512), (256, 9728, 512), (640, 10240, 1024)]


@pytest.mark.parametrize("m,n,k", SHAPES)
@pytest.mark.parametrize("writer", ["quantize", "copy", "cat"])
def test_projection_straight_after_its_weights(m, n, k, writer):
    """B and its scales rewritten by the call right ahead, over and over."""
    gen = wd.device_generator(m + n)
    ws = [hb.hb_quantize_e4m3_block(wd.randn_bf16((n, k), gen, 0.05), block_rows=128) for _ in range(2)]
    raw = [wd.randn_bf16((n, k), gen, 0.05) for _ in range(2)]
    if writer == "quantize":
        ws = [hb.hb_quantize_e4m3_block(w, block_rows=128) for w in raw]
    a, sa = hb.hb_quantize_e4m3_block(wd.randn_bf16((m, k), gen))
    ref = []
    for q, s in ws:
        torch.cuda.synchronize()
        o = torch.empty((m, n), dtype=torch.bfloat16, device="cuda")
        hb.hb_gemm_e4m3_block(a, sa, q, s, o)
        ref.append(o)
    assert not torch.equal(*ref)
    q, s = torch.empty_like(ws[0][0]), torch.empty_like(ws[0][1])
    outs = torch.empty((24, m, n), dtype=torch.bfloat16, device="cuda")
    for i in range(24):
        j = i % 3 % 2
        if writer == "quantize":
            hb.hb_quantize_e4m3_block(raw[j], q, s, block_rows=128)
        elif writer == "copy":
            s.copy_(ws[j][1])
            q.copy_(ws[j][0])
        else:
            torch.add(ws[j][1], 0, out=s)
            torch.cat([ws[j][0][:n // 2], ws[j][0][n // 2:]], out=q)
        hb.hb_gemm_e4m3_block(a, sa, q, s, outs[i])
    hb.hb_check_status()
    for i in range(24):
        assert torch.equal(outs[i], ref[i % 3 % 2]), i


def test_layer_straight_after_its_preparation():
    """The layer called right behind the preparation of its weights, in buffers
    that held other weights before."""
    dims = wl.TINY
    gen = wd.device_generator(77)
    shapes = ((dims.qkv_cols, 256), (256, 256), (dims.d_ff, 256), (dims.d_ff, 256), (256, dims.d_ff), (256,), (256,))
    raws = [[wd.randn_bf16(s, gen, 0.05) for s in shapes] for _ in range(2)]
    T = 40
    hp = hb.hb_plan_batch([], [], [T], [0], [[]], list(range(4)), T, T)
    dp = hb.DevicePlan(hp)
    rope = wd.rope_table_device(64, dims)
    x = wd.randn_bf16((T, 256), gen)
    k, v = (torch.zeros((4, dims.n_kv, 16, dims.d_head), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ws = wd.workspace(hb.hb_layer_workspace_bytes(dims, T, 1, T))
    for fmt in ("e4m3_block", "e4m3", "bf16"):
        ref, outs = [], []
        for i in range(12):
            copies = [t.clone() for t in raws[i % 3 % 2]]
            torch.cuda.synchronize()
            lw = hb.prepare_layer_weights(*copies, fmt=fmt)
            if i < 2:
                torch.cuda.synchronize()
            out = torch.empty_like(x)
            hb.hb_layer_forward(lw, dims, dp, rope, 64, x, out, k, v, T, ws)
            (ref if i < 2 else outs).append(out)
        hb.hb_check_status()
        assert not torch.equal(*ref)
        for i, out in enumerate(outs):
            assert torch.equal(out, ref[(i + 2) % 3 % 2]), (fmt, i)


@pytest.mark.parametrize("m,n,k", [(4, 4096, 4096), (300, 6144, 1024)])
def test_row_scaled_and_bf16_projections_straight_after_their_weights(m, n, k):
    gen = wd.device_generator(m * 3 + n)
    raw = [wd.randn_bf16((n, k), gen, 0.05) for _ in range(2)]
    x = wd.randn_bf16((m, k), gen)
    a, sa = hb.hb_quantize_e4m3(x)
    ones = torch.ones(k, dtype=torch.bfloat16, device="cuda")
    q, s, w = torch.empty((n, k), dtype=torch.uint8, device="cuda"), torch.empty(n, device="cuda"), torch.empty_like(raw[0])
    ref, outs = [], []
    for i in range(20):
        o8, o16 = (torch.empty((m, n), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        hb.hb_quantize_e4m3(raw[i % 3 % 2], q, s)
        if i < 2:
            torch.cuda.synchronize()
        hb.hb_gemm_e4m3(a, sa, q, s, o8)
        hb.hb_fold_gamma(raw[i % 3 % 2], ones, w)
        if i < 2:
            torch.cuda.synchronize()
        hb.hb_gemm(x, w, o16)
        (ref if i < 2 else outs).append((o8, o16))
    hb.hb_check_status()
    for i, (o8, o16) in enumerate(outs):
        r8, r16 = ref[(i + 2) % 3 % 2]
        assert torch.equal(o8, r8) and torch.equal(o16, r16), i


def test_quantize_captured_on_a_stream_that_is_not_the_current_one():
    """Buffers of the call's own, taken while another stream captures: the
    capture is not tied to the current stream's work."""
    gen = wd.device_generator(3)
    x = wd.randn_bf16((130, 512), gen)
    ref = hb.hb_quantize_e4m3_block(x, block_rows=128)
    hb.hb_check_status()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    # relaxed: the other stream's memory comes from cudaMalloc, which a capture otherwise forbids the thread
    with torch.cuda.graph(graph, stream=side, capture_error_mode="relaxed"):
        with torch.cuda.stream(torch.cuda.Stream()):
            q, s = hb.hb_quantize_e4m3_block(x, block_rows=128, stream=side)
    q.zero_()
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(q, ref[0]) and torch.equal(s, ref[1])
