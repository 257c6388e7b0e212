"""hb_kv_append_norm, hb_quantize_e4m3_block and hb_gemm_e4m3_block against
their definitions in 64 bits (GPU).

Quantization is decided by fp32 arithmetic on both sides and compared bit for
bit.  The bounds of the others follow from the arithmetic:

gemm   a code product has 8 significant bits and is exact in fp32.  A block's
       128 products are summed in fp32 on the tensor cores; with every add
       allowed a whole step 2^-23 (truncation) the block's sum is off by at
       most 127 * 2^-23 of the sum of its products' magnitudes.  The product
       of the two scales and the fma that adds block b are each off by half a
       step, 2^-24, and the running sum of B blocks goes through B such adds:
       |err| <= (127 * 2^-23 + (B + 1) * 2^-24) * S,
       S = sum_b sa sb sum_k |a| |b|.
       bf16 outputs add 2^-8 |value|; the residual's fp32 add 2^-24 |value|.
append inv_rms carries the fp32 sum of d squares (half a step each), the
       division, the epsilon add and rsqrt (2 steps): under (d + 8) * 2^-24,
       halved by the root; the two products of the norm, the rotation's
       product and its add 4 half steps more: |err| <= (d / 2 + 16) * 2^-24 *
       (|y_i| + |y_j|) + 2^-8 |value|, y the normed pair.
"""
import numpy as np
import pytest

import oracle.fp8 as of
import oracle.layer as ol
import workloads as wl
from workloads import device as wd

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import chunked_prefill_hybrid_tau_gb300 as hb  # noqa: E402
from chunked_prefill_hybrid_tau_gb300 import _lib as L  # noqa: E402

STORE, RESIDUAL, SWIGLU, F32 = L.HB_EPI_STORE, L.HB_EPI_RESIDUAL, L.HB_EPI_SWIGLU, L.HB_EPI_F32


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(shape, g, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(torch.bfloat16)


# ---------------------------------------------------------------- quantization
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("rows,cols", [(1, 16), (1, 4096), (3, 112), (37, 128), (129, 144), (64, 688), (300, 2064),
                                       (130, 14336), (1030, 256)])
def test_quantize_block_bit_exact(rows, cols, block_rows):
    rng = np.random.default_rng(rows * 31 + cols)
    # groups spread over 2^-60 .. 2^60: subnormal codes and every binade occur
    spread = np.exp2(rng.uniform(-60, 60, (-(-rows // 128), -(-cols // 128))))
    each = np.repeat(np.repeat(spread, 128, 0), 128, 1)[:rows, :cols]
    x = wl.bf16_round((rng.standard_normal((rows, cols)) * each).astype(np.float32))
    if rows > 2:
        x[1] = 0.0
        x[2] = 0.0
        x[2, cols // 2] = -1.5
    q, s = hb.hb_quantize_e4m3_block(wd.bf16_tensor(x), block_rows=block_rows)
    hb.hb_check_status()
    qr, sr = of.quantize_blocks(x, block_rows)
    assert s.shape == sr.shape
    assert np.array_equal(s.cpu().numpy().view(np.uint32), sr.view(np.uint32))
    assert np.array_equal(q.cpu().numpy(), qr)


@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_block_tiny_and_non_finite(block_rows):
    """Values down to bf16's smallest; a NaN or an infinity in one group."""
    x = np.zeros((130, 512), np.float32)
    x[0, 0], x[0, 1] = 1e-38, -2.0 ** -133     # below the floor of a scale, zeros beside them
    x[0, 128] = 2.0 ** -112
    x[0, 256] = np.nan
    x[0, 257] = 3.0
    x[0, 384] = np.inf
    x[0, 385] = 1.0
    x[129, 200] = 7.0
    q, s = hb.hb_quantize_e4m3_block(wd.bf16_tensor(x), block_rows=block_rows)
    hb.hb_check_status()
    q, s = q.cpu().numpy(), s.cpu().numpy()
    xf = x.copy()
    xf[0, 256:] = 0
    qr, sr = of.quantize_blocks(xf, block_rows)
    assert np.array_equal(q[0, :256], qr[0, :256]) and np.array_equal(s[0, :2], sr[0, :2])
    assert np.array_equal(q[129], qr[129]) and s[-1, 1] == sr[-1, 1]
    # a NaN: scale and codes of its group; an infinity: infinite scale, NaN where it stands
    assert np.all((q[0, 256:384] & 0x7F) == 0x7F) and np.isnan(s[0, 2])
    assert (q[0, 384] & 0x7F) == 0x7F and np.isinf(s[0, 3]) and np.all((q[0, 385:] & 0x7F) == 0)


def test_quantize_block_leaves_the_rest_alone():
    """Codes and scales of `rows` rows only; 0 rows do nothing."""
    x = randn((40, 272), gen(3))
    q = torch.full((41, 272), 0xAB, dtype=torch.uint8, device="cuda")
    s = torch.full((41, 3), -5.0, device="cuda")
    hb.hb_quantize_e4m3_block(x, q, s, block_rows=1)
    hb.hb_check_status()
    assert bool((q[40] == 0xAB).all()) and bool((s[40] == -5).all()) and not bool((s[:40] == -5).any())
    hb.hb_quantize_e4m3_block(x[:0], q[40:], s[40:], block_rows=1)
    hb.hb_quantize_e4m3_block(x[:0], q[40:], s[40:], block_rows=128)
    hb.hb_check_status()
    assert bool((q[40] == 0xAB).all()) and bool((s[40] == -5).all())


# ---------------------------------------------------------------- projection
def values(codes):
    return codes.view(torch.float8_e4m3fn).double()


def spread(scale, rows, cols, block_rows):
    return scale.double().repeat_interleave(block_rows, 0)[:rows].repeat_interleave(128, 1)[:, :cols]


def tokens(m, k, g):
    x = (torch.randn((m, k), generator=g, device="cuda") *
         torch.exp(torch.randn((1, k), generator=g, device="cuda"))).to(torch.bfloat16)
    return hb.hb_quantize_e4m3_block(x, block_rows=1)


class Projection:
    """Operands of one projection and its sums in 64 bits."""

    def __init__(self, m, n, k, epi, seed=0):
        g = gen(seed + m * 13 + n + k)
        self.m, self.n, self.k, self.epi = m, n, k, epi
        self.a, self.sa = tokens(m, k, g)
        if epi == SWIGLU:
            f = n // 2
            (qg, sg), (qu, su) = (hb.hb_quantize_e4m3_block(randn((f, k), g, 0.05), block_rows=128) for _ in range(2))
            self.b = torch.stack([qg.view(f // 64, 64, k), qu.view(f // 64, 64, k)], 1).reshape(n, k).contiguous()
            self.sb = torch.cat([sg, su])
            row = torch.arange(n, device="cuda")
            self.sb_row = (row // 128 * 64 + row % 64) // 128 + torch.where(row % 128 >= 64, sg.shape[0], 0)
        else:
            self.b, self.sb = hb.hb_quantize_e4m3_block(randn((n, k), g, 0.05), block_rows=128)
            self.sb_row = torch.arange(n, device="cuda") // 128
        self.r = randn((m, n), g) if epi == RESIDUAL else None

    def out(self):
        cols = self.n // 2 if self.epi == SWIGLU else self.n
        return torch.full((self.m, cols), 7.0, dtype=torch.float32 if self.epi == F32 else torch.bfloat16,
                          device="cuda")

    def run(self, rows=None, out=None):
        rows = rows or slice(None)
        out = self.out()[rows] if out is None else out
        r = None if self.r is None else self.r[rows].contiguous()
        hb.hb_gemm_e4m3_block(self.a[rows].contiguous(), self.sa[rows].contiguous(), self.b, self.sb, out, r, self.epi)
        hb.hb_check_status()
        return out

    def sums(self):
        """-> (P, bound of P's error)."""
        a = values(self.a) * spread(self.sa, self.m, self.k, 1)
        b = values(self.b) * self.sb.double()[self.sb_row].repeat_interleave(128, 1)[:, :self.k]
        blocks = -(-self.k // 128)
        return a @ b.T, (127 * 2.0 ** -23 + (blocks + 1) * 2.0 ** -24) * (a.abs() @ b.abs().T)

    def check(self, got):
        p, e = self.sums()
        if self.epi == SWIGLU:
            def part(t, i):
                return t.view(self.m, self.n // 128, 2, 64)[:, :, i].reshape(self.m, -1)

            gate, up, eg, eu = part(p, 0), part(p, 1), part(e, 0), part(e, 1)
            s = gate * torch.sigmoid(gate)
            ref = s * up
            # |silu'| <= 1.1; exp (2^-21 plus the rounding of its argument,
            # |g| 2^-23), the divide and two products
            bound = 1.1 * eg * (up.abs() + eu) + s.abs() * eu + ref.abs() * (2.0 ** -19 + gate.abs() * 2.0 ** -22)
        else:
            ref, bound = p, e
            if self.epi == RESIDUAL:
                ref = self.r.double() + p
                bound = bound + 2.0 ** -24 * ref.abs()
        if self.epi != F32:
            bound = bound + 2.0 ** -8 * (ref.abs() + bound)
        err = (got.double() - ref).abs()
        bad = err > bound + 1e-30
        assert not bool(bad.any()), (f"{int(bad.sum())} of {bad.numel()} outside, worst "
                                     f"{float((err - bound).max()):.3g} at {bad.nonzero()[0].tolist()}")
        return float(err.norm() / ref.norm())


GEMM_CASES = [
    (1, 8, 16, STORE), (1, 128, 128, STORE), (1, 6144, 4096, STORE), (3, 1000, 688, F32), (16, 128, 272, RESIDUAL),
    (1, 128, 16, SWIGLU), (2, 256, 4096, SWIGLU), (5, 1024, 2064, SWIGLU), (16, 28672, 512, SWIGLU),
    (17, 4096, 1040, RESIDUAL), (32, 4096, 14336, RESIDUAL), (33, 200, 384, F32), (48, 32000, 256, F32),
    (64, 4096, 4096, STORE), (63, 640, 128, SWIGLU), (64, 20000, 640, RESIDUAL),
    (65, 128, 128, STORE), (65, 136, 144, F32), (100, 1000, 688, RESIDUAL), (128, 4096, 4096, SWIGLU),
    (127, 264, 1152, STORE), (128, 512, 16, F32),
    (129, 8, 16, STORE), (129, 136, 2064, RESIDUAL), (200, 6144, 512, STORE), (256, 256, 256, F32),
    (201, 1000, 688, F32), (300, 1024, 384, SWIGLU), (333, 4096, 4096, RESIDUAL), (512, 28672, 4096, SWIGLU),
    (512, 4096, 14336, RESIDUAL), (385, 1160, 400, STORE), (1000, 2176, 1296, SWIGLU), (2050, 3200, 272, F32),
    (1024, 6144, 4096, STORE),
]


@pytest.mark.parametrize("m,n,k,epi", GEMM_CASES)
def test_gemm_block(m, n, k, epi):
    pr = Projection(m, n, k, epi)
    rel = pr.check(pr.run())
    if epi == F32:
        assert rel < 1e-5


@pytest.mark.parametrize("n,k,epi", [(1000, 688, STORE), (4096, 1040, RESIDUAL), (1024, 512, SWIGLU), (520, 400, F32)])
def test_gemm_block_rows_do_not_depend_on_the_batch(n, k, epi):
    """The same rows alone, in small and in large batches: the same bits,
    through every kernel (few tokens, one-CTA and CTA-pair tiles)."""
    pr = Projection(700, n, k, epi)
    whole = pr.run()
    for lo, hi in [(0, 1), (5, 21), (100, 130), (333, 397), (200, 300), (690, 700), (128, 384), (0, 513)]:
        part = pr.run(slice(lo, hi))
        assert torch.equal(part, whole[lo:hi]), (lo, hi)


# More outputs than one wave of tiles of weight rows takes, or nearly so: the 128-row tiles of
# one CTA (65 to 128 tokens) and of CTA pairs, 128 and 256 columns wide.
WIDE_CASES = [
    (65, 4872, 144, F32), (128, 5000, 688, RESIDUAL), (100, 4992, 400, SWIGLU), (127, 8200, 1152, STORE),
    (66, 19592, 2064, STORE), (80, 28672, 4096, SWIGLU), (96, 20000, 272, F32),
    (129, 3256, 272, F32), (200, 4104, 688, RESIDUAL), (201, 6144, 2048, STORE), (300, 2432, 1040, SWIGLU),
    (65, 9736, 144, F32), (128, 10000, 688, RESIDUAL), (127, 12296, 1152, STORE), (129, 6408, 272, F32),
    (200, 5000, 688, RESIDUAL), (385, 5000, 400, STORE), (512, 9728, 656, F32), (700, 10248, 1296, RESIDUAL),
    (1100, 9728, 400, SWIGLU), (293, 10728, 400, RESIDUAL), (600, 7168, 272, STORE), (290, 10752, 1296, SWIGLU),
    (257, 11008, 656, F32),
]


@pytest.mark.parametrize("m,n,k,epi", WIDE_CASES)
def test_gemm_block_many_outputs(m, n, k, epi):
    pr = Projection(m, n, k, epi)
    rel = pr.check(pr.run())
    if epi == F32:
        assert rel < 1e-5


@pytest.mark.parametrize("n,k,epi", [(10248, 528, STORE), (9984, 1168, SWIGLU), (5000, 688, F32),
                                     (20000, 272, RESIDUAL), (10728, 656, RESIDUAL)])
def test_gemm_block_rows_do_not_depend_on_the_batch_many_outputs(n, k, epi):
    pr = Projection(700, n, k, epi)
    whole = pr.run()
    for lo, hi in [(0, 1), (5, 21), (100, 130), (333, 397), (400, 465), (200, 300), (128, 384), (0, 293), (0, 513)]:
        part = pr.run(slice(lo, hi))
        assert torch.equal(part, whole[lo:hi]), (lo, hi)


def test_gemm_block_tokens_in_groups():
    """Few outputs and many tokens: groups of 64 tokens, the last one partly
    empty, neighbours untouched."""
    for m, n, epi in [(65, 8, F32), (1000, 136, STORE), (577, 264, RESIDUAL), (130, 1152, SWIGLU), (4000, 128, SWIGLU),
                      (9730, 8, F32)]:
        pr = Projection(m, n, 400, epi)
        buf = torch.full((m + 1, n // 2 if epi == SWIGLU else n), 7.0, device="cuda",
                         dtype=torch.float32 if epi == F32 else torch.bfloat16)
        pr.check(pr.run(out=buf[:m]))
        assert bool((buf[m] == 7).all())


def test_gemm_block_in_place_residual_and_neighbours():
    """R may be C; rows past M and whatever follows the output stay as they were."""
    for m in (9, 100, 300):
        pr = Projection(m, 264, 400, RESIDUAL)
        buf = torch.full((m + 2, 264), 3.0, dtype=torch.bfloat16, device="cuda")
        buf[1:m + 1] = pr.r
        ref = pr.run()
        hb.hb_gemm_e4m3_block(pr.a, pr.sa, pr.b, pr.sb, buf[1:m + 1], buf[1:m + 1], RESIDUAL)
        hb.hb_check_status()
        assert torch.equal(buf[1:m + 1], ref)
        assert bool((buf[0] == 3).all()) and bool((buf[m + 1] == 3).all())


def test_gemm_block_zero_scales_and_nan_rows():
    """A block of zeros adds nothing; a NaN code spoils its own token only."""
    for m in (8, 70, 300):
        pr = Projection(m, 256, 512, STORE)
        pr.sa[3] = 0
        pr.a[5, 200] = 0x7F
        got = pr.run()
        assert bool((got[3] == 0).all()) and bool(got[5].isnan().all())
        keep = [i for i in range(m) if i not in (3, 5)]
        assert not bool(got[keep].isnan().any())
        pr.a[5, 200] = 0
        pr.check(pr.run())


def test_gemm_block_straight_after_its_weights():
    """The weights may be quantized by the call right ahead on the stream."""
    g = gen(8)
    w = [randn((8192, 4096), g, 0.05) for _ in range(2)]
    a, sa = tokens(4, 4096, g)
    ref = []
    for x in w:
        q, s = hb.hb_quantize_e4m3_block(x, block_rows=128)
        torch.cuda.synchronize()
        o = torch.empty((4, 8192), dtype=torch.bfloat16, device="cuda")
        hb.hb_gemm_e4m3_block(a, sa, q, s, o)
        ref.append(o)
    q, s = torch.empty_like(w[0], dtype=torch.uint8), torch.empty((64, 32), device="cuda")
    for i in (0, 1, 0, 1, 1, 0):
        hb.hb_quantize_e4m3_block(w[i], q, s, block_rows=128)
        o = torch.empty((4, 8192), dtype=torch.bfloat16, device="cuda")
        hb.hb_gemm_e4m3_block(a, sa, q, s, o)
        assert torch.equal(o, ref[i])
    hb.hb_check_status()


# ---------------------------------------------------------------- q/k norm, rotation, append
@pytest.mark.parametrize("T,n_q,n_kv,dh", [(1, 32, 8, 128), (1, 1, 1, 64), (7, 4, 2, 64), (333, 4, 2, 64),
                                           (512, 32, 8, 128), (65, 56, 8, 128), (33, 16, 1, 128), (20, 64, 64, 128),
                                           (5, 128, 64, 64)])
def test_kv_append_norm(T, n_q, n_kv, dh):
    rng = np.random.default_rng(T + n_q * 7 + dh)
    dims = wl.Dims(d_model=n_q * dh, n_q=n_q, n_kv=n_kv, d_head=dh, d_ff=64, eps=1e-6, theta=1e4)
    max_pos, num_pages = 5000, T // 16 + 4
    heads = n_q + 2 * n_kv
    qkv = wl.bf16_round(rng.standard_normal((T, heads, dh)).astype(np.float32) *
                        np.exp2(rng.integers(-20, 20, (T, heads, 1))).astype(np.float32))
    qkv[T // 2, 0] = 0.0                                # a head of zeros
    qkv[T // 3, n_q - 1] = 2.0 ** -100                  # far below the epsilon
    g_q, g_k = (wl.bf16_round(1 + 0.3 * rng.standard_normal(dh).astype(np.float32)) for _ in range(2))
    pos = rng.integers(0, max_pos, T).astype(np.int32)
    pos[-1] = max_pos - 1
    slots = rng.permutation(num_pages * 16)[:T].astype(np.int32)
    if T > 4:
        slots[[1, 3]] = -1                              # padding rows: q only
    k0, v0 = (wl.normal_bf16(rng, (num_pages, n_kv, 16, dh)) for _ in range(2))
    kt, vt = wd.bf16_tensor(k0), wd.bf16_tensor(v0)
    q_out = torch.zeros((T, n_q, dh), dtype=torch.bfloat16, device="cuda")
    rope = wd.rope_table_device(max_pos, dims)
    hb.hb_kv_append_norm(wd.bf16_tensor(qkv.reshape(T, -1)), torch.from_numpy(pos).cuda(),
                         torch.from_numpy(slots).cuda(), rope, max_pos, dims, wd.bf16_tensor(g_q),
                         wd.bf16_tensor(g_k), q_out, kt, vt)
    hb.hb_check_status()
    table = rope.cpu().numpy()
    cos, sin = table[..., 0], table[..., 1]

    def turned(x, g):
        y = ol.head_norm(x, g, dims.eps, np.float64)
        a = np.abs(y)
        pair = np.concatenate([a[..., :dh // 2] + a[..., dh // 2:]] * 2, -1)
        return ol.rope(y, pos, cos, sin, np.float64), pair

    def check(got, ref, pair):
        bound = (dh / 2 + 16) * 2.0 ** -24 * pair
        assert np.all(np.abs(got - ref) <= bound + 2.0 ** -8 * (np.abs(ref) + bound) + 2.0 ** -133)

    qr, pair = turned(qkv[:, :n_q], g_q)
    check(wd.to_numpy(q_out).astype(np.float64), qr, pair)
    kr, pair = turned(qkv[:, n_q:n_q + n_kv], g_k)
    k, v = wd.to_numpy(kt), wd.to_numpy(vt)
    live = np.flatnonzero(slots >= 0)
    pg, off = slots[live] // 16, slots[live] % 16
    check(k[pg, :, off].astype(np.float64), kr[live], pair[live])
    assert np.array_equal(v[pg, :, off], qkv[live, n_q + n_kv:])
    k[pg, :, off], v[pg, :, off] = k0[pg, :, off], v0[pg, :, off]
    assert np.array_equal(k, k0) and np.array_equal(v, v0)     # no other slot changes


def test_kv_append_norm_skips_and_reports_bad_rows():
    """A slot past the pool or a position past the table: that row is left
    out (K/V, or everything) and the status word says so."""
    dims = wl.TINY
    g = gen(5)
    qkv = randn((3, dims.qkv_cols), g)
    gains = randn((64,), g)
    rope = wd.rope_table_device(32, dims)
    for pos, slot in (([0, 32, 2], [0, 1, 2]), ([0, 1, 2], [0, 64, 2]), ([0, -1, 2], [0, 1, 2])):
        k, v = (torch.zeros((4, 2, 16, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        q = torch.zeros((3, 4, 64), dtype=torch.bfloat16, device="cuda")
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        hb.hb_kv_append_norm(qkv, i32(pos), i32(slot), rope, 32, dims, gains, gains, q, k, v)
        with pytest.raises(hb.HBError) as e:
            hb.hb_check_status()
        assert e.value.status == L.HB_ERR_DEVICE
        assert bool((q[0] != 0).any()) and bool((q[2] != 0).any())
        assert bool((q[1] != 0).any()) == (pos[1] == 1)
        assert bool((k[0, :, [0, 2]] != 0).any()) and not bool((k[1:] != 0).any())
        assert not bool((v[0, :, 1] != 0).any())


# ---------------------------------------------------------------- together, other streams, graphs
def test_chain_on_a_side_stream_and_in_a_graph():
    """Quantize, project, norm + rotate + append, as the layer runs them: on a
    side stream and replayed from a graph, the same bits as eagerly."""
    dims = wl.Dims(d_model=512, n_q=8, n_kv=2, d_head=64, d_ff=64, eps=1e-6, theta=1e4)
    T, max_pos = 90, 256
    g = gen(21)
    x = randn((T, 512), g)
    wq, ws = hb.hb_quantize_e4m3_block(randn((dims.qkv_cols, 512), g, 0.05), block_rows=128)
    g_q, g_k = randn((64,), g), randn((64,), g)
    rope = wd.rope_table_device(max_pos, dims)
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    slots = torch.arange(T, dtype=torch.int32, device="cuda")
    bufs = {}

    def chain(stream=None):
        q8, s8, qkv, q, k, v = bufs["b"]
        hb.hb_quantize_e4m3_block(x, q8, s8, 1, stream=stream)
        hb.hb_gemm_e4m3_block(q8, s8, wq, ws, qkv, stream=stream)
        hb.hb_kv_append_norm(qkv, pos, slots, rope, max_pos, dims, g_q, g_k, q, k, v, stream=stream)
        return qkv, q, k, v

    def fresh():
        bf = dict(dtype=torch.bfloat16, device="cuda")
        bufs["b"] = (torch.zeros((T, 512), dtype=torch.uint8, device="cuda"), torch.zeros((T, 4), device="cuda"),
                     torch.zeros((T, dims.qkv_cols), **bf), torch.zeros((T, 8, 64), **bf),
                     torch.zeros((8, 2, 16, 64), **bf), torch.zeros((8, 2, 16, 64), **bf))

    fresh()
    ref = [t.clone() for t in chain()]
    assert float(ref[1].float().norm()) > 0
    side = torch.cuda.Stream()
    fresh()
    side.wait_stream(torch.cuda.current_stream())
    got = chain(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, ref))
    fresh()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = chain()
    x2 = randn((T, 512), g)
    x.copy_(x2)
    graph.replay()
    torch.cuda.synchronize()
    again = [t.clone() for t in got]
    assert not torch.equal(again[0], ref[0])
    graph.replay()
    fresh()
    eager = chain()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(eager, again))
    hb.hb_check_status()


def test_gemm_block_calls_at_once():
    """Every kernel on two streams at a time, and a captured graph replayed
    beside eager calls: the bits of the calls one after the other."""
    cases = [Projection(m, n, k, e) for m, n, k, e in
             [(1, 6144, 4096, STORE), (40, 1000, 688, F32), (64, 4096, 2064, RESIDUAL), (90, 12296, 1152, STORE),
              (300, 2432, 1040, SWIGLU), (600, 10248, 400, RESIDUAL), (1100, 9728, 656, F32)]]
    ref = [pr.run() for pr in cases]
    outs = [[pr.out() for pr in cases] for _ in range(3)]

    def call(pr, out):
        hb.hb_gemm_e4m3_block(pr.a, pr.sa, pr.b, pr.sb, out, pr.r, pr.epi)

    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=streams[0]):
        for pr, out in zip(cases, outs[0]):
            call(pr, out)
    for rep in range(20):
        with torch.cuda.stream(streams[0]):
            graph.replay()
        with torch.cuda.stream(streams[1]):
            for i in range(len(cases)):
                call(cases[-1 - i], outs[1][-1 - i])
        for pr, out in zip(cases, outs[2]):
            call(pr, out)
        torch.cuda.synchronize()
        hb.hb_check_status()
        for got in outs:
            for o, r in zip(got, ref):
                assert torch.equal(o, r), rep
                o.fill_(3)


@pytest.mark.parametrize("m", [65, 80, 128, 200, 520])
def test_gemm_block_behind_quantizations_many_times(m):
    """Projections and the quantizations between them, each launched while its
    predecessors still run, over and over: always the same bits.  (One-CTA
    tiles once took a stage's operands for complete one phase early here.)"""
    g = gen(m)
    x = randn((m, 4096), g)
    up, su = hb.hb_quantize_e4m3_block(randn((28672, 4096), g, 0.02), block_rows=128)
    down, sd = hb.hb_quantize_e4m3_block(randn((10240, 14336), g, 0.02), block_rows=128)
    q, s = hb.hb_quantize_e4m3_block(x)
    a = torch.empty((m, 14336), dtype=torch.bfloat16, device="cuda")
    qa, sa = torch.empty_like(a, dtype=torch.uint8), torch.empty((m, 112), device="cuda")
    first = None
    for _ in range(40):
        out = torch.empty((m, 10240), dtype=torch.bfloat16, device="cuda")
        hb.hb_quantize_e4m3_block(x, q, s)
        hb.hb_gemm_e4m3_block(q, s, up, su, a, epilogue=SWIGLU)
        hb.hb_quantize_e4m3_block(a, qa, sa)
        hb.hb_gemm_e4m3_block(qa, sa, down, sd, out)
        first = out if first is None else first
        assert torch.equal(out, first)
    hb.hb_check_status()
