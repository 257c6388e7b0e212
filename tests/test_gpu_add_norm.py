"""hb_add_rmsnorm against its definition in 64 bits (GPU).

h is decided by one fp32 add and one rounding: bit for bit.  The factor
1 / rms carries the fp32 sum of d squares (half a step each), the division,
the epsilon's add and rsqrt (2 steps), under (d + 8) 2^-24, halved by the
root; the two products of y two half steps more: err = (d / 2 + 8) 2^-24 |y|.
bf16 adds half its step, 2^-8 |y|.  A code's value is within half a step of
E4M3 of the quotient (2^-4 of it, 2^-10 under the smallest normal one), the
factors 448 / top and top / 448 and the product are off by half a step each.
"""
import pytest

from workloads import device as wd

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import e4m3_cache as ec  # noqa: E402

import chunked_prefill_hybrid_tau_gb300 as hb  # noqa: E402
from chunked_prefill_hybrid_tau_gb300 import _lib as L  # noqa: E402

BF = torch.bfloat16
EPS = 1e-6
SIZES = [(1, 16), (1, 4096), (3, 64), (5, 256), (9, 272), (7, 512), (4, 1008), (33, 1024), (2, 1040), (5, 2048), (3, 2064),
         (6, 4096), (2, 4112), (3, 7168), (2, 8192), (3, 14336), (2, 16384), (2, 16400), (1, 32768), (700, 128)]


def inputs(rows, d, seed=0):
    g = wd.device_generator(seed + rows + d)
    size = torch.exp(torch.randn((1, d), generator=g, device="cuda"))
    x, r = ((torch.randn((rows, d), generator=g, device="cuda") * size).to(BF) for _ in range(2))
    return x, r, (1 + 0.3 * torch.randn(d, generator=g, device="cuda")).to(BF)


def check(x, r, gamma, fmt, y, scale):
    h = x if r is None else (x.float() + r.float()).to(BF)
    rows, d = h.shape
    hd = h.cpu().double()
    want = hd / torch.sqrt(hd.square().mean(1, keepdim=True) + EPS) * gamma.cpu().double()
    rel = (d / 2 + 8) * 2.0 ** -24
    if fmt == "bf16":
        assert ((y.cpu().double() - want).abs() <= (rel + ec.HALF_BF16) * want.abs()).all()
        return h
    width = d if fmt == "e4m3" else 128
    s = scale.cpu().double().view(rows, -1)
    for b in range(s.shape[1]):
        part = want[:, b * width:(b + 1) * width]
        amax = part.abs().amax(1)
        assert ((s[:, b] - amax / 448).abs() <= (rel + 2.0 ** -23) * amax / 448).all()
        got = ec.values(y.cpu())[:, b * width:(b + 1) * width] * s[:, b, None]
        room = (ec.HALF_E4M3 + rel + 2.0 ** -21) * part.abs() + ec.HALF_SUB * s[:, b, None]
        assert ((got - part).abs() <= room).all()
    return h


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "e4m3_block"])
@pytest.mark.parametrize("rows,d", SIZES)
def test_add_rmsnorm(rows, d, fmt):
    x, r, gamma = inputs(rows, d)
    h = torch.full_like(x, 9.0)
    y, scale = hb.hb_add_rmsnorm(x, r, gamma, EPS, h, fmt=fmt)
    hb.hb_check_status()
    assert torch.equal(check(x, r, gamma, fmt, y, scale).view(torch.int16), h.view(torch.int16))
    # h not stored, and no residual: the same y from h
    for args in ((x, r, gamma, EPS, None), (h, None, gamma, EPS, None)):
        y2, scale2 = hb.hb_add_rmsnorm(*args, fmt=fmt)
        assert torch.equal(y2.view(torch.uint8), y.view(torch.uint8))
        assert fmt == "bf16" or torch.equal(scale2, scale)


def test_a_width_that_is_no_multiple_of_sixteen():
    for d in (8, 24, 1032, 4104):
        x, r, gamma = inputs(3, d)
        y, _ = hb.hb_add_rmsnorm(x, r, gamma, EPS)
        check(x, r, gamma, "bf16", y, None)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "e4m3_block"])
@pytest.mark.parametrize("which", ["x", "residual"])
def test_h_in_place(fmt, which):
    x, r, gamma = inputs(37, 4096)
    h = torch.empty_like(x)
    want, want_scale = hb.hb_add_rmsnorm(x, r, gamma, EPS, h, fmt=fmt)
    got, scale = hb.hb_add_rmsnorm(x, r, gamma, EPS, x if which == "x" else r, fmt=fmt)
    assert torch.equal((x if which == "x" else r).view(torch.int16), h.view(torch.int16))
    assert torch.equal(got.view(torch.uint8), want.view(torch.uint8))
    assert fmt == "bf16" or torch.equal(scale, want_scale)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "e4m3_block"])
@pytest.mark.parametrize("d", [256, 4096])
def test_rows_do_not_depend_on_each_other(fmt, d):
    x, r, gamma = inputs(65, d)
    x[3, 5], r[40, d - 1] = float("nan"), float("inf")
    x[9], r[9] = 0, 0
    h = torch.empty_like(x)
    y, scale = hb.hb_add_rmsnorm(x, r, gamma, EPS, h, fmt=fmt)
    for i in (0, 2, 4, 9, 39, 41, 64):
        one, s = hb.hb_add_rmsnorm(x[i:i + 1], r[i:i + 1], gamma, EPS, fmt=fmt)
        assert torch.equal(one.view(torch.uint8), y[i:i + 1].view(torch.uint8))
        assert fmt == "bf16" or torch.equal(s, scale[i:i + 1])
    vals = y if fmt == "bf16" else y.view(torch.float8_e4m3fn)
    assert torch.isnan(vals[3].float()).all()
    assert (vals[9].float() == 0).all() and (fmt == "bf16" or (scale[9] == 0).all())
    # an infinity: its own y is a NaN, the others of its row 0
    if fmt == "bf16":
        assert torch.isnan(y[40, d - 1]) and (y[40, :d - 1] == 0).all()
    elif fmt == "e4m3":
        assert torch.isnan(scale[3]) and torch.isnan(scale[40])
    else:
        assert torch.isnan(scale[3]).all() and torch.isnan(scale[40, -1]) and (scale[40, :-1] == 0).all()


def test_codes_feed_the_projections():
    """Codes and scales are the operands of the two E4M3 projections."""
    x, r, gamma = inputs(70, 512)
    g = wd.device_generator(3)
    w = wd.randn_bf16((256, 512), g, 0.05)
    h = torch.empty_like(x)
    want = None
    for fmt in ("bf16", "e4m3", "e4m3_block"):
        y, s = hb.hb_add_rmsnorm(x, r, gamma, EPS, h, fmt=fmt)
        out = torch.empty((70, 256), dtype=torch.float32, device="cuda")
        if fmt == "bf16":
            hb.hb_gemm(y, w, out, epilogue=L.HB_EPI_F32)
            want = out
            continue
        if fmt == "e4m3":
            wq, ws = hb.hb_quantize_e4m3(w)
            hb.hb_gemm_e4m3(y, s, wq, ws, out, epilogue=L.HB_EPI_F32)
            vals = ec.values(y.cpu()) * s.cpu().double()[:, None]
            wd64 = ec.values(wq.cpu()) * ws.cpu().double()[:, None]
        else:
            wq, ws = hb.hb_quantize_e4m3_block(w, block_rows=128)
            hb.hb_gemm_e4m3_block(y, s, wq, ws, out, epilogue=L.HB_EPI_F32)
            vals = ec.values(y.cpu()) * s.cpu().double().repeat_interleave(128, 1)
            wd64 = ec.values(wq.cpu()) * ws.cpu().double().repeat_interleave(128, 0).repeat_interleave(128, 1)
        # 512 products summed in fp32, a step 2^-23 each, and a few scale factors
        room = (512 + 8) * 2.0 ** -23 * (vals.abs() @ wd64.abs().T)
        assert ((out.cpu().double() - vals @ wd64.T).abs() <= room).all()
        # within E4M3's error of the bf16 product: two codes a product, half a step each, and the norm's bf16
        per = 2 * ec.HALF_E4M3 + 2.0 ** -7
        sub = ec.HALF_SUB * 2 * (vals.abs().amax() / 448 * wd64.abs().sum(1).amax() + wd64.abs().amax() / 448 * vals.abs().sum(1).amax())
        assert ((out - want).abs().cpu().double() <= per * 1.1 * (vals.abs() @ wd64.abs().T) + sub).all()
    hb.hb_check_status()


def test_another_stream_and_a_graph():
    x, r, gamma = inputs(300, 4096)
    want, ws = hb.hb_add_rmsnorm(x, r, gamma, EPS, fmt="e4m3_block")
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    got, s = hb.hb_add_rmsnorm(x, r, gamma, EPS, fmt="e4m3_block", stream=st)
    st.synchronize()
    assert torch.equal(got, want) and torch.equal(s, ws)
    y, sc = torch.zeros_like(want), torch.zeros_like(ws)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        hb.hb_add_rmsnorm(x, r, gamma, EPS, None, y, sc, fmt="e4m3_block")
    for sign in (1, -1):
        x.mul_(sign), r.mul_(sign)
        g.replay()
        torch.cuda.synchronize()
        # as values: x + r = 0 is +0 for either sign of the two
        assert torch.equal(ec.values(y) * sign, ec.values(want)) and torch.equal(sc, ws)


@pytest.mark.parametrize("d", [256, 1024, 4096])
@pytest.mark.parametrize("fmt", ["e4m3", "e4m3_block"])
def test_maxima_around_the_smallest_of_a_block(fmt, d):
    """Gains that take a row's largest y to 2^-100 ... 2^-132.  The block form
    counts maxima below 2^-112 as 2^-112, the row form has no smallest one.
    Beside the bounds above, y (its product with the gain) and the scale may be
    subnormal in fp32: off by half a step of those, 2^-150."""
    x, r, gamma = inputs(5, d)
    for e in (100, 110, 111, 112, 113, 114, 118, 119, 120, 126, 130, 132):
        g = (gamma.float() * 2.0 ** -e).to(BF)  # subnormal bf16 gains from 2^-126 on
        y, scale = hb.hb_add_rmsnorm(x, r, g, EPS, fmt=fmt)
        hb.hb_check_status()
        h = (x.float() + r.float()).to(BF).cpu().double()
        want = h / torch.sqrt(h.square().mean(1, keepdim=True) + EPS) * g.cpu().double()
        rel, sub = (d / 2 + 8) * 2.0 ** -24, 2.0 ** -150
        width = d if fmt == "e4m3" else 128
        part = want.view(5, -1, width)
        amax = part.abs().amax(2)
        top = amax if fmt == "e4m3" else torch.where(amax > 0, amax.clamp(min=2.0 ** -112), amax)
        s = scale.cpu().double().view(5, -1)
        assert ((s - top / 448).abs() <= (rel + 2.0 ** -23) * top / 448 + (1 + 1 / 448) * sub).all(), e
        # the codes themselves: a maximum's is 448 (or what 2^-112 leaves of it), the others' by the quotient.  amax is off
        # by rel and half a step, twice the factor's own roundings; a code is within half a step
        q = part * 448 / top[..., None]
        off = (2 * rel + 2.0 ** -21) * q.abs() + (q.abs() + 448) * sub / top[..., None] * 2
        got = ec.values(y.cpu()).view(5, -1, width)
        assert ((got - q).abs() <= ec.HALF_E4M3 * (q.abs() + off) + ec.HALF_SUB + off).all(), e
        if fmt == "e4m3":
            assert (got.abs().amax(2) == 448).all()
