"""hb_logprobs against its definition in 64 bits (GPU).

ids are decided by comparisons: equal.  A term exp(x - m): its argument is
off by half a step of the difference and of its product with log2 e, 2 |d|
2^-24 (weighted by the term: at most the mean of |d| under p, E), the
exponential by 2^-22; a thread adds up to n / 4096 + 16 terms, and 12 joins
and as many rescalings follow, each half a step and the exponential's
error: log s is off by A = 2^-24 (n / 4096 + 16 + 12 * 8 + 4 + 2 E) and 2^-23
|log s|.  A log probability adds half a step of x - m and of itself.  The
entropy's t / s: the terms' errors times |d|, that is A E, and t's adds on top.
"""
import math

import pytest

from workloads import device as wd

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import chunked_prefill_hybrid_tau_gb300 as hb  # noqa: E402

U = 2.0 ** -24


def logits_of(rows, vocab, dtype, extra=0, seed=0, size=3.0, offset=0):
    g = wd.device_generator(seed + rows + vocab)
    flat = torch.full((rows * (vocab + extra) + offset,), 1e9, dtype=dtype, device="cuda")
    x = flat[offset:].view(rows, vocab + extra)[:, :vocab]
    x.copy_(torch.randn((rows, vocab), generator=g, device="cuda") * size)
    return x


def call(x, n_tokens=3, k=5, tokens=None, seed=0):
    rows, vocab = x.shape
    g = wd.device_generator(seed)
    if tokens is None:
        tokens = torch.randint(0, vocab, (rows, n_tokens), generator=g, device="cuda", dtype=torch.int32)
    f32 = dict(dtype=torch.float32, device="cuda")
    lp, ent = torch.full(tokens.shape, 5.0, **f32), torch.full((rows,), 5.0, **f32)
    ids, tlp = torch.full((rows, k), -7, dtype=torch.int32, device="cuda"), torch.full((rows, k), 5.0, **f32)
    hb.hb_logprobs(x, tokens, lp, ent, ids, tlp)
    return tokens, lp, ent, ids, tlp


def check(x, tokens, lp, ent, ids, tlp):
    vocab = x.shape[1]
    x = x.cpu().double()
    m = x.amax(1, keepdim=True)
    d = x - m
    p = torch.exp(d)
    s = p.sum(1, keepdim=True)
    log_s = torch.log(s)
    spread = (p * d.clamp(min=-1e30).abs()).sum(1, keepdim=True) / s
    a = U * (vocab / 4096 + 16 + 12 * 8 + 4 + 2 * spread) + 2 * U * log_s.abs()

    def same(got, at):
        want = d.gather(1, at) - log_s
        room = a + U * (d.gather(1, at).abs() + want.abs())
        got = got.cpu().double()
        hidden = want.float() == -math.inf  # -6e38 is beyond fp32
        assert torch.equal(got == -math.inf, hidden)
        assert ((got - want).abs()[~hidden] <= room[~hidden]).all()

    same(lp, tokens.cpu().long())
    order = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :ids.shape[1]]
    assert torch.equal(ids.cpu().long(), order)
    same(tlp, order)
    want = log_s + spread
    room = a * (2 + 2 * spread) + 2 * U * (log_s.abs() + spread + want)
    assert ((ent.cpu().double()[:, None] - want).abs() <= room).all()


DTYPES = [torch.float32, torch.bfloat16]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,vocab,k", [(1, 1, 1), (1, 2, 2), (3, 7, 7), (2, 31, 31), (1, 64, 32), (5, 100, 32),
                                          (9, 257, 3), (2, 1000, 32), (17, 4097, 20), (1, 32000, 20), (40, 32000, 5),
                                          (65, 32003, 1), (150, 12345, 32), (330, 5001, 8), (2, 152001, 32)])
def test_logprobs(rows, vocab, k, dtype):
    x = logits_of(rows, vocab, dtype)
    check(x, *call(x, k=k))
    hb.hb_check_status()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("extra,offset", [(1, 0), (5, 1), (3, 3), (64, 0), (0, 7)])
def test_strides_and_alignments(dtype, extra, offset):
    x = logits_of(11, 5003, dtype, extra=extra, offset=offset)
    check(x, *call(x, k=9))


@pytest.mark.parametrize("dtype", DTYPES)
def test_equal_logits_and_orders(dtype):
    """Ties go to the lower index; rows in rising and falling order; large ones side by side."""
    vocab = 40000
    rows = [torch.zeros(vocab), torch.full((vocab,), -3.0), torch.arange(vocab).float() / 256,
            -torch.arange(vocab).float() / 256, (torch.arange(vocab) % 2).float(), (torch.arange(vocab) // 5000).float(),
            torch.where(torch.arange(vocab) % 2 == 0, 0.0, -0.0), torch.arange(vocab).float() // 16 % 4]
    block = torch.randn(vocab, generator=torch.Generator().manual_seed(1))
    block[20000:22000] += 20  # the best in a few threads' pieces
    strided = torch.zeros(vocab)
    strided[64::2048] = 5.0
    strided[65::2048] = 5.0
    few = torch.randn(vocab, generator=torch.Generator().manual_seed(2))
    v = torch.arange(vocab) // 4 % 512 // 4
    few[v < 6] += 30  # all the best in six groups of lanes
    x = torch.stack(rows + [block, strided, few]).to(dtype).cuda()
    for k in (1, 20, 32):
        check(x, *call(x, k=k))
        for i in range(x.shape[0]):
            check(x[i:i + 1], *call(x[i:i + 1], k=k))


@pytest.mark.parametrize("dtype", DTYPES)
def test_masked_rows(dtype):
    x = logits_of(6, 9001, dtype)
    g = wd.device_generator(1)
    x.masked_fill_(torch.rand(x.shape, generator=g, device="cuda") < 0.95, -math.inf)
    x[2] = -math.inf
    x[2, 77] = 2.0          # one token left
    x[3] = -math.inf
    x[3, 9000] = -3.0e38
    x[3, 1] = 3.0e38        # a difference that overflows
    x[4, :] = torch.finfo(dtype).min
    tokens = torch.tensor([[0, 77, 9000]] * 6, dtype=torch.int32, device="cuda")
    out = call(x, tokens=tokens, k=32)
    check(x, *out)
    assert out[1][2].tolist() == [-math.inf, 0.0, -math.inf] and out[2][2] == 0


@pytest.mark.parametrize("rows", [1, 40, 700])
@pytest.mark.parametrize("dtype", DTYPES)
def test_rows_without_a_distribution(dtype, rows):
    x = logits_of(rows, 6001, dtype)
    clean = call(x, k=6)
    y = x.clone()
    y[0, 5], y[0, 4001] = math.nan, math.nan
    if rows > 1:
        y[1], y[2, 3000] = -math.inf, math.inf
        y[3, 10], y[3, 9] = -math.nan, math.inf
    tokens, lp, ent, ids, tlp = call(y, k=6)
    hb.hb_check_status()
    bad = list(range(4 if rows > 1 else 1))
    for t in (lp, ent, tlp):
        assert torch.isnan(t[bad]).all()
    best = y[0].float()
    best[torch.isnan(best)] = math.inf
    assert ids[0].tolist() == torch.sort(best, descending=True, stable=True).indices[:6].tolist()
    if rows > 1:
        assert ids[1].tolist() == list(range(6)) and ids[2, 0] == 3000 and ids[3, :2].tolist() == [10, 9]
        for a, b in zip(clean, (tokens, lp, ent, ids, tlp)):
            assert torch.equal(a[4:], b[4:])


@pytest.mark.parametrize("dtype", DTYPES)
def test_rows_do_not_depend_on_the_call(dtype):
    """The same bits whatever the number of rows, which decides how many CTAs share one."""
    x = logits_of(700, 8000, dtype)
    tokens, lp, ent, ids, tlp = call(x, k=7)
    for n in (1, 2, 37, 38, 39, 75, 76, 77, 151, 152, 153, 304, 305, 608, 609):
        _, lp2, ent2, ids2, tlp2 = call(x[:n], tokens=tokens[:n], k=7)
        for a, b in ((lp, lp2), (ent, ent2), (ids, ids2), (tlp, tlp2)):
            assert torch.equal(a[:n], b), n


def test_padding_and_bad_tokens():
    x = logits_of(4, 500, torch.float32)
    tokens = torch.tensor([[1, -1], [-5, 2], [3, 4], [0, 499]], dtype=torch.int32, device="cuda")
    _, lp, *_ = call(x, tokens=tokens, k=0)
    hb.hb_check_status()
    want = torch.log_softmax(x.double(), 1).gather(1, tokens.clamp(min=0).long())
    assert (lp[tokens < 0] == 5.0).all()
    assert torch.allclose(lp[tokens >= 0].double(), want[tokens >= 0], atol=1e-5)
    tokens[2, 1] = 500
    _, lp2, *_ = call(x, tokens=tokens, k=0)
    with pytest.raises(hb.HBError):
        hb.hb_check_status()
    assert lp2[2, 1] == 5.0 and torch.equal(lp2[[0, 1, 3]], lp[[0, 1, 3]])


def test_outputs_left_out():
    x = logits_of(5, 1000, torch.bfloat16)
    tokens, lp, ent, ids, tlp = call(x)
    e = torch.empty_like(ent)
    hb.hb_logprobs(x, entropy=e)
    assert torch.equal(e, ent)
    a, b = torch.empty_like(lp), torch.empty_like(ids)
    hb.hb_logprobs(x, tokens, a)
    assert torch.equal(a, lp)
    c = torch.empty_like(tlp)
    hb.hb_logprobs(x, top_ids=b, top_logprobs=c)
    assert torch.equal(b, ids) and torch.equal(c, tlp)
    hb.hb_logprobs(x)
    hb.hb_logprobs(x[:0], tokens[:0], a[:0], e[:0], b[:0], c[:0])


def test_another_stream_and_a_graph():
    x = logits_of(33, 32000, torch.float32)
    want = call(x)
    torch.cuda.synchronize()
    out = [torch.zeros_like(t) for t in want[1:]]
    st = torch.cuda.Stream()
    hb.hb_logprobs(x, want[0], *out, stream=st)
    st.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want[1:], out))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        hb.hb_logprobs(x, want[0], *out)
    x.copy_(x.flip(0))
    again = call(x, tokens=want[0])
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(again[1:], out))


def test_final_logits_then_logprobs():
    """Behind the LM head, on the same stream, as a server calls them."""
    g = wd.device_generator(9)
    x, w, g_f = (wd.randn_bf16(s, g) for s in ((20, 256), (2048, 256), (256,)))
    rows = torch.tensor([3, 19, 0], dtype=torch.int32, device="cuda")
    logits = torch.empty((3, 2048), dtype=torch.float32, device="cuda")
    hb.hb_final_logits(x, rows, g_f, w, logits, wd.workspace(3 * 256 * 2), 1e-6)
    out = call(logits)
    hb.hb_check_status()
    check(logits, *out)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,vocab", [(1, 152001), (64, 32000), (160, 12345), (700, 5003)])
@pytest.mark.parametrize("allowed", [1, 12, 100])
def test_rows_of_a_few_allowed_tokens(rows, vocab, allowed, dtype):
    """A hard mask: fewer finite logits than best alternatives asked for, or a few more; the rest of
    the alternatives are the first masked tokens."""
    x = logits_of(rows, vocab, dtype)
    g = wd.device_generator(allowed)
    at = torch.stack([torch.randperm(vocab, generator=g, device="cuda")[:allowed] for _ in range(rows)])
    kept = x.gather(1, at)
    x.fill_(-math.inf)
    x.scatter_(1, at, kept)
    check(x, *call(x, tokens=at[:, :1].to(torch.int32), k=20))
    check(x, *call(x, tokens=at[:, -1:].to(torch.int32), k=1))
    hb.hb_check_status()
