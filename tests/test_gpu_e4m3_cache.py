"""hb_kv_append_e4m3 and hb_attention_e4m3 against their definitions in 64
bits (GPU).

append  values are quantized exactly: bit for bit.  Keys are rotated (and
        normed) in fp32 first; with err the bound of that (inv_rms: the sum of
        d squares, half a step each, under (d + 8) 2^-24, halved by the root;
        the norm's products and the rotation's product and add, 4 half steps
        more: (d / 2 + 16) 2^-24 (|y_i| + |y_j|)) a code stands for a value within half a
        step of E4M3 and err of the key, under the scale of the rule unless
        the maximum is within err of a power's limit.
attention  tests/e4m3_cache.py.
"""
import math

import numpy as np
import pytest

import workloads as wl
from gpu_harness import plan_both
from workloads import device as wd

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import e4m3_cache as ec  # noqa: E402

import chunked_prefill_hybrid_tau_gb300 as hb  # noqa: E402


BF = torch.bfloat16


def dims_of(n_q, n_kv, d_head):
    return wl.Dims(d_model=64, n_q=n_q, n_kv=n_kv, d_head=d_head, d_ff=64)


def empty_cache(pages, n_kv, d, fill=0xAA):
    return [torch.full((pages, n_kv, 16, d), fill, dtype=torch.uint8, device="cuda") if i % 2 == 0 else
            torch.full((pages, n_kv, 16), fill, dtype=torch.uint8, device="cuda") for i in range(4)]


# ---------------------------------------------------------------- append
def append(qkv, pos, slots, dims, pages, rope, max_pos, gains=(None, None), cache=None):
    T = qkv.shape[0]
    cache = cache or empty_cache(pages, dims.n_kv, dims.d_head)
    q = torch.full((T, dims.n_q, dims.d_head), 7.0, dtype=BF, device="cuda")
    hb.hb_kv_append_e4m3(qkv, pos, slots, rope, max_pos, dims, q, *cache, *gains)
    return q, cache


@pytest.mark.parametrize("normed", [False, True])
@pytest.mark.parametrize("n_q,n_kv,d,T", [(4, 2, 64, 1), (32, 8, 128, 37), (1, 1, 128, 5), (7, 7, 64, 130),
                                          (16, 1, 128, 300), (64, 8, 128, 700)])
def test_append(n_q, n_kv, d, T, normed):
    dims, max_pos, pages = dims_of(n_q, n_kv, d), 2048, T // 16 + 4
    g = wd.device_generator(n_q + T)
    qkv = wd.randn_bf16((T, n_q + 2 * n_kv, d), g)
    qkv *= torch.exp(torch.randn((T, n_q + 2 * n_kv, 1), generator=g, device="cuda") * 3).to(BF)
    qkv[0, n_q:] = 0  # vectors of zeros
    pos = torch.randint(0, max_pos, (T,), generator=g, device="cuda", dtype=torch.int32)
    slots = torch.randperm(pages * 16, generator=g, device="cuda")[:T].to(torch.int32)
    slots[T // 2] = -1 if T > 1 else slots[0]
    rope = wd.rope_table_device(max_pos, dims)
    gains = [(1 + 0.3 * torch.randn(d, generator=g, device="cuda")).to(BF) for _ in range(2)] if normed else (None, None)
    q, (kc, ks, vc, vs) = append(qkv.view(T, -1), pos, slots, dims, pages, rope, max_pos, gains)
    hb.hb_check_status()

    x = qkv.cpu().double()
    turn = rope.cpu().double()[pos.cpu().long()][:, None]

    def rotated(h, gain):
        if gain is not None:
            h = h / torch.sqrt(h.square().mean(-1, keepdim=True) + dims.eps) * gain.cpu().double()
        a, b, cos, sin = h[..., :d // 2], h[..., d // 2:], turn[..., 0], turn[..., 1]
        size = torch.cat([a.abs() + b.abs()] * 2, -1)
        return torch.cat([a * cos - b * sin, b * cos + a * sin], -1), (d / 2 + 16) * 2.0 ** -24 * size

    want, err = rotated(x[:, :n_q], gains[0])
    assert ((q.cpu().double() - want).abs() <= err + ec.HALF_BF16 * want.abs()).all()

    live = (slots >= 0).cpu()
    page, off = slots.cpu()[live].long() // 16, slots.cpu()[live].long() % 16
    codes, bytes_ = ec.quantize(x[live][:, n_q + n_kv:])
    assert torch.equal(vc.cpu()[page, :, off], codes) and torch.equal(vs.cpu()[page, :, off], bytes_)
    key, err = (t[live] for t in rotated(x[:, n_q:n_q + n_kv], gains[1]))
    got_e = ks.cpu()[page, :, off].double() - 127
    amax, off_by = key.abs().amax(-1), err.amax(-1)
    assert (got_e >= ec.exponent(amax - off_by)).all() and (got_e <= ec.exponent(amax + off_by)).all()
    got = ec.values(kc.cpu()[page, :, off]) * torch.exp2(got_e)[..., None]
    room = ec.HALF_E4M3 * key.abs() + ec.HALF_SUB * torch.exp2(got_e)[..., None]
    assert ((got - key).abs() <= room + err * (1 + ec.HALF_E4M3)).all()
    # nothing else was touched
    kept = torch.ones(pages, 16, dtype=torch.bool)
    kept[page, off] = False
    for t in (kc, ks, vc, vs):
        assert (t.cpu().transpose(1, 2)[kept] == 0xAA).all()


def test_append_extremes():
    """Subnormal, huge, NaN and infinite vectors; each by its own."""
    dims, d = dims_of(1, 1, 64), 64
    rows = torch.zeros(8, 3, d)
    one = torch.linspace(-1, 1, d)
    for i, size in enumerate([2.0 ** -133, 2.0 ** -110, 2.0 ** 127, 448 * 2.0 ** -100, 449 * 2.0 ** 30, 1.0, 1.0, 1.0]):
        rows[i, 2] = one * size
    rows[5, 2, 3] = math.nan
    rows[6, 2, 63] = -math.inf
    qkv = rows.to(BF).cuda()
    slots = torch.arange(8, dtype=torch.int32, device="cuda")
    _, (_, _, vc, vs) = append(qkv.view(8, -1), torch.zeros_like(slots), slots, dims, 1, wd.rope_table_device(4, dims), 4)
    codes, bytes_ = ec.quantize(qkv.cpu()[:, 2:].double())
    assert torch.equal(vc.cpu()[0, 0, :8], codes[:, 0]) and torch.equal(vs.cpu()[0, 0, :8], bytes_[:, 0])
    assert vs[0, 0, 5] == 255 and vs[0, 0, 6] == 255 and vs[0, 0, 7] != 255


def test_append_reports_bad_rows_and_keeps_the_others():
    dims = dims_of(4, 2, 64)
    g = wd.device_generator(5)
    qkv = wd.randn_bf16((4, 8 * 64), g)
    rope = wd.rope_table_device(32, dims)
    i32 = dict(dtype=torch.int32, device="cuda")
    want_q, want = append(qkv, torch.tensor([1, 2, 3, 4], **i32), torch.tensor([0, -1, -1, 3], **i32), dims, 1, rope, 32)
    hb.hb_check_status()
    for pos, slots in (([1, 2, 3, 4], [0, 16, -1, 3]), ([1, 2, 32, 4], [0, -1, 2, 3]), ([1, 2, -1, 4], [0, -1, 2, 3])):
        q, got = append(qkv, torch.tensor(pos, **i32), torch.tensor(slots, **i32), dims, 1, rope, 32)
        with pytest.raises(hb.HBError):
            hb.hb_check_status()
        hb.hb_check_status()
        assert all(torch.equal(a, b) for a, b in zip(got, want)) and torch.equal(q[[0, 3]], want_q[[0, 3]])


# ---------------------------------------------------------------- attention
def batch(dims, dec_ctx, prefills, tau, chunk, seed, size=1.0):
    """A planned iteration and a random cache of its requests.  Every byte of
    the pools that no row may see holds NaN codes and NaN scales."""
    rng = np.random.default_rng(seed)
    st = wl.make_state(rng, dims, dec_ctx, prefills, slack_pages=wl.pages_for(tau) + len(dec_ctx) + 8,
                       random_prefix=False, fill_kv=False)
    hp, _ = plan_both(st, tau, chunk)
    g = wd.device_generator(seed)
    shape = (st.num_pages, dims.n_kv, 16, dims.d_head)
    seen = torch.zeros(st.num_pages, 16, dtype=torch.bool)
    table = hp.block_table.tolist()
    for s, n in enumerate(hp.seq_kv_len):
        t = np.arange(n)
        seen[np.asarray(table[s])[t // 16], t % 16] = True
    cache = []
    for _ in range(2):
        x = torch.randn(shape, generator=g, device="cuda").cpu().double() * size
        x *= torch.exp(torch.randn((st.num_pages, dims.n_kv, 16, 1), generator=torch.Generator().manual_seed(seed)))
        c, e = ec.quantize(x)
        cache += [torch.where(seen[:, None, :, None], c, 0x7f).to(torch.uint8),
                  torch.where(seen[:, None], e, 255).to(torch.uint8)]
    q = wd.randn_bf16((hp.n_rows, dims.n_q, dims.d_head), g)
    return hp, q, cache, table


def attend(hp, q, cache, dims, max_kv=None, stream=None, ws=None, dp=None):
    dp = dp or hb.DevicePlan(hp)
    max_kv = max_kv or int(max(hp.seq_kv_len))
    out = torch.full((hp.n_rows, dims.n_q * dims.d_head), math.nan, dtype=BF, device="cuda")
    if ws is None:
        ws = wd.workspace(hb.hb_attention_e4m3_workspace_bytes(dims, hp.n_rows, hp.n_seqs, max_kv))
        ws.fill_(0xFF)
    hb.hb_attention_e4m3(q, *[t.cuda() for t in cache], dp, dims, max_kv, out, ws, stream)
    return out


def check(dims, dec_ctx, prefills, tau, chunk, seed, size=1.0):
    hp, q, cache, table = batch(dims, dec_ctx, prefills, tau, chunk, seed, size)
    out = attend(hp, q, cache, dims)
    hb.hb_check_status()
    want, bound = ec.attention(q.cpu(), *cache, table, hp.seq_q_start.tolist(), hp.seq_kv_len.tolist())
    got = out.cpu().double()
    assert torch.isfinite(got).all()
    excess = (got - want).abs() - bound
    assert (excess <= 0).all(), (float(excess.max()), np.unravel_index(int(excess.argmax()), excess.shape))
    return hp


HEADS = [(4, 2, 64), (4, 4, 128), (32, 8, 128), (16, 1, 128), (6, 2, 64), (3, 1, 128), (10, 2, 128), (8, 1, 64)]


@pytest.mark.parametrize("n_q,n_kv,d", HEADS)
def test_attention_hybrid(n_q, n_kv, d):
    hp = check(dims_of(n_q, n_kv, d), [0, 1, 14, 15, 16, 127, 128, 255, 256, 300, 1023, 1025], [(600, 100)], 12 + 133, 133,
               seed=n_q + d)
    assert hp.n_rows == 145


@pytest.mark.parametrize("n_q,n_kv,d", [(8, 2, 128), (4, 2, 64), (3, 3, 128)])
@pytest.mark.parametrize("ctx", [[0], [1], [2500], [511, 512, 513], [4095]])
def test_attention_decode_only(n_q, n_kv, d, ctx):
    check(dims_of(n_q, n_kv, d), ctx, [], len(ctx), 1, seed=sum(ctx))


@pytest.mark.parametrize("n_q,n_kv,d", [(8, 2, 128), (4, 2, 64), (3, 1, 128)])
@pytest.mark.parametrize("prefill,chunk", [((2, 0), 2), ((700, 0), 700), ((129, 0), 128), ((900, 515), 257),
                                           ((400, 127), 17)])
def test_attention_one_chunk(n_q, n_kv, d, prefill, chunk):
    check(dims_of(n_q, n_kv, d), [], [prefill], chunk, chunk, seed=chunk)


def test_attention_several_chunks_and_a_one_token_chunk():
    hp = check(dims_of(8, 4, 128), [40, 700], [(300, 50), (90, 0), (500, 499)], 2 + 100 + 90 + 1, 100, seed=4)
    assert sorted(np.diff(hp.seq_q_start).tolist()) == [1, 1, 1, 90, 100]


def test_attention_peaked_scores():
    """Scores of some hundred: one key has nearly all the weight."""
    check(dims_of(8, 2, 128), [5, 700], [(300, 40)], 2 + 130, 130, seed=8, size=40.0)
    check(dims_of(4, 2, 64), [5, 700], [(300, 40)], 2 + 130, 130, seed=8, size=40.0)


@pytest.mark.parametrize("n_q,n_kv,d", [(8, 2, 128), (4, 2, 64)])
def test_attention_nan_scales_reach_their_heads_rows_only(n_q, n_kv, d):
    dims = dims_of(n_q, n_kv, d)
    hp, q, cache, table = batch(dims, [50, 300], [(200, 30)], 2 + 70, 70, seed=11)
    clean = attend(hp, q, cache, dims).view(hp.n_rows, n_q, d)
    cache[3][table[1][2], 1, 5] = 255   # value of key 37 of the second decode, kv head 1
    cache[1][table[2][3], 0, 2] = 255   # key 50 of the chunk's sequence, kv head 0
    got = attend(hp, q, cache, dims).view(hp.n_rows, n_q, d)
    hb.hb_check_status()
    grp = n_q // n_kv
    bad = torch.zeros(hp.n_rows, n_q, dtype=torch.bool, device="cuda")
    bad[1, grp:] = True
    chunk_rows = torch.arange(2, hp.n_rows)
    bad[chunk_rows[chunk_rows - 2 + 30 >= 50], :grp] = True  # rows from position 50 on
    assert torch.isnan(got[bad]).all() and torch.equal(got[~bad], clean[~bad])


def test_attention_rows_do_not_depend_on_the_batch():
    """A sequence alone gives the bits that it gives among others, whatever the hints say."""
    for n_q, n_kv, d in [(8, 2, 128), (4, 2, 64)]:
        dims = dims_of(n_q, n_kv, d)
        hp, q, cache, table = batch(dims, [700, 2100, 33], [(500, 60), (900, 300)], 3 + 2 * 150, 150, seed=13)
        dp = hb.DevicePlan(hp)
        out = attend(hp, q, cache, dims, max_kv=4096, dp=dp)
        dp.hints = (0, 0, 0)
        assert torch.equal(out, attend(hp, q, cache, dims, max_kv=2101, dp=dp))
        for s in range(hp.n_seqs):
            r0, r1 = hp.seq_q_start[s], hp.seq_q_start[s + 1]
            one = hb.DevicePlan(_alone(hp, s))
            o = torch.empty((r1 - r0, n_q * d), dtype=BF, device="cuda")
            ws = wd.workspace(hb.hb_attention_e4m3_workspace_bytes(dims, r1 - r0, 1, 4096))
            hb.hb_attention_e4m3(q[r0:r1].contiguous(), *[t.cuda() for t in cache], one, dims, 4096, o, ws)
            assert torch.equal(o, out[r0:r1]), s
        hb.hb_check_status()


@pytest.mark.parametrize("n_q,n_kv,d", [(8, 2, 128), (5, 1, 64)])
def test_attention_hints_move_work_only(n_q, n_kv, d):
    """Whatever the plan says of its work (SMs of either kind, tiles of a unit)."""
    dims = dims_of(n_q, n_kv, d)
    hp, q, cache, _ = batch(dims, [40, 700, 1300], [(900, 300)], 3 + 290, 290, seed=17)
    dp = hb.DevicePlan(hp)
    want = attend(hp, q, cache, dims, dp=dp)
    seen = [dp.hints, (0, 0, 0), (1, 10 ** 9, 2 ** 20), (10 ** 9, 1, 1), (0, 290 * 600, 290), (10 ** 6, 290 * 600, 10 ** 5)]
    for hints in seen[1:]:
        dp.hints = hints
        assert torch.equal(attend(hp, q, cache, dims, dp=dp), want), hints
    hb.hb_check_status()


@pytest.mark.parametrize("n_q,n_kv,d", [(4, 2, 128), (12, 4, 64), (40, 8, 128)])
@pytest.mark.parametrize("prefills,chunk", [([(1025, 1020)], 5), ([(2048, 2041)], 7), ([(5000, 4990)], 130),
                                            ([(1030, 1000), (9216, 9215 - 126), (2300, 2100)], 200),
                                            ([(9000, 8000)], 300)])
def test_attention_short_chunks_behind_long_prefixes(n_q, n_kv, d, prefills, chunk):
    """Their keys are taken in parts: each row's result is that of its sequence alone."""
    dims = dims_of(n_q, n_kv, d)
    rows = sum(min(chunk, n - done) for n, done in prefills)
    hp = check(dims, [3, 600], prefills, 2 + rows, chunk, seed=rows + n_q)
    assert hp.n_rows == 2 + rows
    hp, q, cache, _ = batch(dims, [3, 600], prefills, 2 + rows, chunk, rows + n_q)
    out = attend(hp, q, cache, dims)
    for s in range(2, hp.n_seqs):
        r0, r1 = hp.seq_q_start[s], hp.seq_q_start[s + 1]
        one = attend(_alone(hp, s), q[r0:r1].contiguous(), cache, dims, max_kv=12000)
        assert torch.equal(one, out[r0:r1]), s
    hb.hb_check_status()


@pytest.mark.parametrize("n_q,n_kv,d", [(4, 1, 128), (3, 1, 64)])
def test_attention_more_chunk_keys_than_are_widened_ahead(n_q, n_kv, d):
    """Sequences behind the end of the workspace's scratch: the same bits as alone."""
    dims = dims_of(n_q, n_kv, d)
    hp, q, cache, table = batch(dims, [900], [(140000, 139990), (122000, 121870), (20000, 19800)],
                              1 + 10 + 130 + 200, 200, seed=19)
    assert sorted(np.diff(hp.seq_q_start).tolist()) == [1, 10, 130, 200]
    out = attend(hp, q, cache, dims)
    hb.hb_check_status()
    want, bound = ec.attention(q.cpu(), *cache, table, hp.seq_q_start.tolist(), hp.seq_kv_len.tolist())
    assert ((out.cpu().double() - want).abs() <= bound).all()
    for s in range(hp.n_seqs):
        r0, r1 = hp.seq_q_start[s], hp.seq_q_start[s + 1]
        one = hb.DevicePlan(_alone(hp, s))
        o = torch.empty((r1 - r0, n_q * d), dtype=BF, device="cuda")
        ws = wd.workspace(hb.hb_attention_e4m3_workspace_bytes(dims, r1 - r0, 1, 140000))
        hb.hb_attention_e4m3(q[r0:r1].contiguous(), *[t.cuda() for t in cache], one, dims, 140000, o, ws)
        assert torch.equal(o, out[r0:r1]), s


def _alone(hp, s):
    import dataclasses
    r0, r1 = int(hp.seq_q_start[s]), int(hp.seq_q_start[s + 1])
    return dataclasses.replace(hp, row_seq=np.zeros(r1 - r0, np.int32), row_pos=hp.row_pos[r0:r1],
                               slot_mapping=hp.slot_mapping[r0:r1], seq_q_start=np.array([0, r1 - r0], np.int32),
                               seq_pos0=hp.seq_pos0[s:s + 1], seq_kv_len=hp.seq_kv_len[s:s + 1],
                               seq_kind=hp.seq_kind[s:s + 1], seq_req=hp.seq_req[s:s + 1],
                               block_table=hp.block_table[s:s + 1], decode_pairs=0, chunk_pairs=0, chunk_rows=0)


def test_attention_reports_bad_plans():
    """Lengths and page ids out of range are found on the device and no access follows them."""
    dims = dims_of(8, 2, 128)
    hp, q, cache, _ = batch(dims, [50, 300], [(200, 30)], 2 + 70, 70, seed=17)

    def bad(change, max_kv=400):
        import copy
        other = copy.deepcopy(hp)
        change(other)
        attend(other, q, cache, dims, max_kv=max_kv)
        with pytest.raises(hb.HBError):
            hb.hb_check_status()
        hb.hb_check_status()

    def page(p, s, i, v):
        p.block_table[s, i] = v

    bad(lambda p: page(p, 0, 1, -1))
    bad(lambda p: page(p, 1, 0, 1 << 30))
    bad(lambda p: page(p, 2, 2, cache[0].shape[0]))
    bad(lambda p: p.seq_kv_len.__setitem__(0, 10 ** 6))
    bad(lambda p: p.seq_kv_len.__setitem__(2, 3))
    bad(lambda p: None, max_kv=299)
    bad(lambda p: p.seq_q_start.__setitem__(1, 0))


def test_attention_streams_and_graphs():
    """Another stream than the current one; two captured calls with workspaces of
    their own, replayed side by side; inputs that change between replays."""
    dims = dims_of(8, 2, 128)
    cases = [batch(dims, [700, 33], [(400, 100)], 2 + 140, 140, seed=s) for s in (21, 22)]
    want = [attend(hp, q, cache, dims) for hp, q, cache, _ in cases]
    side = [torch.cuda.Stream() for _ in cases]
    held, graphs, outs = [], [], []
    for (hp, q, cache, _), st in zip(cases, side):
        dev = [t.cuda() for t in cache]
        dp, ws = hb.DevicePlan(hp), wd.workspace(hb.hb_attention_e4m3_workspace_bytes(dims, hp.n_rows, hp.n_seqs, 800))
        out = torch.zeros((hp.n_rows, dims.n_q * dims.d_head), dtype=BF, device="cuda")
        qs = q.clone()
        torch.cuda.synchronize()
        hb.hb_attention_e4m3(qs, *dev, dp, dims, 800, out, ws, stream=st)
        st.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            hb.hb_attention_e4m3(qs, *dev, dp, dims, 800, out, ws)
        held.append((dev, dp, ws, qs))
        graphs.append(g)
        outs.append(out)
    for i in range(2):
        assert torch.equal(outs[i], want[i])
    for rep in range(4):
        for i in range(2):
            outs[i].zero_()
            held[i][3].copy_(cases[i][1] if rep % 2 == 0 else -cases[i][1])
        torch.cuda.synchronize()
        for g, st in zip(graphs, side):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for i in range(2):
            assert torch.equal(outs[i], want[i]) == (rep % 2 == 0)
    hb.hb_check_status()


def test_attention_large_pool_offsets():
    """Pages whose byte offset is past 2^31 and 2^32."""
    dims = dims_of(8, 8, 128)
    pages = 2 ** 32 // (8 * 16 * 128) + 4
    k, v = (torch.empty((pages, 8, 16, 128), dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.empty((pages, 8, 16), dtype=torch.uint8, device="cuda") for _ in range(2))
    hp, q, cache, table = batch(dims, [100], [(60, 20)], 1 + 40, 40, seed=31)
    moved = np.full_like(hp.block_table, -1)
    ids = [0, pages - 1, pages // 2 + 3, pages - 7, 5, pages // 2 - 1, pages - 20, 17, pages // 4, pages - 31, pages // 3,
           pages - 100]
    for s in range(hp.n_seqs):
        for i in range(-(-int(hp.seq_kv_len[s]) // 16)):
            moved[s, i] = at = ids.pop()
            for big, small in zip((k, ks, v, vs), cache):
                big[at] = small[table[s][i]].cuda()
    want = attend(hp, q, cache, dims)
    hp.block_table[:] = moved
    got = attend(hp, q, [k, ks, v, vs], dims)
    hb.hb_check_status()
    assert torch.equal(got, want)


@pytest.mark.parametrize("n_q,n_kv,d", [(40, 8, 128), (12, 4, 64)])
@pytest.mark.parametrize("prefills,chunk", [([(10000, 9994), (2000, 0)], 2000), ([(2000, 0), (9300, 9300 - 128)], 2000)])
def test_attention_records_of_a_short_chunk_beside_a_long_one(n_q, n_kv, d, prefills, chunk):
    """More rows than sequences of split keys can have: the records go by the
    place in the sequence and not in the plan."""
    dims = dims_of(n_q, n_kv, d)
    rows = sum(min(chunk, n - done) for n, done in prefills)
    hp = check(dims, [], prefills, rows, chunk, seed=n_q)
    assert hp.n_rows == rows
    hp, q, cache, _ = batch(dims, [], prefills, rows, chunk, n_q)
    out = attend(hp, q, cache, dims)
    for s in range(hp.n_seqs):
        r0, r1 = hp.seq_q_start[s], hp.seq_q_start[s + 1]
        assert torch.equal(attend(_alone(hp, s), q[r0:r1].contiguous(), cache, dims, max_kv=12000), out[r0:r1]), s
    hb.hb_check_status()


@pytest.mark.parametrize("n_q,n_kv,d", [(8, 2, 128), (12, 4, 64)])
@pytest.mark.parametrize("dec_ctx,prefills,tau,chunk,pad", [([0], [], 1, 1, 7), ([700], [], 1, 1, 1),
                                                            ([9000], [], 1, 1, 300), ([], [(900, 300)], 130, 130, 62),
                                                            ([], [(9000, 8990)], 10, 10, 6), ([5, 700], [], 2, 1, 6),
                                                            ([40], [(900, 300)], 131, 130, 5)])
def test_attention_rows_behind_the_last_sequence(n_q, n_kv, d, dec_ctx, prefills, tau, chunk, pad):
    """A plan with more rows than its sequences have, one row of one sequence
    among them: the sequences' rows as ever, the others as they were."""
    dims = dims_of(n_q, n_kv, d)
    hp, q, cache, table = batch(dims, dec_ctx, prefills, tau, chunk, seed=pad + n_q)
    n = hp.n_rows
    dp = hb.DevicePlan(hp)
    dp.n_rows = n + pad
    q = torch.cat([q, torch.full((pad, n_q, d), math.nan, dtype=BF, device="cuda")])
    out = torch.full((n + pad, n_q * d), 7.0, dtype=BF, device="cuda")
    ws = wd.workspace(hb.hb_attention_e4m3_workspace_bytes(dims, n + pad, hp.n_seqs, 9500))
    hb.hb_attention_e4m3(q, *[t.cuda() for t in cache], dp, dims, 9500, out, ws)
    hb.hb_check_status()
    want, bound = ec.attention(q[:n].cpu(), *cache, table, hp.seq_q_start.tolist(), hp.seq_kv_len.tolist())
    assert ((out[:n].cpu().double() - want).abs() <= bound).all()
    assert (out[n:] == 7).all()
    if hp.n_seqs > 1 or n > 1:
        assert torch.equal(out[:n], attend(hp, q[:n].contiguous(), cache, dims, max_kv=9500))


@pytest.mark.parametrize("normed", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_append_keys_that_are_not_finite(d, normed):
    """A NaN, an infinity, or a rotation that passes fp32's range: byte 255 and
    NaN codes throughout that head's key; its row's other heads and the other
    rows as without it."""
    dims, rows = dims_of(2, 2, d), 6
    g = wd.device_generator(d)
    clean = wd.randn_bf16((rows, 6, d), g)
    qkv = clean.clone()
    qkv[1, 2, 3] = math.nan
    qkv[2, 3, d - 1] = math.inf
    qkv[3, 2, 0] = -math.inf
    if not normed:
        qkv[4, 3] = 3.38e38  # 3.38e38 (|cos| + |sin|) is past 3.40e38 at any angle off the axes
    pos = torch.tensor([7, 0, 5, 31, 11, 2], dtype=torch.int32, device="cuda")
    slots = torch.tensor([3, 17, 0, 9, 30, 5], dtype=torch.int32, device="cuda")
    gains = [(1 + 0.3 * torch.randn(d, generator=g, device="cuda")).to(BF) for _ in range(2)] if normed else (None, None)
    rope = wd.rope_table_device(32, dims)
    q, cache = append(qkv.view(rows, -1), pos, slots, dims, 2, rope, 32, gains)
    want_q, want = append(clean.view(rows, -1), pos, slots, dims, 2, rope, 32, gains)
    hb.hb_check_status()
    assert torch.equal(q, want_q) and torch.equal(cache[2], want[2]) and torch.equal(cache[3], want[3])
    for r, h in ((1, 0), (2, 1), (3, 0)) + (() if normed else ((4, 1),)):
        page, off = int(slots[r]) // 16, int(slots[r]) % 16
        assert cache[1][page, h, off] == 255 and (cache[0][page, h, off] == 0x7f).all(), (r, h)
        want[1][page, h, off], want[0][page, h, off] = 255, 0x7f
    assert torch.equal(cache[0], want[0]) and torch.equal(cache[1], want[1])
