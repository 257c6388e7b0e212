"""A small model served from the single calls with an E4M3 cache (GPU): chunked
prompts beside decodes over several iterations, the residual stream added and
normed into the projections' operands, tokens chosen and prompts scored by
hb_logprobs.  Every call is checked in 64 bits against the operands that it
really got; then the whole stream of calls is enqueued without a wait in
between, and captured, and has to give the same bits."""
import math

import numpy as np
import pytest

import workloads as wl
from workloads import device as wd

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import e4m3_cache as ec  # noqa: E402
from test_gpu_add_norm import EPS, check as check_norm  # noqa: E402
from test_gpu_logprobs import check as check_logprobs  # noqa: E402

import chunked_prefill_hybrid_tau_gb300 as hb  # noqa: E402
from chunked_prefill_hybrid_tau_gb300 import _lib as L  # noqa: E402

BF = torch.bfloat16
VOCAB, MAX_POS, PAGES, TAU, CHUNK = 1024, 1024, 80, 96, 90
DIMS = wl.Dims(d_model=256, n_q=6, n_kv=2, d_head=64, d_ff=384)
PROMPTS, NEW = [1, 45, 130, 300], [9, 6, 4, 3]  # prompt lengths, new tokens


class Model:
    def __init__(self, layers=2):
        g = wd.device_generator(12)
        d, f, qkv = DIMS.d_model, DIMS.d_ff, (DIMS.n_q + 2 * DIMS.n_kv) * DIMS.d_head

        def gain(n):
            return (1 + 0.3 * torch.randn(n, generator=g, device="cuda")).to(BF)

        def weight(*shape):
            return wd.randn_bf16(shape, g, 1 / math.sqrt(shape[1]))

        self.rope = wd.rope_table_device(MAX_POS, DIMS)
        self.emb, self.lm, self.g_f = wd.randn_bf16((VOCAB, d), g), weight(VOCAB, d), gain(d)
        self.layers = []
        for _ in range(layers):
            gu = torch.empty((2 * f, d), dtype=BF, device="cuda")
            hb.hb_interleave_gate_up(weight(f, d), weight(f, d), gu)
            self.layers.append(dict(
                g1=gain(d), g2=gain(d), g_q=gain(DIMS.d_head), g_k=gain(DIMS.d_head),
                qkv=hb.hb_quantize_e4m3_block(weight(qkv, d), block_rows=128), o=weight(d, DIMS.n_q * DIMS.d_head),
                gu=hb.hb_quantize_e4m3(gu), down=weight(d, f)))

    def cache(self):
        """Pools whose every byte stands for NaN until it is written."""
        return [[torch.full(s, b, dtype=torch.uint8, device="cuda") for s, b in
                 (((PAGES, DIMS.n_kv, 16, DIMS.d_head), 0x7f), ((PAGES, DIMS.n_kv, 16), 255)) * 2] for _ in self.layers]

    def forward(self, ids, next_ids, dp, cache, max_kv, buf, after=lambda name, **kw: None):
        """Enqueues one iteration on the current stream; `after` sees each call's operands."""
        torch.index_select(self.emb, 0, ids, out=buf["x"])
        x, mlp = buf["x"], None
        for n, (w, c) in enumerate(zip(self.layers, cache)):
            before = x.clone()
            if n == 0:
                hb.hb_add_rmsnorm(x, None, w["g1"], EPS, None, buf["c1"], buf["s1"], fmt="e4m3_block")
            else:
                hb.hb_add_rmsnorm(mlp, x, w["g1"], EPS, x, buf["c1"], buf["s1"], fmt="e4m3_block")
            after("norm", x=before if n == 0 else mlp, r=None if n == 0 else before, h=x, gamma=w["g1"],
                  fmt="e4m3_block", y=buf["c1"], scale=buf["s1"])
            hb.hb_gemm_e4m3_block(buf["c1"], buf["s1"], *w["qkv"], buf["qkv"])
            hb.hb_kv_append_e4m3(buf["qkv"], dp.field("row_pos"), dp.field("slot_mapping"), self.rope, MAX_POS, DIMS,
                                 buf["q"], *c, w["g_q"], w["g_k"])
            after("append", w=w, cache=c, qkv=buf["qkv"])
            hb.hb_attention_e4m3(buf["q"], *c, dp, DIMS, max_kv, buf["o"], buf["ws"])
            after("attention", cache=c, q=buf["q"], out=buf["o"])
            hb.hb_gemm(buf["o"], w["o"], buf["proj"])
            before = x.clone()
            hb.hb_add_rmsnorm(buf["proj"], x, w["g2"], EPS, x, buf["c2"], buf["s2"], fmt="e4m3")
            after("norm", x=buf["proj"], r=before, h=x, gamma=w["g2"], fmt="e4m3", y=buf["c2"], scale=buf["s2"])
            hb.hb_gemm_e4m3(buf["c2"], buf["s2"], *w["gu"], buf["act"], epilogue=L.HB_EPI_SWIGLU)
            mlp = buf["mlp"]
            last = n + 1 == len(self.layers)
            hb.hb_gemm(buf["act"], w["down"], x if last else mlp, x if last else None,
                       L.HB_EPI_RESIDUAL if last else L.HB_EPI_STORE)
        hb.hb_final_logits(x, buf["rows"], self.g_f, self.lm, buf["logits"], buf["lws"], EPS)
        hb.hb_logprobs(buf["logits"], next_ids, buf["lp"], buf["ent"], buf["ids"], buf["top"])
        after("logprobs")

    def buffers(self, T, n_seqs, max_kv):
        d, dev = DIMS.d_model, dict(device="cuda")

        def bf(*s):
            return torch.full(s, math.nan, dtype=BF, **dev)

        def f32(*s):
            return torch.full(s, math.nan, dtype=torch.float32, **dev)

        return dict(
            x=bf(T, d), c1=torch.full((T, d), 0x7f, dtype=torch.uint8, **dev), s1=f32(T, 2),
            c2=torch.full((T, d), 0x7f, dtype=torch.uint8, **dev), s2=f32(T),
            qkv=bf(T, (DIMS.n_q + 2 * DIMS.n_kv) * DIMS.d_head), q=bf(T, DIMS.n_q, DIMS.d_head),
            o=bf(T, DIMS.n_q * DIMS.d_head), proj=bf(T, d), act=bf(T, DIMS.d_ff), mlp=bf(T, d),
            ws=wd.workspace(hb.hb_attention_e4m3_workspace_bytes(DIMS, T, n_seqs, max_kv)).fill_(0xFF),
            rows=torch.arange(T, dtype=torch.int32, **dev), logits=f32(T, VOCAB), lws=wd.workspace(T * d * 2),
            lp=f32(T, 1), ent=f32(T), ids=torch.full((T, 4), -7, dtype=torch.int32, **dev), top=f32(T, 4))


def iterations(model, run):
    """Serves PROMPTS with the scheduler; run(ids, next_ids, dp, hp, cache) -> top ids of every row."""
    rng = np.random.default_rng(8)
    text = [list(rng.integers(0, VOCAB, n)) for n in PROMPTS]
    sched, cache, count = hb.Scheduler(TAU, CHUNK, list(rng.permutation(PAGES))), model.cache(), 0
    for n, new in zip(PROMPTS, NEW):
        sched.add(n, new)
    while sched.active():
        hp, req = sched.plan()
        ids = torch.tensor([text[r][p] for r, p in zip(req, hp.row_pos)], dtype=torch.int32, device="cuda")
        nxt = torch.tensor([text[r][p + 1] if p + 1 < PROMPTS[r] else -1 for r, p in zip(req, hp.row_pos)],
                           dtype=torch.int32, device="cuda")
        top = run(ids, nxt[:, None], hb.DevicePlan(hp), hp, cache)
        for s in range(hp.n_seqs):
            row = hp.seq_q_start[s + 1] - 1
            if hp.seq_kv_len[s] >= PROMPTS[req[row]]:
                text[req[row]].append(int(top[row, 0]))
        sched.commit()
        count += 1
    assert sched.free_pages() == PAGES and count > 6
    assert [len(t) for t in text] == [p + n for p, n in zip(PROMPTS, NEW)]
    return text, cache


def test_a_model_served_from_the_calls():
    model, mixed = Model(), []
    kept = {}

    def checked(ids, nxt, dp, hp, cache):
        T, max_kv = hp.n_rows, int(hp.seq_kv_len.max())
        buf = model.buffers(T, hp.n_seqs, max_kv)
        table, start, kv = hp.block_table.tolist(), hp.seq_q_start.tolist(), hp.seq_kv_len.tolist()
        slots = torch.tensor(hp.slot_mapping).long()
        mixed.append((hp.seq_kind == 0).any() and (hp.seq_kind == 1).any())

        def after(name, **a):
            torch.cuda.synchronize()
            if name == "norm":
                h = check_norm(a["x"], a["r"], a["gamma"], a["fmt"], a["y"], a["scale"])
                assert torch.equal(h, a["h"])
            elif name == "append":
                kc, ks, vc, vs = a["cache"]
                x = a["qkv"].cpu().double().view(T, -1, DIMS.d_head)
                codes, e = ec.quantize(x[:, DIMS.n_q + DIMS.n_kv:])
                assert torch.equal(vc.cpu()[slots // 16, :, slots % 16], codes)
                assert torch.equal(vs.cpu()[slots // 16, :, slots % 16], e)
                key = x[:, DIMS.n_q:DIMS.n_q + DIMS.n_kv]
                key = key / torch.sqrt(key.square().mean(-1, keepdim=True) + DIMS.eps) * a["w"]["g_k"].cpu().double()
                turn = model.rope.cpu().double()[torch.tensor(hp.row_pos).long()][:, None]
                u, v, cos, sin = key[..., :32], key[..., 32:], turn[..., 0], turn[..., 1]
                err = (32 + 16) * 2.0 ** -24 * torch.cat([u.abs() + v.abs()] * 2, -1)
                key = torch.cat([u * cos - v * sin, v * cos + u * sin], -1)
                p = ec.powers(ks.cpu()[slots // 16, :, slots % 16])[..., None]
                got = ec.values(kc.cpu()[slots // 16, :, slots % 16]) * p
                room = ec.HALF_E4M3 * key.abs() + ec.HALF_SUB * p + err * (1 + ec.HALF_E4M3)
                assert ((got - key).abs() <= room).all()
            elif name == "attention":
                want, bound = ec.attention(a["q"].cpu(), *[t.cpu() for t in a["cache"]], table, start, kv)
                assert ((a["out"].cpu().double() - want).abs() <= bound).all()
            else:
                known = nxt[:, 0] >= 0
                check_logprobs(buf["logits"][known], nxt[known], *[buf[k][known] for k in ("lp", "ent", "ids", "top")])
                check_logprobs(buf["logits"][~known], torch.zeros_like(nxt[~known]),
                               torch.log_softmax(buf["logits"][~known].double(), 1)[:, :1].float(),
                               *[buf[k][~known] for k in ("ent", "ids", "top")])

        model.forward(ids, nxt, dp, cache, max_kv, buf, after)
        kept[len(kept)] = {k: buf[k].clone() for k in ("x", "lp", "ent", "ids", "top")}
        return buf["ids"]

    text, cache = iterations(model, checked)
    hb.hb_check_status()
    assert any(mixed)

    def same(buf, at):
        for k, t in kept[at].items():
            assert torch.equal(buf[k].view(torch.uint8), t.view(torch.uint8)), (at, k)

    for captured in (False, True):
        at = [0]

        def run(ids, nxt, dp, hp, cache):
            max_kv = int(hp.seq_kv_len.max())
            buf = model.buffers(hp.n_rows, hp.n_seqs, max_kv)
            if captured:
                torch.cuda.synchronize()
                g = torch.cuda.CUDAGraph()
                with torch.cuda.graph(g):
                    model.forward(ids, nxt, dp, cache, max_kv, buf)
                g.replay()
                g.replay()  # writes the same tokens' keys and values again
            else:
                model.forward(ids, nxt, dp, cache, max_kv, buf)
            torch.cuda.synchronize()
            same(buf, at[0])
            at[0] += 1
            return buf["ids"]

        again, cache2 = iterations(model, run)
        hb.hb_check_status()
        assert again == text
        assert all(torch.equal(a, b) for ca, cb in zip(cache, cache2) for a, b in zip(ca, cb))
