"""Measured cases of serving operators around the decoder layer:

  append    rotary positions and the paged K/V write into an E4M3 cache: codes
            with a power-of-two scale per token and kv head
  attend    paged attention of decode rows and prompt chunks over that cache
  norm      residual addition and RMS norm in one pass, with the result in
            bf16 or as E4M3 codes with scales
  logprobs  log probabilities of given tokens, the entropy and the best
            alternatives of every row of logits

A case is a dict; prepare() makes its inputs on the GPU from the seed, run()
is one pass (own: through the library; else in elementary torch operations in
32 bits), exact() the definition in 64 bits.
"""
import math
import types

import torch

own = False

PAGE = 16
BLOCK = 128
E4M3_MAX = 448.0
EPS = 1e-6
AMAX_MIN = 2.0 ** -112  # smallest maximum that the scale of 128 columns is formed from
MIN_EXP = -100          # smallest exponent of a cached vector's scale


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one decode token of a model with normed query and key heads
        dict(name="append_1_row", kind="append", rows=1, decodes=1, n_q=32, n_kv=8, d_head=128, theta=1e6,
             max_pos=32768, pad=0, normed=True),
        # a long prompt in one piece on the widest heads of the workloads
        dict(name="append_prompt_8192", kind="append", rows=8192, decodes=0, n_q=56, n_kv=8, d_head=128, theta=5e6,
             max_pos=32768, pad=0, normed=False),
        # the tiny layer's iteration: a 64-token chunk behind 128 cached tokens and four decodes
        dict(name="attend_tiny_68", kind="attend", n_q=4, n_kv=2, d_head=64, decodes=4, ctx_lo=33, ctx_hi=201,
             chunks=1, chunk=64, prefix_lo=128, prefix_hi=128),
        # one user with a long context: a single row, where latency counts
        dict(name="attend_decode_1x32k", kind="attend", n_q=32, n_kv=8, d_head=128, decodes=1, ctx_lo=32761,
             ctx_hi=32761, chunks=0, chunk=0, prefix_lo=0, prefix_hi=0),
        # a decode-only iteration of a full batch, contexts of ragged lengths
        dict(name="attend_decode_64", kind="attend", n_q=32, n_kv=8, d_head=128, decodes=64, ctx_lo=513,
             ctx_hi=8189, chunks=0, chunk=0, prefix_lo=0, prefix_hi=0),
        # the hybrid iteration of the benchmark: 32 decodes and a 480-token chunk behind 1024 cached tokens
        dict(name="attend_hybrid_512", kind="attend", n_q=32, n_kv=8, d_head=128, decodes=32, ctx_lo=513,
             ctx_hi=4097, chunks=1, chunk=480, prefix_lo=1024, prefix_hi=1024),
        # a late chunk of a long prompt on the widest heads of the workloads
        dict(name="attend_prompt_2048", kind="attend", n_q=56, n_kv=8, d_head=128, decodes=0, ctx_lo=0, ctx_hi=0,
             chunks=1, chunk=2048, prefix_lo=14336, prefix_hi=14336),
        # one decode token's hidden row, codes for a block-scaled projection
        dict(name="norm_1x4096_block", kind="norm", rows=1, d=4096, fmt="e4m3_block"),
        # a long prompt's hidden rows, codes with a scale per row
        dict(name="norm_8192x7168_rows", kind="norm", rows=8192, d=7168, fmt="e4m3"),
        # the sampled token of one request and its twenty best alternatives
        dict(name="logprobs_1x32000", kind="logprobs", rows=1, vocab=32000, extra=0, masked=0.0, dtype="f32", given=1, top=20),
        # the rows of an iteration's LM head: 64 decodes and a prompt's last row
        dict(name="logprobs_65x32000", kind="logprobs", rows=65, vocab=32000, extra=0, masked=0.0, dtype="f32", given=1, top=5),
        # every position of a prompt scored, logits in bf16
        dict(name="logprobs_2048x64000", kind="logprobs", rows=2048, vocab=64000, extra=0, masked=0.0, dtype="bf16",
             given=2, top=8),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


HEADS = [(32, 8, 128), (56, 8, 128), (4, 2, 64), (8, 8, 64), (16, 1, 128), (12, 4, 64), (8, 8, 128), (40, 8, 128),
         (32, 8, 64)]


def draw(rng):
    kind = rng.choice(["append", "attend", "attend", "norm", "logprobs"])
    if kind == "append":
        n_q, n_kv, d_head = rng.choice(HEADS)
        rows = _log_int(rng, 1, 8192)
        return dict(kind="append", rows=rows, decodes=rng.randint(0, min(rows, 64)), n_q=n_q, n_kv=n_kv,
                    d_head=d_head, theta=rng.choice([1e4, 1e6, 5e6]), max_pos=rng.choice([8192, 16384, 32768]),
                    pad=rng.randint(0, min(rows - 1, 7)), normed=rng.random() < 0.5)
    if kind == "attend":
        n_q, n_kv, d_head = rng.choice(HEADS)
        decodes = _log_int(rng, 1, 64) if rng.random() < 0.7 else 0
        chunks = rng.randint(0 if decodes else 1, 2)
        chunk = _log_int(rng, 2, 1024) if chunks else 0
        ctx_hi = _log_int(rng, 1, 32768 if decodes <= 8 else 8192) if decodes else 0
        prefix_hi = _log_int(rng, 1, 14336) - 1 if chunks else 0
        return dict(kind="attend", n_q=n_q, n_kv=n_kv, d_head=d_head, decodes=decodes,
                    ctx_lo=rng.randint(1, ctx_hi) if decodes else 0, ctx_hi=ctx_hi, chunks=chunks, chunk=chunk,
                    prefix_lo=rng.randint(0, prefix_hi) if chunks else 0, prefix_hi=prefix_hi)
    if kind == "norm":
        fmt = rng.choice(["bf16", "e4m3", "e4m3_block"])
        d = 16 * _log_int(rng, 4, 1024)
        return dict(kind="norm", rows=_log_int(rng, 1, 8192 * 7168 // max(d, 7168)), d=d, fmt=fmt)
    vocab = _log_int(rng, 64, 152001)
    return dict(kind="logprobs", rows=_log_int(rng, 1, min(2048, 2048 * 64000 // vocab)), vocab=vocab,
                extra=rng.choice([0, 0, 3, 64]), masked=rng.choice([0.0, 0.0, 0.9]), dtype=rng.choice(["f32", "bf16"]),
                given=rng.randint(0, 4), top=rng.randint(0, 32))


def _spread(lo, hi, n):
    """n lengths from lo to hi, evenly."""
    return [hi if n == 1 else lo + (hi - lo) * i // (n - 1) for i in range(n)]


def _lengths(case):
    """(keys of every decode row, keys ahead of every chunk)."""
    return (_spread(case["ctx_lo"], case["ctx_hi"], case["decodes"]),
            _spread(case["prefix_lo"], case["prefix_hi"], case["chunks"]))


def _groups(n):
    return -(-n // BLOCK)


def work(case):
    if case["kind"] == "append":
        t, h, dh = case["rows"], case["n_q"] + 2 * case["n_kv"], case["d_head"]
        kv = 2 * (t - case["pad"]) * case["n_kv"] * (dh + 1)
        read = t * h * dh * 2 + min(t, case["max_pos"]) * dh * 4 + 8 * t + (4 * dh if case["normed"] else 0)
        return {"bytes": read + t * case["n_q"] * dh * 2 + kv, "flops": (7 * t * (case["n_q"] + case["n_kv"]) + 3 * t *
                                                                         2 * case["n_kv"]) * dh}
    if case["kind"] == "attend":
        ctx, prefix = _lengths(case)
        c, n_q, n_kv, dh = case["chunk"], case["n_q"], case["n_kv"], case["d_head"]
        keys = sum(ctx) + sum(p + c for p in prefix)
        pairs = sum(ctx) + sum(p * c + c * (c + 1) // 2 for p in prefix)
        rows = len(ctx) + c * len(prefix)
        return {"bytes": 2 * keys * n_kv * (dh + 1) + 4 * rows * n_q * dh + 4 * (-(-keys // PAGE)),
                "flops": 4 * pairs * n_q * dh}
    if case["kind"] == "norm":
        n = case["rows"] * case["d"]
        groups = case["rows"] * {"bf16": 0, "e4m3": 1, "e4m3_block": _groups(case["d"])}[case["fmt"]]
        return {"bytes": 6 * n + n * (2 if case["fmt"] == "bf16" else 1) + 4 * groups + 2 * case["d"], "flops": 6 * n}
    n = case["rows"] * case["vocab"]
    return {"bytes": n * (4 if case["dtype"] == "f32" else 2) + case["rows"] * (8 * case["given"] + 4 + 8 * case["top"]),
            "flops": 6 * n}


# ------------------------------------------------------------------ the inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(shape, g, scale=1.0):
    return torch.randn(shape, generator=g, device="cuda") * scale


def _ints(lo, hi, shape, g):
    return torch.randint(lo, hi, shape, generator=g, device="cuda")


def _power(e):
    """2^e in fp32 for whole exponents e of -126 to 127."""
    return ((e + 127) << 23).view(torch.float32)


def _quantize_vectors(y):
    """fp32 vectors (last axis) -> (E4M3 codes, exponent bytes): the scale is
    the smallest power of two, 2^-100 at least, that takes the vector's
    largest magnitude to at most 448; byte 255 where that magnitude is not
    finite."""
    amax = y.abs().amax(-1)
    m, ex = torch.frexp(amax)
    finite = torch.isfinite(amax)
    e = (ex.int() - 9 + (m > 0.875).int()).clamp(min=MIN_EXP)
    e = torch.where(finite, e, torch.zeros_like(e))
    codes = (y * _power(-e)[..., None]).clamp(-E4M3_MAX, E4M3_MAX)
    codes = torch.where(finite[..., None], codes, torch.full_like(codes, math.nan)).to(torch.float8_e4m3fn)
    return codes, torch.where(finite, e + 127, torch.full_like(e, 255)).to(torch.uint8)


def _dims(case):
    n_q, dh = case["n_q"], case["d_head"]
    return types.SimpleNamespace(d_model=n_q * dh, n_q=n_q, n_kv=case["n_kv"], d_head=dh, d_ff=64, page=PAGE, eps=EPS,
                                 theta=case.get("theta", 1e4))


def prepare(case, seed):
    g = _gen(seed)
    return {"append": _prepare_append, "attend": _prepare_attend, "norm": _prepare_norm,
            "logprobs": _prepare_logprobs}[case["kind"]](case, g)


def _pools(pages, n_kv, dh, g):
    """Codes and scale bytes of cached keys and values, channels of different size."""
    out = []
    for _ in range(2):
        x = _randn((pages, n_kv, PAGE, dh), g) * torch.exp(_randn((1, n_kv, 1, dh), g, 0.3))
        codes, scale = _quantize_vectors(x)
        out += [codes.view(torch.uint8), scale]
    return out


def _prepare_append(case, g):
    t, n_dec, n_q, n_kv, dh = case["rows"], case["decodes"], case["n_q"], case["n_kv"], case["d_head"]
    max_pos, half = case["max_pos"], case["d_head"] // 2
    chunk = t - n_dec
    chunk_pages = -(-chunk // PAGE)
    num_pages = chunk_pages + n_dec + 4
    # decode rows: one new token each, anywhere in its context; then the chunk's rows in order
    dec_pos = _ints(0, max_pos, (n_dec,), g)
    start = _ints(0, max(1, (max_pos - chunk) // PAGE), (1,), g) * PAGE
    pos = torch.cat([dec_pos, start + torch.arange(chunk, device="cuda")]).to(torch.int32)
    pages = torch.randperm(num_pages, generator=g, device="cuda")
    i = torch.arange(chunk, device="cuda")
    slots = torch.cat([pages[:n_dec] * PAGE + dec_pos % PAGE, pages[n_dec + i // PAGE] * PAGE + i % PAGE])
    slots = slots.to(torch.int32)
    if case["pad"]:
        slots[t - case["pad"]:] = -1
    ang = torch.arange(max_pos, dtype=torch.float64, device="cuda")[:, None] * \
        case["theta"] ** (-2.0 * torch.arange(half, dtype=torch.float64, device="cuda") / dh)[None, :]
    rope = torch.stack([ang.cos(), ang.sin()], -1).float().contiguous()
    heads = n_q + 2 * n_kv
    # projections of a trained layer: heads of different size
    qkv = (_randn((t, heads, dh), g) * torch.exp(_randn((1, heads, 1), g))).to(torch.bfloat16).view(t, heads * dh)
    g_q = (1 + _randn((dh,), g, 0.2)).to(torch.bfloat16) if case["normed"] else None
    g_k = (1 + _randn((dh,), g, 0.2)).to(torch.bfloat16) if case["normed"] else None
    k, ks, v, vs = _pools(num_pages, n_kv, dh, g)
    q_out = torch.empty((t, n_q, dh), dtype=torch.bfloat16, device="cuda")
    return dict(case=case, qkv=qkv, pos=pos, slots=slots, rope=rope, g_q=g_q, g_k=g_k, k=k, ks=ks, v=v, vs=vs,
                q_out=q_out, dims=_dims(case))


class _Plan:
    """A device plan as a program keeps one: the plan's arrays on the GPU and its sizes."""

    def __init__(self, arrays, n_rows, n_seqs, max_pages, hints):
        self.arrays, self.sizes, self.hints = arrays, (n_rows, n_seqs, max_pages), hints
        self.n_rows, self.n_seqs, self.max_pages = self.sizes

    def struct(self):
        from chunked_prefill_hybrid_tau_gb300 import _lib
        return _lib.hb_device_plan(*self.sizes, *(a.data_ptr() for a in self.arrays), *self.hints)


def _prepare_attend(case, g):
    n_q, n_kv, dh, c = case["n_q"], case["n_kv"], case["d_head"], case["chunk"]
    ctx, prefix = _lengths(case)
    kv_len = ctx + [p + c for p in prefix]
    qlen = [1] * len(ctx) + [c] * len(prefix)
    rows, n_seqs, max_kv = sum(qlen), len(qlen), max(kv_len)
    max_pages = -(-max_kv // PAGE)
    need = [-(-n // PAGE) for n in kv_len]
    num_pages = sum(need) + 3
    k, ks, v, vs = _pools(num_pages, n_kv, dh, g)
    order = torch.randperm(num_pages, generator=g, device="cuda").to(torch.int32)
    first = torch.tensor([0] + need, device="cuda").cumsum(0)[:-1]
    n_pages = torch.tensor(need, device="cuda")
    col = torch.arange(max_pages, device="cuda")[None]
    table = torch.where(col < n_pages[:, None], order[(first[:, None] + col).clamp(max=num_pages - 1)], -1)
    table = table.to(torch.int32).contiguous()
    kv = torch.tensor(kv_len, dtype=torch.int32, device="cuda")
    start = torch.tensor([0] + qlen, device="cuda").cumsum(0).to(torch.int32)
    seq = torch.arange(n_seqs, device="cuda").repeat_interleave(torch.tensor(qlen, device="cuda"))
    pos = (kv[seq] - start[seq + 1] + torch.arange(rows, device="cuda")).to(torch.int32)
    slots = table[seq, (pos // PAGE).long()] * PAGE + pos % PAGE
    pairs = sum(p * c + c * (c + 1) // 2 for p in prefix)
    plan = _Plan([pos, slots.to(torch.int32), start, kv, table], rows, n_seqs, max_pages,
                 (sum(ctx) + (pairs if c == 1 else 0), 0 if c == 1 else pairs, 0 if c == 1 else c * len(prefix)))
    q = _randn((rows, n_q, dh), g).to(torch.bfloat16)
    out = torch.empty((rows, n_q * dh), dtype=torch.bfloat16, device="cuda")
    return dict(case=case, q=q, k=k, ks=ks, v=v, vs=vs, pos=pos, table=table, plan=plan, max_kv=max_kv, out=out,
                dims=_dims(case))


def _prepare_norm(case, g):
    rows, d = case["rows"], case["d"]
    # hidden rows with channels of different size, and the branch that is added to them
    size = torch.exp(_randn((1, d), g, 0.7))
    x = (_randn((rows, d), g) * size).to(torch.bfloat16)
    r = (_randn((rows, d), g) * size * 2).to(torch.bfloat16)
    gamma = (1 + _randn((d,), g, 0.2)).to(torch.bfloat16)
    bf16 = case["fmt"] == "bf16"
    y = torch.empty((rows, d), dtype=torch.bfloat16 if bf16 else torch.uint8, device="cuda")
    groups = (rows,) if case["fmt"] == "e4m3" else (rows, _groups(d))
    scale = None if bf16 else torch.empty(groups, dtype=torch.float32, device="cuda")
    return dict(case=case, x=x, r=r, gamma=gamma, h=torch.empty_like(x), y=y, scale=scale)


def _prepare_logprobs(case, g):
    rows, vocab, given, top = case["rows"], case["vocab"], case["given"], min(case["top"], case["vocab"])
    dtype = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
    # a wide bulk and a few likely tokens; rows of a buffer whose columns may be padded
    full = torch.zeros((rows, vocab + case["extra"]), dtype=dtype, device="cuda")
    logits = full[:, :vocab]
    logits.copy_(_randn((rows, vocab), g, 2.5))
    likely = _ints(0, vocab, (rows, 8), g)
    logits.scatter_add_(1, likely, (6 + 4 * torch.rand((rows, 8), generator=g, device="cuda")).to(dtype))
    if case["masked"]:  # a grammar's mask: tokens that must not come are at -infinity
        logits.masked_fill_(torch.rand((rows, vocab), generator=g, device="cuda") < case["masked"], -math.inf)
        logits[:, 0] = 1.0
    tokens = torch.where(torch.rand((rows, given), generator=g, device="cuda") < 0.7,
                         likely[:, :given], _ints(0, vocab, (rows, given), g)).to(torch.int32)
    f32 = dict(dtype=torch.float32, device="cuda")
    return dict(case=case, logits=logits, tokens=tokens, lp=torch.empty((rows, given), **f32),
                entropy=torch.empty(rows, **f32), ids=torch.empty((rows, top), dtype=torch.int32, device="cuda"),
                top_lp=torch.empty((rows, top), **f32))


# ------------------------------------------------------------------ one pass
def run(state):
    kind = state["case"]["kind"]
    if own:
        return _run_own(kind, state)
    return {"append": _plain_append, "attend": _plain_attend, "norm": _plain_norm, "logprobs": _plain_logprobs}[kind](
        state)


def _run_own(kind, s):
    import chunked_prefill_hybrid_tau_gb300 as hb
    if kind == "append":
        hb.hb_kv_append_e4m3(s["qkv"], s["pos"], s["slots"], s["rope"], s["case"]["max_pos"], s["dims"], s["q_out"],
                             s["k"], s["ks"], s["v"], s["vs"], s["g_q"], s["g_k"])
        return _cached(s["q_out"], s)
    if kind == "attend":
        plan = s["plan"]
        if "ws" not in s:  # the workspace that a program keeps
            s["ws"] = torch.empty(hb.hb_attention_e4m3_workspace_bytes(s["dims"], plan.n_rows, plan.n_seqs, s["max_kv"]),
                                  dtype=torch.uint8, device="cuda")
        hb.hb_attention_e4m3(s["q"], s["k"], s["ks"], s["v"], s["vs"], plan, s["dims"], s["max_kv"], s["out"], s["ws"])
        return s["out"]
    if kind == "norm":
        hb.hb_add_rmsnorm(s["x"], s["r"], s["gamma"], EPS, s["h"], s["y"], s["scale"], fmt=s["case"]["fmt"])
        if s["scale"] is None:
            return s["h"], s["y"]
        return s["h"], s["y"].view(torch.float8_e4m3fn), s["scale"]
    hb.hb_logprobs(s["logits"], s["tokens"], s["lp"], s["entropy"], s["ids"], s["top_lp"])
    return s["lp"], s["entropy"], s["ids"], s["top_lp"]


def _cached(q, s):
    """What the append leaves: q, and the pools as the values that codes and scales stand for."""
    return (q, s["k"].view(torch.float8_e4m3fn), s["ks"].view(torch.float8_e8m0fnu), s["v"].view(torch.float8_e4m3fn),
            s["vs"].view(torch.float8_e8m0fnu))


def _plain_append(s):
    c = s["case"]
    t, n_q, n_kv, dh = c["rows"], c["n_q"], c["n_kv"], c["d_head"]
    x = s["qkv"].view(t, n_q + 2 * n_kv, dh)

    def rotate(h, gain):
        h = h.float()
        if gain is not None:
            h = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS) * gain.float()
        cs = s["rope"][s["pos"].long()][:, None]
        a, b, cos, sin = h[..., :dh // 2], h[..., dh // 2:], cs[..., 0], cs[..., 1]
        return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)

    q = rotate(x[:, :n_q], s["g_q"]).to(torch.bfloat16)
    kept = t - c["pad"]
    page, off = s["slots"][:kept].long() // PAGE, s["slots"][:kept].long() % PAGE
    k, ks = _quantize_vectors(rotate(x[:, n_q:n_q + n_kv], s["g_k"])[:kept])
    v, vs = _quantize_vectors(x[:kept, n_q + n_kv:].float())
    s["k"][page, :, off] = k.view(torch.uint8)
    s["ks"][page, :, off] = ks
    s["v"][page, :, off] = v.view(torch.uint8)
    s["vs"][page, :, off] = vs
    return _cached(q, s)


def _plain_attend(s):
    c = s["case"]
    n_q, n_kv, dh, nd = c["n_q"], c["n_kv"], c["d_head"], c["decodes"]

    def pages(codes, scale, table):
        """[sequences][kv heads][keys][d_head] in fp32"""
        values = codes[table].view(torch.float8_e4m3fn).float() * _power(scale[table].int() - 127)[..., None]
        return values.transpose(1, 2).reshape(table.shape[0], n_kv, -1, dh)

    def attend(q, table, pos):
        """q [sequences][rows][n_q][d_head] at positions pos [sequences][rows]"""
        b, r = pos.shape
        table = table.clamp(min=0).long()
        k, v = pages(s["k"], s["ks"], table), pages(s["v"], s["vs"], table)
        q = q.float().view(b, r, n_kv, n_q // n_kv, dh).permute(0, 2, 3, 1, 4).reshape(b, n_kv, -1, dh)
        score = (q @ k.transpose(2, 3) * dh ** -0.5).view(b, n_kv, n_q // n_kv, r, -1)
        seen = torch.arange(score.shape[-1], device="cuda") <= pos[:, None, None, :, None]
        score = torch.where(seen, score, -math.inf)
        e = torch.exp(score - score.amax(-1, keepdim=True))
        o = (e.view(b, n_kv, -1, e.shape[-1]) @ v).view(*e.shape[:-1], dh) / e.sum(-1, keepdim=True)
        return o.permute(0, 3, 1, 2, 4).reshape(b * r, n_q * dh).to(torch.bfloat16)

    out = []
    if nd:
        out.append(attend(s["q"][:nd, None], s["table"][:nd], s["pos"][:nd, None]))
    if c["chunks"]:
        shape = c["chunks"], c["chunk"]
        out.append(attend(s["q"][nd:].view(*shape, n_q, dh), s["table"][nd:], s["pos"][nd:].view(shape)))
    return torch.cat(out)


def _plain_norm(s):
    h = (s["x"].float() + s["r"].float()).to(torch.bfloat16)
    y = h.float()
    y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) * s["gamma"].float()
    if s["case"]["fmt"] == "bf16":
        return h, y.to(torch.bfloat16)
    if s["case"]["fmt"] == "e4m3":
        codes, scale = _scaled(y[:, None], 0.0)
        return h, codes[:, 0], scale[:, 0]
    rows, d = y.shape
    full = torch.nn.functional.pad(y, (0, -d % BLOCK)).view(rows, -1, BLOCK)
    codes, scale = _scaled(full, AMAX_MIN)
    return h, codes.view(rows, -1)[:, :d].contiguous(), scale


def _scaled(y, smallest):
    """E4M3 codes and fp32 scales of the vectors along the last axis."""
    amax = y.abs().amax(-1)
    zero = amax == 0
    top = torch.full_like(amax, E4M3_MAX)  # tensor by tensor: a divisor that is a number would become a product
    safe = amax.clamp(min=smallest)
    inv = torch.where(zero, 0.0, top / safe)
    codes = (y * inv[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return codes, torch.where(zero, 0.0, safe / top)


def _plain_logprobs(s):
    x = s["logits"].float()
    d = x - x.amax(-1, keepdim=True)
    e = torch.exp(d)
    total = e.sum(-1)
    lse = torch.log(total)
    lp = d.gather(1, s["tokens"].long()) - lse[:, None]
    entropy = lse - torch.where(e > 0, e * d, 0.0).sum(-1) / total
    # the best logits, equal ones by the lower index: one whole number orders both
    bits = (x + 0.0).view(torch.int32)
    order = (bits ^ ((bits >> 31) & 0x7fffffff)).long() * 2 ** 32
    key = order + (2 ** 32 - 1 - torch.arange(x.shape[1], device="cuda"))
    best = torch.topk(key, s["ids"].shape[1], dim=1).values
    ids = 2 ** 32 - 1 - (best & (2 ** 32 - 1))
    return lp, entropy, ids.to(torch.int32), d.gather(1, ids) - lse[:, None]


# ------------------------------------------------------------------ 64 bits
def _e4m3_values():
    """Value of each of the 256 codes: 4 exponent bits (bias 7), 3 mantissa bits."""
    code = torch.arange(256, device="cuda")
    e, f = ((code >> 3) & 15).double(), (code & 7).double()
    mag = torch.where(e == 0, f * 2.0 ** -9, (8 + f) * torch.exp2(e - 10))
    v = torch.where(code >= 128, -mag, mag)
    v[(code & 127) == 127] = math.nan
    return v


def _e4m3_nearest(y):
    """The nearest E4M3 value, ties to the even one, at most 448."""
    mag = y.abs()
    step = torch.exp2(torch.floor(torch.log2(mag.clamp(min=2.0 ** -6))) - 3)
    return torch.copysign((torch.round(mag / step) * step).clamp(max=E4M3_MAX), y)


def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "attend": _exact_attend, "norm": _exact_norm, "logprobs": _exact_logprobs}[
        case["kind"]](case, s)


def _exact_append(case, s):
    t, n_q, n_kv, dh = case["rows"], case["n_q"], case["n_kv"], case["d_head"]
    x = s["qkv"].double().view(t, -1, dh)
    # the table's fp32 cosines and sines are inputs
    turn = torch.view_as_complex(s["rope"].double())[s["pos"].long()][:, None]

    def turned(heads, gain):
        if gain is not None:
            heads = heads / torch.sqrt(heads.square().sum(-1, keepdim=True) / dh + EPS) * gain.double()
        z = torch.complex(heads[..., :dh // 2].contiguous(), heads[..., dh // 2:].contiguous()) * turn
        return torch.cat([z.real, z.imag], -1)

    live = s["slots"] >= 0
    value = _e4m3_values()

    def written(codes, scale, new):
        old = value[codes.int()].transpose(1, 2).reshape(-1, n_kv, dh)
        old_scale = torch.exp2(scale.double() - 127).transpose(1, 2).reshape(-1, n_kv)
        amax = new[live].abs().amax(-1)
        e = torch.floor(torch.log2(amax.clamp(min=2.0 ** -140))) - 8
        e = (e + (amax > E4M3_MAX * torch.exp2(e))).clamp(min=MIN_EXP)
        at = s["slots"][live].long()
        old[at] = _e4m3_nearest(new[live] / torch.exp2(e)[..., None])
        old_scale[at] = torch.exp2(e)
        return old.view(-1, PAGE, n_kv, dh).transpose(1, 2), old_scale.view(-1, PAGE, n_kv).transpose(1, 2)

    k, ks = written(s["k"], s["ks"], turned(x[:, n_q:n_q + n_kv], s["g_k"]))
    v, vs = written(s["v"], s["vs"], x[:, n_q + n_kv:])
    return turned(x[:, :n_q], s["g_q"]), k, ks, v, vs


def _exact_attend(case, s):
    n_q, n_kv, dh = case["n_q"], case["n_kv"], case["d_head"]
    grp = n_q // n_kv
    value = _e4m3_values()
    start, kv = s["plan"].arrays[2].tolist(), s["plan"].arrays[3].tolist()
    out = torch.empty((s["q"].shape[0], n_q, dh), dtype=torch.float64, device="cuda")
    for i, n in enumerate(kv):
        pages = s["table"][i, :-(-n // PAGE)].long()
        rows = slice(start[i], start[i + 1])
        ahead = torch.arange(n, device="cuda")[None] > s["pos"][rows, None]
        for g in range(n_kv):
            k, v = ((value[c[pages, g].int()] * torch.exp2(e[pages, g].double() - 127)[..., None]).reshape(-1, dh)[:n]
                    for c, e in ((s["k"], s["ks"]), (s["v"], s["vs"])))
            for h in range(g * grp, (g + 1) * grp):
                score = s["q"][rows, h].double() @ k.T / math.sqrt(dh)
                out[rows, h] = torch.softmax(score.masked_fill(ahead, -math.inf), -1) @ v
    return out.view(-1, n_q * dh)


def _exact_norm(case, s):
    h = (s["x"].float() + s["r"].float()).to(torch.bfloat16).double()
    y = h / torch.sqrt(h.square().mean(-1, keepdim=True) + EPS) * s["gamma"].double()
    if case["fmt"] == "bf16":
        return h, y
    width = case["d"] if case["fmt"] == "e4m3" else BLOCK
    codes, scales = torch.empty_like(y), []
    for c in range(0, case["d"], width):
        part = y[:, c:c + width]
        amax = part.abs().amax(1)
        scale = torch.where(amax > 0, amax.clamp(min=AMAX_MIN if width == BLOCK else 0.0), amax) / E4M3_MAX
        ratio = torch.where(scale[:, None] > 0, part / scale[:, None], torch.zeros_like(part))
        codes[:, c:c + width] = _e4m3_nearest(ratio)
        scales.append(scale)
    return h, codes, scales[0] if case["fmt"] == "e4m3" else torch.stack(scales, 1)


def _exact_logprobs(case, s):
    out = [torch.empty(t.shape, dtype=torch.float64, device="cuda") for t in (s["lp"], s["entropy"], s["top_lp"])]
    ids = torch.empty(s["ids"].shape, dtype=torch.int64, device="cuda")
    step = max(1, (1 << 25) // case["vocab"])
    for r in range(0, case["rows"], step):
        at = slice(r, r + step)
        x = s["logits"][at].double()
        logp = x - torch.logsumexp(x, 1, keepdim=True)
        out[0][at] = logp.gather(1, s["tokens"][at].long())
        out[1][at] = -(torch.exp(logp) * logp.clamp(min=-1e4)).sum(1)
        ids[at] = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :ids.shape[1]]
        out[2][at] = logp.gather(1, ids[at])
    return out[0], out[1], ids, out[2]
