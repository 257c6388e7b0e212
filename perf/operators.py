"""Measured cases of the decoder layer's operators for models with normed
query/key heads and block-scaled FP8 projections:

  append    RMS norm of every query and key head, the position rotation and
            the paged K/V write, one pass over the packed rows
  quantize  E4M3 codes with one fp32 scale per 128 columns of a row (tokens)
            or per 128 x 128 block (weights)
  gemm      the packed-token projection of such operands, with the store,
            residual, SwiGLU and fp32 epilogues

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
AMAX_MIN = 2.0 ** -112  # smallest group maximum that a scale is formed from


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one decode token, far into its context
        dict(name="append_1_row", kind="append", rows=1, decodes=1, n_q=32, n_kv=8, d_head=128, theta=1e6,
             max_pos=32768, pad=0),
        # the tiny layer's heads, an odd number of rows, some of them padding
        dict(name="append_tiny_333_rows", kind="append", rows=333, decodes=5, n_q=4, n_kv=2, d_head=64, theta=1e4,
             max_pos=4096, pad=3),
        # the hybrid iteration of the benchmark: 32 decodes and a 480-token chunk
        dict(name="append_hybrid_512", kind="append", rows=512, decodes=32, n_q=32, n_kv=8, d_head=128, theta=1e6,
             max_pos=8192, pad=0),
        # a long prompt in one piece on the widest heads of the workloads
        dict(name="append_prompt_8192", kind="append", rows=8192, decodes=0, n_q=56, n_kv=8, d_head=128, theta=5e6,
             max_pos=32768, pad=0),
        # one decode token's hidden row
        dict(name="quantize_1x4096", kind="quantize", rows=1, cols=4096, block_rows=1),
        # the SwiGLU output of a long prompt
        dict(name="quantize_8192x14336", kind="quantize", rows=8192, cols=14336, block_rows=1),
        # weight preparation: the gate and up matrices of one layer
        dict(name="quantize_weight_28672x4096", kind="quantize", rows=28672, cols=4096, block_rows=128),
        # QKV projection of one decode token
        dict(name="gemm_1_qkv", kind="gemm", m=1, n=6144, k=4096, epilogue="store"),
        # down projection of a decode-only iteration
        dict(name="gemm_32_down", kind="gemm", m=32, n=4096, k=14336, epilogue="residual"),
        # odd sizes: rows, output columns and a last K block of 48
        dict(name="gemm_201_odd", kind="gemm", m=201, n=1000, k=688, epilogue="f32"),
        # gate/up projection of the benchmark's hybrid iteration
        dict(name="gemm_512_gate_up", kind="gemm", m=512, n=28672, k=4096, epilogue="swiglu"),
        # QKV projection of a long prompt, the widest hidden size of the workloads
        dict(name="gemm_4096_qkv", kind="gemm", m=4096, n=9216, k=7168, epilogue="store"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["append", "quantize", "gemm", "gemm"])
    if kind == "append":
        n_q, n_kv, d_head = rng.choice([(32, 8, 128), (56, 8, 128), (4, 2, 64), (8, 8, 64), (16, 1, 128),
                                        (12, 4, 64), (1, 1, 128), (40, 5, 128), (64, 8, 64)])
        rows = _log_int(rng, 1, 8192)
        return dict(kind="append", rows=rows, decodes=rng.randint(0, min(rows, 64)), n_q=n_q, n_kv=n_kv,
                    d_head=d_head, theta=rng.choice([1e4, 1e6, 5e6]), max_pos=rng.choice([8192, 16384, 32768]),
                    pad=rng.randint(0, min(rows - 1, 7)))
    if kind == "quantize":
        block_rows = rng.choice([1, 1, 128])
        cols = 16 * _log_int(rng, 1, 896)
        rows = _log_int(rng, 1, min(28672, 8192 * 14336 // cols))
        return dict(kind="quantize", rows=rows, cols=cols, block_rows=block_rows)
    epilogue = rng.choice(["store", "residual", "swiglu", "f32"])
    k = 16 * _log_int(rng, 1, 896)
    n = 128 * _log_int(rng, 1, 224) if epilogue == "swiglu" else 8 * _log_int(rng, 1, 3584)
    return dict(kind="gemm", m=_log_int(rng, 1, min(4096, max(1, 4096 * 9216 * 7168 // (n * k)))), n=n, k=k,
                epilogue=epilogue)


def _blocks(n):
    return -(-n // BLOCK)


def work(case):
    if case["kind"] == "append":
        t, h, dh = case["rows"], case["n_q"] + 2 * case["n_kv"], case["d_head"]
        kv = 2 * (t - case["pad"]) * case["n_kv"] * dh * 2
        read = t * h * dh * 2 + min(t, case["max_pos"]) * dh * 4 + 8 * t + 4 * dh
        rot = t * (case["n_q"] + case["n_kv"]) * dh
        return {"bytes": read + t * case["n_q"] * dh * 2 + kv, "flops": 7 * rot}
    if case["kind"] == "quantize":
        n = case["rows"] * case["cols"]
        return {"bytes": 3 * n + 4 * -(-case["rows"] // case["block_rows"]) * _blocks(case["cols"]), "flops": 2 * n}
    m, n, k, epi = case["m"], case["n"], case["k"], case["epilogue"]
    s = 4 * _blocks(k) * (m + _blocks(n))
    out = m * n * {"store": 2, "residual": 4, "swiglu": 1, "f32": 4}[epi]
    return {"bytes": m * k + n * k + s + out, "flops": 2 * m * n * k}


# ------------------------------------------------------------------ the inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(shape, g, scale=1.0):
    return torch.randn(shape, generator=g, device="cuda") * scale


def _activations(rows, cols, g):
    # channels of different size, as the hidden rows of a trained model have
    return _randn((rows, cols), g) * torch.exp(_randn((1, cols), g))


def _quantize(x, block_rows):
    """fp32 x -> (E4M3 codes, scales) by the rule of hb_quantize_e4m3_block."""
    rows, cols = x.shape
    br, kb = -(-rows // block_rows), _blocks(cols)
    full = torch.zeros((br * block_rows, kb * BLOCK), dtype=torch.float32, device=x.device)
    full[:rows, :cols] = x
    full = full.view(br, block_rows, kb, BLOCK)
    amax = full.abs().amax(dim=(1, 3))
    safe = amax.clamp(min=AMAX_MIN)
    zero = amax == 0
    top = torch.full_like(safe, E4M3_MAX)  # tensor by tensor: a divisor that is a number would become a product
    inv = torch.where(zero, 0.0, top / safe)
    scale = torch.where(zero, 0.0, safe / top)
    y = (full * inv[:, None, :, None]).clamp(-E4M3_MAX, E4M3_MAX)
    codes = y.view(br * block_rows, kb * BLOCK)[:rows, :cols].to(torch.float8_e4m3fn)
    return codes.contiguous(), scale


def prepare(case, seed):
    g = _gen(seed)
    if case["kind"] == "append":
        return _prepare_append(case, g)
    if case["kind"] == "quantize":
        rows, cols, br = case["rows"], case["cols"], case["block_rows"]
        x = _activations(rows, cols, g) if br == 1 else _randn((rows, cols), g, 0.02)
        q = torch.empty((rows, cols), dtype=torch.uint8, device="cuda")
        scale = torch.empty((-(-rows // br), _blocks(cols)), dtype=torch.float32, device="cuda")
        return dict(case=case, x=x.to(torch.bfloat16), q=q, scale=scale)
    m, n, k, epi = case["m"], case["n"], case["k"], case["epilogue"]
    a, sa = _quantize(_activations(m, k, g).to(torch.bfloat16).float(), 1)
    if epi == "swiglu":
        f = n // 2
        gate, sg = _quantize(_randn((f, k), g, 0.02), BLOCK)
        up, su = _quantize(_randn((f, k), g, 0.02), BLOCK)
        # gate and up rows interleaved in blocks of 64, scales of gate then of up
        b = torch.stack([gate.view(torch.uint8).view(f // 64, 64, k), up.view(torch.uint8).view(f // 64, 64, k)], 1)
        b, sb = b.reshape(n, k).contiguous(), torch.cat([sg, su]).contiguous()
    else:
        b, sb = _quantize(_randn((n, k), g, 0.02), BLOCK)
        b = b.view(torch.uint8)
    out_cols = n // 2 if epi == "swiglu" else n
    out = torch.empty((m, out_cols), dtype=torch.float32 if epi == "f32" else torch.bfloat16, device="cuda")
    r = _randn((m, n), g).to(torch.bfloat16) if epi == "residual" else None
    return dict(case=case, a=a.view(torch.uint8), sa=sa, b=b, sb=sb, r=r, out=out)


def _prepare_append(case, g):
    t, n_dec, n_q, n_kv, dh = case["rows"], case["decodes"], case["n_q"], case["n_kv"], case["d_head"]
    max_pos, half = case["max_pos"], case["d_head"] // 2
    chunk = t - n_dec
    chunk_pages = -(-chunk // PAGE)
    num_pages = chunk_pages + n_dec + 4

    def ints(hi, n):
        return torch.randint(0, hi, (n,), generator=g, device="cuda")

    # decode rows: one new token each, anywhere in its context; then the chunk's rows in order
    dec_pos = ints(max_pos, n_dec)
    start = ints(max(1, (max_pos - chunk) // PAGE), 1) * PAGE
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
    g_q = (1 + _randn((dh,), g, 0.2)).to(torch.bfloat16)
    g_k = (1 + _randn((dh,), g, 0.2)).to(torch.bfloat16)
    shape = (num_pages, n_kv, PAGE, dh)
    k_cache, v_cache = (_randn(shape, g).to(torch.bfloat16) for _ in range(2))
    q_out = torch.empty((t, n_q, dh), dtype=torch.bfloat16, device="cuda")
    dims = types.SimpleNamespace(d_model=n_q * dh if (n_q * dh) % 64 == 0 else 64, n_q=n_q, n_kv=n_kv, d_head=dh,
                                 d_ff=64, page=PAGE, eps=EPS, theta=case["theta"])
    return dict(case=case, qkv=qkv, pos=pos, slots=slots, rope=rope, g_q=g_q, g_k=g_k, k=k_cache, v=v_cache,
                q_out=q_out, dims=dims)


# ------------------------------------------------------------------ one pass
def run(state):
    kind = state["case"]["kind"]
    if own:
        return _run_own(kind, state)
    if kind == "append":
        return _plain_append(state)
    if kind == "quantize":
        return _quantize(state["x"].float(), state["case"]["block_rows"])
    return _plain_gemm(state)


def _run_own(kind, s):
    import chunked_prefill_hybrid_tau_gb300 as hb
    if kind == "append":
        hb.hb_kv_append_norm(s["qkv"], s["pos"], s["slots"], s["rope"], s["case"]["max_pos"], s["dims"], s["g_q"],
                             s["g_k"], s["q_out"], s["k"], s["v"])
        return s["q_out"], s["k"], s["v"]
    if kind == "quantize":
        hb.hb_quantize_e4m3_block(s["x"], s["q"], s["scale"], block_rows=s["case"]["block_rows"])
        return s["q"].view(torch.float8_e4m3fn), s["scale"]
    epilogue = ["store", "residual", "swiglu", "f32"].index(s["case"]["epilogue"])
    hb.hb_gemm_e4m3_block(s["a"], s["sa"], s["b"], s["sb"], s["out"], s["r"], epilogue)
    return s["out"]


def _plain_append(s):
    c = s["case"]
    t, n_q, n_kv, dh = c["rows"], c["n_q"], c["n_kv"], c["d_head"]
    x = s["qkv"].view(t, n_q + 2 * n_kv, dh)

    def norm_rotate(h, gain):
        h = h.float()
        h = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS) * gain.float()
        cs = s["rope"][s["pos"].long()][:, None]
        a, b, cos, sin = h[..., :dh // 2], h[..., dh // 2:], cs[..., 0], cs[..., 1]
        return torch.cat([a * cos - b * sin, b * cos + a * sin], -1).to(torch.bfloat16)

    q = norm_rotate(x[:, :n_q], s["g_q"])
    k = norm_rotate(x[:, n_q:n_q + n_kv], s["g_k"])
    kept = t - c["pad"]
    page, off = s["slots"][:kept].long() // PAGE, s["slots"][:kept].long() % PAGE
    s["k"][page, :, off] = k[:kept]
    s["v"][page, :, off] = x[:kept, n_q + n_kv:]
    return q, s["k"], s["v"]


def _spread(scale, rows, cols, block_rows):
    """A block's scale at each of its elements."""
    s = scale.repeat_interleave(block_rows, 0)[:rows] if block_rows > 1 else scale
    return s.repeat_interleave(BLOCK, 1)[:, :cols]


def _plain_gemm(s):
    c = s["case"]
    m, n, k, epi = c["m"], c["n"], c["k"], c["epilogue"]
    a = s["a"].view(torch.float8_e4m3fn).float() * _spread(s["sa"], m, k, 1)
    b = s["b"].view(torch.float8_e4m3fn).float()
    if epi == "swiglu":
        f = n // 2
        b = b.view(f // 64, 2, 64, k)
        half = s["sb"].shape[0] // 2
        gate = a @ (b[:, 0].reshape(f, k) * _spread(s["sb"][:half], f, k, BLOCK)).T
        up = a @ (b[:, 1].reshape(f, k) * _spread(s["sb"][half:], f, k, BLOCK)).T
        return (gate / (1 + torch.exp(-gate)) * up).to(torch.bfloat16)
    y = a @ (b * _spread(s["sb"], n, k, BLOCK)).T
    if epi == "residual":
        y = s["r"].float() + y
    return y if epi == "f32" else y.to(torch.bfloat16)


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
    if case["kind"] == "append":
        return _exact_append(case, s)
    if case["kind"] == "quantize":
        x, br = s["x"].double(), case["block_rows"]
        scale = torch.zeros_like(s["scale"], dtype=torch.float64)
        out = torch.zeros_like(x)
        for j in range(scale.shape[1]):
            cols = x[:, j * BLOCK:(j + 1) * BLOCK]
            amax = cols.abs().amax(1)
            if br > 1:
                amax = torch.nn.functional.pad(amax, (0, -amax.numel() % br)).view(-1, br).amax(1)
            scale[:, j] = torch.where(amax > 0, amax.clamp(min=AMAX_MIN), amax) / E4M3_MAX
            per_row = scale[:, j].repeat_interleave(br)[:x.shape[0]] if br > 1 else scale[:, j]
            out[:, j * BLOCK:(j + 1) * BLOCK] = _e4m3_nearest(
                torch.where(per_row[:, None] > 0, cols / per_row[:, None], torch.zeros_like(cols)))
        return out, scale
    m, n, k, epi = case["m"], case["n"], case["k"], case["epilogue"]
    value = _e4m3_values()
    a = value[s["a"].int()]
    acc = torch.zeros((m, n), dtype=torch.float64, device="cuda")
    row = torch.arange(n, device="cuda")
    if epi == "swiglu":  # scale row of an interleaved row: gate blocks, then up blocks
        f_row = row // 128 * 64 + row % 64
        row = f_row // BLOCK + torch.where(row % 128 >= 64, s["sb"].shape[0] // 2, 0)
    else:
        row = row // BLOCK
    for j in range(_blocks(k)):
        cols = slice(j * BLOCK, min(k, (j + 1) * BLOCK))
        part = a[:, cols] @ value[s["b"][:, cols].int()].T
        acc += part * s["sa"][:, j].double()[:, None] * s["sb"][row, j].double()[None, :]
    if epi == "swiglu":
        acc = acc.view(m, n // 128, 2, 64)
        gate, up = acc[:, :, 0].reshape(m, n // 2), acc[:, :, 1].reshape(m, n // 2)
        return gate * torch.sigmoid(gate) * up
    return acc + s["r"].double() if epi == "residual" else acc


def _exact_append(case, s):
    t, n_q, n_kv, dh = case["rows"], case["n_q"], case["n_kv"], case["d_head"]
    x = s["qkv"].double().view(t, -1, dh)
    i = torch.arange(dh // 2, dtype=torch.float64, device="cuda")
    ang = s["pos"].double()[:, None] * torch.pow(torch.tensor(case["theta"], dtype=torch.float64, device="cuda"),
                                                 -2 * i / dh)
    turn = torch.polar(torch.ones_like(ang), ang)[:, None]

    def normed_turned(heads, gain):
        y = heads / torch.sqrt(heads.square().sum(-1, keepdim=True) / dh + EPS) * gain.double()
        z = torch.complex(y[..., :dh // 2].contiguous(), y[..., dh // 2:].contiguous()) * turn
        return torch.cat([z.real, z.imag], -1)

    live = s["slots"] >= 0

    def written(pool, new):
        flat = pool.double().transpose(1, 2).reshape(-1, n_kv, dh)
        flat[s["slots"][live].long()] = new[live]
        return flat.view(-1, PAGE, n_kv, dh).transpose(1, 2)

    return (normed_turned(x[:, :n_q], s["g_q"]), written(s["k"], normed_turned(x[:, n_q:n_q + n_kv], s["g_k"])),
            written(s["v"], x[:, n_q + n_kv:]))
