"""Refusals of the E4M3 cache, residual norm and log probability calls: operands
that the binding refuses, one condition broken at a time, and argument errors
of the C entry points, found before any device work (no GPU)."""
import ctypes as C

import pytest

import workloads as wl
from chunked_prefill_hybrid_tau_gb300 import _lib as L
from chunked_prefill_hybrid_tau_gb300 import binding as B
from test_binding_operands import OnDevice, Reached

torch = pytest.importorskip("torch")

BF, U8, F32, I32 = torch.bfloat16, torch.uint8, torch.float32, torch.int32
DIMS = wl.TINY  # 4 q and 2 kv heads of 64


class Plan:
    def struct(self):
        return L.hb_device_plan(3, 2, 4, 64, 64, 64, 64, 64, 0, 0, 0)


CACHE = dict(k_cache=((5, 2, 16, 64), U8), k_scale=((5, 2, 16), U8), v_cache=((5, 2, 16, 64), U8),
             v_scale=((5, 2, 16), U8))
CALLS = {
    "append": (lambda o: B.hb_kv_append_e4m3(o["qkv"], o["row_pos"], o["slot_mapping"], o["rope"], 32, DIMS, o["q_out"],
                                             o["k_cache"], o["k_scale"], o["v_cache"], o["v_scale"], o["g_q"], o["g_k"]),
               dict(qkv=((3, DIMS.qkv_cols), BF), row_pos=((3,), I32), slot_mapping=((3,), I32), rope=((32, 32, 2), F32),
                    q_out=((3, 4, 64), BF), g_q=((64,), BF), g_k=((64,), BF), **CACHE)),
    "attention": (lambda o: B.hb_attention_e4m3(o["q"], o["k_cache"], o["k_scale"], o["v_cache"], o["v_scale"], Plan(),
                                                DIMS, 64, o["out"], OnDevice((4096,), U8)),
                  dict(q=((3, 4, 64), BF), out=((3, 256), BF), **CACHE)),
    "norm": (lambda o: B.hb_add_rmsnorm(o["x"], o["residual"], o["gamma"], 1e-6, o["h_out"], o["y"]),
             dict(x=((4, 256), BF), residual=((4, 256), BF), gamma=((256,), BF), h_out=((4, 256), BF), y=((4, 256), BF))),
    "norm rows": (lambda o: B.hb_add_rmsnorm(o["x"], None, o["gamma"], 1e-6, None, o["y"], o["scale"], fmt="e4m3"),
                  dict(x=((4, 256), BF), gamma=((256,), BF), y=((4, 256), U8), scale=((4,), F32))),
    "norm blocks": (lambda o: B.hb_add_rmsnorm(o["x"], None, o["gamma"], 1e-6, None, o["y"], o["scale"],
                                               fmt="e4m3_block"),
                    dict(x=((4, 256), BF), gamma=((256,), BF), y=((4, 256), U8), scale=((4, 2), F32))),
    "logprobs": (lambda o: B.hb_logprobs(o["logits"], o["tokens"], o["token_logprobs"], o["entropy"], o["top_ids"],
                                         o["top_logprobs"]),
                 dict(logits=((4, 100), F32), tokens=((4, 2), I32), token_logprobs=((4, 2), F32), entropy=((4,), F32),
                      top_ids=((4, 5), I32), top_logprobs=((4, 5), F32))),
}
SAME_SIZE = {BF: torch.float16, U8: torch.int8, F32: torch.int32, I32: torch.float32}


@pytest.fixture
def no_library(monkeypatch):
    class Lib:
        def __getattr__(self, name):
            def call(*a):
                raise Reached(name)
            return call

    monkeypatch.setattr(B, "lib", Lib)
    monkeypatch.setattr(B, "_current_stream", lambda: 0)
    monkeypatch.setattr(B, "_current_device", lambda: 0)


def run(call, **changed):
    fn, ops = CALLS[call]
    fn({k: changed.get(k) or OnDevice(*v) for k, v in ops.items()})


@pytest.mark.parametrize("call", CALLS)
def test_good_operands_reach_the_library(call, no_library):
    with pytest.raises(Reached):
        run(call)


def test_codes_scales_and_logits_of_their_other_types(no_library):
    for call, changed in (("append", dict(k_cache=OnDevice((5, 2, 16, 64), torch.float8_e4m3fn))),
                          ("attention", dict(v_scale=OnDevice((5, 2, 16), torch.float8_e8m0fnu))),
                          ("norm rows", dict(y=OnDevice((4, 256), torch.float8_e4m3fn))),
                          ("logprobs", dict(logits=OnDevice((4, 100), BF))),
                          ("logprobs", dict(logits=OnDevice((4, 100), F32, (128, 1))))):
        with pytest.raises(Reached):
            run(call, **changed)


@pytest.mark.parametrize("call,name", [(c, n) for c in CALLS for n in CALLS[c][1]])
def test_each_operand_is_checked(call, name, no_library):
    shape, dtype = CALLS[call][1][name]
    smaller = (shape[0], *shape[1:-1], shape[-1] - 1) if len(shape) > 1 else (shape[0] - 1,)
    bad = {
        "type of the same size": OnDevice(shape, SAME_SIZE[dtype]),
        "wider type": OnDevice(shape, torch.float64),
        "other device": OnDevice(shape, dtype, device=1),
        "host": OnDevice(shape, dtype, device=-1),
    }
    if (call, name) not in (("logprobs", "tokens"), ("logprobs", "top_ids"), ("logprobs", "logits")):
        if not (name in ("x",) and call.startswith("norm")):
            bad["too small"] = OnDevice(smaller, dtype)
        bad["strided"] = OnDevice(shape, dtype, [2 * s for s in torch.empty(shape, device="meta").stride()])
    for what, t in bad.items():
        with pytest.raises(B.HBError) as e:
            run(call, **{name: t})
        assert e.value.status == L.HB_ERR_INVALID_ARG, what


def test_shapes_of_the_log_probabilities(no_library):
    for changed in (dict(logits=OnDevice((4, 100), F32, (1, 4))), dict(logits=OnDevice((4, 100), F32, (99, 1))),
                    dict(tokens=OnDevice((3, 2), I32)), dict(top_ids=OnDevice((20,), I32)),
                    dict(top_ids=OnDevice((5, 4), I32))):
        with pytest.raises(B.HBError):
            run("logprobs", **changed)
    x, t, f = OnDevice((4, 100), F32), OnDevice((4, 2), I32), OnDevice((4, 2), F32)
    for args in (dict(tokens=t), dict(token_logprobs=f), dict(top_ids=t), dict(top_logprobs=f)):
        with pytest.raises(B.HBError):
            B.hb_logprobs(x, **args)
    with pytest.raises(B.HBError):
        B.hb_add_rmsnorm(OnDevice((4, 256), BF), None, OnDevice((256,), BF), 1e-6, fmt="e5m2")


P = C.c_void_p(4096)   # never dereferenced
ODD = C.c_void_p(4100)


def refused(lib, status, word):
    assert status == L.HB_ERR_INVALID_ARG and word in lib.hb_last_error(), lib.hb_last_error()


def test_append_refusals(lib):
    ds = B.dims_struct(DIMS)

    def call(T=1, max_pos=8, pages=1, d=ds, **ch):
        a = [ch.get(n, P) for n in ("qkv", "pos", "slot", "rope", "g_q", "g_k", "q", "k", "ks", "v", "vs")]
        return lib.hb_kv_append_e4m3(a[0], T, a[1], a[2], a[3], max_pos, C.byref(d), *a[4:], pages, None)

    for name in ("qkv", "pos", "slot", "rope", "q", "k", "ks", "v", "vs"):
        refused(lib, call(**{name: None}), b"null")
    refused(lib, call(g_q=None), b"gains")
    refused(lib, call(g_k=None), b"gains")
    for name in ("qkv", "rope", "q", "k", "v", "g_q", "g_k"):
        refused(lib, call(**{name: ODD}), b"alignment")
    for sizes in (dict(T=-1), dict(max_pos=0), dict(pages=0)):
        refused(lib, call(**sizes), b"sizes")
    bad = B.dims_struct(DIMS)
    bad.d_head = 96
    refused(lib, call(d=bad), b"d_head")
    assert call(T=0, qkv=None) == L.HB_OK


def test_attention_refusals(lib):
    ds = B.dims_struct(DIMS)
    need = lib.hb_attention_e4m3_workspace_bytes(C.byref(ds), 3, 2, 100)
    assert need > 0 and lib.hb_attention_e4m3_workspace_bytes(None, 3, 2, 100) == 0

    def call(plan=(3, 2, 4), arrays=(P,) * 5, pages=1, max_kv=100, ws=P, ws_bytes=need, d=ds, no_plan=False, **ch):
        a = [ch.get(n, P) for n in ("q", "k", "ks", "v", "vs")]
        ps = L.hb_device_plan(*plan, *arrays, 0, 0, 0)
        return lib.hb_attention_e4m3(*a, pages, None if no_plan else C.byref(ps), C.byref(d), max_kv, ch.get("out", P), ws,
                                     ws_bytes, None)

    for name in ("q", "k", "ks", "v", "vs", "out"):
        refused(lib, call(**{name: None}), b"null")
        refused(lib, call(**{name: ODD}), b"alignment")
    refused(lib, call(no_plan=True), b"null plan")
    for i in (2, 3, 4):
        refused(lib, call(arrays=tuple(None if j == i else P for j in range(5))), b"plan array")
    for plan in ((-1, 2, 4), (3, -2, 4), (3, 2, 0)):
        refused(lib, call(plan=plan), b"plan sizes")
    refused(lib, call(plan=(1025, 1025, 4)), b"1024")
    refused(lib, call(plan=(1, 2, 4)), b"at least one row")
    refused(lib, call(pages=0), b"num_pages")
    refused(lib, call(max_kv=0), b"max_kv_len")
    refused(lib, call(ws=None), b"workspace")
    refused(lib, call(ws_bytes=need - 1), b"workspace")
    refused(lib, call(ws=C.c_void_p(4096 + 16)), b"256-byte")
    assert call(plan=(0, 0, 1), q=None, ws=None) == L.HB_OK


def test_norm_refusals(lib):
    def call(rows=2, d=256, eps=1e-6, fmt=L.HB_NORM_E4M3, **ch):
        a = [ch.get(n, P) for n in ("x", "r", "g", "h", "y", "s")]
        return lib.hb_add_rmsnorm(*a, rows, d, eps, fmt, None)

    for name in ("x", "g", "y"):
        refused(lib, call(**{name: None}), b"null")
    for name in ("x", "r", "g", "h", "y"):
        refused(lib, call(**{name: ODD}), b"alignment")
    refused(lib, call(s=C.c_void_p(4098)), b"alignment")
    refused(lib, call(s=None), b"scales")
    refused(lib, call(fmt=L.HB_NORM_BF16), b"scales")
    refused(lib, call(fmt=3), b"format")
    for sizes in (dict(rows=-1), dict(d=0), dict(d=264), dict(d=32784), dict(d=8, fmt=L.HB_NORM_E4M3_BLOCK),
                  dict(d=260, fmt=L.HB_NORM_BF16, s=None)):
        refused(lib, call(**sizes), b"multiple")
    refused(lib, call(eps=-1.0), b"eps")
    assert call(rows=0, x=None) == L.HB_OK


def test_logprobs_refusals(lib):
    def call(kind=L.HB_LOGITS_F32, rows=2, vocab=100, stride=100, n=1, k=5, **ch):
        a = {m: ch.get(m, P) for m in ("x", "t", "lp", "e", "ids", "tlp")}
        return lib.hb_logprobs(a["x"], kind, rows, vocab, stride, a["t"], n, a["lp"], a["e"], k, a["ids"], a["tlp"], None)

    for name in ("x", "t", "lp", "ids", "tlp"):
        refused(lib, call(**{name: None}), b"null")
        refused(lib, call(**{name: C.c_void_p(4098)}), b"aligned")
    refused(lib, call(kind=L.HB_LOGITS_BF16, x=C.c_void_p(4097)), b"aligned")
    refused(lib, call(kind=2), b"type")
    for sizes in (dict(rows=-1), dict(vocab=0), dict(stride=99), dict(rows=2 ** 28 + 1)):
        refused(lib, call(**sizes), b"rows")
    refused(lib, call(n=-1), b"n_tokens")
    for k in (-1, 33, 101):
        refused(lib, call(k=k), b"top_k")
    refused(lib, call(vocab=4, k=5), b"top_k")
    assert call(rows=0, x=None) == L.HB_OK
    assert call(n=0, k=0, e=None, t=None, lp=None, ids=None, tlp=None) == L.HB_OK


def test_attention_e4m3_workspace_of_bad_sizes():
    """0, whatever else is given; and never less for more."""
    dims = lambda n_q, n_kv: wl.Dims(d_model=64, n_q=n_q, n_kv=n_kv, d_head=64, d_ff=64)  # noqa: E731
    size = B.hb_attention_e4m3_workspace_bytes
    assert size(dims(0, 1), 10, 2, 100) == 0 and size(dims(4, 0), 10, 2, 100) == 0
    assert size(dims(4, 2), -1, 2, 100) == 0 and size(dims(4, 2), 10, -1, 100) == 0 and size(dims(4, 2), 10, 2, -1) == 0
    for n_q in (1, 4, 75, 77, 160):
        for a in range(3):
            last = 0
            for v in (0, 1, 2, 100, 1000, 5000, 20000, 300000):
                args = [600, 3, 9000]
                args[a] = v
                got = size(dims(n_q, 1), *args)
                assert got >= last, (n_q, args)
                last = got


def test_attention_e4m3_workspace_counts_only_rows_whose_keys_can_be_split():
    """What the sizes ask for, part by part: the keys of decode rows in splits of
    256, the keys of short chunks in parts of up to 128 * (76 / n_q) rows a
    sequence (152 units of a tile and head at least twice), and widened keys."""
    up = lambda n, m: -(-n // m) * m  # noqa: E731
    for n_q, n_kv, d in ((4, 2, 64), (32, 8, 128), (56, 8, 128), (76, 4, 64), (80, 8, 128)):
        dims = wl.Dims(d_model=64, n_q=n_q, n_kv=n_kv, d_head=d, d_ff=64)
        for rows, seqs, kv in ((8192, 2, 32768), (8192, 1, 32768), (2048, 33, 4097), (64, 3, 9000), (130, 130, 9000)):
            splits = -(-kv // 256)
            decode = up(seqs * splits * n_kv * (n_q // n_kv) * (d + 4) * 4, 256)
            parts = max(1, min(8, 152 // n_q, -(-kv // 128) // 8))
            records = min(rows, seqs * 128 * (76 // n_q)) if parts > 1 else 0
            chunk = up(records * n_q * parts * (d + 4) * 4, 256)
            keys = min(min(seqs, rows // 2) * up(kv, 128), max(262144, up(kv, 128)))
            want = 256 + decode + chunk + 2 * keys * n_kv * d * 2
            assert B.hb_attention_e4m3_workspace_bytes(dims, rows, seqs, kv) == want, (n_q, rows, seqs, kv)
