"""Operands of the block-scaled and normed calls that the binding refuses, one
condition broken at a time (no GPU: the tensors are stand-ins that say they
lie on a device, and the library must not be reached)."""
import pytest

import workloads as wl
from chunked_prefill_hybrid_tau_gb300 import _lib as L
from chunked_prefill_hybrid_tau_gb300 import binding as B

torch = pytest.importorskip("torch")


class OnDevice:
    """A tensor as the binding sees one, on device 0."""

    def __init__(self, shape, dtype, strides=None, device=0):
        self.shape, self.dtype, self.where = torch.Size(shape), dtype, device
        self.meta = torch.empty(shape, dtype=dtype, device="meta")
        if strides is not None:
            self.meta = torch.empty_strided(shape, strides, dtype=dtype, device="meta")

    device = property(lambda self: torch.device("cuda", self.where) if self.where >= 0 else torch.device("cpu"))
    is_cuda = True

    def get_device(self):
        return self.where

    def __getattr__(self, name):
        return getattr(self.meta, name)

    def data_ptr(self):
        return 4096


class Reached(Exception):
    pass


@pytest.fixture(autouse=True)
def no_library(monkeypatch):
    class Lib:
        def __getattr__(self, name):
            def call(*a):
                raise Reached(name)
            return call

    monkeypatch.setattr(B, "lib", Lib)
    monkeypatch.setattr(B, "_current_stream", lambda: 0)
    monkeypatch.setattr(B, "_current_device", lambda: 0, raising=False)


BF, U8, F32, I32 = torch.bfloat16, torch.uint8, torch.float32, torch.int32
DIMS = wl.TINY  # 4 q and 2 kv heads of 64
ROWS = DIMS.qkv_cols
CALLS = {
    "quantize": (lambda o: B.hb_quantize_e4m3_block(o["x"], o["q"], o["scale"]),
                 dict(x=((4, 256), BF), q=((4, 256), U8), scale=((4, 2), F32))),
    "gemm": (lambda o: B.hb_gemm_e4m3_block(o["A"], o["s_a"], o["B"], o["s_b"], o["C"], o["R"], L.HB_EPI_RESIDUAL),
             dict(A=((4, 256), U8), s_a=((4, 2), F32), B=((136, 256), U8), s_b=((2, 2), F32), C=((4, 136), BF),
                  R=((4, 136), BF))),
    "append": (lambda o: B.hb_kv_append_norm(o["qkv"], o["row_pos"], o["slot_mapping"], o["rope"], 32, DIMS, o["g_q"],
                                             o["g_k"], o["q_out"], o["k_cache"], o["v_cache"]),
               dict(qkv=((3, ROWS), BF), row_pos=((3,), I32), slot_mapping=((3,), I32), rope=((32, 32, 2), F32),
                    g_q=((64,), BF), g_k=((64,), BF), q_out=((3, 4, 64), BF), k_cache=((5, 2, 16, 64), BF),
                    v_cache=((5, 2, 16, 64), BF))),
}
SAME_SIZE = {BF: torch.float16, U8: torch.int8, F32: torch.int32, I32: torch.float32}


def run(call, **changed):
    fn, ops = CALLS[call]
    fn({k: changed.get(k) or OnDevice(*v) for k, v in ops.items()})


@pytest.mark.parametrize("call", CALLS)
def test_good_operands_reach_the_library(call):
    with pytest.raises(Reached):
        run(call)


def test_codes_may_be_float8():
    for call, name, shape in (("quantize", "q", (4, 256)), ("gemm", "A", (4, 256)), ("gemm", "B", (136, 256))):
        with pytest.raises(Reached):
            run(call, **{name: OnDevice(shape, torch.float8_e4m3fn)})


@pytest.mark.parametrize("call,name", [(c, n) for c in CALLS for n in CALLS[c][1]])
def test_each_operand_is_checked(call, name):
    shape, dtype = CALLS[call][1][name]
    bad = {
        "type of the same size": OnDevice(shape, SAME_SIZE[dtype]),
        "wider type": OnDevice(shape, torch.float64),
        "other device": OnDevice(shape, dtype, device=1),
        "host": OnDevice(shape, dtype, device=-1),
    }
    if len(shape) > 1:
        bad["strided"] = OnDevice(shape, dtype, strides=(2 * shape[-1],) * (len(shape) - 1) + (1,))
    if name not in ("x", "A", "B", "qkv", "k_cache"):  # the operands that give the sizes
        bad["too small"] = OnDevice((shape[0] - 1,) + tuple(shape[1:]), dtype)
    for what, t in bad.items():
        with pytest.raises(B.HBError, match=f"{name} must be a contiguous device tensor") as e:
            run(call, **{name: t})
        assert e.value.status == L.HB_ERR_INVALID_ARG, what


def test_shapes_that_do_not_fit_each_other():
    with pytest.raises(B.HBError, match="rows of 256 codes, B of 384"):
        run("gemm", B=OnDevice((136, 384), U8))
    for cols in (ROWS + 64, ROWS - 64):
        with pytest.raises(B.HBError, match="qkv"):
            run("append", qkv=OnDevice((3, cols), BF))
