"""prepare_layer_weights on a stream of its own (no GPU): the library's calls
are replaced by ones that run late, as a stream does that is behind the
host.  What the preparation returns must not hang on anything that ran
ahead of them, and no buffer that they use may be given out before they
are done with it."""
import numpy as np
import pytest

import oracle.fp8 as of
import workloads as wl
from chunked_prefill_hybrid_tau_gb300 import binding as B

torch = pytest.importorskip("torch")


class LateStream:
    """A stream whose work runs when finish() is called."""
    cuda_stream = 7

    def __init__(self):
        self.queue, self.waited, self.recorded = [], False, []

    def wait_stream(self, other):
        self.waited = True

    def add(self, fn, *tensors):
        self.queue.append((fn, tensors))

    def finish(self):
        for fn, _ in self.queue:
            fn()

    def storages(self):
        return {t.untyped_storage().data_ptr() for _, tensors in self.queue for t in tensors}


def bf16(x):
    return torch.from_numpy(np.asarray(x, np.float32)).to(torch.bfloat16)


@pytest.fixture
def late(monkeypatch):
    s = LateStream()

    def fold(w, gamma, out=None, stream=None):
        out = w if out is None else out
        s.add(lambda: out.copy_((w.float() * gamma.float()).to(torch.bfloat16)), out)
        return out

    def interleave(gate, up, w_gu, stream=None):
        def run():
            f, d = gate.shape
            pad = w_gu.shape[0] // 2 - f
            parts = [torch.cat([t.view(torch.int16), torch.zeros((pad, d), dtype=torch.int16)]).view(-1, 64, d)
                     for t in (gate, up)]
            w_gu.view(torch.int16).copy_(torch.stack(parts, 1).reshape(w_gu.shape))

        s.add(run, gate, up, w_gu)

    def quantize(x, q=None, scale=None, block_rows=None, stream=None):
        rows, cols = x.shape
        shape = (rows,) if block_rows is None else (-(-rows // block_rows), -(-cols // 128))
        q = B._empty((rows, cols), torch.uint8, x.device, stream) if q is None else q
        scale = B._empty(shape, torch.float32, x.device, stream) if scale is None else scale

        def run():
            codes, sc = (of.quantize_rows(x.float().numpy()) if block_rows is None else
                         of.quantize_blocks(x.float().numpy(), block_rows))
            q.copy_(torch.from_numpy(codes))
            scale.copy_(torch.from_numpy(sc))

        s.add(run, x, q, scale)
        return q, scale

    empty = torch.empty

    def poisoned(*a, **k):
        t = empty(*a, **k)
        t.view(torch.uint8).fill_(0x55)
        return t

    monkeypatch.setattr(B, "hb_fold_gamma", fold)
    monkeypatch.setattr(B, "hb_interleave_gate_up", interleave)
    monkeypatch.setattr(B, "hb_quantize_e4m3", quantize)
    monkeypatch.setattr(B, "hb_quantize_e4m3_block", quantize)
    monkeypatch.setattr(B, "_current_stream", lambda: 3)
    monkeypatch.setattr(B, "_capturing", lambda st: False, raising=False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: object())
    monkeypatch.setattr(torch, "empty", poisoned)
    monkeypatch.setattr(torch.Tensor, "record_stream",
                        lambda t, st: s.recorded.append((t.untyped_storage().data_ptr(), st)), raising=False)
    return s


@pytest.mark.parametrize("fmt", ["e4m3_block", "e4m3", "bf16"])
def test_preparation_on_a_late_stream(late, fmt):
    dims = wl.TINY
    w = wl.layer_weights(np.random.default_rng(11), dims)
    names = ("w_qkv", "w_o", "w_g", "w_u", "w_d", "g1", "g2")
    args = [bf16(w[k]) for k in names]
    callers = {t.untyped_storage().data_ptr() for t in args}
    lw = B.prepare_layer_weights(*args, stream=late, fmt=fmt)
    assert late.waited
    kept = {p for p, st in late.recorded if st is late}
    assert late.storages() - callers <= kept  # every buffer of the preparation's own
    late.finish()
    f, d = w["w_g"].shape
    pad = -f % 64

    def interleaved(g, u):
        parts = [np.concatenate([m, np.zeros((pad, d), m.dtype)]).reshape(-1, 64, d) for m in (g, u)]
        return np.stack(parts, 1).reshape(-1, d)

    if fmt == "e4m3_block":
        ref = of.prepare_weights(w, block=True)
        assert np.array_equal(lw.s_gu.numpy(), np.concatenate([ref["g"][1], ref["u"][1]]))
    elif fmt == "e4m3":
        ref = of.prepare_weights(w)
        assert np.array_equal(lw.s_gu.numpy(), interleaved(ref["g"][1][:, None].repeat(d, 1),
                                                           ref["u"][1][:, None].repeat(d, 1))[:, 0])
    if fmt != "bf16":
        assert np.array_equal(lw.w_gu.numpy(), interleaved(ref["g"][0], ref["u"][0]))
        for k in ("qkv", "o", "d"):
            assert np.array_equal(getattr(lw, "w_" + k).numpy(), ref[k][0]), k
            assert np.array_equal(getattr(lw, "s_" + k).numpy(), ref[k][1]), k
    else:
        g, u = ((args[i].float() * args[6].float()).to(torch.bfloat16).float().numpy() for i in (2, 3))
        assert np.array_equal(lw.w_gu.float().numpy(), interleaved(g, u))


def test_own_buffers_on_the_current_stream_need_no_ordering(late, monkeypatch):
    """The current stream's memory, used on the current stream."""
    monkeypatch.setattr(B, "_current_stream", lambda: 7)
    for stream in (None, late, 7):
        B._empty((2, 2), torch.uint8, "cpu", stream)
    assert not late.waited and not late.recorded
