"""Order of the block-scaled calls and what feeds them, on the GPU: weights
prepared on a stream of their own, and operands written by the call right
ahead of the one that reads them."""
import numpy as np
import pytest

import workloads as wl
from workloads import device as wd

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import chunked_prefill_hybrid_tau_gb300 as hb  # noqa: E402


@pytest.mark.parametrize("as_handle", [False, True])
@pytest.mark.parametrize("fmt", ["e4m3_block", "e4m3", "bf16"])
def test_prepare_on_a_side_stream(fmt, as_handle):
    """The weights that the current stream would have prepared, with work on
    the current stream that takes and gives back memory meanwhile."""
    dims = wl.Dims(d_model=1024, n_q=16, n_kv=4, d_head=64, d_ff=2112)
    gen = wd.device_generator(5)
    raw = [wd.randn_bf16(s, gen, 0.05) for s in ((dims.qkv_cols, 1024), (1024, 1024), (2112, 1024), (2112, 1024),
                                                 (1024, 2112), (1024,), (1024,))]
    names = ("w_qkv", "w_o", "w_gu", "w_d") + (() if fmt == "bf16" else ("s_qkv", "s_o", "s_gu", "s_d"))
    ref = hb.prepare_layer_weights(*[t.clone() for t in raw], fmt=fmt)
    side = torch.cuda.Stream()
    handle = side.cuda_stream if as_handle else side
    for _ in range(5):
        churn = [torch.full((3 << 20,), 7.0, device="cuda") for _ in range(4)]
        del churn
        copies = [t.clone() for t in raw]
        side.wait_stream(torch.cuda.current_stream())  # the caller's tensors are the caller's to order
        lw = hb.prepare_layer_weights(*copies, stream=handle, fmt=fmt)
        churn = [torch.full((3 << 20,), 9.0, device="cuda") for _ in range(4)]
        del churn
        side.synchronize()
        for k in names:
            assert torch.equal(getattr(lw, k).view(torch.uint8), getattr(ref, k).view(torch.uint8)), k
        torch.cuda.synchronize()
    hb.hb_check_status()
