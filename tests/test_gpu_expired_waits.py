"""What a CTA does once one of its bounded waits has expired (GPU): the
library's self-test makes them expire after a short limit; nothing hangs or
faults."""
import time

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import chunked_prefill_hybrid_tau_gb300 as hb  # noqa: E402
from chunked_prefill_hybrid_tau_gb300 import _lib as L  # noqa: E402


def clean_status():
    try:
        hb.hb_check_status()
    except hb.HBError:
        pass


def test_a_tile_is_not_stored_when_another_warps_wait_expired():
    """The self-test's first warp has its data, the second one's wait expires:
    an index error instead of the timeout would mean that the first warp had
    taken its own success for the tile's."""
    clean_status()
    hb.hb_selftest_wait_timeout(2000)
    with pytest.raises(hb.HBError) as err:
        hb.hb_check_status()
    assert err.value.status == L.HB_ERR_TIMEOUT
    hb.hb_check_status()


def test_waits_after_an_expired_one_give_up_at_once():
    """Three waits of the limit, then 200 that find the abort flag raised."""
    clean_status()
    hb.hb_selftest_wait_timeout(1000)
    clean_status()
    for limit in (0.002, 0.05):
        t0 = time.perf_counter()
        hb.hb_selftest_wait_timeout(int(limit * 1e6))
        with pytest.raises(hb.HBError) as err:
            hb.hb_check_status()
        took = time.perf_counter() - t0
        print(f"limit {limit * 1e3:.0f} ms: {took * 1e3:.2f} ms")
        assert err.value.status == L.HB_ERR_TIMEOUT
        assert 3 * 0.5 * limit <= took <= 3 * limit + 0.5
    hb.hb_check_status()
