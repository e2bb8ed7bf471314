"""vlaq_check: every status word is read, reported once and cleared, in one
round trip to the device."""
import time

import pytest
import torch

from gpu_helpers import vq

pytestmark = pytest.mark.gpu


def _best_us(call, batches=12, calls=40):
    call()
    best = float("inf")
    for _ in range(batches):
        torch.cuda.synchronize()
        t = time.perf_counter()
        for _ in range(calls):
            call()
        best = min(best, (time.perf_counter() - t) / calls)
    return best * 1e6


def test_check_costs_one_round_trip():
    """Against a kernel, a copy to the host and a wait: 0.9 of it as measured;
    a copy and a wait for each of the four words take four times as long."""
    m = vq()
    x = torch.zeros(1, device="cuda")
    trip = _best_us(lambda: x.add_(1).item())
    check = _best_us(m.vlaq_check)
    assert check < 2 * trip, (check, trip)


@pytest.mark.parametrize("side", [False, True])
def test_words_are_reported_once_whichever_kernel_set_them(side):
    m = vq()
    M, N, K = 5, 136, 400
    x, w = (torch.zeros(r, K, dtype=torch.uint8, device="cuda") for r in (M, N))
    sx, sw = (torch.ones(*s, device="cuda") for s in ((4, M), (2, 4)))
    Y = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    stream = torch.cuda.Stream() if side else torch.cuda.current_stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        m.vlaq_check()
        for set_word in (lambda: m.vlaq_selftest_wait_timeout(),
                         lambda: m.vlaq_selftest_linear_fp8_block(0, 1, 1, x, sx, w, sw, None, Y, M, N, K)):
            set_word()
            with pytest.raises(m.VlaqError) as ei:
                m.vlaq_check()
            assert ei.value.status == 6
            m.vlaq_check()
