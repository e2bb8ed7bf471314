"""The FP8 block linear's kernels when a bounded wait runs out.  The token tiles
arrive incomplete, so every wait for one ends after about 1 ms: no fault, no
hang, the context stays usable."""
import pytest
import torch

from gpu_helpers import to_dev, vq
from test_gpu_block128 import _linear_case

pytestmark = pytest.mark.gpu

COLS, ROWS, PAIR = 0, 1, 2


# a range that fits the stages (its producers never wait) and ones that do not,
# one tile and several per CTA, every kernel and form
@pytest.mark.parametrize("kernel,ctas,M,N,K", [(COLS, 1, 5, 264, 400), (COLS, 1, 1, 37888, 1808), (COLS, 4, 1, 4608, 3584),
                                               (COLS, 8, 20, 136, 2128), (COLS, 2, 64, 264, 4112), (ROWS, 1, 130, 264, 400),
                                               (ROWS, 1, 640, 8192, 1040), (ROWS, 3, 300, 392, 1040),
                                               (ROWS, 8, 70, 136, 4112), (PAIR, 2, 300, 520, 400),
                                               (PAIR, 2, 1024, 12808, 1040), (PAIR, 4, 300, 520, 400),
                                               (PAIR, 4, 700, 1032, 3088)])
@pytest.mark.parametrize("residual", [False, True])
def test_a_call_that_gives_up_lets_its_copies_land_and_stores_no_sums(kernel, ctas, M, N, K, residual):
    """The status is reported once, Y keeps its bytes or, where the CTAs of a
    cluster add their sums, holds NaN; no CTA leaves before
    copies that it issued have had their time to land (2^21 clocks after the
    2 million of the wait, at 1.965 GHz at most), and a call behind it on the
    stream, whose CTAs may start while its last ones end, is right."""
    m = vq()
    gen = torch.Generator(device="cuda")
    gen.manual_seed(K)
    kb, nb = -(-K // 128), -(-N // 128)
    code = [torch.randint(0, 0x60, (r, K), generator=gen, device="cuda", dtype=torch.uint8) for r in (M, N)]
    scale = [torch.rand(*s, generator=gen, device="cuda") for s in ((kb, M), (nb, kb))]
    R = torch.randn(M, N, generator=gen, device="cuda").to(torch.bfloat16) if residual else None
    d = (code[0], scale[0], code[1], scale[1], R)
    want, Y, Z = (torch.full((M, N), 3.0, dtype=torch.bfloat16, device="cuda") for _ in range(3))
    m.vlaq_selftest_linear_fp8_block(kernel, ctas, 0, *d, want, M, N, K)
    torch.cuda.synchronize()
    m.vlaq_check()
    a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    a.record()
    m.vlaq_selftest_linear_fp8_block(kernel, ctas, 1, *d, Y, M, N, K)
    b.record()
    m.vlaq_selftest_linear_fp8_block(kernel, ctas, 0, *d, Z, M, N, K)
    torch.cuda.synchronize()
    with pytest.raises(m.VlaqError) as ei:
        m.vlaq_check()
    assert ei.value.status == 6
    m.vlaq_check()
    if kernel != PAIR and ctas > 1:
        assert torch.isnan(Y).all(), "an incomplete sum looks like a result"
    else:
        assert (Y == 3.0).all(), "an incomplete tile was stored"
    assert torch.equal(Z, want)
    assert a.elapsed_time(b) >= (2_000_000 + 2 ** 21) / 1.965e6, "left before its copies had their time"


def test_every_kernel_gives_up_in_a_graph_and_runs_again():
    """Captured and replayed: the give-up of one replay leaves nothing behind
    for the next."""
    m = vq()
    M, N, K = 48, 264, 1040
    ops, _, _, _ = _linear_case(M, N, K, 3, False)
    d = [to_dev(t) for t in ops]
    for kernel, ctas in ((COLS, 3), (ROWS, 2), (PAIR, 2), (PAIR, 4)):
        want, Y = (torch.zeros(M, N, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        m.vlaq_selftest_linear_fp8_block(kernel, ctas, 0, *d, None, want, M, N, K)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            m.vlaq_selftest_linear_fp8_block(kernel, ctas, 1, *d, None, Y, M, N, K)
            m.vlaq_selftest_linear_fp8_block(kernel, ctas, 0, *d, None, Y, M, N, K)
        for _ in range(2):
            Y.zero_()
            g.replay()
            torch.cuda.synchronize()
            with pytest.raises(m.VlaqError) as ei:
                m.vlaq_check()
            assert ei.value.status == 6 and torch.equal(Y, want)
            m.vlaq_check()
