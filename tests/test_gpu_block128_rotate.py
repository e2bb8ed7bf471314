"""The rotated block quantizer for many blocks by name: few blocks against the
oracle (a call chooses it past 30000 activation blocks), and its give-up."""
import numpy as np
import pytest
import torch

import oracle
import synthetic_inputs as si
from gpu_helpers import bits, vq

pytestmark = pytest.mark.gpu

HAD = 2


# one row; a tile and a row; 64 columns behind the last whole block; more tiles
# than resident CTAs
@pytest.mark.parametrize("rows,K", [(1, 64), (129, 192), (5, 3584), (128, 1088), (300, 18944)])
@pytest.mark.parametrize("weight", [0, 1])
def test_few_blocks_equal_the_oracle(rows, K, weight):
    m = vq()
    X = si.projection_activations(K, rows, 17)
    ref = oracle.quantize_weight_fp8_block(bits(X), HAD) if weight else oracle.quantize_fp8_block(bits(X), None, 1e-6, HAD)
    codes, s = m.alloc_fp8_block(rows, K, weight=bool(weight))
    s.fill_(float("nan"))
    m.vlaq_selftest_rotate_fp8_block(weight, 0, X.cuda(), rows, K, codes, s)
    assert np.array_equal(s.cpu().numpy().view(np.uint32), ref[1].view(np.uint32))
    assert np.array_equal(codes.cpu().numpy(), ref[0])


@pytest.mark.parametrize("rows,K", [(1, 64), (300, 18944)])
@pytest.mark.parametrize("weight", [0, 1])
def test_a_call_that_gives_up_writes_nothing(rows, K, weight):
    """Status once, outputs as they were, no CTA leaves before its copies have
    had their time (2^21 clocks after the 2 million of the wait), and the call
    behind it on the stream is right."""
    m = vq()
    X = si.projection_activations(K, rows, 18).cuda()
    codes, s = m.alloc_fp8_block(rows, K, weight=bool(weight))
    want, ws = m.alloc_fp8_block(rows, K, weight=bool(weight))
    m.vlaq_selftest_rotate_fp8_block(weight, 0, X, rows, K, want, ws)
    codes.fill_(0x11), s.fill_(5.0)
    torch.cuda.synchronize()
    m.vlaq_check()
    a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    a.record()
    m.vlaq_selftest_rotate_fp8_block(weight, 1, X, rows, K, codes, s)
    b.record()
    c2, s2 = torch.empty_like(codes), torch.empty_like(s)
    m.vlaq_selftest_rotate_fp8_block(weight, 0, X, rows, K, c2, s2)
    torch.cuda.synchronize()
    with pytest.raises(m.VlaqError) as ei:
        m.vlaq_check()
    assert ei.value.status == 6
    m.vlaq_check()
    assert (codes == 0x11).all() and (s == 5.0).all()
    assert torch.equal(c2, want) and torch.equal(s2, ws)
    assert a.elapsed_time(b) >= (2_000_000 + 2 ** 21) / 1.965e6
