"""Each kernel of the FP8 block linear by name: every cluster size against the
fp64 product whatever the plan prefers, and the plan that a shape gets."""
import pytest
import torch

import oracle
from gpu_helpers import bits, residual_f64, to_dev, vq
from test_gpu_block128 import _check_gemm, _linear_case

pytestmark = pytest.mark.gpu

COLS, ROWS, PAIR = 0, 1, 2
NAN = float("nan")


# ------------------------------------------------------------ every cluster
# ragged tokens, widths past a tile and a last block of 16, 80 or 112 columns;
# ranges of one block per CTA (nine blocks over eight), of several, uneven ones
@pytest.mark.parametrize("kernel,M,N,K", [(COLS, 1, 136, 1040), (COLS, 16, 264, 2128), (COLS, 29, 392, 1136),
                                          (COLS, 32, 128, 5104), (COLS, 33, 136, 2000), (COLS, 64, 520, 1040),
                                          (ROWS, 40, 264, 4112), (ROWS, 64, 392, 1136), (ROWS, 130, 136, 1040),
                                          (ROWS, 255, 520, 2128), (ROWS, 384, 384, 3584)])
@pytest.mark.parametrize("residual", [False, True])
def test_every_cluster_size_equals_the_fp64_product(kernel, M, N, K, residual):
    m = vq()
    ops, R, dx, dw = _linear_case(M, N, K, 47, residual)
    d = [to_dev(t) for t in ops]
    Rd = None if R is None else R.cuda()
    Y64, mass = oracle.linear_f64(dx, dw, None if R is None else bits(R)), residual_f64(R)
    for ctas in range(1, 9):
        Y = torch.full((M + 8, N), NAN, dtype=torch.bfloat16, device="cuda")
        m.vlaq_selftest_linear_fp8_block(kernel, ctas, 0, *d, Rd, Y, M, N, K)
        torch.cuda.synchronize()
        m.vlaq_check()
        assert torch.isnan(Y[M:]).all(), f"{ctas} CTAs: rows behind the last were written"
        _check_gemm(Y[:M].float().cpu().numpy(), Y64, dx, dw, K, mass, f"kernel {kernel}, {ctas} CTAs")
        if residual:
            Z = Rd.clone()
            m.vlaq_selftest_linear_fp8_block(kernel, ctas, 0, *d, Z, Z, M, N, K)
            assert torch.equal(Z, Y[:M]), f"{ctas} CTAs: in-place residual"


# fewer tokens and columns than a tile, one tile and several, two blocks (one
# for each pair), an odd number of them, a short last one
@pytest.mark.parametrize("M,N,K", [(3, 40, 256), (257, 264, 144), (300, 520, 2128), (130, 1000, 1040), (1, 256, 5104)])
@pytest.mark.parametrize("residual", [False, True])
def test_both_pair_forms_equal_the_fp64_product(M, N, K, residual):
    m = vq()
    ops, R, dx, dw = _linear_case(M, N, K, 53, residual)
    d = [to_dev(t) for t in ops]
    Rd = None if R is None else R.cuda()
    Y64, mass = oracle.linear_f64(dx, dw, None if R is None else bits(R)), residual_f64(R)
    for ctas in (2, 4):
        Y = torch.full((M + 8, N), NAN, dtype=torch.bfloat16, device="cuda")
        m.vlaq_selftest_linear_fp8_block(PAIR, ctas, 0, *d, Rd, Y, M, N, K)
        torch.cuda.synchronize()
        m.vlaq_check()
        assert torch.isnan(Y[M:]).all(), f"{ctas} CTAs: rows behind the last were written"
        _check_gemm(Y[:M].float().cpu().numpy(), Y64, dx, dw, K, mass, f"pairs, {ctas} CTAs")
        if residual:
            Z = Rd.clone()
            m.vlaq_selftest_linear_fp8_block(PAIR, ctas, 0, *d, Z, Z, M, N, K)
            assert torch.equal(Z, Y[:M]), f"{ctas} CTAs: in-place residual"


# --------------------------------------------------------------------- plans
# shapes far from the borders between plans: the kernel, and whether a tile is
# shared by several CTAs (or pairs)
@pytest.mark.parametrize("M,N,K,kernel,shared", [(1, 4608, 3584, COLS, True), (32, 512, 2048, COLS, True),
                                                 (8, 37888, 3584, COLS, False), (64, 512, 512, COLS, True),
                                                 (64, 37888, 3584, ROWS, False), (128, 3584, 3584, ROWS, True),
                                                 (100, 256, 4096, ROWS, True), (512, 3584, 3584, ROWS, False),
                                                 (1024, 8192, 2048, PAIR, False), (512, 3584, 18944, PAIR, True)])
def test_plan_of_a_shape_is_what_a_call_runs(M, N, K, kernel, shared):
    m = vq()
    plan = m.vlaq_linear_fp8_block_plan(M, N, K)
    assert plan[0] == kernel and (plan[1] > (2 if kernel == PAIR else 1)) == shared, plan
    gen = torch.Generator(device="cuda")
    gen.manual_seed(M + N)
    kb, nb = -(-K // 128), -(-N // 128)
    code = [torch.randint(0, 0x60, (r, K), generator=gen, device="cuda", dtype=torch.uint8) for r in (M, N)]
    scale = [torch.rand(*s, generator=gen, device="cuda") for s in ((kb, M), (nb, kb))]
    Y, Z = (torch.empty(M, N, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    m.vlaq_linear_fp8_block(code[0], scale[0], code[1], scale[1], None, Y, M, N, K)
    m.vlaq_selftest_linear_fp8_block(*plan, 0, code[0], scale[0], code[1], scale[1], None, Z, M, N, K)
    assert torch.equal(Y, Z)
