"""What the plan query and the self test of the FP8 block linear refuse,
without a GPU."""
import ctypes

import pytest
import torch

from test_block128_host import FAKE, refused, vq  # noqa: F401  (vq is a fixture)


def _self(vq, kernel, ctas, M=40, N=64, K=1024, starve=0, xq=FAKE, s_x=FAKE, wq=FAKE, s_w=FAKE, R=None, Y=FAKE):
    vq.vlaq_selftest_linear_fp8_block(kernel, ctas, starve, xq, s_x, wq, s_w, R, Y, M, N, K)


def test_plans_that_no_kernel_runs_are_refused(vq):  # noqa: F811
    for kernel, ctas in ((-1, 1), (3, 1), (0, 0), (0, 9), (0, -2), (1, 0), (1, 9), (2, 1), (2, 3), (2, 8)):
        refused(vq, 1, lambda: _self(vq, kernel, ctas), "CTAs per tile")
    refused(vq, 1, lambda: _self(vq, 0, 2, M=65), "CTAs per tile")  # 64 tokens at most
    refused(vq, 1, lambda: _self(vq, 0, 3, K=256), "CTAs per tile")  # two blocks
    refused(vq, 1, lambda: _self(vq, 1, 2, K=128), "CTAs per tile")
    refused(vq, 1, lambda: _self(vq, 2, 4, K=112), "CTAs per tile")


def test_self_test_refuses_what_the_linear_refuses(vq):  # noqa: F811
    refused(vq, 2, lambda: _self(vq, 0, 1, N=60))
    refused(vq, 2, lambda: _self(vq, 0, 1, K=100))
    refused(vq, 1, lambda: _self(vq, 0, 1, M=-1))
    refused(vq, 1, lambda: _self(vq, 0, 1, M=0))
    for a in ("xq", "s_x", "wq", "s_w", "Y"):
        refused(vq, 1, lambda: _self(vq, 1, 2, **{a: None}), a)
        refused(vq, 3, lambda: _self(vq, 1, 2, **{a: FAKE + 8}), a)
    refused(vq, 3, lambda: _self(vq, 1, 2, R=FAKE + 2), "residual")


def test_plan_query_refuses_bad_shapes(vq):  # noqa: F811
    refused(vq, 2, lambda: vq.vlaq_linear_fp8_block_plan(4, 60, 256))
    refused(vq, 2, lambda: vq.vlaq_linear_fp8_block_plan(4, 64, 100))
    refused(vq, 1, lambda: vq.vlaq_linear_fp8_block_plan(-1, 64, 256))
    refused(vq, 1, lambda: vq.vlaq_linear_fp8_block_plan(0, 64, 256))
    n = ctypes.c_int32(7)
    assert vq._lib.vlaq_linear_fp8_block_plan(4, 64, 256, None, ctypes.byref(n)) == 1 and n.value == 7
    assert vq._lib.vlaq_linear_fp8_block_plan(4, 64, 256, ctypes.byref(n), None) == 1 and n.value == 7


def test_no_device_is_an_error(vq):  # noqa: F811
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    for call in (lambda: _self(vq, 1, 2), lambda: _self(vq, 2, 4, starve=1),
                 lambda: vq.vlaq_linear_fp8_block_plan(4, 64, 256)):
        with pytest.raises(vq.VlaqError) as ei:
            call()
        assert ei.value.status in (4, 5)


def test_rotate_self_test_refuses_bad_calls(vq):  # noqa: F811
    f = vq.vlaq_selftest_rotate_fp8_block
    refused(vq, 2, lambda: f(0, 0, FAKE, 0, 256, FAKE, FAKE))
    refused(vq, 2, lambda: f(0, 0, FAKE, 4, 96, FAKE, FAKE))
    refused(vq, 2, lambda: f(1, 0, FAKE, 4, 32832, FAKE, FAKE))
    for i in (2, 5, 6):
        args = [1, 1, FAKE, 4, 256, FAKE, FAKE]
        refused(vq, 1, lambda: f(*(None if j == i else a for j, a in enumerate(args))))
        refused(vq, 3, lambda: f(*(FAKE + 8 if j == i else a for j, a in enumerate(args))))
