"""FP8 block-128 linear, its quantizers and the residual norm, without a GPU:
what the entry points refuse (before any launch), buffer shapes, and the
oracle held to the definitions in fp64 and to hand-made rows."""
import numpy as np
import pytest
import torch

import oracle
import synthetic_inputs as si

FAKE = 0x10000  # never dereferenced: validation fails (or M == 0) before any use


@pytest.fixture(scope="module")
def vq():
    from conftest import build_library
    build_library()
    import vlaq_quantize_act_b200 as vq
    return vq


def refused(vq, status, call, text=None):
    with pytest.raises(vq.VlaqError) as ei:
        call()
    assert ei.value.status == status, ei.value
    if text:
        assert text in ei.value.message


def _norm(vq, fp8=False, H=FAKE, Y=FAKE, M=4, K=256, gp=FAKE, gate=None, gr=0, alpha=1.0, g=FAKE, flags=0, h=FAKE,
          x=FAKE, codes=FAKE, s=FAKE):
    if fp8:
        return vq.vlaq_residual_norm_fp8_block(H, Y, M, K, gp, gate, gr, alpha, g, 1e-6, flags, h, codes, s)
    return vq.vlaq_residual_norm(H, Y, M, K, gp, gate, gr, alpha, g, 1e-6, h, x)


def test_shapes_are_refused(vq):
    refused(vq, 2, lambda: vq.vlaq_quantize_act_fp8_block(FAKE, 4, 3420, None, 1e-6, 0, FAKE, FAKE), "213.75")
    refused(vq, 2, lambda: vq.vlaq_quantize_act_fp8_block(FAKE, 4, 336, None, 1e-6, vq.F_HADAMARD64, FAKE, FAKE))
    refused(vq, 2, lambda: vq.vlaq_quantize_act_fp8_block(FAKE, 4, 65536, None, 1e-6, 0, FAKE, FAKE))
    refused(vq, 2, lambda: vq.vlaq_quantize_act_fp8_block(FAKE, 1 << 31, 256, None, 1e-6, 0, FAKE, FAKE))
    refused(vq, 1, lambda: vq.vlaq_quantize_act_fp8_block(FAKE, -1, 256, None, 1e-6, 0, FAKE, FAKE))
    refused(vq, 2, lambda: vq.vlaq_quantize_weight_fp8_block(FAKE, 0, 256, 0, FAKE, FAKE))
    refused(vq, 2, lambda: vq.vlaq_quantize_weight_fp8_block(FAKE, 64, 96, vq.F_HADAMARD64, FAKE, FAKE))
    refused(vq, 2, lambda: vq.vlaq_linear_fp8_block(FAKE, FAKE, FAKE, FAKE, None, FAKE, 4, 60, 256))
    refused(vq, 2, lambda: vq.vlaq_linear_fp8_block(FAKE, FAKE, FAKE, FAKE, None, FAKE, 4, 64, 100))
    refused(vq, 2, lambda: vq.vlaq_linear_fp8_block(FAKE, FAKE, FAKE, FAKE, None, FAKE, 1 << 30, 1 << 20, 256))
    refused(vq, 1, lambda: vq.vlaq_linear_fp8_block(FAKE, FAKE, FAKE, FAKE, None, FAKE, -1, 64, 256))
    for fp8 in (False, True):
        refused(vq, 2, lambda: _norm(vq, fp8, K=24))
        refused(vq, 2, lambda: _norm(vq, fp8, K=65536))
        refused(vq, 1, lambda: _norm(vq, fp8, M=-2))
    refused(vq, 2, lambda: _norm(vq, True, K=80, flags=vq.F_HADAMARD64))


def test_flags_pointers_and_scalars_are_refused(vq):
    refused(vq, 1, lambda: vq.vlaq_quantize_act_fp8_block(FAKE, 4, 256, None, 1e-6, 4, FAKE, FAKE))
    refused(vq, 1, lambda: vq.vlaq_quantize_act_fp8_block(FAKE, 4, 256, None, 1e-6, vq.F_RMSNORM, FAKE, FAKE))
    refused(vq, 1, lambda: vq.vlaq_quantize_weight_fp8_block(FAKE, 64, 256, vq.F_RMSNORM, FAKE, FAKE))
    refused(vq, 3, lambda: vq.vlaq_quantize_weight_fp8_block(FAKE + 8, 64, 256, 0, FAKE, FAKE))
    refused(vq, 1, lambda: vq.vlaq_linear_fp8_block(FAKE, None, FAKE, FAKE, None, FAKE, 4, 64, 256))
    refused(vq, 3, lambda: vq.vlaq_linear_fp8_block(FAKE, FAKE + 4, FAKE, FAKE, None, FAKE, 4, 64, 256))
    refused(vq, 3, lambda: vq.vlaq_linear_fp8_block(FAKE, FAKE, FAKE, FAKE, FAKE + 2, FAKE, 4, 64, 256))
    for fp8 in (False, True):
        refused(vq, 1, lambda: _norm(vq, fp8, H=None))
        refused(vq, 1, lambda: _norm(vq, fp8, Y=None))
        refused(vq, 1, lambda: _norm(vq, fp8, h=None))
        refused(vq, 1, lambda: _norm(vq, fp8, g=None))
        refused(vq, 3, lambda: _norm(vq, fp8, gp=FAKE + 8))
        refused(vq, 3, lambda: _norm(vq, fp8, gate=FAKE + 8, gr=1))
        refused(vq, 1, lambda: _norm(vq, fp8, gate=FAKE, gr=0), "gate_rows")
        refused(vq, 1, lambda: _norm(vq, fp8, alpha=float("nan")), "alpha")
        refused(vq, 1, lambda: _norm(vq, fp8, alpha=float("inf")), "alpha")
    refused(vq, 3, lambda: _norm(vq, x=FAKE + 8))
    refused(vq, 1, lambda: _norm(vq, True, codes=None))
    refused(vq, 1, lambda: _norm(vq, True, s=None))
    refused(vq, 1, lambda: _norm(vq, True, flags=vq.F_RMSNORM))


def test_no_rows_is_a_noop(vq):
    vq.vlaq_quantize_act_fp8_block(None, 0, 256, None, 1e-6, 0, None, None)
    vq.vlaq_linear_fp8_block(None, None, None, None, None, None, 0, 64, 256)
    _norm(vq, H=None, Y=None, M=0, h=None, x=None, g=None)
    _norm(vq, True, H=None, Y=None, M=0, h=None, codes=None, s=None, g=None)
    assert vq.vlaq_last_error() == ""


def test_no_device_is_an_error(vq):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    for call in (lambda: vq.vlaq_quantize_act_fp8_block(FAKE, 4, 256, None, 1e-6, 0, FAKE, FAKE),
                 lambda: vq.vlaq_quantize_weight_fp8_block(FAKE, 64, 256, 0, FAKE, FAKE),
                 lambda: vq.vlaq_linear_fp8_block(FAKE, FAKE, FAKE, FAKE, None, FAKE, 4, 64, 256),
                 lambda: _norm(vq), lambda: _norm(vq, True), lambda: _norm(vq, x=None, g=None)):
        with pytest.raises(vq.VlaqError) as ei:
            call()
        assert ei.value.status in (4, 5)


def test_alloc_shapes(vq):
    c, s = vq.alloc_fp8_block(5, 336, device="cpu")
    assert c.shape == (5, 336) and s.shape == (3, 5)
    c, s = vq.alloc_fp8_block(129, 336, device="cpu", weight=True)
    assert c.shape == (129, 336) and s.shape == (2, 3)


# ------------------------------------------------------------- oracle pins
def _rows(M, K, seed):
    return si.projection_activations(K, M, seed)


def test_sumsq_tree256_order():
    """A row whose fp32 sum depends on the order: the tree written out here
    with numpy (products of these bf16-like values are exact in fp32, so a
    fused multiply-add is a plain add of the exact product)."""
    rng = np.random.default_rng(1)
    for K in (16, 2048, 2064, 3584, 8192):
        x = (rng.integers(1, 64, K) * 2.0 ** rng.integers(-6, 7, K)).astype(np.float32)
        lane = np.zeros(256, np.float32)
        sq = (x.astype(np.float64) ** 2).astype(np.float32)
        for c in range(K // 16):
            for e in range(16):
                lane[c % 256] = np.float32(lane[c % 256] + sq[16 * c + e])
        g = lane.reshape(8, 32)
        for w in (16, 8, 4, 2, 1):
            g = (g[:, :w] + g[:, w:2 * w]).astype(np.float32)
        g = g[:, 0]
        for _ in range(3):
            g = (g[0::2] + g[1::2]).astype(np.float32)
        assert oracle.sumsq_tree256(x) == g[0], K


@pytest.mark.parametrize("M,K,flags", [(5, 16, 0), (4, 144, 0), (3, 336, 1), (2, 2176, 2), (3, 3584, 3)])
def test_oracle_act_blocks_meet_the_definition(M, K, flags):
    """Scales within the roundings of the transform, codes within half a step
    of the exact quotient (plus what the scale's and the transform's fp32
    roundings move it), the block's largest element at code 448."""
    X = _rows(M, K, 7)
    gam = si.norm_gain(K, 7)
    codes, s = oracle.quantize_fp8_block(si.to_bits(X), si.to_bits(gam), 1e-6, flags)
    x = X.double().numpy()
    if flags & 1:
        x = x / np.sqrt((x ** 2).mean(1, keepdims=True) + 1e-6) * gam.double().numpy()
    if flags & 2:
        i = np.arange(64)
        had = np.array([[(-1) ** bin(a & b).count("1") for b in i] for a in i]) / 8.0
        x = (x.reshape(M, -1, 64) @ had).reshape(M, K)
    # fp32 roundings relative to the block's amax: the sum of squares (K adds
    # of positive terms, halved by the root), five more in the norm, six
    # butterfly stages whose terms sum to at most 64 amax / 8
    u = 2.0 ** -24
    rel = (K / 2 + 5) * u * (flags & 1) + 6 * 8 * u * ((flags >> 1) & 1) + 2 * u
    dec = oracle.decode_fp8_block(codes, s)
    table = np.array([oracle.e4m3_decode(c) for c in range(256)])
    for b in range(-(-K // 128)):
        v = x[:, 128 * b:128 * b + 128]
        amax = np.abs(v).max(1)
        assert np.all(np.abs(s[b] - amax / 448.0) <= (rel + u) * 8 * amax / 448.0)
        q = np.abs(table[codes[:, 128 * b:128 * b + 128]])
        assert np.all(q.max(1) == 448.0)
        err = np.abs(dec[:, 128 * b:128 * b + 128] - v)
        # half a step: 2^-4 of the value, 2^-10 of the scale below 2^-6
        tol = np.maximum(np.abs(v) * 2.0 ** -4, s[b][:, None] * 2.0 ** -10) + 8 * rel * amax[:, None]
        assert np.all(err <= tol)


def test_oracle_weight_blocks_meet_the_definition():
    W = si.projection_weight(336, 200, 3)
    codes, s = oracle.quantize_weight_fp8_block(si.to_bits(W))
    w = W.double().numpy()
    dec = oracle.decode_weight_fp8_block(codes, s)
    for n in range(0, 200, 128):
        for k in range(0, 336, 128):
            v = w[n:n + 128, k:k + 128]
            a = np.float32(np.abs(v).max())
            assert s[n // 128, k // 128] == a / np.float32(448.0)
            sb = float(s[n // 128, k // 128])
            assert np.all(np.abs(dec[n:n + 128, k:k + 128] - v)
                          <= np.maximum(np.abs(v) * 2.0 ** -4, sb * 2.0 ** -10) * (1 + 2.0 ** -20))


def test_oracle_blocks_equal_the_per_row_quantizer_on_one_block():
    """A row of one block is the per-row FP8 quantization of it."""
    X = _rows(9, 128, 5)
    cb, sb = oracle.quantize_fp8_block(si.to_bits(X))
    cr, sr = oracle.quantize_fp8(si.to_bits(X))
    assert np.array_equal(cb, cr) and np.array_equal(sb[0], sr)


def test_oracle_zero_blocks():
    X = torch.zeros(3, 384, dtype=torch.bfloat16)
    X[1, 130] = -2.0
    codes, s = oracle.quantize_fp8_block(si.to_bits(X))
    assert s[1, 1] == np.float32(2.0) / np.float32(448.0) and codes[1, 130] == 0xFE
    assert np.count_nonzero(s) == 1 and np.count_nonzero(codes) == 1


@pytest.mark.parametrize("post,gate_rows,alpha", [(True, 0, 1.0), (False, 1, 0.5), (True, 2, 0.22), (False, 9, 1.0)])
def test_oracle_residual_norm_meets_the_definition(post, gate_rows, alpha):
    M, K = 5, 272
    h, y = _rows(M, K, 11), _rows(M, K, 12)
    gp, g = si.norm_gain(K, 13), si.norm_gain(K, 14)
    gate = torch.randn(-(-M // gate_rows), K).to(torch.bfloat16) if gate_rows else None
    ho, xo = oracle.residual_norm(si.to_bits(h), si.to_bits(y), si.to_bits(gp) if post else None,
                                  None if gate is None else si.to_bits(gate), gate_rows, alpha, si.to_bits(g))

    def norm(v, w):
        return v / np.sqrt((v ** 2).mean(1, keepdims=True) + 1e-6) * w.double().numpy()

    t = y.double().numpy()
    t = norm(t, gp) if post else t
    if gate is not None:
        t = t * gate.double().numpy()[np.arange(M) // gate_rows]
    c = h.double().numpy() + np.float64(np.float32(alpha)) * t
    x = norm(c, g)

    def f(b):
        return torch.from_numpy(b.view(np.int16)).view(torch.bfloat16).double().numpy()

    # one bf16 rounding (2^-8 of the value) on top of fp32 roundings: K / 2
    # for a norm's sum plus a few, relative to the terms of each sum
    u = 2.0 ** -24
    e1 = (K / 2 + 10) * u * (np.abs(t) * alpha + np.abs(h.double().numpy()))
    assert np.all(np.abs(f(ho) - c) <= np.abs(c) * 2.0 ** -8 + 2 * e1 + 1e-30)
    e2 = e1 / np.maximum(np.abs(c), 1e-30) * np.abs(x) + (K + 10) * u * np.abs(x)
    assert np.all(np.abs(f(xo) - x) <= np.abs(x) * 2.0 ** -8 + 2 * e2 + 1e-30)
