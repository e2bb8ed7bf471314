"""The FP8 block-scaled linear, its quantizers and the residual norm: cases.

What is timed are five entry points of the library:

* ``vlaq_linear_fp8_block``        Y = sum_b s_x[b, m] s_w[n / 128, b] sum_{k in b} x w  (+ residual)
* ``vlaq_quantize_act_fp8_block``  bf16 rows -> E4M3 codes, one fp32 scale per 1 x 128 block
* ``vlaq_quantize_weight_fp8_block``  bf16 weight -> E4M3 codes, one fp32 scale per 128 x 128 block
* ``vlaq_residual_norm``           h' = h + alpha gate RMSNorm(y), x = RMSNorm(h'), both bf16
* ``vlaq_residual_norm_fp8_block`` the same with x as E4M3 codes and 1 x 128 block scales

``run`` with ``own`` false computes them with elementary torch operations in
fp32; with ``own`` true it makes the library's calls.  ``exact`` states the
definitions once more in fp64.  Shapes are those of the Qwen2.5-VL-7B
language backbone's projections (hidden 3584, qkv 4608, gate_up 37888, down
18944 -> 3584) at decode and prefill token counts, and ragged ones.
E4M3 codes are returned as ``float8_e4m3fn`` tensors: the values they hold.
"""
import math

import torch

own = False

BLOCK = 128
E4M3_MAX = 448.0
EPS = 1e-6
RMSNORM, HADAMARD64 = 1, 2  # flag bits of the prologue


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one token through the qkv projection: the latency of a decode step
        dict(name="linear M1 qkv", op="linear", M=1, N=4608, K=3584, residual=False),
        # eight tokens (a small decode batch) through down, added to the residual stream
        dict(name="linear M8 down", op="linear", M=8, N=3584, K=18944, residual=True),
        # a short prompt against a ragged projection: no size a multiple of a tile
        dict(name="linear M333 ragged", op="linear", M=333, N=1000, K=1040, residual=True),
        # a prefill chunk through gate_up, the widest projection
        dict(name="linear M1024 gate_up", op="linear", M=1024, N=37888, K=3584, residual=False),
        # the longest prompt (4580 tokens) through down, added to the residual stream
        dict(name="linear M4580 down", op="linear", M=4580, N=3584, K=18944, residual=True),
        # the prologue of one decoded token: RMSNorm and quantization
        dict(name="quant act M1 norm", op="act", M=1, K=3584, flags=RMSNORM),
        # the input of down in a prefill chunk: rotated, then quantized
        dict(name="quant act M1024 rot", op="act", M=1024, K=18944, flags=HADAMARD64),
        # offline weights: qkv, and gate_up (the largest tensor of a layer) rotated
        dict(name="quant weight qkv", op="weight", N=4608, K=3584, flags=0),
        dict(name="quant weight gate_up", op="weight", N=37888, K=3584, flags=HADAMARD64),
        # between the blocks of a decode step: post norm, residual, pre norm, quantized
        dict(name="resnorm M1 fp8", op="resnorm", M=1, K=3584, out="fp8", post=True, gate_rows=0, alpha=1.0, flags=0),
        # a prefill chunk of four sequences, each with its own gate vector, rotated and quantized
        dict(name="resnorm M1024 fp8 gate", op="resnorm", M=1024, K=3584, out="fp8", post=True, gate_rows=256,
             alpha=0.5, flags=HADAMARD64),
        # the longest prompt in bf16: plain pre-norm stream with a learned residual scale per channel
        dict(name="resnorm M4580 bf16", op="resnorm", M=4580, K=3584, out="bf16", post=False, gate_rows=4580,
             alpha=1.0, flags=0),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["linear", "linear", "act", "weight", "resnorm", "resnorm"])
    if op == "linear":
        # 1 .. 4580 tokens, any width (multiple of 8) and depth (multiple of 16) up to the widest projection's
        N = 8 * _log(rng, 8, 4736)
        K = 16 * _log(rng, 8, 1184)
        M = _log(rng, 1, 4580)
        M = max(1, min(M, int(6.0e11 / (2.0 * N * K)), int((2.0e8 - min(1.5e8, N * K)) / (2.0 * N + K))))
        if N * K > 1.3e8:
            N = max(8, int(1.3e8 / K) // 8 * 8)
        return dict(op=op, M=M, N=N, K=K, residual=rng.random() < 0.5)
    if op == "act":
        rot = rng.random() < 0.5
        K = 64 * _log(rng, 2, 296) if rot else 16 * _log(rng, 8, 1184)
        M = max(1, min(_log(rng, 1, 4580), int(1.3e8 / (3 * K))))
        return dict(op=op, M=M, K=K, flags=(HADAMARD64 if rot else 0) | (RMSNORM if rng.random() < 0.5 else 0))
    if op == "weight":
        rot = rng.random() < 0.5
        K = 64 * _log(rng, 2, 296) if rot else 16 * _log(rng, 8, 1184)
        N = max(1, min(_log(rng, 64, 37888), int(1.3e8 / K)))
        return dict(op=op, N=N, K=K, flags=HADAMARD64 if rot else 0)
    out = rng.choice(["fp8", "bf16"])
    rot = out == "fp8" and rng.random() < 0.5
    K = 64 * _log(rng, 2, 128) if rot else 16 * _log(rng, 8, 512)
    M = max(1, min(_log(rng, 1, 4580), int(1.3e8 / (8 * K))))
    gate_rows = rng.choice([0, 1, M, max(1, (M + 2) // 3)])
    return dict(op=op, M=M, K=K, out=out, post=rng.random() < 0.5, gate_rows=gate_rows,
                alpha=rng.choice([1.0, 0.5, 0.22]), flags=HADAMARD64 if rot else 0)


def work(case):
    op, K = case["op"], case["K"]
    blocks = -(-K // BLOCK)
    if op == "linear":
        M, N = case["M"], case["N"]
        b = M * K + N * K + 4 * blocks * (M + -(-N // BLOCK)) + 2 * M * N * (2 if case["residual"] else 1)
        return {"bytes": float(b), "flops": 2.0 * M * N * K}
    if op == "act":
        M = case["M"]
        b = 3 * M * K + 4 * blocks * M + (2 * K if case["flags"] & RMSNORM else 0)
        f = 2 + (4 if case["flags"] & RMSNORM else 0) + (7 if case["flags"] & HADAMARD64 else 0)
        return {"bytes": float(b), "flops": float(f * M * K)}
    if op == "weight":
        N = case["N"]
        b = 3 * N * K + 4 * blocks * -(-N // BLOCK)
        return {"bytes": float(b), "flops": float((2 + (7 if case["flags"] else 0)) * N * K)}
    M, gr = case["M"], case["gate_rows"]
    b = M * K * (2 + 2 + 2) + 2 * K + (2 * K if case["post"] else 0) + (2 * K * -(-M // gr) if gr else 0)
    b += 2 * M * K if case["out"] == "bf16" else M * K + 4 * blocks * M
    f = 2 + 4 + (4 if case["post"] else 0) + (1 if gr else 0) + (2 if case["out"] == "fp8" else 0)
    return {"bytes": float(b), "flops": float((f + (7 if case["flags"] else 0)) * M * K)}


# ----------------------------------------------------------- plain forms
def _hadamard(device, dtype=torch.float32):
    """Normalised Sylvester Hadamard matrix of order 64: (-1)^popcount(i & j) / 8."""
    i = torch.arange(64, device=device)
    b = i[:, None] & i[None, :]
    odd = (b ^ (b >> 1) ^ (b >> 2) ^ (b >> 3) ^ (b >> 4) ^ (b >> 5)) & 1
    return (1 - 2 * odd).to(dtype) / 8


def _rotate(x, had):
    return (x.reshape(-1, 64) @ had).reshape(x.shape)


def _rmsnorm(x, gamma, eps):
    r = 1.0 / torch.sqrt(x.square().mean(-1, keepdim=True) + eps)
    return x * r * gamma.float()


def _pad_last(x, n):
    return torch.nn.functional.pad(x, (0, n - x.shape[-1])) if x.shape[-1] != n else x


def _codes(x, s):
    """E4M3 of x / s (0 where s = 0), s broadcast over x."""
    q = torch.where(s > 0, x / s, torch.zeros_like(x))
    return q.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)


def _quantize_rows(x):
    """fp32 [M, K] -> (codes [M, K], scales [blocks, M])."""
    M, K = x.shape
    blocks = -(-K // BLOCK)
    xb = _pad_last(x, blocks * BLOCK).reshape(M, blocks, BLOCK)
    s = xb.abs().amax(-1) / E4M3_MAX
    codes = _codes(xb, s[:, :, None]).view(torch.uint8).reshape(M, blocks * BLOCK)[:, :K].contiguous()
    return codes.view(torch.float8_e4m3fn), s.t().contiguous()


def _quantize_weight(w):
    """fp32 [N, K] -> (codes [N, K], scales [ceil(N / 128), ceil(K / 128)])."""
    N, K = w.shape
    nb, kb = -(-N // BLOCK), -(-K // BLOCK)
    wp = torch.nn.functional.pad(w, (0, kb * BLOCK - K, 0, nb * BLOCK - N)).reshape(nb, BLOCK, kb, BLOCK)
    s = wp.abs().amax((1, 3)) / E4M3_MAX
    codes = _codes(wp, s[:, None, :, None]).view(torch.uint8).reshape(nb * BLOCK, kb * BLOCK)[:N, :K].contiguous()
    return codes.view(torch.float8_e4m3fn), s


def _linear(xq, sx, wq, sw, residual):
    M, K = xq.shape
    N = wq.shape[0]
    x = xq.float() * sx.t().repeat_interleave(BLOCK, 1)[:, :K]
    w = wq.float() * sw.repeat_interleave(BLOCK, 0)[:N].repeat_interleave(BLOCK, 1)[:, :K]
    y = x @ w.t()
    if residual is not None:
        y = y + residual.float()
    return y.to(torch.bfloat16)


def _residual_norm(s):
    """(h' in fp32, x in fp32)."""
    y = s["y"].float()
    t = _rmsnorm(y, s["gamma_post"], EPS) if s["gamma_post"] is not None else y
    if s["gate"] is not None:
        M = y.shape[0]
        t = t * s["gate"].float().repeat_interleave(s["gate_rows"], 0)[:M]
    h = s["h"].float() + t * s["alpha"]
    return h, _rmsnorm(h, s["gamma_pre"], EPS)


# ------------------------------------------------------------------ inputs
def _gen(seed, stream):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 16 + stream)
    return g


def _acts(M, K, seed, stream):
    """N(0, 1) times a lognormal scale per channel: activations with outlier channels."""
    c = torch.exp(torch.randn(K, generator=_gen(seed, stream), device="cuda"))
    return (torch.randn(M, K, generator=_gen(seed, stream + 1), device="cuda") * c).to(torch.bfloat16)


def _weight(N, K, seed):
    return (torch.randn(N, K, generator=_gen(seed, 4), device="cuda") / math.sqrt(K)).to(torch.bfloat16)


def _gain(K, seed, stream):
    return (0.5 + torch.rand(K, generator=_gen(seed, stream), device="cuda")).to(torch.bfloat16)


def prepare(case, seed):
    op, K = case["op"], case["K"]
    blocks = -(-K // BLOCK)
    s = dict(case)
    if op == "linear":
        M, N = case["M"], case["N"]
        s["xq"], s["sx"] = _quantize_rows(_acts(M, K, seed, 0).float())
        s["wq"], s["sw"] = _quantize_weight(_weight(N, K, seed).float())
        s["residual"] = torch.randn(M, N, generator=_gen(seed, 6), device="cuda").to(torch.bfloat16) \
            if case["residual"] else None
        s["Y"] = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
        return s
    if op == "weight":
        N = case["N"]
        s["W"] = _weight(N, K, seed)
        s["codes"] = torch.empty(N, K, dtype=torch.float8_e4m3fn, device="cuda")
        s["scales"] = torch.empty(-(-N // BLOCK), blocks, device="cuda")
    else:
        M = case["M"]
        s["codes"] = torch.empty(M, K, dtype=torch.float8_e4m3fn, device="cuda")
        s["scales"] = torch.empty(blocks, M, device="cuda")
    if op == "act":
        s["X"] = _acts(M, K, seed, 0)
        s["gamma"] = _gain(K, seed, 2) if case["flags"] & RMSNORM else None
    if op == "resnorm":
        s["h"], s["y"] = _acts(M, K, seed, 0), _acts(M, K, seed, 2)
        s["gamma_post"] = _gain(K, seed, 5) if case["post"] else None
        s["gamma_pre"] = _gain(K, seed, 6)
        gr = case["gate_rows"]
        s["gate"] = (0.1 * torch.randn(-(-M // gr), K, generator=_gen(seed, 7), device="cuda")).to(torch.bfloat16) \
            if gr else None
        s["h_out"] = torch.empty(M, K, dtype=torch.bfloat16, device="cuda")
        s["x_out"] = torch.empty(M, K, dtype=torch.bfloat16, device="cuda")
    s["had"] = _hadamard("cuda") if case["flags"] & HADAMARD64 else None
    return s


# --------------------------------------------------------------------- run
def run(s):
    if own:
        return _run_own(s)
    op = s["op"]
    if op == "linear":
        return {"y": _linear(s["xq"], s["sx"], s["wq"], s["sw"], s["residual"])}
    if op == "act":
        x = s["X"].float()
        if s["gamma"] is not None:
            x = _rmsnorm(x, s["gamma"], EPS)
        codes, scales = _quantize_rows(x if s["had"] is None else _rotate(x, s["had"]))
        return {"codes": codes, "scales": scales}
    if op == "weight":
        w = s["W"].float()
        codes, scales = _quantize_weight(w if s["had"] is None else _rotate(w, s["had"]))
        return {"codes": codes, "scales": scales}
    h, x = _residual_norm(s)
    if s["out"] == "bf16":
        return {"h": h.to(torch.bfloat16), "x": x.to(torch.bfloat16)}
    codes, scales = _quantize_rows(x if s["had"] is None else _rotate(x, s["had"]))
    return {"h": h.to(torch.bfloat16), "codes": codes, "scales": scales}


def _run_own(s):
    import vlaq_quantize_act_b200 as vq

    op, K = s["op"], s["K"]
    if op == "linear":
        vq.vlaq_linear_fp8_block(s["xq"], s["sx"], s["wq"], s["sw"], s["residual"], s["Y"], s["M"], s["N"], K)
        return {"y": s["Y"]}
    if op == "act":
        vq.vlaq_quantize_act_fp8_block(s["X"], s["M"], K, s["gamma"], EPS, s["flags"], s["codes"], s["scales"])
        return {"codes": s["codes"], "scales": s["scales"]}
    if op == "weight":
        vq.vlaq_quantize_weight_fp8_block(s["W"], s["N"], K, s["flags"], s["codes"], s["scales"])
        return {"codes": s["codes"], "scales": s["scales"]}
    if s["out"] == "bf16":
        vq.vlaq_residual_norm(s["h"], s["y"], s["M"], K, s["gamma_post"], s["gate"], s["gate_rows"], s["alpha"],
                              s["gamma_pre"], EPS, s["h_out"], s["x_out"])
        return {"h": s["h_out"], "x": s["x_out"]}
    vq.vlaq_residual_norm_fp8_block(s["h"], s["y"], s["M"], K, s["gamma_post"], s["gate"], s["gate_rows"], s["alpha"],
                                    s["gamma_pre"], EPS, s["flags"], s["h_out"], s["codes"], s["scales"])
    return {"h": s["h_out"], "codes": s["codes"], "scales": s["scales"]}


# ------------------------------------------------------------------- exact
def _e4m3_f64(v):
    """fp64 -> the nearest E4M3 value (ties to even, saturating at 448), in fp64."""
    a = v.abs()
    e = torch.floor(torch.log2(a.clamp_min(2.0 ** -9))).clamp_min(-6.0)
    step = torch.exp2(e - 3.0)
    return torch.sign(v) * (torch.round(a / step) * step).clamp_max(448.0)


def _rot_f64(x):
    """Walsh-Hadamard transform of each 64-group by the doubling recurrence, over 8."""
    t = x.reshape(-1, 64)
    for h in (1, 2, 4, 8, 16, 32):
        p = t.reshape(-1, 64 // (2 * h), 2, h)
        t = torch.stack((p[:, :, 0] + p[:, :, 1], p[:, :, 0] - p[:, :, 1]), 2).reshape(-1, 64)
    return (t / 8.0).reshape(x.shape)


def _blocks_f64(x):
    """(codes, scales [blocks, rows]) of fp64 rows, block by block along K."""
    codes, scales = torch.zeros_like(x), []
    for k in range(0, x.shape[1], 128):
        v = x[:, k:k + 128]
        s = v.abs().amax(1) / 448.0
        codes[:, k:k + 128] = torch.where(s[:, None] > 0, _e4m3_f64(v / s.clamp_min(1e-300)[:, None]), 0.0)
        scales.append(s)
    return codes, torch.stack(scales)


def _norm_f64(x, gamma):
    return x / (x.pow(2).sum(1, keepdim=True) / x.shape[1] + EPS).sqrt() * gamma.double()


def exact(case, seed):
    s = prepare(case, seed)
    op, K = case["op"], case["K"]
    if op == "linear":
        M, N = case["M"], case["N"]
        y = torch.zeros(M, N, dtype=torch.float64, device="cuda")
        for b in range(-(-K // 128)):
            k = slice(128 * b, min(K, 128 * b + 128))
            rows = s["sw"][:, b].double()[torch.arange(N, device="cuda") // 128]
            y += (s["xq"][:, k].double() * s["sx"][b].double()[:, None]) @ (s["wq"][:, k].double() * rows[:, None]).t()
        return {"y": y if s["residual"] is None else y + s["residual"].double()}
    if op == "act":
        x = s["X"].double()
        x = x if s["gamma"] is None else _norm_f64(x, s["gamma"])
        codes, scales = _blocks_f64(_rot_f64(x) if case["flags"] & HADAMARD64 else x)
        return {"codes": codes, "scales": scales}
    if op == "weight":
        w = s["W"].double()
        w = _rot_f64(w) if case["flags"] & HADAMARD64 else w
        codes, scales = torch.empty_like(w), []
        for n in range(0, case["N"], 128):
            row = []
            for k in range(0, K, 128):
                v = w[n:n + 128, k:k + 128]
                row.append(v.abs().amax() / 448.0)
                codes[n:n + 128, k:k + 128] = _e4m3_f64(v / row[-1].clamp_min(1e-300))
            scales.append(torch.stack(row))
        return {"codes": codes, "scales": torch.stack(scales)}
    t = s["y"].double()
    t = t if s["gamma_post"] is None else _norm_f64(t, s["gamma_post"])
    if s["gate"] is not None:
        t = t * s["gate"].double()[torch.arange(case["M"], device="cuda") // case["gate_rows"]]
    h = s["h"].double() + case["alpha"] * t
    x = _norm_f64(h, s["gamma_pre"])
    if case["out"] == "bf16":
        return {"h": h, "x": x}
    codes, scales = _blocks_f64(_rot_f64(x) if case["flags"] & HADAMARD64 else x)
    return {"h": h, "codes": codes, "scales": scales}
