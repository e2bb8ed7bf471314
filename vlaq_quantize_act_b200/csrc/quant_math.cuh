// Arithmetic shared by the quantizer kernels: bf16 unpacking, correctly
// rounded quotients and the scale of a group of values from its amax.  Every
// fp32 operation is an explicitly rounded intrinsic (no contraction).
#pragma once

#include <cstdint>

#include "ptx.cuh"

namespace vlaq {

__device__ __forceinline__ void unpack_bf16x8(const uint4& q, float* v) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = __uint_as_float(w[j] << 16);
    v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
  }
}

// Correctly rounded quotient without a divide per element: Markstein's
// correction step (P. Markstein, "IA-64 and Elementary Functions", 2000:
// with y = RN(1/S) and q0 = RN(x y), the residual x - q0 S is exact under a
// fused multiply-add and RN(q0 + (x - q0 S) y) = RN(x / S)).  The residual
// is formed negated, e' = q0 S - x, so that x = -0 still yields -0.  The
// reciprocal is CUDA's correctly rounded __frcp_rn, once per divisor.  Only
// divisors far from 1 (where the residual or 1/S could leave the normal
// range) and S = 0 take the slow path, behind a warp vote.
struct Divisor {
  float S, y;
  bool slow;  // S = 0 (quotients 0) or S outside [2^-64, 2^64]
};

__device__ __forceinline__ Divisor make_divisor(float S) {
  Divisor d;
  d.S = S;
  const bool ok = S >= 0x1p-64f && S <= 0x1p64f;
  d.y = ok ? __frcp_rn(S) : 0.0f;
  d.slow = !ok;
  return d;
}

__device__ __forceinline__ float markstein_quotient(float x, float S, float y) {
  const float q0 = __fmul_rn(x, y);
  const float e = __fmaf_rn(q0, S, -x);  // q0 S - x, exact
  return __fmaf_rn(-e, y, q0);
}

// RN(v[i] / S) for N values (0 when S = 0).  Executed by the whole warp.
template <int N>
__device__ __forceinline__ void quotients(const float* v, const Divisor& d, float* q) {
  static_assert(N % 2 == 0, "pairs");
  // the same three steps on packed pairs (sm_100a fp32x2 multiply and fused
  // multiply-add, each lane rounded once): q0 = x y, e = q0 S - x (x negated
  // exactly, so -0 stays -0), q = q0 + e (-y)
  const float2 yy = make_float2(d.y, d.y);
  const float2 ny = make_float2(-d.y, -d.y);
  const float2 ss = make_float2(d.S, d.S);
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    const float2 x = make_float2(v[i], v[i + 1]);
    const float2 q0 = __fmul2_rn(x, yy);
    const float2 e = __ffma2_rn(q0, ss, make_float2(-x.x, -x.y));
    const float2 r = __ffma2_rn(e, ny, q0);
    q[i] = r.x;
    q[i + 1] = r.y;
  }
  if (__any_sync(0xffffffffu, d.slow)) {
    if (d.slow) {
#pragma unroll
      for (int i = 0; i < N; ++i) q[i] = (d.S == 0.0f) ? 0.0f : __fdiv_rn(v[i], d.S);
    }
  }
}

// -RN(v[i] / S): the steps of quotients() from the negated product, which
// negate no operand (a packed operand takes an instruction to negate):
// n = x (-y), e = n S + x, r = e (-y) + n.  v = -0 gives +0 and +0 gives -0.
template <int N>
__device__ __forceinline__ void negated_quotients(const float* v, const Divisor& d, float* q) {
  static_assert(N % 2 == 0, "pairs");
  const float2 ny = make_float2(-d.y, -d.y);
  const float2 ss = make_float2(d.S, d.S);
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    const float2 x = make_float2(v[i], v[i + 1]);
    const float2 n = __fmul2_rn(x, ny);
    const float2 e = __ffma2_rn(n, ss, x);
    const float2 r = __ffma2_rn(e, ny, n);
    q[i] = r.x;
    q[i + 1] = r.y;
  }
  if (__any_sync(0xffffffffu, d.slow)) {
    if (d.slow) {
#pragma unroll
      for (int i = 0; i < N; ++i) q[i] = (d.S == 0.0f) ? -0.0f : -__fdiv_rn(v[i], d.S);
    }
  }
}

// E4M3 codes of RN(v[i] / S) for 8 values, element 0 in the low byte.
__device__ __forceinline__ uint2 e4m3_codes8(const float* v, const Divisor& d) {
  float q[8];
  negated_quotients<8>(v, d, q);
  return make_uint2(cvt_e4m3x4(q[0], q[1], q[2], q[3]) ^ 0x80808080u, cvt_e4m3x4(q[4], q[5], q[6], q[7]) ^ 0x80808080u);
}

// The global scale of a row from its amax A >= 0: RN(A / 2688) (NVFP4),
// RN(A / 448) (FP8) or RN(A / 127) (INT8), by the correction step against
// the constant's correctly rounded reciprocal; rows whose amax is tiny
// (quotient near the subnormal range) take a divide.  Uniform per row.
template <int FMT>
__device__ __forceinline__ float row_global(float A) {
  constexpr float c = (FMT == 0) ? 2688.0f : (FMT == 1) ? 448.0f : 127.0f;
  if (A < 0x1p-64f) return __fdiv_rn(A, c);
  return markstein_quotient(A, c, __frcp_rn(c));
}

// Normalised WHT of the 64-block spread over lanes 4 g .. 4 g + 3 (16 values
// each, element 16 (lane % 4) + j): stages h = 1, 2, 4, 8 inside the lane,
// h = 16, 32 across lanes (xor 1, 2), then x 1/8 (exact) -- the stages of the
// sequential butterfly in the same order.  Executed by the whole warp.
// Stages h >= 2 run two butterflies per packed fp32x2 instruction (each lane
// rounded once, so the values are those of the scalar steps): a + b, and
// a - b as fma(b, -1, a), a single rounding of the same exact difference
// (signed zeros included).  Across lanes the new value is p + s v with s = -1
// in the upper lane and +1 in the lower one, again one fused multiply-add.
__device__ __forceinline__ void wht64_lanes(float* v, int lane) {
#pragma unroll
  for (int i = 0; i < 16; i += 2) {
    const float a = v[i], b = v[i + 1];
    v[i] = __fadd_rn(a, b);
    v[i + 1] = __fsub_rn(a, b);
  }
  const float2 m1 = make_float2(-1.0f, -1.0f);
#pragma unroll
  for (int h = 2; h < 16; h <<= 1) {
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
      if ((i & h) == 0) {
        const float2 a = make_float2(v[i], v[i + 1]), b = make_float2(v[i + h], v[i + h + 1]);
        const float2 sum = __fadd2_rn(a, b), dif = __ffma2_rn(b, m1, a);
        v[i] = sum.x;
        v[i + 1] = sum.y;
        v[i + h] = dif.x;
        v[i + h + 1] = dif.y;
      }
    }
  }
#pragma unroll
  for (int x = 1; x < 4; x <<= 1) {
    const float sg = (lane & x) != 0 ? -1.0f : 1.0f;
    const float2 s2 = make_float2(sg, sg);
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
      const float2 p = make_float2(__shfl_xor_sync(0xffffffffu, v[i], x), __shfl_xor_sync(0xffffffffu, v[i + 1], x));
      const float2 r = __ffma2_rn(make_float2(v[i], v[i + 1]), s2, p);
      v[i] = r.x;
      v[i + 1] = r.y;
    }
  }
  const float2 e8 = make_float2(0.125f, 0.125f);
#pragma unroll
  for (int i = 0; i < 16; i += 2) {
    const float2 r = __fmul2_rn(make_float2(v[i], v[i + 1]), e8);
    v[i] = r.x;
    v[i + 1] = r.y;
  }
}

}  // namespace vlaq
