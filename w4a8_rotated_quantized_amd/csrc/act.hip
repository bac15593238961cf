// MLP activations that keep their input as 8-bit codes, and their backward
// pass from those codes (gfx950).
//
// Forward, per row and 64 columns of z (bf16): A = max |z|, r = fl32(127 / A),
// q = clamp(rint(fl32(z r)), -127, 127), s = fl32(A / 127): the symmetric
// quantizer of the library (ROW_GROUP 64, no rotation). y = act(z) comes from
// z itself. Backward: dz = dy act'(s q).
//   GELU       z Phi(z) = z erfc(-z / sqrt 2) / 2;  act' = Phi(z) + z phi(z)
//   GELU_TANH  z sigma(2 t), t = sqrt(2/pi) (z + 0.044715 z^3)
//   SWIGLU     silu(g) u with z = [g | u];  dg = dy u sigma(g)(1 + g(1 - sigma(g))), du = dy g sigma(g)
// erfc keeps the relative precision of the negative tail, where 1 + erf would
// cancel.
#include "common.h"
#include "lora.h"

#include "../../include/convrot.h"

namespace cr {

typedef __bf16 v2bf __attribute__((ext_vector_type(2)));

CR_DEV uint32_t bf16_pair(float lo, float hi) {
  return __builtin_bit_cast(uint32_t, v2bf{(__bf16)lo, (__bf16)hi});   // round half to even, NaN kept
}

// sigma(x) and sigma(-x) from e = exp(-|x|) <= 1: neither overflows, and the
// small one keeps its relative precision.
struct Sigmoid {
  float p, q;
};
CR_DEV Sigmoid sigmoid(float x) {
  const float e = expf(-fabsf(x)), inv = 1.f / (1.f + e), small = e * inv;
  return x < 0.f ? Sigmoid{small, inv} : Sigmoid{inv, small};
}

constexpr float kSqrtHalf = 0.70710678118654752f;
constexpr float kInvSqrt2Pi = 0.39894228040143268f;
constexpr float kTanhA = 1.5957691216057308f;   // 2 sqrt(2 / pi)
constexpr float kTanhB = 0.044715f;

template <int ACT>
CR_DEV float act_value(float z) {
  if constexpr (ACT == CR_ACT_GELU) return z * 0.5f * erfcf(-z * kSqrtHalf);
  else if constexpr (ACT == CR_ACT_GELU_TANH) return z * sigmoid(kTanhA * (z + kTanhB * z * z * z)).p;
  else return z * sigmoid(z).p;
}

template <int ACT>
CR_DEV float act_slope(float z) {
  if constexpr (ACT == CR_ACT_GELU) {
    return 0.5f * erfcf(-z * kSqrtHalf) + z * kInvSqrt2Pi * expf(-0.5f * z * z);
  } else {
    z = z > 20.f ? 20.f : (z < -20.f ? -20.f : z);   // the slope is 1 or 0 beyond; z z could overflow; keeps NaN
    const Sigmoid s = sigmoid(kTanhA * (z + kTanhB * z * z * z));
    return s.p + z * s.p * s.q * kTanhA * (1.f + 3.f * kTanhB * z * z);
  }
}

CR_DEV void unpack8(const u32x4& w, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = bf16_lo(w[i]);
    v[2 * i + 1] = bf16_hi(w[i]);
  }
}

CR_DEV u32x4 pack8(const float (&v)[8]) {
  return u32x4{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]), bf16_pair(v[4], v[5]), bf16_pair(v[6], v[7])};
}

// Codes and scale of the 64 columns that eight consecutive lanes hold (eight
// each). Not-a-number or infinite values make the scale NaN, so that they
// reach the gradient; a group below 127 / FLT_MAX, whose 127 / A has no
// float32 value, is kept as zeros.
CR_DEV void quantize8(const u32x4& w, const float (&v)[8], int8_t* codes, float* scale, bool first) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t lo = w[i] << 16 & 0x7FFF0000u, hi = w[i] & 0x7FFF0000u;
    top = top > lo ? top : lo;
    top = top > hi ? top : hi;
  }
  // the order of magnitudes is that of their bit patterns, infinities and NaN above all
  uint32_t o = (uint32_t)dpp_i<DPP_QUAD_1032>((int)top);
  top = top > o ? top : o;
  o = (uint32_t)dpp_i<DPP_QUAD_2301>((int)top);
  top = top > o ? top : o;
  o = (uint32_t)dpp_i<DPP_HALF_MIRROR>((int)top);
  top = top > o ? top : o;
  const float A = __uint_as_float(top);
  float r = 0.f, s = 0.f;
  if (top >= 0x7F800000u) {
    s = __uint_as_float(0x7FC00000u);
  } else if (A > 3.8e-37f) {
    r = div_rn(127.f, A);
    s = div_rn(A, 127.f);
  }
  uint32_t q[2] = {0, 0};
  if (r != 0.f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float t = fminf(fmaxf(rintf(__fmul_rn(v[i], r)), -127.f), 127.f);
      q[i >> 2] |= ((uint32_t)(int)t & 0xFFu) << (8 * (i & 3));
    }
  }
  *reinterpret_cast<u32x2*>(codes) = u32x2{q[0], q[1]};
  if (first) *scale = s;
}

CR_DEV void dequantize8(const int8_t* codes, float s, float (&v)[8]) {
  const u32x2 q = *reinterpret_cast<const u32x2*>(codes);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = s * (float)(int)(int8_t)(q[i >> 2] >> (8 * (i & 3)));
}

// One thread: eight consecutive columns of one row (of both halves for
// SWIGLU); eight consecutive threads: one scale group.
template <int ACT>
__global__ __launch_bounds__(256) void act_checkpoint_kernel(ActArgs p) {
  const int64_t per_row = p.C / 8;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= p.rows * per_row) return;            // whole groups of eight lanes
  const int64_t m = i / per_row, c = (i % per_row) * 8;
  const bool first = (threadIdx.x & 7) == 0;
  const uint16_t* in = p.in + m * p.ldi + c;
  float v[8], y[8];
  const u32x4 w = *reinterpret_cast<const u32x4*>(in);
  unpack8(w, v);
  if constexpr (ACT == CR_ACT_SWIGLU) {
    const int64_t W = 2 * p.C;
    float u[8];
    const u32x4 wu = *reinterpret_cast<const u32x4*>(in + p.C);
    unpack8(wu, u);
    quantize8(w, v, p.codes + m * W + c, p.scales + (m * W + c) / 64, first);
    quantize8(wu, u, p.codes + m * W + p.C + c, p.scales + (m * W + p.C + c) / 64, first);
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = act_value<ACT>(v[e]) * u[e];
  } else {
    quantize8(w, v, p.codes + m * p.C + c, p.scales + (m * p.C + c) / 64, first);
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = act_value<ACT>(v[e]);
  }
  *reinterpret_cast<u32x4*>(p.out + m * p.ldo + c) = pack8(y);
}

template <int ACT>
__global__ __launch_bounds__(256) void act_backward_kernel(ActArgs p) {
  const int64_t per_row = p.C / 8;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= p.rows * per_row) return;
  const int64_t m = i / per_row, c = (i % per_row) * 8;
  float dy[8], v[8];
  unpack8(*reinterpret_cast<const u32x4*>(p.in + m * p.ldi + c), dy);
  uint16_t* out = p.out + m * p.ldo + c;
  if constexpr (ACT == CR_ACT_SWIGLU) {
    const int64_t W = 2 * p.C;
    float u[8], dg[8], du[8];
    dequantize8(p.codes + m * W + c, p.scales[(m * W + c) / 64], v);
    dequantize8(p.codes + m * W + p.C + c, p.scales[(m * W + p.C + c) / 64], u);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const Sigmoid s = sigmoid(v[e]);
      dg[e] = dy[e] * (u[e] * (s.p * (1.f + v[e] * s.q)));
      du[e] = dy[e] * (v[e] * s.p);
    }
    *reinterpret_cast<u32x4*>(out) = pack8(dg);
    *reinterpret_cast<u32x4*>(out + p.C) = pack8(du);
  } else {
    dequantize8(p.codes + m * p.C + c, p.scales[(m * p.C + c) / 64], v);
#pragma unroll
    for (int e = 0; e < 8; ++e) dy[e] *= act_slope<ACT>(v[e]);
    *reinterpret_cast<u32x4*>(out) = pack8(dy);
  }
}

hipError_t launch_act_checkpoint(const ActArgs& p, hipStream_t s) {
  const dim3 grid((unsigned)((p.rows * (p.C / 8) + 255) / 256));
  switch (p.act) {
    case CR_ACT_GELU: hipLaunchKernelGGL((act_checkpoint_kernel<CR_ACT_GELU>), grid, dim3(256), 0, s, p); break;
    case CR_ACT_GELU_TANH: hipLaunchKernelGGL((act_checkpoint_kernel<CR_ACT_GELU_TANH>), grid, dim3(256), 0, s, p); break;
    default: hipLaunchKernelGGL((act_checkpoint_kernel<CR_ACT_SWIGLU>), grid, dim3(256), 0, s, p); break;
  }
  return hipGetLastError();
}

hipError_t launch_act_backward(const ActArgs& p, hipStream_t s) {
  const dim3 grid((unsigned)((p.rows * (p.C / 8) + 255) / 256));
  switch (p.act) {
    case CR_ACT_GELU: hipLaunchKernelGGL((act_backward_kernel<CR_ACT_GELU>), grid, dim3(256), 0, s, p); break;
    case CR_ACT_GELU_TANH: hipLaunchKernelGGL((act_backward_kernel<CR_ACT_GELU_TANH>), grid, dim3(256), 0, s, p); break;
    default: hipLaunchKernelGGL((act_backward_kernel<CR_ACT_SWIGLU>), grid, dim3(256), 0, s, p); break;
  }
  return hipGetLastError();
}

}  // namespace cr
