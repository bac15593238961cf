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

constexpr float kLog2e = 1.44269504088896341f;
constexpr float kInvSqrt2Pi = 0.39894228040143268f;
constexpr float kTanhA = 1.5957691216057308f;   // 2 sqrt(2 / pi)
constexpr float kTanhB = 0.044715f;

// sigma(x) and sigma(-x) from e = exp(-|x|) <= 1: neither overflows, and the
// small one keeps its relative precision. The hardware reciprocal is within
// one unit in the last place.
struct Sigmoid {
  float p, q;
};
CR_DEV Sigmoid sigmoid(float x) {
  const float e = exp2f(-kLog2e * fabsf(x)), inv = __builtin_amdgcn_rcpf(1.f + e), small = e * inv;
  return x < 0.f ? Sigmoid{small, inv} : Sigmoid{inv, small};
}

// Phi(z) and E = exp(-z^2 / 2). With a = |z|, Phi(-a) = E G(a), where
// G(a) = erfcx(a / sqrt 2) / 2 falls smoothly like 1 / (a sqrt(2 pi)): a
// polynomial in w = 1 / (1 + 0.36308432 a) without constant term, fitted here by
// reweighted least squares on 0 <= a <= 15, has relative error 1.1e-6 in
// float32. Beyond 15, E is below 2^-149.
struct Normal {
  float phi, e;
};
// FLUSH: E below 2^-126 as 0 (the bare instruction). z Phi(z) is below 0.4 E
// there, so a forward value loses less than the smallest normal float32.
template <bool FLUSH>
CR_DEV Normal normal(float z) {
  const float w = __builtin_amdgcn_rcpf(__builtin_fmaf(0.36308431899331844f, fabsf(z), 1.f));
  float g = 0.04788525402545929f;
  g = __builtin_fmaf(g, w, -0.17834912240505219f);
  g = __builtin_fmaf(g, w, 0.1719096153974533f);
  g = __builtin_fmaf(g, w, 0.03162514418363571f);
  g = __builtin_fmaf(g, w, 0.13871920108795166f);
  g = __builtin_fmaf(g, w, 0.1432841569185257f);
  g = __builtin_fmaf(g, w, 0.14492595195770264f);
  const float at = (-0.5f * kLog2e) * (z * z);
  const float e = FLUSH ? __builtin_amdgcn_exp2f(at) : exp2f(at);
  const float t = g * w * e;
  return Normal{z < 0.f ? t : 1.f - t, e};
}

template <int ACT>
CR_DEV float act_value(float z) {
  if constexpr (ACT == CR_ACT_GELU) return z * normal<true>(z).phi;
  else if constexpr (ACT == CR_ACT_GELU_TANH)
    return z * sigmoid(z * __builtin_fmaf(kTanhA * kTanhB, z * z, kTanhA)).p;
  else return z * sigmoid(z).p;
}

template <int ACT>
CR_DEV float act_slope(float z) {
  if constexpr (ACT == CR_ACT_GELU) {
    const Normal n = normal<false>(z);
    return __builtin_fmaf(z * kInvSqrt2Pi, n.e, n.phi);
  } else {
    z = z > 20.f ? 20.f : (z < -20.f ? -20.f : z);   // the slope is 1 or 0 beyond; z z could overflow; keeps NaN
    const float zz = z * z;
    const Sigmoid s = sigmoid(z * __builtin_fmaf(kTanhA * kTanhB, zz, kTanhA));
    return __builtin_fmaf(z * s.p * s.q, __builtin_fmaf(3.f * kTanhA * kTanhB, zz, kTanhA), s.p);
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
    r = 127.f / A;                                 // float32 division: correctly rounded
    s = A / 127.f;
  }
  uint32_t q[2] = {0, 0};
  if (r != 0.f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      // |v r| <= 127 (1 + 2^-23): the rounding stays within the range by itself
      q[i >> 2] |= (__float_as_uint(__fadd_rn(__fmul_rn(v[i], r), CR_MAGIC_RNE)) & 0xFFu) << (8 * (i & 3));
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

// n / d for n < 2^31 and 8 <= d <= 4096: M = ceil(2^(31 + l) / d) with
// 2^(l-1) < d <= 2^l has M d - 2^(31 + l) < 2^l, so n M / 2^(31 + l) has the
// quotient's integer part.
struct RowDiv {
  uint32_t mul;
  int shift;
};
static RowDiv row_div(uint32_t d) {
  int l = 3;
  while ((1u << l) < d) ++l;
  return RowDiv{(uint32_t)((((uint64_t)1 << (31 + l)) + d - 1) / d), l - 1};
}

// One thread: eight consecutive columns of one row (of both halves for
// SWIGLU); eight consecutive threads: one scale group. Nothing is read twice, so
// the copy rate bounds it as long as the arithmetic stays under it: 8192 x 12288,
// forward and backward, tanh GELU 93 and 93 us (5.4 TB/s), GELU 115 and 113,
// SWIGLU 145 and 144 (5.6 TB/s). Two items a thread took longer.
template <int ACT>
__global__ __launch_bounds__(256) void act_checkpoint_kernel(ActArgs p, RowDiv d) {
  const uint32_t per_row = (uint32_t)p.C / 8;
  const uint32_t i = blockIdx.x * 256 + threadIdx.x;
  const uint32_t row = __umulhi(i, d.mul) >> d.shift;
  if (row >= p.rows) return;                    // whole groups of eight lanes
  const int64_t m = row, c = (i - row * per_row) * 8;
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
__global__ __launch_bounds__(256) void act_backward_kernel(ActArgs p, RowDiv d) {
  const uint32_t per_row = (uint32_t)p.C / 8;
  const uint32_t i = blockIdx.x * 256 + threadIdx.x;
  const uint32_t row = __umulhi(i, d.mul) >> d.shift;
  if (row >= p.rows) return;
  const int64_t m = row, c = (i - row * per_row) * 8;
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
      // halved on the way, exactly: the slope reaches 1.1, and u times it could overflow where dg does not
      dg[e] = 2.f * (dy[e] * (u[e] * (0.5f * (s.p * (1.f + v[e] * s.q)))));
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
  const RowDiv d = row_div((uint32_t)(p.C / 8));
  switch (p.act) {
    case CR_ACT_GELU: hipLaunchKernelGGL((act_checkpoint_kernel<CR_ACT_GELU>), grid, dim3(256), 0, s, p, d); break;
    case CR_ACT_GELU_TANH: hipLaunchKernelGGL((act_checkpoint_kernel<CR_ACT_GELU_TANH>), grid, dim3(256), 0, s, p, d); break;
    default: hipLaunchKernelGGL((act_checkpoint_kernel<CR_ACT_SWIGLU>), grid, dim3(256), 0, s, p, d); break;
  }
  return hipGetLastError();
}

hipError_t launch_act_backward(const ActArgs& p, hipStream_t s) {
  const dim3 grid((unsigned)((p.rows * (p.C / 8) + 255) / 256));
  const RowDiv d = row_div((uint32_t)(p.C / 8));
  switch (p.act) {
    case CR_ACT_GELU: hipLaunchKernelGGL((act_backward_kernel<CR_ACT_GELU>), grid, dim3(256), 0, s, p, d); break;
    case CR_ACT_GELU_TANH: hipLaunchKernelGGL((act_backward_kernel<CR_ACT_GELU_TANH>), grid, dim3(256), 0, s, p, d); break;
    default: hipLaunchKernelGGL((act_backward_kernel<CR_ACT_SWIGLU>), grid, dim3(256), 0, s, p, d); break;
  }
  return hipGetLastError();
}

}  // namespace cr
