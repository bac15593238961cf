// One AdamW step over many tensors (gfx950), moments in float32 or in 8 bits.
//
//   g = grad * grad_scale
//   m = b1 m + (1 - b1) g,  v = b2 v + (1 - b2) g^2
//   p = p (1 - lr wd) - lr / (1 - b1^t) * m / (sqrt(v) / sqrt(1 - b2^t) + eps)
// Every operation rounds once to float32. In 8 bits each 256 consecutive elements
// share a scale, the largest magnitude among them:
//   m = s (c / 127) |c / 127|,  c in -127..127
//   sqrt(v) = s (c / 255)^2,    c in 0..255
// The square spends codes where most values of a block lie, far below its
// largest: steps are 2 / c of the value, and sqrt(v) reaches down to s / 65025. Codes are
// rounded up with the chance of what is cut off (a hash of seed, tensor and element
// decides): a moment moves by less than half a step in most steps, so the nearest code
// would never leave its place. A root that is not zero keeps a code of at least
// 1, or m / sqrt(v) would blow up in the next step.
//
// Nothing is read twice, and a block of 256 is one wave's (four elements a lane), so
// its largest magnitude is a reduction in registers: the memory rate is the bound.
// A block takes 1024 elements of one tensor, found in the table of the launch's arguments.
#include "block.h"
#include "common.h"

namespace cr {

typedef __bf16 v2bf __attribute__((ext_vector_type(2)));

CR_DEV uint32_t mix32(uint32_t x) {
  x ^= x >> 16;
  x *= 0x6A09E667u;
  x ^= x >> 15;
  x *= 0xBB67AE85u;
  return x ^ (x >> 16);
}

CR_DEV uint32_t wave_umax(uint32_t v) {
  uint32_t o = (uint32_t)dpp_i<DPP_QUAD_1032>((int)v);
  v = v > o ? v : o;
  o = (uint32_t)dpp_i<DPP_QUAD_2301>((int)v);
  v = v > o ? v : o;
  o = (uint32_t)dpp_i<DPP_HALF_MIRROR>((int)v);
  v = v > o ? v : o;
  o = (uint32_t)dpp_i<DPP_ROW_ROR8>((int)v);
  v = v > o ? v : o;
  o = (uint32_t)__shfl_xor((int)v, 16);
  v = v > o ? v : o;
  o = (uint32_t)__shfl_xor((int)v, 32);
  return v > o ? v : o;
}

// the four elements of a lane, `n` of them inside the tensor
CR_DEV v4f load_f32(const void* base, int64_t i, int n) {
  const float* s = static_cast<const float*>(base) + i;
  if (n == 4) return *reinterpret_cast<const v4f*>(s);
  v4f v = {0.f, 0.f, 0.f, 0.f};
  for (int e = 0; e < 3; ++e)
    if (e < n) v[e] = s[e];
  return v;
}
CR_DEV void store_f32(void* base, int64_t i, int n, v4f v) {
  float* d = static_cast<float*>(base) + i;
  if (n == 4) {
    *reinterpret_cast<v4f*>(d) = v;
  } else {
    for (int e = 0; e < 3; ++e)
      if (e < n) d[e] = v[e];
  }
}
CR_DEV v4f load_bf16(const void* base, int64_t i, int n) {
  const uint16_t* s = static_cast<const uint16_t*>(base) + i;
  if (n == 4) {
    const u32x2 w = *reinterpret_cast<const u32x2*>(s);
    return v4f{bf16_lo(w[0]), bf16_hi(w[0]), bf16_lo(w[1]), bf16_hi(w[1])};
  }
  v4f v = {0.f, 0.f, 0.f, 0.f};
  for (int e = 0; e < 3; ++e)
    if (e < n) v[e] = __uint_as_float((uint32_t)s[e] << 16);
  return v;
}
CR_DEV void store_bf16(void* base, int64_t i, int n, v4f v) {
  uint16_t* d = static_cast<uint16_t*>(base) + i;
  const u32x2 w = {__builtin_bit_cast(uint32_t, v2bf{(__bf16)v[0], (__bf16)v[1]}),
                   __builtin_bit_cast(uint32_t, v2bf{(__bf16)v[2], (__bf16)v[3]})};
  if (n == 4) {
    *reinterpret_cast<u32x2*>(d) = w;
  } else {
    for (int e = 0; e < 3; ++e)
      if (e < n) d[e] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
  }
}
CR_DEV uint32_t load_codes(const void* base, int64_t i, int n) {
  const uint8_t* s = static_cast<const uint8_t*>(base) + i;
  if (n == 4) return *reinterpret_cast<const uint32_t*>(s);
  uint32_t c = 0;
  for (int e = 0; e < 3; ++e)
    if (e < n) c |= (uint32_t)s[e] << (8 * e);
  return c;
}
CR_DEV void store_codes(void* base, int64_t i, int n, uint32_t c) {
  uint8_t* d = static_cast<uint8_t*>(base) + i;
  if (n == 4) {
    *reinterpret_cast<uint32_t*>(d) = c;
  } else {
    for (int e = 0; e < 3; ++e)
      if (e < n) d[e] = (uint8_t)(c >> (8 * e));
  }
}

// values of four codes: the integer c |c| times s / most^2
CR_DEV v4f avg_values(uint32_t c, float s) {
  const float step = s / 16129.f;
  v4f v;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float f = (float)(int)(int8_t)(c >> (8 * e));
    v[e] = f * fabsf(f) * step;
  }
  return v;
}
CR_DEV v4f root_values(uint32_t c, float s) {
  const float step = s / 65025.f;
  v4f v;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float f = (float)((c >> (8 * e)) & 0xFFu);
    v[e] = f * f * step;
  }
  return v;
}

// sqrt(x) rounded once, for 2^-100 <= x <= 1: a step of Goldschmidt's iteration on the root and half
// its reciprocal together, then one of Newton's with the exact residual.
CR_DEV float sqrt_rn(float x) {
  const float y = __builtin_amdgcn_rsqf(x);
  float s = x * y, h = 0.5f * y;
  const float e = __builtin_fmaf(-h, s, 0.5f);
  s = __builtin_fmaf(s, e, s);
  h = __builtin_fmaf(h, e, h);
  return __builtin_fmaf(__builtin_fmaf(-s, s, x), h, s);
}

// Codes of one wave's 256 values and their scale; h16: u in units of 2^-16. SIGNED: c =
// -127..127, else the values are not negative and c = 0..255, at least 1 for a value above 0.
// |x| / s is rounded once: with s scaled to [0.5, 1) and its reciprocal rounded, one
// step from x (1 / s) with the exact remainder gives the rounded quotient (a theorem of
// Markstein's); the library's division takes three times as many instructions. The
// arithmetic bounds the step with 8-bit moments as much as the memory does (5.1 million
// elements: 28 us, of which 22 the vector ALUs, for 92 MB).
template <bool SIGNED>
CR_DEV uint32_t encode(v4f x, const uint32_t (&h16)[4], float* scale) {
  constexpr float most = SIGNED ? 127.f : 255.f;
  uint32_t top = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint32_t b = __float_as_uint(x[e]) & 0x7FFFFFFFu;
    top = top > b ? top : b;
  }
  top = wave_umax(top);
  *scale = top >= 0x7F800000u ? __uint_as_float(0x7FC00000u) : __uint_as_float(top);   // not finite: the block reads as NaN
  if (top == 0 || top >= 0x7F800000u) return 0;
  const int power = __builtin_amdgcn_frexp_expf(__uint_as_float(top));
  const float s = ldexpf(__uint_as_float(top), -power);   // in [0.5, 1)
  const float inv = 1.f / s;
  uint32_t codes = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float a = ldexpf(fabsf(x[e]), -power);
    float q = a * inv;
    q = __builtin_fmaf(__builtin_fmaf(-q, s, a), inv, q);
    // below 2^-100 the root adds less than half a step of u: as good as 2^-100
    const float t = sqrt_rn(fmaxf(q, 0x1p-100f)) * most;
    // t + u: the product by 2^-16 is exact; the sum is not negative, so the conversion is the floor
    float c = fminf(__builtin_fmaf((float)h16[e], 0x1p-16f, t), most);
    if (!SIGNED) c = fmaxf(c, x[e] > 0.f ? 1.f : 0.f);
    const int k = (int)c;
    const int sign = SIGNED ? (int)__float_as_uint(x[e]) >> 31 : 0;
    codes |= (uint32_t)((SIGNED ? (k ^ sign) - sign : k) & 0xFF) << (8 * e);
  }
  return codes;
}

// the entry of a chunk: the last that begins at or before it and holds something
template <typename T>
CR_DEV int entry_of(const T& t, int chunk) {
  int lo = 0, hi = t.count;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (t.t[mid].first <= chunk) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Four consecutive elements a lane, FULL: all inside the tensor.
template <bool G16, int BITS, bool FULL>
CR_DEV void step_chunk(const AdamwEntry& a, const AdamwStep& p, int64_t base, uint32_t key, float gs) {
  const int64_t i = base + threadIdx.x * 4;
  const int64_t left = a.n - i;
  const int n = FULL || left >= 4 ? 4 : left > 0 ? (int)left : 0;
  const int64_t wave0 = i - (threadIdx.x & 63) * 4, block = wave0 / ADAMW_BLOCK;   // a block of 256 is one wave's
  const bool some = FULL || wave0 < a.n;
  v4f w = load_f32(a.param, i, n);
  const v4f grad = G16 ? load_bf16(a.grad, i, n) : load_f32(a.grad, i, n);
  v4f m, v;
  if constexpr (BITS == 8) {
    m = avg_values(load_codes(a.avg, i, n), some ? a.avg_scales[block] : 0.f);
    v = root_values(load_codes(a.sq, i, n), some ? a.sq_scales[block] : 0.f);
    v = v * v;
  } else {
    m = load_f32(a.avg, i, n);
    v = load_f32(a.sq, i, n);
  }
  v4f root;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float g = grad[e] * gs;
    m[e] = m[e] * p.b1 + g * p.c1;
    v[e] = v[e] * p.b2 + g * g * p.c2;
    root[e] = sqrtf(v[e]);
    // the quotient by the hardware's reciprocal: within two units in the last place of the update
    w[e] = w[e] * p.decay - m[e] * __builtin_amdgcn_rcpf(root[e] * p.rsqrt_bias2 + p.eps) * p.rate;
  }
  store_f32(a.param, i, n, w);
  if (a.copy) store_bf16(a.copy, i, n, w);
  if constexpr (BITS == 8) {
    uint32_t um[4], uv[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t h = mix32(mix32((uint32_t)i + e) ^ key);
      um[e] = h & 0xFFFFu;
      uv[e] = h >> 16;
      if (!FULL && e >= n) m[e] = root[e] = 0.f;         // past the end: no part of the largest
    }
    float sm, sv;
    store_codes(a.avg, i, n, encode<true>(m, um, &sm));
    store_codes(a.sq, i, n, encode<false>(root, uv, &sv));
    if (some && (threadIdx.x & 63) == 0) {
      a.avg_scales[block] = sm;
      a.sq_scales[block] = sv;
    }
  } else {
    store_f32(a.avg, i, n, m);
    store_f32(a.sq, i, n, v);
  }
}

template <bool G16, int BITS>
__global__ __launch_bounds__(256) void adamw_step_kernel(AdamwTable t, AdamwStep p) {
  const int which = entry_of(t, (int)blockIdx.x);
  const AdamwEntry& a = t.t[which];
  const int64_t base = (int64_t)((int)blockIdx.x - a.first) * ADAMW_CHUNK;
  const float gs = p.grad_scale ? *p.grad_scale : 1.f;
  const uint32_t key = BITS == 8 ? mix32(p.seed + 0x9E3779B9u * (uint32_t)(t.ordinal + which + 1)) : 0u;
  if (base + ADAMW_CHUNK <= a.n) step_chunk<G16, BITS, true>(a, p, base, key, gs);
  else step_chunk<G16, BITS, false>(a, p, base, key, gs);
}

__global__ __launch_bounds__(256) void adamw_moments_kernel(MomentsTable t, float* avg, float* sq) {
  const MomentsEntry& a = t.t[entry_of(t, (int)blockIdx.x)];
  const int64_t i = (int64_t)((int)blockIdx.x - a.first) * ADAMW_CHUNK + threadIdx.x * 4;
  const int64_t at = a.at;
  const int64_t left = a.n - i;
  const int n = left >= 4 ? 4 : left > 0 ? (int)left : 0;
  if (n == 0) return;
  const v4f m = avg_values(load_codes(a.avg, i, n), a.avg_scales[i / ADAMW_BLOCK]);
  v4f v = root_values(load_codes(a.sq, i, n), a.sq_scales[i / ADAMW_BLOCK]);
  v = v * v;
  if (n == 4 && (at & 3) == 0) {
    *reinterpret_cast<v4f*>(avg + at + i) = m;
    *reinterpret_cast<v4f*>(sq + at + i) = v;
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (e < n) {
        avg[at + i + e] = m[e];
        sq[at + i + e] = v[e];
      }
  }
}

hipError_t launch_adamw_step(const AdamwTable& t, const AdamwStep& p, bool grad_bf16, int bits, int chunks, hipStream_t s) {
  const dim3 grid((unsigned)chunks);
  if (bits == 8) {
    if (grad_bf16) hipLaunchKernelGGL((adamw_step_kernel<true, 8>), grid, dim3(256), 0, s, t, p);
    else hipLaunchKernelGGL((adamw_step_kernel<false, 8>), grid, dim3(256), 0, s, t, p);
  } else {
    if (grad_bf16) hipLaunchKernelGGL((adamw_step_kernel<true, 32>), grid, dim3(256), 0, s, t, p);
    else hipLaunchKernelGGL((adamw_step_kernel<false, 32>), grid, dim3(256), 0, s, t, p);
  }
  return hipGetLastError();
}

hipError_t launch_adamw_moments(const MomentsTable& t, float* avg, float* sq, int chunks, hipStream_t s) {
  hipLaunchKernelGGL(adamw_moments_kernel, dim3((unsigned)chunks), dim3(256), 0, s, t, avg, sq);
  return hipGetLastError();
}

}  // namespace cr
