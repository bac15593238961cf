// Microscaled 4-bit floating point (gfx950): quantization of bf16 rows, with
// or without the ConvRot rotation, and the way back.
//
// The format is the OCP Microscaling one with E2M1 elements: 32 consecutive
// columns share a power of two 2^(b - 127), and each holds one of 0, .5, 1,
// 1.5, 2, 3, 4, 6 with a sign. With A the largest magnitude of the 32,
// b = floor(log2 A) - 2 + 127 (clamped to 0), so A lies in [4, 8) units: what
// rounds above 6 saturates there. The rotation (see rotate.h) is carried out
// unnormalised in float32; its 1 / sqrt(n) is a power of two and goes into b.
//
// Lane layout: that of the rotation. 16 lanes hold 256 columns of a row, 16
// consecutive columns each (the lane's element bits b4..b7 come from its
// number by the DPP-friendly map), so a scale block is a pair of lanes
// (lane ^ 1), a 128-column tile of the output is one half row of 8 lanes, and
// both the rotation and the block maximum stay in registers.
//
// One thread takes 16 columns of one row (64 with the 1024 rotation): 32 bytes
// in, 8 + 1 bytes out. A block covers 16 rows x 256 columns, so that it writes 1 KB
// runs of two tiles; with fewer rows, fewer rows x more columns.
#include "block.h"
#include "common.h"
#include "rotate.h"

namespace cr {

typedef float v2f __attribute__((ext_vector_type(2)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));

// chunks of 256 columns that a lane holds at once, and log2 of sqrt(rotation group)
template <int NR>
struct MxRot {
  static constexpr int chunks = NR == 1024 ? 4 : 1;
  static constexpr int half = NR == 0 ? 0 : NR == 16 ? 2 : NR == 64 ? 3 : NR == 256 ? 4 : 5;
  static constexpr int lanes = NR == 0 ? 256 : NR;   // the lane map's rotation (any for none)
};

CR_DEV uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

// scale byte for the largest magnitude's bits (infinity and NaN: 255)
CR_DEV uint32_t mx_byte(uint32_t top, int half) {
  const int e = (int)(top >> 23);
  if (e == 255) return 255u;
  return (uint32_t)(e - 2 - half > 0 ? e - 2 - half : 0);
}

// eight values -> eight codes, in steps of `unit` (a power of two)
CR_DEV v2bf bf16_pair_of(uint32_t w) { return __builtin_bit_cast(v2bf, w); }
CR_DEV uint32_t codes_bf16(u32x4 w, float unit) {
  uint32_t c = 0;
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, bf16_pair_of(w[0]), unit, 0);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, bf16_pair_of(w[1]), unit, 1);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, bf16_pair_of(w[2]), unit, 2);
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, bf16_pair_of(w[3]), unit, 3);
}
CR_DEV uint32_t codes_f32(const float* v, float unit) {
  uint32_t c = 0;
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[0], v[1], unit, 0);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[2], v[3], unit, 1);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[4], v[5], unit, 2);
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[6], v[7], unit, 3);
}

// Segments (16 lanes) of a block: rpb = 1 << lg_rpb rows x 16 / rpb column
// groups of 256 * chunks.
template <int NR>
__global__ __launch_bounds__(256) void mx_quantize_kernel(MxQuantize p, int lg_rpb, int groups, int across) {
  constexpr int NC = MxRot<NR>::chunks;
  const int seg = threadIdx.x >> 4;
  const LaneRot lr = lane_rot<MxRot<NR>::lanes>(threadIdx.x & 15);
  const uint32_t block = (blockIdx.y << GRID_LG) + blockIdx.x, down = block / (uint32_t)across;
  const int64_t row = ((int64_t)down << lg_rpb) + (seg & ((1 << lg_rpb) - 1));
  const int group = (int)(block - down * across) * (16 >> lg_rpb) + (seg >> lg_rpb);
  if (row >= p.rows || group >= groups) return;        // whole segments: DPP stays inside them
  const int tiles = (int)((p.K + MX_TILE - 1) / MX_TILE);

  u32x4 w[NC][2];
#pragma unroll
  for (int g = 0; g < NC; ++g) {
    const int64_t k0 = ((int64_t)group * NC + g) * 256 + 16 * lr.gL;
    w[g][0] = w[g][1] = u32x4{0, 0, 0, 0};
    if (k0 < p.K) {                                    // K is a multiple of 32
      const u32x4* src = reinterpret_cast<const u32x4*>(p.x + row * p.ldx + k0);
      w[g][0] = src[0];
      w[g][1] = src[1];
    }
  }
  float v[NC][16];
  if constexpr (NR != 0) {
#pragma unroll
    for (int g = 0; g < NC; ++g) {
      if (NR == 1024 && chunk_neg(g)) rotate_group<NR, true>(w[g], lr, v[g]);
      else rotate_group<NR, false>(w[g], lr, v[g]);
    }
    if constexpr (NR == 1024) bfly_chunks<NC>(v);
  }
#pragma unroll
  for (int g = 0; g < NC; ++g) {
    // the block's largest magnitude: bit patterns order magnitudes, infinity and NaN on top
    uint32_t top = 0;
    if constexpr (NR == 0) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t lo = w[g][i >> 2][i & 3] << 16 & 0x7FFF0000u, hi = w[g][i >> 2][i & 3] & 0x7FFF0000u;
        top = umax(top, umax(lo, hi));
      }
    } else {
#pragma unroll
      for (int e = 0; e < 16; ++e) top = umax(top, __float_as_uint(v[g][e]) & 0x7FFFFFFFu);
    }
    top = umax(top, (uint32_t)dpp_i<DPP_QUAD_1032>((int)top));
    const uint32_t byte = mx_byte(top, MxRot<NR>::half);
    const float unit = __uint_as_float((byte + MxRot<NR>::half) << 23);
    u32x2 c;
    if constexpr (NR == 0) {
      c = u32x2{codes_bf16(w[g][0], unit), codes_bf16(w[g][1], unit)};
    } else {
      float t[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const bool neg = (lr.tau < 0.f) != (dreg_neg(e) != (NR == 1024 && chunk_neg(g)));
        t[e] = neg ? -v[g][e] : v[g][e];
      }
      c = u32x2{codes_f32(t, unit), codes_f32(t + 8, unit)};
    }
    if (byte == 255u) c = u32x2{0, 0};
    // the four bytes of a tile's row, gathered in its 8 lanes
    uint32_t s = byte << (8 * ((lr.gL >> 1) & 3));
    s |= (uint32_t)dpp_i<DPP_QUAD_2301>((int)s);
    s |= (uint32_t)dpp_i<DPP_HALF_MIRROR>((int)s);
    const int tile = (group * NC + g) * 2 + (lr.gL >> 3);
    if (tile < tiles) {
      const int64_t at = (int64_t)tile * p.rows + row;
      *reinterpret_cast<u32x2*>(p.codes + at * 64 + (lr.gL & 7) * 8) = c;
      if ((lr.gL & 7) == 0) *reinterpret_cast<uint32_t*>(p.scales + at * 4) = s;
    }
  }
}

// 16 codes -> float32 values of one unit each
CR_DEV void values_fp4(u32x2 c, float (&v)[16]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const v2f a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[h], 1.f, 0);
    const v2f b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[h], 1.f, 1);
    const v2f d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[h], 1.f, 2);
    const v2f f = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[h], 1.f, 3);
    v[8 * h + 0] = a[0]; v[8 * h + 1] = a[1]; v[8 * h + 2] = b[0]; v[8 * h + 3] = b[1];
    v[8 * h + 4] = d[0]; v[8 * h + 5] = d[1]; v[8 * h + 6] = f[0]; v[8 * h + 7] = f[1];
  }
}

template <int NR, bool F32>
__global__ __launch_bounds__(256) void mx_dequantize_kernel(MxDequantize p, int lg_rpb, int groups, int across) {
  constexpr int NC = MxRot<NR>::chunks;
  __shared__ __attribute__((aligned(16))) float lds[F32 ? 16 : 1][F32 ? 256 : 1];
  const int seg = threadIdx.x >> 4;
  const LaneRot lr = lane_rot<MxRot<NR>::lanes>(threadIdx.x & 15);
  const uint32_t block = (blockIdx.y << GRID_LG) + blockIdx.x, down = block / (uint32_t)across;
  const int64_t row = ((int64_t)down << lg_rpb) + (seg & ((1 << lg_rpb) - 1));
  const int group = (int)(block - down * across) * (16 >> lg_rpb) + (seg >> lg_rpb);
  if (row >= p.rows || group >= groups) return;
  float v[NC][16];
#pragma unroll
  for (int g = 0; g < NC; ++g) {
    const int64_t k0 = ((int64_t)group * NC + g) * 256 + 16 * lr.gL;
    u32x2 c = {0, 0};
    uint32_t byte = 0;
    if (k0 < p.K) {
      const int64_t at = (k0 / MX_TILE) * p.rows + row;
      c = *reinterpret_cast<const u32x2*>(p.codes + at * 64 + (lr.gL & 7) * 8);
      byte = p.scales[at * 4 + ((lr.gL >> 1) & 3)];
    }
    values_fp4(c, v[g]);
    // 2^(byte - 127): the smallest is a subnormal float32, 255 is not a number
    const float unit = byte == 255u ? __uint_as_float(0x7FC00000u) : __uint_as_float(byte ? byte << 23 : 0x00400000u);
    const bool cneg = NR == 1024 && chunk_neg(g);
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      v[g][e] = __fmul_rn(v[g][e], unit);
      if (NR != 0 && dreg_neg(e) != cneg) v[g][e] = -v[g][e];
    }
    if constexpr (NR != 0) butterflies<NR>(v[g], lr);
  }
  if constexpr (NR == 1024) bfly_chunks<NC>(v);
#pragma unroll
  for (int g = 0; g < NC; ++g) {
    const int64_t k0 = ((int64_t)group * NC + g) * 256 + 16 * lr.gL;
    if constexpr (NR != 0) {
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const bool neg = (lr.tau < 0.f) != (dreg_neg(e) != (NR == 1024 && chunk_neg(g)));
        v[g][e] = (neg ? -v[g][e] : v[g][e]) * RotSize<NR == 0 ? 256 : NR>::inv_sqrt;
      }
    }
    if constexpr (F32) {
      // 64 bytes a lane would leave as 16-byte pieces 64 bytes apart: through LDS each store covers 256 bytes
      // in a row for every 16 lanes (9216 x 2560 rotated: 33 -> 19 us). Piece q of 16 columns lies at
      // q ^ (gL / 4 % 4), which keeps both sides off the same banks.
      v4f* box = reinterpret_cast<v4f*>(lds[threadIdx.x >> 4]);
#pragma unroll
      for (int q = 0; q < 4; ++q) box[lr.gL * 4 + (q ^ (lr.gL >> 2))] = v4f{v[g][4 * q], v[g][4 * q + 1], v[g][4 * q + 2], v[g][4 * q + 3]};
      // 16 lanes write and read their own box: a wave's LDS accesses are in order
      __builtin_amdgcn_wave_barrier();
      const int L = threadIdx.x & 15;
      float* dst = reinterpret_cast<float*>(p.out) + row * p.ldo + k0 - 16 * lr.gL;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const v4f o = box[(q * 4 + (L >> 2)) * 4 + ((L & 3) ^ q)];
        const int c = q * 64 + L * 4;
        if (k0 - 16 * lr.gL + c < p.K) *reinterpret_cast<v4f*>(dst + c) = o;
      }
      __builtin_amdgcn_wave_barrier();
    } else {
      u32x4 o[2];
#pragma unroll
      for (int e = 0; e < 16; e += 2)
        o[e >> 3][(e & 7) >> 1] = __builtin_bit_cast(uint32_t, v2bf{(__bf16)v[g][e], (__bf16)v[g][e + 1]});
      if (k0 < p.K) {
        u32x4* dst = reinterpret_cast<u32x4*>(reinterpret_cast<uint16_t*>(p.out) + row * p.ldo + k0);
        dst[0] = o[0];
        dst[1] = o[1];
      }
    }
  }
}

struct MxGrid {
  int lg_rpb, groups, across;
  dim3 blocks;
};
// 16 rows a block, fewer where there are fewer; blocks along the columns first
static MxGrid mx_grid(int64_t rows, int64_t K, int chunks) {
  MxGrid g;
  g.lg_rpb = 0;
  while (g.lg_rpb < 4 && ((int64_t)1 << g.lg_rpb) < rows) ++g.lg_rpb;
  g.groups = (int)((K + 256 * chunks - 1) / (256 * chunks));
  const int per = 16 >> g.lg_rpb;
  g.across = (g.groups + per - 1) / per;
  const int64_t rpb = (int64_t)1 << g.lg_rpb;
  g.blocks = long_grid(g.across * ((rows + rpb - 1) / rpb));
  return g;
}

template <int NR>
static hipError_t quantize_nr(const MxQuantize& p, hipStream_t s) {
  const MxGrid g = mx_grid(p.rows, p.K, MxRot<NR>::chunks);
  hipLaunchKernelGGL((mx_quantize_kernel<NR>), g.blocks, dim3(256), 0, s, p, g.lg_rpb, g.groups, g.across);
  return hipGetLastError();
}

template <int NR>
static hipError_t dequantize_nr(const MxDequantize& p, hipStream_t s) {
  const MxGrid g = mx_grid(p.rows, p.K, MxRot<NR>::chunks);
  if (p.out_f32) hipLaunchKernelGGL((mx_dequantize_kernel<NR, true>), g.blocks, dim3(256), 0, s, p, g.lg_rpb, g.groups, g.across);
  else hipLaunchKernelGGL((mx_dequantize_kernel<NR, false>), g.blocks, dim3(256), 0, s, p, g.lg_rpb, g.groups, g.across);
  return hipGetLastError();
}

hipError_t launch_mx_quantize(const MxQuantize& p, hipStream_t s) {
  switch (p.rot_group) {
    case 0: return quantize_nr<0>(p, s);
    case 16: return quantize_nr<16>(p, s);
    case 64: return quantize_nr<64>(p, s);
    case 1024: return quantize_nr<1024>(p, s);
    default: return quantize_nr<256>(p, s);
  }
}

hipError_t launch_mx_dequantize(const MxDequantize& p, hipStream_t s) {
  switch (p.rot_group) {
    case 0: return dequantize_nr<0>(p, s);
    case 16: return dequantize_nr<16>(p, s);
    case 64: return dequantize_nr<64>(p, s);
    case 1024: return dequantize_nr<1024>(p, s);
    default: return dequantize_nr<256>(p, s);
  }
}

}  // namespace cr
