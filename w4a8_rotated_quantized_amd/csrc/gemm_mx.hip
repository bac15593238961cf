// Microscaled 4-bit floating point product (gfx950): out = A W^T + bias with
// both operands as E2M1 codes and one power of two per 32 columns.
//
// v_mfma_scale_f32_32x32x64_f8f6f4 takes the codes and the scale bytes as
// they lie in memory: lane l holds 32 consecutive columns of row l % 32
// (columns 32 (l / 32) .. +31 of the 64) and, in a byte that the instruction
// picks from a register, their power of two. Products of two codes are exact
// and so are the scales, the sums are float32.
//
// Operand layout: codes [ceil(K/128)][rows][64 B], scale bytes
// [ceil(K/128)][rows][4 B]. One 128-column stage of any run of rows is one
// contiguous run of memory for any number of rows, so a block's loads are whole
// lines, and the columns behind K are zeros that the quantizer wrote: the
// loop has no tail.
#include "block.h"
#include "common.h"

namespace cr {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v2f __attribute__((ext_vector_type(2)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
typedef const void __attribute__((address_space(1)))* mx_gptr;
typedef void __attribute__((address_space(3)))* mx_lptr;

constexpr int E2M1 = 4;   // the instruction's format number

CR_DEV v8i mx_operand(u32x4 c) { return v8i{(int)c[0], (int)c[1], (int)c[2], (int)c[3], 0, 0, 0, 0}; }

// s_waitcnt vmcnt(N) lgkmcnt(0)
template <int N>
CR_DEV void mx_wait_vmcnt() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 0xF) | ((N >> 4) << 14) | (0x7 << 4));
}
template <int L>
CR_DEV void mx_wait_stage(int ahead) {   // at most `ahead` later stages (L loads each) left in flight
  if (ahead == 2) mx_wait_vmcnt<2 * L>();
  else if (ahead == 1) mx_wait_vmcnt<L>();
  else mx_wait_vmcnt<0>();
}

// ---------------------------------------------------------------------------
// Block of BM tokens x BN channels, waves of 32 TM x 32 TN, WN waves along the
// channels. A stage is one 128-column tile of both operands, S of them
// rotate in LDS, S - 1 ahead of the one in use. In LDS a row's four 16-byte
// pieces are stored at piece ^ (row / 4 % 4): the 16 rows that one phase of a
// fragment read covers then lie in different banks.
// KG groups of NW waves share a block where blocks are few: group g takes the
// stages g, g + KG, ..., each with a ring of its own, and their sums meet in LDS, in order.
// ---------------------------------------------------------------------------
template <int BM, int BN, int TM, int TN, int S, int MINB, int KG, bool F32>
__global__ __launch_bounds__((BM / (32 * TM)) * (BN / (32 * TN)) * 64 * KG, MINB) void mx_gemm_kernel(MxGemm p) {
  constexpr int WN = BN / (32 * TN);
  constexpr int NW = (BM / (32 * TM)) * WN;
  static_assert(BM % (32 * TM) == 0 && BN % (32 * TN) == 0, "whole wave tiles");
  static_assert(BM % 64 == 0 && BN % 64 == 0, "scale loads take 64 rows");
  static_assert(S >= 2 && S <= 4, "stages in flight ahead of the current one: 0 to 2");
  constexpr int A_ST = BM * 64, W_ST = BN * 64, SC = A_ST + W_ST, STAGE = SC + (BM + BN) * 4;
  constexpr int NC = SC / 1024;                        // 1 KB loads of codes
  constexpr int NS = (BM + BN) / 64;                   // 256-byte loads of scale bytes
  static_assert(NC % NW == 0 && NS <= NW, "even loads");
  static_assert(KG == 1 || (TM == 1 && TN == 1), "sums that meet in LDS: one tile a wave");
  constexpr int LPW = NC / NW;
  constexpr int RS = TN * 64 + 16;                     // epilogue: LDS row stride of a wave's bf16 tile
  constexpr int RF = TN * 128 + 16;                    // ... and of 32 rows in float32
  constexpr int TILE = F32 ? NW * 32 * RF : NW * TM * 32 * RS;
  constexpr int RING = S * STAGE;
  constexpr int SMEM = KG * RING > TILE + (KG - 1) * BM * BN * 4 ? KG * RING : TILE + (KG - 1) * BM * BN * 4;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[SMEM];

  const int tid = threadIdx.x;
  const int l = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6) % NW;
  const int group = KG == 1 ? 0 : __builtin_amdgcn_readfirstlane(tid >> 6) / NW;
  const int wm = wave / WN, wn = wave % WN;

  // block -> tile: consecutive blocks go round robin over the 8 XCDs, so each
  // XCD takes a contiguous range of tiles, in bands of 8 tile rows
  const int ntm = (int)((p.M + BM - 1) / BM);
  const int ntn = (int)((p.N + BN - 1) / BN);
  const int ntiles = ntm * ntn;
  const int xcd = (int)blockIdx.x & 7, q8 = ntiles >> 3, r8 = ntiles & 7;
  const int t = xcd * q8 + min(xcd, r8) + ((int)blockIdx.x >> 3);
  constexpr int GM = 8;
  const int band = t / (GM * ntn);
  const int rows_in_band = min(GM, ntm - band * GM);
  const int within = t - band * GM * ntn;
  const int tn = within / rows_in_band;
  const int tm = band * GM + within % rows_in_band;
  const int64_t m0 = (int64_t)tm * BM, n0 = (int64_t)tn * BN;

  // rows past the end read the last one again; their results are not stored
  const uint8_t* src[LPW];
  int64_t step[LPW];
#pragma unroll
  for (int j = 0; j < LPW; ++j) {
    const int idx = wave + NW * j;
    const int r = idx * 16 + (l >> 2);
    const int piece = ((l & 3) ^ ((l >> 4) & 3)) * 16;
    if (idx < A_ST / 1024) {
      src[j] = p.a + (group * p.M + imin64(m0 + r, p.M - 1)) * 64 + piece;
      step[j] = p.M * 64 * KG;
    } else {
      src[j] = p.w + (group * p.N + imin64(n0 + r - BM, p.N - 1)) * 64 + piece;
      step[j] = p.N * 64 * KG;
    }
  }
  const uint8_t* ssrc;
  int64_t sstep;
  if (wave < BM / 64) {
    ssrc = p.a_scales + (group * p.M + imin64(m0 + wave * 64 + l, p.M - 1)) * 4;
    sstep = p.M * 4 * KG;
  } else {
    ssrc = p.w_scales + (group * p.N + imin64(n0 + wave * 64 + l - BM, p.N - 1)) * 4;
    sstep = p.N * 4 * KG;
  }
  uint8_t* ring = smem + group * RING;
  auto issue = [&](int kb) {                          // the group's stage kb; called in order
    uint8_t* st = ring + (kb % S) * STAGE;
#pragma unroll
    for (int j = 0; j < LPW; ++j) {
      __builtin_amdgcn_global_load_lds((mx_gptr)src[j], (mx_lptr)(st + (wave + NW * j) * 1024), 16, 0, 0);
      src[j] += step[j];
    }
    if (wave < NS) {
      __builtin_amdgcn_global_load_lds((mx_gptr)ssrc, (mx_lptr)(st + SC + wave * 256), 4, 0, 0);
      ssrc += sstep;
    }
  };
  auto wait_stage = [&](int ahead) {
    if (NS == NW || wave < NS) mx_wait_stage<LPW + 1>(ahead);
    else mx_wait_stage<LPW>(ahead);
  };

  v16f acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = v16f{};

  const int h = l >> 5;
  const int piece0 = (h ^ ((l >> 2) & 3)) * 16;        // of the stage's first 64 columns; ^ 32: the second
  const int arow = wm * TM * 32 + (l & 31), wrow = wn * TN * 32 + (l & 31);
  const int nkb = (p.tiles - group + KG - 1) / KG;    // of this group: the first has the most
  const int rounds = (p.tiles + KG - 1) / KG;
#pragma unroll
  for (int s = 0; s < S - 1; ++s)
    if (s < nkb) issue(s);
  for (int kb = 0; kb < rounds; ++kb) {
    if (KG == 1 || kb < nkb) wait_stage(min(S - 2, nkb - 1 - kb));   // this wave's loads of stage kb have landed
    __builtin_amdgcn_s_barrier();                     // ... and every wave's; stage kb - 1 is consumed
    if (KG > 1 && kb >= nkb) break;                   // the last round, and a group without a stage in it
    if (kb + S - 1 < nkb) issue(kb + S - 1);
    const uint8_t* As = ring + (kb % S) * STAGE;
    const uint8_t* Ws = As + A_ST;
    u32x4 av[2][TM], wv[2][TN];
    int as[TM], ws[TN];
#pragma unroll
    for (int kt = 0; kt < 2; ++kt) {
#pragma unroll
      for (int i = 0; i < TM; ++i)
        av[kt][i] = *reinterpret_cast<const u32x4*>(As + (arow + i * 32) * 64 + (piece0 ^ (kt * 32)));
#pragma unroll
      for (int j = 0; j < TN; ++j)
        wv[kt][j] = *reinterpret_cast<const u32x4*>(Ws + (wrow + j * 32) * 64 + (piece0 ^ (kt * 32)));
    }
    // bytes h and 2 + h of a row's four belong to this lane: shifted to bytes 0 and 2
#pragma unroll
    for (int i = 0; i < TM; ++i) as[i] = *reinterpret_cast<const int*>(As + SC + (arow + i * 32) * 4) >> (8 * h);
#pragma unroll
    for (int j = 0; j < TN; ++j) ws[j] = *reinterpret_cast<const int*>(As + SC + (BM + wrow + j * 32) * 4) >> (8 * h);
    // all reads of a stage before its products: left to itself the compiler holds the second half back
    // until the first half's products are under way (8192 x 4096 x 12288: 224 -> 218 us)
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(mx_operand(wv[0][j]), mx_operand(av[0][i]), acc[i][j],
                                                                   E2M1, E2M1, 0, ws[j], 0, as[i]);
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(mx_operand(wv[1][j]), mx_operand(av[1][i]), acc[i][j],
                                                                   E2M1, E2M1, 2, ws[j], 2, as[i]);
  }

  if constexpr (KG > 1) {
    __syncthreads();                                  // every wave is done with the rings
    v4f* meet = reinterpret_cast<v4f*>(smem + TILE) + wave * 256 + l;
    if (group > 0) {
#pragma unroll
      for (int g = 0; g < 4; ++g)
        meet[(group - 1) * NW * 256 + g * 64] = v4f{acc[0][0][4 * g], acc[0][0][4 * g + 1], acc[0][0][4 * g + 2], acc[0][0][4 * g + 3]};
    }
    __syncthreads();
    if (group > 0) return;
#pragma unroll
    for (int o = 0; o < KG - 1; ++o)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const v4f v = meet[o * NW * 256 + g * 64];
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[0][0][4 * g + e] += v[e];
      }
  }
  // lane l of a 32 x 32 result: token l % 32, channels 8 g + 4 (l / 32) + e
  u32x2 bias[TN][4];
#pragma unroll
  for (int j = 0; j < TN; ++j)
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int64_t n = n0 + (wn * TN + j) * 32 + 8 * g + 4 * h;
      bias[j][g] = p.bias && n < p.N ? *reinterpret_cast<const u32x2*>(p.bias + n) : u32x2{0u, 0u};
    }
  if constexpr (F32) {
    // 32 rows at a time through LDS, so that a store covers 128 TN bytes in a row instead of 32
    // (1531 x 2560 x 9216: 32.5 -> 31 us)
    if constexpr (KG == 1) __syncthreads();           // every wave is done with the stages
    uint8_t* tile = smem + wave * (32 * RF);
    constexpr int PR = TN * 8;                        // 16-byte pieces per tile row
#pragma unroll
    for (int i = 0; i < TM; ++i) {
#pragma unroll
      for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int g = 0; g < 4; ++g)
          *reinterpret_cast<v4f*>(tile + (l & 31) * RF + (j * 32 + 8 * g + 4 * h) * 4) =
              v4f{acc[i][j][4 * g] + bf16_lo(bias[j][g][0]), acc[i][j][4 * g + 1] + bf16_hi(bias[j][g][0]),
                  acc[i][j][4 * g + 2] + bf16_lo(bias[j][g][1]), acc[i][j][4 * g + 3] + bf16_hi(bias[j][g][1])};
      // a wave's LDS accesses are in order: its own tile needs no barrier
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int q = 0; q < 32 * PR / 64; ++q) {
        const int pc = q * 64 + l;
        const int r = pc / PR, c = pc % PR;
        const v4f v = *reinterpret_cast<const v4f*>(tile + r * RF + c * 16);
        const int64_t m = m0 + (wm * TM + i) * 32 + r, n = n0 + wn * TN * 32 + c * 4;
        if (m < p.M && n < p.N) *reinterpret_cast<v4f*>(reinterpret_cast<float*>(p.out) + m * p.ldc + n) = v;
      }
      __builtin_amdgcn_wave_barrier();
    }
  } else {
    // the wave's tile passes through LDS, so that stores write whole runs of a row
    if constexpr (KG == 1) __syncthreads();           // every wave is done with the stages
    uint8_t* tile = smem + wave * (TM * 32 * RS);
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const v2bf lo = __builtin_convertvector((v2f{acc[i][j][4 * g] + bf16_lo(bias[j][g][0]),
                                                       acc[i][j][4 * g + 1] + bf16_hi(bias[j][g][0])}), v2bf);
          const v2bf hi = __builtin_convertvector((v2f{acc[i][j][4 * g + 2] + bf16_lo(bias[j][g][1]),
                                                       acc[i][j][4 * g + 3] + bf16_hi(bias[j][g][1])}), v2bf);
          *reinterpret_cast<u32x2*>(tile + (i * 32 + (l & 31)) * RS + (j * 32 + 8 * g + 4 * h) * 2) =
              u32x2{__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi)};
        }
    mx_wait_vmcnt<63>();                              // this wave's tile writes are done
    constexpr int PR = TN * 4;                        // 16-byte pieces per tile row
#pragma unroll
    for (int q = 0; q < TM * 32 * PR / 64; ++q) {
      const int pc = q * 64 + l;
      const int r = pc / PR, c = pc % PR;
      const u32x4 v = *reinterpret_cast<const u32x4*>(tile + r * RS + c * 16);
      const int64_t m = m0 + wm * TM * 32 + r, n = n0 + wn * TN * 32 + c * 8;
      if (m < p.M && n < p.N) *reinterpret_cast<u32x4*>(reinterpret_cast<uint16_t*>(p.out) + m * p.ldc + n) = v;
    }
  }
}

// ---------------------------------------------------------------------------
// Few tokens (M <= 64): the weights are the traffic. A block owns 16 channels,
// its NW waves take the 128-column tiles in turn and read their fragments straight
// from memory: v_mfma_scale_f32_16x16x128_f8f6f4 takes 16 rows x 64 B of a tile,
// which is 1 KB in one piece (lane l: row l % 16, columns 32 (l / 16) .. +31).
// U tiles a wave are loaded before the first is used: with U = 2 all of a matrix up to K = 4096
// (16 waves) or 2048 (8) is on its way at once, a longer one takes further trips, each with a latency
// of its own (K = 2560 with 8 waves: four of them make a second). Tokens past the end are zeros without a load.
// Partial sums meet in LDS in a fixed order.
// ---------------------------------------------------------------------------
template <int FM, int NW, int U, bool F32>
__global__ __launch_bounds__(NW * 64) void mx_few_kernel(MxGemm p) {
  static_assert(FM <= NW, "a wave for each 16 tokens' sums");
  __shared__ __attribute__((aligned(16))) float red[NW][FM][64][4];
  const int l = threadIdx.x & 63, r = l & 15, q = l >> 4;
  const int wave = threadIdx.x >> 6;
  const int64_t n0 = (int64_t)blockIdx.x * 16;
  const int64_t n = imin64(n0 + r, p.N - 1);
  v4f acc[FM];
#pragma unroll
  for (int i = 0; i < FM; ++i) acc[i] = v4f{0.f, 0.f, 0.f, 0.f};

  for (int t0 = wave; t0 < p.tiles; t0 += NW * U) {
    u32x4 wr[U], ar[U][FM];
    int ws[U], as[U][FM];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int t = t0 + u * NW;
      if (t >= p.tiles) break;
      const int64_t at = (int64_t)t * p.N + n;
      wr[u] = *reinterpret_cast<const u32x4*>(p.w + at * 64 + q * 16);
      ws[u] = p.w_scales[at * 4 + q];
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        ar[u][i] = u32x4{0, 0, 0, 0};
        as[u][i] = 0;
        const int64_t m = i * 16 + r;
        if (m < p.M) {
          const int64_t to = (int64_t)t * p.M + m;
          ar[u][i] = *reinterpret_cast<const u32x4*>(p.a + to * 64 + q * 16);
          as[u][i] = p.a_scales[to * 4 + q];
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (t0 + u * NW >= p.tiles) break;
#pragma unroll
      for (int i = 0; i < FM; ++i)
        acc[i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(mx_operand(wr[u]), mx_operand(ar[u][i]), acc[i], E2M1, E2M1,
                                                                  0, ws[u], 0, as[u][i]);
    }
  }
#pragma unroll
  for (int i = 0; i < FM; ++i) *reinterpret_cast<v4f*>(red[wave][i][l]) = acc[i];
  __syncthreads();
  if (wave < FM) {
    v4f y = *reinterpret_cast<const v4f*>(red[0][wave][l]);
#pragma unroll
    for (int w = 1; w < NW; ++w) y += *reinterpret_cast<const v4f*>(red[w][wave][l]);
    // lane l of the 16 x 16 result: token l % 16, channels 4 (l / 16) + e
    const int64_t m = wave * 16 + r, c = n0 + q * 4;
    if (m < p.M && c < p.N) {
      if (p.bias) {
        const u32x2 b = *reinterpret_cast<const u32x2*>(p.bias + c);
        y += v4f{bf16_lo(b[0]), bf16_hi(b[0]), bf16_lo(b[1]), bf16_hi(b[1])};
      }
      if constexpr (F32) {
        *reinterpret_cast<v4f*>(reinterpret_cast<float*>(p.out) + m * p.ldc + c) = y;
      } else {
        const v2bf lo = __builtin_convertvector((v2f{y[0], y[1]}), v2bf), hi = __builtin_convertvector((v2f{y[2], y[3]}), v2bf);
        *reinterpret_cast<u32x2*>(reinterpret_cast<uint16_t*>(p.out) + m * p.ldc + c) =
            u32x2{__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi)};
      }
    }
  }
}

template <int BM, int BN, int TM, int TN, int S, int MINB, int KG, bool F32>
static void launch_tiles(const MxGemm& p, hipStream_t s) {
  const int64_t tiles = ((p.M + BM - 1) / BM) * ((p.N + BN - 1) / BN);
  hipLaunchKernelGGL((mx_gemm_kernel<BM, BN, TM, TN, S, MINB, KG, F32>), dim3((unsigned)tiles),
                     dim3((BM / (32 * TM)) * (BN / (32 * TN)) * 64 * KG), 0, s, p);
}

// 16 waves a block up to one block a compute unit, 8 beyond: 1 x 4096, N = 4096: 4.0 us either way; 1 x 9728,
// N = 2560: 4.9 against 6.2 us; 22 x 2560, N = 9728: 7.5 against 6.2 us
template <int FM, bool F32>
static void launch_few(const MxGemm& p, hipStream_t s) {
  const int64_t blocks = (p.N + 15) / 16;
  if (blocks <= 256) hipLaunchKernelGGL((mx_few_kernel<FM, 16, 2, F32>), dim3((unsigned)blocks), dim3(1024), 0, s, p);
  else hipLaunchKernelGGL((mx_few_kernel<FM, 8, 2, F32>), dim3((unsigned)blocks), dim3(512), 0, s, p);
}

template <bool F32>
static hipError_t launch_out(const MxGemm& p, hipStream_t s) {
  if (p.M <= 64) {
    switch ((p.M + 15) / 16) {
      case 1: launch_few<1, F32>(p, s); break;
      case 2: launch_few<2, F32>(p, s); break;
      case 3: launch_few<3, F32>(p, s); break;
      default: launch_few<4, F32>(p, s); break;
    }
    return hipGetLastError();
  }
  // The block shape with the least time. A compute unit that has n blocks to do takes at least `alone` a
  // stage (one block's own chain of waits) and n times `each` once they fill it, in ns. Measured with K = 4096, the product alone in a row
  // (256 x 256, 128 x 128, 128 x 64, 64 x 64 blocks, in us): 8192 x 12288: 218, 253, -, -; 4096 x 4096: 39, 50, 53, 62;
  // 2048 x 4096: 31, 23, 30, 33; 1024 x 4096: 29, 17, 15, 18; 512 x 4096: 29, 16, 13, 11; and 1531 x 2560, N = 9216:
  // 25, 29, 32, 36.
  auto tiles = [&](int64_t bm, int64_t bn) { return ((p.M + bm - 1) / bm) * ((p.N + bn - 1) / bn); };
  auto cost = [&](int64_t bm, int64_t bn, int64_t alone, int64_t each) {
    const int64_t n = (tiles(bm, bn) + 255) / 256;
    return n * each > alone ? n * each : alone;
  };
  const int64_t c256 = cost(256, 256, 900, 1200), c128 = cost(128, 128, 500, 330), c12864 = cost(128, 64, 390, 230),
                c64 = cost(64, 64, 310, 140);
  if (c256 <= c128 && c256 <= c12864 && c256 <= c64) launch_tiles<256, 256, 4, 2, 4, 1, 1, F32>(p, s);
  else if (c128 <= c12864 && c128 <= c64) launch_tiles<128, 128, 2, 2, 3, 3, 1, F32>(p, s);
  else if (c12864 <= c64) launch_tiles<128, 64, 2, 1, 4, 3, 1, F32>(p, s);
  // one block a compute unit leaves it waiting: four groups share the stages, from where each has some
  // (65 x 4096 x 4096: 9.5 -> 7.5 us, 128 x 9728 x 2560: 18.6 -> 12.5; 300 x 1024 x 328 with 8 stages: 4.4 -> 4.8)
  else if (tiles(64, 64) <= 256 && p.tiles >= 16) launch_tiles<64, 64, 1, 1, 4, 1, 4, F32>(p, s);
  else launch_tiles<64, 64, 1, 1, 4, 4, 1, F32>(p, s);
  return hipGetLastError();
}

hipError_t launch_mx_gemm(const MxGemm& p, hipStream_t s) {
  return p.out_f32 ? launch_out<true>(p, s) : launch_out<false>(p, s);
}

}  // namespace cr
