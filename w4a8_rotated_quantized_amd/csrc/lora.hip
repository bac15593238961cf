// Low-rank adapters of many requests beside one shared projection, forward
// and backward (gfx950, bf16 matrix cores).
//
// The rows of a batch fall into segments, each with an adapter a (or none):
//   la[m, r]   = sum_k x[m, k] down[a][r, k]                      "shrink"
//   out[m, n]  = base[m, n] + c_a sum_r la[m, r] up[a][n, r]       "expand"
// and backward
//   dla[m, r]  = c_a sum_n dy[m, n] up[a][n, r]                    shrink by up
//   dx[m, k]   = dx_base[m, k] + sum_r dla[m, r] down[a][r, k]     expand by down
//   d_up[a]    = c_a sum_m dy[m, :]^T la[m, :]                     "outer"
//   d_down[a]  = sum_m dla[m, :]^T x[m, :]                         outer
// With x saved as rotated INT8 codes, x = (s q) H / sqrt(n) per rotation
// group, so d_down = (sum_m (dla[m, :] s[m])^T q[m, :]) H / sqrt(n): the long
// sum runs on the codes and only the small [R, K] result is rotated back.
//
// la and dla are float32. Where they meet bf16 operands on the matrix cores
// they are split into three bf16 terms (8 + 8 + 8 bits of the 24), whose
// products are exact in float32: the only roundings are those of the float32
// sums and of the stored outputs.
#include "common.h"
#include "lora.h"
#include "rotate.h"

#include <type_traits>

namespace cr {

typedef __bf16 v2bf __attribute__((ext_vector_type(2)));

CR_DEV v4f mfma16(v8bf a, v8bf b, v4f c) { return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0); }

// ---------------------------------------------------------------------------
// segments -> row tiles
// ---------------------------------------------------------------------------
// Boundary v (0 .. S + 2) of the S + 2 stretches that cover all M rows: the
// rows before the first segment, the S segments, and the rows behind the last
// one. Every value lies in [0, M] whatever the offsets hold, so no tile leaves
// the batch. An offset below an earlier one counts as that earlier one: both
// users take the running maximum of these values, so every row lies in exactly
// one stretch and M / T + S + 2 tiles of T rows are enough for any offsets. The
// load is unconditional, its index clamped: loads of several boundaries are
// then under way together.
CR_DEV int seg_bound(const LoraSegments& g, int v) {
  const int at = v - 1;
  int o = g.off[at < 0 ? 0 : (at > g.S ? g.S : at)];
  o = o < 0 ? 0 : (o > g.M ? g.M : o);
  return v <= 0 ? 0 : (v >= g.S + 2 ? g.M : o);
}
CR_DEV int seg_adapter(const LoraSegments& g, int v) {   // adapter of stretch v, or -1
  const int at = v - 1;
  const int a = g.id[at < 0 ? 0 : (at >= g.S ? g.S - 1 : at)];
  return (v < 1 || v > g.S || a < 0 || a >= g.A) ? -1 : a;
}

struct RowTile {
  int lo, hi, a;   // rows [lo, hi) of one stretch and its adapter (-1: none); lo == hi: no tile
};

// inclusive sum over the wave's 64 lanes: within rows of 16, then across them
CR_DEV int wave_scan(int x) {
  x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xF, 0xF, false);   // row_shr:1
  x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xF, 0xF, false);   // row_shr:2
  x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xF, 0xF, false);   // row_shr:4
  x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xF, 0xF, false);   // row_shr:8
  x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xA, 0xF, false);   // row_bcast:15 into rows 1 and 3
  x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xC, 0xF, false);   // row_bcast:31 into rows 2 and 3
  return x;
}

// running maximum over the wave's lanes of values from 0 on
CR_DEV int wave_scan_max(int x) {
  auto with = [&](int o) { x = x > o ? x : o; };
  with(__builtin_amdgcn_update_dpp(0, x, 0x111, 0xF, 0xF, false));   // the same steps
  with(__builtin_amdgcn_update_dpp(0, x, 0x112, 0xF, 0xF, false));
  with(__builtin_amdgcn_update_dpp(0, x, 0x114, 0xF, 0xF, false));
  with(__builtin_amdgcn_update_dpp(0, x, 0x118, 0xF, 0xF, false));
  with(__builtin_amdgcn_update_dpp(0, x, 0x142, 0xA, 0xF, false));
  with(__builtin_amdgcn_update_dpp(0, x, 0x143, 0xC, 0xF, false));
  return x;
}

// Rows [lo, hi) of the lane's stretch v and the running maximum behind the
// wave's last one; top: that of the stretches before.
struct Stretch {
  int lo, hi, top;
};
CR_DEV Stretch seg_rows(const LoraSegments& g, int v, int top) {
  const int start = seg_bound(g, v), end = seg_bound(g, v + 1);
  Stretch r;
  r.lo = wave_scan_max(start > top ? start : top);
  r.hi = end > r.lo ? end : r.lo;
  r.top = __builtin_amdgcn_readlane(r.hi, 63);
  return r;
}

// Tile t of T rows (a power of two), counted through the stretches: each wave scans the tile
// counts of 64 stretches at a time. All 64 lanes take part; the result is
// the same in all of them.
CR_DEV RowTile find_tile(const LoraSegments& g, int t, int T) {
  const int lane = threadIdx.x & 63;
  int top = 0;
  for (int v0 = 0; v0 < g.S + 2; v0 += 64) {
    const int v = v0 + lane;
    const int a = seg_adapter(g, v);
    const Stretch st = seg_rows(g, v, top);        // behind the last stretch: M to M
    top = st.top;
    const int n = (st.hi - st.lo + T - 1) >> __builtin_ctz(T);
    const int upto = wave_scan(n);
    const int total = __builtin_amdgcn_readlane(upto, 63);
    if (t < total) {
      const int src = __builtin_ctzll(__ballot(upto > t));
      const int slo = __builtin_amdgcn_readlane(st.lo, src), shi = __builtin_amdgcn_readlane(st.hi, src);
      const int skip = t - (__builtin_amdgcn_readlane(upto, src) - __builtin_amdgcn_readlane(n, src));
      RowTile r;
      r.lo = slo + skip * T;
      r.hi = r.lo + T < shi ? r.lo + T : shi;
      r.a = __builtin_amdgcn_readlane(a, src);
      return r;
    }
    t -= total;
  }
  return RowTile{0, 0, -1};
}

// tiles of T rows that M rows in S segments can need at most
static unsigned tile_grid(const LoraSegments& g, int T) {
  const int64_t n = (int64_t)g.M / T + g.S + 2;
  return (unsigned)(n < g.M ? n : g.M);
}

// ---------------------------------------------------------------------------
// operand fragments
// ---------------------------------------------------------------------------
CR_DEV v8bf load8(const uint16_t* p, bool ok) {
  const u32x4 z = {0, 0, 0, 0};
  return __builtin_bit_cast(v8bf, ok ? *reinterpret_cast<const u32x4*>(p) : z);
}

// f = hi + mid + lo, each a bf16 value: truncation leaves remainders that are
// exact in float32. An infinity or NaN goes into hi alone. An infinite partner
// of a finite f meets mid and lo too, often zeros: the sum is NaN then where the
// product alone were infinite, not finite in either case.
struct Split {
  uint32_t hi, mid, lo;   // bf16 bits in the upper half
};
CR_DEV Split split3(float f) {
  const uint32_t b = __float_as_uint(f);
  const bool special = (b & 0x7F800000u) == 0x7F800000u;
  Split s;
  s.hi = b & 0xFFFF0000u;
  if ((b & 0x7FFFFFFFu) > 0x7F800000u) s.hi |= 0x00400000u;
  const float r1 = special ? 0.f : f - __uint_as_float(b & 0xFFFF0000u);
  s.mid = __float_as_uint(r1) & 0xFFFF0000u;
  const float r2 = r1 - __uint_as_float(s.mid);
  s.lo = __float_as_uint(r2) & 0xFFFF0000u;
  return s;
}
// bf16 pair from the upper halves of two words
CR_DEV uint32_t upper_pair(uint32_t lo, uint32_t hi) { return __builtin_amdgcn_perm(hi, lo, 0x07060302u); }

// eight values as three operand fragments: hi, mid, lo
CR_DEV void split8(const float (&v)[8], u32x4 (&f)[3]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const Split a = split3(v[2 * i]), b = split3(v[2 * i + 1]);
    f[0][i] = upper_pair(a.hi, b.hi);
    f[1][i] = upper_pair(a.mid, b.mid);
    f[2][i] = upper_pair(a.lo, b.lo);
  }
}

// A float32 [M][R] matrix in the operand order of "outer", whose products run
// over rows: [3 terms][ceil(M / 8)][R][8 rows] of bf16.
CR_DEV int64_t rows8_index(int M, int R, int term, int m, int r) {
  return (((int64_t)term * ((M + 7) / 8) + m / 8) * R + r) * 8 + m % 8;
}
static size_t rows8_bytes(int64_t M, int R) { return (size_t)(3 * ((M + 7) / 8) * 8 * R) * 2; }

// Between LDS accesses of one wave to what its other lanes wrote or will
// write: the hardware keeps their order, the compiler has to as well.
CR_DEV void wave_lds_order() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// ---------------------------------------------------------------------------
// shrink: la[m, r] = (c_a) sum_c x[m, c] w[a][r][c]
// ---------------------------------------------------------------------------
struct ShrinkArgs {
  const uint16_t* x;
  int64_t ldx;
  const uint16_t* w;     // [A][R][C]
  LoraSegments seg;
  const float* scale;    // multiplies the result, or null
  float* la;             // [M][R]
  uint16_t* rows8;       // the result (times row_scales) once more, for "outer", or null
  const float* row_scales;   // [M] or [1] (row_scaled 0), or null
  int row_scaled;
  int R, C;
};

typedef __attribute__((address_space(1))) void* lora_gptr;
typedef __attribute__((address_space(3))) void* lora_lptr;

// s_waitcnt vmcnt(N), other counters untouched (gfx9 encoding: vmcnt[3:0] in
// bits 3:0, vmcnt[5:4] in bits 15:14, expcnt in bits 6:4, lgkmcnt in bits 11:8)
template <int N>
CR_DEV void wait_vmcnt() {
  __builtin_amdgcn_s_waitcnt((N & 0xF) | ((N >> 4) << 14) | (0x7 << 4) | (0xF << 8));
}

template <int RG, int TM, int NW, int DX, int DW>
struct ShrinkLds {
  static constexpr int nx = 2 * TM, nw = 2 * RG;   // loads (KB) of a stage: of x, of the weights
  static constexpr int red = RG * TM * 64;         // 16-byte sums of a wave
  static constexpr int ring = (DX * nx + DW * nw) * 1024 > red * 16 ? (DX * nx + DW * nw) * 1024 : red * 16;
  static constexpr int bytes = NW * ring;
};

// The sums of TM x 16 rows of one segment and 16 RG ranks. A block's NW waves
// share the columns in stages of 64 and add their sums through LDS in a fixed
// order (the caller does: lds holds [NW][RG TM 64] of them). A stage goes straight from memory into the wave's own LDS rings, DX
// stages of x (from memory far away) and DW <= DX of the weights (from L2): one load moves 8 rows x 128 bytes, neighbouring lanes taking
// neighbouring 16 bytes, so that every request is a whole line (the operand
// order of the matrix cores, neighbouring lanes on different rows, reads the
// same bytes from L2 2.6 times slower: 15.5 against 5.9 us for 256 x 512 KB).
// Within a row's 128 bytes, chunk q lies at position q ^ (row % 8), which
// spreads the fragment reads over the banks. 8192 rows, 4096 columns: 23.4 us at
// rank 16 (2.9 TB/s of x), 38 us at rank 64 (1.8 TB/s), where nothing is behind
// the one stage of the rings that is waited for, and the weights, read from L2 for
// every 32 rows, are twice the bytes of x.
//
// WT: the weights lie the other way, [A][C][R]. A load then takes the 16 ranks of
// 32 columns, two lanes a column, and a fragment is gathered two bytes at a
// time; column 8 g + e of the load lies at position 8 g + (e + 2 g) % 8, which
// spreads these reads over the banks. Four times the LDS reads, so it is for
// few ranks only, where a launch that transposes first costs more.
template <int RG, int TM, int NW, int DX, int DW, bool WT>
CR_DEV void shrink_sums(const ShrinkArgs& p, const RowTile& t, int r0, int bx, uint8_t* lds) {
  static_assert(!WT || RG == 1, "a load holds the ranks of one group");
  typedef ShrinkLds<RG, TM, NW, DX, DW> L;
  constexpr int NX = L::nx, NWT = L::nw, RED = L::red;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int i = lane & 15, g = lane >> 4;
  const int lr = lane >> 3, lc = 8 * ((lane & 7) ^ lr);   // row and column of the lane's 16 bytes in a load
  const uint16_t* xr[NX];
  const uint16_t* wr[NWT];
#pragma unroll
  for (int n = 0; n < NX; ++n) {
    const int m = t.lo + 8 * n + lr;
    xr[n] = p.x + (int64_t)(m < t.hi ? m : t.hi - 1) * p.ldx;             // past the tile: computed for nothing
  }
#pragma unroll
  for (int n = 0; n < NWT; ++n) {
    if constexpr (WT) {
      const int r = r0 + 8 * (lane & 1);
      wr[n] = p.w + (int64_t)t.a * p.C * p.R + (r < p.R ? r : 0);
    } else {
      const int r = r0 + 8 * n + lr;
      wr[n] = p.w + ((int64_t)t.a * p.R + (r < p.R ? r : p.R - 1)) * p.C;
    }
  }
  const int wc = (lane >> 4) * 8 + (((lane >> 1) - 2 * (lane >> 4)) & 7);   // WT: the lane's column of a load
  uint8_t* xring = lds + wave * ShrinkLds<RG, TM, NW, DX, DW>::ring;
  uint8_t* wring = xring + DX * NX * 1024;
  const int stages = ((p.C + 63) / 64 - wave + NW - 1) / NW;   // may be 0
  // blocks start at different columns: rows a power of two apart share an L2 channel
  // (rank 64, K = 4096: 21 against 29 us from the cache)
  const int first = stages ? bx % stages : 0;
  auto column = [&](int s) { s += first; return ((s < stages ? s : s - stages) * NW + wave) * 64; };
  auto lane_column = [&](int s) {
    const int c = column(s) + lc;
    return c < p.C ? c : 0;                        // past the last column: loaded for nothing
  };
  auto load_x = [&](int s, int slot) {
    const int c = lane_column(s);
#pragma unroll
    for (int n = 0; n < NX; ++n)
      __builtin_amdgcn_global_load_lds((lora_gptr)(xr[n] + c), (lora_lptr)(xring + (slot * NX + n) * 1024), 16, 0, 0);
  };
  auto load_w = [&](int s, int slot) {
#pragma unroll
    for (int n = 0; n < NWT; ++n) {
      int64_t at = lane_column(s);
      if constexpr (WT) {
        const int c = column(s) + 32 * n + wc;
        at = (int64_t)(c < p.C ? c : 0) * p.R;
      }
      __builtin_amdgcn_global_load_lds((lora_gptr)(wr[n] + at), (lora_lptr)(wring + (slot * NWT + n) * 1024), 16, 0, 0);
    }
  };
  v4f acc[RG][TM];
#pragma unroll
  for (int rg = 0; rg < RG; ++rg)
#pragma unroll
    for (int tm = 0; tm < TM; ++tm) acc[rg][tm] = v4f{0.f, 0.f, 0.f, 0.f};
  // Issue order: x 0 .. DX - DW - 1, then for s = 0, 1, ...: w s, x s + DX - DW.
#pragma unroll
  for (int d = 0; d < DX; ++d) {
    if (d >= DX - DW && d - (DX - DW) < stages) load_w(d - (DX - DW), d - (DX - DW));
    if (d < stages) load_x(d, d);
  }
  int xs = 0, ws = 0;
#pragma unroll 1
  for (int s = 0; s < stages; ++s) {
    // Behind w s and x s in the queue: x s + DX - DW when x s is older than w s, and the
    // DW - 1 pairs after it; fewer at the end, where everything is waited for.
    constexpr int LATER = (DW - 1) * (NWT + NX) + (DX > DW ? NX : 0);
    if (LATER > 0 && s + DX <= stages) wait_vmcnt<LATER>();
    else wait_vmcnt<0>();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    u32x4 xf[TM][2], wf[RG][2];
    const int at = i * 128, sw = i & 7;            // 16 rows of an operand lie one after the other
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int tm = 0; tm < TM; ++tm)
        xf[tm][h] = *reinterpret_cast<const u32x4*>(xring + (xs * NX + 2 * tm) * 1024 + at + ((4 * h + g) ^ sw) * 16);
#pragma unroll
      for (int rg = 0; rg < RG; ++rg) {
        if constexpr (WT) {
          const uint16_t* src = reinterpret_cast<const uint16_t*>(wring + (ws * NWT + h) * 1024) + i;
#pragma unroll
          for (int k = 0; k < 4; ++k)
            wf[rg][h][k] = (uint32_t)src[(8 * g + ((2 * k + 2 * g) & 7)) * 16] |
                           ((uint32_t)src[(8 * g + ((2 * k + 1 + 2 * g) & 7)) * 16] << 16);
        } else {
          wf[rg][h] = *reinterpret_cast<const u32x4*>(wring + (ws * NWT + 2 * rg) * 1024 + at + ((4 * h + g) ^ sw) * 16);
        }
      }
    }
    __builtin_amdgcn_s_waitcnt(0xC07F);            // lgkmcnt(0): read before the slots are filled again
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    if (s + DW < stages) load_w(s + DW, ws);
    if (s + DX < stages) load_x(s + DX, xs);
    xs = xs + 1 == DX ? 0 : xs + 1;
    ws = ws + 1 == DW ? 0 : ws + 1;
    const int c0 = column(s);
    if (c0 + 64 > p.C) {                           // the last columns: zeros past C (C % 8 == 0)
      const u32x4 z = {0, 0, 0, 0};
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const bool ok = c0 + 32 * h + 8 * g < p.C;
#pragma unroll
        for (int tm = 0; tm < TM; ++tm) xf[tm][h] = ok ? xf[tm][h] : z;
#pragma unroll
        for (int rg = 0; rg < RG; ++rg) wf[rg][h] = ok ? wf[rg][h] : z;
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int rg = 0; rg < RG; ++rg)
#pragma unroll
        for (int tm = 0; tm < TM; ++tm)
          acc[rg][tm] = mfma16(__builtin_bit_cast(v8bf, wf[rg][h]), __builtin_bit_cast(v8bf, xf[tm][h]), acc[rg][tm]);
  }
  __syncthreads();                                 // the rings are done with: their memory takes the sums
  v4f* red = reinterpret_cast<v4f*>(lds);
#pragma unroll
  for (int rg = 0; rg < RG; ++rg)
#pragma unroll
    for (int tm = 0; tm < TM; ++tm) red[wave * RED + (rg * TM + tm) * 64 + lane] = acc[rg][tm];
  __syncthreads();
}

// a block: TM x 16 rows of one segment and 16 RG ranks
template <int RG, int TM, int NW, int DX, int DW, bool WT>
CR_DEV void shrink_block(const ShrinkArgs& p, int bx, int by, uint8_t* lds) {
  constexpr int RED = ShrinkLds<RG, TM, NW, DX, DW>::red;
  const int r0 = by * 16 * RG;
  const RowTile t = find_tile(p.seg, bx, 16 * TM);
  if (t.lo >= t.hi) return;
  if (t.a < 0) {                                  // rows without adapter: zeros
    const int nr = p.R - r0 < 16 * RG ? p.R - r0 : 16 * RG;
    for (int k = threadIdx.x; k < (t.hi - t.lo) * nr; k += 64 * NW)
      p.la[(int64_t)(t.lo + k / nr) * p.R + r0 + k % nr] = 0.f;
    return;
  }
  shrink_sums<RG, TM, NW, DX, DW, WT>(p, t, r0, bx, lds);
  const v4f* red = reinterpret_cast<const v4f*>(lds);
  const float cs = p.scale ? p.scale[t.a] : 1.f;
  for (int k = threadIdx.x; k < RED; k += 64 * NW) {
    const int rg = k / 64 / TM, tm = k / 64 % TM, kl = k % 64;
    const int m = t.lo + 16 * tm + (kl & 15), r = r0 + 16 * rg + 4 * (kl >> 4);
    if (m >= t.hi || r >= p.R) continue;           // R % 8 == 0: four ranks in or out together
    v4f s = red[k];
    for (int n = 1; n < NW; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[e] += red[n * RED + k][e];
#pragma unroll
    for (int e = 0; e < 4; ++e) s[e] *= cs;
    *reinterpret_cast<v4f*>(p.la + (int64_t)m * p.R + r) = s;
    if (p.rows8) {
      const float rs = p.row_scales ? p.row_scales[p.row_scaled ? m : 0] : 1.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const Split q = split3(s[e] * rs);
        p.rows8[rows8_index(p.seg.M, p.R, 0, m, r + e)] = (uint16_t)(q.hi >> 16);
        p.rows8[rows8_index(p.seg.M, p.R, 1, m, r + e)] = (uint16_t)(q.mid >> 16);
        p.rows8[rows8_index(p.seg.M, p.R, 2, m, r + e)] = (uint16_t)(q.lo >> 16);
      }
    }
  }
}

template <int RG, int TM, int NW, int DX, int DW>
__global__ __launch_bounds__(64 * NW) void lora_shrink_kernel(ShrinkArgs p) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[ShrinkLds<RG, TM, NW, DX, DW>::bytes];
  shrink_block<RG, TM, NW, DX, DW, false>(p, blockIdx.x, blockIdx.y, lds);
}

static hipError_t launch_shrink(const ShrinkArgs& p, hipStream_t s) {
  const int rg = (p.R + 15) / 16;
  const unsigned t16 = tile_grid(p.seg, 16), t32 = tile_grid(p.seg, 32);
  // 32-row tiles where they make a block for every one of the 256 compute units (rank 128, 7569 rows,
  // K = 952: 12.8 against 14.9 us in 16-row tiles)
  const bool many = p.seg.M / 32 * ((rg + 3) / 4) >= 256;
  // 16 ranks a block while every compute unit gets at most one: more of them take part (64 single
  // rows of rank 64, K = 4096: 3 us less than 64 ranks a block; 256, which make 1024 blocks, 10 us more)
  // (32 ranks a block by the same rule: 1631 rows of rank 64, K = 6768: 15.8 against 20.2 us)
  if (t16 * rg <= 256) hipLaunchKernelGGL((lora_shrink_kernel<1, 1, 16, 2, 2>), dim3(t16, rg), dim3(1024), 0, s, p);
  else if (t16 * ((rg + 1) / 2) <= 256) hipLaunchKernelGGL((lora_shrink_kernel<2, 1, 8, 2, 2>), dim3(t16, (rg + 1) / 2), dim3(512), 0, s, p);
  else if (rg <= 1) hipLaunchKernelGGL((lora_shrink_kernel<1, 1, 8, 3, 2>), dim3(t16), dim3(512), 0, s, p);
  else if (rg <= 2 && !many) hipLaunchKernelGGL((lora_shrink_kernel<2, 1, 8, 2, 2>), dim3(t16), dim3(512), 0, s, p);
  else if (rg <= 2) hipLaunchKernelGGL((lora_shrink_kernel<2, 2, 5, 2, 2>), dim3(t32), dim3(320), 0, s, p);
  else if (!many) hipLaunchKernelGGL((lora_shrink_kernel<4, 1, 8, 1, 1>), dim3(t16, (rg + 3) / 4), dim3(512), 0, s, p);
  else hipLaunchKernelGGL((lora_shrink_kernel<4, 2, 6, 1, 1>), dim3(t32, (rg + 3) / 4), dim3(384), 0, s, p);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// expand: out[m, c] = base[m, c] + sum_r (c_a la[m, r]) w[a][c][r]
// ---------------------------------------------------------------------------
struct ExpandArgs {
  const float* la;
  const uint16_t* w;     // [A][C][R]
  LoraSegments seg;
  const float* scale;    // multiplies la, or null
  const void* base;
  int64_t ldb;
  void* out;
  int64_t ldo;
  int R, C;
  int rows;              // of a tile, a power of two from 16 on (lora_expand_kernel)
  int blocks_x;          // tiles at most
};

template <typename T>
CR_DEV void load_out8(const T* p, float (&v)[8]) {
  if constexpr (sizeof(T) == 2) {
    const u32x4 w = *reinterpret_cast<const u32x4*>(p);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[2 * k] = bf16_lo(w[k]);
      v[2 * k + 1] = bf16_hi(w[k]);
    }
  } else {
    const v4f a = *reinterpret_cast<const v4f*>(p), b = *reinterpret_cast<const v4f*>(p + 4);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[k] = a[k];
      v[4 + k] = b[k];
    }
  }
}
template <typename T>
CR_DEV void store_out8(T* p, const float (&v)[8]) {
  if constexpr (sizeof(T) == 2) {
    u32x4 w;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      w[k] = __builtin_bit_cast(uint32_t, v2bf{(__bf16)v[2 * k], (__bf16)v[2 * k + 1]});   // half to even, NaN kept
    *reinterpret_cast<u32x4*>(p) = w;
  } else {
    *reinterpret_cast<v4f*>(p) = v4f{v[0], v[1], v[2], v[3]};
    *reinterpret_cast<v4f*>(p + 4) = v4f{v[4], v[5], v[6], v[7]};
  }
}

// What one wave does with 16 NJ columns from c0 on.
template <int KS, int NJ, typename T>
struct ExpandWave {
  static constexpr int W = 16 * NJ;
  static constexpr int V = 16 / sizeof(T);        // columns of one 16-byte access of base and out
  static constexpr int CPR = W / V;               // accesses per row
  static constexpr int NB = 16 * CPR / 64;        // accesses per lane and 16 rows
  static constexpr int PITCH = W + 4;             // floats of a row of sums in LDS
  const ExpandArgs& p;
  const RowTile& t;
  int c0, lane;
  // Without a base the loads go to one row of the adapter's weights, which are at
  // hand (R >= 8 values of bf16 per column are longer than a row of out), and the
  // mask makes zeros of them: no branch between a load and its use.
  CR_DEV uint32_t mask() const { return p.base ? ~0u : 0u; }

  // access q: row lane / CPR + q * 64 / CPR, columns column() ..; C % 8 == 0: in or out as a whole
  CR_DEV int row(int q) const { return lane / CPR + q * (64 / CPR); }
  CR_DEV int column() const { return c0 + lane % CPR * V; }
  CR_DEV void load_base(u32x4 (&b)[NB], int mt) const {
    const int c = column() < p.C ? column() : 0;
    const T* from = static_cast<const T*>(p.base ? p.base : static_cast<const void*>(p.w));
    const int64_t ld = p.base ? p.ldb : 0;
#pragma unroll
    for (int q = 0; q < NB; ++q) {
      const int m = mt + row(q);                  // past the tile: its last row, for nothing
      b[q] = *reinterpret_cast<const u32x4*>(from + (int64_t)(m < t.hi ? m : t.hi - 1) * ld + c);
    }
  }
  CR_DEV void store(const u32x4& v, int q, int mt) const {
    const int m = mt + row(q);
    if (m < t.hi && column() < p.C) *reinterpret_cast<u32x4*>(static_cast<T*>(p.out) + (int64_t)m * p.ldo + column()) = v;
  }
  // rows without adapter: the base alone, nothing if that is out itself
  CR_DEV void copy_base() const {
    if (p.base == p.out) return;
    const uint32_t keep = mask();
    for (int mt = t.lo; mt < t.hi; mt += 16) {
      u32x4 b[NB];
      load_base(b, mt);
#pragma unroll
      for (int q = 0; q < NB; ++q) store(u32x4{b[q][0] & keep, b[q][1] & keep, b[q][2] & keep, b[q][3] & keep}, q, mt);
    }
  }
  CR_DEV void load_weights(v8bf (&wf)[NJ][KS]) const {
    const int i = lane & 15, g = lane >> 4;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const int c = c0 + 16 * j + i < p.C ? c0 + 16 * j + i : p.C - 1;
      const uint16_t* w = p.w + ((int64_t)t.a * p.C + c) * p.R;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        const int r = 32 * ks + 8 * g;
        const u32x4 v = *reinterpret_cast<const u32x4*>(w + (r < p.R ? r : 0)), z = {0, 0, 0, 0};
        wf[j][ks] = __builtin_bit_cast(v8bf, r < p.R ? v : z);
      }
    }
  }
  // 16 rows from mt on: la3 holds their lora_act as three bf16 terms ([term][octet of ranks][SUB
  // rows], these from row0 on), sums takes the products and gives them back by rows
  template <int SUB>
  CR_DEV void add_rows(const v8bf (&wf)[NJ][KS], const u32x4 (*la3)[4 * KS][SUB], int row0, float* sums,
                       const u32x4 (&b)[NB], int mt) const {
    const int i = lane & 15, g = lane >> 4;
    const uint32_t keep = mask();
    v4f acc[NJ];
#pragma unroll
    for (int j = 0; j < NJ; ++j) acc[j] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int ks = 0; ks < KS; ++ks)
#pragma unroll
      for (int term = 2; term >= 0; --term) {     // the small terms first
        const v8bf f = __builtin_bit_cast(v8bf, la3[term][4 * ks + g][row0 + i]);
#pragma unroll
        for (int j = 0; j < NJ; ++j) acc[j] = mfma16(wf[j][ks], f, acc[j]);
      }
#pragma unroll
    for (int j = 0; j < NJ; ++j) *reinterpret_cast<v4f*>(sums + i * PITCH + 16 * j + 4 * g) = acc[j];
    wave_lds_order();
#pragma unroll
    for (int q = 0; q < NB; ++q) {
      float d[V];
      const float* src = sums + row(q) * PITCH + lane % CPR * V;
#pragma unroll
      for (int e = 0; e < V; e += 4) {
        const v4f x = *reinterpret_cast<const v4f*>(src + e);
#pragma unroll
        for (int k = 0; k < 4; ++k) d[e + k] = x[k];
      }
      u32x4 o;
      if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int k = 0; k < 4; ++k)                // half to even, NaN kept
          o[k] = __builtin_bit_cast(uint32_t, v2bf{(__bf16)(bf16_lo(b[q][k] & keep) + d[2 * k]),
                                                   (__bf16)(bf16_hi(b[q][k] & keep) + d[2 * k + 1])});
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) o[k] = __float_as_uint(__uint_as_float(b[q][k] & keep) + d[k]);
      }
      store(o, q, mt);
    }
    wave_lds_order();
  }
};

// A block takes p.rows rows of one segment and 64 NJ columns, a wave 16 NJ of
// them, whose weights it holds as operand fragments. lora_act is split once for
// the whole block, up to 32 rows at a time. The sums of a 16 x 16 NJ block go through
// LDS, so that base and out move as whole runs of columns, and the next block's
// base is on its way during the products. Bound by base and out: 8192 x 12288
// float32 of rank 64 176 us (4.6 TB/s), 4622 x 12288 bf16 of rank 16 41.6 us (5.5
// TB/s). Rank 128 leaves room for 64 columns a wave: 8192 x 12288 bf16 131 us (3.1
// TB/s; with 128 columns 133 us, and 4622 x 6096 float32 86 against 68 us).
template <int KS, int NJ, typename T>
struct ExpandLds {
  float sums[4][16 * ExpandWave<KS, NJ, T>::PITCH];
  u32x4 la3[3][4 * KS][32];
};
template <int KS, int NJ, typename T>
CR_DEV void expand_block(const ExpandArgs& p, int bx, int by, ExpandLds<KS, NJ, T>& lds) {
  typedef ExpandWave<KS, NJ, T> Wave;
  constexpr int RO = 4 * KS;                      // rank octets
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const RowTile t = find_tile(p.seg, bx, p.rows);
  if (t.lo >= t.hi) return;
  const Wave w{p, t, (by * 4 + wave) * Wave::W, (int)threadIdx.x & 63};
  if (t.a < 0) {
    w.copy_base();
    return;
  }
  u32x4 bb[2][Wave::NB];
  w.load_base(bb[0], t.lo);
  const float cs = p.scale ? p.scale[t.a] : 1.f;
  v8bf wf[NJ][KS];
  w.load_weights(wf);
  for (int st = t.lo; st < t.hi; st += 32) {
    if (st != t.lo) __syncthreads();              // the last rows' terms have been read
    const int end = st + 32 < t.hi ? st + 32 : t.hi;
    for (int k = threadIdx.x; k < ((end - st + 15) & ~15) * RO; k += 256) {
      const int ro = k % RO, row = k / RO;
      const int64_t m = st + row < t.hi ? st + row : t.hi - 1;
      float v[8];
      load_out8(p.la + m * p.R + (8 * ro < p.R ? 8 * ro : 0), v);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = 8 * ro < p.R ? v[e] * cs : 0.f;
      u32x4 f[3];
      split8(v, f);
#pragma unroll
      for (int term = 0; term < 3; ++term) lds.la3[term][ro][row] = f[term];
    }
    __syncthreads();
    w.load_base(bb[1], st + 16);
    w.add_rows(wf, lds.la3, 0, lds.sums[wave], bb[0], st);
    if (st + 16 < end) {
      w.load_base(bb[0], st + 32);
      w.add_rows(wf, lds.la3, 16, lds.sums[wave], bb[1], st + 16);
    }
  }
}
template <int KS, int NJ, typename T>
__global__ __launch_bounds__(256) void lora_expand_kernel(ExpandArgs p) {
  __shared__ ExpandLds<KS, NJ, T> lds;
  expand_block<KS, NJ, T>(p, blockIdx.x, blockIdx.y, lds);
}

// Tall tiles read the weights less often, short ones end sooner: the tallest
// that still give every one of the 256 compute units two blocks, or one of 64 or
// 32 rows (1531 x 9216 float32 of rank 64: 22.2 us in 64 rows, 32.9 in 16; 2488 x 2280
// of rank 128: 16.0 and 19.8; 2438 x 2816 of rank 64: 13.9 us in 32 rows, 16.6 in 16).
static void expand_tiles(ExpandArgs& p, int NJ) {
  const int64_t columns = (p.C + 64 * NJ - 1) / (64 * NJ);
  p.rows = p.seg.M / 256 * columns >= 512 ? 256
           : p.seg.M / 64 * columns >= 256 ? 64
           : p.seg.M / 32 * columns >= 256 ? 32 : 16;
  p.blocks_x = (int)tile_grid(p.seg, p.rows);
}
template <int KS, int NJ, typename T>
static void launch_expand_k(ExpandArgs p, hipStream_t s) {
  expand_tiles(p, NJ);
  hipLaunchKernelGGL((lora_expand_kernel<KS, NJ, T>), dim3(p.blocks_x, (p.C + 64 * NJ - 1) / (64 * NJ)), dim3(256), 0, s, p);
}
template <typename T>
static void launch_expand_t(const ExpandArgs& p, hipStream_t s) {
  if (p.R <= 32) launch_expand_k<1, 8, T>(p, s);
  else if (p.R <= 64) launch_expand_k<2, 8, T>(p, s);
  else launch_expand_k<4, 4, T>(p, s);
}
static hipError_t launch_expand(const ExpandArgs& p, bool f32, hipStream_t s) {
  if (f32) launch_expand_t<float>(p, s);
  else launch_expand_t<uint16_t>(p, s);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Both in one launch, for few rows: a block takes 16 rows of one segment and
// 2048 columns of out and makes lora_act of the rows for itself (see few_rows).
// ---------------------------------------------------------------------------
template <int RG, typename T>
__global__ __launch_bounds__(1024) void lora_few_kernel(ShrinkArgs sp, ExpandArgs p) {
  constexpr int NW = 16, DX = RG == 1 ? 2 : 1, DW = DX;
  typedef ExpandWave<1, 8, T> Wave;
  typedef ShrinkLds<RG, 1, NW, DX, DW> Lds;
  constexpr int SUMS = NW * 16 * Wave::PITCH * 4;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[Lds::bytes > SUMS ? Lds::bytes : SUMS];
  __shared__ u32x4 la3[3][4][16];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const RowTile t = find_tile(p.seg, blockIdx.x, 16);
  if (t.lo >= t.hi) return;
  const Wave w{p, t, ((int)blockIdx.y * NW + wave) * Wave::W, (int)threadIdx.x & 63};
  if (t.a < 0) {
    if (blockIdx.y == 0)
      for (int k = threadIdx.x; k < (t.hi - t.lo) * p.R; k += 64 * NW) sp.la[(int64_t)t.lo * p.R + k] = 0.f;
    w.copy_base();
    return;
  }
  const float cs = p.scale ? p.scale[t.a] : 1.f;
  u32x4 b[Wave::NB];
  constexpr bool EARLY = RG == 1 || sizeof(T) == 2;   // rank 32 and float32: no registers for it yet
  if constexpr (EARLY) w.load_base(b, t.lo);
  v8bf wf[8][1];
  w.load_weights(wf);
  shrink_sums<RG, 1, NW, DX, DW, false>(sp, t, 0, blockIdx.x, lds);
  if constexpr (!EARLY) w.load_base(b, t.lo);
  const v4f* red = reinterpret_cast<const v4f*>(lds);
  if (threadIdx.x < 128) {                         // 16 rows x 32 ranks, four ranks a thread
    const int rg = threadIdx.x >> 6, row = threadIdx.x & 15, r = 16 * rg + 4 * (threadIdx.x >> 4 & 3);
    v4f s = {0.f, 0.f, 0.f, 0.f};
    if (r < p.R)                                   // R % 8 == 0
      for (int n = 0; n < NW; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[e] += red[n * Lds::red + (threadIdx.x & (64 * RG - 1))][e];
    if (blockIdx.y == 0 && r < p.R && t.lo + row < t.hi)
      *reinterpret_cast<v4f*>(sp.la + (int64_t)(t.lo + row) * p.R + r) = s;
    Split q[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) q[e] = split3(s[e] * cs);
    u32x2* to[3];
#pragma unroll
    for (int term = 0; term < 3; ++term) to[term] = reinterpret_cast<u32x2*>(&la3[term][r >> 3][row]) + (r >> 2 & 1);
    *to[0] = u32x2{upper_pair(q[0].hi, q[1].hi), upper_pair(q[2].hi, q[3].hi)};
    *to[1] = u32x2{upper_pair(q[0].mid, q[1].mid), upper_pair(q[2].mid, q[3].mid)};
    *to[2] = u32x2{upper_pair(q[0].lo, q[1].lo), upper_pair(q[2].lo, q[3].lo)};
  }
  __syncthreads();                                 // also: the shrink's sums are read before lds takes others
  if (w.c0 < p.C) w.add_rows(wf, la3, 0, reinterpret_cast<float*>(lds) + wave * 16 * Wave::PITCH, b, t.lo);
}

// Rows x column groups x weights of the shrink: what the blocks would read of it
// if every row were a tile, at most 64 MiB. GPU time of one launch and of two (host
// calls take 12 and 15.5 us): at the bound, 64 single rows of rank 32, 4096 -> 8192,
// 13.1 and 14.8 us, 128 of rank 16 17.3 and 18.0; below, 128 of rank 16, 4096 -> 4096,
// 10.2 and 13.2; above, 96 of rank 32, 4096 -> 8192 (96 MiB), 22.4 and 19.2, 64 of rank
// 32, 12288 -> 12288, 35.7 and 22.9 (8192 -> 8192, 128 MiB, still 16.3 and 17.4). Long
// segments read less than this counts, in fewer blocks: 256 rows of one adapter,
// rank 32, 4096 -> 4096 (128 MiB as counted), 11.9 and 10.8 us.
static bool few_rows(const LoraSegments& g, int R, int64_t N, int64_t K) {
  return R <= 32 && g.M <= 256 && g.M * ((N + 2047) / 2048) * R * K <= ((int64_t)1 << 25);
}
template <int RG, typename T>
static void launch_few_t(const ShrinkArgs& a, const ExpandArgs& b, hipStream_t s) {
  const dim3 grid(tile_grid(b.seg, 16), (b.C + 2047) / 2048);
  hipLaunchKernelGGL((lora_few_kernel<RG, T>), grid, dim3(1024), 0, s, a, b);
}
static hipError_t launch_few(const ShrinkArgs& a, const ExpandArgs& b, bool f32, hipStream_t s) {
  if (a.R <= 16 && f32) launch_few_t<1, float>(a, b, s);
  else if (a.R <= 16) launch_few_t<1, uint16_t>(a, b, s);
  else if (f32) launch_few_t<2, float>(a, b, s);
  else launch_few_t<2, uint16_t>(a, b, s);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// prepare: what the backward pass reads in another order, in one launch: up
// [A][N][R] -> [A][R][N] and down [A][R][K] -> [A][K][R] (it contracts over the
// other index of each), and lora_act in the row-octet order of "outer". A few
// megabytes: 3 to 5 us, most of it the launch and two trips to memory.
// ---------------------------------------------------------------------------
struct PrepareArgs {
  const uint16_t* up;      // null: not wanted; so down and la
  uint16_t* up_t;
  const uint16_t* down;
  uint16_t* down_t;
  const float* la;
  uint16_t* la8;
  int M, N, K, R, A;
  int up_blocks, down_blocks;
  LoraSegments seg;
};

// rows x cols (at most 64 x 128 or 128 x 64, multiples of 8) of `in` transposed into `out`
template <int THREADS>
CR_DEV void transpose_tile(const uint16_t* in, int64_t ldi, uint16_t* out, int64_t ldo, int rows, int cols,
                           uint16_t* lds) {
  const int pitch = cols + 2;                      // an odd number of words: columns spread over the banks
  const int c8 = cols / 8, r8 = rows / 8;
  for (int k = threadIdx.x; k < rows * c8; k += THREADS) {
    const int r = k / c8, c = k % c8 * 8;
    const u32x4 v = *reinterpret_cast<const u32x4*>(in + r * ldi + c);
    uint32_t* d = reinterpret_cast<uint32_t*>(lds + r * pitch + c);
#pragma unroll
    for (int e = 0; e < 4; ++e) d[e] = v[e];
  }
  __syncthreads();
  for (int k = threadIdx.x; k < cols * r8; k += THREADS) {
    const int c = k / r8, r = k % r8 * 8;
    u32x4 v;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      v[e] = (uint32_t)lds[(r + 2 * e) * pitch + c] | ((uint32_t)lds[(r + 2 * e + 1) * pitch + c] << 16);
    *reinterpret_cast<u32x4*>(out + c * ldo + r) = v;
  }
}

constexpr int kPrepareLds = 128 * 66 > 64 * 130 ? 128 * 66 : 64 * 130;   // 2-byte words
template <int THREADS>
CR_DEV void prepare_block(const PrepareArgs& p, int b, uint16_t* lds) {
  // with more adapters than segments some have no rows, and nothing reads theirs (2 rows, 25 adapters
  // of rank 128, N = 4480: 6.2 against 12.6 us)
  auto unused = [&](int a) {
    if (p.A <= p.seg.S) return false;
    for (int s = 0; s < p.seg.S; s += 64) {
      const int v = s + (threadIdx.x & 63);
      if (__ballot(v < p.seg.S && seg_adapter(p.seg, v + 1) == a)) return false;
    }
    return true;
  };
  if (b < p.up_blocks) {                           // 64 channels and all ranks of one adapter
    const int per = (p.N + 63) / 64;
    const int a = b / per, n0 = b % per * 64;
    if (unused(a)) return;
    const int n = p.N - n0 < 64 ? p.N - n0 : 64;
    transpose_tile<THREADS>(p.up + ((int64_t)a * p.N + n0) * p.R, p.R, p.up_t + (int64_t)a * p.R * p.N + n0, p.N, n, p.R, lds);
    return;
  }
  b -= p.up_blocks;
  if (b < p.down_blocks) {
    const int per = (p.K + 63) / 64;
    const int a = b / per, k0 = b % per * 64;
    if (unused(a)) return;
    const int n = p.K - k0 < 64 ? p.K - k0 : 64;
    transpose_tile<THREADS>(p.down + (int64_t)a * p.R * p.K + k0, p.K, p.down_t + ((int64_t)a * p.K + k0) * p.R, p.R, p.R, n, lds);
    return;
  }
  b -= p.down_blocks;
  const int64_t k = (int64_t)b * THREADS + threadIdx.x;   // one octet of rows and one rank
  const int64_t m8 = k / p.R;
  const int r = (int)(k % p.R);
  if (m8 * 8 >= p.M) return;
  float v[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int64_t m = m8 * 8 + e;
    const float x = p.la[(m < p.M ? m : p.M - 1) * p.R + r];
    v[e] = m < p.M ? x : 0.f;
  }
  u32x4 f[3];
  split8(v, f);
#pragma unroll
  for (int term = 0; term < 3; ++term)
    *reinterpret_cast<u32x4*>(p.la8 + rows8_index(p.M, p.R, term, (int)(m8 * 8), r)) = f[term];
}

__global__ __launch_bounds__(256) void lora_prepare_kernel(PrepareArgs p) {
  __shared__ uint16_t lds[kPrepareLds];
  prepare_block<256>(p, blockIdx.x, lds);
}

static int64_t prepare_blocks(PrepareArgs& p, int threads) {
  p.up_blocks = p.up ? p.A * ((p.N + 63) / 64) : 0;
  p.down_blocks = p.down ? p.A * ((p.K + 63) / 64) : 0;
  return p.up_blocks + p.down_blocks + (p.la ? ((int64_t)((p.M + 7) / 8) * p.R + threads - 1) / threads : 0);
}
static hipError_t launch_prepare(PrepareArgs p, hipStream_t s) {
  const unsigned blocks = (unsigned)prepare_blocks(p, 256);
  hipLaunchKernelGGL(lora_prepare_kernel, dim3(blocks), dim3(256), 0, s, p);
  return hipGetLastError();
}

// prepare and dla in one launch: dla takes up as it lies, and what is left of
// prepare nobody needs before the next launch. A whole call, this way against the
// two launches: 300 rows, 2560 x 4096, rank 8, 21.0 against 24.0 us; 1531 rows, 2560 x 2560,
// rank 32, 24.5 against 26.7; 2 rows, 12288 x 12288, rank 32, 18.8 against 21.0; 8192 rows,
// 4096 x 4096, rank 16, 102.9 against 105.0; 7031 rows, 768 x 7256, rank 16, 69 against 75.
// Ranks above 32 are gathered from lines that several blocks read: 512 rows, 4096 x
// 9216, rank 64 took 31.5 against 29.0 us, 1531 rows of it, two rounds of dla's
// blocks, 42.2 against 36.3 us. The blocks of prepare take as much LDS as those of
// dla, two at most on a compute unit, so there have to be few.
template <int NW, int DX, int DW>
__global__ __launch_bounds__(64 * NW) void lora_first_kernel(ShrinkArgs a, PrepareArgs p, int tiles, int shrink_blocks) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[ShrinkLds<1, 1, NW, DX, DW>::bytes];
  static_assert(sizeof(lds) >= kPrepareLds * 2, "");
  const int b = blockIdx.x;
  if (b < shrink_blocks) shrink_block<1, 1, NW, DX, DW, true>(a, b % tiles, b / tiles, lds);
  else prepare_block<64 * NW>(p, b - shrink_blocks, reinterpret_cast<uint16_t*>(lds));
}
template <int NW, int DX, int DW>
static bool launch_first_k(const ShrinkArgs& a, PrepareArgs p, int64_t tiles, int64_t shrink, hipStream_t s, hipError_t* e) {
  const int64_t prepare = prepare_blocks(p, 64 * NW);
  if (prepare > 512) return false;
  hipLaunchKernelGGL((lora_first_kernel<NW, DX, DW>), dim3((unsigned)(shrink + prepare)), dim3(64 * NW), 0, s, a, p,
                     (int)tiles, (int)shrink);
  *e = hipGetLastError();
  return true;
}
// false: not for these sizes, nothing launched (up: [A][N][R])
static bool launch_first(ShrinkArgs a, const uint16_t* up, PrepareArgs p, hipStream_t s, hipError_t* e) {
  a.w = up;
  p.up = nullptr;
  const int64_t tiles = tile_grid(a.seg, 16), shrink = tiles * ((a.R + 15) / 16);
  if (a.R <= 32 && shrink <= 256) return launch_first_k<16, 2, 2>(a, p, tiles, shrink, s, e);
  if (a.R <= 16) return launch_first_k<8, 3, 2>(a, p, tiles, shrink, s, e);
  return false;
}

// ---------------------------------------------------------------------------
// outer: G[a][r][c] = (c_a) sum over the rows of adapter a of u[m, r] v[m, c]
// ---------------------------------------------------------------------------
struct OuterArgs {
  const uint16_t* u8;     // u in row-octet order (see rows8_index)
  const void* v;          // bf16 or int8 [M][ldv]
  int64_t ldv;
  LoraSegments seg;
  const float* scale;     // multiplies the result, or null
  float* out;             // [A][R][C], or [A][C][R] for up; part q at out + q * part
  int64_t part;
  int P;                  // parts that the rows of an adapter are split into
  int accumulate;         // add to what out holds (P == 1)
  int R, C;
  int blocks;             // of this product in the launch; 0: not wanted
};

// Transposed fragments of an 8 x 8 block: row e of the lane's block holds
// eight columns; fragment j gets column j of the eight rows.
CR_DEV v8bf column_frag(const u32x4 (&row)[8], int j) {
  u32x4 f;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t a = row[2 * k][j >> 1], b = row[2 * k + 1][j >> 1];
    f[k] = __builtin_amdgcn_perm(b, a, (j & 1) ? 0x07060302u : 0x05040100u);
  }
  return __builtin_bit_cast(v8bf, f);
}
CR_DEV v8bf column_frag(const u32x2 (&row)[8], int j) {   // int8 codes, exact in bf16
  u32x4 f;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float a = (float)(int)(int8_t)(row[2 * k][j >> 2] >> (8 * (j & 3)));
    const float b = (float)(int)(int8_t)(row[2 * k + 1][j >> 2] >> (8 * (j & 3)));
    f[k] = upper_pair(__float_as_uint(a), __float_as_uint(b));
  }
  return __builtin_bit_cast(v8bf, f);
}

// A block takes 128 columns, 16 RG ranks and one part of an adapter's rows;
// its four waves take steps of 32 rows in turn and add their sums through LDS in
// a fixed order. Lane i of a 16-lane group holds columns 8 i .. 8 i + 7. During
// the products of a step the next one is on its way: v into registers, the
// fragments of u, which would not fit beside it, into the wave's part of LDS.
template <int RG, bool CODES, bool UP>
CR_DEV void outer_block(const OuterArgs& p, int b, v4f (*red)[RG * 8 * 64]) {
  typedef typename std::conditional<CODES, u32x2, u32x4>::type Row;
  typedef typename std::conditional<CODES, int8_t, uint16_t>::type Elem;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int i = lane & 15, g = lane >> 4;
  const int ct = (p.C + 127) / 128, nrb = (p.R + 16 * RG - 1) / (16 * RG);
  const int c = b % ct * 128 + 8 * i;
  b /= ct;
  const int r0 = b % nrb * 16 * RG;
  b /= nrb;
  const int a = b % p.seg.A, part = b / p.seg.A;
  const bool cok = c < p.C;
  const Elem* vcol = static_cast<const Elem*>(p.v) + (cok ? c : 0);
  const uint16_t* ucol[RG];
#pragma unroll
  for (int rg = 0; rg < RG; ++rg) {
    const int r = r0 + 16 * rg + i;
    ucol[rg] = p.u8 + (r < p.R ? r : p.R - 1) * 8;
  }
  const int64_t term = (int64_t)((p.seg.M + 7) / 8) * p.R * 8;
  v4f acc[RG][8];
#pragma unroll
  for (int rg = 0; rg < RG; ++rg)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[rg][j] = v4f{0.f, 0.f, 0.f, 0.f};

  const float cs = p.scale ? p.scale[a] : 1.f;
  // lane's segment of the 64 that start at s0: its first row and its rows, 0 if
  // it is not of this adapter
  int lo, len, top = 0;                           // top: where the segments before these end
  auto segments = [&](int s0) {
    const int s = s0 + lane;
    const int of = seg_adapter(p.seg, s + 1);
    const Stretch st = seg_rows(p.seg, s + 1, s0 ? top : 0);
    top = st.top;
    lo = st.lo;
    len = s < p.seg.S && of == a ? st.hi - st.lo : 0;
  };
  segments(0);
  int64_t from = 0, to = (int64_t)1 << 62;        // this part of the adapter's rows, counted through its segments
  if (p.P > 1) {
    int64_t n = len;
    for (int s0 = 64; s0 < p.seg.S; s0 += 64) {
      segments(s0);
      n += len;
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) n += __shfl_xor(n, d);
    from = n * part / p.P;
    to = n * (part + 1) / p.P;
    if (p.seg.S > 64) segments(0);
  }

  // rows [mlo, mhi) in steps of 32 that start at multiples of 32; rows of a step
  // outside them count as zeros, whatever they hold
  auto load_v = [&](Row (&row)[8], int m0) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int m = m0 + 8 * g + e;
      row[e] = *reinterpret_cast<const Row*>(vcol + (int64_t)(m < p.seg.M ? m : p.seg.M - 1) * p.ldv);
    }
  };
  u32x4* next_u = reinterpret_cast<u32x4*>(red[0]) + wave * RG * 3 * 64;     // the sums take this memory only after the last step
  auto load_u = [&](int m0) {
    const int m8 = (m0 >> 3) + g < (p.seg.M + 7) / 8 ? (m0 >> 3) + g : 0;
#pragma unroll
    for (int rg = 0; rg < RG; ++rg)
#pragma unroll
      for (int q = 0; q < 3; ++q)
        __builtin_amdgcn_global_load_lds((lora_gptr)(ucol[rg] + q * term + (int64_t)m8 * p.R * 8),
                                         (lora_lptr)(next_u + (rg * 3 + q) * 64), 16, 0, 0);
  };
  // step m0: next holds its v, next_u its u; then those of step m1
  Row next[8];
  auto step = [&](int m0, int m1, int mlo, int mhi) {
    wait_vmcnt<0>();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    u32x4 uf[RG][3];
#pragma unroll
    for (int rg = 0; rg < RG; ++rg)
#pragma unroll
      for (int q = 0; q < 3; ++q) uf[rg][q] = next_u[(rg * 3 + q) * 64 + lane];
    __builtin_amdgcn_s_waitcnt(0xC07F);            // lgkmcnt(0): read before the next step's arrive
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    Row row[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) row[e] = next[e];
    load_u(m1);
    load_v(next, m1);
    if (m0 < mlo || m0 + 32 > mhi) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int m = m0 + 8 * g + 2 * k;
        const bool ok0 = m >= mlo && m < mhi, ok1 = m + 1 >= mlo && m + 1 < mhi;
        const uint32_t keep = (ok0 ? 0xFFFFu : 0u) | (ok1 ? 0xFFFF0000u : 0u);
#pragma unroll
        for (int rg = 0; rg < RG; ++rg)
#pragma unroll
          for (int q = 0; q < 3; ++q) uf[rg][q][k] &= keep;
        const Row z{};
        row[2 * k] = ok0 ? row[2 * k] : z;
        row[2 * k + 1] = ok1 ? row[2 * k + 1] : z;
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const v8bf vf = column_frag(row, j);
#pragma unroll
      for (int q = 2; q >= 0; --q)                 // the small terms first
#pragma unroll
        for (int rg = 0; rg < RG; ++rg) acc[rg][j] = mfma16(__builtin_bit_cast(v8bf, uf[rg][q]), vf, acc[rg][j]);
    }
  };
  // The wave's steps: every fourth of the adapter's, over all runs of rows. A run
  // is one segment of the adapter or several that follow one another, as single
  // rows of one adapter do (95 segments, all but one a row, in 4771 rows of rank 24
  // and one adapter, N = 608: 22 us for the launch against 50 a segment at a time).
  int s0 = 0, turn = 0;                            // turn: steps so far
  int64_t before = 0;                              // rows of the adapter so far
  uint64_t left = __ballot(len > 0);
  int mlo = 0, mhi = 0, m00 = 0, count = 0, k = 0;
  auto advance = [&]() {                           // false behind the last step
    k += 4;
    while (k >= count) {
      while (left == 0) {
        s0 += 64;
        if (s0 >= p.seg.S) return false;
        segments(s0);
        left = __ballot(len > 0);
      }
      int src = __builtin_ctzll(left);
      const int slo = __builtin_amdgcn_readlane(lo, src);
      int slen = __builtin_amdgcn_readlane(len, src);
      for (left &= left - 1; left; left &= left - 1) {
        src = __builtin_ctzll(left);
        if (__builtin_amdgcn_readlane(lo, src) != slo + slen) break;
        slen += __builtin_amdgcn_readlane(len, src);
      }
      const int64_t x0 = from > before ? from - before : 0;
      const int64_t x1 = to - before < slen ? to - before : slen;
      before += slen;
      count = k = 0;
      if (x1 <= x0) continue;
      mlo = slo + (int)x0;
      mhi = slo + (int)x1;
      m00 = mlo & ~31;
      count = (mhi - m00 + 31) >> 5;
      k = (wave - turn) & 3;
      turn += count;
    }
    return true;
  };
  bool more = advance();
  if (more) {
    load_u(m00 + 32 * k);
    load_v(next, m00 + 32 * k);
  }
  // one copy of the step's code: a block runs it a few times only, and fetching it counts
#pragma unroll 1
  while (more) {
    const int m0 = m00 + 32 * k, from_row = mlo, to_row = mhi;
    more = advance();
    step(m0, more ? m00 + 32 * k : m0, from_row, to_row);   // behind the last: itself, for nothing
  }
  float* out = p.out + part * p.part + (int64_t)a * p.R * p.C;
  const int cb = c - 8 * i;
  if (turn == 0) {                                 // no rows: zeros, or what was there
    if (p.accumulate) return;
    const int line = UP ? 4 * RG : 32;
#pragma unroll 1
    for (int k = threadIdx.x; k < 16 * RG * 32; k += 256) {
      const int cc = cb + (UP ? k / line : 4 * (k % line)), r = r0 + (UP ? 4 * (k % line) : k / line);
      if (cc < p.C && r < p.R)
        *reinterpret_cast<v4f*>(out + (UP ? (int64_t)cc * p.R + r : (int64_t)r * p.C + cc)) = v4f{0.f, 0.f, 0.f, 0.f};
    }
    return;
  }
  wait_vmcnt<0>();
  __syncthreads();                                 // every wave's u has arrived and been read
#pragma unroll 1
  for (int n = turn > 2 ? 2 : turn > 1 ? 1 : 0; n >= 1; n >>= 1) {   // waves that had no step hold zeros
    if (wave >= n && wave < 2 * n) {
#pragma unroll
      for (int rg = 0; rg < RG; ++rg)
#pragma unroll
        for (int j = 0; j < 8; ++j) red[wave - n][(rg * 8 + j) * 64 + lane] = acc[rg][j];
    }
    __syncthreads();
    if (wave < n) {
#pragma unroll
      for (int rg = 0; rg < RG; ++rg)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const v4f o = red[wave][(rg * 8 + j) * 64 + lane];
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[rg][j][e] += o[e];
        }
    }
    __syncthreads();
  }
  // The sums go out through LDS, so that neighbouring lanes write neighbouring
  // values (d_up of rank 64 and 4096 channels: 11 us less than lane by lane).
  constexpr int PITCH = UP ? 4 * RG + 1 : 33;      // 16-byte words of a column (up) or of a rank
  constexpr int LINE = UP ? 4 * RG : 32;
  v4f* tile = red[0];
  if (wave == 0) {
#pragma unroll
    for (int rg = 0; rg < RG; ++rg) {
      if constexpr (UP) {
#pragma unroll
        for (int j = 0; j < 8; ++j) tile[(8 * i + j) * PITCH + 4 * rg + g] = acc[rg][j];
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int j = 0; j < 8; j += 4)
            tile[(16 * rg + 4 * g + e) * PITCH + 2 * i + j / 4] =
                v4f{acc[rg][j][e], acc[rg][j + 1][e], acc[rg][j + 2][e], acc[rg][j + 3][e]};
      }
    }
  }
  __syncthreads();
#pragma unroll 1
  for (int k = threadIdx.x; k < 16 * RG * 32; k += 256) {
    const int row = k / LINE, at = k % LINE;
    const int cc = cb + (UP ? row : 4 * at), r = r0 + (UP ? 4 * at : row);
    if (cc >= p.C || r >= p.R) continue;           // C and R are multiples of 8: four values in or out together
    v4f* o = reinterpret_cast<v4f*>(out + (UP ? (int64_t)cc * p.R + r : (int64_t)r * p.C + cc));
    v4f w = {0.f, 0.f, 0.f, 0.f};
    if (p.accumulate) w = *o;
    const v4f x = tile[row * PITCH + at];
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] += x[e] * cs;
    *o = w;
  }
}

// Both weight gradients and dx in one launch: they need the same operands only,
// and the products of the one keep the matrix cores busy while the other waits
// for memory. The first up.blocks blocks make d_up, the next d_down, the rest dx.
// 8192 rows, 4096 x 4096, rank 16: 75 us (402 MB of x, dy, dx_base and dx, 5.4 TB/s);
// 12288 x 4096, rank 64, from codes: 154 us, x and dy read once per 32 ranks.
template <int RG, int KS, int NJ, bool CODES, typename T>
__global__ __launch_bounds__(256) void lora_gradients_kernel(OuterArgs up, OuterArgs down, ExpandArgs dx) {
  constexpr size_t A = sizeof(v4f) * 2 * RG * 8 * 64, B = sizeof(ExpandLds<KS, NJ, T>);
  __shared__ __attribute__((aligned(1024))) uint8_t lds[A > B ? A : B];
  auto red = reinterpret_cast<v4f(*)[RG * 8 * 64]>(lds);
  int b = blockIdx.x;
  if (b < up.blocks) return outer_block<RG, false, true>(up, b, red);
  b -= up.blocks;
  if (b < down.blocks) return outer_block<RG, CODES, false>(down, b, red);
  b -= down.blocks;
  expand_block<KS, NJ, T>(dx, b % dx.blocks_x, b / dx.blocks_x, *reinterpret_cast<ExpandLds<KS, NJ, T>*>(lds));
}

static int outer_blocks(const OuterArgs& p) {
  const int rb = p.R <= 16 ? 16 : 32;
  return (p.C + 127) / 128 * ((p.R + rb - 1) / rb) * p.seg.A * p.P;
}
// Ranks above 32 are made 32 at a time, each reading x or dy again (the second
// time from the caches): the sums of 64 take all registers of half a compute unit,
// too few blocks for dx beside them (8192 rows of rank 64 from codes: 160 us
// together against 91 + 81 us of 64 ranks at a time and dx on its own).
template <int RG, int KS, int NJ, bool CODES, typename T>
static void launch_gradients_k(const OuterArgs& up, const OuterArgs& down, ExpandArgs dx, bool want_dx, hipStream_t s) {
  unsigned blocks = up.blocks + down.blocks;
  if (want_dx) {
    expand_tiles(dx, NJ);
    blocks += (unsigned)dx.blocks_x * ((dx.C + 64 * NJ - 1) / (64 * NJ));
  }
  hipLaunchKernelGGL((lora_gradients_kernel<RG, KS, NJ, CODES, T>), dim3(blocks), dim3(256), 0, s, up, down, dx);
}
template <bool CODES, typename T>
static hipError_t launch_gradients(const OuterArgs& up, const OuterArgs& down, const ExpandArgs& dx, bool want_dx,
                                   hipStream_t s) {
  if (dx.R <= 16) launch_gradients_k<1, 1, 8, CODES, T>(up, down, dx, want_dx, s);
  else if (dx.R <= 32) launch_gradients_k<2, 1, 8, CODES, T>(up, down, dx, want_dx, s);
  else if (dx.R <= 64) launch_gradients_k<2, 2, 8, CODES, T>(up, down, dx, want_dx, s);
  else launch_gradients_k<2, 4, 4, CODES, T>(up, down, dx, want_dx, s);
  return hipGetLastError();
}

// Parts an adapter's rows are split into: as many as keep both gradients' blocks
// in one round on the GPU's 256 compute units, at least 128 rows each were the
// rows even. A block's start and end cost as much as four of its steps (d_up of
// rank 64 and 4096 channels: 28 us in 8 parts, 37 in 16), and the blocks of dx share
// the launch: 8192 rows of rank 16 with 512 blocks 75 us, with 1024 79 us; 1531 rows of
// rank 32 with 384 15.4 us, with 768 16.2 us; 8192 rows of rank 64 from codes with 384 160
// us, with 768 169 us.
static int outer_parts(int64_t M, int64_t N, int64_t K, int R, int A) {
  const int64_t blocks = ((N + 127) / 128 + (K + 127) / 128) * ((R + 31) / 32) * A;
  int64_t P = (R <= 16 ? 512 : 384) / blocks;
  const int64_t most = (M + 127) / 128;
  if (P > most) P = most;
  return P < 1 ? 1 : (int)P;
}

// ---------------------------------------------------------------------------
// join: out = (out +) sum of the P parts, in order. 4 to 5 us: the launch, and the
// parts, which are still in the caches.
// ---------------------------------------------------------------------------
struct JoinArgs {
  const float* part;
  int P;
  int64_t n;              // values of one part
  float* out;
  int accumulate;
  int blocks;             // of this join in the launch; 0: not wanted
};

CR_DEV void join_block(const JoinArgs& p, int b) {
  const int64_t k = ((int64_t)b * 256 + threadIdx.x) * 4;
  if (k >= p.n) return;
  v4f s = *reinterpret_cast<const v4f*>(p.part + k);
  for (int q = 1; q < p.P; q += 8) {               // eight parts on their way at once (38 parts: 4.4 against 11.6 us)
    v4f w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      w[i] = *reinterpret_cast<const v4f*>(p.part + (q + i < p.P ? q + i : q) * p.n + k);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (q + i < p.P)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[e] += w[i][e];
  }
  v4f* o = reinterpret_cast<v4f*>(p.out + k);
  if (p.accumulate) {
    const v4f b = *o;
#pragma unroll
    for (int e = 0; e < 4; ++e) s[e] += b[e];
  }
  *o = s;
}

// The same with every rotation group of NR columns rotated back: sixteen
// lanes hold one row's 256 (NR = 1024: 4 x 256) columns, element 16 gL + e of
// each chunk in register e of its lane.
template <int NR>
CR_DEV void join_rotate_block(const JoinArgs& p, int b) {
  constexpr int GPS = NR == 1024 ? 4 : 1;
  const LaneRot lr = lane_rot<NR>(threadIdx.x & 15);
  const int64_t items = p.n / (256 * GPS);           // rows are whole groups: chunks follow one another
  const int64_t item = (int64_t)b * 16 + (threadIdx.x >> 4);
  const bool ok = item < items;
  const int64_t k0 = (ok ? item : items - 1) * (256 * GPS) + 16 * lr.gL;
  float v[GPS][16];
#pragma unroll
  for (int g = 0; g < GPS; ++g) {
    const float* src = p.part + k0 + 256 * g;
#pragma unroll
    for (int e = 0; e < 16; e += 4) {
      const v4f s = *reinterpret_cast<const v4f*>(src + e);
#pragma unroll
      for (int x = 0; x < 4; ++x) v[g][e + x] = s[x];
    }
    for (int q = 1; q < p.P; q += 4) {
      v4f w[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          w[i][e] = *reinterpret_cast<const v4f*>(src + (q + i < p.P ? q + i : q) * p.n + 4 * e);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (q + i < p.P)
#pragma unroll
          for (int e = 0; e < 16; ++e) v[g][e] += w[i][e >> 2][e & 3];
    }
    const bool cneg = NR == 1024 && chunk_neg(g);
#pragma unroll
    for (int e = 0; e < 16; ++e)
      if (dreg_neg(e) != cneg) v[g][e] = -v[g][e];
    butterflies<NR>(v[g], lr);
  }
  if constexpr (NR == 1024) bfly_chunks<GPS>(v);
  if (!ok) return;
#pragma unroll
  for (int g = 0; g < GPS; ++g) {
    float* dst = p.out + k0 + 256 * g;
#pragma unroll
    for (int e = 0; e < 16; e += 4) {
      v4f s;
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const bool neg = (lr.tau < 0.f) != (dreg_neg(e + x) != (NR == 1024 && chunk_neg(g)));
        s[x] = (neg ? -v[g][e + x] : v[g][e + x]) * RotSize<NR>::inv_sqrt;
      }
      v4f* o = reinterpret_cast<v4f*>(dst + e);
      if (p.accumulate) {
        const v4f b = *o;
#pragma unroll
        for (int x = 0; x < 4; ++x) s[x] += b[x];
      }
      *o = s;
    }
  }
}

// both gradients in one launch, d_up's blocks first; NR: the rotation of
// d_down's columns that is undone (0: none)
template <int NR>
__global__ __launch_bounds__(256) void lora_join_kernel(JoinArgs up, JoinArgs down) {
  const int b = blockIdx.x;
  if (b < up.blocks) join_block(up, b);
  else if constexpr (NR == 0) join_block(down, b - up.blocks);
  else join_rotate_block<NR>(down, b - up.blocks);
}

static int join_blocks(const JoinArgs& p, int rot) {
  return rot == 0 ? (int)((p.n / 4 + 255) / 256) : (int)((p.n / (rot == 1024 ? 1024 : 256) + 15) / 16);
}
static hipError_t launch_join(const JoinArgs& up, const JoinArgs& down, int rot, hipStream_t s) {
  const dim3 grid(up.blocks + down.blocks);
  switch (rot) {
    case 0: hipLaunchKernelGGL((lora_join_kernel<0>), grid, dim3(256), 0, s, up, down); break;
    case 16: hipLaunchKernelGGL((lora_join_kernel<16>), grid, dim3(256), 0, s, up, down); break;
    case 64: hipLaunchKernelGGL((lora_join_kernel<64>), grid, dim3(256), 0, s, up, down); break;
    case 1024: hipLaunchKernelGGL((lora_join_kernel<1024>), grid, dim3(256), 0, s, up, down); break;
    default: hipLaunchKernelGGL((lora_join_kernel<256>), grid, dim3(256), 0, s, up, down); break;
  }
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// entry points
// ---------------------------------------------------------------------------
hipError_t launch_lora_forward(const LoraForward& p, hipStream_t s, int* kernels) {
  const ShrinkArgs a{p.x, p.ldx, p.down, p.seg, nullptr, p.la, nullptr, nullptr, 0, p.R, (int)p.K};
  const ExpandArgs b{p.la, p.up, p.seg, p.scale, p.base, p.ldb, p.out, p.ldo, p.R, (int)p.N, 0, 0};
  const bool few = few_rows(p.seg, p.R, p.N, p.K);
  *kernels = few ? 1 : 2;
  if (few) return launch_few(a, b, p.out_f32 != 0, s);
  const hipError_t e = launch_shrink(a, s);
  if (e != hipSuccess) return e;
  return launch_expand(b, p.out_f32 != 0, s);
}

// workspace: dla [M][R] float32, dla and lora_act in row-octet order, up
// [A][R][N] and down [A][K][R] transposed (bf16), the parts of the two gradients
static size_t pad16(size_t n) { return (n + 15) & ~(size_t)15; }
size_t lora_backward_ws_bytes(int64_t M, int64_t N, int64_t K, int R, int A) {
  return pad16((size_t)M * R * 4) + 2 * rows8_bytes(M, R) + (size_t)A * R * (N + K) * 2 +
         (size_t)outer_parts(M, N, K, R, A) * A * R * (N + K) * 4;
}

hipError_t launch_lora_backward(const LoraBackward& p, hipStream_t s, int* kernels) {
  const int A = p.seg.A, M = p.seg.M, N = (int)p.N, K = (int)p.K;
  const int64_t wn = (int64_t)A * p.R * N, wk = (int64_t)A * p.R * K;
  float* dla = reinterpret_cast<float*>(p.ws);
  uint16_t* dla8 = reinterpret_cast<uint16_t*>(p.ws + pad16((size_t)M * p.R * 4));
  uint16_t* la8 = dla8 + rows8_bytes(M, p.R) / 2;
  uint16_t* up_t = la8 + rows8_bytes(M, p.R) / 2;
  uint16_t* down_t = up_t + wn;
  float* part_up = reinterpret_cast<float*>(down_t + wk);
  const int P = outer_parts(M, N, K, p.R, A);
  float* part_down = part_up + P * wn;
  const bool codes = p.x_scales != nullptr, dla_wanted = p.dx || p.d_down;
  hipError_t e = hipSuccess;
  *kernels = 1;
  const PrepareArgs pre{dla_wanted ? p.up : nullptr, up_t, p.dx ? p.down : nullptr, down_t,
                        p.d_up ? p.la : nullptr, la8, M, N, K, p.R, A, 0, 0, p.seg};
  const ShrinkArgs a{p.dy, p.lddy, up_t, p.seg, p.scale, dla, p.d_down ? dla8 : nullptr,
                     codes ? p.x_scales : nullptr, p.x_row_scales, p.R, N};
  if (dla_wanted && launch_first(a, p.up, pre, s, &e)) {
    if (e != hipSuccess) return e;
  } else {
    if ((e = launch_prepare(pre, s)) != hipSuccess) return e;
    if (dla_wanted) {
      ++*kernels;
      if ((e = launch_shrink(a, s)) != hipSuccess) return e;
    }
  }
  const ExpandArgs ex{dla, down_t, p.seg, nullptr, p.dx_base, p.ldb, p.dx, p.lddx, p.R, K, 0, 0};
  if (!p.d_up && !p.d_down) {
    ++*kernels;
    return launch_expand(ex, p.dx_f32 != 0, s);
  }
  const int rot = codes && p.d_down ? p.rot_group : 0;
  const bool join_up = p.d_up && P > 1, join_down = p.d_down && (P > 1 || rot);
  OuterArgs up{la8, p.dy, p.lddy, p.seg, p.scale, join_up ? part_up : p.d_up, wn, P, !join_up && p.accumulate, p.R, N, 0};
  OuterArgs down{dla8, p.x, p.ldx, p.seg, nullptr, join_down ? part_down : p.d_down, wk, P, !join_down && p.accumulate,
                 p.R, K, 0};
  if (p.d_up) up.blocks = outer_blocks(up);
  if (p.d_down) down.blocks = outer_blocks(down);
  const bool want_dx = p.dx != nullptr, f32 = p.dx_f32 != 0;
  ++*kernels;
  if (codes && f32) e = launch_gradients<true, float>(up, down, ex, want_dx, s);
  else if (codes) e = launch_gradients<true, uint16_t>(up, down, ex, want_dx, s);
  else if (f32) e = launch_gradients<false, float>(up, down, ex, want_dx, s);
  else e = launch_gradients<false, uint16_t>(up, down, ex, want_dx, s);
  if (e != hipSuccess) return e;
  if (join_up || join_down) {
    JoinArgs ju{part_up, P, wn, p.d_up, p.accumulate, 0}, jd{part_down, P, wk, p.d_down, p.accumulate, 0};
    if (join_up) ju.blocks = join_blocks(ju, 0);
    if (join_down) jd.blocks = join_blocks(jd, rot);
    ++*kernels;
    e = launch_join(ju, jd, rot, s);
  }
  return e;
}

}  // namespace cr
