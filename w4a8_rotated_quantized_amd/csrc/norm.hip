// Layer norm of rows with one weight and bias, or one pair per sequence of
// the batch (adaLN modulation), and its gradients (gfx950).
//
//   mean = sum x / C,  rstd = 1 / sqrt(sum (x - mean)^2 / C + eps)
//   xh = (x - mean) rstd,  y = xh w + b
//   g = dy w,  dx = base + rstd (g - sum g / C - xh sum (g xh) / C)
//   dw = sum over the sequence's rows of dy xh,  db = the same of dy
// Both sums of a row run over the values held in registers: x is read once,
// and the variance is that of the differences, which x^2 - mean^2 would lose.
//
// A row is shared by W waves (1 to 16), each lane holding eight consecutive
// columns at a time, V times. The memory rate bounds both directions, so a wave
// keeps a whole row's loads in flight at once.
#include <algorithm>

#include "block.h"
#include "common.h"

namespace cr {

typedef __bf16 v2bf __attribute__((ext_vector_type(2)));

CR_DEV uint32_t pair_of(float lo, float hi) { return __builtin_bit_cast(uint32_t, v2bf{(__bf16)lo, (__bf16)hi}); }

// eight consecutive values as they lie in memory
template <bool F32>
struct Eight {
  u32x4 w[F32 ? 2 : 1];
  CR_DEV void load(const void* base, int64_t at) {
    if constexpr (F32) {
      const u32x4* s = reinterpret_cast<const u32x4*>(static_cast<const float*>(base) + at);
      w[0] = s[0];
      w[1] = s[1];
    } else {
      w[0] = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(base) + at);
    }
  }
  CR_DEV float get(int e) const {
    if constexpr (F32) return __uint_as_float(w[e >> 2][e & 3]);
    else return (e & 1) ? bf16_hi(w[0][e >> 1]) : bf16_lo(w[0][e >> 1]);
  }
};

template <bool F32>
CR_DEV void store8(void* base, int64_t at, const float (&v)[8]) {
  if constexpr (F32) {
    v4f* d = reinterpret_cast<v4f*>(static_cast<float*>(base) + at);
    d[0] = v4f{v[0], v[1], v[2], v[3]};
    d[1] = v4f{v[4], v[5], v[6], v[7]};
  } else {
    *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(base) + at) =
        u32x4{pair_of(v[0], v[1]), pair_of(v[2], v[3]), pair_of(v[4], v[5]), pair_of(v[6], v[7])};
  }
}

// weights and biases are bf16 or float32 by a run-time flag: they come from L2
CR_DEV void load_affine(const void* base, int f32, int64_t at, float (&v)[8]) {
  if (f32) {
    const v4f* s = reinterpret_cast<const v4f*>(static_cast<const float*>(base) + at);
    const v4f a = s[0], b = s[1];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[e] = a[e];
      v[4 + e] = b[e];
    }
  } else {
    const u32x4 w = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(base) + at);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = (e & 1) ? bf16_hi(w[e >> 1]) : bf16_lo(w[e >> 1]);
  }
}

CR_DEV float wave_sum(float v) {
  v += dpp_f<DPP_QUAD_1032>(v);
  v += dpp_f<DPP_QUAD_2301>(v);
  v += dpp_f<DPP_HALF_MIRROR>(v);
  v += dpp_f<DPP_ROW_ROR8>(v);
  v += __shfl_xor(v, 16);
  v += __shfl_xor(v, 32);
  return v;
}

// the sums over the W waves of a row, in a fixed order; `slot` changes from call to call, so one barrier is enough
template <int W>
CR_DEV float row_sum(float v, float* lds, int wave, int slot) {
  v = wave_sum(v);
  if constexpr (W > 1) {
    float* at = lds + slot * W;
    if ((threadIdx.x & 63) == 0) at[wave] = v;
    __syncthreads();
    v = at[0];
#pragma unroll
    for (int w = 1; w < W; ++w) v += at[w];
  }
  return v;
}
template <int W>
CR_DEV void row_sums(float& a, float& b, float2* lds, int wave, int slot) {
  a = wave_sum(a);
  b = wave_sum(b);
  if constexpr (W > 1) {
    float2* at = lds + slot * W;
    if ((threadIdx.x & 63) == 0) at[wave] = float2{a, b};
    __syncthreads();
    a = at[0].x;
    b = at[0].y;
#pragma unroll
    for (int w = 1; w < W; ++w) {
      a += at[w].x;
      b += at[w].y;
    }
  }
}

CR_DEV int wave_max_int(int v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_xor(v, d);
    v = v > o ? v : o;
  }
  return v;
}

// The sequence of a row among S offsets off[0..S], by one wave: the first s, `from`
// on, whose end off[s + 1] lies behind the row, 256 offsets at a time; S: none. An offset
// below an earlier one so counts as that earlier one, and off[s + 1] > row for the s
// found. BEGIN, from the first sequence on: *begin is the sequence's first row, the largest of off[0..s] and 0.
template <bool BEGIN>
CR_DEV int sequence_of(const int32_t* off, int S, int64_t row, int l, int from = 0, int64_t* begin = nullptr) {
  int most = 0;                                        // of the ends before, this lane's
  for (int at = from; at < S; at += 256) {
    int end[4], s = S;
    uint64_t behind[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int i = at + k * 64 + l;
      end[k] = i < S ? off[1 + i] : 0;
      behind[k] = __ballot(i < S && end[k] > row);
    }
#pragma unroll
    for (int k = 3; k >= 0; --k)
      if (behind[k]) s = at + k * 64 + __builtin_ctzll(behind[k]);
    if constexpr (BEGIN) {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (at + k * 64 + l < s && end[k] > most) most = end[k];
    }
    if (s < S) {
      if constexpr (BEGIN) {
        most = wave_max_int(most);
        *begin = most > off[0] ? most : off[0];
      }
      return s;
    }
  }
  return S;
}

// Forward. W == 1: four rows a block, a wave each; otherwise a row a block.
template <int W, int V, bool XF, bool YF>
__global__ __launch_bounds__(W == 1 ? 256 : W * 64) void norm_forward_kernel(NormForward p) {
  __shared__ float lds[2 * W];
  const int l = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t block = ((int64_t)blockIdx.y << GRID_LG) + blockIdx.x, row = W == 1 ? block * 4 + wave : block;
  if (row >= p.rows) return;
  const int lane = W == 1 ? l : threadIdx.x;
  // the row's loads before its sequence is known (8192 x 4096 in 6 sequences: 30.3 -> 28.7 us)
  Eight<XF> x[V];
  const int64_t at = row * p.ldx;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = (v * W * 64 + lane) * 8;
    if (c < p.C) x[v].load(p.x, at + c);
  }
  int s = 0;
  if (p.off) {
    s = sequence_of<false>(p.off, p.S, row, l);
    if (s >= p.S || row < p.off[0]) return;           // in no sequence: left as it is
  }
  float sum = 0.f;
#pragma unroll
  for (int v = 0; v < V; ++v)
    if ((v * W * 64 + lane) * 8 < p.C)
#pragma unroll
      for (int e = 0; e < 8; ++e) sum += x[v].get(e);
  const float mean = row_sum<W>(sum, lds, wave, 0) * p.inv_c;
  float sq = 0.f;
#pragma unroll
  for (int v = 0; v < V; ++v)
    if ((v * W * 64 + lane) * 8 < p.C)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float d = x[v].get(e) - mean;
        sq = __builtin_fmaf(d, d, sq);
      }
  const float rstd = 1.f / sqrtf(row_sum<W>(sq, lds, wave, 1) * p.inv_c + p.eps);
  if (lane == 0) {
    p.mean[row] = mean;
    p.rstd[row] = rstd;
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = (v * W * 64 + lane) * 8;
    if (c >= p.C) continue;
    float y[8], a[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = (x[v].get(e) - mean) * rstd;
    if (p.w) {
      load_affine(p.w, p.w_f32, s * p.ldw + c, a);
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] *= a[e] + p.plus;
    }
    if (p.b) {
      load_affine(p.b, p.w_f32, s * p.ldbias + c, a);
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] += a[e];
    }
    store8<YF>(p.y, row * p.ldy + c, y);
  }
}

CR_DEV void give(float* to, int64_t at, float (&v)[8], int accumulate) {
  if (accumulate) {
    float old[8];
    load_affine(to, 1, at, old);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] += old[e];
  }
  store8<true>(to, at, v);
}

// Backward. The rows are cut into p.parts stretches of p.part_rows, a block each. It
// walks its rows with the sums for dw and db of its columns in registers, the
// next row's loads under way, and writes the sums out where a sequence ends. Those of a
// sequence that lies in one part are the result. Else part q's share of sequence s goes
// to slot q + s of the workspace, which no other pair has, as both only grow along the
// rows, and the last launch adds the sequence's slots in order. For that launch, block 0
// writes down where the sequences begin.
// G groups of W waves take the block's rows in turn, each with sums of its own, added
// through LDS before they are written: rows on their way at once, without a slot for each.
template <int W, int V, int G, bool XF, bool DF>
__global__ __launch_bounds__(G * W * 64) void norm_backward_kernel(NormBackward p) {
  __shared__ float2 lds[G][2 * W];
  __shared__ float4 join[G > 1 ? (G - 1) * W * 64 * 4 : 1];
  const int l = threadIdx.x & 63, wave = threadIdx.x >> 6, group = wave / W;
  const int lane = threadIdx.x - group * W * 64;
  int64_t row = (int64_t)blockIdx.x * p.part_rows;
  const int64_t end = imin64(row + p.part_rows, p.rows);
  if (p.begins && blockIdx.x == 0 && wave == 0) {
    // the largest offset up to each, 256 at a time
    int before = 0;
    for (int at = 0; at < p.S; at += 256) {
      int v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = at + l * 4 + k < p.S ? p.off[at + l * 4 + k] : 0;
#pragma unroll
      for (int k = 1; k < 4; ++k) v[k] = max(v[k], v[k - 1]);
      int upto = v[3];
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(upto, d);
        if (l >= d) upto = max(upto, o);
      }
      const int ahead = __shfl_up(upto, 1);
      before = l ? max(before, ahead) : before;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (at + l * 4 + k < p.S) p.begins[at + l * 4 + k] = max(v[k], before);
      before = max(__shfl(before, 0), __shfl(upto, 63));
    }
  }
  const int64_t part = row;
  if (p.off && row < p.off[0]) row = p.off[0];         // rows in no sequence: nothing is read or written
  Eight<XF> x[V];
  Eight<DF> dy[V];
  float mean = 0.f, rstd = 0.f;
  auto load = [&](int64_t r) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = (v * W * 64 + lane) * 8;
      if (c < p.C) {
        x[v].load(p.x, r * p.ldx + c);
        dy[v].load(p.dy, r * p.lddy + c);
      }
    }
    mean = p.mean[r];
    rstd = p.rstd[r];
  };
  int slot = 0, s = 0;
  int64_t begin = 0;
  if (p.off && row < end) s = sequence_of<true>(p.off, p.S, row, l, 0, &begin);
  while (row < end && s < p.S) {
    const int64_t last = p.off ? imin64(p.rows, p.off[s + 1]) : p.rows, stop = imin64(end, last);
    const bool whole = begin >= part && last <= end;
    float w[V][8], dw[V][8], db[V][8];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = (v * W * 64 + lane) * 8;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        dw[v][e] = db[v][e] = 0.f;
        w[v][e] = 1.f;
      }
      if (p.w && c < p.C) {
        load_affine(p.w, p.w_f32, s * p.ldw + c, w[v]);
#pragma unroll
        for (int e = 0; e < 8; ++e) w[v][e] += p.plus;
      }
    }
    int64_t r = row + group;
    if (r < stop) load(r);
    // the groups meet at the block's barriers: each takes the same number of rounds
    for (int64_t round = row; round < stop; round += G, r += G) {
      const bool some = G == 1 || r < stop;
      // this row's values in float32, then the next row's loads
      const float rs = rstd;
      float a = 0.f, b = 0.f;
      float xh[V][8], d[V][8];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const bool in = some && (v * W * 64 + lane) * 8 < p.C;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          d[v][e] = in ? dy[v].get(e) : 0.f;
          xh[v][e] = in ? (x[v].get(e) - mean) * rs : 0.f;
        }
      }
      if (r + G < stop) load(r + G);
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float g = d[v][e] * w[v][e];
          a += g;
          b = __builtin_fmaf(g, xh[v][e], b);
          dw[v][e] = __builtin_fmaf(d[v][e], xh[v][e], dw[v][e]);
          db[v][e] += d[v][e];
        }
      if (!p.dx) continue;
      row_sums<W>(a, b, lds[group], wave - group * W, slot);
      slot ^= 1;
      a *= p.inv_c;
      b *= p.inv_c;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int c = (v * W * 64 + lane) * 8;
        if (c >= p.C || !some) continue;
        float o[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = rs * (d[v][e] * w[v][e] - a - xh[v][e] * b);
        if (p.base) {
          float t[8];
          load_affine(p.base, p.dx_f32, r * p.ldb + c, t);
#pragma unroll
          for (int e = 0; e < 8; ++e) o[e] += t[e];
        }
        if (p.dx_f32) store8<true>(p.dx, r * p.lddx + c, o);
        else store8<false>(p.dx, r * p.lddx + c, o);
      }
    }
    if (p.parts_w) {
      const int64_t at = ((int64_t)blockIdx.x + s) * p.C;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int c = (v * W * 64 + lane) * 8;
        if constexpr (G > 1) {
          __syncthreads();
          if (group) {
            float4* to = join + (group - 1) * (W * 64 * 4) + lane;
            to[0] = float4{dw[v][0], dw[v][1], dw[v][2], dw[v][3]};
            to[W * 64] = float4{dw[v][4], dw[v][5], dw[v][6], dw[v][7]};
            to[2 * W * 64] = float4{db[v][0], db[v][1], db[v][2], db[v][3]};
            to[3 * W * 64] = float4{db[v][4], db[v][5], db[v][6], db[v][7]};
          }
          __syncthreads();
          if (group == 0) {
#pragma unroll
            for (int o = 0; o < G - 1; ++o)
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                const float4 t = join[(o * 4 + q) * (W * 64) + lane];
                float* to = (q < 2 ? dw[v] : db[v]) + (q & 1) * 4;
                to[0] += t.x;
                to[1] += t.y;
                to[2] += t.z;
                to[3] += t.w;
              }
          }
        }
        if (c >= p.C || group) continue;
        if (!whole) {
          store8<true>(p.parts_w, at + c, dw[v]);
          store8<true>(p.parts_b, at + c, db[v]);
          continue;
        }
        const int64_t to = (int64_t)s * p.C + c;
        if (p.dw) give(p.dw, to, dw[v], p.accumulate);
        if (p.db) give(p.db, to, db[v], p.accumulate);
      }
    }
    // one that begins in this part begins at the row behind the last: no offset between is behind that row
    row = begin = stop;
    if (row < end) s = sequence_of<false>(p.off, p.S, row, l, s + 1);
  }
}

// dw and db of the sequences that have no single part: the slots of the parts that hold a sequence's rows, in
// order, and zeros for those without rows. A wave reads 64 columns of a slot; SHARES waves share the slots, each
// with several on their way, the block's other waves take other columns.
template <int NW, int SHARES>
__global__ __launch_bounds__(64 * NW) void norm_join_kernel(NormBackward p) {
  __shared__ float lds[NW][64];
  const int l = threadIdx.x & 63, wave = threadIdx.x >> 6, share = wave % SHARES;
  const int64_t c = ((int64_t)blockIdx.x * (NW / SHARES) + wave / SHARES) * 64 + l;
  const float* from = blockIdx.z ? p.parts_b : p.parts_w;
  float* to = blockIdx.z ? p.db : p.dw;
  if (!to) return;
  for (int s = blockIdx.y; s < p.S; s += gridDim.y) {
    const int64_t lo = p.off ? p.begins[s] : 0, hi = p.off ? imin64(p.off[s + 1], p.rows) : p.rows;
    int first = 0, last = -1;
    if (lo < hi) {
      first = (int)(lo / p.part_rows);
      last = (int)((hi - 1) / p.part_rows);
      if (first == last) continue;                     // whole in one part, which gave the result
    }
    float sum = 0.f;
    if (c < p.C) {
      const int per = (last - first + SHARES) / SHARES;
      const int q1 = min(first + (share + 1) * per, last + 1);
      const float* at = from + ((int64_t)(first + share * per) + s) * p.C + c;
#pragma unroll 8
      for (int q = first + share * per; q < q1; ++q, at += p.C) sum += *at;
    }
    if constexpr (SHARES > 1) {
      lds[wave][l] = sum;
      __syncthreads();
      if (share == 0) {
#pragma unroll
        for (int o = 1; o < SHARES; ++o) sum += lds[wave + o][l];
      }
      __syncthreads();
    }
    if (share == 0 && c < p.C) {
      float* d = to + (int64_t)s * p.C + c;
      *d = p.accumulate ? *d + sum : sum;
    }
  }
}

// Waves of a row and column groups of a lane: the fewest waves that hold it, as long as the rows fill the chip. In us, by
// waves of a row: 8192 x 2560 in 6 sequences with 1 / 3 / 4 / 5: 21.1, 21.7, 22.7, 25.9, 3000 x 2560: 11.7, 10.8, 11.2, 11.8;
// 8192 x 2048 with 1 / 4: 15.4, 18.8, 1000 x 2048: 6.4, 5.2; 8192 x 3000 with
// 3 / 4: 25.0, 25.8; 8192 x 4096 with 4 / 8: 28.7, 33.5; 8192 x 12288 with 8 / 16: 77, 86. Loading weight and bias along
// with the row instead of behind its sums cost registers: 8192 x 2560 22.7 us for 21.0.
template <bool XF, bool YF>
static hipError_t forward_xy(const NormForward& p, hipStream_t s) {
  const int chunks = (p.C + 7) / 8;
  const dim3 four = long_grid((p.rows + 3) / 4), one = long_grid(p.rows);
#define CR_NF(W, V) hipLaunchKernelGGL((norm_forward_kernel<W, V, XF, YF>), W == 1 ? four : one, dim3(W == 1 ? 256 : W * 64), 0, s, p)
  if (chunks <= 64) CR_NF(1, 1);
  else if (chunks <= 128) CR_NF(1, 2);
  else if (chunks <= 256 && p.rows > 1024) CR_NF(1, 4);
  else if (chunks <= 256) CR_NF(4, 1);
  else if (chunks <= 320 && p.rows > 4096) CR_NF(1, 5);
  else if (chunks <= 384) CR_NF(3, 2);
  else if (chunks <= 512) CR_NF(4, 2);
  else if (chunks <= 1024) CR_NF(4, 4);
  else CR_NF(8, 4);
#undef CR_NF
  return hipGetLastError();
}

hipError_t launch_norm_forward(const NormForward& p, hipStream_t s) {
  if (p.x_f32) return p.y_f32 ? forward_xy<true, true>(p, s) : forward_xy<true, false>(p, s);
  return p.y_f32 ? forward_xy<false, true>(p, s) : forward_xy<false, false>(p, s);
}

// Parts of the backward pass: a block a compute unit, two of narrow rows; whole rounds of a block's groups.
// More parts hide more of a row's latency and make more slots to join.
static int norm_groups(int64_t C) { return C <= 512 ? 8 : C <= 1536 ? 4 : C <= 2048 ? 3 : C <= 4096 ? 2 : 1; }
int norm_parts(int64_t rows, int64_t C, int* part_rows) {
  const int step = norm_groups(C), most = C <= 512 ? 512 : 256;
  int64_t per = (rows + most - 1) / most;
  per = (per + step - 1) / step * step;
  *part_rows = (int)per;
  return (int)((rows + per - 1) / per);
}

size_t norm_backward_ws_bytes(int64_t rows, int64_t C, int S) {
  int per;
  const int parts = norm_parts(rows, C, &per);
  // the slots of dw and of db, then where the sequences begin
  return (size_t)2 * (size_t)(parts + S) * (size_t)C * sizeof(float) + ((size_t)S * sizeof(int) + 15) / 16 * 16;
}

// Waves of a row, eight columns a lane (two times eight from 8192 columns on, where waves end), and the groups that
// make up a block. Sixteen columns a lane, or more blocks instead of groups, leave a block's few waves waiting for their
// row: both launches in us, with 16 columns a lane and one group / 8 and one / 8 and these groups: 1531 x 2560: 19, 16, 13;
// 8192 x 2048: 34, 26, 23; 8192 x 4096: 46, 45, 44; 8192 x 1024: 19, 18, 15.
// The variants of 16 columns a lane keep 21 to 76 registers in scratch (w, dw and db of 16 columns beside the row),
// <8, 1, 2> with x or dy in float32 4 to 10: 8192 x 12288 and x 16384 with a base, x bf16 / float32, run at 4.0 / 3.8 and
// 4.2 / 3.6 TB/s (203 / 265 and 257 / 374 us), 8192 x 8192 at 4.6 / 4.8 (116 / 141), 8192 x 4096 at 4.7 / 4.4 (57 / 77).
template <bool XF, bool DF>
static void backward_xd(const NormBackward& p, hipStream_t s) {
  const dim3 grid((unsigned)p.parts);
#define CR_NB(W, V, G) hipLaunchKernelGGL((norm_backward_kernel<W, V, G, XF, DF>), grid, dim3(G * W * 64), 0, s, p)
  if (p.C <= 512) CR_NB(1, 1, 8);
  else if (p.C <= 1024) CR_NB(2, 1, 4);
  else if (p.C <= 1536) CR_NB(3, 1, 4);
  else if (p.C <= 2048) CR_NB(4, 1, 3);
  else if (p.C <= 3072) CR_NB(6, 1, 2);
  else if (p.C <= 4096) CR_NB(8, 1, 2);
  else if (p.C <= 6144) CR_NB(12, 1, 1);
  else if (p.C <= 8192) CR_NB(16, 1, 1);
  else if (p.C <= 12288) CR_NB(12, 2, 1);
  else CR_NB(16, 2, 1);
#undef CR_NB
}

hipError_t launch_norm_backward(NormBackward p, uint8_t* ws, hipStream_t s, int* kernels) {
  int per;
  p.parts = norm_parts(p.rows, p.C, &per);
  p.part_rows = per;
  if (p.dw || p.db) {
    p.parts_w = reinterpret_cast<float*>(ws);
    p.parts_b = p.parts_w + (size_t)(p.parts + p.S) * p.C;
    if (p.off) p.begins = reinterpret_cast<int*>(p.parts_b + (size_t)(p.parts + p.S) * p.C);
  }
  if (p.x_f32) {
    if (p.dy_f32) backward_xd<true, true>(p, s);
    else backward_xd<true, false>(p, s);
  } else {
    if (p.dy_f32) backward_xd<false, true>(p, s);
    else backward_xd<false, false>(p, s);
  }
  *kernels = 1;
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || !p.parts_w || (p.parts == 1 && !p.off)) return e;
  // Waves that share a sequence's slots: 1 or 4 where it has few (8192 x 4096 in 48 sequences: 45 us with 1, 49 with 4,
  // 64 with 16, for both launches; 1000 x 8192 in 7: 22.5, 22.8, 27.5), else 8 once the blocks are more than one a compute
  // unit (1531 x 2560 in 4 sequences: 15.4 with 8, 16.9 with 16), else 16 (40000 x 128: 22.5, 20.1). Blocks walk
  // the sequences beyond 2048 blocks' worth: most of many lie whole in a part and want nothing here.
  const int slots = p.parts / p.S;
  const unsigned cols = (unsigned)((p.C + 63) / 64), wide = (unsigned)((p.C + 255) / 256);
  auto down = [&](unsigned across) { return (unsigned)std::max(1, std::min(p.S, (int)(1024 / across))); };
  if (slots < 24) hipLaunchKernelGGL((norm_join_kernel<4, 1>), dim3(wide, down(wide), 2), dim3(256), 0, s, p);
  else if (slots < 64) hipLaunchKernelGGL((norm_join_kernel<4, 4>), dim3(cols, (unsigned)p.S, 2), dim3(256), 0, s, p);
  else if (cols * p.S * 2 > 256) hipLaunchKernelGGL((norm_join_kernel<8, 8>), dim3(cols, (unsigned)p.S, 2), dim3(512), 0, s, p);
  else hipLaunchKernelGGL((norm_join_kernel<16, 16>), dim3(cols, (unsigned)p.S, 2), dim3(1024), 0, s, p);
  *kernels = 2;
  return hipGetLastError();
}

}  // namespace cr
