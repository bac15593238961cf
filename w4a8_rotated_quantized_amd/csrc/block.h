// Interface between the host layer (block_abi.cpp) and the kernels of the
// microscaled 4-bit linear (mx.hip, gemm_mx.hip), of layer norm (norm.hip) and
// of the optimizer step (adamw.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/convrot.h"

namespace cr {

// columns of one tile of the 4-bit layout: codes [ceil(K/128)][rows][64 B],
// scale bytes [ceil(K/128)][rows][4 B]
constexpr int MX_TILE = 128;

struct MxQuantize {
  const uint16_t* x;
  int64_t rows, K, ldx;
  int rot_group;
  uint8_t* codes;
  uint8_t* scales;
};
hipError_t launch_mx_quantize(const MxQuantize& p, hipStream_t s);

struct MxDequantize {
  const uint8_t* codes;
  const uint8_t* scales;
  int64_t rows, K;
  int rot_group;
  void* out;
  int out_f32;
  int64_t ldo;
};
hipError_t launch_mx_dequantize(const MxDequantize& p, hipStream_t s);

struct MxGemm {
  const uint8_t* a;         // activations: codes and scale bytes
  const uint8_t* a_scales;
  const uint8_t* w;         // weights
  const uint8_t* w_scales;
  const uint16_t* bias;     // [N] or null
  void* out;
  int64_t ldc;
  int64_t M, N;
  int tiles;                // ceil(K / 128)
  int out_f32;
};
hipError_t launch_mx_gemm(const MxGemm& p, hipStream_t s);

struct NormForward {
  const void* x;
  int64_t ldx;
  const void* w;            // [S][ldw] or null
  const void* b;            // [S][ldbias] or null
  int64_t ldw, ldbias;
  int w_f32;                // of w and b
  float plus;               // added to w
  const int32_t* off;       // [S + 1], or null: one sequence of all rows
  int S;
  void* y;
  int64_t ldy;
  float* mean;
  float* rstd;
  float eps, inv_c;
  int64_t rows;
  int C;
  int x_f32, y_f32;
};
hipError_t launch_norm_forward(const NormForward& p, hipStream_t s);

struct NormBackward {
  const void* dy;
  int64_t lddy;
  const void* x;
  int64_t ldx;
  const float* mean;
  const float* rstd;
  const void* w;            // [S][ldw] or null
  int64_t ldw;
  int w_f32;
  float plus;
  const int32_t* off;
  int S;
  const void* base;         // of dx's type, or null
  int64_t ldb;
  void* dx;                 // or null
  int64_t lddx;
  float* dw;                // [S][C] or null
  float* db;
  int accumulate;
  float inv_c;
  int64_t rows;
  int C;
  int x_f32, dy_f32, dx_f32;
  // set by the launch
  int parts, part_rows;
  float* parts_w;           // [parts + S][C] each
  float* parts_b;
  int* begins;              // [S] first row of each sequence, or null
};
size_t norm_backward_ws_bytes(int64_t rows, int64_t C, int S);
hipError_t launch_norm_backward(NormBackward p, uint8_t* ws, hipStream_t s, int* kernels);

// A launch takes fewer than 2^32 threads along x: blocks beyond 2^20 go on along y.
constexpr int GRID_LG = 20;
inline dim3 long_grid(int64_t blocks) {
  const int64_t most = (int64_t)1 << GRID_LG;
  return blocks <= most ? dim3((unsigned)blocks) : dim3((unsigned)most, (unsigned)((blocks + most - 1) / most));
}

// Tensors of one launch of the optimizer step: their table rides in the kernel's arguments,
// which take 4096 bytes.
constexpr int ADAMW_TENSORS = 63, ADAMW_MOMENTS = 84;
constexpr int ADAMW_CHUNK = 1024;    // elements a block takes
constexpr int ADAMW_CHUNKS = 1 << 21;   // blocks of one launch: those of the longest tensor
constexpr int ADAMW_BLOCK = 256;     // elements that share the scale of an 8-bit moment

struct AdamwEntry {
  void* param;
  const void* grad;
  void* avg;
  void* sq;
  float* avg_scales;
  float* sq_scales;
  void* copy;
  int n;
  int first;                         // chunks of the entries before
};
struct AdamwTable {
  AdamwEntry t[ADAMW_TENSORS];
  int count;
  int ordinal;                       // number of t[0] in the caller's list
};
struct MomentsEntry {
  const void* avg;
  const void* sq;
  const float* avg_scales;
  const float* sq_scales;
  int64_t at;                        // where it begins in the outputs
  int n;
  int first;
};
struct MomentsTable {
  MomentsEntry t[ADAMW_MOMENTS];
  int count;
};
struct AdamwStep {
  float decay, b1, c1, b2, c2, rsqrt_bias2, eps, rate;   // c = 1 - b; rate = lr / (1 - b1^t)
  const float* grad_scale;           // or null
  uint32_t seed;
};
static_assert(sizeof(AdamwTable) + sizeof(AdamwStep) <= 4096 && sizeof(MomentsTable) + 2 * sizeof(float*) <= 4096, "arguments of a launch");
// `chunks` of all entries together
hipError_t launch_adamw_step(const AdamwTable& t, const AdamwStep& p, bool grad_bf16, int bits, int chunks, hipStream_t s);
// moments in 8 bits -> float32
hipError_t launch_adamw_moments(const MomentsTable& t, float* avg, float* sq, int chunks, hipStream_t s);

}  // namespace cr
