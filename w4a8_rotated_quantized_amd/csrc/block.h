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
};
size_t norm_backward_ws_bytes(int64_t rows, int64_t C, int S);
hipError_t launch_norm_backward(NormBackward p, uint8_t* ws, hipStream_t s, int* kernels);

// Tensors of one launch of the optimizer step: their table rides in the kernel's arguments.
constexpr int ADAMW_TENSORS = 48;
constexpr int ADAMW_CHUNK = 1024;    // elements a block takes
constexpr int ADAMW_BLOCK = 256;     // elements that share the scale of an 8-bit moment

struct AdamwTable {
  cr_adamw_tensor t[ADAMW_TENSORS];
  int64_t before[ADAMW_TENSORS];     // elements of t[0] .. t[i - 1]
  int first[ADAMW_TENSORS + 1];      // chunks of t[0] .. t[i - 1]
  int count;
  int ordinal;                       // number of t[0] in the caller's list
};
struct AdamwStep {
  float decay, b1, c1, b2, c2, rsqrt_bias2, eps, rate;   // c = 1 - b; rate = lr / (1 - b1^t)
  const float* grad_scale;           // or null
  uint32_t seed;
  int grad_bf16, bits;
};
hipError_t launch_adamw_step(const AdamwTable& t, const AdamwStep& p, hipStream_t s);
// moments in 8 bits -> float32, tensor after tensor; `at`: where t[0] begins
hipError_t launch_adamw_moments(const AdamwTable& t, int64_t at, float* avg, float* sq, hipStream_t s);

}  // namespace cr
