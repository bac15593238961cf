// Interface between the host layer and the kernels of the batched low-rank
// adapters (lora.hip) and of the 8-bit activation checkpoints (act.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace cr {

// The segments of a batch: rows [off[s], off[s+1]) use adapter id[s].
struct LoraSegments {
  const int32_t* off;   // [S + 1]
  const int32_t* id;    // [S]
  int S, M, A;
};

struct LoraForward {
  const uint16_t* x;
  int64_t ldx;
  const uint16_t* down;   // [A][R][K]
  const uint16_t* up;     // [A][N][R]
  LoraSegments seg;
  const float* scale;     // [A] or null
  const void* base;       // [M][ldb] of the output's type, or null
  int64_t ldb;
  void* out;
  int out_f32;
  int64_t ldo;
  float* la;              // [M][R]
  int R;
  int64_t N, K;
};
hipError_t launch_lora_forward(const LoraForward& p, hipStream_t s, int* kernels);

struct LoraBackward {
  const uint16_t* dy;
  int64_t lddy;
  const float* la;        // [M][R]
  const void* x;          // bf16 [M][ldx], or int8 codes when x_scales is set
  int64_t ldx;
  const float* x_scales;  // null, [1] or [M]
  int x_row_scales;
  int rot_group;
  const uint16_t* down;
  const uint16_t* up;
  LoraSegments seg;
  const float* scale;
  const void* dx_base;
  int64_t ldb;
  void* dx;
  int dx_f32;
  int64_t lddx;
  float* d_down;          // [A][R][K] or null
  float* d_up;            // [A][N][R] or null
  int accumulate;
  int R;
  int64_t N, K;
  uint8_t* ws;
};
hipError_t launch_lora_backward(const LoraBackward& p, hipStream_t s, int* kernels);
size_t lora_backward_ws_bytes(int64_t M, int64_t N, int64_t K, int R, int A);

struct ActArgs {
  const uint16_t* in;     // z (forward) or dy (backward)
  int64_t ldi;
  uint16_t* out;          // y (forward) or dz (backward)
  int64_t ldo;
  int8_t* codes;          // [rows][W], W = C or 2 C
  float* scales;          // [rows][W / 64]
  int64_t rows, C;
  int act;
};
hipError_t launch_act_checkpoint(const ActArgs& p, hipStream_t s);
hipError_t launch_act_backward(const ActArgs& p, hipStream_t s);

}  // namespace cr
