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

}  // namespace cr
