// C-ABI host layer of the batched low-rank adapters and of the 8-bit
// activation checkpoints: argument validation before any HIP call, dispatch.
#include "../../include/convrot.h"
#include "host.h"
#include "lora.h"

namespace {

using cr::host_aligned16;

constexpr int64_t KMAX = 32768;
constexpr int64_t LD_MAX = (int64_t)1 << 31;
constexpr int64_t M_MAX = (int64_t)1 << 26;
constexpr int S_MAX = 65536, A_MAX = 4096;

bool given(const void* p) { return p && host_aligned16(p); }
bool absent_or_aligned(const void* p) { return !p || host_aligned16(p); }
bool bad_ld(int64_t ld, int64_t cols) { return ld < cols || ld % 8 != 0 || ld >= LD_MAX; }

cr_status lora_sizes(int64_t M, int64_t N, int64_t K, int R, int A) {
  if (M < 1 || M >= M_MAX || N < 8 || K < 8 || N % 8 || K % 8 || N > KMAX || K > KMAX) return CR_ERR_UNSUPPORTED_SHAPE;
  if (A < 1 || A > A_MAX) return CR_ERR_UNSUPPORTED_SHAPE;
  if (R < 8 || R > 128 || R % 8) return CR_ERR_UNSUPPORTED_FORMAT;
  return CR_OK;
}

// the output with its optional base
cr_status lora_output(const void* base, int64_t ldb, const void* out, int type, int64_t ldo, int64_t cols) {
  if (!given(out) || !absent_or_aligned(base)) return CR_ERR_INVALID_ARGUMENT;
  if (type < 0 || type > 2) return CR_ERR_INVALID_ARGUMENT;
  if (type == CR_OUT_I32_RAW) return CR_ERR_UNSUPPORTED_FORMAT;
  if (bad_ld(ldo, cols) || (base && bad_ld(ldb, cols))) return CR_ERR_UNSUPPORTED_SHAPE;
  if (base == out && ldb != ldo) return CR_ERR_INVALID_ARGUMENT;
  return CR_OK;
}

bool backward_too_large(int64_t N, int64_t K, int R, int A) {
  return (int64_t)A * R * (N > K ? N : K) >= ((int64_t)1 << 31);
}

}  // namespace

extern "C" {

cr_status convrot_lora_forward(const void* x, int64_t ldx, const void* down, const void* up, int R, int n_adapters,
                               const int32_t* seg_offsets, const int32_t* seg_adapter, int S, const float* scale,
                               const void* base, int64_t ldb, void* out, cr_out out_type, int64_t ldo,
                               float* lora_act, int64_t M, int64_t N, int64_t K, hipStream_t stream) {
  cr::host_tag("convrot_lora_forward", M, N, K, R, n_adapters, out_type);
  if (!given(x) || !given(down) || !given(up) || !given(seg_offsets) || !given(seg_adapter) || !given(lora_act) ||
      !absent_or_aligned(scale))
    return CR_ERR_INVALID_ARGUMENT;
  cr_status st = lora_sizes(M, N, K, R, n_adapters);
  if (st != CR_OK) return st;
  if (S < 1 || S > S_MAX || bad_ld(ldx, K)) return CR_ERR_UNSUPPORTED_SHAPE;
  if ((st = lora_output(base, ldb, out, (int)out_type, ldo, N)) != CR_OK) return st;
  if ((st = cr::host_device_check()) != CR_OK) return st;
  cr::LoraForward p{};
  p.x = static_cast<const uint16_t*>(x);
  p.ldx = ldx;
  p.down = static_cast<const uint16_t*>(down);
  p.up = static_cast<const uint16_t*>(up);
  p.seg = cr::LoraSegments{seg_offsets, seg_adapter, S, (int)M, n_adapters};
  p.scale = scale;
  p.base = base;
  p.ldb = ldb;
  p.out = out;
  p.out_f32 = out_type == CR_OUT_F32;
  p.ldo = ldo;
  p.la = lora_act;
  p.R = R;
  p.N = N;
  p.K = K;
  int kernels = 0;
  const hipError_t e = cr::launch_lora_forward(p, stream, &kernels);
  return cr::host_finish(e, cr::HE_LORA, (uint64_t)kernels);
}

size_t convrot_lora_backward_workspace_size(int64_t M, int64_t N, int64_t K, int R, int n_adapters) {
  if (lora_sizes(M, N, K, R, n_adapters) != CR_OK || backward_too_large(N, K, R, n_adapters)) return 0;
  return cr::lora_backward_ws_bytes(M, N, K, R, n_adapters);
}

cr_status convrot_lora_backward(const void* dy, int64_t lddy, const float* lora_act,
                                const void* x, int64_t ldx, const float* x_scales, cr_gran x_gran, int rot_group,
                                const void* down, const void* up, int R, int n_adapters,
                                const int32_t* seg_offsets, const int32_t* seg_adapter, int S, const float* scale,
                                const void* dx_base, int64_t ldb, void* dx, cr_out dx_type, int64_t lddx,
                                float* d_down, float* d_up, int accumulate,
                                int64_t M, int64_t N, int64_t K,
                                void* workspace, size_t workspace_bytes, hipStream_t stream) {
  cr::host_tag("convrot_lora_backward", M, N, K, R, n_adapters, x_scales ? rot_group : 0);
  if (!given(dy) || !given(down) || !given(up) || !given(seg_offsets) || !given(seg_adapter) || !given(workspace) ||
      !absent_or_aligned(scale) || !absent_or_aligned(lora_act) || !absent_or_aligned(x) ||
      !absent_or_aligned(x_scales) || !absent_or_aligned(d_down) || !absent_or_aligned(d_up))
    return CR_ERR_INVALID_ARGUMENT;
  if (!dx && !d_down && !d_up) return CR_ERR_INVALID_ARGUMENT;
  if ((d_down && !x) || (d_up && !lora_act)) return CR_ERR_INVALID_ARGUMENT;
  cr_status st = lora_sizes(M, N, K, R, n_adapters);
  if (st != CR_OK) return st;
  if (S < 1 || S > S_MAX || bad_ld(lddy, N) || backward_too_large(N, K, R, n_adapters)) return CR_ERR_UNSUPPORTED_SHAPE;
  if (dx && (st = lora_output(dx_base, ldb, dx, (int)dx_type, lddx, K)) != CR_OK) return st;
  if (d_down) {
    if (bad_ld(ldx, K)) return CR_ERR_UNSUPPORTED_SHAPE;
    if (x_scales) {
      if ((int)x_gran < 0 || (int)x_gran > 2) return CR_ERR_INVALID_ARGUMENT;
      if (x_gran == CR_GRAN_ROW_GROUP) return CR_ERR_UNSUPPORTED_FORMAT;
      if (rot_group != 16 && rot_group != 64 && rot_group != 256 && rot_group != 1024) return CR_ERR_UNSUPPORTED_FORMAT;
      if (K % 256 || K % rot_group || ldx % 16) return CR_ERR_UNSUPPORTED_SHAPE;
    }
  }
  if (workspace_bytes < cr::lora_backward_ws_bytes(M, N, K, R, n_adapters)) return CR_ERR_WORKSPACE_TOO_SMALL;
  if ((st = cr::host_device_check()) != CR_OK) return st;
  cr::LoraBackward p{};
  p.dy = static_cast<const uint16_t*>(dy);
  p.lddy = lddy;
  p.la = lora_act;
  p.x = x;
  p.ldx = ldx;
  p.x_scales = x_scales;
  p.x_row_scales = x_gran == CR_GRAN_ROW;
  p.rot_group = rot_group;
  p.down = static_cast<const uint16_t*>(down);
  p.up = static_cast<const uint16_t*>(up);
  p.seg = cr::LoraSegments{seg_offsets, seg_adapter, S, (int)M, n_adapters};
  p.scale = scale;
  p.dx_base = dx_base;
  p.ldb = ldb;
  p.dx = dx;
  p.dx_f32 = dx_type == CR_OUT_F32;
  p.lddx = lddx;
  p.d_down = d_down;
  p.d_up = d_up;
  p.accumulate = accumulate != 0;
  p.R = R;
  p.N = N;
  p.K = K;
  p.ws = static_cast<uint8_t*>(workspace);
  int kernels = 0;
  const hipError_t e = cr::launch_lora_backward(p, stream, &kernels);
  return cr::host_finish(e, cr::HE_LORA, (uint64_t)kernels);
}

static cr_status act_validate(const void* in, const void* out, const void* codes, const void* scales, int64_t rows,
                              int64_t C, int act) {
  if (!given(in) || !given(out) || !given(codes) || !given(scales)) return CR_ERR_INVALID_ARGUMENT;
  if (act < 0 || act > 2) return CR_ERR_INVALID_ARGUMENT;
  // C bounds the product below 2^51 before it is formed
  if (rows < 1 || rows >= LD_MAX || C < 64 || C % 64 || C > KMAX || rows * C >= ((int64_t)1 << 34))
    return CR_ERR_UNSUPPORTED_SHAPE;
  return CR_OK;
}

cr_status convrot_act_checkpoint(const void* z, int64_t ldz, int64_t rows, int64_t C, cr_act act,
                                 void* y, int64_t ldy, void* codes, float* scales, hipStream_t stream) {
  cr::host_tag("convrot_act_checkpoint", rows, C, 0, act, 0, 0);
  cr_status st = act_validate(z, y, codes, scales, rows, C, (int)act);
  if (st != CR_OK) return st;
  if (bad_ld(ldz, act == CR_ACT_SWIGLU ? 2 * C : C) || bad_ld(ldy, C)) return CR_ERR_UNSUPPORTED_SHAPE;
  if ((st = cr::host_device_check()) != CR_OK) return st;
  const cr::ActArgs p{static_cast<const uint16_t*>(z), ldz, static_cast<uint16_t*>(y), ldy,
                      static_cast<int8_t*>(codes), scales, rows, C, act};
  return cr::host_finish(cr::launch_act_checkpoint(p, stream), cr::HE_ACT, 1);
}

cr_status convrot_act_backward(const void* dy, int64_t lddy, const void* codes, const float* scales,
                               int64_t rows, int64_t C, cr_act act, void* dz, int64_t lddz, hipStream_t stream) {
  cr::host_tag("convrot_act_backward", rows, C, 0, act, 0, 0);
  cr_status st = act_validate(dy, dz, codes, scales, rows, C, (int)act);
  if (st != CR_OK) return st;
  if (bad_ld(lddy, C) || bad_ld(lddz, act == CR_ACT_SWIGLU ? 2 * C : C)) return CR_ERR_UNSUPPORTED_SHAPE;
  if ((st = cr::host_device_check()) != CR_OK) return st;
  const cr::ActArgs p{static_cast<const uint16_t*>(dy), lddy, static_cast<uint16_t*>(dz), lddz,
                      static_cast<int8_t*>(const_cast<void*>(codes)), const_cast<float*>(scales), rows, C, act};
  return cr::host_finish(cr::launch_act_backward(p, stream), cr::HE_ACT, 1);
}

}  // extern "C"
