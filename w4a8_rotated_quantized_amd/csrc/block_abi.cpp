// C-ABI host layer of the microscaled 4-bit linear, of layer norm and of the
// optimizer step: argument validation before any HIP call, dispatch.
#include "../../include/convrot.h"
#include "block.h"
#include "host.h"

namespace {

using cr::host_aligned16;

constexpr int64_t KMAX = 32768;
constexpr int64_t LD_MAX = (int64_t)1 << 31;
constexpr int64_t ROWS_MAX = (int64_t)1 << 26;

bool given(const void* p) { return p && host_aligned16(p); }
bool absent_or_aligned(const void* p) { return !p || host_aligned16(p); }
bool bad_ld(int64_t ld, int64_t cols) { return ld < cols || ld % 8 != 0 || ld >= LD_MAX; }

// bf16 or float32 results
cr_status float_output(int type) {
  if (type < 0 || type > 2) return CR_ERR_INVALID_ARGUMENT;
  return type == CR_OUT_I32_RAW ? CR_ERR_UNSUPPORTED_FORMAT : CR_OK;
}

cr_status mx_sizes(int64_t rows, int64_t K, int rot_group) {
  if (rot_group != 0 && rot_group != 16 && rot_group != 64 && rot_group != 256 && rot_group != 1024)
    return CR_ERR_UNSUPPORTED_FORMAT;
  if (rows < 1 || rows >= ROWS_MAX || K < 32 || K % 32 || K > KMAX) return CR_ERR_UNSUPPORTED_SHAPE;
  if (rot_group && K % rot_group) return CR_ERR_UNSUPPORTED_SHAPE;
  return CR_OK;
}

}  // namespace

extern "C" {

cr_status mxfp4_quantize(const void* x, int64_t ldx, int64_t rows, int64_t K, int rot_group,
                         void* codes, void* scales, hipStream_t stream) {
  cr::host_tag("mxfp4_quantize", rows, K, rot_group, 0, 0, 0);
  if (!given(x) || !given(codes) || !given(scales)) return CR_ERR_INVALID_ARGUMENT;
  cr_status st = mx_sizes(rows, K, rot_group);
  if (st != CR_OK) return st;
  if (bad_ld(ldx, K)) return CR_ERR_UNSUPPORTED_SHAPE;
  if ((st = cr::host_device_check()) != CR_OK) return st;
  const cr::MxQuantize p{static_cast<const uint16_t*>(x), rows, K, ldx, rot_group, static_cast<uint8_t*>(codes),
                         static_cast<uint8_t*>(scales)};
  return cr::host_finish(cr::launch_mx_quantize(p, stream), cr::HE_MX, 1);
}

cr_status mxfp4_dequantize(const void* codes, const void* scales, int64_t rows, int64_t K, int rot_group,
                           void* out, cr_out out_type, int64_t ldo, hipStream_t stream) {
  cr::host_tag("mxfp4_dequantize", rows, K, rot_group, out_type, 0, 0);
  if (!given(codes) || !given(scales) || !given(out)) return CR_ERR_INVALID_ARGUMENT;
  cr_status st = float_output((int)out_type);
  if (st != CR_OK) return st;
  if ((st = mx_sizes(rows, K, rot_group)) != CR_OK) return st;
  if (bad_ld(ldo, K)) return CR_ERR_UNSUPPORTED_SHAPE;
  if ((st = cr::host_device_check()) != CR_OK) return st;
  const cr::MxDequantize p{static_cast<const uint8_t*>(codes), static_cast<const uint8_t*>(scales), rows, K, rot_group, out,
                           out_type == CR_OUT_F32, ldo};
  return cr::host_finish(cr::launch_mx_dequantize(p, stream), cr::HE_MX, 1);
}

cr_status mxfp4_gemm(const void* a_codes, const void* a_scales, const void* w_codes, const void* w_scales,
                     const void* bias, void* out, cr_out out_type, int64_t ldc,
                     int64_t M, int64_t N, int64_t K, hipStream_t stream) {
  cr::host_tag("mxfp4_gemm", M, N, K, out_type, bias != nullptr, 0);
  if (!given(a_codes) || !given(a_scales) || !given(w_codes) || !given(w_scales) || !given(out) || !absent_or_aligned(bias))
    return CR_ERR_INVALID_ARGUMENT;
  cr_status st = float_output((int)out_type);
  if (st != CR_OK) return st;
  if ((st = mx_sizes(M, K, 0)) != CR_OK) return st;
  // both below 2^26: the product of the tile counts fits 64 bits
  if (N < 1 || N >= ROWS_MAX || N % 8 || bad_ld(ldc, N) || ((M + 63) / 64) * ((N + 63) / 64) >= LD_MAX)
    return CR_ERR_UNSUPPORTED_SHAPE;
  if ((st = cr::host_device_check()) != CR_OK) return st;
  const cr::MxGemm p{static_cast<const uint8_t*>(a_codes), static_cast<const uint8_t*>(a_scales),
                     static_cast<const uint8_t*>(w_codes), static_cast<const uint8_t*>(w_scales),
                     static_cast<const uint16_t*>(bias), out, ldc, M, N, (int)((K + cr::MX_TILE - 1) / cr::MX_TILE),
                     out_type == CR_OUT_F32};
  return cr::host_finish(cr::launch_mx_gemm(p, stream), cr::HE_MX, 1);
}

}  // extern "C"
