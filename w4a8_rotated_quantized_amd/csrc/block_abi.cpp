// C-ABI host layer of the microscaled 4-bit linear, of layer norm and of the
// optimizer step: argument validation before any HIP call, dispatch.
#include <cmath>

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

constexpr int64_t NORM_COLS = 16384;
constexpr int NORM_SEGMENTS = 4096;

cr_status norm_sizes(int64_t rows, int64_t C, int S) {
  if (rows < 1 || rows >= ROWS_MAX || C < 8 || C % 8 || C > NORM_COLS || S < 1 || S > NORM_SEGMENTS)
    return CR_ERR_UNSUPPORTED_SHAPE;
  return CR_OK;
}

constexpr int ADAMW_COUNT = 65536;
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Entries of a list, `param` to `copy` where `step`, and with 8-bit moments their scales.
cr_status adamw_entries(const cr_adamw_tensor* t, int count, bool step, bool coded) {
  if (!t) return CR_ERR_INVALID_ARGUMENT;
  if (count < 1 || count > ADAMW_COUNT) return CR_ERR_UNSUPPORTED_SHAPE;
  for (int i = 0; i < count; ++i) {
    if (t[i].n < 0 || t[i].n >= LD_MAX) return CR_ERR_UNSUPPORTED_SHAPE;
    if (t[i].n == 0) continue;
    if (!given(t[i].exp_avg) || !given(t[i].exp_avg_sq)) return CR_ERR_INVALID_ARGUMENT;
    if (step && (!given(t[i].param) || !given(t[i].grad) || !absent_or_aligned(t[i].copy))) return CR_ERR_INVALID_ARGUMENT;
    if (coded && (!t[i].avg_scales || !t[i].sq_scales || !aligned4(t[i].avg_scales) || !aligned4(t[i].sq_scales)))
      return CR_ERR_INVALID_ARGUMENT;
  }
  return CR_OK;
}

// Calls launch(table, chunks) for the entries of a list, a table at a time: tables of the same
// number of entries, so that the last launch is no stub. fill(entry, tensor, elements before it).
template <typename Table, int MOST, typename F, typename L>
hipError_t adamw_tables(const cr_adamw_tensor* t, int count, int* kernels, F fill, L launch) {
  *kernels = 0;
  int64_t elements = 0;
  const int tables = (count + MOST - 1) / MOST, per = (count + tables - 1) / tables;
  for (int i = 0; i < count;) {
    Table table;
    table.count = 0;
    const int begin = i;
    int64_t chunks = 0;
    // every entry takes a place, empty ones no chunk, so that their numbers count them
    while (i < count && table.count < per) {
      const int64_t c = (t[i].n + cr::ADAMW_CHUNK - 1) / cr::ADAMW_CHUNK;
      if (table.count && chunks + c > cr::ADAMW_CHUNKS) break;
      auto& e = table.t[table.count++];
      fill(e, t[i], elements);
      e.n = (int)t[i].n;
      e.first = (int)chunks;
      chunks += c;
      elements += t[i].n;
      ++i;
    }
    if (chunks) {
      const hipError_t e = launch(table, begin, (int)chunks);
      if (e != hipSuccess) return e;
      ++*kernels;
    }
  }
  return hipSuccess;
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

cr_status convrot_layer_norm_forward(const void* x, cr_out x_type, int64_t ldx, const void* weight, int64_t ldw,
                                     const void* bias, int64_t ldbias, cr_out affine_type, int one_plus, const int32_t* seg_offsets, int S, double eps,
                                     void* y, cr_out y_type, int64_t ldy, float* mean, float* rstd,
                                     int64_t rows, int64_t C, hipStream_t stream) {
  cr::host_tag("convrot_layer_norm_forward", rows, C, S, x_type, affine_type, y_type);
  if (!given(x) || !given(y) || !given(mean) || !given(rstd) || !absent_or_aligned(weight) || !absent_or_aligned(bias) ||
      !absent_or_aligned(seg_offsets))
    return CR_ERR_INVALID_ARGUMENT;
  if (one_plus < 0 || one_plus > 1 || !(eps >= 0.0) || !(eps < 1e30)) return CR_ERR_INVALID_ARGUMENT;
  if (eps > 0.0 && (float)eps == 0.f) return CR_ERR_INVALID_ARGUMENT;
  cr_status st;
  for (const int type : {(int)x_type, (int)y_type, (int)affine_type})
    if ((st = float_output(type)) != CR_OK) return st;
  if ((st = norm_sizes(rows, C, S)) != CR_OK) return st;
  if (!seg_offsets && S != 1) return CR_ERR_INVALID_ARGUMENT;
  if (bad_ld(ldx, C) || bad_ld(ldy, C) || (S > 1 && ((weight && bad_ld(ldw, C)) || (bias && bad_ld(ldbias, C)))))
    return CR_ERR_UNSUPPORTED_SHAPE;
  if ((st = cr::host_device_check()) != CR_OK) return st;
  cr::NormForward p{};
  p.x = x;
  p.ldx = ldx;
  p.w = weight;
  p.ldw = ldw;
  p.b = bias;
  p.ldbias = ldbias;
  p.w_f32 = affine_type == CR_OUT_F32;
  p.plus = one_plus ? 1.f : 0.f;
  p.off = seg_offsets;
  p.S = S;
  p.y = y;
  p.ldy = ldy;
  p.mean = mean;
  p.rstd = rstd;
  p.eps = (float)eps;
  p.inv_c = 1.f / (float)C;
  p.rows = rows;
  p.C = (int)C;
  p.x_f32 = x_type == CR_OUT_F32;
  p.y_f32 = y_type == CR_OUT_F32;
  return cr::host_finish(cr::launch_norm_forward(p, stream), cr::HE_ACT, 1);
}

size_t convrot_layer_norm_backward_workspace_size(int64_t rows, int64_t C, int S) {
  return norm_sizes(rows, C, S) == CR_OK ? cr::norm_backward_ws_bytes(rows, C, S) : 0;
}

cr_status convrot_layer_norm_backward(const void* dy, cr_out dy_type, int64_t lddy, const void* x, cr_out x_type,
                                      int64_t ldx, const float* mean, const float* rstd, const void* weight, int64_t ldw,
                                      cr_out affine_type, int one_plus, const int32_t* seg_offsets, int S,
                                      const void* dx_base, int64_t ldb, void* dx, cr_out dx_type, int64_t lddx,
                                      float* d_weight, float* d_bias, int accumulate, int64_t rows, int64_t C,
                                      void* workspace, size_t workspace_bytes, hipStream_t stream) {
  cr::host_tag("convrot_layer_norm_backward", rows, C, S, x_type, affine_type, dx_type);
  if (!given(dy) || !given(x) || !given(mean) || !given(rstd) || !absent_or_aligned(weight) ||
      !absent_or_aligned(seg_offsets) || !absent_or_aligned(dx_base) || !absent_or_aligned(dx) ||
      !absent_or_aligned(d_weight) || !absent_or_aligned(d_bias) || !absent_or_aligned(workspace))
    return CR_ERR_INVALID_ARGUMENT;
  if (!dx && !d_weight && !d_bias) return CR_ERR_INVALID_ARGUMENT;
  if (one_plus < 0 || one_plus > 1) return CR_ERR_INVALID_ARGUMENT;
  cr_status st;
  for (const int type : {(int)dy_type, (int)x_type, (int)affine_type, dx ? (int)dx_type : (int)CR_OUT_F32})
    if ((st = float_output(type)) != CR_OK) return st;
  if ((st = norm_sizes(rows, C, S)) != CR_OK) return st;
  if (!seg_offsets && S != 1) return CR_ERR_INVALID_ARGUMENT;
  if (bad_ld(lddy, C) || bad_ld(ldx, C) || (dx && bad_ld(lddx, C)) || (dx && dx_base && bad_ld(ldb, C)) ||
      (S > 1 && weight && bad_ld(ldw, C)))
    return CR_ERR_UNSUPPORTED_SHAPE;
  if (dx && dx_base == dx && ldb != lddx) return CR_ERR_INVALID_ARGUMENT;
  if (d_weight || d_bias) {
    if (!workspace) return CR_ERR_INVALID_ARGUMENT;
    if (workspace_bytes < cr::norm_backward_ws_bytes(rows, C, S)) return CR_ERR_WORKSPACE_TOO_SMALL;
  }
  if ((st = cr::host_device_check()) != CR_OK) return st;
  cr::NormBackward p{};
  p.dy = dy;
  p.lddy = lddy;
  p.x = x;
  p.ldx = ldx;
  p.mean = mean;
  p.rstd = rstd;
  p.w = weight;
  p.ldw = ldw;
  p.w_f32 = affine_type == CR_OUT_F32;
  p.plus = one_plus ? 1.f : 0.f;
  p.off = seg_offsets;
  p.S = S;
  p.base = dx ? dx_base : nullptr;
  p.ldb = ldb;
  p.dx = dx;
  p.lddx = lddx;
  p.dw = d_weight;
  p.db = d_bias;
  p.accumulate = accumulate != 0;
  p.inv_c = 1.f / (float)C;
  p.rows = rows;
  p.C = (int)C;
  p.x_f32 = x_type == CR_OUT_F32;
  p.dy_f32 = dy_type == CR_OUT_F32;
  p.dx_f32 = dx_type == CR_OUT_F32;
  int kernels = 0;
  const hipError_t e = cr::launch_norm_backward(p, static_cast<uint8_t*>(workspace), stream, &kernels);
  return cr::host_finish(e, cr::HE_ACT, (uint64_t)kernels);
}

cr_status convrot_adamw_step(const cr_adamw_tensor* tensors, int count, cr_out grad_type, int state_bits,
                             double lr, double beta1, double beta2, double eps, double weight_decay, int64_t step,
                             const float* grad_scale, uint32_t seed, hipStream_t stream) {
  cr::host_tag("convrot_adamw_step", count, tensors && count > 0 ? tensors[0].n : 0, step, grad_type, state_bits, 0);
  cr_status st = float_output((int)grad_type);
  if (st != CR_OK) return st;
  if (state_bits != 8 && state_bits != 32) return CR_ERR_UNSUPPORTED_FORMAT;
  if (!(lr >= 0.0) || !(eps >= 0.0) || !(weight_decay >= 0.0) || !(beta1 >= 0.0 && beta1 < 1.0) ||
      !(beta2 >= 0.0 && beta2 < 1.0) || step < 1 || !aligned4(grad_scale))
    return CR_ERR_INVALID_ARGUMENT;
  // the kernel multiplies by the denominator's reciprocal, which is infinite where that is eps alone and subnormal
  if (eps > 0.0 && (float)eps < 0x1p-126f) return CR_ERR_INVALID_ARGUMENT;
  if ((st = adamw_entries(tensors, count, true, state_bits == 8)) != CR_OK) return st;
  if ((st = cr::host_device_check()) != CR_OK) return st;
  cr::AdamwStep p;
  p.decay = (float)(1.0 - lr * weight_decay);
  p.b1 = (float)beta1;
  p.c1 = (float)(1.0 - beta1);
  p.b2 = (float)beta2;
  p.c2 = (float)(1.0 - beta2);
  p.rsqrt_bias2 = (float)(1.0 / std::sqrt(1.0 - std::pow(beta2, (double)step)));
  p.eps = (float)eps;
  p.rate = (float)(lr / (1.0 - std::pow(beta1, (double)step)));
  p.grad_scale = grad_scale;
  p.seed = seed;
  const bool grad_bf16 = grad_type == CR_OUT_BF16;
  int kernels = 0;
  const hipError_t e = adamw_tables<cr::AdamwTable, cr::ADAMW_TENSORS>(
      tensors, count, &kernels,
      [](cr::AdamwEntry& d, const cr_adamw_tensor& t, int64_t) {
        d.param = t.param;
        d.grad = t.grad;
        d.avg = t.exp_avg;
        d.sq = t.exp_avg_sq;
        d.avg_scales = t.avg_scales;
        d.sq_scales = t.sq_scales;
        d.copy = t.copy;
      },
      [&](cr::AdamwTable& t, int begin, int chunks) {
        t.ordinal = begin;
        return cr::launch_adamw_step(t, p, grad_bf16, state_bits, chunks, stream);
      });
  return cr::host_finish(e, cr::HE_LORA, (uint64_t)kernels);
}

cr_status convrot_adamw_moments(const cr_adamw_tensor* tensors, int count, float* exp_avg_out, float* exp_avg_sq_out,
                                hipStream_t stream) {
  cr::host_tag("convrot_adamw_moments", count, tensors && count > 0 ? tensors[0].n : 0, 0, 0, 0, 0);
  if (!given(exp_avg_out) || !given(exp_avg_sq_out)) return CR_ERR_INVALID_ARGUMENT;
  cr_status st = adamw_entries(tensors, count, false, true);
  if (st != CR_OK) return st;
  if ((st = cr::host_device_check()) != CR_OK) return st;
  int kernels = 0;
  const hipError_t e = adamw_tables<cr::MomentsTable, cr::ADAMW_MOMENTS>(
      tensors, count, &kernels,
      [](cr::MomentsEntry& d, const cr_adamw_tensor& t, int64_t before) {
        d.avg = t.exp_avg;
        d.sq = t.exp_avg_sq;
        d.avg_scales = t.avg_scales;
        d.sq_scales = t.sq_scales;
        d.at = before;
      },
      [&](const cr::MomentsTable& t, int, int chunks) {
        return cr::launch_adamw_moments(t, exp_avg_out, exp_avg_sq_out, chunks, stream);
      });
  return cr::host_finish(e, cr::HE_LORA, (uint64_t)kernels);
}

}  // extern "C"
