// Stands in for libconvrot.so behind the native module of the Python binding
// (tests/test_binding_cpu.py): no call does anything but wait, five seconds at most, for a
// word from another thread, and answer CR_OK if it came and CR_ERR_HIP if not.
#include <atomic>
#include <chrono>
#include <cstdlib>
#include <thread>

#include "convrot.h"

namespace {
std::atomic<int> g_calls{0}, g_words{0};
std::atomic<int> g_wait{1};
cr_status met() {
  const int call = ++g_calls;
  for (int i = 0; g_wait && i < 5000 && g_words < call; ++i) std::this_thread::sleep_for(std::chrono::milliseconds(1));
  return !g_wait || g_words >= call ? CR_OK : CR_ERR_HIP;
}
}  // namespace

extern "C" {

int stub_calls() { return g_calls; }
void stub_word() { ++g_words; }
void stub_wait(int on) { g_wait = on; }
// The process's end, behind the interpreter's, gives the waiting call its word and stays for half a second.
void stub_linger() {
  std::atexit([] {
    g_words = 1 << 30;
    std::this_thread::sleep_for(std::chrono::milliseconds(500));
  });
}

cr_status mxfp4_quantize(const void*, int64_t, int64_t, int64_t, int, void*, void*, hipStream_t) { return met(); }
cr_status mxfp4_dequantize(const void*, const void*, int64_t, int64_t, int, void*, cr_out, int64_t, hipStream_t) { return met(); }
cr_status mxfp4_gemm(const void*, const void*, const void*, const void*, const void*, void*, cr_out, int64_t, int64_t, int64_t, int64_t,
                     hipStream_t) {
  return met();
}
cr_status convrot_layer_norm_forward(const void*, cr_out, int64_t, const void*, int64_t, const void*, int64_t, cr_out, int, const int32_t*,
                                     int, double, void*, cr_out, int64_t, float*, float*, int64_t, int64_t, hipStream_t) {
  return met();
}
size_t convrot_layer_norm_backward_workspace_size(int64_t, int64_t, int) { return 64; }
cr_status convrot_layer_norm_backward(const void*, cr_out, int64_t, const void*, cr_out, int64_t, const float*, const float*, const void*,
                                      int64_t, cr_out, int, const int32_t*, int, const void*, int64_t, void*, cr_out, int64_t, float*,
                                      float*, int, int64_t, int64_t, void*, size_t, hipStream_t) {
  return met();
}
cr_status convrot_adamw_step(const cr_adamw_tensor*, int, cr_out, int, double, double, double, double, double, int64_t, const float*,
                             uint32_t, hipStream_t) {
  return met();
}
cr_status convrot_adamw_moments(const cr_adamw_tensor*, int, float*, float*, hipStream_t) { return met(); }

}  // extern "C"
