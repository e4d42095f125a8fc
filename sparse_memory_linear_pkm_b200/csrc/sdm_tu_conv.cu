// Entry points and launches of the short causal convolution and its gradient.

#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "sdm_check.h"
#include "sdm_conv.cuh"

namespace sdm_host {

using sdm::bf16;

namespace {

constexpr int kGradSeg = 64;  // tokens of a gradient thread

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

sdm_status_t check_conv(int32_t B, int32_t T, int32_t D, int32_t K, int64_t x_stride, int32_t in_dtype,
                        int32_t w_dtype) {
  if (B < 0 || T < 0 || D < 0) return fail(SDM_ERR_INVALID_ARGUMENT, "B, T and D must be >= 0");
  if (K < 2 || K > sdm::kConvMaxK)
    return fail(SDM_ERR_INVALID_ARGUMENT, "K must be in [2, 8], got " + std::to_string(K));
  if (B > 65535) return fail(SDM_ERR_UNSUPPORTED, "B above 65535");
  if (x_stride != 0 && x_stride < D) return fail(SDM_ERR_INVALID_ARGUMENT, "x_stride must be 0 or at least D");
  // Thread and segment numbers within a sequence are 32-bit.
  if (static_cast<int64_t>(T) + 16 > INT32_MAX || static_cast<int64_t>(D) * ceil_div(T, 8) > INT32_MAX - 1024)
    return fail(SDM_ERR_UNSUPPORTED, "T * D / 8 above 2^31");
  sdm_status_t r;
  if ((r = check_dtype(in_dtype, "in_dtype")) || (r = check_dtype(w_dtype, "w_dtype"))) return r;
  return SDM_OK;
}

// Whether rows of D values at this address and stride are whole units of a thread's channels.
bool whole_units(const void* x, int64_t x_stride, int32_t D, int32_t dtype) {
  constexpr int V = sdm::kConvV;
  return D % V == 0 && x_stride % V == 0 && reinterpret_cast<uintptr_t>(x) % (V * in_size(dtype)) == 0;
}

// Whether a channel's taps are one aligned unit of four.
bool whole_taps(const void* w, int32_t dtype, int32_t K) {
  return K == 4 && reinterpret_cast<uintptr_t>(w) % (4 * in_size(dtype)) == 0;
}

// f(std::integral_constant<int, K>()) for the K in [2, kConvMaxK] of a call.
template <int kTaps = 2, typename F>
void with_taps(int K, const F& f) {
  if constexpr (kTaps < sdm::kConvMaxK) {
    if (K != kTaps) return with_taps<kTaps + 1>(K, f);
  }
  f(std::integral_constant<int, kTaps>());
}

// Tokens of a thread: up to 64 (the K - 1 inputs before a run are read twice),
// fewer while the threads would not fill the device's 148 SMs with 1024 each.
int conv_run(int B, int T, int units) {
  int run = 64;
  while (run > 2 * sdm::kConvAhead && static_cast<int64_t>(B) * units * ceil_div(T, run) < 148 * 1024) run /= 2;
  return run;
}

template <typename T>
void launch_conv(bool vec, const sdm::ConvArgs& a, int B, cudaStream_t st) {
  const dim3 grid(static_cast<unsigned>(ceil_div(a.per_seq, 256)), B);
  with_taps(a.K, [&](auto K) {
    if (vec) sdm::k_short_conv<T, K.value, true><<<grid, 256, 0, st>>>(a);
    else sdm::k_short_conv<T, K.value, false><<<grid, 256, 0, st>>>(a);
  });
}

template <typename T>
void launch_conv_grad(bool vec, const sdm::ConvGradArgs& a, dim3 grid, cudaStream_t st) {
  const dim3 block(sdm::kConvGradLanes, sdm::kConvGradRows);
  with_taps(a.K, [&](auto K) {
    if (vec) sdm::k_short_conv_backward<T, K.value, true><<<grid, block, 0, st>>>(a);
    else sdm::k_short_conv_backward<T, K.value, false><<<grid, block, 0, st>>>(a);
  });
}

struct ConvGradPlan {
  int segs;
  int64_t slots;
  size_t bytes;
};
ConvGradPlan conv_grad_plan(int32_t B, int32_t T, int32_t D, int32_t K) {
  ConvGradPlan p;
  p.segs = static_cast<int>(ceil_div(T, kGradSeg));
  p.slots = ceil_div(static_cast<int64_t>(B) * p.segs, sdm::kConvGradRows);
  p.bytes = align256(static_cast<size_t>(p.slots) * D * (K + 1) * sizeof(float));
  return p;
}

}  // namespace

}  // namespace sdm_host

using namespace sdm_host;

extern "C" {

sdm_status_t sdm_short_conv(const void* x, int64_t x_stride, int32_t in_dtype, const void* w, const void* bias,
                            int32_t w_dtype, int32_t B, int32_t T, int32_t D, int32_t K, int32_t silu, void* state,
                            const int32_t* lengths, void* y, void* stream) {
  sdm_status_t r;
  if ((r = check_conv(B, T, D, K, x_stride, in_dtype, w_dtype)) != SDM_OK) return r;
  const bool any = B > 0 && T > 0 && D > 0;
  if ((r = need_gate(x, "x", any, in_dtype)) || (r = need_gate(w, "w", any, w_dtype)) ||
      (r = need_gate(bias, "bias", any && bias != nullptr, w_dtype)) ||
      (r = need_ptr(state, "state", any && state != nullptr)) ||
      (r = need_gate(lengths, "lengths", any && lengths != nullptr, SDM_F32)) || (r = need_ptr(y, "y", any)))
    return r;
  if (!any) return ok();
  const int64_t stride = x_stride == 0 ? D : x_stride;
  const size_t es = in_size(in_dtype);
  const int64_t tokens = static_cast<int64_t>(B) * T;
  // (Threads read their neighbours' inputs.)
  const size_t row = static_cast<size_t>(D) * es, sb = static_cast<size_t>(B) * (K - 1) * row;
  const size_t ws = in_size(w_dtype) * D;
  const Piece ins[] = {{"x", x, (static_cast<size_t>(tokens - 1) * stride) * es + row},
                       {"w", w, ws * K},
                       {"bias", bias, ws},
                       {"lengths", lengths, B * sizeof(int32_t)}};
  const Piece outs[] = {{"y", y, static_cast<size_t>(tokens) * row}, {"state", state, sb}};
  if ((r = check_apart(outs, 2, ins, 4)) != SDM_OK) return r;
  DeviceInfo* dev;
  if ((r = device_info(&dev)) != SDM_OK) return r;
  const bool vec = whole_units(x, stride, D, in_dtype);
  const int units = static_cast<int>(ceil_div(D, sdm::kConvV)), run = conv_run(B, T, units);
  const sdm::ConvArgs a{x, w, bias, state, lengths, y, stride, T, D, K, units, run,
                        static_cast<unsigned>(units * ceil_div(T, run)), w_dtype == SDM_BF16,
                        whole_taps(w, w_dtype, K), silu != 0, dev->err};
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (in_dtype == SDM_BF16) launch_conv<bf16>(vec, a, B, st);
  else launch_conv<float>(vec, a, B, st);
  if ((r = launch_status("short_conv launch")) != SDM_OK) return r;
  return ok();
}

size_t sdm_short_conv_backward_workspace_bytes(int32_t B, int32_t T, int32_t D, int32_t K) {
  if (check_conv(B, T, D, K, 0, SDM_F32, SDM_F32) != SDM_OK) return 0;
  ok();
  return conv_grad_plan(B, T, D, K).bytes;
}

sdm_status_t sdm_short_conv_backward(const void* x, int64_t x_stride, int32_t in_dtype, const void* w,
                                     const void* bias, int32_t w_dtype, int32_t B, int32_t T, int32_t D, int32_t K,
                                     int32_t silu, const void* state0, const int32_t* lengths, const void* dy,
                                     const void* dstate, void* dx, float* dw, float* dbias, void* dstate0,
                                     void* workspace, size_t workspace_bytes, void* stream) {
  sdm_status_t r;
  if ((r = check_conv(B, T, D, K, x_stride, in_dtype, w_dtype)) != SDM_OK) return r;
  const bool any = B > 0 && T > 0 && D > 0;
  if ((r = need_ptr(dw, "dw", D > 0)) || (r = need_ptr(dbias, "dbias", D > 0 && dbias != nullptr)) ||
      (r = need_ptr(state0, "state0", state0 != nullptr)) || (r = need_ptr(dstate, "dstate", dstate != nullptr)) ||
      (r = need_ptr(dstate0, "dstate0", dstate0 != nullptr)) || (r = need_gate(x, "x", any, in_dtype)) ||
      (r = need_gate(w, "w", any, w_dtype)) || (r = need_gate(bias, "bias", any && bias != nullptr, w_dtype)) ||
      (r = need_gate(lengths, "lengths", any && lengths != nullptr, SDM_F32)) || (r = need_ptr(dy, "dy", any)) ||
      (r = need_ptr(dx, "dx", any)))
    return r;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const size_t es = in_size(in_dtype);
  if (!any) {
    // No token: the parameters get nothing, and the initial state is the final one.
    const size_t sb = static_cast<size_t>(B) * (K - 1) * D * es;
    const Piece first = {"dstate0", dstate0, sb}, last = {"dstate", dstate0 == dstate ? nullptr : dstate, sb};
    if ((r = check_apart(&first, 1, &last, 1)) != SDM_OK) return r;
    cudaError_t e = cudaSuccess;
    if (D > 0) e = cudaMemsetAsync(dw, 0, static_cast<size_t>(D) * K * sizeof(float), st);
    if (e == cudaSuccess && D > 0 && dbias != nullptr) e = cudaMemsetAsync(dbias, 0, D * sizeof(float), st);
    if (e == cudaSuccess && sb > 0 && dstate0 != nullptr && dstate0 != dstate)
      e = dstate != nullptr ? cudaMemcpyAsync(dstate0, dstate, sb, cudaMemcpyDeviceToDevice, st)
                            : cudaMemsetAsync(dstate0, 0, sb, st);
    if (e != cudaSuccess) return fail(SDM_ERR_CUDA, std::string("empty gradient: ") + cudaGetErrorString(e));
    return ok();
  }
  if ((r = need_ptr(workspace, "workspace", true)) != SDM_OK) return r;
  const ConvGradPlan p = conv_grad_plan(B, T, D, K);
  if (workspace_bytes < p.bytes)
    return fail(SDM_ERR_INVALID_ARGUMENT, "workspace is smaller than sdm_short_conv_backward_workspace_bytes");
  const int64_t stride = x_stride == 0 ? D : x_stride;
  const int64_t tokens = static_cast<int64_t>(B) * T;
  const size_t row = static_cast<size_t>(D) * es, nb = static_cast<size_t>(tokens) * row;
  const size_t sb = static_cast<size_t>(B) * (K - 1) * row;
  const Piece ins[] = {{"x", x, (static_cast<size_t>(tokens - 1) * stride) * es + row},
                       {"dy", dy, nb},
                       {"state0", state0, sb},
                       {"dstate", dstate, sb},
                       {"w", w, in_size(w_dtype) * D * K},
                       {"bias", bias, in_size(w_dtype) * D},
                       {"lengths", lengths, B * sizeof(int32_t)}};
  const Piece outs[] = {{"dx", dx, nb},
                        {"dstate0", dstate0, sb},
                        {"dw", dw, sizeof(float) * D * K},
                        {"dbias", dbias, sizeof(float) * D}};
  if ((r = check_apart(outs, 4, ins, 7)) != SDM_OK) return r;
  if (p.slots > 65535) return fail(SDM_ERR_UNSUPPORTED, "B * T above 65535 * 512 tokens");
  DeviceInfo* dev;
  if ((r = device_info(&dev)) != SDM_OK) return r;
  const bool vec = whole_units(x, stride, D, in_dtype);
  float* part = static_cast<float*>(workspace);
  const sdm::ConvGradArgs a{x, w, bias, state0, dy, dstate, lengths, dx, dstate0, part, stride, B, T, D, K,
                            static_cast<int>(ceil_div(D, sdm::kConvV)), p.segs, kGradSeg, w_dtype == SDM_BF16,
                            whole_taps(w, w_dtype, K), silu != 0, dev->err};
  const dim3 grid(static_cast<unsigned>(ceil_div(a.units, sdm::kConvGradLanes)), static_cast<unsigned>(p.slots));
  if (in_dtype == SDM_BF16) launch_conv_grad<bf16>(vec, a, grid, st);
  else launch_conv_grad<float>(vec, a, grid, st);
  if ((r = launch_status("short_conv_backward launch")) != SDM_OK) return r;
  const int64_t n = static_cast<int64_t>(D) * (K + 1);
  sdm::k_short_conv_sums<<<static_cast<unsigned>(ceil_div(n, 32)), dim3(32, 8), 0, st>>>(part, p.slots, D, K, dw,
                                                                                        dbias);
  if ((r = launch_status("short_conv_backward sums launch")) != SDM_OK) return r;
  return ok();
}

}  // extern "C"
