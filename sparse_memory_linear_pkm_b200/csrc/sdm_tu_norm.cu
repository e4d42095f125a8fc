// Entry points and launches of the RMS norm with the residual's addition, its
// 8-bit outputs and its gradient.

#include <algorithm>

#include "sdm_check.h"
#include "sdm_norm.cuh"

namespace sdm_host {

using sdm::bf16;

namespace {

// Threads per row and block size. A row of up to 512 values takes a power-of-two
// part of a warp (several rows a block, no block barrier); a longer one a block.
struct NormPlan {
  bool block;
  int width;  // neighbouring values of a memory access: the widest that rows are whole units of
  int tpr, threads, rpb;
};
NormPlan norm_plan(int32_t d) {
  NormPlan p;
  const int need = (d + 8 * sdm::kNormV - 1) / (8 * sdm::kNormV);
  p.width = d % 8 == 0 ? 8 : (d % 4 == 0 ? 4 : (d % 2 == 0 ? 2 : 1));
  p.block = need > 32;
  if (p.block) {
    p.tpr = (need + 31) / 32 * 32;
    p.threads = p.tpr;
    p.rpb = 1;
  } else {
    p.tpr = 1;
    while (p.tpr < need) p.tpr *= 2;
    if (d % 16 == 0 && p.tpr < 2) p.tpr = 2;  // an 8-bit block is two threads' halves
    p.threads = 128;
    p.rpb = p.threads / p.tpr;
  }
  return p;
}

// Blocks of a launch: as many as the rows need, at most what `per_sm` threads
// on every SM hold (the blocks then loop over the rows).
unsigned norm_grid(const NormPlan& p, int64_t n_rows, int sms, int per_sm) {
  const int64_t need = (n_rows + p.rpb - 1) / p.rpb;
  return static_cast<unsigned>(std::min<int64_t>(need, static_cast<int64_t>(sms) * std::max(1, per_sm / p.threads)));
}

// Threads of the gradient an SM is given: its blocks walk the rows. The kernels for
// a row a block, and those for short rows of whole 16-byte units, take at most 128
// registers, so that all are resident. Short rows of narrower units take 135 to
// 160: an SM holds 384 threads of them, and they run 1.3 waves (65,536 x 500 in
// bf16: 139 us).
constexpr int kGradThreadsPerSm = 512;
constexpr size_t kPlainSmem = 40 * 1024;  // dynamic shared memory beside a little static that needs no attribute

sdm_status_t check_norm(int64_t n_rows, int32_t d, float eps) {
  if (n_rows < 0) return fail(SDM_ERR_INVALID_ARGUMENT, "n_rows must be >= 0");
  if (d < 1) return fail(SDM_ERR_INVALID_ARGUMENT, "d must be >= 1");
  if (d > sdm::kNormMaxD)
    return fail(SDM_ERR_UNSUPPORTED, "d above " + std::to_string(sdm::kNormMaxD));
  if (!(eps >= 0.0f) || eps > 1e30f) return fail(SDM_ERR_INVALID_ARGUMENT, "eps must be finite and >= 0");
  return SDM_OK;
}

// An input that an output may take the place of: nothing to check where it does,
// value for value (a thread reads its values of a row before it writes them).
Piece unless_same(const Piece& in, int32_t in_dtype, const void* out, int32_t out_dtype) {
  return in.p == out && in_dtype == out_dtype ? Piece{in.name, nullptr, 0} : in;
}

template <typename Tx, typename Tr, int kOut, int kW>
void launch_norm_width(const NormPlan& p, unsigned grid, const sdm::NormArgs& a, cudaStream_t st) {
  if (p.block) sdm::k_rmsnorm_residual<Tx, Tr, kOut, true, kW><<<grid, p.threads, 0, st>>>(a);
  else sdm::k_rmsnorm_residual<Tx, Tr, kOut, false, kW><<<grid, p.threads, 0, st>>>(a);
}

template <typename Tx, typename Tr, int kOut>
void launch_norm(const NormPlan& p, unsigned grid, const sdm::NormArgs& a, cudaStream_t st) {
  if (kOut >= sdm::kNormFp8Blk || p.width == 8) {
    launch_norm_width<Tx, Tr, kOut, 8>(p, grid, a, st);
  } else if constexpr (kOut < sdm::kNormFp8Blk) {
    if (p.width == 4) launch_norm_width<Tx, Tr, kOut, 4>(p, grid, a, st);
    else if (p.width == 2) launch_norm_width<Tx, Tr, kOut, 2>(p, grid, a, st);
    else launch_norm_width<Tx, Tr, kOut, 1>(p, grid, a, st);
  }
}

template <typename Tx, typename Tr>
void launch_norm_out(int out, const NormPlan& p, unsigned grid, const sdm::NormArgs& a, cudaStream_t st) {
  switch (out) {
    case sdm::kNormF32: launch_norm<Tx, Tr, sdm::kNormF32>(p, grid, a, st); break;
    case sdm::kNormBf16: launch_norm<Tx, Tr, sdm::kNormBf16>(p, grid, a, st); break;
    case sdm::kNormFp8Blk: launch_norm<Tx, Tr, sdm::kNormFp8Blk>(p, grid, a, st); break;
    default: launch_norm<Tx, Tr, sdm::kNormFp8Row>(p, grid, a, st); break;
  }
}

template <typename T, typename Tdy, int kW>
void launch_norm_grad_width(const NormPlan& p, unsigned grid, const sdm::NormGradArgs& a, cudaStream_t st) {
  if (p.block) {
    const auto kern = sdm::k_rmsnorm_residual_backward<T, Tdy, true, kW>;
    const size_t smem = kW == 8 ? 2 * sdm::kNormGradRowBytes<T, Tdy> * static_cast<size_t>(p.threads) : 0;
    if (smem > kPlainSmem) set_smem(reinterpret_cast<const void*>(kern), smem);
    kern<<<grid, p.threads, smem, st>>>(a);
    return;
  }
  sdm::k_rmsnorm_residual_backward<T, Tdy, false, kW><<<grid, p.threads, 0, st>>>(a);
}

template <typename T, typename Tdy>
void launch_norm_grad(const NormPlan& p, unsigned grid, const sdm::NormGradArgs& a, cudaStream_t st) {
  switch (p.width) {
    case 8: launch_norm_grad_width<T, Tdy, 8>(p, grid, a, st); break;
    case 4: launch_norm_grad_width<T, Tdy, 4>(p, grid, a, st); break;
    case 2: launch_norm_grad_width<T, Tdy, 2>(p, grid, a, st); break;
    default: launch_norm_grad_width<T, Tdy, 1>(p, grid, a, st); break;
  }
}

template <bool kBlocks>
sdm_status_t dequantize(const uint8_t* codes, const void* scales, int64_t units, int units_per_row, void* out,
                        int32_t out_dtype, void* stream) {
  sdm_status_t r;
  DeviceInfo* dev;
  if ((r = device_info(&dev)) != SDM_OK) return r;
  const unsigned grid =
      static_cast<unsigned>(std::min<int64_t>((units + 255) / 256, static_cast<int64_t>(dev->sms) * 64));
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (out_dtype == SDM_BF16)
    sdm::k_dequantize_fp8<bf16, kBlocks><<<grid, 256, 0, st>>>(codes, scales, units, units_per_row,
                                                               static_cast<bf16*>(out));
  else
    sdm::k_dequantize_fp8<float, kBlocks><<<grid, 256, 0, st>>>(codes, scales, units, units_per_row,
                                                                static_cast<float*>(out));
  if ((r = launch_status("dequantize launch")) != SDM_OK) return r;
  return ok();
}

}  // namespace

}  // namespace sdm_host

using namespace sdm_host;

extern "C" {

sdm_status_t sdm_rmsnorm_residual(const void* x, int32_t x_dtype, const void* residual, int32_t res_dtype,
                                  const void* w, int32_t w_dtype, int64_t n_rows, int32_t d, float eps, void* h,
                                  void* y, int32_t y_dtype, void* scales, void* stream) {
  sdm_status_t r;
  if ((r = check_norm(n_rows, d, eps)) || (r = check_dtype(x_dtype, "x_dtype")) ||
      (r = check_dtype(w_dtype, "w_dtype")))
    return r;
  const bool any = n_rows > 0, res = residual != nullptr;
  if (res && (r = check_dtype(res_dtype, "res_dtype"))) return r;
  if (y_dtype < SDM_F32 || y_dtype > SDM_FP8_ROW)
    return fail(SDM_ERR_INVALID_ARGUMENT, "y_dtype is not SDM_F32, SDM_BF16, SDM_FP8_B16 or SDM_FP8_ROW");
  const bool fp8 = y_dtype >= SDM_FP8_B16;
  if (fp8 && d % 16 != 0) return fail(SDM_ERR_INVALID_ARGUMENT, "an 8-bit output needs d a multiple of 16");
  if ((r = need_ptr(x, "x", any)) || (r = need_ptr(w, "w", any)) || (r = need_ptr(residual, "residual", any && res)) ||
      (r = need_ptr(h, "h", any && res)) || (r = need_ptr(y, "y", any)))
    return r;
  if (any && fp8 && scales == nullptr) return fail(SDM_ERR_INVALID_ARGUMENT, "scales is NULL");
  if (any && y_dtype == SDM_FP8_ROW && reinterpret_cast<uintptr_t>(scales) % 4 != 0)
    return fail(SDM_ERR_INVALID_ARGUMENT, "scales is not aligned to its element size");
  if (!any) return ok();
  const size_t n = static_cast<size_t>(n_rows) * d;
  const Piece in_x{"x", x, n * in_size(x_dtype)}, in_r{"residual", residual, n * in_size(res_dtype)};
  const Piece in_w{"w", w, d * in_size(w_dtype)};
  const Piece out_h{"h", res ? h : nullptr, n * in_size(res_dtype)}, out_y{"y", y, fp8 ? n : n * in_size(y_dtype)};
  const Piece out_s{"scales", fp8 ? scales : nullptr,
                    y_dtype == SDM_FP8_ROW ? static_cast<size_t>(n_rows) * sizeof(float) : n / 16};
  const Piece outs[] = {out_h, out_y, out_s}, fixed[] = {in_w};
  const Piece for_h[] = {unless_same(in_x, x_dtype, h, res_dtype), unless_same(in_r, res_dtype, h, res_dtype)};
  const Piece for_y[] = {unless_same(in_x, x_dtype, y, y_dtype), unless_same(in_r, res_dtype, y, y_dtype)};
  const Piece for_s[] = {in_x, in_r};
  if ((r = check_apart(&out_h, 1, for_h, 2)) || (r = check_apart(&out_y, 1, for_y, 2)) ||
      (r = check_apart(&out_s, 1, for_s, 2)) || (r = check_apart(outs, 3, fixed, 1)))
    return r;
  DeviceInfo* dev;
  if ((r = device_info(&dev)) != SDM_OK) return r;
  const NormPlan p = norm_plan(d);
  const sdm::NormArgs a{x, residual, w, h, y, scales, n_rows, d, p.tpr, w_dtype == SDM_BF16, eps};
  const unsigned grid = norm_grid(p, n_rows, dev->sms, 4096);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool rb = res ? res_dtype == SDM_BF16 : true;
  if (x_dtype == SDM_BF16) {
    if (rb) launch_norm_out<bf16, bf16>(y_dtype, p, grid, a, st);
    else launch_norm_out<bf16, float>(y_dtype, p, grid, a, st);
  } else {
    if (rb) launch_norm_out<float, bf16>(y_dtype, p, grid, a, st);
    else launch_norm_out<float, float>(y_dtype, p, grid, a, st);
  }
  if ((r = launch_status("rmsnorm_residual launch")) != SDM_OK) return r;
  return ok();
}

sdm_status_t sdm_dequantize_fp8blk(const uint8_t* codes, const int8_t* exps, int64_t n_blocks, void* out,
                                   int32_t out_dtype, void* stream) {
  sdm_status_t r;
  if (n_blocks < 0) return fail(SDM_ERR_INVALID_ARGUMENT, "n_blocks must be >= 0");
  if ((r = check_dtype(out_dtype, "out_dtype")) != SDM_OK) return r;
  const bool any = n_blocks > 0;
  if ((r = need_ptr(codes, "codes", any)) || (r = need_ptr(out, "out", any))) return r;
  if (any && exps == nullptr) return fail(SDM_ERR_INVALID_ARGUMENT, "exps is NULL");
  if (!any) return ok();
  const size_t n = static_cast<size_t>(n_blocks) * 16;
  const Piece ins[] = {{"codes", codes, n}, {"exps", exps, n / 16}}, outs[] = {{"out", out, n * in_size(out_dtype)}};
  if ((r = check_apart(outs, 1, ins, 2)) != SDM_OK) return r;
  return dequantize<true>(codes, exps, 2 * n_blocks, 2, out, out_dtype, stream);
}

sdm_status_t sdm_dequantize_fp8row(const uint8_t* codes, const float* scales, int64_t n_rows, int32_t d, void* out,
                                   int32_t out_dtype, void* stream) {
  sdm_status_t r;
  if (n_rows < 0) return fail(SDM_ERR_INVALID_ARGUMENT, "n_rows must be >= 0");
  if (d < 16 || d % 16 != 0) return fail(SDM_ERR_INVALID_ARGUMENT, "d must be a multiple of 16");
  if ((r = check_dtype(out_dtype, "out_dtype")) != SDM_OK) return r;
  const bool any = n_rows > 0;
  if ((r = need_ptr(codes, "codes", any)) || (r = need_gate(scales, "scales", any, SDM_F32)) ||
      (r = need_ptr(out, "out", any)))
    return r;
  if (!any) return ok();
  const size_t rows = static_cast<size_t>(n_rows), n = rows * d;
  const Piece ins[] = {{"codes", codes, n}, {"scales", scales, rows * sizeof(float)}};
  const Piece outs[] = {{"out", out, n * in_size(out_dtype)}};
  if ((r = check_apart(outs, 1, ins, 2)) != SDM_OK) return r;
  return dequantize<false>(codes, scales, n_rows * (d / 8), d / 8, out, out_dtype, stream);
}

size_t sdm_rmsnorm_residual_backward_workspace_bytes(int64_t n_rows, int32_t d) {
  if (check_norm(n_rows, d, 0.0f) != SDM_OK) return 0;
  ok();
  if (n_rows == 0) return 0;
  // One slot of d sums per row group of the largest grid of any device (a
  // B200 has 148 SMs; the launch keeps to this many).
  const NormPlan p = norm_plan(d);
  return align256(static_cast<size_t>(norm_grid(p, n_rows, 148, kGradThreadsPerSm)) * p.rpb * d * sizeof(float));
}

sdm_status_t sdm_rmsnorm_residual_backward(const void* h, int32_t h_dtype, const void* w, int32_t w_dtype,
                                           const void* dy, int32_t dy_dtype, const void* dh, int64_t n_rows,
                                           int32_t d, float eps, void* dx, float* dw, void* workspace,
                                           size_t workspace_bytes, void* stream) {
  sdm_status_t r;
  if ((r = check_norm(n_rows, d, eps)) || (r = check_dtype(h_dtype, "h_dtype")) ||
      (r = check_dtype(w_dtype, "w_dtype")) || (r = check_dtype(dy_dtype, "dy_dtype")))
    return r;
  const bool any = n_rows > 0;
  if ((r = need_ptr(dw, "dw", true)) || (r = need_ptr(h, "h", any)) || (r = need_ptr(w, "w", any)) ||
      (r = need_ptr(dy, "dy", any)) || (r = need_ptr(dh, "dh", any && dh != nullptr)) || (r = need_ptr(dx, "dx", any)))
    return r;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (!any) {
    if (cudaMemsetAsync(dw, 0, static_cast<size_t>(d) * sizeof(float), st) != cudaSuccess)
      return launch_status("dw clear");
    return ok();
  }
  if ((r = need_ptr(workspace, "workspace", true)) != SDM_OK) return r;
  if (workspace_bytes < sdm_rmsnorm_residual_backward_workspace_bytes(n_rows, d))
    return fail(SDM_ERR_INVALID_ARGUMENT, "workspace is smaller than sdm_rmsnorm_residual_backward_workspace_bytes");
  const size_t n = static_cast<size_t>(n_rows) * d;
  const Piece in_h{"h", h, n * in_size(h_dtype)}, in_dy{"dy", dy, n * in_size(dy_dtype)};
  const Piece in_dh{"dh", dh, n * in_size(h_dtype)}, in_w{"w", w, d * in_size(w_dtype)};
  const Piece outs[] = {{"dx", dx, n * in_size(h_dtype)}, {"dw", dw, d * sizeof(float)}};
  const Piece for_dx[] = {unless_same(in_h, h_dtype, dx, h_dtype), unless_same(in_dy, dy_dtype, dx, h_dtype),
                          unless_same(in_dh, h_dtype, dx, h_dtype), in_w};
  const Piece for_dw[] = {in_h, in_dy, in_dh, in_w};
  if ((r = check_apart(outs, 1, for_dx, 4)) || (r = check_apart(outs + 1, 1, for_dw, 4)) ||
      (r = check_apart(outs, 2, nullptr, 0)))
    return r;
  const NormPlan p = norm_plan(d);
  const unsigned grid = norm_grid(p, n_rows, 148, kGradThreadsPerSm);
  float* part = static_cast<float*>(workspace);
  const sdm::NormGradArgs a{h, w, dy, dh, dx, part, n_rows, d, p.tpr, w_dtype == SDM_BF16, eps};
  if (h_dtype == SDM_BF16) {
    if (dy_dtype == SDM_BF16) launch_norm_grad<bf16, bf16>(p, grid, a, st);
    else launch_norm_grad<bf16, float>(p, grid, a, st);
  } else {
    if (dy_dtype == SDM_BF16) launch_norm_grad<float, bf16>(p, grid, a, st);
    else launch_norm_grad<float, float>(p, grid, a, st);
  }
  if ((r = launch_status("rmsnorm_residual_backward launch")) != SDM_OK) return r;
  sdm::k_sum_slots<<<(d + 31) / 32, dim3(32, 32), 0, st>>>(part, static_cast<int64_t>(grid) * p.rpb, d, dw);
  if ((r = launch_status("dw sum launch")) != SDM_OK) return r;
  return ok();
}

}  // extern "C"
