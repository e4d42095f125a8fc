// Entry point and launches of the global gradient norm and its clipping.

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <new>
#include <vector>

#include "sdm_check.h"
#include "sdm_clip.cuh"

namespace sdm_host {

namespace {

constexpr int kClipBlocks = 148 * sdm::kClipPerSm;  // at most: what the SMs of a B200 hold at once

struct ClipPlan {
  int64_t total = 0;  // values
  int chunk = 0;
  int launches = 0;
};

bool is_dtype(int32_t d) { return d == SDM_F32 || d == SDM_BF16; }

// One entry of the list. Names are put together only for an error: a list has
// hundreds of entries, and the call is to cost little on the host.
sdm_status_t check_tensor(const sdm_grad_tensor_t& t, int i) {
  auto bad = [i](sdm_status_t s, const char* what) {
    return fail(s, "tensors[" + std::to_string(i) + "]" + what);
  };
  if (t.n < 0) return bad(SDM_ERR_INVALID_ARGUMENT, ".n must be >= 0");
  if (t.n > (int64_t{1} << 40)) return bad(SDM_ERR_UNSUPPORTED, ".n above 2^40");
  if (!is_dtype(t.dtype)) return bad(SDM_ERR_INVALID_ARGUMENT, ".dtype is not SDM_F32 or SDM_BF16");
  if (t.n > 0 && t.grad == nullptr) return bad(SDM_ERR_INVALID_ARGUMENT, ".grad is NULL");
  if (reinterpret_cast<uintptr_t>(t.grad) % in_size(t.dtype) != 0)
    return bad(SDM_ERR_INVALID_ARGUMENT, ".grad is not aligned to its element size");
  if (t.out == nullptr) return SDM_OK;
  if (!is_dtype(t.out_dtype)) return bad(SDM_ERR_INVALID_ARGUMENT, ".out_dtype is not SDM_F32 or SDM_BF16");
  if (reinterpret_cast<uintptr_t>(t.out) % in_size(t.out_dtype) != 0)
    return bad(SDM_ERR_INVALID_ARGUMENT, ".out is not aligned to its element size");
  if (t.out == t.grad && t.out_dtype != t.dtype)
    return bad(SDM_ERR_INVALID_ARGUMENT, " is its own output in another type");
  return SDM_OK;
}

// Outputs must not share a byte with another tensor, whichever of the two the
// list names first: the second pass reads and writes in any order. A sweep over
// all pieces by address, with the two furthest ends of pieces so far that belong
// to different tensors (one is always another's), of all pieces and of outputs.
sdm_status_t check_outputs_apart(const sdm_grad_tensor_t* t, int n) try {
  struct Span {
    uintptr_t begin, end;
    int of;
    bool out;
  };
  std::vector<Span> spans;
  spans.reserve(2 * static_cast<size_t>(n));
  for (int i = 0; i < n; ++i) {
    if (t[i].n == 0) continue;
    const uintptr_t g = reinterpret_cast<uintptr_t>(t[i].grad), o = reinterpret_cast<uintptr_t>(t[i].out);
    if (g != o) spans.push_back({g, g + t[i].n * in_size(t[i].dtype), i, false});
    if (o != 0) spans.push_back({o, o + t[i].n * in_size(t[i].out_dtype), i, true});
  }
  std::sort(spans.begin(), spans.end(), [](const Span& a, const Span& b) { return a.begin < b.begin; });
  struct Ends {
    uintptr_t end[2] = {0, 0};
    int of[2] = {-1, -1};
    void add(uintptr_t e, int i) {
      if (i == of[0]) {
        end[0] = std::max(end[0], e);
      } else if (e > end[0]) {
        end[1] = end[0];
        of[1] = of[0];
        end[0] = e;
        of[0] = i;
      } else if (e > end[1]) {
        end[1] = e;
        of[1] = i;
      }
    }
    int other(uintptr_t begin, int i) const {  // a different tensor that reaches past `begin`, or -1
      const int k = of[0] == i ? 1 : 0;
      return of[k] >= 0 && end[k] > begin ? of[k] : -1;
    }
  } any, outs;
  for (const Span& s : spans) {
    const int hit = (s.out ? any : outs).other(s.begin, s.of);
    if (hit >= 0)
      return fail(SDM_ERR_INVALID_ARGUMENT, "tensors[" + std::to_string(std::max(hit, s.of)) + "] and tensors[" +
                                                std::to_string(std::min(hit, s.of)) + "] overlap in an output");
    // A tensor's own output may be its gradient's memory, but not part of it.
    if (s.out && t[s.of].out != t[s.of].grad) {
      const uintptr_t g = reinterpret_cast<uintptr_t>(t[s.of].grad);
      if (g < s.end && s.begin < g + t[s.of].n * in_size(t[s.of].dtype))
        return fail(SDM_ERR_INVALID_ARGUMENT, "tensors[" + std::to_string(s.of) + "].out overlaps its own grad");
    }
    any.add(s.end, s.of);
    if (s.out) outs.add(s.end, s.of);
  }
  return SDM_OK;
} catch (const std::bad_alloc&) {  // nothing is thrown past a C entry point
  return fail(SDM_ERR_UNSUPPORTED, "not enough host memory to check the list");
}

// Chunks small enough that few values still spread over all blocks, and large
// enough that looking up a chunk's tensor costs nothing against its values.
ClipPlan clip_plan(const sdm_grad_tensor_t* t, int32_t n) {
  ClipPlan p;
  for (int i = 0; i < n; ++i) p.total += t[i].n;
  constexpr int64_t unit = sdm::kClipThreads * sdm::kClipVec;
  const int64_t per = (p.total + kClipBlocks - 1) / kClipBlocks;
  p.chunk = static_cast<int>(std::min<int64_t>(std::max<int64_t>((per + unit - 1) / unit, 1) * unit, 16 * unit));
  p.launches = (n + sdm::kClipTensors - 1) / sdm::kClipTensors;
  return p;
}

// The launch's part of the tensors and its number of blocks (0: no values).
int fill_table(const sdm_grad_tensor_t* t, int32_t n, int chunk, sdm::ClipTable* out) {
  int64_t at = 0;
  for (int i = 0; i < n; ++i) {
    out->grad[i] = t[i].grad;
    out->out[i] = t[i].out;
    out->n[i] = t[i].n;
    out->first[i] = static_cast<int32_t>(at);
    out->type[i] = static_cast<uint8_t>((t[i].dtype == SDM_BF16 ? 1 : 0) |
                                        (t[i].out != nullptr && t[i].out_dtype == SDM_BF16 ? 2 : 0));
    at += (t[i].n + chunk - 1) / chunk;
  }
  out->first[n] = static_cast<int32_t>(at);
  out->tensors = n;
  out->chunk = chunk;
  return static_cast<int>(std::min<int64_t>(at, kClipBlocks));
}

}  // namespace

}  // namespace sdm_host

using namespace sdm_host;

extern "C" {

size_t sdm_grad_norm_clip_workspace_bytes(int32_t n_tensors) {
  if (n_tensors < 0) {
    fail(SDM_ERR_INVALID_ARGUMENT, "n_tensors must be >= 0");
    return 0;
  }
  ok();
  const size_t launches = (static_cast<size_t>(n_tensors) + sdm::kClipTensors - 1) / sdm::kClipTensors;
  return align256(std::max<size_t>(launches, 1) * kClipBlocks * sizeof(double));
}

sdm_status_t sdm_grad_norm_clip(const sdm_grad_tensor_t* tensors, int32_t n_tensors, float max_norm, float eps,
                                float* norm, void* workspace, size_t workspace_bytes, void* stream) {
  sdm_status_t r;
  if (n_tensors < 0) return fail(SDM_ERR_INVALID_ARGUMENT, "n_tensors must be >= 0");
  if (n_tensors > 0 && tensors == nullptr) return fail(SDM_ERR_INVALID_ARGUMENT, "tensors is NULL");
  if (!(max_norm >= 0.0f)) return fail(SDM_ERR_INVALID_ARGUMENT, "max_norm must be >= 0");
  if (!(eps >= 0.0f) || std::isinf(eps)) return fail(SDM_ERR_INVALID_ARGUMENT, "eps must be finite and >= 0");
  bool write = false;
  for (int i = 0; i < n_tensors; ++i) {
    const sdm_grad_tensor_t& t = tensors[i];
    if ((r = check_tensor(t, i)) != SDM_OK) return r;
    write |= t.out != nullptr && t.n > 0;
  }
  if (write && (r = check_outputs_apart(tensors, n_tensors)) != SDM_OK) return r;
  if ((r = need_gate(norm, "norm", true, SDM_F32)) != SDM_OK) return r;
  const ClipPlan p = clip_plan(tensors, n_tensors);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (p.total == 0) {
    const cudaError_t e = cudaMemsetAsync(norm, 0, sizeof(float), st);
    return e == cudaSuccess ? ok() : fail(SDM_ERR_CUDA, std::string("empty norm: ") + cudaGetErrorString(e));
  }
  if (p.total / p.chunk + n_tensors > INT32_MAX) return fail(SDM_ERR_UNSUPPORTED, "too many values");
  if ((r = need_ptr(workspace, "workspace", true)) != SDM_OK) return r;
  if (workspace_bytes < sdm_grad_norm_clip_workspace_bytes(n_tensors))
    return fail(SDM_ERR_INVALID_ARGUMENT, "workspace is smaller than sdm_grad_norm_clip_workspace_bytes");
  // The second pass writes the norm while it reads gradients and writes outputs.
  const Piece own{"norm", norm, sizeof(float)};
  for (int i = 0; i < n_tensors; ++i) {
    const sdm_grad_tensor_t& t = tensors[i];
    const size_t n = static_cast<size_t>(t.n);
    if (overlap(own, {"grad", t.grad, n * in_size(t.dtype)}) || overlap(own, {"out", t.out, n * in_size(t.out_dtype)}))
      return fail(SDM_ERR_INVALID_ARGUMENT, "norm overlaps tensors[" + std::to_string(i) + "]");
  }
  double* slots = static_cast<double*>(workspace);
  sdm::ClipTable table;
  int n_slots = 0;
  for (int l = 0; l < p.launches; ++l) {
    const int first = l * sdm::kClipTensors, n = std::min(n_tensors - first, sdm::kClipTensors);
    const int blocks = fill_table(tensors + first, n, p.chunk, &table);
    if (blocks == 0) continue;
    sdm::k_grad_norm<<<blocks, sdm::kClipThreads, 0, st>>>(table, slots + n_slots);
    n_slots += blocks;
  }
  if ((r = launch_status("grad_norm launch")) != SDM_OK) return r;
  bool told = false;
  for (int l = 0; l < p.launches; ++l) {
    const int first = l * sdm::kClipTensors, n = std::min(n_tensors - first, sdm::kClipTensors);
    if (p.launches > 1) fill_table(tensors + first, n, p.chunk, &table);
    int blocks = std::min(table.first[n], kClipBlocks);
    if (!write) {  // only the norm is wanted: no chunks
      table.first[n] = 0;
      blocks = 1;
    }
    if (blocks == 0) continue;
    sdm::k_grad_clip<<<blocks, sdm::kClipThreads, 0, st>>>(table, slots, n_slots, max_norm, eps,
                                                           told ? nullptr : norm);
    told = true;
    if (!write) break;
  }
  if ((r = launch_status("grad_clip launch")) != SDM_OK) return r;
  return ok();
}

}  // extern "C"
