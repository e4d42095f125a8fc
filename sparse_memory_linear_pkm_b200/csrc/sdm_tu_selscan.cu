// Entry point and launches of the selective state space scan.

#include "sdm_selscan_host.h"

namespace sdm_host {

namespace {

// Tokens a sequence may have for the kernel without shared memory: there each
// token waits for its own loads.
constexpr int kStepTokens = 4;
// The token axis is split until there are so many warps an SM, while a split
// keeps so many tokens. A split costs the time of some ten tokens for its map and
// an unhidden start of its loads, so that short ones pay only where there are few
// warps. Measured in bf16 with N = 16: 64 warps instead of 32, 65,536 x 2048 1385
// -> 1341 us; 64 tokens instead of 128, 1000 x 4096 73 -> 60; 32 tokens instead of
// 64, 384 x 1024 29 -> 20. 64 tokens up to 48 warps: 8192 x 1536 147 -> 155; 32
// tokens up to 48 warps: 4096 x 2048 103 -> 110.
struct SelSplit { int warps, tokens; };
constexpr SelSplit kSelSplits[] = {{64, 128}, {32, 64}, {16, 32}};

struct SelPlan {
  bool step = false;
  int splits = 1, tokens_per_split = 0;
  size_t state_bytes = 0;  // one [B, splits, D, N] fp32 array
};

// Splitting makes every exponential twice, so it pays where the channels leave
// most of the device idle: with w warps an SM one pass takes about 0.95 / w
// clocks per exponential (0.35 at 2.6, 0.143 at 6.9), two take 0.17 to 0.19 once
// some 30 warps an SM are there. At 4.3 warps (B = 5, T = 4096, D = 4096): one
// pass 1068 us, two 871; at 5.2 (B = 6) 1078 and 1028; at 6 and above one pass.
SelPlan sel_plan(const sdm_selscan_shape_t& s) {
  SelPlan p;
  p.step = s.T <= kStepTokens;
  p.tokens_per_split = s.T;
  if (p.step) return p;
  const int64_t warps =
      static_cast<int64_t>(s.B) * s.G * ceil_div(s.D / s.G, sel_channels(s.N)) * (sdm::kSelThreads / 32);
  if (warps >= 6 * kSms) return p;
  int64_t splits = 0;
  for (const SelSplit& l : kSelSplits)
    splits = std::max(splits, std::min<int64_t>(l.warps * kSms / warps, s.T / l.tokens));
  if (splits < 4) return p;
  const int tile = sdm::kSelTile;
  p.tokens_per_split = static_cast<int>(ceil_div(ceil_div(s.T, splits), tile) * tile);
  p.splits = static_cast<int>(ceil_div(s.T, p.tokens_per_split));
  p.state_bytes = align256(static_cast<size_t>(s.B) * p.splits * s.D * s.N * sizeof(float));
  return p;
}

template <typename T, int kMode>
void launch_sel(const sdm::SelScanArgs& a, int B, cudaStream_t st) {
  const dim3 grid(static_cast<unsigned>(a.tiles_per_group) * a.G, a.splits, B);
  if (a.N <= 8) sdm::k_selective_scan<T, 8, 1, kMode><<<grid, sdm::kSelThreads, 0, st>>>(a);
  else if (a.N <= 16) sdm::k_selective_scan<T, 16, 1, kMode><<<grid, sdm::kSelThreads, 0, st>>>(a);
  else if (a.N <= 32) sdm::k_selective_scan<T, 16, 2, kMode><<<grid, sdm::kSelThreads, 0, st>>>(a);
  else sdm::k_selective_scan<T, 16, 4, kMode><<<grid, sdm::kSelThreads, 0, st>>>(a);
}

template <typename T>
void launch_step(const sdm::SelScanArgs& a, int B, cudaStream_t st) {
  const int threads = sdm::kStepThreads;
  auto grid = [&](int lanes) {
    return dim3(static_cast<unsigned>(ceil_div(static_cast<int64_t>(a.D) * lanes, threads)), B);
  };
  if (a.N <= 8) sdm::k_selective_scan_step<T, 8, 1><<<grid(1), threads, 0, st>>>(a);
  else if (a.N <= 16) sdm::k_selective_scan_step<T, 8, 2><<<grid(2), threads, 0, st>>>(a);
  else if (a.N <= 32) sdm::k_selective_scan_step<T, 8, 4><<<grid(4), threads, 0, st>>>(a);
  else sdm::k_selective_scan_step<T, 8, 8><<<grid(8), threads, 0, st>>>(a);
}

}  // namespace

sdm_status_t launch_sel_run(int32_t in_dtype, const sdm::SelScanArgs& a, int B, cudaStream_t st) {
  if (in_dtype == SDM_BF16) launch_sel<bf16, sdm::kSelRun>(a, B, st);
  else launch_sel<float, sdm::kSelRun>(a, B, st);
  return launch_status("selective_scan launch");
}

sdm_status_t launch_sel_states(int32_t in_dtype, sdm::SelScanArgs a, int B, const float* h0, float* ws,
                               cudaStream_t st) {
  a.h_in = nullptr;
  a.in_splits = 0;
  a.h_out = nullptr;
  a.sums = ws;
  if (in_dtype == SDM_BF16) launch_sel<bf16, sdm::kSelSums>(a, B, st);
  else launch_sel<float, sdm::kSelSums>(a, B, st);
  const int64_t per_b = static_cast<int64_t>(a.D) * a.N, total = per_b * B;
  sdm::k_selective_scan_join<<<static_cast<unsigned>(ceil_div(total, 256)), 256, 0, st>>>(
      ws, ws + total * a.splits, h0, per_b, a.splits, total);
  return launch_status("selective_scan state launch");
}

sdm_status_t check_selscan(const sdm_selscan_shape_t* s) {
  if (s == nullptr) return fail(SDM_ERR_INVALID_ARGUMENT, "shape is NULL");
  if (s->B < 0 || s->T < 0 || s->D < 0) return fail(SDM_ERR_INVALID_ARGUMENT, "B, T and D must be >= 0");
  if (s->N < 1 || s->N > 64) return fail(SDM_ERR_INVALID_ARGUMENT, "N must be in [1, 64], got " + std::to_string(s->N));
  if (s->G < 1 || s->D % s->G != 0) return fail(SDM_ERR_INVALID_ARGUMENT, "G must be >= 1 and divide D");
  sdm_status_t r;
  if ((r = check_dtype(s->in_dtype, "in_dtype")) != SDM_OK) return r;
  if (s->reserved != 0) return fail(SDM_ERR_INVALID_ARGUMENT, "reserved must be 0");
  const int64_t gn = static_cast<int64_t>(s->G) * s->N;
  if ((s->x_stride != 0 && s->x_stride < s->D) || (s->dt_stride != 0 && s->dt_stride < s->D) ||
      (s->z_stride != 0 && s->z_stride < s->D))
    return fail(SDM_ERR_INVALID_ARGUMENT, "x_stride, dt_stride and z_stride must be 0 or at least D");
  if ((s->b_stride != 0 && s->b_stride < gn) || (s->c_stride != 0 && s->c_stride < gn))
    return fail(SDM_ERR_INVALID_ARGUMENT, "b_stride and c_stride must be 0 or at least G * N");
  if (s->B > 65535) return fail(SDM_ERR_UNSUPPORTED, "B above 65535");
  if (s->T > INT32_MAX - 4096) return fail(SDM_ERR_UNSUPPORTED, "T above 2^31 - 4096");
  // Thread numbers along the channels are 32-bit (8 lanes a channel at most).
  if (s->D > (1 << 26)) return fail(SDM_ERR_UNSUPPORTED, "D above 2^26");
  return SDM_OK;
}

// The kernels' view of a call's inputs.
sdm::SelScanArgs selscan_args(const sdm_selscan_shape_t& s, const void* x, const void* dt, const float* A,
                              const void* Bm, const void* Cm, const float* Dskip, const void* z,
                              const float* dt_bias, const int32_t* lengths) {
  sdm::SelScanArgs a{};
  a.x = x; a.dt = dt; a.A = A; a.Bm = Bm; a.Cm = Cm; a.Dskip = Dskip; a.z = z; a.bias = dt_bias;
  a.lengths = lengths;
  const int64_t gn = static_cast<int64_t>(s.G) * s.N;
  a.x_stride = s.x_stride ? s.x_stride : s.D;
  a.dt_stride = s.dt_stride ? s.dt_stride : s.D;
  a.z_stride = s.z_stride ? s.z_stride : s.D;
  a.b_stride = s.b_stride ? s.b_stride : gn;
  a.c_stride = s.c_stride ? s.c_stride : gn;
  a.T = s.T; a.D = s.D; a.N = s.N; a.G = s.G;
  a.splits = 1;
  a.tokens_per_split = s.T;
  a.softplus = s.softplus != 0;
  const size_t unit = 4 * in_size(s.in_dtype);
  auto whole = [&](const void* p, int64_t stride) {
    return reinterpret_cast<uintptr_t>(p) % unit == 0 && stride % 4 == 0;
  };
  a.vec_b = s.N % 4 == 0 && whole(Bm, a.b_stride) && whole(Cm, a.c_stride);
  return a;
}

SelInputs selscan_inputs(const sdm_selscan_shape_t& s, const sdm::SelScanArgs& a) {
  const size_t es = in_size(s.in_dtype), last = static_cast<size_t>(s.B) * s.T - 1;
  const size_t gn = static_cast<size_t>(s.G) * s.N, d = s.D;
  return {{{"x", a.x, (last * a.x_stride + d) * es},
           {"dt", a.dt, (last * a.dt_stride + d) * es},
           {"z", a.z, (last * a.z_stride + d) * es},
           {"Bm", a.Bm, (last * a.b_stride + gn) * es},
           {"Cm", a.Cm, (last * a.c_stride + gn) * es},
           {"A", a.A, d * s.N * sizeof(float)},
           {"Dskip", a.Dskip, d * sizeof(float)},
           {"dt_bias", a.bias, d * sizeof(float)},
           {"lengths", a.lengths, s.B * sizeof(int32_t)}}};
}

// The pointers that the scan and its gradient share.
sdm_status_t need_selscan(const sdm_selscan_shape_t& s, bool any, const void* x, const void* dt, const float* A,
                          const void* Bm, const void* Cm, const float* Dskip, const void* z, const float* dt_bias,
                          const int32_t* lengths) {
  sdm_status_t r;
  if ((r = need_gate(x, "x", any, s.in_dtype)) || (r = need_gate(dt, "dt", any, s.in_dtype)) ||
      (r = need_ptr(A, "A", any)) || (r = need_gate(Bm, "Bm", any, s.in_dtype)) ||
      (r = need_gate(Cm, "Cm", any, s.in_dtype)) ||
      (r = need_gate(Dskip, "Dskip", any && Dskip != nullptr, SDM_F32)) ||
      (r = need_gate(z, "z", any && z != nullptr, s.in_dtype)) ||
      (r = need_gate(dt_bias, "dt_bias", any && dt_bias != nullptr, SDM_F32)) ||
      (r = need_gate(lengths, "lengths", any && lengths != nullptr, SDM_F32)))
    return r;
  return SDM_OK;
}

}  // namespace sdm_host

using namespace sdm_host;

extern "C" {

size_t sdm_selective_scan_workspace_bytes(const sdm_selscan_shape_t* shape) {
  if (check_selscan(shape) != SDM_OK) return 0;
  ok();
  if (shape->B == 0 || shape->T == 0 || shape->D == 0) return 0;
  return 2 * sel_plan(*shape).state_bytes;
}

sdm_status_t sdm_selective_scan(const sdm_selscan_shape_t* shape, const void* x, const void* dt, const float* A,
                                const void* Bm, const void* Cm, const float* Dskip, const void* z,
                                const float* dt_bias, const int32_t* lengths, const float* h0, float* hT, void* y,
                                void* workspace, size_t workspace_bytes, void* stream) {
  sdm_status_t r;
  if ((r = check_selscan(shape)) != SDM_OK) return r;
  const sdm_selscan_shape_t& s = *shape;
  const bool any = s.B > 0 && s.T > 0 && s.D > 0, state = s.B > 0 && s.D > 0;
  if ((r = need_selscan(s, any, x, dt, A, Bm, Cm, Dskip, z, dt_bias, lengths)) || (r = need_ptr(y, "y", any)) ||
      (r = need_ptr(h0, "h0", state && h0 != nullptr)) || (r = need_ptr(hT, "hT", state && hT != nullptr)))
    return r;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const size_t states = static_cast<size_t>(s.B) * s.D * s.N * sizeof(float);
  const Piece last = {"hT", hT, states}, start = {"h0", hT == h0 ? nullptr : h0, states};
  if (!any) {
    if ((r = check_apart(&last, 1, &start, 1)) != SDM_OK) return r;
    if (state && hT != nullptr && hT != h0) {
      const cudaError_t e = h0 != nullptr ? cudaMemcpyAsync(hT, h0, states, cudaMemcpyDeviceToDevice, st)
                                          : cudaMemsetAsync(hT, 0, states, st);
      if (e != cudaSuccess) return fail(SDM_ERR_CUDA, std::string("state copy: ") + cudaGetErrorString(e));
    }
    return ok();
  }
  const SelPlan p = sel_plan(s);
  if (p.state_bytes > 0) {
    if ((r = need_ptr(workspace, "workspace", true)) != SDM_OK) return r;
    if (workspace_bytes < 2 * p.state_bytes)
      return fail(SDM_ERR_INVALID_ARGUMENT, "workspace is smaller than sdm_selective_scan_workspace_bytes");
  }
  sdm::SelScanArgs a = selscan_args(s, x, dt, A, Bm, Cm, Dskip, z, dt_bias, lengths);
  const SelInputs in = selscan_inputs(s, a);
  const Piece outs[] = {{"y", y, static_cast<size_t>(s.B) * s.T * s.D * in_size(s.in_dtype)}, last};
  if ((r = check_apart(outs, 2, in.piece, kSelInputs)) || (r = check_apart(outs, 2, &start, 1))) return r;
  DeviceInfo* dev;
  if ((r = device_info(&dev)) != SDM_OK) return r;
  a.err = dev->err;
  a.h_in = h0;
  a.h_out = hT;
  a.y = y;
  if (p.step) {
    if (s.in_dtype == SDM_BF16) launch_step<bf16>(a, s.B, st);
    else launch_step<float>(a, s.B, st);
    r = launch_status("selective_scan step launch");
  } else {
    a.tiles_per_group = static_cast<int>(ceil_div(s.D / s.G, sel_channels(s.N)));
    a.splits = p.splits;
    a.tokens_per_split = p.tokens_per_split;
    if (p.splits > 1) {
      float* ws = static_cast<float*>(workspace);
      if ((r = launch_sel_states(s.in_dtype, a, s.B, h0, ws, st)) != SDM_OK) return r;
      a.h_in = ws + static_cast<int64_t>(s.B) * s.D * s.N * p.splits;
      a.in_splits = 1;
    }
    r = launch_sel_run(s.in_dtype, a, s.B, st);
  }
  if (r != SDM_OK) return r;
  return ok();
}

}  // extern "C"
