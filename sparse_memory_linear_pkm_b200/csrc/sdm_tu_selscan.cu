// Entry point and launches of the selective state space scan.

#include "sdm_selscan_host.h"

namespace sdm_host {

namespace {

// Tokens a sequence may have for the kernel that keeps nothing but the state's
// four values per thread: there its tokens are a serial chain of loads.
constexpr int kStepTokens = 4;

struct SelPlan {
  bool step = false, one_pass = false;
  int ch = 0;               // channels of a block
  int splits = 1, tokens_per_split = 0;
  size_t state_bytes = 0;   // one [B, splits, D, N] fp32 array
};

// Three ways, by how many channels there are to fill 148 SMs with:
//   - many (W = 1): a block takes 64-odd channels and walks the tokens once;
//   - few (W = 8): a block takes an eighth of that and eight warps share the
//     tokens of a tile, at the cost of a second run over each segment;
//   - very few, and a long sequence: the token axis is split over blocks as
//     well, whose maps are joined in between (each exponential twice).
SelPlan sel_plan(const sdm_selscan_shape_t& s) {
  SelPlan p;
  if (s.T <= kStepTokens) {
    p.step = true;
    return p;
  }
  const int L = sel_lanes(s.N), dg = s.D / s.G;
  auto blocks = [&](int ch) { return static_cast<int64_t>(s.B) * s.G * ceil_div(dg, ch); };
  const int wide = 32 / L * kWideGroups, narrow = 32 / L * kTileGroups;
  p.one_pass = blocks(wide) >= 4 * kSms;
  p.ch = p.one_pass ? wide : narrow;
  p.tokens_per_split = s.T;
  if (!p.one_pass) {
    const int64_t base = blocks(narrow);
    const int tiles = static_cast<int>(ceil_div(s.T, kTileTokens));
    const int64_t want = base <= kSms / 4 ? std::min<int64_t>(kSms / base, tiles / 4) : 1;
    if (want > 1) {
      p.tokens_per_split = static_cast<int>(ceil_div(tiles, want)) * kTileTokens;
      p.splits = static_cast<int>(ceil_div(s.T, p.tokens_per_split));
      p.state_bytes = align256(static_cast<size_t>(s.B) * p.splits * s.D * s.N * sizeof(float));
    }
  }
  return p;
}

template <typename T, int L>
sdm_status_t launch_scan_lanes(const SelPlan& p, sdm::SelScanArgs a, int B, const float* h0, float* ws,
                               cudaStream_t st) {
  if (p.step) {
    const int64_t channels = static_cast<int64_t>(B) * a.D;
    sdm::k_selective_scan_step<T, L><<<static_cast<unsigned>(ceil_div(channels * L, 256)), 256, 0, st>>>(a, channels);
    return launch_status("selective_scan step launch");
  }
  if (p.one_pass) {
    launch_sel<T, L, kSegTokens, 1, kWideGroups, sdm::kSelRun>(a, B, st);
    return launch_status("selective_scan launch");
  }
  if (p.splits > 1) {
    sdm::SelScanArgs m = a;
    m.h_in = nullptr;
    m.sums = ws;
    launch_sel<T, L, kSegTokens, kTileWarps, kTileGroups, sdm::kSelSums>(m, B, st);
    const int64_t per_b = static_cast<int64_t>(a.D) * a.N, total = per_b * B;
    float* H = ws + static_cast<int64_t>(B) * a.splits * per_b;
    sdm::k_selective_scan_join<<<static_cast<unsigned>(ceil_div(total, 256)), 256, 0, st>>>(ws, H, h0, per_b,
                                                                                           a.splits, total);
    a.h_in = H;
    a.in_splits = 1;
  }
  launch_sel<T, L, kSegTokens, kTileWarps, kTileGroups, sdm::kSelRun>(a, B, st);
  return launch_status("selective_scan launch");
}

template <typename T>
sdm_status_t launch_scan(int L, const SelPlan& p, const sdm::SelScanArgs& a, int B, const float* h0, float* ws,
                         cudaStream_t st) {
  switch (L) {
    case 2: return launch_scan_lanes<T, 2>(p, a, B, h0, ws, st);
    case 4: return launch_scan_lanes<T, 4>(p, a, B, h0, ws, st);
    case 8: return launch_scan_lanes<T, 8>(p, a, B, h0, ws, st);
    default: return launch_scan_lanes<T, 16>(p, a, B, h0, ws, st);
  }
}

}  // namespace

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
  // Block numbers along the channels are 32-bit, and so is a thread's channel.
  if (static_cast<int64_t>(s->D) * s->B > (int64_t{1} << 34)) return fail(SDM_ERR_UNSUPPORTED, "B * D above 2^34");
  return SDM_OK;
}

// The kernels' view of a call's inputs.
sdm::SelScanArgs selscan_args(const sdm_selscan_shape_t& s, const void* x, const void* dt, const float* A,
                              const void* Bm, const void* Cm, const float* Dskip, const void* z,
                              const float* dt_bias, const int32_t* lengths, unsigned* err) {
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
  a.err = err;
  // Rows read in units of four: address, stride and the group's first channel
  // (and state) on whole units.
  const size_t unit = 4 * in_size(s.in_dtype);
  auto whole = [&](const void* p, int64_t stride) {
    return reinterpret_cast<uintptr_t>(p) % unit == 0 && stride % 4 == 0;
  };
  a.vec_x = (s.D / s.G) % 4 == 0 && whole(x, a.x_stride) && whole(dt, a.dt_stride) &&
            (z == nullptr || whole(z, a.z_stride));
  a.vec_b = s.N % 4 == 0 && whole(Bm, a.b_stride) && whole(Cm, a.c_stride);
  return a;
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
  if (!any) {
    if (state && hT != nullptr && hT != h0) {
      const size_t n = static_cast<size_t>(s.B) * s.D * s.N * sizeof(float);
      const cudaError_t e = h0 != nullptr ? cudaMemcpyAsync(hT, h0, n, cudaMemcpyDeviceToDevice, st)
                                          : cudaMemsetAsync(hT, 0, n, st);
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
  DeviceInfo* dev;
  if ((r = device_info(&dev)) != SDM_OK) return r;
  sdm::SelScanArgs a = selscan_args(s, x, dt, A, Bm, Cm, Dskip, z, dt_bias, lengths, dev->err);
  a.h_in = h0;
  a.h_out = hT;
  a.y = y;
  if (!p.step) {
    a.tiles_per_group = static_cast<int>(ceil_div(s.D / s.G, p.ch));
    a.splits = p.splits;
    a.tokens_per_split = p.tokens_per_split;
  }
  const int L = sel_lanes(s.N);
  float* ws = static_cast<float*>(workspace);
  r = s.in_dtype == SDM_BF16 ? launch_scan<bf16>(L, p, a, s.B, h0, ws, st) : launch_scan<float>(L, p, a, s.B, h0, ws, st);
  if (r != SDM_OK) return r;
  return ok();
}

}  // extern "C"
