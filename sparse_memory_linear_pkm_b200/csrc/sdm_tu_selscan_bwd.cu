// Entry point and launches of the selective scan's gradient.

#include "sdm_selscan_bwd.cuh"
#include "sdm_selscan_host.h"

namespace sdm_host {

namespace {

// A gradient block: 64 tokens by 2 channel groups. Segments of 8 tokens (their
// exponentials and states are 64 registers); the 16 lanes of a wide channel
// exchange 16 tokens' sums at a time, so those take segments of 16.
constexpr int kGradTokens = 64, kGradGroups = 2;
template <int L>
constexpr int kGradSegment = L == 16 ? 16 : 8;

struct SelGradPlan {
  int ch = 0, tiles = 0, tiles_per_group = 0;
  size_t ckpt = 0, part_bc = 0, part_A = 0, part_D = 0;
  size_t total() const { return ckpt + 2 * part_bc + part_A + 2 * part_D; }
};

// Lanes of a channel in the gradient: four states a lane, two lanes at least.
int grad_lanes(int32_t N) {
  int L = 2;
  while (4 * L < N) L *= 2;
  return L;
}

SelGradPlan sel_grad_plan(const sdm_selscan_shape_t& s) {
  SelGradPlan p;
  p.ch = 32 / grad_lanes(s.N) * kGradGroups;
  p.tiles = static_cast<int>(ceil_div(s.T, kGradTokens));
  p.tiles_per_group = static_cast<int>(ceil_div(s.D / s.G, p.ch));
  const size_t f = sizeof(float);
  p.ckpt = align256(2 * static_cast<size_t>(s.B) * p.tiles * s.D * s.N * f);  // decays, states
  p.part_bc = align256(static_cast<size_t>(p.tiles_per_group) * s.B * s.T * s.G * s.N * f);
  p.part_A = align256(static_cast<size_t>(s.B) * s.D * s.N * f);
  p.part_D = align256(static_cast<size_t>(s.B) * s.D * f);
  return p;
}

template <typename T, int L>
sdm_status_t launch_grad_lanes(const SelGradPlan& p, const sdm::SelGradArgs& a, int B, cudaStream_t st) {
  constexpr int S = kGradSegment<L>, W = kGradTokens / S;
  using Tile = sdm::SelGradTile<L, S, W, kGradGroups>;
  constexpr size_t smem = Tile::kSmemFloats * sizeof(float);
  set_smem(reinterpret_cast<const void*>(sdm::k_selective_scan_backward<T, L, S, W, kGradGroups>), smem);
  const dim3 grid(static_cast<unsigned>(p.tiles_per_group) * a.f.G, 1, B);
  sdm::k_selective_scan_backward<T, L, S, W, kGradGroups><<<grid, Tile::kThreads, smem, st>>>(a);
  return launch_status("selective_scan_backward launch");
}

template <typename T>
sdm_status_t launch_grad(int L, const SelGradPlan& p, const sdm::SelGradArgs& a, int B, cudaStream_t st) {
  switch (L) {
    case 2: return launch_grad_lanes<T, 2>(p, a, B, st);
    case 4: return launch_grad_lanes<T, 4>(p, a, B, st);
    case 8: return launch_grad_lanes<T, 8>(p, a, B, st);
    default: return launch_grad_lanes<T, 16>(p, a, B, st);
  }
}

sdm_status_t cleared(void* p, size_t n, cudaStream_t st) {
  if (p == nullptr || n == 0) return SDM_OK;
  const cudaError_t e = cudaMemsetAsync(p, 0, n, st);
  return e == cudaSuccess ? SDM_OK : fail(SDM_ERR_CUDA, std::string("empty gradient: ") + cudaGetErrorString(e));
}

}  // namespace

}  // namespace sdm_host

using namespace sdm_host;

extern "C" {

size_t sdm_selective_scan_backward_workspace_bytes(const sdm_selscan_shape_t* shape) {
  if (check_selscan(shape) != SDM_OK) return 0;
  ok();
  if (shape->B == 0 || shape->T == 0 || shape->D == 0) return 0;
  return sel_grad_plan(*shape).total();
}

sdm_status_t sdm_selective_scan_backward(const sdm_selscan_shape_t* shape, const void* x, const void* dt,
                                         const float* A, const void* Bm, const void* Cm, const float* Dskip,
                                         const void* z, const float* dt_bias, const int32_t* lengths,
                                         const float* h0, const void* dy, const float* dhT, void* dx, void* ddt,
                                         float* dA, void* dB, void* dC, float* dD, void* dz, float* ddt_bias,
                                         float* dh0, void* workspace, size_t workspace_bytes, void* stream) {
  sdm_status_t r;
  if ((r = check_selscan(shape)) != SDM_OK) return r;
  const sdm_selscan_shape_t& s = *shape;
  const bool any = s.B > 0 && s.T > 0 && s.D > 0, par = s.D > 0;
  if ((r = need_selscan(s, any, x, dt, A, Bm, Cm, Dskip, z, dt_bias, lengths)) || (r = need_ptr(dy, "dy", any)) ||
      (r = need_ptr(h0, "h0", any && h0 != nullptr)) || (r = need_ptr(dhT, "dhT", dhT != nullptr)) ||
      (r = need_ptr(dx, "dx", any)) || (r = need_ptr(ddt, "ddt", any)) || (r = need_ptr(dA, "dA", par)) ||
      (r = need_ptr(dB, "dB", any)) || (r = need_ptr(dC, "dC", any)) ||
      (r = need_ptr(dD, "dD", par && (dD != nullptr || Dskip != nullptr))) ||
      (r = need_ptr(dz, "dz", any && z != nullptr)) ||
      (r = need_ptr(ddt_bias, "ddt_bias", par && (ddt_bias != nullptr || dt_bias != nullptr))) ||
      (r = need_ptr(dh0, "dh0", dh0 != nullptr)))
    return r;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const size_t states = static_cast<size_t>(s.B) * s.D * s.N * sizeof(float);
  if (!any) {
    // No token: the parameters get nothing, and dL/dh_0 is dL/dh_T.
    if ((r = cleared(dA, static_cast<size_t>(s.D) * s.N * sizeof(float), st)) ||
        (r = cleared(dD, s.D * sizeof(float), st)) || (r = cleared(ddt_bias, s.D * sizeof(float), st)) ||
        (dhT == nullptr && (r = cleared(dh0, states, st))))
      return r;
    if (states > 0 && dhT != nullptr && dh0 != nullptr && dh0 != dhT &&
        cudaMemcpyAsync(dh0, dhT, states, cudaMemcpyDeviceToDevice, st) != cudaSuccess)
      return launch_status("state gradient copy");
    return ok();
  }
  const SelGradPlan p = sel_grad_plan(s);
  if (p.tiles > 65535) return fail(SDM_ERR_UNSUPPORTED, "T above 65535 * 64 tokens");
  if ((r = need_ptr(workspace, "workspace", true)) != SDM_OK) return r;
  if (workspace_bytes < p.total())
    return fail(SDM_ERR_INVALID_ARGUMENT, "workspace is smaller than sdm_selective_scan_backward_workspace_bytes");
  DeviceInfo* dev;
  if ((r = device_info(&dev)) != SDM_OK) return r;
  sdm::SelGradArgs a{};
  a.f = selscan_args(s, x, dt, A, Bm, Cm, Dskip, z, dt_bias, lengths, dev->err);
  a.f.tiles_per_group = p.tiles_per_group;
  char* ws = static_cast<char*>(workspace);
  auto take = [&](size_t n) {
    float* q = reinterpret_cast<float*>(ws);
    ws += n;
    return q;
  };
  float* ckpt = take(p.ckpt);
  a.part_B = take(p.part_bc);
  a.part_C = take(p.part_bc);
  a.part_A = take(p.part_A);
  a.part_D = take(p.part_D);
  a.part_bias = take(p.part_D);
  a.dy = dy;
  a.dstate = dhT;
  a.dx = dx;
  a.ddt = ddt;
  a.dz = dz;
  a.dstate0 = dh0;
  // States before the tiles: the forward's maps over splits of one tile each.
  sdm::SelScanArgs f = a.f;
  f.tiles_per_group = static_cast<int>(ceil_div(s.D / s.G, sel_channels(s.N)));
  f.splits = p.tiles;
  f.tokens_per_split = kGradTokens;
  if ((r = launch_sel_states(s.in_dtype, f, s.B, h0, ckpt, st)) != SDM_OK) return r;
  a.ckpt = ckpt + static_cast<int64_t>(s.B) * p.tiles * s.D * s.N;
  const int L = grad_lanes(s.N);
  const bool bf = s.in_dtype == SDM_BF16;
  if ((r = bf ? launch_grad<bf16>(L, p, a, s.B, st) : launch_grad<float>(L, p, a, s.B, st)) != SDM_OK) return r;
  const int64_t n = static_cast<int64_t>(s.B) * s.T * s.G * s.N;
  const dim3 grid(static_cast<unsigned>(ceil_div(n, 1024)), 2);
  if (bf)
    sdm::k_selective_scan_sums<bf16><<<grid, 256, 0, st>>>(a.part_B, a.part_C, p.tiles_per_group, n,
                                                           static_cast<bf16*>(dB), static_cast<bf16*>(dC));
  else
    sdm::k_selective_scan_sums<float><<<grid, 256, 0, st>>>(a.part_B, a.part_C, p.tiles_per_group, n,
                                                            static_cast<float*>(dB), static_cast<float*>(dC));
  if ((r = launch_status("selective_scan_backward sums launch")) != SDM_OK) return r;
  auto batch_sum = [&](const float* part, int64_t m, float* out) {
    if (out == nullptr) return;
    sdm::k_selective_scan_batch_sum<<<static_cast<unsigned>(ceil_div(m, 256)), 256, 0, st>>>(part, s.B, m, out);
  };
  batch_sum(a.part_A, static_cast<int64_t>(s.D) * s.N, dA);
  batch_sum(a.part_D, s.D, dD);
  batch_sum(a.part_bias, s.D, ddt_bias);
  if ((r = launch_status("selective_scan_backward parameter sums launch")) != SDM_OK) return r;
  return ok();
}

}  // extern "C"
