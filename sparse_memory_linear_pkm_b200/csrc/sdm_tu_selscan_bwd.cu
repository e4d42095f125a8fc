// Entry point and launches of the selective scan's gradient.

#include "sdm_selscan_bwd.cuh"
#include "sdm_selscan_host.h"

namespace sdm_host {

namespace {

constexpr int kGradSplitTokens = 32;  // a split has at least this many tokens
constexpr int kGradBlocks = 3;        // blocks an SM holds at a time
constexpr int kGradMapTokens = 10;    // tokens that a split's maps and start cost the time of

struct SelGradPlan {
  int NP = 0;                 // states a channel is padded to
  int splits = 1, tokens_per_split = 0, tiles = 0, tiles_per_group = 0;
  size_t split_states = 0, kept = 0, sums = 0, part_bc = 0, part_A = 0, part_D = 0;
  size_t total() const { return 3 * split_states + kept + sums + 2 * part_bc + part_A + part_D; }
};

// The token axis is split into whole tiles so that the blocks come to 1 to 8
// whole waves, of which the cheapest is taken: waves x (tokens of a split + what
// the split itself costs). As many splits as give 24 warps an SM, of 64 tokens at
// least: 2119 us instead of 1940 (3 waves) for B = 4, T = 4096, D = 4096, N = 16,
// 278 instead of 259 (1 wave) for 4096 x 2048, 193 instead of 148 for 1000 x 4096.
SelGradPlan sel_grad_plan(const sdm_selscan_shape_t& s) {
  SelGradPlan p;
  p.NP = s.N <= 8 ? 8 : (s.N <= 16 ? 16 : (s.N <= 32 ? 32 : 64));
  p.tiles_per_group = static_cast<int>(ceil_div(s.D / s.G, sel_channels(s.N)));
  p.tiles = static_cast<int>(ceil_div(s.T, sdm::kGradTile));
  const int64_t blocks = static_cast<int64_t>(s.B) * s.G * p.tiles_per_group, slots = kGradBlocks * kSms;
  int64_t least = INT64_MAX;
  for (int64_t waves = 1; waves <= 8; ++waves) {
    const int64_t want = std::min<int64_t>(waves * slots / blocks, s.T / kGradSplitTokens);
    const int64_t tokens =
        ceil_div(ceil_div(s.T, std::max<int64_t>(1, want)), sdm::kGradTile) * sdm::kGradTile;
    const int64_t splits = ceil_div(s.T, tokens);
    const int64_t cost = ceil_div(splits * blocks, slots) * (tokens + kGradMapTokens);
    if (cost >= least) continue;
    least = cost;
    p.splits = static_cast<int>(splits);
    p.tokens_per_split = static_cast<int>(tokens);
  }
  const size_t f = sizeof(float), row = static_cast<size_t>(s.D) * p.NP * f;
  p.split_states = align256(static_cast<size_t>(s.B) * p.splits * row);
  p.kept = align256(static_cast<size_t>(s.B) * p.tiles * row);
  p.sums = align256(static_cast<size_t>(s.B) * p.tiles * s.D * f);
  p.part_bc = align256(static_cast<size_t>(p.tiles_per_group) * s.B * s.T * s.G * s.N * f);
  p.part_A = align256(static_cast<size_t>(s.B) * p.splits * row);
  p.part_D = align256(2 * static_cast<size_t>(s.B) * p.splits * s.D * f);
  return p;
}

template <typename T, int KS, int L>
sdm_status_t launch_grad_lanes(const sdm::SelGradArgs& a, int B, cudaStream_t st) {
  constexpr int NG = KS * L / 4;
  const dim3 grid(static_cast<unsigned>(a.f.tiles_per_group) * a.f.G, a.f.splits, B);
  sdm::k_selective_scan_grad_maps<T, KS, L><<<grid, sdm::kSelThreads, 0, st>>>(a);
  sdm_status_t r;
  if ((r = launch_status("selective_scan_backward maps launch")) != SDM_OK) return r;
  sdm::k_selective_scan_grad_chain<<<dim3(static_cast<unsigned>(ceil_div(a.f.D, 128)), NG, B), 128, 0, st>>>(a, NG);
  if ((r = launch_status("selective_scan_backward chain launch")) != SDM_OK) return r;
  constexpr size_t smem = sizeof(sdm::GradSmem<KS, L>);
  set_smem(reinterpret_cast<const void*>(sdm::k_selective_scan_grad<T, KS, L>), smem);
  sdm::k_selective_scan_grad<T, KS, L><<<grid, sdm::kSelThreads, smem, st>>>(a);
  return launch_status("selective_scan_backward launch");
}

template <typename T>
sdm_status_t launch_grad(const sdm::SelGradArgs& a, int B, cudaStream_t st) {
  if (a.f.N <= 8) return launch_grad_lanes<T, 8, 1>(a, B, st);
  if (a.f.N <= 16) return launch_grad_lanes<T, 16, 1>(a, B, st);
  if (a.f.N <= 32) return launch_grad_lanes<T, 16, 2>(a, B, st);
  return launch_grad_lanes<T, 16, 4>(a, B, st);
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
  // dh0 may be dhT: one thread reads a value of dhT and writes that of dh0.
  const Piece first = {"dh0", dh0, states}, last = {"dhT", dhT == dh0 ? nullptr : dhT, states};
  if (!any) {
    if ((r = check_apart(&first, 1, &last, 1)) != SDM_OK) return r;
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
  if ((r = need_ptr(workspace, "workspace", true)) != SDM_OK) return r;
  if (workspace_bytes < p.total())
    return fail(SDM_ERR_INVALID_ARGUMENT, "workspace is smaller than sdm_selective_scan_backward_workspace_bytes");
  sdm::SelGradArgs a{};
  a.f = selscan_args(s, x, dt, A, Bm, Cm, Dskip, z, dt_bias, lengths);
  const SelInputs in = selscan_inputs(s, a.f);
  const size_t es = in_size(s.in_dtype), tokens = static_cast<size_t>(s.B) * s.T, rows = tokens * s.D * es;
  const size_t bc = tokens * s.G * s.N * es;
  const size_t row = s.D * sizeof(float);
  const Piece more[] = {{"dy", dy, rows}, {"h0", h0, states}, last};
  const Piece outs[] = {{"dx", dx, rows}, {"ddt", ddt, rows}, {"dz", dz, rows},  {"dB", dB, bc},  {"dC", dC, bc},
                        {"dA", dA, row * s.N}, {"dD", dD, row}, {"ddt_bias", ddt_bias, row}, first};
  if ((r = check_apart(outs, 9, in.piece, kSelInputs)) || (r = check_apart(outs, 9, more, 3))) return r;
  DeviceInfo* dev;
  if ((r = device_info(&dev)) != SDM_OK) return r;
  a.f.err = dev->err;
  a.f.tiles_per_group = p.tiles_per_group;
  a.f.splits = p.splits;
  a.f.tokens_per_split = p.tokens_per_split;
  a.tiles = p.tiles;
  char* ws = static_cast<char*>(workspace);
  auto take = [&](size_t n) {
    float* q = reinterpret_cast<float*>(ws);
    ws += n;
    return q;
  };
  a.P = reinterpret_cast<float4*>(take(p.split_states));
  a.H = reinterpret_cast<float4*>(take(p.split_states));
  a.R = reinterpret_cast<float4*>(take(p.split_states));
  a.kept = reinterpret_cast<float4*>(take(p.kept));
  a.sums = take(p.sums);
  a.part_B = take(p.part_bc);
  a.part_C = take(p.part_bc);
  a.part_A = reinterpret_cast<float4*>(take(p.part_A));
  a.part_D = take(p.part_D);
  a.h0 = h0;
  a.dy = dy;
  a.dstate = dhT;
  a.dx = dx;
  a.ddt = ddt;
  a.dz = dz;
  a.dstate0 = dh0;
  const bool bf = s.in_dtype == SDM_BF16;
  if ((r = bf ? launch_grad<bf16>(a, s.B, st) : launch_grad<float>(a, s.B, st)) != SDM_OK) return r;
  const int64_t n = static_cast<int64_t>(s.B) * s.T * s.G * s.N;
  const dim3 grid(static_cast<unsigned>(ceil_div(n, 1024)), 2);
  if (bf)
    sdm::k_selective_scan_sums<bf16><<<grid, 256, 0, st>>>(a.part_B, a.part_C, p.tiles_per_group, n,
                                                           static_cast<bf16*>(dB), static_cast<bf16*>(dC));
  else
    sdm::k_selective_scan_sums<float><<<grid, 256, 0, st>>>(a.part_B, a.part_C, p.tiles_per_group, n,
                                                            static_cast<float*>(dB), static_cast<float*>(dC));
  if ((r = launch_status("selective_scan_backward sums launch")) != SDM_OK) return r;
  const int NG = p.NP / 4;
  sdm::k_selective_scan_grad_params<<<dim3(static_cast<unsigned>(ceil_div(s.D, 32)), NG + 1), dim3(32, 8), 0, st>>>(
      a, NG, s.B * p.splits, dA, dD, ddt_bias);
  if ((r = launch_status("selective_scan_backward parameter sums launch")) != SDM_OK) return r;
  return ok();
}

}  // extern "C"
