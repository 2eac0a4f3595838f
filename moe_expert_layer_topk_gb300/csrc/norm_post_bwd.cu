// Backward of the norm after a block, with the block's gate.
//
//   n = z r (norm) or z, G = sigmoid(gate), dv = b G dout, dn = dv gain:
//   dz = r (dn - n mean(dn n)) or dn,  dgain = sum_t dv n,  dgate = b dout n gain G (1 - G)
//
// Bound by HBM: rows arrive through the lanes' own rings of shared memory, are read once,
// and the gain's gradient is summed in the registers of a lane that always holds the same
// columns; each block leaves one row of partial sums.
#include "norm_gate.cuh"

namespace moe {
namespace {

struct PostBwdArgs {
  const void* dout;
  const __nv_bfloat16* z;
  const float* gain;
  int norm;
  const float* rstd;
  int gate_kind;
  const void* gate;
  float out_scale;
  int T, H;
  __nv_bfloat16* dz;
  float* part;
  void* dgate;
};

// dz may be z: each vector is read before it is written, by the same thread.
template <typename S, int NV, bool kElement>
struct PostBwd {
  static constexpr int SU = sizeof(Vec8<S>) / 16;                // units of a stream vector
  static constexpr int PER = 1 + SU + (kElement ? 1 : 0);        // z, dout, gate
  static constexpr int UNITS = NV * PER;
};
// As the backward of the norm before a block; with an element's gate a row is held too (two
// blocks an SM), since its sigmoids would be computed twice (8192 x 2048, fp32 stream: 44.5
// against 48.9 us; without that gate, bf16: 29.9 held, 28.5 read twice).
__host__ __device__ constexpr bool holds_row(bool element, bool wide, int nv) { return wide || (element && nv > 1); }
template <typename S, int L, int NV, bool kElement, bool kWide>
__global__ void __launch_bounds__(kWide ? 512 : 256, kWide ? 1 : (holds_row(kElement, kWide, NV) ? 2 : 3))
    post_norm_bwd_kernel(const PostBwdArgs p, int W) {
  pdl_wait();
  pdl_trigger();
  using P = PostBwd<S, NV, kElement>;
  constexpr int SU = P::SU, STAGES = ring_stages(P::UNITS, holds_row(kElement, kWide, NV));
  constexpr bool kHold = holds_row(kElement, kWide, NV);
  __shared__ __align__(16) float sm[kSumFloats];
  extern __shared__ __align__(16) uint8_t ring_smem[];
  RowRing ring(ring_smem, P::UNITS);
  RowGroup<L> rg(sm, W);
  const int H = p.H, nvec = H / 8, T = p.T, lanes = rg.lanes();
  const float inv_h = 1.0f / (float)H;
  const S* dout = static_cast<const S*>(p.dout);
  const long long step = (long long)gridDim.x * rg.rows();
  float acc[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[i][j] = 0.f;
  auto fetch = [&](int stage, long long t) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = rg.l + i * lanes;
      const bool there = t < T && c < nvec;
      const long long at = there ? t * H + 8 * c : 0;
      const int u = i * P::PER;
      ring.fetch(stage, u, p.z + at, there);
      ring.fetch(stage, u + 1, dout + at, there);
      if (kElement) ring.fetch(stage, u + 1 + SU, static_cast<const __nv_bfloat16*>(p.gate) + at, there);
    }
    ring.commit();
  };
  const long long first = (long long)blockIdx.x * rg.rows();
#pragma unroll
  for (int q = 0; q < STAGES - 1; ++q) fetch(q, first + q * step + rg.g);
  int stage = 0;
  for (long long base = first; base < T; base += step) {
    const long long t = base + rg.g;
    const bool live = t < T;
    const float r = p.norm && live ? __ldg(p.rstd + t) : 1.f;
    Gate tok = {1.f, 0.f};
    if (!kElement && p.gate_kind == 1 && live) tok = sigmoid(__ldg(static_cast<const float*>(p.gate) + t));
    fetch(stage == 0 ? STAGES - 1 : stage - 1, t + (STAGES - 1) * step);
    ring.template wait<STAGES - 1>();
    float m = 0.f, dg = 0.f;  // sums of dn n, and of dout n gain
    float n[NV][8], dn[NV][8];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = rg.l + i * lanes, u = i * P::PER;
      const bool there = live && c < nvec;
      const Gain8 w(p.gain, c, c < nvec);
      const Vec8<__nv_bfloat16> zv = ring.template vec<__nv_bfloat16>(stage, u);
      const Vec8<S> d = ring.template vec<S>(stage, u + 1);
      const Vec8<__nv_bfloat16> gv = kElement ? ring.template vec<__nv_bfloat16>(stage, u + 1 + SU) : zero_vec<__nv_bfloat16>();
      float ds[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        n[i][j] = zv.at(j) * r;
        const float e = p.out_scale * d.at(j);
        const Gate G = kElement ? sigmoid(gv.at(j)) : tok;
        const float ew = e * w.at(j);
        acc[i][j] = __fmaf_rn(e * G.g, n[i][j], acc[i][j]);
        dn[i][j] = ew * G.g;
        m = __fmaf_rn(dn[i][j], n[i][j], m);
        if (kElement)
          ds[j] = ew * n[i][j] * G.d;
        else
          dg = __fmaf_rn(ew, n[i][j], dg);
      }
      if (kElement && p.dgate && there) Vec8<__nv_bfloat16>::store(static_cast<__nv_bfloat16*>(p.dgate) + t * H + 8 * c, ds);
    }
    if (!kElement && p.gate_kind == 1 && p.dgate) {
      rg.template sums<true>(m, dg);
      if (live && rg.l == 0) static_cast<float*>(p.dgate)[t] = dg * tok.d;
    } else if (p.norm) {
      m = rg.sum(m);
    }
    m *= inv_h;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = rg.l + i * lanes, u = i * P::PER;
      if (!live || c >= nvec) continue;
      if (!kHold) {
        const Gain8 w(p.gain, c, true);
        const Vec8<__nv_bfloat16> zv = ring.template vec<__nv_bfloat16>(stage, u);
        const Vec8<S> d = ring.template vec<S>(stage, u + 1);
        const Vec8<__nv_bfloat16> gv = kElement ? ring.template vec<__nv_bfloat16>(stage, u + 1 + SU) : zero_vec<__nv_bfloat16>();
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          n[i][j] = zv.at(j) * r;
          dn[i][j] = p.out_scale * d.at(j) * w.at(j) * (kElement ? sigmoid(gv.at(j)).g : tok.g);
        }
      }
      float o[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = p.norm ? r * (dn[i][j] - n[i][j] * m) : dn[i][j];
      Vec8<__nv_bfloat16>::store(p.dz + t * H + 8 * c, o);
    }
    stage = stage + 1 == STAGES ? 0 : stage + 1;
  }
  if (p.part) {  // the ring's memory is free: copies still under way are of rows behind the last, zeros
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
    leave_part<L, NV>(rg, acc, reinterpret_cast<float*>(ring_smem), H, p.part);
  }
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_post_norm_bwd_workspace_size(int T, int H) { return norm_parts_bytes(T, H); }

int moe_post_norm_bwd(const void* dout, int fp32, const void* z, const float* gain, int norm, const float* rstd, int gate_kind,
                      const void* gate, float out_scale, int T, int H, void* dz, float* dgain, void* dgate, int accumulate, void* ws,
                      size_t ws_bytes, void* stream) {
  clear_error();
  const char* fn = "moe_post_norm_bwd";
  if (int rc = check_post(fn, T, H, fp32, norm, gate_kind)) return rc;
  if (dgate && !gate_kind) return fail(MOE_ERR_INVALID_ARG, "%s: dgate without a gate", fn);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (T == 0) {
    if (!dgain || accumulate) return MOE_OK;
    cudaError_t e = cudaMemsetAsync(dgain, 0, sizeof(float) * (size_t)H, s);
    return e == cudaSuccess ? MOE_OK : fail_cuda(fn, e);
  }
  if (!dout || !z || !dz || (norm && !rstd) || (gate_kind && !gate)) return fail(MOE_ERR_INVALID_ARG, "%s: NULL pointer argument", fn);
  if (!aligned16(dout) || !aligned16(z) || !aligned16(gain) || !aligned16(dz))
    return fail(MOE_ERR_ALIGNMENT, "%s: tensors must be 16-byte aligned", fn);
  if (!gate_aligned(gate_kind, gate) || !gate_aligned(gate_kind, dgate)) return fail(MOE_ERR_ALIGNMENT, "%s: gate or dgate is not aligned", fn);
  if (int rc = check_gain_grad(fn, T, H, dgain, ws, ws_bytes)) return rc;
  const PostBwdArgs a = {dout, static_cast<const __nv_bfloat16*>(z), gain, norm, rstd, gate_kind, gate, out_scale, T, H,
                         static_cast<__nv_bfloat16*>(dz), dgain ? static_cast<float*>(ws) : nullptr, dgate};
  auto run = [&](auto type, auto l, auto v, auto wide, auto element) {
    using S = decltype(type);
    constexpr int L = decltype(l)::value, NV = decltype(v)::value;
    constexpr bool kElement = decltype(element)::value, kWide = decltype(wide)::value;
    const RowShape sh = row_shape(H, NV);
    auto kern = post_norm_bwd_kernel<S, L, NV, kElement, kWide>;
    const size_t smem = bwd_smem(PostBwd<S, NV, kElement>::UNITS, NV, sh.threads, holds_row(kElement, kWide, NV));
    const int grid = norm_grid(T, sh.rows, blocks_per_sm(smem, sh.threads, holds_row(kElement, kWide, NV) ? 128 : 80), kNormParts);
    static bool done[kMaxDevices];
    if (int rc = allow_smem(fn, reinterpret_cast<const void*>(kern), smem, done)) return rc;
    launch_pdl(kern, grid, sh.threads, smem, s, a, sh.W);
    if (int rc = check_launch(fn)) return rc;
    return dgain ? launch_gain_sum(fn, static_cast<const float*>(ws), grid, H, dgain, accumulate, s) : MOE_OK;
  };
  auto typed = [&](auto l, auto v, auto wide) {
    if (gate_kind == 2) return fp32 ? run(float(), l, v, wide, std::true_type()) : run(__nv_bfloat16(), l, v, wide, std::true_type());
    return fp32 ? run(float(), l, v, wide, std::false_type()) : run(__nv_bfloat16(), l, v, wide, std::false_type());
  };
  if (H > 4096) return typed(std::integral_constant<int, 0>{}, std::integral_constant<int, 2>{}, std::true_type{});
  if (H > 256) return typed(std::integral_constant<int, 0>{}, std::integral_constant<int, 2>{}, std::false_type{});
  return with_lanes<false>(row_shape(H, 1).L, [&](auto l) { return typed(l, std::integral_constant<int, 1>{}, std::false_type{}); });
}

}  // extern "C"
