// The root-mean-square norm before a block, and its backward.
//
//   r = 1/sqrt(mean x^2 + eps), y = x r gain
//   n = x r, dn = dy gain:  dx = a dres + r (dn - n mean(dn n)),  dgain = sum_t dy n
//
// Bound by HBM: every row is read once into registers, the residual path's gradient
// is added on the way, and the gain's gradient is summed in the registers of a lane
// that always holds the same columns; each block leaves one row of partial sums.
#include "norm.cuh"

namespace moe {
namespace {

// A vector a lane for rows within a warp (registers for eight blocks an SM: 65521 rows of
// 128 with a row stride of 192 take 9.4 us, of which a kernel of one row takes 2.9), up to
// four for longer ones.
template <typename S, int L, int NV>
__global__ void __launch_bounds__(256, NV == 1 ? 8 : 4) pre_norm_kernel(const S* __restrict__ x, long long ldx,
                                                                        const float* __restrict__ gain, float eps, int T, int H, int W,
                                                                        __nv_bfloat16* __restrict__ y, long long ldy,
                                                                        float* __restrict__ rstd) {
  pdl_wait();
  pdl_trigger();
  __shared__ __align__(16) float sm[kSumFloats];
  RowGroup<L> rg(sm, W);
  const int nvec = H / 8, n = rg.lanes(), rows = rg.rows();
  const float inv_h = 1.0f / (float)H;
  for (long long base = (long long)blockIdx.x * rows; base < T; base += (long long)gridDim.x * rows) {
    const long long t = base + rg.g;
    const bool live = t < T;
    Vec8<S> v[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = rg.l + i * n;
      v[i] = zero_vec<S>();
      if (live && c < nvec) v[i].load(x + t * ldx + 8 * c);
    }
    const float r = rg.template rstd<NV>(inv_h, eps, [&](int i, int j) { return v[i].at(j); });
    if (!live) continue;
    if (rstd && rg.l == 0) rstd[t] = r;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = rg.l + i * n;
      if (c >= nvec) continue;
      const Gain8 w(gain, c, true);
      float o[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = v[i].at(j) * r * w.at(j);
      Vec8<__nv_bfloat16>::store(y + t * ldy + 8 * c, o);
    }
  }
}

// dx may be dres, with its row stride: each vector is read before it is written, by the same thread.
template <typename S, int NV>
struct PreBwd {
  static constexpr int SU = sizeof(Vec8<S>) / 16;         // units of a stream vector
  static constexpr int UNITS = NV * (1 + 2 * SU);         // dy, x, dres
};
// A vector a lane for rows within a warp, two for longer ones (kWide: 512 threads, for more
// than 4096 columns).  A row's vectors stay in the ring while it is worked on and are read
// twice: in registers they would leave an SM two blocks instead of three (8192 x 2048: 28.4
// against 31.0 us).  The wide kernel has one block an SM anyway and holds them (2048 x 8192:
// 36.3 against 39.5).
template <typename S, int L, int NV, bool kWide>
__global__ void __launch_bounds__(kWide ? 512 : 256, kWide ? 1 : 3) pre_norm_bwd_kernel(
    const __nv_bfloat16* __restrict__ dy, long long lddy, const S* __restrict__ x, long long ldx, const float* __restrict__ gain,
    const float* __restrict__ rstd, const S* dres, long long lddres, float res_scale, int T, int H, int W, S* dx, long long lddx,
    float* __restrict__ part) {
  pdl_wait();
  pdl_trigger();
  using P = PreBwd<S, NV>;
  constexpr int SU = P::SU, STAGES = ring_stages(P::UNITS, kWide);
  __shared__ __align__(16) float sm[kSumFloats];
  extern __shared__ __align__(16) uint8_t ring_smem[];
  RowRing ring(ring_smem, P::UNITS);
  RowGroup<L> rg(sm, W);
  const int nvec = H / 8, n_lanes = rg.lanes();
  const float inv_h = 1.0f / (float)H;
  const long long step = (long long)gridDim.x * rg.rows();
  float acc[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[i][j] = 0.f;
  auto fetch = [&](int stage, long long t) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = rg.l + i * n_lanes;
      const bool there = t < T && c < nvec;
      const int u = i * (1 + 2 * SU);
      ring.fetch(stage, u, dy + (there ? t * lddy + 8 * c : 0), there);
      ring.fetch(stage, u + 1, x + (there ? t * ldx + 8 * c : 0), there);
      if (dres) ring.fetch(stage, u + 1 + SU, dres + (there ? t * lddres + 8 * c : 0), there);
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
    const float r = live ? __ldg(rstd + t) : 0.f;
    fetch(stage == 0 ? STAGES - 1 : stage - 1, t + (STAGES - 1) * step);
    ring.template wait<STAGES - 1>();
    Vec8<__nv_bfloat16> d[NV];
    Vec8<S> v[NV];
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = rg.l + i * n_lanes, u = i * (1 + 2 * SU);
      d[i] = ring.template vec<__nv_bfloat16>(stage, u);
      v[i] = ring.template vec<S>(stage, u + 1);
      const Gain8 w(gain, c, c < nvec);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float n = v[i].at(j) * r, g = d[i].at(j);
        acc[i][j] = __fmaf_rn(g, n, acc[i][j]);
        m = __fmaf_rn(g * w.at(j), n, m);
      }
    }
    m = rg.sum(m) * inv_h;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = rg.l + i * n_lanes, u = i * (1 + 2 * SU);
      if (!live || c >= nvec) continue;
      if (!kWide) {
        d[i] = ring.template vec<__nv_bfloat16>(stage, u);
        v[i] = ring.template vec<S>(stage, u + 1);
      }
      const Gain8 w(gain, c, true);
      float o[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = r * (d[i].at(j) * w.at(j) - v[i].at(j) * r * m);
      if (dres) {
        const Vec8<S> res = ring.template vec<S>(stage, u + 1 + SU);
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = __fmaf_rn(res_scale, res.at(j), o[j]);
      }
      Vec8<S>::store(dx + t * lddx + 8 * c, o);
    }
    stage = stage + 1 == STAGES ? 0 : stage + 1;
  }
  if (part) {  // the ring's memory is free: copies still under way are of rows behind the last, zeros
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
    leave_part<L, NV>(rg, acc, reinterpret_cast<float*>(ring_smem), H, part);
  }
}

// dgain[h] (+)= the parts' sums: 32 columns a block, four a thread, 64 threads a column,
// each with every 64th of the 512 parts at most, all eight under way at once; their sums in
// a fixed order.
__global__ void __launch_bounds__(512) norm_gain_sum_kernel(const float* __restrict__ part, int parts, int H, float* dgain,
                                                            int accumulate) {
  pdl_wait();
  pdl_trigger();
  __shared__ float s[64][33];
  __shared__ float s2[16][33];
  const int x = threadIdx.x & 7, y = threadIdx.x >> 3, h = blockIdx.x * 32 + 4 * x;
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  if (h < H) {
    float4 a[8];
#pragma unroll
    for (int u = 0; u < 8; ++u)
      a[u] = y + 64 * u < parts ? __ldg(reinterpret_cast<const float4*>(part + (size_t)(y + 64 * u) * H + h)) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int u = 0; u < 8; ++u) v.x += a[u].x, v.y += a[u].y, v.z += a[u].z, v.w += a[u].w;
  }
  s[y][4 * x] = v.x, s[y][4 * x + 1] = v.y, s[y][4 * x + 2] = v.z, s[y][4 * x + 3] = v.w;
  __syncthreads();
  {
    const int c = threadIdx.x & 31, q = threadIdx.x >> 5;
    s2[q][c] = (s[4 * q][c] + s[4 * q + 1][c]) + (s[4 * q + 2][c] + s[4 * q + 3][c]);
  }
  __syncthreads();
  const int c = blockIdx.x * 32 + threadIdx.x;
  if (threadIdx.x < 32 && c < H) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) sum += s2[i][threadIdx.x];
    dgain[c] = accumulate ? dgain[c] + sum : sum;
  }
}

template <class T>
bool row_strides_ok(const T* p, long long ld, int H) {
  const int unit = 16 / (int)sizeof(T);
  return !p || (ld >= H && ld % unit == 0);
}

template <typename S>
int run_pre_norm(const char* fn, const S* x, long long ldx, const float* gain, float eps, int T, int H, __nv_bfloat16* y,
                 long long ldy, float* rstd, cudaStream_t s) {
  const RowShape sh = row_shape(H, 4);
  return with_lanes<true>(sh.L, [&](auto l) {
    constexpr int L = decltype(l)::value, NV = L ? 1 : 4;
    launch_pdl(pre_norm_kernel<S, L, NV>, norm_grid(T, sh.rows, 8, 1 << 30), sh.threads, 0, s, x, ldx, gain, eps, T, H, sh.W, y, ldy,
               rstd);
    return check_launch(fn);
  });
}

template <typename S>
int run_pre_norm_bwd(const char* fn, const __nv_bfloat16* dy, long long lddy, const S* x, long long ldx, const float* gain,
                     const float* rstd, const S* dres, long long lddres, float res_scale, int T, int H, S* dx, long long lddx,
                     float* dgain, int accumulate, float* ws, cudaStream_t s) {
  auto run = [&](auto l, auto v, auto wide) {
    constexpr int L = decltype(l)::value, NV = decltype(v)::value;
    constexpr bool kWide = decltype(wide)::value;
    const RowShape sh = row_shape(H, NV);
    auto kern = pre_norm_bwd_kernel<S, L, NV, kWide>;
    const size_t smem = bwd_smem(PreBwd<S, NV>::UNITS, NV, sh.threads, kWide);
    const int grid = norm_grid(T, sh.rows, blocks_per_sm(smem, sh.threads, kWide ? 128 : 80), kNormParts);
    static bool done[kMaxDevices];
    if (int rc = allow_smem(fn, reinterpret_cast<const void*>(kern), smem, done)) return rc;
    launch_pdl(kern, grid, sh.threads, smem, s, dy, lddy, x, ldx, gain, rstd, dres, lddres, res_scale, T, H, sh.W, dx, lddx,
               dgain ? ws : nullptr);
    if (int rc = check_launch(fn)) return rc;
    return dgain ? launch_gain_sum(fn, ws, grid, H, dgain, accumulate, s) : MOE_OK;
  };
  if (H > 4096) return run(std::integral_constant<int, 0>{}, std::integral_constant<int, 2>{}, std::true_type{});
  if (H > 256) return run(std::integral_constant<int, 0>{}, std::integral_constant<int, 2>{}, std::false_type{});
  return with_lanes<false>(row_shape(H, 1).L, [&](auto l) { return run(l, std::integral_constant<int, 1>{}, std::false_type{}); });
}

}  // namespace

int check_norm(const char* fn, int T, int H, int fp32) {
  if (T < 0 || H <= 0 || (fp32 != 0 && fp32 != 1)) return fail(MOE_ERR_INVALID_ARG, "%s: need T>=0, H>0, fp32 0 or 1", fn);
  if (H % 8 || H > kNormMaxH) return fail(MOE_ERR_UNSUPPORTED_SHAPE, "%s: need H%%8==0, H<=%d (H=%d)", fn, kNormMaxH, H);
  return MOE_OK;
}

int check_gain_grad(const char* fn, int T, int H, const float* dgain, const void* ws, size_t ws_bytes) {
  if (!dgain) return MOE_OK;
  const size_t need = norm_parts_bytes(T, H);
  if (!ws || ws_bytes < need) return fail(MOE_ERR_WORKSPACE, "%s: workspace %zu < %zu bytes", fn, ws ? ws_bytes : (size_t)0, need);
  if (!aligned16(ws) || !aligned16(dgain)) return fail(MOE_ERR_ALIGNMENT, "%s: dgain and ws must be 16-byte aligned", fn);
  return MOE_OK;
}

int allow_smem(const char* fn, const void* kernel, size_t bytes, bool (&done)[kMaxDevices]) {
  const size_t most = 232448 - sizeof(float) * kSumFloats;
  if (bytes > most) return fail(MOE_ERR_UNSUPPORTED_SHAPE, "%s: needs %zu bytes of shared memory", fn, bytes);
  const int dev = current_device();
  if (dev < 0) return fail(MOE_ERR_CUDA, "%s: no current CUDA device", fn);
  if (done[dev]) return MOE_OK;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
  if (e != cudaSuccess) return fail_cuda(fn, e);
  done[dev] = true;
  return MOE_OK;
}

int launch_gain_sum(const char* fn, const float* part, int parts, int H, float* dgain, int accumulate, cudaStream_t s) {
  launch_pdl(norm_gain_sum_kernel, (H + 31) / 32, 512, 0, s, part, parts, H, dgain, accumulate);
  return check_launch(fn);
}

}  // namespace moe

using namespace moe;

extern "C" {

int moe_pre_norm(const void* x, long long ldx, int fp32, const float* gain, float eps, int T, int H, void* y, long long ldy,
                 float* rstd, void* stream) {
  clear_error();
  const char* fn = "moe_pre_norm";
  if (int rc = check_norm(fn, T, H, fp32)) return rc;
  if (!(eps > 0.f && eps <= 3.402823466e+38f)) return fail(MOE_ERR_INVALID_ARG, "%s: need eps>0", fn);
  if (T == 0) return MOE_OK;
  if (!x || !y) return fail(MOE_ERR_INVALID_ARG, "%s: NULL pointer argument", fn);
  auto* yb = static_cast<__nv_bfloat16*>(y);
  const bool strides = (fp32 ? row_strides_ok(static_cast<const float*>(x), ldx, H)
                             : row_strides_ok(static_cast<const __nv_bfloat16*>(x), ldx, H)) &&
                       row_strides_ok(yb, ldy, H);
  if (!strides) return fail(MOE_ERR_INVALID_ARG, "%s: row strides must be at least H and whole 16-byte vectors", fn);
  if (!aligned16(x) || !aligned16(y) || (gain && !aligned16(gain)))
    return fail(MOE_ERR_ALIGNMENT, "%s: x, gain and y must be 16-byte aligned", fn);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return fp32 ? run_pre_norm(fn, static_cast<const float*>(x), ldx, gain, eps, T, H, yb, ldy, rstd, s)
              : run_pre_norm(fn, static_cast<const __nv_bfloat16*>(x), ldx, gain, eps, T, H, yb, ldy, rstd, s);
}

size_t moe_pre_norm_bwd_workspace_size(int T, int H) { return norm_parts_bytes(T, H); }

int moe_pre_norm_bwd(const void* dy, long long lddy, const void* x, long long ldx, int fp32, const float* gain, const float* rstd,
                     const void* dres, long long lddres, float res_scale, int T, int H, void* dx, long long lddx, float* dgain,
                     int accumulate, void* ws, size_t ws_bytes, void* stream) {
  clear_error();
  const char* fn = "moe_pre_norm_bwd";
  if (int rc = check_norm(fn, T, H, fp32)) return rc;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (T == 0) {
    if (!dgain || accumulate) return MOE_OK;
    cudaError_t e = cudaMemsetAsync(dgain, 0, sizeof(float) * (size_t)H, s);
    return e == cudaSuccess ? MOE_OK : fail_cuda(fn, e);
  }
  if (!dy || !x || !rstd || !dx) return fail(MOE_ERR_INVALID_ARG, "%s: NULL pointer argument", fn);
  auto strides = [&](auto type) {
    using S = decltype(type);
    return row_strides_ok(static_cast<const S*>(x), ldx, H) && row_strides_ok(static_cast<const S*>(dres), lddres, H) &&
           row_strides_ok(static_cast<const S*>(dx), lddx, H);
  };
  if (!(fp32 ? strides(float()) : strides(__nv_bfloat16())) || !row_strides_ok(static_cast<const __nv_bfloat16*>(dy), lddy, H))
    return fail(MOE_ERR_INVALID_ARG, "%s: row strides must be at least H and whole 16-byte vectors", fn);
  if (dx == dres && lddx != lddres && T > 1) return fail(MOE_ERR_INVALID_ARG, "%s: dx over dres needs dres's row stride", fn);
  if (!aligned16(dy) || !aligned16(x) || !aligned16(dx) || (dres && !aligned16(dres)) || (gain && !aligned16(gain)))
    return fail(MOE_ERR_ALIGNMENT, "%s: dy, x, gain, dres and dx must be 16-byte aligned", fn);
  if (int rc = check_gain_grad(fn, T, H, dgain, ws, ws_bytes)) return rc;
  auto run = [&](auto type) {
    using S = decltype(type);
    return run_pre_norm_bwd(fn, static_cast<const __nv_bfloat16*>(dy), lddy, static_cast<const S*>(x), ldx, gain, rstd,
                            static_cast<const S*>(dres), lddres, res_scale, T, H, static_cast<S*>(dx), lddx, dgain, accumulate,
                            static_cast<float*>(ws), s);
  };
  return fp32 ? run(float()) : run(__nv_bfloat16());
}

}  // extern "C"
