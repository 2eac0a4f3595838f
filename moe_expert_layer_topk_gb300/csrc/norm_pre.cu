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

template <typename S, int L, int NV>
__global__ void __launch_bounds__(kNormThreads) pre_norm_kernel(const S* __restrict__ x, long long ldx,
                                                                const float* __restrict__ gain, float eps, int T, int H,
                                                                __nv_bfloat16* __restrict__ y, long long ldy,
                                                                float* __restrict__ rstd) {
  pdl_wait();
  pdl_trigger();
  __shared__ float sm[16];
  RowGroup<L> rg(sm);
  const int nvec = H / 8;
  const float inv_h = 1.0f / (float)H;
  for (long long base = (long long)blockIdx.x * rg.kRows; base < T; base += (long long)gridDim.x * rg.kRows) {
    const long long t = base + rg.g;
    const bool live = t < T;
    Vec8<S> v[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = rg.l + i * L;
      v[i] = zero_vec<S>();
      if (live && c < nvec) v[i].load(x + t * ldx + 8 * c);
    }
    const float r = rg.template rstd<NV>(inv_h, eps, [&](int i, int j) { return v[i].at(j); });
    if (!live) continue;
    if (rstd && rg.l == 0) rstd[t] = r;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = rg.l + i * L;
      if (c >= nvec) continue;
      const Gain8 w(gain, c, true);
      float o[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = v[i].at(j) * r * w.at(j);
      Vec8<__nv_bfloat16>::store(y + t * ldy + 8 * c, o);
    }
  }
}

// dx may be dres: a row's vectors are read before they are written by the same lane.
template <typename S, int L, int NV>
__global__ void __launch_bounds__(kNormThreads) pre_norm_bwd_kernel(
    const __nv_bfloat16* __restrict__ dy, long long lddy, const S* __restrict__ x, long long ldx, const float* __restrict__ gain,
    const float* __restrict__ rstd, const S* dres, long long lddres, float res_scale, int T, int H, S* dx, long long lddx,
    float* __restrict__ part) {
  pdl_wait();
  pdl_trigger();
  __shared__ float sm[16];
  __shared__ float fold[kNormThreads * NV * 8];
  RowGroup<L> rg(sm);
  const int nvec = H / 8;
  const float inv_h = 1.0f / (float)H;
  float acc[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[i][j] = 0.f;
  for (long long base = (long long)blockIdx.x * rg.kRows; base < T; base += (long long)gridDim.x * rg.kRows) {
    const long long t = base + rg.g;
    const bool live = t < T;
    Vec8<S> v[NV], res[NV];
    Vec8<__nv_bfloat16> d[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = rg.l + i * L;
      v[i] = zero_vec<S>();
      res[i] = zero_vec<S>();
      d[i] = zero_vec<__nv_bfloat16>();
      if (live && c < nvec) {
        v[i].load(x + t * ldx + 8 * c);
        d[i].load(dy + t * lddy + 8 * c);
        if (dres) res[i].load(dres + t * lddres + 8 * c);
      }
    }
    const float r = live ? __ldg(rstd + t) : 0.f;
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = rg.l + i * L;
      const Gain8 w(gain, c, c < nvec);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float n = v[i].at(j) * r, g = d[i].at(j);
        acc[i][j] = __fmaf_rn(g, n, acc[i][j]);
        m = __fmaf_rn(g * w.at(j), n, m);
      }
    }
    m = rg.sum(m) * inv_h;
    if (!live) continue;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = rg.l + i * L;
      if (c >= nvec) continue;
      const Gain8 w(gain, c, true);
      float o[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float n = v[i].at(j) * r;
        o[j] = r * (d[i].at(j) * w.at(j) - n * m);
        if (dres) o[j] = __fmaf_rn(res_scale, res[i].at(j), o[j]);
      }
      Vec8<S>::store(dx + t * lddx + 8 * c, o);
    }
  }
  if (part) leave_part<L, NV>(acc, fold, H, part);
}

// dgain[h] (+)= the parts' sums, in their order: 32 columns a block, eight threads a
// column, each every eighth part.
__global__ void __launch_bounds__(256) norm_gain_sum_kernel(const float* __restrict__ part, int parts, int H, float* dgain,
                                                            int accumulate) {
  pdl_wait();
  pdl_trigger();
  __shared__ float s[8][33];
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5, h = blockIdx.x * 32 + x;
  float v = 0.f;
  if (h < H)
    for (int p = y; p < parts; p += 8) v += __ldg(part + (size_t)p * H + h);
  s[y][x] = v;
  __syncthreads();
  if (y == 0 && h < H) {
    v = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) v += s[i][x];
    dgain[h] = accumulate ? dgain[h] + v : v;
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
  return with_row_shape(H, [&](auto l, auto nv) {
    constexpr int L = decltype(l)::value, NV = decltype(nv)::value;
    launch_pdl(pre_norm_kernel<S, L, NV>, norm_grid(T, kNormThreads / L, 8, 1 << 30), kNormThreads, 0, s, x, ldx, gain, eps, T, H,
               y, ldy, rstd);
    return check_launch(fn);
  });
}

template <typename S>
int run_pre_norm_bwd(const char* fn, const __nv_bfloat16* dy, long long lddy, const S* x, long long ldx, const float* gain,
                     const float* rstd, const S* dres, long long lddres, float res_scale, int T, int H, S* dx, long long lddx,
                     float* dgain, int accumulate, float* ws, cudaStream_t s) {
  return with_row_shape(H, [&](auto l, auto nv) {
    constexpr int L = decltype(l)::value, NV = decltype(nv)::value;
    const int grid = norm_grid(T, kNormThreads / L, 2, kNormParts);
    launch_pdl(pre_norm_bwd_kernel<S, L, NV>, grid, kNormThreads, 0, s, dy, lddy, x, ldx, gain, rstd, dres, lddres, res_scale, T, H,
               dx, lddx, dgain ? ws : nullptr);
    if (int rc = check_launch(fn)) return rc;
    return dgain ? launch_gain_sum(fn, ws, grid, H, dgain, accumulate, s) : MOE_OK;
  });
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

int launch_gain_sum(const char* fn, const float* part, int parts, int H, float* dgain, int accumulate, cudaStream_t s) {
  launch_pdl(norm_gain_sum_kernel, (H + 31) / 32, 256, 0, s, part, parts, H, dgain, accumulate);
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
