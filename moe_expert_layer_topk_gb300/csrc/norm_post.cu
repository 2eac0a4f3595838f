// The norm after a block with the block's gate, the residual and a scale for each;
// alone or on the weighted combine of the experts' rows, with the next block's norm
// of the result where it is asked for, and its backward.
//
//   n = z r (norm) or z, G = sigmoid(gate):  out = a residual + b G n gain
//   dv = b G dout, dn = dv gain:  dz = r (dn - n mean(dn n)),  dgain = sum_t dv n,
//   dgate = b dout n gain G (1 - G)
//
// Bound by HBM: a token's row stays in the registers of its lanes from the experts'
// rows to the next block's input.
#include "norm.cuh"

namespace moe {
namespace {

struct PostArgs {
  const __nv_bfloat16* z;  // the block's output, or the experts' rows
  const float* topk_w;     // combine: [T,k]
  const int32_t* row_of_slot;
  int k, R;
  const void* residual;
  const float* gain;
  int norm;
  float eps;
  int gate_kind;
  const void* gate;
  float res_scale, out_scale;
  int T, H;
  __nv_bfloat16* z_out;
  void* out;
  float* rstd;
  const float* next_gain;
  __nv_bfloat16* next_y;
  float* next_rstd;
  int* status;
};

// sigmoid(x) and its derivative, from e^-|x|: neither loses digits at either end.
struct Gate {
  float g, d;
};
__device__ __forceinline__ Gate sigmoid(float x) {
  const float e = __expf(-fabsf(x)), t = __fdividef(1.0f, 1.0f + e);
  return {x >= 0.f ? t : e * t, e * t * t};
}

template <typename S, int L, int NV, bool kCombine>
__global__ void __launch_bounds__(kNormThreads) post_norm_kernel(const PostArgs p) {
  pdl_wait();
  pdl_trigger();
  __shared__ float sm[16];
  RowGroup<L> rg(sm);
  const int H = p.H, nvec = H / 8, T = p.T;
  const float inv_h = 1.0f / (float)H;
  const S* residual = static_cast<const S*>(p.residual);
  S* out = static_cast<S*>(p.out);
  for (long long base = (long long)blockIdx.x * rg.kRows; base < T; base += (long long)gridDim.x * rg.kRows) {
    const long long t = base + rg.g;
    const bool live = t < T;
    float z[NV][8];
    Vec8<S> res[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = rg.l + i * L;
      res[i] = zero_vec<S>();
      if (residual && live && c < nvec) res[i].load(residual + t * H + 8 * c);
#pragma unroll
      for (int j = 0; j < 8; ++j) z[i][j] = 0.f;
    }
    if constexpr (kCombine) {
      constexpr int KB = NV == 1 ? 8 : (NV == 2 ? 4 : 2);
      for (int j0 = 0; j0 < p.k; j0 += KB) {
        uint4 buf[KB][NV];
        float w[KB];
#pragma unroll
        for (int u = 0; u < KB; ++u) {
          const bool slot = live && j0 + u < p.k;
          const int row = slot ? __ldg(p.row_of_slot + t * p.k + j0 + u) : -1;
          const bool there = row >= 0 && row < p.R;
          if (slot && !there) set_status(p.status, MOE_STATUS_BAD_INDEX);
          w[u] = there ? __ldg(p.topk_w + t * p.k + j0 + u) : 0.f;
#pragma unroll
          for (int i = 0; i < NV; ++i) {
            const int c = rg.l + i * L;
            buf[u][i] = there && c < nvec ? __ldg(reinterpret_cast<const uint4*>(p.z + (size_t)row * H) + c) : make_uint4(0, 0, 0, 0);
          }
        }
#pragma unroll
        for (int u = 0; u < KB; ++u)
#pragma unroll
          for (int i = 0; i < NV; ++i) {
            float f[8];
            unpack8(buf[u][i], f);
#pragma unroll
            for (int j = 0; j < 8; ++j) z[i][j] = __fmaf_rn(w[u], f[j], z[i][j]);
          }
      }
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = rg.l + i * L;
        if (live && c < nvec) unpack8(*(reinterpret_cast<const uint4*>(p.z + t * H) + c), z[i]);
      }
    }
    float r = 1.f;
    if (p.norm) {
      r = rg.template rstd<NV>(inv_h, p.eps, [&](int i, int j) { return z[i][j]; });
      if (p.rstd && live && rg.l == 0) p.rstd[t] = r;
    }
    float tok = p.out_scale;
    if (p.gate_kind == 1 && live) tok *= sigmoid(__ldg(static_cast<const float*>(p.gate) + t)).g;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = rg.l + i * L;
      const bool there = live && c < nvec;
      if (!there) continue;
      if (kCombine && p.z_out) Vec8<__nv_bfloat16>::store(p.z_out + t * H + 8 * c, z[i]);
      const Gain8 w(p.gain, c, true);
      float g[8];
      if (p.gate_kind == 2) unpack8(__ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.gate) + t * H) + c), g);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float v = z[i][j] * r * w.at(j) * tok;
        if (p.gate_kind == 2) v *= sigmoid(g[j]).g;
        if (residual) v = __fmaf_rn(p.res_scale, res[i].at(j), v);
        z[i][j] = v;
      }
      Vec8<S>::store(out + t * H + 8 * c, z[i]);
      if (sizeof(S) == 2) {  // the next norm is of what is stored
#pragma unroll
        for (int j = 0; j < 8; ++j) z[i][j] = __bfloat162float(__float2bfloat16_rn(z[i][j]));
      }
    }
    if (p.next_y) {
      const float q = rg.template rstd<NV>(inv_h, p.eps, [&](int i, int j) { return z[i][j]; });
      if (p.next_rstd && live && rg.l == 0) p.next_rstd[t] = q;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = rg.l + i * L;
        if (!live || c >= nvec) continue;
        const Gain8 w(p.next_gain, c, true);
        float o[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = z[i][j] * q * w.at(j);
        Vec8<__nv_bfloat16>::store(p.next_y + t * H + 8 * c, o);
      }
    }
  }
}

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

// dz may be z: a row's vectors are read before they are written by the same lane.
template <typename S, int L, int NV>
__global__ void __launch_bounds__(kNormThreads) post_norm_bwd_kernel(const PostBwdArgs p) {
  pdl_wait();
  pdl_trigger();
  __shared__ float sm[16];
  __shared__ float fold[kNormThreads * NV * 8];
  RowGroup<L> rg(sm);
  const int H = p.H, nvec = H / 8, T = p.T;
  const float inv_h = 1.0f / (float)H;
  const S* dout = static_cast<const S*>(p.dout);
  const __nv_bfloat16* gate2 = p.gate_kind == 2 ? static_cast<const __nv_bfloat16*>(p.gate) : nullptr;
  float acc[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[i][j] = 0.f;
  for (long long base = (long long)blockIdx.x * rg.kRows; base < T; base += (long long)gridDim.x * rg.kRows) {
    const long long t = base + rg.g;
    const bool live = t < T;
    Vec8<__nv_bfloat16> zv[NV], gv[NV];
    Vec8<S> d[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = rg.l + i * L;
      zv[i] = gv[i] = zero_vec<__nv_bfloat16>();
      d[i] = zero_vec<S>();
      if (live && c < nvec) {
        zv[i].load(p.z + t * H + 8 * c);
        d[i].load(dout + t * H + 8 * c);
        if (gate2) gv[i].load(gate2 + t * H + 8 * c);
      }
    }
    const float r = p.norm && live ? __ldg(p.rstd + t) : 1.f;
    Gate tok = {1.f, 0.f};
    if (p.gate_kind == 1 && live) tok = sigmoid(__ldg(static_cast<const float*>(p.gate) + t));
    float m = 0.f, dg = 0.f;  // sums of dn n, and of dout n gain
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = rg.l + i * L;
      const bool there = live && c < nvec;
      const Gain8 w(p.gain, c, c < nvec);
      float ds[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float n = zv[i].at(j) * r, e = p.out_scale * d[i].at(j);
        const Gate G = gate2 ? sigmoid(gv[i].at(j)) : tok;
        const float dv = e * G.g;
        acc[i][j] = __fmaf_rn(dv, n, acc[i][j]);
        m = __fmaf_rn(dv * w.at(j), n, m);
        dg = __fmaf_rn(e * w.at(j), n, dg);
        ds[j] = e * w.at(j) * n * G.d;
      }
      if (gate2 && p.dgate && there) Vec8<__nv_bfloat16>::store(static_cast<__nv_bfloat16*>(p.dgate) + t * H + 8 * c, ds);
    }
    if (p.norm) m = rg.sum(m) * inv_h;
    if (p.gate_kind == 1 && p.dgate) {
      dg = rg.sum(dg);
      if (live && rg.l == 0) static_cast<float*>(p.dgate)[t] = dg * tok.d;
    }
    if (!live) continue;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = rg.l + i * L;
      if (c >= nvec) continue;
      const Gain8 w(p.gain, c, true);
      float o[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float dn = p.out_scale * d[i].at(j) * (gate2 ? sigmoid(gv[i].at(j)).g : tok.g) * w.at(j);
        o[j] = p.norm ? r * (dn - zv[i].at(j) * r * m) : dn;
      }
      Vec8<__nv_bfloat16>::store(p.dz + t * H + 8 * c, o);
    }
  }
  if (p.part) leave_part<L, NV>(acc, fold, H, p.part);
}

// The combine keeps a token's k rows in flight in each lane: one vector a lane as
// long as a block's lanes can hold the row.
template <class F>
int with_combine_shape(int H, F&& f) {
  using std::integral_constant;
  if (H <= 256) return f(integral_constant<int, 32>{}, integral_constant<int, 1>{});
  if (H <= 512) return f(integral_constant<int, 64>{}, integral_constant<int, 1>{});
  if (H <= 1024) return f(integral_constant<int, 128>{}, integral_constant<int, 1>{});
  if (H <= 2048) return f(integral_constant<int, 256>{}, integral_constant<int, 1>{});
  if (H <= 4096) return f(integral_constant<int, 256>{}, integral_constant<int, 2>{});
  return f(integral_constant<int, 256>{}, integral_constant<int, 4>{});
}

template <typename S>
int run_post_norm(const char* fn, const PostArgs& a, bool combine, cudaStream_t s) {
  if (combine)
    return with_combine_shape(a.H, [&](auto l, auto nv) {
      constexpr int L = decltype(l)::value, NV = decltype(nv)::value;
      launch_pdl(post_norm_kernel<S, L, NV, true>, norm_grid(a.T, kNormThreads / L, 8, 1 << 30), kNormThreads, 0, s, a);
      return check_launch(fn);
    });
  return with_row_shape(a.H, [&](auto l, auto nv) {
    constexpr int L = decltype(l)::value, NV = decltype(nv)::value;
    launch_pdl(post_norm_kernel<S, L, NV, false>, norm_grid(a.T, kNormThreads / L, 8, 1 << 30), kNormThreads, 0, s, a);
    return check_launch(fn);
  });
}

int check_post(const char* fn, int T, int H, int fp32, int norm, int gate_kind) {
  if (int rc = check_norm(fn, T, H, fp32)) return rc;
  if ((norm != 0 && norm != 1) || gate_kind < 0 || gate_kind > 2)
    return fail(MOE_ERR_INVALID_ARG, "%s: need norm 0 or 1, gate_kind 0, 1 or 2", fn);
  return MOE_OK;
}

bool gate_aligned(int kind, const void* gate) {
  return kind == 2 ? aligned16(gate) : (reinterpret_cast<uintptr_t>(gate) & 3u) == 0;
}

// The arguments that both forward calls check.
int check_post_fwd(const char* fn, const PostArgs& a) {
  if (!(a.eps > 0.f && a.eps <= 3.402823466e+38f)) return fail(MOE_ERR_INVALID_ARG, "%s: need eps>0", fn);
  if (a.T == 0) return MOE_OK;
  if (!a.z || !a.out || (a.gate_kind && !a.gate)) return fail(MOE_ERR_INVALID_ARG, "%s: NULL pointer argument", fn);
  if (!a.next_y && (a.next_gain || a.next_rstd)) return fail(MOE_ERR_INVALID_ARG, "%s: next_gain and next_rstd need next_y", fn);
  for (const void* q : {static_cast<const void*>(a.z), a.residual, static_cast<const void*>(a.gain), static_cast<const void*>(a.z_out),
                        static_cast<const void*>(a.out), static_cast<const void*>(a.next_gain), static_cast<const void*>(a.next_y)})
    if (!aligned16(q)) return fail(MOE_ERR_ALIGNMENT, "%s: tensors must be 16-byte aligned", fn);
  if (!gate_aligned(a.gate_kind, a.gate)) return fail(MOE_ERR_ALIGNMENT, "%s: gate is not aligned", fn);
  return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

int moe_post_norm(const void* z, const void* residual, int fp32, const float* gain, int norm, float eps, int gate_kind,
                  const void* gate, float res_scale, float out_scale, int T, int H, void* out, float* rstd, const float* next_gain,
                  void* next_y, float* next_rstd, void* stream) {
  clear_error();
  const char* fn = "moe_post_norm";
  if (int rc = check_post(fn, T, H, fp32, norm, gate_kind)) return rc;
  PostArgs a = {static_cast<const __nv_bfloat16*>(z), nullptr, nullptr, 0, 0, residual, gain, norm, eps, gate_kind, gate, res_scale,
                out_scale, T, H, nullptr, out, rstd, next_gain, static_cast<__nv_bfloat16*>(next_y), next_rstd, nullptr};
  if (int rc = check_post_fwd(fn, a)) return rc;
  if (T == 0) return MOE_OK;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return fp32 ? run_post_norm<float>(fn, a, false, s) : run_post_norm<__nv_bfloat16>(fn, a, false, s);
}

int moe_combine_post_norm(const void* y_perm, const float* topk_w, const int32_t* row_of_slot, const void* residual, int fp32,
                          const float* gain, int norm, float eps, int gate_kind, const void* gate, float res_scale, float out_scale,
                          int T, int H, int k, void* z, void* out, float* rstd, const float* next_gain, void* next_y,
                          float* next_rstd, void* stream) {
  clear_error();
  const char* fn = "moe_combine_post_norm";
  if (k <= 0) return fail(MOE_ERR_INVALID_ARG, "%s: need k>0", fn);
  if (int rc = check_post(fn, T, H, fp32, norm, gate_kind)) return rc;
  if (H % 64 || k > kMaxTopK || (long long)T * k >= (1ll << 31))
    return fail(MOE_ERR_UNSUPPORTED_SHAPE, "%s: need H%%64==0, k<=32, T*k<2^31", fn);
  PostArgs a = {static_cast<const __nv_bfloat16*>(y_perm), topk_w, row_of_slot, k, T * k, residual, gain, norm, eps, gate_kind, gate,
                res_scale, out_scale, T, H, static_cast<__nv_bfloat16*>(z), out, rstd, next_gain, static_cast<__nv_bfloat16*>(next_y),
                next_rstd, nullptr};
  if (int rc = check_post_fwd(fn, a)) return rc;
  if (T == 0) return MOE_OK;
  if (!topk_w || !row_of_slot) return fail(MOE_ERR_INVALID_ARG, "%s: NULL pointer argument", fn);
  a.status = status_word();
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return fp32 ? run_post_norm<float>(fn, a, true, s) : run_post_norm<__nv_bfloat16>(fn, a, true, s);
}

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
  return with_row_shape(H, [&](auto l, auto nv) {
    constexpr int L = decltype(l)::value, NV = decltype(nv)::value;
    const int grid = norm_grid(T, kNormThreads / L, 2, kNormParts);
    if (fp32)
      launch_pdl(post_norm_bwd_kernel<float, L, NV>, grid, kNormThreads, 0, s, a);
    else
      launch_pdl(post_norm_bwd_kernel<__nv_bfloat16, L, NV>, grid, kNormThreads, 0, s, a);
    if (int rc = check_launch(fn)) return rc;
    return dgain ? launch_gain_sum(fn, static_cast<const float*>(ws), grid, H, dgain, accumulate, s) : MOE_OK;
  });
}

}  // extern "C"
