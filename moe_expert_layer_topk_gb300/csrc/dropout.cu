// Dropout whose mask is computed from a counter and never stored: alone, in
// the weighted combine (with the residual added), and in the combine's
// backward.
//
// Mask: Philox4x32-10 (Salmon, Moraes, Dror, Shaw, "Parallel random numbers:
// as easy as 1, 2, 3", SC 2011), key = rng[0], 64-bit counter = rng[1] + i/8
// for element i of the tensor in row-major order.  One evaluation's 128 bits
// are eight 16-bit numbers, one per element of a 16-byte bf16 vector, so a
// thread evaluates the generator once per vector it already holds and the
// backward recomputes the same bits from the same (key, counter).  Sixteen
// bits an element halve the generator's work against 32; the drop
// probability is the multiple of 2^-16 nearest to p, and the scale
// 65536/(65536 - drop) is that probability's own, so the expectation is
// exact.
//
// A dropped element is selected away, not multiplied by zero: an infinity or
// a NaN under the mask does not reach the output.
#include "common.cuh"

namespace moe {
namespace {

// drop counts 16-bit numbers: element i stays when its number is >= drop.
struct DropParams {
  uint32_t drop;  // 0..65536
  float scale;    // 65536 / (65536 - drop), 0 when everything is dropped
};

struct PhiloxKey {
  uint32_t k0, k1;
  unsigned long long base;  // counter of the tensor's first eight elements
};

__device__ __forceinline__ PhiloxKey load_key(const unsigned long long* rng) {
  const unsigned long long s = __ldg(rng), o = __ldg(rng + 1);
  return {(uint32_t)s, (uint32_t)(s >> 32), o};
}

// The eight 16-bit numbers of elements 8b .. 8b+7, two to a word, lowest first.
__device__ __forceinline__ uint4 philox8(const PhiloxKey& k, unsigned long long b) {
  const unsigned long long ctr = k.base + b;
  uint32_t c0 = (uint32_t)ctr, c1 = (uint32_t)(ctr >> 32), c2 = 0, c3 = 0;
  uint32_t k0 = k.k0, k1 = k.k1;
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const unsigned long long p0 = (unsigned long long)0xD2511F53u * c0;
    const unsigned long long p1 = (unsigned long long)0xCD9E8D57u * c2;
    c0 = (uint32_t)(p1 >> 32) ^ c1 ^ k0;
    c1 = (uint32_t)p1;
    c2 = (uint32_t)(p0 >> 32) ^ c3 ^ k1;
    c3 = (uint32_t)p0;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return make_uint4(c0, c1, c2, c3);
}

// Whether element i (0..7) of a generator block stays.
__device__ __forceinline__ bool stays(const uint4& w, int i, uint32_t drop) {
  const uint32_t v = i < 2 ? w.x : (i < 4 ? w.y : (i < 6 ? w.z : w.w));
  return ((i & 1) ? v >> 16 : v & 0xFFFFu) >= drop;
}

// ------------------------------------------------------------- elementwise
// out = residual + D(x), fp32 arithmetic, one rounding.
// Eight elements as they lie in memory.
template <typename T>
struct Vec8;
template <>
struct Vec8<__nv_bfloat16> {
  uint4 q;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { q = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ float at(int i) const {
    const uint32_t w = i < 2 ? q.x : (i < 4 ? q.y : (i < 6 ? q.z : q.w));
    return (i & 1) ? bf16hi(w) : bf16lo(w);
  }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, const float (&f)[8]) {
    *reinterpret_cast<uint4*>(p) = pack8(f);
  }
  static __device__ __forceinline__ float one(const __nv_bfloat16* p) { return __bfloat162float(*p); }
  static __device__ __forceinline__ __nv_bfloat16 round(float v) { return __float2bfloat16_rn(v); }
};
template <>
struct Vec8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ float at(int i) const {
    const float4& v = i < 4 ? a : b;
    return (i & 3) == 0 ? v.x : ((i & 3) == 1 ? v.y : ((i & 3) == 2 ? v.z : v.w));
  }
  static __device__ __forceinline__ void store(float* p, const float (&f)[8]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
  }
  static __device__ __forceinline__ float one(const float* p) { return *p; }
  static __device__ __forceinline__ float round(float v) { return v; }
};

// x may be out (every element is read before it is written by its thread).
// One generator block of eight elements a thread, their vectors held as they lie
// in memory (16.8 M bf16 elements with a residual: 15.1 us, 6.7 TB/s, fp32 30.8;
// unpacked first 16.8, and then with two blocks a thread 18.3, four 19.4: the
// registers they take cost more warps than their loads are worth).
template <typename T>
__global__ void __launch_bounds__(256) dropout_kernel(const T* x, const T* residual, long long n, DropParams dp,
                                                      const unsigned long long* __restrict__ rng, T* out) {
  pdl_wait();
  pdl_trigger();
  const PhiloxKey key = load_key(rng);
  const long long nb = (n + 7) / 8, whole = n / 8;
  for (long long b = blockIdx.x * (long long)blockDim.x + threadIdx.x; b < nb; b += (long long)gridDim.x * blockDim.x) {
    if (b < whole) {
      Vec8<T> v, r;
      v.load(x + 8 * b);
      if (residual) r.load(residual + 8 * b);
      const uint4 w = philox8(key, b);
      float o[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float d = stays(w, i, dp.drop) ? v.at(i) * dp.scale : 0.f;
        o[i] = residual ? r.at(i) + d : d;
      }
      Vec8<T>::store(out + 8 * b, o);
    } else {  // the last, partial block
      const uint4 w = philox8(key, b);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const long long j = 8 * b + i;
        if (j < n) {
          const float d = stays(w, i, dp.drop) ? Vec8<T>::one(x + j) * dp.scale : 0.f;
          out[j] = Vec8<T>::round(residual ? Vec8<T>::one(residual + j) + d : d);
        }
      }
    }
  }
}

// ----------------------------------------------------------------- combine
// Thread = two 16-byte vectors (16 columns) of one token: the fp32 sum over the
// slots in order (KB of them loaded at a time), dropout on that sum, the
// residual, one bf16 rounding.  Two persistent CTAs an SM; the row ids and
// weights of a thread's next batch are under way while this one is summed.
//
// Bound by HBM: what counts is bytes in flight, 256 a thread at KB = 8.
// Measured at 8192 x 2048, top-8: 55.9 us (6.0 TB/s); one vector a thread and a
// CTA for each 256 of them 61.7 (12.4 against 13.8 us at 2000 tokens, whose
// rows the L2 holds); top-2 30.3 against 40.5.
template <int KB>
__global__ void __launch_bounds__(256, 2) combine_dropout_kernel(
    const __nv_bfloat16* __restrict__ y_perm, const float* __restrict__ topk_w,
    const int32_t* __restrict__ row_of_slot, const __nv_bfloat16* residual, int T, int H, int k, int R,
    DropParams dp, const unsigned long long* __restrict__ rng, __nv_bfloat16* y, int* status) {
  pdl_wait();
  pdl_trigger();
  const PhiloxKey key = load_key(rng);
  constexpr int NV = 2;
  const int nvec = H / (8 * NV);
  // thread -> (token, piece), advanced by the grid without a division
  const size_t gid = (size_t)blockIdx.x * blockDim.x + threadIdx.x, step = (size_t)gridDim.x * blockDim.x;
  long long t = (long long)(gid / nvec);
  int v = (int)(gid % nvec);
  const int dt = (int)(step / nvec), dv = (int)(step % nvec);
  int next_row[KB];
  float next_w[KB];
  auto fetch = [&](long long t, int j0) {
#pragma unroll
    for (int u = 0; u < KB; ++u) {
      next_row[u] = -1;
      next_w[u] = 0.f;
      if (t < T && j0 + u < k) {
        next_row[u] = __ldg(row_of_slot + (size_t)t * k + j0 + u);
        next_w[u] = __ldg(topk_w + (size_t)t * k + j0 + u);
      }
    }
  };
  fetch(t, 0);
  while (t < T) {
    const int c0 = v * 8 * NV;
    const long long here = t;
    const size_t at = (size_t)here * H + c0;
    v += dv;
    t += dt + (v >= nvec);  // the thread's next piece
    if (v >= nvec) v -= nvec;
    uint4 res[NV];
#pragma unroll
    for (int q = 0; q < NV; ++q)
      res[q] = residual ? reinterpret_cast<const uint4*>(residual + at)[q] : make_uint4(0, 0, 0, 0);
    float acc[8 * NV];
#pragma unroll
    for (int i = 0; i < 8 * NV; ++i) acc[i] = 0.f;
    for (int j0 = 0; j0 < k; j0 += KB) {
      uint4 buf[KB][NV];
      float w[KB];
#pragma unroll
      for (int u = 0; u < KB; ++u) {
        const int row = next_row[u];
        const bool there = row >= 0 && row < R;
        if (j0 + u < k && !there) set_status(status, MOE_STATUS_BAD_INDEX);
        w[u] = there ? next_w[u] : 0.f;
#pragma unroll
        for (int q = 0; q < NV; ++q)
          buf[u][q] = there ? __ldg(reinterpret_cast<const uint4*>(y_perm + (size_t)row * H + c0) + q) : make_uint4(0, 0, 0, 0);
      }
      if (j0 + KB < k)
        fetch(here, j0 + KB);
      else
        fetch(t, 0);
#pragma unroll
      for (int u = 0; u < KB; ++u) {
        if (j0 + u < k) {
#pragma unroll
          for (int q = 0; q < NV; ++q) {
            float f[8];
            unpack8(buf[u][q], f);
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[8 * q + i] = __fmaf_rn(w[u], f[i], acc[8 * q + i]);
          }
        }
      }
    }
#pragma unroll
    for (int q = 0; q < NV; ++q) {
      const uint4 bits = philox8(key, at / 8 + q);
      float r[8], o[8];
      unpack8(res[q], r);
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = r[i] + (stays(bits, i, dp.drop) ? acc[8 * q + i] * dp.scale : 0.f);
      reinterpret_cast<uint4*>(y + at)[q] = pack8(o);
    }
  }
}

// bf16 element pairs of a vector with the dropped ones replaced by zero
__device__ __forceinline__ uint4 select8(uint4 v, const uint4& bits, uint32_t drop) {
  uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] &= (stays(bits, 2 * i, drop) ? 0xFFFFu : 0u) | (stays(bits, 2 * i + 1, drop) ? 0xFFFF0000u : 0u);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// A warp's sum of dy . y_perm over the elements that stay, both rows' dropped
// elements selected away: added up as the kernel below does.
__device__ __noinline__ float dot_of_kept(const uint4* dy, const uint4* y, const unsigned long long* rng, uint32_t drop,
                                          unsigned long long block0, int nvec) {
  const PhiloxKey key = load_key(rng);
  float sum = 0.f;
#pragma unroll 1
  for (int v0 = 0; v0 < nvec; v0 += 256) {
    float p = 0.f;
#pragma unroll 1
    for (int v = v0 + (threadIdx.x & 31); v < min(nvec, v0 + 256); v += 32) {
      const uint4 bits = philox8(key, block0 + v);
      float g[8], yv[8];
      unpack8(select8(__ldg(dy + v), bits, drop), g);
      unpack8(select8(__ldg(y + v), bits, drop), yv);
#pragma unroll
      for (int i = 0; i < 8; ++i) p = __fmaf_rn(g[i], yv[i], p);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) p += __shfl_xor_sync(0xffffffffu, p, off);
    sum += p;
  }
  return sum;
}

// Warp per token: the token's dy row with its dropped elements zeroed sits in
// registers; for every slot the warp writes dy_perm[row] = (w scale) dy[t] and
// reduces dy[t] . y_perm[row]; the scale is applied to the sum once.  A dropped
// element of y_perm meets a zero of dy there, which an infinity or a NaN turns
// into NaN: a sum that is not finite is taken again over the elements that stay
// (selecting them away each time cost 6% at 2048 columns, 26% at 512).
//
// Bound by HBM at 2048 columns (8192 tokens, top-8: 89.6 us, 6.4 TB/s; top-2
// 31.1).  The eight vectors a lane holds are 2048 columns: narrower rows leave
// some of them empty, and a token's slots follow one another (top-8: 1024 columns
// 57.0 us, 512 43.7, 256 27.9, 128 25.9, of which HBM needs 42, 21, 11 and 5).
__global__ void __launch_bounds__(64) combine_dropout_bwd_kernel(
    const __nv_bfloat16* __restrict__ dy, const __nv_bfloat16* __restrict__ y_perm,
    const float* __restrict__ topk_w, const int32_t* __restrict__ row_of_slot, int T, int H, int k, int R,
    DropParams dp, const unsigned long long* __restrict__ rng, __nv_bfloat16* __restrict__ dy_perm,
    float* __restrict__ d_w, int* status) {
  pdl_wait();
  pdl_trigger();
  const PhiloxKey key = load_key(rng);
  const int lane = threadIdx.x & 31;
  const int nvec = H / 8;
  const unsigned nw = (gridDim.x * blockDim.x) >> 5;
  for (unsigned t = (blockIdx.x * blockDim.x + threadIdx.x) >> 5; t < (unsigned)T; t += nw) {
    int my_row = lane < k ? __ldg(row_of_slot + (size_t)t * k + lane) : -1;
    const float my_w = lane < k ? __ldg(topk_w + (size_t)t * k + lane) * dp.scale : 0.f;
    if (lane < k && (my_row < 0 || my_row >= R)) {
      set_status(status, MOE_STATUS_BAD_INDEX);
      my_row = -1;
    }
    float my_dw = 0.f;
    for (int v0 = 0; v0 < nvec; v0 += 256) {
      uint4 gp[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int v = v0 + u * 32 + lane;
        gp[u] = v < nvec ? __ldg(reinterpret_cast<const uint4*>(dy + (size_t)t * H) + v) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int v = v0 + u * 32 + lane;
        if (v < nvec) gp[u] = select8(gp[u], philox8(key, (unsigned long long)t * nvec + v), dp.drop);
      }
      for (int j = 0; j < k; ++j) {
        const int row = __shfl_sync(0xffffffffu, my_row, j);
        const float w = __shfl_sync(0xffffffffu, my_w, j);
        if (row < 0) continue;  // uniform across the warp
        uint4 yb[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const int v = v0 + u * 32 + lane;
          yb[u] = v < nvec ? __ldg(reinterpret_cast<const uint4*>(y_perm + (size_t)row * H) + v)
                           : make_uint4(0, 0, 0, 0);
        }
        float p = 0.f;
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const int v = v0 + u * 32 + lane;
          float g[8], yv[8], o[8];
          unpack8(gp[u], g);
          unpack8(yb[u], yv);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            o[i] = w * g[i];
            p = __fmaf_rn(g[i], yv[i], p);
          }
          if (v < nvec) reinterpret_cast<uint4*>(dy_perm + (size_t)row * H)[v] = pack8(o);
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) p += __shfl_xor_sync(0xffffffffu, p, off);
        if (lane == j) my_dw += p;
      }
    }
    for (unsigned again = __ballot_sync(0xffffffffu, !isfinite(my_dw)); again; again &= again - 1) {
      const int j = __ffs(again) - 1, row = __shfl_sync(0xffffffffu, my_row, j);
      const float p = dot_of_kept(reinterpret_cast<const uint4*>(dy + (size_t)t * H), reinterpret_cast<const uint4*>(y_perm + (size_t)row * H),
                                  rng, dp.drop, (unsigned long long)t * nvec, nvec);
      if (lane == j) my_dw = p;
    }
    if (lane < k) d_w[(size_t)t * k + lane] = my_dw * dp.scale;
  }
}

// --------------------------------------------------------------- host side

int drop_params(const char* fn, double p, const void* rng, DropParams* dp) {
  if (!(p >= 0.0 && p <= 1.0)) return fail(MOE_ERR_INVALID_ARG, "%s: need 0 <= p <= 1", fn);
  if (!rng) return fail(MOE_ERR_INVALID_ARG, "%s: NULL pointer argument", fn);
  if (!aligned16(rng)) return fail(MOE_ERR_ALIGNMENT, "%s: rng must be 16-byte aligned", fn);
  dp->drop = (uint32_t)(p * 65536.0 + 0.5);
  dp->scale = dp->drop < 65536u ? (float)(65536.0 / (65536.0 - dp->drop)) : 0.f;
  return MOE_OK;
}

int grid_for(size_t work, int per_block, int per_sm) {
  const size_t b = (work + per_block - 1) / per_block;
  const size_t cap = (size_t)(sm_count() > 0 ? sm_count() : 148) * per_sm;
  return (int)(b < cap ? (b > 0 ? b : 1) : cap);
}

int check_combine(const char* fn, int T, int H, int k) {
  if (T < 0 || H <= 0 || k <= 0) return fail(MOE_ERR_INVALID_ARG, "%s: need T>=0, H>0, k>0", fn);
  if (H % 64 != 0 || k > kMaxTopK || (long long)T * k >= (1ll << 31))
    return fail(MOE_ERR_UNSUPPORTED_SHAPE, "%s: need H%%64==0, k<=32, T*k<2^31", fn);
  return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

int moe_dropout(const void* x, const void* residual, long long n, int fp32, double p, const int64_t* rng, void* out,
                void* stream) {
  clear_error();
  const char* fn = "moe_dropout";
  DropParams dp;
  if (n < 0 || (fp32 != 0 && fp32 != 1)) return fail(MOE_ERR_INVALID_ARG, "%s: need n>=0, fp32 0 or 1", fn);
  if (n == 0) return MOE_OK;
  if (int rc = drop_params(fn, p, rng, &dp)) return rc;
  if (!x || !out) return fail(MOE_ERR_INVALID_ARG, "%s: NULL pointer argument", fn);
  if (!aligned16(x) || !aligned16(out) || (residual && !aligned16(residual)))
    return fail(MOE_ERR_ALIGNMENT, "%s: x, residual and out must be 16-byte aligned", fn);
  const int grid = grid_for((size_t)(n + 7) / 8, 256, 16);
  const auto* r = reinterpret_cast<const unsigned long long*>(rng);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (fp32)
    launch_pdl(dropout_kernel<float>, grid, 256, 0, s, static_cast<const float*>(x),
               static_cast<const float*>(residual), n, dp, r, static_cast<float*>(out));
  else
    launch_pdl(dropout_kernel<__nv_bfloat16>, grid, 256, 0, s, static_cast<const __nv_bfloat16*>(x),
               static_cast<const __nv_bfloat16*>(residual), n, dp, r, static_cast<__nv_bfloat16*>(out));
  return check_launch(fn);
}

int moe_combine_dropout(const void* y_perm, const float* topk_w, const int32_t* row_of_slot, const void* residual,
                        int T, int H, int k, double p, const int64_t* rng, void* y, void* stream) {
  clear_error();
  const char* fn = "moe_combine_dropout";
  DropParams dp;
  if (int rc = check_combine(fn, T, H, k)) return rc;
  if (T == 0) return MOE_OK;
  if (int rc = drop_params(fn, p, rng, &dp)) return rc;
  if (!y_perm || !topk_w || !row_of_slot || !y) return fail(MOE_ERR_INVALID_ARG, "%s: NULL pointer argument", fn);
  if (!aligned16(y_perm) || !aligned16(y) || (residual && !aligned16(residual)))
    return fail(MOE_ERR_ALIGNMENT, "%s: y_perm, residual and y must be 16-byte aligned", fn);
  auto run = [&](auto kern) {
    launch_pdl(kern, grid_for((size_t)T * (H / 16), 256, 2), 256, 0, static_cast<cudaStream_t>(stream),
               static_cast<const __nv_bfloat16*>(y_perm), topk_w, row_of_slot,
               static_cast<const __nv_bfloat16*>(residual), T, H, k, T * k, dp,
               reinterpret_cast<const unsigned long long*>(rng), static_cast<__nv_bfloat16*>(y), status_word());
  };
  if (k <= 2)
    run(combine_dropout_kernel<2>);
  else if (k <= 4)
    run(combine_dropout_kernel<4>);
  else
    run(combine_dropout_kernel<8>);
  return check_launch(fn);
}

int moe_combine_dropout_bwd(const void* dy, const void* y_perm, const float* topk_w, const int32_t* row_of_slot,
                            int T, int H, int k, double p, const int64_t* rng, void* dy_perm, float* d_w,
                            void* stream) {
  clear_error();
  const char* fn = "moe_combine_dropout_bwd";
  DropParams dp;
  if (int rc = check_combine(fn, T, H, k)) return rc;
  if (T == 0) return MOE_OK;
  if (int rc = drop_params(fn, p, rng, &dp)) return rc;
  if (!dy || !y_perm || !topk_w || !row_of_slot || !dy_perm || !d_w)
    return fail(MOE_ERR_INVALID_ARG, "%s: NULL pointer argument", fn);
  if (!aligned16(dy) || !aligned16(y_perm) || !aligned16(dy_perm))
    return fail(MOE_ERR_ALIGNMENT, "%s: dy, y_perm and dy_perm must be 16-byte aligned", fn);
  launch_pdl(combine_dropout_bwd_kernel, grid_for((size_t)T * 32, 64, 32), 64, 0, static_cast<cudaStream_t>(stream),
             static_cast<const __nv_bfloat16*>(dy), static_cast<const __nv_bfloat16*>(y_perm), topk_w, row_of_slot, T,
             H, k, T * k, dp, reinterpret_cast<const unsigned long long*>(rng),
             static_cast<__nv_bfloat16*>(dy_perm), d_w, status_word());
  return check_launch(fn);
}

}  // extern "C"
