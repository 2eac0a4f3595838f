// Activations kept in 8 bits: packing bf16 rows, bringing them back, and the
// experts' permuted rows made from tokens kept either way.  The experts' products
// that write and read such rows are kinds of the grouped GEMMs.
//
// Format: whole numbers of 8 bits with one bf16 scale for each 32 columns of a row,
// 1.0625 bytes an element.  For normally distributed columns the error is 0.5% of
// their size (relative L2), against 2.6% for e4m3 codes with any scale.
//
// All three are bound by HBM.
#include "common.cuh"

namespace moe {
namespace {

// Thread = sixteen columns; the two threads of a group of 32 share its amax.  8192 x 2048
// and back: 16.4 us, with eight columns a thread 18.1.
__global__ void __launch_bounds__(256) ckpt_pack_kernel(const __nv_bfloat16* __restrict__ a, size_t n16, uint4* __restrict__ q,
                                                        __nv_bfloat16* __restrict__ scale) {
  pdl_wait();
  pdl_trigger();
  const size_t step = (size_t)gridDim.x * blockDim.x;
  for (size_t first = blockIdx.x * (size_t)blockDim.x + (threadIdx.x & ~31u); first < n16; first += step) {
    const size_t v = first + (threadIdx.x & 31);
    float f[8], g[8];
    const uint4* p = reinterpret_cast<const uint4*>(a) + 2 * v;
    unpack8(v < n16 ? __ldg(p) : make_uint4(0, 0, 0, 0), f);
    unpack8(v < n16 ? __ldg(p + 1) : make_uint4(0, 0, 0, 0), g);
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = amax_nan(amax_nan(m, f[i]), g[i]);
    m = amax_nan(m, __shfl_xor_sync(0xffffffffu, m, 1));
    const float s = ckpt_scale(m), inv = __frcp_rn(s);
    if (v < n16) {
      q[v] = make_uint4(ckpt_codes4(f[0], f[1], f[2], f[3], inv), ckpt_codes4(f[4], f[5], f[6], f[7], inv),
                        ckpt_codes4(g[0], g[1], g[2], g[3], inv), ckpt_codes4(g[4], g[5], g[6], g[7], inv));
      if ((v & 1) == 0) scale[v >> 1] = __ushort_as_bfloat16((unsigned short)(__float_as_uint(s) >> 16));
    }
  }
}

__device__ __forceinline__ uint4 unpack_codes8(uint2 w, uint32_t scale_bits) {
  const float s = bf16_bits(scale_bits);
  float a[4], b[4];
  ckpt_decode4(w.x, s, a);
  ckpt_decode4(w.y, s, b);
  return make_uint4(pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3]), pack_bf16x2(b[0], b[1]), pack_bf16x2(b[2], b[3]));
}

__global__ void __launch_bounds__(256) ckpt_unpack_kernel(const uint2* __restrict__ q, const unsigned short* __restrict__ scale,
                                                          size_t nvec, uint4* __restrict__ a) {
  pdl_wait();
  pdl_trigger();
  for (size_t v = blockIdx.x * (size_t)blockDim.x + threadIdx.x; v < nvec; v += (size_t)gridDim.x * blockDim.x)
    a[v] = unpack_codes8(__ldg(q + v), __ldg(scale + (v >> 2)));
}

// Warp = 64 vectors (512 columns) of one token, written to its k rows, whose ids its
// lanes hold.  8192 x 2048 from codes, top-8: 47.4 us (6.1 TB/s); a vector a lane 50.2, with
// the ids read by every thread 51.5; four vectors 47.7, eight 49.0.
template <bool kCodes>
__global__ void __launch_bounds__(256) dispatch_rows_kernel(const void* __restrict__ x, const unsigned short* __restrict__ scale,
                                                            const int32_t* __restrict__ row_of_slot, const float* __restrict__ topk_w,
                                                            int T, int H, int k, int R, uint4* __restrict__ x_perm,
                                                            float* __restrict__ row_w, int* status) {
  pdl_wait();
  pdl_trigger();
  constexpr int NV = 2;
  const int lane = threadIdx.x & 31, nvec = H / 8, pieces = (nvec + 32 * NV - 1) / (32 * NV);
  const size_t total = (size_t)T * pieces, nw = (size_t)gridDim.x * 8;
  for (size_t i = blockIdx.x * (size_t)8 + (threadIdx.x >> 5); i < total; i += nw) {
    const size_t t = i / pieces;
    const int v0 = (int)(i - t * pieces) * 32 * NV + lane;
    int row = lane < k ? __ldg(row_of_slot + t * k + lane) : 0;
    uint4 val[NV];
#pragma unroll
    for (int q = 0; q < NV; ++q) {
      const int v = v0 + 32 * q;
      val[q] = make_uint4(0, 0, 0, 0);
      if (v < nvec) {
        const size_t at = t * nvec + v;
        val[q] = kCodes ? unpack_codes8(__ldg(static_cast<const uint2*>(x) + at), __ldg(scale + (at >> 2))) : __ldg(static_cast<const uint4*>(x) + at);
      }
    }
    if (row < 0 || row >= R) {
      set_status(status, MOE_STATUS_BAD_INDEX);
      row = -1;
    }
    if (v0 == lane && row_w && lane < k && row >= 0) row_w[row] = __ldg(topk_w + t * k + lane);
    for (int j = 0; j < k; ++j) {
      const int r = __shfl_sync(0xffffffffu, row, j);
      if (r < 0) continue;
#pragma unroll
      for (int q = 0; q < NV; ++q)
        if (v0 + 32 * q < nvec) x_perm[(size_t)r * nvec + v0 + 32 * q] = val[q];
    }
  }
}

// Rows within less than a warp's 32 vectors (H < 256): thread = one vector of a token, the ids
// read by each.  65536 tokens, top-2, from codes: H = 64 5.6 us, 128 13.1; with the kernel
// above, whose lanes are then mostly idle, 14.7 and 17.0 (H = 256, top-4: 17.3 against 16.1).
template <bool kCodes>
__global__ void __launch_bounds__(256) dispatch_short_rows_kernel(const void* __restrict__ x, const unsigned short* __restrict__ scale,
                                                            const int32_t* __restrict__ row_of_slot, const float* __restrict__ topk_w,
                                                            int T, int H, int k, int R, uint4* __restrict__ x_perm,
                                                            float* __restrict__ row_w, int* status) {
  pdl_wait();
  pdl_trigger();
  const int nvec = H / 8;
  const size_t total = (size_t)T * nvec;
  for (size_t i = blockIdx.x * (size_t)blockDim.x + threadIdx.x; i < total; i += (size_t)gridDim.x * blockDim.x) {
    const size_t t = i / nvec;
    const int v = (int)(i - t * nvec);
    uint4 val;
    if (kCodes)
      val = unpack_codes8(__ldg(static_cast<const uint2*>(x) + i), __ldg(scale + (i >> 2)));
    else
      val = __ldg(static_cast<const uint4*>(x) + i);
    for (int j = 0; j < k; ++j) {
      const int row = __ldg(row_of_slot + t * k + j);
      if (row < 0 || row >= R) {
        if (v == 0) set_status(status, MOE_STATUS_BAD_INDEX);
        continue;
      }
      x_perm[(size_t)row * nvec + v] = val;
      if (v == 0 && row_w) row_w[row] = __ldg(topk_w + t * k + j);
    }
  }
}

int grid_of(size_t work, int per_sm) {
  const size_t b = (work + 255) / 256, cap = (size_t)(sm_count() > 0 ? sm_count() : 148) * per_sm;
  return (int)(b < cap ? b : cap);
}

int check_rows(const char* fn, int rows, int cols) {
  if (rows < 0 || cols <= 0) return fail(MOE_ERR_INVALID_ARG, "%s: need rows>=0, cols>0", fn);
  if (cols % kCkptGroup) return fail(MOE_ERR_UNSUPPORTED_SHAPE, "%s: need cols%%32==0 (cols=%d)", fn, cols);
  return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

int moe_ckpt_pack(const void* a, int rows, int cols, void* q, void* scale, void* stream) {
  clear_error();
  const char* fn = "moe_ckpt_pack";
  if (int rc = check_rows(fn, rows, cols)) return rc;
  if (rows == 0) return MOE_OK;
  if (!a || !q || !scale) return fail(MOE_ERR_INVALID_ARG, "%s: NULL pointer argument", fn);
  if (!aligned16(a) || !aligned16(q) || !aligned16(scale)) return fail(MOE_ERR_ALIGNMENT, "%s: tensors must be 16-byte aligned", fn);
  const size_t nvec = (size_t)rows * (cols / 8);
  launch_pdl(ckpt_pack_kernel, grid_of(nvec / 2, 16), 256, 0, static_cast<cudaStream_t>(stream), static_cast<const __nv_bfloat16*>(a), nvec / 2,
             static_cast<uint4*>(q), static_cast<__nv_bfloat16*>(scale));
  return check_launch(fn);
}

int moe_ckpt_unpack(const void* q, const void* scale, int rows, int cols, void* a, void* stream) {
  clear_error();
  const char* fn = "moe_ckpt_unpack";
  if (int rc = check_rows(fn, rows, cols)) return rc;
  if (rows == 0) return MOE_OK;
  if (!a || !q || !scale) return fail(MOE_ERR_INVALID_ARG, "%s: NULL pointer argument", fn);
  if (!aligned16(a) || !aligned16(q) || !aligned16(scale)) return fail(MOE_ERR_ALIGNMENT, "%s: tensors must be 16-byte aligned", fn);
  const size_t nvec = (size_t)rows * (cols / 8);
  launch_pdl(ckpt_unpack_kernel, grid_of(nvec, 16), 256, 0, static_cast<cudaStream_t>(stream), static_cast<const uint2*>(q),
             static_cast<const unsigned short*>(scale), nvec, static_cast<uint4*>(a));
  return check_launch(fn);
}

int moe_dispatch_rows(const void* x, const void* scale, const int32_t* row_of_slot, const float* topk_w, int T, int H, int k,
                      void* x_perm, float* row_w, void* stream) {
  clear_error();
  const char* fn = "moe_dispatch_rows";
  if (T < 0 || H <= 0 || k <= 0) return fail(MOE_ERR_INVALID_ARG, "%s: need T>=0, H>0, k>0", fn);
  if (H % 64 || k > kMaxTopK || (long long)T * k >= (1ll << 31))
    return fail(MOE_ERR_UNSUPPORTED_SHAPE, "%s: need H%%64==0, k<=32, T*k<2^31", fn);
  if (T == 0) return MOE_OK;
  if (!x || !row_of_slot || !x_perm) return fail(MOE_ERR_INVALID_ARG, "%s: NULL pointer argument", fn);
  if (!topk_w != !row_w) return fail(MOE_ERR_INVALID_ARG, "%s: topk_w and row_w are given together", fn);
  if (!aligned16(x) || !aligned16(x_perm) || (scale && !aligned16(scale)))
    return fail(MOE_ERR_ALIGNMENT, "%s: tensors must be 16-byte aligned", fn);
  auto run = [&](auto kern, size_t threads) {
    launch_pdl(kern, grid_of(threads, 16), 256, 0, static_cast<cudaStream_t>(stream), x, static_cast<const unsigned short*>(scale),
               row_of_slot, topk_w, T, H, k, T * k, static_cast<uint4*>(x_perm), row_w, status_word());
  };
  if (H < 256)
    run(scale ? dispatch_short_rows_kernel<true> : dispatch_short_rows_kernel<false>, (size_t)T * (H / 8));
  else
    run(scale ? dispatch_rows_kernel<true> : dispatch_rows_kernel<false>, (size_t)T * ((H / 8 + 63) / 64) * 32);
  return check_launch(fn);
}

}  // extern "C"
