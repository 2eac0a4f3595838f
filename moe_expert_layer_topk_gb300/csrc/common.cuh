// Shared host and device helpers of the MoE expert-layer library (sm_103a).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <utility>

#include "moe_topk.h"

namespace moe {

// ----------------------------------------------------------------- host side

// Records a printf-style message for moe_last_error_string() and returns `code`.
int fail(int code, const char* fmt, ...);
// Clears the calling thread's last error.
void clear_error();
// Device address of the status word for the current device (nullptr on failure).
int* status_word();
// Multiprocessor count of the current device (cached; 0 on failure).
int sm_count();
// Current device ordinal (-1 on failure).
int current_device();

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Launches `kern` on `s` with programmatic dependent launch allowed: the
// kernel may be scheduled while its predecessor in the stream is finishing;
// every kernel of this library starts with pdl_wait(), which returns once
// the predecessor has completed and its memory is visible.
template <typename... KArgs, typename... Args>
inline cudaError_t launch_pdl(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem,
                              cudaStream_t s, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...);
}

inline int check_launch(const char* what) {
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(MOE_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
  return MOE_OK;
}
// the same, naming the entry point and the kernel of a multi-kernel call
inline int check_launch(const char* fn, const char* kernel) {
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(MOE_ERR_CUDA, "%s: %s: %s", fn, kernel, cudaGetErrorString(e));
  return MOE_OK;
}

// Reports an error that a runtime call returned, and takes it off the runtime:
// left there, the next call's check would report it as its own.
inline int fail_cuda(const char* fn, cudaError_t e) {
  cudaGetLastError();
  return fail(MOE_ERR_CUDA, "%s: %s", fn, cudaGetErrorString(e));
}

constexpr int kMaxExperts = 1024;
constexpr int kMaxTopK = 32;
constexpr int kMaxSegments = 1024;
// tokens per ranking chunk: the router's top-k CTA and the dispatch row CTA
// each cover one chunk, and the route's chunk prefixes are per chunk
constexpr int kRouteChunk = 16;

// Internal entry points shared between translation units (not exported).
struct GroupedSegs {
  int num_seg;
  const int32_t* seg_offsets;
  const int32_t* seg_expert;  // may be null (identity)
};

// Dense "row" GEMM with K-major A [M,K] and K-major B [N,K], both bf16, one
// segment [0,M) and fp32 accumulation; epilogue out[m,n] = bf16(acc + add[m,n])
// with `add` fp32 [M,N] (row stride N).  Used by the router backward.
int launch_dense_add_bf16(const void* A, const void* B, const float* add, void* out, int M, int N,
                          int K, cudaStream_t stream);
// out[g] (fp32 [groups, M, N]) = sum over the K rows of segment g of A^T B,
// with A [K_rows, M] and B [K_rows, N] bf16 row-major (both MN-major).  Used
// by the router backward (split-K partials, overwrite).  `maps` is device
// scratch of dw_split_maps_bytes(num_seg) bytes, 128-byte aligned, for the
// per-segment TMA descriptors.
size_t dw_split_maps_bytes(int num_seg);
int launch_dw_split(const void* A, const void* B, int K_rows, int M, int N,
                    const int32_t* seg_offsets, int num_seg, float* out, void* maps,
                    cudaStream_t stream);

// ---------------------------------------------------------------- device side

// Programmatic dependent launch: wait for the predecessor grid (its writes
// visible), then let the successor grid be scheduled.
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_trigger() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

__device__ __forceinline__ float bf16lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf16hi(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);  // round to nearest even
  return *reinterpret_cast<uint32_t*>(&p);
}

// eight bf16 values of a 16-byte vector <-> fp32
__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  f[0] = bf16lo(v.x); f[1] = bf16hi(v.x); f[2] = bf16lo(v.y); f[3] = bf16hi(v.y);
  f[4] = bf16lo(v.z); f[5] = bf16hi(v.z); f[6] = bf16lo(v.w); f[7] = bf16hi(v.w);
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}

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

__device__ __forceinline__ void set_status(int* status, int bits) {
  if (status) atomicOr(status, bits);
}

// e4m3 row quantisation ("TorchTitan FSDP2 完全指南", performance table: FP8
// matmuls; the recipe is the reading stated in moe_topk.h): the largest |a|
// of eight bf16 values, the row scale from the row's largest |a|, and eight
// codes e4m3(a / s) (IEEE division, round to nearest even, saturated).
__device__ __forceinline__ float amax_bf16x8(uint4 v, float m) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) m = fmaxf(m, fmaxf(fabsf(bf16lo(w[i])), fabsf(bf16hi(w[i]))));
  return m;
}
__device__ __forceinline__ float e4m3_row_scale(float amax) { return amax > 0.0f ? __fdiv_rn(amax, 448.0f) : 1.0f; }
__device__ __forceinline__ uint2 e4m3_codes8(uint4 v, float s) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t out[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const float2 a = make_float2(__fdiv_rn(bf16lo(w[2 * h]), s), __fdiv_rn(bf16hi(w[2 * h]), s));
    const float2 b = make_float2(__fdiv_rn(bf16lo(w[2 * h + 1]), s), __fdiv_rn(bf16hi(w[2 * h + 1]), s));
    const uint32_t ca = __nv_cvt_float2_to_fp8x2(a, __NV_SATFINITE, __NV_E4M3);
    const uint32_t cb = __nv_cvt_float2_to_fp8x2(b, __NV_SATFINITE, __NV_E4M3);
    out[h] = (ca & 0xFFFFu) | (cb << 16);
  }
  return make_uint2(out[0], out[1]);
}

// Activations kept in 8 bits: 32 columns share a bf16 scale s, the smallest bf16
// number that is at least amax/127 (and 2^-126, whose reciprocal is finite), and
// are whole numbers of at most 7 bits and a sign times it.
constexpr int kCkptGroup = 32;

// The larger magnitude, or NaN where there is one.
__device__ __forceinline__ float amax_nan(float m, float a) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(m), "f"(fabsf(a)));
  return r;
}
// An amax that is infinite or NaN gives a NaN: all the group's values come back as NaN.
// A scale above 2^121 becomes 2.125 * 2^120: the largest values, up to 256 * 2^120, then
// have codes of at most 120, which stand for 255 * 2^120, bf16's largest, where 127 of
// the scale 2.015625 * 2^120 would be rounded to an infinity.
__device__ __forceinline__ float ckpt_scale(float amax) {
  const float q = __fdiv_rn(amax, 127.0f);
  const float up = __uint_as_float((__float_as_uint(q) + 0xFFFFu) & 0xFFFF0000u);
  if (!(q <= 3.402823466e+38f)) return __uint_as_float(0x7FC00000u);
  return up < 0x1p-126f ? 0x1p-126f : (up > 0x1p121f ? 0x1.1p121f : up);
}
// Four codes, lowest first: a * inv rounded to nearest even by adding 1.5 * 2^23,
// whose lowest byte is then the two's complement code (|a * inv| is at most 127
// and a few units of the last place).
__device__ __forceinline__ uint32_t ckpt_codes4(float a, float b, float c, float d, float inv) {
  const uint32_t x = __float_as_uint(__fadd_rn(__fmul_rn(a, inv), 12582912.0f));
  const uint32_t y = __float_as_uint(__fadd_rn(__fmul_rn(b, inv), 12582912.0f));
  const uint32_t z = __float_as_uint(__fadd_rn(__fmul_rn(c, inv), 12582912.0f));
  const uint32_t w = __float_as_uint(__fadd_rn(__fmul_rn(d, inv), 12582912.0f));
  return __byte_perm(__byte_perm(x, y, 0x0040), __byte_perm(z, w, 0x0040), 0x5410);
}
// The values of four codes: the byte with its sign bit flipped is code + 128, put
// into the low mantissa bits of 2^23, whose difference from 2^23 + 128 is exact.
__device__ __forceinline__ void ckpt_decode4(uint32_t w, float s, float (&f)[4]) {
  const uint32_t v = w ^ 0x80808080u;
  f[0] = (__uint_as_float(__byte_perm(v, 0x4B000000u, 0x7440)) - 8388736.0f) * s;
  f[1] = (__uint_as_float(__byte_perm(v, 0x4B000000u, 0x7441)) - 8388736.0f) * s;
  f[2] = (__uint_as_float(__byte_perm(v, 0x4B000000u, 0x7442)) - 8388736.0f) * s;
  f[3] = (__uint_as_float(__byte_perm(v, 0x4B000000u, 0x7443)) - 8388736.0f) * s;
}
__device__ __forceinline__ float bf16_bits(uint32_t h) { return __uint_as_float(h << 16); }

}  // namespace moe
