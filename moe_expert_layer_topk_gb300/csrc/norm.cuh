// Rows spread over groups of lanes, their sums, and the root-mean-square norm's
// statistics: shared by the norms before and after a block.
#pragma once

#include <type_traits>

#include "common.cuh"

namespace moe {

constexpr int kNormThreads = 256;
constexpr int kNormMaxH = 8192;
// rows of partial gain gradients that a backward leaves at most
constexpr int kNormParts = 512;

// A row belongs to L lanes (a part of a warp, a warp, or several warps), lane l of
// them holding the 16-byte vectors l, l + L, ... of it (NV at most).  A block of 256
// threads works on 256/L rows; every thread of a block makes the same number of
// steps, so that full-warp shuffles and the rows' barriers always meet.
template <int L>
struct RowGroup {
  static constexpr int kRows = kNormThreads / L;
  int g, l, slot;
  float* sm;  // [2][8]
  __device__ __forceinline__ explicit RowGroup(float* s) : g(threadIdx.x / L), l(threadIdx.x % L), slot(0), sm(s) {}
  // The row's sum in each of its lanes, always added in the same order.  Two slots:
  // a warp writes one again only behind the next sum's barrier, which the row's other
  // warps reach with this sum read.
  __device__ __forceinline__ float sum(float v) {
#pragma unroll
    for (int off = (L < 32 ? L : 32) / 2; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    if constexpr (L > 32) {
      constexpr int W = L / 32;
      const int warp = threadIdx.x >> 5;
      float* p = sm + 8 * slot;
      slot ^= 1;
      if ((threadIdx.x & 31) == 0) p[warp] = v;
      asm volatile("bar.sync %0, %1;" ::"r"(1 + g), "n"(L) : "memory");
      v = 0.f;
#pragma unroll
      for (int i = 0; i < W; ++i) v += p[g * W + i];
    }
    return v;
  }
  // 1/sqrt(mean + eps) of the squares of a row's values, at(i, j) for element j of this
  // lane's i-th vector (0 where it has none).  Squares beyond fp32's range are added
  // again of values times 2^-80 (8192 of the largest, 2^48 each, add up to 2^109); eps
  // is nothing beside those.  An infinity gives 0, a NaN NaN.
  template <int NV, class At>
  __device__ __forceinline__ float rstd(float inv_h, float eps, At&& at) {
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = __fmaf_rn(at(i, j), at(i, j), ss);
    ss = sum(ss);
    float r = __frsqrt_rn(__fmaf_rn(ss, inv_h, eps));
    const bool big = !(ss <= 3.402823466e+38f);
    if (L <= 32 ? __any_sync(0xffffffffu, big) : big) {
      float s2 = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float v = at(i, j) * 0x1p-80f;
          s2 = __fmaf_rn(v, v, s2);
        }
      s2 = sum(s2);
      if (big) r = __frsqrt_rn(s2 * inv_h) * 0x1p-80f;
    }
    return r;
  }
};

// A thread's own stretch of shared memory, through which the 16-byte vectors of its
// next rows arrive while it works on one: no other thread reads it, so that waiting
// for one's own copies is all the synchronisation there is.  A stage holds `units`
// vectors.
constexpr int kRingUnitBytes = kNormThreads * 16;  // a vector of each thread
struct RowRing {
  uint8_t* mine;
  int units;
  __device__ __forceinline__ RowRing(uint8_t* smem, int units) : mine(smem + threadIdx.x * 16), units(units) {}
  // unit u of `stage` = the 16 bytes at src, or zeros
  __device__ __forceinline__ void fetch(int stage, int u, const void* src, bool there) {
    const uint32_t dst = (uint32_t)__cvta_generic_to_shared(mine + (stage * units + u) * kRingUnitBytes);
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
  }
  __device__ __forceinline__ void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
  // all but the last BUT stages' copies have arrived
  template <int BUT>
  __device__ __forceinline__ void wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(BUT) : "memory");
  }
  __device__ __forceinline__ const uint4& at(int stage, int u) const {
    return *reinterpret_cast<const uint4*>(mine + (stage * units + u) * kRingUnitBytes);
  }
  // the vector whose (first) unit is u
  template <typename S>
  __device__ __forceinline__ Vec8<S> vec(int stage, int u) const {
    Vec8<S> v;
    uint4* w = reinterpret_cast<uint4*>(&v);
#pragma unroll
    for (int i = 0; i < (int)(sizeof(Vec8<S>) / 16); ++i) w[i] = at(stage, u + i);
    return v;
  }
};
// stages that leave room for two blocks an SM (up to 12 units)
__host__ __device__ constexpr int ring_stages(int units) { return units <= 6 ? 4 : (units <= 8 ? 3 : 2); }

template <typename S>
__device__ __forceinline__ Vec8<S> zero_vec() {
  Vec8<S> v;
  memset(&v, 0, sizeof v);
  return v;
}

// Eight gains (ones without a tensor).
struct Gain8 {
  float4 a, b;
  __device__ __forceinline__ Gain8(const float* gain, int vec, bool there) {
    a = b = make_float4(1.f, 1.f, 1.f, 1.f);
    if (gain && there) {
      a = __ldg(reinterpret_cast<const float4*>(gain) + 2 * vec);
      b = __ldg(reinterpret_cast<const float4*>(gain) + 2 * vec + 1);
    }
  }
  __device__ __forceinline__ float at(int i) const {
    const float4& v = i < 4 ? a : b;
    return (i & 3) == 0 ? v.x : ((i & 3) == 1 ? v.y : ((i & 3) == 2 ? v.z : v.w));
  }
};

// Leaves this block's sums over its rows, acc of each lane's vectors, as one row of
// part [blocks][H].  fold: shared, 256 * NV * 8 floats.
template <int L, int NV>
__device__ __forceinline__ void leave_part(const float (&acc)[NV][8], float* fold, int H, float* part) {
  constexpr int kCols = L * NV * 8;
  const int g = threadIdx.x / L, l = threadIdx.x % L;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) fold[g * kCols + (l + i * L) * 8 + j] = acc[i][j];
  __syncthreads();
  for (int c = threadIdx.x; c < H; c += kNormThreads) {
    float v = 0.f;
    for (int r = 0; r < RowGroup<L>::kRows; ++r) v += fold[r * kCols + c];
    part[(size_t)blockIdx.x * H + c] = v;
  }
}

// Calls f(lanes of a row, vectors of a lane) for rows of H elements.
template <class F>
int with_row_shape(int H, F&& f) {
  using std::integral_constant;
  if (H <= 64) return f(integral_constant<int, 8>{}, integral_constant<int, 1>{});
  if (H <= 128) return f(integral_constant<int, 16>{}, integral_constant<int, 1>{});
  if (H <= 256) return f(integral_constant<int, 32>{}, integral_constant<int, 1>{});
  if (H <= 512) return f(integral_constant<int, 32>{}, integral_constant<int, 2>{});
  if (H <= 1024) return f(integral_constant<int, 32>{}, integral_constant<int, 4>{});
  if (H <= 2048) return f(integral_constant<int, 64>{}, integral_constant<int, 4>{});
  if (H <= 4096) return f(integral_constant<int, 128>{}, integral_constant<int, 4>{});
  return f(integral_constant<int, 256>{}, integral_constant<int, 4>{});
}

// Blocks an SM that a backward kernel's registers leave room for.
__host__ __device__ constexpr int bwd_blocks(int nv) { return nv == 4 ? 1 : 2; }

// The same for the backward kernels, which hold the gain's gradient of their columns as
// well: fewer vectors a lane.
template <class F>
int with_bwd_shape(int H, F&& f) {
  using std::integral_constant;
  if (H <= 64) return f(integral_constant<int, 8>{}, integral_constant<int, 1>{});
  if (H <= 128) return f(integral_constant<int, 16>{}, integral_constant<int, 1>{});
  if (H <= 256) return f(integral_constant<int, 32>{}, integral_constant<int, 1>{});
  if (H <= 512) return f(integral_constant<int, 32>{}, integral_constant<int, 2>{});
  if (H <= 1024) return f(integral_constant<int, 64>{}, integral_constant<int, 2>{});
  if (H <= 2048) return f(integral_constant<int, 128>{}, integral_constant<int, 2>{});
  if (H <= 4096) return f(integral_constant<int, 256>{}, integral_constant<int, 2>{});
  return f(integral_constant<int, 256>{}, integral_constant<int, 4>{});
}

inline int norm_grid(long long T, int rows_per_block, int per_sm, int most) {
  const long long b = (T + rows_per_block - 1) / rows_per_block;
  const long long cap = (long long)(sm_count() > 0 ? sm_count() : 148) * per_sm;
  long long g = b < cap ? b : cap;
  if (g > most) g = most;
  return (int)(g > 0 ? g : 1);
}

inline size_t norm_parts_bytes(int T, int H) {
  if (T <= 0 || H <= 0) return 0;
  return (size_t)(T < kNormParts ? T : kNormParts) * H * sizeof(float);
}

// shared memory of a backward: its ring, in which the gain's gradients are folded too
constexpr size_t norm_smem(int units, int nv) {
  const size_t ring = (size_t)units * ring_stages(units) * kRingUnitBytes, fold = sizeof(float) * kNormThreads * 8 * nv;
  return ring > fold ? ring : fold;
}
// blocks of so much shared memory that an SM holds (228 KB, 1 KB of it a block's own)
inline int blocks_per_sm(size_t smem, int most) {
  const int n = (int)(228 * 1024 / (smem + 1024));
  return n < most ? (n > 0 ? n : 1) : most;
}
// lets a kernel have that much (an attribute of the kernel, set on every call: cheap, and right on every device)
int allow_smem(const char* fn, const void* kernel, size_t bytes);

// H, eps and a call's gradient of the gain
int check_norm(const char* fn, int T, int H, int fp32);
int check_gain_grad(const char* fn, int T, int H, const float* dgain, const void* ws, size_t ws_bytes);
// dgain (+)= sum over the rows of part
int launch_gain_sum(const char* fn, const float* part, int parts, int H, float* dgain, int accumulate, cudaStream_t s);

}  // namespace moe
