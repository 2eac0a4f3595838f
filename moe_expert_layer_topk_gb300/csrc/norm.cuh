// Rows spread over groups of lanes, their sums, the root-mean-square norm's
// statistics, and rings of rows in shared memory: shared by the norms before and
// after a block.
#pragma once

#include <type_traits>

#include "common.cuh"

namespace moe {

constexpr int kNormMaxH = 8192;
// rows of partial gain gradients that a backward leaves at most
constexpr int kNormParts = 512;

// floats of shared memory that a block's row sums take: two slots of two sums, for each
// group of at most eight places for sixteen warps
constexpr int kSumFloats = 2 * 2 * 8 * 16;

// A row belongs to a group of lanes: L of them (8, 16 or 32, parts of a warp), or W
// whole warps (L = 0); lane l of n holds the 16-byte vectors l, l + n, ... of it.  Every
// thread of a block makes the same number of steps, so that full-warp shuffles and the
// groups' barriers always meet.
template <int L>
struct RowGroup {
  int W, g, l, slot;
  float* sm;
  __device__ __forceinline__ RowGroup(float* s, int w) : W(w), slot(0), sm(s) {
    const int n = lanes();
    g = threadIdx.x / n;
    l = threadIdx.x - g * n;
    if constexpr (L == 0) {  // places of warps that a group does not have stay zero
      for (int i = threadIdx.x; i < kSumFloats; i += blockDim.x) sm[i] = 0.f;
      __syncthreads();
    }
  }
  __device__ __forceinline__ int lanes() const { return L ? L : 32 * W; }
  __device__ __forceinline__ int rows() const { return blockDim.x / lanes(); }
  // The row's sums of a and b in each of its lanes, always added in the same order.  Two
  // slots: a warp writes one again only behind the next sum's barrier, which the row's
  // other warps reach with this sum read.
  template <bool kTwo>
  __device__ __forceinline__ void sums(float& a, float& b) {
#pragma unroll
    for (int off = (L ? L : 32) / 2; off > 0; off >>= 1) {
      a += __shfl_xor_sync(0xffffffffu, a, off);
      if (kTwo) b += __shfl_xor_sync(0xffffffffu, b, off);
    }
    if constexpr (L == 0) {
      if (W == 1) return;
      float* p = sm + slot * (kSumFloats / 2) + g * 16;
      slot ^= 1;
      const int w = (threadIdx.x >> 5) - g * W;
      if ((threadIdx.x & 31) == 0) {
        p[w] = a;
        if (kTwo) p[w + kSumFloats / 4] = b;
      }
      asm volatile("bar.sync %0, %1;" ::"r"(1 + g), "r"(32 * W) : "memory");
      a = places(p);
      if (kTwo) b = places(p + kSumFloats / 4);
    }
  }
  __device__ __forceinline__ float places(const float* p) const {
    const float4* q = reinterpret_cast<const float4*>(p);
    const float4 x = q[0], y = q[1];
    float v = ((x.x + x.y) + (x.z + x.w)) + ((y.x + y.y) + (y.z + y.w));
    if (W > 8) {
      const float4 z = q[2], u = q[3];
      v += ((z.x + z.y) + (z.z + z.w)) + ((u.x + u.y) + (u.z + u.w));
    }
    return v;
  }
  __device__ __forceinline__ float sum(float v) {
    float none = 0.f;
    sums<false>(v, none);
    return v;
  }
  // 1/sqrt(mean + eps) of the squares of a row's values, at(i, j) for element j of this
  // lane's i-th vector (0 where it has none).  Where mean + eps, or the squares' sum, leaves
  // fp32's range they are formed again of values times 2^-80 (8192 of the largest, 2^48 each,
  // add up to 2^109) and eps times 2^-160; below 2^-90, where squares of eps's size lose
  // digits, of values times 2^64 (at most 2^51 each then) and eps times 2^128.  An infinity
  // gives 0, a NaN NaN.
  template <int NV, class At>
  __device__ __forceinline__ float rstd(float inv_h, float eps, At&& at) {
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = __fmaf_rn(at(i, j), at(i, j), ss);
    ss = sum(ss);
    const float ms = __fmaf_rn(ss, inv_h, eps);
    float r = __frsqrt_rn(ms);
    const bool again = !(ms <= 3.402823466e+38f && ms >= 0x1p-90f);
    if (L ? __any_sync(0xffffffffu, again) : again) {
      const float scale = ms < 0x1p-90f ? 0x1p64f : 0x1p-80f;
      float s2 = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float v = at(i, j) * scale;
          s2 = __fmaf_rn(v, v, s2);
        }
      s2 = sum(s2);
      if (again) r = __frsqrt_rn(__fmaf_rn(s2, inv_h, eps * scale * scale)) * scale;
    }
    return r;
  }
};

template <typename S>
__device__ __forceinline__ Vec8<S> zero_vec() {
  Vec8<S> v;
  memset(&v, 0, sizeof v);
  return v;
}

// A thread's own stretch of shared memory, through which the 16-byte vectors of its
// next rows arrive while it works on one: no other thread reads it, so that waiting
// for one's own copies is all the synchronisation there is.  A stage holds `units`
// vectors.
struct RowRing {
  uint32_t mine;  // shared-memory address
  int pitch, stage_bytes;
  __device__ __forceinline__ RowRing(uint8_t* smem, int units)
      : mine((uint32_t)__cvta_generic_to_shared(smem) + threadIdx.x * 16), pitch(blockDim.x * 16), stage_bytes(units * pitch) {}
  // units u, u + 1 .. of `stage` = the vector of S at src, or zeros.  The two halves of eight
  // fp32 values lie in one 32-byte sector, which each of two warp-wide copies touches: by way
  // of L1 it is fetched once (8192 x 2048 in fp32, backwards: 44.4 us against 56.1, with an
  // element gate 38.0 against 43.9); a bf16 vector goes past it (in the combine 66.9 against
  // 86.4).
  template <typename S>
  __device__ __forceinline__ void fetch(int stage, int u, const S* src, bool there) {
    const uint32_t dst = mine + stage * stage_bytes + u * pitch;
    if constexpr (sizeof(Vec8<S>) == 16) {
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
    } else {
      asm volatile("cp.async.ca.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
      asm volatile("cp.async.ca.shared.global [%0], [%1], 16, %2;" ::"r"(dst + pitch), "l"(src + 4), "r"(there ? 16 : 0) : "memory");
    }
  }
  __device__ __forceinline__ void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
  // all but the last BUT stages' copies have arrived
  template <int BUT>
  __device__ __forceinline__ void wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(BUT) : "memory");
  }
  __device__ __forceinline__ uint4 at(int stage, int u) const {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(mine + stage * stage_bytes + u * pitch)
                 : "memory");
    return v;
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
// Stages of a backward's ring.  What the rings of an SM's blocks leave of its 256 KB caches
// the gains: 8192 x 2048, three blocks an SM, with three stages of 24 KB in each takes 31.2
// us, with two 28.4.  hold: two blocks an SM at most.
__host__ __device__ constexpr int ring_stages(int units, bool hold) { return !hold ? 2 : (units <= 4 ? 4 : (units <= 6 ? 3 : 2)); }

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
// part [blocks][H].  fold: shared, 8 NV floats a thread.
template <int L, int NV>
__device__ __forceinline__ void leave_part(const RowGroup<L>& rg, const float (&acc)[NV][8], float* fold, int H, float* part) {
  const int n = rg.lanes(), cols = n * NV * 8, rows = rg.rows();
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) fold[rg.g * cols + (rg.l + i * n) * 8 + j] = acc[i][j];
  __syncthreads();
  for (int c = threadIdx.x; c < H; c += blockDim.x) {
    float v = 0.f;
    for (int r = 0; r < rows; ++r) v += fold[r * cols + c];
    part[(size_t)blockIdx.x * H + c] = v;
  }
}

// How rows of H elements lie: lanes of a row (0: whole warps, W of them), rows and
// threads of a block.
struct RowShape {
  int L, W, rows, threads;
};
// nv vectors a lane; blocks of about 256 threads
inline RowShape row_shape(int H, int nv) {
  const int nvec = H / 8;
  if (nvec <= 8) return {8, 1, 32, 256};
  if (nvec <= 16) return {16, 1, 16, 256};
  if (nvec <= 32) return {32, 1, 8, 256};
  const int W = (nvec + 32 * nv - 1) / (32 * nv), rows = W >= 8 ? 1 : 8 / W;
  return {0, W, rows, 32 * W * rows};
}
// Calls f(L) for the lanes of a row (kLong: rows of whole warps too).
template <bool kLong, class F>
int with_lanes(int L, F&& f) {
  using std::integral_constant;
  if (L == 8) return f(integral_constant<int, 8>{});
  if (L == 16) return f(integral_constant<int, 16>{});
  if constexpr (kLong) {
    if (L == 0) return f(integral_constant<int, 0>{});
  }
  return f(integral_constant<int, 32>{});
}

// Blocks that an SM holds: 228 KB of shared memory (1 KB of it a block's own), registers
// of `regs` a thread, and 2048 threads.
inline int blocks_per_sm(size_t smem, int threads, int regs) {
  int n = 2048 / threads;
  const int by_smem = (int)(228 * 1024 / (smem + 1024 + sizeof(float) * kSumFloats)), by_regs = 65536 / (regs * threads);
  n = n < by_smem ? n : by_smem;
  n = n < by_regs ? n : by_regs;
  return n > 0 ? n : 1;
}
inline int norm_grid(long long T, int rows_per_block, int per_sm, int most) {
  const long long b = (T + rows_per_block - 1) / rows_per_block;
  const long long cap = (long long)(sm_count() > 0 ? sm_count() : 148) * per_sm;
  long long g = b < cap ? b : cap;
  if (g > most) g = most;
  return (int)(g > 0 ? g : 1);
}
// shared memory of a backward: its ring, in which the gain's gradients are folded too
inline size_t bwd_smem(int units, int nv, int threads, bool hold) {
  const size_t ring = (size_t)units * ring_stages(units, hold) * threads * 16, fold = sizeof(float) * 8 * nv * threads;
  return ring > fold ? ring : fold;
}

inline size_t norm_parts_bytes(int T, int H) {
  if (T <= 0 || H <= 0) return 0;
  return (size_t)(T < kNormParts ? T : kNormParts) * H * sizeof(float);
}

// Lets a kernel that is launched with `bytes` of shared memory have what a block can
// have beside its static sums; done: the kernel's own flags, one a device.
constexpr int kMaxDevices = 64;
int allow_smem(const char* fn, const void* kernel, size_t bytes, bool (&done)[kMaxDevices]);
// H, and a call's gradient of the gain
int check_norm(const char* fn, int T, int H, int fp32);
int check_gain_grad(const char* fn, int T, int H, const float* dgain, const void* ws, size_t ws_bytes);
// dgain (+)= sum over the rows of part
int launch_gain_sum(const char* fn, const float* part, int parts, int H, float* dgain, int accumulate, cudaStream_t s);

}  // namespace moe
