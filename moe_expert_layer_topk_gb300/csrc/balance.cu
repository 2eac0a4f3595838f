// Load-balance loss and router z-loss of masked, packed tokens, the slots of
// every expert, and the gradient of the router logits.
//
// Token t of sequence q (mask m_t): p_t = softmax(l_t), lse_t its
// log-sum-exp; n_q = sum m_t, n = sum n_q, c_qe = slots of q's tokens routed
// to expert e, P_qe = sum m_t p_te.
//   balance = 1/n sum_q E/(k n_q) sum_e c_qe P_qe     z = 1/n sum_t m_t lse_t^2
//   dl_te   = m_t p_te (a E/(k n_q n) (c_qe - sum_j c_qj p_tj) + 2 b/n lse_t)
// The slot counts carry no gradient, so the gradient needs the counts but not
// P: after a pass over topk_idx (the smallest tensor) one pass over the
// logits gives the gradient and the sums P together.
//
// Deterministic: the token range is cut into one chunk per CTA, a chunk that
// reaches into several sequences leaves one partial row per sequence, and the
// rows of a sequence are added in chunk order.  (chunk c, sequence q) sits in
// row c + q: along the token axis every new pair raises one of the two, so no
// two pairs share a row.  Integer counts use atomics, whose order does not
// matter.
#include <cfloat>

#include "common.cuh"

namespace moe {
namespace {

constexpr int kMaxSeq = kMaxSegments;
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

struct Tokens {  // the packed token axis, cut into chunks
  int T, E, k, num_seq, chunk;
  const int32_t* seq_offsets;  // null: one sequence of all tokens
  const uint8_t* mask;         // null: every token counts
};

// The sequence table in shared memory, made monotone and clamped to [0, T]
// (a table that is not is reported): off[0..num_seq].
__device__ __forceinline__ void load_table(const Tokens& k, int* off, int* status) {
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    int carry = 0;
    for (int b = 0; b <= k.num_seq; b += 32) {
      const int s = b + lane;
      int v = 0;
      if (s <= k.num_seq) {
        v = k.seq_offsets ? k.seq_offsets[s] : (s == 0 ? 0 : k.T);
        if (v < 0 || v > k.T) {
          set_status(status, MOE_STATUS_BAD_SEGMENTS);
          v = v < 0 ? 0 : k.T;
        }
      }
      int m = v;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, m, d);
        if (lane >= d) m = max(m, o);
      }
      m = max(m, carry);
      if (s <= k.num_seq) {
        if (m != v) set_status(status, MOE_STATUS_BAD_SEGMENTS);
        off[s] = m;
      }
      carry = __shfl_sync(0xffffffffu, m, 31);
    }
  }
  __syncthreads();
}

// The sequence that token t lies in, given off[0] <= t < off[num_seq].
__device__ __forceinline__ int seq_of(const int* off, int num_seq, int t) {
  int lo = 0, hi = num_seq - 1;  // last s with off[s] <= t
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (off[mid] <= t) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// f(seq, first token, end) for every non-empty piece of [t0, t1) inside a sequence.
template <class F>
__device__ __forceinline__ void for_each_piece(const int* off, int num_seq, int t0, int t1, F&& f) {
  int a = max(t0, off[0]);
  const int end = min(t1, off[num_seq]);
  if (a >= end) return;
  int s = seq_of(off, num_seq, a);
  while (a < end) {
    const int b = min(end, off[s + 1]);
    if (b > a) f(s, a, b);
    a = max(a, b);
    ++s;
  }
}

// ------------------------------------------------------------------ counts
// counts[q][e], tokens[q] (zeroed before): shared-memory histogram of the
// chunk, added to the sequence's row.
__global__ void __launch_bounds__(kThreads) balance_count_kernel(const Tokens tk, const int32_t* __restrict__ topk_idx,
                                                                 int32_t* __restrict__ counts,
                                                                 int32_t* __restrict__ tokens, int* status) {
  pdl_wait();
  pdl_trigger();
  extern __shared__ int sm[];
  int* off = sm;                      // [num_seq + 1]
  int* hist = sm + tk.num_seq + 1;    // [E]
  __shared__ int live;
  load_table(tk, off, status);
  const int t0 = blockIdx.x * tk.chunk, t1 = min(tk.T, t0 + tk.chunk);
  for_each_piece(off, tk.num_seq, t0, t1, [&](int s, int a, int b) {
    for (int e = threadIdx.x; e < tk.E; e += kThreads) hist[e] = 0;
    if (threadIdx.x == 0) live = 0;
    __syncthreads();
    int mine = 0;
    if (tk.mask) {
      for (int t = a + threadIdx.x; t < b; t += kThreads) mine += tk.mask[t] != 0;
    } else if (threadIdx.x == 0) {
      mine = b - a;
    }
    if (mine) atomicAdd(&live, mine);
    const long long q1 = (long long)b * tk.k;
    for (long long q = (long long)a * tk.k + threadIdx.x; q < q1; q += kThreads) {
      if (tk.mask && !tk.mask[q / tk.k]) continue;
      const int e = topk_idx[q];
      if (e >= 0 && e < tk.E)
        atomicAdd(&hist[e], 1);
      else
        set_status(status, MOE_STATUS_BAD_INDEX);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < tk.E; e += kThreads)
      if (hist[e]) atomicAdd(counts + (size_t)s * tk.E + e, hist[e]);
    if (threadIdx.x == 0 && live) atomicAdd(tokens + s, live);
    __syncthreads();
  });
}

// ------------------------------------------------------------- main kernel
//
// LPT lanes hold one token's logits (VEC consecutive values NQ times, VEC LPT
// apart), a warp 32/LPT tokens side by side; kU of a lane's tokens are loaded
// before the first is used.  The lane's share of P stays in registers over
// the piece and is added over the warp's token groups and the warps at its
// end.
struct Grad {
  float a, b;            // coefficients of the two losses
  const float* dloss;    // their upstream gradients on the device, or null
  float* dlogits;
};

template <int LPT, int VEC, int NQ, bool kSum, bool kGrad>
__global__ void __launch_bounds__(kThreads) balance_main_kernel(const Tokens tk, const float* __restrict__ logits,
                                                                const int32_t* __restrict__ counts,
                                                                const int32_t* __restrict__ tokens, const Grad gr,
                                                                float* __restrict__ part, float* __restrict__ zpart,
                                                                unsigned* __restrict__ ticket, int* status) {
  constexpr int NV = NQ * VEC;       // values per lane
  constexpr int TPW = 32 / LPT;      // tokens per warp side by side
  constexpr int kU = NV <= 4 ? 4 : (NV <= 8 ? 2 : 1);
  pdl_wait();
  pdl_trigger();
  extern __shared__ int sm[];
  int* off = sm;                                                       // [num_seq + 1]
  float* red = reinterpret_cast<float*>(sm + ((tk.num_seq + 4) & ~3));  // kSum: [kWarps][E + 1]
  __shared__ int s_n;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = lane / LPT, el = lane % LPT;
  const int E = tk.E;
  if (threadIdx.x == 0) {
    s_n = 0;
    if (kSum && blockIdx.x == 0) *ticket = 0;  // read by the finishing kernel only
  }
  load_table(tk, off, status);
  const int t0 = blockIdx.x * tk.chunk, t1 = min(tk.T, t0 + tk.chunk);
  float ga = 0.f, gb = 0.f;
  if constexpr (kGrad) {
    int n = 0;
    for (int s = threadIdx.x; s < tk.num_seq; s += kThreads) n += tokens[s];
    if (n) atomicAdd(&s_n, n);
    __syncthreads();
    const float rn = 1.f / (float)max(s_n, 1);
    ga = gr.a * (gr.dloss ? gr.dloss[0] : 1.f) * ((float)E / (float)tk.k) * rn;
    gb = gr.b * (gr.dloss ? gr.dloss[1] : 1.f) * 2.f * rn;
    // tokens outside every sequence get no gradient
    const int lo = min(t1, max(t0, off[0])), hi = max(t0, min(t1, off[tk.num_seq]));
    for (size_t i = (size_t)t0 * E + threadIdx.x; i < (size_t)lo * E; i += kThreads) gr.dlogits[i] = 0.f;
    for (size_t i = (size_t)max(lo, hi) * E + threadIdx.x; i < (size_t)t1 * E; i += kThreads) gr.dlogits[i] = 0.f;
  }
  const unsigned gmask = LPT == 32 ? 0xffffffffu : (((1u << (LPT & 31)) - 1u) << (sub * LPT));
  auto gmax = [&](float v) {
#pragma unroll
    for (int d = LPT / 2; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor_sync(gmask, v, d));
    return v;
  };
  auto gsum = [&](float v) {
#pragma unroll
    for (int d = LPT / 2; d > 0; d >>= 1) v += __shfl_xor_sync(gmask, v, d);
    return v;
  };
  auto col = [&](int i) { return (i / VEC) * VEC * LPT + el * VEC + i % VEC; };

  for_each_piece(off, tk.num_seq, t0, t1, [&](int s, int a, int b) {
    float cf[kGrad ? NV : 1], acc[kSum ? NV : 1];
    float ga_s = 0.f, z = 0.f;
    if constexpr (kGrad) {
      ga_s = ga / (float)max(tokens[s], 1);
#pragma unroll
      for (int i = 0; i < NV; ++i) cf[i] = col(i) < E ? (float)counts[(size_t)s * E + col(i)] : 0.f;
    }
    if constexpr (kSum) {
#pragma unroll
      for (int i = 0; i < NV; ++i) acc[i] = 0.f;
    }
    const int step = kWarps * TPW;
    for (int tb = a + warp * TPW + sub; tb < b; tb += kU * step) {
      float l[kU][NV];
      bool on[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int t = tb + u * step;
        on[u] = t < b && (!tk.mask || tk.mask[t]);
#pragma unroll
        for (int q = 0; q < NQ; ++q) {
          const int c0 = q * VEC * LPT + el * VEC;
          if constexpr (VEC == 4) {
            float4 v = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
            if (on[u] && c0 < E) v = __ldg(reinterpret_cast<const float4*>(logits + (size_t)t * E + c0));
            l[u][4 * q] = v.x; l[u][4 * q + 1] = v.y; l[u][4 * q + 2] = v.z; l[u][4 * q + 3] = v.w;
          } else {
            l[u][q] = on[u] && c0 < E ? __ldg(logits + (size_t)t * E + c0) : -INFINITY;
          }
        }
      }
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int t = tb + u * step;
        if (t >= b) break;
        float dl[NV];
        if (on[u]) {
          float m = l[u][0];
#pragma unroll
          for (int i = 1; i < NV; ++i) m = fmaxf(m, l[u][i]);
          m = gmax(m);
          float sum = 0.f, dot = 0.f;
#pragma unroll
          for (int i = 0; i < NV; ++i) {
            // lanes past the last expert hold -inf; a real logit may be +inf or NaN, whose NaN has to show
            l[u][i] = col(i) < E ? expf(l[u][i] - m) : 0.f;
            sum += l[u][i];
            if constexpr (kGrad) dot = fmaf(cf[i], l[u][i], dot);
          }
          sum = gsum(sum);
          const float r = 1.f / sum;
          const float lse = m + logf(sum);
          if constexpr (kSum) {
#pragma unroll
            for (int i = 0; i < NV; ++i) acc[i] = fmaf(l[u][i], r, acc[i]);
            if (el == 0) z = fmaf(lse, lse, z);
          }
          if constexpr (kGrad) {
            dot = gsum(dot) * r;
            const float w = gb * lse - ga_s * dot;
#pragma unroll
            for (int i = 0; i < NV; ++i) dl[i] = l[u][i] * r * fmaf(ga_s, cf[i], w);
          }
        } else {
#pragma unroll
          for (int i = 0; i < NV; ++i) dl[i] = 0.f;
        }
        if constexpr (kGrad) {
#pragma unroll
          for (int q = 0; q < NQ; ++q) {
            const int c0 = q * VEC * LPT + el * VEC;
            if (c0 < E) {
              float* o = gr.dlogits + (size_t)t * E + c0;
              if constexpr (VEC == 4)
                *reinterpret_cast<float4*>(o) = make_float4(dl[4 * q], dl[4 * q + 1], dl[4 * q + 2], dl[4 * q + 3]);
              else
                *o = dl[q];
            }
          }
        }
      }
    }
    if constexpr (kSum) {
      __syncwarp();
#pragma unroll
      for (int d = LPT; d < 32; d <<= 1) {
#pragma unroll
        for (int i = 0; i < NV; ++i) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], d);
      }
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) z += __shfl_xor_sync(0xffffffffu, z, d);
      if (sub == 0) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
          if (col(i) < E) red[warp * (E + 1) + col(i)] = acc[i];
      }
      if (lane == 0) red[warp * (E + 1) + E] = z;
      __syncthreads();
      const size_t row = (size_t)(blockIdx.x + s);
      for (int e = threadIdx.x; e <= E; e += kThreads) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) v += red[w * (E + 1) + e];
        if (e < E)
          part[row * E + e] = v;
        else
          zpart[row] = v;
      }
      __syncthreads();
    }
  });
}

// -------------------------------------------------------------- finish kernel
// CTA (sequence q, 32 experts): P_qe from the partial rows in order (32 row
// groups side by side, added in order), and their share of the two losses;
// the last CTA to finish adds the shares in order.
__global__ void __launch_bounds__(1024) balance_finish_kernel(const Tokens tk, const float* __restrict__ part,
                                                              const float* __restrict__ zpart,
                                                              const int32_t* __restrict__ counts,
                                                              const int32_t* __restrict__ tokens,
                                                              float* __restrict__ prob_sum, float2* __restrict__ share,
                                                              unsigned* __restrict__ ticket, float* __restrict__ loss,
                                                              int* status) {
  pdl_wait();
  pdl_trigger();
  extern __shared__ int sm[];
  int* off = sm;
  __shared__ float red[32][33];
  __shared__ float zred[32];
  __shared__ int s_n;
  __shared__ bool last;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int q = blockIdx.x, e = blockIdx.y * 32 + lane;
  if (threadIdx.x == 0) s_n = 0;
  load_table(tk, off, status);
  int n = 0;
  for (int s = threadIdx.x; s < tk.num_seq; s += 1024) n += tokens[s];
  if (n) atomicAdd(&s_n, n);
  const int a = off[q], b = off[q + 1];
  const int c0 = a / tk.chunk, c1 = b > a ? (b - 1) / tk.chunk + 1 : c0;
  float v = 0.f;
  if (e < tk.E) {
#pragma unroll 4
    for (int c = c0 + warp; c < c1; c += 32) v += part[(size_t)(c + q) * tk.E + e];
  }
  red[warp][lane] = v;
  float z = 0.f;
  if (blockIdx.y == 0) {
    for (int c = c0 + threadIdx.x; c < c1; c += 1024) z += zpart[c + q];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) z += __shfl_xor_sync(0xffffffffu, z, d);
    if (lane == 0) zred[warp] = z;
  }
  __syncthreads();
  if (warp == 0) {
    float p = 0.f, zz = 0.f;
    for (int w = 0; w < 32; ++w) p += red[w][lane];
    if (e < tk.E) prob_sum[(size_t)q * tk.E + e] = p;
    float t = e < tk.E ? p * (float)counts[(size_t)q * tk.E + e] : 0.f;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) t += __shfl_xor_sync(0xffffffffu, t, d);
    if (blockIdx.y == 0)
      for (int w = 0; w < 32; ++w) zz += zred[w];
    if (lane == 0) {
      const float rn = 1.f / (float)max(s_n, 1), nq = (float)max(tokens[q], 1);
      share[(size_t)q * gridDim.y + blockIdx.y] =
          make_float2(t * ((float)tk.E / (float)tk.k) / nq * rn, zz * rn);
      __threadfence();
      last = atomicAdd(ticket, 1u) == gridDim.x * gridDim.y - 1;
    }
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  const int total = gridDim.x * gridDim.y;
  float lb = 0.f, lz = 0.f;
  for (int i = threadIdx.x; i < total; i += 1024) {
    const float2 h = __ldcg(share + i);
    lb += h.x;
    lz += h.y;
  }
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    lb += __shfl_xor_sync(0xffffffffu, lb, d);
    lz += __shfl_xor_sync(0xffffffffu, lz, d);
  }
  if (lane == 0) {
    red[0][warp] = lb;
    red[1][warp] = lz;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    lb = lz = 0.f;
    for (int w = 0; w < 32; ++w) {
      lb += red[0][w];
      lz += red[1][w];
    }
    loss[0] = lb;
    loss[1] = lz;
  }
}

// --------------------------------------------------------------- host side

size_t align256(size_t b) { return (b + 255) & ~size_t(255); }

// Chunks: enough for four CTAs per SM, at least 16 tokens each.
constexpr int kMaxChunks = 608;
int chunk_tokens(int T) {
  const int c = (T + kMaxChunks - 1) / kMaxChunks;
  return c < 16 ? 16 : c;
}

struct Layout {
  int chunk, nchunk;
  size_t part, zpart, share, ticket, total;
};
Layout layout(int T, int E, int num_seq) {
  Layout L;
  L.chunk = chunk_tokens(T);
  L.nchunk = (T + L.chunk - 1) / L.chunk;
  const size_t rows = (size_t)L.nchunk + num_seq;
  size_t at = 0;
  L.part = at; at += align256(rows * E * sizeof(float));
  L.zpart = at; at += align256(rows * sizeof(float));
  L.share = at; at += align256((size_t)num_seq * ((E + 31) / 32) * sizeof(float2));
  L.ticket = at; at += 256;
  L.total = at;
  return L;
}

template <bool kSum, bool kGrad>
struct Main {
  template <int LPT, int VEC, int NQ>
  static void go(const Layout& L, const Tokens& tk, const float* logits, const int32_t* counts, const int32_t* tokens,
                 const Grad& gr, float* part, float* zpart, unsigned* ticket, cudaStream_t s) {
    const size_t smem = sizeof(int) * ((tk.num_seq + 4) & ~3) + (kSum ? sizeof(float) * kWarps * (tk.E + 1) : 0);
    launch_pdl(balance_main_kernel<LPT, VEC, NQ, kSum, kGrad>, L.nchunk, kThreads, smem, s, tk, logits, counts, tokens,
               gr, part, zpart, ticket, status_word());
  }
  template <class... A>
  static void pick(int E, A&&... a) {
    if (E % 4 == 0) {
      if (E <= 4) go<1, 4, 1>(a...);
      else if (E <= 8) go<2, 4, 1>(a...);
      else if (E <= 16) go<4, 4, 1>(a...);
      else if (E <= 32) go<8, 4, 1>(a...);
      else if (E <= 64) go<16, 4, 1>(a...);
      else if (E <= 128) go<32, 4, 1>(a...);
      else if (E <= 256) go<32, 4, 2>(a...);
      else if (E <= 512) go<32, 4, 4>(a...);
      else go<32, 4, 8>(a...);
    } else {
      if (E <= 4) go<4, 1, 1>(a...);
      else if (E <= 16) go<16, 1, 1>(a...);
      else if (E <= 32) go<32, 1, 1>(a...);
      else if (E <= 64) go<32, 1, 2>(a...);
      else if (E <= 128) go<32, 1, 4>(a...);
      else if (E <= 256) go<32, 1, 8>(a...);
      else if (E <= 512) go<32, 1, 16>(a...);
      else go<32, 1, 32>(a...);
    }
  }
};

int check_balance(const char* fn, const float* logits, int T, int E, int k, int num_seq, const int32_t* seq_offsets) {
  if (T < 0 || E <= 0 || k <= 0 || num_seq <= 0)
    return fail(MOE_ERR_INVALID_ARG, "%s: need T>=0, E>0, k>0, num_seg>0", fn);
  if (E > kMaxExperts || k > kMaxTopK || k > E || num_seq > kMaxSeq || (long long)T * k >= (1ll << 31))
    return fail(MOE_ERR_UNSUPPORTED_SHAPE, "%s: need E<=1024, k<=min(E,32), num_seg<=%d, T*k<2^31 (E=%d k=%d num_seg=%d)",
                fn, kMaxSeq, E, k, num_seq);
  if (num_seq > 1 && !seq_offsets) return fail(MOE_ERR_INVALID_ARG, "%s: seg_offsets is NULL", fn);
  if (T > 0 && !logits) return fail(MOE_ERR_INVALID_ARG, "%s: NULL pointer argument", fn);
  if (!aligned16(logits)) return fail(MOE_ERR_ALIGNMENT, "%s: logits must be 16-byte aligned", fn);
  return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_balance_loss_workspace_size(int T, int E, int num_seg) {
  if (T < 0 || E <= 0 || num_seg <= 0) return 0;
  return layout(T, E, num_seg).total;
}

int moe_balance_loss(const float* logits, const int32_t* topk_idx, const uint8_t* mask, int T, int E, int k,
                     int num_seg, const int32_t* seg_offsets, int32_t* counts, int32_t* tokens, float* prob_sum,
                     float* loss, float balance_coef, float z_coef, float* dlogits, void* ws, size_t ws_bytes,
                     void* stream) {
  clear_error();
  const char* fn = "moe_balance_loss";
  if (int rc = check_balance(fn, logits, T, E, k, num_seg, seg_offsets)) return rc;
  if (!counts || !tokens || !prob_sum || !loss || !ws || (T > 0 && !topk_idx))
    return fail(MOE_ERR_INVALID_ARG, "%s: NULL pointer argument", fn);
  if (!aligned16(ws) || (dlogits && !aligned16(dlogits)))
    return fail(MOE_ERR_ALIGNMENT, "%s: dlogits and ws must be 16-byte aligned", fn);
  const Layout L = layout(T, E, num_seg);
  if (ws_bytes < L.total) return fail(MOE_ERR_WORKSPACE, "%s: workspace %zu < %zu bytes", fn, ws_bytes, L.total);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaMemsetAsync(counts, 0, sizeof(int32_t) * (size_t)num_seg * E, s);
  if (e == cudaSuccess) e = cudaMemsetAsync(tokens, 0, sizeof(int32_t) * (size_t)num_seg, s);
  if (e == cudaSuccess && T == 0) e = cudaMemsetAsync(prob_sum, 0, sizeof(float) * (size_t)num_seg * E, s);
  if (e == cudaSuccess && T == 0) e = cudaMemsetAsync(loss, 0, 2 * sizeof(float), s);
  if (e != cudaSuccess) return fail(MOE_ERR_CUDA, "%s: %s", fn, cudaGetErrorString(e));
  if (T == 0) return MOE_OK;
  const Tokens tk{T, E, k, num_seg, L.chunk, seg_offsets, mask};
  char* base = static_cast<char*>(ws);
  auto* part = reinterpret_cast<float*>(base + L.part);
  auto* zpart = reinterpret_cast<float*>(base + L.zpart);
  auto* share = reinterpret_cast<float2*>(base + L.share);
  auto* ticket = reinterpret_cast<unsigned*>(base + L.ticket);
  const size_t table = sizeof(int) * (size_t)(num_seg + 1);
  launch_pdl(balance_count_kernel, L.nchunk, kThreads, table + sizeof(int) * (size_t)E, s, tk, topk_idx, counts, tokens,
             status_word());
  if (int rc = check_launch(fn, "count kernel")) return rc;
  const Grad gr{balance_coef, z_coef, nullptr, dlogits};
  if (dlogits)
    Main<true, true>::pick(E, L, tk, logits, counts, tokens, gr, part, zpart, ticket, s);
  else
    Main<true, false>::pick(E, L, tk, logits, counts, tokens, gr, part, zpart, ticket, s);
  if (int rc = check_launch(fn, "main kernel")) return rc;
  launch_pdl(balance_finish_kernel, dim3(num_seg, (E + 31) / 32), 1024, table, s, tk, part, zpart, counts, tokens,
             prob_sum, share, ticket, loss, status_word());
  return check_launch(fn, "finish kernel");
}

int moe_balance_loss_bwd(const float* logits, const uint8_t* mask, int T, int E, int k, int num_seg,
                         const int32_t* seg_offsets, const int32_t* counts, const int32_t* tokens, float balance_coef,
                         float z_coef, const float* dloss, float* dlogits, void* stream) {
  clear_error();
  const char* fn = "moe_balance_loss_bwd";
  if (int rc = check_balance(fn, logits, T, E, k, num_seg, seg_offsets)) return rc;
  if (T == 0) return MOE_OK;
  if (!counts || !tokens || !dlogits) return fail(MOE_ERR_INVALID_ARG, "%s: NULL pointer argument", fn);
  if (!aligned16(dlogits)) return fail(MOE_ERR_ALIGNMENT, "%s: dlogits must be 16-byte aligned", fn);
  const Layout L = layout(T, E, num_seg);
  const Tokens tk{T, E, k, num_seg, L.chunk, seg_offsets, mask};
  const Grad gr{balance_coef, z_coef, dloss, dlogits};
  Main<false, true>::pick(E, L, tk, logits, counts, tokens, gr, static_cast<float*>(nullptr),
                          static_cast<float*>(nullptr), static_cast<unsigned*>(nullptr),
                          static_cast<cudaStream_t>(stream));
  return check_launch(fn);
}

}  // extern "C"
