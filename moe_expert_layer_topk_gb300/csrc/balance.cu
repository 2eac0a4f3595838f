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
// Two kernels: the slots are counted per chunk of the token axis, then one CTA
// per (finer) chunk adds up its sequences' counts, walks its tokens and leaves
// its partial sums; the CTA that delivers a sequence's last partial adds them
// and the sequence's losses up, and the one that delivers the last sequence
// writes the totals.  A few tokens are done by a single CTA.
//
// Deterministic: a chunk that reaches into several sequences leaves one partial
// row per sequence, and the rows of a sequence are added in chunk order by
// whichever CTA comes last.  (chunk c, sequence q) sits in row c + q: along the
// token axis every new pair raises one of the two, so no two pairs share a row.
//
// Up to about 65536 tokens x 128 experts a chain of latencies bounds the call
// (two launches, the counts' rows, a piece's sums, its ticket, the last rows:
// 11.5 us at 8192 x 128, 19.0 at 65519 x 128 in one sequence, of which the tokens
// are 7), above it HBM (300000 x 128: 61.7 us, 5.1 TB/s).
#include <cfloat>

#include "common.cuh"
#include "packed_cut.cuh"

namespace moe {
namespace {

constexpr int kMaxSeq = kMaxSegments;
constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;

struct Tokens {  // the packed token axis, cut into chunks
  int T, E, k, num_seq;
  int count_chunks; // chunks of the counting kernel
  const int32_t* seq_offsets;  // null: one sequence of all tokens
  const uint8_t* mask;         // null: every token counts
};

struct Work {                  // in the caller's workspace
  int32_t* cnt_part;           // [count chunk + sequence][E]
  int32_t* tok_part;           // [count chunk + sequence]
  int32_t* tok_chunk;          // [count chunk]
  float* part;                 // [chunk + sequence][E]
  float* zpart;                // [chunk + sequence]
  float2* share;               // [sequence] its part of the two losses
  unsigned* ticket;            // [num_seq + 1] partials delivered, sequences finished
};

struct Out {
  int32_t* counts;
  int32_t* tokens;
  float* prob_sum;
  float* loss;
};

// The sequence table in shared memory, made monotone and clamped to [0, T]
// (a table that is not is reported): off[0..num_seq], and the number of
// sequences with tokens before each, nb[0..num_seq].
__device__ __forceinline__ void load_table(const Tokens& k, int* off, int* nb, int* status) {
  bool bad = false;
  for (int s = threadIdx.x; s <= k.num_seq; s += kThreads) {
    int v = k.seq_offsets ? __ldg(k.seq_offsets + s) : (s == 0 ? 0 : k.T);
    if (v < 0 || v > k.T) {
      bad = true;
      v = v < 0 ? 0 : k.T;
    }
    off[s] = v;
  }
  __syncthreads();
  if (k.num_seq > 1 && threadIdx.x < 32) {
    const int lane = threadIdx.x;
    int carry = 0, full = 0;
    for (int b = 0; b <= k.num_seq; b += 32) {
      const int s = b + lane, v = s <= k.num_seq ? off[s] : 0;
      int m = v;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, m, d);
        if (lane >= d) m = max(m, o);
      }
      m = max(m, carry);
      int before = __shfl_up_sync(0xffffffffu, m, 1);
      if (lane == 0) before = carry;
      const unsigned more = __ballot_sync(0xffffffffu, s > 0 && s <= k.num_seq && m > before);
      if (s <= k.num_seq) {
        bad |= m != v;
        off[s] = m;
        nb[s] = full + __popc(more & (0xffffffffu >> (31 - lane)));
      }
      full += __popc(more);
      carry = __shfl_sync(0xffffffffu, m, 31);
    }
  } else if (k.num_seq == 1 && threadIdx.x == 0) {
    if (off[1] < off[0]) {
      bad = true;
      off[1] = off[0];
    }
    nb[0] = 0;
    nb[1] = off[1] > off[0];
  }
  if (bad) set_status(status, MOE_STATUS_BAD_SEGMENTS);
  __syncthreads();
}

// ------------------------------------------------------------------ counts
// hist[e], *live: the slots and tokens of [a, b) that count (all threads).
// Four slots' loads are under way before the first is counted; a token is
// counted with its first slot.
__device__ __forceinline__ void count_slots(const Tokens& tk, const int32_t* __restrict__ topk_idx, unsigned a, unsigned b, int* hist,
                                            int* live, int* status) {
  constexpr int kSlots = 4;
  for (int e = threadIdx.x; e < tk.E; e += kThreads) hist[e] = 0;
  if (threadIdx.x == 0) *live = 0;
  __syncthreads();
  int mine = 0;
  const unsigned q1 = b * tk.k;  // T k < 2^31
  for (unsigned q0 = a * tk.k + threadIdx.x; q0 < q1; q0 += kSlots * kThreads) {
    int e[kSlots];
    bool on[kSlots];
#pragma unroll
    for (int u = 0; u < kSlots; ++u) {
      const unsigned q = q0 + u * kThreads;
      e[u] = q < q1 ? __ldg(topk_idx + q) : 0;
      on[u] = q < q1;
      if (tk.mask && on[u]) {
        const unsigned t = q / (unsigned)tk.k;
        on[u] = __ldg(tk.mask + t) != 0;
        mine += on[u] && q == t * (unsigned)tk.k;
      }
    }
#pragma unroll
    for (int u = 0; u < kSlots; ++u) {
      if (!on[u]) continue;
      if (e[u] >= 0 && e[u] < tk.E)
        atomicAdd(&hist[e[u]], 1);
      else
        set_status(status, MOE_STATUS_BAD_INDEX);
    }
  }
  if (tk.mask) {
    mine = __reduce_add_sync(0xffffffffu, mine);
    if ((threadIdx.x & 31) == 0 && mine) atomicAdd(live, mine);
  } else if (threadIdx.x == 0) {
    *live = (int)(b - a);
  }
  __syncthreads();
}

// A sequence without tokens: everything about it is zero.
__device__ __forceinline__ void zero_sequence(const Tokens& tk, const Out& o, int s) {
  for (int e = threadIdx.x; e < tk.E; e += kThreads) {
    o.counts[(size_t)s * tk.E + e] = 0;
    o.prob_sum[(size_t)s * tk.E + e] = 0.f;
  }
  if (threadIdx.x == 0) o.tokens[s] = 0;
}

// A piece costs about as much as so many tokens of the count (none: 24.6 us at
// 65519 x 128 in 37 sequences, 128: 23.3).
constexpr int kCountPad = 128;

__global__ void __launch_bounds__(kThreads) balance_count_kernel(const Tokens tk, const int32_t* __restrict__ topk_idx,
                                                                 const Work w, const Out o, int* status) {
  pdl_wait();
  pdl_trigger();
  extern __shared__ int sm[];
  int* off = sm;                      // [num_seq + 1]
  int* nb = off + tk.num_seq + 1;     // [num_seq + 1]
  int* hist = nb + tk.num_seq + 1;    // [E]
  __shared__ int live;
  load_table(tk, off, nb, status);
  const int c = blockIdx.x;
  int total = 0;
  Cut(off, nb, tk.num_seq, gridDim.x, kCountPad).pieces(c, [&](int s, unsigned a, unsigned b) {
    count_slots(tk, topk_idx, a, b, hist, &live, status);
    for (int e = threadIdx.x; e < tk.E; e += kThreads) w.cnt_part[(size_t)(c + s) * tk.E + e] = hist[e];
    if (threadIdx.x == 0) w.tok_part[c + s] = live;
    total += live;
    __syncthreads();
  });
  if (threadIdx.x == 0) w.tok_chunk[c] = total;
  for (int s = c; s < tk.num_seq; s += gridDim.x)
    if (off[s + 1] == off[s]) {
      zero_sequence(tk, o, s);
      if (threadIdx.x == 0) w.share[s] = make_float2(0.f, 0.f);
    }
  if (c == 0) {  // for the main kernel, which starts after this one
    for (int s = threadIdx.x; s <= tk.num_seq; s += kThreads) w.ticket[s] = 0;
    if (threadIdx.x < 2) o.loss[threadIdx.x] = 0.f;
  }
}

// e^x, x <= 0, through the hardware's base-2 exponential: a product's rounding
// more than expf (relative error below 2^-23 |x| + 2^-22) at a third of its
// instructions, which lie on every token's path: 65519 x 128 in 37 sequences 23.3
// us against 24.5 with expf, 65519 x 60 16.1 against 18.6, nothing where HBM binds.
// All outputs are as far from their float64 values either way (8192 and 65519 x
// 128: gradient 8e-8 to 1e-7, sums 5e-8 to 7e-8, losses 4e-8 to 7e-8).
__device__ __forceinline__ float exp_of(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x * 1.4426950408889634f));
  return y;
}

// largest of a warp's values (all lanes converged)
__device__ __forceinline__ float warp_max(float v) {
  float m;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(v));
  return m;
}

// ------------------------------------------------------------- main kernel
//
// LPT lanes hold one token's logits (VEC consecutive values NQ times, VEC LPT
// apart; 16 values a lane where the experts allow it), a warp 32/LPT tokens
// side by side: with a token over all 32 lanes the three reductions' shuffles
// and the per-token instructions bound the kernel (230 issued a token at 128
// experts).  The next token's loads are under way while one is worked on.  The
// lane's share of P stays in registers over the piece and is added over the
// warp's token groups and the warps at its end.  kFull: the lanes' columns are
// the experts exactly.
//
// kInline: one CTA does everything, counting included.
struct Grad {
  float a, b;            // coefficients of the two losses
  const float* dloss;    // their upstream gradients on the device, or null
  float* dlogits;
};

// A piece's counts, sums and ticket cost about as much as so many steps of its
// warps over tokens (2: 25.0 us at 65519 x 128 in 37 sequences, 4: 23.3, 6: 23.9);
// without sums, one.
constexpr int kPieceSteps = 4;

template <int LPT, int VEC, int NQ, bool kFull, bool kSum, bool kGrad, bool kInline>
__global__ void __launch_bounds__(kThreads, 1) balance_main_kernel(const Tokens tk, const float* __restrict__ logits,
                                                                const int32_t* __restrict__ topk_idx, const Work w,
                                                                const Out o, const Grad gr, int* status) {
  constexpr int NV = NQ * VEC;       // values per lane
  constexpr int TPW = 32 / LPT;      // tokens per warp side by side
  // After a counting kernel of the same call, which waited for everything before
  // it, the logits and the table may be read at once; only the counts are waited for.
  constexpr bool kCounted = kSum && !kInline;
  if (!kCounted) pdl_wait();
  pdl_trigger();
  extern __shared__ int sm[];
  int* off = sm;                                                        // [num_seq + 1]
  int* nb = sm + tk.num_seq + 1;                                        // [num_seq + 1]
  int* cnt = sm + ((2 * tk.num_seq + 5) & ~3);                          // [E] the sequence's counts
  float* red = reinterpret_cast<float*>(cnt + ((tk.E + 3) & ~3));       // kSum: [kWarps][E + 1]
  // kSum: every kFold tokens a lane's running sums are moved to sums of sums, so
  // that no fp32 sum takes more than about the square root of a long piece's
  // tokens (16.8 M equal rows in one run: 8e-5 off without)
  float* fold = red + kWarps * (tk.E + 1) + threadIdx.x;                // [NV] kThreads apart
  constexpr int kFold = 64;
  __shared__ int s_n, s_tok;
  __shared__ bool s_last;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = lane / LPT, el = lane % LPT;
  const int E = tk.E;
  load_table(tk, off, nb, status);
  const int chunk = blockIdx.x;
  const int step = kWarps * TPW;
  const Cut cut(off, nb, tk.num_seq, gridDim.x, (kSum ? kPieceSteps : 1) * step);
  const Cut counted(off, nb, tk.num_seq, kCounted ? tk.count_chunks : 1, kCountPad);
  if constexpr (kGrad) {  // tokens outside every sequence get no gradient
    const size_t lo = (size_t)off[0] * E, hi = (size_t)off[tk.num_seq] * E, n = (size_t)tk.T * E;
    const size_t i0 = (size_t)chunk * kThreads + threadIdx.x, di = (size_t)gridDim.x * kThreads;
    for (size_t i = i0; i < lo; i += di) gr.dlogits[i] = 0.f;
    for (size_t i = hi + i0; i < n; i += di) gr.dlogits[i] = 0.f;
  }
  if constexpr (kInline) {
    for (int s = 0; s < tk.num_seq; ++s)
      if (off[s + 1] == off[s]) zero_sequence(tk, o, s);
    if (threadIdx.x < 2) o.loss[threadIdx.x] = 0.f;
  }
  float ga = 0.f, gb = 0.f, rn = 0.f;   // set with the first piece
  float loss_b = 0.f, loss_z = 0.f;     // kInline: thread 0's running totals
  bool ready = false;
  unsigned finished = 0;                // thread 0: sequences this CTA finished
  const unsigned gmask = LPT == 32 ? 0xffffffffu : (((1u << (LPT & 31)) - 1u) << (sub * LPT));
  // over a token's lanes
  auto gmax = [&](float v) {
    if constexpr (LPT == 32) {
      return warp_max(v);
    } else {
#pragma unroll
      for (int d = LPT / 2; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor_sync(gmask, v, d));
      return v;
    }
  };
  auto gsum = [&](float v) {
#pragma unroll
    for (int d = LPT / 2; d > 0; d >>= 1) v += __shfl_xor_sync(gmask, v, d);
    return v;
  };
  auto col = [&](int i) { return (i / VEC) * VEC * LPT + el * VEC + i % VEC; };
  auto has = [&](int i) { return kFull || col(i) < E; };

  // The lane's share of the next token; the rows of tokens that do not count are
  // read and replaced.
  float ln[NV];
  bool onn = false;
  auto load = [&](unsigned t) {
    onn = !tk.mask || __ldg(tk.mask + t);
    const float* src = logits + (size_t)t * E + el * VEC;
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      if constexpr (VEC == 4) {
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (has(4 * q)) v = __ldg(reinterpret_cast<const float4*>(src + q * VEC * LPT));
        ln[4 * q] = v.x; ln[4 * q + 1] = v.y; ln[4 * q + 2] = v.z; ln[4 * q + 3] = v.w;
      } else {
        ln[q] = has(q) ? __ldg(src + q * LPT) : 0.f;
      }
    }
  };

  cut.pieces(chunk, [&](int s, unsigned a, unsigned b) {
    float acc[kSum ? NV : 1];
    float cf[kGrad ? NV : 1];
    float z = 0.f, z_fold = 0.f;
    int since = 0;
    bool folded = false;
    TokenWalk walk{a + warp * TPW + sub, b, (unsigned)step};
    if (walk.more()) load(walk.t);  // under way while the counts are added up
    const int cc0 = kCounted ? counted.first(s) : 0, cc1 = kCounted ? counted.last(s) + 1 : 0;
    if constexpr (kCounted)
      if (!ready) pdl_wait();
    // this sequence's counts and, with the first piece, the call's tokens and sequences
    if (threadIdx.x == 0) s_tok = 0;
    if (!ready && threadIdx.x == 0) s_n = 0;
    if constexpr (kSum && !kInline) {
      int tok = 0, n = 0;
      for (int c = cc0 + threadIdx.x; c < cc1; c += kThreads) tok += __ldcg(w.tok_part + c + s);
      if (!ready)
        for (int c = threadIdx.x; c < tk.count_chunks; c += kThreads) n += __ldcg(w.tok_chunk + c);
      int iv[NV];
#pragma unroll
      for (int i = 0; i < NV; ++i) iv[i] = 0;
      constexpr int kR = NV <= 16 ? 2 : 1;  // rows in flight
      for (int r0 = cc0 + warp * TPW + sub; r0 < cc1; r0 += kR * step) {
#pragma unroll
        for (int u = 0; u < kR; ++u) {
          const int c = r0 + u * step;
#pragma unroll
          for (int q = 0; q < NQ; ++q) {
            const int e0 = q * VEC * LPT + el * VEC;
            const int32_t* src = w.cnt_part + (size_t)(c + s) * E + e0;
            if (c < cc1 && e0 < E) {
              if constexpr (VEC == 4) {
                const int4 f = __ldcg(reinterpret_cast<const int4*>(src));
                iv[4 * q] += f.x; iv[4 * q + 1] += f.y; iv[4 * q + 2] += f.z; iv[4 * q + 3] += f.w;
              } else {
                iv[q] += __ldcg(src);
              }
            }
          }
        }
      }
      __syncwarp();
#pragma unroll
      for (int d = LPT; d < 32; d <<= 1) {
#pragma unroll
        for (int i = 0; i < NV; ++i) iv[i] += __shfl_xor_sync(0xffffffffu, iv[i], d);
      }
      int* rows = reinterpret_cast<int*>(red);
      if (sub == 0) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
          if (has(i)) rows[warp * E + col(i)] = iv[i];
      }
      tok = __reduce_add_sync(0xffffffffu, tok);
      n = __reduce_add_sync(0xffffffffu, n);
      __syncthreads();
      if (lane == 0 && tok) atomicAdd(&s_tok, tok);
      if (lane == 0 && n) atomicAdd(&s_n, n);
      for (int e = threadIdx.x; e < E; e += kThreads) {
        int v = 0;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) v += rows[i * E + e];
        cnt[e] = v;
      }
      __syncthreads();
    } else if (!ready) {
      __syncthreads();
      int n = 0;
      if constexpr (kInline) {
        if (tk.mask) {
          for (int t = off[0] + threadIdx.x; t < off[tk.num_seq]; t += kThreads) n += __ldg(tk.mask + t) != 0;
        } else if (threadIdx.x == 0) {
          n = off[tk.num_seq] - off[0];
        }
      } else {
        for (int q = threadIdx.x; q < tk.num_seq; q += kThreads) n += o.tokens[q];
      }
      n = __reduce_add_sync(0xffffffffu, n);
      if (lane == 0 && n) atomicAdd(&s_n, n);
      __syncthreads();
    }
    if constexpr (kInline) count_slots(tk, topk_idx, a, b, cnt, &s_tok, status);
    if (!ready) {
      rn = 1.f / (float)max(s_n, 1);
      if constexpr (kGrad) {
        ga = gr.a * (gr.dloss ? gr.dloss[0] : 1.f) * ((float)E / (float)tk.k) * rn;
        gb = gr.b * (gr.dloss ? gr.dloss[1] : 1.f) * 2.f * rn;
      }
      ready = true;
    }
    float ga_s = 0.f;
    if constexpr (kGrad) {
      ga_s = ga / (float)max(kSum ? s_tok : o.tokens[s], 1);
#pragma unroll
      for (int i = 0; i < NV; ++i)
        cf[i] = has(i) ? (float)(kSum ? cnt[col(i)] : o.counts[(size_t)s * E + col(i)]) : 0.f;
    }
    if constexpr (kSum) {
#pragma unroll
      for (int i = 0; i < NV; ++i) acc[i] = 0.f;
    }
    while (walk.more()) {
      float l[NV];
      const bool on = onn;
#pragma unroll
      for (int i = 0; i < NV; ++i) l[i] = has(i) ? ln[i] : -INFINITY;
      if (!on) {
#pragma unroll
        for (int i = 0; i < NV; ++i) l[i] = 0.f;
      }
      const unsigned here = walk.t;
      walk.next();
      if (walk.more()) load(walk.t);
      float m = l[0], sum = 0.f, dot = 0.f;
#pragma unroll
      for (int i = 1; i < NV; ++i) m = fmaxf(m, l[i]);
      m = gmax(m);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        // a real logit may be +inf or NaN, whose NaN has to show
        l[i] = has(i) ? exp_of(l[i] - m) : 0.f;
        sum += l[i];
        if constexpr (kGrad) dot = fmaf(cf[i], l[i], dot);
      }
      sum = gsum(sum);
      if constexpr (kGrad) dot = gsum(dot);
      const float r = on ? 1.f / sum : 0.f;
      const float lse = m + logf(sum);
      if constexpr (kSum) {
#pragma unroll
        for (int i = 0; i < NV; ++i) acc[i] = fmaf(l[i], r, acc[i]);
        if (el == 0 && on) z = fmaf(lse, lse, z);
        if (++since == kFold) {
          since = 0;
#pragma unroll
          for (int i = 0; i < NV; ++i) {
            fold[i * kThreads] = folded ? fold[i * kThreads] + acc[i] : acc[i];
            acc[i] = 0.f;
          }
          z_fold += z;
          z = 0.f;
          folded = true;
        }
      }
      if constexpr (kGrad) {
        const float ar = ga_s * r, c = (gb * lse - ga_s * dot * r) * r;
        float* d = gr.dlogits + (size_t)here * E + el * VEC;
#pragma unroll
        for (int q = 0; q < NQ; ++q) {
          if (has(VEC * q)) {
            float dl[VEC];
#pragma unroll
            for (int i = 0; i < VEC; ++i) dl[i] = l[VEC * q + i] * fmaf(ar, cf[VEC * q + i], c);
            if constexpr (VEC == 4)
              *reinterpret_cast<float4*>(d + q * VEC * LPT) = make_float4(dl[0], dl[1], dl[2], dl[3]);
            else
              d[q * LPT] = dl[0];
          }
        }
      }
    }
    if constexpr (kSum) {
      if (folded) {
#pragma unroll
        for (int i = 0; i < NV; ++i) acc[i] += fold[i * kThreads];
        z += z_fold;
      }
      // acc and z over the warp's token groups and the warps: red[0..E)
      auto gather = [&]() {
        __syncwarp();
#pragma unroll
        for (int d = LPT; d < 32; d <<= 1) {
#pragma unroll
          for (int i = 0; i < NV; ++i) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], d);
        }
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) z += __shfl_xor_sync(0xffffffffu, z, d);
        __syncthreads();  // red is free
        if (sub == 0) {
#pragma unroll
          for (int i = 0; i < NV; ++i)
            if (has(i)) red[warp * (E + 1) + col(i)] = acc[i];
        }
        if (lane == 0) red[warp * (E + 1) + E] = z;
        __syncthreads();
        for (int e = threadIdx.x; e <= E; e += kThreads) {
          float v = 0.f;
#pragma unroll
          for (int i = 0; i < kWarps; ++i) v += red[i * (E + 1) + e];
          red[e] = v;
        }
      };
      gather();
      bool finish = true;
      const int c0 = cut.first(s), c1 = cut.last(s) + 1;
      if (!kInline && c1 - c0 > 1) {  // a sequence wholly in this chunk needs no others' partials
        for (int e = threadIdx.x; e <= E; e += kThreads) {  // each thread its own sums
          if (e < E)
            w.part[(size_t)(chunk + s) * E + e] = red[e];
          else
            w.zpart[chunk + s] = red[e];
        }
        __threadfence();
        __syncthreads();
        if (threadIdx.x == 0) s_last = atomicAdd(w.ticket + s, 1u) == (unsigned)(c1 - c0 - 1);
        __syncthreads();
        finish = s_last;
        if (finish) {
          // this CTA delivered the sequence's last partial: all of them, in chunk
          // order, rows taken like tokens
          __threadfence();
          z = 0.f;
#pragma unroll
          for (int i = 0; i < NV; ++i) acc[i] = 0.f;
          for (int c = c0 + threadIdx.x; c < c1; c += kThreads) z += __ldcg(w.zpart + c + s);
          constexpr int kR = NV <= 16 ? 2 : 1;
          for (int r0 = c0 + warp * TPW + sub; r0 < c1; r0 += kR * step) {
            float v[kR][NV];
#pragma unroll
            for (int u = 0; u < kR; ++u) {
              const int c = r0 + u * step;
#pragma unroll
              for (int q = 0; q < NQ; ++q) {
                const int e0 = q * VEC * LPT + el * VEC;
                const float* src = w.part + (size_t)(c + s) * E + e0;
                if constexpr (VEC == 4) {
                  float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
                  if (c < c1 && e0 < E) f = __ldcg(reinterpret_cast<const float4*>(src));
                  v[u][4 * q] = f.x; v[u][4 * q + 1] = f.y; v[u][4 * q + 2] = f.z; v[u][4 * q + 3] = f.w;
                } else {
                  v[u][q] = c < c1 && e0 < E ? __ldcg(src) : 0.f;
                }
              }
            }
#pragma unroll
            for (int u = 0; u < kR; ++u)
#pragma unroll
              for (int i = 0; i < NV; ++i) acc[i] += v[u][i];
          }
          gather();
        }
      }
      if (finish) {
        __syncthreads();
        float dot = 0.f;
        for (int e = threadIdx.x; e < E; e += kThreads) {
          o.prob_sum[(size_t)s * E + e] = red[e];
          o.counts[(size_t)s * E + e] = cnt[e];
          dot = fmaf(red[e], (float)cnt[e], dot);
        }
        const float zz = red[E];
        __syncthreads();
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) dot += __shfl_xor_sync(0xffffffffu, dot, d);
        if (lane == 0) red[warp] = dot;
        __syncthreads();
        if (threadIdx.x == 0) {
          float t = 0.f;
          for (int i = 0; i < kWarps; ++i) t += red[i];
          o.tokens[s] = s_tok;
          const float2 sh = make_float2(t * ((float)E / (float)tk.k) / (float)max(s_tok, 1) * rn, zz * rn);
          if constexpr (kInline) {
            loss_b += sh.x;
            loss_z += sh.y;
            o.loss[0] = loss_b;
            o.loss[1] = loss_z;
          } else if (tk.num_seq == 1) {
            o.loss[0] = sh.x;
            o.loss[1] = sh.y;
          } else {
            __stcg(w.share + s, sh);
            ++finished;
          }
        }
      }
      __syncthreads();
    }
  });
  if constexpr (kCounted) {
    // a CTA without a piece still may not end before the counting kernel does
    if (!ready) pdl_wait();
    if (tk.num_seq > 1) {  // the CTA that finishes the last sequence adds the shares up in order
      if (threadIdx.x == 0) {
        s_last = false;
        if (finished > 0) {
          __threadfence();
          s_last = atomicAdd(w.ticket + tk.num_seq, finished) + finished == (unsigned)nb[tk.num_seq];
        }
      }
      __syncthreads();
      if (!s_last) return;
      __threadfence();
      float lb = 0.f, lz = 0.f;
      for (int i = threadIdx.x; i < tk.num_seq; i += kThreads) {
        const float2 h = __ldcg(w.share + i);
        lb += h.x;
        lz += h.y;
      }
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        lb += __shfl_xor_sync(0xffffffffu, lb, d);
        lz += __shfl_xor_sync(0xffffffffu, lz, d);
      }
      if (lane == 0) {
        red[2 * warp] = lb;
        red[2 * warp + 1] = lz;
      }
      __syncthreads();
      if (threadIdx.x == 0) {
        lb = lz = 0.f;
        for (int i = 0; i < kWarps; ++i) {
          lb += red[2 * i];
          lz += red[2 * i + 1];
        }
        o.loss[0] = lb;
        o.loss[1] = lz;
      }
    }
  }
}

// --------------------------------------------------------------- host side

size_t align256(size_t b) { return (b + 255) & ~size_t(255); }

// Main chunks: one CTA per SM, about 64 tokens each at least (what a CTA of 128
// experts works on at a time); counting chunks fewer, since every main CTA adds
// their rows up.
constexpr int kMaxChunks = 152, kMaxCountChunks = 304;
// One CTA does the whole of a problem of up to so many logits (and few sequences).
constexpr int kInlineLogits = 8192, kInlineSeqs = 4;

int chunks(int T, int num_seq, int most) {
  const int c = T / 64 + (T % 64 != 0) + num_seq - 1;
  return c < most ? c : most;
}

bool is_inline(int T, int E, int num_seq) { return (long long)T * E <= kInlineLogits && num_seq <= kInlineSeqs; }

struct Layout {
  int nchunk, ncount;
  size_t cnt, tok, tokc, part, zpart, share, ticket, total;
};
Layout layout(int T, int E, int num_seq) {
  Layout L;
  L.nchunk = chunks(T, num_seq, kMaxChunks);
  L.ncount = chunks(T, num_seq, kMaxCountChunks);
  const size_t rows = (size_t)L.nchunk + num_seq, crows = (size_t)L.ncount + num_seq;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += align256(bytes);
    return here;
  };
  L.cnt = take(crows * E * sizeof(int32_t));
  L.tok = take(crows * sizeof(int32_t));
  L.tokc = take((size_t)L.ncount * sizeof(int32_t));
  L.part = take(rows * E * sizeof(float));
  L.zpart = take(rows * sizeof(float));
  L.share = take((size_t)num_seq * sizeof(float2));
  L.ticket = take((size_t)(num_seq + 1) * sizeof(unsigned));
  L.total = at;
  return L;
}

template <bool kSum, bool kGrad, bool kInline>
struct Main {
  // nv: values a lane holds
  static constexpr size_t smem_bytes(int num_seq, int E, int nv) {
    return sizeof(int) * (((2 * num_seq + 5) & ~3) + ((E + 3) & ~3)) + (kSum ? sizeof(float) * (kWarps * (E + 1) + nv * kThreads) : 0);
  }
  template <int LPT, int VEC, int NQ, bool kFull>
  static int go(const char* fn, int grid, const Tokens& tk, const float* logits, const int32_t* idx, const Work& w, const Out& o,
                const Grad& gr, cudaStream_t s) {
    const size_t smem = smem_bytes(tk.num_seq, tk.E, VEC * NQ);
    auto kern = balance_main_kernel<LPT, VEC, NQ, kFull, kSum, kGrad, kInline>;
    // Asked for once per device whatever this call's size: beside the kernel's
    // static variables even 48 KB of dynamic shared memory are more than a launch
    // has unasked.  The most that an accepted shape takes is below it.
    constexpr size_t kMost = 160 * 1024;
    static_assert(smem_bytes(kMaxSeq, kMaxExperts, VEC * NQ) <= kMost, "shared memory limit exceeded");
    static bool set[64] = {};
    const int dev = current_device();
    if (dev < 0) return fail(MOE_ERR_CUDA, "%s: no current CUDA device", fn);
    if (!set[dev]) {
      const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMost);
      if (e != cudaSuccess) return fail_cuda(fn, e);
      set[dev] = true;
    }
    launch_pdl(kern, grid, kThreads, smem, s, tk, logits, idx, w, o, gr, status_word());
    return check_launch(fn, "main kernel");
  }
  // experts in fours; full: they fill the lanes' columns (a single CTA is latency-bound either way)
  template <int LPT, int NQ, class... A>
  static int fours(const char* fn, int grid, const Tokens& tk, A&&... a) {
    if constexpr (!kInline)
      if (tk.E == 4 * LPT * NQ) return go<LPT, 4, NQ, true>(fn, grid, tk, a...);
    return go<LPT, 4, NQ, false>(fn, grid, tk, a...);
  }
  template <class... A>
  static int pick(const char* fn, int grid, const Tokens& tk, A&&... a) {
    const int E = tk.E;
    if (E % 4 == 0) {
      if (E <= 16) return fours<1, 4>(fn, grid, tk, a...);
      if (E <= 32) return fours<2, 4>(fn, grid, tk, a...);
      if (E <= 64) return fours<4, 4>(fn, grid, tk, a...);
      if (E <= 128) return fours<8, 4>(fn, grid, tk, a...);
      if (E <= 256) return fours<16, 4>(fn, grid, tk, a...);
      if (E <= 512) return fours<32, 4>(fn, grid, tk, a...);
      return fours<32, 8>(fn, grid, tk, a...);
    }
    if (E <= 16) return go<4, 1, 4, false>(fn, grid, tk, a...);
    if (E <= 64) return go<16, 1, 4, false>(fn, grid, tk, a...);
    if (E <= 256) return go<32, 1, 8, false>(fn, grid, tk, a...);
    return go<32, 1, 32, false>(fn, grid, tk, a...);
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
  if (T == 0) {
    cudaError_t e = cudaMemsetAsync(counts, 0, sizeof(int32_t) * (size_t)num_seg * E, s);
    if (e == cudaSuccess) e = cudaMemsetAsync(tokens, 0, sizeof(int32_t) * (size_t)num_seg, s);
    if (e == cudaSuccess) e = cudaMemsetAsync(prob_sum, 0, sizeof(float) * (size_t)num_seg * E, s);
    if (e == cudaSuccess) e = cudaMemsetAsync(loss, 0, 2 * sizeof(float), s);
    if (e != cudaSuccess) return fail_cuda(fn, e);
    return MOE_OK;
  }
  const Tokens tk{T, E, k, num_seg, L.ncount, seg_offsets, mask};
  char* base = static_cast<char*>(ws);
  const Work w{reinterpret_cast<int32_t*>(base + L.cnt),  reinterpret_cast<int32_t*>(base + L.tok),
               reinterpret_cast<int32_t*>(base + L.tokc), reinterpret_cast<float*>(base + L.part),
               reinterpret_cast<float*>(base + L.zpart),  reinterpret_cast<float2*>(base + L.share),
               reinterpret_cast<unsigned*>(base + L.ticket)};
  const Out o{counts, tokens, prob_sum, loss};
  const Grad gr{balance_coef, z_coef, nullptr, dlogits};
  if (is_inline(T, E, num_seg))
    return dlogits ? Main<true, true, true>::pick(fn, 1, tk, logits, topk_idx, w, o, gr, s)
                   : Main<true, false, true>::pick(fn, 1, tk, logits, topk_idx, w, o, gr, s);
  launch_pdl(balance_count_kernel, L.ncount, kThreads, sizeof(int) * (size_t)(2 * num_seg + 2 + E), s, tk, topk_idx, w, o,
             status_word());
  if (int rc = check_launch(fn, "count kernel")) return rc;
  return dlogits ? Main<true, true, false>::pick(fn, L.nchunk, tk, logits, topk_idx, w, o, gr, s)
                 : Main<true, false, false>::pick(fn, L.nchunk, tk, logits, topk_idx, w, o, gr, s);
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
  const Tokens tk{T, E, k, num_seg, L.ncount, seg_offsets, mask};
  const Out o{const_cast<int32_t*>(counts), const_cast<int32_t*>(tokens), nullptr, nullptr};  // read only
  const Grad gr{balance_coef, z_coef, dloss, dlogits};
  return Main<false, true, false>::pick(fn, L.nchunk, tk, logits, static_cast<const int32_t*>(nullptr), Work{}, o, gr,
                                        static_cast<cudaStream_t>(stream));
}

}  // extern "C"
