// A projection shared by all requests plus a low-rank adapter for each
// request, forward and backward.
//
// Row t of a request with adapter a:
//   y_t  = W x_t + B_a v_t,        v_t = s_a A_a x_t
//   dx_t = W^T dy_t + A_a^T u_t,   u_t = s_a B_a^T dy_t
//   dA_a = sum_t u_t x_t^T,        dB_a = sum_t dy_t v_t^T
// Rows of requests without an adapter leave the second terms out.
//
// Two products per direction.  The narrow one (v or u, r <= 128 columns,
// bound by reading x or dy) writes its fp32 result as three bf16 parts whose
// sum is that value (8 bits each), so the products that take it stay on the
// tensor cores without losing what the first one computed: the gradients of
// A and B and the wide product take all three.  The wide one appends the
// adapter to the shared projection's reduction: after the W blocks, the same
// accumulator tile takes v_t's parts times B_a for every run of rows with one
// adapter, with the tile's other rows switched off by the MMA's lane mask
// (tcgen05.mma disable-output-lane).  A tile may so hold any mix of requests,
// no row is computed for another request's adapter, and a non-finite value in
// one request's row or adapter reaches no other row.
//
// Measured (r = 16 unless said; graph replays, cold L2 not forced):
//   1 row, 2048 x 2048, one request                7.2 us   launches and latency
//   64 rows of 64 requests, 48 adapters            11.5     masked MMAs, one run a row
//   517 rows, mixed, r = 64, 768 x 2048            26.0     the same
//   16381 rows, 2048 x 4096, r = 32                170-181  tensor cores: 0.28 TFLOP of the
//                                                  wide product in 149, narrow 24 before it
//   8192 rows, 2048 x 2048, backward               121.8 with the forward: narrow 14 and
//                                                  wide 44 each way, gradients 18 + 6, in part
//                                                  beside them (r = 64: 149.1)
//
// With v and u at 16 bits in the wide product (two parts) these took 11.9 (12.3
// now, in turn with it), 23.6 (26.6), 177.3 (180.1), 120.7 (121.8) and 140.5
// (149.1); but where W x cancels the adapter's term, those 16 bits were all that
// y had.
#include <cuda.h>

#include "tc_common.cuh"

namespace moe {
namespace tc {
namespace {

constexpr int kPlanes = 3;        // bf16 parts of v, u
constexpr int kMaxRank = 128;
constexpr int kMaxAdapters = 1024;

__host__ __device__ constexpr int round_up(int v, int to) { return (v + to - 1) / to * to; }
// Columns of one part in the hidden tensor: whole 16-wide MMA steps when all
// parts fit two 64-column blocks (and no part crosses from one to the next),
// else whole 64-column blocks.
__host__ __device__ constexpr bool parts_packed(int r) { return r <= 32; }
__host__ __device__ constexpr int plane_cols(int r) { return parts_packed(r) ? round_up(r, 16) : round_up(r, 64); }
// Columns of all parts, and of a row of the hidden tensor (whole 64-column
// blocks; what pads a row is never used).
__host__ __device__ constexpr int hidden_cols(int r) { return kPlanes * plane_cols(r); }
__host__ __device__ constexpr int hidden_pitch(int r) { return round_up(hidden_cols(r), 64); }
// 64-column blocks that hold the parts of up to 64 ranks.
__host__ __device__ constexpr int hidden_blocks(int r) { return parts_packed(r) ? hidden_pitch(r) / 64 : kPlanes; }

// ------------------------------------------------------------ request table

struct Reqs {
  int T, num_seg, num_adapters;
  const int32_t* offsets;  // [num_seg + 1]
  const int32_t* adapter;  // [num_seg], negative: none
};

__host__ __device__ constexpr size_t table_bytes(int num_seg) { return (size_t)(num_seg + 2) * 4 + (size_t)(num_seg + 2) * 2; }

// Shared-memory copy: offsets made monotone and clamped to [0, T], adapter ids
// out of range replaced by -1 (both reported).  off[num_seg + 1], ad[num_seg].
// Threads from `from` on (a multiple of 32) read it, that warp closes it.
__device__ __forceinline__ void load_requests(const Reqs& q, int* off, int16_t* ad, int* status, int from = 0) {
  if (q.num_seg == 0) {  // there may be no table at all
    if (threadIdx.x == 0) off[0] = 0;
    __syncthreads();
    return;
  }
  bool bad = false;
  for (int s = (int)threadIdx.x - from; s >= 0 && s <= q.num_seg; s += blockDim.x - from) {
    int v = __ldg(q.offsets + s);
    if (v < 0 || v > q.T) {
      bad = true;
      v = v < 0 ? 0 : q.T;
    }
    off[s] = v;
    if (s < q.num_seg) {
      int a = __ldg(q.adapter + s);
      if (a >= q.num_adapters || a < -1) {
        bad = true;
        a = -1;
      }
      ad[s] = (int16_t)a;
    }
  }
  __syncthreads();
  if ((int)threadIdx.x >= from && (int)threadIdx.x < from + 32) {
    const int lane = threadIdx.x & 31;
    int carry = 0;
    for (int b = 0; b <= q.num_seg; b += 32) {
      const int s = b + lane, v = s <= q.num_seg ? off[s] : 0;
      int m = v;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, m, d);
        if (lane >= d) m = max(m, o);
      }
      m = max(m, carry);
      if (s <= q.num_seg) {
        bad |= m != v;
        off[s] = m;
      }
      carry = __shfl_sync(0xffffffffu, m, 31);
    }
  }
  if (bad) set_status(status, MOE_STATUS_BAD_SEGMENTS);
  __syncthreads();
}

// First request that ends after row t.
__device__ __forceinline__ int first_request(const int* off, int num_seg, int t) {
  int lo = 0, hi = num_seg;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (off[mid + 1] > t) hi = mid; else lo = mid + 1;
  }
  return lo;
}

// A run: rows lo <= row - m0 < hi of a tile with one adapter;
// neighbouring requests with the same adapter are one run.
struct Run {
  int lo, hi, a;
};
__device__ __forceinline__ Run unpack_run(uint32_t v) {
  return {(int)(v & 0xFFu), (int)((v >> 8) & 0xFFu) + 1, (int)(v >> 16)};
}

// Adapter of row t, -1: none.
__device__ __forceinline__ int adapter_of_row(const int* off, const int16_t* ad, int num_seg, int t) {
  const int s = first_request(off, num_seg, t);
  return s < num_seg && off[s] <= t ? ad[s] : -1;
}

// The runs of a tile of 32 NW rows into list (32 NW entries), in row order, from
// the adapters of rows 32 w + lane (-1: none); returns how many.  A warp's
// common work: run starts are found and numbered by ballots (walking the table
// request by request took 0.07 us a request, more than the run's products).
template <int NW>
__device__ __forceinline__ int list_runs(const int (&a)[NW], uint32_t* list) {
  const int lane = threadIdx.x & 31;
  __syncwarp();  // the list's last reader is done
  uint32_t start[NW], brk[NW];
  int before = -1;  // adapter of the row before this word
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    const int up = __shfl_up_sync(0xffffffffu, a[w], 1);
    const int prev = lane == 0 ? before : up;
    start[w] = __ballot_sync(0xffffffffu, a[w] >= 0 && a[w] != prev);
    brk[w] = start[w] | __ballot_sync(0xffffffffu, a[w] < 0);
    before = __shfl_sync(0xffffffffu, a[w], 31);
  }
  int n = 0;
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    if ((start[w] >> lane) & 1u) {
      const uint32_t later = lane == 31 ? 0u : brk[w] & (0xffffffffu << (lane + 1));
      int hi = later ? 32 * w + __ffs(later) - 1 : -1;
#pragma unroll
      for (int v = 0; v < NW; ++v)
        if (v > w && hi < 0 && brk[v]) hi = 32 * v + __ffs(brk[v]) - 1;
      if (hi < 0) hi = 32 * NW;
      list[n + __popc(start[w] & ((1u << lane) - 1u))] = (uint32_t)(32 * w + lane) | (uint32_t)(hi - 1) << 8 | (uint32_t)a[w] << 16;
    }
    n += __popc(start[w]);
  }
  __syncwarp();
  return n;
}

// The same from the request table, for the rows of [m0, m1).
template <int NW>
__device__ __forceinline__ int build_runs(const int* off, const int16_t* ad, int num_seg, int m0, int m1, uint32_t* list) {
  int a[NW];
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    const int t = m0 + 32 * w + (threadIdx.x & 31);
    a[w] = t < m1 ? adapter_of_row(off, ad, num_seg, t) : -1;
  }
  return list_runs<NW>(a, list);
}

// Word w of the MMA's lane mask (1 = lane off) that leaves rows [lo, hi) on.
__device__ __forceinline__ uint32_t lanes_off(int lo, int hi, int w) {
  const int a = max(lo - 32 * w, 0);
  uint32_t on;
  asm("bmsk.clamp.b32 %0, %1, %2;" : "=r"(on) : "r"(a), "r"(max(min(hi - 32 * w, 32) - a, 0)));
  return ~on;
}

// Lane mask of a tile of 128 rows (one CTA) or 256 (a pair: the second CTA's
// 128 lanes in words 4..7).
template <int CTAS>
struct LaneMask {
  uint32_t w[4 * CTAS];
};
template <int CTAS>
__device__ __forceinline__ LaneMask<CTAS> lane_mask(int lo, int hi) {
  LaneMask<CTAS> m;
#pragma unroll
  for (int i = 0; i < 4 * CTAS; ++i) m.w[i] = lanes_off(lo, hi, i);
  return m;
}

// D (+)= A B that leaves the accumulator rows of masked lanes as they are.
__device__ __forceinline__ void mma_lanes(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate,
                                          const LaneMask<1>& m) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, {%5, %6, %7, %8}, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(m.w[0]), "r"(m.w[1]), "r"(m.w[2]), "r"(m.w[3])
      : "memory");
}
__device__ __forceinline__ void mma_lanes(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate,
                                          const LaneMask<2>& m) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, {%5, %6, %7, %8, %9, %10, %11, %12}, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(m.w[0]), "r"(m.w[1]), "r"(m.w[2]), "r"(m.w[3]), "r"(m.w[4]),
      "r"(m.w[5]), "r"(m.w[6]), "r"(m.w[7])
      : "memory");
}

template <int CTAS>
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0, int c1, int c2,
                                            int c3) {
  if constexpr (CTAS == 1)
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
        : "memory");
}

__device__ __forceinline__ void st_cluster(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
__device__ __forceinline__ float ld_cluster(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr));
  return v;
}

// True in one lane of a converged warp.  The compiler knows such a branch for
// one thread's and keeps its values in uniform registers: the MMA loop under
// it issues a block's four MMAs in about 0.2 us less than under lane == 0.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred P;\n\telect.sync _|P, 0xffffffff;\n\tselp.u32 %0, 1, 0, P;\n\t}" : "=r"(p));
  return p != 0;
}

__device__ __forceinline__ uint32_t align1k(uint32_t a) { return (a + 1023u) & ~1023u; }

constexpr float kLargestBf16 = 0x1.FEp127f;

// v split into kPlanes bf16 parts, largest first, 8 columns: one 16-byte vector a part
__device__ __forceinline__ void split8(const float (&v)[8], uint4 (&out)[kPlanes]) {
  float rest[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) rest[i] = v[i];
#pragma unroll
  for (int p = 0; p < kPlanes; ++p) {
    float h[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      // A finite value above the largest bf16 number starts with that one (the
      // nearest would be infinity); of an infinity or a NaN, whose difference would
      // be NaN, only the first part is kept.
      const bool finite = isfinite(rest[i]);
      h[i] = __bfloat162float(__float2bfloat16_rn(finite ? fminf(fmaxf(rest[i], -kLargestBf16), kLargestBf16) : rest[i]));
      rest[i] = finite ? rest[i] - h[i] : 0.f;
    }
    out[p] = pack8(h);
  }
}

// ------------------------------------------------- narrow product, tensor cores
//
// hidden[t] = parts of s_a F_a . in[t] for 128 rows a cluster; the cluster's
// CTAs share the reduction (a K slice each) and add their fp32 accumulators
// through distributed shared memory.  F_a is A_a [r, K] (K-major operand) or
// B_a^T, read from B_a [N, r] as it lies (MN-major operand).  One row tile's
// runs follow one another for every block of the reduction, each with the
// lanes of the other runs off, so x is read once whatever the mix of requests.
// With few runs it is bound by reading x (8192 x 2048: 13 us, 2.6 TB/s with the
// start and the sums across the cluster), with many by issuing their MMAs.
struct ShrinkParams {
  Reqs q;
  int red;              // reduction length
  int nrank;            // CTAs of a cluster
  int r, rN;            // rank, MMA columns (rank up to a multiple of 16)
  int f_bytes;          // shared-memory bytes of one F block
  int f_rows;           // rows of F's 2-D view per adapter
  int x_stages, f_stages;  // steps of x and of F in flight
  int f_runs;              // runs a step of F holds
  const float* scale;   // [num_adapters] or null
  __nv_bfloat16* hidden;
  uint32_t idesc;
  uint32_t tmem_cols;
  int* status;
};
constexpr int kShrinkK = 2;                  // 64-column blocks of the reduction a step
constexpr int kShrinkX = 3, kShrinkF = 12;   // steps of x in flight, of F at most
constexpr int kShrinkXBytes = kShrinkK * BM * BK * 2;

struct ShrinkCtl {
  unsigned long long xfull[kShrinkX], xempty[kShrinkX], ffull[kShrinkF], fempty[kShrinkF], done;
  uint32_t tmem_base;
  int abort_flag;
  int row_ad[BM];
  float row_scale[BM];
  uint32_t runs[2][BM];  // the loading warp's and the MMA warp's
};

template <bool kMN>
__global__ void __launch_bounds__(192) adapter_shrink_kernel(const __grid_constant__ CUtensorMap tmX,
                                                             const __grid_constant__ CUtensorMap tmF,
                                                             const ShrinkParams p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ ShrinkCtl ctl;
  const uint32_t base = align1k(smem_u32(smem_raw));
  uint8_t* bytes = smem_raw + (base - smem_u32(smem_raw));
  const int f_run = kShrinkK * p.f_bytes, f_stage = p.f_runs * f_run;
  const uint32_t sX = base, sF = base + p.x_stages * kShrinkXBytes;
  // the slices' sums of this CTA's share of the rows: [slice][rN][rows]
  float* sums = reinterpret_cast<float*>(bytes + p.x_stages * kShrinkXBytes + p.f_stages * f_stage);
  int* off = reinterpret_cast<int*>(sums + p.rN * BM);
  int16_t* ad = reinterpret_cast<int16_t*>(off + p.q.num_seg + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nrank = p.nrank, rank = (int)cluster_rank();
  const int m0 = (int)(blockIdx.x / nrank) * BM, m1 = min(p.q.T, m0 + BM);
  const int nkb = p.red / BK;
  const int kb0 = (int)((long long)nkb * rank / nrank), kb1 = (int)((long long)nkb * (rank + 1) / nrank);
  auto load_x = [&](int kb, int xs) {
    const int nb = min(kShrinkK, kb1 - kb);
    const uint32_t xb = smem_u32(&ctl.xfull[xs]);
    mbar_arrive_expect_tx(xb, nb * (BM * BK * 2));
    for (int i = 0; i < nb; ++i) tma_load_2d(sX + xs * kShrinkXBytes + i * (BM * BK * 2), &tmX, xb, (kb + i) * BK, m0);
  };
  // one warp sets the barriers up and sends for the first blocks, one takes the
  // tensor memory, the others read the request table
  if (warp == 0) {
    for (int i = lane; i < p.x_stages; i += 32) {
      mbar_init(smem_u32(&ctl.xfull[i]), 1);
      mbar_init(smem_u32(&ctl.xempty[i]), 1);
    }
    for (int i = lane; i < p.f_stages; i += 32) {
      mbar_init(smem_u32(&ctl.ffull[i]), 1);
      mbar_init(smem_u32(&ctl.fempty[i]), 1);
    }
    if (lane == 0) {
      mbar_init(smem_u32(&ctl.done), 1);
      ctl.abort_flag = 0;
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    __syncwarp();
    if (elect_one()) {
      prefetch_tmap(&tmX);
      prefetch_tmap(&tmF);
    }
    pdl_wait();  // (so far nothing that an earlier kernel writes or needs)
    __syncwarp();
    if (elect_one()) {
      for (int i = 0; i < p.x_stages && kb0 + i * kShrinkK < kb1; ++i) load_x(kb0 + i * kShrinkK, i);
    }
  } else {
    pdl_wait();
    if (warp == 1) tmem_alloc_n<1>(smem_u32(&ctl.tmem_base), p.tmem_cols);
  }
  load_requests(p.q, off, ad, p.status, 64);
  if (threadIdx.x < BM) {
    const int t = m0 + threadIdx.x;
    const int a = t < m1 ? adapter_of_row(off, ad, p.q.num_seg, t) : -1;
    ctl.row_ad[threadIdx.x] = a;
    ctl.row_scale[threadIdx.x] = a >= 0 && p.scale ? __ldg(p.scale + a) : 1.f;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // only now may the next kernel of the stream start beside this one: it must
  // not take the tensor memory that this one still has to allocate
  pdl_trigger();
  // (waited for before the first access to a peer's shared memory: it has to run by then)
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  const uint32_t tmem = ctl.tmem_base;
  auto runs_to = [&](uint32_t* list) {
    const int a[4] = {ctl.row_ad[lane], ctl.row_ad[32 + lane], ctl.row_ad[64 + lane], ctl.row_ad[96 + lane]};
    return list_runs<4>(a, list);
  };

  if (warp == 0) {
    const int n = runs_to(ctl.runs[0]);
    if (elect_one()) {
      int xs = 0, fs = 0;
      uint32_t xp = 0, fp = 0;
      bool ok = true;
      for (int kb = kb0; ok && kb < kb1; kb += kShrinkK) {
        if (kb >= kb0 + p.x_stages * kShrinkK) {
          if (!wait_bar(smem_u32(&ctl.xempty[xs]), xp ^ 1u, &ctl.abort_flag, p.status)) break;
          load_x(kb, xs);
        }
        if (++xs == p.x_stages) { xs = 0; xp ^= 1u; }
        const int nb = min(kShrinkK, kb1 - kb);
        for (int i = 0; i < n; i += p.f_runs) {
          if (!(ok = wait_bar(smem_u32(&ctl.fempty[fs]), fp ^ 1u, &ctl.abort_flag, p.status))) break;
          const int here = min(p.f_runs, n - i);
          const uint32_t fb = smem_u32(&ctl.ffull[fs]);
          mbar_arrive_expect_tx(fb, here * nb * p.f_bytes);
          for (int g = 0; g < here; ++g) {
            const int a = unpack_run(ctl.runs[0][i + g]).a;
            for (int j = 0; j < nb; ++j) {
              const uint32_t dst = sF + fs * f_stage + g * f_run + j * p.f_bytes;
              if (kMN) {
                for (int c = 0; c < p.r; c += 64) tma_load_2d(dst + c * 128, &tmF, fb, c, a * p.f_rows + (kb + j) * BK);
              } else {
                tma_load_2d(dst, &tmF, fb, (kb + j) * BK, a * p.f_rows);
              }
            }
          }
          if (++fs == p.f_stages) { fs = 0; fp ^= 1u; }
        }
      }
    }
  } else if (warp == 1) {
    const int n = runs_to(ctl.runs[1]);
    if (elect_one()) {
      int xs = 0, fs = 0;
      uint32_t xp = 0, fp = 0;
      bool ok = true;
      for (int kb = kb0; ok && kb < kb1; kb += kShrinkK) {
        if (!(ok = wait_bar(smem_u32(&ctl.xfull[xs]), xp, &ctl.abort_flag, p.status))) break;
        const uint64_t xd = sdesc(sX + xs * kShrinkXBytes, 16, 1024);
        const int nb = min(kShrinkK, kb1 - kb);
        for (int i = 0; i < n; i += p.f_runs) {
          if (!(ok = wait_bar(smem_u32(&ctl.ffull[fs]), fp, &ctl.abort_flag, p.status))) break;
          tc_fence_after();
          const int here = min(p.f_runs, n - i);
          for (int g = 0; g < here; ++g) {
            const Run run = unpack_run(ctl.runs[1][i + g]);
            const LaneMask<1> m = lane_mask<1>(run.lo, run.hi);
            // (descriptors count 16-byte units: blocks and steps add to their low word)
            const uint32_t b0 = sF + fs * f_stage + g * f_run;
            const uint64_t bd = kMN ? sdesc(b0, CHUNK_BYTES, 1024) : sdesc(b0, 16, 1024);
#pragma unroll
            for (int j = 0; j < kShrinkK; ++j) {
              if (j >= nb) break;
              const uint64_t bj = bd + (uint64_t)(j * (p.f_bytes >> 4));
#pragma unroll
              for (int kk = 0; kk < BK / 16; ++kk)
                mma_lanes(tmem, xd + (uint64_t)(j * (BM * BK * 2 / 16) + kk * 2), bj + (uint64_t)(kk * (kMN ? 128 : 2)), p.idesc,
                          kb > kb0 || j > 0 || kk > 0, m);
            }
          }
          mma_commit(smem_u32(&ctl.fempty[fs]));
          if (++fs == p.f_stages) { fs = 0; fp ^= 1u; }
        }
        mma_commit(smem_u32(&ctl.xempty[xs]));
        if (++xs == p.x_stages) { xs = 0; xp ^= 1u; }
      }
      mma_commit(smem_u32(&ctl.done));
    }
  }
  __syncwarp();  // the two roles' other lanes do not spin beside them
  // every MMA of this CTA has ended (on an abort: those issued)
  const bool fine = __all_sync(0xffffffffu, wait_bar(smem_u32(&ctl.done), 0, &ctl.abort_flag, p.status));
  tc_fence_after();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  const int per = BM / nrank;  // rows of a CTA's share
  if (warp >= 2 && fine) {
    // each row's sums go straight to the CTA that finishes the row
    const int row = (warp & 3) * 32 + lane;
    const uint32_t dst = map_to_rank(smem_u32(sums + (size_t)rank * p.rN * per + row % per), row / per);
    for (int c = 0; c < p.rN; c += 16) {
      uint32_t v[16];
      asm volatile(
          "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
          "%15}, [%16];"
          : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
            "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
          : "r"(tmem + ((uint32_t)((warp & 3) * 32) << 16) + (uint32_t)c));
      tmem_wait_ld();
#pragma unroll
      for (int i = 0; i < 16; ++i) st_cluster(dst + (uint32_t)((c + i) * per) * 4, f32(v[i]));
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc_n<1>(tmem, p.tmem_cols);
  cluster_sync();  // all slices' sums have arrived; nothing remote follows
  // the slices' sums in order, scaled and split
  const int rp = plane_cols(p.r), hp = hidden_pitch(p.r);
  for (int i = threadIdx.x; i < per * (rp / 8); i += blockDim.x) {
    const int row = rank * per + i % per, c = i / per * 8;
    if (m0 + row >= p.q.T) continue;
    const int a = ctl.row_ad[row];
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (a >= 0 && c < p.r) {
      for (int k = 0; k < nrank; ++k) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] += sums[((size_t)k * p.rN + c + j) * per + i % per];
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] *= ctl.row_scale[row];
    }
    uint4 o[kPlanes];
    split8(v, o);
#pragma unroll
    for (int k = 0; k < kPlanes; ++k)
      *reinterpret_cast<uint4*>(p.hidden + (size_t)(m0 + row) * hp + k * rp + c) = o[k];
  }
}

// ------------------------------------------------- narrow product, few rows
//
// v_t for requests of a row or a few: one warp a (row, kGemvRanks ranks), the
// lanes along the reduction, fp32 throughout.  Bound by reading each row's own
// A_a once, which spreads over all SMs here; on the tensor cores one 128-row
// tile would walk its adapters one after the other.
constexpr int kGemvRanks = 2, kGemvWarps = 4;

struct GemvParams {
  Reqs q;
  const __nv_bfloat16* x;
  long long ldx;
  const __nv_bfloat16* A;
  const float* scale;
  int K, r;
  __nv_bfloat16* hidden;
  int* status;
};

__global__ void __launch_bounds__(kGemvWarps * 32) adapter_gemv_kernel(const GemvParams p) {
  pdl_wait();
  pdl_trigger();
  extern __shared__ int tab[];
  int* off = tab;
  int16_t* ad = reinterpret_cast<int16_t*>(off + p.q.num_seg + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t = blockIdx.x;
  const int j0 = (blockIdx.y * kGemvWarps + warp) * kGemvRanks;
  const uint4* x = reinterpret_cast<const uint4*>(p.x + (size_t)t * p.ldx);
  const int nv = p.K / 8;
  uint4 xv[4];  // the row's first values, on their way while the table is read
#pragma unroll
  for (int u = 0; u < 4; ++u) xv[u] = u * 32 + lane < nv ? __ldg(x + u * 32 + lane) : make_uint4(0, 0, 0, 0);
  load_requests(p.q, off, ad, p.status);
  const int a = adapter_of_row(off, ad, p.q.num_seg, t);
  const int rp = plane_cols(p.r), hp = hidden_pitch(p.r);
  if (j0 >= rp) return;
  float sum[kGemvRanks] = {0.f, 0.f};
  if (a >= 0 && j0 < p.r) {
    const uint4* f = reinterpret_cast<const uint4*>(p.A + ((size_t)a * p.r + j0) * p.K);
    for (int v0 = 0; v0 < nv; v0 += 128) {
      uint4 fv[kGemvRanks][4];
#pragma unroll
      for (int j = 0; j < kGemvRanks; ++j)
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int v = v0 + u * 32 + lane;
          fv[j][u] = v < nv ? __ldg(f + (size_t)j * nv + v) : make_uint4(0, 0, 0, 0);
        }
      if (v0 > 0) {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int v = v0 + u * 32 + lane;
          xv[u] = v < nv ? __ldg(x + v) : make_uint4(0, 0, 0, 0);
        }
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        float xf[8];
        unpack8(xv[u], xf);
#pragma unroll
        for (int j = 0; j < kGemvRanks; ++j) {
          float ff[8];
          unpack8(fv[j][u], ff);
#pragma unroll
          for (int i = 0; i < 8; ++i) sum[j] = fmaf(xf[i], ff[i], sum[j]);
        }
      }
    }
  }
#pragma unroll
  for (int j = 0; j < kGemvRanks; ++j) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum[j] += __shfl_xor_sync(0xffffffffu, sum[j], d);
  }
  if (lane < kGemvRanks) {  // ranks are even in number, columns past them are zero
    float v[8] = {(lane == 0 ? sum[0] : sum[1]) * (a >= 0 && p.scale ? __ldg(p.scale + a) : 1.f), 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    uint4 o[kPlanes];
    split8(v, o);
#pragma unroll
    for (int k = 0; k < kPlanes; ++k)
      p.hidden[(size_t)t * hp + k * rp + j0 + lane] = __ushort_as_bfloat16((unsigned short)(o[k].x & 0xFFFFu));
  }
}

// ------------------------------------------------------------- wide product
//
// out[128 rows x BN] = in W^T (kMN: in W) + hidden F.  A TMA warp streams the
// blocks of in and W and then, run by run, those of F; one warp lists the next
// tile's runs (a search that cost 2.4 us a tile where the TMA and MMA warps did
// it themselves) and loads hidden's blocks of the tile, once, whatever the
// number of runs; one warp issues the MMAs; four warps write the tile out.
//
// Whole tiles (kSplit false): persistent over the tiles, two accumulators, so
// that a tile's epilogue runs beside the next one's MMAs.  256-column tiles run
// as CTA pairs on 256 rows (tcgen05 cta_group::2: each CTA holds its 128 rows
// of in and half of W's columns, the leader issues the MMAs): one CTA per
// 128 x 256 tile was bound by the 48 KB it loads per block, 18 TB/s over all
// SMs, where a pair's CTA loads 32.  When their last wave would fill less than
// half of the SMs it is given out as 128-column halves.
//
// kSplit: for so few rows that the tiles do not fill the SMs.  A cluster shares
// one tile: each CTA takes a slice of the reduction and every nrank-th run, and
// the fp32 accumulators are added through distributed shared memory, each CTA
// writing a share of the columns.  Blocks of in hold only the rows there are.
struct WideParams {
  Reqs q;
  int red, r;
  int f_rows;          // K-major F: rows of its 2-D view per adapter
  int n_tiles;         // tiles along the columns
  int units;           // whole tiles and halves (kSplit: unused)
  int full;            // units that are whole tiles
  int a_rows;          // rows of a block of in and hidden
  int stages;
  int has_hidden;      // a narrow kernel of the same call wrote hidden
  uint32_t idesc, idesc_half;
  __nv_bfloat16* out;  // kSplit
  long long ldo;
  int* status;
};

constexpr int kWideStagesMax = 12;
constexpr int kWideThreads = 224;

template <int BN, bool kSplit>
struct WideCfg {
  static constexpr int CTAS = BN == 256 ? 2 : 1;
  static constexpr int B_BYTES = BN / CTAS * BK * 2;       // a CTA's share of a block of W
  static constexpr int WB = BN / CTAS > 64 && CTAS == 1 ? BN : 64;  // W rows (columns) of one TMA box
  static constexpr int EP_BYTES = kSplit ? 0 : 4 * EP_SLOTS * EP_BOX_BYTES;
  // three blocks of hidden cost the wider tiles' ring a stage (with two held and
  // the third part in a pass of its own, F's blocks loaded again, 8192 rows forward
  // and backward at r = 64 took 153.7 us instead of 149.1, 517 mixed rows 30.8
  // instead of 26.6)
  static constexpr int stages(int vblocks) { return BN == 64 ? 6 : (vblocks <= 2 ? 5 : 4); }
  static constexpr size_t smem(int a_rows, int vblocks, int stages) {
    // the MMA reads 128 rows from a hidden block's start, however few it holds
    return 1024 + (size_t)stages * (a_rows * BK * 2 + B_BYTES) + (size_t)((vblocks - 1) * a_rows + BM) * BK * 2 + EP_BYTES +
           table_bytes(kMaxSegments);
  }
  static constexpr bool fits(int vblocks);
};
constexpr size_t kAdapterSmem = kSmemMax - 4096;  // dynamic; the rest is for static tables
template <int BN, bool kSplit>
constexpr bool WideCfg<BN, kSplit>::fits(int vblocks) {
  return smem(BM, vblocks, stages(vblocks)) <= kAdapterSmem;
}
static_assert(WideCfg<256, false>::fits(2) && WideCfg<256, false>::fits(3) && WideCfg<128, false>::fits(2) &&
                  WideCfg<128, false>::fits(3) && WideCfg<64, false>::fits(3) && WideCfg<64, true>::fits(3),
              "shared memory budget exceeded");

struct WideCtl {
  unsigned long long full[kWideStagesMax], empty[kWideStagesMax], tfull[2], tempty[2], lfull[2], lempty[2], vfull, vempty, drain;
  uint32_t tmem_base;
  int abort_flag;
  int num_runs[2];
  uint32_t runs[2][2 * BM];  // of this tile and the next
};

template <int BN, bool kMN, bool kSplit>
__global__ void __launch_bounds__(kWideThreads, 1) adapter_wide_kernel(const __grid_constant__ CUtensorMap tmX,
                                                                       const __grid_constant__ CUtensorMap tmW,
                                                                       const __grid_constant__ CUtensorMap tmH,
                                                                       const __grid_constant__ CUtensorMap tmF,
                                                                       const __grid_constant__ CUtensorMap tmO,
                                                                       const WideParams p) {
  using C = WideCfg<BN, kSplit>;
  constexpr int CTAS = C::CTAS;
  // The narrow kernel of this call waited for everything before it and lets
  // this one start early; x, W and the request table are older than it, so only
  // hidden has to be waited for.
  if (!p.has_hidden) pdl_wait();
  extern __shared__ uint8_t smem_raw[];
  __shared__ WideCtl ctl;
  const uint32_t base = align1k(smem_u32(smem_raw));
  uint8_t* bytes = smem_raw + (base - smem_u32(smem_raw));
  const int a_bytes = kSplit ? p.a_rows * (BK * 2) : BM * BK * 2;
  const int nst = p.stages;
  const int stage_bytes = a_bytes + C::B_BYTES;
  const uint32_t sV = base + nst * stage_bytes;
  uint8_t* ep = bytes + (size_t)nst * stage_bytes + (hidden_blocks(p.r) - 1) * a_bytes + BM * BK * 2;
  int* off = reinterpret_cast<int*>(ep + C::EP_BYTES);
  int16_t* ad = reinterpret_cast<int16_t*>(off + p.q.num_seg + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int pair_rank = CTAS == 2 ? (int)cluster_rank() : 0;
  const bool leader = pair_rank == 0;
  constexpr int kTmem = kSplit ? BN : 2 * BN;
  // one warp sets the barriers up, one takes the tensor memory, the others read the request table
  if (warp == 0) {
    if (lane < nst) {
      mbar_init(smem_u32(&ctl.full[lane]), 1);
      mbar_init(smem_u32(&ctl.empty[lane]), 1);
    }
    if (lane < 2) {
      mbar_init(smem_u32(&ctl.tfull[lane]), 1);
      mbar_init(smem_u32(&ctl.tempty[lane]), 4 * CTAS);
      mbar_init(smem_u32(&ctl.lfull[lane]), 1);
      mbar_init(smem_u32(&ctl.lempty[lane]), leader ? 2 : 1);  // a pair's second CTA issues no MMAs
    }
    if (lane == 0) {
      mbar_init(smem_u32(&ctl.vfull), 1);
      mbar_init(smem_u32(&ctl.vempty), 1);
      mbar_init(smem_u32(&ctl.drain), 1);
      ctl.abort_flag = 0;
      prefetch_tmap(&tmX);
      prefetch_tmap(&tmW);
      prefetch_tmap(&tmH);
      prefetch_tmap(&tmF);
      if (!kSplit) prefetch_tmap(&tmO);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  } else if (warp == 1) {
    tmem_alloc_n<CTAS>(smem_u32(&ctl.tmem_base), kTmem);
  }
  load_requests(p.q, off, ad, p.status, 64);
  tc_fence_before();
  __syncthreads();
  if constexpr (CTAS == 2) cluster_sync();  // peer barriers initialised before any remote signal
  tc_fence_after();
  // With a narrow kernel before it the next kernel may start only once that one
  // has ended (below): what follows may then take hidden without waiting for this one.
  if (!p.has_hidden) pdl_trigger();
  const uint32_t tmem = ctl.tmem_base;
  const int nrank = kSplit ? (int)gridDim.x : 1, rank = kSplit ? (int)blockIdx.x : 0;
  const int nkb = p.red / BK;
  const int kb0 = kSplit ? (int)((long long)nkb * rank / nrank) : 0;
  const int kb1 = kSplit ? (int)((long long)nkb * (rank + 1) / nrank) : nkb;
  // Passes: 64 ranks of F at a time, with the blocks that hold hidden's three
  // parts of them.
  const int rp = plane_cols(p.r);
  const bool packed = parts_packed(p.r);
  const int passes = (p.r + 63) / 64;
  const int vblocks = hidden_blocks(p.r), vcol = packed ? 64 : rp;  // columns from one block to the next
  // A stage holds F's blocks of several runs: one in W's place, the others in in's
  // (a barrier wait and a commit a run cost about what its MMAs do).
  const int per_stage = 1 + a_bytes / C::B_BYTES;
  auto run_slot = [&](int j) { return j == 0 ? a_bytes : (j - 1) * C::B_BYTES; };

  struct Unit {
    int m0, n0, bn;  // the tile's first row (of the pair's 256) and column, its columns
  };
  constexpr int TM = BM * CTAS;
  auto unit_at = [&](int u) -> Unit {
    if (kSplit) return {(int)blockIdx.z * BM, (int)blockIdx.y * BN, BN};
    if (BN < 256 || u < p.full) return {u / p.n_tiles * TM, u % p.n_tiles * BN, BN};
    const int t = p.full + (u - p.full) / 2;
    return {t / p.n_tiles * TM, t % p.n_tiles * BN + ((u - p.full) & 1) * (BN / 2), BN / 2};
  };
  const int u0 = kSplit ? 0 : (int)blockIdx.x / CTAS, u1 = kSplit ? 1 : p.units, du = kSplit ? 1 : (int)gridDim.x / CTAS;
  // this CTA's (pair's) runs of a tile: every nrank-th
  const int r0 = rank, dr = nrank;
  const bool listed = p.q.num_seg > 0;
  auto at_leader = [&](uint32_t bar) { return CTAS == 2 ? map_to_rank(bar, 0) : bar; };

  if (warp == 0) {
    if (elect_one()) {
      int st = 0, local = 0;
      uint32_t ph = 0;
      bool ok = true;
      auto next = [&]() { if (++st == nst) { st = 0; ph ^= 1u; } };
      for (int u = u0; ok && u < u1; u += du, ++local) {
        const Unit t = unit_at(u);
        const int lb = local & 1;
        const uint32_t b_bytes = (uint32_t)t.bn / CTAS * BK * 2;
        const int row = t.m0 + pair_rank * BM, col = t.n0 + pair_rank * (t.bn / CTAS), nbox = t.bn / CTAS / C::WB;
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!(ok = wait_bar(smem_u32(&ctl.empty[st]), ph ^ 1u, &ctl.abort_flag, p.status))) break;
          const uint32_t fb = at_leader(smem_u32(&ctl.full[st])), sA = base + st * stage_bytes, sB = sA + a_bytes;
          if (leader) mbar_arrive_expect_tx(smem_u32(&ctl.full[st]), CTAS * (a_bytes + b_bytes));
          tma_load<CTAS>(sA, &tmX, fb, kb * BK, row);
          for (int h = 0; h < nbox; ++h) {
            if (kMN)
              tma_load_mn<CTAS>(sB + h * (C::WB * BK * 2), &tmW, fb, kb * BK, col / 64 + h * (C::WB / 64));
            else
              tma_load<CTAS>(sB + h * (C::WB * BK * 2), &tmW, fb, kb * BK, col + h * C::WB);
          }
          next();
        }
        if (!ok || !listed) continue;
        if (!(ok = wait_bar(smem_u32(&ctl.lfull[lb]), (local >> 1) & 1, &ctl.abort_flag, p.status))) break;
        const int n = ctl.num_runs[lb];
        for (int ps = 0; ok && ps < passes; ++ps) {
          const int c = ps * 64;  // F's columns (ranks) of this pass
          for (int i = r0; i < n; i += dr * per_stage) {
            if (!(ok = wait_bar(smem_u32(&ctl.empty[st]), ph ^ 1u, &ctl.abort_flag, p.status))) break;
            const int here = min(per_stage, (n - i + dr - 1) / dr);
            const uint32_t fb = at_leader(smem_u32(&ctl.full[st])), sA = base + st * stage_bytes;
            if (leader) mbar_arrive_expect_tx(smem_u32(&ctl.full[st]), CTAS * here * b_bytes);
            for (int j = 0; j < here; ++j) {
              const int a = unpack_run(ctl.runs[lb][i + j * dr]).a;
              const uint32_t sB = sA + run_slot(j);
              for (int h = 0; h < nbox; ++h) {
                if (kMN)
                  tma_load_4d<CTAS>(sB + h * (C::WB * BK * 2), &tmF, fb, 0, c, col / 64 + h * (C::WB / 64), a);
                else
                  tma_load<CTAS>(sB + h * (C::WB * BK * 2), &tmF, fb, c, a * p.f_rows + col + h * C::WB);
              }
            }
            next();
          }
        }
        mbar_arrive(smem_u32(&ctl.lempty[lb]));
      }
    }
  } else if (warp == 6) {
    if (p.has_hidden) {
      uint32_t ph = 0;
      int local = 0;
      bool ok = true, waited = false;
      for (int u = u0; ok && u < u1; u += du, ++local) {
        const Unit t = unit_at(u);
        const int lb = local & 1;
        ok = __all_sync(0xffffffffu, wait_bar(smem_u32(&ctl.lempty[lb]), ((local >> 1) & 1) ^ 1, &ctl.abort_flag, p.status));
        if (!ok) break;
        const int n = build_runs<4 * CTAS>(off, ad, p.q.num_seg, t.m0, min(p.q.T, t.m0 + TM), ctl.runs[lb]);
        if (lane == 0) {
          ctl.num_runs[lb] = n;
          mbar_arrive(smem_u32(&ctl.lfull[lb]));
        }
        if (!waited) {
          pdl_wait();
          pdl_trigger();
          waited = true;
        }
        if (lane == 0 && n > r0) {
          for (int ps = 0; ps < passes; ++ps, ph ^= 1u) {
            if (!(ok = wait_bar(smem_u32(&ctl.vempty), ph ^ 1u, &ctl.abort_flag, p.status))) break;
            const uint32_t fb = at_leader(smem_u32(&ctl.vfull));
            if (leader) mbar_arrive_expect_tx(smem_u32(&ctl.vfull), CTAS * vblocks * a_bytes);
            for (int v = 0; v < vblocks; ++v)
              tma_load<CTAS>(sV + v * a_bytes, &tmH, fb, v * vcol + ps * 64, t.m0 + pair_rank * BM);
          }
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
      }
      if (!waited) {  // the grid may not end before the narrow kernel does
        pdl_wait();
        pdl_trigger();
      }
    }
  } else if (warp == 1) {
    // a pair's second CTA only keeps its tensor memory
    if (leader && elect_one()) {
      int st = 0, local = 0;
      uint32_t ph = 0, vph = 0;
      bool ok = true;
      auto next = [&]() { if (++st == nst) { st = 0; ph ^= 1u; } };
      for (int u = u0; ok && u < u1; u += du, ++local) {
        const Unit t = unit_at(u);
        const uint32_t idesc = t.bn == BN ? p.idesc : p.idesc_half;
        const int buf = local & 1;
        if (!(ok = wait_bar(smem_u32(&ctl.tempty[buf]), ((local >> 1) & 1) ^ 1, &ctl.abort_flag, p.status))) break;
        tc_fence_after();
        const uint32_t d = tmem + buf * BN;
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!(ok = wait_bar(smem_u32(&ctl.full[st]), ph, &ctl.abort_flag, p.status))) break;
          tc_fence_after();
          const uint32_t a0 = base + st * stage_bytes, b0 = a0 + a_bytes;
#pragma unroll
          for (int kk = 0; kk < BK / 16; ++kk)
            mma_issue<CTAS>(d, sdesc(a0 + kk * 32, 16, 1024),
                            kMN ? sdesc(b0 + kk * 2048, CHUNK_BYTES, 1024) : sdesc(b0 + kk * 32, 16, 1024), idesc,
                            kb > kb0 || kk > 0);
          mma_commit_to<CTAS>(smem_u32(&ctl.empty[st]));
          next();
        }
        if (!ok) break;
        if (listed) {
          const int lb = local & 1;
          if (!(ok = wait_bar(smem_u32(&ctl.lfull[lb]), (local >> 1) & 1, &ctl.abort_flag, p.status))) break;
          const int n = ctl.num_runs[lb];
          for (int ps = 0; ok && n > r0 && ps < passes; ++ps, vph ^= 1u) {
            if (!(ok = wait_bar(smem_u32(&ctl.vfull), vph, &ctl.abort_flag, p.status))) break;
            const int steps = min(4, (p.r - ps * 64 + 15) / 16);  // 16-wide steps of this block of F
            // where the parts of hidden start, in the descriptors' 16-byte units
            const uint64_t vd = sdesc(sV, 16, 1024);
            const uint64_t vp[kPlanes] = {vd, vd + (uint64_t)((packed ? rp * 2 : a_bytes) >> 4),
                                          vd + (uint64_t)((packed ? (rp == 16 ? 64 : a_bytes) : 2 * a_bytes) >> 4)};
            for (int i = r0; i < n; i += dr * per_stage) {
              if (!(ok = wait_bar(smem_u32(&ctl.full[st]), ph, &ctl.abort_flag, p.status))) break;
              tc_fence_after();
              const int here = min(per_stage, (n - i + dr - 1) / dr);
              for (int j = 0; j < here; ++j) {
                const Run run = unpack_run(ctl.runs[lb][i + j * dr]);
                const LaneMask<CTAS> m = lane_mask<CTAS>(run.lo, run.hi);
                const uint32_t b0 = base + st * stage_bytes + run_slot(j);
                // (descriptors count 16-byte units: a step adds to their low word)
                const uint64_t bd = kMN ? sdesc(b0, CHUNK_BYTES, 1024) : sdesc(b0, 16, 1024);
#pragma unroll
                for (int kk = 0; kk < BK / 16; ++kk) {
                  if (kk >= steps) break;
#pragma unroll
                  for (int pl = 0; pl < kPlanes; ++pl)
                    mma_lanes(d, vp[pl] + (uint64_t)(kk * 2), bd + (uint64_t)(kk * (kMN ? 128 : 2)), idesc, 1u, m);
                }
              }
              mma_commit_to<CTAS>(smem_u32(&ctl.empty[st]));
              next();
            }
            if (ok) mma_commit_to<CTAS>(smem_u32(&ctl.vempty));
          }
          if (!ok) break;
          mbar_arrive(smem_u32(&ctl.lempty[lb]));
        }
        mma_commit_to<CTAS>(smem_u32(&ctl.tfull[buf]));
      }
      if (!ok) {  // drain MMAs still in flight before TMEM is released
        mma_commit_to<CTAS>(smem_u32(&ctl.drain));
        const unsigned long long t0 = globaltimer();
        while (!mbar_try_wait(smem_u32(&ctl.drain), 0) && globaltimer() - t0 < TIMEOUT_NS) {
        }
      }
    }
  } else if constexpr (kSplit) {
    // the slice's accumulator, column by column, over the ring (all of it consumed)
    const int q = warp & 3;
    float* acc = reinterpret_cast<float*>(bytes);  // [BN][BM]
    if (__all_sync(0xffffffffu, wait_bar(smem_u32(&ctl.tfull[0]), 0, &ctl.abort_flag, p.status)) && q * 32 < p.a_rows) {
      tc_fence_after();
      for (int c = 0; c < BN; c += 32) {
        uint32_t v[32];
        tmem_ld32(tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)c, v);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 32; ++i) acc[(c + i) * BM + q * 32 + lane] = f32(v[i]);
      }
    }
  } else {
    const int q = warp & 3;
    EpRing<EP_SLOTS> ring{ep + (size_t)(warp - 2) * EP_SLOTS * EP_BOX_BYTES, 0, lane};
    const uint32_t tempty[2] = {at_leader(smem_u32(&ctl.tempty[0])), at_leader(smem_u32(&ctl.tempty[1]))};
    int local = 0;
    for (int u = u0; u < u1; u += du, ++local) {
      const Unit t = unit_at(u);
      const int rb = t.m0 + pair_rank * BM + q * 32;
      const int buf = local & 1;
      if (!__all_sync(0xffffffffu, wait_bar(smem_u32(&ctl.tfull[buf]), (local >> 1) & 1, &ctl.abort_flag, p.status))) break;
      tc_fence_after();
      if (rb < p.q.T) {
        for (int c = 0; c < t.bn; c += 32) {
          uint32_t v[32];
          tmem_ld32(tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(buf * BN + c), v);
          tmem_wait_ld();
          uint8_t* box = ring.acquire();
#pragma unroll
          for (int i = 0; i < 4; ++i)
            ring.put(box, i, make_uint4(pack_bf16x2(f32(v[8 * i]), f32(v[8 * i + 1])), pack_bf16x2(f32(v[8 * i + 2]), f32(v[8 * i + 3])),
                                        pack_bf16x2(f32(v[8 * i + 4]), f32(v[8 * i + 5])), pack_bf16x2(f32(v[8 * i + 6]), f32(v[8 * i + 7]))));
          ring.issue(box, &tmO, t.n0 + c, rb);  // rows past the last token are clipped by the map
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (CTAS == 1)
          mbar_arrive(tempty[buf]);
        else
          asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(tempty[buf]) : "memory");
      }
    }
    ring.drain();
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (CTAS == 2) cluster_sync();  // neither CTA frees tensor memory while the pair still uses it
  tc_fence_after();
  if (warp == 1) tmem_dealloc_n<CTAS>(tmem, kTmem);
  if constexpr (kSplit) {
    cluster_sync();
    // this CTA's share of the columns: the slices' sums in order
    const int m0 = blockIdx.z * BM, per = BN / nrank;
    const int rows = min(p.a_rows, p.q.T - m0);
    const uint32_t local = base;
    for (int i = threadIdx.x; i < rows * (per / 8); i += kWideThreads) {
      const int row = i % rows, c = rank * per + i / rows * 8;
      float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      for (int k = 0; k < nrank; ++k) {
        const uint32_t peer = map_to_rank(local + (uint32_t)(c * BM + row) * 4, k);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] += ld_cluster(peer + j * BM * 4);
      }
      *reinterpret_cast<uint4*>(p.out + (size_t)(m0 + row) * p.ldo + (int)blockIdx.y * BN + c) = pack8(v);
    }
    cluster_sync();  // a peer may still read this CTA's accumulator
  }
}

// ------------------------------------------------------- adapters' gradients
//
// dA_a^T [K, r] = sum over a's rows of x^T u, dB_a [N, r] = sum of dy^T v: a
// tile is 128 rows of the output (columns of x or dy) times the hidden columns
// of all parts, over at most part_rows of the adapter's rows; the parts'
// products are added in the epilogue.  An adapter's rows are those of all its
// requests in order, neighbouring ones as one run.  A run's last block may reach into the next request's
// rows: those are overwritten with zeros in shared memory.
//
// Bound by reading x and dy once, 67 MB at 8192 x (2048 + 2048): 17 us, 3.9 TB/s
// (tensor cores 9% busy; a CTA's ring waits for its loads).  Parts of 512 rows:
// fewer leave more sums to add up, more leave SMs idle (128, 256 and 384 rows
// were slower).  All three parts of u and v are taken: with two the gradients
// were further from the exact ones than with products of fp32 tensors.
struct GradParams {
  Reqs q;
  int K, N, r;
  int part_rows;
  int tiles_a, tiles_b;   // 128-row tiles of dA^T and of dB
  float* dA;              // [num_adapters, r, K]
  float* dB;              // [num_adapters, N, r]
  float* part;            // [parts][r K + N r]
  int accumulate;
  uint32_t idesc;
  int stages;
  int* status;
};

constexpr int kGradStagesMax = 6;
// two accumulators up to 96 hidden columns, one beyond
__host__ __device__ constexpr uint32_t grad_tmem_cols(int r) {
  const int hc = hidden_cols(r);
  return hc <= 64 ? 128 : (hc <= 192 ? 256 : 512);
}
struct GradCtl {
  unsigned long long full[kGradStagesMax], empty[kGradStagesMax], tfull[2], tempty[2], drain;
  uint32_t tmem_base;
  int abort_flag;
};

// Sums of a warp's values over all adapters, 32 at a time: v[a] becomes f(v[a]),
// f(0) + ... + f(v[a]) or the sum before it; returns the whole.
template <bool kBefore, class F>
__device__ __forceinline__ int scan_adapters(int n, const int* v, int* out, F&& f) {
  const int lane = threadIdx.x & 31;
  int carry = 0;
  for (int b = 0; b < n; b += 32) {
    const int a = b + lane, x = a < n ? f(v[a]) : 0;
    int m = x;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, m, d);
      if (lane >= d) m += o;
    }
    if (a < n) out[a] = carry + m - (kBefore ? x : 0);
    carry += __shfl_sync(0xffffffffu, m, 31);
  }
  return carry;
}

// Shared-memory tables (all threads call it): the rows of each adapter and from
// them its first part, first[num_adapters] all parts.
// kRuns: also its rows as runs, requests that follow one another with one adapter
// taken together: list[begin[a]..begin[a + 1]) are a's, in row order, each its
// first request and the one past its last (walking all requests for each tile made
// the kernel's time grow with their number: 1000 requests over 48 adapters 637 us,
// 345 with the runs).  They are counted, then placed from the last request back,
// where the end of each is known.
template <bool kRuns>
__device__ __forceinline__ void load_parts(const Reqs& q, const int* off, const int16_t* ad, int part_rows, int* rows, int* first,
                                           int* begin = nullptr, uint32_t* list = nullptr) {
  for (int a = threadIdx.x; a < q.num_adapters; a += blockDim.x) {
    rows[a] = 0;
    if (kRuns) begin[a] = 0;
  }
  __syncthreads();
  for (int s = threadIdx.x; s < q.num_seg; s += blockDim.x) {
    const int a = ad[s];
    if (a < 0) continue;
    if (off[s + 1] > off[s]) atomicAdd(&rows[a], off[s + 1] - off[s]);
    if (kRuns && (s == 0 || ad[s - 1] != a)) atomicAdd(&begin[a], 1);
  }
  __syncthreads();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp == 0) {
    const int parts = scan_adapters<true>(q.num_adapters, rows, first, [&](int n) { return (n + part_rows - 1) / part_rows; });
    if (lane == 0) first[q.num_adapters] = parts;
  }
  if (kRuns && warp == 2) {
    const int runs = scan_adapters<false>(q.num_adapters, begin, begin, [](int n) { return n; });  // where they end
    if (lane == 0) begin[q.num_adapters] = runs;
    __syncwarp();
    int after = q.num_seg;  // the next request with another adapter
    for (int b = (q.num_seg - 1) / 32 * 32; b >= 0; b -= 32) {
      const int s = b + lane, a = s < q.num_seg ? ad[s] : -1;
      const unsigned other = __ballot_sync(0xffffffffu, s < q.num_seg && (s == 0 || ad[s - 1] != a));
      const bool start = ((other >> lane) & 1u) && a >= 0;
      const unsigned above = lane == 31 ? 0u : 0xffffffffu << (lane + 1), later = other & above;
      const unsigned peers = __match_any_sync(0xffffffffu, start ? a : -1 - lane);
      if (start)
        list[begin[a] - 1 - __popc(peers & above)] = (uint32_t)s | (uint32_t)(later ? b + __ffs(later) - 1 : after) << 16;
      __syncwarp();
      if (start && (peers & ((1u << lane) - 1u)) == 0) begin[a] -= __popc(peers);
      __syncwarp();
      if (other) after = b + __ffs(other) - 1;
    }
  }
  __syncthreads();
}

// f(first row, valid rows <= 64) -> bool for the blocks of part `part` of the adapter with runs [i0, i1).
template <class F>
__device__ __forceinline__ void for_each_block(const int* off, const uint32_t* list, int i0, int i1, int part, int part_rows, F&& f) {
  const long long lo = (long long)part * part_rows, hi = lo + part_rows;
  long long at = 0;  // adapter rows before this run
  for (int i = i0; i < i1 && at < hi; ++i) {
    const uint32_t run = list[i];
    const int first = off[run & 0xffffu], n = off[run >> 16] - first;
    const int b = (int)max(lo - at, 0ll), e = (int)min(hi - at, (long long)n);
    for (int t = b; t < e; t += BK)
      if (!f(first + t, min(BK, e - t))) return;
    at += n;
  }
}

__device__ __forceinline__ int adapter_of_part(const int* first, int num_adapters, int part) {
  int lo = 0, hi = num_adapters - 1;  // last a with first[a] <= part
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (first[mid] <= part) lo = mid; else hi = mid - 1;
  }
  return lo;
}

__global__ void __launch_bounds__(192) adapter_grad_kernel(const __grid_constant__ CUtensorMap tmX,
                                                           const __grid_constant__ CUtensorMap tmU,
                                                           const __grid_constant__ CUtensorMap tmDy,
                                                           const __grid_constant__ CUtensorMap tmV,
                                                           const GradParams p) {
  // The wide kernel before this one lets it start once u is there, and neither
  // needs the other: this one fills the SMs that the other's last tiles leave.
  extern __shared__ uint8_t smem_raw[];
  __shared__ GradCtl ctl;
  const uint32_t base = align1k(smem_u32(smem_raw));
  uint8_t* bytes = smem_raw + (base - smem_u32(smem_raw));
  const int hc = hidden_cols(p.r), rp = plane_cols(p.r);
  const int nck = hidden_pitch(p.r) / 64;            // 64-column chunks of hidden
  const int nmma = hc > 256 ? 2 : 1;                 // MMAs (column halves) of a step
  const int stage_bytes = BM * BK * 2 + nck * CHUNK_BYTES;
  int* off = reinterpret_cast<int*>(bytes + (size_t)p.stages * stage_bytes);
  int16_t* ad = reinterpret_cast<int16_t*>(off + p.q.num_seg + 1);
  int* rows = reinterpret_cast<int*>(ad + (p.q.num_seg + 1) / 2 * 2);
  int* first = rows + p.q.num_adapters;
  int* begin = first + p.q.num_adapters + 1;
  uint32_t* runs = reinterpret_cast<uint32_t*>(begin + p.q.num_adapters + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int bufs = hc <= 96 ? 2 : 1;
  const uint32_t cols = grad_tmem_cols(p.r);
  if (threadIdx.x == 160) {
    for (int i = 0; i < p.stages; ++i) {
      mbar_init(smem_u32(&ctl.full[i]), 1);
      mbar_init(smem_u32(&ctl.empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&ctl.tfull[i]), 1);
      mbar_init(smem_u32(&ctl.tempty[i]), 4);
    }
    mbar_init(smem_u32(&ctl.drain), 1);
    ctl.abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    prefetch_tmap(&tmX);
    prefetch_tmap(&tmU);
    prefetch_tmap(&tmDy);
    prefetch_tmap(&tmV);
  }
  if (warp == 1) tmem_alloc_n<1>(smem_u32(&ctl.tmem_base), cols);
  load_requests(p.q, off, ad, p.status);
  load_parts<true>(p.q, off, ad, p.part_rows, rows, first, begin, runs);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_trigger();
  const uint32_t tmem = ctl.tmem_base;
  const int per = p.tiles_a + p.tiles_b;
  const long long items = (long long)first[p.q.num_adapters] * per;

  if (warp == 0) {
    if (lane == 0) {
      int st = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (long long it = blockIdx.x; ok && it < items; it += gridDim.x) {
        const int part = (int)(it / per), mt = (int)(it % per);
        const int a = adapter_of_part(first, p.q.num_adapters, part);
        const bool is_a = mt < p.tiles_a;
        const CUtensorMap* ml = is_a ? &tmX : &tmDy;
        const CUtensorMap* mr = is_a ? &tmU : &tmV;
        const int ck = (is_a ? mt : mt - p.tiles_a) * 2;
        for_each_block(off, runs, begin[a], begin[a + 1], part - first[a], p.part_rows, [&](int row, int) {
          if (!(ok = wait_bar(smem_u32(&ctl.empty[st]), ph ^ 1u, &ctl.abort_flag, p.status))) return false;
          const uint32_t fb = smem_u32(&ctl.full[st]), sA = base + st * stage_bytes;
          mbar_arrive_expect_tx(fb, stage_bytes);
          tma_load_3d(sA, ml, fb, 0, row, ck);
          tma_load_3d(sA + BM * BK * 2, mr, fb, 0, row, 0);
          if (++st == p.stages) { st = 0; ph ^= 1u; }
          return true;
        });
      }
    }
  } else if (warp == 1) {
    int st = 0, local = 0;
    uint32_t ph = 0;
    bool ok = true;
    for (long long it = blockIdx.x; ok && it < items; it += gridDim.x, ++local) {
      const int part = (int)(it / per);
      const int a = adapter_of_part(first, p.q.num_adapters, part);
      const int buf = local % bufs, use = local / bufs;
      ok = __all_sync(0xffffffffu, wait_bar(smem_u32(&ctl.tempty[buf]), (use & 1) ^ 1, &ctl.abort_flag, p.status));
      if (!ok) break;
      tc_fence_after();
      const uint32_t d = tmem + buf * (cols / bufs);
      uint32_t started = 0;
      for_each_block(off, runs, begin[a], begin[a + 1], part - first[a], p.part_rows, [&](int, int valid) {
        ok = __all_sync(0xffffffffu, wait_bar(smem_u32(&ctl.full[st]), ph, &ctl.abort_flag, p.status));
        if (!ok) return false;
        const int steps = (valid + 15) / 16;
        const uint32_t a0 = base + st * stage_bytes, b0 = a0 + BM * BK * 2;
        if (valid & 15) {  // rows of the last step past the run: zeros in both operands
          uint8_t* blk = bytes + (size_t)st * stage_bytes;
          const int nz = (steps * 16 - valid) * 8;
          for (int c = 0; c < 2 + nck; ++c)
            for (int i = lane; i < nz; i += 32)
              *reinterpret_cast<uint4*>(blk + c * CHUNK_BYTES + valid * 128 + i * 16) = make_uint4(0, 0, 0, 0);
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
        }
        tc_fence_after();
        if (elect_one()) {
          for (int kk = 0; kk < steps; ++kk) {
            for (int h = 0; h < nmma; ++h)
              mma_bf16(d + h * (hc / 2), sdesc(a0 + kk * 2048, CHUNK_BYTES, 1024),
                       sdesc(b0 + h * (nck / 2 * CHUNK_BYTES) + kk * 2048, CHUNK_BYTES, 1024), p.idesc,
                       started || kk > 0);
          }
          mma_commit(smem_u32(&ctl.empty[st]));
        }
        started = 1;
        __syncwarp();
        if (++st == p.stages) { st = 0; ph ^= 1u; }
        return true;
      });
      if (!ok) break;
      if (elect_one()) mma_commit(smem_u32(&ctl.tfull[buf]));
      __syncwarp();
    }
    if (!ok) {
      if (lane == 0) mma_commit(smem_u32(&ctl.drain));
      __syncwarp();
      const unsigned long long t0 = globaltimer();
      while (!mbar_try_wait(smem_u32(&ctl.drain), 0) && globaltimer() - t0 < TIMEOUT_NS) {
      }
    }
  } else {
    const int q = warp & 3;
    int local = 0;
    const size_t part_sz = (size_t)p.r * (p.K + p.N);
    for (long long it = blockIdx.x; it < items; it += gridDim.x, ++local) {
      const int part = (int)(it / per), mt = (int)(it % per);
      const int a = adapter_of_part(first, p.q.num_adapters, part);
      const bool is_a = mt < p.tiles_a;
      const int m = (is_a ? mt : mt - p.tiles_a) * BM + q * 32 + lane;
      const bool direct = first[a + 1] - first[a] == 1 && !p.accumulate;
      const int buf = local % bufs, use = local / bufs;
      if (!__all_sync(0xffffffffu, wait_bar(smem_u32(&ctl.tfull[buf]), use & 1, &ctl.abort_flag, p.status))) break;
      tc_fence_after();
      const uint32_t d = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(buf * (cols / bufs));
      float* dst;
      if (is_a)
        dst = (direct ? p.dA + (size_t)a * p.r * p.K : p.part + (size_t)part * part_sz) + m;
      else
        dst = (direct ? p.dB + (size_t)a * p.N * p.r : p.part + (size_t)part * part_sz + (size_t)p.r * p.K) + (size_t)m * p.r;
      for (int c = 0; c < p.r; c += 8) {
        float s[8];
#pragma unroll
        for (int pl = 0; pl < kPlanes; ++pl) {
          uint32_t v[8];
          asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                       : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                       : "r"(d + (uint32_t)(pl * rp + c)));
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 8; ++i) s[i] = pl == 0 ? f32(v[i]) : s[i] + f32(v[i]);
        }
        if (is_a) {
          if (m < p.K) {
#pragma unroll
            for (int i = 0; i < 8; ++i) dst[(size_t)(c + i) * p.K] = s[i];
          }
        } else if (m < p.N) {
          *reinterpret_cast<float4*>(dst + c) = make_float4(s[0], s[1], s[2], s[3]);
          *reinterpret_cast<float4*>(dst + c + 4) = make_float4(s[4], s[5], s[6], s[7]);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&ctl.tempty[buf]));
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc_n<1>(tmem, cols);
  pdl_wait();  // this grid may not end before the wide kernel does
}

// dA, dB of the adapters whose rows were not one part: the parts' sums in
// order, zero for an adapter without rows, added to the old values when
// accumulating.
__global__ void __launch_bounds__(256) adapter_grad_sum_kernel(const GradParams p) {
  extern __shared__ int tab[];
  int* off = tab;
  int16_t* ad = reinterpret_cast<int16_t*>(off + p.q.num_seg + 1);
  int* rows = reinterpret_cast<int*>(ad + (p.q.num_seg + 1) / 2 * 2);
  int* first = rows + p.q.num_adapters;
  load_requests(p.q, off, ad, p.status);
  load_parts<false>(p.q, off, ad, p.part_rows, rows, first);
  pdl_wait();  // (the request table is older than the call's first kernel, which waited for it)
  pdl_trigger();
  const int a = blockIdx.y;
  const int n = first[a + 1] - first[a];
  if (n == 1 && !p.accumulate) return;
  const size_t na = (size_t)p.r * p.K, sz = na + (size_t)p.r * p.N;
  const float4* src = reinterpret_cast<const float4*>(p.part + (size_t)first[a] * sz);
  for (size_t i = blockIdx.x * (size_t)blockDim.x + threadIdx.x; i < sz / 4; i += (size_t)gridDim.x * blockDim.x) {
    float4* dst = reinterpret_cast<float4*>(4 * i < na ? p.dA + (size_t)a * na + 4 * i : p.dB + (size_t)a * (sz - na) + (4 * i - na));
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int k = 0; k < n; ++k) {
      const float4 w = __ldcg(src + (size_t)k * (sz / 4) + i);
      v = make_float4(v.x + w.x, v.y + w.y, v.z + w.z, v.w + w.w);
    }
    if (p.accumulate) {
      const float4 o = *dst;
      v = make_float4(o.x + v.x, o.y + v.y, o.z + v.z, o.w + v.w);
    }
    *dst = v;
  }
}

// --------------------------------------------------------------- host side

// bf16 map of rank <= 4: dims and box innermost first, pitches (elements) of dims 1..
int make_map(CUtensorMap* m, const void* ptr, int rank, const uint64_t* dims, const uint64_t* pitch, const uint32_t* box,
             CUtensorMapSwizzle swz = CU_TENSOR_MAP_SWIZZLE_128B) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return fail(MOE_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
  cuuint64_t d[4], s[3];
  cuuint32_t b[4], es[4] = {1, 1, 1, 1};
  for (int i = 0; i < rank; ++i) {
    d[i] = dims[i] > 0 ? dims[i] : 1;
    b[i] = box[i];
    if (i > 0) s[i - 1] = pitch[i - 1] * 2;
  }
  const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(ptr), d, s, b, es,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, swz, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS)
    return fail(MOE_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d) for an adapter operand of %llu columns", (int)r, (unsigned long long)dims[0]);
  return MOE_OK;
}
int map2(CUtensorMap* m, const void* ptr, uint64_t inner, uint64_t outer, uint64_t pitch, uint32_t bi, uint32_t bo,
         CUtensorMapSwizzle swz = CU_TENSOR_MAP_SWIZZLE_128B) {
  const uint64_t d[2] = {inner, outer}, s[1] = {pitch};
  const uint32_t b[2] = {bi, bo};
  return make_map(m, ptr, 2, d, s, b, swz);
}
// MN-major operand: [rows, cols] as {64 columns, rows, chunks of 64 columns}
int map_mn(CUtensorMap* m, const void* ptr, uint64_t cols, uint64_t rows, uint64_t pitch, uint32_t chunks) {
  const uint64_t d[3] = {cols < 64 ? cols : 64, rows, (cols + 63) / 64}, s[2] = {pitch, 64};
  const uint32_t b[3] = {64, 64, chunks};
  return make_map(m, ptr, 3, d, s, b);
}

int set_smem(const void* kern, bool* done, const char* fn, size_t most = kAdapterSmem) {
  const int dev = current_device();
  if (dev < 0) return fail(MOE_ERR_CUDA, "%s: no current CUDA device", fn);
  if (done[dev]) return MOE_OK;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
  if (e != cudaSuccess) return fail_cuda(fn, e);
  done[dev] = true;
  return MOE_OK;
}

template <typename... KArgs, typename... Args>
int launch_adapter(const char* fn, void (*kern)(KArgs...), dim3 grid, int threads, size_t smem, int cluster_x,
                   cudaStream_t s, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = threads;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cluster_x;
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cluster_x > 0 ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...);
  if (e != cudaSuccess) return fail_cuda(fn, e);
  return check_launch(fn);
}

// hidden = parts of scale F . in.  kMN false: F = A [nA, r, red]; true: F = B^T, B [nA, red, r].
template <bool kMN>
int run_shrink(const char* fn, const Reqs& q, const void* in, long long ld, const void* F, const float* scale, int red, int r,
               void* hidden, cudaStream_t s) {
  static bool attr[64] = {};
  auto kern = adapter_shrink_kernel<kMN>;
  if (int rc = set_smem(reinterpret_cast<const void*>(kern), attr, fn)) return rc;
  const int tiles = (q.T + BM - 1) / BM, nkb = red / BK, sms = sm_count() > 0 ? sm_count() : 148;
  const int rN = round_up(r, 16), f_bytes = kMN ? (r + 63) / 64 * CHUNK_BYTES : r * 128;
  // as many slices as run at a time: two CTAs an SM where both fit (r = 64, of which one fits, with slices
  // for two: 159 us instead of 150 for 8192 x 2048 x 2048 in both directions, 113.5 instead of 107.6 for
  // the forward of 16384 x 2048 x 2048)
  const int least = 1024 + 2 * kShrinkXBytes + rN * BM * 4 + (int)table_bytes(q.num_seg) + 2 * kShrinkK * f_bytes;
  const bool two = least <= 110 * 1024;
  int cs = 1;
  while (cs < 8 && cs * 2 <= nkb && tiles * cs * 2 <= (two ? 2 : 1) * sms) cs *= 2;
  CUtensorMap tx, tf;
  if (int rc = map2(&tx, in, red, q.T, ld, BK, BM)) return rc;
  if (kMN) {
    if (int rc = map2(&tf, F, r, (uint64_t)q.num_adapters * red, r, 64, 64)) return rc;
  } else {
    if (int rc = map2(&tf, F, red, (uint64_t)q.num_adapters * r, red, BK, r)) return rc;
  }
  ShrinkParams p{};
  p.q = q;
  p.red = red;
  p.nrank = cs;
  p.r = r;
  p.rN = rN;
  p.f_bytes = f_bytes;
  p.f_rows = kMN ? red : r;
  // Tiles of many runs want many blocks of F in flight: as many as fit where a CTA has its SM alone.
  // Otherwise two CTAs share one, with two steps of x in flight each (three: one CTA an SM; 18 us instead
  // of 13 for 8192 x 2048).
  const bool alone = !two || tiles * cs <= sms;
  // more runs than rows of tiles: several share a step of F, its barrier wait and its commit
  p.f_runs = q.num_seg <= 2 * tiles ? 1 : (kShrinkK * p.f_bytes <= 8192 ? 4 : (kShrinkK * p.f_bytes <= 16384 ? 2 : 1));
  const int f_stage = p.f_runs * kShrinkK * p.f_bytes;
  const int steps = ((nkb + cs - 1) / cs + kShrinkK - 1) / kShrinkK;
  p.x_stages = r <= 64 && alone ? kShrinkX : 2;
  if (steps < p.x_stages) p.x_stages = steps;
  const int fixed = 1024 + p.x_stages * kShrinkXBytes + p.rN * BM * 4 + (int)table_bytes(q.num_seg);
  const int f_room = alone ? (int)kAdapterSmem - fixed : 8192;
  p.f_stages = f_room / f_stage < 2 ? 2 : (f_room / f_stage > kShrinkF ? kShrinkF : f_room / f_stage);
  p.scale = scale;
  p.hidden = static_cast<__nv_bfloat16*>(hidden);
  p.idesc = make_idesc(p.rN, BM, false, kMN);
  p.tmem_cols = p.rN <= 32 ? 32 : (p.rN <= 64 ? 64 : 128);
  p.status = status_word();
  // (an F block of r rows is read as rN: the last one reads into the sums, whose columns past r are not used)
  const size_t smem = (size_t)fixed + (size_t)p.f_stages * f_stage;
  return launch_adapter(fn, kern, dim3(cs * tiles), 192, smem, cs, s, tx, tf, p);
}

template <int BN, bool kMN, bool kSplit>
int run_wide_bn(const char* fn, const Reqs& q, const void* in, long long ld, const void* W, const void* hidden, const void* F,
                int red, int out_cols, int r, void* out, long long ldo, bool has_hidden, int nrank, cudaStream_t s) {
  using C = WideCfg<BN, kSplit>;
  static bool attr[64] = {};
  auto kern = adapter_wide_kernel<BN, kMN, kSplit>;
  if (int rc = set_smem(reinterpret_cast<const void*>(kern), attr, fn)) return rc;
  const int sms = sm_count();
  if (sms <= 0) return fail(MOE_ERR_CUDA, "%s: cannot query the SM count", fn);
  WideParams p{};
  p.a_rows = kSplit && q.T < BM ? round_up(q.T, 8) : BM;
  CUtensorMap tx, tw, th, tf, to;
  if (int rc = map2(&tx, in, red, q.T, ld, BK, p.a_rows)) return rc;
  const int hp = hidden_pitch(r);
  if (kMN) {
    if (int rc = map_mn(&tw, W, out_cols, red, out_cols, C::WB / 64)) return rc;
  } else {
    if (int rc = map2(&tw, W, red, out_cols, red, BK, C::WB)) return rc;
  }
  th = tx;
  tf = tw;
  if (has_hidden) {
    if (int rc = map2(&th, hidden, hp, q.T, hp, 64, p.a_rows)) return rc;
    if (kMN) {
      const uint64_t d[4] = {64, (uint64_t)r, (uint64_t)out_cols / 64, (uint64_t)q.num_adapters};
      const uint64_t pt[3] = {(uint64_t)out_cols, 64, (uint64_t)r * out_cols};
      const uint32_t b[4] = {64, 64, C::WB / 64, 1};
      if (int rc = make_map(&tf, F, 4, d, pt, b)) return rc;
    } else {
      if (int rc = map2(&tf, F, r, (uint64_t)q.num_adapters * out_cols, r, 64, C::WB)) return rc;
    }
  }
  to = tx;
  if (!kSplit)
    if (int rc = map2(&to, out, out_cols, q.T, ldo, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B)) return rc;
  p.q = q;
  p.red = red;
  p.r = r;
  p.f_rows = out_cols;
  p.n_tiles = out_cols / BN;
  const int tm = BM * C::CTAS, rows = (q.T + tm - 1) / tm, tiles = rows * p.n_tiles, places = sms / C::CTAS;
  const int rest = BN == 256 ? tiles % places : 0;
  p.full = rest > 0 && 2 * rest <= places ? tiles - rest : tiles;
  p.units = p.full + 2 * (tiles - p.full);
  p.has_hidden = has_hidden;
  p.idesc = make_idesc(BN, tm, false, kMN);
  p.idesc_half = make_idesc(BN / 2, tm, false, kMN);
  p.out = static_cast<__nv_bfloat16*>(out);
  p.ldo = ldo;
  p.status = status_word();
  const int vblocks = hidden_blocks(r);
  p.stages = C::stages(vblocks);
  if (kSplit) {
    // a slice's blocks all in flight where they fit; four hold the accumulator afterwards
    while (p.stages < kWideStagesMax && C::smem(p.a_rows, vblocks, p.stages + 1) <= kAdapterSmem) ++p.stages;
    return launch_adapter(fn, kern, dim3(nrank, p.n_tiles, rows), kWideThreads, C::smem(p.a_rows, vblocks, p.stages), nrank, s, tx,
                          tw, th, tf, to, p);
  }
  return launch_adapter(fn, kern, dim3((p.units < places ? p.units : places) * C::CTAS), kWideThreads, C::smem(BM, vblocks, p.stages),
                        C::CTAS == 2 ? 2 : 0, s, tx, tw, th, tf,
                        to, p);
}

template <bool kMN>
int run_wide(const char* fn, const Reqs& q, const void* in, long long ld, const void* W, const void* hidden, const void* F,
             int red, int out_cols, int r, void* out, long long ldo, bool has_hidden, cudaStream_t s) {
  const int sms = sm_count() > 0 ? sm_count() : 148, rows = (q.T + BM - 1) / BM;
  // where even the narrowest tiles leave half of the SMs idle: clusters along the reduction
  const int tiles = rows * (out_cols / 64);
  int nrank = 1;
  while (nrank < 8 && nrank * 2 <= red / BK && tiles * nrank * 2 <= sms) nrank *= 2;
  if (nrank > 1)
    return run_wide_bn<64, kMN, true>(fn, q, in, ld, W, hidden, F, red, out_cols, r, out, ldo, has_hidden, nrank, s);
  // else the tile whose waves cost least: a block's time goes with the columns it multiplies plus half of
  // the 128 rows it loads; a pair's last wave may be one of halves, which cost what a 128-column tile does
  // (forward, narrow product included: 517 rows of 40 requests, 768 x 2048, r = 16: 18.5 us on 128 columns,
  // 20.6 on halves of 256, 18.0 on 64 with four times the loads; r = 64: 26.8, 27.6, 24.2, since the
  // adapters' MMAs, which the rule does not count, weigh more; 8192 rows, 2048 x 2048, r = 16: 50.5 on 256
  // and a wave of halves, 64.1 on 128, 102 on 64)
  int best = (tiles + sms - 1) / sms * (64 + 64), bn = 64;
  if (out_cols % 128 == 0) {
    const int w128 = (tiles / 2 + sms - 1) / sms * (128 + 64);
    if (w128 <= best) best = w128, bn = 128;
  }
  if (out_cols % 256 == 0) {
    const int places = sms / 2, t256 = (q.T + 2 * BM - 1) / (2 * BM) * (out_cols / 256), rest = t256 % places;
    const int w256 = t256 / places * (256 + 64) + (rest == 0 ? 0 : (2 * rest <= places ? 128 + 64 : 256 + 64));
    if (w256 < best) bn = 256;
  }
  if (bn == 256)
    return run_wide_bn<256, kMN, false>(fn, q, in, ld, W, hidden, F, red, out_cols, r, out, ldo, has_hidden, 1, s);
  if (bn == 128)
    return run_wide_bn<128, kMN, false>(fn, q, in, ld, W, hidden, F, red, out_cols, r, out, ldo, has_hidden, 1, s);
  return run_wide_bn<64, kMN, false>(fn, q, in, ld, W, hidden, F, red, out_cols, r, out, ldo, has_hidden, 1, s);
}

// v of requests of a row or a few.
int run_gemv(const char* fn, const Reqs& q, const void* x, long long ldx, const void* A, const float* scale, int K, int r,
             void* hidden, cudaStream_t s) {
  const GemvParams p{q, static_cast<const __nv_bfloat16*>(x), ldx, static_cast<const __nv_bfloat16*>(A), scale, K, r,
                     static_cast<__nv_bfloat16*>(hidden), status_word()};
  const dim3 grid(q.T, (plane_cols(r) + kGemvWarps * kGemvRanks - 1) / (kGemvWarps * kGemvRanks));
  return launch_adapter(fn, adapter_gemv_kernel, grid, kGemvWarps * 32, table_bytes(q.num_seg), 0, s, p);
}

int check_adapter(const char* fn, const Reqs& q, int K, int N, int r, long long ldx, long long ldy) {
  if (q.T < 0 || K <= 0 || N <= 0 || r <= 0 || q.num_adapters <= 0 || q.num_seg < 0)
    return fail(MOE_ERR_INVALID_ARG, "%s: need T>=0, K>0, N>0, r>0, num_adapters>0, num_seg>=0", fn);
  if (K % 64 || N % 64 || r % 8 || r > kMaxRank || q.num_adapters > kMaxAdapters || q.num_seg > kMaxSegments ||
      (long long)q.num_adapters * (N > r ? N : r) >= (1ll << 31))
    return fail(MOE_ERR_UNSUPPORTED_SHAPE,
                "%s: need K%%64==0, N%%64==0, r%%8==0, r<=%d, num_adapters<=%d, num_seg<=%d (K=%d N=%d r=%d)", fn, kMaxRank,
                kMaxAdapters, kMaxSegments, K, N, r);
  if (ldx < K || ldy < N || ldx % 8 || ldy % 8 || ldx >= (1ll << 31) || ldy >= (1ll << 31))
    return fail(MOE_ERR_UNSUPPORTED_SHAPE, "%s: row strides must be multiples of 8 and at least the row length", fn);
  if (q.num_seg > 0 && (!q.offsets || !q.adapter)) return fail(MOE_ERR_INVALID_ARG, "%s: NULL request table", fn);
  return MOE_OK;
}

size_t align256(size_t b) { return (b + 255) & ~size_t(255); }

// Rows of one part of an adapter's gradient sum (see adapter_grad_kernel).
constexpr int kPartRows = 512;

struct BwdLayout {
  size_t u, part, total;
};
BwdLayout bwd_layout(int T, int K, int N, int r, int num_seg) {
  BwdLayout L;
  // an adapter's last part may be short: at most one a request more than whole parts
  const size_t parts = (size_t)T / kPartRows + (size_t)num_seg;
  size_t at = 0;
  L.u = at; at += align256((size_t)T * hidden_pitch(r) * 2);
  L.part = at; at += align256(parts * r * (size_t)(K + N) * sizeof(float));
  L.total = at > 256 ? at : 256;
  return L;
}

}  // namespace
}  // namespace tc
}  // namespace moe

using namespace moe;
using namespace moe::tc;

extern "C" {

size_t moe_adapter_hidden_size(int T, int r) {
  if (T < 0 || r <= 0 || r > kMaxRank) return 0;
  const size_t n = align256((size_t)T * hidden_pitch(r) * 2);
  return n > 0 ? n : 256;
}

size_t moe_adapter_linear_bwd_workspace_size(int T, int K, int N, int r, int num_seg) {
  if (T < 0 || K <= 0 || N <= 0 || r <= 0 || r > kMaxRank || num_seg < 0) return 0;
  return bwd_layout(T, K, N, r, num_seg).total;
}

int moe_adapter_linear(const void* x, long long ldx, const void* W, const void* A, const void* B, const float* scale,
                       int num_seg, const int32_t* seg_offsets, const int32_t* seg_adapter, int T, int K, int N, int r,
                       int num_adapters, void* hidden, size_t hidden_bytes, void* y, long long ldy, void* stream) {
  clear_error();
  const char* fn = "moe_adapter_linear";
  const Reqs q{T, num_seg, num_adapters, seg_offsets, seg_adapter};
  if (int rc = check_adapter(fn, q, K, N, r, ldx, ldy)) return rc;
  if (T == 0) return MOE_OK;
  if (!x || !W || !A || !B || !hidden || !y) return fail(MOE_ERR_INVALID_ARG, "%s: NULL pointer argument", fn);
  if (!aligned16(x) || !aligned16(W) || !aligned16(A) || !aligned16(B) || !aligned16(hidden) || !aligned16(y))
    return fail(MOE_ERR_ALIGNMENT, "%s: tensors must be 16-byte aligned", fn);
  if (hidden_bytes < moe_adapter_hidden_size(T, r))
    return fail(MOE_ERR_WORKSPACE, "%s: hidden %zu < %zu bytes", fn, hidden_bytes, moe_adapter_hidden_size(T, r));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (num_seg > 0) {
    const bool few = T <= 4 * num_seg || T <= 16;
    if (int rc = few ? run_gemv(fn, q, x, ldx, A, scale, K, r, hidden, s)
                     : run_shrink<false>(fn, q, x, ldx, A, scale, K, r, hidden, s))
      return rc;
  }
  return run_wide<false>(fn, q, x, ldx, W, hidden, B, K, N, r, y, ldy, num_seg > 0, s);
}

int moe_adapter_linear_bwd(const void* dy, long long lddy, const void* x, long long ldx, const void* W, const void* A,
                           const void* B, const float* scale, const void* hidden, size_t hidden_bytes, int num_seg,
                           const int32_t* seg_offsets, const int32_t* seg_adapter, int T, int K, int N, int r,
                           int num_adapters, void* dx, long long lddx, float* dA, float* dB, int accumulate, void* ws,
                           size_t ws_bytes, void* stream) {
  clear_error();
  const char* fn = "moe_adapter_linear_bwd";
  const Reqs q{T, num_seg, num_adapters, seg_offsets, seg_adapter};
  if (int rc = check_adapter(fn, q, K, N, r, ldx, lddy)) return rc;
  if (lddx < K || lddx % 8 || lddx >= (1ll << 31))
    return fail(MOE_ERR_UNSUPPORTED_SHAPE, "%s: row strides must be multiples of 8 and at least the row length", fn);
  if (!dA || !dB || !ws || (T > 0 && (!dy || !x || !W || !A || !B || !hidden || !dx)))
    return fail(MOE_ERR_INVALID_ARG, "%s: NULL pointer argument", fn);
  if (!aligned16(dy) || !aligned16(x) || !aligned16(W) || !aligned16(A) || !aligned16(B) || !aligned16(hidden) ||
      !aligned16(dx) || !aligned16(dA) || !aligned16(dB) || !aligned16(ws))
    return fail(MOE_ERR_ALIGNMENT, "%s: tensors must be 16-byte aligned", fn);
  if (T > 0 && hidden_bytes < moe_adapter_hidden_size(T, r))
    return fail(MOE_ERR_WORKSPACE, "%s: hidden %zu < %zu bytes", fn, hidden_bytes, moe_adapter_hidden_size(T, r));
  const BwdLayout L = bwd_layout(T, K, N, r, num_seg);
  if (ws_bytes < L.total) return fail(MOE_ERR_WORKSPACE, "%s: workspace %zu < %zu bytes", fn, ws_bytes, L.total);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (T == 0 || num_seg == 0) {
    if (!accumulate) {
      cudaError_t e = cudaMemsetAsync(dA, 0, sizeof(float) * (size_t)num_adapters * r * K, s);
      if (e == cudaSuccess) e = cudaMemsetAsync(dB, 0, sizeof(float) * (size_t)num_adapters * r * N, s);
      if (e != cudaSuccess) return fail_cuda(fn, e);
    }
    if (T == 0) return MOE_OK;
    return run_wide<true>(fn, q, dy, lddy, W, nullptr, A, N, K, r, dx, lddx, false, s);
  }
  char* base = static_cast<char*>(ws);
  void* u = base + L.u;
  if (int rc = run_shrink<true>(fn, q, dy, lddy, B, scale, N, r, u, s)) return rc;
  if (int rc = run_wide<true>(fn, q, dy, lddy, W, u, A, N, K, r, dx, lddx, true, s)) return rc;

  GradParams p{};
  p.q = q;
  p.K = K;
  p.N = N;
  p.r = r;
  p.part_rows = kPartRows;
  p.tiles_a = (K + BM - 1) / BM;
  p.tiles_b = (N + BM - 1) / BM;
  p.dA = dA;
  p.dB = dB;
  p.part = reinterpret_cast<float*>(base + L.part);
  p.accumulate = accumulate;
  const int hp = hidden_pitch(r), hc = hidden_cols(r), nck = hp / 64;
  p.idesc = make_idesc(hc > 256 ? hc / 2 : hc, BM, true, true);
  p.stages = nck == 1 ? 4 : (nck == 2 ? 3 : (nck == 3 ? 5 : 3));
  p.status = status_word();
  static bool attr[64] = {};
  if (int rc = set_smem(reinterpret_cast<const void*>(adapter_grad_kernel), attr, fn, kSmemMax - 1024)) return rc;
  CUtensorMap tx, tu, td, tv;
  if (int rc = map_mn(&tx, x, K, T, ldx, 2)) return rc;
  if (int rc = map_mn(&tu, u, hp, T, hp, nck)) return rc;
  if (int rc = map_mn(&td, dy, N, T, lddy, 2)) return rc;
  if (int rc = map_mn(&tv, hidden, hp, T, hp, nck)) return rc;
  const size_t table = table_bytes(num_seg) + sizeof(int) * (size_t)(2 * num_adapters + 2);
  const size_t smem = 1024 + (size_t)p.stages * (BM * BK * 2 + nck * CHUNK_BYTES) + table + sizeof(int) * (size_t)(num_adapters + 1 + num_seg);
  const int per_sm = nck <= 2 ? 2 : 1;
  const long long most = ((long long)T / kPartRows + num_seg) * (p.tiles_a + p.tiles_b);
  const int sms = sm_count() > 0 ? sm_count() : 148;
  const int grid = (int)(most < (long long)sms * per_sm ? most : (long long)sms * per_sm);
  if (int rc = launch_adapter(fn, adapter_grad_kernel, dim3(grid), 192, smem, 0, s, tx, tu, td, tv, p)) return rc;
  const size_t vec = (size_t)r * (K + N) / 4;
  const int gx = (int)((vec + 255) / 256 < 256 ? (vec + 255) / 256 : 256);
  return launch_adapter(fn, adapter_grad_sum_kernel, dim3(gx, num_adapters), 256, table, 0, s, p);
}

}  // extern "C"
