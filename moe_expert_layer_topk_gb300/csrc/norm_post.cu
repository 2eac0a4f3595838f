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
// (The approximate instructions themselves: each is off by 2^-22 or so, and what is below
// 2^-126 is 0.)
__device__ __forceinline__ Gate sigmoid(float x) {
  float e, t;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(fabsf(x) * -1.44269504f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(t) : "f"(1.0f + e));
  return {x >= 0.f ? t : e * t, e * t * t};
}

// The two gains of a lane's vectors: kept in registers where that is one vector (the
// same for every row), else read for each row.
template <int L, int NV>
struct Gains {
  Gain8 own, next;
  __device__ __forceinline__ Gains(const PostArgs& p, int l)
      : own(p.gain, l, NV == 1 && l < p.H / 8), next(p.next_gain, l, NV == 1 && l < p.H / 8) {}
  __device__ __forceinline__ Gain8 of(const PostArgs& p, int c) const { return NV == 1 ? own : Gain8(p.gain, c, true); }
  __device__ __forceinline__ Gain8 of_next(const PostArgs& p, int c) const { return NV == 1 ? next : Gain8(p.next_gain, c, true); }
};

// What follows a row's z: norm, gate, residual, and the next norm.  res, gate2: the row's
// vectors of the residual and of an element's gate (zeros without).
template <typename S, int L, int NV>
__device__ __forceinline__ void finish_row(const PostArgs& p, RowGroup<L>& rg, const Gains<L, NV>& gains, long long t, float (&z)[NV][8],
                                           const Vec8<S> (&res)[NV], const uint4 (&gate2)[NV], float tok_logit) {
  const int H = p.H, nvec = H / 8;
  const float inv_h = 1.0f / (float)H;
  const bool live = t < p.T;
  float r = 1.f;
  if (p.norm) {
    r = rg.template rstd<NV>(inv_h, p.eps, [&](int i, int j) { return z[i][j]; });
    if (p.rstd && live && rg.l == 0) p.rstd[t] = r;
  }
  const float tok = p.gate_kind == 1 ? p.out_scale * sigmoid(tok_logit).g : p.out_scale;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = rg.l + i * L;
    if (!live || c >= nvec) continue;
    const Gain8 w = gains.of(p, c);
    float g[8];
    unpack8(gate2[i], g);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float v = z[i][j] * r * w.at(j) * tok;
      if (p.gate_kind == 2) v *= sigmoid(g[j]).g;
      if (p.residual) v = __fmaf_rn(p.res_scale, res[i].at(j), v);
      z[i][j] = v;
    }
    Vec8<S>::store(static_cast<S*>(p.out) + t * H + 8 * c, z[i]);
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
      const Gain8 w = gains.of_next(p, c);
      float o[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = z[i][j] * q * w.at(j);
      Vec8<__nv_bfloat16>::store(p.next_y + t * H + 8 * c, o);
    }
  }
}

// The row's vectors of the residual and of an element's gate.
template <typename S, int L, int NV>
__device__ __forceinline__ void load_sides(const PostArgs& p, const RowGroup<L>& rg, long long t, Vec8<S> (&res)[NV], uint4 (&gate2)[NV]) {
  const int nvec = p.H / 8;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = rg.l + i * L;
    const bool there = t < p.T && c < nvec;
    res[i] = zero_vec<S>();
    gate2[i] = make_uint4(0, 0, 0, 0);
    if (p.residual && there) res[i].load(static_cast<const S*>(p.residual) + t * p.H + 8 * c);
    if (p.gate_kind == 2 && there)
      gate2[i] = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.gate) + t * p.H) + c);
  }
}

template <typename S, int L, int NV>
__global__ void __launch_bounds__(kNormThreads) post_norm_kernel(const PostArgs p) {
  pdl_wait();
  pdl_trigger();
  __shared__ float sm[16];
  RowGroup<L> rg(sm);
  const Gains<L, NV> gains(p, rg.l);
  const int nvec = p.H / 8;
  for (long long base = (long long)blockIdx.x * rg.kRows; base < p.T; base += (long long)gridDim.x * rg.kRows) {
    const long long t = base + rg.g;
    float z[NV][8];
    Vec8<S> res[NV];
    uint4 gate2[NV], zv[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = rg.l + i * L;
      zv[i] = t < p.T && c < nvec ? __ldg(reinterpret_cast<const uint4*>(p.z + t * p.H) + c) : make_uint4(0, 0, 0, 0);
    }
    load_sides<S, L, NV>(p, rg, t, res, gate2);
    const float logit = p.gate_kind == 1 && t < p.T ? __ldg(static_cast<const float*>(p.gate) + t) : 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) unpack8(zv[i], z[i]);
    finish_row<S, L, NV>(p, rg, gains, t, z, res, gate2, logit);
  }
}

// Combine: the rows of a token's first eight slots, its residual and its element gate come
// through the lanes' own rings of shared memory while the token before is summed (a
// token's further slots are read when their turn comes); the row ids, a token further
// ahead, and the weights sit in registers, lane j of a warp holding slot j's.
template <typename S, int NV>
struct CombineRing {
  static constexpr int KB = NV == 4 ? 4 : 8;  // four vectors a lane: the first four slots
  static constexpr int SU = sizeof(Vec8<S>) / 16;
  static constexpr int STAGES = 2;
  // a vector's units: rows, residual, element gate
  static __host__ __device__ int per(int gate_kind) { return KB + SU + (gate_kind == 2 ? 1 : 0); }
  static size_t bytes(int gate_kind) { return (size_t)NV * per(gate_kind) * STAGES * kRingUnitBytes; }
};
template <typename S, int L, int NV>
__global__ void __launch_bounds__(kNormThreads, NV == 1 ? 3 : 1) combine_post_norm_kernel(const PostArgs p) {
  pdl_wait();
  pdl_trigger();
  using C = CombineRing<S, NV>;
  constexpr int KB = C::KB, SU = C::SU, STAGES = C::STAGES;
  __shared__ float sm[16];
  extern __shared__ __align__(16) uint8_t ring_smem[];
  const int per = C::per(p.gate_kind);
  RowRing ring(ring_smem, NV * per);
  RowGroup<L> rg(sm);
  const Gains<L, NV> gains(p, rg.l);
  const int H = p.H, nvec = H / 8, k = p.k, lane = threadIdx.x & 31;
  const long long step = (long long)gridDim.x * rg.kRows;
  // this lane's slot of token t; a row out of range counts as none
  auto ids = [&](long long t, int& row, float& w) {
    row = -1;
    w = 0.f;
    if (t < p.T && lane < k) {
      row = __ldg(p.row_of_slot + t * k + lane);
      w = __ldg(p.topk_w + t * k + lane);
    }
  };
  auto checked = [&](long long t, int& row, float& w) {
    if (t < p.T && lane < k && (row < 0 || row >= p.R)) {
      set_status(p.status, MOE_STATUS_BAD_INDEX);
      row = -1;
      w = 0.f;
    }
  };
  auto fetch = [&](int stage, long long t, int row) {
#pragma unroll
    for (int u = 0; u < KB; ++u) {
      if (u >= k) break;
      const int q = __shfl_sync(0xffffffffu, row, u);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = rg.l + i * L;
        const bool there = q >= 0 && c < nvec;
        ring.fetch(stage, i * per + u, p.z + (there ? (size_t)q * H + 8 * c : 0), there);
      }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = rg.l + i * L;
      const bool there = t < p.T && c < nvec;
      const size_t at = there ? (size_t)t * H + 8 * c : 0;
      if (p.residual) {
#pragma unroll
        for (int v = 0; v < SU; ++v)
          ring.fetch(stage, i * per + KB + v, reinterpret_cast<const uint4*>(static_cast<const S*>(p.residual) + at) + v, there);
      }
      if (p.gate_kind == 2) ring.fetch(stage, i * per + KB + SU, static_cast<const __nv_bfloat16*>(p.gate) + at, there);
    }
    ring.commit();
  };
  const long long first = (long long)blockIdx.x * rg.kRows + rg.g;
  float w[STAGES];  // of the token in hand and the STAGES - 1 behind it
  int ahead_row;
  float ahead_w;
#pragma unroll
  for (int q = 0; q < STAGES - 1; ++q) {
    int row;
    ids(first + q * step, row, w[q]);
    checked(first + q * step, row, w[q]);
    fetch(q, first + q * step, row);
  }
  ids(first + (STAGES - 1) * step, ahead_row, ahead_w);
  float logit = p.gate_kind == 1 && first < p.T ? __ldg(static_cast<const float*>(p.gate) + first) : 0.f;
  int stage = 0;
  for (long long base = (long long)blockIdx.x * rg.kRows; base < p.T; base += step) {
    const long long t = base + rg.g;
    checked(t + (STAGES - 1) * step, ahead_row, ahead_w);
    fetch(stage == 0 ? STAGES - 1 : stage - 1, t + (STAGES - 1) * step, ahead_row);
    w[STAGES - 1] = ahead_w;
    ids(t + STAGES * step, ahead_row, ahead_w);
    const float gate = logit;
    logit = p.gate_kind == 1 && t + step < p.T ? __ldg(static_cast<const float*>(p.gate) + t + step) : 0.f;
    ring.template wait<STAGES - 1>();
    float z[NV][8];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) z[i][j] = 0.f;
#pragma unroll
    for (int u = 0; u < KB; ++u) {
      if (u >= k) break;
      const float wu = __shfl_sync(0xffffffffu, w[0], u);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float f[8];
        unpack8(ring.at(stage, i * per + u), f);
#pragma unroll
        for (int j = 0; j < 8; ++j) z[i][j] = __fmaf_rn(wu, f[j], z[i][j]);
      }
    }
    if (k > KB) {
      int row;
      float unused;
      ids(t, row, unused);
      if (row >= p.R) row = -1;
      for (int j0 = KB; j0 < k; j0 += 4) {
        uint4 buf[4][NV];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int q = __shfl_sync(0xffffffffu, row, (j0 + u) & 31);
#pragma unroll
          for (int i = 0; i < NV; ++i) {
            const int c = rg.l + i * L;
            buf[u][i] = j0 + u < k && q >= 0 && c < nvec ? __ldg(reinterpret_cast<const uint4*>(p.z + (size_t)q * H) + c)
                                                         : make_uint4(0, 0, 0, 0);
          }
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const float wu = __shfl_sync(0xffffffffu, w[0], (j0 + u) & 31);
          if (j0 + u >= k) break;
#pragma unroll
          for (int i = 0; i < NV; ++i) {
            float f[8];
            unpack8(buf[u][i], f);
#pragma unroll
            for (int j = 0; j < 8; ++j) z[i][j] = __fmaf_rn(wu, f[j], z[i][j]);
          }
        }
      }
    }
    Vec8<S> res[NV];
    uint4 gate2[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      res[i] = p.residual ? ring.template vec<S>(stage, i * per + KB) : zero_vec<S>();
      gate2[i] = p.gate_kind == 2 ? ring.at(stage, i * per + KB + SU) : make_uint4(0, 0, 0, 0);
    }
    stage = stage + 1 == STAGES ? 0 : stage + 1;
#pragma unroll
    for (int q = 0; q + 1 < STAGES; ++q) w[q] = w[q + 1];
    if (p.z_out && t < p.T) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = rg.l + i * L;
        if (c < nvec) Vec8<__nv_bfloat16>::store(p.z_out + t * H + 8 * c, z[i]);
      }
    }
    finish_row<S, L, NV>(p, rg, gains, t, z, res, gate2, gate);
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

// dz may be z: each vector is read before it is written, by the same thread.
template <typename S, int L, int NV, bool kElement>
struct PostBwd {
  static constexpr int SU = sizeof(Vec8<S>) / 16;                // units of a stream vector
  static constexpr int PER = 1 + SU + (kElement ? 1 : 0);        // z, dout, gate
  static constexpr int UNITS = NV * PER;
};
template <typename S, int L, int NV, bool kElement>
__global__ void __launch_bounds__(kNormThreads, bwd_blocks(NV)) post_norm_bwd_kernel(const PostBwdArgs p) {
  pdl_wait();
  pdl_trigger();
  using P = PostBwd<S, L, NV, kElement>;
  constexpr int SU = P::SU, STAGES = ring_stages(P::UNITS);
  __shared__ float sm[16];
  extern __shared__ __align__(16) uint8_t ring_smem[];
  RowRing ring(ring_smem, P::UNITS);
  RowGroup<L> rg(sm);
  const int H = p.H, nvec = H / 8, T = p.T;
  const float inv_h = 1.0f / (float)H;
  const S* dout = static_cast<const S*>(p.dout);
  const long long step = (long long)gridDim.x * rg.kRows;
  float acc[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[i][j] = 0.f;
  auto fetch = [&](int stage, long long t) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = rg.l + i * L;
      const bool there = t < T && c < nvec;
      const long long at = there ? t * H + 8 * c : 0;
      const int u = i * P::PER;
      ring.fetch(stage, u, p.z + at, there);
#pragma unroll
      for (int q = 0; q < SU; ++q) ring.fetch(stage, u + 1 + q, reinterpret_cast<const uint4*>(dout + at) + q, there);
      if (kElement) ring.fetch(stage, u + 1 + SU, static_cast<const __nv_bfloat16*>(p.gate) + at, there);
    }
    ring.commit();
  };
  const long long first = (long long)blockIdx.x * rg.kRows;
#pragma unroll
  for (int q = 0; q < STAGES - 1; ++q) fetch(q, first + q * step + rg.g);
  int stage = 0;
  for (long long base = first; base < T; base += step) {
    const long long t = base + rg.g;
    const bool live = t < T;
    const float r = p.norm && live ? __ldg(p.rstd + t) : 1.f;
    Gate tok = {1.f, 0.f};
    if (!kElement && p.gate_kind == 1 && live) tok = sigmoid(__ldg(static_cast<const float*>(p.gate) + t));
    ring.template wait<STAGES - 2>();
    const int cur = stage;
    float m = 0.f, dg = 0.f;  // sums of dn n, and of dout n gain
    float n[NV][8], dn[NV][8];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = rg.l + i * L, u = i * P::PER;
      const bool there = live && c < nvec;
      const Gain8 w(p.gain, c, c < nvec);
      const Vec8<__nv_bfloat16> zv = ring.template vec<__nv_bfloat16>(cur, u);
      const Vec8<S> d = ring.template vec<S>(cur, u + 1);
      const Vec8<__nv_bfloat16> gv = kElement ? ring.template vec<__nv_bfloat16>(cur, u + 1 + SU) : zero_vec<__nv_bfloat16>();
      float ds[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        n[i][j] = zv.at(j) * r;
        const float e = p.out_scale * d.at(j), en = e * n[i][j];
        const Gate G = kElement ? sigmoid(gv.at(j)) : tok;
        const float dv = e * G.g;
        acc[i][j] = __fmaf_rn(dv, n[i][j], acc[i][j]);
        dn[i][j] = dv * w.at(j);
        m = __fmaf_rn(dn[i][j], n[i][j], m);
        if (kElement)
          ds[j] = en * w.at(j) * G.d;
        else
          dg = __fmaf_rn(en, w.at(j), dg);
      }
      if (kElement && p.dgate && there) Vec8<__nv_bfloat16>::store(static_cast<__nv_bfloat16*>(p.dgate) + t * H + 8 * c, ds);
    }
    fetch(stage == 0 ? STAGES - 1 : stage - 1, t + (STAGES - 1) * step);
    stage = stage + 1 == STAGES ? 0 : stage + 1;
    if (p.norm) m = rg.sum(m) * inv_h;
    if (!kElement && p.gate_kind == 1 && p.dgate) {
      dg = rg.sum(dg);
      if (live && rg.l == 0) static_cast<float*>(p.dgate)[t] = dg * tok.d;
    }
    if (!live) continue;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = rg.l + i * L;
      if (c >= nvec) continue;
      float o[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = p.norm ? r * (dn[i][j] - n[i][j] * m) : dn[i][j];
      Vec8<__nv_bfloat16>::store(p.dz + t * H + 8 * c, o);
    }
  }
  if (p.part) {  // the ring's memory is free: copies still under way are of rows behind the last, zeros
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
    leave_part<L, NV>(acc, reinterpret_cast<float*>(ring_smem), H, p.part);
  }
}

// Lanes of a token's row and vectors of a lane in the combine.
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
      auto kern = combine_post_norm_kernel<S, L, NV>;
      const size_t smem = CombineRing<S, NV>::bytes(a.gate_kind);
      if (int rc = allow_smem(fn, reinterpret_cast<const void*>(kern), smem)) return rc;
      launch_pdl(kern, norm_grid(a.T, kNormThreads / L, blocks_per_sm(smem, NV == 1 ? 3 : 1), 1 << 30), kNormThreads, smem, s, a);
      return check_launch(fn);
    });
  return with_row_shape(a.H, [&](auto l, auto nv) {
    constexpr int L = decltype(l)::value, NV = decltype(nv)::value;
    launch_pdl(post_norm_kernel<S, L, NV>, norm_grid(a.T, kNormThreads / L, 8, 1 << 30), kNormThreads, 0, s, a);
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
  return with_bwd_shape(H, [&](auto l, auto nv) {
    constexpr int L = decltype(l)::value, NV = decltype(nv)::value;
    int grid = 0;
    auto run = [&](auto type, auto element) {
      using S = decltype(type);
      constexpr bool kElement = decltype(element)::value;
      auto kern = post_norm_bwd_kernel<S, L, NV, kElement>;
      const size_t smem = norm_smem(PostBwd<S, L, NV, kElement>::UNITS, NV);
      grid = norm_grid(T, kNormThreads / L, blocks_per_sm(smem, bwd_blocks(NV)), kNormParts);
      if (int rc = allow_smem(fn, reinterpret_cast<const void*>(kern), smem)) return rc;
      launch_pdl(kern, grid, kNormThreads, smem, s, a);
      return check_launch(fn);
    };
    const int rc = gate_kind == 2 ? (fp32 ? run(float(), std::true_type()) : run(__nv_bfloat16(), std::true_type()))
                                  : (fp32 ? run(float(), std::false_type()) : run(__nv_bfloat16(), std::false_type()));
    if (rc) return rc;
    return dgain ? launch_gain_sum(fn, static_cast<const float*>(ws), grid, H, dgain, accumulate, s) : MOE_OK;
  });
}

}  // extern "C"
