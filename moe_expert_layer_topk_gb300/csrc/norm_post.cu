// The norm after a block with the block's gate, the residual and a scale for each;
// alone or on the weighted combine of the experts' rows, with the next block's norm
// of the result where it is asked for.
//
//   n = z r (norm) or z, G = sigmoid(gate):  out = a residual + b G n gain
//
// Bound by HBM: a token's row stays in the registers of its lanes from the experts'
// rows to the next block's input.
#include "norm_gate.cuh"

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

// The two gains of a lane's vectors: kept in registers where that is one vector (the
// same for every row), else read for each row.
template <int NV>
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
__device__ __forceinline__ void finish_row(const PostArgs& p, RowGroup<L>& rg, const Gains<NV>& gains, long long t, float (&z)[NV][8],
                                           const Vec8<S> (&res)[NV], const uint4 (&gate2)[NV], float tok_logit) {
  const int H = p.H, nvec = H / 8, n = rg.lanes();
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
    const int c = rg.l + i * n;
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
      const int c = rg.l + i * n;
      if (!live || c >= nvec) continue;
      const Gain8 w = gains.of_next(p, c);
      float o[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = z[i][j] * q * w.at(j);
      Vec8<__nv_bfloat16>::store(p.next_y + t * H + 8 * c, o);
    }
  }
}

// Alone: as the norm before a block, a vector a lane within a warp, up to four beyond.
template <typename S, int L, int NV>
__global__ void __launch_bounds__(256, L ? 4 : (sizeof(S) == 2 ? 3 : 2)) post_norm_kernel(const PostArgs p, int W) {
  pdl_wait();
  pdl_trigger();
  __shared__ __align__(16) float sm[kSumFloats];
  RowGroup<L> rg(sm, W);
  const Gains<NV> gains(p, rg.l);
  const int nvec = p.H / 8, n = rg.lanes();
  for (long long base = (long long)blockIdx.x * rg.rows(); base < p.T; base += (long long)gridDim.x * rg.rows()) {
    const long long t = base + rg.g;
    float z[NV][8];
    Vec8<S> res[NV];
    uint4 gate2[NV], zv[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = rg.l + i * n;
      const bool there = t < p.T && c < nvec;
      zv[i] = gate2[i] = make_uint4(0, 0, 0, 0);
      res[i] = zero_vec<S>();
      if (there) zv[i] = __ldg(reinterpret_cast<const uint4*>(p.z + t * p.H) + c);
      if (there && p.residual) res[i].load(static_cast<const S*>(p.residual) + t * p.H + 8 * c);
      if (there && p.gate_kind == 2)
        gate2[i] = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.gate) + t * p.H) + c);
    }
    const float logit = p.gate_kind == 1 && t < p.T ? __ldg(static_cast<const float*>(p.gate) + t) : 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) unpack8(zv[i], z[i]);
    finish_row<S, L, NV>(p, rg, gains, t, z, res, gate2, logit);
  }
}

// The rows of a token's first slots (eight; four where a lane has two vectors), its
// residual and its element gate come through the lanes' own rings of shared memory,
// STAGES - 1 tokens ahead of the one that is summed; a token's further slots are read when
// their turn comes.  The row ids, a token further ahead, and the weights sit in registers,
// lane j of a warp holding slot j's.
//
// Bound by HBM.  8192 x 2048, top-8, token gate, next norm: 67.4 us (6.0 TB/s) on three
// blocks of 256 threads an SM with two stages; two blocks with three stages 75; rows in
// registers instead of shared memory 88.5 to 109.
template <typename S, int NV>
struct PostRing {
  static constexpr int KB = NV == 1 ? 8 : 4;
  static constexpr int SU = sizeof(Vec8<S>) / 16;
  // a vector's units: rows, residual, element gate
  static __host__ __device__ int rows(int k) { return k < KB ? k : KB; }
  static __host__ __device__ int per(int k, int gate_kind) { return rows(k) + SU + (gate_kind == 2 ? 1 : 0); }
};
// threads of a block at most, and the registers a thread that its blocks an SM leave
template <int NV, bool kWide>
struct PostBlock {
  static constexpr int THREADS = kWide ? 512 : 256, BLOCKS = kWide ? 1 : 3, REGS = kWide ? 128 : 80;
};
template <typename S, int L, int NV, bool kWide, int STAGES>
__global__ void __launch_bounds__(PostBlock<NV, kWide>::THREADS, PostBlock<NV, kWide>::BLOCKS) combine_post_norm_kernel(const PostArgs p, int W) {
  pdl_wait();
  pdl_trigger();
  using C = PostRing<S, NV>;
  constexpr int KB = C::KB, SU = C::SU;
  __shared__ __align__(16) float sm[kSumFloats];
  extern __shared__ __align__(16) uint8_t ring_smem[];
  const int k = p.k, kr = C::rows(k), per = C::per(k, p.gate_kind);
  RowRing ring(ring_smem, NV * per);
  RowGroup<L> rg(sm, W);
  const Gains<NV> gains(p, rg.l);
  const int H = p.H, nvec = H / 8, n = rg.lanes(), lane = threadIdx.x & 31;
  const long long step = (long long)gridDim.x * rg.rows();
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
      if (u >= kr) break;
      const int q = __shfl_sync(0xffffffffu, row, u);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = rg.l + i * n;
        const bool there = q >= 0 && c < nvec;
        ring.fetch(stage, i * per + u, p.z + (there ? (size_t)q * H + 8 * c : 0), there);
      }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = rg.l + i * n;
      const bool there = t < p.T && c < nvec;
      const size_t at = there ? (size_t)t * H + 8 * c : 0;
      if (p.residual) ring.fetch(stage, i * per + kr, static_cast<const S*>(p.residual) + at, there);
      if (p.gate_kind == 2) ring.fetch(stage, i * per + kr + SU, static_cast<const __nv_bfloat16*>(p.gate) + at, there);
    }
    ring.commit();
  };
  const long long block0 = (long long)blockIdx.x * rg.rows(), first = block0 + rg.g;
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
  auto token_gate = [&](long long t) { return p.gate_kind == 1 && t < p.T ? __ldg(static_cast<const float*>(p.gate) + t) : 0.f; };
  float logit = token_gate(first);
  int stage = 0;
  for (long long base = block0; base < p.T; base += step) {
    const long long t = base + rg.g;
    checked(t + (STAGES - 1) * step, ahead_row, ahead_w);
    fetch(stage == 0 ? STAGES - 1 : stage - 1, t + (STAGES - 1) * step, ahead_row);
    w[STAGES - 1] = ahead_w;
    ids(t + STAGES * step, ahead_row, ahead_w);
    const float gate = logit;
    logit = token_gate(t + step);
    ring.template wait<STAGES - 1>();
    float z[NV][8];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) z[i][j] = 0.f;
#pragma unroll
    for (int u = 0; u < KB; ++u) {
      if (u >= kr) break;
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
            const int c = rg.l + i * n;
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
      res[i] = p.residual ? ring.template vec<S>(stage, i * per + kr) : zero_vec<S>();
      gate2[i] = p.gate_kind == 2 ? ring.at(stage, i * per + kr + SU) : make_uint4(0, 0, 0, 0);
    }
    stage = stage + 1 == STAGES ? 0 : stage + 1;
#pragma unroll
    for (int q = 0; q + 1 < STAGES; ++q) w[q] = w[q + 1];
    if (p.z_out && t < p.T) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = rg.l + i * n;
        if (c < nvec) Vec8<__nv_bfloat16>::store(p.z_out + t * H + 8 * c, z[i]);
      }
    }
    finish_row<S, L, NV>(p, rg, gains, t, z, res, gate2, gate);
  }
}

template <typename S>
int run_post_norm(const char* fn, const PostArgs& a, cudaStream_t s) {
  const RowShape sh = row_shape(a.H, 4);
  return with_lanes<true>(sh.L, [&](auto l) {
    constexpr int L = decltype(l)::value, NV = L ? 1 : 4;
    launch_pdl(post_norm_kernel<S, L, NV>, norm_grid(a.T, sh.rows, 8, 1 << 30), sh.threads, 0, s, a, sh.W);
    return check_launch(fn);
  });
}

// A vector a lane in 256 threads up to 2048 columns and in 512 up to 4096, two in 512
// beyond.  With up to three rows a token, tokens are small and four stages are held (two
// beyond 4096 columns: 224 KB of shared memory at most).
template <typename S>
int run_combine_post_norm(const char* fn, const PostArgs& a, cudaStream_t s) {
  auto run = [&](auto l, auto v, auto wide, auto stages) {
    constexpr int L = decltype(l)::value, NV = decltype(v)::value, STAGES = decltype(stages)::value;
    constexpr bool kWide = decltype(wide)::value;
    RowShape sh = row_shape(a.H, NV);
    if (L == 32) sh = {32, 1, 8, 256};  // short rows too: a warp's lanes hold a token's slots
    auto kern = combine_post_norm_kernel<S, L, NV, kWide, STAGES>;
    const size_t smem = (size_t)NV * PostRing<S, NV>::per(a.k, a.gate_kind) * STAGES * sh.threads * 16;
    static bool done[kMaxDevices];
    if (int rc = allow_smem(fn, reinterpret_cast<const void*>(kern), smem, done)) return rc;
    launch_pdl(kern, norm_grid(a.T, sh.rows, blocks_per_sm(smem, sh.threads, PostBlock<NV, kWide>::REGS), 1 << 30), sh.threads, smem, s, a,
               sh.W);
    return check_launch(fn);
  };
  using std::integral_constant;
  auto shaped = [&](auto stages) {
    if (a.H <= 256) return run(integral_constant<int, 32>{}, integral_constant<int, 1>{}, std::false_type{}, stages);
    if (a.H <= 2048) return run(integral_constant<int, 0>{}, integral_constant<int, 1>{}, std::false_type{}, stages);
    return run(integral_constant<int, 0>{}, integral_constant<int, 1>{}, std::true_type{}, stages);
  };
  if (a.H > 4096) return run(integral_constant<int, 0>{}, integral_constant<int, 2>{}, std::true_type{}, integral_constant<int, 2>{});
  return a.k <= 3 ? shaped(integral_constant<int, 4>{}) : shaped(integral_constant<int, 2>{});
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
  return fp32 ? run_post_norm<float>(fn, a, s) : run_post_norm<__nv_bfloat16>(fn, a, s);
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
  return fp32 ? run_combine_post_norm<float>(fn, a, s) : run_combine_post_norm<__nv_bfloat16>(fn, a, s);
}

}  // extern "C"
