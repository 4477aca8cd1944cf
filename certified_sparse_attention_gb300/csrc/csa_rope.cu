// Per-head norms of queries and keys with the position rotation, and the
// new rows' way into the cache, in one pass (csa_qk_norm_rope).
//
// For a row x of d channels at position p:
//   x <- x (mean x_c^2 + eps)^(-1/2) w_c,
//   (x_a, x_b) <- (x_a cos - x_b sin, x_a sin + x_b cos) for each pair,
// float32 throughout, one rounding at the end.  The angle of pair i is
// p f_i.  The table holds f_i / (2 pi) as a 64-bit fraction of a turn, so
// p times it modulo 2^64 is the angle's exact fraction of a turn at any
// position, and one sincospif on it (|argument| <= 1) has no range
// reduction to lose digits in.
//
// Every row is read once and written once.  A row is held by lanes with two
// vectors of 4 (8: bf16, 16 bytes) channels each.  With split pairs
// (i, i + rot / 2) the two vectors of a lane are partners, so the rotation
// needs no exchange between lanes; with adjacent pairs the partners are in one
// vector.  A lane's sines and cosines serve every head of the token that its
// group processes, and the norm's weights are multiplied into them, so that an
// element costs two multiplications and one fused one.
//
// A prompt of 16K tokens x 48 heads x 128 in bf16, into a cache: 69 us for
// 403 MB, 5.8 TB/s or 86% of the copy bandwidth.  Single tokens: 4.2 us, the
// latency of one launch and of three loads that depend on one another.
#include <cmath>

#include "csa_args.cuh"

namespace csa {

struct RopeArgs {
  const void* q;
  const void* k;
  const void* v;
  csa_strides qs, ks, vs;
  const int64_t* len;
  const int64_t* n_new;
  const void* wq;
  const void* wk;
  const uint64_t* turns;
  void* q_out;
  void* K;
  void* V;
  unsigned* status;
  int64_t n_max;
  int B, T, Hq, Hkv;
  int heads;          // heads to process: q, k and, when given, v
  int rot, interleaved, to_cache;
  int heads_per;      // heads of a token that one group of lanes processes
  int nchunk;         // groups per token
  float eps;
};

// VEC consecutive elements
template <typename E, int VEC> struct Vec;
template <> struct Vec<float, 4> {
  typedef float4 Raw;
  static __device__ __forceinline__ void widen(const Raw& r, float (&x)[4]) { x[0] = r.x; x[1] = r.y; x[2] = r.z; x[3] = r.w; }
  static __device__ __forceinline__ Raw narrow(const float (&x)[4]) { return make_float4(x[0], x[1], x[2], x[3]); }
};
__device__ __forceinline__ unsigned bf16_pair(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const unsigned*>(&v);
}
template <> struct Vec<__nv_bfloat16, 4> {
  typedef uint2 Raw;
  static __device__ __forceinline__ void widen(const Raw& r, float (&x)[4]) {
    x[0] = __uint_as_float(r.x << 16); x[1] = __uint_as_float(r.x & 0xFFFF0000u);
    x[2] = __uint_as_float(r.y << 16); x[3] = __uint_as_float(r.y & 0xFFFF0000u);
  }
  static __device__ __forceinline__ Raw narrow(const float (&x)[4]) { return make_uint2(bf16_pair(x[0], x[1]), bf16_pair(x[2], x[3])); }
};
template <> struct Vec<__nv_bfloat16, 8> {
  typedef uint4 Raw;
  static __device__ __forceinline__ void widen(const Raw& r, float (&x)[8]) {
    const unsigned u[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(i & 1 ? u[i / 2] & 0xFFFF0000u : u[i / 2] << 16);
  }
  static __device__ __forceinline__ Raw narrow(const float (&x)[8]) {
    return make_uint4(bf16_pair(x[0], x[1]), bf16_pair(x[2], x[3]), bf16_pair(x[4], x[5]), bf16_pair(x[6], x[7]));
  }
};

// The elements of a lane's pair i: of split pairs, channel i of both vectors;
// of adjacent ones, channels 2 i and 2 i + 1 of the two vectors in a row.
template <bool INTER, int VEC>
__device__ __forceinline__ float& pair_a(float (&x)[VEC], float (&y)[VEC], int i) {
  return !INTER ? x[i] : i < VEC / 2 ? x[2 * i] : y[2 * i - VEC];
}
template <bool INTER, int VEC>
__device__ __forceinline__ float& pair_b(float (&x)[VEC], float (&y)[VEC], int i) {
  return !INTER ? y[i] : i < VEC / 2 ? x[2 * i + 1] : y[2 * i + 1 - VEC];
}

// Sequence b's first new position and number of new tokens; false (nothing
// to do, flagged by the caller) when they are out of range.
__device__ __forceinline__ bool new_tokens(const int64_t* len, const int64_t* n_new, int b, int T, int64_t cap,
                                           int64_t& start, int64_t& m) {
  const int64_t n = len[b];
  m = n_new ? n_new[b] : (int64_t)T;
  start = n - m;
  return m >= 0 && m <= T && start >= 0 && n <= cap;
}

constexpr int kRopeThreads = 128;
// rows of a group of lanes in flight (a prompt: 2 rows 88 us, 4 69 us, 8 74 us)
constexpr int kRopeBatch = 4;

template <int D, int VEC, bool INTER, typename E>
__global__ void __launch_bounds__(kRopeThreads, 4) qk_norm_rope_kernel(const RopeArgs a) {
  pdl_entry();
  typedef Vec<E, VEC> Vx;
  typedef typename Vx::Raw Raw;
  constexpr int LPR = D / (2 * VEC);         // lanes per row
  constexpr int RPB = kRopeThreads / LPR;    // groups of lanes per CTA
  const int j = threadIdx.x % LPR;
  const int64_t cap = a.to_cache ? a.n_max : INT64_MAX;
  if (a.status && blockIdx.x == 0 && threadIdx.x < 32) {
    bool bad = false;
    for (int b = threadIdx.x; b < a.B; b += 32) {
      int64_t s0, m0;
      bad |= !new_tokens(a.len, a.n_new, b, a.T, cap, s0, m0);
    }
    const unsigned any = __any_sync(0xffffffffu, bad);
    if (threadIdx.x == 0) *a.status = any ? 8u : 0u;
  }
  const int64_t item = (int64_t)blockIdx.x * RPB + threadIdx.x / LPR;
  const int64_t tok = item / a.nchunk;
  const int chunk = (int)(item - tok * a.nchunk);
  const int b = (int)(tok / a.T), t = (int)(tok - (int64_t)b * a.T);
  // (a group of lanes leaves as a whole; the shuffles below name its lanes)
  int64_t start = 0, m = 0;
  if (b >= a.B || !new_tokens(a.len, a.n_new, b, a.T, cap, start, m) || t >= m) return;
  const int64_t pos = start + t;

  const bool turns_here = 2 * VEC * j < a.rot;
  // first channels of the two vectors: split pairs sit rot / 2 apart
  const int c0 = !INTER && turns_here ? VEC * j : 2 * VEC * j;
  const int c1 = !INTER && turns_here ? c0 + a.rot / 2 : c0 + VEC;
  const int h_lo = chunk * a.heads_per, h_hi = min(h_lo + a.heads_per, a.heads);
  const unsigned group_mask = (unsigned)((1ull << LPR) - 1) << (threadIdx.x % 32 / LPR * LPR);

  float cs[VEC], sn[VEC];

  // the chunk's heads of q, of k and of v in turn
  bool have_turns = false;
#pragma unroll 1
  for (int part = 0; part < 3; ++part) {
    const int first = part == 0 ? 0 : part == 1 ? a.Hq : a.Hq + a.Hkv;      // the part's first head
    const int lo = max(h_lo, first) - first;
    const int hi = min(h_hi, part == 0 ? a.Hq : first + a.Hkv) - first;
    if (lo >= hi) continue;
    const csa_strides& st = part == 0 ? a.qs : part == 1 ? a.ks : a.vs;
    const E* src = reinterpret_cast<const E*>(part == 0 ? a.q : part == 1 ? a.k : a.v) + b * st.b + t * st.t + lo * st.h;
    Raw r0[kRopeBatch], r1[kRopeBatch];
    const auto load = [&](int h) {
#pragma unroll
      for (int i = 0; i < kRopeBatch; ++i) {
        if (h + i >= hi) continue;
        r0[i] = *reinterpret_cast<const Raw*>(src + c0);
        r1[i] = *reinterpret_cast<const Raw*>(src + c1);
        src += st.h;
      }
    };
    load(lo);       // (on their way during the sines and cosines)
    E* dst = reinterpret_cast<E*>(part == 0 ? a.q_out : part == 1 ? a.K : a.V);
    int64_t dstep = D;
    if (part == 0) {
      dst += (((int64_t)b * a.T + t) * a.Hq + lo) * D;
    } else if (a.to_cache) {
      dst += (((int64_t)b * a.Hkv + lo) * a.n_max + pos) * D;
      dstep = a.n_max * D;
    } else {
      dst += (((int64_t)b * a.T + t) * a.Hkv + lo) * D;
    }
    // pair i of the lane: (x_a, x_b) <- (x_a wa cos - x_b wb sin, x_a wa sin + x_b wb cos)
    float ac[VEC], bs[VEC], as[VEC], bc[VEC];
    const void* wt = part == 0 ? a.wq : a.wk;
    if (part < 2) {
      float w0[VEC], w1[VEC];
#pragma unroll
      for (int c = 0; c < VEC; ++c) w0[c] = w1[c] = 1.0f;
      if (wt) {
        Vx::widen(*reinterpret_cast<const Raw*>(reinterpret_cast<const E*>(wt) + c0), w0);
        Vx::widen(*reinterpret_cast<const Raw*>(reinterpret_cast<const E*>(wt) + c1), w1);
      }
      if (!have_turns) {
        have_turns = true;
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          cs[i] = 1.0f;
          sn[i] = 0.0f;
          if (turns_here) {
            const long long frac = (long long)((unsigned long long)pos * a.turns[VEC * j + i]);   // signed: [-1/2, 1/2) turn
            sincospif((float)frac * 1.0842021724855044e-19f, &sn[i], &cs[i]);                     // 2^-63: in units of pi
          }
        }
      }
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const float wa = pair_a<INTER, VEC>(w0, w1, i), wb = pair_b<INTER, VEC>(w0, w1, i);
        ac[i] = wa * cs[i]; bs[i] = wb * sn[i]; as[i] = wa * sn[i]; bc[i] = wb * cs[i];
      }
    }
#pragma unroll 1
    for (int h = lo; h < hi; h += kRopeBatch) {
      if (h != lo) load(h);
#pragma unroll
      for (int i = 0; i < kRopeBatch; ++i) {
        if (h + i >= hi) continue;
        if (part < 2) {
          float x[VEC], y[VEC];
          Vx::widen(r0[i], x);
          Vx::widen(r1[i], y);
          if (wt) {
            float ss = 0.0f;
#pragma unroll
            for (int c = 0; c < VEC; ++c) ss += x[c] * x[c] + y[c] * y[c];
#pragma unroll
            for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(group_mask, ss, o);
            const float inv = rsqrtf(ss * (1.0f / D) + a.eps);
#pragma unroll
            for (int c = 0; c < VEC; ++c) { x[c] *= inv; y[c] *= inv; }
          }
#pragma unroll
          for (int c = 0; c < VEC; ++c) {
            float &xa = pair_a<INTER, VEC>(x, y, c), &xb = pair_b<INTER, VEC>(x, y, c);
            if (turns_here) {
              const float u = xa * ac[c] - xb * bs[c];
              xb = xa * as[c] + xb * bc[c];
              xa = u;
            } else {          // (no partner: one that is infinite would reach it through 0 times infinity)
              xa *= ac[c];
              xb *= bc[c];
            }
          }
          r0[i] = Vx::narrow(x);
          r1[i] = Vx::narrow(y);
        }
        *reinterpret_cast<Raw*>(dst + c0) = r0[i];
        *reinterpret_cast<Raw*>(dst + c1) = r1[i];
        dst += dstep;
      }
    }
  }
}

template <int D, int VEC, typename E>
cudaError_t launch_rope(RopeArgs a, int64_t tokens, cudaStream_t st) {
  constexpr int RPB = kRopeThreads / (D / (2 * VEC));
  // heads of a token to a group of lanes: the more, the fewer sines and
  // cosines (all 48 of a prompt 69 us, at most 16 of them 100 us); but first
  // enough groups for four CTAs on every SM
  const int64_t per = tokens * a.heads / ((int64_t)sm_count() * 4 * RPB);
  a.heads_per = (int)(per < 1 ? 1 : per > 64 ? 64 : per);
  a.nchunk = (a.heads + a.heads_per - 1) / a.heads_per;
  const int64_t blocks = (tokens * a.nchunk + RPB - 1) / RPB;
  if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
  const dim3 grid((unsigned)blocks), block(kRopeThreads);
  if (a.interleaved) launch_pdl(qk_norm_rope_kernel<D, VEC, true, E>, grid, block, 0, st, a);
  else launch_pdl(qk_norm_rope_kernel<D, VEC, false, E>, grid, block, 0, st, a);
  return cudaGetLastError();
}

}  // namespace csa

using namespace csa;

extern "C" {

csa_status csa_rope_turns(const double* inv_freq, int n, uint64_t* turns) {
  if (!inv_freq || !turns || n < 0) return CSA_ERR_INVALID_ARG;
  // 1 / (2 pi) as the sum of two doubles
  const double hi = 0x1.45f306dc9c883p-3, lo = -0x1.6b01ec5417056p-57;
  for (int i = 0; i < n; ++i) {
    const double f = std::fabs(inv_freq[i]);
    if (!(f <= 1048576.0)) return CSA_ERR_INVALID_ARG;
    const double p = f * hi;
    const double e = std::fma(f, hi, -p) + f * lo;      // f / (2 pi) = p + e
    const double t = std::ldexp(p - std::floor(p), 64);  // exact, below 2^64
    const uint64_t u = (uint64_t)t;
    const uint64_t turn = u + (uint64_t)(int64_t)std::nearbyint((t - (double)u) + std::ldexp(e, 64));
    turns[i] = inv_freq[i] < 0.0 ? 0u - turn : turn;
  }
  return CSA_OK;
}

csa_status csa_qk_norm_rope(const csa_shape* shape, int T, const csa_norm_rope* params, const void* q,
                            const csa_strides* qs, const void* k, const csa_strides* ks, const void* v,
                            const csa_strides* vs, const int64_t* len, const int64_t* n_new, void* q_out, void* K,
                            void* V, int to_cache, uint32_t* status, void* stream) {
  if (!shape_ok(shape) || !params || T < 1 || !q || !k || !len || !q_out || !K || (v && !V) ||
      (to_cache != 0 && to_cache != 1))
    return CSA_ERR_INVALID_ARG;
  const csa_status su = shape_supported(shape);
  if (su != CSA_OK) return su;
  const int d = shape->d;
  if (params->rot_dim < 0 || params->rot_dim > d || params->rot_dim % 8 != 0 || (params->rot_dim && !params->turns) ||
      (params->interleaved != 0 && params->interleaved != 1) || !(params->norm_eps >= 0.f) ||
      !std::isfinite(params->norm_eps))
    return CSA_ERR_INVALID_ARG;
  const bool bf16 = shape->dtype == CSA_BF16;
  const int64_t unit = bf16 ? 8 : 4;
  if (!strides_ok(qs, unit, shape->B, T, shape->Hq) || !strides_ok(ks, unit, shape->B, T, shape->Hkv) ||
      (v && !strides_ok(vs, unit, shape->B, T, shape->Hkv)))
    return CSA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(q_out) || !aligned16(K) || !aligned16(V) ||
      !aligned16(params->wq) || !aligned16(params->wk))
    return CSA_ERR_INVALID_ARG;
  RopeArgs a = {};
  a.q = q; a.k = k; a.v = v; a.qs = *qs; a.ks = *ks;
  if (v) a.vs = *vs;
  a.len = len; a.n_new = n_new; a.wq = params->wq; a.wk = params->wk; a.turns = params->turns;
  a.q_out = q_out; a.K = K; a.V = V; a.status = status; a.n_max = shape->n_max;
  a.B = shape->B; a.T = T; a.Hq = shape->Hq; a.Hkv = shape->Hkv;
  a.rot = params->rot_dim; a.interleaved = params->interleaved; a.to_cache = to_cache; a.eps = params->norm_eps;
  a.heads = shape->Hq + (v ? 2 : 1) * shape->Hkv;
  const int64_t tokens = (int64_t)shape->B * T;
  add_launches(1);
  cudaStream_t st = (cudaStream_t)stream;
  // bf16: 16-byte accesses where the rotated part divides into them
  const bool wide = params->rot_dim % 16 == 0;
  cudaError_t e;
  if (d == 128)
    e = !bf16 ? launch_rope<128, 4, float>(a, tokens, st)
        : wide ? launch_rope<128, 8, __nv_bfloat16>(a, tokens, st) : launch_rope<128, 4, __nv_bfloat16>(a, tokens, st);
  else
    e = !bf16 ? launch_rope<64, 4, float>(a, tokens, st)
        : wide ? launch_rope<64, 8, __nv_bfloat16>(a, tokens, st) : launch_rope<64, 4, __nv_bfloat16>(a, tokens, st);
  return e == cudaSuccess ? CSA_OK : CSA_ERR_CUDA;
}

}  // extern "C"
