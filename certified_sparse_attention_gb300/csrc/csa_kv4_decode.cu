// Decode attention over the 4-bit K/V cache (csa_kv4_decode):
//   o = softmax(q K^T / sqrt d) V
// for the last T tokens of every sequence, K and V the values the cache
// stands for (whole blocks of 64 tokens in codes, the incomplete last block
// in full precision).
//
// Work is split over the long axis by units of one block of one (sequence,
// KV head): the units of the whole batch, in order, are dealt to the CTAs in
// equal runs, whatever the lengths, which are read on the device.  A CTA
// walks its run item by item (an item: one (sequence, KV head)); its warps
// take the blocks in turn, each with its own running maximum and sums, and
// merge them in shared memory.  An item that lies in one CTA is finished
// there; the parts of the others (at most two per CTA: its first and its
// last item) go to the workspace, and a second kernel joins them, one CTA
// for each item that was cut.
//
// The rows of an item are its T * G query vectors (G query heads share the
// KV head); a warp handles a tile of 8 rows, so with more than 8 rows the
// warps of a CTA form teams of 2, 4 or 8 that share the blocks.
#include <cmath>

#include "csa_args.cuh"

namespace csa {

struct Kv4DecodeArgs {
  csa_kv4 c;
  const void* q;
  csa_strides qs;
  const int64_t* len;
  const int64_t* n_q;
  float* o;
  float* lse;
  unsigned* status;
  float* part;          // [2 * CTAs][rows][D + 2]: m, l, acc[D]
  int64_t n_max, nblk_max;
  int B, T, Hq, Hkv, G;
  float rs;             // log2(e) / sqrt(d): scores in units of log 2
};

constexpr int kKdWarps = 8;
constexpr int kKdTile = 8;        // query rows of a warp

// units of one (sequence, KV head) of n tokens (at least one: somebody has to
// write the output of an empty sequence)
__device__ __forceinline__ int64_t kd_units(int64_t n) { return n > 0 ? (n + kBlock - 1) / kBlock : 1; }
__device__ __forceinline__ int64_t kd_len(const Kv4DecodeArgs& a, int b) {
  return min(max(a.len[b], (int64_t)0), a.n_max);
}
__device__ __forceinline__ int64_t kd_nq(const Kv4DecodeArgs& a, int b) {
  return a.n_q ? min(max(a.n_q[b], (int64_t)0), (int64_t)a.T) : (int64_t)a.T;
}

// s_pref[b] = units of the sequences before b (s_pref[B]: all), by warp 0
__device__ __forceinline__ void kd_prefix(const Kv4DecodeArgs& a, int64_t* s_pref) {
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    int64_t u[4], sum = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int b = lane * 4 + i;
      u[i] = b < a.B ? kd_units(kd_len(a, b)) * a.Hkv : 0;
      sum += u[i];
    }
    int64_t x = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    int64_t before = x - sum;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      s_pref[lane * 4 + i] = before;
      before += u[i];
    }
    if (lane == 31) s_pref[kMaxB] = before;
  }
  __syncthreads();
}

// the sequence that holds unit u: the last b with s_pref[b] <= u (sequences
// past B hold no units and start at the end)
__device__ __forceinline__ int kd_find(const int64_t* s_pref, int B, int64_t u) {
  int lo = 0, hi = B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (s_pref[mid] <= u) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// writes one finished row
template <int D>
__device__ __forceinline__ void kd_store(const Kv4DecodeArgs& a, int b, int g, int r, int c, float M, float l, float v) {
  const int t = r / a.G, h = g * a.G + r % a.G;
  const int64_t row = ((int64_t)b * a.T + t) * a.Hq + h;
  // l = 0 only where nothing was attended to
  a.o[row * D + c] = l == 0.0f ? 0.0f : v / l;
  if (c == 0 && a.lse) a.lse[row] = l == 0.0f ? -INFINITY : (M + log2f(l)) * 0.69314718055994531f;
}

template <int D>
struct KdState {
  float m[kKdTile], l[kKdTile], acc[kKdTile][D / 32];
};

// one online-softmax step of a warp over eight tokens: lane holds channels
// [lane * D / 32, ...) of the eight rows; tok(lane & 7) is the position of
// the token whose score the lane ends up with; row r sees positions below
// s_end[r]
template <int D>
__device__ __forceinline__ void kd_step(KdState<D>& st, const float (&kv)[8][D / 32], const float (&vv)[8][D / 32],
                                        const float* s_q, const int64_t* s_end, int64_t pos, int rows) {
  constexpr int CPL = D / 32;
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int r = 0; r < kKdTile; ++r) {
    if (r >= rows) break;
    float part[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float p[CPL];
#pragma unroll
      for (int c = 0; c < CPL; ++c) p[c] = kv[i][c] * s_q[r * D + lane * CPL + c];
      part[i] = local_tree<CPL>(p);
    }
    float s = reduce8_rows(part);
    const bool seen = pos < s_end[r];
    if (!seen) s = -INFINITY;
    float mx = s;
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
    const float mn = fmaxf(st.m[r], mx);
    const unsigned who = __ballot_sync(0xffffffffu, seen) & 0xffu;
    if (who == 0u) continue;
    const float ref = mn > -INFINITY ? mn : 0.0f;
    const float sc = exp2f(st.m[r] - ref);
    const float p = seen ? exp2f(s - ref) : 0.0f;
    float ps = p;
    ps += __shfl_xor_sync(0xffffffffu, ps, 1);
    ps += __shfl_xor_sync(0xffffffffu, ps, 2);
    ps += __shfl_xor_sync(0xffffffffu, ps, 4);
    st.l[r] = st.l[r] * sc + ps;
    st.m[r] = mn;
#pragma unroll
    for (int c = 0; c < CPL; ++c) st.acc[r][c] *= sc;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float pi = __shfl_sync(0xffffffffu, p, i);
      // an unseen token's value may be anything: it is left out, not
      // multiplied by zero
      if (who >> i & 1u) {
#pragma unroll
        for (int c = 0; c < CPL; ++c) st.acc[r][c] += pi * vv[i][c];
      }
    }
  }
}

template <int D, typename E>
__global__ void __launch_bounds__(kKdWarps * 32) kv4_decode_kernel(const Kv4DecodeArgs a) {
  pdl_entry();
  constexpr int CPL = D / 32;
  __shared__ int64_t s_pref[kMaxB + 1];
  __shared__ int64_t s_end[CSA_KV4_MAX_ROWS];
  __shared__ float s_m[kKdWarps][kKdTile], s_l[kKdWarps][kKdTile];
  extern __shared__ __align__(16) float dyn[];
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int R = a.T * a.G, Rp = (R + kKdTile - 1) / kKdTile * kKdTile;
  float* s_q = dyn;                         // [Rp][D]
  float* s_acc = dyn + Rp * D;              // [warps][8][D]
  // teams: warps that share a block, one tile of rows each
  const int ntile = Rp / kKdTile;
  const int team = ntile <= 1 ? 1 : ntile <= 2 ? 2 : ntile <= 4 ? 4 : 8;
  const int nteam = kKdWarps / team, my_team = w / team, tile = w % team;
  const int rows = min(kKdTile, R - tile * kKdTile);      // <= 0: a warp with no rows
  kd_prefix(a, s_pref);
  if (blockIdx.x == 0 && tid < 32) {
    bool bad = false;
    for (int b = lane; b < a.B; b += 32) {
      bad |= a.len[b] < 0 || a.len[b] > a.n_max;
      if (a.n_q) bad |= a.n_q[b] < 0 || a.n_q[b] > a.T;
    }
    const unsigned any = __any_sync(0xffffffffu, bad);
    if (lane == 0) *a.status = any ? 8u : 0u;
  }
  const int64_t total = s_pref[kMaxB];
  const int64_t per = (total + gridDim.x - 1) / gridDim.x;
  const int64_t u0 = (int64_t)blockIdx.x * per, u1 = min(total, u0 + per);

  for (int64_t u = u0; u < u1;) {
    const int b = kd_find(s_pref, a.B, u);
    const int64_t n = kd_len(a, b), ub = kd_units(n), rem = u - s_pref[b];
    const int g = (int)(rem / ub);
    const int64_t blk0 = rem - (int64_t)g * ub, cnt = min(ub - blk0, u1 - u);
    const int64_t nfull = n / kBlock, bg = (int64_t)b * a.Hkv + g;
    const int64_t nq = kd_nq(a, b);
    __syncthreads();
    for (int i = tid; i < Rp * D; i += kKdWarps * 32) {
      const int r = i / D, c = i - r * D;
      const int t = r / a.G;
      float x = 0.0f;
      if (t < nq)
        x = Elem<E>::get(reinterpret_cast<const E*>(a.q) + b * a.qs.b + t * a.qs.t + (int64_t)(g * a.G + r % a.G) * a.qs.h, c) * a.rs;
      s_q[i] = x;
    }
    if (tid < Rp) s_end[tid] = tid / a.G < nq ? n - nq + tid / a.G + 1 : 0;
    __syncthreads();
    KdState<D> st;
#pragma unroll
    for (int r = 0; r < kKdTile; ++r) {
      st.m[r] = -INFINITY; st.l[r] = 0.0f;
#pragma unroll
      for (int c = 0; c < CPL; ++c) st.acc[r][c] = 0.0f;
    }
    if (rows > 0) {
      const float* q = s_q + tile * kKdTile * D;
      const int64_t* end = s_end + tile * kKdTile;
      // groups of eight tokens, in turn over the teams
      for (int64_t x = my_team; x < cnt * 8; x += nteam) {
        const int64_t blk = blk0 + x / 8;
        const int grp = (int)(x % 8);
        const int64_t p0 = blk * kBlock;
        float kv[8][CPL], vv[8][CPL];
        if (blk < nfull) {
          const int64_t at = bg * a.nblk_max + blk;
          float mn[CPL], dl[CPL];
          unsigned vw[CPL];
#pragma unroll
          for (int c = 0; c < CPL; ++c) {
            mn[c] = a.c.bounds[at * 2 * D + lane * CPL + c];
            dl[c] = a.c.bounds[at * 2 * D + D + lane * CPL + c];
            vw[c] = reinterpret_cast<const unsigned*>(a.c.V4)[(at * D + lane * CPL + c) * 8 + grp];
          }
          // word grp of a V4 row: tokens 32 i + 16 u + 8 v + 2 w + e with
          // i = grp & 1, w = grp >> 1, nibble 4 e + 2 u + v
          const int base = 32 * (grp & 1) + 2 * (grp >> 1);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int t = base + 16 * ((i >> 1) & 1) + 8 * (i & 1) + (i >> 2);
            const float2 sc = reinterpret_cast<const float2*>(a.c.vscale)[at * kBlock + t];
            const uint8_t* kr = a.c.K4 + (at * kBlock + t) * (D / 2) + lane * CPL / 2;
#pragma unroll
            for (int c = 0; c < CPL; ++c) {
              kv[i][c] = fadd(fmul((float)((kr[c / 2] >> (4 * (c & 1))) & 15), dl[c]), mn[c]);
              vv[i][c] = fadd(fmul((float)((vw[c] >> (4 * i)) & 15u), sc.y), sc.x);
            }
          }
          const int i = lane & 7;
          kd_step<D>(st, kv, vv, q, end, p0 + base + 16 * ((i >> 1) & 1) + 8 * (i & 1) + (i >> 2), rows);
        } else {
          if (p0 + 8 * grp >= n) continue;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int t = 8 * grp + i;
            const bool there = p0 + t < n;
            const E* kr = reinterpret_cast<const E*>(a.c.Kt) + (bg * kBlock + t) * D + lane * CPL;
            const E* vr = reinterpret_cast<const E*>(a.c.Vt) + (bg * kBlock + t) * D + lane * CPL;
#pragma unroll
            for (int c = 0; c < CPL; ++c) {
              kv[i][c] = there ? Elem<E>::get(kr, c) : 0.0f;
              vv[i][c] = there ? Elem<E>::get(vr, c) : 0.0f;
            }
          }
          kd_step<D>(st, kv, vv, q, end, p0 + 8 * grp + (lane & 7), rows);
        }
      }
    }
    // merge the teams
#pragma unroll
    for (int r = 0; r < kKdTile; ++r) {
      if (lane == 0) { s_m[w][r] = st.m[r]; s_l[w][r] = st.l[r]; }
#pragma unroll
      for (int c = 0; c < CPL; ++c) s_acc[(w * kKdTile + r) * D + lane * CPL + c] = st.acc[r][c];
    }
    __syncthreads();
    const bool done = cnt == ub;
    float* part = a.part + (2 * (int64_t)blockIdx.x + (u == u0 ? 0 : 1)) * R * (D + 2);
    for (int i = tid; i < R * D; i += kKdWarps * 32) {
      const int r = i / D, c = i - r * D;
      float M = -INFINITY, l = 0.0f, v = 0.0f;
      for (int k = 0; k < nteam; ++k) M = fmaxf(M, s_m[k * team + r / kKdTile][r % kKdTile]);
      for (int k = 0; k < nteam; ++k) {
        const int x = k * team + r / kKdTile;
        const float mx = s_m[x][r % kKdTile];
        const float e = mx > -INFINITY ? exp2f(mx - M) : s_l[x][r % kKdTile] == 0.0f ? 0.0f : 1.0f;
        l += e * s_l[x][r % kKdTile];
        v += e * s_acc[(x * kKdTile + r % kKdTile) * D + c];
      }
      if (done) {
        if (r / a.G < nq) kd_store<D>(a, b, g, r, c, M, l, v);
      } else {
        if (c == 0) { part[r * (D + 2)] = M; part[r * (D + 2) + 1] = l; }
        part[r * (D + 2) + 2 + c] = v;
      }
    }
    u += cnt;
  }
}

// Joins the parts of the items that were cut: CTA j owns the item that holds
// the border between the runs of CTAs j and j + 1, if j is the first CTA of
// that item.
template <int D>
__global__ void __launch_bounds__(256) kv4_join_kernel(const Kv4DecodeArgs a, int ncta) {
  pdl_entry();
  __shared__ int64_t s_pref[kMaxB + 1];
  kd_prefix(a, s_pref);
  const int64_t total = s_pref[kMaxB], per = (total + ncta - 1) / ncta;
  const int64_t x = ((int64_t)blockIdx.x + 1) * per;
  if (x >= total) return;
  const int b = kd_find(s_pref, a.B, x);
  const int64_t n = kd_len(a, b), ub = kd_units(n), rem = x - s_pref[b];
  const int g = (int)(rem / ub);
  const int64_t first = s_pref[b] + g * ub, last = first + ub - 1;
  if (first == x || first / per != (int64_t)blockIdx.x) return;
  const int c0 = (int)blockIdx.x, c1 = (int)(last / per);
  const int R = a.T * a.G;
  const int64_t nq = kd_nq(a, b);
  const int64_t stride = (int64_t)R * (D + 2);
  const float* p0 = a.part + (2 * (int64_t)c0 + (first == c0 * per ? 0 : 1)) * stride;
  for (int i = threadIdx.x; i < R * D; i += 256) {
    const int r = i / D, c = i - r * D;
    if (r / a.G >= nq) continue;
    float M = -INFINITY, l = 0.0f, v = 0.0f;
    for (int k = c0; k <= c1; ++k) M = fmaxf(M, (k == c0 ? p0 : a.part + 2 * k * stride)[r * (D + 2)]);
    for (int k = c0; k <= c1; ++k) {
      const float* p = (k == c0 ? p0 : a.part + 2 * k * stride) + r * (D + 2);
      const float e = p[0] > -INFINITY ? exp2f(p[0] - M) : p[1] == 0.0f ? 0.0f : 1.0f;
      l += e * p[1];
      v += e * p[2 + c];
    }
    kd_store<D>(a, b, g, r, c, M, l, v);
  }
}

namespace {

// CTAs of the decode kernel: one per SM, no more than there can be units
int kd_ctas(const csa_shape* s) {
  const int64_t units = (int64_t)s->B * s->Hkv * ((s->n_max + kBlock - 1) / kBlock);
  const int nsm = sm_count();
  return (int)(units < nsm ? units : nsm);
}

size_t kd_workspace(const csa_shape* s, int T) {
  const int R = T * (s->Hq / s->Hkv);
  return 256 + (size_t)2 * kd_ctas(s) * R * (s->d + 2) * 4;
}

template <int D, typename E>
cudaError_t launch_kv4_decode(const Kv4DecodeArgs& a, int ncta, cudaStream_t st) {
  const int Rp = (a.T * a.G + kKdTile - 1) / kKdTile * kKdTile;
  const int smem = (Rp + kKdWarps * kKdTile) * D * 4;
  const cudaError_t e = cudaFuncSetAttribute(kv4_decode_kernel<D, E>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  launch_pdl(kv4_decode_kernel<D, E>, dim3(ncta), dim3(kKdWarps * 32), smem, st, a);
  if (ncta > 1) launch_pdl(kv4_join_kernel<D>, dim3(ncta - 1), dim3(256), 0, st, a, ncta);
  return cudaGetLastError();
}

bool kd_args_ok(const csa_shape* s, int T, csa_status* st) {
  if (!shape_ok(s) || T < 1) { *st = CSA_ERR_INVALID_ARG; return false; }
  *st = shape_supported(s);
  if (*st == CSA_OK && (T > CSA_KV4_MAX_T || T * (s->Hq / s->Hkv) > CSA_KV4_MAX_ROWS)) *st = CSA_ERR_UNSUPPORTED;
  return *st == CSA_OK;
}

}  // namespace
}  // namespace csa

using namespace csa;

extern "C" {

size_t csa_kv4_workspace_size(const csa_shape* shape, int T) {
  csa_status st;
  return kd_args_ok(shape, T, &st) ? kd_workspace(shape, T) : 0;
}

csa_status csa_kv4_decode(const csa_shape* shape, const csa_kv4* cache, int T, const void* q, const csa_strides* qs,
                          const int64_t* len, const int64_t* n_q, float* o, float* lse, void* workspace,
                          size_t workspace_bytes, void* stream) {
  csa_status su;
  if (!shape_ok(shape) || !kv4_cache_ok(cache) || T < 1 || !q || !len || !o) return CSA_ERR_INVALID_ARG;
  if (!kd_args_ok(shape, T, &su)) return su;
  const bool bf16 = shape->dtype == CSA_BF16;
  if (!strides_ok(qs, bf16 ? 8 : 4, shape->B, T, shape->Hq) || !aligned16(q) || !aligned16(o)) return CSA_ERR_INVALID_ARG;
  if (!workspace || workspace_bytes < kd_workspace(shape, T) || ((uintptr_t)workspace % 256)) return CSA_ERR_WORKSPACE;
  Kv4DecodeArgs a = {};
  a.c = *cache; a.q = q; a.qs = *qs; a.len = len; a.n_q = n_q; a.o = o; a.lse = lse;
  a.status = (unsigned*)workspace; a.part = (float*)((char*)workspace + 256);
  a.n_max = shape->n_max; a.nblk_max = (shape->n_max + kBlock - 1) / kBlock;
  a.B = shape->B; a.T = T; a.Hq = shape->Hq; a.Hkv = shape->Hkv; a.G = shape->Hq / shape->Hkv;
  a.rs = (float)(1.4426950408889634 / std::sqrt((double)shape->d));
  const int ncta = kd_ctas(shape);
  add_launches(ncta > 1 ? 2 : 1);
  cudaStream_t st = (cudaStream_t)stream;
  const cudaError_t e = shape->d == 128 ? (bf16 ? launch_kv4_decode<128, __nv_bfloat16>(a, ncta, st) : launch_kv4_decode<128, float>(a, ncta, st))
                                        : (bf16 ? launch_kv4_decode<64, __nv_bfloat16>(a, ncta, st) : launch_kv4_decode<64, float>(a, ncta, st));
  return e == cudaSuccess ? CSA_OK : CSA_ERR_CUDA;
}

}  // extern "C"
