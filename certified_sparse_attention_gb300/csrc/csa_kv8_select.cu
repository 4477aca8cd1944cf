// The choice of blocks by a cheap score (csa_kv8_select).
//
// A cluster of CTAs takes up to 16 query rows of one (sequence, KV head): the
// query heads of 16 / G tokens.  Scores are exact whole numbers before their two
// roundings:
//   I = sum_c q_c (q_c >= 0 ? hi_c : lo_c) = sum_c q+_c hi_c + sum_c q-_c lo_c,
// q+ and q- the positive and negative parts of the query's 8-bit codes: one
// product of 2 d channels, on the tensor cores in half precision (codes and their
// products are whole, sums stay below 2^24), 16 rows x 8 blocks x 16 channels an
// instruction.  The blocks' spans go from memory to the operands' registers, 16
// bytes a lane, each read once per cluster.  A token's scores are collected, as
// ordered integers, in the shared memory of one CTA of the cluster, which then
// finds the n_sel-th largest digit by digit and writes the blocks above it, and
// the first ones equal to it, in ascending order.
#include <cuda_fp16.h>

#include "csa_rows.cuh"

namespace csa {

struct Kv8SelectArgs {
  csa_kv8 c;
  const void* q;
  csa_strides qs;
  const int64_t* len;
  const int64_t* n_q;
  int32_t* blocks;
  int32_t* count;
  unsigned* status;
  int64_t n_max, nblk_max;
  int B, T, Hkv, G;
  int n_sel, n_first, n_last;
  int tokens;              // of a cluster
  int cluster;             // CTAs of a cluster
};

constexpr int kSelThreads = 256, kSelWarps = kSelThreads / 32;
constexpr int kSelRows = 16;
constexpr unsigned kSelForced = 0xFFFFFFFFu;      // above every score

__device__ __forceinline__ unsigned cluster_rank() {
  unsigned r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;\n" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;\n" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;\n" ::: "memory"); }
// store to the same place in the shared memory of CTA `rank` of the cluster
__device__ __forceinline__ void store_cluster(unsigned* p, unsigned rank, unsigned v) {
  unsigned at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("st.shared::cluster.u32 [%0], %1;\n" ::"r"(at), "r"(v) : "memory");
}
__device__ __forceinline__ void mma_rows(float (&d)[4], const unsigned (&a)[4], unsigned b0, unsigned b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ unsigned half2_bits(__half2 h) { return *reinterpret_cast<const unsigned*>(&h); }
// two of a word's four codes as half-precision numbers (a byte under the
// exponent of 1024, minus 1152)
__device__ __forceinline__ unsigned two_codes(unsigned word, int sel) {
  const unsigned u = __byte_perm(word, 0x64646464u, sel);
  return half2_bits(__hsub2(*reinterpret_cast<const __half2*>(&u),
                            __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480))));
}
// a score as an ordered integer; a NaN counts as +infinity, -0 as 0
__device__ __forceinline__ unsigned score_key(float s) { return ord_of(s == s ? s + 0.0f : INFINITY); }

// The n_sel largest of the keys [0, n), n > n_sel, equal ones from the lowest:
// their places to out, ascending.  By the whole CTA.
__device__ void select_keys(const unsigned* key, int n, int n_sel, int32_t* out) {
  __shared__ unsigned s_hist[256];
  __shared__ unsigned s_found[2];
  __shared__ int s_gt[kSelWarps], s_eq[kSelWarps];
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int end = (n + kSelThreads - 1) / kSelThreads * kSelThreads;
  unsigned prefix = 0, mask = 0;
  int need = n_sel;
  for (int shift = 24; shift >= 0; shift -= 8) {
    s_hist[tid] = 0;
    __syncthreads();
    for (int i = tid; i < end; i += kSelThreads) {
      // (neighbouring scores share their first digits: one addition for each
      // different digit of a warp)
      const bool in = i < n && (key[i] & mask) == prefix;
      const unsigned digit = in ? key[i] >> shift & 255u : 256u;
      const unsigned peers = __match_any_sync(0xffffffffu, digit);
      if (in && lane == __ffs(peers) - 1) atomicAdd(&s_hist[digit], __popc(peers));
    }
    __syncthreads();
    if (w == 0) {
      // the digit at which the keys from the largest down reach `need`
      unsigned h[8], sum = 0;
#pragma unroll
      for (int k = 0; k < 8; ++k) { h[k] = s_hist[255 - (lane * 8 + k)]; sum += h[k]; }
      unsigned upto = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned y = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += y;
      }
      unsigned above = upto - sum;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (above < (unsigned)need && above + h[k] >= (unsigned)need) {
          s_found[0] = 255 - (lane * 8 + k);
          s_found[1] = above;
        }
        above += h[k];
      }
    }
    __syncthreads();
    prefix |= s_found[0] << shift;
    mask |= 255u << shift;
    need -= (int)s_found[1];
    __syncthreads();
  }
  // keys above prefix, and the first `need` of those equal to it
  const int per = end / kSelWarps, i0 = w * per;
  int gt = 0, eq = 0;
  for (int i = i0 + lane; i < i0 + per; i += 32) {
    const unsigned k = i < n ? key[i] : 0u;
    gt += __popc(__ballot_sync(0xffffffffu, i < n && k > prefix));
    eq += __popc(__ballot_sync(0xffffffffu, i < n && k == prefix));
  }
  if (lane == 0) { s_gt[w] = gt; s_eq[w] = eq; }
  __syncthreads();
  gt = eq = 0;
  for (int i = 0; i < w; ++i) { gt += s_gt[i]; eq += s_eq[i]; }
  const unsigned below = (1u << lane) - 1u;
  for (int i = i0 + lane; i < i0 + per; i += 32) {
    const unsigned k = i < n ? key[i] : 0u;
    const bool isg = i < n && k > prefix, ise = i < n && k == prefix;
    const unsigned mg = __ballot_sync(0xffffffffu, isg), me = __ballot_sync(0xffffffffu, ise);
    const int before = eq + __popc(me & below);
    if (isg || (ise && before < need)) out[gt + __popc(mg & below) + min(before, need)] = i;
    gt += __popc(mg);
    eq += __popc(me);
  }
  __syncthreads();
}

template <int D, typename E>
__global__ void __launch_bounds__(kSelThreads) kv8_select_kernel(const Kv8SelectArgs a) {
  pdl_entry();
  constexpr int CPL = D / 32, KS = D / 64;
  typedef typename Row<CPL, E>::T RowT;
  __shared__ __align__(16) __half s_code[kSelRows][D + 8];
  __shared__ float s_step[kSelRows];
  extern __shared__ __align__(16) unsigned s_key[];     // [tokens of this CTA][nblk_max]
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5, gid = lane >> 2, tig = lane & 3;
  const int rank = a.cluster > 1 ? (int)cluster_rank() : 0;
  const int tile = blockIdx.x / a.cluster, g = blockIdx.y, b = blockIdx.z;
  if (a.status && blockIdx.x == 0 && g == 0 && b == 0 && w == 0) {
    bool bad = false;
    for (int i = lane; i < a.B; i += 32) {
      const int64_t n = a.len[i], m = a.n_q ? a.n_q[i] : a.T;
      bad |= n < 0 || n > a.n_max || m < 0 || m > a.T;
    }
    report_range(a.status, nullptr, bad);
  }
  // (what follows returns or goes on for a whole cluster)
  const int64_t n = a.len[b], m = a.n_q ? a.n_q[b] : (int64_t)a.T;
  if (n < 0 || n > a.n_max || m < 0 || m > a.T) return;
  const int t0 = tile * a.tokens, tokens = min((int)m - t0, a.tokens);
  if (tokens <= 0) return;
  const int64_t pos0 = n - m + t0, last = pos0 + tokens - 1;
  const int own = last < 0 ? -1 : (int)(last / kBlock);          // the last token's
  const int64_t bg = (int64_t)b * a.Hkv + g;
  if (own >= a.n_sel) {
    // blocks [0, own) are whole (and every token's own block is chosen anyway)
    if (a.cluster > 1) cluster_arrive();
    for (int r = w; r < kSelRows; r += kSelWarps) {
      const int t = r / a.G;
      float x[CPL], top = 0.0f;
#pragma unroll
      for (int c = 0; c < CPL; ++c) x[c] = 0.0f;
      if (t < tokens) {
        const E* src = reinterpret_cast<const E*>(a.q) + b * a.qs.b + (int64_t)(t0 + t) * a.qs.t +
                       (int64_t)(g * a.G + r % a.G) * a.qs.h + lane * CPL;
        row_floats<CPL>(*reinterpret_cast<const RowT*>(src), x, E());
      }
#pragma unroll
      for (int c = 0; c < CPL; ++c) top = max_nan(top, fabsf(x[c]));
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
      float step = fdiv(top, 127.0f);
      if (step == 0.0f) step = 1.0f;
#pragma unroll
      for (int c = 0; c < CPL; ++c) {
        const float y = rintf(fdiv(x[c], step));
        s_code[r][lane * CPL + c] = __float2half_rn(y == y ? fminf(fmaxf(y, -127.0f), 127.0f) : 0.0f);
      }
      if (lane == 0) s_step[r] = step;
    }
    __syncthreads();
    // operands: channels 64 h + 16 tig + 4 s + (0..3) of rows gid, gid + 8; the
    // positive parts against the upper ends, the negative ones against the lower
    unsigned qa[2][KS][4][4];
    const __half2 zero = __float2half2_rn(0.0f);
#pragma unroll
    for (int h = 0; h < KS; ++h)
#pragma unroll
      for (int s = 0; s < 4; ++s)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const __half2 c = *reinterpret_cast<const __half2*>(&s_code[gid + (e & 1) * 8][64 * h + 16 * tig + 4 * s + (e >> 1) * 2]);
          qa[0][h][s][e] = half2_bits(__hmax2(c, zero));
          qa[1][h][s][e] = half2_bits(__hmin2(c, zero));
        }
    const float step0 = s_step[gid], step1 = s_step[gid + 8];
    if (a.cluster > 1) cluster_wait();            // every CTA of the cluster has begun
    const uint8_t* span = a.c.span + bg * a.nblk_max * 2 * D + 16 * tig;
    const float2* scale = reinterpret_cast<const float2*>(a.c.scale) + bg * a.nblk_max;
    const int tok0 = gid / a.G, tok1 = (gid + 8) / a.G;
    const bool put0 = gid % a.G == 0 && tok0 < tokens, put1 = gid % a.G == 0 && tok1 < tokens;
    for (int j0 = (rank * kSelWarps + w) * 8; j0 < own; j0 += a.cluster * kSelWarps * 8) {
      const uint8_t* src = span + (int64_t)min(j0 + gid, own - 1) * 2 * D;
      uint4 k[2][KS];
#pragma unroll
      for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int h = 0; h < KS; ++h) k[p][h] = *reinterpret_cast<const uint4*>(src + p * D + 64 * h);
      const int ja = j0 + 2 * tig, jb = ja + 1;
      const float sa = scale[min(ja, own - 1)].x, sb = scale[min(jb, own - 1)].x;
      float x[2][4];
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        x[p][0] = x[p][1] = x[p][2] = x[p][3] = 0.0f;
#pragma unroll
        for (int h = 0; h < KS; ++h)
#pragma unroll
          for (int s = 0; s < 4; ++s) {
            const unsigned word = s == 0 ? k[p][h].x : s == 1 ? k[p][h].y : s == 2 ? k[p][h].z : k[p][h].w;
            mma_rows(x[p], qa[p][h][s], two_codes(word, 0x4140), two_codes(word, 0x4342));
          }
      }
      float v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = fmul(fmul(x[0][e] + x[1][e], e & 1 ? sb : sa), e < 2 ? step0 : step1);
      for (int o = 1; o < a.G; o <<= 1)
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = max_nan(v[e], __shfl_xor_sync(0xffffffffu, v[e], 4 * o));
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int j = e & 1 ? jb : ja, tok = e < 2 ? tok0 : tok1;
        if ((e < 2 ? put0 : put1) && j < own) {
          unsigned* at = s_key + (int64_t)(tok / a.cluster) * a.nblk_max + j;
          if (a.cluster > 1) store_cluster(at, tok % a.cluster, score_key(v[e]));
          else *at = score_key(v[e]);
        }
      }
    }
    if (a.cluster > 1) { cluster_arrive(); cluster_wait(); }
    else __syncthreads();
  }
  for (int tok = rank; tok < tokens; tok += a.cluster) {
    const int64_t pos = pos0 + tok, row = ((int64_t)b * a.T + t0 + tok) * a.Hkv + g;
    const int n_cand = pos < 0 ? 0 : (int)(pos / kBlock) + 1;
    int32_t* out = a.blocks + row * a.n_sel;
    if (tid == 0) a.count[row] = min(n_cand, a.n_sel);
    if (n_cand <= a.n_sel) {
      for (int i = tid; i < a.n_sel; i += kSelThreads) out[i] = i < n_cand ? i : -1;
    } else {
      unsigned* key = s_key + (int64_t)(tok / a.cluster) * a.nblk_max;
      for (int i = tid; i < a.n_first; i += kSelThreads) key[i] = kSelForced;
      for (int i = tid; i < a.n_last; i += kSelThreads) key[n_cand - 1 - i] = kSelForced;
      __syncthreads();
      select_keys(key, n_cand, a.n_sel, out);
    }
  }
}

namespace {

// shared memory for the scores of a CTA's tokens: one row of
// CSA_KV8_MAX_SELECT_TOKENS / 64 blocks at most, more rows of fewer
constexpr int kSelShared = CSA_KV8_MAX_SELECT_TOKENS / kBlock * 4;

template <int D, typename E>
cudaError_t launch_select(Kv8SelectArgs a, cudaStream_t st) {
  const int row = (int)a.nblk_max * 4;
  int tokens = kSelRows / a.G < a.T ? kSelRows / a.G : a.T, cluster = 1;
  // More CTAs to a cluster while the card has room for them and each of their
  // warps has blocks to score.
  while (cluster < 8 && a.nblk_max > 64 * cluster &&
         (int64_t)a.B * a.Hkv * ((a.T + tokens - 1) / tokens) * cluster <= sm_count())
    cluster *= 2;
  const int fit = kSelShared / row * cluster;
  if (tokens > fit) tokens = fit;
  a.tokens = tokens;
  a.cluster = cluster;
  cudaError_t e = cudaFuncSetAttribute(kv8_select_kernel<D, E>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSelShared);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((a.T + tokens - 1) / tokens * cluster, a.Hkv, a.B);
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = (size_t)((tokens + cluster - 1) / cluster) * row;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  e = cudaLaunchKernelEx(&cfg, kv8_select_kernel<D, E>, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace
}  // namespace csa

using namespace csa;

extern "C" {

csa_status csa_kv8_select(const csa_shape* shape, const csa_kv8* cache, int T, const void* q, const csa_strides* qs,
                          const int64_t* len, const int64_t* n_q, int n_sel, int n_first, int n_last, int32_t* blocks,
                          int32_t* count, uint32_t* status, void* stream) {
  if (!shape_ok(shape) || !kv8_cache_ok(cache) || T < 1 || !q || !len || !blocks || !count || n_sel < 1 || n_first < 0 ||
      n_last < 1 || n_first > n_sel - n_last || ((uintptr_t)blocks | (uintptr_t)count) % 4)
    return CSA_ERR_INVALID_ARG;
  const csa_status su = shape_supported(shape);
  if (su != CSA_OK) return su;
  const int G = shape->Hq / shape->Hkv;
  if (T > CSA_KV4_MAX_T || T * G > CSA_KV4_MAX_ROWS || n_sel > CSA_KV8_MAX_SEL || shape->n_max > CSA_KV8_MAX_SELECT_TOKENS)
    return CSA_ERR_UNSUPPORTED;
  const bool bf16 = shape->dtype == CSA_BF16;
  if (!strides_ok(qs, bf16 ? 8 : 4, shape->B, T, shape->Hq) || !aligned16(q)) return CSA_ERR_INVALID_ARG;
  Kv8SelectArgs a = {};
  a.c = *cache; a.q = q; a.qs = *qs; a.len = len; a.n_q = n_q; a.blocks = blocks; a.count = count; a.status = status;
  a.n_max = shape->n_max; a.nblk_max = (shape->n_max + kBlock - 1) / kBlock;
  a.B = shape->B; a.T = T; a.Hkv = shape->Hkv; a.G = G;
  a.n_sel = n_sel; a.n_first = n_first; a.n_last = n_last;
  add_launches(1);
  cudaStream_t st = (cudaStream_t)stream;
  const cudaError_t e = shape->d == 128 ? (bf16 ? launch_select<128, __nv_bfloat16>(a, st) : launch_select<128, float>(a, st))
                                        : (bf16 ? launch_select<64, __nv_bfloat16>(a, st) : launch_select<64, float>(a, st));
  return e == cudaSuccess ? CSA_OK : CSA_ERR_CUDA;
}

}  // extern "C"
