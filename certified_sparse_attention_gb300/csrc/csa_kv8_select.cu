// The choice of blocks by a cheap score (csa_kv8_select).
//
// A cluster of CTAs takes up to 8 query rows of one (sequence, KV head): the
// query heads of 8 / G tokens.  Scores are exact whole numbers before their two
// roundings:
//   I = sum_c q_c (q_c >= 0 ? hi_c : lo_c) = sum_c q+_c hi_c + sum_c q-_c lo_c,
// q+ and q- the positive and negative parts of the query's 8-bit codes: one
// product of 2 d channels, on the tensor cores in half precision, 16 blocks x 8 rows x
// 16 channels an instruction (with rows and blocks the other way round, half of each
// instruction idle, 4 x 128K tokens took 17 us, now 12).  The codes enter 1152 too
// large, which the sums of q+ and q- correct; each sum is over 64 channels, below
// 64 127 1279 < 2^24, so all of it is exact.  The blocks' spans go from memory to
// shared memory by bulk copies and from there to the operands' registers, 16 bytes
// a lane, each once per cluster.  A token's scores are collected, as ordered
// integers, in the shared memory of one CTA of the cluster, which then finds the
// n_sel-th largest by histograms and writes the blocks above it, and the first ones
// equal to it, in ascending order.
//
// d = 128, 32 / 8 heads: 64 sequences of 2K to 16K tokens 12.6 us, one of 1M 23.5:
// the latency of phases that depend on one another (query codes, operands, scores,
// ranking: about half of the last), not the 17 or 35 MB of spans.
#include <algorithm>

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
  int clog;                // log2 of the CTAs of a cluster
  int stages;              // chunks of spans in shared memory at once
  int chunk;               // blocks of a chunk
};

constexpr int kSelStages = 2;
constexpr int kSelRows = 8;       // query rows of a cluster at most

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
// two of a word's four codes as half-precision numbers 1152 larger: a byte under the
// exponent of 1024
__device__ __forceinline__ unsigned two_codes(unsigned word, int sel) { return __byte_perm(word, 0x64646464u, sel); }
// a score as an ordered integer; a NaN counts as +infinity, -0 as 0
__device__ __forceinline__ unsigned score_key(float s) { return ord_of(s == s ? s + 0.0f : INFINITY); }

// four bins to a thread
template <int NT> constexpr int kSelBinLog = NT == 256 ? 10 : 11;
template <int NT>
struct SelShared {
  uint4 hist[NT];                             // from the uppermost bins down
  unsigned lo[NT / 32], hi[NT / 32];
  unsigned sum[NT / 32];
  unsigned bin, above, count;
  int gt[NT / 32], eq[NT / 32];
};

// The n_sel best blocks of [0, n), n > n_sel: the first n_first, the last n_last and
// those of the largest keys, equal ones from the lowest; to out, ascending.  By the
// whole CTA of NT threads.  The keys' own range is cut into 4 NT bins (digits of the
// number would put most of them in a few, one addition after the other), the one at
// which they reach the number wanted is cut again, and so on: two times as a rule.
template <int NT>
__device__ void select_keys(SelShared<NT>& sh, const unsigned* key, int n, int n_sel, int n_first, int n_last, int32_t* out) {
  constexpr int NW = NT / 32, bins = 4 * NT, N = 8;
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  // N keys to a thread at a time: with one, a pass waited for shared memory once
  // for each
  const auto each = [&](int from, int to, const auto& f) {
    for (int i0 = from + tid; i0 < to; i0 += N * NT) {
      unsigned k[N];
#pragma unroll
      for (int j = 0; j < N; ++j) k[j] = i0 + j * NT < to ? key[i0 + j * NT] : 0u;
#pragma unroll
      for (int j = 0; j < N; ++j)
        if (i0 + j * NT < to) f(k[j]);
    }
  };
  const int end = n - n_last;                 // keys [n_first, end) compete
  unsigned need = n_sel - n_first - n_last;
  unsigned lo = 0xFFFFFFFFu, hi = 0u;
  each(n_first, end, [&](unsigned k) {
    lo = min(lo, k);
    hi = max(hi, k);
  });
  lo = __reduce_min_sync(0xffffffffu, lo);
  hi = __reduce_max_sync(0xffffffffu, hi);
  if (lane == 0) { sh.lo[w] = lo; sh.hi[w] = hi; }
  sh.hist[tid] = make_uint4(0u, 0u, 0u, 0u);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < NW; ++i) { lo = min(lo, sh.lo[i]); hi = max(hi, sh.hi[i]); }
  // keys of [lo, hi] are in play, those above are chosen; none is wanted of a range
  // if need is 0
  int shift = max(32 - __clz(hi - lo) - kSelBinLog<NT>, 0);
  while (need) {
    const unsigned span = hi - lo;
    unsigned* hist = reinterpret_cast<unsigned*>(sh.hist) + (bins - 1);
    each(n_first, end, [&](unsigned k) {
      const unsigned off = k - lo;
      if (k >= lo && off <= span) atomicAdd(hist - (int)(off >> shift), 1u);
    });
    __syncthreads();
    // the bin at which the keys from the largest down reach `need`
    const uint4 h4 = sh.hist[tid];
    sh.hist[tid] = make_uint4(0u, 0u, 0u, 0u);
    const unsigned h[4] = {h4.x, h4.y, h4.z, h4.w}, sum = h4.x + h4.y + h4.z + h4.w;
    unsigned upto = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned y = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += y;
    }
    if (lane == 31) sh.sum[w] = upto;
    __syncthreads();
    unsigned above = upto - sum;
#pragma unroll
    for (int i = 0; i < NW; ++i) above += i < w ? sh.sum[i] : 0u;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (above < need && above + h[k] >= need) {
        sh.bin = bins - 1 - (tid * 4 + k);
        sh.above = above;
        sh.count = h[k];
      }
      above += h[k];
    }
    __syncthreads();
    need -= sh.above;
    lo += sh.bin << shift;
    hi = min(hi, lo + ((1u << shift) - 1u));
    if (shift == 0 || sh.count == need) break;
    shift = max(shift - kSelBinLog<NT>, 0);
    // (what has been found is read by all before the next pass writes it)
    __syncthreads();
  }
  // keys above hi, and the first `need` of [lo, hi]
  constexpr int M = 4;
  const int per = (n + M * NT - 1) / (M * NT) * M * 32, i0 = w * per, i1 = min(i0 + per, n);
  const auto rank = [&](int i, unsigned k, bool& isg, bool& ise) {
    isg = i < n && (i < n_first || i >= end || k > hi);
    ise = i < n && !isg && need && k >= lo;
  };
  int gt = 0, eq = 0;
  for (int i = i0 + lane; i < i1 + lane; i += 32 * M) {
    unsigned k[M];
#pragma unroll
    for (int j = 0; j < M; ++j) k[j] = i + 32 * j < n ? key[i + 32 * j] : 0u;
#pragma unroll
    for (int j = 0; j < M; ++j) {
      bool isg, ise;
      rank(i + 32 * j, k[j], isg, ise);
      gt += __popc(__ballot_sync(0xffffffffu, isg));
      eq += __popc(__ballot_sync(0xffffffffu, ise));
    }
  }
  if (lane == 0) { sh.gt[w] = gt; sh.eq[w] = eq; }
  __syncthreads();
  gt = eq = 0;
#pragma unroll
  for (int i = 0; i < NW; ++i) {
    gt += i < w ? sh.gt[i] : 0;
    eq += i < w ? sh.eq[i] : 0;
  }
  const unsigned below = (1u << lane) - 1u;
  for (int i = i0 + lane; i < i1 + lane; i += 32 * M) {
    unsigned k[M];
#pragma unroll
    for (int j = 0; j < M; ++j) k[j] = i + 32 * j < n ? key[i + 32 * j] : 0u;
#pragma unroll
    for (int j = 0; j < M; ++j) {
      bool isg, ise;
      rank(i + 32 * j, k[j], isg, ise);
      const unsigned mg = __ballot_sync(0xffffffffu, isg), me = __ballot_sync(0xffffffffu, ise);
      const int before = eq + __popc(me & below);
      if (isg || (ise && before < (int)need)) out[gt + __popc(mg & below) + min(before, (int)need)] = i + 32 * j;
      gt += __popc(mg);
      eq += __popc(me);
    }
  }
  __syncthreads();
}

template <int D, int NT, typename E>
__global__ void __launch_bounds__(NT, NT == 256 ? 2 : 1) kv8_select_kernel(const Kv8SelectArgs a) {
  pdl_entry();
  constexpr int CPL = D / 32, KS = D / 64, NW = NT / 32;
  typedef typename Row<CPL, E>::T RowT;
  __shared__ __align__(16) __half s_code[kSelRows][D + 8];
  __shared__ float s_step[kSelRows], s_extra[kSelRows][2][KS];   // (1152 times the sums of q+, q- over 64 channels)
  __shared__ SelShared<NT> s_sel;
  __shared__ __align__(8) unsigned long long s_bar[2 * kSelStages];      // chunks full, empty
  extern __shared__ __align__(128) uint8_t s_dyn[];     // [stages] chunks, [tokens of this CTA][nblk_max] keys
  const unsigned chunk_bytes = a.chunk * 2 * D;
  unsigned* s_key = reinterpret_cast<unsigned*>(s_dyn + a.stages * chunk_bytes);
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5, gid = lane >> 2, tig = lane & 3;
  const int cluster = 1 << a.clog, rank = cluster > 1 ? (int)cluster_rank() : 0;
  const int tile = blockIdx.x >> a.clog, g = blockIdx.y, b = blockIdx.z;
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
  const int t0 = tile * a.tokens;
  // the rows' query elements: row r = w is head r % G of token t0 + r / G (sent for
  // before the lengths are known; tokens past T are not there)
  RowT raw = RowT();
  const int glog = 31 - __clz(a.G);
  if (w < kSelRows && (w >> glog) < a.tokens && t0 + (w >> glog) < a.T)
    raw = *reinterpret_cast<const RowT*>(reinterpret_cast<const E*>(a.q) + b * a.qs.b + (int64_t)(t0 + (w >> glog)) * a.qs.t +
                                         (int64_t)(g * a.G + (w & (a.G - 1))) * a.qs.h + lane * CPL);
  if (n < 0 || n > a.n_max || m < 0 || m > a.T) return;
  const int tokens = min((int)m - t0, a.tokens);
  if (tokens <= 0) return;
  const int64_t pos0 = n - m + t0, last = pos0 + tokens - 1;
  const int own = last < 0 ? -1 : (int)(last / kBlock);          // the last token's
  const int64_t bg = (int64_t)b * a.Hkv + g;
  if (own >= a.n_sel) {
    // blocks [0, own) are whole (and every token's own block is chosen anyway)
    if (cluster > 1) cluster_arrive();
    // chunks rank, rank + cluster, ... of the blocks are this CTA's, sixteen blocks
    // of each a warp's
    const uint8_t* span = a.c.span + bg * a.nblk_max * 2 * D;
    const float2* scale = reinterpret_cast<const float2*>(a.c.scale) + bg * a.nblk_max;
    const int chunks = ((own + a.chunk - 1) / a.chunk - rank + cluster - 1) >> a.clog;
    const unsigned full = smem_u32(s_bar), empty = full + 8 * kSelStages, data = smem_u32(s_dyn);
    bool dead = false;
    const auto send = [&](int c, int stage) {
      const int j = (rank + (c << a.clog)) * a.chunk;
      const unsigned size = (unsigned)min(a.chunk, own - j) * 2 * D;
      mbar_expect_tx(full + 8 * stage, size);
      asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n" ::"r"(
                       data + stage * chunk_bytes),
                   "l"(span + (int64_t)j * 2 * D), "r"(size), "r"(full + 8 * stage)
                   : "memory");
    };
    if (tid == 0) {
      for (int i = 0; i < a.stages; ++i) {
        mbar_init(full + 8 * i, 1);
        mbar_init(empty + 8 * i, NW);
      }
      fence_barrier_init();
      for (int c = 0; c < min(chunks, a.stages); ++c) send(c, c);
    }
    // the steps of the lane's two blocks of a chunk, sent for a chunk ahead
    const auto step_of = [&](int c, int e) {
      return scale[min((rank + (c << a.clog)) * a.chunk + w * 16 + gid + 8 * e, own - 1)].x;
    };
    float next_a = step_of(0, 0), next_b = step_of(0, 1);
    if (w < kSelRows) {
      const int r = w;
      float x[CPL], top = 0.0f;
      row_floats<CPL>(raw, x, E());
#pragma unroll
      for (int c = 0; c < CPL; ++c) top = max_nan(top, fabsf(x[c]));
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
      float step = fdiv(top, 127.0f);
      if (step == 0.0f) step = 1.0f;
      float plus = 0.0f, minus = 0.0f;
#pragma unroll
      for (int c = 0; c < CPL; ++c) {
        float y = rintf(fdiv(x[c], step));
        y = y == y ? fminf(fmaxf(y, -127.0f), 127.0f) : 0.0f;
        s_code[r][lane * CPL + c] = __float2half_rn(y);
        plus += fmaxf(y, 0.0f);
        minus += fminf(y, 0.0f);
      }
#pragma unroll
      for (int o = 1; o < 32 / KS; o <<= 1) {
        plus += __shfl_xor_sync(0xffffffffu, plus, o);
        minus += __shfl_xor_sync(0xffffffffu, minus, o);
      }
      if (lane % (32 / KS) == 0) {
        s_extra[r][0][lane / (32 / KS)] = 1152.0f * plus;
        s_extra[r][1][lane / (32 / KS)] = 1152.0f * minus;
      }
      if (lane == 0) s_step[r] = step;
    }
    __syncthreads();
    // operands: channels 64 h + 16 tig + 4 s + (0..3) of row gid; the positive parts
    // against the upper ends, the negative ones against the lower
    unsigned qb[2][KS][4][2];
    const __half2 zero = __float2half2_rn(0.0f);
#pragma unroll
    for (int h = 0; h < KS; ++h)
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const uint2 u = *reinterpret_cast<const uint2*>(&s_code[gid][64 * h + 16 * tig + 4 * s]);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const unsigned x = e ? u.y : u.x;
          const __half2 c = *reinterpret_cast<const __half2*>(&x);
          qb[0][h][s][e] = half2_bits(__hmax2(c, zero));
          qb[1][h][s][e] = half2_bits(__hmin2(c, zero));
        }
      }
    // the lane's scores are of the rows 2 tig, 2 tig + 1
    float extra[2][2][KS], row_step[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      row_step[e] = s_step[2 * tig + e];
#pragma unroll
      for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int h = 0; h < KS; ++h) extra[e][p][h] = s_extra[2 * tig + e][p][h];
    }
    if (cluster > 1) cluster_wait();            // every CTA of the cluster has begun
    int stage = 0, phase = 0, before = 0;         // of the chunk, and the stage of the one before
    for (int c = 0; c < chunks; ++c) {
      const int j0 = (rank + (c << a.clog)) * a.chunk + w * 16;
      if (tid == 0 && c > 0 && c - 1 + a.stages < chunks) {
        // the chunk before has been read
        if (!mbar_wait(empty + 8 * before, stage ? phase : phase ^ 1)) dead = true;
        send(c - 1 + a.stages, before);
      }
      const float fa = next_a, fb = next_b;
      next_a = step_of(c + 1, 0);
      next_b = step_of(c + 1, 1);
      __syncwarp();
      if (!mbar_wait(full + 8 * stage, phase)) dead = true;
      if (w * 16 < a.chunk && j0 < own) {
        const uint8_t* src = s_dyn + stage * chunk_bytes + (w * 16 + gid) * 2 * D + 16 * tig;
        float x[2][KS][4];
#pragma unroll
        for (int h = 0; h < KS; ++h)
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            const uint4 k0 = *reinterpret_cast<const uint4*>(src + p * D + 64 * h), k1 = *reinterpret_cast<const uint4*>(src + 16 * D + p * D + 64 * h);
            x[p][h][0] = x[p][h][1] = x[p][h][2] = x[p][h][3] = 0.0f;
#pragma unroll
            for (int s = 0; s < 4; ++s) {
              const unsigned w0 = s == 0 ? k0.x : s == 1 ? k0.y : s == 2 ? k0.z : k0.w, w1 = s == 0 ? k1.x : s == 1 ? k1.y : s == 2 ? k1.z : k1.w;
              const unsigned op[4] = {two_codes(w0, 0x4140), two_codes(w1, 0x4140), two_codes(w0, 0x4342), two_codes(w1, 0x4342)};
              mma_rows(x[p][h], op, qb[p][h][s][0], qb[p][h][s][1]);
            }
          }
        // v[e]: block gid (+ 8 with e / 2), row 2 tig + e % 2
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float sum = 0.0f;
#pragma unroll
          for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int h = 0; h < KS; ++h) sum += x[p][h][e] - extra[e & 1][p][h];
          v[e] = fmul(fmul(sum, e < 2 ? fa : fb), row_step[e & 1]);
        }
        // the largest over a token's rows
        if (a.G >= 2) {
          v[0] = max_nan(v[0], v[1]);
          v[2] = max_nan(v[2], v[3]);
          for (int o = 1; 2 * o < a.G; o <<= 1) {
            v[0] = max_nan(v[0], __shfl_xor_sync(0xffffffffu, v[0], o));
            v[2] = max_nan(v[2], __shfl_xor_sync(0xffffffffu, v[2], o));
          }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int j = j0 + gid + (e & 2) * 4, r = 2 * tig + (e & 1), tok = r >> glog;
          if ((r & (a.G - 1)) == 0 && tok < tokens && j < own) {
            unsigned* at = s_key + (int64_t)(tok >> a.clog) * a.nblk_max + j;
            if (cluster > 1) store_cluster(at, tok & (cluster - 1), score_key(v[e]));
            else *at = score_key(v[e]);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(empty + 8 * stage);
      before = stage;
      if (++stage == a.stages) { stage = 0; phase ^= 1; }
    }
    // (each wait is bounded; what was sent for has landed when the last chunk's has
    // been waited for, or is waited for here)
    if (dead) {
      for (int i = 0; i < 2 * a.stages; ++i) mbar_wait(full + 8 * (i >> 1), i & 1);
      if (a.status) atomicOr(a.status, 4u);
    }
    if (cluster > 1) { cluster_arrive(); cluster_wait(); }
    else __syncthreads();
  }
  for (int tok = rank; tok < tokens; tok += cluster) {
    const int64_t pos = pos0 + tok, row = ((int64_t)b * a.T + t0 + tok) * a.Hkv + g;
    const int n_cand = pos < 0 ? 0 : (int)(pos / kBlock) + 1;
    int32_t* out = a.blocks + row * a.n_sel;
    if (tid == 0) a.count[row] = min(n_cand, a.n_sel);
    if (n_cand <= a.n_sel) {
      for (int i = tid; i < a.n_sel; i += NT) out[i] = i < n_cand ? i : -1;
    } else {
      select_keys<NT>(s_sel, s_key + (int64_t)(tok >> a.clog) * a.nblk_max, n_cand, a.n_sel, a.n_first, a.n_last, out);
    }
  }
}

namespace {

// dynamic shared memory there can be: the scores of one token of
// CSA_KV8_MAX_SELECT_TOKENS / 64 blocks, or of more tokens of fewer, and a chunk of 64
// spans
constexpr int kSelShared = CSA_KV8_MAX_SELECT_TOKENS / kBlock * 4 + 64 * 2 * 128;

template <int D, int NT, typename E>
cudaError_t launch_select_t(const Kv8SelectArgs& a, size_t smem, cudaStream_t st) {
  const int cluster = 1 << a.clog;
  cudaError_t e = cudaFuncSetAttribute(kv8_select_kernel<D, NT, E>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSelShared);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((a.T + a.tokens - 1) / a.tokens * cluster, a.Hkv, a.B);
  cfg.blockDim = dim3(NT);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  e = cudaLaunchKernelEx(&cfg, kv8_select_kernel<D, NT, E>, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}
template <int D, typename E>
cudaError_t launch_select(Kv8SelectArgs a, cudaStream_t st) {
  int tokens = kSelRows / a.G < a.T ? kSelRows / a.G : a.T, cluster = 1, clog = 0;
  // More CTAs to a cluster while the card has room for them and each of their
  // warps has blocks to score.
  const int64_t tiles = (int64_t)a.B * a.Hkv * ((a.T + tokens - 1) / tokens);
  while (cluster < 8 && a.nblk_max > 64 * cluster && tiles * cluster <= sm_count()) {
    cluster *= 2;
    ++clog;
  }
  // room for a chunk of 64 blocks and the tokens' scores
  constexpr int64_t least = 64 * 2 * D;
  const int64_t fit = (kSelShared - least) / (a.nblk_max * 4) * cluster;
  if (tokens > fit) tokens = (int)fit;
  const int64_t rows = (tokens + cluster - 1) / cluster * a.nblk_max * 4;
  // Sixteen warps to a CTA where the context is long and there are CTAs for half
  // of the SMs at most (clusters of eight lie within groups of SMs, and a card full
  // of them, one CTA to an SM, takes two rounds); all of them at work where there is
  // room for their chunk.  Sixteen / eight, us: 1 sequence of 128K tokens 8.4 / 8.1,
  // 256K 10.5 / 11.8, 1M 24 / 33; 2 sequences (a full card) 128K 12 / 9, 256K 16 / 13.
  const bool wide = 2 * tiles * cluster <= sm_count() && a.nblk_max >= 4096 && rows + 4 * least <= kSelShared;
  a.tokens = tokens;
  a.clog = clog;
  a.chunk = wide ? 256 : rows + 2 * least <= kSelShared ? 128 : 64;
  const int64_t chunks = (a.nblk_max + a.chunk * cluster - 1) / (a.chunk * cluster);
  a.stages = (int)std::min(std::min((int64_t)kSelStages, chunks), (kSelShared - rows) / (a.chunk * 2 * D));
  const size_t smem = (size_t)(rows + a.stages * a.chunk * 2 * D);
  return wide ? launch_select_t<D, 512, E>(a, smem, st) : launch_select_t<D, 256, E>(a, smem, st);
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
