// Decode attention over the 8-bit K/V cache, over all of it (csa_kv8_decode) or
// over listed blocks (csa_kv8_decode_blocks):
//   o = softmax(q K^T / sqrt d) V
// for the last T tokens of every sequence, K and V the values the cache
// stands for (whole blocks of 64 tokens in codes, the incomplete last block
// in full precision).
//
// Work is dealt to the CTAs in equal runs of units of about one block (KdBatch),
// whatever the lengths, which are read on the device; a CTA walks its run item by
// item, its warps take the blocks in turn, each with its own running maximum and
// sums, and merge them in shared memory.  Items that were cut are joined by a
// second kernel; few small ones are shared by clusters of CTAs instead, which join
// their sums in shared memory (k8_clog).  An item is a sequence and KV head with its
// T * G query rows; over lists, where each token has blocks of its own, a token's G.
//
// A warp handles one tile of 8 rows, or two; with more the warps of a CTA form teams
// that share the blocks.  Codes become half-precision numbers exactly (a
// byte under the exponent of 1024, minus 1152), the other operand is split into
// two half-precision parts: the 16 rows of a matrix instruction (m16n8k16) are
// the high parts of the 8 query rows, or weights, and their low parts, 2^12
// larger, so that float32 accuracy costs no more instructions than a single part
// would.  The layouts of K8 and V8 are the instruction's operand orders: lane (gid
// = lane / 4, tid = lane % 4) reads 16 consecutive bytes, lanes side by side,
// and holds the scores of the tokens 16 tid .. 16 tid + 15 of row gid, which are
// its weights' places in the second product: nothing is exchanged between lanes
// but a row's maximum.
//
// Matrix instructions truncate their sums: a block's sums start from zero and are
// added to the running ones in float32, where the values' step comes in.  Weights
// are relative to the block's own maximum, so that their parts' floor is 2^-37 of
// that whatever came before.
//
// Each warp has a slot of shared memory for a block's keys and one for its values
// (a team shares its two).  As it is done with one it sends for the next block's
// itself, a bulk copy that completes on an mbarrier, into the next item too.  Two
// further warps fetch the next items' queries and merge the sums of those done with;
// the run's first queries and last sums are all warps' work.
//
// What bounds it, bf16, d = 128: with one tile of rows and long contexts memory (4 x
// 128K tokens, 32 / 8 heads: 1.07 GB in 166 us, 6.5 TB/s); with many items also an
// item's start and end, 1.5 to 3 us of a CTA beside 0.36 us a block (64 sequences of
// 1K to 8K tokens, 64 / 8 heads: 115 us, 5.5 TB/s; 128 of 960: 54 us); with more
// tiles the latency of the warps, whose issue slots and tensor pipe are a third
// busy (8 sequences of up to 20000 tokens, 24 rows: 104 us, 2.1 TB/s); short ones
// the chain of lengths, queries, a round of blocks and the merges (1000
// tokens, 32 / 8 heads: 8.2 us).  A warp that sends for all (218 us for 4 x 128K),
// three slots a warp (188) and two blocks ahead were slower.
#include <algorithm>
#include <cmath>

#include "csa_decode.cuh"

namespace csa {

// W: consumer warps of a CTA, MT: tiles of 8 rows to each
constexpr int kK8Warps = 10;      // W for one tile of rows
constexpr int kK8Side = 2;        // ... and warps that fetch the queries and merge the sums
// (MT = 2: and two that only fill a warpgroup, from which registers move to the
// consumers': the launch has 168 a thread)
template <int W, int MT> constexpr int kK8Threads = (W + kK8Side * MT) * 32;
constexpr int kK8RegsConsumer = 208, kK8RegsSide = 88;
static_assert(2 * kK8RegsConsumer + kK8RegsSide <= 3 * 168, "more registers than the launch has");
constexpr int kK8Items = 3;       // items whose queries are there at once
// high parts of x and y, and what is left of them in units of 2^-12
__device__ __forceinline__ void k8_parts(float x, float y, unsigned& hi, unsigned& lo) {
  hi = half_pair(x, y);
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hi));
  lo = half_pair((x - f.x) * 4096.0f, (y - f.y) * 4096.0f);
}

template <bool LIST>
struct Kv8DecodeArgs : DecodeArgs {
  csa_kv8 c;
  const int32_t* blocks;  // LIST: [B][T][Hkv][n_sel], count [B][T][Hkv]
  const int32_t* count;
  int n_sel;
  int clog;               // whole: log2 of the CTAs that share an item
  // Fitted to the times of single CTAs (batch of 64, 8 query heads to a KV head: a
  // block 0.355 us, an item 1.5 to 3 us, its incomplete block 1.5 us).  Leads of 5
  // and of 12 take the same time there; 128 sequences of up to 2000 tokens take 101,
  // 94 and 92 us with 5, 8 and 12, one CTA's worth of drafts 115, 116 and 118.
  static constexpr int kLead = 8, kTailBase = 4, kTailStep = 64;
  static constexpr bool kPerToken = LIST, kPlainQ = true, kTop = false;
  static constexpr int kMaxCtas = 256;     // one per SM
  // Query rows as the matrix instructions' operand: of each tile of 8 rows, the
  // channels 64 h + 16 tid + 4 s + (0..3) of row gid are 16 bytes, (h, s, lane) in
  // that order: high parts of the first two, their low parts, the same of the others.
  template <int D>
  static __device__ __forceinline__ void put(float* q, int r, int lane, const float (&x)[D / 32], float up) {
    const int c = lane * (D / 32);
    unsigned* at = reinterpret_cast<unsigned*>(q + (r & ~7) * D) + ((c / 64 * 4 + c % 16 / 4) * 32 + (r & 7) * 4 + c % 64 / 16) * 4 + c % 4;
#pragma unroll
    for (int i = 0; i < D / 32; i += 2) {
      unsigned hi, lo;
      k8_parts(x[i] * up, x[i + 1] * up, hi, lo);
      *reinterpret_cast<uint2*>(at + i) = make_uint2(hi, lo);
    }
  }
};

// ------------------------------------------------------ tensor-core blocks

constexpr float kLowUnit = 0x1p-12f;     // what a low part's unit stands for

// codes of four bytes as two pairs of half-precision numbers
__device__ __forceinline__ void k8_numbers(unsigned word, unsigned& b0, unsigned& b1) {
  const __half2 off = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));     // 1152
  const unsigned u0 = __byte_perm(word, 0x64646464u, 0x4140), u1 = __byte_perm(word, 0x64646464u, 0x4342);
  const __half2 h0 = __hsub2(*reinterpret_cast<const __half2*>(&u0), off), h1 = __hsub2(*reinterpret_cast<const __half2*>(&u1), off);
  b0 = *reinterpret_cast<const unsigned*>(&h0);
  b1 = *reinterpret_cast<const unsigned*>(&h1);
}
__device__ __forceinline__ unsigned word_of(const uint4& v, int s) { return s == 0 ? v.x : s == 1 ? v.y : s == 2 ? v.z : v.w; }

// The state of a warp over the blocks of an item; the lane's row is gid.
template <int D>
struct K8Fast {
  float inv;                   // undoes the row's scale
  float r;                     // reference of the sums: the running maximum, or up to 8 below it
  float l;                     // sum of the lane's own tokens' weights
  float o[D / 8][2];           // channels 8 i + 2 tid, + 1
};

// What a row takes from a block whose scores are up to `top` in this lane: ref is
// the row's largest, share = 2^(ref - f.r), both 0 where it sees nothing of the
// block (and takes nothing from it, whatever the block's step).
struct K8Share {
  float ref, share;
  bool seen;
};
template <int D>
__device__ __forceinline__ K8Share k8_share(K8Fast<D>& f, float top) {
  top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
  // The sums' reference moves only when a block's maximum exceeds it by more
  // than 8 (weights up to 2^8).
  if (__builtin_expect(__any_sync(0xffffffffu, top > f.r + 8.0f), 0)) {
    const float r = top > f.r + 8.0f ? top : f.r, e = r == f.r ? 1.0f : ex2(f.r - r);
    f.r = r;
    f.l *= e;
#pragma unroll
    for (int i = 0; i < D / 8; ++i) { f.o[i][0] *= e; f.o[i][1] *= e; }
  }
  K8Share s;
  s.seen = top > -INFINITY;
  s.ref = s.seen ? top : 0.0f;
  s.share = s.seen ? ex2(top - f.r) : 0.0f;
  return s;
}

// One block for MT tiles of rows, whose codes are converted once: query operands at
// qa (put; the lane's), 2 D apart, keys at kt, values at vt, steps ks and vs;
// between() is called when the keys have been read and before the values are.  The
// lane's rows see the block's tokens below end; masked: some row does not see all of
// them.
template <int D, int MT, typename Between>
__device__ __forceinline__ void k8_block(K8Fast<D> (&f)[MT], const uint4* qa, const uint8_t* kt, const uint8_t* vt, float ks, float vs,
                                         bool masked, const int (&end)[MT], Between between) {
  const int lane = threadIdx.x & 31, tid = lane & 3;
  float x[MT][8][4];
#pragma unroll
  for (int t = 0; t < MT; ++t)
#pragma unroll
    for (int j = 0; j < 8; ++j) x[t][j][0] = x[t][j][1] = x[t][j][2] = x[t][j][3] = 0.0f;
#pragma unroll 1
  for (int h = 0; h < D / 64; ++h) {
    uint4 q[MT][4];
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int s = 0; s < 4; ++s) q[t][s] = qa[2 * D * t + (h * 4 + s) * 32];
#pragma unroll
    for (int j0 = 0; j0 < 8; j0 += 4) {
      uint4 k[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) k[j] = *reinterpret_cast<const uint4*>(kt + ((j0 + j) * (D / 64) + h) * 512 + lane * 16);
#pragma unroll
      for (int s = 0; s < 4; ++s)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          unsigned b0, b1;
          k8_numbers(word_of(k[j], s), b0, b1);
#pragma unroll
          for (int t = 0; t < MT; ++t) mma_f16(x[t][j0 + j], q[t][s].x, q[t][s].y, q[t][s].z, q[t][s].w, b0, b1);
        }
    }
  }
  between();
  unsigned p[MT][4][4];
  float weight[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    // scores: x[t][j][e] of token 16 tid + 2 j + e
    const float unit = ks * f[t].inv;
    float top = -INFINITY, top1 = -INFINITY;
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int e = 0; e < 2; ++e) x[t][j][e] = fmaf(x[t][j][e + 2], kLowUnit, x[t][j][e]) * unit;
    if (__builtin_expect(masked, 0)) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          if (16 * tid + 2 * j + e >= end[t]) x[t][j][e] = -INFINITY;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) { top = fmaxf(top, x[t][j][0]); top1 = fmaxf(top1, x[t][j][1]); }
    const K8Share sh = k8_share<D>(f[t], fmaxf(top, top1));
    weight[t] = sh.seen ? sh.share * vs : 0.0f;
    float sum = 0.0f, sum1 = 0.0f;
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const float pa = ex2(x[t][2 * s + u][0] - sh.ref), pb = ex2(x[t][2 * s + u][1] - sh.ref);
        sum += pa;
        sum1 += pb;
        k8_parts(pa, pb, p[t][s][2 * u], p[t][s][2 * u + 1]);
      }
    f[t].l = fmaf(sum + sum1, sh.share, f[t].l);
  }
  constexpr int N = 4 / MT;              // n-tiles of channels at a time
#pragma unroll
  for (int i0 = 0; i0 < D / 8; i0 += N) {
    uint4 v[N];
    float y[MT][N][4];
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = *reinterpret_cast<const uint4*>(vt + (i0 + i) * 512 + lane * 16);
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int i = 0; i < N; ++i) {
        unsigned b0, b1;
        k8_numbers(word_of(v[i], s), b0, b1);
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          if (s == 0) mma_f16_first(y[t][i], p[t][s][0], p[t][s][1], p[t][s][2], p[t][s][3], b0, b1);
          else mma_f16(y[t][i], p[t][s][0], p[t][s][1], p[t][s][2], p[t][s][3], b0, b1);
        }
      }
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int i = 0; i < N; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          f[t].o[i0 + i][e] = fmaf(fmaf(y[t][i][e + 2], kLowUnit, y[t][i][e]), weight[t], f[t].o[i0 + i][e]);
  }
}

// ---------------------------------------------------- the incomplete block

__device__ __forceinline__ void mma_bf16(float (&d)[4], unsigned a0, unsigned a1, unsigned a2, unsigned a3, unsigned b0,
                                         unsigned b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ unsigned bf16_pair(float x, float y) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
  return *reinterpret_cast<const unsigned*>(&h);
}
__device__ __forceinline__ float bf16_low(unsigned u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf16_high(unsigned u) { return __uint_as_float(u & 0xFFFF0000u); }
// x and y as N bf16 parts each: the rounded pair, the rounded remainders, ...
template <int N>
__device__ __forceinline__ void bf16_parts(float x, float y, unsigned (&p)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    p[i] = bf16_pair(x, y);
    if (i + 1 < N) { x -= bf16_low(p[i]); y -= bf16_high(p[i]); }
  }
}
// two channels of a row
template <typename E> struct PairOf { typedef unsigned T; };
template <> struct PairOf<float> { typedef float2 T; };
__device__ __forceinline__ float2 pair_of(const __nv_bfloat16* p) {
  const unsigned u = *reinterpret_cast<const unsigned*>(p);
  return make_float2(bf16_low(u), bf16_high(u));
}
__device__ __forceinline__ float2 pair_of(const float* p) { return *reinterpret_cast<const float2*>(p); }
// four channels
__device__ __forceinline__ float4 four_of(const __nv_bfloat16* p) { return Elem<__nv_bfloat16>::get4(p); }
__device__ __forceinline__ float4 four_of(const float* p) { return Elem<float>::get4(p); }
// infinities, NaNs and float32 numbers that bf16 rounds to infinity
__device__ __forceinline__ bool odd_number(float x) { return !(fabsf(x) < 0x1.FFp127f); }

constexpr int kK8Few = 8;         // tokens of the incomplete block at a time
// Scores of up to eight tokens at K, channel by channel: the lane's row with tokens
// 2 tid, 2 tid + 1.  (Not inline: its registers would cost float32 drafts of 20 rows 1.0
// of 68 us, the call costs 0.4.)
template <int D, typename E>
__device__ __noinline__ float2 k8_scores(const uint4* qa, const E* K, int tokens, float inv) {
  const int tid = threadIdx.x & 3;
  float2 out = make_float2(0.0f, 0.0f);
#pragma unroll 1
  for (int t = 0; t < tokens; ++t) {
    float s = 0.0f;
#pragma unroll 1
    for (int c = 0; c < D / 16; ++c) {
      const uint4 q = qa[c * 32];
      const float4 k = four_of(K + t * D + 64 * (c / 4) + 16 * tid + 4 * (c % 4));
      const float2 x0 = __half22float2(*reinterpret_cast<const __half2*>(&q.x)), y0 = __half22float2(*reinterpret_cast<const __half2*>(&q.y));
      const float2 x1 = __half22float2(*reinterpret_cast<const __half2*>(&q.z)), y1 = __half22float2(*reinterpret_cast<const __half2*>(&q.w));
      s = fmaf(fmaf(y0.x, kLowUnit, x0.x) * inv, k.x, s);
      s = fmaf(fmaf(y0.y, kLowUnit, x0.y) * inv, k.y, s);
      s = fmaf(fmaf(y1.x, kLowUnit, x1.x) * inv, k.z, s);
      s = fmaf(fmaf(y1.y, kLowUnit, x1.y) * inv, k.w, s);
    }
    s += __shfl_xor_sync(0xffffffffu, s, 1);
    s += __shfl_xor_sync(0xffffffffu, s, 2);
    if (t == 2 * tid) out.x = s;
    if (t == 2 * tid + 1) out.y = s;
  }
  return out;
}

// Eight tokens of the incomplete block at K, V, `left` of them there, of which the
// lane's row sees those below end; on the tensor cores too.  Keys and queries are
// split into bf16 parts (a bf16 number is one; float32 ones are three, whose
// products are all summed), weights into three: the instruction's 16 rows are
// the high and middle parts, and the low ones stand in its second eight tokens,
// which are the first ones again.
template <int D, typename E>
__device__ __forceinline__ void k8_rows(K8Fast<D>& f, const uint4* qa, const E* K, const E* V, int left, int end) {
  constexpr int N = sizeof(E) == 2 ? 1 : 3;
  const int lane = threadIdx.x & 31, gid = lane >> 2, tid = lane & 3;
  const bool in = gid < left;
  const E* kr = K + gid * D + 16 * tid;
  const E* vr = V + gid * D + 2 * tid;
  typename PairOf<E>::T vraw[D / 8];       // (on their way while the scores are made)
#pragma unroll
  for (int i = 0; i < D / 8; ++i) vraw[i] = in ? *reinterpret_cast<const typename PairOf<E>::T*>(vr + 8 * i) : typename PairOf<E>::T();
  float s4[2][4] = {{0.0f, 0.0f, 0.0f, 0.0f}, {0.0f, 0.0f, 0.0f, 0.0f}};      // (two sums in turn: less to wait for)
#pragma unroll
  for (int h = 0; h < D / 64; ++h)
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      float(&s)[4] = s4[c & 1];
      const uint4 q = qa[(h * 4 + c) * 32];
      const float4 k = in ? four_of(kr + 64 * h + 4 * c) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      unsigned a[2][N], b[2][N];
      bf16_parts<N>(k.x, k.y, b[0]);
      bf16_parts<N>(k.z, k.w, b[1]);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const unsigned hi = e ? q.z : q.x, lo = e ? q.w : q.y;
        const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&hi)), y = __half22float2(*reinterpret_cast<const __half2*>(&lo));
        bf16_parts<N>(fmaf(y.x, kLowUnit, x.x), fmaf(y.y, kLowUnit, x.y), a[e]);
      }
#pragma unroll
      for (int i = N - 1; i >= 0; --i) {
        mma_bf16(s, a[0][0], N > 1 ? a[0][N / 2] : 0u, a[1][0], N > 1 ? a[1][N / 2] : 0u, b[0][i], b[1][i]);
        if (N > 1) mma_bf16(s, a[0][N - 1], 0u, a[1][N - 1], 0u, b[0][i], b[1][i]);
      }
    }
  float sa = (s4[0][0] + s4[1][0] + (s4[0][2] + s4[1][2])) * f.inv, sb = (s4[0][1] + s4[1][1] + (s4[0][3] + s4[1][3])) * f.inv;
  // An infinite key (or one that bf16 rounds to infinity) has met zeros, the rows that
  // are not there or other parts, and made NaNs of its token's scores: those are taken
  // again, channel by channel
  if (__builtin_expect(__any_sync(0xffffffffu, odd_number(sa) || odd_number(sb)), 0)) {
    const float2 s = k8_scores<D, E>(qa, K, min(left, kK8Few), f.inv);
    if (odd_number(sa)) sa = s.x;
    if (odd_number(sb)) sb = s.y;
  }
  if (2 * tid >= end) sa = -INFINITY;
  if (2 * tid + 1 >= end) sb = -INFINITY;
  const K8Share sh = k8_share<D>(f, fmaxf(sa, sb));
  const float pa = ex2(sa - sh.ref), pb = ex2(sb - sh.ref);
  f.l = fmaf(pa + pb, sh.share, f.l);
  unsigned p[3];
  bf16_parts<3>(pa, pb, p);
  bool odd = false;
#pragma unroll
  for (int i = 0; i < D / 8; ++i) {
    const float2 v = pair_of(reinterpret_cast<const E*>(&vraw[i]));
    // (what is no number of bf16 parts is left to the loop below)
    const bool ox = odd_number(v.x), oy = odd_number(v.y);
    odd = odd || ox || oy;
    unsigned b[N];
    bf16_parts<N>(ox ? 0.0f : v.x, oy ? 0.0f : v.y, b);
    float y[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int k = N - 1; k >= 0; --k) {
      const unsigned t = transpose8(b[k]);
      mma_bf16(y, p[0], p[1], p[2], 0u, t, t);
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) f.o[i][e] = fmaf(y[e] + y[e + 2], sh.share, f.o[i][e]);
  }
  // what a row does not see must not reach it, and parts that are 0 would make
  // NaNs of infinities: those values are taken one by one
  if (__builtin_expect(__any_sync(0xffffffffu, odd), 0)) {
#pragma unroll 1
    for (int t = 0; t < kK8Few; ++t) {
      const float w = __shfl_sync(0xffffffffu, t & 1 ? pb : pa, lane & 28 | t >> 1) * sh.share;
      if (t >= left || t >= end) continue;
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        const float2 v = pair_of(V + t * D + 8 * i + 2 * tid);
        if (odd_number(v.x)) f.o[i][0] = fmaf(w, v.x, f.o[i][0]);
        if (odd_number(v.y)) f.o[i][1] = fmaf(w, v.y, f.o[i][1]);
      }
    }
    __syncwarp();
  }
}
// the rows of tokens [first, first + 8) below left on their way to the cache
template <int D, typename E>
__device__ __forceinline__ void k8_rows_ahead(const E* K, const E* V, int first, int left) {
  const int lane = threadIdx.x & 31;
  constexpr int lines = D * (int)sizeof(E) / 128;       // 128-byte lines of a row
  for (int x = lane; x < 2 * kK8Few * lines; x += 32) {
    const int row = first + x / lines % kK8Few;
    if (row < left)
      asm volatile("prefetch.global.L2 [%0];\n" ::"l"((const char*)((x < kK8Few * lines ? K : V) + row * D) + x % lines * 128));
  }
}

// --------------------------------------------------------------- the sums

// rows of a warp's sums in shared memory lie D + 8 floats apart (bank offsets; with
// two tiles there is room for D + 4)
template <int D, int MT> constexpr int kK8Pitch = D + 8 / MT;

// the warp's sums as rows [8] of m, l and acc[D] in shared memory
template <int D, int MT>
__device__ __forceinline__ void k8_store(K8Fast<D>& f, float* s_m, float* s_l, float* s_acc) {
  const int lane = threadIdx.x & 31, gid = lane >> 2, tid = lane & 3;
  f.l += __shfl_xor_sync(0xffffffffu, f.l, 1);
  f.l += __shfl_xor_sync(0xffffffffu, f.l, 2);
  if (tid == 0) { s_m[gid] = f.r; s_l[gid] = f.l; }
#pragma unroll
  for (int i = 0; i < D / 8; ++i)
    *reinterpret_cast<float2*>(s_acc + gid * kK8Pitch<D, MT> + 8 * i + 2 * tid) = make_float2(f.o[i][0], f.o[i][1]);
}
// factor of sums relative to m where they become relative to M
__device__ __forceinline__ float k8_factor(float m, float l, float M) { return m > -INFINITY ? ex2(m - M) : l == 0.0f ? 0.0f : 1.0f; }

// --------------------------------------------------------------- the kernel

// shared memory: barriers (keys and values full, empty, items full, sums full,
// empty), items, their list entries, sums of W * MT tiles, q rows, the slots
template <int D, int W, int MT, typename A>
struct K8Layout {
  static constexpr int item = (4 * W + kK8Items + 3) * 8;
  static constexpr int ids = item + kK8Items * (int)sizeof(KdItem<A>);
  static constexpr int m = ids + (A::kPerToken ? kK8Items * kKdIds * 4 : 0);
  static constexpr int l = m + W * MT * 8 * 4;
  static constexpr int acc = (l + W * MT * 8 * 4 + 15) / 16 * 16;
  static constexpr int q = acc + W * MT * 8 * kK8Pitch<D, MT> * 4;
  static constexpr __host__ __device__ int slots(int rows) { return (q + kK8Items * rows * D * 4 + 127) / 128 * 128; }     // (padded rows)
};

// whether the phase of parity `parity` is complete, for a whole warp
__device__ __forceinline__ bool mbar_test(unsigned bar, unsigned parity) {
  unsigned done;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(done)
      : "r"(bar), "r"(parity)
      : "memory");
  return __all_sync(0xffffffffu, done);
}
__device__ __forceinline__ void k8_send(unsigned to, const uint8_t* from, unsigned bytes, unsigned bar) {
  mbar_expect_tx(bar, bytes);
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n" ::"r"(to), "l"(from),
               "r"(bytes), "r"(bar)
               : "memory");
}
// where block x of an item lies
template <typename A>
__device__ __forceinline__ int64_t k8_at(const A& a, const KdSegOf<A>& s, const int32_t* s_ids, int x) {
  if constexpr (A::kPerToken) {
    const int id = x < kKdIds ? s_ids[x] : a.blocks[(((int64_t)s.b * a.T + s.t) * a.Hkv + s.g) * a.n_sel + s.blk0 + x];
    return s.bg * a.nblk_max + id;
  } else {
    return s.bg * a.nblk_max + s.blk0 + x;
  }
}

// D / 32 floats at p (a lane's channels of a row)
template <int CPL>
__device__ __forceinline__ void floats_in(float (&x)[CPL], const float* p) {
  if (CPL == 4) {
    const float4 v = *reinterpret_cast<const float4*>(p);
    x[0] = v.x; x[1] = v.y; x[CPL - 2] = v.z; x[CPL - 1] = v.w;
  } else {
    const float2 v = *reinterpret_cast<const float2*>(p);
    x[0] = v.x; x[1] = v.y;
  }
}
template <int CPL>
__device__ __forceinline__ void floats_out(float* p, const float (&x)[CPL]) {
  if (CPL == 4) *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[CPL - 2], x[CPL - 1]);
  else *reinterpret_cast<float2*>(p) = make_float2(x[0], x[1]);
}

// shared memory of CTA `rank` of the cluster
__device__ __forceinline__ unsigned cluster_at(unsigned own, unsigned rank) {
  unsigned at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(at) : "r"(own), "r"(rank));
  return at;
}
__device__ __forceinline__ float4 cluster_load4(unsigned at) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];\n" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ float2 cluster_load2(unsigned at) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0,%1}, [%2];\n" : "=f"(v.x), "=f"(v.y) : "r"(at) : "memory");
  return v;
}
// all threads of the cluster that have not ended
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}

// a finished row: the lane's D / 32 channels
template <int D, typename A>
__device__ __forceinline__ void k8_out(const A& a, const KdSegOf<A>& s, int r, float M, float l, float (&v)[D / 32]) {
  constexpr int CPL = D / 32;
  const int lane = threadIdx.x & 31, glog = 31 - __clz(a.G);
  int t = r >> glog;
  const int h = s.g * a.G + (r & (a.G - 1));
  if constexpr (A::kPerToken) t = s.t;
  if (t >= s.nq) return;
  const int64_t row = ((int64_t)s.b * a.T + t) * a.Hq + h;
  // l = 0 only where nothing was attended to
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
  for (int c = 0; c < CPL; ++c) v[c] = l == 0.0f ? 0.0f : v[c] * inv;
  floats_out<CPL>(a.o + row * D + lane * CPL, v);
  if (lane == 0 && a.lse) a.lse[row] = l == 0.0f ? -INFINITY : (M + log2f(l)) * 0.69314718055994531f;
}

// The item's sums from its teams' (team_rows rows each), by a side warp: rows
// [r0, r1), four at a time.  First a lane to a team, then D / 32 channels to a lane.
// Where the CTA has a part of the item only they go to the workspace, or to `keep`
// (rows of D, then m and l of each) for the other CTAs of the cluster.
template <int D, int MT, typename A>
__device__ __forceinline__ void k8_merge(const A& a, const KdSegOf<A>& s, int nteam, int team_rows, const float* s_m, const float* s_l,
                                         const float* s_acc, float* keep, int r0, int r1) {
  constexpr int CPL = D / 32, N = 4;
  const int lane = threadIdx.x & 31, R = kd_rows(a);
  float* part = a.part + (2 * (int64_t)blockIdx.x + (s.cut0 ? 0 : 1)) * R * (D + 4) + lane * CPL;
  for (int r = r0; r < min(r1, R); r += N) {
    float M[N], l[N], f[N], v[N][CPL];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int x = lane * team_rows + r + i;
      const bool in = lane < nteam;
      M[i] = f[i] = in ? s_m[x] : -INFINITY;
      l[i] = in ? s_l[x] : 0.0f;
    }
#pragma unroll
    for (int o = 1; o < 16; o <<= 1)
#pragma unroll
      for (int i = 0; i < N; ++i) M[i] = fmaxf(M[i], __shfl_xor_sync(0xffffffffu, M[i], o));
#pragma unroll
    for (int i = 0; i < N; ++i) {
      M[i] = __shfl_sync(0xffffffffu, M[i], 0);
      f[i] = k8_factor(f[i], l[i], M[i]);
      l[i] *= f[i];
#pragma unroll
      for (int c = 0; c < CPL; ++c) v[i][c] = 0.0f;
    }
#pragma unroll
    for (int o = 1; o < 16; o <<= 1)
#pragma unroll
      for (int i = 0; i < N; ++i) l[i] += __shfl_xor_sync(0xffffffffu, l[i], o);
#pragma unroll 2
    for (int y = 0; y < nteam; ++y) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        float z[CPL];
        floats_in<CPL>(z, s_acc + (y * team_rows + r + i) * kK8Pitch<D, MT> + lane * CPL);
        const float w = __shfl_sync(0xffffffffu, f[i], y);
#pragma unroll
        for (int c = 0; c < CPL; ++c) v[i][c] = fmaf(w, z[c], v[i][c]);
      }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      l[i] = __shfl_sync(0xffffffffu, l[i], 0);
      if (r + i >= R) continue;
      if constexpr (A::kPerToken) {
        if (s.bad) {
          M[i] = 0.0f;
          l[i] = NAN;
#pragma unroll
          for (int c = 0; c < CPL; ++c) v[i][c] = NAN;
        }
      }
      if (a.clog) {
        floats_out<CPL>(keep + (r + i) * D + lane * CPL, v[i]);
        if (lane == 0) *reinterpret_cast<float2*>(keep + R * D + 2 * (r + i)) = make_float2(M[i], l[i]);
      } else if (s.cut0 || s.cut1) {
        float* to = part + (r + i) * (D + 4);
        floats_out<CPL>(to, v[i]);
        if (lane == 0) { to[D] = M[i]; to[D + 1] = l[i]; }
      } else {
        k8_out<D>(a, s, r + i, M[i], l[i], v[i]);
      }
    }
  }
}

// The share of CTA `rank` of the 2^clog that take an item together: whole blocks in
// order, and of the incomplete one's tokens, eight at a time, those from k8_first on
// (from the last CTA to the first, as the first shares of blocks are the smallest);
// with up to 16 rows, of which a CTA does eight times eight tokens at once, rank 0
// takes it all (8 items, 500 tokens, 64 rows: 16.3 us, all to one CTA 22.3; 20 rows
// 11.0 and 12.4; but 32 items, 1000 tokens, 4 rows 9.5 and 9.1, 16 rows 14.2 and 13.4).
__device__ __forceinline__ int k8_first(int tokens, int rank, int clog) {
  return kK8Few * ((tokens + kK8Few - 1) / kK8Few * ((1 << clog) - 1 - rank) >> clog);
}
template <typename S>
__device__ __forceinline__ void k8_take(S& s, int rank, int clog, bool spread) {
  const int lo = (int)((int64_t)s.nfast * rank >> clog), hi = (int)((int64_t)s.nfast * (rank + 1) >> clog);
  s.blk0 += lo;
  s.nfast = hi - lo;
  s.clear = min(max(s.clear - lo, 0), s.nfast);
  if (rank) s.left = spread ? min(s.left, k8_first(s.left, rank - 1, clog)) : 0;
}
// The item's sums from its CTAs' (keep), by warp `part` of `parts` of CTA `rank`: rows
// rank, rank + the CTAs, ...  First a lane to a CTA, then D / 32 channels to a lane.
template <int D, typename A>
__device__ __forceinline__ void k8_join(const A& a, const KdSegOf<A>& s, const float* keep, int rank, int part, int parts) {
  constexpr int CPL = D / 32, N = 8;
  const int lane = threadIdx.x & 31, R = kd_rows(a), n = 1 << a.clog;
  const unsigned at = smem_u32(keep);
  for (int r = rank + part * n; r < R; r += parts * n) {
    float z[N][CPL];
#pragma unroll
    for (int k = 0; k < N; ++k)
      if (k < n) {
        const unsigned from = cluster_at(at + (r * D + lane * CPL) * 4, k);
        if (CPL == 4) {
          const float4 y = cluster_load4(from);
          z[k][0] = y.x; z[k][1] = y.y; z[k][CPL - 2] = y.z; z[k][CPL - 1] = y.w;
        } else {
          const float2 y = cluster_load2(from);
          z[k][0] = y.x; z[k][1] = y.y;
        }
      }
    const float2 ml = lane < n ? cluster_load2(cluster_at(at + (R * D + 2 * r) * 4, lane)) : make_float2(-INFINITY, 0.0f);
    float M = ml.x;
#pragma unroll
    for (int o = 1; o < N; o <<= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    M = __shfl_sync(0xffffffffu, M, 0);
    const float f = k8_factor(ml.x, ml.y, M);
    float l = ml.y * f, v[CPL];
#pragma unroll
    for (int o = 1; o < N; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    l = __shfl_sync(0xffffffffu, l, 0);
#pragma unroll
    for (int c = 0; c < CPL; ++c) v[c] = 0.0f;
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const float w = __shfl_sync(0xffffffffu, f, k);
      if (k < n) {
#pragma unroll
        for (int c = 0; c < CPL; ++c) v[c] = fmaf(w, z[k][c], v[c]);
      }
    }
    k8_out<D>(a, s, r, M, l, v);
  }
}

template <int D, int W, int MT, typename E, typename A>
__global__ void __launch_bounds__(kK8Threads<W, MT>, 1) kv8_decode_kernel(const A a) {
  pdl_entry();
  using Lt = K8Layout<D, W, MT, A>;
  constexpr unsigned bytes = kBlock * D;
  __shared__ KdBatch batch;
  extern __shared__ __align__(128) uint8_t k8_sm[];
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int R = kd_rows(a), Rp = (R + 8 * MT - 1) / (8 * MT) * (8 * MT);
  // teams: warps that share a block, MT tiles of rows each (those left over idle)
  const int team = W == kK8Warps ? 1 : Rp / (8 * MT), nteam = W / team;
  const unsigned bars = smem_u32(k8_sm), item_full = bars + 4 * W * 8, sums_full = item_full + 8 * kK8Items, sums_empty = sums_full + 8;
  KdItem<A>* items = reinterpret_cast<KdItem<A>*>(k8_sm + Lt::item);
  int32_t* s_ids = reinterpret_cast<int32_t*>(k8_sm + Lt::ids);
  float* s_q = reinterpret_cast<float*>(k8_sm + Lt::q);        // [items][rows, padded][D]
  float* s_m = reinterpret_cast<float*>(k8_sm + Lt::m);        // [warps][8]
  float* s_l = reinterpret_cast<float*>(k8_sm + Lt::l);
  float* s_acc = reinterpret_cast<float*>(k8_sm + Lt::acc);    // [warps][8][kK8Pitch]
  if (tid >= 32 && tid < 32 + 2 * W) {
    const int i = tid - 32;
    mbar_init(bars + 8 * i, 1);                                // full: keys, values of the teams in turn
    mbar_init(bars + 8 * (2 * W + i), team);                   // empty
    if (i < kK8Items) mbar_init(item_full + 8 * i, kK8Side);
    if (i == 0) {
      mbar_init(sums_full, W);
      mbar_init(sums_empty, kK8Side);
    }
    fence_barrier_init();
  }
  kd_batch(a, batch);
  const int64_t per = kd_run(batch, gridDim.x >> a.clog);
  const int rank = blockIdx.x & ((1 << a.clog) - 1);
  int64_t u0 = (int64_t)(blockIdx.x >> a.clog) * per, u1 = min(batch.pref[kMaxB], u0 + per);
  kd_trim(a, batch, u0, u1);
  // (Each wait is bounded: one that gives up marks the call, and the warp goes
  // on without waiting.)
  bool dead = false;
  // An item's part of the run that begins at u, its queries (rows [r0, r1)) and what
  // else is known of it; writer: by the warp that writes what is the item's.
  KdSegOf<A> sg;
  const auto fetch = [&](int64_t u, int buf, bool writer, int r0, int r1) {
    KdItem<A>& it = items[buf];
    sg = u == u0 ? kd_seg(a, batch, u, u1) : kd_next(a, batch, sg, u, u1);
    const int32_t* ids = nullptr;
    if constexpr (A::kPerToken) ids = kd_list(a, sg);
    if (a.clog) k8_take(sg, rank, a.clog, R > 16);
    if constexpr (A::kPerToken) {
      ids += sg.blk0;
      if (writer)
        for (int x = lane; x < min(sg.nfast, kKdIds); x += 32) s_ids[buf * kKdIds + x] = ids[x];
    }
    if (lane == 0 && writer) it.seg = sg;
    kd_item_queries<D, E>(a, sg, it, s_q + buf * Rp * D, r0, r1);
  };
  // the first item's by all warps
  if (u0 < u1) {
    const int each = (Rp + W + kK8Side - 1) / (W + kK8Side);
    if (w < W + kK8Side) fetch(u0, 0, w == W, min(w * each, Rp), min((w + 1) * each, Rp));
  }
  __syncthreads();

  if (w >= W) {
    // The side warps: the next items' queries and what else is known of them, ahead
    // of the sums, which they merge while the others are at the items after.
    if constexpr (MT == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kK8RegsSide));
    const int part = w - W;
    if (part >= kK8Side) return;
    if (blockIdx.x == 0 && part == 1) {
      bool bad = false;
      for (int b = lane; b < a.B; b += 32) {
        bad |= a.len[b] < 0 || a.len[b] > a.n_max;
        if (a.n_q) bad |= a.n_q[b] < 0 || a.n_q[b] > a.T;
      }
      const unsigned any = __any_sync(0xffffffffu, bad);
      // (a wait that gives up flags the word two seconds later at the earliest)
      if (lane == 0) *a.status = any ? 8u : 0u;
    }
    int64_t u = u0;
    const auto ahead = [&](int buf) {
      if (u >= u1) return;
      if (u > u0) fetch(u, buf, part == 0, part * (Rp / kK8Side), (part + 1) * (Rp / kK8Side));
      __syncwarp();
      if (lane == 0) mbar_arrive(item_full + 8 * buf);
      u += sg.step;
    };
    for (int buf = 0; buf < kK8Items; ++buf) ahead(buf);
    int64_t done = u0;
    for (int k = 0, buf = 0; done < u1; ++k) {
      const KdSegOf<A> s = items[buf].seg;
      done += s.step;
      if (done >= u1) break;                      // the last one's sums are merged by the others
      if (!dead) dead = __any_sync(0xffffffffu, !mbar_wait(sums_full, k & 1));
      k8_merge<D, MT>(a, s, nteam, team * MT * 8, s_m, s_l, s_acc, nullptr, part * (Rp / kK8Side), (part + 1) * (Rp / kK8Side));
      __syncwarp();
      if (lane == 0) mbar_arrive(sums_empty);
      bar_sync(1, kK8Side * 32);                  // both have read the item
      ahead(buf);
      if (++buf == kK8Items) buf = 0;
    }
    if (dead && lane == 0) atomicOr(a.status, 4u);
    return;
  }

  if constexpr (MT == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(kK8RegsConsumer));
  const int my_team = w / team, tile = w % team;
  const bool works = my_team < nteam;             // (a warp with rows)
  const int r0 = works ? tile * 8 * MT : 0;
  // the team's slots and barriers: keys, values
  const uint8_t* kt = k8_sm + Lt::slots(Rp) + 2 * min(my_team, nteam - 1) * bytes;
  const uint8_t* vt = kt + bytes;
  const unsigned full = bars + 16 * my_team, empty = full + 16 * W;
  // An item's work goes to the teams in turn, its blocks and then its incomplete
  // block by eight tokens, and on with the next item.
  int x = my_team;                                // the team's next turn in the item
  int phase = 0;                                  // parity of its slots
  bool sent = false;                              // the team's first warp has sent for that block,
  float2 step = make_float2(0.0f, 0.0f);          // and its steps are known
  int k = 0, buf = 0, turn = 0, last = 0;         // number of the item, its place, its parity there, the last one's place

  for (int64_t u = u0; u < u1; ++k) {
    if (!dead) dead = __any_sync(0xffffffffu, !mbar_wait(item_full + 8 * buf, turn));
    if (dead) {
      // the way through the items does not hang on the side warps
      if (lane == 0) items[buf].seg = kd_seg(a, batch, u, u1);
      __syncwarp();
    }
    const int buf1 = buf + 1 == kK8Items ? 0 : buf + 1, turn1 = buf1 ? turn : turn ^ 1;      // the next item's
    const KdItem<A>& it = items[buf];
    const int n = my_team < nteam ? it.seg.nfast : 0, left = it.seg.left;
    const uint4* qa = reinterpret_cast<const uint4*>(s_q + (buf * Rp + r0) * D) + lane;
    // (the incomplete block, if it is to be done here)
    const int64_t tail0 = it.seg.n / kBlock * kBlock;
    const E* Kt = reinterpret_cast<const E*>(a.c.Kt) + it.seg.bg * kBlock * D;
    const E* Vt = reinterpret_cast<const E*>(a.c.Vt) + it.seg.bg * kBlock * D;
    const int first = a.clog && R > 16 ? min(k8_first((int)(it.seg.n % kBlock), rank, a.clog), left) : 0;
    const int turns = n + (left - first + kK8Few - 1) / kK8Few;
    const int x1 = x < turns ? x + (turns - x + nteam - 1) / nteam * nteam - turns : x - turns;   // the team's first turn in the next item
    const int few = !works ? kBlock : first + kK8Few * ((x < n ? x + (n - x + nteam - 1) / nteam * nteam : x) - n);
    if (few < left) k8_rows_ahead<D>(Kt, Vt, few, left);
    if (x < n && !sent && !dead) {
      const int64_t at = k8_at(a, it.seg, s_ids + buf * kKdIds, x);
      if (tile == 0 && lane == 0) {
        // (the team's other warps are done with both slots: nothing was sent for since)
        if (team > 1) {
          mbar_wait(empty, phase ^ 1);
          mbar_wait(empty + 8, phase ^ 1);
        }
        k8_send(smem_u32(kt), a.c.K8 + at * bytes, bytes, full);
        k8_send(smem_u32(vt), a.c.V8 + at * bytes, bytes, full + 8);
      }
      step = *reinterpret_cast<const float2*>(a.c.scale + at * 2);
    }
    __syncwarp();
    K8Fast<D> f[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      f[t].inv = it.inv[r0 + 8 * t + (lane >> 2)];
      f[t].r = -INFINITY;
      f[t].l = 0.0f;
#pragma unroll
      for (int i = 0; i < D / 8; ++i) f[t].o[i][0] = f[t].o[i][1] = 0.0f;
    }
    // the end of what the lane's row of tile t sees, from position p on, up to `most`
    const auto end_of = [&](int t, int64_t p, int most) {
      return (int)min(max(it.end[r0 + 8 * t + (lane >> 2)] - p, (int64_t)0), (int64_t)most);
    };
    const int64_t u_next = u + it.seg.step;
    while (x < n) {
      if (!dead) dead = __any_sync(0xffffffffu, !mbar_wait(full, phase));
      const float ks = step.x, vs = step.y;
      int64_t at = 0;
      // The keys are read: the next block's, of this item or the next one, if
      // that is known.
      const auto between = [&]() {
        __syncwarp();
        sent = x + nteam < n;
        if (sent) {
          at = k8_at(a, it.seg, s_ids + buf * kKdIds, x + nteam);
        } else if (u_next < u1 && mbar_test(item_full + 8 * buf1, turn1)) {
          const KdSegOf<A>& next = items[buf1].seg;
          sent = x1 < next.nfast;
          if (sent) at = k8_at(a, next, s_ids + buf1 * kKdIds, x1);
        }
        sent = sent && !dead;
        if (team > 1 && lane == 0) mbar_arrive(empty);
        if (sent) {
          if (tile == 0 && lane == 0) {
            if (team > 1) mbar_wait(empty, phase);
            k8_send(smem_u32(kt), a.c.K8 + at * bytes, bytes, full);
          }
          step = *reinterpret_cast<const float2*>(a.c.scale + at * 2);
        }
        __syncwarp();
        if (!dead) dead = __any_sync(0xffffffffu, !mbar_wait(full + 8, phase));
      };
      const int64_t p0 = [&] {
        if constexpr (A::kPerToken) return it.seg.own;
        else return (it.seg.blk0 + x) * kBlock;
      }();
      const bool masked = x >= it.seg.clear;
      int end[MT];
#pragma unroll
      for (int t = 0; t < MT; ++t) end[t] = masked ? end_of(t, p0, kBlock) : 0;
      k8_block<D, MT>(f, qa, kt, vt, ks, vs, masked, end, between);
      __syncwarp();
      if (team > 1 && lane == 0) mbar_arrive(empty + 8);
      if (sent && tile == 0 && lane == 0) {
        if (team > 1) mbar_wait(empty + 8, phase);
        k8_send(smem_u32(vt), a.c.V8 + at * bytes, bytes, full + 8);
      }
      __syncwarp();
      phase ^= 1;
      x += nteam;
    }
    if (few < left) {
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        const int end = end_of(t, tail0, left);
#pragma unroll 1
        for (int i = few; i < left; i += kK8Few * nteam) k8_rows<D, E>(f[t], qa + 2 * D * t, Kt + i * D, Vt + i * D, left - i, end - i);
      }
    }
    x = x1;
    // the sums, once those of the item before have been merged
    if (k > 0 && !dead) dead = __any_sync(0xffffffffu, !mbar_wait(sums_empty, (k - 1) & 1));
#pragma unroll
    for (int t = 0; t < MT; ++t)
      k8_store<D, MT>(f[t], s_m + (w * MT + t) * 8, s_l + (w * MT + t) * 8, s_acc + (w * MT + t) * 8 * kK8Pitch<D, MT>);
    __syncwarp();
    if (u_next < u1 && lane == 0) mbar_arrive(sums_full);        // (and the item's place may be filled again)
    u = u_next;
    last = buf;
    buf = buf1;
    turn = turn1;
  }
  if (dead) {
    // copies in flight land before the CTA can end (of whichever phase)
    for (int i = 0; i < 4; ++i) mbar_wait(full + 8 * (i & 1), i >> 1);
    if (lane == 0) atomicOr(a.status, 4u);
  }
  if (u0 >= u1) return;
  bar_sync(2, W * 32);
  const KdSegOf<A> s = items[last].seg;
  float* keep = s_q + Rp * D;                     // (with a.clog there is one item: the other places are free)
  for (int r = 4 * w; r < R; r += 4 * W) k8_merge<D, MT>(a, s, nteam, team * MT * 8, s_m, s_l, s_acc, keep, r, r + 4);
  if (a.clog) {
    cluster_sync();
    k8_join<D>(a, s, keep, rank, w, W);
    cluster_sync();                               // (its shared memory has been read)
  }
}

namespace {

// How items are dealt out: whole, one CTA each; shared by clusters of CTAs; or cut
// wherever the CTAs' equal runs end, and joined by a second kernel.  us, bf16, d = 128,
// lengths all the same, whole / shared / cut:
//                    300 tokens       1000             2000             4000             8000
//    8 items,  4 rows   8 /  -  / 10   11 /  8 / 11     17 /  8 / 11     27 / 10 / 13     46 / 12 / 13
//             20 rows  13 / 10  / 13   22 / 11 / 14     36 / 12 / 15     64 / 16 / 16    119 / 22 / 20
//             64 rows  27 / 19  / 23   48 / 20 / 25     77 / 23 / 25    141 / 31 / 28    263 / 45 / 34
//   32 items,  4 rows   8 /  -  / 11   12 /  9 / 13     17 / 10 / 13     28 / 13 / 16     48 / 19 / 19
//             16 rows  15 / 13  / 16   19 / 13 / 18     27 / 16 / 20     43 / 20 / 22     72 / 25 / 28
//   64 items,  8 rows   8 /  -  / 13   12 / 11 / 16     18 / 13 / 17     28 / 19 / 22     49 / 31 / 34
//             32 rows  18 / 17  / 23   28 / 21 / 28     43 / 30 / 36     76 / 46 / 48    140 / 79 / 78
//  160 items,  8 rows  13 /  -  / 16   19 /  - / 20     29 /  - / 25     51 /  - / 42     90 /  - / 64
//  512 items,  8 rows  23 /  -  / 28   38 /  - / 43     54 /  - / 58     94 /  - / 96    173 /  - / 168
// Lengths that differ favour cut items: whole and shared ones take as long as the
// longest (512 items of up to 2000 tokens: 56 us, cut 52).
//
// Whole: where the blocks are one round of a CTA's warps at most, and up to 16
// blocks where there are items for a quarter of the SMs.
constexpr int64_t kK8WholeBlocks = 16;
int64_t k8_blocks(const csa_shape* s, int n_sel) {
  const int64_t blocks = (s->n_max + kBlock - 1) / kBlock;
  return n_sel && n_sel < blocks ? n_sel : blocks;
}
int64_t k8_items(const csa_shape* s, int T, int n_sel) { return (int64_t)s->B * s->Hkv * (n_sel ? T : 1); }
int k8_rows_of(const csa_shape* s, int T, int n_sel) { return (n_sel ? 1 : T) * (s->Hq / s->Hkv); }
// Shared by 2, 4 or 8 CTAs, as the SMs allow (eight only for half of them: a card full
// of such clusters, which lie within groups of SMs, takes two rounds).  They are doubled
// while each still has more than 2 blocks of a tile, beside the incomplete one's up to
// eight turns, of lists more than 10: each is left with more than 1, of lists 5 (1000
// tokens, 4 rows: 8.2 us, doubled only from 10 blocks 9.9); up to 6 blocks stay
// together (300 tokens: 7.7 us, shared 8.1).  And up to
// three rounds of their warps; with CTAs for more than half of the SMs, where cutting
// has less to gain, six, or sixteen of lists, which are mostly of one length (64
// items of 256 blocks: 65 us, cut 70).
int k8_clog(const csa_shape* s, int T, int n_sel) {
  const int tiles = (k8_rows_of(s, T, n_sel) + 7) / 8, least = n_sel || 2 * tiles > kK8Warps ? kK8Warps : 2 * tiles;
  const int64_t items = k8_items(s, T, n_sel), work = k8_blocks(s, n_sel) * tiles;
  int clog = 0;
  if (work <= 6) return 0;
  while (clog < 3 && (items << (clog + 1)) <= (clog < 2 ? sm_count() : sm_count() / 2) && work > ((int64_t)least << clog)) ++clog;
  const int rounds = 2 * (items << clog) <= sm_count() ? 3 : n_sel ? 16 : 6;
  return work <= ((int64_t)rounds * kK8Warps << clog) ? clog : 0;
}
int k8_whole(const csa_shape* s, int T, int n_sel) {
  const int64_t blocks = k8_blocks(s, n_sel);
  return blocks * ((k8_rows_of(s, T, n_sel) + 7) / 8) <= kK8Warps ||
         (blocks <= kK8WholeBlocks && 4 * k8_items(s, T, n_sel) > sm_count()) || k8_clog(s, T, n_sel);
}

// CTAs of the decode kernel: one per SM, no more than there can be units
int k8_ctas(const csa_shape* s, int T, int n_sel) {
  if (k8_clog(s, T, n_sel)) return (int)k8_items(s, T, n_sel) << k8_clog(s, T, n_sel);
  const int64_t units = k8_items(s, T, n_sel) * (k8_whole(s, T, n_sel) ? 1 : k8_blocks(s, n_sel));
  const int nsm = sm_count() < Kv8DecodeArgs<true>::kMaxCtas ? sm_count() : Kv8DecodeArgs<true>::kMaxCtas;
  return (int)(units < nsm ? units : nsm);
}

size_t k8_workspace(const csa_shape* s, int T, int n_sel) {
  const size_t rows = 2 * (size_t)k8_ctas(s, T, n_sel) * k8_rows_of(s, T, n_sel);
  return 256 + (k8_whole(s, T, n_sel) ? 0 : rows * (s->d + 4) * 4);
}

// Dynamic shared memory there can be: a CTA's 227 KB without the kernel's own.
// The limit is set to this on every call, whatever the call needs: it belongs to
// the function, and another host thread's call may lie between the setting and
// the launch.
constexpr int kK8SharedBytes = 232448 - ((int)sizeof(KdBatch) + 127) / 128 * 128;
template <int D, int W, int MT, typename E, typename A>
cudaError_t launch_kv8_decode_t(const A& a, int ncta, cudaStream_t st) {
  const int R = kd_rows(a), Rp = (R + 8 * MT - 1) / (8 * MT) * (8 * MT), nteam = W / (Rp / (8 * MT));
  constexpr int least = W == 14 ? 24 : 8 * MT;     // padded rows there are at least: the most teams
  static_assert(K8Layout<D, W, MT, A>::slots(least) + 2 * (W * 8 * MT / least) * kBlock * D <= kK8SharedBytes, "shared memory");
  const int smem = K8Layout<D, W, MT, A>::slots(Rp) + 2 * nteam * kBlock * D;
  const cudaError_t e =
      cudaFuncSetAttribute(kv8_decode_kernel<D, W, MT, E, A>, cudaFuncAttributeMaxDynamicSharedMemorySize, kK8SharedBytes);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ncta);
  cfg.blockDim = dim3(kK8Threads<W, MT>);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 1 << a.clog;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = a.clog ? 2 : 1;
  const cudaError_t le = cudaLaunchKernelEx(&cfg, kv8_decode_kernel<D, W, MT, E, A>, a);
  if (le != cudaSuccess) return le;
  if (ncta > 1 && !a.whole)
    launch_pdl(decode_join_kernel<D, A>, dim3(ncta - 1, (R + kKdJoinWarps - 1) / kKdJoinWarps), dim3(kKdJoinWarps * 32), 0, st, a, ncta);
  return cudaGetLastError();
}
// Ten warps for one tile of rows.  With more, eight warps of two tiles each, whose
// codes are converted once for both, where eight are shared out evenly, i.e. with 2,
// 4 or 8 tiles, else fourteen of one.  8 sequences of up to 20,000 tokens, d = 128,
// eight of two against fourteen of one in us: 16 rows 72 against 80, 24 rows 121
// against 104, 32 rows 122 against 139, 40 rows 213 against 192, 48 rows 213 against
// 196, 56 rows 230 against 233, 64 rows 232 against 307.
template <int D, typename E, typename A>
cudaError_t launch_kv8_decode_w(const A& a, int ncta, cudaStream_t st) {
  if constexpr (!A::kPerToken)         // (lists have one tile)
    if (kd_rows(a) > 8) {
      const int tiles = (kd_rows(a) + 7) / 8;
      return (tiles & (tiles - 1)) == 0 ? launch_kv8_decode_t<D, 8, 2, E>(a, ncta, st) : launch_kv8_decode_t<D, 14, 1, E>(a, ncta, st);
    }
  return launch_kv8_decode_t<D, kK8Warps, 1, E>(a, ncta, st);
}
template <typename A>
cudaError_t launch_kv8_decode(const A& a, int d, bool bf16, int ncta, cudaStream_t st) {
  return d == 128 ? (bf16 ? launch_kv8_decode_w<128, __nv_bfloat16>(a, ncta, st) : launch_kv8_decode_w<128, float>(a, ncta, st))
                  : (bf16 ? launch_kv8_decode_w<64, __nv_bfloat16>(a, ncta, st) : launch_kv8_decode_w<64, float>(a, ncta, st));
}

bool k8_args_ok(const csa_shape* s, int T, csa_status* st) {
  if (!shape_ok(s) || T < 1) { *st = CSA_ERR_INVALID_ARG; return false; }
  *st = shape_supported(s);
  if (*st == CSA_OK && (T > CSA_KV4_MAX_T || T * (s->Hq / s->Hkv) > CSA_KV4_MAX_ROWS)) *st = CSA_ERR_UNSUPPORTED;
  return *st == CSA_OK;
}

template <bool LIST>
csa_status k8_decode(const csa_shape* shape, const csa_kv8* cache, int T, const void* q, const csa_strides* qs,
                     const int64_t* len, const int64_t* n_q, const int32_t* blocks, const int32_t* count, int n_sel, float* o,
                     float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  csa_status su;
  if (!shape_ok(shape) || !kv8_cache_ok(cache) || T < 1 || !q || !len || !o) return CSA_ERR_INVALID_ARG;
  if (LIST && (!blocks || !count || n_sel < 1 || ((uintptr_t)blocks | (uintptr_t)count) % 4)) return CSA_ERR_INVALID_ARG;
  if (!k8_args_ok(shape, T, &su)) return su;
  if (LIST && n_sel > CSA_KV8_MAX_SEL) return CSA_ERR_UNSUPPORTED;
  const bool bf16 = shape->dtype == CSA_BF16;
  if (!strides_ok(qs, bf16 ? 8 : 4, shape->B, T, shape->Hq) || !aligned16(q) || !aligned16(o)) return CSA_ERR_INVALID_ARG;
  if (!workspace || workspace_bytes < k8_workspace(shape, T, n_sel) || ((uintptr_t)workspace % 256)) return CSA_ERR_WORKSPACE;
  Kv8DecodeArgs<LIST> a = {};
  a.c = *cache; a.q = q; a.qs = *qs; a.len = len; a.n_q = n_q; a.o = o; a.lse = lse;
  a.blocks = blocks; a.count = count; a.n_sel = n_sel;
  a.status = (unsigned*)workspace; a.part = (float*)((char*)workspace + 256);
  a.n_max = shape->n_max; a.nblk_max = (shape->n_max + kBlock - 1) / kBlock;
  a.B = shape->B; a.T = T; a.Hq = shape->Hq; a.Hkv = shape->Hkv; a.G = shape->Hq / shape->Hkv;
  a.rs = (float)(1.4426950408889634 / std::sqrt((double)shape->d));
  const int ncta = k8_ctas(shape, T, n_sel);
  a.whole = k8_whole(shape, T, n_sel);
  a.clog = k8_clog(shape, T, n_sel);
  add_launches(ncta > 1 && !a.whole ? 2 : 1);
  const cudaError_t e = launch_kv8_decode(a, shape->d, bf16, ncta, (cudaStream_t)stream);
  return e == cudaSuccess ? CSA_OK : CSA_ERR_CUDA;
}

}  // namespace
}  // namespace csa

using namespace csa;

extern "C" {

size_t csa_kv8_workspace_size(const csa_shape* shape, int T, int n_sel) {
  csa_status st;
  if (n_sel < 0 || n_sel > CSA_KV8_MAX_SEL || !k8_args_ok(shape, T, &st)) return 0;
  // Fewer tokens may need more: their lists are fewer items, which are cut where
  // more of them share CTAs (16 sequences and KV heads, 121 blocks: one token 0.6 MB,
  // two 256 bytes).  With fewer blocks, the tokens the same, items are never cut
  // that were not with more.
  size_t most = 0;
  for (int t = 1; t <= T; ++t) most = std::max(most, k8_workspace(shape, t, n_sel));
  return most;
}

csa_status csa_kv8_decode(const csa_shape* shape, const csa_kv8* cache, int T, const void* q, const csa_strides* qs,
                          const int64_t* len, const int64_t* n_q, float* o, float* lse, void* workspace,
                          size_t workspace_bytes, void* stream) {
  return k8_decode<false>(shape, cache, T, q, qs, len, n_q, nullptr, nullptr, 0, o, lse, workspace, workspace_bytes, stream);
}

csa_status csa_kv8_decode_blocks(const csa_shape* shape, const csa_kv8* cache, int T, const void* q, const csa_strides* qs,
                                 const int64_t* len, const int64_t* n_q, const int32_t* blocks, const int32_t* count,
                                 int n_sel, float* o, float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  return k8_decode<true>(shape, cache, T, q, qs, len, n_q, blocks, count, n_sel, o, lse, workspace, workspace_bytes, stream);
}

}  // extern "C"
