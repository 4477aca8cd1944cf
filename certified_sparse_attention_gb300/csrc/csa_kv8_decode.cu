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
// second kernel.  An item is a sequence and KV head with its T * G query rows;
// over lists, where each token has blocks of its own, a token's G rows.
//
// A warp handles a tile of 8 rows; with more the warps of a CTA form teams of 2
// to 8 that share the blocks.  Codes become half-precision numbers exactly (a
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
// Blocks come by bulk copies into two rings of shared memory, keys and values,
// each slot on an mbarrier; producer warps run ahead over the items.
#include <cmath>

#include "csa_decode.cuh"

namespace csa {

constexpr int kK8Warps = 8;       // consumer warps of a CTA: two warpgroups; a third one's
                                  // warps send for the blocks and the queries
constexpr int kK8Threads = (kK8Warps + 4) * 32;
// registers: 384 threads start with 168 each; the producers give theirs up
constexpr int kK8RegsConsumer = 200, kK8RegsProducer = 104;
static_assert(2 * kK8RegsConsumer + kK8RegsProducer <= 3 * 168, "more registers than the launch has");
constexpr int kK8MaxStages = 32;  // slots of a ring
// warps of a team, for 1 .. 8 tiles
__host__ __device__ constexpr int k8_team(int ntile) { return ntile <= 2 ? ntile : ntile <= 4 ? 4 : 8; }

template <bool LIST>
struct Kv8DecodeArgs : DecodeArgs {
  csa_kv8 c;
  const int32_t* blocks;  // LIST: [B][T][Hkv][n_sel], count [B][T][Hkv]
  const int32_t* count;
  int n_sel;
  int slotsK, slotsV;     // slots of the two rings: multiples of the number of teams
  static constexpr int kLead = 8, kTailBase = 3, kTailStep = 8;
  static constexpr bool kPerToken = LIST, kPlainQ = true;
  template <int D>
  static __device__ __forceinline__ int top(int c) { return c; }
};

// -------------------------------------------------------- moving the blocks

// A producer warp: sends for the keys' or the values' codes of the CTA's whole
// blocks in order, as slots come free, by one bulk copy each (and a block's two
// steps beside its keys).
template <int D, typename A>
__device__ __forceinline__ void k8_produce(const A& a, const KdBatch& batch, int64_t u0, int64_t u1, const KdRing& ring,
                                           unsigned side, bool keys) {
  constexpr unsigned codes = kBlock * D;
  const int lane = threadIdx.x & 31;
  const uint8_t* src = keys ? a.c.K8 : a.c.V8;
  const unsigned data = smem_u32(ring.data);
  int i = 0, slot = 0, phase = 0;
  bool dead = false;
  kd_trim(a, batch, u0, u1);
  for (int64_t u = u0; u < u1 && !dead;) {
    KdSeg s = kd_seg(a, batch, u, u1);
    const int32_t* ids = nullptr;
    if constexpr (A::kPerToken) ids = kd_list(a, s);
    int id = 0;
    for (int x = 0; x < s.nfast; ++x) {
      int64_t at = s.bg * a.nblk_max;
      if constexpr (A::kPerToken) {
        if ((x & 31) == 0) id = x + lane < s.nfast ? ids[s.blk0 + x + lane] : 0;
        at += __shfl_sync(0xffffffffu, id, x & 31);
      } else {
        at += s.blk0 + x;
      }
      dead = !mbar_wait(ring.empty + 8 * slot, phase ^ 1);    // (a new barrier's "phase -1" is complete)
      dead = __any_sync(0xffffffffu, dead);
      if (dead) break;
      if (lane == 0) {
        const unsigned bar = ring.full + 8 * slot;
        mbar_expect_tx(bar, codes);
        asm volatile(
            "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n" ::"r"(data + slot * codes),
            "l"(src + at * codes), "n"(codes), "r"(bar)
            : "memory");
        if (keys) {
          asm volatile("cp.async.ca.shared.global [%0], [%1], 8;\n" ::"r"(side + slot * 8), "l"(a.c.scale + at * 2) : "memory");
          asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];\n" ::"r"(bar) : "memory");
        }
      }
      ++i;
      if (++slot == ring.slots) { slot = 0; phase ^= 1; }
    }
    u += s.step;
  }
  // all copies land before the CTA can end
  for (int k = max(0, i - ring.slots); k < i; ++k)
    if (!mbar_wait(ring.full + 8 * (k % ring.slots), (k / ring.slots) & 1)) dead = true;
  if (dead && lane == 0) atomicOr(a.status, 4u);
}

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
// high parts of x and y, and what is left of them in units of 2^-12
__device__ __forceinline__ void k8_parts(float x, float y, unsigned& hi, unsigned& lo) {
  hi = half_pair(x, y);
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hi));
  lo = half_pair((x - f.x) * 4096.0f, (y - f.y) * 4096.0f);
}

// The state of a warp over the tensor-core blocks of an item; the lane's row is
// gid.
template <int D>
struct K8Fast {
  unsigned qa[D / 64][4][4];   // query operand: channels 64 h + 16 tid + 4 s + (0..3), high and low parts
  float inv;                   // undoes the row's scale
  float r;                     // reference of the sums: the running maximum, or up to 8 below it
  float l;                     // sum of the lane's own tokens' weights
  float o[D / 8][2];           // channels 8 i + 2 tid, + 1
};

template <int D>
__device__ __forceinline__ void k8_init(K8Fast<D>& f, const float* s_q, const float* s_inv) {
  const int lane = threadIdx.x & 31, gid = lane >> 2, tid = lane & 3;
#pragma unroll
  for (int h = 0; h < D / 64; ++h)
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const float4 x = *reinterpret_cast<const float4*>(s_q + kd_q<D>(gid, 64 * h + 16 * tid) + 4 * s);
      k8_parts(x.x, x.y, f.qa[h][s][0], f.qa[h][s][1]);
      k8_parts(x.z, x.w, f.qa[h][s][2], f.qa[h][s][3]);
    }
  f.inv = s_inv[gid];
  f.r = -INFINITY;
  f.l = 0.0f;
#pragma unroll
  for (int i = 0; i < D / 8; ++i) f.o[i][0] = f.o[i][1] = 0.0f;
}

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

// One block: its keys at kt, its values at vt, steps ks and vs; between() is
// called when the keys have been read and before the values are.  MASK: the
// lane's row sees the block's tokens below end only.
template <int D, bool MASK, typename Between>
__device__ __forceinline__ void k8_block(K8Fast<D>& f, const uint8_t* kt, const uint8_t* vt, float ks, float vs, int end,
                                         Between between) {
  const int lane = threadIdx.x & 31, tid = lane & 3;
  float x[8][4];
#pragma unroll
  for (int j = 0; j < 8; ++j) x[j][0] = x[j][1] = x[j][2] = x[j][3] = 0.0f;
#pragma unroll
  for (int h = 0; h < D / 64; ++h)
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
          k8_numbers(s == 0 ? k[j].x : s == 1 ? k[j].y : s == 2 ? k[j].z : k[j].w, b0, b1);
          mma_f16(x[j0 + j], f.qa[h][s][0], f.qa[h][s][1], f.qa[h][s][2], f.qa[h][s][3], b0, b1);
        }
    }
  between();
  // scores: x[j][e] of token 16 tid + 2 j + e
  const float unit = ks * f.inv;
  float top = -INFINITY;
#pragma unroll
  for (int j = 0; j < 8; ++j)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      x[j][e] = fmaf(x[j][e + 2], kLowUnit, x[j][e]) * unit;
      if (MASK && 16 * tid + 2 * j + e >= end) x[j][e] = -INFINITY;
      top = fmaxf(top, x[j][e]);
    }
  const K8Share sh = k8_share<D>(f, top);
  const float ref = sh.ref, share = sh.share, weight = sh.seen ? share * vs : 0.0f;
  unsigned p[4][4];
  float sum = 0.0f;
#pragma unroll
  for (int s = 0; s < 4; ++s)
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const float pa = ex2(x[2 * s + u][0] - ref), pb = ex2(x[2 * s + u][1] - ref);
      sum += pa + pb;
      k8_parts(pa, pb, p[s][2 * u], p[s][2 * u + 1]);
    }
  f.l = fmaf(sum, share, f.l);
#pragma unroll
  for (int i0 = 0; i0 < D / 8; i0 += 4) {
    uint4 v[4];
    float y[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = *reinterpret_cast<const uint4*>(vt + (i0 + i) * 512 + lane * 16);
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        unsigned b0, b1;
        k8_numbers(s == 0 ? v[i].x : s == 1 ? v[i].y : s == 2 ? v[i].z : v[i].w, b0, b1);
        if (s == 0) mma_f16_first(y[i], p[s][0], p[s][1], p[s][2], p[s][3], b0, b1);
        else mma_f16(y[i], p[s][0], p[s][1], p[s][2], p[s][3], b0, b1);
      }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e) f.o[i0 + i][e] = fmaf(fmaf(y[i][e + 2], kLowUnit, y[i][e]), weight, f.o[i0 + i][e]);
  }
}

// the warp's sums as rows [8] of m, l and acc[D] in shared memory
template <int D>
__device__ __forceinline__ void k8_fast_store(K8Fast<D>& f, float* s_m, float* s_l, float* s_acc) {
  const int lane = threadIdx.x & 31, gid = lane >> 2, tid = lane & 3;
  f.l += __shfl_xor_sync(0xffffffffu, f.l, 1);
  f.l += __shfl_xor_sync(0xffffffffu, f.l, 2);
  if (tid == 0) { s_m[gid] = f.r; s_l[gid] = f.l; }
#pragma unroll
  for (int i = 0; i < D / 8; ++i)
    *reinterpret_cast<float2*>(s_acc + gid * D + 8 * i + 2 * tid) = make_float2(f.o[i][0], f.o[i][1]);
}

// ---------------------------------------------------- the incomplete block

__device__ __forceinline__ void mma_bf16_first(float (&d)[4], unsigned a0, unsigned a1, unsigned a2, unsigned a3, unsigned b0,
                                               unsigned b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};\n"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}
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

// Eight tokens of the incomplete block in bf16, on the tensor cores too: keys and
// queries as they are (products of two bf16 numbers are exact), weights in
// three bf16 parts.  The rows come straight from memory, sent for before the
// item's blocks are worked on, zeros past the last one.
constexpr int kK8Few = 8;
template <int D>
struct K8Rows {
  uint4 k[D / 32];        // token gid: channels 64 h + 16 tid + (0..15)
  unsigned v[D / 8];      // token gid: channels 8 i + 2 tid, + 1
};
template <int D>
__device__ __forceinline__ void k8_rows_load(K8Rows<D>& x, const __nv_bfloat16* K, const __nv_bfloat16* V, int first, int left) {
  const int lane = threadIdx.x & 31, gid = lane >> 2, tid = lane & 3;
  const bool in = first + gid < left;
  const uint4* k = reinterpret_cast<const uint4*>(K + (first + gid) * D + 16 * tid);
  const unsigned* v = reinterpret_cast<const unsigned*>(V + (first + gid) * D + 2 * tid);
#pragma unroll
  for (int i = 0; i < D / 32; ++i) x.k[i] = in ? k[i / 2 * 8 + i % 2] : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
  for (int i = 0; i < D / 8; ++i) x.v[i] = in ? v[4 * i] : 0u;
}
// ... which the lane's row sees below end (of the tokens from first on)
template <int D>
__device__ __forceinline__ void k8_rows(K8Fast<D>& f, K8Rows<D>& x, const float* s_q, int end, const __nv_bfloat16* V, int left) {
  const int lane = threadIdx.x & 31, gid = lane >> 2, tid = lane & 3;
  float s[4];
#pragma unroll
  for (int h = 0; h < D / 64; ++h)
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const float4 q = *reinterpret_cast<const float4*>(s_q + kd_q<D>(gid, 64 * h + 16 * tid) + 4 * c);
      const uint4 k = x.k[2 * h + c / 2];
      const unsigned a0 = bf16_pair(q.x, q.y), a2 = bf16_pair(q.z, q.w);
      if (h == 0 && c == 0) mma_bf16_first(s, a0, 0u, a2, 0u, k.x, k.y);
      else mma_bf16(s, a0, 0u, a2, 0u, c & 1 ? k.z : k.x, c & 1 ? k.w : k.y);
    }
  const int t0 = 2 * tid;
  const float sa = t0 < end ? s[0] * f.inv : -INFINITY, sb = t0 + 1 < end ? s[1] * f.inv : -INFINITY;
  const K8Share sh = k8_share<D>(f, fmaxf(sa, sb));
  const float pa = ex2(sa - sh.ref), pb = ex2(sb - sh.ref);
  f.l = fmaf(pa + pb, sh.share, f.l);
  // infinities and NaNs: what a row does not see must not reach it, and parts
  // that are 0 would make NaNs of infinities
  unsigned most = 0u;
#pragma unroll
  for (int i = 0; i < D / 8; ++i) {
    const unsigned u = x.v[i] & 0x7FFF7FFFu;
    most = __vmaxu2(most, u);
  }
  const bool odd = (most & 0xFFFFu) >= 0x7F80u || (most >> 16) >= 0x7F80u;
  if (__builtin_expect(__any_sync(0xffffffffu, odd), 0)) {
#pragma unroll 1
    for (int t = 0; t < kK8Few; ++t) {
      const float p = __shfl_sync(0xffffffffu, t & 1 ? pb : pa, lane & 28 | t >> 1);
      if (t >= left || t >= end) continue;
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        const unsigned u = *reinterpret_cast<const unsigned*>(V + t * D + 8 * i + 2 * tid);
        if ((u & 0x7F80u) == 0x7F80u) f.o[i][0] = fmaf(p * sh.share, bf16_low(u), f.o[i][0]);
        if ((u & 0x7F800000u) == 0x7F800000u) f.o[i][1] = fmaf(p * sh.share, bf16_high(u), f.o[i][1]);
      }
    }
#pragma unroll
    for (int i = 0; i < D / 8; ++i) {
      if ((x.v[i] & 0x7F80u) == 0x7F80u) x.v[i] &= 0xFFFF0000u;
      if ((x.v[i] & 0x7F800000u) == 0x7F800000u) x.v[i] &= 0xFFFFu;
    }
    __syncwarp();
  }
  const unsigned hi = bf16_pair(pa, pb);
  const float ra = pa - bf16_low(hi), rb = pb - bf16_high(hi);
  const unsigned mid = bf16_pair(ra, rb), lo = bf16_pair(ra - bf16_low(mid), rb - bf16_high(mid));
  // rows: high and middle parts; the second eight of the 16 summed tokens are
  // the same ones again, with the low parts
#pragma unroll
  for (int i = 0; i < D / 8; ++i) {
    const unsigned v = transpose8(x.v[i]);
    float y[4];
    mma_bf16_first(y, hi, mid, lo, 0u, v, v);
#pragma unroll
    for (int e = 0; e < 2; ++e) f.o[i][e] = fmaf(y[e] + y[e + 2], sh.share, f.o[i][e]);
  }
}

// float32: the incomplete block's tokens that fall to the warp, RT rows of its tile: first
// the ones at first, then those at step further, and so on below left.
template <int D, int RT, typename E>
__device__ __forceinline__ void k8_tail(const E* K, const E* V, int first, int step, int left, const float* q, const float* inv,
                                        const int64_t* end, int64_t p0, float* my_m, float* my_l, float* my_acc) {
  constexpr int CPL = D / 32;
  const int lane = threadIdx.x & 31;
  // the state moves on to lanes that hold channels
  __syncwarp();
  KdState<D, RT> st;
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    st.m[r] = my_m[r]; st.l[r] = my_l[r];
#pragma unroll
    for (int c = 0; c < CPL; ++c) st.acc[r][c] = my_acc[r * D + lane * CPL + c];
  }
  __syncwarp();
  // (my_acc is free until the state returns to it)
  for (int t0 = kKdStep<RT> * first; t0 < left; t0 += kKdStep<RT> * step)
    kd_step<D, RT, E>(st, K + t0 * D, V + t0 * D, min(kKdStep<RT>, left - t0), q, inv, end, p0 + t0, my_acc);
  __syncwarp();
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    if (lane == 0) { my_m[r] = st.m[r]; my_l[r] = st.l[r]; }
#pragma unroll
    for (int c = 0; c < CPL; ++c) my_acc[r * D + lane * CPL + c] = st.acc[r][c];
  }
}

// shared memory: barriers (keys full, empty, values full, empty, items full,
// empty), items, warp sums, q rows of two items, steps of the keys' slots, the rings
template <int D>
struct K8Layout {
  static constexpr int item = (4 * kK8MaxStages + 4) * 8;
  static constexpr int m = item + 2 * (int)sizeof(KdItem);
  static constexpr int l = m + kK8Warps * 8 * 4;
  static constexpr int acc = (l + kK8Warps * 8 * 4 + 15) / 16 * 16;
  static constexpr int side = acc + kK8Warps * 8 * D * 4;
  static constexpr int q = side + kK8MaxStages * 8;
  static __host__ __device__ int ring(int rows) { return (q + 2 * ((rows + 7) / 8 * 8) * (D + 16) * 4 + 127) / 128 * 128; }
};

template <int D, typename E, typename A>
__global__ void __launch_bounds__(kK8Threads, 1) kv8_decode_kernel(const A a) {
  pdl_entry();
  using Lt = K8Layout<D>;
  constexpr int W = kK8Warps;
  __shared__ KdBatch batch;
  extern __shared__ __align__(128) uint8_t k8_sm[];
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int R = kd_rows(a), Rp = (R + 7) / 8 * 8;
  // teams: warps that share a block, one tile of rows each
  const int team = k8_team(Rp / 8), nteam = W / team;
  KdRing keys, values;
  keys.full = smem_u32(k8_sm);
  keys.empty = keys.full + kK8MaxStages * 8;
  values.full = keys.empty + kK8MaxStages * 8;
  values.empty = values.full + kK8MaxStages * 8;
  const unsigned item_full = values.empty + kK8MaxStages * 8, item_empty = item_full + 16;
  keys.slots = a.slotsK;
  values.slots = a.slotsV;
  keys.data = k8_sm + Lt::ring(R);
  values.data = keys.data + a.slotsK * kBlock * D;
  KdItem* items = reinterpret_cast<KdItem*>(k8_sm + Lt::item);
  float* s_q = reinterpret_cast<float*>(k8_sm + Lt::q);        // two of [rows, padded] (kd_q)
  if (tid >= 32 && tid < 32 + kK8MaxStages) {
    // (keys full: one arrival with the codes' bytes, one of the steps' copy)
    const int i = tid - 32;
    mbar_init(keys.full + 8 * i, 2);
    mbar_init(keys.empty + 8 * i, team);
    mbar_init(values.full + 8 * i, 1);
    mbar_init(values.empty + 8 * i, team);
    if (i < 2) {
      mbar_init(item_full + 8 * i, kKdQueryWarps<8>);
      mbar_init(item_empty + 8 * i, W);
    }
    fence_barrier_init();
  }
  kd_batch(a, batch);
  const int64_t per = kd_run(batch, gridDim.x);
  int64_t u0 = (int64_t)blockIdx.x * per, u1 = min(batch.pref[kMaxB], u0 + per);

  if (w >= W) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kK8RegsProducer));
    if (blockIdx.x == 0 && w == W + 1) {
      bool bad = false;
      for (int b = lane; b < a.B; b += 32) {
        bad |= a.len[b] < 0 || a.len[b] > a.n_max;
        if (a.n_q) bad |= a.n_q[b] < 0 || a.n_q[b] > a.T;
      }
      const unsigned any = __any_sync(0xffffffffu, bad);
      // (a wait that gives up flags the word two seconds later at the earliest)
      if (lane == 0) *a.status = any ? 8u : 0u;
    }
    if (w == W) k8_produce<D>(a, batch, u0, u1, keys, smem_u32(k8_sm) + Lt::side, true);
    else if (w == W + 1) k8_produce<D>(a, batch, u0, u1, values, 0, false);
    else kd_queries<D, 8, E>(a, batch, u0, u1, items, s_q, item_full, item_empty, w - W - 2);
    return;
  }
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(kK8RegsConsumer));

  float* s_m = reinterpret_cast<float*>(k8_sm + Lt::m);        // [warps][8]
  float* s_l = reinterpret_cast<float*>(k8_sm + Lt::l);
  float* s_acc = reinterpret_cast<float*>(k8_sm + Lt::acc);    // [warps][8][D]
  const float2* side = reinterpret_cast<const float2*>(k8_sm + Lt::side);
  const int my_team = w / team, tile = w % team;
  const int rows = min(8, R - tile * 8);          // <= 0: a warp with no rows
  const int r0 = tile * 8 < Rp ? tile * 8 : 0;
  // (Each wait is bounded: one that gives up marks the call, and the warp goes
  // on without waiting.)
  bool dead = false;
  int base = 0;                                   // number of the item's first block
  int i = my_team;                                // the team's next block, its slots and their parities
  int sk = my_team, sv = my_team, pk = 0, pv = 0;
  int k = 0;                                      // number of the item
  kd_trim(a, batch, u0, u1);

  for (int64_t u = u0; u < u1; ++k) {
    const int buf = k & 1;
    if (!dead && !mbar_wait(item_full + 8 * buf, (k >> 1) & 1)) dead = true;
    dead = __any_sync(0xffffffffu, dead);
    if (dead) {
      // the way through the items does not hang on the producer
      if (lane == 0) items[buf].seg = kd_seg(a, batch, u, u1);
      __syncwarp();
    }
    const KdItem& it = items[buf];
    const float* q = s_q + kd_q<D>(buf * Rp + r0, 0);
    float* my_m = s_m + w * 8;
    float* my_l = s_l + w * 8;
    float* my_acc = s_acc + w * 8 * D;
    // the incomplete block, if it is to be done here: the teams go on in turn
    // where the blocks ended, a few tokens at a time
    const int64_t tail0 = it.seg.n / kBlock * kBlock, at = it.seg.bg * kBlock * D;
    const int left = it.seg.left, to = base + it.seg.nfast, clear = base + it.seg.clear;
    const E* Kt = reinterpret_cast<const E*>(a.c.Kt) + at;
    const E* Vt = reinterpret_cast<const E*>(a.c.Vt) + at;
    {
      K8Fast<D> f;
      k8_init<D>(f, q, it.inv + r0);
      constexpr bool few = sizeof(E) == 2;
      K8Rows<D> few_rows;
      int few_at = kBlock;
      if constexpr (few) {
        if (left > 0 && rows > 0) few_at = kK8Few * ((i < to ? i + (to - i + nteam - 1) / nteam * nteam : i) - to);
        if (few_at < left) k8_rows_load<D>(few_rows, Kt, Vt, few_at, left);
      }
      while (i < to) {
        if (!dead && !mbar_wait(keys.full + 8 * sk, pk)) dead = true;
        const float2 step = side[sk];
        const auto between = [&]() {
          __syncwarp();
          if (lane == 0) mbar_arrive(keys.empty + 8 * sk);
          if (!dead && !mbar_wait(values.full + 8 * sv, pv)) dead = true;
        };
        const uint8_t* kt = keys.data + sk * kBlock * D;
        const uint8_t* vt = values.data + sv * kBlock * D;
        if (rows <= 0) {
          between();
        } else if (i < clear) {
          k8_block<D, false>(f, kt, vt, step.x, step.y, 0, between);
        } else {
          const int64_t p0 = A::kPerToken ? it.seg.own : (it.seg.blk0 + (i - base)) * kBlock;
          k8_block<D, true>(f, kt, vt, step.x, step.y, (int)min(max(it.end[r0 + (lane >> 2)] - p0, (int64_t)0), (int64_t)kBlock),
                            between);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(values.empty + 8 * sv);
        i += nteam;
        if ((sk += nteam) >= keys.slots) { sk = my_team; pk ^= 1; }
        if ((sv += nteam) >= values.slots) { sv = my_team; pv ^= 1; }
      }
      base = to;
      if constexpr (few) {
        const int end = (int)min(max(it.end[r0 + (lane >> 2)] - tail0, (int64_t)0), (int64_t)left);
        while (few_at < left) {
          k8_rows<D>(f, few_rows, q, end - few_at, Vt + few_at * D, left - few_at);
          few_at += kK8Few * nteam;
          if (few_at < left) k8_rows_load<D>(few_rows, Kt, Vt, few_at, left);
        }
      }
      k8_fast_store<D>(f, my_m, my_l, my_acc);
    }
    if constexpr (sizeof(E) == 4) {
      if (rows > 4 && kKdStep<8> * (i - base) < left)
        k8_tail<D, 8, E>(Kt, Vt, i - base, nteam, left, q, it.inv + r0, it.end + r0, tail0, my_m, my_l, my_acc);
      else if (rows > 0 && rows <= 4 && kKdStep<4> * (i - base) < left)
        k8_tail<D, 4, E>(Kt, Vt, i - base, nteam, left, q, it.inv + r0, it.end + r0, tail0, my_m, my_l, my_acc);
    }
    bar_sync(1, W * 32);
    // merge the teams, four channels of a row to a thread
    float* part = a.part + (2 * (int64_t)blockIdx.x + (it.seg.cut0 ? 0 : 1)) * R * (D + 4);
    for (int e = tid; e < R * (D / 4); e += W * 32) {
      const int r = e / (D / 4), c = e % (D / 4) * 4;
      float M = -INFINITY, l = 0.0f;
      float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      for (int x = r; x < W * 8; x += team * 8) M = fmaxf(M, s_m[x]);   // (the row in each team)
      for (int x = r; x < W * 8; x += team * 8) {
        const float s = s_m[x] > -INFINITY ? ex2(s_m[x] - M) : s_l[x] == 0.0f ? 0.0f : 1.0f;
        const float4 y = *reinterpret_cast<const float4*>(s_acc + x * D + c);
        l = fmaf(s, s_l[x], l);
        v.x = fmaf(s, y.x, v.x); v.y = fmaf(s, y.y, v.y); v.z = fmaf(s, y.z, v.z); v.w = fmaf(s, y.w, v.w);
      }
      if (A::kPerToken && it.seg.bad) { M = 0.0f; l = v.x = v.y = v.z = v.w = NAN; }
      if (!it.seg.cut0 && !it.seg.cut1) {
        if (A::kPerToken || r / a.G < it.seg.nq) kd_store<D>(a, it.seg, r, c, M, l, v);
      } else {
        *reinterpret_cast<float4*>(part + r * (D + 4) + c) = v;
        if (c == 0) { part[r * (D + 4) + D] = M; part[r * (D + 4) + D + 1] = l; }
      }
    }
    u += it.seg.step;
    bar_sync(1, W * 32);
    if (lane == 0) mbar_arrive(item_empty + 8 * buf);
  }
  if (dead && lane == 0) atomicOr(a.status, 4u);
}

namespace {

// Items of up to this many blocks stay whole.
constexpr int64_t kK8WholeBlocks = 2 * kK8Warps;
int64_t k8_blocks(const csa_shape* s, int n_sel) {
  const int64_t blocks = (s->n_max + kBlock - 1) / kBlock;
  return n_sel && n_sel < blocks ? n_sel : blocks;
}
int k8_whole(const csa_shape* s, int n_sel) { return k8_blocks(s, n_sel) <= kK8WholeBlocks; }

// CTAs of the decode kernel: one per SM, no more than there can be units
int k8_ctas(const csa_shape* s, int T, int n_sel) {
  const int64_t units = (int64_t)s->B * s->Hkv * (n_sel ? T : 1) * (k8_whole(s, n_sel) ? 1 : k8_blocks(s, n_sel));
  const int nsm = sm_count() < kKdMaxCtas ? sm_count() : kKdMaxCtas;
  return (int)(units < nsm ? units : nsm);
}

size_t k8_workspace(const csa_shape* s, int T, int n_sel) {
  const int R = (n_sel ? 1 : T) * (s->Hq / s->Hkv);
  return 256 + (k8_whole(s, n_sel) ? 0 : (size_t)2 * k8_ctas(s, T, n_sel) * R * (s->d + 4) * 4);
}

// Dynamic shared memory there can be: a CTA's 227 KB without the kernel's own.
// The limit is set to this on every call, whatever the call needs: it belongs to
// the function, and another host thread's call may lie between the setting and
// the launch.
constexpr int kK8SharedBytes = 232448 - ((int)sizeof(KdBatch) + 127) / 128 * 128;
template <int D, typename E, typename A>
cudaError_t launch_kv8_decode_t(A a, int ncta, cudaStream_t st) {
  const int R = kd_rows(a), rest = K8Layout<D>::ring(R);
  // one slot per team in each ring (an SM's shared memory holds that for every
  // number of rows), then more while there is room: keys first, whose copies
  // have less time (the values' come while the warp is at the keys)
  constexpr int bytes = kBlock * D;
  const int nteam = kK8Warps / k8_team((R + 7) / 8);
  int nk = 1, nv = 1;
  for (bool more = true; more;) {
    more = false;
    if ((nk + 1) * nteam <= kK8MaxStages && nteam * (nk + 1 + nv) * bytes <= kK8SharedBytes - rest) { ++nk; more = true; }
    if ((nv + 1) * nteam <= kK8MaxStages && nteam * (nk + nv + 1) * bytes <= kK8SharedBytes - rest) { ++nv; more = true; }
  }
  a.slotsK = nk * nteam;
  a.slotsV = nv * nteam;
  const int smem = rest + (a.slotsK + a.slotsV) * bytes;
  const cudaError_t e =
      cudaFuncSetAttribute(kv8_decode_kernel<D, E, A>, cudaFuncAttributeMaxDynamicSharedMemorySize, kK8SharedBytes);
  if (e != cudaSuccess) return e;
  launch_pdl(kv8_decode_kernel<D, E, A>, dim3(ncta), dim3(kK8Threads), smem, st, a);
  if (ncta > 1 && !a.whole)
    launch_pdl(decode_join_kernel<D, A>, dim3(ncta - 1, (R + kKdJoinWarps - 1) / kKdJoinWarps), dim3(kKdJoinWarps * 32), 0, st, a, ncta);
  return cudaGetLastError();
}
template <typename A>
cudaError_t launch_kv8_decode(const A& a, int d, bool bf16, int ncta, cudaStream_t st) {
  return d == 128 ? (bf16 ? launch_kv8_decode_t<128, __nv_bfloat16>(a, ncta, st) : launch_kv8_decode_t<128, float>(a, ncta, st))
                  : (bf16 ? launch_kv8_decode_t<64, __nv_bfloat16>(a, ncta, st) : launch_kv8_decode_t<64, float>(a, ncta, st));
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
  a.whole = k8_whole(shape, n_sel);
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
  return n_sel >= 0 && n_sel <= CSA_KV8_MAX_SEL && k8_args_ok(shape, T, &st) ? k8_workspace(shape, T, n_sel) : 0;
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
