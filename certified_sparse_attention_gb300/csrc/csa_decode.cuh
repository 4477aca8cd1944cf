// Decode attention over a K/V cache whose whole blocks of 64 tokens are held
// in codes and whose incomplete last block is held in full precision: what the
// kernels for the different codes share.  That is how the batch's work is dealt
// to the CTAs, the queries of an item, the rows' outputs and the join of items
// that were cut.
//
// The argument block A of a kernel is derived from DecodeArgs and says
//   kLead, kTailBase, kTailStep   what an item and its incomplete block cost, in
//                                 units of one whole block (kd_tail)
//   kPerToken                     an item is one query token (of one sequence and
//                                 KV head), which attends to a list of blocks of
//                                 its own, n_sel at most; otherwise an item is
//                                 all tokens of a sequence, over all its blocks
//   kMaxCtas                      CTAs of a call at most
//   kPlainQ                       query rows keep their own digits: log2(e) /
//                                 sqrt(d) goes into what undoes a row's scale
//   put<D>(q, r, lane, x, up)     lays channels lane D / 32 ... of query row r,
//                                 x up, down in shared memory
//   kTop, top<D>(c)               whether the kernel wants to know of the channel c
//                                 of a row's largest query element, and what
#pragma once

#include <type_traits>

#include <cuda_fp16.h>

#include "csa_args.cuh"

namespace csa {

struct DecodeArgs {
  const void* q;
  csa_strides qs;
  const int64_t* len;
  const int64_t* n_q;
  float* o;
  float* lse;
  unsigned* status;
  float* part;          // [2 * CTAs][rows][D + 4]: acc[D], m, l, unused
  int64_t n_max, nblk_max;
  int B, T, Hq, Hkv, G;
  int whole;            // items are not cut: one unit each
  float rs;             // log2(e) / sqrt(d): scores in units of log 2
};

// rows of an item
template <typename A>
__host__ __device__ __forceinline__ int kd_rows(const A& a) { return A::kPerToken ? a.G : a.T * a.G; }

// What the kernels know of the batch.  An item is one sequence and KV head
// (kPerToken: and query token, of those below n_q).
// Its units of work, in order: kLead for its own cost (its queries, the
// merge), its whole blocks, and what its incomplete block costs.
struct KdBatch {
  int64_t pref[kMaxB + 1];    // units of the sequences before b (pref[B]: all)
  int64_t len[kMaxB];
  int nq[kMaxB];
};

// units of the incomplete block (an empty item has one)
template <typename A>
__device__ __forceinline__ int kd_tail(int64_t n) {
  const int left = (int)(n % kBlock);
  return left ? A::kTailBase + left / A::kTailStep : n == 0;
}
// whole blocks of an item (kPerToken: there can be in its list)
template <typename A>
__device__ __forceinline__ int64_t kd_blocks(const A& a, int64_t n) {
  if constexpr (A::kPerToken) return min(n / kBlock, (int64_t)a.n_sel);
  else return n / kBlock;
}
template <typename A>
__device__ __forceinline__ int64_t kd_units(const A& a, int64_t n) {
  return a.whole ? 1 : A::kLead + kd_blocks(a, n) + kd_tail<A>(n);
}

// by warp 0, then a barrier of the CTA
template <typename A>
__device__ __forceinline__ void kd_batch(const A& a, KdBatch& s) {
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    int64_t u[4], sum = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int b = lane * 4 + i;
      u[i] = 0;
      if (b < a.B) {
        const int64_t n = min(max(a.len[b], (int64_t)0), a.n_max);
        s.len[b] = n;
        s.nq[b] = a.n_q ? (int)min(max(a.n_q[b], (int64_t)0), (int64_t)a.T) : a.T;
        u[i] = kd_units(a, n) * a.Hkv;
        if constexpr (A::kPerToken) u[i] *= s.nq[b];
      }
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
      s.pref[lane * 4 + i] = before;
      before += u[i];
    }
    if (lane == 31) s.pref[kMaxB] = before;
  }
  __syncthreads();
}

// the part of an item that lies in the run [u, u1) of a CTA
struct KdSeg {
  int64_t bg, n, blk0;     // its first block
  int64_t step;            // its units
  int64_t start, last;     // the item's first and last units that stand for work done where they lie
  int b, g, nq;
  int nfast;               // whole blocks
  int clear;               // of those, the first `clear` are seen in full by every row
  int left;                // tokens of the incomplete block
  bool any;                // there is something to do
  bool cut0, cut1;         // the item has parts in the run before, in the one after
};
// ... of one query token
struct KdTokenSeg : KdSeg {
  int t;                   // the query token
  bool bad;                // its list is not one (kd_list)
  int64_t own;             // first position of the token's own block
};
template <typename A>
using KdSegOf = std::conditional_t<A::kPerToken, KdTokenSeg, KdSeg>;

// item i of sequence b, whose units begin at v0 of them at unit u
template <typename A>
__device__ __forceinline__ KdSegOf<A> kd_seg_at(const A& a, const KdBatch& batch, int b, int i, int64_t units, int64_t v0, int64_t u,
                                                int64_t u1) {
  KdSegOf<A> s;
  s.b = b;
  s.n = batch.len[b];
  s.nq = batch.nq[b];
  const int64_t whole = kd_blocks(a, s.n), v1 = min(units, v0 + (u1 - u));
  s.g = i;
  if constexpr (A::kPerToken) {
    s.t = s.g / a.Hkv;
    s.g -= s.t * a.Hkv;
    s.bad = false;
  }
  s.bg = (int64_t)s.b * a.Hkv + s.g;
  s.step = v1 - v0;
  // Work begins with the first block; the incomplete block is done where the
  // middle of its units lies.
  const int tail = kd_tail<A>(s.n);
  const int64_t w0 = a.whole ? 0 : A::kLead, w1 = a.whole ? 0 : A::kLead + whole + (tail ? tail / 2 : -1);
  s.start = u - v0 + w0;
  s.last = u - v0 + w1;
  s.any = v0 <= w1 && v1 > w0;
  s.cut0 = v0 > w0;
  s.cut1 = v1 <= w1;
  s.blk0 = a.whole ? 0 : min(max(v0 - A::kLead, (int64_t)0), whole);
  s.nfast = (int)((a.whole ? whole : min(max(v1 - A::kLead, (int64_t)0), whole)) - s.blk0);
  s.left = v0 <= w1 && w1 < v1 ? (int)(s.n % kBlock) : 0;
  // the first row sees positions below n - nq + 1
  const int64_t clear = max(s.n - s.nq + 1, (int64_t)0) / kBlock - s.blk0;
  s.clear = (int)min(max(clear, (int64_t)0), (int64_t)s.nfast);
  return s;
}
template <typename A>
__device__ __forceinline__ KdSegOf<A> kd_seg(const A& a, const KdBatch& batch, int64_t u, int64_t u1) {
  // the last b with pref[b] <= u (sequences past B hold no units)
  int lo = 0, hi = a.B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (batch.pref[mid] <= u) lo = mid; else hi = mid - 1;
  }
  const int64_t units = kd_units(a, batch.len[lo]), rem = u - batch.pref[lo];
  const int i = (rem | units) >> 32 ? (int)(rem / units) : (int)((unsigned)rem / (unsigned)units);
  return kd_seg_at(a, batch, lo, i, units, rem - i * units, u, u1);
}
// the one after s, at its end u < u1
template <typename A>
__device__ __forceinline__ KdSegOf<A> kd_next(const A& a, const KdBatch& batch, const KdSegOf<A>& s, int64_t u, int64_t u1) {
  int b = s.b, i = s.g + 1;
  if constexpr (A::kPerToken) i += s.t * a.Hkv;
  if (u >= batch.pref[b + 1]) {
    i = 0;
    do ++b;
    while (u >= batch.pref[b + 1]);
  }
  return kd_seg_at(a, batch, b, i, kd_units(a, batch.len[b]), 0, u, u1);
}

// kPerToken: list entries of an item that its queries' warps leave in shared memory
constexpr int kKdIds = 128;
// kPerToken: the item's list of blocks, of which [blk0, blk0 + nfast) are the
// run's; by a whole warp.  A list is ascending and ends at the token's own block
// at the latest, so only its last entry can be the incomplete block, or a whole
// one that the token does not see in full.
template <typename A>
__device__ __forceinline__ const int32_t* kd_list(const A& a, KdTokenSeg& s) {
  const int lane = threadIdx.x & 31;
  const int64_t row = ((int64_t)s.b * a.T + s.t) * a.Hkv + s.g, pos = s.n - s.nq + s.t;
  const int32_t* ids = a.blocks + row * a.n_sel;
  const int64_t own = pos < 0 ? -1 : pos / kBlock;
  // (entries are looked at from `count` on too, so that nothing waits for it)
  const int count = a.count[row];
  bool bad = count < 0 || count > a.n_sel;
  int end = -1;
  for (int x = lane; x < a.n_sel; x += 32) {
    const int id = ids[x], before = x ? ids[x - 1] : -1;
    bad |= x < count && (id <= before || id > own);
    if (x == count - 1) end = id;
  }
  s.bad = __any_sync(0xffffffffu, bad);
  const int64_t last = s.bad ? -1 : __reduce_max_sync(0xffffffffu, end);
  const bool tail = last == s.n / kBlock;
  const int coded = s.bad ? 0 : count - tail;
  s.own = own * kBlock;
  s.nfast = (int)max(min(s.blk0 + s.nfast, (int64_t)coded) - s.blk0, (int64_t)0);
  s.clear = (int)min(max(coded - (last == own && !tail) - s.blk0, (int64_t)0), (int64_t)s.nfast);
  if (!tail) s.left = 0;
  return ids;
}

// units of a CTA's run
__device__ __forceinline__ int64_t kd_run(const KdBatch& batch, int ncta) {
  return (batch.pref[kMaxB] + ncta - 1) / ncta;
}
// the run without what is nothing to do at its ends: the units of an item whose
// work lies in the run before or in the one after
template <typename A>
__device__ __forceinline__ void kd_trim(const A& a, const KdBatch& batch, int64_t& u0, int64_t& u1) {
  if (a.whole || u0 >= u1) return;
  const KdSegOf<A> s = kd_seg(a, batch, u0, u1), e = kd_seg(a, batch, u1 - 1, u1);
  if (e.start >= u1) u1 = max(u0, e.start - A::kLead);
  if (!s.any) u0 = min(u1, u0 + s.step);
}

// writes four channels of a finished row
template <int D, typename A>
__device__ __forceinline__ void kd_store(const A& a, const KdSegOf<A>& s, int r, int c, float M, float l, float4 v) {
  int t = r / a.G, h = s.g * a.G + r % a.G;
  if constexpr (A::kPerToken) { t = s.t; h = s.g * a.G + r; }
  const int64_t row = ((int64_t)s.b * a.T + t) * a.Hq + h;
  // l = 0 only where nothing was attended to
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  if (l == 0.0f) v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  *reinterpret_cast<float4*>(a.o + row * D + c) = make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv);
  if (c == 0 && a.lse) a.lse[row] = l == 0.0f ? -INFINITY : (M + log2f(l)) * 0.69314718055994531f;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// ------------------------------------------------------ tensor-core blocks

__device__ __forceinline__ void mma_f16(float (&d)[4], unsigned a0, unsigned a1, unsigned a2, unsigned a3, unsigned b0,
                                        unsigned b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// the same with d = 0 before
__device__ __forceinline__ void mma_f16_first(float (&d)[4], unsigned a0, unsigned a1, unsigned a2, unsigned a3, unsigned b0,
                                              unsigned b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};\n"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}
__device__ __forceinline__ unsigned transpose8(unsigned x) {
  unsigned y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(y) : "r"(x));
  return y;
}
// two float32 numbers as half-precision parts: hi = the rounded pair (x low,
// y high), lo = the rounded remainders
__device__ __forceinline__ unsigned half_pair(float x, float y) {
  const __half2 h = __floats2half2_rn(x, y);
  return *reinterpret_cast<const unsigned*>(&h);
}
// 2^k, -126 <= k <= 127
__device__ __forceinline__ float pow2i(int k) { return __int_as_float((127 + k) << 23); }
// exponent of x > 0 (subnormals: -127)
__device__ __forceinline__ int exponent(float x) { return (int)(__float_as_uint(x) >> 23) - 127; }
// The queries of an item and what else its warps need of it: filled by producer
// warps, four rows at a time, ahead of the sums.  Query rows are log2(e) / sqrt(d) q
// (kPlainQ: q) times a power of two that puts the row's largest at 2^11 .. 2^12
// (undone by inv), laid out by A::put.
template <typename A>
struct KdPlainItem {
  KdSegOf<A> seg;
  int64_t end[CSA_KV4_MAX_ROWS];    // row r sees positions below end[r]
  float inv[CSA_KV4_MAX_ROWS];      // undoes the scale of row r
};
template <typename A>
struct KdTopItem : KdPlainItem<A> {
  int top[CSA_KV4_MAX_ROWS];        // of the channel of the largest of row r: A::top
};
template <typename A>
using KdItem = std::conditional_t<A::kTop, KdTopItem<A>, KdPlainItem<A>>;

// the rows [r0, r1) of an item, but for it.seg
template <int D, typename E, typename A>
__device__ __forceinline__ void kd_item_queries(const A& a, const KdSegOf<A>& sg, KdItem<A>& it, float* q, int r0, int r1) {
  constexpr int CPL = D / 32;
  const int lane = threadIdx.x & 31;
  const E* base = reinterpret_cast<const E*>(a.q) + sg.b * a.qs.b + (int64_t)sg.g * a.G * a.qs.h + lane * CPL;
#pragma unroll 4
  for (int r = r0; r < r1; ++r) {
    int t = r / a.G;
    if constexpr (A::kPerToken) t = r < a.G ? sg.t : a.T;
    float x[CPL];
#pragma unroll
    for (int c = 0; c < CPL; ++c) x[c] = 0.0f;
    if (t < sg.nq) {
      const E* src = base + t * a.qs.t + (A::kPerToken ? r : r - t * a.G) * a.qs.h;
      if (CPL == 4) {
        const float4 v = Elem<E>::get4(src);
        x[0] = v.x; x[1] = v.y; x[CPL - 2] = v.z; x[CPL - 1] = v.w;
      } else {
        const float2 v = Elem<E>::get2(src);
        x[0] = v.x; x[1] = v.y;
      }
    }
    // the row's largest in magnitude, without its last 7 bits, and (kTop) its channel
    unsigned key = 0;
#pragma unroll
    for (int c = 0; c < CPL; ++c) {
      if constexpr (!A::kPlainQ) x[c] *= a.rs;
      key = max(key, (__float_as_uint(x[c]) & 0x7fffff80u) + (A::kTop ? lane * CPL + c : 0));
    }
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) key = max(key, __shfl_xor_sync(0xffffffffu, key, m));
    const float top = __uint_as_float(key & ~127u);
    const int e = top > 0.0f && top < INFINITY ? min(max(11 - exponent(top), -100), 100) : 0;
    const float up = pow2i(e);
    A::template put<D>(q, r, lane, x, up);
    if (lane == 0) {
      if constexpr (A::kTop) it.top[r] = A::template top<D>((int)(key & 127));
      it.inv[r] = A::kPlainQ ? a.rs * pow2i(-e) : pow2i(-e);
      it.end[r] = t < sg.nq ? sg.n - sg.nq + t + 1 : 0;
    }
  }
}

// Joins the parts of the items that were cut: CTAs (j, y) own the item of
// which CTA j of the decode kernel did the beginning, if it did not do all of
// it; a warp to a row, eight rows to a CTA.  Which item that is depends on the
// lengths alone, so it is found before the wait for the decode kernel (whose
// own wait has seen the lengths written; CTAs with nothing to do wait too:
// the next kernel takes this grid's end for the decode kernel's).  Weights and
// the first eight parts are read at once: done one after the other, eight rows
// to a CTA's eight warps in turn, the join took 10 us after a batch of 64 and
// 17 after drafts of 24 rows.
constexpr int kKdJoinWarps = 8;
template <int D, typename A>
__global__ void __launch_bounds__(kKdJoinWarps * 32) decode_join_kernel(const A a, int ncta) {
  __shared__ KdBatch batch;
  __shared__ float s_w[kKdJoinWarps][A::kMaxCtas];
  kd_batch(a, batch);
  if (A::kPerToken && batch.pref[kMaxB] == 0) {      // no query token at all
    pdl_entry();
    return;
  }
  const int64_t per = kd_run(batch, ncta), x = min(((int64_t)blockIdx.x + 1) * per, batch.pref[kMaxB] - 1);
  const KdSegOf<A> s = kd_seg(a, batch, x, x + 1);
  const int c0 = (int)(s.start / per), parts = (int)(s.last / per) - c0 + 1;
  const int R = kd_rows(a), lane = threadIdx.x & 31, w = threadIdx.x >> 5, r = blockIdx.y * kKdJoinWarps + w;
  pdl_entry();
  if (c0 != (int)blockIdx.x || parts == 1 || r >= R || (!A::kPerToken && r / a.G >= s.nq)) return;
  // part 0 is the last one of its CTA, the others the first ones
  const int64_t stride = (int64_t)R * (D + 4);
  const float* part0 = a.part + (2 * (int64_t)c0 + 1) * stride + r * (D + 4);
  const float* part1 = a.part + 2 * (int64_t)c0 * stride + r * (D + 4);
  const auto at = [&](int k) { return k ? part1 + 2 * k * stride : part0; };
  const int c = lane % (D / 4) * 4;
  float4 y[8];
#pragma unroll
  for (int k = 0; k < 8; ++k)
    if (k < parts) y[k] = *reinterpret_cast<const float4*>(at(k) + c);
  float M = -INFINITY, l = 0.0f;
  for (int k = lane; k < parts; k += 32) {
    const float2 ml = *reinterpret_cast<const float2*>(at(k) + D);
    // (the running maximum of the lane's own parts)
    const float top = fmaxf(M, ml.x), ref = top > -INFINITY ? top : 0.0f;
    l = l * ex2(M - ref) + ml.y * (ml.x > -INFINITY ? ex2(ml.x - ref) : ml.y == 0.0f ? 0.0f : 1.0f);
    M = top;
    s_w[w][k] = ml.x > -INFINITY ? ml.x : ml.y == 0.0f ? -INFINITY : NAN;
  }
  float top = M;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  const float ref = top > -INFINITY ? top : 0.0f;
  l *= ex2(M - ref);
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  __syncwarp();
  float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int k0 = 0; k0 < parts; k0 += 8) {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k0 && k0 + k < parts) y[k] = *reinterpret_cast<const float4*>(at(k0 + k) + c);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (k0 + k >= parts) continue;
      const float e = ex2(s_w[w][k0 + k] - ref);
      v[0] = fmaf(e, y[k].x, v[0]); v[1] = fmaf(e, y[k].y, v[1]); v[2] = fmaf(e, y[k].z, v[2]); v[3] = fmaf(e, y[k].w, v[3]);
    }
  }
  if (lane < D / 4) kd_store<D>(a, s, r, c, top, l, make_float4(v[0], v[1], v[2], v[3]));
}

}  // namespace csa
