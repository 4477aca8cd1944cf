// Decode attention over the 4-bit K/V cache (csa_kv4_decode):
//   o = softmax(q K^T / sqrt d) V
// for the last T tokens of every sequence, K and V the values the cache
// stands for (whole blocks of 64 tokens in codes, the incomplete last block
// in full precision).
//
// Work is split over the long axis by units of about one block of one
// (sequence, KV head), an item: the units of the whole batch, in order, are
// dealt to the CTAs in equal runs, whatever the lengths, which are read on the
// device.  A CTA walks its run item by item; its warps take the blocks in
// turn, each with its own running maximum and sums, and merge them in shared
// memory.  An item that lies in one CTA is finished there; the parts of the
// others (at most two per CTA, of its first and its last item) go to the
// workspace, and a second kernel joins them.  Where no sequence can be longer
// than 24 blocks, items are not cut and there is no second kernel.
//
// The rows of an item are its T * G query vectors (G query heads share the
// KV head).  A warp handles a tile of 4 or 8 rows; with more than 8 rows the
// warps of a CTA form teams of 2 to 8 that share the blocks.
//
// Whole blocks go through the tensor cores with the codes themselves as one
// operand.  A key is k_c = m_c + Delta_c n_c, so
//   q.k = sum_c q_c m_c + sum_c (q_c Delta_c) n_c,
// and a value row is v = m_t + Delta_t n, so
//   sum_t p_t v_t = sum_t p_t m_t + sum_t (p_t Delta_t) n_t :
// no code is ever converted or scaled.  A nibble in a zeroed 16-bit word is
// already a half-precision number (n 2^-17 in bits 7..10), which matrix
// instructions multiply exactly: eight codes cost four shifts and four ANDs.
// The instructions line products up by their operands' exponents and count
// leading zeros as digits, so nibbles stand as high as they can (at bits 0..3
// and 4..7, two shifts less, the 128K-token output was off by 2.3e-5), and they
// truncate their sums, so the small parts below have sums of their own.
// The other operand, q_c Delta_c or p_t Delta_t, is scaled by a power of two
// to the top of the half-precision range and split into two halves (22 bits:
// a single one would leave 2^-12 of every score), and the products are
// summed in float32.  Each row has scales of its own, which follow the products
// themselves (kd_rescale, kd_scale_fit): what a row does not attend to, and
// channels that its query is small in, cost it no digits.  Over 40 random
// shapes the outputs' error against 64 bits is 0.88 times that of the same
// attention in float32 (mean of the ratios; the largest 2.0).  With up to 4
// rows the two parts fill the 8 columns of one instruction (m16n8k16: codes are
// the 16-row side); with 8 rows each part takes an instruction.  The incomplete
// block takes a plain path (kd_step).
//
// Blocks come by bulk copies into two rings of shared memory, keys and values,
// each slot on an mbarrier; producer warps run ahead over the items, so the
// first blocks and the queries of the next item are on their way while the
// current one is merged.
//
// What bounds it: neither the memory (15 to 58% busy) nor the tensor pipe (21 to
// 34%) nor the issue slots (48 to 54%), but latency: a block is a chain of about
// 1300 instructions of its warp, with 8 rows 1600, and registers allow three
// such warps to a scheduler.  (With d = 128, 8 rows spill 136 bytes a thread, 100
// without the producers' code, and 4 rows of float32 queries 80.)  Four
// sequences of 128K tokens, 8 KV heads, 4 query heads each: 136 us for 638 MB,
// 4.7 TB/s, 69% of the copy bandwidth.  Batch of 64, up to 8K tokens, 8 query
// heads each: 131 us for 369 MB, 2.8 TB/s.  Before the codes went through the
// tensor cores those were 1250 and 1217 us.
#include <cmath>

#include "csa_decode.cuh"

namespace csa {

constexpr int kKdWarps = 12;      // consumer warps of a CTA: three warpgroups; a fourth
                                  // one's warps send for the blocks and the queries
constexpr int kKdThreads = (kKdWarps + 4) * 32;
// registers: 512 threads start with 128 each; the producers give theirs up
constexpr int kKdRegsConsumer = 152, kKdRegsProducer = 56;
static_assert(3 * kKdRegsConsumer + kKdRegsProducer <= 4 * 128, "more registers than the launch has");
constexpr int kKdMaxStages = 24;  // slots of a ring
// warps of a team, for 1 .. 8 tiles (above 6 tiles: one team, four warps left
// over)
__host__ __device__ constexpr int kd_team(int ntile) { return ntile <= 4 ? ntile : ntile <= 6 ? 6 : 8; }

// One block in shared memory: the keys' part (codes, bounds) in one ring, the
// values' (codes, token scales) in another.  The bounds lie in eight pieces 16
// bytes apart, so that the four channel ranges of a warp's lanes start in
// different banks (in one piece they would start in the same ones).
template <int D>
struct KdStage {
  static constexpr int PIECE = D;                       // bytes: D / 4 floats
  static constexpr int PITCH = PIECE + 16;
  static constexpr int B = kBlock * D / 2;              // keys: codes, then the bounds
  static constexpr int bytesK = B + 8 * PITCH;
  static constexpr int S = kBlock * D / 2;              // values: codes, then the token scales
  static constexpr int bytesV = S + kBlock * 8;
};

// The query rows of an item in shared memory: row r starts at r (D + 16), its
// channels in four pieces 4 floats apart (bank offsets, as for the bounds).
template <int D> __host__ __device__ __forceinline__ constexpr int kd_q(int r, int c) { return r * (D + 16) + c + c / (D / 4) * 4; }

struct Kv4DecodeArgs : DecodeArgs {
  csa_kv4 c;
  int slotsK, slotsV;   // slots of the two rings: multiples of the number of teams

  // What an item and its incomplete block cost, in blocks (KdBatch).  The weights
  // follow fits to the times of single CTAs (batch of 64, 8 query heads to a KV
  // head: a block 0.30 us, an item 3.8 to 4.6 us, an incomplete block 1.7 us and
  // 0.06 us a token).  With 16 units for an item and one for its incomplete
  // block the last CTA of that batch took 144 us where the mean was 119; a lead
  // of 8 and of 12 with lighter incomplete blocks took 133 and 131 us for the
  // call, this 128 (drafts of 24 rows 116, 117 and 120).  The fit is that batch's,
  // twelve teams of one warp; larger teams, whose blocks weigh more beside an
  // item's own cost, have the same weights and would want a smaller lead.  An item
  // whose sequence has no query token (n_q = 0) is walked like any other.
  static constexpr int kLead = 16, kTailBase = 6, kTailStep = 4;
  static constexpr bool kPerToken = false, kPlainQ = false, kTop = true;
  static constexpr int kMaxCtas = 256;     // one per SM
  template <int D>
  static __device__ __forceinline__ void put(float* q, int r, int lane, const float (&x)[D / 32], float up) {
#pragma unroll
    for (int c = 0; c < D / 32; ++c) q[kd_q<D>(r, lane * (D / 32)) + c] = x[c] * up;
  }
  // where a block holds Delta_c
  template <int D>
  static __device__ __forceinline__ int top(int c) {
    return KdStage<D>::B + (4 + c / (D / 4)) * KdStage<D>::PITCH + c % (D / 4) * 4;
  }
};

// what the high parts hi of x and y (half_pair) leave out
__device__ __forceinline__ unsigned half_rest(float x, float y, unsigned hi) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hi));
  return half_pair(x - f.x, y - f.y);
}
// the pair (x low, y high) in half precision, truncated
__device__ __forceinline__ unsigned half_pair_rz(float x, float y) {
  unsigned r;
  asm("cvt.rz.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(y), "f"(x));
  return r;
}

template <int D, int RT>
struct KdState {
  float m[RT], l[RT], acc[RT][D / 32];
};

// CNT consecutive elements (16 bytes aligned) as floats
template <int CNT>
__device__ __forceinline__ void kd_floats(const float* p, float (&x)[CNT]) {
#pragma unroll
  for (int i = 0; i < CNT; i += 4) {
    const float4 v = *reinterpret_cast<const float4*>(p + i);
    x[i] = v.x; x[i + 1] = v.y; x[i + 2] = v.z; x[i + 3] = v.w;
  }
}
template <int CNT>
__device__ __forceinline__ void kd_floats(const __nv_bfloat16* p, float (&x)[CNT]) {
#pragma unroll
  for (int i = 0; i < CNT; i += 8) {
    const uint4 v = *reinterpret_cast<const uint4*>(p + i);
    const unsigned u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 8; ++e) x[i + e] = __uint_as_float(e & 1 ? u[e / 2] & 0xFFFF0000u : u[e / 2] << 16);
  }
}

// One online-softmax step of a warp over `have` <= NT full-precision tokens at
// K, V (rows of D), the first at position pos.  Scores: lane (gid,
// tid) takes token gid and the channels [tid NC, (tid + 1) NC) of every query
// row; values: a lane takes the channels [lane D / 32, ...) of the state st, the
// weights come through s_p ([NT][RT] floats).  Row r sees positions below
// s_end[r].
//
// With 8 rows four tokens to a step, so that more warps share a block's tokens
// (batch of 64: 128 us, with eight 130; drafts of 24 rows 120 and 123); with 4
// rows, where a step costs half, eight (one sequence of 1000 tokens: 12.5 us,
// with four 14.4: some warps then have steps after their second block).
template <int RT> constexpr int kKdStep = RT == 8 ? 4 : 8;
template <int D, int RT, typename E>
__device__ __forceinline__ void kd_step(KdState<D, RT>& st, const E* K, const E* V, int have, const float* s_q,
                                        const float* s_inv, const int64_t* s_end, int64_t pos, float* s_p) {
  constexpr int CPL = D / 32, NT = kKdStep<RT>, LPT = 32 / NT, NC = D / LPT;
  const int lane = threadIdx.x & 31, gid = lane / LPT, tid = lane % LPT;
  float vv[NT][CPL];
#pragma unroll
  for (int e = 0; e < NT; ++e) {
#pragma unroll
    for (int c = 0; c < CPL; ++c) vv[e][c] = 0.0f;
    if (e < have) {
      if (CPL == 4) {
        const float4 v = Elem<E>::get4(V + e * D + lane * CPL);
        vv[e][0] = v.x; vv[e][1] = v.y; vv[e][CPL - 2] = v.z; vv[e][CPL - 1] = v.w;
      } else {
        const float2 v = Elem<E>::get2(V + e * D + lane * CPL);
        vv[e][0] = v.x; vv[e][1] = v.y;
      }
    }
  }
  float k[NC], s[RT];
  kd_floats<NC>(K + (gid < have ? gid : 0) * D + tid * NC, k);
  bool cut = have < NT;                   // some row does not see some token
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    float even = 0.0f, odd = 0.0f;
#pragma unroll
    for (int i = 0; i < NC; i += 4) {
      const float4 q = *reinterpret_cast<const float4*>(s_q + kd_q<D>(r, tid * NC) + i);
      even = fmaf(k[i], q.x, even); odd = fmaf(k[i + 1], q.y, odd);
      even = fmaf(k[i + 2], q.z, even); odd = fmaf(k[i + 3], q.w, odd);
    }
    s[r] = (even + odd) * s_inv[r];
    cut = cut || s_end[r] < pos + NT;
  }
#pragma unroll
  for (int m = 1; m < LPT; m <<= 1)
#pragma unroll
    for (int r = 0; r < RT; ++r) s[r] += __shfl_xor_sync(0xffffffffu, s[r], m);
  float top[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    if (gid >= have || pos + gid >= s_end[r]) s[r] = -INFINITY;
    top[r] = s[r];
  }
#pragma unroll
  for (int m = LPT; m < 32; m <<= 1)
#pragma unroll
    for (int r = 0; r < RT; ++r) top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], m));
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    const float mn = fmaxf(st.m[r], top[r]), ref = mn > -INFINITY ? mn : 0.0f;
    const float old = ex2(st.m[r] - ref);
    st.m[r] = mn;
    st.l[r] *= old;
#pragma unroll
    for (int c = 0; c < CPL; ++c) st.acc[r][c] *= old;
    // an unseen token is marked
    const bool seen = gid < have && pos + gid < s_end[r];
    if (r * LPT / RT == tid) s_p[gid * RT + r] = seen ? ex2(s[r] - ref) : -1.0f;
  }
  __syncwarp();
#pragma unroll
  for (int e = 0; e < NT; ++e) {
    float p[RT];
#pragma unroll
    for (int r = 0; r < RT; r += 4) {
      const float4 v = *reinterpret_cast<const float4*>(s_p + e * RT + r);
      p[r] = v.x; p[r + 1] = v.y; p[r + 2] = v.z; p[r + 3] = v.w;
    }
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      // an unseen token's value may be anything: it is left out, not
      // multiplied by zero
      if (!cut || !(p[r] < 0.0f)) {
        st.l[r] += p[r];
#pragma unroll
        for (int c = 0; c < CPL; ++c) st.acc[r][c] = fmaf(p[r], vv[e][c], st.acc[r][c]);
      }
    }
  }
  __syncwarp();
}

// ------------------------------------------------------- moving the blocks

// A ring of slots with full and empty barriers.  Block i sits in slot i %
// slots and is taken by team i % teams; slots is a multiple of teams, so a
// slot serves one team, which has seen its last phase when it waits for the
// next.
struct KdRing {
  uint8_t* data;
  unsigned full, empty;
  int slots;
};

// A producer warp: sends for the keys' or the values' parts of the CTA's
// tensor-core blocks in order, as slots come free: the codes by one bulk
// copy, the bounds or token scales by 16-byte copies of the lanes (eight bulk
// copies of 128 bytes, one for each piece of the bounds, held the 128K-token
// step at 62% of the memory's rate).
template <int D>
__device__ __forceinline__ void kd_produce(const Kv4DecodeArgs& a, const KdBatch& batch, int64_t u0, int64_t u1,
                                           const KdRing& ring, bool keys) {
  using St = KdStage<D>;
  constexpr int codes = kBlock * D / 2;
  const int lane = threadIdx.x & 31;
  const unsigned size = keys ? St::bytesK : St::bytesV;
  const unsigned side = keys ? 8 * D : kBlock * 8;        // bytes of the bounds, of the scales
  const uint8_t* src = keys ? a.c.K4 : a.c.V4;
  const uint8_t* side_src = reinterpret_cast<const uint8_t*>(keys ? a.c.bounds : a.c.vscale) + lane * 16;
  // where the lane's 16 bytes go, and (keys, d = 128) its other 16: 512 bytes on
  const unsigned to0 = codes + (keys ? lane * 16 / St::PIECE * St::PITCH + lane * 16 % St::PIECE : lane * 16);
  const unsigned to1 = codes + (lane * 16 + 512) / St::PIECE * St::PITCH + lane * 16 % St::PIECE;
  const bool two = side > 512;
  const unsigned data = smem_u32(ring.data);
  int i = 0, slot = 0, phase = 0;
  bool dead = false;
  for (int64_t u = u0; u < u1 && !dead;) {
    const KdSeg s = kd_seg(a, batch, u, u1);
    const int64_t at = s.bg * a.nblk_max + s.blk0;
    const uint8_t* from = src + at * codes;
    const uint8_t* side_from = side_src + at * side;
    for (int x = 0; x < s.nfast; ++x) {
      dead = !mbar_wait(ring.empty + 8 * slot, phase ^ 1);    // (a new barrier's "phase -1" is complete)
      dead = __any_sync(0xffffffffu, dead);
      if (dead) break;
      const unsigned to = data + slot * size, bar = ring.full + 8 * slot;
      if (lane == 0) {
        mbar_expect_tx(bar, codes);
        asm volatile(
            "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n" ::"r"(to),
            "l"(from), "n"(codes), "r"(bar)
            : "memory");
      }
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(to + to0), "l"(side_from) : "memory");
      if (two) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(to + to1), "l"(side_from + 512) : "memory");
      asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];\n" ::"r"(bar) : "memory");
      from += codes;
      side_from += side;
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

// A nibble of a half word in bits 7..10: n 2^-17 (bit 10 is the lowest exponent
// bit, where the subnormal numbers go on as normal ones of the same spacing)
constexpr unsigned kNib = 0x07800780u;
// nibbles 2 z and 2 z + 1 of the half words of a and b
__device__ __forceinline__ void kd_key_operand(unsigned a, unsigned b, int z, unsigned (&op)[4]) {
  op[0] = (z ? a >> 1 : a << 7) & kNib;
  op[1] = (z ? b >> 1 : b << 7) & kNib;
  op[2] = (z ? a >> 5 : a << 3) & kNib;
  op[3] = (z ? b >> 5 : b << 3) & kNib;
}
constexpr int kKdChains = 4;      // sums of values in turn
constexpr float kCodeUnit = 131072.0f;   // 2^17

// The state of a warp over the tensor-core blocks of an item.  Lane (gid =
// lane / 4, tid = lane % 4) works on query row gid % RT (RT = 4: lanes with
// gid >= 4 have the same rows and supply the low parts) and its channels
// [tid D / 4, (tid + 1) D / 4).  Softmax state: rows ra, ra + 1 with ra = 2
// (tid % (RT / 2)); the sums l are over the lane's own tokens, om too (RT =
// 4: and those of lane ^ 2).
template <int D, int RT>
struct KdFast {
  float qinv;             // undoes the scale of the lane's row
  float xs;               // scale of the lane's row's q_c Delta_c, a power of two
  float most;             // Delta_c from which some row's may be too large
  int at;                 // where a block holds Delta_c of the lane's row's largest q_c
  float csA, csB;         // unit of the code sums of rows ra, ra + 1
  float rA, rB;           // reference (running maximum, or up to 8 below it)
  float lA, lB, omA, omB;
  float svA, svB;         // scale of p_t Delta_t, a power of two (0: not set)
  float wide;             // p_t Delta_t up to which both hold
  float o[D / 16][4];     // channels 16 i + gid (+ 8) x operand columns 2 tid, 2 tid + 1
  bool newA, newB;        // the row has seen no token yet
};

// The scale sv of a row's operands p_t Delta_t, from what is summed: the
// largest of them, weights included, that the row has met since sv was set
// lies in [2^5, 2^15) / sv, so the two halves' floor of 2^-25 is 2^-30 of it
// or less.  (A scale from Delta_t alone cost a row up to 2^-9 of its output
// beside a token of values 2^20 times larger at no weight.)
constexpr int kKdScaleMin = -109, kKdScaleMax = 110;     // exponents of sv
// first p_t Delta_t that sv is too large for, 2^15 / sv; below zero for sv = 0
__device__ __forceinline__ float kd_scale_end(float sv) { return __uint_as_float(0x86800000u - __float_as_uint(sv)); }
// sv fitted to a block whose largest p_t Delta_t is top; returns the sums' factor
__device__ __forceinline__ float kd_scale_fit(float& sv, float top) {
  if (!(top > 0.0f && top >= kd_scale_end(sv))) return 1.0f;
  const float to = pow2i(min(max(5 - exponent(top), kKdScaleMin), kKdScaleMax));
  const float up = sv == 0.0f ? 1.0f : __fdividef(to, sv);        // (powers of two: exact)
  sv = to;
  return up;
}
// The row's reference moves up by d, its sums shrink by e = 2^-d: sv follows.
// Returns the sums' factor.
__device__ __forceinline__ float kd_scale_follow(float& sv, float d, float e) {
  if (e == 0.0f) sv = 0.0f;      // (nothing is left of the sums)
  if (sv == 0.0f) return e;
  const float up = pow2i(min((int)fminf(d, 120.0f), kKdScaleMax - exponent(sv)));
  sv *= up;
  return e * up;
}

// The scale xs of a row's operands q_c Delta_c: the largest in a block lies in
// [2, 2^15) / xs, so the two halves' floor of 2^-25 is 2^-26 of it or less.
// A row's largest q_c lies in [2^11, 2^12) (kd_q), which says that without a
// look at the products where no step of the block is 2^3 / xs or more and the
// one of that channel is 2^-10 / xs or more: xs stays 1 for usual keys.
// Otherwise this looks at them, row by row.  (A scale from the steps alone, kept
// when they got smaller, lost every digit of the scores beside a channel of
// large keys and small queries.)
constexpr float kKdMost = 8.0f, kKdLeast = 0x1p-10f;
template <int D, int RT>
__device__ __forceinline__ void kd_rescale(KdFast<D, RT>& f, const float* sq, const float* sd) {
  float mx = 0.0f;
#pragma unroll 1
  for (int i = 0; i < D / 4; i += 4) {
    const float4 q = *reinterpret_cast<const float4*>(sq + i), dl = *reinterpret_cast<const float4*>(sd + i);
    mx = fmaxf(mx, fmaxf(fmaxf(fabsf(q.x * dl.x), fabsf(q.y * dl.y)), fmaxf(fabsf(q.z * dl.z), fabsf(q.w * dl.w))));
  }
  mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
  mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
  if (mx > 0.0f && mx < INFINITY && !(mx * f.xs >= 2.0f && mx * f.xs < 32768.0f)) {
    const int e = exponent(mx);
    f.xs = e >= 1 && e < 15 ? 1.0f : pow2i(min(max(11 - e, -120), 120));
  }
  const float high = __uint_as_float(__reduce_max_sync(0xffffffffu, mx > 0.0f ? __float_as_uint(f.xs) : 0u));
  if (mx == 0.0f && high > 0.0f) f.xs = high;       // (a row of zeros, for instance a padded one)
  f.most = high > 0.0f ? kKdMost / high : kKdMost;
  const float c = pow2i(min(max(17 + exponent(f.qinv) - exponent(f.xs), -126), 127));
  const int ra = 2 * (threadIdx.x % 4 % (RT / 2));
  f.csA = __shfl_sync(0xffffffffu, c, 4 * ra);
  f.csB = __shfl_sync(0xffffffffu, c, 4 * ra + 4);
}

template <int D, int RT>
__device__ __forceinline__ void kd_fast_init(KdFast<D, RT>& f, const float* s_inv, const int* s_top) {
  const int lane = threadIdx.x & 31, gid = lane >> 2, ra = 2 * (lane % 4 % (RT / 2));
  f.qinv = s_inv[gid % RT];
  f.xs = 1.0f;
  f.most = kKdMost;
  // (within the block also when a wait gave up and nobody filled the item in)
  f.at = (int)(min((unsigned)s_top[gid % RT], (unsigned)KdStage<D>::bytesK - 4) & ~3u);
  f.csA = kCodeUnit * s_inv[ra];
  f.csB = kCodeUnit * s_inv[ra + 1];
  f.rA = f.rB = f.lA = f.lB = f.omA = f.omB = 0.0f;
  f.svA = f.svB = 0.0f;
  f.wide = kd_scale_end(0.0f);
#pragma unroll
  for (int i = 0; i < D / 16; ++i) f.o[i][0] = f.o[i][1] = f.o[i][2] = f.o[i][3] = 0.0f;
  f.newA = f.newB = true;
}

// One block: its keys' part at st, its values' part at vt; between() is
// called when the one has been read and before the other is.  MASK: row ra
// sees the block's tokens below endA only, row ra + 1 those below endB.  The
// channels go through a loop that stays a loop: unrolled, the code was more
// than the instruction caches could feed to warps that are each at another
// place of it (at 8 rows the warps spent a third of their time waiting for
// instructions).
template <int D, int RT, bool MASK, typename Between>
__device__ __forceinline__ void kd_fast_block(KdFast<D, RT>& f, const uint8_t* st, const uint8_t* vt, const float* s_q,
                                              int endA, int endB, Between between) {
  using St = KdStage<D>;
  constexpr int NC = D / 4;        // channels of a lane
  constexpr int NW = D / 32;       // code words of a lane in a key row
  constexpr int HL = RT == 8 ? 2 : 1;   // instructions per operand (parts in columns with RT = 4)
  const int lane = threadIdx.x & 31, gid = lane >> 2, tid = lane & 3;
  const bool upper = RT == 4 && tid >= 2;
  const int ra = 2 * (tid % (RT / 2));

  // q_c Delta_c, and sum_c q_c m_c
  const float* sq = s_q + kd_q<D>(gid % RT, tid * NC);
  const float* sm = reinterpret_cast<const float*>(st + St::B + tid * St::PITCH);
  const float* sd = reinterpret_cast<const float*>(st + St::B + (4 + tid) * St::PITCH);
  float top;
  if (D == 128) {
    const float4 dl = *reinterpret_cast<const float4*>(st + St::B + (4 + (lane >> 3)) * St::PITCH + (lane & 7) * 16);
    top = fmaxf(fmaxf(dl.x, dl.y), fmaxf(dl.z, dl.w));
  } else {
    const float2 dl = *reinterpret_cast<const float2*>(st + St::B + (4 + (lane >> 3)) * St::PITCH + (lane & 7) * 8);
    top = fmaxf(dl.x, dl.y);
  }
  const float own = *reinterpret_cast<const float*>(st + f.at);
  if (__builtin_expect(__any_sync(0xffffffffu, top >= f.most || own * f.xs < kKdLeast), 0)) kd_rescale<D, RT>(f, sq, sd);
  // Scores of the four tiles of 16 tokens, two code words (16 channels of a
  // lane) at a time: q_c Delta_c as the operand (column gid, channel pairs (8
  // w + 0, 4), (1, 5), (2, 6), (3, 7); high part = the leading 11 bits, low
  // part = the rest), and sum_c q_c m_c beside it, in float32.  (RT = 4: the
  // lanes gid and gid + 4 take half of the channels of that each.)  Matrix
  // instructions truncate their sums: they start from zero.
  float t[4][4], low[4][4];
  if (RT == 8) {
#pragma unroll
    for (int y = 0; y < 4; ++y) t[y][0] = t[y][1] = t[y][2] = t[y][3] = low[y][0] = low[y][1] = low[y][2] = low[y][3] = 0.0f;
  }
  float qm = 0.0f, qm1 = 0.0f;
  const unsigned cut = RT == 8 || gid >= 4 ? 0xffffe000u : 0u;
  if constexpr (RT == 4) {
    // (the low part is truncated too: a quarter of a step more, to half of one, takes most of the bias away)
    const float up = gid >= 4 ? 1.0f + 0x1p-12f : 1.0f;
    float x[NC];
#pragma unroll
    for (int i = 0; i < NC; i += 4) {
      const float4 q = *reinterpret_cast<const float4*>(sq + i), dl = *reinterpret_cast<const float4*>(sd + i);
      x[i] = q.x * dl.x; x[i + 1] = q.y * dl.y; x[i + 2] = q.z * dl.z; x[i + 3] = q.w * dl.w;
    }
    if (__builtin_expect(f.xs != 1.0f, 0)) {
#pragma unroll
      for (int i = 0; i < NC; ++i) x[i] *= f.xs;
    }
    unsigned bq[NW][4];
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const int h = 8 * w + (gid >> 2) * 4;
      const float4 q = *reinterpret_cast<const float4*>(sq + h), mn = *reinterpret_cast<const float4*>(sm + h);
      qm = fmaf(q.x, mn.x, qm); qm1 = fmaf(q.y, mn.y, qm1);
      qm = fmaf(q.z, mn.z, qm); qm1 = fmaf(q.w, mn.w, qm1);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float u = x[8 * w + e], v = x[8 * w + e + 4];
        bq[w][e] = half_pair_rz((u - __uint_as_float(__float_as_uint(u) & cut)) * up, (v - __uint_as_float(__float_as_uint(v) & cut)) * up);
      }
    }
#pragma unroll
    for (int pr = 0; pr < 4; pr += 2) {
      unsigned k[2 * 2][NW];
#pragma unroll
      for (int j = 0; j < 2 * 2; ++j) {
        const uint8_t* kr = st + (16 * pr + 8 * j + gid) * (D / 2) + tid * (D / 8);
        if (D == 128) {
          const uint4 u = *reinterpret_cast<const uint4*>(kr);
          k[j][0] = u.x; k[j][1] = u.y; k[j][NW - 2] = u.z; k[j][NW - 1] = u.w;
        } else {
          const uint2 u = *reinterpret_cast<const uint2*>(kr);
          k[j][0] = u.x; k[j][1] = u.y;
        }
      }
#pragma unroll
      for (int w = 0; w < NW; ++w)
#pragma unroll
        for (int z = 0; z < 2; ++z)
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            unsigned op[4];
            kd_key_operand(k[2 * y][w], k[2 * y + 1][w], z, op);
            if (w == 0 && z == 0) mma_f16_first(t[pr + y], op[0], op[1], op[2], op[3], bq[w][2 * z], bq[w][2 * z + 1]);
            else mma_f16(t[pr + y], op[0], op[1], op[2], op[3], bq[w][2 * z], bq[w][2 * z + 1]);
          }
    }
  } else
#pragma unroll 1
  for (int wp = 0; wp < NW / 2; ++wp) {
    unsigned bq[HL][2][4];
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
      const int c = wp * 16 + i;
      const float4 q = *reinterpret_cast<const float4*>(sq + c), dl = *reinterpret_cast<const float4*>(sd + c);
      const float4 mn = *reinterpret_cast<const float4*>(sm + c);
      x[i] = q.x * dl.x; x[i + 1] = q.y * dl.y; x[i + 2] = q.z * dl.z; x[i + 3] = q.w * dl.w;
      qm = fmaf(q.x, mn.x, qm); qm1 = fmaf(q.y, mn.y, qm1);
      qm = fmaf(q.z, mn.z, qm); qm1 = fmaf(q.w, mn.w, qm1);
    }
    if (__builtin_expect(f.xs != 1.0f, 0)) {
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] *= f.xs;
    }
#pragma unroll
    for (int w = 0; w < 2; ++w)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float u = x[8 * w + e], v = x[8 * w + e + 4];
        bq[0][w][e] = half_pair_rz(u, v);
        bq[HL - 1][w][e] = half_pair(u - __uint_as_float(__float_as_uint(u) & cut), v - __uint_as_float(__float_as_uint(v) & cut));
      }
    uint2 k[8];                          // rows gid, gid + 8 of the tiles
#pragma unroll
    for (int j = 0; j < 8; ++j) k[j] = *reinterpret_cast<const uint2*>(st + (8 * j + gid) * (D / 2) + tid * (D / 8) + wp * 8);
#pragma unroll
    for (int w = 0; w < 2; ++w)
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        unsigned op[4][4];
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          kd_key_operand(w ? k[2 * y].y : k[2 * y].x, w ? k[2 * y + 1].y : k[2 * y + 1].x, z, op[y]);
        }
#pragma unroll
        for (int y = 0; y < 4; ++y)      // (four independent sums in turn: one has to wait 31 cycles for its last)
          mma_f16(low[y], op[y][0], op[y][1], op[y][2], op[y][3], bq[HL - 1][w][2 * z], bq[HL - 1][w][2 * z + 1]);
#pragma unroll
        for (int y = 0; y < 4; ++y) mma_f16(t[y], op[y][0], op[y][1], op[y][2], op[y][3], bq[0][w][2 * z], bq[0][w][2 * z + 1]);
      }
  }
  if (RT == 8) {
#pragma unroll
    for (int y = 0; y < 4; ++y)
#pragma unroll
      for (int k = 0; k < 4; ++k) t[y][k] += low[y][k];
  }
  between();
  qm = (qm + qm1) * f.qinv;
  qm += __shfl_xor_sync(0xffffffffu, qm, 1);
  qm += __shfl_xor_sync(0xffffffffu, qm, 2);
  if (RT == 4) qm += __shfl_xor_sync(0xffffffffu, qm, 16);
  const float sA = __shfl_sync(0xffffffffu, qm, 4 * ra), sB = __shfl_sync(0xffffffffu, qm, 4 * ra + 4);
  // The scores.  (Not yet relative to rA, rB: the difference is rounded to the
  // digits of the larger, and a reference that is about to move may be far
  // from the scores.)  RT = 4: the two parts are added; the lane
  // has token 16 y + gid (+ 8 in the upper lanes), rows ra, ra + 1, in
  // t[y][0], t[y][1]; RT = 8: tokens gid and gid + 8 in t[y][0..1], t[y][2..3].
  constexpr int TK = RT == 8 ? 2 : 1;    // tokens of a tile in a lane
  const auto token = [&](int y, int k) { return 16 * y + gid + (RT == 8 ? 8 * k : upper ? 8 : 0); };
  float2 sc[4][TK];                      // token scales
  float xA = -INFINITY, xB = -INFINITY, wide = 0.0f;
#pragma unroll
  for (int y = 0; y < 4; ++y) {
    if (RT == 4) {
      const float g0 = __shfl_xor_sync(0xffffffffu, upper ? t[y][0] : t[y][2], 2);
      const float g1 = __shfl_xor_sync(0xffffffffu, upper ? t[y][1] : t[y][3], 2);
      t[y][0] = fmaf((upper ? t[y][2] : t[y][0]) + g0, f.csA, sA);
      t[y][1] = fmaf((upper ? t[y][3] : t[y][1]) + g1, f.csB, sB);
    } else {
      t[y][0] = fmaf(t[y][0], f.csA, sA); t[y][1] = fmaf(t[y][1], f.csB, sB);
      t[y][2] = fmaf(t[y][2], f.csA, sA); t[y][3] = fmaf(t[y][3], f.csB, sB);
    }
#pragma unroll
    for (int k = 0; k < TK; ++k) sc[y][k] = *reinterpret_cast<const float2*>(vt + St::S + token(y, k) * 8);
  }
  if (MASK) {
    // an unseen token's value may be anything
#pragma unroll
    for (int y = 0; y < 4; ++y)
#pragma unroll
      for (int k = 0; k < TK; ++k) {
        if (token(y, k) >= endA) t[y][2 * k] = -INFINITY;
        if (token(y, k) >= endB) t[y][2 * k + 1] = -INFINITY;
        if (token(y, k) >= max(endA, endB)) sc[y][k] = make_float2(0.0f, 0.0f);
      }
  }
#pragma unroll
  for (int y = 0; y < 4; ++y)
#pragma unroll
    for (int k = 0; k < TK; ++k) {
      xA = fmaxf(xA, t[y][2 * k]);
      xB = fmaxf(xB, t[y][2 * k + 1]);
      wide = fmaxf(wide, sc[y][k].y);
    }
  // The reference moves only when a score exceeds it by more than 8 (weights
  // up to 2^8), and the value scale only when it or a p_t Delta_t asks for
  // it; the lane's largest weight times its largest step says that none does.
  // Both are rare after the first block.
  const float big = fmaxf(xA - f.rA, xB - f.rB);
  if (__builtin_expect(__any_sync(0xffffffffu, f.newA || f.newB || big > 8.0f || ex2(big) * wide >= f.wide), 0)) {
    float tA = 0.0f, tB = 0.0f;
#pragma unroll
    for (int m = (RT == 4 ? 2 : 4); m < 32; m <<= 1) {
      xA = fmaxf(xA, __shfl_xor_sync(0xffffffffu, xA, m));
      xB = fmaxf(xB, __shfl_xor_sync(0xffffffffu, xB, m));
    }
    // the references move up to the maximum
    const float nA = f.newA ? (xA > -INFINITY ? xA : 0.0f) : fmaxf(f.rA, xA);
    const float nB = f.newB ? (xB > -INFINITY ? xB : 0.0f) : fmaxf(f.rB, xB);
    const float dA = f.newA ? 0.0f : nA - f.rA, dB = f.newB ? 0.0f : nB - f.rB;
    const float eA = ex2(-dA), eB = ex2(-dB);
    float upA = kd_scale_follow(f.svA, dA, eA), upB = kd_scale_follow(f.svB, dB, eB);
    f.lA *= eA; f.lB *= eB;
    f.omA *= eA; f.omB *= eB;
    f.rA = nA; f.rB = nB;
    f.newA = f.newA && !(xA > -INFINITY);
    f.newB = f.newB && !(xB > -INFINITY);
#pragma unroll
    for (int y = 0; y < 4; ++y)
#pragma unroll
      for (int k = 0; k < TK; ++k) {
        const float wA = ex2(t[y][2 * k] - nA) * sc[y][k].y, wB = ex2(t[y][2 * k + 1] - nB) * sc[y][k].y;
        if ((!MASK || token(y, k) < endA) && wA < INFINITY) tA = fmaxf(tA, wA);
        if ((!MASK || token(y, k) < endB) && wB < INFINITY) tB = fmaxf(tB, wB);
      }
#pragma unroll
    for (int m = (RT == 4 ? 2 : 4); m < 32; m <<= 1) {
      tA = fmaxf(tA, __shfl_xor_sync(0xffffffffu, tA, m));
      tB = fmaxf(tB, __shfl_xor_sync(0xffffffffu, tB, m));
    }
    upA *= kd_scale_fit(f.svA, tA);
    upB *= kd_scale_fit(f.svB, tB);
    f.wide = fminf(kd_scale_end(f.svA), kd_scale_end(f.svB));
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
      f.o[i][0] *= upA; f.o[i][1] *= upB;
      f.o[i][2] *= upA; f.o[i][3] *= upB;
    }
  }
  // Weights and the second operand: column gid, token pairs.  The tokens gid +
  // 8 of a tile enter as 15 - n with the opposite sign, and with m + 15 Delta
  // for m: the sums of codes, all positive, would outgrow the differences that
  // the output consists of (values around zero) and leave them their rounding
  // errors.
  float omA = 0.0f, omB = 0.0f;
  unsigned bp[HL][4][2];
#pragma unroll
  for (int y = 0; y < 4; ++y) {
    unsigned hi[TK], lo[TK];
#pragma unroll
    for (int k = 0; k < TK; ++k) {
      const float pA = ex2(t[y][2 * k] - f.rA), pB = ex2(t[y][2 * k + 1] - f.rB);
      f.lA += pA; f.lB += pB;
      const bool turned = RT == 8 ? k == 1 : upper;
      const float dl = sc[y][k].y, m = fmaf(dl, turned ? 15.0f : 0.0f, sc[y][k].x);
      float wA = pA * dl * (turned ? -f.svA : f.svA), wB = pB * dl * (turned ? -f.svB : f.svB);
      if (MASK) {
        // left out, not multiplied by zero
        if (token(y, k) >= endA) wA = 0.0f; else omA = fmaf(pA, m, omA);
        if (token(y, k) >= endB) wB = 0.0f; else omB = fmaf(pB, m, omB);
      } else {
        omA = fmaf(pA, m, omA);
        omB = fmaf(pB, m, omB);
      }
      hi[k] = half_pair(wA, wB);
      lo[k] = half_rest(wA, wB, hi[k]);
    }
    if (RT == 4) {
      const unsigned got = __shfl_xor_sync(0xffffffffu, upper ? hi[0] : lo[0], 2);
      bp[0][y][0] = transpose8(upper ? got : hi[0]);
      bp[0][y][1] = transpose8(upper ? lo[0] : got);
    } else {
      bp[0][y][0] = transpose8(hi[0]);
      bp[0][y][1] = transpose8(hi[TK - 1]);
      bp[HL - 1][y][0] = transpose8(lo[0]);
      bp[HL - 1][y][1] = transpose8(lo[TK - 1]);
    }
  }
  // (the two halves of a tile's tokens cancel: RT = 4 has them in lane pairs)
  if (RT == 4) {
    omA += __shfl_xor_sync(0xffffffffu, omA, 2);
    omB += __shfl_xor_sync(0xffffffffu, omB, 2);
  }
  f.omA += omA;
  f.omB += omB;
#pragma unroll
  for (int i = 0; i < D / 16; i += kKdChains) {
    uint2 v[2 * kKdChains];              // channels gid, gid + 8 of the tiles i, i + 1, ...
#pragma unroll
    for (int j = 0; j < 2 * kKdChains; ++j)
      v[j] = *reinterpret_cast<const uint2*>(vt + (16 * i + 8 * j + gid) * (kBlock / 2) + tid * 8);
    float u[kKdChains][4];
#pragma unroll
    for (int y = 0; y < 4; ++y) {
      unsigned op[kKdChains][4];
#pragma unroll
      for (int z = 0; z < kKdChains; ++z) {
        const unsigned a = y < 2 ? v[2 * z].x : v[2 * z].y, b = y < 2 ? v[2 * z + 1].x : v[2 * z + 1].y;
        op[z][0] = (y & 1 ? a >> 1 : a << 7) & kNib; op[z][1] = (y & 1 ? b >> 1 : b << 7) & kNib;
        op[z][2] = ~(y & 1 ? a >> 5 : a << 3) & kNib; op[z][3] = ~(y & 1 ? b >> 5 : b << 3) & kNib;
      }
#pragma unroll
      for (int h = HL - 1; h >= 0; --h)
#pragma unroll
        for (int z = 0; z < kKdChains; ++z) {
          if (y == 0 && h == HL - 1) mma_f16_first(u[z], op[z][0], op[z][1], op[z][2], op[z][3], bp[h][y][0], bp[h][y][1]);
          else mma_f16(u[z], op[z][0], op[z][1], op[z][2], op[z][3], bp[h][y][0], bp[h][y][1]);
        }
    }
#pragma unroll
    for (int z = 0; z < kKdChains; ++z)
#pragma unroll
      for (int e = 0; e < 4; ++e) f.o[i + z][e] += u[z][e];
  }
}

// the warp's sums as rows [RT] of m, l and acc[D] in shared memory
template <int D, int RT>
__device__ __forceinline__ void kd_fast_store(KdFast<D, RT>& f, float* s_m, float* s_l, float* s_acc) {
  const int lane = threadIdx.x & 31, gid = lane >> 2, tid = lane & 3;
  const bool upper = RT == 4 && tid >= 2;
  const int ra = 2 * (tid % (RT / 2));
  if (RT == 4) {
    f.lA += __shfl_xor_sync(0xffffffffu, f.lA, 2);
    f.lB += __shfl_xor_sync(0xffffffffu, f.lB, 2);
  }
#pragma unroll
  for (int m = 4; m < 32; m <<= 1) {
    f.lA += __shfl_xor_sync(0xffffffffu, f.lA, m);
    f.lB += __shfl_xor_sync(0xffffffffu, f.lB, m);
    f.omA += __shfl_xor_sync(0xffffffffu, f.omA, m);
    f.omB += __shfl_xor_sync(0xffffffffu, f.omB, m);
  }
  if (gid == 0 && !upper) {
    s_m[ra] = f.newA ? -INFINITY : f.rA; s_m[ra + 1] = f.newB ? -INFINITY : f.rB;
    s_l[ra] = f.lA; s_l[ra + 1] = f.lB;
  }
  const float backA = f.svA == 0.0f ? 0.0f : kCodeUnit / f.svA, backB = f.svB == 0.0f ? 0.0f : kCodeUnit / f.svB;
#pragma unroll
  for (int i = 0; i < D / 16; ++i) {
    if (RT == 4) {
      const float g0 = __shfl_xor_sync(0xffffffffu, upper ? f.o[i][0] : f.o[i][2], 2);
      const float g1 = __shfl_xor_sync(0xffffffffu, upper ? f.o[i][1] : f.o[i][3], 2);
      const int c = 16 * i + gid + (upper ? 8 : 0);
      s_acc[ra * D + c] = fmaf((upper ? f.o[i][2] : f.o[i][0]) + g0, backA, f.omA);
      s_acc[(ra + 1) * D + c] = fmaf((upper ? f.o[i][3] : f.o[i][1]) + g1, backB, f.omB);
    } else {
      const int c = 16 * i + gid;
      s_acc[ra * D + c] = fmaf(f.o[i][0], backA, f.omA);
      s_acc[(ra + 1) * D + c] = fmaf(f.o[i][1], backB, f.omB);
      s_acc[ra * D + c + 8] = fmaf(f.o[i][2], backA, f.omA);
      s_acc[(ra + 1) * D + c + 8] = fmaf(f.o[i][3], backB, f.omB);
    }
  }
}


// Queries come by one producer warp, tiles of 8 by two, half of the rows each (one
// took 12 us for 64 rows; drafts of 24 rows 114 us, with one 121, the batch of 64
// with 8 rows 126 and 128).
template <int RT> constexpr int kKdQueryWarps = RT == 8 ? 2 : 1;

template <int D, int RT, typename E>
__device__ __forceinline__ void kd_queries(const Kv4DecodeArgs& a, const KdBatch& batch, int64_t u0, int64_t u1,
                                           KdItem<Kv4DecodeArgs>* items, float* s_q, unsigned full, unsigned empty, int part) {
  const int lane = threadIdx.x & 31;
  const int R = a.T * a.G, Rp = (R + RT - 1) / RT * RT, per = Rp / kKdQueryWarps<RT>;
  int k = 0;
  bool dead = false;
  kd_trim(a, batch, u0, u1);
  for (int64_t u = u0; u < u1 && !dead; ++k) {
    const int buf = k & 1;
    dead = !mbar_wait(empty + 8 * buf, ((k >> 1) & 1) ^ 1);
    dead = __any_sync(0xffffffffu, dead);
    if (dead) break;
    KdItem<Kv4DecodeArgs>& it = items[buf];
    const KdSeg sg = kd_seg(a, batch, u, u1);
    if (lane == 0 && part == 0) it.seg = sg;
    kd_item_queries<D, E>(a, sg, it, s_q + buf * kd_q<D>(Rp, 0), part * per, (part + 1) * per);
    __syncwarp();
    if (lane == 0) mbar_arrive(full + 8 * buf);
    u += sg.step;
  }
  if (dead && lane == 0) atomicOr(a.status, 4u);
}

// shared memory: barriers (keys full, empty, values full, empty, items full,
// empty), items, warp sums, q rows of two items, the rings
template <int D, int RT>
struct KdLayout {
  static constexpr int item = (4 * kKdMaxStages + 4) * 8;
  static constexpr int m = item + 2 * (int)sizeof(KdItem<Kv4DecodeArgs>);
  static constexpr int l = m + kKdWarps * RT * 4;
  static constexpr int acc = (l + kKdWarps * RT * 4 + 15) / 16 * 16;
  static constexpr int q = acc + kKdWarps * RT * D * 4;
  static __host__ __device__ int ring(int rows) { return q + 2 * ((rows + RT - 1) / RT * RT) * (D + 16) * 4; }
};

template <int D, int RT, typename E>
__global__ void __launch_bounds__(kKdThreads, 1) kv4_decode_kernel(const Kv4DecodeArgs a) {
  pdl_entry();
  using St = KdStage<D>;
  using Lt = KdLayout<D, RT>;
  constexpr int CPL = D / 32, W = kKdWarps;
  __shared__ KdBatch batch;
  extern __shared__ __align__(128) uint8_t kd_sm[];
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int R = a.T * a.G, Rp = (R + RT - 1) / RT * RT;
  // teams: warps that share a block, one tile of rows each
  const int ntile = Rp / RT;
  const int team = kd_team(ntile), nteam = W / team;
  KdRing keys, values;
  keys.full = smem_u32(kd_sm);
  keys.empty = keys.full + kKdMaxStages * 8;
  values.full = keys.empty + kKdMaxStages * 8;
  values.empty = values.full + kKdMaxStages * 8;
  const unsigned item_full = values.empty + kKdMaxStages * 8, item_empty = item_full + 16;
  keys.slots = a.slotsK;
  values.slots = a.slotsV;
  keys.data = kd_sm + Lt::ring(R);
  values.data = keys.data + a.slotsK * St::bytesK;
  KdItem<Kv4DecodeArgs>* items = reinterpret_cast<KdItem<Kv4DecodeArgs>*>(kd_sm + Lt::item);
  float* s_q = reinterpret_cast<float*>(kd_sm + Lt::q);        // two of [rows, padded] (kd_q)
  if (tid >= 32 && tid < 32 + kKdMaxStages) {
    // (full: one arrival with the codes' bytes, one of each lane of the producer)
    const int i = tid - 32;
    mbar_init(keys.full + 8 * i, 33);
    mbar_init(keys.empty + 8 * i, team);
    mbar_init(values.full + 8 * i, 33);
    mbar_init(values.empty + 8 * i, team);
    if (i < 2) {
      mbar_init(item_full + 8 * i, kKdQueryWarps<RT>);
      mbar_init(item_empty + 8 * i, W);
    }
    fence_barrier_init();
  }
  kd_batch(a, batch);
  const int64_t per = kd_run(batch, gridDim.x);
  int64_t u0 = (int64_t)blockIdx.x * per, u1 = min(batch.pref[kMaxB], u0 + per);

  if (w >= W) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kKdRegsProducer));
    const auto report = [&]() {
      bool bad = false;
      for (int b = lane; b < a.B; b += 32) {
        bad |= a.len[b] < 0 || a.len[b] > a.n_max;
        if (a.n_q) bad |= a.n_q[b] < 0 || a.n_q[b] > a.T;
      }
      const unsigned any = __any_sync(0xffffffffu, bad);
      // (a wait that gives up flags the word two seconds later at the earliest)
      if (lane == 0) *a.status = any ? 8u : 0u;
    };
    // (one order of the branches for both made the consumers of 4 rows spill: the
    // 128K-token batch took 144 us, not 134)
    if constexpr (kKdQueryWarps<RT> == 1) {
      if (w == W) kd_produce<D>(a, batch, u0, u1, keys, true);
      else if (w == W + 1) kd_produce<D>(a, batch, u0, u1, values, false);
      else if (w == W + 2) kd_queries<D, RT, E>(a, batch, u0, u1, items, s_q, item_full, item_empty, 0);
      else if (blockIdx.x == 0) report();
    } else {
      if (blockIdx.x == 0 && w == W + 1) report();
      if (w == W) kd_produce<D>(a, batch, u0, u1, keys, true);
      else if (w == W + 1) kd_produce<D>(a, batch, u0, u1, values, false);
      else kd_queries<D, RT, E>(a, batch, u0, u1, items, s_q, item_full, item_empty, w - W - 2);
    }
    return;
  }
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(kKdRegsConsumer));

  float* s_m = reinterpret_cast<float*>(kd_sm + Lt::m);        // [warps][RT]
  float* s_l = reinterpret_cast<float*>(kd_sm + Lt::l);
  float* s_acc = reinterpret_cast<float*>(kd_sm + Lt::acc);    // [warps][RT][D]
  const int my_team = w / team, tile = w % team;
  const int rows = my_team < nteam ? min(RT, R - tile * RT) : 0;    // <= 0: a warp with no rows
  const int r0 = tile * RT < Rp ? tile * RT : 0;
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
    const KdItem<Kv4DecodeArgs>& it = items[buf];
    const float* q = s_q + kd_q<D>(buf * Rp + r0, 0);
    float* my_m = s_m + w * RT;
    float* my_l = s_l + w * RT;
    float* my_acc = s_acc + w * RT * D;
    {
      KdFast<D, RT> f;
      kd_fast_init<D, RT>(f, it.inv + r0, it.top + r0);
      const int to = base + it.seg.nfast, clear = base + it.seg.clear;
      while (my_team < nteam && i < to) {
        if (!dead && !mbar_wait(keys.full + 8 * sk, pk)) dead = true;
        const auto between = [&]() {
          __syncwarp();
          if (lane == 0) mbar_arrive(keys.empty + 8 * sk);
          if (!dead && !mbar_wait(values.full + 8 * sv, pv)) dead = true;
        };
        const uint8_t* kt = keys.data + sk * St::bytesK;
        const uint8_t* vt = values.data + sv * St::bytesV;
        if (rows <= 0) {
          between();
        } else if (i < clear) {
          kd_fast_block<D, RT, false>(f, kt, vt, q, 0, 0, between);
        } else {
          const int ra = 2 * (lane % 4 % (RT / 2));
          const int64_t p0 = (it.seg.blk0 + (i - base)) * kBlock;
          kd_fast_block<D, RT, true>(f, kt, vt, q, (int)min(max(it.end[r0 + ra] - p0, (int64_t)0), (int64_t)kBlock),
                                     (int)min(max(it.end[r0 + ra + 1] - p0, (int64_t)0), (int64_t)kBlock), between);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(values.empty + 8 * sv);
        i += nteam;
        if ((sk += nteam) >= keys.slots) { sk = my_team; pk ^= 1; }
        if ((sv += nteam) >= values.slots) { sv = my_team; pv ^= 1; }
      }
      base = to;
      kd_fast_store<D, RT>(f, my_m, my_l, my_acc);
    }
    // the incomplete block, if it is to be done here
    const int64_t p0 = it.seg.n / kBlock * kBlock;
    const int left = it.seg.left;
    if (rows > 0 && kKdStep<RT> * (i - base) < left) {
      // a few tokens at a time: the state moves on to lanes that hold channels
      __syncwarp();
      KdState<D, RT> st;
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        st.m[r] = my_m[r]; st.l[r] = my_l[r];
#pragma unroll
        for (int c = 0; c < CPL; ++c) st.acc[r][c] = my_acc[r * D + lane * CPL + c];
      }
      __syncwarp();
      // (the teams go on in turn where the blocks ended; my_acc is free until
      // the state returns to it)
      for (int t0 = kKdStep<RT> * (i - base); t0 < left; t0 += kKdStep<RT> * nteam) {
        const int64_t at = (it.seg.bg * kBlock + t0) * D;
        kd_step<D, RT, E>(st, reinterpret_cast<const E*>(a.c.Kt) + at, reinterpret_cast<const E*>(a.c.Vt) + at,
                          min(kKdStep<RT>, left - t0), q, it.inv + r0, it.end + r0, p0 + t0, my_acc);
      }
      __syncwarp();
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        if (lane == 0) { my_m[r] = st.m[r]; my_l[r] = st.l[r]; }
#pragma unroll
        for (int c = 0; c < CPL; ++c) my_acc[r * D + lane * CPL + c] = st.acc[r][c];
      }
    }
    bar_sync(1, W * 32);
    // merge the teams, four channels of a row to a thread
    float* part = a.part + (2 * (int64_t)blockIdx.x + (it.seg.cut0 ? 0 : 1)) * R * (D + 4);
    for (int e = tid; e < R * (D / 4); e += W * 32) {
      const int r = e / (D / 4), c = e % (D / 4) * 4;
      float M = -INFINITY, l = 0.0f;
      float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      for (int x = r; x < nteam * team * RT; x += team * RT) M = fmaxf(M, s_m[x]);   // (the row in each team)
      for (int x = r; x < nteam * team * RT; x += team * RT) {
        const float s = s_m[x] > -INFINITY ? ex2(s_m[x] - M) : s_l[x] == 0.0f ? 0.0f : 1.0f;
        const float4 y = *reinterpret_cast<const float4*>(s_acc + x * D + c);
        l = fmaf(s, s_l[x], l);
        v.x = fmaf(s, y.x, v.x); v.y = fmaf(s, y.y, v.y); v.z = fmaf(s, y.z, v.z); v.w = fmaf(s, y.w, v.w);
      }
      if (!it.seg.cut0 && !it.seg.cut1) {
        if (r / a.G < it.seg.nq) kd_store<D>(a, it.seg, r, c, M, l, v);
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

// Items of up to this many blocks stay whole: with tiles of one warp two rounds
// of the twelve teams, which take less time than a second kernel where there are
// items for most SMs.  Whole / cut, us, bf16, d = 128:
//                     500 tokens    1000 tokens    1500 tokens
//   128 items,  4 rows  14 / 19       15 / 22        19 / 25
//               8 rows  16 / 25       19 / 27        22 / 30
//              24 rows  31 / 40       37 / 47        44 / 51
//              64 rows  79 / 96       99 / 116      116 / 128
//     8 items,  4 rows  12 / 13       13 / 14        15 / 14
//               8 rows  14 / 17       18 / 16        19 / 16
//              24 rows  28 / 27       34 / 26        38 / 23
//              64 rows  73 / 58       87 / 54       101 / 47
// So the rule is right for a batch, and costs few items of many rows up to
// twice their time: it knows neither the number of items nor that of teams.
constexpr int64_t kKdWholeBlocks = 2 * kKdWarps;
int kd_whole(const csa_shape* s) { return (s->n_max + kBlock - 1) / kBlock <= kKdWholeBlocks; }

// CTAs of the decode kernel: one per SM, no more than there can be units
int kd_ctas(const csa_shape* s) {
  const int64_t blocks = (s->n_max + kBlock - 1) / kBlock;
  const int64_t units = (int64_t)s->B * s->Hkv * (kd_whole(s) ? 1 : blocks);
  const int nsm = sm_count() < Kv4DecodeArgs::kMaxCtas ? sm_count() : Kv4DecodeArgs::kMaxCtas;
  return (int)(units < nsm ? units : nsm);
}

size_t kd_workspace(const csa_shape* s, int T) {
  const int R = T * (s->Hq / s->Hkv);
  return 256 + (kd_whole(s) ? 0 : (size_t)2 * kd_ctas(s) * R * (s->d + 4) * 4);
}

// Dynamic shared memory there can be: a CTA's 227 KB without the kernel's own.
// The limit is set to this on every call, whatever the call needs: it belongs to
// the function, and another host thread's call may lie between the setting and
// the launch.
constexpr int kKdSharedBytes = 232448 - ((int)sizeof(KdBatch) + 127) / 128 * 128;
template <int D, int RT, typename E>
cudaError_t launch_kv4_decode_t(Kv4DecodeArgs a, int ncta, cudaStream_t st) {
  const int rest = KdLayout<D, RT>::ring(a.T * a.G);
  // one slot per team in each ring (an SM's shared memory holds that for every
  // RT and d), then more while there is room: keys first, whose copies have
  // less time (the values' come while the warp is at the keys)
  constexpr int K = KdStage<D>::bytesK, V = KdStage<D>::bytesV;
  const int ntile = (a.T * a.G + RT - 1) / RT;
  const int nteam = kKdWarps / kd_team(ntile);
  int nk = 1, nv = 1;
  for (bool more = true; more;) {
    more = false;
    if ((nk + 1) * nteam <= kKdMaxStages && nteam * ((nk + 1) * K + nv * V) <= kKdSharedBytes - rest) { ++nk; more = true; }
    if ((nv + 1) * nteam <= kKdMaxStages && nteam * (nk * K + (nv + 1) * V) <= kKdSharedBytes - rest) { ++nv; more = true; }
  }
  a.slotsK = nk * nteam;
  a.slotsV = nv * nteam;
  const int smem = rest + a.slotsK * K + a.slotsV * V;
  const cudaError_t e =
      cudaFuncSetAttribute(kv4_decode_kernel<D, RT, E>, cudaFuncAttributeMaxDynamicSharedMemorySize, kKdSharedBytes);
  if (e != cudaSuccess) return e;
  launch_pdl(kv4_decode_kernel<D, RT, E>, dim3(ncta), dim3(kKdThreads), smem, st, a);
  if (ncta > 1 && !a.whole) launch_pdl(decode_join_kernel<D, Kv4DecodeArgs>, dim3(ncta - 1, (a.T * a.G + kKdJoinWarps - 1) / kKdJoinWarps), dim3(kKdJoinWarps * 32), 0, st, a, ncta);
  return cudaGetLastError();
}
template <int D, typename E>
cudaError_t launch_kv4_decode(const Kv4DecodeArgs& a, int ncta, cudaStream_t st) {
  return a.T * a.G <= 4 ? launch_kv4_decode_t<D, 4, E>(a, ncta, st) : launch_kv4_decode_t<D, 8, E>(a, ncta, st);
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
  a.whole = kd_whole(shape);
  add_launches(ncta > 1 && !a.whole ? 2 : 1);
  cudaStream_t st = (cudaStream_t)stream;
  const cudaError_t e = shape->d == 128 ? (bf16 ? launch_kv4_decode<128, __nv_bfloat16>(a, ncta, st) : launch_kv4_decode<128, float>(a, ncta, st))
                                        : (bf16 ? launch_kv4_decode<64, __nv_bfloat16>(a, ncta, st) : launch_kv4_decode<64, float>(a, ncta, st));
  return e == cudaSuccess ? CSA_OK : CSA_ERR_CUDA;
}

}  // extern "C"
