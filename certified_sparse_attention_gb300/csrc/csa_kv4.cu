// The 4-bit K/V cache (csa.h "a K/V cache held in 4 bits"): appending rows
// and reading rows back.
//
// append: one CTA per (sequence, KV head, block of 64 positions that the new
// tokens touch).  A block that becomes whole is gathered in registers (its
// first rows may lie in the kept rows Kt, Vt, the others among the new ones)
// and coded; the rows of the block that stays incomplete are copied to
// Kt, Vt.  When a call both completes a block and leaves a new incomplete
// one, the CTA of the first block writes the kept rows, after it has read
// the old ones: nobody else reads or writes them.
//
// unpack: one CTA per (sequence, KV head, block of the wanted range).
//
// The code arithmetic is quantize_block's of csa_internal.cuh: explicitly
// rounded float32 operations, so that the codes are reproducible bit for
// bit.
#include "csa_rows.cuh"

namespace csa {

struct Kv4AppendArgs {
  csa_kv4 c;
  const void* k;
  const void* v;
  csa_strides ks, vs;
  const int64_t* len;
  const int64_t* n_new;
  unsigned* status;
  int64_t n_max, nblk_max;
  int B, T, Hkv;
};

struct Kv4UnpackArgs {
  csa_kv4 c;
  const int64_t* first;
  const int64_t* len;
  void* K;
  void* V;
  unsigned* status;
  int64_t rows, n_max, nblk_max;
  int B, Hkv;
};

// clamp(rint(fl(fl(x - m) / step)), 0, 15); 0 for a NaN
__device__ __forceinline__ unsigned code4(float x, float m, float step) {
  return (unsigned)fminf(fmaxf(rintf(fdiv(fsub(x, m), step)), 0.0f), 15.0f);
}
constexpr int kKv4Threads = 256;

// Codes of CPL values, each on top of kCodeBase.  Where the step is in the normal range the
// product with the reciprocal, off by less than 1e-5 (a quotient up to 15,
// three roundings), decides unless it lies that close to the middle between
// two codes; only then is the quotient itself computed (on 16-bit inputs, whose
// quotients are often exactly half way, for about one value in a thousand).
// The division on every value doubled the time of a long append.  Adding
// 3 * 2^22 rounds to an integer, which then stands in the low bits.
constexpr float kCodeRound = 12582912.0f;
constexpr unsigned kCodeBase = 0x4B400000u;      // the bits of kCodeRound
template <int CPL>
__device__ __forceinline__ void codes4(const float (&x)[CPL], const float (&m)[CPL], const float (&step)[CPL],
                                           const float (&inv)[CPL], bool plain, unsigned (&code)[CPL]) {
  float off = 0.0f;
#pragma unroll
  for (int c = 0; c < CPL; ++c) {
    const float y = fsub(x[c], m[c]) * inv[c];
    const float q = fadd(y, kCodeRound);
    off = fmaxf(off, fabsf(fsub(y, fsub(q, kCodeRound))));
    code[c] = __float_as_uint(fminf(q, kCodeRound + 15.0f));
  }
  if (!(plain && off < 0.49999f)) {
#pragma unroll
    for (int c = 0; c < CPL; ++c) code[c] = kCodeBase + code4(x[c], m[c], step[c]);
  }
}

// v[e] (e = 0 .. 7): value of row e in this lane.  Returns in v[0] op over the
// warp of row lane % 8.
template <typename U, typename Op>
__device__ __forceinline__ void reduce8(U (&v)[8], const Op op) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int s = 0; s < 3; ++s) {
    const bool hi = (lane >> s) & 1;
#pragma unroll
    for (int i = 0; i < (4 >> s); ++i) {
      const U send = hi ? v[2 * i] : v[2 * i + 1], keep = hi ? v[2 * i + 1] : v[2 * i];
      v[i] = op(keep, __shfl_xor_sync(0xffffffffu, send, 1 << s));
    }
  }
  v[0] = op(v[0], __shfl_xor_sync(0xffffffffu, v[0], 8));
  v[0] = op(v[0], __shfl_xor_sync(0xffffffffu, v[0], 16));
}

// lo, hi: over the warp, minimum and maximum of row lane % 8 of eight rows of
// which each lane holds a part
__device__ __forceinline__ void rows_minmax(const unsigned (&r)[8], float& lo, float& hi) {
  // (minimum, -maximum) of a row as a pair, so that one minimum serves both
  unsigned v[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const unsigned neg = r[e] ^ 0x80008000u;
    v[e] = min2_nan(__byte_perm(r[e], neg, 0x5410), __byte_perm(r[e], neg, 0x7632));
  }
  reduce8(v, [](unsigned a, unsigned b) { return min2_nan(a, b); });
  lo = __uint_as_float(v[0] << 16);
  hi = -__uint_as_float(v[0] & 0xFFFF0000u);
}
__device__ __forceinline__ void rows_minmax(const uint2 (&r)[8], float& lo, float& hi) {
  unsigned v[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const unsigned a = min2_nan(r[e].x, r[e].y), b = max2_nan(r[e].x, r[e].y) ^ 0x80008000u;
    v[e] = min2_nan(__byte_perm(a, b, 0x5410), __byte_perm(a, b, 0x7632));
  }
  reduce8(v, [](unsigned a, unsigned b) { return min2_nan(a, b); });
  lo = __uint_as_float(v[0] << 16);
  hi = -__uint_as_float(v[0] & 0xFFFF0000u);
}
__device__ __forceinline__ void reduce_both(float (&l)[8], float (&h)[8], float& lo, float& hi) {
  reduce8(l, [](float a, float b) { return min_nan(a, b); });
  reduce8(h, [](float a, float b) { return max_nan(a, b); });
  lo = l[0];
  hi = h[0];
}
__device__ __forceinline__ void rows_minmax(const float2 (&r)[8], float& lo, float& hi) {
  float l[8], h[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) { l[e] = min_nan(r[e].x, r[e].y); h[e] = max_nan(r[e].x, r[e].y); }
  reduce_both(l, h, lo, hi);
}
__device__ __forceinline__ void rows_minmax(const float4 (&r)[8], float& lo, float& hi) {
  float l[8], h[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    l[e] = min_nan(min_nan(r[e].x, r[e].y), min_nan(r[e].z, r[e].w));
    h[e] = max_nan(max_nan(r[e].x, r[e].y), max_nan(r[e].z, r[e].w));
  }
  reduce_both(l, h, lo, hi);
}

// Warp w takes the eight tokens of word w of the value rows, 32 i + 16 u + 8 v
// + 2 (w / 2) + e with i = w % 2, of which lane l holds the channels [l D / 32,
// (l + 1) D / 32): all 16 rows (K and V) are loaded at once, a row by one
// access of the warp, and stay in registers.  A key channel's minimum and
// maximum go over the warps (shared memory), a value row's over the lanes.
//
// 32K tokens x 8 heads x 128, bf16: 52 us for 134 MB read and 42 MB written,
// a little over a third of the copy bandwidth.  It is the instructions that
// count (35 an element of K and V on a thread at first, 25 now, issue slots
// 62% busy): a code costs nine, minimum and maximum of bf16 are taken in pairs
// (72 -> 52 us, with the addresses of a block whose rows are all new).  Three
// CTAs on an SM; two, with no limit on registers, took 62 us, four 51 with
// spills.  float32 rows need twice the registers: two CTAs.
template <int D, typename E>
__global__ void __launch_bounds__(kKv4Threads, sizeof(E) == 2 ? 3 : 2) kv4_append_kernel(const Kv4AppendArgs a) {
  pdl_entry();
  constexpr int CPL = D / 32;
  typedef typename Row<CPL, E>::T RowT;
  __shared__ __align__(16) RowT s_lo[8][32], s_hi[8][32];
  __shared__ __align__(16) unsigned s_v[8][D];
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int g = blockIdx.y, b = blockIdx.z;
  if ((a.status || a.c.refused) && blockIdx.x == 0 && g == 0 && b == 0 && tid < 32) {
    bool bad = false;
    for (int i = tid; i < a.B; i += 32) {
      const int64_t n = a.len[i], m = a.n_new ? a.n_new[i] : a.T;
      bad |= m < 0 || m > a.T || n < m || n > a.n_max;
    }
    report_range(a.status, a.c.refused, bad);
  }
  const int64_t n = a.len[b], m = a.n_new ? a.n_new[b] : (int64_t)a.T;
  if (m <= 0 || m > a.T || n < m || n > a.n_max) return;
  const int64_t start = n - m, blk0 = start / kBlock, whole = n / kBlock;   // blocks [0, whole) are whole
  const int64_t blk = blk0 + blockIdx.x;
  // CTAs: the blocks that become whole, or (when none does) the first one,
  // which then only keeps rows
  if (blk > blk0 && blk >= whole) return;
  const int64_t bg = (int64_t)b * a.Hkv + g;
  E* Kt = reinterpret_cast<E*>(a.c.Kt) + bg * kBlock * D;
  E* Vt = reinterpret_cast<E*>(a.c.Vt) + bg * kBlock * D;
  const E* kn = reinterpret_cast<const E*>(a.k) + b * a.ks.b + g * a.ks.h;
  const E* vn = reinterpret_cast<const E*>(a.v) + b * a.vs.b + g * a.vs.h;
  if (blk < whole) {
    const int64_t p0 = blk * kBlock, at = bg * a.nblk_max + blk;
    const int t0 = 32 * (w & 1) + 2 * (w >> 1);
    RowT rk[8], rv[8];
    if (p0 >= start) {          // all rows are new
      const E* k = kn + (p0 - start + t0) * a.ks.t + lane * CPL;
      const E* v = vn + (p0 - start + t0) * a.vs.t + lane * CPL;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int t = 16 * ((e >> 1) & 1) + 8 * (e & 1) + (e >> 2);
        rk[e] = *reinterpret_cast<const RowT*>(k + t * a.ks.t);
        rv[e] = *reinterpret_cast<const RowT*>(v + t * a.vs.t);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int t = t0 + 16 * ((e >> 1) & 1) + 8 * (e & 1) + (e >> 2);
        const int64_t p = p0 + t;
        const E* k = p < start ? Kt + t * D : kn + (p - start) * a.ks.t;
        const E* v = p < start ? Vt + t * D : vn + (p - start) * a.vs.t;
        rk[e] = *reinterpret_cast<const RowT*>(k + lane * CPL);
        rv[e] = *reinterpret_cast<const RowT*>(v + lane * CPL);
      }
    }
    // keys: one (m, Delta) per channel
    RowT klo = rk[0], khi = rk[0];
#pragma unroll
    for (int e = 1; e < 8; ++e) { klo = pick<false>(klo, rk[e]); khi = pick<true>(khi, rk[e]); }
    s_lo[w][lane] = klo;
    s_hi[w][lane] = khi;
    // values: one (m, Delta) per token, over the lanes meanwhile
    float x[CPL], vm, vhi;
    rows_minmax(rv, vm, vhi);
    const float vstep = fdiv(fsub(vhi, vm), 15.0f), vinv = approx_rcp(vstep);
    if (lane < 8)
      reinterpret_cast<float2*>(a.c.vscale)[at * kBlock + t0 + 16 * ((lane >> 1) & 1) + 8 * (lane & 1) + (lane >> 2)] =
          make_float2(vm, vstep);
    unsigned word[CPL], code[CPL];
#pragma unroll
    for (int c = 0; c < CPL; ++c) word[c] = 0u - kCodeBase * 0x11111111u;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float me[CPL], de[CPL], ie[CPL];
      me[0] = __shfl_sync(0xffffffffu, vm, e);
      de[0] = __shfl_sync(0xffffffffu, vstep, e);
      ie[0] = __shfl_sync(0xffffffffu, vinv, e);
#pragma unroll
      for (int c = 1; c < CPL; ++c) { me[c] = me[0]; de[c] = de[0]; ie[c] = ie[0]; }
      row_floats<CPL>(rv[e], x, E());
      codes4<CPL>(x, me, de, ie, step_plain(de[0]), code);       // (Delta = 0: 0/0, code 0)
#pragma unroll
      for (int c = 0; c < CPL; ++c) word[c] += code[c] << (4 * e);
    }
#pragma unroll
    for (int c = 0; c < CPL; ++c) s_v[w][lane * CPL + c] = word[c];
    __syncthreads();
    klo = s_lo[0][lane];
    khi = s_hi[0][lane];
#pragma unroll
    for (int i = 1; i < 8; ++i) { klo = pick<false>(klo, s_lo[i][lane]); khi = pick<true>(khi, s_hi[i][lane]); }
    float lo[CPL], hi[CPL], inv[CPL];
    row_floats<CPL>(klo, lo, E());
    row_floats<CPL>(khi, hi, E());
    bool plain = true;
#pragma unroll
    for (int c = 0; c < CPL; ++c) {
      hi[c] = fdiv(fsub(hi[c], lo[c]), 15.0f);     // the step from here on
      if (hi[c] == 0.0f) hi[c] = 1.0f;
      inv[c] = approx_rcp(hi[c]);
      plain = plain && step_plain(hi[c]);
    }
    if (w == 0) {
#pragma unroll
      for (int c = 0; c < CPL; ++c) {
        a.c.bounds[at * 2 * D + lane * CPL + c] = lo[c];
        a.c.bounds[at * 2 * D + D + lane * CPL + c] = hi[c];
      }
    }
    uint8_t* K4 = a.c.K4 + at * kBlock * (D / 2) + lane * (CPL / 2);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int t = t0 + 16 * ((e >> 1) & 1) + 8 * (e & 1) + (e >> 2);
      row_floats<CPL>(rk[e], x, E());
      codes4<CPL>(x, lo, hi, inv, plain, code);
      unsigned all = 0u - (unsigned)(((1ull << 4 * CPL) - 1) / 15 * kCodeBase);
#pragma unroll
      for (int c = 0; c < CPL; ++c) all += code[c] << (4 * c);
      if (CPL == 4) *reinterpret_cast<uint16_t*>(K4 + t * (D / 2)) = (uint16_t)all;
      else K4[t * (D / 2)] = (uint8_t)all;
    }
    // value words, four of a channel's eight by a thread
    if (tid < 2 * D) {
      const int c = tid >> 1, q = (tid & 1) * 4;
      reinterpret_cast<uint4*>(a.c.V4 + at * D * (kBlock / 2))[tid] =
          make_uint4(s_v[q][c], s_v[q + 1][c], s_v[q + 2][c], s_v[q + 3][c]);
    }
  }
  // the rows of the block that stays incomplete (after every warp has read
  // the old ones: they are all in registers since the barrier above)
  if (blk == blk0) {
    const int64_t p0 = max(start, whole * kBlock);
    const int left = (int)(n - p0);       // below 64
    for (int r = w; r < left; r += kKv4Threads / 32) {
      const int64_t p = p0 + r;
      const RowT k = *reinterpret_cast<const RowT*>(kn + (p - start) * a.ks.t + lane * CPL);
      const RowT v = *reinterpret_cast<const RowT*>(vn + (p - start) * a.vs.t + lane * CPL);
      *reinterpret_cast<RowT*>(Kt + (p % kBlock) * D + lane * CPL) = k;
      *reinterpret_cast<RowT*>(Vt + (p % kBlock) * D + lane * CPL) = v;
    }
  }
}

// Code k of a word as a float: the nibble under the exponent of 2^23, minus
// 2^23.  lo = word & 0x0F0F0F0F, hi = word >> 4 & 0x0F0F0F0F.
__device__ __forceinline__ float nibble(unsigned lo, unsigned hi, int k) {
  return __uint_as_float(__byte_perm(k & 1 ? hi : lo, 0x4B000000u, 0x7440 + k / 2)) - 8388608.0f;
}
// Half of the threads take the keys, half the values; a thread produces eight
// channels of a row at a time.  Keys: the eight channels' bounds stay in
// registers while the thread walks down the rows, one code word a row.
// Values: eight words, one of each channel, hold eight tokens of eight
// channels; the codes pass through shared memory, eight rows 260 bytes apart
// so that the threads of a row read different banks, and the tokens' scales
// are on their way meanwhile (loaded after the barrier: 151 us where it is 126).
//
// Bound by memory: 128K tokens x 8 heads x 128 to bf16, 696 MB in 126 us,
// 5.5 TB/s or 81% of the copy bandwidth.  Stores marked as streaming made no
// difference.
template <int D, typename E>
__global__ void __launch_bounds__(kKv4Threads) kv4_unpack_kernel(const Kv4UnpackArgs a) {
  pdl_entry();
  constexpr int CG = D / 8;                         // groups of eight channels
  constexpr int HALF = kKv4Threads / 2;
  __shared__ unsigned s_v[CG * 65];
  const int tid = threadIdx.x;
  const int g = blockIdx.y, b = blockIdx.z;
  if (a.status && blockIdx.x == 0 && g == 0 && b == 0 && tid < 32) {
    bool bad = false;
    for (int i = tid; i < a.B; i += 32) {
      const int64_t n = a.len[i], f = a.first ? a.first[i] : 0;
      bad |= n < 0 || n > a.n_max || f < 0;
    }
    report_range(a.status, nullptr, bad);
  }
  const int64_t n = a.len[b], first = a.first ? a.first[b] : 0;
  if (n < 0 || n > a.n_max || first < 0 || first >= n) return;
  const int64_t end = n - first < a.rows ? n : first + a.rows;
  const int64_t blk = first / kBlock + blockIdx.x;
  const int64_t p0 = max(first, blk * kBlock), p1 = min(end, (blk + 1) * kBlock);
  if (p0 >= p1) return;
  const int r0 = (int)(p0 - blk * kBlock), r1 = (int)(p1 - blk * kBlock);     // rows [r0, r1) of the block
  const int64_t bg = (int64_t)b * a.Hkv + g;
  const int64_t at = bg * a.nblk_max + blk;
  // row r of the block is row blk * 64 + r - first of the output
  const int64_t out = (bg * a.rows + blk * kBlock - first) * D;
  E* Ko = reinterpret_cast<E*>(a.K) + out;
  E* Vo = reinterpret_cast<E*>(a.V) + out;
  const int cg = tid % CG;
  if (blk >= n / kBlock) {
    const int half = tid / HALF;
    const E* src = reinterpret_cast<const E*>(half ? a.c.Vt : a.c.Kt) + bg * kBlock * D;
    E* dst = half ? Vo : Ko;
    constexpr int Q = 8 * sizeof(E) / 16;
    for (int r = r0 + tid % HALF / CG; r < r1; r += HALF / CG) {
#pragma unroll
      for (int i = 0; i < Q; ++i)
        reinterpret_cast<uint4*>(dst + r * D + cg * 8)[i] = reinterpret_cast<const uint4*>(src + r * D + cg * 8)[i];
    }
    return;
  }
  const unsigned* V4 = reinterpret_cast<const unsigned*>(a.c.V4 + at * D * (kBlock / 2));
  for (int i = tid; i < D * 8; i += kKv4Threads) s_v[i / 64 * 65 + i % 64] = V4[i];
  constexpr int STEP = HALF / CG;                   // groups of threads, each of which holds all channels of a row
  const int sub = tid % HALF / CG;
  if (tid < HALF) {
    float m[8], dl[8];
    const float* bp = a.c.bounds + at * 2 * D + cg * 8;
#pragma unroll
    for (int i = 0; i < 8; i += 4) {
      const float4 u = *reinterpret_cast<const float4*>(bp + i), v = *reinterpret_cast<const float4*>(bp + D + i);
      m[i] = u.x; m[i + 1] = u.y; m[i + 2] = u.z; m[i + 3] = u.w;
      dl[i] = v.x; dl[i + 1] = v.y; dl[i + 2] = v.z; dl[i + 3] = v.w;
    }
    const unsigned* K4 = reinterpret_cast<const unsigned*>(a.c.K4 + at * kBlock * (D / 2));
    unsigned word[kBlock / STEP];
#pragma unroll
    for (int j = 0; j < kBlock / STEP; ++j) word[j] = K4[(sub + j * STEP) * CG + cg];
    bar_sync(1, kKv4Threads);
    E* dst = Ko + sub * D + cg * 8;
#pragma unroll
    for (int j = 0; j < kBlock / STEP; ++j) {
      const int r = sub + j * STEP;
      const unsigned lo = word[j] & 0x0F0F0F0Fu, hi = word[j] >> 4 & 0x0F0F0F0Fu;
      float x[8];
#pragma unroll
      for (int c = 0; c < 8; ++c) x[c] = fadd(fmul(nibble(lo, hi, c), dl[c]), m[c]);
      if (r >= r0 && r < r1) store8<E>(dst + j * STEP * D, x);
    }
  } else {
    // word wi: tokens 32 i + 16 u + 8 v + 2 w + e, i = wi % 2, w = wi / 2
    constexpr int N = 8 / STEP > 1 ? 8 / STEP : 1;  // words of a thread
    float2 sc[N][8];
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int wi = sub + k * STEP, t0 = 32 * (wi & 1) + 2 * (wi >> 1 & 3);
#pragma unroll
      for (int u = 0; u < 4; ++u) {                 // two tokens' (m, Delta), e = 0 and 1, side by side
        const float4 two = *reinterpret_cast<const float4*>(a.c.vscale + (at * kBlock + t0 + 16 * (u >> 1) + 8 * (u & 1)) * 2);
        sc[k][u] = make_float2(two.x, two.y);
        sc[k][u + 4] = make_float2(two.z, two.w);
      }
    }
    bar_sync(1, kKv4Threads);
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int wi = sub + k * STEP;
      if (wi >= 8) break;                           // (d = 64: sixteen groups)
      unsigned lo[8], hi[8];
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const unsigned word = s_v[cg * 65 + c * 8 + wi];
        lo[c] = word & 0x0F0F0F0Fu;
        hi[c] = word >> 4 & 0x0F0F0F0Fu;
      }
      const int t0 = 32 * (wi & 1) + 2 * (wi >> 1);
      E* dst = Vo + t0 * D + cg * 8;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int dr = 16 * ((e >> 1) & 1) + 8 * (e & 1) + (e >> 2), r = t0 + dr;
        float x[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) x[c] = fadd(fmul(nibble(lo[c], hi[c], e), sc[k][e].y), sc[k][e].x);
        if (r >= r0 && r < r1) store8<E>(dst + dr * D, x);
      }
    }
  }
}

namespace {

template <int D, typename E>
cudaError_t launch_append(const Kv4AppendArgs& a, dim3 grid, cudaStream_t st) {
  launch_pdl(kv4_append_kernel<D, E>, grid, dim3(kKv4Threads), 0, st, a);
  return cudaGetLastError();
}

template <int D, typename E>
cudaError_t launch_unpack(const Kv4UnpackArgs& a, dim3 grid, cudaStream_t st) {
  launch_pdl(kv4_unpack_kernel<D, E>, grid, dim3(kKv4Threads), 0, st, a);
  return cudaGetLastError();
}

}  // namespace

bool kv4_cache_ok(const csa_kv4* c) {
  return c && c->K4 && c->bounds && c->V4 && c->vscale && c->Kt && c->Vt && aligned16(c->K4) && aligned16(c->bounds) &&
         aligned16(c->V4) && aligned16(c->vscale) && aligned16(c->Kt) && aligned16(c->Vt) &&
         ((uintptr_t)c->refused & 3) == 0;
}

}  // namespace csa

using namespace csa;

extern "C" {

csa_status csa_kv4_append(const csa_shape* shape, const csa_kv4* cache, int T, const void* k, const csa_strides* ks,
                          const void* v, const csa_strides* vs, const int64_t* len, const int64_t* n_new,
                          uint32_t* status, void* stream) {
  if (!shape_ok(shape) || !kv4_cache_ok(cache) || T < 1 || !k || !v || !len) return CSA_ERR_INVALID_ARG;
  const csa_status su = shape_supported(shape);
  if (su != CSA_OK) return su;
  const bool bf16 = shape->dtype == CSA_BF16;
  const int64_t unit = bf16 ? 8 : 4;
  if (!strides_ok(ks, unit, shape->B, T, shape->Hkv) || !strides_ok(vs, unit, shape->B, T, shape->Hkv) ||
      !aligned16(k) || !aligned16(v))
    return CSA_ERR_INVALID_ARG;
  Kv4AppendArgs a = {};
  a.c = *cache; a.k = k; a.v = v; a.ks = *ks; a.vs = *vs; a.len = len; a.n_new = n_new; a.status = status;
  a.n_max = shape->n_max; a.nblk_max = (shape->n_max + kBlock - 1) / kBlock;
  a.B = shape->B; a.T = T; a.Hkv = shape->Hkv;
  // blocks that T tokens can touch
  const int64_t nb = ((int64_t)T + 2 * kBlock - 2) / kBlock;
  dim3 grid((unsigned)(nb < a.nblk_max ? nb : a.nblk_max), (unsigned)shape->Hkv, (unsigned)shape->B);
  add_launches(1);
  cudaStream_t st = (cudaStream_t)stream;
  const cudaError_t e = shape->d == 128 ? (bf16 ? launch_append<128, __nv_bfloat16>(a, grid, st) : launch_append<128, float>(a, grid, st))
                                        : (bf16 ? launch_append<64, __nv_bfloat16>(a, grid, st) : launch_append<64, float>(a, grid, st));
  return e == cudaSuccess ? CSA_OK : CSA_ERR_CUDA;
}

csa_status csa_kv4_unpack(const csa_shape* shape, const csa_kv4* cache, int64_t rows, const int64_t* first,
                          const int64_t* len, void* K, void* V, uint32_t* status, void* stream) {
  if (!shape_ok(shape) || !kv4_cache_ok(cache) || rows < 1 || rows > (int64_t)1 << 31 || !len || !K || !V ||
      !aligned16(K) || !aligned16(V))
    return CSA_ERR_INVALID_ARG;
  const csa_status su = shape_supported(shape);
  if (su != CSA_OK) return su;
  const bool bf16 = shape->dtype == CSA_BF16;
  Kv4UnpackArgs a = {};
  a.c = *cache; a.first = first; a.len = len; a.K = K; a.V = V; a.status = status; a.rows = rows;
  a.n_max = shape->n_max; a.nblk_max = (shape->n_max + kBlock - 1) / kBlock;
  a.B = shape->B; a.Hkv = shape->Hkv;
  const int64_t nb = (rows + 2 * kBlock - 2) / kBlock;
  dim3 grid((unsigned)(nb < a.nblk_max ? nb : a.nblk_max), (unsigned)shape->Hkv, (unsigned)shape->B);
  add_launches(1);
  cudaStream_t st = (cudaStream_t)stream;
  const cudaError_t e = shape->d == 128 ? (bf16 ? launch_unpack<128, __nv_bfloat16>(a, grid, st) : launch_unpack<128, float>(a, grid, st))
                                        : (bf16 ? launch_unpack<64, __nv_bfloat16>(a, grid, st) : launch_unpack<64, float>(a, grid, st));
  return e == cudaSuccess ? CSA_OK : CSA_ERR_CUDA;
}

}  // extern "C"
