// The 8-bit K/V cache (csa.h "a K/V cache held in 8 bits"): appending rows
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
// Steps and codes are explicitly rounded float32 operations, so that they are
// reproducible bit for bit.
//
// d = 128, bf16, 8 KV heads: 4 sequences' up to 8191 new tokens are appended in 41
// us (15 instructions an element, issue slots 55% busy) and read back in 31; one
// token to each of 64 in 4.2 us; 4 x 32K rows are read back in 122 us, 6.6 TB/s,
// what a copy reaches.
#include "csa_rows.cuh"

namespace csa {

struct Kv8AppendArgs {
  csa_kv8 c;
  const void* k;
  const void* v;
  csa_strides ks, vs;
  const int64_t* len;
  const int64_t* n_new;
  unsigned* status;
  int64_t n_max, nblk_max;
  int B, T, Hkv;
};

struct Kv8UnpackArgs {
  csa_kv8 c;
  const int64_t* first;
  const int64_t* len;
  void* K;
  void* V;
  unsigned* status;
  int64_t rows, n_max, nblk_max;
  int B, Hkv;
};

constexpr int kKv8Threads = 256;
constexpr int kKv8Warps = kKv8Threads / 32;

// the step of values up to `top` in magnitude
__device__ __forceinline__ float step8(float top) {
  const float step = fdiv(top, 127.0f);
  return step == 0.0f ? 1.0f : step;
}
// clamp(rint(fl(x / step)), -127, 127) + 128; 128 for a NaN
__device__ __forceinline__ unsigned code8(float x, float step) {
  const float q = rintf(fdiv(x, step));
  return (unsigned)((q == q ? fminf(fmaxf(q, -127.0f), 127.0f) : 0.0f) + 128.0f);
}

// Codes of CPL values, in the low byte of each word (what is above it is not
// theirs).  Where the step is in the normal range the product with the
// reciprocal decides unless it lies within 3e-5 of the middle between two codes
// (a quotient up to 127: the reciprocal's unit in the last place is 1.6e-5 of it,
// the quotient's own rounding 0.8e-5); only then is the quotient itself computed.
// Adding 3 * 2^22 + 128 rounds to an integer and leaves it, plus 128, in the low
// byte.
constexpr float kCode8Round = 12582912.0f + 128.0f;
template <int CPL>
__device__ __forceinline__ void codes8(const float (&x)[CPL], float step, float inv, bool plain, unsigned (&code)[CPL]) {
  float off = 0.0f;
#pragma unroll
  for (int c = 0; c < CPL; ++c) {
    const float q = fmaf(x[c], inv, kCode8Round);
    off = fmaxf(off, fabsf(fmaf(x[c], inv, kCode8Round - q)));
    code[c] = __float_as_uint(q);
  }
  if (!(plain && off < 0.49997f)) {
#pragma unroll
    for (int c = 0; c < CPL; ++c) code[c] = code8(x[c], step);
  }
}
// low bytes side by side
template <int CPL>
__device__ __forceinline__ unsigned bytes_of(const unsigned (&code)[CPL]) {
  const unsigned lo = __byte_perm(code[0], code[1], 0x0040);
  return CPL == 2 ? lo : __byte_perm(lo, __byte_perm(code[CPL - 2], code[CPL - 1], 0x0040), 0x5410);
}
template <int CPL> struct Codes { typedef uint32_t T; };
template <> struct Codes<2> { typedef uint16_t T; };

__device__ __forceinline__ float warp_max_nan(float x) {
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) x = max_nan(x, __shfl_xor_sync(0xffffffffu, x, m));
  return x;
}
template <int CPL>
__device__ __forceinline__ float top_of(const float (&lo)[CPL], const float (&hi)[CPL]) {
  float t = 0.0f;
#pragma unroll
  for (int c = 0; c < CPL; ++c) t = max_nan(t, max_nan(fabsf(lo[c]), fabsf(hi[c])));
  return t;
}

// Warp w takes the tokens 8 w .. 8 w + 7, of which lane l holds the channels
// [l D / 32, (l + 1) D / 32): all 16 rows (K and V) are loaded at once, a row by
// one access of the warp, and stay in registers.  Extremes go over the warps
// through shared memory, once: each channel's of the keys (whose span is
// coded like the keys themselves, rounding being monotone), one number of the
// values.  Value codes pass through shared memory into channel rows.
template <int D, typename E>
__global__ void __launch_bounds__(kKv8Threads, sizeof(E) == 2 ? 3 : 2) kv8_append_kernel(const Kv8AppendArgs a) {
  pdl_entry();
  constexpr int CPL = D / 32, PITCH = kBlock + 8;
  typedef typename Row<CPL, E>::T RowT;
  __shared__ __align__(16) RowT s_lo[kKv8Warps][32], s_hi[kKv8Warps][32];
  __shared__ float s_top[kKv8Warps];
  __shared__ __align__(16) uint8_t s_v[D * PITCH];       // [channel][token], rows 72 bytes apart
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
    const int t0 = 8 * w;
    RowT rk[8], rv[8];
    if (p0 >= start) {          // all rows are new
      const E* k = kn + (p0 - start + t0) * a.ks.t + lane * CPL;
      const E* v = vn + (p0 - start + t0) * a.vs.t + lane * CPL;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        rk[e] = *reinterpret_cast<const RowT*>(k + e * a.ks.t);
        rv[e] = *reinterpret_cast<const RowT*>(v + e * a.vs.t);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int t = t0 + e;
        const int64_t p = p0 + t;
        const E* k = p < start ? Kt + t * D : kn + (p - start) * a.ks.t;
        const E* v = p < start ? Vt + t * D : vn + (p - start) * a.vs.t;
        rk[e] = *reinterpret_cast<const RowT*>(k + lane * CPL);
        rv[e] = *reinterpret_cast<const RowT*>(v + lane * CPL);
      }
    }
    RowT klo = rk[0], khi = rk[0], vlo = rv[0], vhi = rv[0];
#pragma unroll
    for (int e = 1; e < 8; ++e) {
      klo = pick<false>(klo, rk[e]); khi = pick<true>(khi, rk[e]);
      vlo = pick<false>(vlo, rv[e]); vhi = pick<true>(vhi, rv[e]);
    }
    s_lo[w][lane] = klo;
    s_hi[w][lane] = khi;
    float lo[CPL], hi[CPL], x[CPL];
    row_floats<CPL>(vlo, lo, E());
    row_floats<CPL>(vhi, hi, E());
    const float vtop = warp_max_nan(top_of<CPL>(lo, hi));
    if (lane == 0) s_top[w] = vtop;
    __syncthreads();
    klo = s_lo[0][lane];
    khi = s_hi[0][lane];
    float top = s_top[0];
#pragma unroll
    for (int i = 1; i < kKv8Warps; ++i) {
      klo = pick<false>(klo, s_lo[i][lane]);
      khi = pick<true>(khi, s_hi[i][lane]);
      top = max_nan(top, s_top[i]);
    }
    row_floats<CPL>(klo, lo, E());
    row_floats<CPL>(khi, hi, E());
    const float kstep = step8(warp_max_nan(top_of<CPL>(lo, hi))), vstep = step8(top);
    const float kinv = approx_rcp(kstep), vinv = approx_rcp(vstep);
    const bool kplain = step_plain(kstep), vplain = step_plain(vstep);
    unsigned code[CPL];
    if (w == 0) {
      typedef typename Codes<CPL>::T CT;
      CT* span = reinterpret_cast<CT*>(a.c.span + at * 2 * D) + lane;
      codes8<CPL>(hi, kstep, kinv, kplain, code);
      span[0] = (CT)bytes_of<CPL>(code);
      codes8<CPL>(lo, kstep, kinv, kplain, code);
      span[32] = (CT)bytes_of<CPL>(code);
      if (lane == 0) reinterpret_cast<float2*>(a.c.scale)[at] = make_float2(kstep, vstep);
    }
    // values: eight tokens of a channel side by side
    unsigned v8[CPL][2];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      row_floats<CPL>(rv[e], x, E());
      codes8<CPL>(x, vstep, vinv, vplain, code);
#pragma unroll
      for (int c = 0; c < CPL; ++c) {
        const int sel = e % 4 == 0 ? 0x3214 : e % 4 == 1 ? 0x3240 : e % 4 == 2 ? 0x3410 : 0x4210;
        v8[c][e / 4] = __byte_perm(e % 4 ? v8[c][e / 4] : 0u, code[c], sel);
      }
    }
#pragma unroll
    for (int c = 0; c < CPL; ++c)
      *reinterpret_cast<uint2*>(s_v + (lane * CPL + c) * PITCH + t0) = make_uint2(v8[c][0], v8[c][1]);
    // keys: token 8 w + e is row (j, g) = (4 (w % 2) + e / 2, 2 (w / 2) + e % 2)
    uint8_t* K8 = a.c.K8 + at * kBlock * D + (lane * CPL / 64 * 8) * 64 + lane * CPL % 64;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      row_floats<CPL>(rk[e], x, E());
      codes8<CPL>(x, kstep, kinv, kplain, code);
      const int j = 4 * (w & 1) + e / 2, r = 2 * (w >> 1) + (e & 1);
      *reinterpret_cast<typename Codes<CPL>::T*>(K8 + (j * (D / 64) * 8 + r) * 64) = (typename Codes<CPL>::T)bytes_of<CPL>(code);
    }
    __syncthreads();
    uint2* V8 = reinterpret_cast<uint2*>(a.c.V8 + at * kBlock * D);
#pragma unroll
    for (int i = tid; i < D * 8; i += kKv8Threads) V8[i] = *reinterpret_cast<const uint2*>(s_v + (i >> 3) * PITCH + (i & 7) * 8);
  }
  // the rows of the block that stays incomplete (after every warp has read
  // the old ones: they are all in registers since the barriers above)
  if (blk == blk0) {
    const int64_t p0 = max(start, whole * kBlock);
    const int left = (int)(n - p0);       // below 64
    for (int r = w; r < left; r += kKv8Warps) {
      const int64_t p = p0 + r;
      const RowT k = *reinterpret_cast<const RowT*>(kn + (p - start) * a.ks.t + lane * CPL);
      const RowT v = *reinterpret_cast<const RowT*>(vn + (p - start) * a.vs.t + lane * CPL);
      *reinterpret_cast<RowT*>(Kt + (p % kBlock) * D + lane * CPL) = k;
      *reinterpret_cast<RowT*>(Vt + (p % kBlock) * D + lane * CPL) = v;
    }
  }
}

// Byte k of a word as the number it stands for: under the exponent of 2^23,
// minus 2^23 + 128.
__device__ __forceinline__ float number8(unsigned word, int k) {
  return __uint_as_float(__byte_perm(word, 0x4B000000u, 0x7440 + k)) - 8388736.0f;
}

// Half of the threads take the keys, half the values; a thread produces eight
// channels of a row at a time.  Value codes pass through shared memory, eight
// channel rows 516 bytes apart so that the threads of a row read different banks.
template <int D, typename E>
__global__ void __launch_bounds__(kKv8Threads) kv8_unpack_kernel(const Kv8UnpackArgs a) {
  pdl_entry();
  constexpr int CG = D / 8;                         // groups of eight channels
  constexpr int HALF = kKv8Threads / 2;
  __shared__ unsigned s_v[CG * 129];
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
  const float2 step = reinterpret_cast<const float2*>(a.c.scale)[at];
  const unsigned* V8 = reinterpret_cast<const unsigned*>(a.c.V8 + at * kBlock * D);
#pragma unroll
  for (int i = tid; i < D * 16; i += kKv8Threads) s_v[i / 128 * 129 + i % 128] = V8[i];
  constexpr int STEP = HALF / CG;                   // groups of threads, each of which holds all channels of a row
  const int sub = tid % HALF / CG;
  if (tid < HALF) {
    const uint2* K8 = reinterpret_cast<const uint2*>(a.c.K8 + at * kBlock * D);
    uint2 word[kBlock / STEP];
#pragma unroll
    for (int i = 0; i < kBlock / STEP; ++i) {
      const int t = sub + i * STEP, j = (t & 15) >> 1, r = (t >> 4) * 2 + (t & 1);
      word[i] = K8[((j * (D / 64) + cg / 8) * 8 + r) * 8 + cg % 8];
    }
    bar_sync(1, kKv8Threads);
#pragma unroll
    for (int i = 0; i < kBlock / STEP; ++i) {
      const int r = sub + i * STEP;
      float x[8];
#pragma unroll
      for (int c = 0; c < 8; ++c) x[c] = fmul(number8(c < 4 ? word[i].x : word[i].y, c & 3), step.x);
      if (r >= r0 && r < r1) store8<E>(Ko + r * D + cg * 8, x);
    }
  } else {
    bar_sync(1, kKv8Threads);
#pragma unroll
    for (int wi = sub; wi < 16; wi += STEP) {       // tokens 4 wi .. 4 wi + 3
      unsigned word[8];
#pragma unroll
      for (int c = 0; c < 8; ++c) word[c] = s_v[cg * 129 + c * 16 + wi];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = 4 * wi + e;
        float x[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) x[c] = fmul(number8(word[c], e), step.y);
        if (r >= r0 && r < r1) store8<E>(Vo + r * D + cg * 8, x);
      }
    }
  }
}

namespace {

template <int D, typename E>
cudaError_t launch_append8(const Kv8AppendArgs& a, dim3 grid, cudaStream_t st) {
  launch_pdl(kv8_append_kernel<D, E>, grid, dim3(kKv8Threads), 0, st, a);
  return cudaGetLastError();
}

template <int D, typename E>
cudaError_t launch_unpack8(const Kv8UnpackArgs& a, dim3 grid, cudaStream_t st) {
  launch_pdl(kv8_unpack_kernel<D, E>, grid, dim3(kKv8Threads), 0, st, a);
  return cudaGetLastError();
}

}  // namespace

bool kv8_cache_ok(const csa_kv8* c) {
  return c && c->K8 && c->V8 && c->scale && c->span && c->Kt && c->Vt && aligned16(c->K8) && aligned16(c->V8) &&
         aligned16(c->scale) && aligned16(c->span) && aligned16(c->Kt) && aligned16(c->Vt) &&
         ((uintptr_t)c->refused & 3) == 0;
}

}  // namespace csa

using namespace csa;

extern "C" {

csa_status csa_kv8_append(const csa_shape* shape, const csa_kv8* cache, int T, const void* k, const csa_strides* ks,
                          const void* v, const csa_strides* vs, const int64_t* len, const int64_t* n_new,
                          uint32_t* status, void* stream) {
  if (!shape_ok(shape) || !kv8_cache_ok(cache) || T < 1 || !k || !v || !len) return CSA_ERR_INVALID_ARG;
  const csa_status su = shape_supported(shape);
  if (su != CSA_OK) return su;
  const bool bf16 = shape->dtype == CSA_BF16;
  const int64_t unit = bf16 ? 8 : 4;
  if (!strides_ok(ks, unit, shape->B, T, shape->Hkv) || !strides_ok(vs, unit, shape->B, T, shape->Hkv) ||
      !aligned16(k) || !aligned16(v))
    return CSA_ERR_INVALID_ARG;
  Kv8AppendArgs a = {};
  a.c = *cache; a.k = k; a.v = v; a.ks = *ks; a.vs = *vs; a.len = len; a.n_new = n_new; a.status = status;
  a.n_max = shape->n_max; a.nblk_max = (shape->n_max + kBlock - 1) / kBlock;
  a.B = shape->B; a.T = T; a.Hkv = shape->Hkv;
  // blocks that T tokens can touch
  const int64_t nb = ((int64_t)T + 2 * kBlock - 2) / kBlock;
  dim3 grid((unsigned)(nb < a.nblk_max ? nb : a.nblk_max), (unsigned)shape->Hkv, (unsigned)shape->B);
  add_launches(1);
  cudaStream_t st = (cudaStream_t)stream;
  const cudaError_t e = shape->d == 128 ? (bf16 ? launch_append8<128, __nv_bfloat16>(a, grid, st) : launch_append8<128, float>(a, grid, st))
                                        : (bf16 ? launch_append8<64, __nv_bfloat16>(a, grid, st) : launch_append8<64, float>(a, grid, st));
  return e == cudaSuccess ? CSA_OK : CSA_ERR_CUDA;
}

csa_status csa_kv8_unpack(const csa_shape* shape, const csa_kv8* cache, int64_t rows, const int64_t* first,
                          const int64_t* len, void* K, void* V, uint32_t* status, void* stream) {
  if (!shape_ok(shape) || !kv8_cache_ok(cache) || rows < 1 || rows > (int64_t)1 << 31 || !len || !K || !V ||
      !aligned16(K) || !aligned16(V))
    return CSA_ERR_INVALID_ARG;
  const csa_status su = shape_supported(shape);
  if (su != CSA_OK) return su;
  const bool bf16 = shape->dtype == CSA_BF16;
  Kv8UnpackArgs a = {};
  a.c = *cache; a.first = first; a.len = len; a.K = K; a.V = V; a.status = status; a.rows = rows;
  a.n_max = shape->n_max; a.nblk_max = (shape->n_max + kBlock - 1) / kBlock;
  a.B = shape->B; a.Hkv = shape->Hkv;
  const int64_t nb = (rows + 2 * kBlock - 2) / kBlock;
  dim3 grid((unsigned)(nb < a.nblk_max ? nb : a.nblk_max), (unsigned)shape->Hkv, (unsigned)shape->B);
  add_launches(1);
  cudaStream_t st = (cudaStream_t)stream;
  const cudaError_t e = shape->d == 128 ? (bf16 ? launch_unpack8<128, __nv_bfloat16>(a, grid, st) : launch_unpack8<128, float>(a, grid, st))
                                        : (bf16 ? launch_unpack8<64, __nv_bfloat16>(a, grid, st) : launch_unpack8<64, float>(a, grid, st));
  return e == cudaSuccess ? CSA_OK : CSA_ERR_CUDA;
}

}  // extern "C"
