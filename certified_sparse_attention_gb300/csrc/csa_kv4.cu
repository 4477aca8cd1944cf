// The 4-bit K/V cache (csa.h "a K/V cache held in 4 bits"): appending rows
// and reading rows back.
//
// append: one CTA per (sequence, KV head, block of 64 positions that the new
// tokens touch).  A block that becomes whole is gathered in shared memory
// (its first rows may lie in the kept rows Kt, Vt, the others among the new
// ones) and coded; the rows of the block that stays incomplete are copied to
// Kt, Vt.  When a call both completes a block and leaves a new incomplete
// one, the CTA of the first block writes the kept rows, after it has read
// the old ones: nobody else reads or writes them.
//
// unpack: one CTA per (sequence, KV head, block of the wanted range).
//
// The code arithmetic is quantize_block's of csa_internal.cuh: explicitly
// rounded float32 operations, so that the codes are reproducible bit for
// bit.
#include "csa_args.cuh"

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

// Place of token t of a block among the 64 nibbles of a V4 row, and back.
__host__ __device__ __forceinline__ int v4_place(int t) {
  return 16 * ((t >> 1) & 3) + 8 * (t >> 5) + 4 * (t & 1) + 2 * ((t >> 4) & 1) + ((t >> 3) & 1);
}
__host__ __device__ __forceinline__ int v4_token(int p) {
  return 32 * ((p >> 3) & 1) + 16 * ((p >> 1) & 1) + 8 * (p & 1) + 2 * (p >> 4) + ((p >> 2) & 1);
}

// minimum and maximum that keep a NaN
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// clamp(rint(fl(fl(x - m) / step)), 0, 15); 0 for a NaN
__device__ __forceinline__ unsigned code4(float x, float m, float step) {
  return (unsigned)fminf(fmaxf(rintf(fdiv(fsub(x, m), step)), 0.0f), 15.0f);
}
__device__ __forceinline__ float value4(unsigned code, float m, float step) {
  return fadd(fmul((float)code, step), m);
}

template <typename E> __device__ __forceinline__ E to_elem(float x);
template <> __device__ __forceinline__ float to_elem<float>(float x) { return x; }
template <> __device__ __forceinline__ __nv_bfloat16 to_elem<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

constexpr int kKv4Threads = 256;

// the status word of a call: set by one warp of its first CTA
__device__ __forceinline__ void report_range(unsigned* status, bool bad) {
  const unsigned any = __any_sync(0xffffffffu, bad);
  if ((threadIdx.x & 31) == 0) *status = any ? 8u : 0u;
}

template <int D, typename E>
__global__ void __launch_bounds__(kKv4Threads) kv4_append_kernel(const Kv4AppendArgs a) {
  pdl_entry();
  extern __shared__ __align__(16) uint8_t sm_raw[];
  float* s_x = reinterpret_cast<float*>(sm_raw);                 // [64][D + 1]
  float* s_mn = s_x + kBlock * (D + 1);                          // [D]
  float* s_dl = s_mn + D;                                        // [D]
  const int tid = threadIdx.x;
  const int g = blockIdx.y, b = blockIdx.z;
  if (a.status && blockIdx.x == 0 && g == 0 && b == 0 && tid < 32) {
    bool bad = false;
    for (int i = tid; i < a.B; i += 32) {
      const int64_t n = a.len[i], m = a.n_new ? a.n_new[i] : a.T;
      bad |= m < 0 || m > a.T || n < m || n > a.n_max;
    }
    report_range(a.status, bad);
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
    const int64_t p0 = blk * kBlock;
    const int64_t at = bg * a.nblk_max + blk;
    for (int i = tid; i < kBlock * D; i += kKv4Threads) {
      const int r = i / D, c = i - r * D;
      const int64_t p = p0 + r;
      s_x[r * (D + 1) + c] = Elem<E>::get(p < start ? Kt + r * D : kn + (p - start) * a.ks.t, c);
    }
    __syncthreads();
    // keys: one (m, Delta) per channel
    if (tid < D) {
      float mn = INFINITY, mx = -INFINITY;
      for (int r = 0; r < kBlock; ++r) {
        mn = min_nan(mn, s_x[r * (D + 1) + tid]);
        mx = max_nan(mx, s_x[r * (D + 1) + tid]);
      }
      float dl = fdiv(fsub(mx, mn), 15.0f);
      if (dl == 0.0f) dl = 1.0f;
      s_mn[tid] = mn; s_dl[tid] = dl;
      a.c.bounds[at * 2 * D + tid] = mn;
      a.c.bounds[at * 2 * D + D + tid] = dl;
    }
    __syncthreads();
    unsigned* K4 = reinterpret_cast<unsigned*>(a.c.K4 + at * kBlock * (D / 2));
    for (int i = tid; i < kBlock * D / 8; i += kKv4Threads) {
      const int r = i / (D / 8), c = (i - r * (D / 8)) * 8;
      unsigned w = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) w |= code4(s_x[r * (D + 1) + c + e], s_mn[c + e], s_dl[c + e]) << (4 * e);
      K4[i] = w;
    }
    __syncthreads();
    for (int i = tid; i < kBlock * D; i += kKv4Threads) {
      const int r = i / D, c = i - r * D;
      const int64_t p = p0 + r;
      s_x[r * (D + 1) + c] = Elem<E>::get(p < start ? Vt + r * D : vn + (p - start) * a.vs.t, c);
    }
    __syncthreads();
    // values: one (m, Delta) per token
    if (tid < kBlock) {
      float mn = INFINITY, mx = -INFINITY;
      for (int c = 0; c < D; ++c) {
        mn = min_nan(mn, s_x[tid * (D + 1) + c]);
        mx = max_nan(mx, s_x[tid * (D + 1) + c]);
      }
      const float dl = fdiv(fsub(mx, mn), 15.0f);
      s_mn[tid] = mn; s_dl[tid] = dl;
      reinterpret_cast<float2*>(a.c.vscale)[at * kBlock + tid] = make_float2(mn, dl);
    }
    __syncthreads();
    unsigned* V4 = reinterpret_cast<unsigned*>(a.c.V4 + at * D * (kBlock / 2));
    for (int i = tid; i < kBlock * D / 8; i += kKv4Threads) {
      const int c = i / (kBlock / 8), p = (i - c * (kBlock / 8)) * 8;
      unsigned w = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int t = v4_token(p + e);
        w |= code4(s_x[t * (D + 1) + c], s_mn[t], s_dl[t]) << (4 * e);   // (Delta = 0: 0/0, code 0)
      }
      V4[i] = w;
    }
    __syncthreads();
  }
  // the rows of the block that stays incomplete
  if (blk == blk0) {
    const int64_t p0 = max(start, whole * kBlock);
    for (int64_t i = tid; i < (n - p0) * D; i += kKv4Threads) {
      const int64_t p = p0 + i / D;
      const int c = (int)(i % D);
      Kt[(p % kBlock) * D + c] = kn[(p - start) * a.ks.t + c];
      Vt[(p % kBlock) * D + c] = vn[(p - start) * a.vs.t + c];
    }
  }
}

template <int D, typename E>
__global__ void __launch_bounds__(kKv4Threads) kv4_unpack_kernel(const Kv4UnpackArgs a) {
  pdl_entry();
  const int tid = threadIdx.x;
  const int g = blockIdx.y, b = blockIdx.z;
  if (a.status && blockIdx.x == 0 && g == 0 && b == 0 && tid < 32) {
    bool bad = false;
    for (int i = tid; i < a.B; i += 32) {
      const int64_t n = a.len[i], f = a.first ? a.first[i] : 0;
      bad |= n < 0 || n > a.n_max || f < 0;
    }
    report_range(a.status, bad);
  }
  const int64_t n = a.len[b], first = a.first ? a.first[b] : 0;
  if (n < 0 || n > a.n_max || first < 0 || first >= n) return;
  const int64_t end = n - first < a.rows ? n : first + a.rows;
  const int64_t blk = first / kBlock + blockIdx.x;
  const int64_t p0 = max(first, blk * kBlock), p1 = min(end, (blk + 1) * kBlock);
  if (p0 >= p1) return;
  const int64_t bg = (int64_t)b * a.Hkv + g;
  const int64_t at = bg * a.nblk_max + blk;
  const bool coded = blk < n / kBlock;
  E* Ko = reinterpret_cast<E*>(a.K) + bg * a.rows * D;
  E* Vo = reinterpret_cast<E*>(a.V) + bg * a.rows * D;
  const int count = (int)(p1 - p0) * D;
  for (int i = tid; i < count; i += kKv4Threads) {
    const int64_t p = p0 + i / D;
    const int r = (int)(p % kBlock), c = i % D;
    const int64_t out = (p - first) * D + c;
    if (!coded) {
      Ko[out] = reinterpret_cast<const E*>(a.c.Kt)[(bg * kBlock + r) * D + c];
      Vo[out] = reinterpret_cast<const E*>(a.c.Vt)[(bg * kBlock + r) * D + c];
      continue;
    }
    const unsigned kb = a.c.K4[(at * kBlock + r) * (D / 2) + c / 2];
    Ko[out] = to_elem<E>(value4((kb >> (4 * (c & 1))) & 15u, a.c.bounds[at * 2 * D + c], a.c.bounds[at * 2 * D + D + c]));
    const int pl = v4_place(r);
    const unsigned vb = a.c.V4[(at * D + c) * (kBlock / 2) + pl / 2];
    const float2 sc = reinterpret_cast<const float2*>(a.c.vscale)[at * kBlock + r];
    Vo[out] = to_elem<E>(value4((vb >> (4 * (pl & 1))) & 15u, sc.x, sc.y));
  }
}

namespace {

template <int D, typename E>
cudaError_t launch_append(const Kv4AppendArgs& a, dim3 grid, cudaStream_t st) {
  const int smem = (kBlock * (D + 1) + 2 * D) * 4;
  const cudaError_t e = cudaFuncSetAttribute(kv4_append_kernel<D, E>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  launch_pdl(kv4_append_kernel<D, E>, grid, dim3(kKv4Threads), smem, st, a);
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
         aligned16(c->V4) && aligned16(c->vscale) && aligned16(c->Kt) && aligned16(c->Vt);
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
