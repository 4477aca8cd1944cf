// Rows of keys and values on their way into a cache held in codes, and back:
// what the kernels for the different codes share.
#pragma once

#include "csa_args.cuh"

namespace csa {

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

// the status word of a call and the word that keeps refusals (either may be
// null): set by one warp of its first CTA
__device__ __forceinline__ void report_range(unsigned* status, unsigned* refused, bool bad) {
  const unsigned any = __any_sync(0xffffffffu, bad);
  if ((threadIdx.x & 31) == 0) {
    if (status) *status = any ? 8u : 0u;
    if (refused && any) *refused = 8u;
  }
}

// steps whose reciprocal and its products stay in the normal range
__device__ __forceinline__ bool step_plain(float step) { return step > 1e-30f && step < 1e30f; }
// 1 / x to one unit in the last place
__device__ __forceinline__ float approx_rcp(float x) {
  float r;
  asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

template <int CPL, typename E> struct Row {};      // CPL consecutive elements
template <> struct Row<4, __nv_bfloat16> { typedef uint2 T; };
template <> struct Row<2, __nv_bfloat16> { typedef unsigned T; };
template <> struct Row<4, float> { typedef float4 T; };
template <> struct Row<2, float> { typedef float2 T; };
template <int CPL>
__device__ __forceinline__ void row_floats(const typename Row<CPL, __nv_bfloat16>::T& r, float (&x)[CPL], __nv_bfloat16) {
  const unsigned* u = reinterpret_cast<const unsigned*>(&r);
#pragma unroll
  for (int c = 0; c < CPL; ++c) x[c] = __uint_as_float(c & 1 ? u[c / 2] & 0xFFFF0000u : u[c / 2] << 16);
}
template <int CPL>
__device__ __forceinline__ void row_floats(const typename Row<CPL, float>::T& r, float (&x)[CPL], float) {
  const float* f = reinterpret_cast<const float*>(&r);
#pragma unroll
  for (int c = 0; c < CPL; ++c) x[c] = f[c];
}

// element by element; bf16 in pairs, which loses nothing
__device__ __forceinline__ unsigned min2_nan(unsigned a, unsigned b) {
  unsigned r;
  asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ unsigned max2_nan(unsigned a, unsigned b) {
  unsigned r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
template <bool MAX> __device__ __forceinline__ float pick(float a, float b) { return MAX ? max_nan(a, b) : min_nan(a, b); }
template <bool MAX> __device__ __forceinline__ unsigned pick(unsigned a, unsigned b) { return MAX ? max2_nan(a, b) : min2_nan(a, b); }
template <bool MAX> __device__ __forceinline__ uint2 pick(uint2 a, uint2 b) { return make_uint2(pick<MAX>(a.x, b.x), pick<MAX>(a.y, b.y)); }
template <bool MAX> __device__ __forceinline__ float2 pick(float2 a, float2 b) { return make_float2(pick<MAX>(a.x, b.x), pick<MAX>(a.y, b.y)); }
template <bool MAX> __device__ __forceinline__ float4 pick(float4 a, float4 b) {
  return make_float4(pick<MAX>(a.x, b.x), pick<MAX>(a.y, b.y), pick<MAX>(a.z, b.z), pick<MAX>(a.w, b.w));
}

// eight channels of a row, rounded to its type
template <typename E>
__device__ __forceinline__ void store8(E* dst, const float (&x)[8]);
template <> __device__ __forceinline__ void store8<float>(float* dst, const float (&x)[8]) {
  reinterpret_cast<float4*>(dst)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4*>(dst)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
template <> __device__ __forceinline__ void store8<__nv_bfloat16>(__nv_bfloat16* dst, const float (&x)[8]) {
  unsigned u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    u[i] = *reinterpret_cast<const unsigned*>(&v);
  }
  *reinterpret_cast<uint4*>(dst) = make_uint4(u[0], u[1], u[2], u[3]);
}

}  // namespace csa
