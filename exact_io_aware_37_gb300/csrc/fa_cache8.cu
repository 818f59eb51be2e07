// Writing and reading the 8-bit key/value cache (format: fa_cache8.cuh).
//
// Both kernels move rows once and compute next to nothing, so HBM traffic
// bounds them.  A thread owns eight elements of one row (16 bytes of a 16-bit
// tensor, 8 codes); D / 8 neighbouring threads share a row and find its
// largest magnitude with xor shuffles.  Keys and values go through one launch.
#include <math.h>

#include "fa_cache8.cuh"
#include "fa_internal.cuh"

namespace fa {
namespace {

constexpr int kThreads = 256;
constexpr int kElems = 8;  // elements per thread

template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&x)[8]) {
  if constexpr (sizeof(T) == 4) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  } else {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float2 f;
      if constexpr (__is_same(T, __half))
        f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      else
        f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]));
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&x)[8]) {
  if constexpr (sizeof(T) == 4) {
    reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (__is_same(T, __half)) {
        const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
      } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
      }
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// Rows [start, start + count) of sequence b in the cache; count = -1 when they
// do not fit (reported by the caller, and the sequence skipped).
struct Range {
  int start, count;
};
__device__ __forceinline__ Range seq_rows(const CacheRows& a, int b) {
  Range r{a.start ? a.start[b] : 0, a.count ? a.count[b] : a.n};
  if (r.count < 0 || r.count > a.n || r.start < 0 || r.start > a.cap - r.count) r.count = -1;
  return r;
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) cache_write_kernel(const CacheRows a) {
  constexpr int kLanes = D / kElems;  // threads per row
  const long long t = (long long)blockIdx.x * kThreads + threadIdx.x;
  const uint32_t row = (uint32_t)(t / kLanes);  // over [B, H, n]
  if (row >= a.rows) return;                    // a row's threads leave together
  const int lane = threadIdx.x % kLanes;
  const uint32_t bh = row / (uint32_t)a.n;
  const int i = (int)(row - bh * (uint32_t)a.n);
  const Range r = seq_rows(a, (int)(bh / (uint32_t)a.H));
  if (r.count < 0 && lane == 0) atomicOr(a.status, kDevBadSeqlens);
  if (i >= r.count) return;  // so do a row's threads here
  const bool is_v = blockIdx.y != 0;
  float x[8];
  load8(static_cast<const T*>(is_v ? a.v : a.k) + (long long)row * D + lane * kElems, x);
  float amax = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) amax = fmaxf(amax, c8::finite_abs(x[e]));
  // the shuffle's mask is the row's own threads: other rows of the warp may have left
  const unsigned group = (kLanes == 16 ? 0xffffu : 0xffu) << ((threadIdx.x & 31) / kLanes * kLanes);
#pragma unroll
  for (int m = kLanes / 2; m >= 1; m >>= 1) amax = fmaxf(amax, __shfl_xor_sync(group, amax, m));
  const int eb = c8::exp_byte(amax);
  const float f = c8::inv_scale(eb);
  uint2 out;
  out.x = c8::encode2(x[0] * f, x[1] * f) | c8::encode2(x[2] * f, x[3] * f) << 16;
  out.y = c8::encode2(x[4] * f, x[5] * f) | c8::encode2(x[6] * f, x[7] * f) << 16;
  const long long dst = (long long)bh * a.cap + r.start + i;
  *reinterpret_cast<uint2*>((is_v ? a.v_codes : a.k_codes) + dst * D + lane * kElems) = out;
  if (lane == 0) (is_v ? a.v_exp : a.k_exp)[dst] = (uint8_t)eb;
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(const CacheRows a) {
  constexpr int kLanes = D / kElems;
  const long long t = (long long)blockIdx.x * kThreads + threadIdx.x;
  const uint32_t row = (uint32_t)(t / kLanes);
  if (row >= a.rows) return;
  const int lane = threadIdx.x % kLanes;
  const uint32_t bh = row / (uint32_t)a.n;
  const int i = (int)(row - bh * (uint32_t)a.n);
  const Range r = seq_rows(a, (int)(bh / (uint32_t)a.H));
  if (r.count < 0) {
    if (lane == 0) atomicOr(a.status, kDevBadSeqlens);
    return;
  }
  const bool is_v = blockIdx.y != 0;
  float x[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = 0.f;
  if (i < r.count) {
    const long long src = (long long)bh * a.cap + r.start + i;
    const uint2 u = *reinterpret_cast<const uint2*>((is_v ? a.v_codes : a.k_codes) + src * D + lane * kElems);
    const float f = c8::scale((is_v ? a.v_exp : a.k_exp)[src]);
    const uint32_t w[4] = {u.x, u.x >> 16, u.y, u.y >> 16};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 y = c8::decode2(w[e]);
      x[2 * e] = y.x * f;
      x[2 * e + 1] = y.y * f;
    }
  }
  store8(static_cast<T*>(const_cast<void*>(is_v ? a.v : a.k)) + (long long)row * D + lane * kElems, x);
}

template <typename T, int D>
cudaError_t launch_td(const CacheRows& a, bool write, cudaStream_t s) {
  const long long threads = (long long)a.rows * (D / kElems);
  const dim3 grid((unsigned)((threads + kThreads - 1) / kThreads), 2);
  if (write)
    cache_write_kernel<T, D><<<grid, kThreads, 0, s>>>(a);
  else
    cache_read_kernel<T, D><<<grid, kThreads, 0, s>>>(a);
  note_launches(1);
  return note_error(write ? "cache write launch" : "cache read launch", cudaGetLastError());
}

template <typename T>
cudaError_t launch_t(const CacheRows& a, int D, bool write, cudaStream_t s) {
  return D == 64 ? launch_td<T, 64>(a, write, s) : launch_td<T, 128>(a, write, s);
}

}  // namespace

cudaError_t launch_cache8(const CacheRows& a, int D, fa_dtype dt, bool write, cudaStream_t s) {
  if (dt == FA_F32) return launch_t<float>(a, D, write, s);
  if (dt == FA_F16) return launch_t<__half>(a, D, write, s);
  return launch_t<__nv_bfloat16>(a, D, write, s);
}

}  // namespace fa
