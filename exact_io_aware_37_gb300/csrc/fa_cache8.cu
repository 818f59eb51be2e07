// Writing and reading the 8-bit key/value cache (format: fa_cache8.cuh).
//
// Both kernels move rows once and compute next to nothing, so HBM traffic
// bounds them: 4096 new rows of B2 H32 D128 bf16 are written in 30.4 us (6.6 TB/s), 8192 rows of B4 read
// back in 118 us (6.9 TB/s).  D / 16 neighbouring threads share a row, sixteen elements each in
// pieces of 16 bytes of the dense tensor, piece p of lane x at (p D / 16 + x) pieces, so that every access of
// a warp covers whole rows; a write finds the row's largest magnitude with xor shuffles.
// A thread has kRows rows in flight at once, its loads ahead of the look-up of where they go.
// Keys and values go through one launch.
#include <math.h>

#include <type_traits>

#include "fa_cache8.cuh"
#include "fa_internal.cuh"

namespace fa {
namespace {

constexpr int kThreads = 256;

// n / d by multiplication, exact for n < 2^31 (m = ceil(2^p / d) with 2^(p - 31) >= d).
struct FastDiv {
  uint32_t d, m;
  int p;
  explicit FastDiv(uint32_t d_) : d(d_) {
    int log = 0;
    while ((1ull << log) < d) ++log;
    p = 31 + log;
    m = (uint32_t)(((1ull << p) + d - 1) / d);
  }
  __device__ __forceinline__ uint32_t operator()(uint32_t n) const { return (uint32_t)(((uint64_t)n * m) >> p); }
};

struct Params {
  CacheRows a;
  FastDiv by_n, by_h;
};

template <typename T, int D>
struct Rows {
  static constexpr int kLanes = D / 16;           // threads of a row
  static constexpr int kPiece = 16 / sizeof(T);   // elements of 16 bytes
  static constexpr int kPieces = 16 / kPiece;
  static constexpr int kRows = sizeof(T) == 4 ? 2 : 4;  // rows of a thread
  static constexpr int kBlockRows = kThreads / kLanes * kRows;
};

template <typename T>
__device__ __forceinline__ void unpack(const uint4& u, float (&x)[16 / sizeof(T)]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (std::is_same<T, float>::value) {
      x[i] = __uint_as_float(w[i]);
    } else {
      float2 f;
      if constexpr (std::is_same<T, __half>::value)
        f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      else
        f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]));
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
}
template <typename T>
__device__ __forceinline__ uint4 pack(const float (&x)[16 / sizeof(T)]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (std::is_same<T, float>::value) {
      w[i] = __float_as_uint(x[i]);
    } else if constexpr (std::is_same<T, __half>::value) {
      const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    } else {
      const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Where dense row `row` lies in the cache: its row number there, -1 past the
// sequence's count, -2 for a sequence whose range does not fit (reported).
__device__ __forceinline__ long long cache_row(const Params& p, uint32_t row) {
  const CacheRows& a = p.a;
  const uint32_t bh = p.by_n(row), b = p.by_h(bh);
  const int i = (int)(row - bh * p.by_n.d);
  const int start = a.start ? __ldg(a.start + b) : 0, count = a.count ? __ldg(a.count + b) : a.n;
  if (count < 0 || count > a.n || start < 0 || start > a.cap - count) {
    atomicOr(a.status, kDevBadSeqlens);
    return -2;
  }
  return i < count ? (long long)bh * a.cap + start + i : -1;
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) cache_write_kernel(const Params p) {
  using R = Rows<T, D>;
  const CacheRows& a = p.a;
  const bool is_v = blockIdx.y != 0;
  const int lane = threadIdx.x % R::kLanes;
  const uint32_t row0 = blockIdx.x * R::kBlockRows + threadIdx.x / R::kLanes;  // then every kThreads / kLanes-th
  const T* src = static_cast<const T*>(is_v ? a.v : a.k);
  uint4 u[R::kRows][R::kPieces];
#pragma unroll
  for (int r = 0; r < R::kRows; ++r) {
    const uint32_t row = row0 + r * (kThreads / R::kLanes);
    if (row < a.rows)
#pragma unroll
      for (int i = 0; i < R::kPieces; ++i)
        u[r][i] = __ldcs(reinterpret_cast<const uint4*>(src + (long long)row * D) + i * R::kLanes + lane);
  }
#pragma unroll
  for (int r = 0; r < R::kRows; ++r) {
    const uint32_t row = row0 + r * (kThreads / R::kLanes);
    if (row >= a.rows) return;  // a row's threads leave together, and so they do below
    const long long dst = cache_row(p, row);
    if (dst < 0) continue;
    float x[R::kPieces][R::kPiece], amax = 0.f;
#pragma unroll
    for (int i = 0; i < R::kPieces; ++i) {
      unpack<T>(u[r][i], x[i]);
#pragma unroll
      for (int e = 0; e < R::kPiece; ++e) amax = fmaxf(amax, fabsf(x[i][e]));  // (NaN counts as nothing)
    }
    // the shuffle's mask is the row's own threads: other rows of the warp may have left
    const unsigned group = ((1u << R::kLanes) - 1) << ((threadIdx.x & 31) / R::kLanes * R::kLanes);
#pragma unroll
    for (int m = R::kLanes / 2; m >= 1; m >>= 1) amax = fmaxf(amax, __shfl_xor_sync(group, amax, m));
    // Infinities count as nothing too, and the conversion, which would saturate them, is to see NaN: mended where a
    // row holds one.  (A test of every element made the ALU the bound: 35.7 us, and 30.4 without, for 4096 new rows of B2
    // H32 D128 bf16.)
    if (amax == INFINITY) {
      amax = 0.f;
#pragma unroll
      for (int i = 0; i < R::kPieces; ++i)
#pragma unroll
        for (int e = 0; e < R::kPiece; ++e) {
          if (fabsf(x[i][e]) == INFINITY) x[i][e] = __uint_as_float(0x7fffffffu);
          amax = fmaxf(amax, fabsf(x[i][e]));
        }
#pragma unroll
      for (int m = R::kLanes / 2; m >= 1; m >>= 1) amax = fmaxf(amax, __shfl_xor_sync(group, amax, m));
    }
    const int eb = c8::exp_byte(amax);
    const float f = c8::inv_scale(eb);
    uint8_t* codes = (is_v ? a.v_codes : a.k_codes) + dst * D;
#pragma unroll
    for (int i = 0; i < R::kPieces; ++i) {
      uint32_t w[R::kPiece / 4];
#pragma unroll
      for (int e = 0; e < R::kPiece; e += 4)
        w[e / 4] = c8::encode2(x[i][e] * f, x[i][e + 1] * f) | c8::encode2(x[i][e + 2] * f, x[i][e + 3] * f) << 16;
      if constexpr (R::kPiece == 8)
        reinterpret_cast<uint2*>(codes)[i * R::kLanes + lane] = make_uint2(w[0], w[1]);
      else
        reinterpret_cast<uint32_t*>(codes)[i * R::kLanes + lane] = w[0];
    }
    if (lane == 0) (is_v ? a.v_exp : a.k_exp)[dst] = (uint8_t)eb;
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(const Params p) {
  using R = Rows<T, D>;
  const CacheRows& a = p.a;
  const bool is_v = blockIdx.y != 0;
  const int lane = threadIdx.x % R::kLanes;
  const uint32_t row0 = blockIdx.x * R::kBlockRows + threadIdx.x / R::kLanes;
  T* out = static_cast<T*>(const_cast<void*>(is_v ? a.v : a.k));
  const uint8_t* codes = is_v ? a.v_codes : a.k_codes;
  const uint8_t* exps = is_v ? a.v_exp : a.k_exp;
  uint32_t w[R::kRows][R::kPieces][R::kPiece / 4];
  int eb[R::kRows];
  long long src[R::kRows];
#pragma unroll
  for (int r = 0; r < R::kRows; ++r) {
    const uint32_t row = row0 + r * (kThreads / R::kLanes);
    src[r] = row < a.rows ? cache_row(p, row) : -2;
    eb[r] = 0;
#pragma unroll
    for (int i = 0; i < R::kPieces; ++i) {
#pragma unroll
      for (int e = 0; e < R::kPiece / 4; ++e) w[r][i][e] = 0;  // rows past the count: zeros
      if (src[r] >= 0) {
        if constexpr (R::kPiece == 8) {
          const uint2 y = __ldcs(reinterpret_cast<const uint2*>(codes + src[r] * D) + i * R::kLanes + lane);
          w[r][i][0] = y.x;
          w[r][i][1] = y.y;
        } else {
          w[r][i][0] = __ldcs(reinterpret_cast<const uint32_t*>(codes + src[r] * D) + i * R::kLanes + lane);
        }
      }
    }
    if (src[r] >= 0) eb[r] = exps[src[r]];
  }
#pragma unroll
  for (int r = 0; r < R::kRows; ++r) {
    if (src[r] == -2) continue;
    const uint32_t row = row0 + r * (kThreads / R::kLanes);
    const float f = c8::scale(eb[r]);
#pragma unroll
    for (int i = 0; i < R::kPieces; ++i) {
      float x[R::kPiece];
#pragma unroll
      for (int e = 0; e < R::kPiece; e += 2) {
        const float2 y = c8::decode2(w[r][i][e / 4] >> (e & 2) * 8);
        x[e] = y.x * f;
        x[e + 1] = y.y * f;
      }
      reinterpret_cast<uint4*>(out + (long long)row * D)[i * R::kLanes + lane] = pack<T>(x);
    }
  }
}

template <typename T, int D>
cudaError_t launch_td(const CacheRows& a, bool write, cudaStream_t s) {
  const Params p{a, FastDiv((uint32_t)a.n), FastDiv((uint32_t)a.H)};
  const dim3 grid((a.rows + Rows<T, D>::kBlockRows - 1) / Rows<T, D>::kBlockRows, 2);
  if (write)
    cache_write_kernel<T, D><<<grid, kThreads, 0, s>>>(p);
  else
    cache_read_kernel<T, D><<<grid, kThreads, 0, s>>>(p);
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
