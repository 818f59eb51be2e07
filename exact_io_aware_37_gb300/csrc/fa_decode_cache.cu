// Decoding steps over a cache whose sequences have their own lengths, with
// grouped heads: fa_decode_cache (the 8-bit cache) and fa_decode_shared (a
// prefix that the whole batch shares, then each sequence's own rows, 16-bit or
// 8-bit).  Query head h reads key head h / (H / Hk); row i of the nq new
// queries sits at position total - nq + i of its sequence's total = np + len
// keys, so causal allows key j iff j <= i + total - nq.
//
// As in fa_decode.cu the keys of a (sequence, key head) are split across CTAs,
// each keeps the running state (m, l, u) of its rows, and a second kernel
// joins the states: m = max m_s, l = sum l_s 2^(m_s - m), u = sum u_s 2^(m_s - m).
#include <math.h>

#include "fa_cache8.cuh"
#include "fa_internal.cuh"

namespace fa {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kG = 8;  // query rows per CTA

// Factor of a state with maximum m joined under the maximum mm >= m: 1 for
// equal maxima, -inf among them (that state holds nothing, or only NaN).
__device__ __forceinline__ float join_factor(float m, float mm) { return m == mm ? 1.f : exp2f(m - mm); }

template <typename T, int E>
__device__ __forceinline__ void load_row(const T* p, float (&x)[E]) {
#pragma unroll
  for (int e = 0; e < E; ++e) x[e] = ld_elem(p, e);
}
template <int E>
__device__ __forceinline__ void load_codes(const uint8_t* p, float f, float (&x)[E]) {
#pragma unroll
  for (int e = 0; e < E; e += 2) {
    const float2 y = c8::decode2(*reinterpret_cast<const uint16_t*>(p + e));
    x[e] = y.x * f;
    x[e + 1] = y.y * f;
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) serve_split_kernel(const ServeArgs a) {
  constexpr int E = D / 32;
  __shared__ float s_m[kWarps][kG], s_l[kWarps][kG];
  __shared__ float s_u[kWarps][kG][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int split = blockIdx.x % a.splits, g0 = (blockIdx.x / a.splits) * kG;
  const int hk = blockIdx.y, b = blockIdx.z;
  const int rows = a.group * a.nq;
  const int len = a.lens ? a.lens[b] : a.max_len;
  if (len < 0 || len > a.max_len) {
    if (threadIdx.x == 0) atomicOr(a.status, kDevBadSeqlens);
    return;
  }
  const int total = a.np + len;
  const long long k0 = (long long)split * a.keys_per_split, k1 = min((long long)total, k0 + a.keys_per_split);
  const long long bh = (long long)b * a.Hk + hk;
  const T* q = static_cast<const T*>(a.q) + (bh * rows + g0) * D;

  float qv[kG][E], m[kG], l[kG], u[kG][E];
  int last[kG];
#pragma unroll
  for (int g = 0; g < kG; ++g) {
    m[g] = -INFINITY;
    l[g] = 0.f;
    last[g] = g0 + g < rows ? (a.causal ? total - a.nq + (g0 + g) % a.nq : total - 1) : -1;
#pragma unroll
    for (int e = 0; e < E; ++e) qv[g][e] = u[g][e] = 0.f;
    if (g0 + g < rows) load_row<T, E>(q + (long long)g * D + lane * E, qv[g]);
#pragma unroll
    for (int e = 0; e < E; ++e) qv[g][e] *= a.c2;
  }
  for (long long j = k0 + warp; j < k1; j += kWarps) {
    float kr[E], vr[E];
    if (j < a.np) {
      const long long r = (long long)hk * a.np + j;
      load_row<T, E>(static_cast<const T*>(a.kp) + r * D + lane * E, kr);
      load_row<T, E>(static_cast<const T*>(a.vp) + r * D + lane * E, vr);
    } else {
      const long long r = bh * a.cap + (j - a.np);
      if (a.k_exp) {
        load_codes<E>(static_cast<const uint8_t*>(a.k) + r * D + lane * E, c8::scale(a.k_exp[r]), kr);
        load_codes<E>(static_cast<const uint8_t*>(a.v) + r * D + lane * E, c8::scale(a.v_exp[r]), vr);
      } else {
        load_row<T, E>(static_cast<const T*>(a.k) + r * D + lane * E, kr);
        load_row<T, E>(static_cast<const T*>(a.v) + r * D + lane * E, vr);
      }
    }
#pragma unroll
    for (int g = 0; g < kG; ++g) {
      if (j > last[g]) continue;
      float s = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) s = fmaf(qv[g][e], kr[e], s);
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
      const float m_new = fmaxf(m[g], s), ref = m_new == -INFINITY ? 0.f : m_new;  // a score of -inf weighs nothing
      const float alpha = exp2f(m[g] - ref), p = exp2f(s - ref);
      l[g] = l[g] * alpha + p;
#pragma unroll
      for (int e = 0; e < E; ++e) u[g][e] = u[g][e] * alpha + p * vr[e];
      m[g] = m_new;
    }
  }
#pragma unroll
  for (int g = 0; g < kG; ++g) {
    if (lane == 0) {
      s_m[warp][g] = m[g];
      s_l[warp][g] = l[g];
    }
#pragma unroll
    for (int e = 0; e < E; ++e) s_u[warp][g][lane * E + e] = u[g][e];
  }
  __syncthreads();
  for (int idx = threadIdx.x; idx < min(kG, rows - g0) * D; idx += kThreads) {
    const int g = idx / D, d = idx % D;
    float mm = -INFINITY, ll = 0.f, uu = 0.f;
    for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, s_m[w][g]);
    for (int w = 0; w < kWarps; ++w) {
      const float f = join_factor(s_m[w][g], mm);
      ll += s_l[w][g] * f;
      uu += s_u[w][g][d] * f;
    }
    const long long row = (split * (long long)a.B * a.Hk + bh) * rows + g0 + g;
    a.part_u[row * D + d] = uu;
    if (d == 0) {
      a.part_ml[row * 2] = mm;
      a.part_ml[row * 2 + 1] = ll;
    }
  }
}

template <typename T>
__global__ void serve_merge_kernel(const ServeArgs a, int D) {
  const long long row = blockIdx.x, rows = (long long)a.B * a.Hk * a.group * a.nq;
  const int len = a.lens ? a.lens[row / ((long long)a.Hk * a.group * a.nq)] : a.max_len;
  if (len < 0 || len > a.max_len) return;
  const int splits = min(a.splits, (a.np + len + a.keys_per_split - 1) / a.keys_per_split);
  float mm = -INFINITY, ll = 0.f, uu = 0.f;
  for (int s = 0; s < splits; ++s) mm = fmaxf(mm, a.part_ml[(s * rows + row) * 2]);
  for (int s = 0; s < splits; ++s) {
    const long long r = s * rows + row;
    const float f = join_factor(a.part_ml[r * 2], mm);
    ll += a.part_ml[r * 2 + 1] * f;
    uu += a.part_u[r * D + threadIdx.x] * f;
  }
  st_elem(static_cast<T*>(a.o), row * D + threadIdx.x, ll == 0.f ? 0.f : uu / ll);  // l = 0: no key; NaN goes through
  if (threadIdx.x == 0) a.lse[row] = ll == 0.f ? -INFINITY : (mm + log2f(ll)) * kLn2;
}

template <typename T>
cudaError_t launch_t(const ServeArgs& a, int D, cudaStream_t s) {
  const int groups = (a.group * a.nq + kG - 1) / kG;
  const dim3 grid((unsigned)(a.splits * groups), a.Hk, a.B);
  if (D == 64)
    serve_split_kernel<T, 64><<<grid, kThreads, 0, s>>>(a);
  else
    serve_split_kernel<T, 128><<<grid, kThreads, 0, s>>>(a);
  note_launches(1);
  cudaError_t e = note_error("cached decoding launch", cudaGetLastError());
  if (e != cudaSuccess) return e;
  serve_merge_kernel<T><<<(unsigned)((long long)a.B * a.Hk * a.group * a.nq), D, 0, s>>>(a, D);
  note_launches(1);
  return note_error("cached decoding merge launch", cudaGetLastError());
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

DecodeSplit serve_split(int B, int Hk, long long keys) {
  // about 1024 CTAs, no split shorter than 256 keys
  long long want = (1024 + (long long)B * Hk - 1) / ((long long)B * Hk);
  const long long most = (keys + 255) / 256;
  if (want > most) want = most;
  if (want < 1) want = 1;
  DecodeSplit sp;
  sp.keys_per_split = (int)((keys + want - 1) / want);
  if (sp.keys_per_split < 1) sp.keys_per_split = 1;
  sp.splits = (int)((keys + sp.keys_per_split - 1) / sp.keys_per_split);
  if (sp.splits < 1) sp.splits = 1;
  return sp;
}

}  // namespace

size_t serve_workspace_bytes(int B, int H, int Hk, int nq, int np, int max_len, int D) {
  const DecodeSplit sp = serve_split(B, Hk, (long long)np + max_len);
  const size_t rows = (size_t)sp.splits * B * H * nq;
  return up256(rows * D * sizeof(float)) + up256(rows * 2 * sizeof(float));
}

cudaError_t launch_serve(ServeArgs& a, int D, fa_dtype dt, void* workspace, cudaStream_t s) {
  const DecodeSplit sp = serve_split(a.B, a.Hk, (long long)a.np + a.max_len);
  a.splits = sp.splits;
  a.keys_per_split = sp.keys_per_split;
  const size_t rows = (size_t)sp.splits * a.B * a.Hk * a.group * a.nq;
  a.part_u = static_cast<float*>(workspace);
  a.part_ml = reinterpret_cast<float*>(static_cast<char*>(workspace) + up256(rows * D * sizeof(float)));
  return dt == FA_F16 ? launch_t<__half>(a, D, s) : launch_t<__nv_bfloat16>(a, D, s);
}

}  // namespace fa
