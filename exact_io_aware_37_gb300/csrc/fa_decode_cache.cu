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
#include "fa_serve.cuh"
#include "ptx.cuh"

namespace fa {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kG = 8;  // query rows per CTA

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

// Joins the states of every query row: a warp a row.
constexpr int kMergeWarps = 8;

struct MergeParams {
  ServeArgs a;
  int tile, tile_rows, row_groups;  // of the pass over the own rows
};

template <typename T, int D>
__global__ void __launch_bounds__(kMergeWarps * 32) merge_kernel(const __grid_constant__ MergeParams p) {
  constexpr int E = D / 32;
  const ServeArgs& a = p.a;
  const int lane = threadIdx.x & 31;
  const int rows = a.group * a.nq;
  const long long row = (long long)blockIdx.x * kMergeWarps + (threadIdx.x >> 5);
  if (row >= (long long)a.B * a.Hk * rows) return;
  const long long slab = row / rows;
  const int r = (int)(row - slab * rows), b = (int)(slab / a.Hk), hk = (int)(slab - (long long)b * a.Hk);
  const int len = raw_len(a, b);
  if (!len_ok(a, len)) return;
  ptx::grid_wait();
  float m = -INFINITY, mu = -INFINITY, l = 0.f, u[E];
#pragma unroll
  for (int e = 0; e < E; ++e) u[e] = 0.f;
  auto join = [&](const float* pu, const float4* pml) {
    const float4 s = *pml;
    const float m_new = fmaxf(m, s.x), mu_new = fmaxf(mu, s.z);
    l = l * join_factor(m, m_new) + s.y * join_factor(s.x, m_new);
    const float f = join_factor(mu, mu_new), g = join_factor(s.z, mu_new);
#pragma unroll
    for (int e = 0; e < E; ++e) u[e] = u[e] * f + pu[lane * E + e] * g;
    m = m_new;
    mu = mu_new;
  };
  const int nt = own_tiles(len, p.tile);
  if (nt > 0) {
    const int rg = r / p.tile_rows;
    const long long per = a.plan[0];
    const long long t0 = a.plan[1 + b] + ((long long)hk * p.row_groups + rg) * nt;
    const long long c0 = t0 / per, c1 = (t0 + nt - 1) / per;
    if (c0 == c1) {
      join(a.row_u + row * D, a.row_ml + row);
    } else {
      for (long long c = c0; c <= c1; ++c) {
        const long long at = (c * 2 + (c == c0 ? 1 : 0)) * p.tile_rows + (r - rg * p.tile_rows);
        join(a.cut_u + at * D, a.cut_ml + at);
      }
    }
  }
  // l = 0: no key; NaN goes through
  const float f = l == 0.f ? 0.f : exp2f(mu - m);
#pragma unroll
  for (int e = 0; e < E; ++e) st_elem(static_cast<T*>(a.o), row * D + lane * E + e, l == 0.f ? 0.f : u[e] / l * f);
  if (lane == 0) a.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

template <typename T>
cudaError_t launch_merge(const MergeParams& p, int D, cudaStream_t s) {
  const long long rows = (long long)p.a.B * p.a.Hk * p.a.group * p.a.nq;
  const int ctas = (int)((rows + kMergeWarps - 1) / kMergeWarps);
  return note_error("cached decoding merge launch",
                    launch_serve_kernel(D == 64 ? merge_kernel<T, 64> : merge_kernel<T, 128>, ctas, kMergeWarps * 32, 0,
                                        true, s, p));
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

namespace {

// Carves the workspace from `base`; returns the bytes taken.
size_t carve(ServeArgs& a, int D, char* base) {
  size_t at = 0;
  auto take = [&](size_t bytes) {
    char* p = base + at;
    at += up256(bytes);
    return p;
  };
  const size_t rows = (size_t)a.B * a.Hk * a.group * a.nq;
  const size_t cut = (size_t)kOwnCtas * 2 * 16 * own_row_tiles(a.group * a.nq);
  a.plan = reinterpret_cast<long long*>(take((size_t)(a.B + 1) * sizeof(long long)));
  a.row_u = reinterpret_cast<float*>(take(rows * D * sizeof(float)));
  a.row_ml = reinterpret_cast<float4*>(take(rows * sizeof(float4)));
  a.cut_u = reinterpret_cast<float*>(take(cut * D * sizeof(float)));
  a.cut_ml = reinterpret_cast<float4*>(take(cut * sizeof(float4)));
  return at;
}

}  // namespace

size_t serve_workspace_bytes(int B, int H, int Hk, int nq, int np, int max_len, int D) {
  if (np > 0) {
    const DecodeSplit sp = serve_split(B, Hk, (long long)np + max_len);
    const size_t rows = (size_t)sp.splits * B * H * nq;
    return up256(rows * D * sizeof(float)) + up256(rows * 2 * sizeof(float));
  }
  ServeArgs a{};
  a.B = B;
  a.Hk = Hk;
  a.group = H / Hk;
  a.nq = nq;
  return carve(a, D, nullptr);
}

cudaError_t launch_serve(ServeArgs& a, int D, fa_dtype dt, void* workspace, cudaStream_t s) {
  if (a.np > 0) {
    const DecodeSplit sp = serve_split(a.B, a.Hk, (long long)a.np + a.max_len);
    a.splits = sp.splits;
    a.keys_per_split = sp.keys_per_split;
    const size_t rows = (size_t)sp.splits * a.B * a.Hk * a.group * a.nq;
    a.part_u = static_cast<float*>(workspace);
    a.part_ml = reinterpret_cast<float*>(static_cast<char*>(workspace) + up256(rows * D * sizeof(float)));
    return dt == FA_F16 ? launch_t<__half>(a, D, s) : launch_t<__nv_bfloat16>(a, D, s);
  }
  carve(a, D, static_cast<char*>(workspace));
  const int wr = own_row_tiles(a.group * a.nq);
  MergeParams m;
  m.tile = own_stage_keys(a.k_exp ? D : 2 * D) * (4 / wr);
  m.tile_rows = 16 * wr;
  m.row_groups = (a.group * a.nq + m.tile_rows - 1) / m.tile_rows;
  if (a.max_len > 0) {
    const cudaError_t e = a.k_exp ? launch_own_e4m3(a, D, dt == FA_F16, false, s) : launch_own_16(a, D, dt == FA_F16, false, s);
    if (e != cudaSuccess) return e;
  }
  m.a = a;
  return dt == FA_F16 ? launch_merge<__half>(m, D, s) : launch_merge<__nv_bfloat16>(m, D, s);
}

}  // namespace fa
