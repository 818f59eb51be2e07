// Decoding steps over a cache whose sequences have their own lengths, with
// grouped heads: fa_decode_cache (the 8-bit cache) and fa_decode_shared (a
// prefix that the whole batch shares, then each sequence's own rows, 16-bit or
// 8-bit).  Query head h reads key head h / (H / Hk); row i of the nq new
// queries sits at position total - nq + i of its sequence's total = np + len
// keys, so causal allows key j iff j <= i + total - nq.
//
// A step is up to three launches: the pass over the prefix (fa_tc_prefix.cu), the
// pass over the own rows (fa_serve_own.cuh), and the join of the states they
// leave, here: m = max m_s, l = sum l_s 2^(m_s - m), u = sum u_s 2^(mu_s - mu),
// O = u 2^(mu - m) / l, L = (m + log2 l) ln 2.  Each launch may start while the one
// in front of it drains.
#include <math.h>

#include <type_traits>

#include "fa_internal.cuh"
#include "fa_serve.cuh"
#include "ptx.cuh"

namespace fa {
namespace {

// Joins the states of every query row: a warp a row.
constexpr int kMergeWarps = 8;

struct MergeParams {
  ServeArgs a;
  int cta_rows, row_groups;  // of the pass over the own rows
  PrefixPlan pre;
};

// E (2 or 4) elements, rounded once, in one store.
template <int E, typename T>
__device__ __forceinline__ void store_row(T* p, const float (&x)[E]) {
  uint32_t w[E / 2];
#pragma unroll
  for (int i = 0; i < E / 2; ++i) w[i] = ptx::pack16x2<std::is_same<T, __half>::value>(x[2 * i], x[2 * i + 1]);
  if constexpr (E == 4)
    *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  else
    *reinterpret_cast<uint32_t*>(p) = w[0];
}

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
  // ---- where the row's states are: n_pre of the prefix, then n_own of the own rows
  const long long x = (long long)b * rows + r;  // row of the key head
  const int unit = hk * p.pre.pairs + (int)(x / (2 * kPrefixRows)), slots = p.pre.split ? 2 : 1;
  long long pre_at = 0;
  int n_pre = 0, n_own = 0;
  if (a.np > 0) {
    const int c0 = (int)((long long)unit * p.pre.steps / p.pre.per_cta);
    const int c1 = (int)(((long long)(unit + 1) * p.pre.steps - 1) / p.pre.per_cta);
    pre_at = ((long long)unit * p.pre.parts * 2 + ((int)(x / kPrefixRows) & 1)) * kPrefixRows + x % kPrefixRows;
    n_pre = (c1 - c0 + 1) * slots;
  }
  const int nt = own_tiles(len), rg = r / p.cta_rows;
  long long c0 = 0;
  if (nt > 0) {
    const long long per = a.plan[0];
    const long long t0 = a.plan[1 + b] + ((long long)hk * p.row_groups + rg) * own_cost(nt) + kRunCost;
    c0 = t0 / per;
    n_own = (int)((t0 + nt - 1) / per - c0) + 1;
  }
  const bool whole = n_own == 1;
  auto state = [&](int i, const float*& u) -> const float4* {
    if (i < n_pre) {
      // part i / slots of the unit; with halved keys both slots hold the row
      const long long at = pre_at + ((long long)(i / slots) * 2 + i % slots) * kPrefixRows;
      u = a.pre_u + at * D;
      return a.pre_ml + at;
    }
    if (whole) {
      u = a.row_u + row * D;
      return a.row_ml + row;
    }
    const int c = i - n_pre;
    const long long at = ((c0 + c) * 2 + (c == 0 ? 1 : 0)) * p.cta_rows + (r - rg * p.cta_rows);
    u = a.cut_u + at * D;
    return a.cut_ml + at;
  };

  // ---- 32 states at a time: a lane finds one state's share, then all lanes add the rows up
  using Vec = typename std::conditional<E == 4, float4, float2>::type;
  float m = -INFINITY, mu = -INFINITY, l = 0.f, u[E];
#pragma unroll
  for (int e = 0; e < E; ++e) u[e] = 0.f;
  const int n = n_pre + n_own;
  for (int i0 = 0; i0 < n; i0 += 32) {
    const float* pu = nullptr;
    float4 s = make_float4(-INFINITY, 0.f, -INFINITY, 0.f);
    if (i0 + lane < n) s = *state(i0 + lane, pu);
    const bool some = s.y != 0.f;  // a state without a key may not even have its u; NaN is not 0
    const float m_new = fmaxf(m, ptx::warp_max(some ? s.x : -INFINITY));
    const float mu_new = fmaxf(mu, ptx::warp_max(some ? s.z : -INFINITY));
    float share = some ? s.y * join_factor(s.x, m_new) : 0.f;
    const float g = join_factor(s.z, mu_new);
#pragma unroll
    for (int x = 16; x >= 1; x >>= 1) share += __shfl_xor_sync(0xffffffffu, share, x);
    l = l * join_factor(m, m_new) + share;
    const float f = join_factor(mu, mu_new);
#pragma unroll
    for (int e = 0; e < E; ++e) u[e] *= f;
    m = m_new;
    mu = mu_new;
    unsigned todo = __ballot_sync(0xffffffffu, some);
    while (todo) {
      constexpr int kTogether = 4;  // rows read before the first is used
      Vec v[kTogether];
      float w[kTogether];
#pragma unroll
      for (int k = 0; k < kTogether; ++k) {
        const int i = todo ? __ffs(todo) - 1 : 0;
        w[k] = __shfl_sync(0xffffffffu, g, i);
        const float* at = reinterpret_cast<const float*>(
            __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(pu), i));
        if (todo)
          v[k] = reinterpret_cast<const Vec*>(at)[lane];
        else
          w[k] = 0.f, v[k] = Vec{};
        todo &= todo - 1;
      }
#pragma unroll
      for (int k = 0; k < kTogether; ++k) {
        const float* y = reinterpret_cast<const float*>(&v[k]);
#pragma unroll
        for (int e = 0; e < E; ++e) u[e] = fmaf(y[e], w[k], u[e]);
      }
    }
  }
  // l = 0: no key; NaN goes through
  const float f = l == 0.f ? 0.f : exp2f(mu - m);
#pragma unroll
  for (int e = 0; e < E; ++e) u[e] = l == 0.f ? 0.f : u[e] / l * f;
  store_row<E>(static_cast<T*>(a.o) + row * D + lane * E, u);
  if (lane == 0) a.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

template <typename T>
cudaError_t launch_merge(const MergeParams& p, int D, cudaStream_t s) {
  const long long rows = (long long)p.a.B * p.a.Hk * p.a.group * p.a.nq;
  const int ctas = (int)((rows + kMergeWarps - 1) / kMergeWarps);
  return note_error("cached decoding merge launch",
                    launch_serve_kernel(D == 64 ? merge_kernel<T, 64> : merge_kernel<T, 128>, ctas, kMergeWarps * 32, 0,
                                        p.a.np > 0 || p.a.max_len > 0, s, p));
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

// Carves the workspace from `base`; returns the bytes taken.
size_t carve(ServeArgs& a, int D, const PrefixPlan& pre, char* base) {
  size_t at = 0;
  auto take = [&](size_t bytes) {
    char* p = base + at;
    at += up256(bytes);
    return p;
  };
  const size_t rows = (size_t)a.B * a.Hk * a.group * a.nq;
  const size_t cut = (size_t)kOwnCtas * 2 * own_rows(a.group * a.nq);
  if (a.np > 0) {
    const size_t states = (size_t)pre.units * pre.parts * 2 * kPrefixRows;
    a.pre_u = reinterpret_cast<float*>(take(states * D * sizeof(float)));
    a.pre_ml = reinterpret_cast<float4*>(take(states * sizeof(float4)));
  }
  if (a.max_len == 0) return at;
  a.plan = reinterpret_cast<long long*>(take((size_t)(a.B + 1) * sizeof(long long)));
  a.row_u = reinterpret_cast<float*>(take(rows * D * sizeof(float)));
  a.row_ml = reinterpret_cast<float4*>(take(rows * sizeof(float4)));
  a.cut_u = reinterpret_cast<float*>(take(cut * D * sizeof(float)));
  a.cut_ml = reinterpret_cast<float4*>(take(cut * sizeof(float4)));
  return at;
}

}  // namespace

size_t serve_workspace_bytes(int B, int H, int Hk, int nq, int np, int max_len, int D) {
  ServeArgs a{};
  a.B = B;
  a.Hk = Hk;
  a.group = H / Hk;
  a.nq = nq;
  a.np = np;
  a.max_len = max_len;
  return carve(a, D, prefix_plan(B, Hk, a.group * nq, np), nullptr);
}

cudaError_t launch_serve(ServeArgs& a, int D, fa_dtype dt, void* workspace, cudaStream_t s) {
  const bool f16 = dt == FA_F16;
  MergeParams m;
  m.cta_rows = own_rows(a.group * a.nq);
  m.row_groups = (a.group * a.nq + m.cta_rows - 1) / m.cta_rows;
  m.pre = prefix_plan(a.B, a.Hk, a.group * a.nq, a.np);
  carve(a, D, m.pre, static_cast<char*>(workspace));
  cudaError_t e = cudaSuccess;
  if (a.np > 0) e = launch_prefix(a, m.pre, D, f16, s);
  if (e == cudaSuccess && a.max_len > 0)
    e = a.k_exp ? launch_own_e4m3(a, D, f16, a.np > 0, s) : launch_own_16(a, D, f16, a.np > 0, s);
  if (e != cudaSuccess) return e;
  m.a = a;
  return f16 ? launch_merge<__half>(m, D, s) : launch_merge<__nv_bfloat16>(m, D, s);
}

}  // namespace fa
