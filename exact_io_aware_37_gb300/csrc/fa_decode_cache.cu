// Decoding steps over a cache whose sequences have their own lengths, with
// grouped heads: fa_decode_cache (the 8-bit cache) and fa_decode_shared (a
// prefix that the whole batch shares, then each sequence's own rows, 16-bit or
// 8-bit).  Query head h reads key head h / (H / Hk); row i of the nq new
// queries sits at position total - nq + i of its sequence's total = np + len
// keys, so causal allows key j iff j <= i + total - nq.
//
// A step is up to three launches: the pass over the own rows (fa_serve_own.cuh), the
// pass over the prefix (fa_tc_prefix.cu), and the join of the states they
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
  // ---- where the prefix's states are (nothing here hangs on the kernels in front)
  const int slots = p.pre.split ? 2 : 1;
  int n_pre = 0;
  const float* pre_u = nullptr;
  const float4* pre_ml = nullptr;
  if (a.np > 0) {
    const long long x = (long long)b * rows + r;  // row of the key head
    const int unit = hk * p.pre.pairs + (int)(x / (2 * kPrefixRows));
    const int c0 = (int)((long long)unit * p.pre.steps / p.pre.per_cta);
    const int c1 = (int)(((long long)(unit + 1) * p.pre.steps - 1) / p.pre.per_cta);
    const long long tile = (long long)unit * p.pre.parts * 2 + ((int)(x / kPrefixRows) & 1);
    n_pre = (c1 - c0 + 1) * slots;
    // lane i reads state i's share; its own columns (groups of eight) of any state
    pre_ml = a.pre_ml + tile * kPrefixRows + x % kPrefixRows;
    pre_u = a.pre_u + tile * kPrefixRows * D + x % kPrefixRows * 8 + lane * E / 8 * (kPrefixRows * 8) + lane * E % 8;
  }
  const int len = raw_len(a, b);
  if (!len_ok(a, len)) return;
  const int nt = own_tiles(len), rg = r / p.cta_rows;
  ptx::grid_wait();
  long long per = 0, base = 0;
  if (nt > 0) {
    per = a.plan[0];
    base = a.plan[1 + b];
  }

  using Vec = typename std::conditional<E == 4, float4, float2>::type;
  float m = -INFINITY, mu = -INFINITY, l = 0.f, u[E];
#pragma unroll
  for (int e = 0; e < E; ++e) u[e] = 0.f;
  // Adds n states: 32 at a time, a lane finds one state's share (s: its own of the first 32), then all
  // lanes add the rows up.  at(i): where state i is, in steps from ml and pu.
  const float4 none = make_float4(-INFINITY, 0.f, -INFINITY, 0.f);
  auto join = [&](int n, float4 s, const float4* ml, const float* pu, long long ml_step, long long u_step, auto at) {
    for (int i0 = 0; i0 < n; i0 += 32) {
      if (i0 > 0) s = i0 + lane < n ? ml[at(i0 + lane) * ml_step] : none;
      const bool some = s.y != 0.f;  // a state without a key may not even have its u; NaN is not 0
      const float m_new = fmaxf(m, ptx::warp_max(some ? s.x : -INFINITY));
      const float mu_new = fmaxf(mu, ptx::warp_max(some ? s.z : -INFINITY));
      float share = some ? s.y * join_factor(s.x, m_new) : 0.f;
      const float g = join_factor(s.z, mu_new);
      unsigned todo = __ballot_sync(0xffffffffu, some);
#pragma unroll
      for (int x = 16; x >= 1; x >>= 1) share += __shfl_xor_sync(0xffffffffu, share, x);
      l = l * join_factor(m, m_new) + share;
      const float f = join_factor(mu, mu_new);
#pragma unroll
      for (int e = 0; e < E; ++e) u[e] *= f;
      m = m_new;
      mu = mu_new;
      while (todo) {
        constexpr int kTogether = 8;  // rows read before the first is used
        Vec v[kTogether];
        float w[kTogether];
#pragma unroll
        for (int k = 0; k < kTogether; ++k) {
          const int i = todo ? __ffs(todo) - 1 : 0;
          w[k] = todo ? __shfl_sync(0xffffffffu, g, i) : 0.f;
          v[k] = todo ? *reinterpret_cast<const Vec*>(pu + at(i0 + i) * u_step) : Vec{};
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
  };
  // part i / slots of the unit; with halved keys both slots hold the row
  const auto pre_at = [&](int i) -> long long { return (long long)(i / slots) * 2 + i % slots; };
  const float4 pre_s = lane < n_pre ? pre_ml[pre_at(lane) * kPrefixRows] : none;
  // the own rows' first shares are on their way while the prefix's states are added
  int n_own = 0;
  const float4* own_ml = a.row_ml + row;
  const float* own_u = a.row_u + row * D + lane * E;
  if (nt > 0) {
    const long long t0 = base + ((long long)hk * p.row_groups + rg) * own_cost(a, nt) + a.run_cost;
    const long long c0 = t0 / per;
    n_own = (int)((t0 + nt - 1) / per - c0) + 1;
    if (n_own > 1) {
      const long long first = c0 * 2 * p.cta_rows + (r - rg * p.cta_rows);
      own_ml = a.cut_ml + first;
      own_u = a.cut_u + first * D + lane * E;
    }
  }
  const auto own_at = [&](int i) -> long long { return n_own == 1 ? 0 : i == 0 ? 1 : 2 * (long long)i; };
  const float4 own_s = lane < n_own ? own_ml[own_at(lane) * p.cta_rows] : none;
  join(n_pre, pre_s, pre_ml, pre_u, kPrefixRows, (long long)kPrefixRows * D, pre_at);
  join(n_own, own_s, own_ml, own_u, p.cta_rows, (long long)p.cta_rows * D, own_at);
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
  a.run_cost = own_run_cost(a.k_exp ? 1 : 2, D);
  MergeParams m;
  m.cta_rows = own_rows(a.group * a.nq);
  m.row_groups = (a.group * a.nq + m.cta_rows - 1) / m.cta_rows;
  m.pre = prefix_plan(a.B, a.Hk, a.group * a.nq, a.np);
  carve(a, D, m.pre, static_cast<char*>(workspace));
  cudaError_t e = cudaSuccess;
  // The own rows first: where their shares end unevenly the prefix's CTAs, all alike, move in.
  if (a.max_len > 0) e = a.k_exp ? launch_own_e4m3(a, D, f16, s) : launch_own_16(a, D, f16, s);
  if (e == cudaSuccess && a.np > 0) e = launch_prefix(a, m.pre, D, f16, a.max_len > 0, s);
  if (e != cudaSuccess) return e;
  m.a = a;
  return f16 ? launch_merge<__half>(m, D, s) : launch_merge<__nv_bfloat16>(m, D, s);
}

}  // namespace fa
