// Decoding steps over a cache whose sequences have their own lengths, with
// grouped heads: fa_decode_cache (the 8-bit cache) and fa_decode_shared (a
// prefix that the whole batch shares, then each sequence's own rows, 16-bit or
// 8-bit).  Query head h reads key head h / (H / Hk); row i of the nq new
// queries sits at position total - nq + i of its sequence's total = np + len
// keys, so causal allows key j iff j <= i + total - nq.
//
// A step is up to three launches: the pass over the prefix (fa_tc_prefix.cu), the
// pass over the own rows (fa_serve_own.cuh), beside it, and the join of the states they
// leave, here: m = max m_s, l = sum l_s 2^(m_s - m), u = sum u_s 2^(mu_s - mu),
// O = u 2^(mu - m) / l, L = (m + log2 l) ln 2.  Each launch may start while the one
// in front of it drains.
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "fa_internal.cuh"
#include "fa_serve.cuh"
#include "ptx.cuh"

namespace fa {
namespace {

// Joins the states of every query row: D / 8 lanes a row, eight columns each, one
// whole sector of a state's row.  The join waits for L2 more than it moves bytes, so
// where few rows have many states kGroups groups of lanes share a row's.  Four groups and one, us a step: behind a prefix
// of 16384 keys 512 rows 32 and 62, 2048 rows 32 and 46, 4096 rows 45 and 47, 8192 rows 72 and 65; 4096 rows behind 1024
// keys 19 and 20, 8192 rows 26 and 18.  Of the own rows alone, 16384 keys: 32 rows (about 38 states each) 15 and 20, 128 rows (9)
// 31 and 32, 256 rows (4) and 512 rows (2) alike.
constexpr int kMergeThreads = 256;
constexpr long long kFewRows = 4096;
constexpr int kManyStates = 6;

struct MergeParams {
  ServeArgs a;
  int cta_rows, row_groups, own_ctas;  // of the pass over the own rows
  PrefixPlan pre;
};

template <typename T, int D, int kGroups>
__global__ void __launch_bounds__(kMergeThreads) merge_kernel(const __grid_constant__ MergeParams p) {
  constexpr int kLanes = D / 8, kTogether = 4;  // lanes of a row; states' rows read before the first is used
  const ServeArgs& a = p.a;
  const int lane = threadIdx.x % kLanes;
  const int rows = a.group * a.nq;
  constexpr int kBlockRows = kMergeThreads / kLanes / kGroups;
  const int group = threadIdx.x / kLanes % kGroups, in_block = threadIdx.x / kLanes / kGroups;
  const long long row = (long long)blockIdx.x * kBlockRows + in_block;
  const bool there = row < (long long)a.B * a.Hk * rows;  // every lane stays for the shuffles
  const long long slab = there ? row / rows : 0;
  const int r = there ? (int)(row - slab * rows) : 0, b = (int)(slab / a.Hk), hk = (int)(slab - (long long)b * a.Hk);
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
    pre_ml = a.pre_ml + tile * kPrefixRows + x % kPrefixRows;
    pre_u = a.pre_u + tile * kPrefixRows * D + x % kPrefixRows * 8 + lane * (kPrefixRows * 8);
  }
  const int len = raw_len(a, b);
  const bool valid = there && len_ok(a, len);
  const int nt = valid ? own_tiles(len) : 0, rg = r / p.cta_rows;
  if (!valid) n_pre = 0;
  ptx::grid_wait();
  // part i / slots of the unit; with halved keys both slots hold the row
  // (this group's are i kGroups + group)
  const auto mine = [&](int n) { return (n - group + kGroups - 1) / kGroups; };
  const auto pre_at = [&](int i) -> long long {
    i = i * kGroups + group;
    return (long long)(i / slots) * 2 + i % slots;
  };
  n_pre = mine(n_pre);
  const float4 none = make_float4(-INFINITY, 0.f, -INFINITY, 0.f);
  const float4 pre_s = lane < n_pre ? pre_ml[pre_at(lane) * kPrefixRows] : none;
  int n_own = 0;
  const float4* own_ml = a.row_ml + row;
  const float* own_u = a.row_u + row * D + lane * 8;
  if (nt > 0) {
    const long long per = a.plan[0];
    const long long t0 = a.plan[1 + b] + ((long long)hk * p.row_groups + rg) * own_cost(a, nt) + a.run_cost;
    const long long c0 = t0 / per;
    n_own = (int)((t0 + nt - 1) / per - c0) + 1;
    if (n_own > 1) {
      const long long first = c0 * 2 * p.cta_rows + (r - rg * p.cta_rows);
      own_ml = a.cut_ml + first;
      own_u = a.cut_u + first * D + lane * 8;
    }
  }
  const bool whole = n_own == 1;
  const auto own_at = [&](int i) -> long long {
    i = i * kGroups + group;
    return whole ? 0 : i == 0 ? 1 : 2 * (long long)i;
  };
  n_own = mine(n_own);
  const float4 own_s = lane < n_own ? own_ml[own_at(lane) * p.cta_rows] : none;  // on its way while the prefix's are added

  float m = -INFINITY, mu = -INFINITY, l = 0.f, u[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) u[e] = 0.f;
  // Adds n states, kLanes at a time: a lane finds one state's share (s: its own of the first kLanes), then
  // all lanes add the rows up.  at(i): where state i is, in steps from ml and pu.
  auto join = [&](int n, float4 s, const float4* ml, const float* pu, long long ml_step, long long u_step, auto at) {
    const int most = __reduce_max_sync(0xffffffffu, n);  // the warp's rows go together
    for (int i0 = 0; i0 < most; i0 += kLanes) {
      if (i0 > 0) s = i0 + lane < n ? ml[at(i0 + lane) * ml_step] : none;
      const bool some = s.y != 0.f;  // a state without a key may not even have its u; NaN is not 0
      float m_new = some ? s.x : -INFINITY, mu_new = some ? s.z : -INFINITY;
#pragma unroll
      for (int x = kLanes / 2; x >= 1; x >>= 1) {
        m_new = fmaxf(m_new, __shfl_xor_sync(0xffffffffu, m_new, x));
        mu_new = fmaxf(mu_new, __shfl_xor_sync(0xffffffffu, mu_new, x));
      }
      m_new = fmaxf(m, m_new);
      mu_new = fmaxf(mu, mu_new);
      float share = some ? s.y * join_factor(s.x, m_new) : 0.f;
#pragma unroll
      for (int x = kLanes / 2; x >= 1; x >>= 1) share += __shfl_xor_sync(0xffffffffu, share, x);
      l = l * join_factor(m, m_new) + share;
      const float f = join_factor(mu, mu_new), g = join_factor(s.z, mu_new);
#pragma unroll
      for (int e = 0; e < 8; ++e) u[e] *= f;
      m = m_new;
      mu = mu_new;
      const unsigned has = __ballot_sync(0xffffffffu, some) >> (threadIdx.x % 32 / kLanes * kLanes);
      for (int k0 = 0; k0 < min(kLanes, most - i0); k0 += kTogether) {
        float4 v[kTogether][2];
        float w[kTogether];
#pragma unroll
        for (int k = 0; k < kTogether; ++k) {
          const int i = k0 + k;
          const bool take = (has >> i) & 1;
          w[k] = __shfl_sync(0xffffffffu, g, i, kLanes);
          if (!take) w[k] = 0.f;
          const float4* from = reinterpret_cast<const float4*>(pu + at(i0 + i) * u_step);
          v[k][0] = take ? from[0] : make_float4(0.f, 0.f, 0.f, 0.f);
          v[k][1] = take ? from[1] : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int k = 0; k < kTogether; ++k)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            u[4 * h] = fmaf(v[k][h].x, w[k], u[4 * h]);
            u[4 * h + 1] = fmaf(v[k][h].y, w[k], u[4 * h + 1]);
            u[4 * h + 2] = fmaf(v[k][h].z, w[k], u[4 * h + 2]);
            u[4 * h + 3] = fmaf(v[k][h].w, w[k], u[4 * h + 3]);
          }
      }
    }
  };
  join(n_pre, pre_s, pre_ml, pre_u, kPrefixRows, (long long)kPrefixRows * D, pre_at);
  join(n_own, own_s, own_ml, own_u, p.cta_rows, (long long)p.cta_rows * D, own_at);
  if constexpr (kGroups > 1) {
    __shared__ float4 s_s[kBlockRows][kGroups];
    __shared__ float4 s_u[kBlockRows][kGroups][2][kLanes];
    if (lane == 0) s_s[in_block][group] = make_float4(m, l, mu, 0.f);
    s_u[in_block][group][0][lane] = make_float4(u[0], u[1], u[2], u[3]);
    s_u[in_block][group][1][lane] = make_float4(u[4], u[5], u[6], u[7]);
    __syncthreads();
    if (group != 0) return;
#pragma unroll
    for (int x = 1; x < kGroups; ++x) {
      const float4 t = s_s[in_block][x];
      if (t.y == 0.f) continue;
      const float m_new = fmaxf(m, t.x), mu_new = fmaxf(mu, t.z);
      l = l * join_factor(m, m_new) + t.y * join_factor(t.x, m_new);
      const float f = join_factor(mu, mu_new), g = join_factor(t.z, mu_new);
      const float* y = reinterpret_cast<const float*>(&s_u[in_block][x][0][lane]);
      const float* z = reinterpret_cast<const float*>(&s_u[in_block][x][1][lane]);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        u[e] = u[e] * f + y[e] * g;
        u[4 + e] = u[4 + e] * f + z[e] * g;
      }
      m = m_new;
      mu = mu_new;
    }
  }
  if (!valid) {
    if (there && lane == 0) atomicOr(a.status, kDevBadSeqlens);
    return;
  }
  // l = 0: no key; NaN goes through
  const float f = l == 0.f ? 0.f : exp2f(mu - m);
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < 8; ++e) u[e] = l == 0.f ? 0.f : u[e] / l * f;
#pragma unroll
  for (int e = 0; e < 4; ++e) w[e] = ptx::pack16x2<std::is_same<T, __half>::value>(u[2 * e], u[2 * e + 1]);
  *reinterpret_cast<uint4*>(static_cast<T*>(a.o) + row * D + lane * 8) = make_uint4(w[0], w[1], w[2], w[3]);
  if (lane == 0) a.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

template <typename T>
cudaError_t launch_merge(const MergeParams& p, int D, cudaStream_t s) {
  const long long rows = (long long)p.a.B * p.a.Hk * p.a.group * p.a.nq;
  // states of a row, about: the prefix's parts, and the CTAs that share a unit of the own rows
  const long long units = (long long)p.a.B * p.a.Hk * p.row_groups;
  const long long states = (p.a.np > 0 ? (p.pre.steps / p.pre.per_cta + 1) * (p.pre.split ? 2 : 1) : 0) +
                           std::min<long long>(p.own_ctas / units, own_tiles(p.a.max_len));
  const bool few = rows <= kFewRows && states >= kManyStates;
  const int per = kMergeThreads / (D / 8) / (few ? 4 : 1);
  auto* kernel = few ? (D == 64 ? merge_kernel<T, 64, 4> : merge_kernel<T, 128, 4>)
                     : (D == 64 ? merge_kernel<T, 64, 1> : merge_kernel<T, 128, 1>);
  return note_error("cached decoding merge launch",
                    launch_serve_kernel(kernel, (int)((rows + per - 1) / per), kMergeThreads, 0,
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
  // the layout depends on whether the own rows are 8-bit; the size covers both
  size_t most = 0;
  for (int elem = 1; elem <= 2; ++elem) {
    const size_t bytes = carve(a, D, serve_plan(B, Hk, a.group * nq, np, max_len, D, elem).pre, nullptr);
    if (bytes > most) most = bytes;
  }
  return most;
}

cudaError_t launch_serve(ServeArgs& a, int D, fa_dtype dt, void* workspace, cudaStream_t s) {
  const bool f16 = dt == FA_F16;
  MergeParams m;
  m.cta_rows = own_rows(a.group * a.nq);
  a.run_cost = own_run_cost(m.cta_rows, a.k_exp ? 1 : 2, D);
  m.row_groups = (a.group * a.nq + m.cta_rows - 1) / m.cta_rows;
  const ServePlan plan = serve_plan(a.B, a.Hk, a.group * a.nq, a.np, a.max_len, D, a.k_exp ? 1 : 2);
  m.pre = plan.pre;
  m.own_ctas = plan.own_sms * own_per_sm(m.cta_rows, a.k_exp ? 1 : 2, D);
  carve(a, D, m.pre, static_cast<char*>(workspace));
  cudaError_t e = cudaSuccess;
  if (a.np > 0) e = launch_prefix(a, m.pre, D, f16, s);
  if (e == cudaSuccess && a.max_len > 0)
    e = a.k_exp ? launch_own_e4m3(a, D, f16, plan.own_sms, plan.together, s)
                : launch_own_16(a, D, f16, plan.own_sms, plan.together, s);
  if (e != cudaSuccess) return e;
  m.a = a;
  return f16 ? launch_merge<__half>(m, D, s) : launch_merge<__nv_bfloat16>(m, D, s);
}

}  // namespace fa
