// The router's choice by scores, with a bias for balance and groups of experts, and its gradient
// for the logits.
//
//   s[e] = 1 / (1 + exp(-l[e]))  or  softmax(l)[e]          c[e] = s[e] + bias[e]
//   groups of E / G experts: a group's worth is the sum of its best one or two c; the Gk groups of
//   most worth are kept, and the k largest c in them are the picks (ties: the lower id)
//   w[j] = scale s[e_j] (/ sum_i s[e_i])
//
// Whole numbers hang on c, so c and the worths are float64 by definition. Few rows need it: c is
// formed in float32 (or, where c grows with l alone, l itself is compared) with a bound on its
// error, and a row in which two neighbours of the result's order lie closer than their bounds
// allow is done again in float64 by its wave (row_exact). At T 65,536, E 256 of random logits that
// is one row in a thousand.
#include <algorithm>

#include "device_common.h"
#include "launch.h"
#include "mok.h"

namespace mok {
namespace {

constexpr int RS_NT = 256, RS_LPR = 16;          // lanes of a row: one DPP row
constexpr int RS_MAXE = 1024, RS_MAXK = 64;

struct RsArgs {
  const float* logits;
  const float* bias;
  int32_t* idx;
  float* w;
  int64_t T;
  int E, k, G, Gk, top;                          // experts of a group: E / G
  int sigmoid, renorm;
  float scale;
};

// ----------------------------------------------------------------- float64, one wave a row

// Doubles in the order of unsigned numbers, from 2 up; NaN above all. 1: -inf (an expert that is
// left out while there are others), 0: not available (its group is not kept, or taken).
MOK_DEV uint64_t order_key(double v) {
  if (v == -INFINITY) return 1;
  if (v != v) return ~0ull;
  const uint64_t u = (uint64_t)__double_as_longlong(v);
  return (u >> 63) ? ~u : u | (1ull << 63);
}
MOK_DEV double key_value(uint64_t k) {
  if (k == 1) return -INFINITY;
  if (k == ~0ull) return NAN;
  return __longlong_as_double((long long)((k >> 63) ? k & ~(1ull << 63) : ~k));
}

// Orders the wave's LDS accesses before this point against those behind it.
MOK_DEV void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

MOK_DEV double wave_sum(double v) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) v += __shfl_xor(v, m, kWave);
  return v;
}

// The lane's best (key, id) -> the wave's: the largest key, of equal ones the least id.
MOK_DEV void wave_best(uint64_t& key, int& id) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) {
    const uint64_t ok = shfl_xor_u64(key, m);
    const int oi = __shfl_xor(id, m, kWave);
    if (ok > key || (ok == key && oi < id)) { key = ok; id = oi; }
  }
}

// Row t by one wave. key [E], worth [G]: LDS of the wave's own.
MOK_DEV void row_exact(const RsArgs& a, int64_t t, uint64_t* key, uint64_t* worth) {
  const int lane = lane_id(), gs = a.E / a.G;
  const float* l = a.logits + t * a.E;
  double top = -INFINITY, inv = 0.0;
  if (!a.sigmoid) {
    double sum = 0.0;
    for (int e = lane; e < a.E; e += 64) top = fmax(top, (double)l[e]);
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) top = fmax(top, __shfl_xor(top, m, kWave));
    if (top > -INFINITY) {
      for (int e = lane; e < a.E; e += 64) sum += exp((double)l[e] - top);
      inv = 1.0 / wave_sum(sum);
    }
  }
  auto score = [&](float v) {
    if (a.sigmoid) return 1.0 / (1.0 + exp(-(double)v));
    return top > -INFINITY ? exp((double)v - top) * inv : (v != v ? (double)v : 0.0);
  };
  for (int e = lane; e < a.E; e += 64) {
    const float v = l[e];
    const double c = a.bias ? score(v) + (double)a.bias[e] : score(v);
    key[e] = v == -INFINITY ? 1 : order_key(c);
  }
  wave_sync();
  if (a.Gk < a.G) {
    for (int g = lane; g < a.G; g += 64) {
      uint64_t m1 = 1, m2 = 1;
      for (int e = g * gs; e < (g + 1) * gs; ++e) {
        const uint64_t c = key[e];
        if (c > m1) { m2 = m1; m1 = c; }
        else if (c > m2) m2 = c;
      }
      worth[g] = m1 == 1 || m2 == 1 || a.top == 1 ? m1 : order_key(key_value(m1) + key_value(m2));
    }
    wave_sync();
    for (int r = 0; r < a.Gk; ++r) {
      uint64_t best = 0;
      int id = a.G;
      for (int g = lane; g < a.G; g += 64)
        if (worth[g] > best) { best = worth[g]; id = g; }
      wave_best(best, id);
      if ((id & 63) == lane) worth[id] = 0;        // taken
      wave_sync();
    }
    for (int e = lane; e < a.E; e += 64)
      if (worth[e / gs] != 0) key[e] = 0;
    wave_sync();
  }
  int mine = 0;                                    // lane j: pick j
  for (int j = 0; j < a.k; ++j) {
    uint64_t best = 0;
    int id = a.E;
    for (int e = lane; e < a.E; e += 64)
      if (key[e] > best) { best = key[e]; id = e; }
    wave_best(best, id);
    if ((id & 63) == lane) key[id] = 0;
    if (lane == j) mine = id;
    wave_sync();
  }
  double s = 0.0;
  if (lane < a.k) s = score(l[mine]);
  if (a.renorm) {
    double sum = 0.0;
    for (int j = 0; j < a.k; ++j) sum += __shfl(s, j, kWave);
    s = sum == 0.0 ? 0.0 : s / sum;
  }
  if (lane < a.k) {
    a.idx[t * a.k + lane] = mine;
    a.w[t * a.k + lane] = (float)(a.scale * s);
  }
}

__global__ __launch_bounds__(RS_NT) void k_topk_scored_exact(const RsArgs a) {
  __shared__ uint64_t key[RS_NT / 64][RS_MAXE], worth[RS_NT / 64][RS_MAXE];
  const int wv = threadIdx.x >> 6;
  const int64_t t = blockIdx.x * (int64_t)(RS_NT / 64) + wv;
  if (t < a.T) row_exact(a, t, key[wv], worth[wv]);
}

// ------------------------------------------------------------------------------- gradient
// out = in + d loss / d logits. The picks' shares are scattered into the rows' place in LDS (an
// expert named twice adds up, in pick order), then the rows go through once.

struct RsBwd {
  const float* logits;
  const int32_t* idx;
  const float* dw;
  const float* in;
  float* out;
  int64_t T;
  int E, k, sigmoid, renorm, rows;               // rows of a workgroup
  float scale;
};

template <int LK>                                // lanes of a row's picks: a power of two >= k
MOK_DEV double pick_sum(double v) {
#pragma unroll
  for (int m = 1; m < LK; m <<= 1) v += __shfl_xor(v, m, kWave);
  return v;
}
template <int LK>
MOK_DEV float pick_max(float v) {
#pragma unroll
  for (int m = 1; m < LK; m <<= 1) v = fmaxf(v, __shfl_xor(v, m, kWave));
  return v;
}

// The picks of rows t0 .. t0 + n: dl at each pick into st [rows, E] (FULL: the gradient of its
// score; dot [rows] takes the sum over the picks of that times the score).
template <int LK, bool FULL>
MOK_DEV void scatter_picks(const RsBwd& a, int64_t t0, int n, float* st, const float* top,
                           const float* inv, float* dot) {
  const int l = threadIdx.x % LK;
  for (int r0 = 0; r0 < n; r0 += RS_NT / LK) {
    const int r = r0 + threadIdx.x / LK;
    const bool live = r < n && l < a.k;
    const int64_t at = (t0 + r) * a.k + l;
    const int e = live ? a.idx[at] : -1;
    const bool ok = live && e >= 0 && e < a.E;
    const float lg = ok ? a.logits[(t0 + r) * a.E + e] : -INFINITY;
    const double dw = ok ? (double)a.dw[at] : 0.0;
    double g;
    if constexpr (FULL) {
      g = a.scale * dw;
      const double s = ok && top[r] > -INFINITY ? exp((double)lg - (double)top[r]) * (double)inv[r] : 0.0;
      const double d = pick_sum<LK>(g * s);
      if (l == 0 && r < n) dot[r] = (float)d;
    } else {
      // s up to a factor that renormalising cancels; one: ds / dl = s one
      double s, one;
      if (a.sigmoid) {
        const double x = exp(-fabs((double)lg)), y = 1.0 / (1.0 + x);
        s = lg < 0.0f ? x * y : y;
        one = lg < 0.0f ? y : x * y;
      } else {
        const float m = pick_max<LK>(lg);
        s = m > -INFINITY ? exp((double)lg - (double)m) : 0.0;
        one = 1.0;
      }
      if (a.renorm) {
        const double sum = pick_sum<LK>(s), d = pick_sum<LK>(s * dw);
        g = sum == 0.0 ? 0.0 : a.scale * (s / sum) * (dw - d / sum) * one;
      } else {
        g = a.scale * dw * s * one;
      }
    }
    if (!ok) g = 0.0;
    // the first pick of an expert brings the shares of all that name it
    bool first = true;
    double all = g;
    for (int j = 0; j < a.k; ++j) {
      const int ej = __shfl(e, j, LK);
      const double gj = __shfl(g, j, LK);
      if (ej == e && j < l) first = false;
      if (ej == e && j > l) all += gj;
    }
    if (ok && first) st[r * a.E + e] = (float)all;
  }
}

// Softmax renormalised over the picks, and sigmoid: the gradient is zero outside the picks.
template <int LK>
__global__ __launch_bounds__(RS_NT) void k_topk_scored_bwd(const RsBwd a) {
  extern __shared__ float st[];
  const int64_t t0 = blockIdx.x * (int64_t)a.rows;
  const int n = (int)min((int64_t)a.rows, a.T - t0);
  const int elems = n * a.E;
  for (int i = threadIdx.x; i < elems; i += RS_NT) st[i] = 0.0f;
  __syncthreads();
  scatter_picks<LK, false>(a, t0, n, st, nullptr, nullptr, nullptr);
  __syncthreads();
  const int64_t base = t0 * a.E;
  for (int i = threadIdx.x; i < elems; i += RS_NT)
    a.out[base + i] = (a.in ? a.in[base + i] : 0.0f) + st[i];
}

// Softmax as it is: dl = s (ds - sum_picks ds s) for every expert of the row.
template <int LK>
__global__ __launch_bounds__(RS_NT) void k_topk_scored_bwd_full(const RsBwd a) {
  extern __shared__ float st[];
  __shared__ float top[RS_NT], inv[RS_NT], dot[RS_NT];
  const int64_t t0 = blockIdx.x * (int64_t)a.rows, base = t0 * a.E;
  const int n = (int)min((int64_t)a.rows, a.T - t0);
  const int elems = n * a.E, lane = lane_id();
  for (int i = threadIdx.x; i < elems; i += RS_NT) st[i] = 0.0f;
  for (int r = threadIdx.x >> 6; r < n; r += RS_NT / 64) {
    const float* l = a.logits + base + r * a.E;
    float m = -INFINITY;
    for (int e = lane; e < a.E; e += 64) m = fmaxf(m, l[e]);
#pragma unroll
    for (int q = 1; q < 64; q <<= 1) m = fmaxf(m, __shfl_xor(m, q, kWave));
    double s = 0.0;
    for (int e = lane; e < a.E; e += 64) s += (double)expf(l[e] - m);
    s = wave_sum(s);
    if (lane == 0) {
      top[r] = m;
      inv[r] = (float)(1.0 / s);
    }
  }
  __syncthreads();
  scatter_picks<LK, true>(a, t0, n, st, top, inv, dot);
  __syncthreads();
  for (int i = threadIdx.x; i < elems; i += RS_NT) {
    const int r = i / a.E;
    // a row of nothing but -inf has no probabilities and no gradient
    const float l = a.logits[base + i];
    const float p = top[r] == -INFINITY ? (l != l ? l : 0.0f) : expf(l - top[r]) * inv[r];
    a.out[base + i] = (a.in ? a.in[base + i] : 0.0f) + p * (st[i] - dot[r]);
  }
}

int rs_check(int64_t T, int32_t E, int32_t k, int32_t score) {
  if (T < 0 || E < 1 || E > RS_MAXE || k < 1 || k > E || k > RS_MAXK) return MOK_EINVAL;
  if (T * (int64_t)k >= (int64_t)1 << 31) return MOK_EINVAL;
  return score == MOK_SCORE_SOFTMAX || score == MOK_SCORE_SIGMOID ? MOK_OK : MOK_EINVAL;
}
int rs_check_groups(int32_t E, int32_t k, int32_t G, int32_t Gk, int32_t top, float scale) {
  if (G < 1 || G > E || E % G || Gk < 1 || Gk > G || k > (int64_t)Gk * (E / G)) return MOK_EINVAL;
  return top >= 1 && top <= 2 && fabsf(scale) < INFINITY ? MOK_OK : MOK_EINVAL;
}

hipError_t launch_scored(const RsArgs& a, hipStream_t s) {
  launch_k(k_topk_scored_exact, dim3((unsigned)((a.T + 3) / 4)), dim3(RS_NT), 0, s, nullptr,
           nullptr, a);
  return hipGetLastError();
}

}  // namespace
}  // namespace mok

using namespace mok;

extern "C" {

int mok_topk_scored(const float* logits, int64_t T, int32_t E, int32_t k, int32_t score,
                    const float* bias, int32_t n_groups, int32_t topk_groups, int32_t group_top,
                    int32_t renorm, float scale, int32_t* topk_idx, float* topk_w, void* stream) {
  int st = rs_check(T, E, k, score);
  if (st == MOK_OK) st = rs_check_groups(E, k, n_groups, topk_groups, group_top, scale);
  if (st != MOK_OK) return st;
  if (T == 0) return MOK_OK;
  if (!logits || !topk_idx || !topk_w) return MOK_EINVAL;
  const RsArgs a = {logits, bias, topk_idx, topk_w, T, E, k, n_groups, topk_groups, group_top,
                    score == MOK_SCORE_SIGMOID, renorm != 0, scale};
  return launch_scored(a, (hipStream_t)stream) == hipSuccess ? MOK_OK : MOK_EHIP;
}

int mok_route_scored(const void* x, const void* w_router, int64_t T, int32_t d, int32_t E,
                     int32_t k, int32_t io_dtype, int32_t score, const float* bias,
                     int32_t n_groups, int32_t topk_groups, int32_t group_top, int32_t renorm,
                     float scale, float* logits, int32_t* topk_idx, float* topk_w, void* stream) {
  int st = rs_check(T, E, k, score);
  if (st == MOK_OK) st = rs_check_groups(E, k, n_groups, topk_groups, group_top, scale);
  if (st != MOK_OK) return st;
  if (d < 1 || (io_dtype != MOK_FP32 && io_dtype != MOK_BF16)) return MOK_EINVAL;
  if (T == 0) return MOK_OK;
  if (!x || !w_router || !logits || !topk_idx || !topk_w) return MOK_EINVAL;
  const hipError_t e = launch_router_logits(x, w_router, T, d, E, io_dtype == MOK_BF16, logits,
                                            (hipStream_t)stream);
  if (e != hipSuccess) return MOK_EHIP;
  return mok_topk_scored(logits, T, E, k, score, bias, n_groups, topk_groups, group_top, renorm,
                         scale, topk_idx, topk_w, stream);
}

int mok_topk_scored_backward(const float* logits, const int32_t* topk_idx, const float* dtopk_w,
                             const float* dlogits_in, int64_t T, int32_t E, int32_t k,
                             int32_t score, int32_t renorm, float scale, float* dlogits,
                             void* stream) {
  const int st = rs_check(T, E, k, score);
  if (st != MOK_OK) return st;
  if (!(fabsf(scale) < INFINITY)) return MOK_EINVAL;
  if (T == 0) return MOK_OK;
  if (!logits || !topk_idx || !dtopk_w || !dlogits) return MOK_EINVAL;
  RsBwd a = {logits, topk_idx, dtopk_w, dlogits_in, dlogits, T, E, k, score == MOK_SCORE_SIGMOID,
             renorm != 0, 0, scale};
  // rows of a workgroup: 16 KB of their place in LDS, at most 64
  a.rows = std::max(1, std::min(64, 4096 / E));
  const dim3 grid((unsigned)((T + a.rows - 1) / a.rows));
  const uint32_t lds = (uint32_t)(a.rows * E * sizeof(float));
  hipStream_t s = (hipStream_t)stream;
  const bool full = score == MOK_SCORE_SOFTMAX && !renorm;
  auto go = [&](auto LK) {
    launch_k(full ? k_topk_scored_bwd_full<LK()> : k_topk_scored_bwd<LK()>, grid, dim3(RS_NT), lds,
             s, nullptr, nullptr, a);
  };
  if (k <= 8) go(std::integral_constant<int, 8>{});
  else go(std::integral_constant<int, 64>{});
  return hipGetLastError() == hipSuccess ? MOK_OK : MOK_EHIP;
}

}  // extern "C"
