// The router's choice by scores, with a bias for balance and groups of experts, and its gradient
// for the logits.
//
//   s[e] = 1 / (1 + exp(-l[e]))  or  softmax(l)[e]          c[e] = s[e] + bias[e]
//   groups of E / G experts: a group's worth is the sum of its best one or two c; the Gk groups of
//   most worth are kept, and the k largest c in them are the picks (ties: the lower id)
//   w[j] = scale s[e_j] (/ sum_i s[e_i])
//
// Whole numbers hang on c, so c and the worths are float64 by definition. Few rows need it: k_topk_scored
// orders a row by float32 values (c, or l itself where c grows with l alone) whose error is bounded. Where
// neighbours of that order lie closer than the bound allows, c of those up to the next clear step (16 at
// most) is formed in float64 and they are ordered by it; rows with groups that close, with NaN, with scores
// at float64's ends or with nothing left are done in float64 from the start by their wave (row_exact).
//
// Bound by the vector unit for many rows (T 65,536, E 256, 8 groups: 41 to 49 us, 89% of them vector instructions
// (a row's sort, rounds and float64 weights), against 13 for reading the logits; the whole row in float64 took
// 537) and by latency for few (one row: 7 us with its launch). 16 lanes a row and not 64: four rows share the rounds' instructions. The gradient
// is a stream of dlogits (30 us there against 27 for its bytes).
#include <algorithm>

#include "device_common.h"
#include "launch.h"
#include "mok.h"

namespace mok {
namespace {

constexpr int RS_NT = 256, RS_LPR = 16;          // lanes of a row: one DPP row
constexpr int RS_MAXE = 1024, RS_MAXK = 64;
constexpr int64_t RS_MAXT = 1 << 25;             // a launch's 2^32 threads, 64 a row

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

MOK_DEV double wave_sum(double v) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) v += __shfl_xor(v, m, kWave);
  return v;
}

template <int CTRL> MOK_DEV uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, true);
}
// The lane's best (key, id) -> the wave's: the largest key, of equal ones the least id. Within the rows of
// 16 lanes by rotations, then across them.
MOK_DEV void wave_best(uint64_t& key, int& id) {
  auto step = [&](uint32_t lo, uint32_t hi, int oi) {
    const uint64_t ok = ((uint64_t)hi << 32) | lo;
    const bool better = ok > key || (ok == key && oi < id);
    key = better ? ok : key;
    id = better ? oi : id;
  };
  step(dpp<0x128>((uint32_t)key), dpp<0x128>((uint32_t)(key >> 32)), (int)dpp<0x128>((uint32_t)id));
  step(dpp<0x124>((uint32_t)key), dpp<0x124>((uint32_t)(key >> 32)), (int)dpp<0x124>((uint32_t)id));
  step(dpp<0x122>((uint32_t)key), dpp<0x122>((uint32_t)(key >> 32)), (int)dpp<0x122>((uint32_t)id));
  step(dpp<0x121>((uint32_t)key), dpp<0x121>((uint32_t)(key >> 32)), (int)dpp<0x121>((uint32_t)id));
#pragma unroll
  for (int m = 16; m < 64; m <<= 1) {
    const uint64_t ok = shfl_xor_u64(key, m);
    step((uint32_t)ok, (uint32_t)(ok >> 32), __shfl_xor(id, m, kWave));
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
    // P lanes a group: each its share of the members, then the best two of all
    const int P = a.G > 32 ? 1 : 64 >> (32 - __clz(a.G - 1));
    for (int g0 = 0; g0 < a.G; g0 += 64 / P) {
      const int g = g0 + lane / P;
      uint64_t m1 = 1, m2 = 1;
      if (g < a.G)
        for (int e = g * gs + lane % P; e < (g + 1) * gs; e += P) {
          const uint64_t c = key[e];
          m2 = max(m2, min(m1, c));
          m1 = max(m1, c);
        }
      for (int m = 1; m < P; m <<= 1) {
        const uint64_t o1 = shfl_xor_u64(m1, m), o2 = shfl_xor_u64(m2, m);
        m2 = max(min(m1, o1), max(m2, o2));
        m1 = max(m1, o1);
      }
      if (g < a.G && lane % P == 0)
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
    if (!a.sigmoid && inv == inv) {                // from the picks' largest, as it may be far below the row's
      const double x = lane < a.k ? (double)l[mine] : -INFINITY;
      double most = x;
#pragma unroll
      for (int m = 1; m < 64; m <<= 1) most = fmax(most, __shfl_xor(most, m, kWave));
      s = most > -INFINITY ? exp(x - most) : 0.0;
    }
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

// ----------------------------------------------------------------------- float32, four rows a wave
// A row is 16 lanes, lane l with the C = ceil(E / 16) <= Q values from l C on. Every value becomes a key:
// the float32's bits in the order of unsigned numbers, the lowest four or five of them replaced by its
// place in the lane. A lane sorts its 8 largest; k rounds then take the row's largest of 16 heads.

// Over the row's 16 lanes, the result in each (rotations by 8, 4, 2, 1).
MOK_DEV uint32_t row_max(uint32_t v) {
  v = max(v, dpp<0x128>(v));
  v = max(v, dpp<0x124>(v));
  v = max(v, dpp<0x122>(v));
  return max(v, dpp<0x121>(v));
}
MOK_DEV float row_maxf(float v) {
  v = fmaxf(v, __uint_as_float(dpp<0x128>(__float_as_uint(v))));
  v = fmaxf(v, __uint_as_float(dpp<0x124>(__float_as_uint(v))));
  v = fmaxf(v, __uint_as_float(dpp<0x122>(__float_as_uint(v))));
  return fmaxf(v, __uint_as_float(dpp<0x121>(__float_as_uint(v))));
}
MOK_DEV double row_sum(double v) {
#pragma unroll
  for (int m = 1; m < RS_LPR; m <<= 1) v += __shfl_xor(v, m, kWave);
  return v;
}

// exp(x) for x <= 0 within 2^-35 of itself, 0 below -700 (float32 holds none of it): 2^n e^r, |r| <= ln 2 / 2, by
// the series up to r^9. A softmax that is not renormalised takes one of every expert.
MOK_DEV double exp_down(double x) {
  const double n = rint(x * 1.4426950408889634);
  const double r = fma(n, -0.6931471805599453, x);
  double p = 1.0 / 362880;
  p = fma(p, r, 1.0 / 40320);
  p = fma(p, r, 1.0 / 5040);
  p = fma(p, r, 1.0 / 720);
  p = fma(p, r, 1.0 / 120);
  p = fma(p, r, 1.0 / 24);
  p = fma(p, r, 1.0 / 6);
  p = fma(p, r, 0.5);
  p = fma(p, r, 1.0);
  p = fma(p, r, 1.0);
  return x > -700.0 ? __builtin_amdgcn_ldexp(p, (int)n) : 0.0;
}

MOK_DEV uint32_t key_of(float v) {
  const uint32_t u = __float_as_uint(v);
  return u ^ ((uint32_t)((int)u >> 31) | 0x80000000u);
}
MOK_DEV float value_of(uint32_t k) {
  return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}
constexpr uint32_t kLeftOut = 0x007FFFFFu;         // key_of(-inf): keys up to this are left-out experts'

MOK_DEV void order2(uint32_t& a, uint32_t& b) {    // the larger first
  const uint32_t m = max(a, b);
  b = min(a, b);
  a = m;
}
// Sorts K[0 .. 8) (N = 8) or [0 .. 4), largest first.
template <int N> MOK_DEV void sort_keys(uint32_t* K) {
  auto c = [&](int i, int j) { order2(K[i], K[j]); };
  if constexpr (N == 4) {
    c(0, 1); c(2, 3); c(0, 2); c(1, 3); c(1, 2);
  } else {
    c(0, 1); c(2, 3); c(4, 5); c(6, 7); c(0, 2); c(1, 3); c(4, 6); c(5, 7); c(1, 2); c(5, 6);
    c(0, 4); c(1, 5); c(2, 6); c(3, 7); c(2, 4); c(3, 5); c(1, 2); c(3, 4); c(5, 6);
  }
}
// A = the 8 largest of two sorted eights, sorted: the larger of A[i] and B[7 - i] are they, a bitonic row.
MOK_DEV void merge8(uint32_t* A, const uint32_t* B) {
#pragma unroll
  for (int i = 0; i < 8; ++i) A[i] = max(A[i], B[7 - i]);
#pragma unroll
  for (int d = 4; d > 0; d >>= 1)
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (!(i & d)) order2(A[i], A[i + d]);
}

template <int Q>
__global__ __launch_bounds__(RS_NT) void k_topk_scored(const RsArgs a, bool by_logit) {
  constexpr int H = Q < 8 ? Q : 8;                 // heads a lane keeps
  constexpr uint32_t PLACE = Q > 16 ? 31u : 15u;
  __shared__ int picks[RS_NT / RS_LPR][RS_LPR];
  // a wave's: float64 keys of a row, or the values of its four rows
  __shared__ uint64_t xkey[RS_NT / 64][32 * Q], xworth[RS_NT / 64][RS_LPR];
  const int l = threadIdx.x & 15, row = threadIdx.x >> 4, wv = threadIdx.x >> 6;
  const int64_t t = blockIdx.x * (int64_t)(RS_NT / RS_LPR) + row;
  const bool live = t < a.T;
  const float* lg = a.logits + min(t, a.T - 1) * a.E;
  const int C = (a.E + RS_LPR - 1) / RS_LPR, e0 = l * C, n = max(0, min(C, a.E - e0));
  float v[Q], bias[Q];
  auto load = [&](const float* p, float (&to)[Q], float none) {
    if (a.E == RS_LPR * Q && ((uintptr_t)p & 15) == 0) {
#pragma unroll
      for (int q = 0; q < Q; q += 4) {
        const float4 u = *(const float4*)(p + e0 + q);
        to[q] = u.x; to[q + 1] = u.y; to[q + 2] = u.z; to[q + 3] = u.w;
      }
    } else {
#pragma unroll
      for (int q = 0; q < Q; ++q) to[q] = q < n ? p[e0 + q] : none;
    }
  };
  load(lg, v, -INFINITY);
  if (a.bias) load(a.bias, bias, 0.0f);
  // c, or l. A row with NaN or +inf is done in float64.
  bool redo = false;
#pragma unroll
  for (int q = 0; q < Q; ++q) redo |= !(v[q] < INFINITY);
  float top = -INFINITY;
  double sum = 1.0;                                // softmax that is not renormalised: its sum
  if (!a.sigmoid) {
#pragma unroll
    for (int q = 0; q < Q; ++q) top = fmaxf(top, v[q]);
    top = row_maxf(top);
    if (!a.renorm && top > -INFINITY) {
      double s = 0.0;                              // (the weights are float64's, rounded once)
#pragma unroll
      for (int q = 0; q < Q; ++q) s += exp_down((double)v[q] - (double)top);
      sum = row_sum(s);
    }
  }
  // margin of a value x, m0 + m1 |x|: pairs further apart than this are in the order of float64. The bits
  // that make room for the place count less than 2^-19 (2^-18) of x, both ways the same; c is rounded by
  // 2^-24. A sigmoid is off by 1 unit of 2^-24 for its argument and exponential, 1 for 1 + x and 2 for the
  // reciprocal: two of them by less than 6e-7. A softmax by 2^-24 of its argument (d e^-d < 0.4), 2 for the
  // exponential, and by a factor of the sum's, common to the row, of less than 1.5e-6.
  float m0 = by_logit ? 1e-6f : a.sigmoid ? 6e-7f : 3e-6f, m1 = Q > 16 ? 4.4e-6f : 2.4e-6f;
  if (!by_logit) {
    if (a.sigmoid) {
#pragma unroll
      for (int q = 0; q < Q; ++q) v[q] = v[q] == -INFINITY ? v[q] : __builtin_amdgcn_rcpf(1.0f + __expf(-v[q]));
    } else {
      float s = 0.0f;
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        const float x = __expf(v[q] - top);
        s += x;
        v[q] = v[q] == -INFINITY ? v[q] : x;
      }
      const float inv = (float)(1.0 / row_sum((double)s));
#pragma unroll
      for (int q = 0; q < Q; ++q) v[q] *= inv;
      if (!a.bias) { m0 = 0.0f; m1 += 4e-5f; }
    }
    if (a.bias) {
#pragma unroll
      for (int q = 0; q < Q; ++q) v[q] += bias[q];
#pragma unroll
      for (int q = 0; q < Q; ++q) redo |= !(v[q] < INFINITY);
    }
  }
  uint32_t kept = 0xFFFFFFFFu;                     // lane's values that are available
  if (a.Gk < a.G) {
    const int gs = a.E / a.G, L = gs / C;
    float w1 = -INFINITY, w2 = -INFINITY;
    const bool aligned = a.E == RS_LPR * C && gs % C == 0 && (L & (L - 1)) == 0;
    int g;                                         // the group whose worth this lane has (G: none)
    if (aligned) {
#pragma unroll
      for (int q = 0; q < Q; ++q)
        if (q < C) {
          w2 = fmaxf(w2, fminf(w1, v[q]));
          w1 = fmaxf(w1, v[q]);
        }
      for (int m = 1; m < L; m <<= 1) {
        const float o1 = __shfl_xor(w1, m, kWave), o2 = __shfl_xor(w2, m, kWave);
        w2 = fmaxf(fminf(w1, o1), fmaxf(w2, o2));
        w1 = fmaxf(w1, o1);
      }
      g = l / L;
    } else {
      // through LDS: lane g goes over group g
      float* const f = (float*)xkey[wv] + (row & 3) * (16 * Q);
#pragma unroll
      for (int q = 0; q < Q; ++q)
        if (q < n) f[e0 + q] = v[q];
      wave_sync();
      g = l < a.G ? l : a.G;
      if (l < a.G)
        for (int e = l * gs; e < (l + 1) * gs; ++e) {
          w2 = fmaxf(w2, fminf(w1, f[e]));
          w1 = fmaxf(w1, f[e]);
        }
      wave_sync();
    }
    const float w = a.top == 1 || w2 == -INFINITY ? w1 : w1 + w2;
    const int step = aligned ? L : 1;
    int rank = 0;
    for (int r = 1; r < a.G; ++r) {
      // group (g + r) % G
      const int og = g + r >= a.G ? g + r - a.G : g + r;
      const float o = __shfl(w, min(og * step, 15), RS_LPR);
      rank += o > w || (o == w && og < g);
    }
    const bool in = g < a.G && rank < a.Gk, out = g < a.G && !in;
    const float least = -row_maxf(in ? -w : -INFINITY), most = row_maxf(out ? w : -INFINITY);
    // (worths carry no places: m0 of each member, and roundings; by_logit they are logits themselves. A bias
    // may be any number, and members of other signs leave a worth far smaller than what was rounded)
    const float size = a.bias ? row_maxf((w1 > -INFINITY ? fabsf(w1) : 0.0f) + (w2 > -INFINITY ? fabsf(w2) : 0.0f))
                              : fabsf(least);
    const float near = by_logit ? m0 * fmaxf(1.0f, fabsf(least)) : 2.0f * m0 + (m0 == 0.0f ? 9e-5f : 4e-7f) * size;
    redo |= most > -INFINITY && least - most < near;
    redo |= a.bias && !(size < INFINITY);          // worths past float32
    if (by_logit && most > -INFINITY)              // where float64 scores may be equal
      redo |= a.sigmoid ? most > 20.0f || least < -700.0f : least - top < -700.0f;
    if (aligned) {
      kept = in ? kept : 0;
    } else {
      const uint32_t mask = (uint32_t)(ballot(in) >> (threadIdx.x & 48)) & 0xFFFFu;
      kept = 0;
      int gg = e0 / gs, left = (gg + 1) * gs - e0;           // group of value q, values left of it
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        kept |= ((mask >> min(gg, 31)) & 1u) << q;
        if (--left == 0) { ++gg; left = gs; }
      }
    }
  }
  uint32_t K[Q < 8 ? 8 : Q];
#pragma unroll
  for (int q = 0; q < Q; ++q)
    K[q] = q < n && ((kept >> q) & 1u) ? (key_of(v[q]) & ~PLACE) | (uint32_t)q : 0u;
#pragma unroll
  for (int q = 0; q < Q; q += H) sort_keys<H>(K + q);
#pragma unroll
  for (int q = 8; q < Q; q += 8) merge8(K, K + q);
  // Rounds: the row's candidates in the order of their keys, k and on to the first that lies clear of the
  // one before it. near: two of them do not, and their order has to be found.
  float prev = INFINITY;
  int used = 0, n_cand = 0;
  bool near = false;
  for (int j = 0; j <= RS_LPR; ++j) {
    const uint32_t m = row_max(K[0]);
    const uint32_t hits = (uint32_t)(ballot(K[0] == m) >> (threadIdx.x & 48)) & 0xFFFFu;
    const float x = value_of(m | PLACE);
    const bool left_out = (m & ~PLACE) <= kLeftOut;
    // (nothing left, and experts that are left out behind others, are clear)
    const bool clear = m == 0 || j == 0 || prev - x > (by_logit ? m0 * fmaxf(1.0f, fabsf(prev)) : m0) + m1 * fabsf(prev);
    if (j >= a.k && clear && n_cand == 0) n_cand = j;
    if (ballot(n_cand == 0) == 0 || j == RS_LPR) break;
    if (n_cand == 0) {
      near |= !clear;
      if (j < a.k) {
        if (by_logit && !left_out)                 // where float64 scores may be equal
          redo |= a.sigmoid ? x > 20.0f || x < -700.0f : x - top < -700.0f;
        if (m0 == 0.0f) redo |= !left_out && x < 1e-30f;         // near float32's end
      }
      if (l == __ffs(hits) - 1) {
        picks[row][j] = e0 + (int)(m & PLACE);
#pragma unroll
        for (int i = 0; i + 1 < H; ++i) K[i] = K[i + 1];
        K[H - 1] = 0;
        ++used;
      }
      prev = x;
    }
  }
  redo |= n_cand == 0;                             // more than 16 that have to be told apart
  if (H < Q) redo |= used >= H;                    // a lane may have had more
  redo |= near && !a.sigmoid && a.bias;            // c needs the softmax's sum in float64
  redo &= live;
  wave_sync();
  // lane j has candidate j; the picks are those of rank below k
  const bool any = ((ballot(redo) >> (threadIdx.x & 48)) & 0xFFFFu) != 0;
  const bool cand = l < n_cand && !any;
  const int e = cand ? picks[row][l] : 0;
  const float x = cand ? lg[e] : -INFINITY;
  double s = a.sigmoid ? 1.0 / (1.0 + exp(-(double)x)) : 0.0;
  int slot = l;
  if (ballot(near && cand)) {
    double c = a.sigmoid ? s : exp((double)x - (double)top);
    if (a.bias) c += cand ? (double)a.bias[e] : 0.0;
    if (x == -INFINITY) c = -INFINITY;
    const int id = cand ? e : RS_MAXE + l;
    int rank = 0;
#pragma unroll
    for (int r = 1; r < RS_LPR; ++r) {
      const double o = __shfl(c, l + r, RS_LPR);
      const int oi = __shfl(id, l + r, RS_LPR);
      rank += o > c || (o == c && oi < id);
    }
    slot = rank;
  }
  const bool has = cand && slot < a.k;
  if (!a.sigmoid) {
    const float base = a.renorm ? row_maxf(has ? x : -INFINITY) : top;
    s = base > -INFINITY ? exp((double)x - (double)base) / sum : 0.0;
  }
  if (!has) s = 0.0;
  if (a.renorm) {
    const double all = row_sum(s);
    s = all == 0.0 ? 0.0 : s / all;
  }
  if (has && live) {
    a.idx[t * a.k + slot] = e;
    a.w[t * a.k + slot] = (float)(a.scale * s);
  }
  uint64_t rows = ballot(any);
  while (rows) {
    const int r = (__ffsll((unsigned long long)rows) - 1) >> 4;
    rows &= ~(0xFFFFull << (16 * r));
    row_exact(a, blockIdx.x * (int64_t)(RS_NT / RS_LPR) + 4 * wv + r, xkey[wv], xworth[wv]);
    wave_sync();
  }
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
        if (lg < 0.0f && x < 0x1p-1024) s = 0.0;   // the forward's, where exp(-l) is past float64
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
// V: 4 values a thread where rows and addresses allow, or 1. The loads of dlogits_in go first, over the
// picks' work.
template <int LK, int V>
__global__ __launch_bounds__(RS_NT) void k_topk_scored_bwd(const RsBwd a) {
  typedef float Vec __attribute__((ext_vector_type(V)));
  extern __shared__ __attribute__((aligned(16))) float st[];
  const int64_t t0 = blockIdx.x * (int64_t)a.rows, base = t0 * a.E;
  const int n = (int)min((int64_t)a.rows, a.T - t0), elems = n * a.E / V;
  constexpr int U = 4;
  Vec in[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int i = threadIdx.x + u * RS_NT;
    in[u] = a.in && i < elems ? ((const Vec*)(a.in + base))[i] : Vec(0.0f);
  }
  for (int i = threadIdx.x; i < elems; i += RS_NT) ((Vec*)st)[i] = Vec(0.0f);
  __syncthreads();
  scatter_picks<LK, false>(a, t0, n, st, nullptr, nullptr, nullptr);
  __syncthreads();
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int i = threadIdx.x + u * RS_NT;
    if (i < elems) ((Vec*)(a.out + base))[i] = in[u] + ((Vec*)st)[i];
  }
  for (int i = threadIdx.x + U * RS_NT; i < elems; i += RS_NT)
    ((Vec*)(a.out + base))[i] = (a.in ? ((const Vec*)(a.in + base))[i] : Vec(0.0f)) + ((Vec*)st)[i];
}

// Softmax as it is: dl = s (ds - sum_picks ds s) for every expert of the row.
template <int LK>
__global__ __launch_bounds__(RS_NT) void k_topk_scored_bwd_full(const RsBwd a) {
  extern __shared__ __attribute__((aligned(16))) float st[];
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
  if (T >= (int64_t)1 << 31 || T * (int64_t)k >= (int64_t)1 << 31) return MOK_EINVAL;
  return score == MOK_SCORE_SOFTMAX || score == MOK_SCORE_SIGMOID ? MOK_OK : MOK_EINVAL;
}
int rs_check_groups(int32_t E, int32_t k, int32_t G, int32_t Gk, int32_t top, float scale) {
  if (G < 1 || G > E || E % G || Gk < 1 || Gk > G || k > (int64_t)Gk * (E / G)) return MOK_EINVAL;
  return top >= 1 && top <= 2 && fabsf(scale) < INFINITY ? MOK_OK : MOK_EINVAL;
}

hipError_t launch_scored(const RsArgs& a, hipStream_t s) {
  // k_topk_scored holds 32 values and the 8 best a lane, and a group a lane (T 65,536, E 256, 8 groups: k 8 41 to 49 us;
  // k 9, by a wave a row in float64, 429)
  if (a.E > 512 || a.k > 8 || (a.G > RS_LPR && a.Gk < a.G)) {
    launch_k(k_topk_scored_exact, dim3((unsigned)((a.T + 3) / 4)), dim3(RS_NT), 0, s, nullptr, nullptr, a);
  } else {
    // c grows with l alone: no bias, and no sums of two
    const bool by_logit = !a.bias && (a.Gk == a.G || a.top == 1);
    const int C = (a.E + RS_LPR - 1) / RS_LPR;
    auto k = C <= 4 ? k_topk_scored<4> : C <= 8 ? k_topk_scored<8> : C <= 16 ? k_topk_scored<16>
             : C <= 24 ? k_topk_scored<24> : k_topk_scored<32>;
    constexpr int rows = RS_NT / RS_LPR;
    launch_k(k, dim3((unsigned)((a.T + rows - 1) / rows)), dim3(RS_NT), 0, s, nullptr, nullptr, a, by_logit);
  }
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
  if (T > RS_MAXT) return MOK_EUNSUPPORTED;
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
  if (T > RS_MAXT) return MOK_EUNSUPPORTED;
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
  if (T > RS_MAXT) return MOK_EUNSUPPORTED;
  RsBwd a = {logits, topk_idx, dtopk_w, dlogits_in, dlogits, T, E, k, score == MOK_SCORE_SIGMOID,
             renorm != 0, 0, scale};
  // rows of a workgroup: at most 16 KB of their place in LDS, 64, and what leaves 1024 workgroups
  a.rows = (int)std::max<int64_t>(1, std::min<int64_t>(std::min(64, 4096 / E), T / 1024));
  const dim3 grid((unsigned)((T + a.rows - 1) / a.rows));
  const uint32_t lds = (uint32_t)(a.rows * E * sizeof(float));
  hipStream_t s = (hipStream_t)stream;
  const bool full = score == MOK_SCORE_SOFTMAX && !renorm;
  const bool vec = E % 4 == 0 && (((uintptr_t)dlogits_in | (uintptr_t)dlogits) & 15) == 0;
  auto go = [&](auto LK) {
    launch_k(full ? k_topk_scored_bwd_full<LK()> : vec ? k_topk_scored_bwd<LK(), 4> : k_topk_scored_bwd<LK(), 1>,
             grid, dim3(RS_NT), lds, s, nullptr, nullptr, a);
  };
  if (k <= 8) go(std::integral_constant<int, 8>{});
  else go(std::integral_constant<int, 64>{});
  return hipGetLastError() == hipSuccess ? MOK_OK : MOK_EHIP;
}

}  // extern "C"
