// Products with 4-bit weights in groups along K, for a few rows, and the experts' FFNs of the MoE
// layer on such weights.
//
//   W[n,k] = (q[n,k] - z[n,k / g]) s[n,k / g],  q 0 .. 15, two codes a byte, 2i in the low nibble
//   C[m,n] = sum_groups s (sum_{k in group} x[m,k] (q - z))
//
// Bound by streaming the codes once. A weight's 16 rows and 128 columns are one 16-byte load a lane
// (lane (kq, n): row n, 32 codes), and enter the 16x16x32 bf16 MFMA as integers: a nibble 0 .. 15 is,
// as an E4M3 byte, q 2^-9 (its first two binades are evenly spaced), so one AND for four codes and a
// conversion for two give exact bf16 integers, about one VALU operation a code. x is the other
// operand. A second MFMA with the constant -z beside each takes the zero point off inside the same
// float32 sum; the group's sum is scaled in float32. Rows of x past M are zero: up to 16 rows cost
// what one does.
//
// A workgroup's waves split K (KC columns each), and keep their part of x in registers while they
// walk the workgroup's tiles of 16 weight rows, so that only weights are loaded in the loop, up to R
// tiles ahead; the waves' sums meet in LDS in a fixed order. K past 8 KC goes in rounds, whose sums
// stay in LDS.
//
// The MoE's first launch pairs the gate and up rows of a tile and writes H = silu(gate) up in
// float32; its second reads H as two bf16 planes (16 significant bits) that take rows 0 .. 7 and
// 8 .. 15 of the MFMA's 16, which keeps the result as exact as float32 H would to 2^-17; a third adds
// a token's experts in the order of its picks.
#include <algorithm>

#include "device_common.h"
#include "launch.h"
#include "mok.h"

namespace mok {
namespace {

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));

constexpr int W4_MAXW = 8;           // waves of a workgroup
constexpr int W4_TILES = 8;          // tiles of a workgroup
constexpr int W4_SCAN = 1024;        // routes up to which a workgroup finds its rows by itself
enum { W4_DENSE = 0, W4_UP = 1, W4_DOWN = 2 };

struct W4Mat {
  const uint8_t* codes;              // [experts, N, K / 2]
  const uint16_t* scales;            // [experts, N, K / g] bf16
  const uint8_t* zeros;              // the same shape; NULL: 8
};

struct W4Args {
  W4Mat w[2];
  const void* x;                     // rows: bf16 [M, K], or H float32 [routes, K]
  void* out;                         // dense: bf16 or float32 [M, N]; up: H; down: P float32
  int64_t M;                         // dense
  int N, K;
  int tiles, tpw, waves, out_f32;
  // MoE
  const int32_t* idx;                // [T k]
  const float* tw;
  const int32_t *offsets, *route_ids;   // the plan (more than W4_SCAN routes), else NULL
  int64_t routes;
  int k, e0, El;
};

// Lane groups of 16 <-> registers: afterwards w[j] of lane group q is what w[q] of group j was.
MOK_DEV void transpose4(uint32_t (&w)[4]) {
  auto s32 = [](uint32_t& a, uint32_t& b) {
    const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
    a = r[0]; b = r[1];
  };
  auto s16 = [](uint32_t& a, uint32_t& b) {
    const auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
    a = r[0]; b = r[1];
  };
  s32(w[0], w[2]);
  s32(w[1], w[3]);
  s16(w[0], w[1]);
  s16(w[2], w[3]);
}

// 8 codes of a word as bf16 integers, in the order 0 2 4 6 1 3 5 7.
MOK_DEV bf16x8_t unpack8(uint32_t w) {
  const uint32_t lo = w & 0x0F0F0F0Fu, hi = (w >> 4) & 0x0F0F0F0Fu;
  const bf16x2_t a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 512.0f, false);
  const bf16x2_t b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 512.0f, true);
  const bf16x2_t c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 512.0f, false);
  const bf16x2_t d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 512.0f, true);
  return bf16x8_t{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// 8 consecutive values in that order.
MOK_DEV bf16x8_t order8(const uint4 v) {
  uint4 o;
  o.x = __builtin_amdgcn_perm(v.y, v.x, 0x05040100u);
  o.y = __builtin_amdgcn_perm(v.w, v.z, 0x05040100u);
  o.z = __builtin_amdgcn_perm(v.y, v.x, 0x07060302u);
  o.w = __builtin_amdgcn_perm(v.w, v.z, 0x07060302u);
  return __builtin_bit_cast(bf16x8_t, o);
}

typedef uint32_t u32_any __attribute__((aligned(1)));

// One tile's weights of a wave: codes, scales and zero points of its KC columns.
template <int G, bool Z, int KC>
struct W4Unit {
  static constexpr int NL = KC / 128, NS = KC / G;      // loads, groups
  uint4 q[NL];
  uint32_t s[NS / 2];
  uint32_t z[Z ? (NS + 3) / 4 : 1];

  // m: the matrix, its row n (of lane) at codes offset row_c; kb: the wave's first column
  MOK_DEV void load(const W4Mat& m, int64_t row, int K, int kb, int kq) {
    const uint8_t* c = m.codes + row * (K / 2);
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      const int k = kb + 128 * i + 32 * kq;
      q[i] = *(const uint4*)(c + (k < K ? k / 2 : 0));   // x is zero there
    }
    const int ng = K / G, g0 = kb / G;
    const uint16_t* sp = m.scales + row * ng + g0;
    const uint8_t* zp = Z ? m.zeros + row * ng + g0 : nullptr;
    if (kb + KC <= K) {
#pragma unroll
      for (int i = 0; i < NS / 2; ++i) s[i] = ((const u32_any*)sp)[i];
      if constexpr (Z)
#pragma unroll
        for (int i = 0; i < NS / 4; ++i) z[i] = ((const u32_any*)zp)[i];
    } else {
#pragma unroll
      for (int i = 0; i < NS / 2; ++i) {
        const uint32_t lo = g0 + 2 * i < ng ? sp[2 * i] : 0, hi = g0 + 2 * i + 1 < ng ? sp[2 * i + 1] : 0;
        s[i] = lo | (hi << 16);
      }
      if constexpr (Z)
#pragma unroll
        for (int i = 0; i < NS / 4; ++i) {
          z[i] = 0;
#pragma unroll
          for (int b = 0; b < 4; ++b)
            if (g0 + 4 * i + b < ng) z[i] |= (uint32_t)zp[4 * i + b] << (8 * b);
        }
    }
  }

  MOK_DEV f32x4_t product(const bf16x8_t (&a)[KC / 32]) const {
    f32x4_t total = {0, 0, 0, 0}, acc = {0, 0, 0, 0};
    bf16x8_t zb = __builtin_bit_cast(bf16x8_t, make_uint4(0xC100C100u, 0xC100C100u, 0xC100C100u, 0xC100C100u));
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      uint32_t w[4] = {q[i].x, q[i].y, q[i].z, q[i].w};
      if constexpr (G < 128) transpose4(w);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int k = 128 * i + 32 * j, g = k / G;
        if constexpr (Z)
          if (k % G == 0) {
            const float zf = -(float)((z[g / 4] >> (8 * (g % 4))) & 0xFF);
            const uint32_t zz = pack_bf16x2(zf, zf);
            zb = __builtin_bit_cast(bf16x8_t, make_uint4(zz, zz, zz, zz));
          }
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[4 * i + j], unpack8(w[j]), acc, 0, 0, 0);
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[4 * i + j], zb, acc, 0, 0, 0);
        if ((k + 32) % G == 0) {
          const float sc = __uint_as_float(g % 2 ? s[g / 2] & 0xFFFF0000u : s[g / 2] << 16);
          total += acc * sc;
          acc = f32x4_t{0, 0, 0, 0};
        }
      }
    }
    return total;
  }
};

// Workgroup (x, y): tiles x tpw .., of M rows y 16 .. (dense) or of expert slot y (MoE).
template <int G, bool Z, int KC, int MODE>
__global__ __launch_bounds__(64 * W4_MAXW) void k_w4(const W4Args p) {
  constexpr int S = MODE == W4_UP ? 2 : 1;             // matrices of a tile
  constexpr int MR = MODE == W4_DOWN ? 8 : 16;         // rows of a pass
  constexpr int R = S == 2 ? 2 : 3;                    // units in registers
  __shared__ float red[2][W4_MAXW][S][256];
  __shared__ float part[W4_TILES][S][256];
  __shared__ int16_t list[MODE == W4_DENSE ? 1 : W4_SCAN];
  const int tid = threadIdx.x, lane = lane_id(), wv = uniform(tid >> 6), kq = lane >> 4, ln = lane & 15;
  int64_t expert = 0, count, plan_at = 0;
  if constexpr (MODE == W4_DENSE) {
    count = min((int64_t)MR, p.M - (int64_t)blockIdx.y * MR);
  } else if (p.offsets) {
    expert = blockIdx.y;
    plan_at = p.offsets[expert];
    count = p.offsets[expert + 1] - plan_at;
    if (count <= 0) return;
  } else {
    // more local experts than routes: a slot is a route, and serves its expert if no earlier route
    // names it; otherwise a slot is an expert
    const bool by_route = p.routes < p.El;
    int e = p.e0 + (int)blockIdx.y;
    if (by_route) e = p.idx[blockIdx.y];
    if (e < p.e0 || e >= p.e0 + p.El) return;
    expert = e - p.e0;
    int n = 0;
    for (int r0 = 0; r0 < (int)p.routes; r0 += 64) {
      const int r = r0 + lane;
      const bool hit = r < p.routes && p.idx[r] == e;
      const uint64_t mask = ballot(hit);
      if (by_route && n == 0 && mask && r0 + __ffsll((unsigned long long)mask) - 1 < (int)blockIdx.y) return;
      if (hit && wv == 0) list[n + __popcll(mask & lanemask_lt())] = (int16_t)r;
      n += __popcll(mask);
    }
    count = n;
    if (count == 0) return;
    __syncthreads();
  }
  const int t0 = blockIdx.x * p.tpw, nt = min(p.tpw, p.tiles - t0);
  const int span = p.waves * KC, rounds = (p.K + span - 1) / span;
  const int units = nt * S;
  int turn = 0;                        // the half of red that the next tile's sums take
  auto route_of = [&](int64_t m) -> int64_t {
    return p.offsets ? p.route_ids[plan_at + m] : (int64_t)list[m];
  };
  for (int64_t m0 = 0; m0 < count; m0 += MR) {
    const int rows = (int)min((int64_t)MR, count - m0);
    // the row of x that this lane's MFMA row is
    const int am = ln % MR;
    int64_t row = -1;
    if (am < rows) {
      if constexpr (MODE == W4_DENSE) row = (int64_t)blockIdx.y * MR + am;
      else if constexpr (MODE == W4_UP) row = route_of(m0 + am) / p.k;
      else row = route_of(m0 + am);
    }
    for (int rd = 0; rd < rounds; ++rd) {
      const int kb = rd * span + wv * KC;
      W4Unit<G, Z, KC> u[R];
      auto fetch = [&](W4Unit<G, Z, KC>& to, int i) {
        const int n = min((t0 + i / S) * 16 + ln, p.N - 1);
        to.load(p.w[S == 2 ? i % 2 : 0], expert * p.N + n, p.K, kb < p.K ? kb : 0, kq);
      };
#pragma unroll
      for (int q = 0; q + 1 < R; ++q)
        if (q < units) fetch(u[q], q);
      bf16x8_t a[KC / 32];
#pragma unroll
      for (int f = 0; f < KC / 32; ++f) {
        const int k = kb + 128 * (f / 4) + (G < 128 ? 32 * (f % 4) + 8 * kq : 32 * kq + 8 * (f % 4));
        const bool ok = row >= 0 && k < p.K;
        if constexpr (MODE != W4_DOWN) {
          uint4 v = make_uint4(0, 0, 0, 0);
          if (ok) v = *(const uint4*)((const bf16_t*)p.x + row * p.K + k);
          a[f] = order8(v);
        } else {
          float4 v0 = make_float4(0, 0, 0, 0), v1 = v0;
          if (ok) {
            v0 = *(const float4*)((const float*)p.x + row * p.K + k);
            v1 = *(const float4*)((const float*)p.x + row * p.K + k + 4);
          }
          const float v[8] = {v0.x, v0.z, v1.x, v1.z, v0.y, v0.w, v1.y, v1.w};
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const __bf16 hi = (__bf16)v[i];
            a[f][i] = ln < 8 ? hi : (__bf16)(v[i] - (float)hi);
          }
        }
      }
      f32x4_t sum[S];
      for (int i0 = 0; i0 < units; i0 += R) {
#pragma unroll
        for (int q = 0; q < R; ++q) {
          const int i = i0 + q;
          if (i >= units) break;
          if (i + R - 1 < units) fetch(u[(q + R - 1) % R], i + R - 1);
          __builtin_amdgcn_sched_barrier(0);
          const int s = S == 2 ? q % 2 : 0, t = i / S;
          sum[s] = u[q].product(a);
          if (s + 1 < S) continue;
          // the waves' sums, in their order
#pragma unroll
          for (int c = 0; c < S; ++c)
#pragma unroll
            for (int e = 0; e < 4; ++e) red[turn][wv][c][(4 * kq + e) * 16 + ln] = sum[c][e];
          __syncthreads();
          for (int o = tid; o < rows * 16; o += blockDim.x) {
            float v[S];
#pragma unroll
            for (int c = 0; c < S; ++c) {
              v[c] = 0.0f;
              for (int w = 0; w < p.waves; ++w) {
                v[c] += red[turn][w][c][o];
                if constexpr (MR == 8) v[c] += red[turn][w][c][128 + o];
              }
              if (rounds > 1) {
                if (rd > 0) v[c] += part[t][c][o];
                part[t][c][o] = v[c];
              }
            }
            const int m = o >> 4, n = (t0 + t) * 16 + (o & 15);
            if (rd + 1 < rounds || n >= p.N) continue;
            if constexpr (MODE == W4_DENSE) {
              const int64_t at = ((int64_t)blockIdx.y * MR + m) * p.N + n;
              if (p.out_f32) ((float*)p.out)[at] = v[0];
              else ((bf16_t*)p.out)[at] = f32_to_bf16(v[0]);
            } else {
              const int64_t r = route_of(m0 + m);
              if constexpr (MODE == W4_UP) ((float*)p.out)[r * p.N + n] = silu(v[0]) * v[S - 1];
              else ((float*)p.out)[r * p.N + n] = p.tw[r] * v[0];
            }
          }
          turn ^= 1;
        }
      }
    }
  }
}

// y[t] = y_in[t] + sum of the local experts' P[t k + j], j ascending; 4 columns a thread.
__global__ __launch_bounds__(256) void k_w4_combine(const float* __restrict__ P,
                                                    const int32_t* __restrict__ idx,
                                                    const uint2* y_in, int64_t T, int k, int e0,
                                                    int El, int d4, uint2* y) {
  const int64_t i = blockIdx.x * (int64_t)256 + threadIdx.x;
  const int64_t t = i / d4;
  if (t >= T) return;
  float4 v = make_float4(0, 0, 0, 0);
  if (y_in) {
    const uint2 u = y_in[i];
    v = make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u),
                    __uint_as_float(u.y << 16), __uint_as_float(u.y & 0xFFFF0000u));
  }
  const float4* p = (const float4*)P + t * k * d4 + (i - t * d4);
#pragma unroll 4
  for (int j = 0; j < k; ++j) {
    const int e = idx[t * k + j] - e0;
    if (e < 0 || e >= El) continue;
    const float4 q = p[(int64_t)j * d4];
    v.x += q.x; v.y += q.y; v.z += q.z; v.w += q.w;
  }
  y[i] = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
}

// ------------------------------------------------------------------------------- quantiser
// A thread a group: its range, then its codes.
template <int G>
__global__ __launch_bounds__(256) void k_quantize_int4(const bf16_t* __restrict__ src,
                                                       int64_t groups, uint8_t* __restrict__ codes,
                                                       uint16_t* __restrict__ scales,
                                                       uint8_t* __restrict__ zeros) {
  const int64_t g = blockIdx.x * (int64_t)256 + threadIdx.x;
  if (g >= groups) return;
  const uint4* p = (const uint4*)(src + g * G);
  float lo = 0.0f, hi = 0.0f;
  bool bad = false;
  auto values = [&](int i, float (&v)[8]) {
    const uint4 q = p[i];
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = __uint_as_float(w[j] << 16);
      v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
    }
  };
  for (int i = 0; i < G / 8; ++i) {
    float v[8];
    values(i, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      lo = fminf(lo, v[j]);
      hi = fmaxf(hi, v[j]);
      bad |= !(fabsf(v[j]) < INFINITY);
    }
  }
  // |w| up to 7 steps below the zero point and 7 above; with zero points 15 steps over the range
  const float range = zeros ? __fdiv_rn(hi, 15.0f) - __fdiv_rn(lo, 15.0f)
                            : __fdiv_rn(fmaxf(hi, -lo), 7.0f);
  uint16_t sb = f32_to_bf16(range);
  if (bad) sb = 0x7FC0;
  const float s = bf16_to_f32(sb);
  const bool flat = !(s > 0.0f);                  // zeros (or no numbers): all codes the zero point
  float z = 8.0f;
  if (zeros) z = flat ? 0.0f : fminf(fmaxf(rintf(__fdiv_rn(-lo, s)), 0.0f), 15.0f);
  scales[g] = sb;
  if (zeros) zeros[g] = (uint8_t)z;
  uint32_t* out = (uint32_t*)(codes + g * (G / 2));
  for (int i = 0; i < G / 8; ++i) {
    float v[8];
    values(i, v);
    uint32_t w = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float c = flat ? z : fminf(fmaxf(rintf(__fdiv_rn(v[j], s)) + z, 0.0f), 15.0f);
      w |= (uint32_t)c << (4 * j);
    }
    out[i] = w;
  }
}

bool group_ok(int g) { return g == 32 || g == 64 || g == 128; }
bool al16(const void* p) { return (uintptr_t)p % 16 == 0; }

template <int MODE>
hipError_t launch_w4(W4Args a, int g, unsigned slots, hipStream_t s) {
  // KC columns a wave: 512, or 1024 where 8 waves of 512 do not cover K (groups of 32 would hold too
  // many scales)
  const bool wide = a.K > 512 * W4_MAXW && g >= 64;
  const int kc = wide ? 1024 : 512;
  a.waves = std::min(W4_MAXW, (a.K + kc - 1) / kc);
  a.tiles = (a.N + 15) / 16;
  // as many tiles a workgroup as leave one for every CU
  a.tpw = (int)std::max<int64_t>(1, std::min<int64_t>(W4_TILES, (int64_t)a.tiles * slots / 256));
  const dim3 grid((a.tiles + a.tpw - 1) / a.tpw, slots), block(64 * a.waves);
  auto go = [&](auto G, auto Z) {
    if constexpr (G() >= 64)
      if (wide) return launch_k(k_w4<G(), Z(), 1024, MODE>, grid, block, 0, s, nullptr, nullptr, a);
    launch_k(k_w4<G(), Z(), 512, MODE>, grid, block, 0, s, nullptr, nullptr, a);
  };
  auto pick = [&](auto G) {
    if (a.w[0].zeros) go(G, std::true_type{});
    else go(G, std::false_type{});
  };
  if (g == 32) pick(std::integral_constant<int, 32>{});
  else if (g == 64) pick(std::integral_constant<int, 64>{});
  else pick(std::integral_constant<int, 128>{});
  return hipGetLastError();
}

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

// Places in the workspace of a MoE call.
struct MoeW4Plan {
  bool plan;                 // routes grouped by a plan (else every workgroup scans them)
  size_t H, P, counts, offsets, ranks, ids, blk, total;
};
MoeW4Plan moe_w4_plan(const mok_moe_w4_args& a) {
  MoeW4Plan p = {};
  const int64_t n = a.T * a.k;
  p.plan = n > W4_SCAN;
  size_t at = 0;
  auto put = [&](size_t bytes) { const size_t o = at; at += up256(bytes); return o; };
  p.H = put((size_t)n * a.I * sizeof(float));
  p.P = put((size_t)n * a.d * sizeof(float));
  if (p.plan) {
    p.counts = put((size_t)a.E_l * 4);
    p.offsets = put((size_t)(a.E_l + 1) * 4);
    p.ranks = put((size_t)a.E_l * 4);
    p.ids = put((size_t)n * 4);
    p.blk = put((size_t)4 << 16);      // the most that a plan's chunk histograms take
  }
  p.total = std::max<size_t>(at, 256);
  return p;
}

int moe_w4_check(const mok_moe_w4_args* a) {
  if (!a || a->T < 0 || a->d < 1 || a->I < 1 || !group_ok(a->group)) return MOK_EINVAL;
  if (a->d % a->group || a->I % a->group || a->d > (1 << 22) || a->I > (1 << 22)) return MOK_EINVAL;
  if (a->E < 1 || a->k < 1 || a->k > a->E || a->k > 64 || a->e0 < 0 || a->E_l < 1 || a->E_l > 1024 ||
      a->E_l > a->E - a->e0)
    return MOK_EINVAL;
  return a->T * (int64_t)a->k < (int64_t)1 << 31 ? MOK_OK : MOK_EINVAL;
}

}  // namespace
}  // namespace mok

using namespace mok;

extern "C" {

int mok_quantize_int4(const void* src_bf16, int64_t rows, int32_t K, int32_t group, uint8_t* codes,
                      void* scales, uint8_t* zeros, void* stream) {
  if (rows < 0 || K < 1 || !group_ok(group) || K % group) return MOK_EINVAL;
  if (rows == 0) return MOK_OK;
  if (!src_bf16 || !codes || !scales || !al16(src_bf16) || (uintptr_t)codes % 4) return MOK_EINVAL;
  const int64_t groups = rows * (K / group), blocks = (groups + 255) / 256;
  if (blocks * 256 >= (int64_t)1 << 32) return MOK_EUNSUPPORTED;
  auto k = group == 32 ? k_quantize_int4<32> : group == 64 ? k_quantize_int4<64> : k_quantize_int4<128>;
  launch_k(k, dim3((unsigned)blocks), dim3(256), 0, (hipStream_t)stream, nullptr, nullptr,
           (const bf16_t*)src_bf16, groups, codes, (uint16_t*)scales, zeros);
  return hipGetLastError() == hipSuccess ? MOK_OK : MOK_EHIP;
}

int mok_w4_gemm(const void* x, const uint8_t* codes, const void* scales, const uint8_t* zeros,
                int64_t M, int64_t N, int32_t K, int32_t group, int32_t out_dtype, void* c,
                void* stream) {
  if (M < 0 || N < 0 || M >= (int64_t)1 << 31 || N >= (int64_t)1 << 31 || !group_ok(group)) return MOK_EINVAL;
  if (K < group || K % group || K > (1 << 22)) return MOK_EINVAL;
  if (out_dtype != MOK_BF16 && out_dtype != MOK_FP32) return MOK_EINVAL;
  if (M == 0 || N == 0) return MOK_OK;
  if (!x || !codes || !scales || !c || !al16(x) || !al16(codes) || (uintptr_t)scales % 2) return MOK_EINVAL;
  if ((uintptr_t)c % (out_dtype == MOK_FP32 ? 4 : 2)) return MOK_EINVAL;
  W4Args a = {};
  a.w[0] = {codes, (const uint16_t*)scales, zeros};
  a.x = x; a.out = c; a.M = M; a.N = (int)N; a.K = K; a.out_f32 = out_dtype == MOK_FP32;
  const int64_t slots = (M + 15) / 16;
  if (slots > 65535 || N > (int64_t)1 << 26) return MOK_EUNSUPPORTED;
  return launch_w4<W4_DENSE>(a, group, (unsigned)slots, (hipStream_t)stream) == hipSuccess ? MOK_OK
                                                                                          : MOK_EHIP;
}

int mok_moe_w4_workspace_bytes(const mok_moe_w4_args* args, size_t* bytes) {
  if (!bytes || moe_w4_check(args) != MOK_OK) return MOK_EINVAL;
  *bytes = moe_w4_plan(*args).total;
  return MOK_OK;
}

int mok_moe_w4_forward(const mok_moe_w4_args* args, void* stream) {
  const int st = moe_w4_check(args);
  if (st != MOK_OK) return st;
  const mok_moe_w4_args& a = *args;
  if (a.T == 0) return MOK_OK;
  if (!a.x || !a.topk_idx || !a.topk_w || !a.y) return MOK_EINVAL;
  const void* const cs[] = {a.gate_codes, a.up_codes, a.down_codes};
  const void* const ss[] = {a.gate_scales, a.up_scales, a.down_scales};
  for (int i = 0; i < 3; ++i)
    if (!cs[i] || !ss[i] || !al16(cs[i]) || (uintptr_t)ss[i] % 2) return MOK_EINVAL;
  const bool z = a.gate_zeros;
  if (z != (a.up_zeros != nullptr) || z != (a.down_zeros != nullptr)) return MOK_EINVAL;
  if (!al16(a.x) || (uintptr_t)a.y % 8 || (uintptr_t)a.y_in % 8) return MOK_EINVAL;
  const MoeW4Plan p = moe_w4_plan(a);
  if (!a.workspace || a.workspace_bytes < p.total || !al16(a.workspace)) return MOK_EWORKSPACE;
  char* const ws = (char*)a.workspace;
  hipStream_t s = (hipStream_t)stream;
  const int64_t n = a.T * a.k, blocks = (a.T * (a.d / 4) + 255) / 256;
  if (blocks * 256 >= (int64_t)1 << 32) return MOK_EUNSUPPORTED;
  if (p.plan) {
    const hipError_t e = launch_plan(a.topk_idx, a.T, a.k, a.e0, a.E_l, a.T, (int32_t*)(ws + p.counts),
                                     (int32_t*)(ws + p.offsets), (int32_t*)(ws + p.ranks),
                                     (int32_t*)(ws + p.ids), (int32_t*)(ws + p.blk), n, s);
    if (e != hipSuccess) return MOK_EHIP;
  }
  W4Args w = {};
  w.idx = a.topk_idx; w.tw = a.topk_w; w.routes = n; w.k = a.k; w.e0 = a.e0; w.El = a.E_l;
  if (p.plan) {
    w.offsets = (const int32_t*)(ws + p.offsets);
    w.route_ids = (const int32_t*)(ws + p.ids);
  }
  const unsigned slots = (unsigned)(p.plan ? a.E_l : std::min<int64_t>(n, a.E_l));
  w.w[0] = {a.gate_codes, (const uint16_t*)a.gate_scales, a.gate_zeros};
  w.w[1] = {a.up_codes, (const uint16_t*)a.up_scales, a.up_zeros};
  w.x = a.x; w.out = ws + p.H; w.N = a.I; w.K = a.d;
  if (launch_w4<W4_UP>(w, a.group, slots, s) != hipSuccess) return MOK_EHIP;
  w.w[0] = {a.down_codes, (const uint16_t*)a.down_scales, a.down_zeros};
  w.x = ws + p.H; w.out = ws + p.P; w.N = a.d; w.K = a.I;
  if (launch_w4<W4_DOWN>(w, a.group, slots, s) != hipSuccess) return MOK_EHIP;
  launch_k(k_w4_combine, dim3((unsigned)blocks), dim3(256), 0, s, nullptr, nullptr,
           (const float*)(ws + p.P), a.topk_idx, (const uint2*)a.y_in, a.T, a.k, a.e0, a.E_l, a.d / 4,
           (uint2*)a.y);
  return hipGetLastError() == hipSuccess ? MOK_OK : MOK_EHIP;
}

}  // extern "C"
