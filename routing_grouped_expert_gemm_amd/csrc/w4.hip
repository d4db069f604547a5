// Products with 4-bit weights in groups along K, for a few rows, and the experts' FFNs of the MoE
// layer on such weights.
//
//   W[n,k] = (q[n,k] - z[n,k / g]) s[n,k / g],  q 0 .. 15, two codes a byte, 2i in the low nibble
//   C[m,n] = sum_groups s (sum_{k in group} x[m,k] (q - z))
//
// Bound by streaming the codes, and by the start of each workgroup; the vector unit, which has to take
// every code apart, is busy for a fifth to a half of the time. A weight's 16 rows and 128 columns are one 16-byte
// load a lane (lane (kq, n): row n, 32 codes). A wave takes one tile (16 weight rows; of the MoE's first product
// gate and up tiles in turn) and one of KS parts of K and streams it in bodies of 512 columns: the loads of the
// next body are in flight while this one's are used, each issued as its register becomes free. A workgroup is
// 8 waves: 8 / KS tiles by KS parts, whose sums meet in LDS in a fixed order. (Streamed alone, the codes of T 1,
// d 7168, I 2048, k 8 come at 5.3 TB/s with one wave a tile and 32 KB a CU in flight, 4.7 with two and 64 KB.)
//
// Whole passes: T 1, d 7168, I 2048, k 8 of 256 experts 49 us for 182 MB, where each of the two launches starts
// up for 5 to 7 us (x to LDS, the first codes); 48 tokens there on 32 of the experts with zero points 190 to
// 204 us, by the routing, for 602 MB; T 48, d 2048, I 1408, k 6 of 64 (bf16 rows) 103 us for 283 MB. (Fewer
// operations for the zero points, -z times the sums of x's bytes as the accumulators' start, changed nothing.)
//
//  k_w4_few   up to 4 rows of x a pass: integers. x is cut into 30-bit integers with one exponent for a
//    row's group (what is lost is below 2^-30 of the group's largest value, less than a float32 sum of the
//    group loses; bf16 values within 2^-22 of it, and float32 values within 2^-6, are exact) and those into four
//    signed bytes, which are rows 4 m .. 4 m + 3 of the 16-row int8 MFMA. A code less its zero point is a
//    byte: 4 (with zero points 7) vector operations for 8 codes. The bytes' sums are exact; a lane's
//    accumulators are those of row kq and column n, joined to the group's sum in float32.
//  k_w4_token the same, of all the experts of one token.
//  k_w4_rows  up to 16 rows: the bf16 MFMA. A nibble 0 .. 15 is, as an E4M3 byte, q 2^-9 (its first two
//    binades are evenly spaced), so one AND for four codes and a conversion for two give exact bf16
//    integers. x's products with a constant (-8, or 1, times -z) begin a group's float32 sum, which takes
//    the zero point off; the sum is scaled in float32.
//  k_w4_split the same for at most a tile a CU: x from the caches, up to 16 parts of K.
//
// The MoE's first launch writes H = silu(gate) up in float32, its second reads it (k_w4_rows: as three bf16
// planes, all of its bits); a third adds a token's experts in the order of its picks.
#include <algorithm>

#include "device_common.h"
#include "launch.h"
#include "mok.h"
#include "w4_shape.h"

namespace mok {
namespace {

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));

constexpr int W4_LOADS = W4_BODY / 128;
constexpr int W4_STEP = 256, W4_PARTS = 16;   // k_w4_split: columns of a wave's step, most parts of K
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
  int tiles, tpw, ks;                // tiles of a workgroup, parts of K
  int cap;                           // bytes of LDS for x
  int out_f32;
  // MoE
  const int32_t* idx;                // [T k]
  const float* tw;
  const int32_t *offsets, *route_ids;   // the plan (more than W4_SCAN routes), else NULL
  int64_t routes;
  int k, e0, El;
  const void* y_in;                  // k_w4_token: bf16 [T, N] or NULL; out: y bf16 [T, N]
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

// The same for halves of the wave: afterwards w[0], w[1] of every lane come from the first and second
// lane group (columns 0 .. 63 of 128), w[2], w[3] from the others.
MOK_DEV void swap2(uint32_t (&w)[4]) {
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const auto r = __builtin_amdgcn_permlane32_swap(w[j], w[2 + j], false, false);
    w[j] = r[0];
    w[2 + j] = r[1];
  }
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
typedef uint16_t u16_any __attribute__((aligned(1)));

// The scales and zero points of a wave's tile row (of the lane) for one step (of BODY columns).
template <int G, bool Z, int BODY = W4_BODY>
struct W4Groups {
  static constexpr int NG = BODY / G, ZW = (NG + 3) / 4;
  uint32_t s[NG / 2];
  uint32_t z[Z ? ZW : 1];
  MOK_DEV void load(const W4Mat& m, int64_t row, int K, int k) {
    const int ng = K / G, g0 = k / G;
    const uint16_t* sp = m.scales + row * ng + g0;
    const uint8_t* zp = Z ? m.zeros + row * ng + g0 : nullptr;
    if (k + BODY <= K) {
#pragma unroll
      for (int i = 0; i < NG / 2; ++i) s[i] = ((const u32_any*)sp)[i];
      if constexpr (Z)
#pragma unroll
        for (int i = 0; i < ZW; ++i) z[i] = NG < 4 ? *(const u16_any*)zp : ((const u32_any*)zp)[i];
    } else {
#pragma unroll
      for (int i = 0; i < NG / 2; ++i) {
        const uint32_t lo = g0 + 2 * i < ng ? sp[2 * i] : 0, hi = g0 + 2 * i + 1 < ng ? sp[2 * i + 1] : 0;
        s[i] = lo | (hi << 16);
      }
      if constexpr (Z)
#pragma unroll
        for (int i = 0; i < ZW; ++i) {
          z[i] = 0;
#pragma unroll
          for (int b = 0; b < 4 && 4 * i + b < NG; ++b)
            if (g0 + 4 * i + b < ng) z[i] |= (uint32_t)zp[4 * i + b] << (8 * b);
        }
    }
  }
  MOK_DEV float scale(int g) const {
    return __uint_as_float(g % 2 ? s[g / 2] & 0xFFFF0000u : s[g / 2] << 16);
  }
  MOK_DEV uint32_t zero_byte(int g) const { return (z[g / 4] >> (8 * (g % 4))) & 0xFF; }
  MOK_DEV float zero(int g) const { return Z ? (float)zero_byte(g) : 8.0f; }
};

// total += the products of 128 columns (load i of a body), whose x are the sums of a[0 .. A)[0 .. 3].
template <int G, bool Z, int S, int A, int BODY>
MOK_DEV void w4_step(const uint4 (&q)[S], const W4Groups<G, Z, BODY> (&gr)[S], int i, const bf16x8_t (&a)[A][4],
                     f32x4_t (&total)[S]) {
  constexpr int J = G < 128 ? G / 32 : 4;            // instructions of a group
  const uint32_t c = Z ? 0x3F803F80u : 0xC100C100u;  // 1 or -8
  const bf16x8_t cv = __builtin_bit_cast(bf16x8_t, make_uint4(c, c, c, c));
  uint32_t w[S][4];
#pragma unroll
  for (int s = 0; s < S; ++s) {
    w[s][0] = q[s].x; w[s][1] = q[s].y; w[s][2] = q[s].z; w[s][3] = q[s].w;
    if constexpr (G < 128) transpose4(w[s]);
  }
#pragma unroll
  for (int j0 = 0; j0 < 4; j0 += J) {
    const int g = (128 * i + 32 * j0) / G;
    f32x4_t x = {0, 0, 0, 0};
#pragma unroll
    for (int j = j0; j < j0 + J; ++j)
#pragma unroll
      for (int n = 0; n < A; ++n) x = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[n][j], cv, x, 0, 0, 0);
#pragma unroll
    for (int s = 0; s < S; ++s) {
      f32x4_t acc = x;
      if constexpr (Z) acc *= -gr[s].zero(g);
#pragma unroll
      for (int j = j0; j < j0 + J; ++j) {
        const bf16x8_t b = unpack8(w[s][j]);
#pragma unroll
        for (int n = 0; n < A; ++n) acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[n][j], b, acc, 0, 0, 0);
      }
      const float sc = gr[s].scale(g);
#pragma unroll
      for (int e = 0; e < 4; ++e) total[s][e] = fmaf(acc[e], sc, total[s][e]);
    }
  }
}

// The rows of an expert slot (MoE), found by every wave for itself (the same values): false if none.
struct W4Rows {
  int64_t expert = 0, count = 0, plan_at = 0;
  const int32_t* ids = nullptr;      // the plan's, or NULL: list
  const int16_t* list = nullptr;
  MOK_DEV bool find(const W4Args& p, int slot, int16_t* own) {
    const int lane = lane_id();
    if (p.offsets) {
      expert = slot;
      plan_at = p.offsets[expert];
      count = p.offsets[expert + 1] - plan_at;
      ids = p.route_ids;
      return count > 0;
    }
    // more local experts than routes: a slot is a route, and serves its expert if no earlier route
    // names it; otherwise a slot is an expert
    const bool by_route = p.routes < p.El;
    int n = 0;
    if (p.routes <= 64) {                  // one load
      const int32_t mine = lane < p.routes ? p.idx[lane] : -1;
      const int e = by_route ? __builtin_amdgcn_readlane(mine, slot) : p.e0 + slot;
      if (e < p.e0 || e >= p.e0 + p.El) return false;
      expert = e - p.e0;
      const bool hit = mine == e && lane < p.routes;
      const uint64_t mask = ballot(hit);
      if (by_route && __ffsll((unsigned long long)mask) - 1 < slot) return false;
      // every wave writes the list for itself (the same values), so that none waits
      if (hit) own[__popcll(mask & lanemask_lt())] = (int16_t)lane;
      n = __popcll(mask);
    } else {
      const int e = by_route ? uniform(p.idx[slot]) : p.e0 + slot;
      if (e < p.e0 || e >= p.e0 + p.El) return false;
      expert = e - p.e0;
      for (int r0 = 0; r0 < (int)p.routes; r0 += 256) {
        bool hit[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int r = r0 + 64 * q + lane;
          hit[q] = r < p.routes && p.idx[r] == e;
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int r = r0 + 64 * q;
          const uint64_t mask = ballot(hit[q]);
          if (by_route && n == 0 && mask && r + __ffsll((unsigned long long)mask) - 1 < slot) return false;
          if (hit[q]) own[n + __popcll(mask & lanemask_lt())] = (int16_t)(r + lane);
          n += __popcll(mask);
        }
      }
    }
    count = n;
    list = own;
    wave_sync();
    return n > 0;
  }
  MOK_DEV int32_t route(int64_t m) const { return ids ? ids[plan_at + m] : (int32_t)list[m]; }
};

// Row of x of the pass's row m: a token, or a route.
template <int MODE>
MOK_DEV int64_t w4_x_row(const W4Args& p, const W4Rows& rows, int64_t m) {
  if constexpr (MODE == W4_DENSE) return m;
  else if constexpr (MODE == W4_UP) return rows.route(m) / p.k;
  else return rows.route(m);
}

// A result v of row m (of rows) and column n.
template <int MODE, int S>
MOK_DEV void w4_store(const W4Args& p, const W4Rows& rows, int64_t m, int n, const float (&v)[S]) {
  if constexpr (MODE == W4_DENSE) {
    if (p.out_f32) ((float*)p.out)[m * p.N + n] = v[0];
    else ((bf16_t*)p.out)[m * p.N + n] = f32_to_bf16(v[0]);
  } else if constexpr (MODE == W4_UP) {
    ((float*)p.out)[(int64_t)rows.route(m) * p.N + n] = silu(v[0]) * v[S - 1];
  } else {
    const int64_t r = rows.route(m);
    ((float*)p.out)[r * p.N + n] = p.tw[r] * v[0];
  }
}

// The parts' sums of the workgroup's tiles, in order: red [wave][S][16 rows][16 columns]. PL > 1: row m's are those
// of row m and of row lo_row + m.
template <int MODE, int S, int PL>
MOK_DEV void w4_join(const W4Args& p, const W4Rows& rows, const float* red, int64_t m0, int n_rows,
                     int lo_row, int t0, int nt) {
  for (int o = threadIdx.x; o < n_rows * nt * 16; o += blockDim.x) {
    const int m = o / (nt * 16), c = o - m * (nt * 16), n = t0 * 16 + c;
    float v[S];
#pragma unroll
    for (int s = 0; s < S; ++s) {
      v[s] = 0.0f;
      for (int w = 0; w < p.ks; ++w) {
        const float* r = red + (((c >> 4) * p.ks + w) * S + s) * 256 + m * 16 + (c & 15);
        v[s] += r[0];
        if constexpr (PL > 1) v[s] += r[lo_row * 16];
      }
    }
    if (n < p.N) w4_store<MODE, S>(p, rows, m0 + m, n, v);
  }
}

// A wave's place: its tile's codes and its lane's row in them.
template <int S>
struct W4Tile {
  const uint8_t* code[S];
  uint32_t row_at, row_end;          // the lane's first bytes of a body; the last 16 bytes of its row
  int64_t row;
  MOK_DEV W4Tile(const W4Mat* w, int N, int K, int64_t expert, int n0) {
    const int lane = lane_id(), lr = min(lane & 15, N - 1 - n0);
    row = expert * N + n0 + lr;
#pragma unroll
    for (int s = 0; s < S; ++s) code[s] = w[s].codes + (expert * N + n0) * (int64_t)(K / 2);
    row_at = lr * (uint32_t)(K / 2) + 16 * (lane >> 4);
    row_end = lr * (uint32_t)(K / 2) + K / 2 - 16;
  }
  // load i of the body at column k; past K, where x is zero, the row's last codes
  MOK_DEV uint4 load(int s, int i, int k) const {
    return *(const uint4*)(code[s] + min(row_at + (uint32_t)(k / 2 + 64 * i), row_end));
  }
};

typedef int i32x4_t __attribute__((ext_vector_type(4)));

// 8 codes of a word less their zero point as bytes, the even ones, then the odd ones; without zero points
// (z the constant 8) times 16, which x's exponents take off.
template <bool Z>
MOK_DEV void code_bytes(uint32_t w, uint32_t zc, int& even, int& odd) {
  if constexpr (Z) {                                   // 0x80 + q - z carries into no other byte
    even = (int)(((w & 0x0F0F0F0Fu) + zc) ^ 0x80808080u);
    odd = (int)((((w >> 4) & 0x0F0F0F0Fu) + zc) ^ 0x80808080u);
  } else {                                             // q ^ 8 is q - 8 in two's complement
    w ^= 0x88888888u;
    even = (int)((w << 4) & 0xF0F0F0F0u);
    odd = (int)(w & 0xF0F0F0F0u);
  }
}

// The bytes of n as signed digits, -128 .. 127 each: half a place's worth goes to every place but the highest.
MOK_DEV uint32_t signed_bytes(int n) { return ((uint32_t)n + 0x00808080u) ^ 0x00808080u; }

// The least bytes of four words (the first's lowest), .., their highest.
MOK_DEV void bytes_by_place(uint32_t a, uint32_t b, uint32_t c, uint32_t d, uint32_t& p0, uint32_t& p1, uint32_t& p2,
                            uint32_t& p3) {
  const uint32_t ab = __builtin_amdgcn_perm(b, a, 0x05010400u), AB = __builtin_amdgcn_perm(b, a, 0x07030602u);
  const uint32_t cd = __builtin_amdgcn_perm(d, c, 0x05010400u), CD = __builtin_amdgcn_perm(d, c, 0x07030602u);
  p0 = __builtin_amdgcn_perm(cd, ab, 0x05040100u);
  p1 = __builtin_amdgcn_perm(cd, ab, 0x07060302u);
  p2 = __builtin_amdgcn_perm(CD, AB, 0x05040100u);
  p3 = __builtin_amdgcn_perm(CD, AB, 0x07060302u);
}

// x's rows in LDS, as bytes: [rows][4][ck + 16], then the groups' exponents [rows][ck / G]. XF: 16 bytes that
// 8 values take (bf16: 1, float32: 2).
template <int G, bool Z, int XF>
struct W4Bytes {
  static constexpr int XU = 2;         // units of 8 values that a thread has in flight
  static constexpr int SHIFT = (Z ? 156 : 160) - 16;   // of an exponent: the integers' place, 16, the sums' 65536
  int8_t* xb;
  const void* x;
  int K, n_rows, ck, ld, ng, cw, units;
  float* ex;
  uint4 xv[XU][XF];
  MOK_DEV W4Bytes(int8_t* lds, const void* x_, int K_, int rows, int ck_)
      : xb(lds), x(x_), K(K_), n_rows(rows), ck(ck_), ld(ck_ + 16), ng(ck_ / G), cw(ck_ / 8), units(rows * (ck_ / 8)),
        ex((float*)(lds + rows * 4 * (ck_ + 16))) {}
  // the columns c ck .. : row_of(r) is where row r lies in x, in rows
  template <class Row> MOK_DEV void load(int c, int u0, Row&& row_of) {
#pragma unroll
    for (int j = 0; j < XU; ++j) {
      const int u = u0 + j * (int)blockDim.x, r = min(u / cw, n_rows - 1), k = c * ck + (u - r * cw) * 8;
      const int64_t at = (int64_t)row_of(r) * K + min(k, K - 8);
#pragma unroll
      for (int i = 0; i < XF; ++i) {
        const uint4 v = XF == 1 ? *(const uint4*)((const bf16_t*)x + at) : *(const uint4*)((const float*)x + at + 4 * i);
        xv[j][i] = k < K ? v : make_uint4(0, 0, 0, 0);
      }
    }
  }
  // A group is G / 8 neighbouring lanes (a row's units fill whole waves).
  MOK_DEV void store(int u0) {
#pragma unroll
    for (int j = 0; j < XU; ++j) {
      const int u = u0 + j * (int)blockDim.x;
      if (u >= units) break;
      const int r = u / cw, o = (u - r * cw) * 8;
      float v[8];
      const uint4 q = xv[j][0];
      if constexpr (XF == 1) {
        const uint32_t t[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[2 * i] = __uint_as_float(t[i] << 16);
          v[2 * i + 1] = __uint_as_float(t[i] & 0xFFFF0000u);
        }
      } else {
        const uint4 h = xv[j][XF - 1];
        const uint32_t t[8] = {q.x, q.y, q.z, q.w, h.x, h.y, h.z, h.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(t[i]);
      }
      uint32_t top = 0;                              // exponent field of the largest; 255: not finite
#pragma unroll
      for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(v[i]) & 0x7FFFFFFFu);
#pragma unroll
      for (int m = 1; m < G / 8; m <<= 1) top = max(top, (uint32_t)__shfl_xor((int)top, m, kWave));
      const int e = max((int)(top >> 23), 1);
      if (u % (G / 8) == 0)
        ex[r * ng + o / G] = e == 255 ? NAN : __builtin_amdgcn_ldexpf(1.0f, e - SHIFT);
      uint32_t n[8], d[4][2];
#pragma unroll
      for (int i = 0; i < 8; ++i)                    // |v| < 2^30
        n[i] = e == 255 ? 0 : signed_bytes((int)rintf(__builtin_amdgcn_ldexpf(v[i], 156 - e)));
#pragma unroll
      for (int h = 0; h < 2; ++h) bytes_by_place(n[h], n[2 + h], n[4 + h], n[6 + h], d[3][h], d[2][h], d[1][h], d[0][h]);
#pragma unroll
      for (int q = 0; q < 4; ++q) *(uint2*)(xb + (r * 4 + q) * ld + o) = make_uint2(d[q][0], d[q][1]);
    }
  }
  // Chunk c into LDS; loaded: the first units are in xv.
  template <class Row> MOK_DEV void fill(int c, bool loaded, Row&& row_of) {
    for (int u = threadIdx.x;;) {
      if (!loaded || u != (int)threadIdx.x) load(c, u, row_of);
      store(u);
      u += XU * (int)blockDim.x;
      if (u - (int)threadIdx.x >= units) break;
    }
  }
  // Where the lane's row of the MFMA lies: byte ln % 4 of row first + ln / 4 (rows past the last are not looked
  // at), with its columns' place in 128; and the exponents of row first + kq.
  MOK_DEV const int8_t* fragment(int first) const {
    const int kq = lane_id() >> 4, ln = lane_id() & 15;
    return xb + (min(first + (ln >> 2), n_rows - 1) * 4 + (ln & 3)) * ld +
           (G == 128 ? 32 * kq : G == 64 ? 32 * (kq & 1) + 16 * (kq >> 1) : 8 * kq);
  }
  MOK_DEV const float* exponents(int first) const { return ex + min(first + (lane_id() >> 4), n_rows - 1) * ng; }
};

// total += a body's products; xl, xe: x's place at its first column. The registers q take the codes of the body at
// column kn of tile w as they become free. A group's sum times its exponent is exact (short of float32's largest
// value), so that a large scale of small values, or a small one, loses nothing.
template <int G, bool Z>
MOK_DEV void w4_few_body(uint4 (&q)[W4_LOADS], const W4Groups<G, Z>& gr, const int8_t* xl, const float* xe,
                         const W4Tile<1>& w, int kn, float& total) {
#pragma unroll
  for (int l = 0; l < W4_LOADS; ++l) {
    uint32_t t[4] = {q[l].x, q[l].y, q[l].z, q[l].w};
    if constexpr (G == 64) swap2(t);
    if constexpr (G == 32) transpose4(t);
    constexpr int NG = 128 / G, W = 4 / NG;          // groups of the load, words of a group
    i32x4_t acc[NG];
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      const uint32_t zc = Z ? 0x80808080u - gr.zero_byte(l * NG + g) * 0x01010101u : 0;
      acc[g] = i32x4_t{0, 0, 0, 0};
#pragma unroll
      for (int j = 0; j < W; j += W > 1 ? 2 : 1) {
        int lo[2], hi[2];
        code_bytes<Z>(t[W * g + j], zc, lo[0], hi[0]);
        if constexpr (W > 1) {
          code_bytes<Z>(t[W * g + j + 1], zc, lo[1], hi[1]);
          const i32x4_t a = *(const i32x4_t*)(xl + 128 * l + (G == 128 ? 8 * j : 64 * g));
          acc[g] = __builtin_amdgcn_mfma_i32_16x16x64_i8(a, i32x4_t{lo[0], hi[0], lo[1], hi[1]}, acc[g], 0, 0, 0);
        } else {
          const long a = *(const long*)(xl + 128 * l + 32 * g);
          acc[g] = __builtin_amdgcn_mfma_i32_16x16x32_i8(a, (long)(uint32_t)lo[0] | ((long)hi[0] << 32), acc[g], 0, 0, 0);
        }
      }
    }
    q[l] = w.load(0, l, kn);
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      const float v = fmaf((float)((acc[g][2] << 8) + acc[g][3]), 1.0f / 65536, (float)((acc[g][0] << 8) + acc[g][1]));
      total = fmaf(v * xe[l * NG + g], gr.scale(l * NG + g), total);
    }
  }
}

// Workgroup (x, y): tpw tiles, rows y MR .. (dense) or expert slot y (MoE).
template <int G, bool Z, int MODE>
__global__ __launch_bounds__(64 * W4_MAXW, 4) void k_w4_few(const W4Args p) {
  constexpr int S = MODE == W4_UP ? 2 : 1, MR = 4;
  extern __shared__ __attribute__((aligned(16))) int8_t xb[];
  __shared__ float red[W4_MAXW * 64];
  __shared__ int16_t list[MODE == W4_DENSE ? 1 : W4_SCAN];
  const int tid = threadIdx.x, lane = lane_id(), wv = uniform(tid >> 6);
  W4Rows rows;
  if constexpr (MODE == W4_DENSE) rows.count = p.M;
  else if (!rows.find(p, blockIdx.y, list)) return;
  // S tiles, of gate and up, are a pair's; a workgroup has whole pairs
  const int tile = wv / p.ks, part = wv - tile * p.ks, t0 = blockIdx.x * (p.tpw / S);
  const int nt = min(p.tpw / S, p.tiles - t0);                          // pairs of the workgroup
  const bool idle = tile >= nt * S;
  const W4Mat& mat = p.w[S == 2 ? tile % 2 : 0];
  const W4Tile<1> w(&mat, p.N, p.K, rows.expert, idle ? 0 : (t0 + tile / S) * 16);
  const int64_t m_first = MODE == W4_DENSE ? (int64_t)blockIdx.y * MR : 0;
  const int64_t m_end = MODE == W4_DENSE ? min(rows.count, m_first + MR) : rows.count;
  for (int64_t m0 = m_first; m0 < m_end; m0 += MR) {
    const int n_rows = (int)min((int64_t)MR, m_end - m0);
    // bodies of a chunk and part; chunks
    const int bodies = (p.K + W4_BODY - 1) / W4_BODY, bw = W4_BODY * p.ks;
    const int bpc = w4_bodies(bodies, p.ks, p.cap, w4_body_bytes(true, G, 1), n_rows);
    const int ck = bpc * bw, chunks = (p.K + ck - 1) / ck;
    auto column = [&](int c, int b) { return min(c * ck + (part * bpc + b) * W4_BODY, p.K); };
    auto row_of = [&](int r) { return w4_x_row<MODE>(p, rows, m0 + r); };
    W4Bytes<G, Z, MODE == W4_DOWN ? 2 : 1> x(xb, p.x, p.K, n_rows, ck);
    uint4 q[W4_LOADS];
    W4Groups<G, Z> gr;
    x.load(0, tid, row_of);                            // x first: waiting for it must not wait for the codes
    __builtin_amdgcn_sched_barrier(0);
    if (!idle) {
      gr.load(mat, w.row, p.K, column(0, 0));
#pragma unroll
      for (int l = 0; l < W4_LOADS; ++l) q[l] = w.load(0, l, column(0, 0));
    }
    __builtin_amdgcn_sched_barrier(0);
    const int8_t* const xl = x.fragment(0) + part * bpc * W4_BODY;
    const float* const xe = x.exponents(0) + part * bpc * (W4_BODY / G);
    float total = 0.0f;
    for (int c = 0; c < chunks; ++c) {
      __syncthreads();                                 // the chunk (or the sums) before is done with
      x.fill(c, c == 0, row_of);
      __syncthreads();
      if (idle) continue;
      for (int b = 0; b < bpc; ++b) {
        // the next body (behind the last, and past K: the row's last codes once more)
        const int kn = b + 1 < bpc ? column(c, b + 1) : column(c + 1, 0);
        W4Groups<G, Z> gn;
        gn.load(mat, w.row, p.K, kn);
        w4_few_body<G, Z>(q, gr, xl + b * W4_BODY, xe + b * (W4_BODY / G), w, kn, total);
        gr = gn;
      }
    }
    red[wv * 64 + lane] = total;
    __syncthreads();
    // the parts' sums, in order
    for (int o = tid; o < n_rows * nt * 16; o += blockDim.x) {
      const int m = o / (nt * 16), c = o - m * (nt * 16), n = t0 * 16 + c, t = c >> 4;
      float v[S];
#pragma unroll
      for (int s = 0; s < S; ++s) {
        v[s] = 0.0f;
        for (int j = 0; j < p.ks; ++j) v[s] += red[((t * S + s) * p.ks + j) * 64 + m * 16 + (c & 15)];
      }
      if (n < p.N) w4_store<MODE, S>(p, rows, m0 + m, n, v);
    }
  }
}

// The down projection of a token whose experts hardly any other token shares: workgroup (x, y) takes tile x of
// all the k <= 8 routes of token y, a wave a route (and part of K), and writes y itself, which saves P's way
// through memory and a launch (T 1, d 7168, I 2048, k 8 of 256 experts: 51.5 -> 49 us; d 2048, I 1408, k 6 of
// 64: 20.3 -> 18.0).
template <int G, bool Z>
__global__ __launch_bounds__(64 * W4_MAXW, 4) void k_w4_token(const W4Args p) {
  extern __shared__ __attribute__((aligned(16))) int8_t xb[];
  __shared__ float red[W4_MAXW * 16];
  const int tid = threadIdx.x, lane = lane_id(), wv = uniform(tid >> 6);
  const int j = wv / p.ks, part = wv - j * p.ks;
  const int64_t t = blockIdx.y;
  const int n0 = blockIdx.x * 16;
  // bodies of a chunk and part; chunks
  const int bodies = (p.K + W4_BODY - 1) / W4_BODY, bw = W4_BODY * p.ks;
  const int bpc = w4_bodies(bodies, p.ks, p.cap, w4_body_bytes(true, G, 1), p.k);
  const int ck = bpc * bw, chunks = (p.K + ck - 1) / ck;
  auto column = [&](int c, int b) { return min(c * ck + (part * bpc + b) * W4_BODY, p.K); };
  auto row_of = [&](int r) { return t * p.k + r; };
  const int e = uniform(p.idx[t * p.k + j]) - p.e0;
  const bool idle = e < 0 || e >= p.El;
  W4Bytes<G, Z, 2> x(xb, p.x, p.K, p.k, ck);
  x.load(0, tid, row_of);                              // (rows of routes to other experts hold anything)
  __builtin_amdgcn_sched_barrier(0);
  uint4 q[W4_LOADS];
  W4Groups<G, Z> gr;
  const W4Tile<1> w(p.w, p.N, p.K, idle ? 0 : e, n0);
  if (!idle) {
    gr.load(p.w[0], w.row, p.K, column(0, 0));
#pragma unroll
    for (int l = 0; l < W4_LOADS; ++l) q[l] = w.load(0, l, column(0, 0));
  }
  __builtin_amdgcn_sched_barrier(0);
  const int8_t* const xl = x.fragment(j) + part * bpc * W4_BODY;
  const float* const xe = x.exponents(j) + part * bpc * (W4_BODY / G);
  float total = 0.0f;
  for (int c = 0; c < chunks; ++c) {
    if (c > 0) __syncthreads();
    x.fill(c, c == 0, row_of);
    __syncthreads();
    if (idle) continue;
    for (int b = 0; b < bpc; ++b) {
      const int kn = b + 1 < bpc ? column(c, b + 1) : column(c + 1, 0);
      W4Groups<G, Z> gn;
      gn.load(p.w[0], w.row, p.K, kn);
      w4_few_body<G, Z>(q, gr, xl + b * W4_BODY, xe + b * (W4_BODY / G), w, kn, total);
      gr = gn;
    }
  }
  // the wave's route is row 0 of its MFMA: lanes 0 .. 15 have its columns
  if (lane < 16) red[wv * 16 + lane] = idle ? 0.0f : total;
  __syncthreads();
  const int n = n0 + tid;
  if (tid < 16 && n < p.N) {
    float v = p.y_in ? bf16_to_f32(((const bf16_t*)p.y_in)[t * p.N + n]) : 0.0f;
    for (int r = 0; r < p.k; ++r) {
      const int er = p.idx[t * p.k + r] - p.e0;
      if (er < 0 || er >= p.El) continue;
      float s = 0.0f;
      for (int i = 0; i < p.ks; ++i) s += red[(r * p.ks + i) * 16 + tid];
      v += p.tw[t * p.k + r] * s;
    }
    ((bf16_t*)p.out)[t * p.N + n] = f32_to_bf16(v);
  }
}

// The same for up to 16 rows of the MFMA, x in LDS for the whole workgroup. H, which is float32, is three bf16
// values, the bits of its significand in order: 8 rows of H are the MFMA's rows m (first) and 8 + m (second),
// and of another MFMA on the same codes half the third in both. The accumulators' rows m and 8 + m add up.
template <int G, bool Z, int MODE>
__global__ __launch_bounds__(64 * W4_MAXW) void k_w4_rows(const W4Args p) {
  constexpr int S = MODE == W4_UP ? 2 : 1, PL = MODE == W4_DOWN ? 3 : 1;
  constexpr int MR = PL == 1 ? 16 : 8, A = PL == 1 ? 1 : 2;          // rows of a pass, MFMAs of a fragment
  extern __shared__ __attribute__((aligned(16))) bf16_t xs[];   // [rows PL][ck + 8]; then the waves' sums
  __shared__ int16_t list[MODE == W4_DENSE ? 1 : W4_SCAN];
  const int tid = threadIdx.x, lane = lane_id(), wv = uniform(tid >> 6), kq = lane >> 4, ln = lane & 15;
  W4Rows rows;
  if constexpr (MODE == W4_DENSE) rows.count = p.M;
  else if (!rows.find(p, blockIdx.y, list)) return;
  const int tile = wv / p.ks, part = wv - tile * p.ks, t0 = blockIdx.x * p.tpw;
  const int nt = min(p.tpw, p.tiles - t0);
  const bool idle = tile >= nt;
  const W4Tile<S> w(p.w, p.N, p.K, rows.expert, idle ? 0 : (t0 + tile) * 16);
  const int64_t m_first = MODE == W4_DENSE ? (int64_t)blockIdx.y * MR : 0;
  const int64_t m_end = MODE == W4_DENSE ? min(rows.count, m_first + MR) : rows.count;
  for (int64_t m0 = m_first; m0 < m_end; m0 += MR) {
    const int n_rows = (int)min((int64_t)MR, m_end - m0);
    // bodies of a chunk and part; chunks
    const int bodies = (p.K + W4_BODY - 1) / W4_BODY, bw = W4_BODY * p.ks;
    const int bpc = w4_bodies(bodies, p.ks, p.cap, w4_body_bytes(false, G, PL), n_rows);
    const int ck = bpc * bw, chunks = (p.K + ck - 1) / ck, ld = ck + 8;
    auto column = [&](int c, int b) { return c * ck + (part * bpc + b) * W4_BODY; };
    // x's columns c ck .. to LDS, 8 at a time, in unpack8's order: XU loads of a thread in flight
    constexpr int XU = PL == 1 ? 4 : 2, XF = PL == 1 ? 1 : 2;          // XF: 16 bytes of 8 values
    const int cw = ck / 8, units = n_rows * cw;
    uint4 xv[XU][XF];
    auto x_load = [&](int c, int u0) {
#pragma unroll
      for (int j = 0; j < XU; ++j) {
        const int u = u0 + j * (int)blockDim.x, r = min(u / cw, n_rows - 1), k = c * ck + (u - r * cw) * 8;
        const int64_t at = w4_x_row<MODE>(p, rows, m0 + r) * p.K + min(k, p.K - 8);
#pragma unroll
        for (int i = 0; i < XF; ++i) {
          const uint4 v = PL == 1 ? *(const uint4*)((const bf16_t*)p.x + at) : *(const uint4*)((const float*)p.x + at + 4 * i);
          xv[j][i] = k < p.K ? v : make_uint4(0, 0, 0, 0);
        }
      }
    };
    auto x_store = [&](int u0) {
#pragma unroll
      for (int j = 0; j < XU; ++j) {
        const int u = u0 + j * (int)blockDim.x, r = u / cw;
        if (u >= units) break;
        bf16_t* const to = xs + r * ld + (u - r * cw) * 8;
        if constexpr (PL == 1) {
          *(bf16x8_t*)to = order8(xv[j][0]);
        } else {
          const uint4 a = xv[j][0], b = xv[j][XF - 1];
          const uint32_t w[8] = {a.x, a.z, b.x, b.z, a.y, a.w, b.y, b.w};
          uint32_t p[3][4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t t[3][2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {              // cut off, not rounded: the rest fits the next, exactly
              float v = __uint_as_float(w[2 * i + h]);
              t[0][h] = __float_as_uint(v) >> 16;
              v -= __uint_as_float(t[0][h] << 16);
              t[1][h] = __float_as_uint(v) >> 16;
              v -= __uint_as_float(t[1][h] << 16);
              t[2][h] = __float_as_uint(0.5f * v) >> 16;
            }
#pragma unroll
            for (int q = 0; q < 3; ++q) p[q][i] = t[q][0] | (t[q][1] << 16);
          }
#pragma unroll
          for (int q = 0; q < 3; ++q) *(uint4*)(to + q * n_rows * ld) = make_uint4(p[q][0], p[q][1], p[q][2], p[q][3]);
        }
      }
    };
    // the row of xs that is this lane's of the MFMA's 16 (those past the rows are not looked at)
    const bf16_t* const xl = xs + (PL > 1 ? min(ln & 7, n_rows - 1) + (ln >> 3) * n_rows : min(ln, n_rows - 1)) * ld;
    const int third = (PL > 1 ? 2 - (ln >> 3) : 0) * n_rows * ld;      // from there to H's third part
    uint4 q[W4_LOADS][S];
    W4Groups<G, Z> gr[S];
    f32x4_t total[S];
#pragma unroll
    for (int s = 0; s < S; ++s) total[s] = f32x4_t{0, 0, 0, 0};
    x_load(0, tid);                                    // x first: waiting for it must not wait for the codes
    __builtin_amdgcn_sched_barrier(0);
    if (!idle)
#pragma unroll
      for (int s = 0; s < S; ++s) {
        gr[s].load(p.w[s], w.row, p.K, min(column(0, 0), p.K));
#pragma unroll
        for (int l = 0; l < W4_LOADS; ++l) q[l][s] = w.load(s, l, column(0, 0));
      }
    __builtin_amdgcn_sched_barrier(0);
    for (int c = 0; c < chunks; ++c) {
      __syncthreads();                                 // the chunk (or the sums) before is done with
      for (int u = tid;;) {
        if (c > 0 || u != tid) x_load(c, u);
        x_store(u);
        u += XU * (int)blockDim.x;
        if (u - tid >= units) break;
      }
      __syncthreads();
      if (idle) continue;
      for (int b = 0; b < bpc; ++b) {
        // the next body (behind the last, and past K: the row's last codes once more)
        const int kn = min(b + 1 < bpc ? column(c, b + 1) : column(c + 1, 0), p.K);
        W4Groups<G, Z> gn[S];
#pragma unroll
        for (int s = 0; s < S; ++s) gn[s].load(p.w[s], w.row, p.K, kn);
        const bf16_t* const xb = xl + (part * bpc + b) * W4_BODY;
        bf16x8_t a[2][A][4];
        auto read = [&](int l) {
#pragma unroll
          for (int n = 0; n < A; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j)
              a[l & 1][n][j] = *(const bf16x8_t*)(xb + n * third + 128 * l + (G < 128 ? 32 * j + 8 * kq : 32 * kq + 8 * j));
        };
        read(0);
#pragma unroll
        for (int l = 0; l < W4_LOADS; ++l) {
          if (l + 1 < W4_LOADS) read(l + 1);
          w4_step<G, Z, S, A, W4_BODY>(q[l], gr, l, a[l & 1], total);
#pragma unroll
          for (int s = 0; s < S; ++s) q[l][s] = w.load(s, l, kn);
        }
#pragma unroll
        for (int s = 0; s < S; ++s) gr[s] = gn[s];
      }
    }
    __syncthreads();
    float* const red = (float*)xs;
    if (!idle)
#pragma unroll
      for (int s = 0; s < S; ++s)
#pragma unroll
        for (int e = 0; e < 4; ++e) red[(wv * S + s) * 256 + (4 * kq + e) * 16 + ln] = total[s][e];
    __syncthreads();
    w4_join<MODE, S, PL>(p, rows, red, m0, n_rows, 8, t0, nt);
  }
}

// The dense product of up to 16 rows with few tiles: a workgroup is one tile in up to 16 parts of K, and every
// wave loads its own x, whose fragments are 16 bytes a lane, from the caches: with one tile a workgroup LDS would
// be read once as well. A wave's step is W4_STEP columns; the next step's codes are in flight meanwhile.
template <int G, bool Z>
__global__ __launch_bounds__(64 * W4_PARTS) void k_w4_split(const W4Args p) {
  constexpr int L = W4_STEP / 128;
  __shared__ float red[W4_PARTS * 256];
  const int lane = lane_id(), part = uniform(threadIdx.x >> 6), kq = lane >> 4, ln = lane & 15;
  const int64_t m0 = (int64_t)blockIdx.y * 16;
  const int n_rows = (int)min((int64_t)16, p.M - m0), steps = (p.K + W4_STEP - 1) / W4_STEP;
  const int t0 = blockIdx.x, per = (steps + p.ks - 1) / p.ks, last = min(steps, (part + 1) * per);
  const W4Tile<1> w(p.w, p.N, p.K, 0, t0 * 16);
  const bf16_t* const x = (const bf16_t*)p.x + (m0 + min(ln, n_rows - 1)) * p.K;   // rows past the last: not looked at
  struct Codes {
    uint4 q[L][1];
    W4Groups<G, Z, W4_STEP> gr[1];
  };
  auto load = [&](Codes& t, int i) {                   // past K: the row's last codes once more
    const int k0 = min(i * W4_STEP, p.K);
    t.gr[0].load(p.w[0], w.row, p.K, k0);
#pragma unroll
    for (int l = 0; l < L; ++l) t.q[l][0] = w.load(0, l, k0);
  };
  f32x4_t total[1] = {{0, 0, 0, 0}};
  Codes now, next;
  if (part * per < last) load(now, part * per);
  for (int i = part * per; i < last; ++i) {
    uint4 v[L][4];
#pragma unroll
    for (int l = 0; l < L; ++l)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int k = i * W4_STEP + 128 * l + (G < 128 ? 32 * j + 8 * kq : 32 * kq + 8 * j);
        const uint4 u = *(const uint4*)(x + min(k, p.K - 8));
        v[l][j] = k < p.K ? u : make_uint4(0, 0, 0, 0);
      }
    load(next, i + 1);
#pragma unroll
    for (int l = 0; l < L; ++l) {
      bf16x8_t a[1][4];
#pragma unroll
      for (int j = 0; j < 4; ++j) a[0][j] = order8(v[l][j]);
      w4_step<G, Z, 1, 1, W4_STEP>(now.q[l], now.gr, l, a, total);
    }
    now = next;
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) red[part * 256 + (4 * kq + e) * 16 + ln] = total[0][e];
  __syncthreads();
  w4_join<W4_DENSE, 1, 1>(p, W4Rows{}, red, m0, n_rows, 0, t0, 1);
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

hipError_t launch_w4_split(W4Args a, int g, int64_t slots, hipStream_t s) {
  const int steps = (a.K + W4_STEP - 1) / W4_STEP;
  const int per = (steps + W4_PARTS - 1) / W4_PARTS;
  a.ks = (steps + per - 1) / per;
  const dim3 grid((unsigned)a.tiles, (unsigned)slots), block(64 * a.ks);
  auto go = [&](auto G) {
    launch_k(a.w[0].zeros ? k_w4_split<G(), true> : k_w4_split<G(), false>, grid, block, 0, s, nullptr, nullptr, a);
  };
  if (g == 32) go(std::integral_constant<int, 32>{});
  else if (g == 64) go(std::integral_constant<int, 64>{});
  else go(std::integral_constant<int, 128>{});
  return hipGetLastError();
}

// tokens: the rows of an expert (or the product) whose tokens name it once; most: those that it can have; mean:
// how many it has on average.
template <int MODE>
hipError_t launch_w4(W4Args a, int g, int64_t slots, int64_t tokens, int64_t most, double mean, hipStream_t s) {
  constexpr int S = MODE == W4_UP ? 2 : 1, PL = MODE == W4_DOWN ? 3 : 1;
  // one in twenty experts of 2 rows has a second pass. Whole passes, bf16 rows and integers: 64 experts of d 2048,
  // I 1408, k 6 at a mean of 1.5, 2, 2.5 and 4 rows 83 and 72, 87 and 82, 90 and 90, 102 and 113 us; 32 of 256 of
  // d 7168, I 2048, k 8 with zero points at 1.5, 2, 2.5 and 4: 200 and 190, 225 and 214, 245 and 250, 297 and 330
  const bool few = tokens <= 4 || mean <= 2.0;
  a.tiles = (a.N + 15) / 16;
  const int mr = few ? 4 : PL > 1 ? 8 : 16;
  if (MODE == W4_DENSE) slots = (a.M + mr - 1) / mr;
  // at most a tile a CU (13 and 5 rows, N 4096, K 7168, groups of 32 with zero points: 20.5 -> 12.2 and 11.1 ->
  // 9.4 us; 13 rows, N 8192, with two: 21.8 -> 22.4, groups of 128 16.4 -> 19.3)
  if (MODE == W4_DENSE && !few && a.tiles * slots <= 256) return launch_w4_split(a, g, slots, s);
  const int pair = few ? S : 1;                   // gate and up tiles come in pairs of waves
  const W4Shape f = w4_shape(few, g, PL, a.K, (int64_t)a.tiles * pair * slots, pair, few ? 0 : S * 1024,
                             (int)std::min<int64_t>(tokens, mr), (int)std::min<int64_t>(most, mr));
  a.ks = f.ks; a.tpw = f.tpw; a.cap = f.cap;
  const dim3 grid((unsigned)((a.tiles * pair + a.tpw - 1) / a.tpw), (unsigned)slots), block(64 * a.tpw * a.ks);
  auto go = [&](auto G, auto Z) {
    launch_k(few ? k_w4_few<G(), Z(), MODE> : k_w4_rows<G(), Z(), MODE>, grid, block, (uint32_t)f.lds, s, nullptr,
             nullptr, a);
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

hipError_t launch_w4_token(W4Args a, int g, int64_t T, hipStream_t s) {
  a.tiles = (a.N + 15) / 16;
  const W4Shape f = w4_token_shape(g, a.K, a.k);
  a.ks = f.ks; a.cap = f.cap;
  const dim3 grid((unsigned)a.tiles, (unsigned)T), block(64 * a.k * a.ks);
  auto go = [&](auto G) {
    launch_k(a.w[0].zeros ? k_w4_token<G(), true> : k_w4_token<G(), false>, grid, block, (uint32_t)f.lds, s, nullptr,
             nullptr, a);
  };
  if (g == 32) go(std::integral_constant<int, 32>{});
  else if (g == 64) go(std::integral_constant<int, 64>{});
  else go(std::integral_constant<int, 128>{});
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
  if (!a || a->T < 0 || a->T >= (int64_t)1 << 31 || a->d < 1 || a->I < 1 || !group_ok(a->group)) return MOK_EINVAL;
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
  if (rows >= (int64_t)1 << 32) return MOK_EUNSUPPORTED;
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
  if (M > 1 << 20 || N > 1 << 26) return MOK_EUNSUPPORTED;
  return launch_w4<W4_DENSE>(a, group, 0, M, M, (double)M, (hipStream_t)stream) == hipSuccess ? MOK_OK : MOK_EHIP;
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
  const int64_t slots = p.plan ? a.E_l : std::min<int64_t>(n, a.E_l);
  const double mean = (double)n / a.E;
  w.w[0] = {a.gate_codes, (const uint16_t*)a.gate_scales, a.gate_zeros};
  w.w[1] = {a.up_codes, (const uint16_t*)a.up_scales, a.up_zeros};
  w.x = a.x; w.out = ws + p.H; w.N = a.I; w.K = a.d;
  if (launch_w4<W4_UP>(w, a.group, slots, a.T, n, mean, s) != hipSuccess) return MOK_EHIP;
  w.w[0] = {a.down_codes, (const uint16_t*)a.down_scales, a.down_zeros};
  w.x = ws + p.H; w.N = a.d; w.K = a.I;
  // few routes an expert: nearly all of its tokens' products would be one row (mean 0.25: one in eight
  // experts that are picked serves two); and all experts here, or waves would be idle. Whole passes without and
  // with it: 128 experts of d 512, I 256, k 8 at a mean of 0.25 17.4 and 13.2 us; 64 of d 2048, I 1408, k 6 at 0.19
  // and 0.47 26.5 and 23.1, 40.3 and 38.2; 256 of d 7168, I 2048, k 8 at 0.03, 0.06, 0.12 and 0.25 51.5 and 48.8,
  // 87 and 87, 148 and 154, 259 and 284, where the weights that two tokens share count for more than a launch
  if (!p.plan && a.k <= W4_MAXW && a.E_l == a.E && mean <= 0.25) {
    w.out = a.y;
    w.y_in = a.y_in;
    return launch_w4_token(w, a.group, a.T, s) == hipSuccess ? MOK_OK : MOK_EHIP;
  }
  w.out = ws + p.P;
  if (launch_w4<W4_DOWN>(w, a.group, slots, a.T, n, mean, s) != hipSuccess) return MOK_EHIP;
  launch_k(k_w4_combine, dim3((unsigned)blocks), dim3(256), 0, s, nullptr, nullptr,
           (const float*)(ws + p.P), a.topk_idx, (const uint2*)a.y_in, a.T, a.k, a.e0, a.E_l, a.d / 4,
           (uint2*)a.y);
  return hipGetLastError() == hipSuccess ? MOK_OK : MOK_EHIP;
}

}  // extern "C"
