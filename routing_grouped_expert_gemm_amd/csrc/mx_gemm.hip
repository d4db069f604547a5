// Product of two microscaled operands: C[m,n] = sum_k A[m,k] B[n,k], A [M, K] and B [N, K] in
// MXFP8 (E4M3) or MXFP4 (E2M1), one E8M0 scale per 32 values along K, both in the layout that the
// mok_quantize_mx* entry points write (row-major codes and scales); C in bf16 or float32.
//
// Everything runs on the scaled MFMA 32x32x64, which takes the codes and the scales as they are
// and accumulates in float32. Its operands: a lane (h, r) = (lane / 32, lane % 32) carries row r
// and the scale of the instruction's 32-value block h. An E2M1 lane holds block h's 16 code
// bytes; an E4M3 lane holds 16 of the 32 values of block 0 (its half h) and 16 of block 1. K may
// be permuted freely as long as both operands agree, so the instructions of a step of 256 values
// pair block s with block 4 + s (s = 0 .. 3): lane half h then needs the scales 4 h .. 4 h + 3 of
// its row, one aligned word, and instruction s picks byte s of it (op_sel).
// B is the first operand, so a lane's accumulators hold 4 consecutive columns of C's row r.
//
// Two forms:
//  k_mx_tile  LDS tiles, for many rows: bound by the MFMA rate and its LDS feeding.
//  k_mx_rows  up to 64 rows (single tokens and small batches): bound by streaming B once.
#include <algorithm>
#include <utility>

#include "device_common.h"
#include "launch.h"
#include "lds_dma.h"
#include "mok.h"

namespace mok {
namespace {

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
constexpr int F8 = 0, F4 = 4;                     // the MFMA's operand format codes

template <int F> constexpr int code_bytes(int n) { return F == F8 ? n : n / 2; }

struct MxArgs {
  const uint8_t *a, *as, *b, *bs;
  void* c;                 // bf16 or float32 [M, N]; partial sums: float32 [splits, M, N]
  int M, N, K;
  int out_f32;
  int tiles_m, tiles_n;
  int splits;              // K ranges (grid z of k_mx_tile)
  int steps_per_split;
};

template <int N, class F, int... I>
MOK_DEV void static_for_(F&& f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>{}), ...);
}
template <int N, class F> MOK_DEV void static_for(F&& f) {
  static_for_<N>(f, std::make_integer_sequence<int, N>{});
}

// A lane's operand of one MFMA: 16 bytes (E2M1) or 32 (E4M3).
template <int F> struct Frag {
  uint4 q[F == F8 ? 2 : 1];
  MOK_DEV void zero() {
    q[0] = make_uint4(0, 0, 0, 0);
    if constexpr (F == F8) q[1] = make_uint4(0, 0, 0, 0);
  }
  MOK_DEV i32x8_t regs() const {
    i32x8_t v = {0, 0, 0, 0, 0, 0, 0, 0};
    v[0] = q[0].x; v[1] = q[0].y; v[2] = q[0].z; v[3] = q[0].w;
    if constexpr (F == F8) { v[4] = q[1].x; v[5] = q[1].y; v[6] = q[1].z; v[7] = q[1].w; }
    return v;
  }
};

template <int FA, int FB, int SEL>
MOK_DEV f32x16_t mfma(const Frag<FB>& b, const Frag<FA>& a, f32x16_t acc, uint32_t bsc,
                      uint32_t asc) {
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(b.regs(), a.regs(), acc, FB, FA, SEL,
                                                         (int)bsc, SEL, (int)asc);
}

// The instruction adds the products of a 32-value block on a grid 13 bits below the largest sum of
// two exponents (a subnormal has its type's least exponent) and cuts each product off there, towards
// zero, then rounds to float32 (so measured for every pair of two values). A block thus loses less
// than 32 2^-13 = 2^-8 of its largest product, subnormals counted as their type's smallest normal.
// E2M1 products span 8 bits and are exact. An E4M3 operand spans 18 binades: on normal rows two of
// them leave 1.5e-5 of the result's norm, one beside an E2M1 operand 5e-6. In the mixed pair (X) the
// E4M3 operand can be split at 4 into two, and the products are two instructions, both exact:
//   below 4: exponents -6 .. 1, multiples of 2^-9; with E2M1 (exponents 0 .. 2, multiples of 1/2) the
//     products are multiples of 2^-10 and the grid is at most 2^(1 + 2 - 13);
//   4 to 448: exponents 2 .. 8, products multiples of 2^-2, the grid at most 2^(8 + 2 - 13).
// (Split at 8, values below 2^-6 lost their last bit beside 4 to 7.5. Two E4M3 operands would need
// twelve instructions.) That is done for float32 results, and for up to 64 rows, where it costs next to
// nothing (MXFP8 x MXFP4, bf16 results, N 4096, K 7168, M 64: 20.5 and 21.4 us, M 1, N 7168, K 2048: 8.3
// and 8.4). Above, bf16 results take one instruction: two double the time (M 1000: 32 and 65 us, M 8192:
// 175 and 327), and 5e-6 is a 300th of what the rounding to bf16 leaves (0.4% of the results are the
// neighbour of the exact sum's rounding).
MOK_DEV Frag<F8> large_of(const Frag<F8>& v) {
  Frag<F8> o;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t w[4] = {v.q[i].x, v.q[i].y, v.q[i].z, v.q[i].w};
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      // per byte: all ones where the code without its sign is at least 0x48 (the value 4)
      const uint32_t ge = (((w[n] & 0x7F7F7F7Fu) + 0x38383838u) >> 7) & 0x01010101u;
      w[n] &= (ge << 8) - ge;
    }
    o.q[i] = make_uint4(w[0], w[1], w[2], w[3]);
  }
  return o;
}
MOK_DEV Frag<F8> without(const Frag<F8>& v, const Frag<F8>& u) {
  Frag<F8> o;
#pragma unroll
  for (int i = 0; i < 2; ++i)
    o.q[i] = make_uint4(v.q[i].x ^ u.q[i].x, v.q[i].y ^ u.q[i].y, v.q[i].z ^ u.q[i].z,
                        v.q[i].w ^ u.q[i].w);
  return o;
}
// The products of one a with N b's; after(j) follows the j-th.
template <int FA, int FB, int SEL, bool X, int N, class After>
MOK_DEV void mfma_row(const Frag<FB> (&b)[N], const Frag<FA>& a, f32x16_t (&acc)[N],
                      const uint32_t (&bsc)[N], uint32_t asc, After&& after) {
  if constexpr (X && FA == F8 && FB == F4) {
    const Frag<F8> hi = large_of(a), lo = without(a, hi);
#pragma unroll
    for (int j = 0; j < N; ++j) {
      acc[j] = mfma<FA, FB, SEL>(b[j], lo, acc[j], bsc[j], asc);
      acc[j] = mfma<FA, FB, SEL>(b[j], hi, acc[j], bsc[j], asc);
      after(j);
    }
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      if constexpr (X && FA == F4 && FB == F8) {
        const Frag<F8> hi = large_of(b[j]), lo = without(b[j], hi);
        acc[j] = mfma<FA, FB, SEL>(lo, a, acc[j], bsc[j], asc);
        acc[j] = mfma<FA, FB, SEL>(hi, a, acc[j], bsc[j], asc);
      } else {
        acc[j] = mfma<FA, FB, SEL>(b[j], a, acc[j], bsc[j], asc);
      }
      after(j);
    }
  }
}

// A 4-byte word at any address.
MOK_DEV uint32_t load_word(const uint8_t* p) {
  uint32_t v;
  __builtin_memcpy(&v, p, 4);
  return v;
}
// The scales of blocks b0 .. b0 + 3 of a row of n blocks: past the row, the last one's (their
// codes are taken as zero).
MOK_DEV uint32_t scales_at(const uint8_t* row, int b0, int n) {
  if (b0 + 4 <= n) return load_word(row + b0);
  uint32_t v = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) v |= (uint32_t)row[min(b0 + i, n - 1)] << (8 * i);
  return v;
}

// 4 consecutive columns n .. n + 3 of row m of C.
MOK_DEV void store4(const MxArgs& p, void* c, bool f32, int m, int n, float4 v) {
  if (m >= p.M || n >= p.N) return;
  const int64_t at = (int64_t)m * p.N + n;
  if (p.N % 4 == 0) {
    if (f32) *(float4*)((float*)c + at) = v;
    else *(uint2*)((bf16_t*)c + at) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
  } else {
    const float q[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n + i < p.N) {
        if (f32) ((float*)c)[at + i] = q[i];
        else ((bf16_t*)c)[at + i] = f32_to_bf16(q[i]);
      }
  }
}

// ------------------------------------------------------------------------- few rows
// A workgroup computes 32 columns (rows of B) x 32 MT rows; its KS waves take every KS-th step
// of 256 along K, straight from memory into registers, and add their sums through LDS in wave
// order. B is read once over the grid.
constexpr int KS = 8;

template <int FA, int FB, int MT>
__global__ __launch_bounds__(64 * KS) void k_mx_rows(const MxArgs p) {
  constexpr bool X = FA != FB;
  __shared__ float4 red[KS][MT][4][64];
  const int lane = lane_id(), w = uniform(threadIdx.x >> 6), h = lane >> 5, r = lane & 31;
  const int n0 = blockIdx.x * 32, m0 = blockIdx.y * 32 * MT;
  const int KB = p.K / 32;
  const int64_t rb = min(n0 + r, p.N - 1);
  const uint8_t* b = p.b + rb * code_bytes<FB>(p.K);
  const uint8_t* bs = p.bs + rb * KB;
  const uint8_t *a[MT], *as[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int64_t ra = min(m0 + 32 * i + r, p.M - 1);
    a[i] = p.a + ra * code_bytes<FA>(p.K);
    as[i] = p.as + ra * KB;
  }
  f32x16_t acc[MT][1] = {};
  // this lane's part of the MFMA of blocks b0 + s and b0 + 4 + s
  auto frag = [&](auto f, const uint8_t* row, int b0, int s) {
    Frag<f()> v;
    const int blk = b0 + 4 * h + s;
    if constexpr (f() == F4) {
      v.q[0] = *(const uint4*)(row + 16 * min(blk, KB - 1));
      if (blk >= KB) v.zero();
    } else {
      const int x0 = b0 + s, x1 = b0 + 4 + s;
      v.q[0] = *(const uint4*)(row + 32 * min(x0, KB - 1) + 16 * h);
      v.q[1] = *(const uint4*)(row + 32 * min(x1, KB - 1) + 16 * h);
      if (x0 >= KB) v.q[0] = make_uint4(0, 0, 0, 0);
      if (x1 >= KB) v.q[1] = make_uint4(0, 0, 0, 0);
    }
    return v;
  };
  std::integral_constant<int, FA> fa;
  std::integral_constant<int, FB> fb;
  for (int b0 = 8 * w; b0 < KB; b0 += 8 * KS) {
    Frag<FB> vb[4][1];
    Frag<FA> va[MT][4];
    uint32_t sb[1] = {scales_at(bs, b0 + 4 * h, KB)}, sa[MT];
#pragma unroll
    for (int s = 0; s < 4; ++s) vb[s][0] = frag(fb, b, b0, s);
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      sa[i] = scales_at(as[i], b0 + 4 * h, KB);
#pragma unroll
      for (int s = 0; s < 4; ++s) va[i][s] = frag(fa, a[i], b0, s);
    }
    static_for<4>([&](auto s) {
#pragma unroll
      for (int i = 0; i < MT; ++i)
        mfma_row<FA, FB, s(), X>(vb[s()], va[i][s()], acc[i], sb, sa[i], [](int) {});
    });
  }
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int q = 0; q < 4; ++q)
      red[w][i][q][lane] = make_float4(acc[i][0][4 * q], acc[i][0][4 * q + 1],
                                       acc[i][0][4 * q + 2], acc[i][0][4 * q + 3]);
  __syncthreads();
  for (int t = threadIdx.x; t < 256 * MT; t += 64 * KS) {
    const int l = t & 63, q = (t >> 6) & 3, i = t >> 8;
    float4 v = red[0][i][q][l];
#pragma unroll
    for (int k = 1; k < KS; ++k) {
      const float4 x = red[k][i][q][l];
      v.x += x.x; v.y += x.y; v.z += x.z; v.w += x.w;
    }
    store4(p, p.c, p.out_f32, m0 + 32 * i + (l & 31), n0 + 8 * q + 4 * (l >> 5), v);
  }
}

// ------------------------------------------------------------------------- LDS tiles
// BM x BN tiles, WM x WN waves of BM/WM x BN/WN: 2 x 2 (two waves a SIMD were no faster: 2 x 4 and
// 4 x 2 were within 2% at 256 x 256 and 10 to 20% slower at 128 x 128, where two groups of 2 x 2 that
// share a step's K were 3 to 17% slower). K steps of KT values go to one of ST LDS buffers by
// LDS-DMA (16-byte chunks; chunk c of row r at slot c ^ swz(r), so that the 16 rows that a quarter
// of a wave reads at one chunk hit distinct banks). A step's last sub-step follows the
// barrier that publishes the next step's buffer: its MFMAs cover the next step's first LDS reads,
// and the DMA of the step ST steps on, into the buffer just read, is issued among them.
// 128 x 128 tiles leave room for 4 buffers: their steps are shorter than a load's way from memory (3,
// 5 and 6 buffers took the same time). One tile a CU pays for its loads beside its MFMAs: M 1000, N
// 4096, K 7168 MXFP8 x MXFP4 takes 33 us, 26 without its code loads, 29 without its scale loads, 20
// with the MFMAs alone.
// AL: K % 512 == 0, so that 16-byte pieces of the scale rows are aligned and also go by DMA.
template <int FA_, int FB_, int BM_, int BN_, int WM_, int WN_, bool AL_, bool X_>
struct Tile {
  static constexpr int WM = WM_, WN = WN_, NW = WM * WN;          // waves over rows and columns
  static constexpr int FA = FA_, FB = FB_, BM = BM_, BN = BN_;
  static constexpr bool AL = AL_, X = X_;
  static constexpr int KT = FA == F4 && FB == F4 ? 256 : 128;
  static constexpr int ST = AL && BM == 128 ? 4 : 2;
  static constexpr int SUB = KT / 64;
  static constexpr int FM = BM / WM / 32, FN = BN / WN / 32;
  static constexpr int RBA = code_bytes<FA>(KT), RBB = code_bytes<FB>(KT);   // bytes of a row
  static constexpr int QA = BM * RBA / 1024 / NW, QB = BN * RBB / 1024 / NW;   // DMA instructions a wave
};

template <int RB> MOK_DEV constexpr int swz(int r) {
  return RB == 128 ? (r >> 1) & 7 : (r >> 2) & 3;
}

template <class C>
__global__ __launch_bounds__(64 * C::NW) void k_mx_tile(const MxArgs p) {
  constexpr int FA = C::FA, FB = C::FB, FM = C::FM, FN = C::FN, SUB = C::SUB, KT = C::KT;
  constexpr int ST = C::ST;
  constexpr int A_B = C::BM * C::RBA, B_B = C::BN * C::RBB, S_B = (C::BM + C::BN) * 32;   // bytes
  constexpr int OUT_B = C::NW * 32 * (C::BN / C::WN * 4 + 16);      // the epilogue's rows
  constexpr int NSB = ST > 2 ? 4 : 2;                               // buffers of scales
  __shared__ __align__(1024) char lds[std::max(ST * (A_B + B_B) + NSB * S_B, OUT_B)];
  char* const lds_b0 = lds + ST * A_B;
  char* const lds_s0 = lds_b0 + ST * B_B;
  auto buf_a = [&](int kt) { return (uint4*)(lds + kt % ST * A_B); };
  auto buf_b = [&](int kt) { return (uint4*)(lds_b0 + kt % ST * B_B); };
  auto buf_s = [&](int g) { return (uint32_t*)(lds_s0 + (g & (NSB - 1)) * S_B); };
  const int tid = threadIdx.x, lane = tid & 63, wid = uniform(tid >> 6);
  const int wm = wid / C::WN, wn = wid % C::WN, h = lane >> 5, r = lane & 31;
  // XCD x takes consecutive tiles, 8 M tiles deep, so that its L2 holds their operands
  const int tiles = p.tiles_m * p.tiles_n;
  const int per = (tiles + 7) / 8;
  const int tile = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
  if (tile >= tiles || (int)(blockIdx.x >> 3) >= per) return;
  const int band = tile / (8 * p.tiles_n), in = tile % (8 * p.tiles_n);
  const int bh = min(8, p.tiles_m - 8 * band);
  const int m0 = (8 * band + in % bh) * C::BM, n0 = in / bh * C::BN;
  const int KB = p.K / 32;
  const int step0 = blockIdx.z * p.steps_per_split;
  const int nk = min(p.steps_per_split, (p.K + KT - 1) / KT - step0);
  const int64_t lda = code_bytes<FA>(p.K), ldb = code_bytes<FB>(p.K);

  // DMA instruction q of this wave fills LDS rows (wid Q + q) RPI + lane / CH of an operand's
  // buffer, lane % CH being the slot: its row's byte offset from the tile's first row (rows past
  // the operand: its last) is kept; the slot's chunk alternates between two with q.
  constexpr int CHA = C::RBA / 16, CHB = C::RBB / 16, RPA = 64 / CHA, RPB = 64 / CHB;
  uint32_t off_a[C::QA], off_b[C::QB];
  int ch_a[2], ch_b[2];
#pragma unroll
  for (int q = 0; q < C::QA; ++q) {
    const int row = (wid * C::QA + q) * RPA + lane / CHA;
    off_a[q] = (uint32_t)((min(m0 + row, p.M - 1) - m0) * lda);
    if (q < 2) ch_a[q] = ((lane % CHA) ^ swz<C::RBA>(row)) * 16;
  }
#pragma unroll
  for (int q = 0; q < C::QB; ++q) {
    const int row = (wid * C::QB + q) * RPB + lane / CHB;
    off_b[q] = (uint32_t)((min(n0 + row, p.N - 1) - n0) * ldb);
    if (q < 2) ch_b[q] = ((lane % CHB) ^ swz<C::RBB>(row)) * 16;
  }
  const uint8_t* base_a = uniform_ptr(p.a + m0 * lda);
  const uint8_t* base_b = uniform_ptr(p.b + n0 * ldb);
  const uint32_t to_a = uniform(lds_addr(lds)), to_b = to_a + ST * A_B, to_s = to_b + ST * B_B;
  // chunks past K: the row's last (cleared in LDS before they are read)
  auto issue = [&](int kt, int q) {
    __builtin_amdgcn_sched_barrier(0);
    const int g = step0 + kt;
    if (q < C::QA) {
      const int ch = min(ch_a[q & 1], (int)lda - 16 - g * C::RBA);
      dma_b128(base_a + g * C::RBA, off_a[q] + ch,
               to_a + kt % ST * A_B + (wid * C::QA + q) * 1024);
    } else {
      const int ch = min(ch_b[(q - C::QA) & 1], (int)ldb - 16 - g * C::RBB);
      dma_b128(base_b + g * C::RBB, off_b[q - C::QA] + ch,
               to_b + kt % ST * B_B + (wid * C::QB + q - C::QA) * 1024);
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  constexpr int NQ = C::QA + C::QB, NM = FM * FN;
  auto issue_all = [&](int kt) {
#pragma unroll
    for (int q = 0; q < NQ; ++q) issue(kt, q);
  };
  // Scales go through LDS in groups of SG steps: 32 bytes of each of the tile's BM + BN rows (A's
  // first), NSB buffers. (Read from memory by every lane for its own rows and step, a word at a
  // time, they touched as many cache lines as the codes: M 8192, N 4096, K 7168 took 155 us,
  // against 126 without any scales.) 16-byte half x of row r lies at half x ^ (r >> 3 & 1), which
  // spreads a column of words over the banks. Step kt loads a piece of the group SG steps on from
  // step kt + ST - 1's: with ST 2 the last piece lands with the step before that group's first, with
  // ST 4, where two steps' loads stay in flight, two steps earlier, hence more buffers.
  // The first half of the waves loads A's rows, the second B's. A piece is 32 rows a wave, 16 bytes a
  // lane, P pieces a group, then over again (the same bytes); or (WORDS) 8 rows, a word a lane, where
  // those are a step's share: a fourth of the cache lines (M 1000, N 4096, K 7168, MXFP8 by MXFP4:
  // 34.1 -> 32.9 us, by MXFP8: 35.1 -> 33.3; two such loads a step were no faster, 22.5 against 21.8
  // for MXFP4 operands).
  constexpr int SG = 32 / (KT / 32), SH = C::NW / 2, P = C::BM / (32 * SH);
  constexpr bool WORDS = C::AL && C::BM == 8 * SH * SG;
  static_assert(C::BM == C::BN, "both operands' scales in the same number of pieces");
  const bool tiny = KB < 16;
  const uint8_t* base_sc = uniform_ptr(wid < SH ? p.as + (int64_t)m0 * KB : p.bs + (int64_t)n0 * KB);
  const int sc_last = uniform(wid < SH ? p.M - 1 - m0 : p.N - 1 - n0);      // the operand's last row
  const int sc_r = wid % SH * 32 + lane / 2;                               // row in piece 0
  auto sc_at = [&](int t) { return (uint32_t)min(t * 32 * SH + sc_r, sc_last) * (uint32_t)KB; };
  const int sc_half = (lane ^ (sc_r >> 3)) & 1;       // the half of the row that slot lane & 1 holds
  const int sc_byte = step0 * (KT / 32) + 16 * sc_half;
  const int sc_to = wid / SH * C::BM + wid % SH * 32;                      // LDS row of piece 0
  // AL: past the row's end: its last 16 bytes
  auto sc_dma = [&](int g, int t) {
    __builtin_amdgcn_sched_barrier(0);
    dma_b128(base_sc, sc_at(t) + min(sc_byte + g * 32, KB - 16),
             to_s + (g & (NSB - 1)) * S_B + (sc_to + t * 32 * SH) * 32);
    __builtin_amdgcn_sched_barrier(0);
  };
  auto sc_words = [&](int g, int t) {
    __builtin_amdgcn_sched_barrier(0);
    const int e = t * SH + wid % SH;                       // the 8 rows
    const uint32_t row = (uint32_t)min(e * 8 + lane / 8, sc_last) * (uint32_t)KB;
    const int w = (lane % 8) ^ (4 * (e & 1));
    dma_b32(base_sc, row + min(step0 * (KT / 32) + g * 32 + 4 * w, KB - 4),
            to_s + (g & (NSB - 1)) * S_B + (wid / SH * C::BM + e * 8) * 32);
    __builtin_amdgcn_sched_barrier(0);
  };
  auto sc_piece = [&](int g, int t) {
    if constexpr (WORDS) sc_words(g, t); else sc_dma(g, t % P);
  };
  // else through registers: 16 bytes from the row's byte, or the row's last 16 where it ends
  // before, then shifted down by the bytes that it starts early. Rows of fewer than 16 blocks:
  // byte by byte (one group; the steps' loads then read the codes, and are not used).
  auto sc_load = [&](int g, int t) {
    uint4 v;
    __builtin_memcpy(&v, tiny ? p.a : base_sc + (sc_at(t) + min(sc_byte + g * 32, KB - 16)), 16);
    return v;
  };
  auto sc_put = [&](int g, int t, uint4 v) {
    *(uint4*)&buf_s(g)[(sc_to + t * 32 * SH) * 8 + lane * 4] = v;
  };
  auto sc_store = [&](int g, int t, uint4 v) {
    const int early = max(sc_byte + g * 32 - (KB - 16), 0), by = early & 3, wd = early >> 2;
    uint32_t w0 = __builtin_amdgcn_alignbyte(v.y, v.x, by), w1 = __builtin_amdgcn_alignbyte(v.z, v.y, by),
             w2 = __builtin_amdgcn_alignbyte(v.w, v.z, by), w3 = __builtin_amdgcn_alignbyte(0u, v.w, by);
    const bool s1 = wd & 1, s2 = wd & 2;
    w0 = s1 ? w1 : w0; w1 = s1 ? w2 : w1; w2 = s1 ? w3 : w2; w3 = s1 ? 0u : w3;
    w0 = s2 ? w2 : w0; w1 = s2 ? w3 : w1; w2 = s2 ? 0u : w2; w3 = s2 ? 0u : w3;
    sc_put(g, t, make_uint4(w0, w1, w2, w3));
  };
  auto sc_short = [&](int t) {
    uint32_t w[4] = {0, 0, 0, 0};
    const uint8_t* q = base_sc + sc_at(t);
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (16 * sc_half + i < KB) w[i >> 2] |= (uint32_t)q[16 * sc_half + i] << (8 * (i & 3));
    sc_put(0, t, make_uint4(w[0], w[1], w[2], w[3]));
  };
  // a step's scale words of this lane's rows. KT 256: lane half h takes blocks 4 h .. 4 h + 3,
  // byte s for sub-step s; KT 128: blocks 0 .. 3, shifted by h, byte 2 s.
  uint32_t asc[FM], bsc[FN], asc_n[FM], bsc_n[FN];
  auto read_scales = [&](int kt) {
    const int w = (KT == 256 ? 2 * (kt % SG) + h : kt % SG) ^ (4 * ((r >> 3) & 1));
    const uint32_t* S = buf_s(kt / SG);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < FM; ++i) asc_n[i] = S[(wm * (C::BM / C::WM) + 32 * i + r) * 8 + w];
#pragma unroll
    for (int j = 0; j < FN; ++j) bsc_n[j] = S[(C::BM + wn * (C::BN / C::WN) + 32 * j + r) * 8 + w];
    __builtin_amdgcn_sched_barrier(0);
  };
  auto take_scales = [&]() {
#pragma unroll
    for (int i = 0; i < FM; ++i) asc[i] = KT == 256 ? asc_n[i] : asc_n[i] >> (8 * h);
#pragma unroll
    for (int j = 0; j < FN; ++j) bsc[j] = KT == 256 ? bsc_n[j] : bsc_n[j] >> (8 * h);
  };
  // blocks of step kt that K holds (KT / 32, fewer in a ragged last step)
  auto left = [&](int kt) { return KB - (step0 + kt) * (KT / 32); };
  // a ragged last step: the codes past K, which the DMA filled with the row's last chunk, are
  // cleared where this wave's DMA put them (after it landed, before the barrier that publishes it)
  auto clear_tail = [&](auto F_, auto RB_, auto Q_, uint4* buf, int kt) {
    constexpr int F = F_(), RB = RB_(), Q = Q_(), CH = RB / 16, RPI = 64 / CH;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const int row = (wid * Q + q) * RPI + lane / CH;
      const int c = (lane % CH) ^ swz<RB>(row);             // the chunk at this lane's slot
      if ((F == F8 ? c / 2 : c) >= left(kt))
        buf[(wid * Q + q) * 64 + lane] = make_uint4(0, 0, 0, 0);
    }
  };
  // Step kt is whole in LDS: every wave's DMA of it has landed (all but the OUT vector-memory
  // instructions that it issued last: vmcnt counts in order) and its LDS reads are back. LAST: kt
  // may be the ragged last step.
  auto publish = [&](int kt, auto OUT, auto LAST) {
    static_assert(OUT() < 64, "vmcnt range");
    __builtin_amdgcn_s_waitcnt((OUT() & 15) | ((OUT() >> 4) << 14) | (7 << 4));   // lgkmcnt(0)
    if constexpr (LAST()) {
      if (left(kt) < KT / 32) {
        clear_tail(std::integral_constant<int, FA>{}, std::integral_constant<int, C::RBA>{},
                   std::integral_constant<int, C::QA>{}, buf_a(kt), kt);
        clear_tail(std::integral_constant<int, FB>{}, std::integral_constant<int, C::RBB>{},
                   std::integral_constant<int, C::QB>{}, buf_b(kt), kt);
        __builtin_amdgcn_s_waitcnt(0x70);
      }
    }
    lds_barrier();
  };
  Frag<FA> fa[2][FM];
  Frag<FB> fb[2][FN];
  // block pairs of sub-step s: (s, 4 + s) of 8 blocks (KT 256) or (2 s, 2 s + 1) of 4 (KT 128)
  auto blk = [](int s, int x) { return KT == 256 ? 4 * x + s : 2 * s + x; };
  auto read = [&](auto f, auto RB_, const uint4* buf, int row, int s) {
    constexpr int RB = RB_(), CH = RB / 16;
    Frag<f()> v;
    const uint4* base = buf + row * CH;
    if constexpr (f() == F4) {
      v.q[0] = base[blk(s, h) ^ swz<RB>(row)];
    } else {
      v.q[0] = base[(2 * blk(s, 0) + h) ^ swz<RB>(row)];
      v.q[1] = base[(2 * blk(s, 1) + h) ^ swz<RB>(row)];
    }
    return v;
  };
  // in the order in which the MFMAs first use them
  auto frags = [&](int kt, int s, int f) {
    const uint4 *A = buf_a(kt), *B = buf_b(kt);
    auto a_at = [&](int i) {
      fa[f][i] = read(std::integral_constant<int, FA>{}, std::integral_constant<int, C::RBA>{}, A,
                      wm * (C::BM / C::WM) + 32 * i + r, s);
    };
    __builtin_amdgcn_sched_barrier(0);
    a_at(0);
#pragma unroll
    for (int j = 0; j < FN; ++j)
      fb[f][j] = read(std::integral_constant<int, FB>{}, std::integral_constant<int, C::RBB>{}, B,
                      wn * (C::BN / C::WN) + 32 * j + r, s);
#pragma unroll
    for (int i = 1; i < FM; ++i) a_at(i);
    __builtin_amdgcn_sched_barrier(0);
  };
  f32x16_t acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.0f;
  auto mfmas = [&](auto s, auto&& after) {
    constexpr int SEL = KT == 256 ? s() : 2 * s(), F = s() & 1;
#pragma unroll
    for (int i = 0; i < FM; ++i)
      mfma_row<FA, FB, SEL, C::X>(fb[F], fa[F][i], acc[i], bsc, asc[i],
                                  [&](int j) { after(i * FN + j); });
    __builtin_amdgcn_sched_barrier(0);
  };
  // One K step. MORE: a step follows; LAST: it may be the last one; DMA: the loads of step kt + ST
  // and one scale piece are issued here (LATE: also what the step before left of its loads), and
  // OUT vector-memory instructions may stay in flight at the barrier. No branches inside the main
  // loop's form: the compiler moves MFMAs past them.
  // A step's loads are issued among the MFMAs of the last sub-step and, where the buffers give
  // them the time to land, of the next step's first: NQ of them in one sub-step hold up its MFMAs.
  constexpr bool SPREAD = SUB == 4 || ST > 2;
  constexpr int H1 = SPREAD ? (NQ + 1) / 2 : NQ, H2 = NQ - H1;
  auto step = [&](int kt, auto MORE, auto LAST, auto DMA, auto LATE, auto OUT) {
    const int u = kt + ST - 1, sg = u / SG + 1, st = u % SG;     // the scale piece on its way
    uint4 sv;
    if constexpr (DMA() && !C::AL) sv = sc_load(sg, st % P);
    static_for<SUB - 1>([&](auto s) {
      mfmas(s, [&](int n) {
        if (n == NM / 2 - 1) frags(kt, s() + 1, (s() + 1) & 1);
        if constexpr (LATE() && H2 > 0 && s() == 0) {
#pragma unroll
          for (int q = n * H2 / NM; q < (n + 1) * H2 / NM; ++q) issue(kt - 1 + ST, H1 + q);
        }
      });
    });
    if constexpr (MORE()) publish(kt + 1, OUT, LAST);     // and all reads of step kt are back
    mfmas(std::integral_constant<int, SUB - 1>{}, [&](int n) {
      if constexpr (MORE()) {
        if (n == 0) read_scales(kt + 1);
        if (n == NM / 2 - 1) frags(kt + 1, 0, 0);
      }
      if constexpr (DMA()) {
        if (n == 1) {
          if constexpr (C::AL) sc_piece(sg, st); else sc_store(sg, st % P, sv);
        }
#pragma unroll
        for (int q = n * H1 / NM; q < (n + 1) * H1 / NM; ++q) issue(kt + ST, q);
      }
    });
    if constexpr (MORE()) take_scales();
  };
  constexpr std::integral_constant<bool, true> yes{};
  constexpr std::integral_constant<bool, false> no{};
  constexpr std::integral_constant<int, 0> none{};
#pragma unroll
  for (int t = 0; t < P; ++t) {
    if constexpr (C::AL) {
      sc_dma(0, t);
    } else {
      if (tiny) sc_short(t);
      else sc_store(0, t, sc_load(0, t));
    }
  }
  if constexpr (C::AL) {
#pragma unroll
    for (int u = 0; u < ST - 1; ++u) sc_piece(1, u);
  } else {
    if (KB > 32) sc_store(1, 0, sc_load(1, 0));
  }
  issue_all(0);
  if (nk >= ST) {
#pragma unroll
    for (int i = 1; i < ST; ++i) {
#pragma unroll
      for (int q = 0; q < (i == ST - 1 ? H1 : NQ); ++q) issue(i, q);
    }
    publish(0, std::integral_constant<int, (ST - 1) * NQ - H2>{}, yes);
  } else {
    for (int i = 1; i < nk; ++i) issue_all(i);
    publish(0, none, yes);
  }
  read_scales(0);
  take_scales();
  frags(0, 0, 0);
  // (ST - 2) NQ of a step's NQ + 1: the prologue's steps have no scale piece among their loads, so
  // that with (ST - 2) (NQ + 1) the first steps' last loads could still be on their way.
  int kt = 0;
  for (; kt < nk - ST; ++kt)
    step(kt, yes, no, yes, yes, std::integral_constant<int, (ST - 2) * NQ>{});
  if (nk >= ST) step(kt++, yes, yes, no, yes, none);
  if constexpr (ST > 2) {
    for (; kt < nk - 1; ++kt) step(kt, yes, yes, no, no, none);
  }
  if (kt < nk) step(kt, no, no, no, no, none);

  void* c = p.c;
  bool f32 = p.out_f32;
  if (p.splits > 1) {
    c = (float*)p.c + (int64_t)blockIdx.z * p.M * p.N;
    f32 = true;
  }
  if (p.N % 8 == 0) {
    // Each wave puts its blocks of 32 rows through its own part of the operand buffers and writes
    // whole row segments, 16 bytes a lane (straight from the accumulators, 8 bytes a lane and 32
    // rows an instruction, the stores took 34 of 149 us at M 8192, N 4096, K 7168).
    constexpr int WN = C::BN / C::WN;
    char* mine = lds + wid * (32 * (WN * 4 + 16));
    __syncthreads();                              // every wave is past its last fragment reads
    // the lane made opaque again: what derives from it is computed here, not held over the K loop
    const int lane_ = opaque(threadIdx.x) & 63;
    auto out = [&, lane = lane_, r = lane_ & 31, h = lane_ >> 5](auto F32) {
      constexpr int es = F32() ? 4 : 2, ld = WN * es + 16;
      constexpr int seg = WN * es / 16, at_once = 64 / seg;    // lanes a row, rows a store
      const int piece = lane % seg, col = n0 + wn * WN + piece * (16 / es);
#pragma unroll
      for (int i = 0; i < FM; ++i) {
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            char* at = mine + r * ld + (32 * j + 8 * q + 4 * h) * es;
            const f32x16_t& v = acc[i][j];
            if constexpr (F32())
              *(float4*)at = make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
            else
              *(uint2*)at = make_uint2(pack_bf16x2(v[4 * q], v[4 * q + 1]),
                                       pack_bf16x2(v[4 * q + 2], v[4 * q + 3]));
          }
        const int row0 = m0 + wm * (C::BM / C::WM) + 32 * i;
#pragma unroll
        for (int x0 = 0; x0 < 32; x0 += at_once) {
          const int x = x0 + lane / seg;
          const u32x4_t v = *(const u32x4_t*)(mine + x * ld + piece * 16);
          // non-temporal: C would push the operands out of the L2 (121 -> 116 us)
          if (row0 + x < p.M && col < p.N)
            __builtin_nontemporal_store(v, (u32x4_t*)((char*)c + ((int64_t)(row0 + x) * p.N + col) * es));
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    if (f32) out(yes); else out(no);
    return;
  }
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        store4(p, c, f32, m0 + wm * (C::BM / C::WM) + 32 * i + r,
               n0 + wn * (C::BN / C::WN) + 32 * j + 8 * q + 4 * h,
               make_float4(acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2],
                           acc[i][j][4 * q + 3]));
}

// C = the K ranges' partial sums in ascending order.
__global__ __launch_bounds__(256) void k_mx_join(const float* __restrict__ part, int splits,
                                                 int64_t elems, int f32, void* c) {
  for (int64_t i = blockIdx.x * (int64_t)256 + threadIdx.x; i < elems;
       i += (int64_t)gridDim.x * 256) {
    float v = 0.0f;
#pragma unroll 4
    for (int q = 0; q < splits; ++q) v += part[q * elems + i];
    if (f32) ((float*)c)[i] = v;
    else ((bf16_t*)c)[i] = f32_to_bf16(v);
  }
}

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

constexpr int kRowsMax = 64;      // rows up to which k_mx_rows streams B

// The tiling of a product, from its sizes alone.
struct Plan {
  bool rows;               // k_mx_rows
  int tile;                // 256 or 128
  int splits;
};
Plan plan_of(int64_t M, int64_t N, int64_t K) {
  Plan t;
  t.rows = M <= kRowsMax;
  t.tile = cdiv(M, 256) * cdiv(N, 256) >= 192 ? 256 : 128;
  const int64_t tiles = cdiv(M, t.tile) * cdiv(N, t.tile), steps = cdiv(K, 256);
  // K ranges: where 256 CUs have 32 tiles or fewer and at least 16 steps each; every range keeps 4
  // steps, and all their sums 8 MB, since writing and adding them costs as much as 10 steps (M 256,
  // N 2048, K 7168: 17.8 us in one range, 11.7 to 13.6 in 7 to 3; M 256, N 4096: 17.9 in one, 18.3
  // in 4; M 256, N 7168, K 2048: 7.8 in one, 19.8 in 2).
  t.splits = 1;
  if (!t.rows && tiles <= 32 && steps >= 16)
    t.splits = (int)std::max<int64_t>(
        1, std::min({256 / tiles, steps / 4, ((int64_t)8 << 20) / (M * N * 4)}));
  return t;
}

template <int FA, int FB, bool X>
hipError_t run_mx(MxArgs p, const Plan& t, float* part, void* c, hipStream_t s) {
  if (t.rows) {
    p.c = c;
    auto k = p.M <= 32 ? k_mx_rows<FA, FB, 1> : k_mx_rows<FA, FB, 2>;
    launch_k(k, dim3((unsigned)cdiv(p.N, 32)), dim3(64 * KS), 0, s, nullptr, nullptr, p);
    return hipGetLastError();
  }
  p.tiles_m = (int)cdiv(p.M, t.tile);
  p.tiles_n = (int)cdiv(p.N, t.tile);
  constexpr int KT = Tile<FA, FB, 128, 128, 2, 2, true, X>::KT;
  const int64_t steps = cdiv(p.K, KT);
  p.steps_per_split = (int)cdiv(cdiv(steps, t.splits), 4) * 4;   // whole aligned scale pieces
  p.splits = (int)cdiv(steps, p.steps_per_split);       // every range has a step
  p.c = p.splits > 1 ? part : c;
  const int64_t tiles = (int64_t)p.tiles_m * p.tiles_n;
  const dim3 grid((unsigned)(8 * cdiv(tiles, 8)), 1, p.splits);
  const bool al = p.K % 512 == 0 && (uintptr_t)p.as % 16 == 0 && (uintptr_t)p.bs % 16 == 0;
  auto k = t.tile == 256 ? (al ? k_mx_tile<Tile<FA, FB, 256, 256, 2, 2, true, X>>
                               : k_mx_tile<Tile<FA, FB, 256, 256, 2, 2, false, X>>)
                         : (al ? k_mx_tile<Tile<FA, FB, 128, 128, 2, 2, true, X>>
                               : k_mx_tile<Tile<FA, FB, 128, 128, 2, 2, false, X>>);
  launch_k(k, grid, dim3(256), 0, s, nullptr, nullptr, p);
  if (hipGetLastError() != hipSuccess) return hipErrorLaunchFailure;
  if (p.splits > 1) {
    const int64_t elems = (int64_t)p.M * p.N;
    launch_k(k_mx_join, dim3((unsigned)std::min<int64_t>(cdiv(elems, 256), 8192)), dim3(256), 0, s,
             nullptr, nullptr, (const float*)part, p.splits, elems, p.out_f32, c);
  }
  return hipGetLastError();
}

int mx_check(int64_t M, int64_t N, int64_t K) {
  if (M < 0 || N < 0 || K < 32 || K % 32 || K > (1 << 22)) return MOK_EINVAL;
  if (M >= (int64_t)1 << 31 || N >= (int64_t)1 << 31) return MOK_EINVAL;
  return MOK_OK;
}

}  // namespace
}  // namespace mok

using namespace mok;

extern "C" {

int mok_mx_gemm_workspace_bytes(int64_t M, int64_t N, int32_t K, size_t* bytes) {
  if (!bytes || mx_check(M, N, K) != MOK_OK) return MOK_EINVAL;
  *bytes = 0;
  if (M == 0 || N == 0) return MOK_OK;
  const Plan t = plan_of(M, N, K);
  if (t.splits > 1) *bytes = (size_t)t.splits * M * N * sizeof(float);
  return MOK_OK;
}

int mok_mx_gemm(const uint8_t* a_codes, const uint8_t* a_scales, int32_t a_dtype,
                const uint8_t* b_codes, const uint8_t* b_scales, int32_t b_dtype, int64_t M,
                int64_t N, int32_t K, int32_t out_dtype, void* c, void* ws, size_t ws_bytes,
                void* stream) {
  const int st = mx_check(M, N, K);
  if (st != MOK_OK) return st;
  if ((a_dtype != MOK_MXFP8 && a_dtype != MOK_MXFP4) || (b_dtype != MOK_MXFP8 && b_dtype != MOK_MXFP4))
    return MOK_EINVAL;
  if (out_dtype != MOK_FP32 && out_dtype != MOK_BF16) return MOK_EINVAL;
  if (M == 0 || N == 0) return MOK_OK;
  if (!a_codes || !a_scales || !b_codes || !b_scales || !c) return MOK_EINVAL;
  if ((uintptr_t)a_codes % 16 || (uintptr_t)b_codes % 16 || (uintptr_t)c % 16) return MOK_EINVAL;
  const Plan t = plan_of(M, N, K);
  // a launch counts its threads in 32 bits
  const int64_t threads = t.rows ? cdiv(N, 32) * 64 * KS : cdiv(M, t.tile) * cdiv(N, t.tile) * 256;
  if (threads >= (int64_t)1 << 31) return MOK_EUNSUPPORTED;
  size_t need = 0;
  mok_mx_gemm_workspace_bytes(M, N, K, &need);
  if (need && (!ws || ws_bytes < need || (uintptr_t)ws % 16)) return MOK_EWORKSPACE;
  MxArgs p = {};
  p.a = a_codes; p.as = a_scales; p.b = b_codes; p.bs = b_scales;
  p.M = (int)M; p.N = (int)N; p.K = K;
  p.out_f32 = out_dtype == MOK_FP32;
  hipStream_t s = (hipStream_t)stream;
  hipError_t e;
  float* part = (float*)ws;
  const bool f32 = p.out_f32;
  if (a_dtype == MOK_MXFP4 && b_dtype == MOK_MXFP4) e = run_mx<F4, F4, false>(p, t, part, c, s);
  else if (a_dtype == MOK_MXFP8 && b_dtype == MOK_MXFP8) e = run_mx<F8, F8, false>(p, t, part, c, s);
  else if (a_dtype == MOK_MXFP8)
    e = f32 ? run_mx<F8, F4, true>(p, t, part, c, s) : run_mx<F8, F4, false>(p, t, part, c, s);
  else
    e = f32 ? run_mx<F4, F8, true>(p, t, part, c, s) : run_mx<F4, F8, false>(p, t, part, c, s);
  return e == hipSuccess ? MOK_OK : MOK_EHIP;
}

}  // extern "C"
