// Gradients through the router: from the gradients of the routing weights (and of the logits, as
// the balance loss gives them) to the router's input and its weight.
//
//   dl[t,e]  = dlogits[t,e] + sum_{j: idx[t,j] = e} w[t,j] (dw[t,j] - sum_i w[t,i] dw[t,i])
//   dx[t,i]  = dx_in[t,i] + sum_e dl[t,e] W[e,i]
//   dW[e,i]  = sum_t dl[t,e] x[t,i]
//
// (w = softmax over a token's picks, so its gradient is the softmax's.) The picks are held
// fixed. dW's token sum is cut into ranges whose partial sums a last launch adds in order: no
// atomics, the same bits every run. Three forms:
//
//  k_route_bwd_any  any type, size and alignment: 64 x 64 tiles of both products on the float32 MFMA
//    (operands and sums in float32), 4 waves of 32 x 32, K steps of 32 through LDS, the next step's
//    values loaded into registers under the MFMAs. dl is written once in float32 (DL), or, where
//    T d E < 2^27, built by each workgroup in LDS from the given dlogits and the picks, which saves
//    a launch (float32, T 257, d 272, E 20: 12 against 15 us; T 508, d 4864, E 182: 63 against 46).
//  k_route_bwd_few  float32, up to 16 experts (8 of narrow rows), large: a stream.
//  k_route_bwd_tile  bf16 rows of d % 8 == 0, or of any d where there is much to do, x and the weight
//    then copied to such rows (k_route_bwd_pad): dl is written once as three bf16 planes that sum to
//    it (8 + 8 + 8 significant bits: 24, all of float32's), and both products run on the bf16
//    MFMA with float32 sums: dW on all three planes, dx, which is rounded to 8 bits, on two.
#include <algorithm>

#include "device_common.h"
#include "launch.h"
#include "lds_dma.h"
#include "mok.h"

namespace mok {
namespace {

constexpr int RB_NT = 256, RB_TILE = 64, RB_K = 32, RB_PAD = 4;

struct RbArgs {
  const void *x, *w;
  const int32_t* idx;
  const float *tw, *dtw, *dlogits;
  const void* dx_in;
  const float* dl;    // dl [Tp, EP], zero past T and E
  void* dx;
  float* dw;          // dW itself (one range) or its partial sums [ranges, E, d]
  int64_t T;
  int d, E, k, EP;
  int tiles_d;        // tiles of 64 columns
  int64_t dx_tiles;   // workgroups of the dx product; the rest are dW's
  int tiles_e;
  int64_t t_range;    // tokens of one dW range (a multiple of RB_K)
};

// add(e, g) for each pick e of token t inside [0, E), in pick order, with its share of dl:
// g = w (dw - sum_i w_i dw_i). The picks come 8 at a time, their loads in flight together.
template <class Add>
MOK_DEV void each_pick(const RbArgs& a, int64_t t, Add&& add) {
  float s = 0.0f;
  int32_t e[8];
  float w[8], g[8];
  auto fetch = [&](int j0) {
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const bool ok = j0 + q < a.k;
      e[q] = ok ? a.idx[t * a.k + j0 + q] : -1;
      w[q] = ok ? a.tw[t * a.k + j0 + q] : 0.0f;
      g[q] = ok ? a.dtw[t * a.k + j0 + q] : 0.0f;
    }
  };
  for (int j0 = 0; j0 < a.k; j0 += 8) {
    fetch(j0);
#pragma unroll
    for (int q = 0; q < 8; ++q)
      if (e[q] >= 0 && e[q] < a.E) s += w[q] * g[q];
  }
  for (int j0 = 0; j0 < a.k; j0 += 8) {
    if (a.k > 8) fetch(j0);
#pragma unroll
    for (int q = 0; q < 8; ++q)
      if (e[q] >= 0 && e[q] < a.E) add(e[q], w[q] * (g[q] - s));
  }
}

// acc += A^T B over one K step: A and B lie as [RB_K][RB_TILE + pad] in LDS, the wave's block is
// rows am .. am + 32 of A and columns bn .. bn + 32 of B.
MOK_DEV void mma_step(const float* A, const float* B, int am, int bn, f32x16_t& acc) {
  const int h = lane_id() >> 5, l = lane_id() & 31;
#pragma unroll
  for (int kk = 0; kk < RB_K; kk += 2) {
    const float av = A[(kk + h) * (RB_TILE + RB_PAD) + am + l];
    const float bv = B[(kk + h) * (RB_TILE + RB_PAD) + bn + l];
    acc = __builtin_amdgcn_mfma_f32_32x32x2f32(av, bv, acc, 0, 0, 0);
  }
}

// One 64 x 64 tile of dx or of a range of dW per workgroup.
template <class T, bool DL>
__global__ __launch_bounds__(RB_NT) void k_route_bwd_any(const RbArgs a) {
  __shared__ float A[RB_K * (RB_TILE + RB_PAD)], B[RB_K * (RB_TILE + RB_PAD)];
  constexpr int LD = RB_TILE + RB_PAD;
  const int lane = lane_id(), w = threadIdx.x >> 6, h = lane >> 5, l = lane & 31;
  const int am = (w >> 1) * 32, bn = (w & 1) * 32;
  const bool is_dx = blockIdx.x < a.dx_tiles;
  const int64_t b = is_dx ? blockIdx.x : blockIdx.x - a.dx_tiles;
  const int c0 = (int)(b % a.tiles_d) * RB_TILE;
  const int64_t rest = b / a.tiles_d;
  f32x16_t acc = {};
  constexpr int N = RB_K * RB_TILE / RB_NT;       // values of an operand a thread holds
  float ra[N], rb[N];
  // dx: A row = expert k0 + e, column = token; dW: A row = token k0 + t, column = expert
  const int64_t t0 = rest * RB_TILE;              // dx: first token
  const int e0 = (int)(rest % a.tiles_e) * RB_TILE;               // dW: first expert
  const int64_t range = rest / a.tiles_e;                         // dW: range of tokens
  const int64_t k_begin = is_dx ? 0 : range * a.t_range;
  const int64_t k_end = is_dx ? a.E : min(a.T, k_begin + a.t_range);
  const T* const src = (const T*)(is_dx ? a.w : a.x);             // B rows: experts or tokens
  auto load = [&](int64_t k0) {
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int i = threadIdx.x + n * RB_NT;
      const int64_t t = is_dx ? t0 + i / RB_K : k0 + i / RB_TILE;
      const int e = is_dx ? (int)k0 + i % RB_K : e0 + i % RB_TILE;
      if constexpr (DL) ra[n] = a.dl[t * a.EP + e];
      else ra[n] = a.dlogits && t < a.T && e < a.E ? a.dlogits[t * a.E + e] : 0.0f;
      const int c = c0 + i % RB_TILE;
      const int64_t r = k0 + i / RB_TILE;
      rb[n] = r < k_end && c < a.d ? load_as_f32(src + r * a.d + c) : 0.0f;
    }
  };
  if (k_begin < k_end) load(k_begin);
  for (int64_t k0 = k_begin; k0 < k_end; k0 += RB_K) {
    __syncthreads();                              // every wave is past the previous step's reads
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int i = threadIdx.x + n * RB_NT;
      A[is_dx ? i % RB_K * LD + i / RB_K : i / RB_TILE * LD + i % RB_TILE] = ra[n];
      B[i / RB_TILE * LD + i % RB_TILE] = rb[n];
    }
    __syncthreads();
    if constexpr (!DL) {                          // the picks' share: a thread a token
      const int64_t t = (is_dx ? t0 : k0) + threadIdx.x;
      if (threadIdx.x < (is_dx ? RB_TILE : RB_K) && t < a.T) {
        const int eb = is_dx ? (int)k0 : e0, ne = is_dx ? RB_K : RB_TILE;
        each_pick(a, t, [&](int e, float g) {     // a repeated expert adds up
          e -= eb;
          if (e >= 0 && e < ne) A[is_dx ? e * LD + threadIdx.x : threadIdx.x * LD + e] += g;
        });
      }
      __syncthreads();
    }
    if (k0 + RB_K < k_end) load(k0 + RB_K);
    mma_step(A, B, am, bn, acc);
  }
  if (is_dx) {
#pragma unroll
    for (int v = 0; v < 16; ++v) {
      const int64_t t = t0 + am + 8 * (v >> 2) + 4 * h + (v & 3);
      const int c = c0 + bn + l;
      if (t < a.T && c < a.d) {
        const int64_t at = t * a.d + c;
        const float in = a.dx_in ? load_as_f32((const T*)a.dx_in + at) : 0.0f;
        ((T*)a.dx)[at] = f32_to<T>(in + acc[v]);
      }
    }
  } else {
    float* out = a.dw + range * a.E * a.d;
#pragma unroll
    for (int v = 0; v < 16; ++v) {
      const int e = e0 + am + 8 * (v >> 2) + 4 * h + (v & 3), c = c0 + bn + l;
      if (e < a.E && c < a.d) out[(int64_t)e * a.d + c] = acc[v];
    }
  }
}

// ------------------------------------------------------------------------- few experts
// Float32 rows, up to EC experts: both products are a stream of x, dx_in and dx with E multiply-adds
// a value each, so a thread holds a column (its E weights and E sums of dW) and walks over the tokens
// of range blockIdx.y, 8 tokens' loads in flight; dl of 64 tokens at a time lies in LDS. (The 64 x 64
// tiles do a full tile's products for any E: T 3757, d 6119, float32 took 186 us in them for E 4 and
// 136 for E 16, in this 71 and 98; T 1300, d 379, E 4: 12 and 16, hence T d >= 2^22.)
template <int EC>
__global__ __launch_bounds__(RB_NT) void k_route_bwd_few(const RbArgs a) {
  constexpr int U = 8;
  __shared__ float dls[64][EC];
  const int tid = threadIdx.x, c = blockIdx.x * RB_NT + tid;
  const bool in = c < a.d;
  const float* x = a.dw ? (const float*)a.x : nullptr;
  const float* dx_in = a.dx ? (const float*)a.dx_in : nullptr;
  float* dx = (float*)a.dx;
  float wv[EC], acc[EC];
#pragma unroll
  for (int e = 0; e < EC; ++e) {
    wv[e] = dx && in && e < a.E ? ((const float*)a.w)[(int64_t)e * a.d + c] : 0.0f;
    acc[e] = 0.0f;
  }
  const int64_t tb = blockIdx.y * a.t_range, te = min(a.T, tb + a.t_range);
  for (int64_t t0 = tb; t0 < te; t0 += 64) {
    __syncthreads();                  // the last tokens' dl has been read
    if (tid < 64) {
      const int64_t t = t0 + tid;
#pragma unroll
      for (int e = 0; e < EC; ++e)
        dls[tid][e] = a.dlogits && t < te && e < a.E ? a.dlogits[t * a.E + e] : 0.0f;
      if (t < te) each_pick(a, t, [&](int e, float g) { dls[tid][e] += g; });
    }
    __syncthreads();
    const int nt = (int)min((int64_t)64, te - t0);
    for (int u0 = 0; u0 < nt; u0 += U) {
      float xv[U], o[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const bool ok = in && u0 + u < nt;
        const int64_t at = (t0 + u0 + u) * a.d + c;
        xv[u] = x && ok ? x[at] : 0.0f;
        o[u] = dx_in && ok ? dx_in[at] : 0.0f;
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float s = 0.0f;
#pragma unroll
        for (int e = 0; e < EC; ++e) {
          const float g = dls[u0 + u][e];
          acc[e] += g * xv[u];
          s += g * wv[e];
        }
        if (dx && in && u0 + u < nt) dx[(t0 + u0 + u) * a.d + c] = o[u] + s;
      }
    }
  }
  if (!a.dw || !in) return;
  float* out = a.dw + ((int64_t)blockIdx.y * a.E) * a.d + c;
#pragma unroll
  for (int e = 0; e < EC; ++e)
    if (e < a.E) out[(int64_t)e * a.d] = acc[e];
}

// ------------------------------------------------------------------------- bf16 planes
// dl [Tp][EP], zero past T tokens and E experts, 8 experts a thread: in float32, or (PLANES) as bf16
// planes P0 + P1 + P2 [3][Tp][EP], each the rounding of what the ones before leave, so that the sum
// holds 24 bits.
template <bool PLANES>
__global__ __launch_bounds__(256) void k_route_bwd_dl(const RbArgs a, int EP, int64_t Tp,
                                                      void* __restrict__ out) {
  const int per = EP / 8;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t t = i / per;
  const int e0 = (int)(i - t * per) * 8;
  if (t >= Tp) return;
  float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  if (t < a.T) {
    if (a.dlogits) {
      const float* q = a.dlogits + t * a.E + e0;
#pragma unroll
      for (int n = 0; n < 8; ++n)
        if (e0 + n < a.E) v[n] = q[n];
    }
    each_pick(a, t, [&](int e, float g) {
#pragma unroll
      for (int m = 0; m < 8; ++m) v[m] += m == e - e0 ? g : 0.0f;
    });
  }
  if constexpr (!PLANES) {
    float* q = (float*)out + t * EP + e0;
    *(float4*)q = make_float4(v[0], v[1], v[2], v[3]);
    *(float4*)(q + 4) = make_float4(v[4], v[5], v[6], v[7]);
    return;
  }
#pragma unroll
  for (int p = 0; p < 3; ++p) {
    uint32_t w[4];
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      w[n] = pack_bf16x2(v[2 * n], v[2 * n + 1]);
      const float lo = __uint_as_float(w[n] << 16), hi = __uint_as_float(w[n] & 0xFFFF0000u);
      v[2 * n] = fabsf(lo) == INFINITY ? 0.0f : v[2 * n] - lo;     // an infinity stays one
      v[2 * n + 1] = fabsf(hi) == INFINITY ? 0.0f : v[2 * n + 1] - hi;
    }
    *(uint4*)((bf16_t*)out + ((int64_t)p * Tp + t) * EP + e0) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// The n (at most 8) bf16 values at p, zeros behind them, and back: p on any value's address. Whole
// pieces in one access (with 8 of 2 bytes each T 8192, d 2050, E 64 took 104 us, with these 57).
MOK_DEV u32x4 load_part(const bf16_t* p, int n) {
  u32x4 v = {0, 0, 0, 0};
  if (n >= 8) {
    __builtin_memcpy(&v, p, 16);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < n) v[e / 2] |= (uint32_t)p[e] << (16 * (e & 1));
  }
  return v;
}
MOK_DEV void store_part(bf16_t* p, int n, u32x4 v) {
  if (n >= 8) {
    __builtin_memcpy(p, &v, 16);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < n) p[e] = (bf16_t)(v[e / 2] >> (16 * (e & 1)));
  }
}

// Rows of d bf16 values, d % 8 != 0, laid out in rows of ld = d rounded up to 8, zeros behind them:
// x's T rows, then the router weight's E (either may be left out).
__global__ __launch_bounds__(256) void k_route_bwd_pad(const bf16_t* __restrict__ x, int64_t T,
                                                       const bf16_t* __restrict__ w, int E, int d,
                                                       int ld, bf16_t* __restrict__ out) {
  const int per = ld / 8;
  const int64_t n = (T + E) * per;
  for (int64_t i = blockIdx.x * (int64_t)256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
    const int64_t row = i / per;
    const int c = (int)(i - row * per) * 8;
    const bf16_t* src = row < T ? x : w;
    if (!src) continue;
    src += (row < T ? row : row - T) * d;
    *(u32x4*)(out + row * ld + c) = load_part(src + c, d - c);
  }
}

struct RbTile {
  const bf16_t *x, *w, *dx_in, *planes;
  bf16_t* dx;
  float* dw;            // dW itself (one range) or the partial sums [ranges, E, d]
  int64_t T, Tp;
  int d, E, EP;
  int ld;               // row of x and w: d, or d rounded up to 8 where x and w are padded copies
  int tiles_d;          // tiles of XC columns
  int tiles_e;          // tiles of EM experts
  int dw_tiles, dx_tiles;
  int dw_blocks;        // workgroups of dW (the first ones, a multiple of 8); the rest are dx's
  int64_t t_range;      // tokens of a dW range, a multiple of 64
};

// An operand whose K is the slow dimension, in LDS: K rows of CH 16-byte chunks, chunk c of row kr
// at slot c ^ tswz(kr). ds_read_b64_tr_b16 turns it into K-contiguous fragments: in each group of
// 16 lanes, lane p addresses 4 columns (4 (p % 4) further on) of K row p / 4, and lane i receives
// column i of the 4 K rows; two reads give a lane its 8 K values. A half wave reads 4 rows x 4
// chunks at once: the swizzle puts them on 16 distinct slots of the 64 banks.
template <int CH> MOK_DEV constexpr int tswz(int kr) {
  return CH == 8 ? 4 * ((kr >> 1) & 1) : 4 * (kr & 3);
}
template <int CH>
MOK_DEV bf16x8_t frag_t(uint32_t tile, int blk, int s, int lane) {
  typedef short v4i16 __attribute__((ext_vector_type(4)));
  typedef __attribute__((address_space(3))) v4i16 lds_v4;
  const int g = lane >> 4, p = lane & 15;
  const int m = blk + 16 * (g & 1) + 4 * (p & 3);
  v4i16 v[2];
#pragma unroll
  for (int kb = 0; kb < 2; ++kb) {
    const int kr = 16 * s + 8 * (g >> 1) + 4 * kb + (p >> 2);
    const int off = kr * CH * 16 + (((m >> 3) ^ tswz<CH>(kr)) << 4) + (m & 7) * 2;
    v[kb] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4*)(uintptr_t)(tile + off));
  }
  return __builtin_bit_cast(bf16x8_t, __builtin_shufflevector(v[0], v[1], 0, 1, 2, 3, 4, 5, 6, 7));
}

// Both products in one launch, so that dx's streaming runs beside dW's matrix work. 256 threads.
//  dW: EM experts x XC columns over a range of tokens, K steps of 32 tokens: three planes and x
//      through two LDS buffers by LDS-DMA.
//  dx: 128 tokens x XC columns, K steps of 32 experts: two planes (K-contiguous rows of 64 bytes,
//      chunk c of row r at slot c ^ (r >> 2 & 3)) and the weight's rows, through three buffers or,
//      where EM is 64 (two steps) or XC 256 (LDS), two. The tile goes through LDS in float32, half of
//      its rows at a time, so that dx_in is read and dx written in whole row segments; dx_in is
//      loaded before the product. Both pass the caches by (T 8192, d 2048, E 64: 36 -> 33 us).
// PAD: x and w are copies in rows of ld, dx_in, dx and dW have rows of d, d % 8 != 0 (a form of its
// own: decided in the kernel it cost the aligned one 5%).
// 40 to 80 KB of LDS: 2 or 3 workgroups a CU cover each other's loads (256 experts a workgroup and
// steps of 64, 112 KB and one workgroup a CU, took 113 us at T 4096, d 7168, E 256 where this takes
// 93). There the tiles do 75 GFLOP, and wait for L2 most: 24 to 31% of the cycles are MFMAs, 37%
// waits for loads, a quarter of the reads miss L2.
template <int EM, int XC, bool PAD>
__global__ __launch_bounds__(RB_NT, 2) void k_route_bwd_tile(const RbTile a) {
  constexpr int KT = 32;
  constexpr int PB = KT * EM * 2, XB = KT * XC * 2, WST = 3 * PB + XB;      // bytes of a dW step
  constexpr int DST = 2 * 128 * 64 + XB;                                // bytes of a dx step
  constexpr int OLD = XC + 4;                                             // floats of a staged row
  constexpr int DN = XC == 256 || EM == 64 ? 2 : 3;               // buffers of dx
  constexpr int BYTES = std::max(std::max(2 * WST, DN * DST), 64 * OLD * 4);
  __shared__ __align__(1024) char lds[BYTES];
  const uint32_t lds0 = uniform(lds_addr(lds));
  constexpr int FC = XC / 64, QX = XB / 4096;
  constexpr std::integral_constant<int, XC / 8> CX{};
  const int tid = threadIdx.x, lane = tid & 63, wid = uniform(tid >> 6);
  const int h = lane >> 5, l = lane & 31;
  // every wave's DMA has landed and its LDS reads are back
  auto publish = [&]() {
    __builtin_amdgcn_s_waitcnt(0x70);   // vmcnt(0) lgkmcnt(0)
    lds_barrier();
  };
  // LDS-DMA of K rows x CH chunks (row-major source, ld bytes a row): this wave's instruction q of Q
  // covers rows kr(q) on. at(q): the lane's byte offset; a step whose source ends at row `last`
  // before the step's last row clamps the rows (their products are with zeros of dl). Offsets are
  // made once.
  auto row_of = [&](auto CH_, int Q, int q) { return (wid * Q + q) * (64 / CH_()) + lane / CH_(); };
  auto col_of = [&](auto CH_, int kr, int c0, int cols) {
    return (uint32_t)min(c0 + 8 * ((lane % CH_()) ^ tswz<CH_()>(kr)), cols - 8) * 2;
  };
  // XCD x takes an eighth of each product's tiles, neighbours in order: they share a range of dl's
  // planes (dW) or tokens and, with time, the weight (dx), which its L2 then holds (T 8192, d 2048,
  // E 64: 33 -> 31 us)
  auto tile_of = [](int b, int blocks) { return (b & 7) * (blocks / 8) + (b >> 3); };
  if ((int)blockIdx.x < a.dw_blocks) {
    constexpr int FE = EM / 64;                  // waves: 2 x 2
    const int b = tile_of(blockIdx.x, a.dw_blocks);
    if (b >= a.dw_tiles) return;
    const int c0 = b % a.tiles_d * XC, rest = b / a.tiles_d;
    const int e0 = rest % a.tiles_e * EM;
    const int64_t range = rest / a.tiles_e, tb = range * a.t_range;
    const int64_t te = min(a.T, tb + a.t_range);
    const int nk = te > tb ? (int)((te - tb + KT - 1) / KT) : 0;
    const int we = (wid >> 1) * 32 * FE, wc = (wid & 1) * 32 * FC;
    constexpr int QP = PB / 4096;
    static_assert(QP > 0 && QX > 0, "whole instructions a wave");
    constexpr std::integral_constant<int, EM / 8> CP{};
    const uint32_t ldp = a.EP * 2, ldx = a.ld * 2;
    uint32_t offp[QP], offx[QX], colx[QX];
#pragma unroll
    for (int q = 0; q < QP; ++q) {
      const int kr = row_of(CP, QP, q);
      offp[q] = kr * ldp + col_of(CP, kr, 0, EM);
    }
#pragma unroll
    for (int q = 0; q < QX; ++q) {
      const int kr = row_of(CX, QX, q);
      colx[q] = col_of(CX, kr, c0, a.ld);
      offx[q] = kr * ldx + colx[q];
    }
    auto issue = [&](int kt) {
      const uint32_t to = lds0 + (kt & 1) * WST + wid * 1024 * QP;
      const int64_t t0 = tb + (int64_t)kt * KT;
#pragma unroll
      for (int p = 0; p < 3; ++p) {
        const bf16_t* base = uniform_ptr(a.planes + ((int64_t)p * a.Tp + t0) * a.EP + e0);
#pragma unroll
        for (int q = 0; q < QP; ++q) dma_b128(base, offp[q], to + p * PB + q * 1024);
      }
      const bf16_t* base = uniform_ptr(a.x + t0 * a.ld);
      const uint32_t tx = lds0 + (kt & 1) * WST + 3 * PB + wid * 1024 * QX;
      const int last = (int)min((int64_t)KT - 1, a.T - 1 - t0);
      if (last == KT - 1) {
#pragma unroll
        for (int q = 0; q < QX; ++q) dma_b128(base, offx[q], tx + q * 1024);
      } else {
#pragma unroll
        for (int q = 0; q < QX; ++q)
          dma_b128(base, min(row_of(CX, QX, q), last) * ldx + colx[q], tx + q * 1024);
      }
    };
    f32x16_t acc[FE][FC] = {};
    if (nk > 0) issue(0);
    for (int kt = 0; kt < nk; ++kt) {
      publish();
      if (kt + 1 < nk) issue(kt + 1);
      const uint32_t at = lds0 + (kt & 1) * WST;
#pragma unroll
      for (int s = 0; s < KT / 16; ++s) {
        bf16x8_t fx[FC];
#pragma unroll
        for (int j = 0; j < FC; ++j) fx[j] = frag_t<XC / 8>(at + 3 * PB, wc + 32 * j, s, lane);
#pragma unroll
        for (int p = 2; p >= 0; --p)           // the smallest plane first
#pragma unroll
          for (int i = 0; i < FE; ++i) {
            const bf16x8_t fp = frag_t<EM / 8>(at + p * PB, we + 32 * i, s, lane);
#pragma unroll
            for (int j = 0; j < FC; ++j)
              acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fx[j], fp, acc[i][j], 0, 0, 0);
          }
      }
    }
    float* out = a.dw + range * a.E * a.d;
#pragma unroll
    for (int i = 0; i < FE; ++i)
#pragma unroll
      for (int j = 0; j < FC; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int e = e0 + we + 32 * i + l, c = c0 + wc + 32 * j + 8 * q + 4 * h;
          float* at = out + (int64_t)e * a.d + c;
          if (e < a.E && c < a.d) {
            const float4 v = make_float4(acc[i][j][4 * q], acc[i][j][4 * q + 1],
                                         acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]);
            if constexpr (!PAD) {
              *(float4*)at = v;
            } else if (c + 4 <= a.d) {
              __builtin_memcpy(at, &v, 16);
            } else {
              at[0] = v.x;
              if (c + 1 < a.d) at[1] = v.y;
              if (c + 2 < a.d) at[2] = v.z;
            }
          }
        }
    return;
  }
  const int b = tile_of(blockIdx.x - a.dw_blocks, gridDim.x - a.dw_blocks);
  if (b >= a.dx_tiles) return;
  const int c0 = b % a.tiles_d * XC;
  const int64_t t0 = (int64_t)(b / a.tiles_d) * 128;
  constexpr int TR = XC / 8, RP = RB_NT / TR, NI = 128 / RP;   // threads a row, rows a pass, passes
  u32x4 in[NI];                          // dx_in and dx pass once: non-temporal
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int64_t t = t0 + i * RP + tid / TR;
    const int c = c0 + tid % TR * 8;
    in[i] = u32x4{0, 0, 0, 0};
    if (a.dx_in && t < a.T && c < a.d) {
      const bf16_t* at = a.dx_in + t * a.d + c;
      if constexpr (PAD) in[i] = load_part(at, a.d - c);
      else in[i] = __builtin_nontemporal_load((const u32x4*)at);
    }
  }
  const int wt = (wid >> 1) * 64, wc = (wid & 1) * 32 * FC;
  const int nk = (a.E + 31) / 32;       // every step holds an expert
  const uint32_t ldw = a.ld * 2;
  uint32_t offp[2], offw[QX], colw[QX];
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int r = (wid * 2 + q) * 16 + (lane >> 2);
    offp[q] = (r * a.EP + 8 * ((lane & 3) ^ ((r >> 2) & 3))) * 2;
  }
#pragma unroll
  for (int q = 0; q < QX; ++q) {
    const int kr = row_of(CX, QX, q);
    colw[q] = col_of(CX, kr, c0, a.ld);
    offw[q] = kr * ldw + colw[q];
  }
  auto issue = [&](int kt) {
    const uint32_t at = lds0 + kt % DN * DST, to = at + wid * 2048;
    const uint32_t tw = at + 16384 + wid * 1024 * QX;
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const bf16_t* base = uniform_ptr(a.planes + ((int64_t)p * a.Tp + t0) * a.EP + kt * 32);
#pragma unroll
      for (int q = 0; q < 2; ++q) dma_b128(base, offp[q], to + p * 8192 + q * 1024);
    }
    const bf16_t* base = uniform_ptr(a.w + (int64_t)kt * 32 * a.ld);
    const int last = min(31, a.E - 1 - kt * 32);
    if (last == 31) {
#pragma unroll
      for (int q = 0; q < QX; ++q) dma_b128(base, offw[q], tw + q * 1024);
    } else {
#pragma unroll
      for (int q = 0; q < QX; ++q)
        dma_b128(base, min(row_of(CX, QX, q), last) * ldw + colw[q], tw + q * 1024);
    }
  };
  f32x16_t acc[2][FC] = {};
  for (int kt = 0; kt < DN - 1 && kt < nk; ++kt) issue(kt);
  for (int kt = 0; kt < nk; ++kt) {
    if (DN == 3 && kt + 1 < nk) {       // the next step's instructions may stay in flight
      __builtin_amdgcn_s_waitcnt((4 + QX) | (7 << 4));
      lds_barrier();
    } else {
      publish();
    }
    if (kt + DN - 1 < nk) issue(kt + DN - 1);
    const uint32_t at = lds0 + kt % DN * DST;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      bf16x8_t fw[FC];
#pragma unroll
      for (int j = 0; j < FC; ++j) fw[j] = frag_t<XC / 8>(at + 16384, wc + 32 * j, s, lane);
#pragma unroll
      for (int p = 1; p >= 0; --p)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int r = wt + 32 * i + l;
          const int off = (int)(at - lds0) + p * 8192 + r * 64 + (((2 * s + h) ^ ((r >> 2) & 3)) << 4);
          const bf16x8_t fp = *(const bf16x8_t*)(lds + off);
#pragma unroll
          for (int j = 0; j < FC; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fw[j], fp, acc[i][j], 0, 0, 0);
        }
    }
  }
  float* st = (float*)lds;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    __syncthreads();                    // the operands, or the first half, have been read
    if ((wid >> 1) == half) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < FC; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q)
            *(float4*)(st + (32 * i + l) * OLD + wc + 32 * j + 8 * q + 4 * h) =
                make_float4(acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2],
                            acc[i][j][4 * q + 3]);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NI / 2; ++i) {
      const int r = i * RP + tid / TR;
      const int64_t t = t0 + half * 64 + r;
      const int c = c0 + tid % TR * 8;
      if (t >= a.T || c >= a.d) continue;
      const float* q = st + r * OLD + tid % TR * 8;
      const float4 u = *(const float4*)q, v = *(const float4*)(q + 4);
      const u32x4 w = in[half * (NI / 2) + i];
      const float s[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
      u32x4 o;
#pragma unroll
      for (int n = 0; n < 4; ++n)
        o[n] = pack_bf16x2(__uint_as_float(w[n] << 16) + s[2 * n],
                           __uint_as_float(w[n] & 0xFFFF0000u) + s[2 * n + 1]);
      bf16_t* at = a.dx + t * a.d + c;
      if constexpr (PAD) store_part(at, a.d - c, o);
      else __builtin_nontemporal_store(o, (u32x4*)at);
    }
  }
}

// out = the n partial sums of each element, in ascending order (n == 0: zeros).
__global__ __launch_bounds__(256) void k_route_bwd_sum(const float* __restrict__ part, int n,
                                                       int64_t elems, float* __restrict__ out) {
  for (int64_t i = blockIdx.x * (int64_t)256 + threadIdx.x; i < elems;
       i += (int64_t)gridDim.x * 256) {
    float v = 0.0f;
#pragma unroll 8
    for (int q = 0; q < n; ++q) v += part[q * elems + i];
    out[i] = v;
  }
}

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// The any-size form's shapes: dl (if written) padded to whole tiles; dW's token ranges, as many as
// give about two workgroups a CU, each of at least 64 tokens.
struct RbAny {
  bool few;                           // k_route_bwd_few
  bool write_dl;
  int EP;
  int64_t Tp, ranges, t_range;
  size_t dl, total;                   // bytes; the partial sums follow dl
};
RbAny rb_any(int64_t T, int d, int E, bool f32) {
  RbAny p;
  p.EP = (int)cdiv(E, RB_TILE) * RB_TILE;
  p.Tp = cdiv(T, RB_TILE) * RB_TILE;
  const int64_t tiles = cdiv(d, RB_TILE) * cdiv(E, RB_TILE);
  // a column a thread: narrow rows leave threads idle, which costs the form of 16 experts most
  // (float32, few and any-size form: T 70,000, d 61, E 5: 57 and 56 us, E 16: 85 and 56; T 40,000, d 128,
  // E 4: 46 and 52, E 16: 65 and 53; T 24,000, d 192, E 16: 40 and 50; T 300,000, d 16, E 4: 110 and 139)
  p.few = f32 && (E <= 8 || (E <= 16 && d > 128)) && T * d >= (int64_t)1 << 22;
  const int64_t n = std::max<int64_t>(
      1, std::min(p.few ? cdiv(1024, cdiv(d, RB_NT)) : cdiv(512, tiles), cdiv(T, 64)));
  const int unit = p.few ? 64 : RB_K;
  p.t_range = std::max<int64_t>(1, cdiv(cdiv(T, n), unit)) * unit;
  p.ranges = std::max<int64_t>(1, cdiv(T, p.t_range));
  p.write_dl = !p.few && (double)T * d * E >= (double)(1 << 27);
  p.dl = p.write_dl ? (size_t)p.Tp * p.EP * sizeof(float) : 0;
  p.total = std::max<size_t>(256, p.dl + (p.ranges > 1 ? (size_t)p.ranges * E * d * sizeof(float) : 0));
  return p;
}

// The plane form's shapes: experts padded to the tile EM, tokens to dx's tiles, dW's ranges.
struct RbPlan {
  int EM, EP, XC;                     // XC: a tile's columns
  int64_t Tp, ranges, t_range;
  int ld;                             // a row of x and w, as the tiles read them
  size_t planes, copies, total;       // bytes: dl's planes, padded x and w, then the partial sums
};
RbPlan rb_plan(int64_t T, int d, int E) {
  RbPlan p;
  p.EP = (int)cdiv(E, 64) * 64;
  if (p.EP > 64) p.EP = (int)cdiv(E, 128) * 128;
  p.EM = p.EP == 64 ? 64 : 128;
  p.Tp = cdiv(T, 128) * 128;
  // tiles of 256 columns read a third less into LDS, but fill the chip only with three dx tiles a CU
  // (128 against 256 columns: T 4096, d 7168, E 256: 101 and 93 us; T 16384, d 4096, E 32: 101 and
  // 89; T 8192, d 4096, E 128: 72 and 71; T 4096, d 2048, E 128: 30 and 31; T 512, d 2048, E 128:
  // 18 and 23)
  p.XC = cdiv(T, 128) * cdiv(d, 256) >= 768 ? 256 : 128;
  // dW workgroups: one a CU of 128 columns (T 8192, d 2048, E 64: 38 us with 112 of them, 31 with
  // 256, 36 with 300), fewer of 256, whose partial sums cost more (T 4096, d 7168, E 256: 112 us
  // with 112, 93 with 168, 99 with 224)
  const int64_t tiles = cdiv(d, p.XC) * (p.EP / p.EM);
  const int64_t n = std::max<int64_t>(1, std::min(cdiv(p.XC == 256 ? 160 : 256, tiles), cdiv(T, 256)));
  p.t_range = cdiv(cdiv(T, n), 64) * 64;
  p.ranges = cdiv(T, p.t_range);
  p.planes = (size_t)3 * p.Tp * p.EP * 2;
  p.ld = (int)cdiv(d, 8) * 8;
  p.copies = p.ld == d ? 0 : (size_t)(T + E) * p.ld * 2;
  p.total = p.planes + p.copies + (p.ranges > 1 ? (size_t)p.ranges * E * d * sizeof(float) : 0);
  return p;
}

// bf16 rows that the plane form takes: whole pieces of 16 bytes, or, where the products outweigh a
// launch more and a copy of x and the weight in such rows, any (T 257, d 275, E 20: 12.6 us in the
// any-size form, 15.9 in this; T 512, d 1069, E 64: 19.4 and 18.8; T 5536, d 1069, E 212: 153 and 53;
// T 2100, d 2003, E 1: 44 and 25).
bool rb_tiled(int64_t T, int d, int E) {
  return d % 8 == 0 || T * d >= 1 << 22 || (double)T * d * E >= (double)(1 << 25);
}

int rb_check(int64_t T, int32_t d, int32_t E, int32_t k, int32_t io_dtype) {
  if (T < 0 || d < 1 || d > (1 << 24) || E < 1 || E > 1024 || k < 1 || k > E || k > 64)
    return MOK_EINVAL;
  if (T * (int64_t)k >= (int64_t)1 << 31) return MOK_EINVAL;
  return io_dtype == MOK_FP32 || io_dtype == MOK_BF16 ? MOK_OK : MOK_EINVAL;
}

}  // namespace
}  // namespace mok

using namespace mok;

extern "C" {

int mok_route_backward_workspace_bytes(int64_t T, int32_t d, int32_t E, int32_t io_dtype,
                                       size_t* bytes) {
  if (!bytes || rb_check(T, d, E, 1, io_dtype) != MOK_OK) return MOK_EINVAL;
  size_t need = rb_any(T, d, E, io_dtype == MOK_FP32).total;
  if (io_dtype == MOK_BF16 && T > 0 && rb_tiled(T, d, E)) need = std::max(need, rb_plan(T, d, E).total);
  *bytes = need;
  return MOK_OK;
}

int mok_route_backward(const void* x, const void* w_router, const int32_t* topk_idx,
                       const float* topk_w, const float* dtopk_w, const float* dlogits,
                       const void* dx_in, int64_t T, int32_t d, int32_t E, int32_t k,
                       int32_t io_dtype, void* dx, float* dw_router, void* ws, size_t ws_bytes,
                       void* stream) {
  const int st = rb_check(T, d, E, k, io_dtype);
  if (st != MOK_OK) return st;
  if (!dx && !dw_router && T > 0) return MOK_EINVAL;
  if (T > 0 && (!topk_idx || !topk_w || !dtopk_w || (dx && !w_router) || (dw_router && !x)))
    return MOK_EINVAL;
  size_t need = 0;
  mok_route_backward_workspace_bytes(T, d, E, io_dtype, &need);
  if (!ws || ws_bytes < need || (uintptr_t)ws % 16) return MOK_EWORKSPACE;
  hipStream_t s = (hipStream_t)stream;
  const int64_t elems = (int64_t)E * d;
  const unsigned sum_grid = (unsigned)std::min<int64_t>(cdiv(elems, 256), 4096);
  if (T == 0) {
    if (dw_router)
      launch_k(k_route_bwd_sum, dim3(sum_grid), dim3(256), 0, s, nullptr, nullptr,
               (const float*)ws, 0, elems, dw_router);
    return hipGetLastError() == hipSuccess ? MOK_OK : MOK_EHIP;
  }
  RbArgs a = {};
  a.x = x; a.w = w_router; a.idx = topk_idx; a.tw = topk_w; a.dtw = dtopk_w; a.dlogits = dlogits;
  a.dx_in = dx_in; a.dx = dx; a.T = T; a.d = d; a.E = E; a.k = k;
  auto al16 = [](const void* p) { return (uintptr_t)p % 16 == 0; };
  const bool aligned = al16(x) && al16(w_router) && al16(dx_in) && al16(dx) && al16(dw_router);
  if (io_dtype == MOK_BF16 && rb_tiled(T, d, E) && (aligned || d % 8)) {
    const RbPlan p = rb_plan(T, d, E);
    RbTile t;
    t.x = (const bf16_t*)x; t.w = (const bf16_t*)w_router; t.dx_in = (const bf16_t*)dx_in;
    t.planes = (const bf16_t*)ws; t.dx = (bf16_t*)dx;
    t.dw = p.ranges > 1 ? (float*)((char*)ws + p.planes + p.copies) : dw_router;
    t.ld = p.ld;
    t.T = T; t.Tp = p.Tp; t.d = d; t.E = E; t.EP = p.EP;
    t.tiles_d = (int)cdiv(d, p.XC);
    t.tiles_e = p.EP / p.EM;
    t.t_range = p.t_range;
    const int64_t n_dw = dw_router ? p.ranges * t.tiles_e * t.tiles_d : 0;
    const int64_t n_dx = dx ? p.Tp / 128 * t.tiles_d : 0, n_pl = cdiv(p.Tp * (p.EP / 8), 256);
    const int64_t n = cdiv(n_dw, 8) * 8 + cdiv(n_dx, 8) * 8;
    if (n * RB_NT >= (int64_t)1 << 32 || n_pl * 256 >= (int64_t)1 << 32) return MOK_EUNSUPPORTED;
    t.dw_tiles = (int)n_dw;
    t.dx_tiles = (int)n_dx;
    t.dw_blocks = (int)(cdiv(n_dw, 8) * 8);
    launch_k(k_route_bwd_dl<true>, dim3((unsigned)n_pl), dim3(256), 0, s, nullptr, nullptr, a, p.EP,
             p.Tp, ws);
    if (hipGetLastError() != hipSuccess) return MOK_EHIP;
    if (p.copies) {
      bf16_t* const to = (bf16_t*)((char*)ws + p.planes);
      launch_k(k_route_bwd_pad, dim3((unsigned)std::min<int64_t>(cdiv((T + E) * (p.ld / 8), 256), 8192)),
               dim3(256), 0, s, nullptr, nullptr, dw_router ? t.x : nullptr, T, dx ? t.w : nullptr, E,
               d, p.ld, to);
      if (hipGetLastError() != hipSuccess) return MOK_EHIP;
      t.x = to;
      t.w = to + T * p.ld;
    }
    auto pick = [&](auto PAD) {
      constexpr bool pad = PAD();
      return p.XC == 256
                 ? (p.EM == 64 ? k_route_bwd_tile<64, 256, pad> : k_route_bwd_tile<128, 256, pad>)
                 : (p.EM == 64 ? k_route_bwd_tile<64, 128, pad> : k_route_bwd_tile<128, 128, pad>);
    };
    auto k = p.copies ? pick(std::true_type{}) : pick(std::false_type{});
    launch_k(k, dim3((unsigned)n), dim3(RB_NT), 0, s, nullptr, nullptr, t);
    if (hipGetLastError() != hipSuccess) return MOK_EHIP;
    if (dw_router && p.ranges > 1)
      launch_k(k_route_bwd_sum, dim3(sum_grid), dim3(256), 0, s, nullptr, nullptr,
               (const float*)t.dw, (int)p.ranges, elems, dw_router);
    return hipGetLastError() == hipSuccess ? MOK_OK : MOK_EHIP;
  }
  const RbAny p = rb_any(T, d, E, io_dtype == MOK_FP32);
  a.dl = (const float*)ws;
  a.EP = p.EP;
  a.tiles_d = (int)cdiv(d, RB_TILE);
  a.tiles_e = p.EP / RB_TILE;
  a.dx_tiles = dx ? p.Tp / RB_TILE * a.tiles_d : 0;
  a.t_range = p.t_range;
  float* const part = (float*)((char*)ws + p.dl);
  a.dw = p.ranges > 1 ? part : dw_router;
  if (p.few) {
    if (!dw_router) a.dw = nullptr;
    auto kern = E <= 4 ? k_route_bwd_few<4> : E <= 8 ? k_route_bwd_few<8> : k_route_bwd_few<16>;
    launch_k(kern, dim3((unsigned)cdiv(d, RB_NT), (unsigned)p.ranges), dim3(RB_NT), 0, s, nullptr,
             nullptr, a);
    if (hipGetLastError() != hipSuccess) return MOK_EHIP;
    if (dw_router && p.ranges > 1)
      launch_k(k_route_bwd_sum, dim3(sum_grid), dim3(256), 0, s, nullptr, nullptr,
               (const float*)part, (int)p.ranges, elems, dw_router);
    return hipGetLastError() == hipSuccess ? MOK_OK : MOK_EHIP;
  }
  const int64_t grid = a.dx_tiles + (dw_router ? p.ranges * a.tiles_e * a.tiles_d : 0);
  const int64_t n_dl = cdiv(p.Tp * (p.EP / 8), 256);
  if (grid * RB_NT >= (int64_t)1 << 32 || n_dl * 256 >= (int64_t)1 << 32) return MOK_EUNSUPPORTED;
  if (p.write_dl) {
    launch_k(k_route_bwd_dl<false>, dim3((unsigned)n_dl), dim3(256), 0, s, nullptr, nullptr, a,
             p.EP, p.Tp, ws);
    if (hipGetLastError() != hipSuccess) return MOK_EHIP;
  }
  const bool bf = io_dtype == MOK_BF16;
  auto kern = p.write_dl ? (bf ? k_route_bwd_any<bf16_t, true> : k_route_bwd_any<float, true>)
                         : (bf ? k_route_bwd_any<bf16_t, false> : k_route_bwd_any<float, false>);
  launch_k(kern, dim3((unsigned)grid), dim3(RB_NT), 0, s, nullptr, nullptr, a);
  if (hipGetLastError() != hipSuccess) return MOK_EHIP;
  if (dw_router && p.ranges > 1)
    launch_k(k_route_bwd_sum, dim3(sum_grid), dim3(256), 0, s, nullptr, nullptr, (const float*)part,
             (int)p.ranges, elems, dw_router);
  return hipGetLastError() == hipSuccess ? MOK_OK : MOK_EHIP;
}

}  // extern "C"
