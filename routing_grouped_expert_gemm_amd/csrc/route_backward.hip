// Gradients through the router: from the gradients of the routing weights (and of the logits, as
// the balance loss gives them) to the router's input and its weight.
//
//   dl[t,e]  = dlogits[t,e] + sum_{j: idx[t,j] = e} w[t,j] (dw[t,j] - sum_i w[t,i] dw[t,i])
//   dx[t,i]  = dx_in[t,i] + sum_e dl[t,e] W[e,i]
//   dW[e,i]  = sum_t dl[t,e] x[t,i]
//
// (w = softmax over a token's picks, so its gradient is the softmax's.) The picks are held
// fixed. dl is never written out as a whole: a workgroup builds the part it needs in LDS from the
// picks and the given dlogits.
//
// This form takes any size and alignment: 64 x 64 tiles of both products on the float32 MFMA
// (operands and sums in float32), 4 waves of 32 x 32, K steps of 32 through LDS. dW's token sum
// is cut into ranges (one per grid z) whose partial sums a second launch adds in order: no
// atomics, the same bits every run.
#include <algorithm>

#include "device_common.h"
#include "launch.h"
#include "mok.h"

namespace mok {
namespace {

constexpr int RB_NT = 256, RB_TILE = 64, RB_K = 32, RB_PAD = 4;

struct RbArgs {
  const void *x, *w;
  const int32_t* idx;
  const float *tw, *dtw, *dlogits;
  const void* dx_in;
  void* dx;
  float* dw;          // dW itself (one range) or its partial sums [ranges, E, d]
  int64_t T;
  int d, E, k;
  int tiles_d;        // tiles of 64 columns
  int64_t dx_tiles;   // workgroups of the dx product; the rest are dW's
  int tiles_e;
  int64_t t_range;    // tokens of one dW range (a multiple of RB_K)
};

// sum_i w[t,i] dw[t,i] over the token's picks inside [0, E), in pick order.
MOK_DEV float pick_dot(const RbArgs& a, int64_t t) {
  float s = 0.0f;
  for (int j = 0; j < a.k; ++j) {
    const int32_t e = a.idx[t * a.k + j];
    if (e >= 0 && e < a.E) s += a.tw[t * a.k + j] * a.dtw[t * a.k + j];
  }
  return s;
}

// dl of tokens [t0, t0 + nt) and experts [e0, e0 + ne), zero past the tensors, at
// buf[row * ld + column] (E_MAJOR: row = expert). nt <= RB_NT. Ends with a barrier.
template <bool E_MAJOR>
MOK_DEV void build_dl(const RbArgs& a, int64_t t0, int nt, int e0, int ne, float* buf, int ld) {
  for (int i = threadIdx.x; i < nt * ne; i += RB_NT) {
    const int e = i % ne, t = i / ne;
    const bool ok = t0 + t < a.T && e0 + e < a.E;
    buf[E_MAJOR ? e * ld + t : t * ld + e] =
        ok && a.dlogits ? a.dlogits[(t0 + t) * a.E + e0 + e] : 0.0f;
  }
  __syncthreads();
  if ((int)threadIdx.x < nt && t0 + threadIdx.x < a.T) {
    const int64_t t = t0 + threadIdx.x;
    const float s = pick_dot(a, t);
    for (int j = 0; j < a.k; ++j) {          // in pick order: a repeated expert adds up
      const int e = a.idx[t * a.k + j] - e0;
      if (e >= 0 && e < ne && e0 + e < a.E) {
        float* q = &buf[E_MAJOR ? e * ld + threadIdx.x : threadIdx.x * ld + e];
        *q += a.tw[t * a.k + j] * (a.dtw[t * a.k + j] - s);
      }
    }
  }
  __syncthreads();
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
template <class T>
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
  // rows of B: T or E rows of `src` [.., d] from row k0, columns c0 ..
  auto load_b = [&](const T* src, int64_t k0, int64_t rows) {
    for (int i = threadIdx.x; i < RB_K * RB_TILE; i += RB_NT) {
      const int c = i % RB_TILE, r = i / RB_TILE;
      B[r * LD + c] = k0 + r < rows && c0 + c < a.d ? load_as_f32(src + (k0 + r) * a.d + c0 + c)
                                                    : 0.0f;
    }
  };
  if (is_dx) {
    const int64_t t0 = rest * RB_TILE;
    for (int e0 = 0; e0 < a.E; e0 += RB_K) {
      load_b((const T*)a.w, e0, a.E);
      build_dl<true>(a, t0, RB_TILE, e0, RB_K, A, LD);
      mma_step(A, B, am, bn, acc);
      __syncthreads();
    }
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
    const int e0 = (int)(rest % a.tiles_e) * RB_TILE;
    const int64_t range = rest / a.tiles_e;
    const int64_t t_end = min(a.T, (range + 1) * a.t_range);
    for (int64_t t0 = range * a.t_range; t0 < t_end; t0 += RB_K) {
      load_b((const T*)a.x, t0, a.T);
      build_dl<false>(a, t0, RB_K, e0, RB_TILE, A, LD);
      mma_step(A, B, am, bn, acc);
      __syncthreads();
    }
    float* out = a.dw + range * a.E * a.d;
#pragma unroll
    for (int v = 0; v < 16; ++v) {
      const int e = e0 + am + 8 * (v >> 2) + 4 * h + (v & 3), c = c0 + bn + l;
      if (e < a.E && c < a.d) out[(int64_t)e * a.d + c] = acc[v];
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

// Token ranges of dW: as many as give about two workgroups a CU, each of at least 256 tokens.
int64_t any_ranges(int64_t T, int d, int E) {
  const int64_t tiles = cdiv(d, RB_TILE) * cdiv(E, RB_TILE);
  return std::max<int64_t>(1, std::min(cdiv(512, tiles), cdiv(T, 256)));
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
  const int64_t n = any_ranges(T, d, E);
  *bytes = n > 1 ? (size_t)n * E * d * sizeof(float) : 256;
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
  if (dw_router && (!ws || ws_bytes < need || (uintptr_t)ws % 16)) return MOK_EWORKSPACE;
  hipStream_t s = (hipStream_t)stream;
  const int64_t elems = (int64_t)E * d;
  const unsigned sum_grid = (unsigned)std::min<int64_t>(cdiv(elems, 256), 4096);
  if (T == 0) {
    if (dw_router)
      launch_k(k_route_bwd_sum, dim3(sum_grid), dim3(256), 0, s, nullptr, nullptr,
               (const float*)ws, 0, elems, dw_router);
    return hipGetLastError() == hipSuccess ? MOK_OK : MOK_EHIP;
  }
  RbArgs a;
  a.x = x; a.w = w_router; a.idx = topk_idx; a.tw = topk_w; a.dtw = dtopk_w; a.dlogits = dlogits;
  a.dx_in = dx_in; a.dx = dx; a.T = T; a.d = d; a.E = E; a.k = k;
  a.tiles_d = (int)cdiv(d, RB_TILE);
  a.tiles_e = (int)cdiv(E, RB_TILE);
  a.dx_tiles = dx ? cdiv(T, RB_TILE) * a.tiles_d : 0;
  const int64_t ranges = dw_router ? any_ranges(T, d, E) : 0;
  a.t_range = ranges ? cdiv(cdiv(T, ranges), RB_K) * RB_K : RB_K;
  a.dw = ranges > 1 ? (float*)ws : dw_router;
  const int64_t grid = a.dx_tiles + ranges * a.tiles_e * a.tiles_d;
  if (grid * RB_NT >= (int64_t)1 << 32) return MOK_EUNSUPPORTED;
  if (io_dtype == MOK_BF16)
    launch_k(k_route_bwd_any<bf16_t>, dim3((unsigned)grid), dim3(RB_NT), 0, s, nullptr, nullptr, a);
  else
    launch_k(k_route_bwd_any<float>, dim3((unsigned)grid), dim3(RB_NT), 0, s, nullptr, nullptr, a);
  if (hipGetLastError() != hipSuccess) return MOK_EHIP;
  if (ranges > 1)
    launch_k(k_route_bwd_sum, dim3(sum_grid), dim3(256), 0, s, nullptr, nullptr, (const float*)ws,
             (int)ranges, elems, dw_router);
  return hipGetLastError() == hipSuccess ? MOK_OK : MOK_EHIP;
}

}  // extern "C"
