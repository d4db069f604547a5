// Residual addition + root-mean-square norm, with an output in the storage type, in MXFP8, or
// both, and the norm's backward.
//
//   h = x + residual (rounded to the storage type: the residual stream)
//   rstd[t] = 1 / sqrt(mean_i h[t,i]^2 + eps)          y[t,i] = h[t,i] rstd[t] weight[i]
//   backward, g = dy weight, n = h rstd:
//   dx[t,i] = rstd (g[t,i] - n[t,i] mean_j(g[t,j] n[t,j])) + dh[t,i]
//   dweight[i] = sum_t dy[t,i] n[t,i]
//
// The norm reads h as it is stored, so the backward, which is given the stored h, differentiates
// exactly the function that the forward computed. The sum of squares and rstd are float64 and y is
// h w rstd rounded once to float32 (then to the output type): every value of a row hangs on rstd,
// and codes next to a border of two would flip with its last bit. Gradients are float32, each
// output rounded once. MXFP8 codes come from the float32 y, by the rules of mok_quantize_mxfp8_f32.
//
// HBM streams: a row stays in registers between its sum of squares and its output, so each input
// is read once and each output written once. TPR threads hold a row in NC pieces of 8 values.
#include <algorithm>

#include "device_common.h"
#include "launch.h"
#include "mok.h"
#include "norm_common.h"

namespace mok {
namespace {

// The 8 E4M3 codes of a lane's piece and its 32-value block's scale byte (the aligned quad of
// lanes holds the block). A block with an infinity or a NaN is NaN: code 0x7F, scale 0xFF.
MOK_DEV uint2 mx8_codes(const float (&v)[8], uint8_t* scale) {
  bool bad = false;
#pragma unroll
  for (int i = 0; i < 8; ++i) bad |= !(fabsf(v[i]) < INFINITY);
  int b = bad;
  b |= __shfl_xor(b, 1, kWave);
  b |= __shfl_xor(b, 2, kWave);
  int s;
  uint2 c = quantize_quad8_f32(v, &s);
  if (b) {
    c = make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
    s = 128;
  }
  *scale = (uint8_t)(s + 127);
  return c;
}

// A workgroup of max(TPR, 256) threads holds 256 / TPR rows (at least one). res, h_out, rstd, y,
// codes (with scales): NULL where not wanted.
template <class T, int TPR, int NC>
__global__ __launch_bounds__(TPR > NORM_NT ? TPR : NORM_NT) void k_rmsnorm(
    const T* x, const T* res, const T* __restrict__ weight, int64_t rows, int d, float eps,
    T* h_out, float* __restrict__ rstd_out, T* y, uint8_t* __restrict__ codes,
    uint8_t* __restrict__ scales) {
  constexpr int NT = TPR > NORM_NT ? TPR : NORM_NT, RPB = NT / TPR;
  __shared__ double sh[NT / 64];
  const int l = threadIdx.x % TPR;
  const int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR;
  const bool live = row < rows;
  const int64_t at = row * d;
  float h[NC][8];
  double ss = 0.0;
#pragma unroll
  for (int n = 0; n < NC; ++n) {
    const int c = (n * TPR + l) * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) h[n][i] = 0.0f;
    if (live && c < d) {
      Piece<T>::load(x + at + c, h[n]);
      if (res) {
        float r[8];
        Piece<T>::load(res + at + c, r);
#pragma unroll
        for (int i = 0; i < 8; ++i) h[n][i] = as_stored<T>(h[n][i] + r[i]);
      }
    }
  }
#pragma unroll
  for (int n = 0; n < NC; ++n) {
    const int c = (n * TPR + l) * 8;
    if (h_out && live && c < d) Piece<T>::store(h_out + at + c, h[n]);
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fma((double)h[n][i], (double)h[n][i], ss);
  }
  const double rd = 1.0 / sqrt(row_total<TPR>(ss, sh) / d + eps);
  const RowScale rs(rd);
  if (rstd_out && live && l == 0) rstd_out[row] = (float)rd;
#pragma unroll
  for (int n = 0; n < NC; ++n) {
    const int c = (n * TPR + l) * 8;
    const bool ok = live && c < d;
    float w[8] = {0, 0, 0, 0, 0, 0, 0, 0}, v[8];
    if (ok) Piece<T>::load(weight + c, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = norm_value<T>(h[n][i], w[i], rs);
    if (y && ok) Piece<T>::store(y + at + c, v);
    if (codes) {                   // d % 32 == 0: a quad's four lanes are all inside the row
      uint8_t s;
      const uint2 q = mx8_codes(v, &s);
      if (ok) {
        *(uint2*)(codes + at + c) = q;
        if ((l & 3) == 0) scales[(at + c) >> 5] = s;
      }
    }
  }
}

// Any d and alignment: one workgroup a row, one value a thread and step (one 32-value block a
// thread for the codes). The second pass reads back what the first stored in h_out.
template <class T, int NT>
__global__ __launch_bounds__(NT) void k_rmsnorm_any(
    const T* x, const T* res, const T* weight, int64_t rows, int d, float eps, T* h_out,
    float* rstd_out, T* y, uint8_t* codes, uint8_t* scales) {
  __shared__ double sh[NT / 64];
  const int64_t row = blockIdx.x, at = row * d;
  auto sum_at = [&](int i) {
    const float v = load_as_f32(x + at + i);
    return res ? as_stored<T>(v + load_as_f32(res + at + i)) : v;
  };
  double ss = 0.0;
  for (int i = threadIdx.x; i < d; i += NT) {
    const float v = sum_at(i);
    if (h_out) h_out[at + i] = f32_to<T>(v);
    ss = fma((double)v, (double)v, ss);
  }
  ss = row_total<NT>(ss, sh);
  __syncthreads();                 // the row's h is written: other threads read it below
  const double rd = 1.0 / sqrt(ss / d + eps);
  const RowScale rs(rd);
  if (rstd_out && threadIdx.x == 0) rstd_out[row] = (float)rd;
  auto h_at = [&](int i) { return h_out ? load_as_f32(h_out + at + i) : sum_at(i); };
  auto y_at = [&](int i) { return norm_value<T>(h_at(i), load_as_f32(weight + i), rs); };
  if (codes) {
    for (int b = threadIdx.x; b < d / 32; b += NT) {
      float amax = 0.0f;
      bool bad = false;
      for (int i = 0; i < 32; ++i) {
        const float v = fabsf(y_at(32 * b + i));
        bad |= !(v < INFINITY);
        amax = fmaxf(amax, v);
      }
      const int s = mx_shared_exp(amax);
      for (int i = 0; i < 32; ++i)
        codes[at + 32 * b + i] = bad ? 0x7F : (uint8_t)e4m3_encode(y_at(32 * b + i), s);
      scales[(at >> 5) + b] = bad ? 0xFF : (uint8_t)(s + 127);
    }
    __syncthreads();               // y may be x: its first write follows the codes' last read
  }
  if (y)
    for (int i = threadIdx.x; i < d; i += NT) y[at + i] = f32_to<T>(y_at(i));
}

// Backward over rows blockIdx.x * RPB + ..., stepping by the whole grid: dweight's sums stay in
// registers from row to row. part [gridDim.x, d]: this workgroup's share of dweight (NULL: none).
template <class T, int TPR, int NC>
__global__ __launch_bounds__(TPR > NORM_NT ? TPR : NORM_NT) void k_rmsnorm_bwd(
    const T* dy, const T* __restrict__ h, const float* __restrict__ rstd,
    const T* __restrict__ weight, const T* dh, int64_t rows, int d, T* dx,
    float* __restrict__ part) {
  constexpr int NT = TPR > NORM_NT ? TPR : NORM_NT, RPB = NT / TPR;
  __shared__ float sh[2][NT / 64];
  __shared__ double shd[NT / 64];
  __shared__ float fold[RPB > 1 ? RPB : 1][RPB > 1 ? TPR * NC * 8 : 1];
  const int l = threadIdx.x % TPR, r = threadIdx.x / TPR;
  float w[NC][8], acc[NC][8];
#pragma unroll
  for (int n = 0; n < NC; ++n) {
    const int c = (n * TPR + l) * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) w[n][i] = acc[n][i] = 0.0f;
    if (c < d) Piece<T>::load(weight + c, w[n]);
  }
  // The next row's loads are issued before this row's sum: a workgroup walks only a few rows, and
  // a row's loads, sum and store in sequence left the memory idle in between.
  typedef typename Piece<T>::Raw Raw;
  Raw hq[NC], gq[NC], oq[NC];
  auto fetch = [&](int64_t row) {
    const bool live = row < rows;
#pragma unroll
    for (int n = 0; n < NC; ++n) {
      const int c = (n * TPR + l) * 8;
      const int64_t at = row * d + c;
      const bool ok = live && c < d;
      hq[n] = ok ? Piece<T>::raw(h + at) : Piece<T>::none();
      gq[n] = ok ? Piece<T>::raw(dy + at) : Piece<T>::none();
      oq[n] = ok && dh ? Piece<T>::raw(dh + at) : Piece<T>::none();
    }
    return live ? rstd[row] : 0.0f;
  };
  int turn = 0;
  const int64_t stride = (int64_t)gridDim.x * RPB;
  float rs_next = fetch((int64_t)blockIdx.x * RPB + r);
  for (int64_t r0 = (int64_t)blockIdx.x * RPB; r0 < rows; r0 += stride) {
    const int64_t row = r0 + r, at = row * d;
    const bool live = row < rows;
    float n_[NC][8], g[NC][8], o[NC][8], dot = 0.0f;
#pragma unroll
    for (int n = 0; n < NC; ++n) {
      Piece<T>::widen(hq[n], n_[n]);
      Piece<T>::widen(gq[n], g[n]);
      Piece<T>::widen(oq[n], o[n]);
    }
    const BwdScale q(rs_next, d, [&] {
      double ss = 0.0;
#pragma unroll
      for (int n = 0; n < NC; ++n)
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fma((double)n_[n][i], (double)n_[n][i], ss);
      return row_total<TPR>(ss, shd);         // the sum of dot lies between two uses of shd
    });
    const float rs = q.rs;
    if (q.scale != 1.0f)
#pragma unroll
      for (int n = 0; n < NC; ++n)
#pragma unroll
        for (int i = 0; i < 8; ++i) n_[n][i] *= q.scale;
    rs_next = fetch(row + stride);
#pragma unroll
    for (int n = 0; n < NC; ++n)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        n_[n][i] *= rs;
        acc[n][i] += g[n][i] * n_[n][i];
        g[n][i] *= w[n][i];
        dot += g[n][i] * n_[n][i];
      }
    dot = row_total<TPR>(dot, sh[turn]) / (float)d;
    turn ^= 1;
#pragma unroll
    for (int n = 0; n < NC; ++n) {
      const int c = (n * TPR + l) * 8;
      if (live && c < d) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float v = g[n][i] - n_[n][i] * dot;
          o[n][i] = q.scale == 1.0f ? fmaf(rs, v, o[n][i]) : fmaf(q.scale, rs * v, o[n][i]);
        }
        Piece<T>::store(dx + at + c, o[n]);
      }
    }
  }
  if (!part) return;
  float* out = part + (int64_t)blockIdx.x * d;
  if constexpr (RPB == 1) {
#pragma unroll
    for (int n = 0; n < NC; ++n) {
      const int c = (n * TPR + l) * 8;
      if (c < d) Piece<float>::store(out + c, acc[n]);
    }
  } else {
#pragma unroll
    for (int n = 0; n < NC; ++n) Piece<float>::store(&fold[r][(n * TPR + l) * 8], acc[n]);
    __syncthreads();
    for (int c = threadIdx.x; c < d; c += NT) {
      float v = fold[0][c];
#pragma unroll
      for (int q = 1; q < RPB; ++q) v += fold[q][c];
      out[c] = v;
    }
  }
}

// Any d and alignment, first launch: workgroup (x, y) sums dweight's columns 256 x .. over the
// rows y, y + gridDim.y, ... It runs before dx is written, which may lie where dy does.
template <class T>
__global__ __launch_bounds__(NORM_NT) void k_rmsnorm_dw_any(const T* dy, const T* h,
                                                            const float* rstd, int64_t rows, int d,
                                                            float* part) {
  __shared__ double shd[NORM_NT / 64];
  const int c = blockIdx.x * NORM_NT + threadIdx.x, at = min(c, d - 1);
  float v = 0.0f, top = 0.0f;                 // top: the largest rstd, the same in every thread
  for (int64_t row = blockIdx.y; row < rows; row += gridDim.y) {
    const float rs = rstd[row];
    top = fmaxf(top, rs);
    v += load_as_f32(dy + row * d + at) * (load_as_f32(h + row * d + at) * rs);
  }
  if (top == INFINITY) {                      // once more, with rstd from h where it is an infinity
    v = 0.0f;
    for (int64_t row = blockIdx.y; row < rows; row += gridDim.y) {
      const BwdScale q(rstd[row], d, [&] {
        __syncthreads();                      // shd of a row before has been read
        return row_total<NORM_NT>(squares<NORM_NT>(h + row * d, d), shd);
      });
      v += load_as_f32(dy + row * d + at) * (load_as_f32(h + row * d + at) * q.scale * q.rs);
    }
  }
  if (c < d) part[(int64_t)blockIdx.y * d + c] = v;
}

template <class T, int NT>
__global__ __launch_bounds__(NT) void k_rmsnorm_bwd_any(const T* dy, const T* h,
                                                             const float* rstd, const T* weight,
                                                             const T* dh, int d, T* dx) {
  __shared__ float sh[NT / 64];
  __shared__ double shd[NT / 64];
  const int64_t row = blockIdx.x, at = row * d;
  auto rest = [&](float rs, auto SCALED, float scale) {
    auto h_at = [&](int i) {
      const float v = load_as_f32(h + at + i);
      return SCALED() ? v * scale : v;
    };
    float dot = 0.0f;
    for (int i = threadIdx.x; i < d; i += NT)
      dot += load_as_f32(dy + at + i) * load_as_f32(weight + i) * (h_at(i) * rs);
    dot = row_total<NT>(dot, sh) / (float)d;
    for (int i = threadIdx.x; i < d; i += NT) {
      const float g = load_as_f32(dy + at + i) * load_as_f32(weight + i);
      float o = rs * (g - h_at(i) * rs * dot);
      if constexpr (SCALED()) o *= scale;
      dx[at + i] = f32_to<T>(o + (dh ? load_as_f32(dh + at + i) : 0.0f));
    }
  };
  const float rs = rstd[row];
  if (rs != INFINITY) {
    rest(rs, std::integral_constant<bool, false>{}, 1.0f);
  } else {
    const BwdScale q(rs, d, [&] { return row_total<NT>(squares<NT>(h + at, d), shd); });
    rest(q.rs, std::integral_constant<bool, true>{}, q.scale);
  }
}

// out[c] = sum of part[0 .. n)[c]: a workgroup takes 16 columns (one 64-byte segment of each row)
// and 64 groups of rows, each group's rows in ascending order, then the groups in a fixed tree.
// n == 0 writes zeros. (64 columns and 16 groups left 32 workgroups for 2,048 columns and took
// 11.4 us for 512 rows of them; this took 5 us.)
__global__ __launch_bounds__(1024) void k_column_sum(const float* __restrict__ part, int n, int d,
                                                     float* __restrict__ out) {
  __shared__ float sh[64][17];
  const int l = threadIdx.x & 15, g = threadIdx.x >> 4, c = blockIdx.x * 16 + l;
  float v = 0.0f;
  if (c < d)
    for (int i = g; i < n; i += 64) v += part[(int64_t)i * d + c];
  sh[g][l] = v;
  __syncthreads();
#pragma unroll
  for (int m = 32; m > 0; m >>= 1) {
    if (g < m) sh[g][l] += sh[g + m][l];
    __syncthreads();
  }
  if (g == 0 && c < d) out[c] = sh[0][l];
}

template <class T>
hipError_t run_norm(const T* x, const T* res, const T* weight, int64_t rows, int d, float eps,
                    T* h, float* rstd, T* y, uint8_t* codes, uint8_t* scales, hipStream_t s) {
  const bool vec = d % 8 == 0 && d <= 16384 && al16(x) && al16(res) && al16(weight) && al16(h) &&
                   al16(y) && (uintptr_t)codes % 8 == 0;
  if (rows > kMaxLaunchRows) {
    const int64_t n = kMaxLaunchRows, o = n * d;
    const hipError_t e = run_norm(x, res, weight, n, d, eps, h, rstd, y, codes, scales, s);
    if (e != hipSuccess) return e;
    auto skip = [](auto* p, int64_t k) { return p ? p + k : p; };
    return run_norm(x + o, skip(res, o), weight, rows - n, d, eps, skip(h, o), skip(rstd, n),
                    skip(y, o), skip(codes, o), skip(scales, o / 32), s);
  }
  auto go = [&](auto TPR, auto NC) {
    constexpr int nt = TPR() > NORM_NT ? TPR() : NORM_NT, rpb = nt / TPR();
    launch_k(k_rmsnorm<T, TPR(), NC()>, dim3((unsigned)((rows + rpb - 1) / rpb)), dim3(nt), 0, s,
             nullptr, nullptr, x, res, weight, rows, d, eps, h, rstd, y, codes, scales);
  };
  auto c = [](auto v) { return v; };
#define MOK_NORM(TPR, NC) go(c(std::integral_constant<int, TPR>{}), c(std::integral_constant<int, NC>{}))
  if (!vec)
    launch_k(d > 2048 ? k_rmsnorm_any<T, 1024> : k_rmsnorm_any<T, 256>, dim3((unsigned)rows),
             dim3(d > 2048 ? 1024 : 256), 0, s, nullptr, nullptr, x, res, weight, rows, d, eps, h,
             rstd, y, codes, scales);
  else if (d <= 512) MOK_NORM(64, 1);
  // few rows (fewer workgroups than CUs): more threads a row, for the row's latency
  else if (rows <= 256 && d <= 2048) MOK_NORM(256, 1);
  else if (rows <= 256 && d <= 8192) MOK_NORM(1024, 1);
  else if (d <= 1024) MOK_NORM(64, 2);
  else if (d <= 2048) MOK_NORM(64, 4);
  else if (d <= 4096) MOK_NORM(256, 2);
  else if (d <= 8192) MOK_NORM(256, 4);
  else MOK_NORM(1024, 2);
#undef MOK_NORM
  return hipGetLastError();
}

template <class T>
hipError_t run_bwd(const T* dy, const T* h, const float* rstd, const T* weight, const T* dh,
                   int64_t rows, int d, T* dx, float* dweight, float* part, hipStream_t s) {
  const int blocks = bwd_blocks(rows);
  const bool vec = d % 8 == 0 && d <= 8192 && al16(dy) && al16(h) && al16(weight) && al16(dh) &&
                   al16(dx);
  float* p = dweight ? part : nullptr;
  int n_part = rows > 0 ? blocks : 0;
  auto go = [&](auto TPR, auto NC) {
    constexpr int nt = TPR() > NORM_NT ? TPR() : NORM_NT, rpb = nt / TPR();
    const int grid = (int)std::min<int64_t>(dweight ? blocks : 1 << 16, (rows + rpb - 1) / rpb);
    n_part = grid;
    launch_k(k_rmsnorm_bwd<T, TPR(), NC()>, dim3(grid), dim3(nt), 0, s, nullptr, nullptr, dy,
             h, rstd, weight, dh, rows, d, dx, p);
  };
  auto c = [](auto v) { return v; };
#define MOK_NORM(TPR, NC) go(c(std::integral_constant<int, TPR>{}), c(std::integral_constant<int, NC>{}))
  if (rows == 0) {
  } else if (!vec) {
    if (p)
      launch_k(k_rmsnorm_dw_any<T>, dim3((d + NORM_NT - 1) / NORM_NT, blocks), dim3(NORM_NT), 0, s,
               nullptr, nullptr, dy, h, rstd, rows, d, p);
    for (int64_t r = 0; r < rows; r += kMaxLaunchRows) {
      const int64_t n = std::min(rows - r, kMaxLaunchRows), o = r * d;
      launch_k(d > 2048 ? k_rmsnorm_bwd_any<T, 1024> : k_rmsnorm_bwd_any<T, 256>, dim3((unsigned)n),
               dim3(d > 2048 ? 1024 : 256), 0, s, nullptr, nullptr, dy + o, h + o, rstd + r, weight,
               dh ? dh + o : dh, d, dx + o);
    }
  } else if (d <= 512) MOK_NORM(64, 1);
  else if (d <= 1024) MOK_NORM(64, 2);
  else if (d <= 2048) MOK_NORM(256, 1);
  else if (d <= 4096) MOK_NORM(256, 2);
  else MOK_NORM(1024, 1);        // (256, 4) needs 256 registers: one wave a SIMD
#undef MOK_NORM
  if (dweight)
    launch_k(k_column_sum, dim3((d + 15) / 16), dim3(1024), 0, s, nullptr, nullptr,
             (const float*)part, n_part, d, dweight);
  return hipGetLastError();
}

int norm_check(int64_t rows, int32_t d, int32_t io_dtype) {
  if (rows < 0 || rows >= (int64_t)1 << 31 || d < 1 || d > (1 << 24)) return MOK_EINVAL;
  return io_dtype == MOK_FP32 || io_dtype == MOK_BF16 ? MOK_OK : MOK_EINVAL;
}

}  // namespace
}  // namespace mok

using namespace mok;

extern "C" {

int mok_rmsnorm(const void* x, const void* residual, const void* weight, int64_t rows, int32_t d,
                int32_t io_dtype, float eps, void* h, float* rstd, void* y, uint8_t* codes,
                uint8_t* scales, void* stream) {
  const int st = norm_check(rows, d, io_dtype);
  if (st != MOK_OK) return st;
  if (!(eps >= 0.0f) || (codes != nullptr) != (scales != nullptr) || (codes && d % 32))
    return MOK_EINVAL;
  if (rows == 0) return MOK_OK;
  if (!x || !weight || (!h && !rstd && !y && !codes)) return MOK_EINVAL;
  hipStream_t s = (hipStream_t)stream;
  const hipError_t e =
      io_dtype == MOK_BF16
          ? run_norm((const bf16_t*)x, (const bf16_t*)residual, (const bf16_t*)weight, rows, d, eps,
                     (bf16_t*)h, rstd, (bf16_t*)y, codes, scales, s)
          : run_norm((const float*)x, (const float*)residual, (const float*)weight, rows, d, eps,
                     (float*)h, rstd, (float*)y, codes, scales, s);
  return e == hipSuccess ? MOK_OK : MOK_EHIP;
}

int mok_rmsnorm_backward_workspace_bytes(int64_t rows, int32_t d, size_t* bytes) {
  if (!bytes || norm_check(rows, d, MOK_FP32) != MOK_OK) return MOK_EINVAL;
  *bytes = (size_t)bwd_blocks(rows) * d * sizeof(float);
  return MOK_OK;
}

int mok_rmsnorm_backward(const void* dy, const void* h, const float* rstd, const void* weight,
                         const void* dh, int64_t rows, int32_t d, int32_t io_dtype, void* dx,
                         float* dweight, void* ws, size_t ws_bytes, void* stream) {
  const int st = norm_check(rows, d, io_dtype);
  if (st != MOK_OK) return st;
  if (rows > 0 && (!dy || !h || !rstd || !weight || !dx)) return MOK_EINVAL;
  if (rows == 0 && !dweight) return MOK_OK;
  size_t need = 0;
  mok_rmsnorm_backward_workspace_bytes(rows, d, &need);
  if (dweight && (!ws || ws_bytes < need || (uintptr_t)ws % 16)) return MOK_EWORKSPACE;
  hipStream_t s = (hipStream_t)stream;
  const hipError_t e =
      io_dtype == MOK_BF16
          ? run_bwd((const bf16_t*)dy, (const bf16_t*)h, rstd, (const bf16_t*)weight,
                    (const bf16_t*)dh, rows, d, (bf16_t*)dx, dweight, (float*)ws, s)
          : run_bwd((const float*)dy, (const float*)h, rstd, (const float*)weight, (const float*)dh,
                    rows, d, (float*)dx, dweight, (float*)ws, s);
  return e == hipSuccess ? MOK_OK : MOK_EHIP;
}

}  // extern "C"
