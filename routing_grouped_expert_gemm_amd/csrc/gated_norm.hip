// The join of a block's output to the residual stream: a norm of the output, a gate, the scales of
// the sum, and the norm that the next block reads, in one pass; and the backward.
//
//   u = y rstd_y w_post        (w_post NULL: u = y)           rstd = 1 / sqrt(mean of squares + eps)
//   h = alpha res + beta gate u, rounded to the storage type   (gate NULL: 1)
//   n = h rstd_h w_pre         (w_pre NULL: no n)
//
//   backward, from dh and dn (the norm reads h as it is stored, and the rounding passes gradients):
//   dt = dh + rstd_h (g - nh mean(g nh)),  g = dn w_pre, nh = h rstd_h;   dw_pre = sum_t dn nh
//   dres = alpha dt;   dgate = beta dt u (summed over the rows that share a gate)
//   q = beta dt gate;  dw_post = sum_t q v,  v = y rstd_y;   dy = rstd_y (p - v mean(p v)), p = q w_post
//
// Statistics are float64 as in the residual RMS norm (every value of a row hangs on them), the rest
// float32, each output rounded once. HBM streams: a row stays in registers from its first sum to
// its last output, each input read once and each output written once; TPR threads hold a row in NC
// pieces of 8 values. The weights' gradients stay in registers from row to row of a workgroup, whose
// shares a second launch adds in a fixed order: no atomics. Rows that are not whole 16-byte pieces, or lie
// at other addresses, take the same kernels with loads and stores of single values' alignment and a last
// piece value by value (float32, T 1001, d 1111 both ways: one value a thread and step, three passes over
// memory and four launches, 38 us; so 24). That one-value form is left for rows past 16,384 values (8,192 in
// the backward) or, forward, 2^21 rows. Whole passes, bf16, T 8192: forward d 7168 103 us for 470 MB, both
// directions d 2048 90 us for 436 MB, 4.6 and 4.8 TB/s (under the profiler the kernels' own times come to 108
// and 95).
#include <algorithm>

#include "device_common.h"
#include "launch.h"
#include "mok.h"
#include "norm_common.h"

namespace mok {
namespace {

// A row's piece of 8 values at p, of which the row has `left`. AL: whole 16-byte pieces at 16-byte addresses.
typedef uint4 uint4_any __attribute__((aligned(2)));
typedef float4 float4_any __attribute__((aligned(4)));
template <class T, bool AL>
MOK_DEV typename Piece<T>::Raw piece_load(const T* p, int left) {
  if constexpr (AL) return Piece<T>::raw(p);
  if (left >= 8) {
    if constexpr (sizeof(T) == 2) return *(const uint4_any*)p;
    else return {*(const float4_any*)p, *(const float4_any*)(p + 4)};
  }
  T v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = i < left ? p[i] : T(0);
  return __builtin_bit_cast(typename Piece<T>::Raw, v);
}
template <class T, bool AL>
MOK_DEV void piece_store(T* p, int left, const float (&v)[8]) {
  if constexpr (AL) {
    Piece<T>::store(p, v);
  } else if (left >= 8) {
    if constexpr (sizeof(T) == 2)
      *(uint4_any*)p = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                  pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
    else {
      *(float4_any*)p = make_float4(v[0], v[1], v[2], v[3]);
      *(float4_any*)(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < left) p[i] = f32_to<T>(v[i]);
  }
}

struct GnArgs {
  const void *y, *res, *w_post, *gate, *w_pre;
  void *h, *n;
  float *rstd_y, *rstd_h;
  int64_t rows;
  int d;
  int gate_ld;            // 0: one gate row for all
  float eps, alpha, beta;
};

template <class T, int TPR, int NC, bool AL>
__global__ __launch_bounds__(TPR > NORM_NT ? TPR : NORM_NT) void k_gated_norm(const GnArgs a) {
  constexpr int NT = TPR > NORM_NT ? TPR : NORM_NT, RPB = NT / TPR;
  typedef Piece<T> P;
  __shared__ double sh[2][NT / 64];
  const int l = threadIdx.x % TPR, d = a.d;
  const int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR;
  const bool live = row < a.rows;
  const int64_t at = row * d;
  typename P::Raw rq[NC], gq[NC];
  float u[NC][8];
  auto ok = [&](int n) { return live && (n * TPR + l) * 8 < d; };
#pragma unroll
  for (int n = 0; n < NC; ++n) {
    const int c = (n * TPR + l) * 8;
    P::widen(ok(n) ? piece_load<T, AL>((const T*)a.y + at + c, d - c) : P::none(), u[n]);
    rq[n] = ok(n) ? piece_load<T, AL>((const T*)a.res + at + c, d - c) : P::none();
    gq[n] = ok(n) && a.gate ? piece_load<T, AL>((const T*)a.gate + row * a.gate_ld + c, d - c) : P::none();
  }
  if (a.w_post) {
    double ss = 0.0;
#pragma unroll
    for (int n = 0; n < NC; ++n)
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fma((double)u[n][i], (double)u[n][i], ss);
    const double rd = 1.0 / sqrt(row_total<TPR>(ss, sh[0]) / d + a.eps);
    const RowScale rs(rd);
    if (a.rstd_y && live && l == 0) a.rstd_y[row] = (float)rd;
#pragma unroll
    for (int n = 0; n < NC; ++n) {
      float w[8] = {0, 0, 0, 0, 0, 0, 0, 0};
      const int c = (n * TPR + l) * 8;
      if (ok(n)) P::widen(piece_load<T, AL>((const T*)a.w_post + c, d - c), w);
#pragma unroll
      for (int i = 0; i < 8; ++i) u[n][i] = norm_value<T>(u[n][i], w[i], rs);
    }
  }
#pragma unroll
  for (int n = 0; n < NC; ++n) {
    float r[8], g[8];
    P::widen(rq[n], r);
    P::widen(gq[n], g);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float v = a.gate ? g[i] * u[n][i] : u[n][i];
      u[n][i] = as_stored<T>(fmaf(a.beta, v, a.alpha * r[i]));
    }
    const int c = (n * TPR + l) * 8;
    if (ok(n)) piece_store<T, AL>((T*)a.h + at + c, d - c, u[n]);
  }
  if (!a.w_pre) return;
  double ss = 0.0;
#pragma unroll
  for (int n = 0; n < NC; ++n)
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fma((double)u[n][i], (double)u[n][i], ss);
  const double rd = 1.0 / sqrt(row_total<TPR>(ss, sh[1]) / d + a.eps);
  const RowScale rs(rd);
  if (a.rstd_h && live && l == 0) a.rstd_h[row] = (float)rd;
  if (!a.n) return;
#pragma unroll
  for (int n = 0; n < NC; ++n) {
    if (!ok(n)) continue;
    const int c = (n * TPR + l) * 8;
    float w[8];
    P::widen(piece_load<T, AL>((const T*)a.w_pre + c, d - c), w);
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = norm_value<T>(u[n][i], w[i], rs);
    piece_store<T, AL>((T*)a.n + at + c, d - c, w);
  }
}

// Rows that the form above does not hold, or too many for it: one workgroup a row, one value a thread and step.
template <class T, int NT>
__global__ __launch_bounds__(NT) void k_gated_norm_any(const GnArgs a, int64_t row0) {
  __shared__ double sh[2][NT / 64];
  const int d = a.d;
  const int64_t row = row0 + blockIdx.x, at = row * d;
  const T *y = (const T*)a.y + at, *res = (const T*)a.res + at, *wp = (const T*)a.w_post,
          *gate = a.gate ? (const T*)a.gate + row * a.gate_ld : nullptr;
  T* h = (T*)a.h + at;
  double rd = 1.0;
  if (wp) {
    double ss = 0.0;
    for (int i = threadIdx.x; i < d; i += NT) {
      const double v = load_as_f32(y + i);
      ss = fma(v, v, ss);
    }
    rd = 1.0 / sqrt(row_total<NT>(ss, sh[0]) / d + a.eps);
    if (a.rstd_y && threadIdx.x == 0) a.rstd_y[row] = (float)rd;
  }
  const RowScale ry(rd);
  double ss = 0.0;
  for (int i = threadIdx.x; i < d; i += NT) {
    float u = load_as_f32(y + i);
    if (wp) u = norm_value<T>(u, load_as_f32(wp + i), ry);
    if (gate) u *= load_as_f32(gate + i);
    const float v = as_stored<T>(fmaf(a.beta, u, a.alpha * load_as_f32(res + i)));
    h[i] = f32_to<T>(v);
    ss = fma((double)v, (double)v, ss);
  }
  if (!a.w_pre) return;
  rd = 1.0 / sqrt(row_total<NT>(ss, sh[1]) / d + a.eps);
  const RowScale rh(rd);
  if (a.rstd_h && threadIdx.x == 0) a.rstd_h[row] = (float)rd;
  if (!a.n) return;
  for (int i = threadIdx.x; i < d; i += NT)      // a thread reads the h that it wrote
    ((T*)a.n)[at + i] = f32_to<T>(norm_value<T>(load_as_f32(h + i),
                                                load_as_f32((const T*)a.w_pre + i), rh));
}

struct GnBwd {
  const void *dh, *dn, *y, *h, *w_post, *gate, *w_pre;
  const float *rstd_y, *rstd_h;
  void *dres, *dy, *dgate;          // dgate: NULL where the gate is shared (its sum is p_gate)
  int64_t rows;
  int d, gate_ld;
  float alpha, beta;
  float *p_gate, *p_post, *p_pre;   // shares of the column sums, [workgroups, d] each, or NULL
  float* stat;                      // any form: 5 floats a row
};

// A value of the norm that the backward multiplies by: v scale rs.
MOK_DEV float unit(float v, const BwdScale& q) { return q.scale == 1.0f ? v * q.rs : v * q.scale * q.rs; }

template <class T, int TPR, int NC, bool AL>
__global__ __launch_bounds__(TPR > NORM_NT ? TPR : NORM_NT) void k_gated_norm_bwd(const GnBwd a) {
  constexpr int NT = TPR > NORM_NT ? TPR : NORM_NT, RPB = NT / TPR;
  typedef Piece<T> P;
  typedef typename P::Raw Raw;
  __shared__ float sh[2][2][NT / 64];
  __shared__ double shd[2][NT / 64];
  __shared__ float fold[RPB > 1 ? RPB : 1][RPB > 1 ? TPR * NC * 8 : 1];
  const int l = threadIdx.x % TPR, r = threadIdx.x / TPR, d = a.d;
  float aa[NC][8], ab[NC][8], ag[NC][8];
  Raw wa[NC], wb[NC];
  const T one = f32_to<T>(1.0f);
  T ones[8] = {one, one, one, one, one, one, one, one};
  // hq .. gq: the next row's, whose loads are issued before this row's sums (gq: or the gate of all rows)
  constexpr bool AHEAD = TPR < 1024 || sizeof(T) == 2;      // float32 rows of 1024 threads: no registers for it
  Raw hq[NC], nq[NC], oq[NC], yq[NC], gq[NC];
#pragma unroll
  for (int n = 0; n < NC; ++n) {
    const int c = (n * TPR + l) * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) aa[n][i] = ab[n][i] = ag[n][i] = 0.0f;
    wa[n] = wb[n] = gq[n] = __builtin_bit_cast(Raw, ones);
    if (c < d) {
      if (a.w_post) wa[n] = piece_load<T, AL>((const T*)a.w_post + c, d - c);
      if (a.w_pre) wb[n] = piece_load<T, AL>((const T*)a.w_pre + c, d - c);
      if (a.gate && !a.gate_ld) gq[n] = piece_load<T, AL>((const T*)a.gate + c, d - c);
    }
  }
  float ry = 0.0f, rh = 0.0f;
  auto fetch = [&](int64_t row) {
    const bool live = row < a.rows;
#pragma unroll
    for (int n = 0; n < NC; ++n) {
      const int c = (n * TPR + l) * 8;
      const int64_t at = row * d + c;
      const bool ok = live && c < d;
      oq[n] = ok && a.dh ? piece_load<T, AL>((const T*)a.dh + at, d - c) : P::none();
      hq[n] = ok && a.dn ? piece_load<T, AL>((const T*)a.h + at, d - c) : P::none();
      nq[n] = ok && a.dn ? piece_load<T, AL>((const T*)a.dn + at, d - c) : P::none();
      yq[n] = ok ? piece_load<T, AL>((const T*)a.y + at, d - c) : P::none();
      if (a.gate_ld) gq[n] = ok ? piece_load<T, AL>((const T*)a.gate + at, d - c) : P::none();
    }
    ry = live && a.w_post ? a.rstd_y[row] : 0.0f;
    rh = live && a.dn ? a.rstd_h[row] : 0.0f;
  };
  auto squares_of = [&](const float (&v)[NC][8], double* slot) {
    if constexpr (TPR > 64) __syncthreads();        // the slot of a row before has been read
    double ss = 0.0;
#pragma unroll
    for (int n = 0; n < NC; ++n)
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fma((double)v[n][i], (double)v[n][i], ss);
    return row_total<TPR>(ss, slot);
  };
  int turn = 0;
  const int64_t stride = (int64_t)gridDim.x * RPB;
  if (AHEAD) fetch((int64_t)blockIdx.x * RPB + r);
  for (int64_t r0 = (int64_t)blockIdx.x * RPB; r0 < a.rows; r0 += stride) {
    const int64_t row = r0 + r, at = row * d;
    const bool live = row < a.rows;
    float h[NC][8], g[NC][8], o[NC][8], v[NC][8], dot = 0.0f;
    if (!AHEAD) fetch(row);
#pragma unroll
    for (int n = 0; n < NC; ++n) {
      P::widen(hq[n], h[n]);
      P::widen(nq[n], g[n]);
      P::widen(oq[n], o[n]);
      P::widen(yq[n], v[n]);
    }
    const float cy = ry, ch = rh;
    Raw gc[NC];
#pragma unroll
    for (int n = 0; n < NC; ++n) gc[n] = gq[n];
    if (AHEAD) fetch(row + stride);
    if (a.dn) {
      const BwdScale q(ch, d, [&] { return squares_of(h, shd[0]); });
#pragma unroll
      for (int n = 0; n < NC; ++n) {
        float w[8];
        P::widen(wb[n], w);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          h[n][i] = unit(h[n][i], q);
          ab[n][i] += g[n][i] * h[n][i];
          g[n][i] *= w[i];
          dot += g[n][i] * h[n][i];
        }
      }
      dot = row_total<TPR>(dot, sh[turn][0]) / (float)d;
#pragma unroll
      for (int n = 0; n < NC; ++n)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float w = g[n][i] - h[n][i] * dot;
          o[n][i] = q.scale == 1.0f ? fmaf(q.rs, w, o[n][i]) : fmaf(q.scale, q.rs * w, o[n][i]);
        }
    }
    if (a.dres) {
#pragma unroll
      for (int n = 0; n < NC; ++n) {
        const int c = (n * TPR + l) * 8;
        if (!live || c >= d) continue;
        float w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = a.alpha * o[n][i];
        piece_store<T, AL>((T*)a.dres + at + c, d - c, w);
      }
    }
    const BwdScale q(a.w_post ? cy : 1.0f, d, [&] { return squares_of(v, shd[1]); });
    dot = 0.0f;
#pragma unroll
    for (int n = 0; n < NC; ++n) {
      const int c = (n * TPR + l) * 8;
      float dg[8], w[8], gt[8];
      P::widen(wa[n], w);
      P::widen(gc[n], gt);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float b = a.beta * o[n][i];
        v[n][i] = unit(v[n][i], q);
        dg[i] = b * (v[n][i] * w[i]);
        ag[n][i] += dg[i];
        o[n][i] = b * gt[i];                                  // the gradient of u
        aa[n][i] += o[n][i] * v[n][i];
        o[n][i] *= w[i];
        dot += o[n][i] * v[n][i];
      }
      if (a.dgate && live && c < d) piece_store<T, AL>((T*)a.dgate + at + c, d - c, dg);
    }
    if (a.dy) {
      if (a.w_post) dot = row_total<TPR>(dot, sh[turn][1]) / (float)d;
#pragma unroll
      for (int n = 0; n < NC; ++n) {
        const int c = (n * TPR + l) * 8;
        if (!live || c >= d) continue;
        if (a.w_post) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float w = q.rs * (o[n][i] - v[n][i] * dot);
            o[n][i] = q.scale == 1.0f ? w : q.scale * w;
          }
        }
        piece_store<T, AL>((T*)a.dy + at + c, d - c, o[n]);
      }
    }
    turn ^= 1;
  }
  auto share = [&](float* part, const float (&acc)[NC][8]) {
    if (!part) return;
    float* out = part + (int64_t)blockIdx.x * d;
    if constexpr (RPB == 1) {
#pragma unroll
      for (int n = 0; n < NC; ++n) {
        const int c = (n * TPR + l) * 8;
        if (c < d) piece_store<float, AL>(out + c, d - c, acc[n]);
      }
    } else {
      __syncthreads();
#pragma unroll
      for (int n = 0; n < NC; ++n) Piece<float>::store(&fold[r][(n * TPR + l) * 8], acc[n]);
      __syncthreads();
      for (int c = threadIdx.x; c < d; c += NT) {
        float s = fold[0][c];
#pragma unroll
        for (int q = 1; q < RPB; ++q) s += fold[q][c];
        out[c] = s;
      }
    }
  };
  share(a.p_gate, ag);
  share(a.p_post, aa);
  share(a.p_pre, ab);
}

// The same for rows that it does not hold. First launch: a workgroup a row; what its columns' sums need of the row
// (both rstd and their scales, the mean of g nh) goes to stat.
template <class T, int NT>
__global__ __launch_bounds__(NT) void k_gated_norm_bwd_any(const GnBwd a, int64_t row0) {
  __shared__ float sh[2][NT / 64];
  __shared__ double shd[2][NT / 64];
  const int d = a.d;
  const int64_t row = row0 + blockIdx.x, at = row * d;
  const T *h = (const T*)a.h + at, *y = (const T*)a.y + at;
  const BwdScale qh(a.dn ? a.rstd_h[row] : 1.0f, d,
                    [&] { return row_total<NT>(squares<NT>(h, d), shd[0]); });
  const BwdScale qy(a.w_post ? a.rstd_y[row] : 1.0f, d,
                    [&] { return row_total<NT>(squares<NT>(y, d), shd[1]); });
  auto g_at = [&](int i) {
    return load_as_f32((const T*)a.dn + at + i) * load_as_f32((const T*)a.w_pre + i);
  };
  float m = 0.0f;
  if (a.dn) {
    for (int i = threadIdx.x; i < d; i += NT) m += g_at(i) * unit(load_as_f32(h + i), qh);
    m = row_total<NT>(m, sh[0]) / (float)d;
  }
  auto dt_at = [&](int i) {
    float o = a.dh ? load_as_f32((const T*)a.dh + at + i) : 0.0f;
    if (a.dn) {
      const float w = qh.rs * (g_at(i) - unit(load_as_f32(h + i), qh) * m);
      o += qh.scale == 1.0f ? w : qh.scale * w;
    }
    return o;
  };
  auto wa_at = [&](int i) { return a.w_post ? load_as_f32((const T*)a.w_post + i) : 1.0f; };
  auto gate_at = [&](int i) {
    return a.gate ? load_as_f32((const T*)a.gate + row * a.gate_ld + i) : 1.0f;
  };
  float dot = 0.0f;
  for (int i = threadIdx.x; i < d; i += NT) {
    const float o = dt_at(i), b = a.beta * o, v = unit(load_as_f32(y + i), qy);
    if (a.dres) ((T*)a.dres)[at + i] = f32_to<T>(a.alpha * o);
    if (a.dgate) ((T*)a.dgate)[at + i] = f32_to<T>(b * (v * wa_at(i)));
    dot += b * gate_at(i) * wa_at(i) * v;
  }
  if (a.w_post) dot = row_total<NT>(dot, sh[1]) / (float)d;
  else dot = 0.0f;
  if (a.dy)
    for (int i = threadIdx.x; i < d; i += NT) {
      const float p = a.beta * dt_at(i) * gate_at(i) * wa_at(i);
      float o = p;
      if (a.w_post) {
        o = qy.rs * (p - unit(load_as_f32(y + i), qy) * dot);
        if (qy.scale != 1.0f) o *= qy.scale;
      }
      ((T*)a.dy)[at + i] = f32_to<T>(o);
    }
  if (a.stat && threadIdx.x == 0) {
    float* s = a.stat + row * 5;
    s[0] = qh.rs; s[1] = qh.scale; s[2] = qy.rs; s[3] = qy.scale; s[4] = m;
  }
}

// Second launch: workgroup (x, y) sums the columns 256 x .. over the rows y, y + gridDim.y, ...
template <class T>
__global__ __launch_bounds__(NORM_NT) void k_gated_norm_cols_any(const GnBwd a) {
  const int c = blockIdx.x * NORM_NT + threadIdx.x, d = a.d;
  if (c >= d) return;
  const float wa = a.w_post ? load_as_f32((const T*)a.w_post + c) : 1.0f;
  const float wb = a.w_pre ? load_as_f32((const T*)a.w_pre + c) : 1.0f;
  float sg = 0.0f, sa = 0.0f, sb = 0.0f;
  for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
    const float* s = a.stat + row * 5;
    const int64_t at = row * d + c;
    float o = a.dh ? load_as_f32((const T*)a.dh + at) : 0.0f;
    if (a.dn) {
      const float dn = load_as_f32((const T*)a.dn + at);
      const float nh = load_as_f32((const T*)a.h + at) * s[1] * s[0];
      sb += dn * nh;
      o += s[1] * (s[0] * (dn * wb - nh * s[4]));
    }
    const float b = a.beta * o, v = load_as_f32((const T*)a.y + at) * s[3] * s[2];
    sg += b * (v * wa);
    sa += b * (a.gate ? load_as_f32((const T*)a.gate + row * a.gate_ld + c) : 1.0f) * v;
  }
  const int64_t at = (int64_t)blockIdx.y * d + c;
  if (a.p_gate) a.p_gate[at] = sg;
  if (a.p_post) a.p_post[at] = sa;
  if (a.p_pre) a.p_pre[at] = sb;
}

// out[c] = sum over the n shares of column c, for up to three sums (grid y): 16 columns a
// workgroup, 64 groups of shares, each in ascending order, then the groups in a fixed tree.
struct GnSums {
  const float* part[3];
  float* out[3];
};
__global__ __launch_bounds__(1024) void k_gated_norm_sum(const GnSums a, int n, int d) {
  __shared__ float sh[64][17];
  const float* part = a.part[blockIdx.y];
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
  if (g == 0 && c < d) a.out[blockIdx.y][c] = sh[0][l];
}

template <int TPR, int NC> struct Form {
  static constexpr int tpr = TPR, nc = NC, nt = TPR > NORM_NT ? TPR : NORM_NT, rpb = nt / TPR;
};

template <class T>
hipError_t run_gated(const GnArgs& a, hipStream_t s) {
  const int d = a.d;
  const bool al = d % 8 == 0 && al16(a.y) && al16(a.res) && al16(a.w_post) && al16(a.gate) &&
                  al16(a.w_pre) && al16(a.h) && al16(a.n);
  auto go = [&](auto F) {
    launch_k(al ? k_gated_norm<T, F.tpr, F.nc, true> : k_gated_norm<T, F.tpr, F.nc, false>,
             dim3((unsigned)((a.rows + F.rpb - 1) / F.rpb)), dim3(F.nt), 0, s, nullptr, nullptr, a);
  };
  if (d > 16384 || a.rows > kMaxLaunchRows) {
    const bool wide = d > 2048;
    for (int64_t r = 0; r < a.rows; r += kMaxLaunchRows)
      launch_k(wide ? k_gated_norm_any<T, 1024> : k_gated_norm_any<T, 256>,
               dim3((unsigned)std::min(a.rows - r, kMaxLaunchRows)), dim3(wide ? 1024 : 256), 0, s,
               nullptr, nullptr, a, r);
  } else if (d <= 512) go(Form<64, 1>{});
  // 256 threads a row beyond 1024 values (float32 T 1001, d 1111: 9.3 us, with 64 threads 12.8; bf16 T 8192,
  // d 2048: 39 and 41), and for few rows (fewer workgroups than CUs) before that, for the row's latency
  else if (d <= 2048 && (d > 1024 || a.rows <= 256)) go(Form<256, 1>{});
  else if (d <= 1024) go(Form<64, 2>{});
  else if (a.rows <= 256 && d <= 8192) go(Form<1024, 1>{});
  else if (d <= 4096) go(Form<256, 2>{});
  // (bf16 T 8192, d 7168, under the profiler: 108 us, with 512 threads a row 109, with 1024 145)
  else if (d <= 8192) go(Form<256, 4>{});
  else go(Form<1024, 2>{});
  return hipGetLastError();
}

template <class T>
hipError_t run_gated_bwd(GnBwd a, float* dgate_all, float* dw_post, float* dw_pre, float* ws,
                         hipStream_t s) {
  const int d = a.d, blocks = bwd_blocks(a.rows);
  const bool al = d % 8 == 0 && al16(a.dh) && al16(a.dn) && al16(a.y) && al16(a.h) &&
                   al16(a.w_post) && al16(a.gate) && al16(a.w_pre) && al16(a.dres) && al16(a.dy) &&
                   al16(a.dgate);
  const size_t part = (size_t)blocks * d;
  GnSums sums = {};
  int n_sums = 0, n_part = a.rows > 0 ? blocks : 0;
  auto want = [&](float* out, int slot) {
    if (!out) return (float*)nullptr;
    sums.part[n_sums] = ws + slot * part;
    sums.out[n_sums++] = out;
    return ws + slot * part;
  };
  a.p_gate = want(dgate_all, 0);
  a.p_post = want(dw_post, 1);
  a.p_pre = want(dw_pre, 2);
  a.stat = n_sums ? ws + 3 * part : nullptr;
  auto go = [&](auto F) {
    n_part = (int)std::min<int64_t>(n_sums ? blocks : 1 << 16, (a.rows + F.rpb - 1) / F.rpb);
    launch_k(al ? k_gated_norm_bwd<T, F.tpr, F.nc, true> : k_gated_norm_bwd<T, F.tpr, F.nc, false>,
             dim3(n_part), dim3(F.nt), 0, s, nullptr, nullptr, a);
  };
  if (a.rows == 0) {
  } else if (d > 8192) {
    for (int64_t r = 0; r < a.rows; r += kMaxLaunchRows)
      launch_k(k_gated_norm_bwd_any<T, 1024>, dim3((unsigned)std::min(a.rows - r, kMaxLaunchRows)), dim3(1024), 0, s,
               nullptr, nullptr, a, r);
    if (n_sums)
      launch_k(k_gated_norm_cols_any<T>, dim3((d + NORM_NT - 1) / NORM_NT, blocks), dim3(NORM_NT),
               0, s, nullptr, nullptr, a);
  } else if (d <= 512) go(Form<64, 1>{});
  else if (d <= 1024) go(Form<64, 2>{});
  else if (d <= 2048) go(Form<256, 1>{});
  else if (d <= 4096) go(Form<512, 1>{});      // (256, 2) leaves one wave a SIMD
  else go(Form<1024, 1>{});
  if (n_sums)
    launch_k(k_gated_norm_sum, dim3((d + 15) / 16, n_sums), dim3(1024), 0, s, nullptr, nullptr,
             sums, n_part, d);
  return hipGetLastError();
}

int gn_check(int64_t rows, int32_t d, int32_t io_dtype, float alpha, float beta) {
  if (rows < 0 || rows >= (int64_t)1 << 31 || d < 1 || d > (1 << 24)) return MOK_EINVAL;
  if (!(fabsf(alpha) < INFINITY) || !(fabsf(beta) < INFINITY)) return MOK_EINVAL;
  return io_dtype == MOK_FP32 || io_dtype == MOK_BF16 ? MOK_OK : MOK_EINVAL;
}

}  // namespace
}  // namespace mok

using namespace mok;

extern "C" {

int mok_gated_norm(const void* y, const void* w_post, const void* gate, int32_t gate_per_row,
                   const void* residual, const void* w_pre, int64_t rows, int32_t d,
                   int32_t io_dtype, float eps, float alpha, float beta, void* h, void* n,
                   float* rstd_y, float* rstd_h, void* stream) {
  const int st = gn_check(rows, d, io_dtype, alpha, beta);
  if (st != MOK_OK) return st;
  if (!(eps >= 0.0f) || (!w_post && rstd_y) || (!w_pre && (n || rstd_h))) return MOK_EINVAL;
  if (rows == 0) return MOK_OK;
  if (!y || !residual || !h) return MOK_EINVAL;
  const GnArgs a = {y, residual, w_post, gate, w_pre, h, n, rstd_y, rstd_h, rows, d,
                    gate && gate_per_row ? d : 0, eps, alpha, beta};
  const hipError_t e = io_dtype == MOK_BF16 ? run_gated<bf16_t>(a, (hipStream_t)stream)
                                            : run_gated<float>(a, (hipStream_t)stream);
  return e == hipSuccess ? MOK_OK : MOK_EHIP;
}

int mok_gated_norm_backward_workspace_bytes(int64_t rows, int32_t d, size_t* bytes) {
  if (!bytes || gn_check(rows, d, MOK_FP32, 1.0f, 1.0f) != MOK_OK) return MOK_EINVAL;
  *bytes = ((size_t)3 * bwd_blocks(rows) * d + (size_t)5 * rows) * sizeof(float);
  return MOK_OK;
}

int mok_gated_norm_backward(const void* dh, const void* dn, const void* y, const void* h,
                            const void* w_post, const void* gate, int32_t gate_per_row,
                            const void* w_pre, const float* rstd_y, const float* rstd_h,
                            int64_t rows, int32_t d, int32_t io_dtype, float alpha, float beta,
                            void* dres, void* dy, void* dgate, float* dw_post, float* dw_pre,
                            void* ws, size_t ws_bytes, void* stream) {
  const int st = gn_check(rows, d, io_dtype, alpha, beta);
  if (st != MOK_OK) return st;
  if ((dgate && !gate) || (dw_post && !w_post) || (dw_pre && !w_pre) || (dn && !w_pre))
    return MOK_EINVAL;
  const bool per_row = gate && gate_per_row;
  float* const dgate_all = per_row ? nullptr : (float*)dgate;
  const bool sums = dgate_all || dw_post || dw_pre;
  if (!dres && !dy && !dgate && !sums) return MOK_EINVAL;
  if (rows > 0 && ((!dh && !dn) || !y || (w_post && !rstd_y) || (dn && (!h || !rstd_h))))
    return MOK_EINVAL;
  if (rows == 0 && !sums) return MOK_OK;
  size_t need = 0;
  mok_gated_norm_backward_workspace_bytes(rows, d, &need);
  if (sums && (!ws || ws_bytes < need || (uintptr_t)ws % 16)) return MOK_EWORKSPACE;
  GnBwd a = {};
  a.dh = dh; a.dn = dn; a.y = y; a.h = h; a.w_post = w_post; a.gate = gate; a.w_pre = w_pre;
  a.rstd_y = rstd_y; a.rstd_h = rstd_h; a.dres = dres; a.dy = dy;
  a.dgate = per_row ? dgate : nullptr;
  a.rows = rows; a.d = d; a.gate_ld = per_row ? d : 0; a.alpha = alpha; a.beta = beta;
  hipStream_t s = (hipStream_t)stream;
  const hipError_t e = io_dtype == MOK_BF16
                           ? run_gated_bwd<bf16_t>(a, dgate_all, dw_post, dw_pre, (float*)ws, s)
                           : run_gated_bwd<float>(a, dgate_all, dw_post, dw_pre, (float*)ws, s);
  return e == hipSuccess ? MOK_OK : MOK_EHIP;
}

}  // extern "C"
