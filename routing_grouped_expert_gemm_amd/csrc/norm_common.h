// What the norms share: pieces of 8 values, the row's sum over its threads, the norm of a value and
// the backward's rstd.
#pragma once
#include "device_common.h"

namespace mok {
namespace {

constexpr int NORM_NT = 256;

template <class T> struct Piece;             // 8 consecutive values; Raw: as they lie in memory
template <> struct Piece<bf16_t> {
  typedef uint4 Raw;
  MOK_DEV static Raw raw(const bf16_t* p) { return *(const uint4*)p; }
  MOK_DEV static Raw none() { return make_uint4(0, 0, 0, 0); }
  MOK_DEV static void load(const bf16_t* p, float (&v)[8]) { widen(raw(p), v); }
  MOK_DEV static void widen(const Raw& q, float (&v)[8]) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  MOK_DEV static void store(bf16_t* p, const float (&v)[8]) {
    *(uint4*)p = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                            pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
  }
};
template <> struct Piece<float> {
  struct Raw { float4 a, b; };
  MOK_DEV static Raw raw(const float* p) { return {*(const float4*)p, *(const float4*)(p + 4)}; }
  MOK_DEV static Raw none() { return {make_float4(0, 0, 0, 0), make_float4(0, 0, 0, 0)}; }
  MOK_DEV static void load(const float* p, float (&v)[8]) { widen(raw(p), v); }
  MOK_DEV static void widen(const Raw& q, float (&v)[8]) {
    const float4 a = q.a, b = q.b;
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
  MOK_DEV static void store(float* p, const float (&v)[8]) {
    *(float4*)p = make_float4(v[0], v[1], v[2], v[3]);
    *(float4*)(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
  }
};

template <class T> MOK_DEV float as_stored(float v);     // v rounded to the storage type
template <> MOK_DEV float as_stored<float>(float v) { return v; }
template <> MOK_DEV float as_stored<bf16_t>(float v) { return bf16_to_f32(f32_to_bf16(v)); }

// rstd as the norm multiplies by it: y = (h scale) w (r + rl), scale the power of two that brings the
// row's root mean square to 0.5 .. 1, so that neither h w nor rstd leaves float32's range where y
// does not (rows of 1e38 with a weight above 3; rows of 1e-40 with eps 0).
struct RowScale {
  float scale, r, rl;
  MOK_DEV explicit RowScale(double rd) {
    const int e = min(max((int)(__double2hiint(rd) >> 20) - 1023, -126), 126);
    scale = __int_as_float((e + 127) << 23);
    const double v = rd * (double)__int_as_float((127 - e) << 23);
    r = (float)v;
    rl = (float)(v - r);
  }
};

// h w rstd in float32, rstd = r + rl: the rounding errors of the products, by fma, added back. h w
// is exact for bf16 operands. (Contracted, y + e would become fma(p, r, e) and count the error
// twice.)
template <class T>
MOK_DEV float norm_value(float h, float w, const RowScale& q) {
#pragma clang fp contract(off)
  const float r = q.r, rl = q.rl;
  h *= q.scale;
  const float p = h * w;
  const float y = p * r;
  float e = __builtin_fmaf(p, rl, __builtin_fmaf(p, r, -y));
  if constexpr (sizeof(T) == 4) e = __builtin_fmaf(__builtin_fmaf(h, w, -p), r, e);
  return fabsf(y) < INFINITY ? y + e : y;
}

// Sum over the row's TPR threads, the same value in each (xor order within a wave, then the
// waves in ascending order). slot: LDS words of this call, one per wave; two calls in a row use
// two slots, so one barrier each is enough.
template <int TPR, class V>
MOK_DEV V row_total(V v, V* slot) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) v += __shfl_xor(v, m, kWave);
  if constexpr (TPR > 64) {
    if (lane_id() == 0) slot[threadIdx.x >> 6] = v;
    __syncthreads();
    v = slot[0];
#pragma unroll
    for (int w = 1; w < TPR / 64; ++w) v += slot[w];
  }
  return v;
}

// The backward's rstd of a row: the forward's, or, where that is an infinity (a root mean square below
// 3e-39, which needs eps 0), what the norm multiplied by, from sum(), the row's sum of squares in
// float64: h is then taken times scale. Every thread that meets in sum() is given the same rstd.
struct BwdScale {
  float rs, scale;
  template <class Sum> MOK_DEV BwdScale(float rstd, int d, Sum&& sum) : rs(rstd), scale(1.0f) {
    if (rstd == INFINITY) {
      const RowScale q(1.0 / sqrt(sum() / d));
      rs = q.r;
      scale = q.scale;
    }
  }
};

// A thread's share of a row's sum of squares, NT threads to a row.
template <int NT, class T> MOK_DEV double squares(const T* h, int d) {
  double ss = 0.0;
  for (int i = threadIdx.x; i < d; i += NT) {
    const double v = load_as_f32(h + i);
    ss = fma(v, v, ss);
  }
  return ss;
}

// Workgroups of a backward that keep a share of the weights' gradients each.
inline int bwd_blocks(int64_t rows) {
  return (int)(rows < 1 ? 1 : rows < 512 ? rows : 512);
}

// Rows of one launch that takes a workgroup a row: a launch counts its threads in 32 bits.
constexpr int64_t kMaxLaunchRows = (int64_t)1 << 21;

inline bool al16(const void* p) { return (uintptr_t)p % 16 == 0; }

}  // namespace
}  // namespace mok
