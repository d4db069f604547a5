// How the 4-bit products lay x out in LDS: what a launch asks for and what a workgroup addresses. Plain C++, so
// that the two can be held against each other without a GPU.
#pragma once
#include <stddef.h>
#include <stdint.h>

#ifndef MOK_HOSTDEV
#define MOK_HOSTDEV inline
#endif

namespace mok {

constexpr int W4_BODY = 512;         // columns of a wave's step
constexpr int W4_MAXW = 8;           // waves of a workgroup
constexpr int W4_LDS_FEW = 70 * 1024, W4_LDS_ROWS = 72 * 1024;   // for x: two workgroups a CU

// LDS of a body's columns of one row of x. few: four bytes a value and a float32 exponent a group; else bf16,
// pl planes of it. Behind each plane's columns lie 16 bytes more.
MOK_HOSTDEV int w4_body_bytes(bool few, int g, int pl) { return few ? 4 * W4_BODY + W4_BODY / g * 4 : 2 * pl * W4_BODY; }
MOK_HOSTDEV int w4_pad_bytes(bool few, int pl) { return 16 * (few ? 4 : pl); }

// Bodies of a chunk and part that a workgroup takes at a time: cap bytes (which hold one body of every row and
// part at least) over rows of body_bytes, ks parts.
MOK_HOSTDEV int w4_bodies(int bodies, int ks, int cap, int body_bytes, int rows) {
  const int all = (bodies + ks - 1) / ks, fit = cap / (body_bytes * rows * ks);
  return all < fit ? all : fit > 1 ? fit : 1;
}

// What a workgroup with that many rows addresses for x.
inline size_t w4_x_bytes(bool few, int g, int pl, int bodies, int ks, int cap, int rows) {
  const int b = w4_body_bytes(few, g, pl), n = w4_bodies(bodies, ks, cap, b, rows) * ks;
  return (size_t)rows * (b * n + w4_pad_bytes(few, pl));
}

struct W4Shape {
  int ks, tpw, cap;                  // parts of K, tiles of a workgroup, bytes of LDS for x's bodies
  size_t lds;                        // dynamic LDS of the launch
};

// rows: the rows that a workgroup mostly has at a time, most: those that it can have (an expert that tokens name
// more than once has more rows than there are tokens). waves: of the launch with one part of K, tile pairs of
// `pair` waves; red: bytes of LDS that a wave's sums take there (0: they lie elsewhere).
inline W4Shape w4_shape(bool few, int g, int pl, int K, int64_t waves, int pair, int red, int rows, int most) {
  W4Shape s;
  const int bodies = (K + W4_BODY - 1) / W4_BODY, b = w4_body_bytes(few, g, pl);
  const int lds_x = few ? W4_LDS_FEW : W4_LDS_ROWS;
  // twice as much for the bf16 rows of few workgroups, which have a CU each
  for (int room = few ? lds_x : 2 * lds_x;; room = lds_x) {
    int parts = W4_MAXW / pair;
    if (parts > bodies) parts = bodies;
    if (parts > room / (b * most)) parts = room / (b * most);       // one body of every row and part has to fit
    // as many parts of K as give every SIMD two waves
    if (waves < 1) waves = 1;
    const int64_t want = (2048 + waves - 1) / waves;
    s.ks = want < parts ? (int)want : parts;
    s.ks = (bodies + (bodies + s.ks - 1) / s.ks - 1) / ((bodies + s.ks - 1) / s.ks);
    s.tpw = W4_MAXW / s.ks / pair * pair;
    if (room == lds_x || waves <= (int64_t)256 * s.tpw) break;
  }
  s.cap = b * rows * s.ks * w4_bodies(bodies, s.ks, lds_x, b, rows);
  if (s.cap < b * most * s.ks) s.cap = b * most * s.ks;
  const size_t x = (size_t)s.cap + (size_t)w4_pad_bytes(few, pl) * most, sums = (size_t)s.tpw * s.ks * red;
  s.lds = x > sums ? x : sums;
  return s;
}

// The same of a workgroup of one token's k routes, a wave a route and part.
inline W4Shape w4_token_shape(int g, int K, int k) {
  W4Shape s;
  const int bodies = (K + W4_BODY - 1) / W4_BODY, b = w4_body_bytes(true, g, 1) * k;
  s.tpw = k;
  s.ks = W4_MAXW / k;
  if (s.ks > bodies) s.ks = bodies;
  if (s.ks > W4_LDS_FEW / b) s.ks = W4_LDS_FEW / b;
  if (s.ks < 1) s.ks = 1;
  s.ks = (bodies + (bodies + s.ks - 1) / s.ks - 1) / ((bodies + s.ks - 1) / s.ks);
  s.cap = b * s.ks * w4_bodies(bodies, s.ks, W4_LDS_FEW, b, 1);
  s.lds = (size_t)s.cap + (size_t)w4_pad_bytes(true, 1) * k;
  return s;
}

}  // namespace mok
