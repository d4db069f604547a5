// Balance loss of the router: expert counts, mean router probabilities, the loss and its
// gradient for the logits, over one batch or packed sequences.
//
//   p[t,e] = softmax(logits[t,:])_e        c[s,e] = picks of expert e in sequence s
//   f[s,e] = E c[s,e] / (k n_s)            P[s,e] = (1/n_s) sum_{t in s} p[t,e]
//   loss   = (alpha / S) sum_s sum_e f[s,e] P[s,e]
//   dlogits[t,e] = dloss (alpha / (S n_s)) p[t,e] (f[s,e] - sum_e' f[s,e'] p[t,e'])
//
// The gradient goes through P only (the counts are piecewise constant), so it needs the counts
// and the token's own row, nothing else of the forward.
//
// Both directions stream the logits once: memory bound. A workgroup takes a chunk of
// consecutive tokens; L lanes hold a row (16 for up to 64 experts with 16-byte loads, so a wave
// holds 4 rows and each softmax reduction is 4 shuffles), and a lane keeps the same columns for
// every row, so the sums over tokens stay in its registers. Chunks meet sequences in a
// staircase: the pairs (chunk c, sequence s) that share tokens have distinct c + s, which is
// the slot of the pair's partial sums, so ragged sequences need no sort and no float atomics.
// A second launch adds each sequence's slots in ascending order and forms the loss; its last
// workgroup (an integer ticket) adds the workgroups' loss terms in order. Same bits every run.
#include <algorithm>

#include "device_common.h"
#include "launch.h"
#include "mok.h"

namespace mok {
namespace {

constexpr int BAL_NT = 256;                // threads of the row kernels: 4 waves
constexpr int BAL_W = BAL_NT / 64;

// Tokens of a chunk: at most `most` chunks, and at least 16 tokens, a workgroup's rows in one step
// of the 16-lane form. Forward: 1024 chunks, which all run at once and keep the second launch's
// sums short (2048 took as long here, and 2 us more there: T 262,144, E 256). Backward, which has
// nothing to join: 2048, 8 a CU.
constexpr int kChunksFwd = 1024, kChunksBwd = 2048;
int64_t bal_chunk(int64_t T, int most = kChunksFwd) {
  const int64_t c = (T + most - 1) / most;
  return std::max<int64_t>(16, (c + 15) / 16 * 16);
}
int64_t bal_chunks(int64_t T) { return (T + bal_chunk(T) - 1) / bal_chunk(T); }

// Workspace: [ticket (256 B)] [loss terms: double per (sequence, 64 experts)]
//            [prob partials: float (chunks + S) x E] [count partials: int32, same]
struct BalWs {
  size_t terms, prob, count, total;
};
BalWs bal_ws(int64_t T, int E, int64_t S) {
  BalWs w;
  auto up = [](size_t v) { return (v + 255) / 256 * 256; };
  const size_t slots = (size_t)(bal_chunks(T) + S);
  w.terms = 256;
  w.prob = w.terms + up((size_t)S * ((E + 63) / 64) * sizeof(double));
  w.count = w.prob + up(slots * E * sizeof(float));
  w.total = w.count + up(slots * E * sizeof(int32_t));
  return w;
}

// Offset of sequence s, held inside [0, T] so that no offset can address past the tokens.
MOK_DEV int64_t seq_at(const int32_t* off, int64_t s, int64_t T) {
  if (!off) return s == 0 ? 0 : T;
  const int64_t v = off[s];
  return v < 0 ? 0 : (v > T ? T : v);
}

// First sequence that ends behind token t (S if none does).
MOK_DEV int first_seq(const int32_t* off, int S, int64_t T, int64_t t) {
  int lo = 0, hi = S;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (seq_at(off, mid + 1, T) > t) hi = mid; else lo = mid + 1;
  }
  return lo;
}

template <int L> MOK_DEV float row_max(float v) {
#pragma unroll
  for (int m = 1; m < L; m <<= 1) v = fmaxf(v, __shfl_xor(v, m, kWave));
  return v;
}
template <int L> MOK_DEV float row_sum(float v) {
#pragma unroll
  for (int m = 1; m < L; m <<= 1) v += __shfl_xor(v, m, kWave);
  return v;
}

// A row in L lanes: column of value (n, i) of lane l is (n L + l) W + i. W = 4 needs E % 4 == 0
// and 16-byte rows.
template <int W, int L, int NC>
struct Row {
  float v[NC][W];
  MOK_DEV void load(const float* p, int E, int l, bool ok) {
#pragma unroll
    for (int n = 0; n < NC; ++n) {
      const int c = (n * L + l) * W;
      if constexpr (W == 4) {
        float4 q = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
        if (ok && c < E) q = *(const float4*)(p + c);
        v[n][0] = q.x; v[n][1] = q.y; v[n][2] = q.z; v[n][3] = q.w;
      } else {
        v[n][0] = ok && c < E ? p[c] : -INFINITY;
      }
    }
  }
  // The softmax in place. A row with no logit above -inf has no probabilities: zeros. A NaN or
  // +inf makes the row NaN.
  MOK_DEV void softmax() {
    float m = -INFINITY;
#pragma unroll
    for (int n = 0; n < NC; ++n)
#pragma unroll
      for (int i = 0; i < W; ++i) m = fmaxf(m, v[n][i]);
    m = row_max<L>(m);
    if (m == -INFINITY) m = 0.0f;
    float s = 0.0f;
#pragma unroll
    for (int n = 0; n < NC; ++n)
#pragma unroll
      for (int i = 0; i < W; ++i) {
        v[n][i] = __expf(v[n][i] - m);
        s += v[n][i];
      }
    s = row_sum<L>(s);
    const float r = s == 0.0f ? 0.0f : 1.0f / s;
#pragma unroll
    for (int n = 0; n < NC; ++n)
#pragma unroll
      for (int i = 0; i < W; ++i) v[n][i] *= r;
  }
};

// Loads in flight per lane: about 16 values (T 262,144, E 256: the reading launch takes 85 us, 61 at
// least, with one row at a time 96, 86 at least).
constexpr int row_unroll(int values) { return values >= 16 ? 1 : values >= 8 ? 2 : 4; }

template <int W, int L, int NC>
__global__ __launch_bounds__(BAL_NT) void k_balance_rows(
    const float* __restrict__ logits, const int32_t* __restrict__ idx, int64_t T, int E, int k,
    const int32_t* __restrict__ off, int S, int64_t chunk, float* __restrict__ prob,
    int32_t* __restrict__ count, int32_t* __restrict__ ticket) {
  constexpr int R = 64 / L;                       // rows a wave holds
  constexpr int U = row_unroll(NC * W);           // ... and loads before it uses the first
  __shared__ float sum_sh[BAL_W][NC * L * W];
  __shared__ int32_t hist[1024];
  const int lane = lane_id(), w = threadIdx.x >> 6, l = lane % L, r = lane / L;
  if (blockIdx.x == 0 && threadIdx.x == 0) *ticket = 0;
  const int64_t lo = blockIdx.x * chunk, hi = min(T, lo + chunk);
  for (int s = first_seq(off, S, T, lo); s < S; ++s) {
    const int64_t a0 = seq_at(off, s, T);
    if (a0 >= hi) break;
    const int64_t a = max(lo, a0), b = min(hi, seq_at(off, s + 1, T));
    if (a >= b) continue;
    for (int e = threadIdx.x; e < E; e += BAL_NT) hist[e] = 0;
    __syncthreads();
    for (int64_t i = a * k + threadIdx.x; i < b * k; i += BAL_NT) {
      const int32_t e = idx[i];
      if (e >= 0 && e < E) atomicAdd(&hist[e], 1);
    }
    float acc[NC][W] = {};
    for (int64_t t0 = a + w * R; t0 < b; t0 += BAL_W * R * U) {
      Row<W, L, NC> x[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t t = t0 + u * BAL_W * R + r;
        x[u].load(logits + t * E, E, l, t < b);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        x[u].softmax();
#pragma unroll
        for (int n = 0; n < NC; ++n)
#pragma unroll
          for (int i = 0; i < W; ++i) acc[n][i] += x[u].v[n][i];
      }
    }
#pragma unroll
    for (int n = 0; n < NC; ++n)
#pragma unroll
      for (int i = 0; i < W; ++i) {
#pragma unroll
        for (int m = L; m < 64; m <<= 1) acc[n][i] += __shfl_xor(acc[n][i], m, kWave);
        if (r == 0) sum_sh[w][(n * L + l) * W + i] = acc[n][i];
      }
    __syncthreads();
    const int64_t slot = (int64_t)blockIdx.x + s;
    for (int e = threadIdx.x; e < E; e += BAL_NT) {
      float v = sum_sh[0][e];
#pragma unroll
      for (int q = 1; q < BAL_W; ++q) v += sum_sh[q][e];
      prob[slot * E + e] = v;
      count[slot * E + e] = hist[e];
    }
    __syncthreads();
  }
}

// Workgroup (x, s): CW experts of sequence s, 1024 / CW groups over its chunks. Few sequences take
// narrow workgroups, which share out the chunks; many take one workgroup each, since every
// workgroup pays for the ticket.
template <int CW>
__global__ __launch_bounds__(1024) void k_balance_sum(
    const float* __restrict__ prob, const int32_t* __restrict__ count, int T, int E, int k,
    const int32_t* __restrict__ off, int S, int chunk, float alpha, double* terms,
    int32_t* __restrict__ ticket, float* __restrict__ loss, int32_t* __restrict__ counts,
    float* __restrict__ mean_prob) {
  constexpr int G = 1024 / CW;
  __shared__ float psh[G][CW];
  __shared__ int32_t csh[G][CW];
  __shared__ double tsh[CW / 64];
  __shared__ int last;
  const int tid = threadIdx.x, lane = lane_id(), col = tid % CW, g = tid / CW;
  const int e = blockIdx.x * CW + col, s = blockIdx.y;
  const int a = (int)seq_at(off, s, T), b = (int)seq_at(off, s + 1, T);
  float p = 0.0f;
  int32_t c = 0;
  if (a < b && e < E) {
    const int c1 = (b - 1) / chunk;
#pragma unroll 4
    for (int ch = a / chunk + g; ch <= c1; ch += G) {
      p += prob[(int64_t)(ch + s) * E + e];
      c += count[(int64_t)(ch + s) * E + e];
    }
  }
  psh[g][col] = p;
  csh[g][col] = c;
  __syncthreads();
  if (tid < CW) {
#pragma unroll
    for (int q = 1; q < G; ++q) {
      p += psh[q][col];
      c += csh[q][col];
    }
    double term = 0.0;
    if (e < E) {
      const double n = (double)(b - a);
      const double mean = a < b ? p / n : 0.0;
      counts[(int64_t)s * E + e] = c;
      mean_prob[(int64_t)s * E + e] = (float)mean;
      if (a < b) term = (double)c * E / ((double)k * n) * mean;
    }
    for (int m = 1; m < 64; m <<= 1) term += __shfl_xor(term, m, kWave);
    if (lane == 0) tsh[col / 64] = term;
  }
  __syncthreads();
  const int n_terms = gridDim.x * gridDim.y;
  if (tid == 0) {
    double term = tsh[0];
#pragma unroll
    for (int q = 1; q < CW / 64; ++q) term += tsh[q];
    __hip_atomic_store(&terms[s * gridDim.x + blockIdx.x], term, __ATOMIC_RELAXED,
                       __HIP_MEMORY_SCOPE_AGENT);
    const int t = __hip_atomic_fetch_add(ticket, 1, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT);
    last = t == n_terms - 1;
  }
  __syncthreads();
  if (last && tid < 64) {           // every term is written: the loss, in a fixed order
    double v = 0.0;
    for (int i = lane; i < n_terms; i += 64)
      v += __hip_atomic_load(&terms[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    for (int m = 1; m < 64; m <<= 1) v += __shfl_xor(v, m, kWave);
    if (lane == 0) *loss = (float)((double)alpha / S * v);
  }
}

__global__ __launch_bounds__(64) void k_balance_empty(float* loss, int32_t* counts,
                                                      float* mean_prob, int64_t n) {
  if (blockIdx.x == 0 && threadIdx.x == 0) *loss = 0.0f;
  for (int64_t i = blockIdx.x * 64 + threadIdx.x; i < n; i += gridDim.x * 64) {
    counts[i] = 0;
    mean_prob[i] = 0.0f;
  }
}

template <int W, int L, int NC>
__global__ __launch_bounds__(BAL_NT) void k_balance_bwd(
    const float* __restrict__ logits, const int32_t* __restrict__ counts, int64_t T, int E, int k,
    const int32_t* __restrict__ off, int S, int64_t chunk, float alpha,
    const float* __restrict__ dloss, float* __restrict__ dlogits) {
  constexpr int R = 64 / L;
  const int lane = lane_id(), w = threadIdx.x >> 6, l = lane % L, r = lane / L;
  const int64_t lo = blockIdx.x * chunk, hi = min(T, lo + chunk);
  auto zero = [&](int64_t a, int64_t b) {         // tokens of no sequence
    for (int64_t i = a * E + threadIdx.x; i < b * E; i += BAL_NT) dlogits[i] = 0.0f;
  };
  int64_t done = lo;
  const float up = *dloss * alpha / (float)S;
  for (int s = first_seq(off, S, T, lo); s < S; ++s) {
    const int64_t a0 = seq_at(off, s, T), b0 = seq_at(off, s + 1, T);
    if (a0 >= hi) break;
    const int64_t a = max(done, a0), b = min(hi, b0);
    if (a >= b) continue;
    zero(done, a);
    // f counted from the mean count, to the nearest: sum_e p = 1, so the gradient is the same, but
    // where the counts are nearly equal nothing cancels (all equal, k = E for one: zeros, not rounding
    // errors of p; one token, 5 of 6 experts: counted from 0, 1 - p of the sixth lost p's bits)
    const float n = (float)(b0 - a0);
    const int32_t mean = (int32_t)(((b0 - a0) * k + E / 2) / E);
    float f[NC][W];
#pragma unroll
    for (int q = 0; q < NC; ++q)
#pragma unroll
      for (int i = 0; i < W; ++i) {
        const int e = (q * L + l) * W + i;
        f[q][i] = e < E ? (float)(counts[(int64_t)s * E + e] - mean) * ((float)E / ((float)k * n)) : 0.0f;
      }
    const float c = up / n;
    for (int64_t t0 = a + w * R; t0 < b; t0 += BAL_W * R) {
      const int64_t t = t0 + r;
      Row<W, L, NC> x;
      x.load(logits + t * E, E, l, t < b);
      x.softmax();
      float dot = 0.0f;
#pragma unroll
      for (int q = 0; q < NC; ++q)
#pragma unroll
        for (int i = 0; i < W; ++i) dot += f[q][i] * x.v[q][i];
      dot = row_sum<L>(dot);
      if (t < b) {
        float* out = dlogits + t * E;
#pragma unroll
        for (int q = 0; q < NC; ++q) {
          const int e = (q * L + l) * W;
          if (e < E) {
            if constexpr (W == 4) {
              *(float4*)(out + e) = make_float4(
                  c * x.v[q][0] * (f[q][0] - dot), c * x.v[q][1] * (f[q][1] - dot),
                  c * x.v[q][2] * (f[q][2] - dot), c * x.v[q][3] * (f[q][3] - dot));
            } else {
              out[e] = c * x.v[q][0] * (f[q][0] - dot);
            }
          }
        }
      }
    }
    done = b;
  }
  zero(done, hi);
}

// The row form for E experts: 16-byte columns where every row starts on 16 bytes.
template <class F>
void pick_row(int E, bool vec, F&& f) {
  auto c = [](auto v) { return v; };
#define MOK_ROW(W, L, NC)                                                        \
  return f(c(std::integral_constant<int, W>{}), c(std::integral_constant<int, L>{}), \
           c(std::integral_constant<int, NC>{}))
  if (vec) {
    if (E <= 64) MOK_ROW(4, 16, 1);
    if (E <= 128) MOK_ROW(4, 32, 1);
    if (E <= 256) MOK_ROW(4, 64, 1);
    if (E <= 512) MOK_ROW(4, 64, 2);
    MOK_ROW(4, 64, 4);
  }
  if (E <= 16) MOK_ROW(1, 16, 1);
  if (E <= 64) MOK_ROW(1, 64, 1);
  if (E <= 128) MOK_ROW(1, 64, 2);
  if (E <= 256) MOK_ROW(1, 64, 4);
  if (E <= 512) MOK_ROW(1, 64, 8);
  MOK_ROW(1, 64, 16);
#undef MOK_ROW
}

bool bal_vec(int E, const void* p) { return E % 4 == 0 && (uintptr_t)p % 16 == 0; }

int bal_check(int64_t T, int32_t E, int32_t k, const int32_t* off, int32_t S) {
  if (T < 0 || E < 1 || E > 1024 || k < 1 || k > E || k > 64 || S < 1 || S > 65535)
    return MOK_EINVAL;
  if (!off && S != 1) return MOK_EINVAL;
  if (T * (int64_t)k >= (int64_t)1 << 31) return MOK_EINVAL;
  return MOK_OK;
}

}  // namespace
}  // namespace mok

using namespace mok;

extern "C" {

int mok_balance_loss_workspace_bytes(int64_t T, int32_t E, int32_t n_seq, size_t* bytes) {
  if (!bytes || T < 0 || T >= (int64_t)1 << 31 || E < 1 || E > 1024 || n_seq < 1 || n_seq > 65535)
    return MOK_EINVAL;
  *bytes = bal_ws(T, E, n_seq).total;
  return MOK_OK;
}

int mok_balance_loss(const float* logits, const int32_t* topk_idx, int64_t T, int32_t E, int32_t k,
                     const int32_t* seq_offsets, int32_t n_seq, float alpha, float* loss,
                     int32_t* counts, float* mean_prob, void* ws, size_t ws_bytes, void* stream) {
  const int st = bal_check(T, E, k, seq_offsets, n_seq);
  if (st != MOK_OK) return st;
  if (!loss || !counts || !mean_prob || (T > 0 && (!logits || !topk_idx))) return MOK_EINVAL;
  const BalWs w = bal_ws(T, E, n_seq);
  if (!ws || ws_bytes < w.total || (uintptr_t)ws % 8) return MOK_EWORKSPACE;
  hipStream_t s = (hipStream_t)stream;
  if (T == 0) {
    const int64_t n = (int64_t)n_seq * E;
    launch_k(k_balance_empty, dim3((unsigned)std::min<int64_t>((n + 63) / 64, 1024)), dim3(64), 0,
             s, nullptr, nullptr, loss, counts, mean_prob, n);
    return hipGetLastError() == hipSuccess ? MOK_OK : MOK_EHIP;
  }
  char* base = (char*)ws;
  int32_t* ticket = (int32_t*)base;
  double* terms = (double*)(base + w.terms);
  float* prob = (float*)(base + w.prob);
  int32_t* count = (int32_t*)(base + w.count);
  const int64_t chunk = bal_chunk(T), n_chunks = bal_chunks(T);
  pick_row(E, bal_vec(E, logits), [&](auto W, auto L, auto NC) {
    launch_k(k_balance_rows<W(), L(), NC()>, dim3((unsigned)n_chunks), dim3(BAL_NT), 0, s, nullptr,
             nullptr, logits, topk_idx, T, E, k, seq_offsets, n_seq, chunk, prob, count, ticket);
  });
  if (hipGetLastError() != hipSuccess) return MOK_EHIP;
  const bool few = (int64_t)n_seq * ((E + 63) / 64) <= 32;
  const int cw = few || E <= 64 ? 64 : E <= 256 ? 256 : 1024;
  auto sum = cw == 64 ? k_balance_sum<64> : cw == 256 ? k_balance_sum<256> : k_balance_sum<1024>;
  launch_k(sum, dim3((E + cw - 1) / cw, n_seq), dim3(1024), 0, s, nullptr, nullptr, prob, count,
           (int)T, E, k, seq_offsets, n_seq, (int)chunk, alpha, terms, ticket, loss, counts,
           mean_prob);
  return hipGetLastError() == hipSuccess ? MOK_OK : MOK_EHIP;
}

int mok_balance_loss_backward(const float* logits, const int32_t* counts, int64_t T, int32_t E,
                              int32_t k, const int32_t* seq_offsets, int32_t n_seq, float alpha,
                              const float* dloss, float* dlogits, void* stream) {
  const int st = bal_check(T, E, k, seq_offsets, n_seq);
  if (st != MOK_OK) return st;
  if (T == 0) return MOK_OK;
  if (!logits || !counts || !dloss || !dlogits) return MOK_EINVAL;
  hipStream_t s = (hipStream_t)stream;
  const int64_t chunk = bal_chunk(T, kChunksBwd), n_chunks = (T + chunk - 1) / chunk;
  pick_row(E, bal_vec(E, logits) && bal_vec(E, dlogits), [&](auto W, auto L, auto NC) {
    launch_k(k_balance_bwd<W(), L(), NC()>, dim3((unsigned)n_chunks), dim3(BAL_NT), 0, s,
             nullptr, nullptr, logits, counts, T, E, k, seq_offsets, n_seq, chunk, alpha, dloss,
             dlogits);
  });
  return hipGetLastError() == hipSuccess ? MOK_OK : MOK_EHIP;
}

}  // extern "C"
