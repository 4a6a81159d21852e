// Short causal depthwise convolution over the tokens, with SiLU, for gfx950.
//
//   z_t = bias + sum_j w_j x_{t-K+1+j},  y_t = silu(z_t)  (or z_t); rows before a sequence's first from x_init or zero
//   backward  dz = dY silu'(z),  dx_s = sum_j w_j dz_{s+K-1-j} (+ dx_final),  dw_j = sum_t dz_t x_{t-K+1+j},  dbias = sum_t dz_t
//
// Bound by HBM: x is read once and y written once.  A thread has 16 bytes of channels and walks over a run of tokens
// with the last K rows in registers (named in turn, so that none is moved), the next K rows' loads under way; a run
// reads the K - 1 rows before it again.  Sums are fp32, those of gradients over runs fp64.  65,536 x 6144 in bf16, K = 4: 253
// us, 6.4 TB/s; backward of 16,458 x 2304: 54 us, 4.2 TB/s; a step of 256 rows x 6144: 7 us.
#include "delta.hpp"
#include "norm.hpp"
#include "slots.hpp"

namespace ttt {
namespace {

constexpr int kConvThreads = 256;

// p = 1 / (1 + exp(-z)) and q = 1 - p.  fp32: both from exp(-|z|) and a reciprocal put right by one step of Newton's, off by
// some 2^-22 of themselves also far from zero; the hardware's own, which bf16 takes, are off by |z| 2^-24 and more (2^-18 at
// 60), far below its rounding.
struct Sigmoid {
  float p, q;
};
template <typename T> __device__ __forceinline__ Sigmoid sigmoid_of(float z) {
  if constexpr (sizeof(T) == 2) {
    const float p = sigmoid_f(z);
    return {p, 1.f - p};
  } else {
    const float t = exp_neg(-fabsf(z)), d = 1.f + t, r0 = __builtin_amdgcn_rcpf(d), r = fmaf(fmaf(-d, r0, 1.f), r0, r0);
    return z >= 0.f ? Sigmoid{r, t * r} : Sigmoid{t * r, r};
  }
}

// Which channels and which run (or sequence) a thread has: cv threads in a row along the channels, a wave at most,
// the rest along the runs.
struct ConvPlace {
  int64_t run;
  int c;                          // first channel
  bool in;
};
__device__ __forceinline__ ConvPlace conv_place(int cv, int blocks_c, int VEC, int d, int64_t block) {
  const int per = kConvThreads / cv;
  ConvPlace p;
  p.c = ((int)(block % blocks_c) * cv + (int)threadIdx.x % cv) * VEC;
  p.run = block / blocks_c * per + threadIdx.x / cv;
  p.in = p.c < d;
  return p;
}

// A thread's taps and bias, widened; channels past d are zero.
template <typename T, bool RAG, int K, int VEC>
__device__ __forceinline__ void load_taps(const T* w, const T* bias, int c, int d, float (&tap)[K][VEC], float (&b)[VEC]) {
  if constexpr (!RAG) {
    float v[K * VEC];             // the taps of a channel lie together
#pragma unroll
    for (int i = 0; i < K; ++i)
      widen(*reinterpret_cast<const Pack<T, VEC>*>(w + (int64_t)c * K + i * VEC), v + i * VEC);
#pragma unroll
    for (int j = 0; j < VEC; ++j)
#pragma unroll
      for (int k = 0; k < K; ++k) tap[k][j] = v[j * K + k];
#pragma unroll
    for (int j = 0; j < VEC; ++j) b[j] = 0.f;
    if (bias) widen(*reinterpret_cast<const Pack<T, VEC>*>(bias + c), b);
  } else {
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      const bool in = c + j < d;
      b[j] = bias && in ? to_f32(bias[c + j]) : 0.f;
#pragma unroll
      for (int k = 0; k < K; ++k) tap[k][j] = in ? to_f32(w[(int64_t)(c + j) * K + k]) : 0.f;
    }
  }
}

// Row r of a sequence whose first token lies at `first` (its channels c..), r < 0: of its earlier rows.
template <typename T, int K, bool RAG, int VEC = Vec<T>::V>
__device__ __forceinline__ Pack<T, VEC> conv_row(const T* first, int64_t pitch, const T* init, int d, int c, int r) {
  if (r >= 0) return load_pack<T, VEC, RAG>(first + r * pitch, d - c);
  if (init) return load_pack<T, VEC, RAG>(init + (int64_t)(r + K - 1) * d + c, d - c);
  Pack<T, VEC> z;
  __builtin_memset(&z, 0, sizeof(z));
  return z;
}

// The parts of sequences that tokens [t0, t1) of batch row b hold, in order: f(sequence, its first token, its end, from,
// to).  Packed starts may have any values: they are brought into 0..n, an end before its start counts as the start,
// and no token is gone back to.
template <typename F>
__device__ __forceinline__ void conv_parts(const DeltaSeqs& q, int b, int t0, int t1, F f) {
  if (!q.starts) {
    f(b, 0, q.n, t0, t1);
    return;
  }
  int lo = 0, hi = q.num;         // the last sequence that starts at or before t0
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (seq_start(q, mid) <= t0) lo = mid; else hi = mid;
  }
  int t = t0;
  for (int i = lo; i < q.num && t < t1; ++i) {
    const int a = seq_start(q, i), e = max(seq_start(q, i + 1), a);
    if (a >= t1) break;
    t = max(t, a);
    const int to = min(e, t1);
    if (t < to) {
      f(i, a, e, t, to);
      t = to;
    }
  }
}

template <typename T, bool RAG, int K, bool STREAM>
__global__ __launch_bounds__(kConvThreads) void k_conv(ConvArgs a, ConvPlan p) {
  constexpr int VEC = Vec<T>::V;
  using V = Pack<T, VEC>;
  const int d = a.d;
  const T* x = (const T*)a.x;
  if ((int64_t)blockIdx.x >= p.blocks) {          // every sequence's last K - 1 rows
    const ConvPlace at = conv_place(p.cv, p.blocks_c, VEC, d, blockIdx.x - p.blocks);
    if (!at.in || at.run >= p.seqs) return;
    const int s = (int)at.run;
    int len = a.seqs.n;
    const T* first = x + s * a.sx.b + at.c;
    if (a.seqs.starts) {
      const int from = seq_start(a.seqs, s);
      len = max(seq_start(a.seqs, s + 1), from) - from;
      first = x + from * a.sx.t + at.c;
    }
    const T* init = a.x_init ? (const T*)a.x_init + (int64_t)s * (K - 1) * d : nullptr;
#pragma unroll
    for (int j = 0; j < K - 1; ++j)
      store_pack<T, VEC, RAG>((T*)a.x_final + ((int64_t)s * (K - 1) + j) * d + at.c,
                              conv_row<T, K, RAG>(first, a.sx.t, init, d, at.c, len - (K - 1) + j), d - at.c);
    return;
  }
  const ConvPlace at = conv_place(p.cv, p.blocks_c, VEC, d, blockIdx.x);
  const int64_t row = at.run / p.runs;
  if (!at.in || row >= a.batch) return;
  const int b = (int)row, t0 = (int)(at.run - row * p.runs) * p.run;
  float tap[K][VEC], bias[VEC];
  load_taps<T, RAG, K, VEC>((const T*)a.w, (const T*)a.bias, at.c, d, tap, bias);
  T* y = (T*)a.Y + b * a.sy.b + at.c;
  conv_parts(a.seqs, b, t0, min(t0 + p.run, a.seqs.n), [&](int seq, int begin, int, int from, int to)
                                                           __attribute__((always_inline)) {
    const T* first = x + b * a.sx.b + begin * a.sx.t + at.c;
    const T* init = a.x_init ? (const T*)a.x_init + (int64_t)seq * (K - 1) * d : nullptr;
    float win[K][VEC];            // row r is in place (r - (from - begin)) mod K
    V next[K];
#pragma unroll
    for (int j = 0; j < K - 1; ++j) widen(conv_row<T, K, RAG>(first, a.sx.t, init, d, at.c, from - begin - (K - 1) + j), win[j + 1]);
#pragma unroll
    for (int u = 0; u < K; ++u)
      if (from + u < to) next[u] = load_pack<T, VEC, RAG, STREAM>(first + (from + u - begin) * a.sx.t, d - at.c);
    for (int t = from; t < to; t += K) {
      V now[K];
#pragma unroll
      for (int u = 0; u < K; ++u) now[u] = next[u];
#pragma unroll
      for (int u = 0; u < K; ++u)
        if (t + K + u < to) next[u] = load_pack<T, VEC, RAG, STREAM>(first + (t + K + u - begin) * a.sx.t, d - at.c);
#pragma unroll
      for (int u = 0; u < K; ++u) {
        if (t + u < to) {
          widen(now[u], win[u]);
          float o[VEC];
#pragma unroll
          for (int j = 0; j < VEC; ++j) {
            float z = bias[j];
#pragma unroll
            for (int k = 0; k < K; ++k) z += tap[k][j] * win[(u + 1 + k) % K][j];
            o[j] = a.silu ? z * sigmoid_of<T>(z).p : z;
          }
          V out;
          narrow(o, out);
          store_pack<T, VEC, RAG, STREAM>(y + (t + u) * a.sy.t, out, d - at.c);
        }
      }
    }
  });
}

// dz from z and dY.
template <typename T> __device__ __forceinline__ float conv_dz(float z, float g, bool silu) {
  if (!silu) return g;
  const Sigmoid s = sigmoid_of<T>(z);
  return g * (s.p + z * s.p * s.q);
}

// Channels of a thread: 8 of bf16 would take more than half of the registers, for one wave a SIMD.
constexpr int kGradVec = 4;

// The taps' and the bias's gradient of a workgroup's runs goes to part[][K + 1][d].  Over a run's tokens, 64 at most, it is
// summed in fp32 (fp64 would take K + 1 registers more a channel, for two waves a SIMD), over runs in fp64 but for lanes
// side by side and the rounding of a workgroup's.
template <typename T, bool RAG, int K>
__global__ __launch_bounds__(kConvThreads) void k_conv_grad(ConvGradArgs g, ConvPlan p) {
  constexpr int VEC = kGradVec;
  using V = Pack<T, VEC>;
  const ConvArgs& a = g.f;
  const int d = a.d;
  const T* x = (const T*)a.x;
  const T* dY = (const T*)g.dY;
  float tap[K][VEC], bias[VEC];
  if ((int64_t)blockIdx.x >= p.blocks) {          // the gradient of every sequence's earlier rows
    const ConvPlace at = conv_place(p.cv, p.blocks_c, VEC, d, blockIdx.x - p.blocks);
    if (!at.in || at.run >= p.seqs) return;
    load_taps<T, RAG, K, VEC>((const T*)a.w, (const T*)a.bias, at.c, d, tap, bias);
    const int s = (int)at.run;
    int len = a.seqs.n;
    const T *first = x + s * a.sx.b + at.c, *dfirst = dY + s * g.sdy.b + at.c;
    if (a.seqs.starts) {
      const int from = seq_start(a.seqs, s);
      len = max(seq_start(a.seqs, s + 1), from) - from;
      first = x + from * a.sx.t + at.c;
      dfirst = dY + from * g.sdy.t + at.c;
    }
    const T* init = a.x_init ? (const T*)a.x_init + (int64_t)s * (K - 1) * d : nullptr;
    float o[K][VEC];              // row i of the K - 1: i = t + j
#pragma unroll
    for (int i = 0; i < K - 1; ++i) {
#pragma unroll
      for (int j = 0; j < VEC; ++j) o[i][j] = 0.f;
      if (g.dx_final && i >= len)
        widen(load_pack<T, VEC, RAG>((const T*)g.dx_final + ((int64_t)s * (K - 1) + i - len) * d + at.c, d - at.c), o[i]);
    }
#pragma unroll
    for (int t = 0; t < K - 1; ++t) {
      if (t < len) {
        float z[VEC], dy[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) z[j] = bias[j];
#pragma unroll
        for (int k = 0; k < K; ++k) {
          float r[VEC];
          widen(conv_row<T, K, RAG, VEC>(first, a.sx.t, init, d, at.c, t - (K - 1) + k), r);
#pragma unroll
          for (int j = 0; j < VEC; ++j) z[j] += tap[k][j] * r[j];
        }
        widen(load_pack<T, VEC, RAG>(dfirst + t * g.sdy.t, d - at.c), dy);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const float dz = conv_dz<T>(z[j], dy[j], a.silu);
#pragma unroll
          for (int k = 0; k < K - 1; ++k)
            if (t + k < K - 1) o[t + k][j] += tap[k][j] * dz;
        }
      }
    }
#pragma unroll
    for (int i = 0; i < K - 1; ++i) {
      V out;
      narrow(o[i], out);
      store_pack<T, VEC, RAG>((T*)g.dx_init + ((int64_t)s * (K - 1) + i) * d + at.c, out, d - at.c);
    }
    return;
  }
  const ConvPlace at = conv_place(p.cv, p.blocks_c, VEC, d, blockIdx.x);
  const int64_t row = at.run / p.runs;
  const bool live = at.in && row < a.batch;
  if (live) load_taps<T, RAG, K, VEC>((const T*)a.w, (const T*)a.bias, at.c, d, tap, bias);
  const int b = (int)row, t0 = (int)(at.run - row * p.runs) * p.run;
  float dw[K][VEC], db[VEC];
#pragma unroll
  for (int j = 0; j < VEC; ++j) {
    db[j] = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k) dw[k][j] = 0.f;
  }
  T* dx = (T*)g.dx + b * g.sdx.b + at.c;
  if (live) conv_parts(a.seqs, b, t0, min(t0 + p.run, a.seqs.n), [&](int seq, int begin, int end, int from, int to)
                                                           __attribute__((always_inline)) {
    const T* first = x + b * a.sx.b + begin * a.sx.t + at.c;
    const T* dfirst = dY + b * g.sdy.b + begin * g.sdy.t + at.c;
    const T* init = a.x_init ? (const T*)a.x_init + (int64_t)seq * (K - 1) * d : nullptr;
    const int last = min(to + K - 1, end);        // dz of the K - 1 tokens behind enter the run's dx too
    float win[K][VEC], pend[K][VEC];              // row r, and dx of it so far, in place (r - (from - begin)) mod K
#pragma unroll
    for (int j = 0; j < K - 1; ++j) {
      widen(conv_row<T, K, RAG, VEC>(first, a.sx.t, init, d, at.c, from - begin - (K - 1) + j), win[j + 1]);
    }
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int j = 0; j < VEC; ++j) pend[k][j] = 0.f;
    V nx[K], ny[K];
    auto load = [&](int t) __attribute__((always_inline)) {
#pragma unroll
      for (int u = 0; u < K; ++u)
        if (t + u < last) {
          nx[u] = load_pack<T, VEC, RAG>(first + (t + u - begin) * a.sx.t, d - at.c);
          ny[u] = load_pack<T, VEC, RAG>(dfirst + (t + u - begin) * g.sdy.t, d - at.c);
        }
    };
    load(from);
    for (int t = from; t < to + K - 1; t += K) {
      V rx[K], ry[K];
#pragma unroll
      for (int u = 0; u < K; ++u) {
        rx[u] = nx[u];
        ry[u] = ny[u];
      }
      load(t + K);
#pragma unroll
      for (int u = 0; u < K; ++u) {
        float dz[VEC];
        if (t + u < last) {
          float dy[VEC];
          widen(rx[u], win[u]);
          widen(ry[u], dy);
#pragma unroll
          for (int j = 0; j < VEC; ++j) {
            float z = bias[j];
#pragma unroll
            for (int k = 0; k < K; ++k) z += tap[k][j] * win[(u + 1 + k) % K][j];
            dz[j] = conv_dz<T>(z, dy[j], a.silu);
          }
          if (t + u < to) {
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
              db[j] += dz[j];
#pragma unroll
              for (int k = 0; k < K; ++k) dw[k][j] += dz[j] * win[(u + 1 + k) % K][j];
            }
          }
        } else {
#pragma unroll
          for (int j = 0; j < VEC; ++j) dz[j] = 0.f;
        }
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
#pragma unroll
          for (int k = 0; k < K - 1; ++k) pend[(u + 1 + k) % K][j] += tap[k][j] * dz[j];
          pend[u][j] = tap[K - 1][j] * dz[j];     // row t + u: its first
        }
        const int s = t + u - (K - 1);            // the row that no later token reaches
        if (s >= from && s < to) {
          float(&o)[VEC] = pend[(u + 1) % K];
          if (g.dx_final && s >= end - (K - 1)) {
            float f[VEC];
            widen(load_pack<T, VEC, RAG>((const T*)g.dx_final + ((int64_t)seq * (K - 1) + s - end + K - 1) * d + at.c, d - at.c), f);
#pragma unroll
            for (int j = 0; j < VEC; ++j) o[j] += f[j];
          }
          V out;
          narrow(o, out);
          store_pack<T, VEC, RAG>(dx + s * g.sdx.t, out, d - at.c);
        }
      }
    }
  });
  __shared__ float red[kConvThreads / 64][K + 1][64][VEC];
  const int lane = lane_id(), w = wave_id(), cv = p.cv;
#pragma unroll
  for (int k = 0; k <= K; ++k) {
    float v[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) v[j] = k < K ? dw[k][j] : db[j];
    for (int r = cv; r < 64; r *= 2)
#pragma unroll
      for (int j = 0; j < VEC; ++j) v[j] += __shfl_xor(v[j], r, 64);
    if (lane < cv)
#pragma unroll
      for (int j = 0; j < VEC; ++j) red[w][k][lane][j] = v[j];
  }
  __syncthreads();
  const int c0 = (int)(blockIdx.x % p.blocks_c) * cv * VEC;
  float* part = g.part + (int64_t)(blockIdx.x / p.blocks_c) * (K + 1) * d;
  for (int i = threadIdx.x; i < (K + 1) * cv * VEC; i += kConvThreads) {
    const int k = i / (cv * VEC), c = i % (cv * VEC);
    double v = 0.0;
#pragma unroll
    for (int r = 0; r < kConvThreads / 64; ++r) v += red[r][k][c / VEC][c % VEC];
    if (c0 + c < d) part[(int64_t)k * d + c0 + c] = (float)v;
  }
}

// dw[c][k] and dbias[c]: the parts' sums in fp64 in a fixed order, 16 channels of a tap a workgroup, each of its 64 rows of
// threads every 64th part, joined in LDS.
__global__ __launch_bounds__(1024) void k_conv_sum(const float* __restrict__ part, int64_t parts, int d, int K,
                                                   float* __restrict__ dw, float* __restrict__ db) {
  __shared__ double sum[64][17];
  const int j = threadIdx.x & 15, r = threadIdx.x >> 4, c = blockIdx.x * 16 + j, k = blockIdx.y;
  if (k == K && db == nullptr) return;
  double s = 0.0;
  if (c < d) {
#pragma unroll 4
    for (int64_t g = r; g < parts; g += 64) s += part[(g * (K + 1) + k) * d + c];
  }
  sum[r][j] = s;
  __syncthreads();
  if (r == 0 && c < d) {
    s = 0.0;
#pragma unroll
    for (int i = 0; i < 64; ++i) s += sum[i][j];
    if (k < K)
      dw[(int64_t)c * K + k] = (float)s;
    else
      db[c] = (float)s;
  }
}

// One token for every row of a serving batch: a workgroup has one row and some channels.  Rows that name the same
// earlier rows take them one after the other, in row order: the first of them carries them through all.
template <typename T, bool RAG, int K>
__global__ __launch_bounds__(kConvThreads) void k_conv_step(ConvStepArgs p) {
  constexpr int VEC = Vec<T>::V;
  using V = Pack<T, VEC>;
  const int d = p.d, blocks_c = (d + kConvThreads * VEC - 1) / (kConvThreads * VEC);
  int r = blockIdx.x / blocks_c;
  const int c = ((int)(blockIdx.x % blocks_c) * kConvThreads + (int)threadIdx.x) * VEC;
  const bool in = c < d;
  const int64_t slot = p.slots ? (int64_t)p.slots[r] : (int64_t)r;
  if (slot < 0 || slot >= p.pool) {               // a padding row: its output is zero
    V z;
    __builtin_memset(&z, 0, sizeof(z));
    if (in) store_pack<T, VEC, RAG>((T*)p.Y + (int64_t)r * d + c, z, d - c);
    return;
  }
  T* halo = (T*)p.halo + slot * (K - 1) * d + c;
  V line[K];
  float tap[K][VEC], bias[VEC];
  if (in) {
#pragma unroll
    for (int k = 0; k < K - 1; ++k) line[k] = load_pack<T, VEC, RAG>(halo + (int64_t)k * d, d - c);
    line[K - 1] = load_pack<T, VEC, RAG>((const T*)p.x + (int64_t)r * d + c, d - c);
    load_taps<T, RAG, K, VEC>((const T*)p.w, (const T*)p.bias, c, d, tap, bias);
  }
  if (p.slots && next_row(p.slots, r, 0, (int)slot) < r) return;
  for (;;) {
    if (in) {
      float o[VEC];
#pragma unroll
      for (int j = 0; j < VEC; ++j) o[j] = bias[j];
#pragma unroll
      for (int k = 0; k < K; ++k) {
        float v[VEC];
        widen(line[k], v);
#pragma unroll
        for (int j = 0; j < VEC; ++j) o[j] += tap[k][j] * v[j];
      }
      if (p.silu)
#pragma unroll
        for (int j = 0; j < VEC; ++j) o[j] *= sigmoid_of<T>(o[j]).p;
      V out;
      narrow(o, out);
      store_pack<T, VEC, RAG>((T*)p.Y + (int64_t)r * d + c, out, d - c);
#pragma unroll
      for (int k = 0; k < K - 1; ++k) line[k] = line[k + 1];
    }
    r = p.slots ? next_row(p.slots, p.rows, r + 1, (int)slot) : p.rows;
    if (r >= p.rows) break;
    if (in) line[K - 1] = load_pack<T, VEC, RAG>((const T*)p.x + (int64_t)r * d + c, d - c);
  }
  if (in) {
#pragma unroll
    for (int k = 0; k < K - 1; ++k) store_pack<T, VEC, RAG>(halo + (int64_t)k * d, line[k], d - c);
  }
}

// Runs of `run` tokens a batch row, and the grid over them and the channels.
ConvPlan conv_plan(const ConvArgs& a, int VEC, int most) {
  ConvPlan p;
  const int units = (a.d + VEC - 1) / VEC;
  p.cv = 1;
  while (p.cv < units && p.cv < 64) p.cv *= 2;
  p.blocks_c = (units + p.cv - 1) / p.cv;
  // Runs are shortened until the chip has some 4 waves a SIMD.
  p.run = most;
  while (p.run > 8 && (int64_t)a.batch * ((a.seqs.n + p.run - 1) / p.run) * p.blocks_c * p.cv < 256 * 16 * 64) p.run /= 2;
  p.runs = (a.seqs.n + p.run - 1) / p.run;
  const int per = kConvThreads / p.cv;
  p.seqs = a.seqs.starts ? a.seqs.num : a.batch;
  p.blocks = ((int64_t)a.batch * p.runs + per - 1) / per * p.blocks_c;
  p.seq_blocks = (p.seqs + per - 1) / per * p.blocks_c;
  return p;
}

// Tokens of a run, at most.  Forward: short ones, so that a wave's rows lie in few pages, and longer where more rows before a
// run are read again (65,536 x 6144 in bf16, us for runs of 8, 12, 16, 24, 48: K = 2 253, 275, 285, 290, 307; K = 4 265, 253,
// 262, 274, 302; K = 6 327, 277, 266, 278, 297; K = 8 375, 318, 292, 299, 301); backward: each costs a sum of dw (16,458 x
// 2304: 64 59 us, 24 65 us).
int forward_run(int K) { return std::max(8, 3 * K); }
constexpr int kGradRun = 64;

template <typename F>
hipError_t with_taps(int K, F f) {
  using std::integral_constant;
  switch (K) {
    case 1: return f(integral_constant<int, 1>());
    case 2: return f(integral_constant<int, 2>());
    case 3: return f(integral_constant<int, 3>());
    case 4: return f(integral_constant<int, 4>());
    case 5: return f(integral_constant<int, 5>());
    case 6: return f(integral_constant<int, 6>());
    case 7: return f(integral_constant<int, 7>());
    case 8: return f(integral_constant<int, 8>());
  }
  return hipErrorInvalidValue;
}

template <typename F>
hipError_t with_variant(bool rag, int K, F f) {
  return with_taps(K, [&](auto k) { return rag ? f(std::true_type(), k) : f(std::false_type(), k); });
}

}  // namespace

template <typename T>
hipError_t launch_conv(const ConvArgs& a, hipStream_t s) {
  const ConvPlan p = conv_plan(a, Vec<T>::V, forward_run(a.K));
  const int64_t grid = p.blocks + (a.K > 1 ? p.seq_blocks : 0);
  if (grid == 0) return hipSuccess;
  const bool stream = (int64_t)a.batch * a.seqs.n * a.d * 2 * (int)sizeof(T) > kStreamBytes;
  return with_variant(a.rag, a.K, [&](auto rag, auto k) {
    constexpr bool RAG = decltype(rag)::value;
    constexpr int K = decltype(k)::value;
    if (!RAG && stream)
      k_conv<T, RAG, K, !RAG><<<dim3((unsigned)grid), kConvThreads, 0, s>>>(a, p);
    else
      k_conv<T, RAG, K, false><<<dim3((unsigned)grid), kConvThreads, 0, s>>>(a, p);
    return hipGetLastError();
  });
}

template <typename T>
int64_t conv_blocks(const ConvArgs& a, bool grad) {
  const ConvPlan p = grad ? conv_plan(a, kGradVec, kGradRun) : conv_plan(a, Vec<T>::V, forward_run(a.K));
  return p.blocks + p.seq_blocks;
}

template <typename T>
int64_t conv_grad_parts(const ConvArgs& a) {
  const ConvPlan p = conv_plan(a, kGradVec, kGradRun);
  return p.blocks / p.blocks_c;
}

template <typename T>
hipError_t launch_conv_grad(const ConvGradArgs& a, hipStream_t s) {
  const ConvPlan p = conv_plan(a.f, kGradVec, kGradRun);
  const int64_t grid = p.blocks + (a.dx_init && a.f.K > 1 ? p.seq_blocks : 0);
  if (grid > 0) {
    hipError_t e = with_variant(a.f.rag, a.f.K, [&](auto rag, auto k) {
      k_conv_grad<T, decltype(rag)::value, decltype(k)::value><<<dim3((unsigned)grid), kConvThreads, 0, s>>>(a, p);
      return hipGetLastError();
    });
    if (e != hipSuccess) return e;
  }
  k_conv_sum<<<dim3((unsigned)((a.f.d + 15) / 16), a.f.K + 1), 1024, 0, s>>>(a.part, p.blocks / p.blocks_c, a.f.d,
                                                                             a.f.K, a.dw, a.dbias);
  return hipGetLastError();
}

template <typename T>
hipError_t launch_conv_step(const ConvStepArgs& a, hipStream_t s) {
  constexpr int C = kConvThreads * Vec<T>::V;
  const int64_t grid = (int64_t)a.rows * ((a.d + C - 1) / C);
  return with_variant(a.rag, a.K, [&](auto rag, auto k) {
    k_conv_step<T, decltype(rag)::value, decltype(k)::value><<<dim3((unsigned)grid), kConvThreads, 0, s>>>(a);
    return hipGetLastError();
  });
}

#define TTT_CONV(T)                                                      \
  template hipError_t launch_conv<T>(const ConvArgs&, hipStream_t);      \
  template int64_t conv_blocks<T>(const ConvArgs&, bool);                \
  template int64_t conv_grad_parts<T>(const ConvArgs&);                   \
  template hipError_t launch_conv_grad<T>(const ConvGradArgs&, hipStream_t); \
  template hipError_t launch_conv_step<T>(const ConvStepArgs&, hipStream_t);
TTT_CONV(bf16)
TTT_CONV(float)

}  // namespace ttt
