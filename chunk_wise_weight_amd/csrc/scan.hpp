// What the kernels of the selective scan share (gfx950).
//
// Tokens go in chunks of 64.  Within a chunk, r the rates, b the running sum of the log decays A r, S the state [P, N]
// before the chunk, u_j = r_j x_j:
//   O_i = exp(b_i) S C_i + sum_{j <= i} (C_i . B_j) exp(b_i - b_j) u_j + D x_i
//   S'  = exp(b_63) S + sum_j exp(b_63 - b_j) u_j B_j^T
// A wave keeps 16 CT rows of a head's state (its transpose's columns) in registers and walks over the chunks.  Sequences
// are cut into segments of whole chunks so that the walks fill the chip: a first pass makes every segment's state from
// zero, a second adds them up over each sequence's segments, and the last has each segment's walk begin where it should.
//
// Operands are as in delta.hpp (Mat, Panels): a product's result is the next one's operand without leaving the
// registers.  The outputs are made transposed, rows of P by tokens, so that a lane has consecutive features of a token.
//
// Precision (bf16 inputs).  x, B and C enter as they are.  What is fp32 enters as sums of bf16 values: the scaled x of
// the state's update as three (2^-24), the state and the decayed C B^T of the outputs as two (2^-17), so that the state
// is fp32's own and O off by its own rounding.  Running sums of log decays are fp64; differences of them are taken from
// two fp32 parts, the first a multiple of 2^-8, whose differences are exact.
#pragma once
#include "delta.hpp"
#include "scan_rate.hpp"

namespace ttt {

// Where a segment slot's tokens lie; len <= 0: the slot has none.  Slots are dealt as the chunks' of delta.hpp, with
// segments of `seg` tokens in place of 64.
struct SegPlace {
  int b, tok0, len, seq;
  bool first, last;             // of its sequence
};
inline __host__ __device__ int64_t seg_slots(const DeltaSeqs& q, int batch, int seg) {
  if (q.starts) return q.num > 0 ? (int64_t)q.n / seg + q.num : 0;
  return (int64_t)batch * (((int64_t)q.n + seg - 1) / seg);
}
__device__ __forceinline__ SegPlace seg_place(const DeltaSeqs& q, int seg, int slot) {
  if (!q.starts) {
    const int m = (int)(((int64_t)q.n + seg - 1) / seg), b = slot / m, c = slot - b * m;
    return {b, c * seg, min(seg, q.n - c * seg), b, c == 0, c == m - 1};
  }
  int lo = 0, hi = q.num;       // the last sequence whose first slot is not past this one
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (seq_start(q, mid) / seg + mid <= slot) lo = mid; else hi = mid;
  }
  const int a = seq_start(q, lo), e = max(seq_start(q, lo + 1), a), c = slot - (a / seg + lo);
  if (c < 0 || (int64_t)c * seg >= e - a) return {0, 0, 0, lo, false, false};
  return {0, a + c * seg, min(seg, e - a - c * seg), lo, c == 0, (int64_t)(c + 1) * seg >= e - a};
}
// First slot of sequence s and its segments.
struct SeqSlots {
  int first, count;
};
__device__ __forceinline__ SeqSlots seq_slots(const DeltaSeqs& q, int seg, int s) {
  if (!q.starts) {
    const int m = (int)(((int64_t)q.n + seg - 1) / seg);
    return {s * m, m};
  }
  const int a = seq_start(q, s), e = max(seq_start(q, s + 1), a);
  return {a / seg + s, (int)(((int64_t)(e - a) + seg - 1) / seg)};
}

__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }

// A chunk's gates for one head in LDS, base 2 logarithms: b in two parts, exp(b), the rates, and exp(b_63 - b) r.
struct Gates {
  float hi[kDC], lo[kDC], eb[kDC], r[kDC], w[kDC];
};

// A chunk's gates from its lanes' dt (one wave; tokens past len leave the state alone).  Log decays below kResetDecay
// are taken as that: exp of them is zero either way, and sums of 64 stay where `hi` is exact.  rest: exp(b_63 - b), if
// wanted.  Returns the chunk's sum.
__device__ __forceinline__ double make_gates(float dt, float A, float bias, bool softplus, int len, Gates* o,
                                             float* rest = nullptr) {
  const int lane = lane_id();
  const float r = lane < len ? scan_rate(dt, bias, softplus) : 0.f;
  double b = lane < len ? fmax((double)A * r, (double)kResetDecay) * 1.4426950408889634 : 0.0;
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) {
    const double up = __shfl_up(b, m, 64);
    if (lane >= m) b += up;
  }
  const double last = __shfl(b, 63, 64);
  const float hi = rintf((float)b * 256.f) * (1.f / 256.f);
  o->hi[lane] = hi;
  o->lo[lane] = (float)(b - (double)hi);
  o->eb[lane] = exp2_hw((float)b);
  o->r[lane] = r;
  const float f = exp2_hw((float)(last - b));
  o->w[lane] = r * f;
  if (rest) rest[lane] = f;
  return last;
}

// Values as three bf16 operands.
__device__ __forceinline__ void split3(const float (&v)[8], u32x4& h, u32x4& m, u32x4& l) {
  f32x4 c[2] = {{v[0], v[1], v[2], v[3]}, {v[4], v[5], v[6], v[7]}};
  h = Mat<bf16>::frag(c);
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const u32x4 w = k ? m : h;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        c[i][2 * j] -= __uint_as_float(w[2 * i + j] << 16);
        c[i][2 * j + 1] -= __uint_as_float(w[2 * i + j] & 0xffff0000u);
      }
    (k ? l : m) = Mat<bf16>::frag(c);
  }
}

// An operand of tokens (contraction over 16 bytes of them) times their weights, as parts whose sum it is.
template <typename T> struct Scaled {
  static constexpr int kParts = sizeof(T) == 2 ? 3 : 1;
  u32x4 part[kParts];
  __device__ __forceinline__ Scaled(u32x4 x, const float* w) {
    if constexpr (sizeof(T) == 2) {
      float v[8];
      unpack8(x, v);
      const f32x4 a = *reinterpret_cast<const f32x4*>(w), b = *reinterpret_cast<const f32x4*>(w + 4);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[i] *= a[i];
        v[4 + i] *= b[i];
      }
      split3(v, part[0], part[1], part[2]);
    } else {
      const f32x4 a = *reinterpret_cast<const f32x4*>(w);
#pragma unroll
      for (int i = 0; i < 4; ++i) part[0][i] = __float_as_uint(__uint_as_float(x[i]) * a[i]);
    }
  }
  __device__ __forceinline__ f32x4 mma(u32x4 a, f32x4 c) const {
#pragma unroll
    for (int i = 0; i < kParts; ++i) c = Mat<T>::mma(a, part[kParts - 1 - i], c);
    return c;
  }
};

// The heads' waves of a workgroup: HW heads of a group, PW waves with 16 CT rows of the state each.
template <typename T, int DN_, int HW_, int PW_> struct ScanShape {
  static constexpr int DN = DN_, HW = HW_, PW = PW_, W = HW * PW;
  static constexpr int CT = DN <= 128 ? 2 : 1;              // blocks of P a wave has
  static constexpr int NT = DN / 16, NS = DN / Mat<T>::KB, CS = kDC / Mat<T>::KB;
  static constexpr int cols = 16 * CT * PW;                 // of P, of a workgroup's heads
  static constexpr int kLine = 128 / (int)sizeof(T), DX = cols < kLine ? kLine : cols;
  static constexpr int kB = Panels<T>::bytes(DN), kX = Panels<T>::bytes(DX);
  static constexpr int kM = Mat<T>::kTri * 1024 * (Mat<T>::kSplit ? 2 : 1);
};

// State rows of a wave: element p = row(ct, lane & 15) of its rows, n = Mat::row(nt, 4 g + 0..3).
template <typename T, int CT, int NT> struct StateRows {
  f32x4 s[CT][NT];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int c = 0; c < CT; ++c)
#pragma unroll
      for (int t = 0; t < NT; ++t) s[c][t] = (f32x4){0.f, 0.f, 0.f, 0.f};
  }
  // tile0: the wave's first block of 16 among the head's P rows
  __device__ __forceinline__ void load(const float* S, int tile0, int P, int N) {
    const int m = lane_id() & 15, g = lane_id() >> 4;
#pragma unroll
    for (int c = 0; c < CT; ++c) {
      const int p = Mat<T>::row(tile0 + c, m);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const int n = Mat<T>::row(t, 4 * g);
        s[c][t] = p < P && n < N ? *reinterpret_cast<const f32x4*>(S + (int64_t)p * N + n) : (f32x4){0.f, 0.f, 0.f, 0.f};
      }
    }
  }
  __device__ __forceinline__ void store(float* S, int tile0, int P, int N) const {
    const int m = lane_id() & 15, g = lane_id() >> 4;
#pragma unroll
    for (int c = 0; c < CT; ++c) {
      const int p = Mat<T>::row(tile0 + c, m);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const int n = Mat<T>::row(t, 4 * g);
        if (p < P && n < N) *reinterpret_cast<f32x4*>(S + (int64_t)p * N + n) = s[c][t];
      }
    }
  }
  // += the weighted outer products of a step's tokens: x[c] their features of this wave's blocks, `cols` their rows of N
  // in LDS.  All blocks of P at once, so that an operand is read once.
  __device__ __forceinline__ void add(const u32x4 (&x)[CT], const char* cols, int step, const float* weights, int N) {
    static_assert(CT <= 2, "blocks");
    const Scaled<T> u0(x[0], weights), u1(x[CT - 1], weights);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      if (t / Mat<T>::TPS * Mat<T>::KB < N) {
        const u32x4 f = Panels<T>::frag_t(cols, t, step, lane_id());
        s[0][t] = u0.mma(f, s[0][t]);
        if (CT == 2) s[CT - 1][t] = u1.mma(f, s[CT - 1][t]);
      }
    }
  }
  // A decay that is zero in fp32 empties the state, whatever it holds.
  __device__ __forceinline__ void decay(float a) {
    if (a == 0.f) {
      zero();
    } else {
#pragma unroll
      for (int c = 0; c < CT; ++c)
#pragma unroll
        for (int t = 0; t < NT; ++t) s[c][t] *= a;
    }
  }
};

}  // namespace ttt
