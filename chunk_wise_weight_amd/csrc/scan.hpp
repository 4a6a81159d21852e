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
// Operands are as in delta.hpp (Mat): a product's result is the next one's operand without leaving the registers.  The outputs are made transposed, rows of P by tokens, so that a lane has consecutive features of a token.
//
// Precision (bf16 inputs).  x, B and C enter as they are.  What is fp32 enters as sums of bf16 values: the scaled x of
// the state's update as three (24 bits), the state and the decayed C B^T of the outputs as two (17 bits), so that the
// state is fp32's own and O off by its own rounding.  Running sums of log decays are fp64.
#pragma once
#include "delta.hpp"
#include "scan_rate.hpp"

namespace ttt {

// Where a segment slot's tokens lie; len <= 0: the slot has none.  Slots are dealt as the chunks' of delta.hpp, with
// segments of `seg` tokens in place of 64.  Cuts between segments are numbered without those between sequences: segment c of
// a packed sequence that starts at a has a / seg + c behind it, since it has c + 1 segments more of a row's n tokens only if
// they hold as many times seg.
struct SegPlace {
  int b, tok0, len, seq;
  int cut;                      // behind it; the one before it is cut - 1
  bool first, last;             // of its sequence
};
inline __host__ __device__ int64_t seg_slots(const DeltaSeqs& q, int batch, int seg) {
  if (q.starts) return q.num > 0 ? (int64_t)q.n / seg + q.num : 0;
  return (int64_t)batch * (((int64_t)q.n + seg - 1) / seg);
}
inline int64_t seg_cuts(const DeltaSeqs& q, int batch, int seg) {
  if (q.starts) return q.num > 0 ? q.n / seg : 0;
  return q.n > 0 ? (int64_t)batch * ((q.n - 1) / seg) : 0;
}
__device__ __forceinline__ SegPlace seg_place(const DeltaSeqs& q, int seg, int slot) {
  if (!q.starts) {
    const int m = (int)(((int64_t)q.n + seg - 1) / seg), b = slot / m, c = slot - b * m;
    return {b, c * seg, min(seg, q.n - c * seg), b, b * (m - 1) + c, c == 0, c == m - 1};
  }
  int lo = 0, hi = q.num;       // the last sequence whose first slot is not past this one
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (seq_start(q, mid) / seg + mid <= slot) lo = mid; else hi = mid;
  }
  const int a = seq_start(q, lo), e = max(seq_start(q, lo + 1), a), c = slot - (a / seg + lo);
  if (c < 0 || (int64_t)c * seg >= e - a) return {0, 0, 0, lo, 0, false, false};
  return {0, a + c * seg, min(seg, e - a - c * seg), lo, a / seg + c, c == 0, (int64_t)(c + 1) * seg >= e - a};
}
// First cut of sequence s and its segments.
struct SeqCuts {
  int first, count;
};
__device__ __forceinline__ SeqCuts seq_cuts(const DeltaSeqs& q, int seg, int s) {
  if (!q.starts) {
    const int m = (int)(((int64_t)q.n + seg - 1) / seg);
    return {s * (m - 1), m};
  }
  const int a = seq_start(q, s), e = max(seq_start(q, s + 1), a);
  return {a / seg, (int)(((int64_t)(e - a) + seg - 1) / seg)};
}

// Row block and step of a triangular matrix's fragment.
template <typename T> __device__ __forceinline__ void tri_place(int f, int* t, int* s) {
  if constexpr (sizeof(T) == 2) {
    *t = f < 2 ? f : 2 + ((f - 2) >> 1);
    *s = f < 2 ? 0 : (f - 2) & 1;
  } else {
    *t = f < 1 ? 0 : f < 3 ? 1 : f < 6 ? 2 : 3;
    *s = f - *t * (*t + 1) / 2;
  }
}

__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }

// Tiles in LDS: panels of 64 rows of 128 bytes, the 16-byte chunk c of row r in slot c ^ row_swz(r).  Rows are read 16 a
// time (row(t, .) differ in bits 0, 1, 3 and 4; LDS serves lanes 0-3 and 12-15 of a group with 4-11 of the next, whose
// slots differ by 1), columns by transposing reads of 8 bytes from 4 rows a lane group, a whole 32 bytes of each: all fall
// into different banks.
constexpr int kPanel64 = 64 * 128;
__device__ __forceinline__ int row_swz(int r) { return ((r >> 1) & 1) << 1 ^ ((r >> 3) & 1) << 2 ^ ((r >> 4) & 1) * 5; }
template <typename T> constexpr int tile_bytes(int cols) { return cols * (int)sizeof(T) * 64; }

// DMA of a tile of DK columns by NW waves, 8 rows of a panel an instruction.  Rows >= len and columns >= row_bytes read
// as zero; the lanes' offsets are the same for every chunk of a walk and made once.
template <typename T, int DK, int NW> struct TileLoader {
  static constexpr int N = tile_bytes<T>(DK) / 1024 / NW;
  static_assert(N >= 1, "an instruction a wave");
  unsigned off[N];
  __device__ __forceinline__ TileLoader(unsigned pitch, unsigned row_bytes) {
    const int L = lane_id(), w = wave_id() % NW;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int i = j * NW + w, b = i % 8, r = b * 8 + (L >> 3);
      const unsigned byte = (unsigned)(((L & 7) ^ row_swz(r)) << 4) + (unsigned)(i / 8) * 128u;
      off[j] = byte < row_bytes ? (unsigned)r * pitch + byte : kOOB;
    }
  }
  __device__ __forceinline__ void issue(const void* rows, int len, char* t) const {
#if __HIP_DEVICE_COMPILE__
    const __amdgpu_buffer_rsrc_t rs = rows_rsrc(rows);
    const int L = lane_id(), w = wave_id() % NW;
    if (len >= 64) {
#pragma unroll
      for (int j = 0; j < N; ++j)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_ptr_t)(t + (j * NW + w) * 1024), 16, off[j], 0, 0, 0);
    } else {
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const int i = j * NW + w;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_ptr_t)(t + i * 1024), 16,
                                                 (i % 8) * 8 + (L >> 3) < len ? off[j] : kOOB, 0, 0, 0);
      }
    }
#endif
  }
};

// Where a lane reads operands of a tile: the parts that depend on it, in registers; blocks and steps are offsets (or flip
// bits of the slot) from there.
//   place, frag  16 bytes of row(t, lane & 15) at step s of the columns
//   halves       the same with the columns in the order in which two blocks of results hold them: 4 g + 0..3 of each
//   cols         column 16 t + (lane & 15), rows of step s (as a contraction over rows takes them); cols_row: row(t, .)
//   at, at_row   columns 16 ct + 4 g + 0..3, row(ct, 4 g + 0..3), of row(t, lane & 15)
template <typename T> struct LaneAt;
template <> struct LaneAt<bf16> {
  unsigned f, c, n, h;
  __device__ __forceinline__ explicit LaneAt(int lane) {
    const int m = lane & 15, g = lane >> 4, r = (m >> 2) * 8 + (m & 3), rt = g * 8 + (m >> 2);
    f = r * 128 + ((g ^ row_swz(r)) << 4);
    h = r * 128 + (((g >> 1) ^ row_swz(r)) << 4) + (g & 1) * 8;
    c = rt * 128 + (((m & 3) ^ row_swz(rt)) << 4);
    n = rt * 128 + ((((m >> 1) & 1) ^ row_swz(rt)) << 4) + (m & 1) * 8;
    asm volatile("" : "+v"(f), "+v"(c), "+v"(n), "+v"(h));
  }
  __device__ static __forceinline__ int rows(int t) { return (t >> 1) * 4096 + (t & 1) * 512; }
  __device__ static __forceinline__ u32x4 pair(u32x2 a, u32x2 b) { return (u32x4){a[0], a[1], b[0], b[1]}; }
  __device__ static __forceinline__ u32x4 read_t(const char* q) {
    return pair(__builtin_bit_cast(u32x2, lds_read_tr16(q)), __builtin_bit_cast(u32x2, lds_read_tr16(q + 512)));
  }
  __device__ __forceinline__ char* place(char* p, int t, int s) const {
    return p + (f ^ (unsigned)(s & 1) << 6) + ((s >> 1) * kPanel64 + rows(t));
  }
  __device__ __forceinline__ u32x4 frag(const char* p, int t, int s) const {
    return *reinterpret_cast<const u32x4*>(place(const_cast<char*>(p), t, s));
  }
  __device__ __forceinline__ u32x4 halves(const char* p, int t, int s) const {
    const int o = (s >> 1) * kPanel64 + rows(t);
    return pair(*reinterpret_cast<const u32x2*>(p + (h ^ (unsigned)(s & 1) << 6) + o),
                *reinterpret_cast<const u32x2*>(p + (h ^ (unsigned)(s & 1) << 6 ^ 32u) + o));
  }
  __device__ __forceinline__ u32x4 cols(const char* p, int t, int s) const {
    return read_t(p + (n ^ (unsigned)(t & 3) << 5) + ((t >> 2) * kPanel64 + s * 4096));
  }
  __device__ __forceinline__ u32x4 cols_row(const char* p, int t, int s) const {
    return read_t(p + (c ^ (unsigned)((t >> 1) & 1) << 6) + ((t >> 2) * kPanel64 + s * 4096 + (t & 1) * 8));
  }
  __device__ __forceinline__ f32x4 at(const char* p, int t, int ct) const {
    return load4((const bf16*)(p + (h ^ (unsigned)(ct & 3) << 5) + ((ct >> 2) * kPanel64 + rows(t))));
  }
  __device__ __forceinline__ f32x4 at_row(const char* p, int t, int ct) const {
    return load4((const bf16*)(p + (f ^ (unsigned)((ct >> 1) & 1) << 6) + ((ct >> 2) * kPanel64 + (ct & 1) * 8 + rows(t))));
  }
};
// fp32: row(t, i) is 16 t + i, and a step's contraction goes over 16.
template <> struct LaneAt<float> {
  unsigned f, c;
  __device__ __forceinline__ explicit LaneAt(int lane) {
    const int m = lane & 15, g = lane >> 4;
    f = m * 128 + ((g ^ row_swz(m)) << 4);
    c = g * 512 + (((m >> 2) ^ row_swz(4 * g)) << 4) + (m & 3) * 4;
    asm volatile("" : "+v"(f), "+v"(c));
  }
  __device__ __forceinline__ char* place(char* p, int t, int s) const {
    return p + (f ^ (unsigned)(s & 1) << 6 ^ (unsigned)(t & 1) * 0x50u) + ((s >> 1) * kPanel64 + t * 2048);
  }
  __device__ __forceinline__ u32x4 frag(const char* p, int t, int s) const {
    return *reinterpret_cast<const u32x4*>(place(const_cast<char*>(p), t, s));
  }
  __device__ __forceinline__ u32x4 halves(const char* p, int t, int s) const { return frag(p, t, s); }
  __device__ __forceinline__ u32x4 cols(const char* p, int t, int s) const {
    const unsigned q = c ^ (unsigned)(t & 1) << 6 ^ (unsigned)(s & 1) * 0x50u;
    const int o = (t >> 1) * kPanel64 + s * 2048;
    const char *q0 = p + q + o, *q1 = p + (q ^ 32u) + o;
    return (u32x4){*reinterpret_cast<const unsigned*>(q0), *reinterpret_cast<const unsigned*>(q0 + 128),
                   *reinterpret_cast<const unsigned*>(q1 + 256), *reinterpret_cast<const unsigned*>(q1 + 384)};
  }
  __device__ __forceinline__ u32x4 cols_row(const char* p, int t, int s) const { return cols(p, t, s); }
  __device__ __forceinline__ f32x4 at(const char* p, int t, int ct) const { return __builtin_bit_cast(f32x4, frag(p, t, ct)); }
  __device__ __forceinline__ f32x4 at_row(const char* p, int t, int ct) const { return at(p, t, ct); }
};

// A chunk's gates for one head, base 2 logarithms, a lane for each token (one wave; tokens past len leave the state
// alone).  Log decays below kLeastLog are taken as that: exp of them is zero either way.
constexpr double kLeastLog = -120.0;
struct LaneGates {
  double b, sum;                      // running sum of the log decays, the chunk's
  float r;
};
// Lane i's x added to lane i + by, within the rows of 16 (by < 16) or from row to row (row_bcast), nothing where no lane is.
template <int CTRL, int ROWS> __device__ __forceinline__ double dpp_add(double x) {
  const u32x2 v = __builtin_bit_cast(u32x2, x);
  const u32x2 up = {(unsigned)__builtin_amdgcn_update_dpp(0, (int)v[0], CTRL, ROWS, 0xf, false),
                    (unsigned)__builtin_amdgcn_update_dpp(0, (int)v[1], CTRL, ROWS, 0xf, false)};
  return x + __builtin_bit_cast(double, up);
}
__device__ __forceinline__ LaneGates make_gates(float dt, float A, float bias, bool softplus, int len) {
  const int lane = lane_id();
  LaneGates v;
  v.r = lane < len ? scan_rate(dt, bias, softplus) : 0.f;
  double b = lane < len ? fmax((double)A * v.r, kLeastLog) * 1.4426950408889634 : 0.0;
  b = dpp_add<0x111, 0xf>(b);         // row_shr 1, 2, 4, 8
  b = dpp_add<0x112, 0xf>(b);
  b = dpp_add<0x114, 0xf>(b);
  b = dpp_add<0x118, 0xf>(b);
  b = dpp_add<0x142, 0xa>(b);         // row_bcast 15 into rows 1 and 3, 31 into 2 and 3
  b = dpp_add<0x143, 0xc>(b);
  const u32x2 w = __builtin_bit_cast(u32x2, b);
  const u32x2 l = {(unsigned)__builtin_amdgcn_readlane((int)w[0], 63), (unsigned)__builtin_amdgcn_readlane((int)w[1], 63)};
  v.b = b;
  v.sum = __builtin_bit_cast(double, l);
  return v;
}
// b in two parts, the first a multiple of 2^-8 below 2^14: differences of first parts are exact.
__device__ __forceinline__ void two_parts(double b, float* hi, float* lo) {
  *hi = rintf((float)b * 256.f) * (1.f / 256.f);
  *lo = (float)(b - (double)*hi);
}

// Gates as they lie in LDS: b in two parts, exp(b), the rates, and exp(b_63 - b) r.  bf16 outputs take one fp32 b, lo 0, where
// the chunk's sum stays above kOnePart: differences of two such are off by 2^-16 at most, as the products are.  Sums of 64
// reach 2^14 (tokens that empty the state), where one part would be off by 2^-10.
constexpr double kOnePart = -256.0;
struct Gates {
  float hi[kDC], lo[kDC], eb[kDC], r[kDC], w[kDC];
};
template <typename T> __device__ __forceinline__ void put_gates(const LaneGates& v, Gates* o) {
  const int lane = lane_id();
  float hi, lo;
  two_parts(v.b, &hi, &lo);
  const bool one = sizeof(T) == 2 && v.sum >= kOnePart;
  o->hi[lane] = one ? (float)v.b : hi;
  o->lo[lane] = one ? 0.f : lo;
  o->eb[lane] = exp2_hw((float)v.b);
  o->r[lane] = v.r;
  o->w[lane] = v.r * exp2_hw((float)(v.sum - v.b));
}
// Whether lo may be other than 0 (hi of the last token is off by 2^-9 at most), the same for all lanes.
template <typename T> __device__ __forceinline__ bool two_part_gates(const Gates& g) {
  return sizeof(T) == 4 ||
         __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(g.hi[kDC - 1]))) < (float)kOnePart + 0.5f;
}
// The same as the backward pass keeps them for its chunk-local part, b in two parts, with exp(b_63 - b) and the rate's
// derivative by dt.
struct KeptGates {
  Gates g;
  float rest[kDC], slope[kDC];
};

// fp32 results to operands of bf16 values whose sum they are.  What a rounding leaves is made by the matrix cores: a
// result plus (-1 at its own place) times the rounded operand, exact, and off the vector units, which bound these kernels
// (16 vector instructions less for each operand and part).
template <typename T> struct Split {
  u32x4 minus[2];                     // -1 at row(u, lane & 15), u the block of a step
  __device__ __forceinline__ explicit Split(int lane) {
    const int m = lane & 15, g = lane >> 4;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int e = 4 * u + (m & 3);
#pragma unroll
      for (int i = 0; i < 4; ++i) minus[u][i] = g == m >> 2 && i == e >> 1 ? 0xbf80u << (16 * (e & 1)) : 0u;
    }
    asm volatile("" : "+v"(minus[0]), "+v"(minus[1]));
  }
  __device__ __forceinline__ void rest(f32x4* c, u32x4 h) const {
#pragma unroll
    for (int u = 0; u < 2; ++u) c[u] = Mat<T>::mma(minus[u], h, c[u]);
  }
  __device__ __forceinline__ void two(const f32x4* v, u32x4& h, u32x4& l) const {
    f32x4 c[2] = {v[0], v[1]};
    h = Mat<T>::frag(c);
    rest(c, h);
    l = Mat<T>::frag(c);
  }
};
template <> struct Split<float> {
  __device__ __forceinline__ explicit Split(int) {}
  __device__ __forceinline__ void two(const f32x4* v, u32x4& h, u32x4&) const { h = Mat<float>::frag(v); }
};

// An operand of tokens (contraction over 16 bytes of them) times their weights, as parts whose sum it is: bf16 three, 24
// bits in all.
template <typename T> struct Scaled {
  static constexpr int kParts = sizeof(T) == 2 ? 3 : 1;
  u32x4 part[kParts];
  __device__ __forceinline__ Scaled(const Split<T>& sp, u32x4 x, const float* w) {
    const f32x4 a = *reinterpret_cast<const f32x4*>(w);
    if constexpr (sizeof(T) == 2) {
      const f32x4 b = *reinterpret_cast<const f32x4*>(w + 4);
      float v[8];
      unpack8(x, v);
      f32x4 c[2];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        c[0][i] = v[i] * a[i];
        c[1][i] = v[4 + i] * b[i];
      }
#pragma unroll
      for (int k = 0; k < 3; ++k) {
        part[k] = Mat<T>::frag(c);
        if (k < 2) sp.rest(c, part[k]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) part[0][i] = __float_as_uint(__uint_as_float(x[i]) * a[i]);
    }
  }
};

// Blocks of P that a wave has: two read B and C from LDS half as often, where the registers hold two (fp32 has its
// operands in three parts at once).
template <typename T, int DN> constexpr int kBlocks = sizeof(T) == 2 && DN <= 128 ? 2 : 1;

// Whether a state's columns from `col` on, zero past N, may be left out: looked at where a branch costs less than what it
// saves, every 16 columns in fp32, whose products take eight times as long, every 64 of the widest in bf16.
template <typename T, int DN> __device__ __forceinline__ bool past(int col, int N) {
  return (sizeof(T) == 4 ? col > 0 : DN > 128 && col % 64 == 0) && col >= N;
}

// The heads' waves of a workgroup: HW heads of a group, PW waves with CT blocks of 16 rows of the state each.
template <typename T, int DN_, int HW_, int PW_, int CT_ = kBlocks<T, DN_>> struct ScanShape {
  static constexpr int DN = DN_, HW = HW_, PW = PW_, W = HW * PW;
  static constexpr int CT = CT_;
  static constexpr int NT = DN / 16, NS = DN / Mat<T>::KB, CS = kDC / Mat<T>::KB;
  static constexpr int cols = 16 * CT * PW;                 // of P, of a workgroup's heads
  static constexpr int kLine = 128 / (int)sizeof(T), DX = cols < kLine ? kLine : cols;
  static constexpr int kB = tile_bytes<T>(DN), kX = tile_bytes<T>(DX);
  static constexpr int kM = Mat<T>::kTri * 1024 * (Mat<T>::kSplit ? 2 : 1);
};

// The row of P that index i of block `tile` stands for: two blocks of bf16 a wave are dealt such that 8 of a result's rows
// follow one another.
template <typename T, int CT> __device__ __forceinline__ int state_row(int tile, int i) {
  return CT == 2 ? Mat<T>::row(tile, i) : tile * 16 + i;
}
// The operand of their columns, rows of step s.
template <typename T, int CT> __device__ __forceinline__ u32x4 state_cols(const LaneAt<T>& L, const char* x, int tile, int s) {
  return CT == 2 ? L.cols_row(x, tile, s) : L.cols(x, tile, s);
}

// State rows of a wave: element p = state_row(tile, lane & 15), n = 16 nt + 4 g + 0..3.
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
      const int p = state_row<T, CT>(tile0 + c, m);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const int n = t * 16 + 4 * g;
        s[c][t] = p < P && n < N ? *reinterpret_cast<const f32x4*>(S + (int64_t)p * N + n) : (f32x4){0.f, 0.f, 0.f, 0.f};
      }
    }
  }
  __device__ __forceinline__ void store(float* S, int tile0, int P, int N) const {
    const int m = lane_id() & 15, g = lane_id() >> 4;
#pragma unroll
    for (int c = 0; c < CT; ++c) {
      const int p = state_row<T, CT>(tile0 + c, m);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const int n = t * 16 + 4 * g;
        if (p < P && n < N) *reinterpret_cast<f32x4*>(S + (int64_t)p * N + n) = s[c][t];
      }
    }
  }
  // += the weighted outer products of a step's tokens: x[c] their features of this wave's blocks, `cols` their rows of N
  // in LDS.  All blocks of P at once, so that an operand is read once.
  __device__ __forceinline__ void add(const LaneAt<T>& L, const Split<T>& sp, const u32x4 (&x)[CT], const char* cols,
                                      int step, const float* weights, int N) {
    static_assert(CT <= 2, "blocks");
    const Scaled<T> u0(sp, x[0], weights), u1(sp, x[CT - 1], weights);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      if (past<T, NT * 16>(t * 16, N)) break;
      const u32x4 f = L.cols(cols, t, step);
#pragma unroll
      for (int k = Scaled<T>::kParts - 1; k >= 0; --k) {
        s[0][t] = Mat<T>::mma(f, u0.part[k], s[0][t]);
        if (CT == 2) s[CT - 1][t] = Mat<T>::mma(f, u1.part[k], s[CT - 1][t]);
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
