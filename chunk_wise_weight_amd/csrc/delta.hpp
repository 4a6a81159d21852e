// What the kernels of the gated delta rule share (gfx950).
//
// Tokens go in chunks of 64.  Within a chunk, b is the running sum of the log
// decays, S the state [dk, dv] (W^T) before the chunk, and row i a token:
//   L_ij = (k_i . k_j) exp(b_i - b_j)  (j < i),   T = (I + L diag(beta))^-1
//   E    = T (V - exp(b) K S)                     the tokens' errors before beta
//   O    = scale exp(b) Q S + P E,  P_ij = scale (q_i . k_j) exp(b_i - b_j) beta_j  (j <= i)
//   S'   = exp(b_63) S + K^T (exp(b_63 - b) beta E)
// T and P depend on the inputs alone and are made for all chunks at once
// (k_delta_chunks); the walk over the chunks (k_delta_walk) keeps a slice of
// the state's columns in registers.
//
// Operands.  Every product is made of 16 x 16 MFMA blocks whose operand lanes
// hold row lane & 15 and 16 bytes along the contraction.  Result rows are
// dealt to the blocks such (Mat::row) that the registers a lane holds of a
// result are, in order, the operand of the next product contracted over those
// rows: state, errors and their scaled forms go from product to product
// without leaving the registers.
//
// Precision (bf16 inputs).  A product's bf16 operand that comes from fp32
// registers is a pair hi + lo of bf16 values (2^-17 relative), with hi x hi,
// hi x lo and lo x hi summed in fp32: the fp32 state is off by 3e-6 of its norm
// after 64K tokens, and O by its own rounding (1.7e-3; from the exact O rounded,
// 1e-4 to 2e-4).  Of the state's 3e-6 nearly all comes from the two operands of T
// R and K^T E; a third bf16 value for those would leave 8e-7 (emulated in fp64) at
// 22 products and 80 vector instructions more in a chunk's chain of 82 and 250.
// Two keep it hundreds of times closer than the bf16 inputs are to what they
// stand for.  One operand is rounded once: the state in Q S for heads past 128,
// whose pairs LDS has no room for (O off by up to 2.2e-3, where decays are weak).
#pragma once
#include <type_traits>

#include "gemm.hpp"
#include "launch.hpp"

namespace ttt {

constexpr int kDC = 64;          // tokens of a chunk
constexpr float kResetDecay = -200.f;   // log decays below it empty the state

template <typename T> struct Mat;

template <> struct Mat<bf16> {
  static constexpr int KB = 32;            // contraction per product step
  static constexpr int TPS = 2;            // result blocks whose rows make one step
  static constexpr int kTri = 6;           // operand fragments of a lower triangular 64 x 64 matrix
  static constexpr bool kSplit = true;
  // Row of the matrix that block `tile`, block row m stands for: lane group g
  // holds rows g * 8 + 0..3 of a step in its even block and + 4..7 in its odd one.
  __device__ static __forceinline__ int row(int tile, int m) {
    return ((tile >> 1) << 5) + ((m >> 2) << 3) + ((tile & 1) << 2) + (m & 3);
  }
  // steps of a triangular matrix that block `tile` has
  __device__ static constexpr int steps(int tile) { return (tile >> 1) + 1; }
  __device__ static constexpr int tri(int tile, int s) { return tile < 2 ? tile : 2 + (tile - 2) * 2 + s; }
  // the same of an upper triangular one: steps first(tile) .. 64 / KB - 1
  __device__ static constexpr int first(int tile) { return tile >> 1; }
  __device__ static constexpr int triu(int tile, int s) { return tile < 2 ? tile * 2 + s : 4 + (tile - 2); }
  __device__ static __forceinline__ f32x4 mma(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                   0, 0);
  }
  // The operand made of a step's result blocks, rounded to bf16.
  __device__ static __forceinline__ u32x4 frag(const f32x4* c) {
    return (u32x4){pack2_bf16(c[0][0], c[0][1]), pack2_bf16(c[0][2], c[0][3]), pack2_bf16(c[1][0], c[1][1]),
                   pack2_bf16(c[1][2], c[1][3])};
  }
  // Values and what their rounding to bf16 left.
  __device__ static __forceinline__ void split(const f32x4* c, u32x4& hi, u32x4& lo) {
    hi = frag(c);
    f32x4 r[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const unsigned w = hi[2 * i + j];
        r[i][2 * j] = c[i][2 * j] - __uint_as_float(w << 16);
        r[i][2 * j + 1] = c[i][2 * j + 1] - __uint_as_float(w & 0xffff0000u);
      }
    lo = frag(r);
  }
};

template <> struct Mat<float> {
  static constexpr int KB = 16, TPS = 1, kTri = 10;
  static constexpr bool kSplit = false;
  __device__ static __forceinline__ int row(int tile, int m) { return tile * 16 + m; }
  __device__ static constexpr int steps(int tile) { return tile + 1; }
  __device__ static constexpr int tri(int tile, int s) { return tile * (tile + 1) / 2 + s; }
  __device__ static constexpr int first(int tile) { return tile; }
  __device__ static constexpr int triu(int tile, int s) { return tile * 4 - tile * (tile - 1) / 2 + (s - tile); }
  // lane group g holds contraction indices 4 g + r; instruction r takes index 4 g + r of every group
  __device__ static __forceinline__ f32x4 mma(u32x4 a, u32x4 b, f32x4 c) {
#pragma unroll
    for (int r = 0; r < 4; ++r)
      c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a[r]), __uint_as_float(b[r]), c, 0, 0, 0);
    return c;
  }
  __device__ static __forceinline__ u32x4 frag(const f32x4* c) { return __builtin_bit_cast(u32x4, c[0]); }
  __device__ static __forceinline__ void split(const f32x4* c, u32x4& hi, u32x4& lo) {
    hi = frag(c);
    lo = (u32x4){0, 0, 0, 0};
  }
};

// c + a b with b = hi + lo and a exact.
template <typename T>
__device__ __forceinline__ f32x4 mma_split(u32x4 a, u32x4 bh, u32x4 bl, f32x4 c) {
  c = Mat<T>::mma(a, bh, c);
  if (Mat<T>::kSplit) c = Mat<T>::mma(a, bl, c);
  return c;
}

// What k_delta_chunks leaves of a chunk and value head, in operand order
// (fragment, lane, 16 bytes): T (hi, then lo), the gates, P (hi, then lo).  In
// bf16 a fragment on the diagonal is zero in the lanes whose 8 columns lie
// behind their row (lane group g > (lane & 15) >> 2): it is kept as its 40
// other lanes, dealt such that the lanes that LDS serves together (0-3 and 12-15
// of a group with 4-11 of the next) lie in different banks, and 16 bytes of zeros.
template <typename T> struct ChunkRec {
  static constexpr bool kPacked = sizeof(T) == 2;
  static constexpr int kDiag = 41 * 16;
  static constexpr int kPart = kPacked ? 4 * kDiag + 2 * 1024 : Mat<T>::kTri * 1024;  // one triangular matrix
  static constexpr int kTl = kPart;
  static constexpr int kGate = Mat<T>::kSplit ? 2 * kPart : kPart;   // exp(b), beta exp(b_63 - b): 64 floats each
  static constexpr int kP = kGate + (kPacked ? 512 : 1024), kPl = kP + kPart;
  static constexpr int kBytes = (Mat<T>::kSplit ? 2 * kGate + 512 : kGate + 1024 + kPart) + 1023 & ~1023;
  // KB that hold T and the gates, and the gates and P
  static constexpr int kLoadT = (kP + 1023) / 1024, kLoadP = (kBytes - kGate + 1023) / 1024;
  // A lane's place in the fragments of a part: on the diagonal, elsewhere.
  __device__ static __forceinline__ int diag(int lane) {
    const int g = lane >> 4, m = lane & 15;
    if (!kPacked) return lane * 16;
    return (g > m >> 2 ? 40 : g == 0 ? m : g == 1 ? 16 + m : g == 2 ? 32 + ((m & 7) ^ 4) : 4 + m) * 16;
  }
  // The same for a loop over chunks: kept in a register, not made again at every turn.
  __device__ static __forceinline__ int diag_kept(int lane) {
    int d = diag(lane);
    asm volatile("" : "+v"(d));
    return d;
  }
  // Where fragment (t, s) is in a part, from the lane's place on.
  __device__ static constexpr bool on_diag(int t, int s) { return kPacked && s == t >> 1; }
  __device__ static constexpr int at(int t, int s) {
    return !kPacked ? Mat<T>::tri(t, s) * 1024 : on_diag(t, s) ? t * kDiag : 4 * kDiag + (t - 2) * 1024;
  }
  // A lane's operand of fragment (t, s): part + diag(lane), part + 16 lane.
  __device__ static __forceinline__ u32x4 frag(const char* d, const char* f, int t, int s) {
    return *reinterpret_cast<const u32x4*>((on_diag(t, s) ? d : f) + at(t, s));
  }
};
static_assert(ChunkRec<bf16>::kBytes == 19 * 1024 && ChunkRec<float>::kBytes == 21 * 1024, "the header states them");
// The same for the backward pass: the transposes of T and P (hi, lo each), the gates, and b itself (64 doubles).
template <typename T> struct ChunkRecT {
  static constexpr int kFrag = Mat<T>::kTri * 1024;
  static constexpr int kTl = kFrag;
  static constexpr int kP = Mat<T>::kSplit ? 2 * kFrag : kFrag;
  static constexpr int kPl = kP + kFrag;
  static constexpr int kGate = 2 * kP;
  static constexpr int kBytes = kGate + 1024;
};

// Rows from `base` on: loads through it test rows and columns themselves.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_rsrc(const void* base) { return make_rsrc(base, kOOB); }

// R (64) rows of up to DK elements in LDS: panels of 128 bytes a row, the 16-byte
// chunk c of row r in slot c ^ panel_swz(r).  The 16 rows of an operand read
// (Mat::row: rows 0-3, 8-11, 16-19, 24-27 of a step, or the other four of each
// eight) differ in row & 1 and the three bits used here, so they fall into 16
// different 16-byte bank groups.
__device__ __forceinline__ int panel_swz(int r) { return ((r >> 1) & 1) | (((r >> 3) & 3) << 1); }
template <typename T, int R = kDC> struct Panels {
  static constexpr int kPanel = R * 128;
  static constexpr int bytes(int DK) { return DK * (int)sizeof(T) * R; }
  // 16 bytes of row r at contraction step s, lane group g
  __device__ static __forceinline__ u32x4 frag(const char* t, int r, int s, int g) {
    return *reinterpret_cast<const u32x4*>(t + (s >> 1) * kPanel + r * 128 + (((4 * (s & 1) + g) ^ panel_swz(r)) << 4));
  }
  // The transpose's operand: row = column Mat::row(tile, lane & 15), contraction over the rows, step s.
  __device__ static __forceinline__ u32x4 frag_t(const char* t, int tile, int s, int lane) {
    const int j = lane & 15, g = lane >> 4;
    if constexpr (sizeof(T) == 2) {
      // ds_read_b64_tr_b16: lane j of a 16-lane group addresses 4 columns of row j >> 2 and receives
      // column j of the 16 addressed, rows 0..3
      const int col = ((tile >> 1) << 5) + ((j & 3) << 3), r = s * 32 + g * 8 + (j >> 2);
      const char* p = t + (col >> 6) * kPanel + ((tile & 1) << 3);
      const int c = (col & 63) >> 3;
      const s16x4 x = lds_read_tr16(p + r * 128 + ((c ^ panel_swz(r)) << 4));
      const s16x4 y = lds_read_tr16(p + (r + 4) * 128 + ((c ^ panel_swz(r + 4)) << 4));
      const u32x2 a = __builtin_bit_cast(u32x2, x), b = __builtin_bit_cast(u32x2, y);
      return (u32x4){a[0], a[1], b[0], b[1]};
    } else {
      const int col = tile * 16 + j, c = (col & 31) >> 2;
      u32x4 o;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = s * 16 + g * 4 + i;
        o[i] = *reinterpret_cast<const unsigned*>(t + (col >> 5) * kPanel + r * 128 + ((c ^ panel_swz(r)) << 4) +
                                                  ((col & 3) << 2));
      }
      return o;
    }
  }
  // place of element (r, col)
  __device__ static __forceinline__ int at(int r, int col) {
    const int byte = col * (int)sizeof(T);
    return (byte >> 7) * kPanel + r * 128 + ((((byte & 127) >> 4) ^ panel_swz(r)) << 4) + (byte & 15);
  }
};

// DMA of all panels by NW waves, 8 rows of a panel an instruction.  Rows >= len and columns >= row_bytes read as
// zero; the lanes' offsets are the same for every chunk of a walk and made once.
template <typename T, int DK, int NW, int R = kDC> struct PanelLoader {
  static constexpr int N = DK * (int)sizeof(T) * R / 1024 / NW;
  unsigned off[N];
  __device__ __forceinline__ PanelLoader(unsigned pitch, unsigned row_bytes) {
    const int L = lane_id(), w = wave_id() % NW;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int i = j * NW + w, b = i % (R / 8);
      const unsigned byte = (unsigned)(((L & 7) ^ ((L >> 4) & 1) ^ ((b & 3) << 1)) << 4) + (unsigned)(i / (R / 8)) * 128u;
      off[j] = byte < row_bytes ? (unsigned)(b * 8 + (L >> 3)) * pitch + byte : kOOB;
    }
  }
  // (left out of the host's pass, which drops kernels that call it from here)
  __device__ __forceinline__ void issue(const void* rows, int len, char* t) const {
#if __HIP_DEVICE_COMPILE__
    const __amdgpu_buffer_rsrc_t rs = rows_rsrc(rows);
    const int L = lane_id(), w = wave_id() % NW;
    if (len >= R) {
#pragma unroll
      for (int j = 0; j < N; ++j)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_ptr_t)(t + w * 1024 + j * (NW * 1024)), 16, off[j], 0, 0, 0);
    } else {
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const int i = j * NW + w;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_ptr_t)(t + i * 1024), 16,
                                                 (i % (R / 8)) * 8 + (L >> 3) < len ? off[j] : kOOB, 0, 0, 0);
      }
    }
#endif
  }
};

// 64 rows of a wave group's own columns: NW waves with 16 columns each, row by row.
template <typename T, int NW> struct Columns {
  static constexpr int kPitch = 16 * NW * (int)sizeof(T), kBytes = kDC * kPitch;
  static constexpr int N = kBytes / 1024, GPR = kPitch / 16, RPI = 64 / GPR;   // 16-byte pieces a row, rows a load
  unsigned off[N];
  // cols: valid columns from this group's first on
  __device__ __forceinline__ Columns(unsigned pitch, int cols) {
    const int L = lane_id(), c = L % GPR;
#pragma unroll
    for (int j = 0; j < N; ++j)
      off[j] = c * (16 / (int)sizeof(T)) < cols ? (unsigned)(j * RPI + L / GPR) * pitch + c * 16u : kOOB;
  }
  __device__ __forceinline__ void issue(const void* rows, int len, char* t) const {
    const __amdgpu_buffer_rsrc_t rs = rows_rsrc(rows);
    const int L = lane_id();
#pragma unroll
    for (int j = 0; j < N; ++j)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_ptr_t)(t + j * 1024), 16,
                                               j * RPI + L / GPR < len ? off[j] : kOOB, 0, 0, 0);
  }
  // Column lane & 15 of wave w's, rows Mat::row(tile, 4 g + 0..3), as it lies in LDS and widened.
  using Raw = typename std::conditional<sizeof(T) == 2, u32x2, f32x4>::type;
  __device__ static __forceinline__ Raw read(const char* t, int w, int tile, int lane) {
    const int m = lane & 15, r = Mat<T>::row(tile, (lane >> 4) * 4);
    if constexpr (sizeof(T) == 2) {
      return __builtin_bit_cast(u32x2, lds_read_tr16(t + (r + (m >> 2)) * kPitch + w * 32 + (m & 3) * 8));
    } else {
      f32x4 o;
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = *reinterpret_cast<const float*>(t + (r + i) * kPitch + (w * 16 + m) * 4);
      return o;
    }
  }
  __device__ static __forceinline__ f32x4 wide(u32x2 x) {
    return (f32x4){__uint_as_float(x[0] << 16), __uint_as_float(x[0] & 0xffff0000u), __uint_as_float(x[1] << 16),
                   __uint_as_float(x[1] & 0xffff0000u)};
  }
  __device__ static __forceinline__ f32x4 wide(f32x4 x) { return x; }
};

// `N` KB that lie one after the other, by one wave; bytes from `most` on read as zero.
template <int N>
__device__ __forceinline__ void load_block(const void* base, char* t, int most = N * 1024) {
  const __amdgpu_buffer_rsrc_t rs = make_rsrc(base, most);
#pragma unroll
  for (int i = 0; i < N; ++i)
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_ptr_t)(t + i * 1024), 16, (unsigned)(i * 1024 + lane_id() * 16),
                                             0, 0, 0);
}

// Waits until at most N of this wave's memory operations are under way.
template <int N> __device__ __forceinline__ void wait_vm() {
  static_assert(N < 64, "vmcnt has 6 bits");
  __builtin_amdgcn_s_waitcnt(0x0f70 | (N & 15) | ((N >> 4) << 14));
}

// A turn's barrier; with one stage another before it, when the stage has been read.
template <int STAGES> __device__ __forceinline__ void next_turn(bool first) {
  if (STAGES == 1 && !first) __syncthreads();
  __syncthreads();
}

// The DMA wave of a walk: issue(i) brings what the i-th turn works on.  With
// two stages turn i's work hides turn i + 1's loads, with one they follow one
// another.
template <int STAGES, typename I>
__device__ __forceinline__ void dma_wave(int turns, I issue) {
  if (STAGES == 2 && turns > 0) issue(0);
  for (int i = 0; i < turns; ++i) {
    if (STAGES == 1) {
      if (i > 0) __syncthreads();
      issue(i);
    }
    wait_vm<0>();
    __syncthreads();
    if (STAGES == 2 && i + 1 < turns) issue(i + 1);
  }
}
// Which (sequence, value head, part of dv) a workgroup of a walk has.  The
// workgroups of a key head read the same K (and Q): they go to one XCD, whose
// L2 then brings it once; the key heads (of all sequences, in order) are dealt
// to the XCDs in turn, so that long sequences spread over the chip.
struct WalkPlace {
  int seq, h, part;
};
inline __host__ __device__ int64_t walk_blocks(int64_t units, int64_t per) { return (units + 7) / 8 * 8 * per; }
__device__ __forceinline__ bool walk_place(int bid, int sequences, int Hk, int group, int parts, WalkPlace* o) {
  const int per = group * parts, unit = bid / 8 / per * 8 + (bid & 7), j = bid / 8 % per;
  if (unit >= sequences * Hk) return false;
  *o = {unit / Hk, unit % Hk * group + j / parts, j % parts};
  return true;
}

// ------------------------------------------------------------------ sequences and their chunks

// Packed rows: sequence i's chunks take the slots from starts[i] / 64 + i on.
// That leaves every sequence room for its chunks (a sequence touches at most
// one more 64-token cell than it has full chunks) and needs no prefix sum: the
// slots number n / 64 + num, and none where there is no sequence (the single
// start has no end behind it to read).  Starts are brought into 0..n and an end
// before its start counts as the start, so no value of theirs leads out of the
// rows.
__device__ __forceinline__ int seq_start(const DeltaSeqs& q, int i) { return min(max(q.starts[i], 0), q.n); }
inline __host__ __device__ int64_t delta_slots(const DeltaSeqs& q, int batch) {
  if (q.starts) return q.num > 0 ? (int64_t)q.n / kDC + q.num : 0;
  return (int64_t)batch * ((q.n + kDC - 1) / kDC);
}

// Where sequence s lies: batch row, first token, tokens, first chunk slot.
struct SeqPlace {
  int b, tok0, len, slot0;
};
__device__ __forceinline__ SeqPlace seq_place(const DeltaSeqs& q, int s) {
  if (q.starts) {
    const int a = seq_start(q, s), e = max(seq_start(q, s + 1), a);
    return {0, a, e - a, a / kDC + s};
  }
  return {s, 0, q.n, s * ((q.n + kDC - 1) / kDC)};
}

// Where a chunk slot's tokens lie; len <= 0: the slot has none.
struct ChunkPlace {
  int b, tok0, len;
  int seq;
  bool first, last;             // of its sequence
};
__device__ __forceinline__ ChunkPlace chunk_place(const DeltaSeqs& q, int slot) {
  if (!q.starts) {
    const int m = (q.n + kDC - 1) / kDC, b = slot / m, c = slot - b * m;
    return {b, c * kDC, min(kDC, q.n - c * kDC), b, c == 0, c == m - 1};
  }
  int lo = 0, hi = q.num;       // the last sequence whose first slot is not past this one
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (seq_start(q, mid) / kDC + mid <= slot) lo = mid; else hi = mid;
  }
  const int a = seq_start(q, lo), e = max(seq_start(q, lo + 1), a), c = slot - (a / kDC + lo);
  if (c < 0 || c * kDC >= e - a) return {0, 0, 0, lo, false, false};
  return {0, a + c * kDC, min(kDC, e - a - c * kDC), lo, c == 0, (c + 1) * kDC >= e - a};
}

}  // namespace ttt
