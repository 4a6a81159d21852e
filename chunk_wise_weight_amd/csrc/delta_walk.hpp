// The kernels that the gated delta rule's forward and backward pass share
// (gfx950); the mathematics and the operand layout are in delta.hpp.
#pragma once
#include "delta.hpp"

namespace ttt {
namespace {

// ------------------------------------------------------------------ T, P and the gates of every chunk

// One workgroup of 4 waves per chunk slot and value head.  Wave w makes row
// block w (16 tokens) of K K^T and Q K^T, the decays in fp64 (differences of
// sums that may have grown large), then T: the four 16 x 16 diagonal blocks by
// substitution, one a wave, and the blocks below them column by column,
//   T_ij = -T_ii sum_{j <= l < i} A_il T_lj,   A = L diag(beta),
// wave j taking column j: fp32 MFMA products, the running block column staying
// in registers as the next product's operand.  64K tokens of 32 heads of 128:
// 356 us (an earlier form's 419: the operands' loads and products about
// 150, the inverse 100, the exponentials 30, the stores 60): each workgroup is a
// chain of short phases, so the more of them a CU holds the better.  Forward: operands of two
// steps at a time and four waves a SIMD (an earlier form's 372 us; four steps and three waves
// 419); the backward's form, with twice the stores, is better off with the
// latter (70 us for 4 x 4096 tokens of 16 heads; 79).
constexpr int kChunkThreads = 256;
constexpr int kLd = 68;           // pitch of a 64 x 64 fp32 matrix in LDS

__device__ __forceinline__ f32x4 mma_f32(const float* a, f32x4 b, f32x4 c) {
  return Mat<float>::mma(*reinterpret_cast<const u32x4*>(a), __builtin_bit_cast(u32x4, b), c);
}

// The lower triangle X (or, with TRANS, its transpose) to memory in operand
// order, in T's type, for bf16 with what that leaves: whole fragments, by waves.
template <typename T, bool TRANS>
__device__ __forceinline__ void put_fragments(const float* X, char* hi, char* lo) {
  constexpr int E = 16 / sizeof(T);
  const int lane = lane_id(), m = lane & 15, g = lane >> 4;
#pragma unroll
  for (int t = 0; t < 4; ++t)
#pragma unroll
    for (int s = 0; s < kDC / Mat<T>::KB; ++s) {
      if (TRANS ? s < Mat<T>::first(t) : s >= Mat<T>::steps(t)) continue;
      const int f = TRANS ? Mat<T>::triu(t, s) : Mat<T>::tri(t, s);
      if ((f & 3) != wave_id()) continue;
      const int r = Mat<T>::row(t, m), k = s * Mat<T>::KB + g * E;
      f32x4 v[E / 4];
#pragma unroll
      for (int i = 0; i < E; ++i) v[i / 4][i % 4] = TRANS ? X[(k + i) * kLd + r] : X[r * kLd + k + i];
      u32x4 h, l;
      Mat<T>::split(v, h, l);
      *reinterpret_cast<u32x4*>(hi + f * 1024 + lane * 16) = h;
      if (Mat<T>::kSplit) *reinterpret_cast<u32x4*>(lo + f * 1024 + lane * 16) = l;
    }
}

// The lower triangle X as a part of ChunkRec: in bf16 its 16 bytes one after the other, by threads.
template <typename T>
__device__ __forceinline__ void put_triangle(const float* X, char* hi, char* lo) {
  using R = ChunkRec<T>;
  if constexpr (!R::kPacked) {
    put_fragments<T, false>(X, hi, lo);
  } else {
    for (int i = threadIdx.x; i < R::kPart / 16; i += kChunkThreads) {
      int t, s = 0, lane;
      if (i < 4 * 41) {                                    // on the diagonal; diag()'s inverse
        t = i / 41;
        s = t >> 1;
        const int p = i - t * 41;
        lane = p < 16 ? p : p < 20 ? 48 + p - 4 : p < 32 ? p : 32 + 8 + ((p - 32) ^ 4);
        if (p == 40) {                                     // the zeros: four rows' columns behind the diagonal
          t &= 2;
          lane = 48;
        }
      } else {
        t = 2 + (i - 4 * 41) / 64;
        lane = (i - 4 * 41) & 63;
      }
      const float* x = X + Mat<T>::row(t, lane & 15) * kLd + s * 32 + (lane >> 4) * 8;
      const f32x4 v[2] = {*reinterpret_cast<const f32x4*>(x), *reinterpret_cast<const f32x4*>(x + 4)};
      u32x4 h, l;
      Mat<T>::split(v, h, l);
      *reinterpret_cast<u32x4*>(hi + i * 16) = h;
      *reinterpret_cast<u32x4*>(lo + i * 16) = l;
    }
  }
}

// With BACK, T goes to rec and the transposes of T and P to rect.
template <typename T, bool BACK>
__global__ __launch_bounds__(kChunkThreads) __attribute__((amdgpu_waves_per_eu(BACK ? 3 : 4))) void k_delta_chunks(
    DeltaArgs p, char* rec, char* rect) {
  constexpr int KB = Mat<T>::KB;
  __shared__ __attribute__((aligned(16))) float A[kDC * kLd], X[kDC * kLd];   // X: P, then T
  __shared__ double b[kDC];
  __shared__ float beta[kDC];
  const int id = xcd_remap(blockIdx.x, gridDim.x);
  const int h = id % p.Hv, slot = id / p.Hv;
  const ChunkPlace c = chunk_place(p.seqs, slot);
  if (c.len <= 0) return;
  char* out = rec + (int64_t)id * ChunkRec<T>::kBytes;
  const int w = wave_id(), lane = lane_id(), m = lane & 15, g = lane >> 4;
  const int kh = h / (p.Hv / p.Hk);

  // Rows of this wave's block against all blocks up to it, GS steps' operands at a time straight from memory, the
  // first of them under way while the gates are made.  Columns past dk read as zero.
  constexpr int GS = BACK ? 4 : 2;
  f32x4 kk[4], qk[4];
#pragma unroll
  for (int t = 0; t < 4; ++t) kk[t] = qk[t] = (f32x4){0.f, 0.f, 0.f, 0.f};
  const __amdgpu_buffer_rsrc_t rk = rows_rsrc((const T*)p.k + c.b * p.sk.b + kh * p.sk.h + c.tok0 * p.sk.t);
  const __amdgpu_buffer_rsrc_t rq = rows_rsrc((const T*)p.q + c.b * p.sq.b + kh * p.sq.h + c.tok0 * p.sq.t);
  const unsigned row_bytes = p.dk * sizeof(T), kp = p.sk.t * sizeof(T), qp = p.sq.t * sizeof(T);
  u32x4 fk[GS][4], fq[GS];
  auto load = [&](int s0) __attribute__((always_inline)) {
#pragma unroll
    for (int s = 0; s < GS; ++s) {
      const unsigned byte = (s0 + s) * 64 + g * 16;
      const int r = w * 16 + m;
      fq[s] = __builtin_amdgcn_raw_buffer_load_b128(rq, r < c.len && byte < row_bytes ? r * qp + byte : kOOB, 0, 0);
#pragma unroll
      for (int t = 0; t < 4; ++t)
        if (t <= w) {
          const int j = t * 16 + m;
          fk[s][t] = __builtin_amdgcn_raw_buffer_load_b128(rk, j < c.len && byte < row_bytes ? j * kp + byte : kOOB, 0, 0);
        }
    }
  };
  load(0);
  if (w == 0) {
    float gi = 0.f, bi = 0.f;
    if (lane < c.len) {
      gi = p.g[c.b * p.sg.b + h * p.sg.h + (c.tok0 + lane) * p.sg.t];
      bi = p.beta[c.b * p.sbeta.b + h * p.sbeta.h + (c.tok0 + lane) * p.sbeta.t];
    }
    // exp(-200) is zero in fp32: a decay of -inf (a state reset) keeps the running sum finite
    double s = gi < kResetDecay ? kResetDecay : gi;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const double up = __shfl_up(s, d, 64);
      if (lane >= d) s += up;
    }
    const double last = __shfl(s, 63, 64);
    b[lane] = s;
    beta[lane] = bi;
    float* gate = reinterpret_cast<float*>(out + ChunkRec<T>::kGate);
    const float up = __expf((float)s), left = bi * __expf((float)(last - s));
    gate[lane] = up;
    gate[64 + lane] = left;
    if (BACK) {
      gate = reinterpret_cast<float*>(rect + (int64_t)id * ChunkRecT<T>::kBytes + ChunkRecT<T>::kGate);
      gate[lane] = up;
      gate[64 + lane] = left;
      reinterpret_cast<double*>(gate + 128)[lane] = s;
    }
  }

  for (int s0 = 0; s0 * KB < p.dk; s0 += GS) {
    if (s0 > 0) load(s0);
#pragma unroll
    for (int s = 0; s < GS; ++s) {
      u32x4 mine = fk[s][0];
#pragma unroll
      for (int t = 1; t < 4; ++t)
        if (t == w) mine = fk[s][t];
#pragma unroll
      for (int t = 0; t < 4; ++t)
        if (t <= w) {
          kk[t] = Mat<T>::mma(mine, fk[s][t], kk[t]);
          qk[t] = Mat<T>::mma(fq[s], fk[s][t], qk[t]);
        }
    }
  }
  __syncthreads();
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    if (t > (w | 1)) continue;      // a block above the diagonal is zero where a fragment holds it too
    const int j = t * 16 + m;
    const float bj = beta[j];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int i = w * 16 + g * 4 + r;
      const float d = i >= j ? __expf((float)(b[i] - b[j])) * bj : 0.f;
      A[i * kLd + j] = i > j ? kk[t][r] * d : 0.f;
      X[i * kLd + j] = i >= j ? p.scale * qk[t][r] * d : 0.f;
    }
  }
  __syncthreads();
  // P to memory in operand order
  char* outt = rect + (int64_t)id * ChunkRecT<T>::kBytes;
  if (BACK)
    put_fragments<T, true>(X, outt + ChunkRecT<T>::kP, outt + ChunkRecT<T>::kPl);
  else
    put_triangle<T>(X, out + ChunkRec<T>::kP, out + ChunkRec<T>::kPl);
  // the diagonal block's inverse: lane m has column m; x_i = [i = m] - sum_{l < i} A_il x_l
  float x[16];
  {
    const float* a = A + (w * 16) * kLd + w * 16;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float v = i == m ? 1.f : 0.f;
#pragma unroll
      for (int l = 0; l < i; ++l) v -= a[i * kLd + l] * x[l];
      x[i] = v;
    }
  }
  __syncthreads();                // P has left X
  if (g == 0)
#pragma unroll
    for (int i = 0; i < 16; ++i) X[(w * 16 + i) * kLd + w * 16 + m] = x[i];
  if ((w & 1) == 0)
#pragma unroll
    for (int i = 0; i < 4; ++i) X[(w * 16 + g * 4 + i) * kLd + w * 16 + 16 + m] = 0.f;
  __syncthreads();
  f32x4 col[4];                   // blocks T_lj of this wave's column j = w, rows g * 4 + r
#pragma unroll
  for (int j = 0; j < 3; ++j) {
    if (w != j) continue;
#pragma unroll
    for (int r = 0; r < 4; ++r) col[j][r] = X[(j * 16 + g * 4 + r) * kLd + j * 16 + m];
#pragma unroll
    for (int i = j + 1; i < 4; ++i) {
      f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int l = j; l < i; ++l) acc = mma_f32(A + (i * 16 + m) * kLd + l * 16 + g * 4, col[l], acc);
      acc = -acc;
      col[i] = mma_f32(X + (i * 16 + m) * kLd + i * 16 + g * 4, acc, (f32x4){0.f, 0.f, 0.f, 0.f});
#pragma unroll
      for (int r = 0; r < 4; ++r) X[(i * 16 + g * 4 + r) * kLd + j * 16 + m] = col[i][r];
    }
  }
  __syncthreads();
  put_triangle<T>(X, out, out + ChunkRec<T>::kTl);
  if (BACK) put_fragments<T, true>(X, outt, outt + ChunkRecT<T>::kTl);
}

// ------------------------------------------------------------------ the walk over the chunks

// Fragments of one wave's 16 state columns to memory as rows of W [dv, dk].
template <typename T, int SS>
__device__ __forceinline__ void put_state(const u32x4 (&S)[SS], T* W, int dk, bool in) {
  const int g = lane_id() >> 4;
#pragma unroll
  for (int s = 0; s < SS; ++s) {
    const int d = s * Mat<T>::KB + g * (16 / (int)sizeof(T));
    if (in && d < dk) *reinterpret_cast<u32x4*>(W + d) = S[s];
  }
}

// O of a chunk's tokens at 16 columns, from operands of the state (Sl: what Sh
// leaves, LO) and the errors (fp32): the columns in the instruction's rows,
// tokens in its columns, so that a lane gets 4 columns of one token.  gp: the
// chunk's gates and P, diag: the lane's place in P; Q in panels at q, or from memory through rq.
template <typename T, int SS, bool LO, int TB, bool QLDS = true>
__device__ __forceinline__ void make_outputs(const u32x4 (&Sh)[SS], const u32x4 (&Sl)[SS], const f32x4 (&e)[4],
                                             const char* gp, int diag, const char* q, float scale, int len, bool in,
                                             int64_t pitch, T* out, const void* q_rows = nullptr, unsigned qp = 0, unsigned qrow = 0) {
  using M = Mat<T>;
  constexpr int CS = kDC / M::KB;
  const int lane = lane_id(), m = lane & 15, g = lane >> 4;
  u32x4 Eh[CS], El[CS];
#pragma unroll
  for (int s = 0; s < CS; ++s) M::split(e + s * M::TPS, Eh[s], El[s]);
  using R = ChunkRec<T>;
  const char *pd = gp + R::kP - R::kGate + diag, *pf = gp + R::kP - R::kGate + lane * 16;
#pragma unroll
  for (int t0 = 0; t0 < 4; t0 += TB) {
    f32x4 o[TB];
    u32x4 f[TB][SS];
#pragma unroll
    for (int i = 0; i < TB; ++i) {
      const int r = M::row(t0 + i, m);
      o[i] = (f32x4){0.f, 0.f, 0.f, 0.f};
      if constexpr (QLDS) {
#pragma unroll
        for (int s = 0; s < SS; ++s) f[i][s] = Panels<T>::frag(q, r, s, g);
      } else {
        const __amdgpu_buffer_rsrc_t rq = rows_rsrc(q_rows);
#pragma unroll
        for (int s = 0; s < SS; ++s) {
          const unsigned byte = s * 64u + g * 16u;
          const unsigned at = r < len && byte < qrow ? (unsigned)r * qp + byte : kOOB;
          f[i][s] = __builtin_amdgcn_raw_buffer_load_b128(rq, at, 0, 0);
        }
      }
    }
#pragma unroll
    for (int s = 0; s < SS; ++s)
#pragma unroll
      for (int l = 0; l < (LO ? 2 : 1); ++l)
#pragma unroll
        for (int i = 0; i < TB; ++i) o[i] = M::mma(l ? Sl[s] : Sh[s], f[i][s], o[i]);
#pragma unroll
    for (int i = 0; i < TB; ++i) o[i] *= scale * reinterpret_cast<const float*>(gp)[M::row(t0 + i, m)];
#pragma unroll
    for (int s = 0; s < CS; ++s) {
      u32x4 ph[TB], pl[TB];
#pragma unroll
      for (int i = 0; i < TB; ++i)
        if (s < M::steps(t0 + i)) {
          ph[i] = R::frag(pd, pf, t0 + i, s);
          if (M::kSplit) pl[i] = R::frag(pd + R::kPart, pf + R::kPart, t0 + i, s);
        }
#pragma unroll
      for (int l = 0; l < (M::kSplit ? 3 : 1); ++l)
#pragma unroll
        for (int i = 0; i < TB; ++i)
          if (s < M::steps(t0 + i)) o[i] = M::mma(l == 1 ? El[s] : Eh[s], l == 2 ? pl[i] : ph[i], o[i]);
    }
#pragma unroll
    for (int i = 0; i < TB; ++i) {
      const int r = M::row(t0 + i, m);
      if (r < len && in) store4(out + (int64_t)r * pitch, o[i][0], o[i][1], o[i][2], o[i][3]);
    }
  }
}

// A workgroup walks one sequence of one value head with NW state waves, each
// keeping 16 columns of the state (dv), which need nothing of the others.
// Waves 0 and 1 bring each chunk's K, T, gates and the group's columns of V to
// LDS by DMA while the chunk before is worked on (two stages; the widest heads
// have room for one only).  One wave takes longer to issue all of a chunk's
// loads: 1.77 instead of 1.69 ms for 64K tokens of 32 heads; the backward's
// walks, whose workgroups fill the chip, are better off with one (233 instead
// of 247 us for 4 x 4K of 16).
// A state wave's chunk is a chain of dependent products (K S, T R, K^T E) with
// the splitting of operands between them: 82 MFMAs and about 250 vector
// instructions, 1.33 us with every load taken out; that bounds the walk.  One
// barrier a chunk.  By OUT:
//   kHelped  as many helper waves, one chunk behind, make O from the state and
//            the errors that the state waves left in LDS, their Q and P coming
//            with the DMA too where there is room, else straight from memory:
//            the shortest chain, for walks that do not fill the chip
//   kOwn     the state waves make O themselves: four of them to a workgroup,
//            one a SIMD, for walks that do
//   kKeep    (the backward's recompute) no O: the states before each chunk and
//            the errors go to memory
enum { kKeep = 0, kHelped = 1, kOwn = 2 };
template <typename T, int DK, int NW, int STAGES, int OUT, bool QLDS> struct Walk {
  static constexpr int SS = DK / Mat<T>::KB;
  static constexpr int kK = 0, kRec = Panels<T>::bytes(DK), kV = kRec + ChunkRec<T>::kLoadT * 1024;
  static constexpr int kStage = kV + Columns<T, NW>::kBytes;
  // the helpers' stages: gates and P, then Q
  static constexpr int kG = STAGES * kStage, kQ = ChunkRec<T>::kLoadP * 1024;
  static constexpr int kStageQ = OUT != kKeep && QLDS ? kQ + Panels<T>::bytes(DK) : 0;
  static constexpr int kSwap = kG + STAGES * kStageQ;      // a state wave's state operands and errors (fp32), twice
  // whether O takes the state as a pair: for all but the bf16 heads past 128, for which LDS has no room
  static constexpr bool kLo = Mat<T>::kSplit && DK <= 128;
  static constexpr int kSwapE = SS * (kLo ? 2048 : 1024), kSwapBytes = kSwapE + 4096;
  static constexpr int kSmem = kSwap + (OUT == kHelped ? 2 * NW * kSwapBytes : 0);
  static constexpr int kThreads = 64 * (2 + NW * (OUT == kHelped ? 2 : 1));   // kKeep: with one DMA wave, 64 fewer
  static constexpr int kLag = OUT == kHelped ? 1 : 0;      // turns that O is behind
  // Blocks of 16 tokens that O's sums go by at a time, so that they (and loads of Q from memory) do not wait for each
  // other.  1, 2, 4 blocks: helped, bf16 128 x 128, 64K tokens of 32 heads 1.70, 1.73, 1.68 ms; own, 64 x 64, 8 x 2K
  // 74, 71, 73 us; Q from memory, 4096 tokens of 8 fp32 heads of 256 x 512 2.02, 1.84, 1.73 ms; of 16 of 128 526, 439,
  // 488 us.
  static constexpr int kTB = QLDS ? (!Mat<T>::kSplit ? 1 : OUT == kHelped ? 4 : 2) : DK > 128 ? 4 : 2;
  static constexpr bool kHoist = SS <= 4;                  // whether a chunk's operands fit in registers
  static constexpr bool kLateK = OUT == kOwn && kLo;       // K^T's only behind O, which needs the state's low parts
};

template <typename T, int DK, int NW, int STAGES, int OUT, bool QLDS>
__device__ __forceinline__ void walk_loads(const DeltaArgs& p, int parts, const char* rec, const WalkPlace& at,
                                           const SeqPlace& sp) {
  extern __shared__ __attribute__((aligned(16))) char smem[];
  using G = Walk<T, DK, NW, STAGES, OUT, QLDS>;
  const int first = at.part * NW * 16, kh = at.h / (p.Hv / p.Hk), chunks = (sp.len + kDC - 1) / kDC;
  const unsigned kp = p.sk.t * sizeof(T), qp = p.sq.t * sizeof(T), vp = p.sv.t * sizeof(T), row = p.dk * sizeof(T);
  const T* k0 = (const T*)p.k + sp.b * p.sk.b + kh * p.sk.h + sp.tok0 * p.sk.t;
  const T* q0 = (const T*)p.q + sp.b * p.sq.b + kh * p.sq.h + sp.tok0 * p.sq.t;
  const T* v0 = (const T*)p.v + sp.b * p.sv.b + at.h * p.sv.h + sp.tok0 * p.sv.t + first;
  const char* rec0 = rec + ((int64_t)sp.slot0 * p.Hv + at.h) * ChunkRec<T>::kBytes;
  const int64_t rstep = (int64_t)p.Hv * ChunkRec<T>::kBytes;
  const PanelLoader<T, DK, 1> kload(kp, row), qload(qp, row);
  const Columns<T, NW> vload(vp, p.dv - first);
  // turn c: the state waves at chunk c, O at chunk c - kLag
  auto issue = [&](int c) __attribute__((always_inline)) {
    const int d = c - G::kLag, len = min(kDC, sp.len - c * kDC);
    char* st = smem + c % STAGES * G::kStage;
    char* sq = smem + G::kG + d % STAGES * G::kStageQ;
    const bool out = OUT != kKeep && QLDS && d >= 0;
    if (parts & 1) {
      if (c < chunks) {
        kload.issue(k0 + (int64_t)c * kDC * p.sk.t, len, st + G::kK);
      }
      if (out)
        load_block<G::kQ / 1024>(rec0 + d * rstep + ChunkRec<T>::kGate, sq, ChunkRec<T>::kBytes - ChunkRec<T>::kGate);
    }
    if (parts & 2) {
      if (c < chunks) {
        load_block<ChunkRec<T>::kLoadT>(rec0 + c * rstep, st + G::kRec);
        vload.issue(v0 + (int64_t)c * kDC * p.sv.t, len, st + G::kV);
      }
      if (out) qload.issue(q0 + (int64_t)d * kDC * p.sq.t, min(kDC, sp.len - d * kDC), sq + G::kQ);
    }
  };
  dma_wave<STAGES>(chunks > 0 ? chunks + G::kLag : 0, issue);
}

template <typename T, int DK, int NW, int STAGES, int OUT, bool QLDS>
__device__ __forceinline__ void walk_states(const DeltaArgs& p, int w, void* states, void* errors, const WalkPlace& at,
                                            const SeqPlace& sp) {
  extern __shared__ __attribute__((aligned(16))) char smem[];
  using M = Mat<T>;
  using G = Walk<T, DK, NW, STAGES, OUT, QLDS>;
  constexpr int ST = DK / 16, SS = G::SS, CS = kDC / M::KB;   // state blocks, steps over dk, steps over the tokens
  const int lane = lane_id(), m = lane & 15, g = lane >> 4, h = at.h, seq = at.seq;
  const int col = (at.part * NW + w) * 16 + m, chunks = (sp.len + kDC - 1) / kDC;
  // state block t, register r: dk = row(t, 4 g + r), dv = col
  f32x4 S[ST];
  const int64_t wbase = (((int64_t)seq * p.Hv + h) * p.dv + col) * p.dk;
  // A sequence that begins with a reset takes nothing from W_init, whatever values it holds.
  const bool resumed =
      p.W_init && !(sp.len > 0 && p.g[sp.b * p.sg.b + h * p.sg.h + sp.tok0 * p.sg.t] < kResetDecay);
#pragma unroll
  for (int t = 0; t < ST; ++t) {
    const int d = M::row(t, g * 4);
    S[t] = (f32x4){0.f, 0.f, 0.f, 0.f};
    if (resumed && d < p.dk && col < p.dv) S[t] = *reinterpret_cast<const f32x4*>(p.W_init + wbase + d);
  }

  const int diag = ChunkRec<T>::diag_kept(lane);
  for (int c = 0; c < chunks; ++c) {
    const char* st = smem + c % STAGES * G::kStage;
    next_turn<STAGES>(c == 0);
    const float* gate = reinterpret_cast<const float*>(st + G::kRec + ChunkRec<T>::kGate);
    [[maybe_unused]] char* swap = smem + G::kSwap + ((c & 1) * NW + w) * G::kSwapBytes + lane * 16;
    const int64_t slot = (int64_t)(sp.slot0 + c) * p.Hv + h;

    // Reads from LDS go out ahead of the arithmetic that hides them: one wave a SIMD has nobody else to do it.
    u32x4 Kf[G::kHoist ? 4 : 1][SS], Th[M::kTri], Tl[M::kSplit ? M::kTri : 1];
    typename Columns<T, NW>::Raw v[4];
    f32x4 up[4], left[4];
    auto read_k = [&](int t, u32x4 (&f)[SS]) __attribute__((always_inline)) {
      const int r = M::row(t, m);
#pragma unroll
      for (int s = 0; s < SS; ++s) f[s] = Panels<T>::frag(st + G::kK, r, s, g);
    };
    if constexpr (G::kHoist)
#pragma unroll
      for (int t = 0; t < 4; ++t) read_k(t, Kf[t]);
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      v[t] = Columns<T, NW>::read(st + G::kV, w, t, lane);
      up[t] = *reinterpret_cast<const f32x4*>(gate + M::row(t, g * 4));
      left[t] = *reinterpret_cast<const f32x4*>(gate + 64 + M::row(t, g * 4));
    }
    const float decay = gate[63];
    __builtin_amdgcn_sched_barrier(0);
    u32x4 Sh[SS], Sl[SS];
#pragma unroll
    for (int s = 0; s < SS; ++s) M::split(S + s * M::TPS, Sh[s], Sl[s]);
    if constexpr (OUT == kKeep) {
      put_state<T, SS>(Sh, (T*)states + (slot * p.dv + col) * p.dk, p.dk, col < p.dv);
    }
    // V - exp(b) K S
    f32x4 e[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) e[t] = (f32x4){0.f, 0.f, 0.f, 0.f};
    if constexpr (G::kHoist) {
#pragma unroll
      for (int s = 0; s < SS; ++s)
#pragma unroll
        for (int i = 0; i < (M::kSplit ? 2 : 1); ++i)
#pragma unroll
          for (int t = 0; t < 4; ++t) e[t] = M::mma(Kf[t][s], i ? Sl[s] : Sh[s], e[t]);
    } else {
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        read_k(t, Kf[0]);
#pragma unroll
        for (int s = 0; s < SS; ++s) e[t] = mma_split<T>(Kf[0][s], Sh[s], Sl[s], e[t]);
      }
    }
    // Behind K's reads, under the products: before them 16K tokens of 32 heads take 449 us instead of 432.
    if constexpr (OUT == kHelped) {
#pragma unroll
      for (int s = 0; s < SS; ++s) {
        *reinterpret_cast<u32x4*>(swap + s * 1024) = Sh[s];
        if (G::kLo) *reinterpret_cast<u32x4*>(swap + (SS + s) * 1024) = Sl[s];
      }
    }
    const char *td = st + G::kRec + diag, *tf = st + G::kRec + lane * 16;
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int s = 0; s < M::steps(t); ++s) {
        Th[M::tri(t, s)] = ChunkRec<T>::frag(td, tf, t, s);
        if (M::kSplit) Tl[M::tri(t, s)] = ChunkRec<T>::frag(td + ChunkRec<T>::kTl, tf + ChunkRec<T>::kTl, t, s);
      }
    u32x4 Kt[G::kHoist ? ST : 1][CS];
    if constexpr (G::kHoist && !G::kLateK)
#pragma unroll
      for (int t = 0; t < ST; ++t)
#pragma unroll
        for (int s = 0; s < CS; ++s) Kt[t][s] = Panels<T>::frag_t(st + G::kK, t, s, lane);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int t = 0; t < ST; ++t) S[t] *= decay;
#pragma unroll
    for (int t = 0; t < 4; ++t) e[t] = Columns<T, NW>::wide(v[t]) - up[t] * e[t];
    u32x4 Rh[CS], Rl[CS];
#pragma unroll
    for (int s = 0; s < CS; ++s) M::split(e + s * M::TPS, Rh[s], Rl[s]);
    // E = T (V - exp(b) K S)
#pragma unroll
    for (int t = 0; t < 4; ++t) e[t] = (f32x4){0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s = 0; s < CS; ++s)
#pragma unroll
      for (int i = 0; i < (M::kSplit ? 3 : 1); ++i)
#pragma unroll
        for (int t = 0; t < 4; ++t)
          if (s < M::steps(t)) {
            const int f = M::tri(t, s);
            e[t] = M::mma(i == 2 ? Tl[M::kSplit ? f : 0] : Th[f], i == 1 ? Rl[s] : Rh[s], e[t]);
          }
    if constexpr (OUT == kHelped) {
#pragma unroll
      for (int t = 0; t < 4; ++t) *reinterpret_cast<f32x4*>(swap + G::kSwapE + t * 1024) = e[t];
    } else if constexpr (OUT == kOwn) {
      const char* sq = smem + G::kG + c % STAGES * G::kStageQ;
      const int len = min(kDC, sp.len - c * kDC), col0 = (at.part * NW + w) * 16 + g * 4;
      T* o = (T*)p.O + sp.b * p.so.b + h * p.so.h + (int64_t)(sp.tok0 + c * kDC) * p.so.t + col0;
      make_outputs<T, SS, G::kLo, G::kTB>(Sh, Sl, e, sq, diag, sq + G::kQ, p.scale, len, col0 < p.dv, p.so.t, o);
    } else {
      T* E = (T*)errors + (slot * p.dv + col) * kDC + g * (16 / (int)sizeof(T));
#pragma unroll
      for (int s = 0; s < CS; ++s)
        if (col < p.dv) *reinterpret_cast<u32x4*>(E + s * M::KB) = M::frag(e + s * M::TPS);
    }
    if constexpr (G::kHoist && G::kLateK) {
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int t = 0; t < ST; ++t)
#pragma unroll
        for (int s = 0; s < CS; ++s) Kt[t][s] = Panels<T>::frag_t(st + G::kK, t, s, lane);
    }
    // S = exp(b_63) S + K^T (exp(b_63 - b) beta E)
#pragma unroll
    for (int t = 0; t < 4; ++t) e[t] *= left[t];
#pragma unroll
    for (int s = 0; s < CS; ++s) M::split(e + s * M::TPS, Rh[s], Rl[s]);
#pragma unroll
    for (int s = 0; s < CS; ++s)
#pragma unroll
      for (int t = 0; t < ST; ++t) {
        const u32x4 f = G::kHoist ? Kt[G::kHoist ? t : 0][s] : Panels<T>::frag_t(st + G::kK, t, s, lane);
        S[t] = M::mma(f, Rh[s], S[t]);
        if (M::kSplit) S[t] = M::mma(f, Rl[s], S[t]);
      }
  }
  if (OUT == kHelped && chunks > 0) next_turn<STAGES>(false);   // the helpers' last one
  if (p.W_final) {
#pragma unroll
    for (int t = 0; t < ST; ++t) {
      const int d = M::row(t, g * 4);
      if (d < p.dk && col < p.dv) *reinterpret_cast<f32x4*>(p.W_final + wbase + d) = S[t];
    }
  }
}

// The helpers' side: O of chunk c while the state waves are at chunk c + 1.
template <typename T, int DK, int NW, int STAGES, bool QLDS>
__device__ __forceinline__ void walk_outputs(const DeltaArgs& p, const char* rec, int w, const WalkPlace& at,
                                             const SeqPlace& sp) {
  extern __shared__ __attribute__((aligned(16))) char smem[];
  using G = Walk<T, DK, NW, STAGES, kHelped, QLDS>;
  constexpr int SS = G::SS;
  const int lane = lane_id(), g = lane >> 4, h = at.h;
  const int col0 = (at.part * NW + w) * 16 + g * 4;
  const int kh = h / (p.Hv / p.Hk), chunks = (sp.len + kDC - 1) / kDC;
  const unsigned qp = p.sq.t * sizeof(T), qrow = p.dk * sizeof(T);
  const T* q0 = (const T*)p.q + sp.b * p.sq.b + kh * p.sq.h + sp.tok0 * p.sq.t;
  T* o0 = (T*)p.O + sp.b * p.so.b + h * p.so.h + sp.tok0 * p.so.t + col0;
  const char* rec0 = rec + ((int64_t)sp.slot0 * p.Hv + h) * ChunkRec<T>::kBytes + ChunkRec<T>::kGate;
  const int64_t rstep = (int64_t)p.Hv * ChunkRec<T>::kBytes;
  const int diag = ChunkRec<T>::diag_kept(lane);
  if (chunks > 0) next_turn<STAGES>(true);
  for (int c = 0; c < chunks; ++c) {
    next_turn<STAGES>(false);
    const int len = min(kDC, sp.len - c * kDC);
    const char* swap = smem + G::kSwap + ((c & 1) * NW + w) * G::kSwapBytes + lane * 16;
    const char* st = smem + G::kG + c % STAGES * G::kStageQ;
    const char* gp = QLDS ? st : rec0 + c * rstep;           // gates, P
    u32x4 Sh[SS], Sl[SS];
#pragma unroll
    for (int s = 0; s < SS; ++s) {
      Sh[s] = *reinterpret_cast<const u32x4*>(swap + s * 1024);
      if (G::kLo) Sl[s] = *reinterpret_cast<const u32x4*>(swap + (SS + s) * 1024);
    }
    f32x4 e[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) e[t] = *reinterpret_cast<const f32x4*>(swap + G::kSwapE + t * 1024);
    make_outputs<T, SS, G::kLo, G::kTB, QLDS>(Sh, Sl, e, gp, diag, st + G::kQ, p.scale, len, col0 < p.dv, p.so.t,
                                              o0 + (int64_t)c * kDC * p.so.t, q0 + (int64_t)c * kDC * p.sq.t, qp, qrow);
  }
}

}  // namespace
}  // namespace ttt
