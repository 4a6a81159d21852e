// The backward pass of the gated delta rule (gfx950).  Notation of delta.hpp;
// dS' is the gradient of the state after a chunk.
//
// Within a chunk, with bE = beta E the step each token takes,
//   dbE = P0^T dO + exp(b_63 - b) K dS'             (P = P0 diag(beta))
//   X   = T^T (beta dbE)                            = dV, the residual's gradient
//   dS  = exp(b_63) dS' + Q^T (scale exp(b) dO) - K^T (exp(b) X)
// so a reverse walk over the chunks needs T^T, P^T and the gates alone, as the
// forward one does, and the two walks do not need each other: one launch runs
// both (the forward one to remake the states S before each chunk and the
// errors E).  They leave S, dS', E and X in memory, and the rest is local to a
// chunk (k_delta_grads):
//   Mq_ij = scale D_ij beta_j (dO_i . E_j)   j <= i,  D_ij = exp(b_i - b_j)
//   Mk_ij =      -D_ij beta_j (X_i . E_j)    j <  i
//   dQ = scale exp(b) dO S^T + Mq K
//   dK = Mq^T Q + (Mk + Mk^T) K - exp(b) X S^T + exp(b_63 - b) beta E dS'^T
//   dbeta_j = (sum_i Mq_ij q_i.k_j + Mk_ij k_i.k_j) / beta_j + exp(b_63 - b_j) k_j.(dS'^T E_j)
//   dg_t = sum_{j < t <= i} N_ij + sum_{i >= t} exp(b_i) (scale q_i.(S dO_i) - k_i.(S X_i))
//          + sum_{j < t} exp(b_63 - b_j) beta_j k_j.(dS'^T E_j) + exp(b_63) <S, dS'>,
//   N_ij = Mq_ij q_i.k_j + Mk_ij k_i.k_j   (j < i)
// (the division is by a factor of the summands, which are taken without it).
// Every term of dg_t has exp(g_t) in its decay: the sums are made so that no
// other terms come in that would have to cancel, and a strong decay's small
// gradient keeps its digits.
// Gradients of a key head sum over its value heads, one after the other in one
// workgroup: no atomics.
//
// Rounding (bf16).  The walks' states are fp32 with operands in pairs, as in
// the forward pass, so dW_init keeps fp32's digits; what they leave in memory
// is bf16, each value rounded once, and so are Mq and Mk: they feed only
// gradients that are bf16 themselves, or sums.  Off by, of a gradient's norm: dv
// 1.7e-3, which is its own rounding; dq and dk 2.7e-3 to 3.2e-3; dg and dbeta
// 2e-3 to 4e-3 over a hundred tokens or more, but up to 6e-3 and 1.3e-2 over a
// sequence of a few, where a gate's gradient is a handful of dots of those
// roundings that cancel in part.  Of dq's and dk's error that of E and that of
// Mq and Mk are the larger parts, of dg's that of S and dS' under weak decays;
// X's matters little.  Pairs in memory would write and read twice the 400 MB that
// S, dS', E and X are at the size below, 160 us at a copy's rate.
//
// Workspace (delta_grad_workspace_bytes): 140 KB a chunk and value head of 128 x
// 128 in bf16: 44 KB of records, 64 of S and dS', 32 of E and X.
//
// 4 x 4096 tokens, 16 value heads of 128: walks 235 us, chunk-local gradients
// 219 us (56 KB of operands a head and dv block; bound by those and by LDS).
// 16384 tokens, 8 value heads of 256 x 512, bf16: walks 1.93 ms, gradients 0.56.
#include "delta_walk.hpp"

namespace ttt {
namespace {

// ------------------------------------------------------------------ the reverse walk

template <typename T, int DK, int NW, int STAGES> struct WalkBack {
  static constexpr int SS = DK / Mat<T>::KB;
  static constexpr int kK = 0, kQ = Panels<T>::bytes(DK), kRec = 2 * kQ, kD = kRec + ChunkRecT<T>::kBytes;
  static constexpr int kStage = kD + Columns<T, NW>::kBytes;
  static constexpr int kSmem = STAGES * kStage;
  static constexpr bool kHoist = SS <= 4;
};

template <typename T, int DK, int NW, int STAGES>
__device__ __forceinline__ void walk_back_loads(const DeltaGradArgs& a, const WalkPlace& at, const SeqPlace& sp) {
  extern __shared__ __attribute__((aligned(16))) char smem[];
  using G = WalkBack<T, DK, NW, STAGES>;
  const DeltaArgs& p = a.f;
  const int first = at.part * NW * 16, kh = at.h / (p.Hv / p.Hk), chunks = (sp.len + kDC - 1) / kDC;
  const unsigned kp = p.sk.t * sizeof(T), qp = p.sq.t * sizeof(T), dp = a.sdo.t * sizeof(T), row = p.dk * sizeof(T);
  const T* k0 = (const T*)p.k + sp.b * p.sk.b + kh * p.sk.h + sp.tok0 * p.sk.t;
  const T* q0 = (const T*)p.q + sp.b * p.sq.b + kh * p.sq.h + sp.tok0 * p.sq.t;
  const T* d0 = (const T*)a.dO + sp.b * a.sdo.b + at.h * a.sdo.h + sp.tok0 * a.sdo.t + first;
  const char* rec0 = a.rect + ((int64_t)sp.slot0 * p.Hv + at.h) * ChunkRecT<T>::kBytes;
  const int64_t rstep = (int64_t)p.Hv * ChunkRecT<T>::kBytes;
  const PanelLoader<T, DK, 1> kload(kp, row), qload(qp, row);
  const Columns<T, NW> dload(dp, p.dv - first);
  auto issue = [&](int turn) __attribute__((always_inline)) {
    const int c = chunks - 1 - turn, len = min(kDC, sp.len - c * kDC);
    char* st = smem + turn % STAGES * G::kStage;
    kload.issue(k0 + (int64_t)c * kDC * p.sk.t, len, st + G::kK);
    qload.issue(q0 + (int64_t)c * kDC * p.sq.t, len, st + G::kQ);
    load_block<ChunkRecT<T>::kBytes / 1024>(rec0 + c * rstep, st + G::kRec);
    dload.issue(d0 + (int64_t)c * kDC * a.sdo.t, len, st + G::kD);
  };
  dma_wave<STAGES>(chunks, issue);
}

template <typename T, int DK, int NW, int STAGES>
__device__ __forceinline__ void walk_back(const DeltaGradArgs& a, int w, const WalkPlace& at, const SeqPlace& sp) {
  extern __shared__ __attribute__((aligned(16))) char smem[];
  using M = Mat<T>;
  using G = WalkBack<T, DK, NW, STAGES>;
  const DeltaArgs& p = a.f;
  constexpr int ST = DK / 16, SS = G::SS, CS = kDC / M::KB;
  const int lane = lane_id(), m = lane & 15, g = lane >> 4, h = at.h, seq = at.seq;
  const int col = (at.part * NW + w) * 16 + m, chunks = (sp.len + kDC - 1) / kDC;
  void *dstates = a.dstates, *xs = a.xs;
  f32x4 S[ST];                    // dS': block t, register r: dk = row(t, 4 g + r), dv = col
  const int64_t wbase = (((int64_t)seq * p.Hv + h) * p.dv + col) * p.dk;
#pragma unroll
  for (int t = 0; t < ST; ++t) {
    const int d = M::row(t, g * 4);
    S[t] = (f32x4){0.f, 0.f, 0.f, 0.f};
    if (a.dW_final && d < p.dk && col < p.dv) S[t] = *reinterpret_cast<const f32x4*>(a.dW_final + wbase + d);
  }

  for (int c = chunks - 1; c >= 0; --c) {
    const char* st = smem + (chunks - 1 - c) % STAGES * G::kStage;
    next_turn<STAGES>(c == chunks - 1);
    const float* gate = reinterpret_cast<const float*>(st + G::kRec + ChunkRecT<T>::kGate);
    const int64_t slot = (int64_t)(sp.slot0 + c) * p.Hv + h;
    // As in the forward walk, reads from LDS go out a stage of arithmetic ahead.
    u32x4 Kf[G::kHoist ? 4 : 1][SS];
    typename Columns<T, NW>::Raw raw[4];
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
      raw[t] = Columns<T, NW>::read(st + G::kD, w, t, lane);
      up[t] = *reinterpret_cast<const f32x4*>(gate + M::row(t, g * 4));
      left[t] = *reinterpret_cast<const f32x4*>(gate + 64 + M::row(t, g * 4));
    }
    const float decay = gate[63];
    __builtin_amdgcn_sched_barrier(0);
    u32x4 Sh[SS], Sl[SS];
#pragma unroll
    for (int s = 0; s < SS; ++s) M::split(S + s * M::TPS, Sh[s], Sl[s]);
    put_state<T, SS>(Sh, (T*)dstates + (slot * p.dv + col) * p.dk, p.dk, col < p.dv);
    // beta dbE = beta exp(b_63 - b) K dS' + P^T dO
    f32x4 x[4], d[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) x[t] = (f32x4){0.f, 0.f, 0.f, 0.f};
    if constexpr (G::kHoist) {
#pragma unroll
      for (int s = 0; s < SS; ++s)
#pragma unroll
        for (int i = 0; i < (M::kSplit ? 2 : 1); ++i)
#pragma unroll
          for (int t = 0; t < 4; ++t) x[t] = M::mma(Kf[t][s], i ? Sl[s] : Sh[s], x[t]);
    } else {
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        read_k(t, Kf[0]);
#pragma unroll
        for (int s = 0; s < SS; ++s) x[t] = mma_split<T>(Kf[0][s], Sh[s], Sl[s], x[t]);
      }
    }
    const char* rl = st + G::kRec + lane * 16;
    u32x4 Ph[M::kTri], Pl[M::kSplit ? M::kTri : 1], Qt[G::kHoist ? ST : 1][CS];
#pragma unroll
    for (int f = 0; f < M::kTri; ++f) {
      Ph[f] = *reinterpret_cast<const u32x4*>(rl + ChunkRecT<T>::kP + f * 1024);
      if (M::kSplit) Pl[f] = *reinterpret_cast<const u32x4*>(rl + ChunkRecT<T>::kPl + f * 1024);
    }
    if constexpr (G::kHoist)
#pragma unroll
      for (int t = 0; t < ST; ++t)
#pragma unroll
        for (int s = 0; s < CS; ++s) Qt[t][s] = Panels<T>::frag_t(st + G::kQ, t, s, lane);
    __builtin_amdgcn_sched_barrier(0);
    u32x4 D[CS], Dh[CS], Dl[CS];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      d[t] = Columns<T, NW>::wide(raw[t]);
      x[t] *= left[t];
    }
#pragma unroll
    for (int s = 0; s < CS; ++s) D[s] = M::frag(d + s * M::TPS);       // exact: dO is of type T
#pragma unroll
    for (int s = 0; s < CS; ++s)
#pragma unroll
      for (int i = 0; i < (M::kSplit ? 2 : 1); ++i)
#pragma unroll
        for (int t = 0; t < 4; ++t)
          if (s >= M::first(t)) x[t] = M::mma(i ? Pl[M::kSplit ? M::triu(t, s) : 0] : Ph[M::triu(t, s)], D[s], x[t]);
    // dS = exp(b_63) dS' + Q^T (scale exp(b) dO) - K^T (exp(b) X): the second term has nothing to wait for
#pragma unroll
    for (int t = 0; t < 4; ++t) d[t] *= p.scale * up[t];
#pragma unroll
    for (int s = 0; s < CS; ++s) M::split(d + s * M::TPS, Dh[s], Dl[s]);
#pragma unroll
    for (int t = 0; t < ST; ++t) S[t] *= decay;
#pragma unroll
    for (int s = 0; s < CS; ++s)
#pragma unroll
      for (int t = 0; t < ST; ++t) {
        const u32x4 f = G::kHoist ? Qt[G::kHoist ? t : 0][s] : Panels<T>::frag_t(st + G::kQ, t, s, lane);
        S[t] = M::mma(f, Dh[s], S[t]);
        if (M::kSplit) S[t] = M::mma(f, Dl[s], S[t]);
      }
    u32x4 Th[M::kTri], Tl[M::kSplit ? M::kTri : 1], Kt[G::kHoist ? ST : 1][CS];
#pragma unroll
    for (int f = 0; f < M::kTri; ++f) {
      Th[f] = *reinterpret_cast<const u32x4*>(rl + f * 1024);
      if (M::kSplit) Tl[f] = *reinterpret_cast<const u32x4*>(rl + ChunkRecT<T>::kTl + f * 1024);
    }
    if constexpr (G::kHoist)
#pragma unroll
      for (int t = 0; t < ST; ++t)
#pragma unroll
        for (int s = 0; s < CS; ++s) Kt[t][s] = Panels<T>::frag_t(st + G::kK, t, s, lane);
    __builtin_amdgcn_sched_barrier(0);
    u32x4 Rh[CS], Rl[CS];
#pragma unroll
    for (int s = 0; s < CS; ++s) M::split(x + s * M::TPS, Rh[s], Rl[s]);
    // X = T^T (beta dbE)
#pragma unroll
    for (int t = 0; t < 4; ++t) x[t] = (f32x4){0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s = 0; s < CS; ++s)
#pragma unroll
      for (int i = 0; i < (M::kSplit ? 3 : 1); ++i)
#pragma unroll
        for (int t = 0; t < 4; ++t)
          if (s >= M::first(t)) {
            const int f = M::triu(t, s);
            x[t] = M::mma(i == 2 ? Tl[M::kSplit ? f : 0] : Th[f], i == 1 ? Rl[s] : Rh[s], x[t]);
          }
    T* xo = (T*)xs + (slot * p.dv + col) * kDC + g * (16 / (int)sizeof(T));
#pragma unroll
    for (int s = 0; s < CS; ++s)
      if (col < p.dv) *reinterpret_cast<u32x4*>(xo + s * M::KB) = M::frag(x + s * M::TPS);
#pragma unroll
    for (int t = 0; t < 4; ++t) x[t] *= -up[t];
#pragma unroll
    for (int s = 0; s < CS; ++s) M::split(x + s * M::TPS, Rh[s], Rl[s]);
#pragma unroll
    for (int s = 0; s < CS; ++s)
#pragma unroll
      for (int t = 0; t < ST; ++t) {
        const u32x4 f = G::kHoist ? Kt[G::kHoist ? t : 0][s] : Panels<T>::frag_t(st + G::kK, t, s, lane);
        S[t] = M::mma(f, Rh[s], S[t]);
        if (M::kSplit) S[t] = M::mma(f, Rl[s], S[t]);
      }
  }
  if (a.dW_init) {
#pragma unroll
    for (int t = 0; t < ST; ++t) {
      const int d = M::row(t, g * 4);
      if (d < p.dk && col < p.dv) *reinterpret_cast<f32x4*>(a.dW_init + wbase + d) = S[t];
    }
  }
}

// Both walks: the first half of the workgroups goes forward, the second back.
template <typename T, int DK, int NW, int SF, int SB>
__global__ __launch_bounds__(64 * (1 + NW)) void k_delta_walks(DeltaGradArgs a, int sequences) {
  const DeltaArgs& p = a.f;
  const int half = gridDim.x / 2;
  const bool back = (int)blockIdx.x >= half;
  WalkPlace at;
  if (!walk_place(back ? blockIdx.x - half : blockIdx.x, sequences, p.Hk, p.Hv / p.Hk,
                  (p.dv + 16 * NW - 1) / (16 * NW), &at))
    return;
  const SeqPlace sp = seq_place(p.seqs, at.seq);
  const int w = wave_id();
  if (back) {
    if (w == 0)
      walk_back_loads<T, DK, NW, SB>(a, at, sp);
    else
      walk_back<T, DK, NW, SB>(a, w - 1, at, sp);
  } else if (w == 0) {
    walk_loads<T, DK, NW, SF, kKeep, false>(p, 3, a.rec, at, sp);
  } else {
    walk_states<T, DK, NW, SF, kKeep, false>(p, w - 1, a.states, a.errors, at, sp);
  }
}

// ------------------------------------------------------------------ what is local to a chunk

// One workgroup of 8 waves per chunk slot and key head; waves w and w + 4 make
// the rows of tokens row(w, .), each half of the features.  Every product has the tokens as the instruction's
// columns and the features (dk, or the other token) as its rows, so that a
// lane holds 4 consecutive features of one token.  dv goes by in blocks of 128
// bytes: the block's rows of S and dS' ([dv, dk]) and of E and X ([dv, 64])
// and the block of dO come to LDS; what is contracted over dv in them is read
// transposed.
template <typename T, int DK> struct Grads {
  static constexpr int BV = 128 / (int)sizeof(T);            // columns of a dv block
  using Rows = Panels<T, BV>;                                // its rows of S, dS', E, X
  static constexpr int kS = 0, kDS = Rows::bytes(DK), kE = 2 * kDS, kX = kE + Rows::bytes(kDC), kD = kX + Rows::bytes(kDC);
  static constexpr int kBlock = kD + Panels<T>::bytes(BV), kQK = 2 * Panels<T>::bytes(DK);
  // Where LDS has room Q and K have a place of their own, and where it has more, a block comes while the one before
  // is worked on; the widest fp32 heads load Q and K in the place of S and dS' after a head's last block.
  static constexpr int kLds = 160 * 1024 - 6144;             // but for the arrays of single values
  static constexpr bool kOwnQ = kBlock + kQK <= kLds, kTwo = 2 * kBlock + kQK <= kLds;
  static constexpr int kQ = kOwnQ ? (kTwo ? 2 : 1) * kBlock : 0, kK = kQ + kQK / 2;
  static constexpr int kSmem = kOwnQ ? kQ + kQK : (kBlock > kQK + kBlock - kE ? kBlock : kQK + kBlock - kE);
  static constexpr int kShift = kOwnQ ? 0 : (kQK > kE ? kQK - kE : 0);   // E, X and dO lie behind Q and K then
  // Mq and Mk take the place of E, X and dO: both at once, where there is room
  static constexpr int kM = kE + kShift, kMBytes = Panels<T>::bytes(kDC);
  static constexpr bool kBoth = kBlock - kE >= 2 * kMBytes;
};

// x of the lane groups in front of group g (lanes of equal lane & 15), summed.
__device__ __forceinline__ float groups_before(float x, int g) {
  float up = __shfl_up(x, 16, 64);
  if (g >= 1) x += up;
  up = __shfl_up(x, 32, 64);
  if (g >= 2) x += up;
  up = __shfl_up(x, 16, 64);
  return g >= 1 ? up : 0.f;
}

template <typename T, int DK>
__global__ __launch_bounds__(512) void k_delta_grads(DeltaGradArgs a) {
  using M = Mat<T>;
  using G = Grads<T, DK>;
  using Rows = typename G::Rows;
  constexpr int HT = DK / 32, SS = DK / M::KB, CS = kDC / M::KB, E = 16 / (int)sizeof(T);   // HT: half the blocks of dk
  constexpr int VS = G::BV / M::KB;                          // steps over a dv block: 2
  extern __shared__ __attribute__((aligned(16))) char smem[];
  __shared__ double b[kDC];
  __shared__ float beta[kDC], colsum[2][4][kDC], half[2][4][kDC], part[8];   // colsum: of N_ij / beta_j; dg's
  const DeltaArgs& p = a.f;
  const int id = xcd_remap(blockIdx.x, gridDim.x);
  const int kh = id % p.Hk, slot = id / p.Hk, group = p.Hv / p.Hk;
  const ChunkPlace c = chunk_place(p.seqs, slot);
  if (c.len <= 0) return;
  const int wave = wave_id(), w = wave & 3, hf = wave >> 2, lane = lane_id(), m = lane & 15, g = lane >> 4;
  const int t0 = hf * HT, j0 = hf * 2;                       // first block of dk, of the other tokens
  const int i = M::row(w, m);                                // this lane's token
  const unsigned row = p.dk * sizeof(T);
  const PanelLoader<T, DK, 8, G::BV> sload(row, row);
  const PanelLoader<T, kDC, 8, G::BV> eload(kDC * sizeof(T), kDC * sizeof(T));
  const PanelLoader<T, DK, 8> qload(p.sq.t * sizeof(T), row), kload(p.sk.t * sizeof(T), row);
  const int blocks = (p.dv + G::BV - 1) / G::BV;             // of a head; n counts them over all heads
  auto load_qk = [&]() __attribute__((always_inline)) {
    qload.issue((const T*)p.q + c.b * p.sq.b + kh * p.sq.h + c.tok0 * p.sq.t, c.len, smem + G::kQ);
    kload.issue((const T*)p.k + c.b * p.sk.b + kh * p.sk.h + c.tok0 * p.sk.t, c.len, smem + G::kK);
  };
  auto load_block = [&](int n) __attribute__((always_inline)) {
    char* st = smem + (G::kTwo ? (n & 1) * G::kBlock : 0);
    const int h = kh * group + n / blocks, v0 = n % blocks * G::BV, rows = min(G::BV, p.dv - v0);
    const int64_t sh = (int64_t)slot * p.Hv + h, so = (sh * p.dv + v0) * p.dk, eo = (sh * p.dv + v0) * kDC;
    sload.issue((const T*)a.states + so, rows, st + G::kS);
    sload.issue((const T*)a.dstates + so, rows, st + G::kDS);
    eload.issue((const T*)a.errors + eo, rows, st + G::kE + G::kShift);
    eload.issue((const T*)a.xs + eo, rows, st + G::kX + G::kShift);
    const PanelLoader<T, G::BV, 8> dload(a.sdo.t * sizeof(T), rows * sizeof(T));
    dload.issue((const T*)a.dO + c.b * a.sdo.b + h * a.sdo.h + c.tok0 * a.sdo.t + v0, c.len, st + G::kD + G::kShift);
  };
  if (G::kOwnQ) load_qk();
  if (G::kTwo) load_block(0);
  f32x4 dq[HT], dk[HT];
#pragma unroll
  for (int t = 0; t < HT; ++t) dq[t] = dk[t] = (f32x4){0.f, 0.f, 0.f, 0.f};

  for (int h = kh * group; h < (kh + 1) * group; ++h) {
    const int64_t sh = (int64_t)slot * p.Hv + h;
    __syncthreads();                                         // the head before is done with LDS
    if (wave == 0) {
      const char* gate = a.rect + sh * ChunkRecT<T>::kBytes + ChunkRecT<T>::kGate;
      b[lane] = reinterpret_cast<const double*>(gate + 512)[lane];
      beta[lane] =
          lane < c.len ? p.beta[c.b * p.sbeta.b + h * p.sbeta.h + (c.tok0 + lane) * p.sbeta.t] : 0.f;
    }
    f32x4 os[HT], xs[HT], es[HT];                            // S dO, S X, dS' E by token
#pragma unroll
    for (int t = 0; t < HT; ++t) os[t] = xs[t] = es[t] = (f32x4){0.f, 0.f, 0.f, 0.f};
    f32x4 oe[2], xe[2];                                      // E_j . dO_i, E_j . X_i: j = row(j0 + t, 4 g + r)
#pragma unroll
    for (int t = 0; t < 2; ++t) oe[t] = xe[t] = (f32x4){0.f, 0.f, 0.f, 0.f};
    float ss = 0.f;                                          // <S, dS'>
    for (int v0 = 0; v0 < p.dv; v0 += G::BV) {
      const int rows = min(G::BV, p.dv - v0), n = (h - kh * group) * blocks + v0 / G::BV;
      if (!G::kTwo) {
        if (v0 > 0) __syncthreads();
        load_block(n);
      }
      wait_vm<0>();
      __syncthreads();
      if (G::kTwo && n + 1 < group * blocks) load_block(n + 1);
      const char* st = smem + (G::kTwo ? (n & 1) * G::kBlock : 0);
      u32x4 fo[VS], fx[VS], fe[VS];                          // this lane's token, contraction over the block
#pragma unroll
      for (int s = 0; s < VS; ++s) {
        fo[s] = Panels<T>::frag(st + G::kD + G::kShift, i, s, g);
        fx[s] = Rows::frag_t(st + G::kX + G::kShift, w, s, lane);
        fe[s] = Rows::frag_t(st + G::kE + G::kShift, w, s, lane);
      }
      // dV = X
      if (i < c.len) {
        T* o = (T*)a.dv + c.b * a.sdv.b + h * a.sdv.h + (int64_t)(c.tok0 + i) * a.sdv.t + v0 + g * E;
#pragma unroll
        for (int s = 0; s < VS; ++s)
          if (s == hf && s * M::KB + g * E < rows) *reinterpret_cast<u32x4*>(o + s * M::KB) = fx[s];
      }
#pragma unroll
      for (int t = 0; t < HT; ++t)
#pragma unroll
        for (int s = 0; s < VS; ++s) {
          const u32x4 fs = Rows::frag_t(st + G::kS, t0 + t, s, lane);
          os[t] = M::mma(fs, fo[s], os[t]);
          xs[t] = M::mma(fs, fx[s], xs[t]);
          es[t] = M::mma(Rows::frag_t(st + G::kDS, t0 + t, s, lane), fe[s], es[t]);
        }
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int s = 0; s < VS; ++s) {
          const u32x4 f = Rows::frag_t(st + G::kE + G::kShift, j0 + t, s, lane);
          oe[t] = M::mma(f, fo[s], oe[t]);
          xe[t] = M::mma(f, fx[s], xe[t]);
        }
      // rows past the block's are zero in LDS; the same slots of both panels hold the same element
      for (int at = threadIdx.x * 16; at < Rows::bytes(DK); at += 512 * 16) {
        const u32x4 x = *reinterpret_cast<const u32x4*>(st + G::kS + at);
        const u32x4 y = *reinterpret_cast<const u32x4*>(st + G::kDS + at);
        if constexpr (sizeof(T) == 2) {
          float u[8], v[8];
          unpack8(x, u);
          unpack8(y, v);
#pragma unroll
          for (int j = 0; j < 8; ++j) ss += u[j] * v[j];
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) ss += __uint_as_float(x[j]) * __uint_as_float(y[j]);
        }
      }
    }
    __syncthreads();                                         // the block has been read
    if (!G::kOwnQ) {
      load_qk();
      wait_vm<0>();
      __syncthreads();
    }
    const int m0 = G::kM + (G::kTwo ? ((h + 1 - kh * group) * blocks - 1 & 1) * G::kBlock : 0);   // Mq, Mk
    // q_i . k_j and k_i . k_j
    f32x4 qk[2], kk[2];
    {
      u32x4 fq[SS], fk[SS];
#pragma unroll
      for (int s = 0; s < SS; ++s) {
        fq[s] = Panels<T>::frag(smem + G::kQ, i, s, g);
        fk[s] = Panels<T>::frag(smem + G::kK, i, s, g);
      }
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        qk[t] = kk[t] = (f32x4){0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < SS; ++s) {
          const u32x4 f = Panels<T>::frag(smem + G::kK, M::row(j0 + t, m), s, g);
          qk[t] = M::mma(f, fq[s], qk[t]);
          kk[t] = M::mma(f, fk[s], kk[t]);
        }
      }
    }
    const double bi = b[i], last = b[kDC - 1];
    f32x4 mq[2], mk[2];
    float sums[16];                                          // [t, r]: N_ij / beta_j (j <= i), then dg's part of row i
    float N[2][4], total[2];                                 // N_ij, j < i, and its sums over r
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      total[t] = 0.f;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int j = M::row(j0 + t, g * 4 + r);
        const float bj = beta[j], d = j <= i ? __expf((float)(bi - b[j])) : 0.f;
        const float uq = j <= i ? p.scale * d * oe[t][r] : 0.f, uk = j < i ? -d * xe[t][r] : 0.f;
        mq[t][r] = uq * bj;
        mk[t][r] = uk * bj;
        const float n = uq * qk[t][r] + uk * kk[t][r];
        sums[t * 4 + r] = n;
        N[t][r] = j < i ? n * bj : 0.f;
        total[t] += N[t][r];
      }
    }
    // Row i's part of dg_j: the sum of N_ij' over this half's j' < j, where j <= i.
    const float rows = total[0] + total[1];
    {
      float before[2];
      if constexpr (M::TPS == 2) {                           // a lane's j: g * 8 + 0..7
        before[0] = groups_before(rows, g);
        before[1] = before[0] + total[0];
      } else {                                               // t * 16 + g * 4 + 0..3
        before[0] = groups_before(total[0], g);
        before[1] = groups_before(total[1], g) + __shfl(before[0] + total[0], 48 + m, 64);
      }
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          sums[8 + t * 4 + r] = M::row(j0 + t, g * 4 + r) <= i ? before[t] : 0.f;
          before[t] += N[t][r];
        }
    }
    auto put_m = [&](const f32x4 (&x)[2], int to) __attribute__((always_inline)) {   // rows of tokens i, columns j
#pragma unroll
      for (int t = 0; t < 2; ++t)
        store4(reinterpret_cast<T*>(smem + to + Panels<T>::at(i, M::row(j0 + t, g * 4))), x[t][0], x[t][1], x[t][2],
               x[t][3]);
    };
    put_m(mq, m0);
    if (G::kBoth) put_m(mk, m0 + G::kMBytes);
    // Summed over this wave's 16 tokens: each step halves the sums that a lane holds, and lane m ends with the m-th.
#pragma unroll
    for (int d = 8; d > 0; d >>= 1)
#pragma unroll
      for (int x = 0; x < d; ++x) {
        const float other = __shfl_xor((m & d) ? sums[x] : sums[x + d], d, 64);
        sums[x] = ((m & d) ? sums[x + d] : sums[x]) + other;
      }
    colsum[m >> 3][w][M::row(j0 + ((m >> 2) & 1), g * 4 + (m & 3))] = sums[0];
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) ss += __shfl_xor(ss, d, 64);
    if (lane == 0) part[wave] = ss;
    // this token's own products: scale exp(b) q.(S dO), exp(b) k.(S X), k.(dS' E), over this wave's half of dk
    float own[4] = {rows, 0.f, 0.f, 0.f};
#pragma unroll
    for (int t = 0; t < HT; ++t) {
      const int at = Panels<T>::at(i, M::row(t0 + t, g * 4));
      const f32x4 q = load4(reinterpret_cast<const T*>(smem + G::kQ + at));
      const f32x4 k = load4(reinterpret_cast<const T*>(smem + G::kK + at));
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        own[1] += q[r] * os[t][r];
        own[2] += k[r] * xs[t][r];
        own[3] += k[r] * es[t][r];
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      own[j] += __shfl_xor(own[j], 16, 64);
      own[j] += __shfl_xor(own[j], 32, 64);
      if (g == 0) half[hf][j][i] = own[j];
    }
    const float up = __expf((float)bi), left = __expf((float)(last - bi)), bet = beta[i];
    const float us = p.scale * up, le = left * bet;
#pragma unroll
    for (int t = 0; t < HT; ++t) {
      dq[t] += us * os[t];
      dk[t] += le * es[t] - up * xs[t];
    }
    __syncthreads();                                         // Mq, Mk, the sums
    if (wave == 0) {                                         // lane: token
      const float qos = half[0][1][lane] + half[1][1][lane];
      const float kxs = half[0][2][lane] + half[1][2][lane], kes = half[0][3][lane] + half[1][3][lane];
      const float n = colsum[0][0][lane] + colsum[0][1][lane] + colsum[0][2][lane] + colsum[0][3][lane];
      const float up = __expf((float)b[lane]), left = __expf((float)(last - b[lane]));
      float after = p.scale * up * qos - up * kxs;           // summed over the tokens from this one on
      float low = half[0][0][lane];                          // N_ij over the first half's j: of the second half's dg
      float end = left * beta[lane] * kes;                   // summed over the tokens before this one
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const float x = __shfl_down(after, d, 64), y = __shfl_down(low, d, 64), z = __shfl_up(end, d, 64);
        if (lane + d < 64) {
          after += x;
          low += y;
        }
        if (lane >= d) end += z;
      }
      end = __shfl_up(end, 1, 64);
      const float all = part[0] + part[1] + part[2] + part[3] + part[4] + part[5] + part[6] + part[7];
      const float dg = after + (lane > 0 ? end : 0.f) + (lane >= 32 ? low : 0.f) + __expf((float)last) * all +
                       (colsum[1][0][lane] + colsum[1][1][lane] + colsum[1][2][lane] + colsum[1][3][lane]);
      if (lane < c.len) {
        const int64_t t = c.tok0 + lane;
        const int64_t og = c.b * a.sdg.b + h * a.sdg.h + t * a.sdg.t;
        const int64_t ob = c.b * a.sdbeta.b + h * a.sdbeta.h + t * a.sdbeta.t;
        const float db = n + left * kes;
        if (a.gates_f32) {
          ((float*)a.dg)[og] = dg;
          ((float*)a.dbeta)[ob] = db;
        } else {
          ((T*)a.dg)[og] = from_f32<T>(dg);
          ((T*)a.dbeta)[ob] = from_f32<T>(db);
        }
      }
    }
    // dQ += Mq K; dK += Mk K + Mk^T K + Mq^T Q
    {
      u32x4 a_q[CS], a_k[CS], t_q[CS], t_k[CS];
#pragma unroll
      for (int s = 0; s < CS; ++s) {
        a_q[s] = Panels<T>::frag(smem + m0, i, s, g);
        t_q[s] = Panels<T>::frag_t(smem + m0, w, s, lane);
      }
      if (!G::kBoth) {
        __syncthreads();
        put_m(mk, m0);
        __syncthreads();
      }
#pragma unroll
      for (int s = 0; s < CS; ++s) {
        a_k[s] = Panels<T>::frag(smem + m0 + (G::kBoth ? G::kMBytes : 0), i, s, g);
        t_k[s] = Panels<T>::frag_t(smem + m0 + (G::kBoth ? G::kMBytes : 0), w, s, lane);
      }
#pragma unroll
      for (int t = 0; t < HT; ++t)
#pragma unroll
        for (int s = 0; s < CS; ++s) {
          const u32x4 fk = Panels<T>::frag_t(smem + G::kK, t0 + t, s, lane);
          const u32x4 fq = Panels<T>::frag_t(smem + G::kQ, t0 + t, s, lane);
          dq[t] = M::mma(fk, a_q[s], dq[t]);
          dk[t] = M::mma(fk, a_k[s], dk[t]);
          dk[t] = M::mma(fk, t_k[s], dk[t]);
          dk[t] = M::mma(fq, t_q[s], dk[t]);
        }
    }
  }
  if (i < c.len) {
    T* oq = (T*)a.dq + c.b * a.sdq.b + kh * a.sdq.h + (int64_t)(c.tok0 + i) * a.sdq.t;
    T* ok = (T*)a.dk + c.b * a.sdk.b + kh * a.sdk.h + (int64_t)(c.tok0 + i) * a.sdk.t;
#pragma unroll
    for (int t = 0; t < HT; ++t) {
      const int d = M::row(t0 + t, g * 4);
      if (d < p.dk) {
        store4(oq + d, dq[t][0], dq[t][1], dq[t][2], dq[t][3]);
        store4(ok + d, dk[t][0], dk[t][1], dk[t][2], dk[t][3]);
      }
    }
  }
}

constexpr size_t kAlign = 256;
size_t up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

// The workspace: both records, S, dS' (T), E, X (T), in this order.
template <typename T>
size_t place(DeltaGradArgs& a) {
  const size_t n = (size_t)delta_slots(a.f.seqs, a.f.batch) * a.f.Hv;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    char* r = a.f.ws + at;
    at += up(bytes);
    return r;
  };
  a.rec = take(n * ChunkRec<T>::kBytes);
  a.rect = take(n * ChunkRecT<T>::kBytes);
  a.states = take(n * a.f.dv * a.f.dk * sizeof(T));
  a.dstates = take(n * a.f.dv * a.f.dk * sizeof(T));
  a.errors = take(n * a.f.dv * kDC * sizeof(T));
  a.xs = take(n * a.f.dv * kDC * sizeof(T));
  return at;
}

template <typename T, int DK, int NW>
hipError_t launch_sizes(const DeltaGradArgs& a, int64_t slots, int sequences, hipStream_t s) {
  constexpr int kMax = 160 * 1024;
  constexpr int SF = Walk<T, DK, NW, 2, kKeep, false>::kSmem <= kMax ? 2 : 1;
  constexpr int SB = WalkBack<T, DK, NW, 2>::kSmem <= kMax ? 2 : 1;
  constexpr int F = Walk<T, DK, NW, SF, kKeep, false>::kSmem, B = WalkBack<T, DK, NW, SB>::kSmem, W = F > B ? F : B;
  static_assert(W <= kMax && Grads<T, DK>::kSmem <= Grads<T, DK>::kLds, "LDS of a CU");
  auto walks = k_delta_walks<T, DK, NW, SF, SB>;
  auto grads = k_delta_grads<T, DK>;
  if (sequences > 0) {
    const int64_t blocks =
        walk_blocks((int64_t)sequences * a.f.Hk, a.f.Hv / a.f.Hk * ((a.f.dv + 16 * NW - 1) / (16 * NW)));
    walks<<<dim3((unsigned)(2 * blocks)), 64 * (1 + NW), W, s>>>(a, sequences);
    if (hipError_t e = hipGetLastError()) return e;
  }
  if (slots > 0) grads<<<dim3((unsigned)(slots * a.f.Hk)), 512, Grads<T, DK>::kSmem, s>>>(a);
  return hipGetLastError();
}

}  // namespace

template <typename T>
size_t delta_grad_workspace_bytes(const DeltaArgs& f) {
  DeltaGradArgs a{};
  a.f = f;
  a.f.ws = nullptr;
  return place<T>(a);
}

template <typename T>
hipError_t launch_delta_grad(const DeltaGradArgs& given, hipStream_t s) {
  DeltaGradArgs a = given;
  place<T>(a);
  const int64_t slots = a.f.seqs.n > 0 ? delta_slots(a.f.seqs, a.f.batch) : 0;
  if (slots > 0) {
    k_delta_chunks<T, true><<<dim3((unsigned)(slots * a.f.Hv)), kChunkThreads, 0, s>>>(a.f, a.rec, a.rect);
    if (hipError_t e = hipGetLastError()) return e;
  }
  const int sequences = a.f.seqs.starts ? a.f.seqs.num : a.f.batch;
  if (a.f.dk <= 64) return launch_sizes<T, 64, 4>(a, slots, sequences, s);
  if (a.f.dk <= 128) return launch_sizes<T, 128, 4>(a, slots, sequences, s);
  return launch_sizes<T, 256, sizeof(T) == 2 ? 4 : 2>(a, slots, sequences, s);
}

template size_t delta_grad_workspace_bytes<bf16>(const DeltaArgs&);
template size_t delta_grad_workspace_bytes<float>(const DeltaArgs&);
template hipError_t launch_delta_grad<bf16>(const DeltaGradArgs&, hipStream_t);
template hipError_t launch_delta_grad<float>(const DeltaGradArgs&, hipStream_t);

}  // namespace ttt
