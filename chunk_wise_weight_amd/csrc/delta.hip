// The gated delta rule over whole sequences, forward (gfx950); the mathematics
// and the operand layout are in delta.hpp.
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
// in registers as the next product's operand.
constexpr int kChunkThreads = 256;
constexpr int kLd = 68;           // pitch of a 64 x 64 fp32 matrix in LDS

__device__ __forceinline__ f32x4 mma_f32(const float* a, f32x4 b, f32x4 c) {
  return Mat<float>::mma(*reinterpret_cast<const u32x4*>(a), __builtin_bit_cast(u32x4, b), c);
}

template <typename T>
__global__ __launch_bounds__(kChunkThreads) void k_delta_chunks(DeltaArgs p, char* rec) {
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

  if (w == 0) {
    float gi = 0.f, bi = 0.f;
    if (lane < c.len) {
      gi = p.g[c.b * p.sg.b + h * p.sg.h + (c.tok0 + lane) * p.sg.t];
      bi = p.beta[c.b * p.sbeta.b + h * p.sbeta.h + (c.tok0 + lane) * p.sbeta.t];
    }
    // exp(-200) is zero in fp32: a decay of -inf (a state reset) keeps the running sum finite
    double s = gi < -200.f ? -200.0 : (double)gi;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const double up = __shfl_up(s, d, 64);
      if (lane >= d) s += up;
    }
    const double last = __shfl(s, 63, 64);
    b[lane] = s;
    beta[lane] = bi;
    float* gate = reinterpret_cast<float*>(out + ChunkRec<T>::kGate);
    gate[lane] = __expf((float)s);
    gate[64 + lane] = bi;
    gate[128 + lane] = __expf((float)(last - s));
  }

  // rows of this wave's block against all blocks up to it
  f32x4 kk[4], qk[4];
#pragma unroll
  for (int t = 0; t < 4; ++t) kk[t] = qk[t] = (f32x4){0.f, 0.f, 0.f, 0.f};
  const __amdgpu_buffer_rsrc_t rk =
      make_rsrc((const T*)p.k + c.b * p.sk.b + kh * p.sk.h + c.tok0 * p.sk.t, (uint64_t)kOOB);
  const __amdgpu_buffer_rsrc_t rq =
      make_rsrc((const T*)p.q + c.b * p.sq.b + kh * p.sq.h + c.tok0 * p.sq.t, (uint64_t)kOOB);
  const unsigned row_bytes = p.dk * sizeof(T), kp = p.sk.t * sizeof(T), qp = p.sq.t * sizeof(T);
  for (int s = 0; s * KB < p.dk; ++s) {
    const unsigned byte = s * 64 + g * 16;
    const int r = w * 16 + m;
    const u32x4 fq =
        __builtin_amdgcn_raw_buffer_load_b128(rq, r < c.len && byte < row_bytes ? r * qp + byte : kOOB, 0, 0);
    u32x4 fk[4];
#pragma unroll
    for (int t = 0; t < 4; ++t)
      if (t <= w) {
        const int j = t * 16 + m;
        fk[t] = __builtin_amdgcn_raw_buffer_load_b128(rk, j < c.len && byte < row_bytes ? j * kp + byte : kOOB, 0, 0);
      }
    u32x4 mine = fk[0];
#pragma unroll
    for (int t = 1; t < 4; ++t)
      if (t == w) mine = fk[t];
#pragma unroll
    for (int t = 0; t < 4; ++t)
      if (t <= w) {
        kk[t] = Mat<T>::mma(mine, fk[t], kk[t]);
        qk[t] = Mat<T>::mma(fq, fk[t], qk[t]);
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
  constexpr int E = 16 / sizeof(T);
  for (int f = w; f < Mat<T>::kTri; f += 4) {
    int t = 0;
    while (Mat<T>::tri(t, Mat<T>::steps(t) - 1) < f) ++t;
    const int s = f - Mat<T>::tri(t, 0);
    const float* x = X + Mat<T>::row(t, m) * kLd + s * KB + g * E;
    u32x4 hi;
    if constexpr (sizeof(T) == 2) {
      const f32x4 v[2] = {*reinterpret_cast<const f32x4*>(x), *reinterpret_cast<const f32x4*>(x + 4)};
      hi = Mat<T>::frag(v);
    } else {
      hi = *reinterpret_cast<const u32x4*>(x);
    }
    *reinterpret_cast<u32x4*>(out + ChunkRec<T>::kP + f * 1024 + lane * 16) = hi;
  }
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
  for (int f = w; f < Mat<T>::kTri; f += 4) {
    int t = 0;
    while (Mat<T>::tri(t, Mat<T>::steps(t) - 1) < f) ++t;
    const int s = f - Mat<T>::tri(t, 0);
    const float* y = X + Mat<T>::row(t, m) * kLd + s * KB + g * E;
    char* o = out + f * 1024 + lane * 16;
    if constexpr (sizeof(T) == 2) {
      const f32x4 v[2] = {*reinterpret_cast<const f32x4*>(y), *reinterpret_cast<const f32x4*>(y + 4)};
      u32x4 hi, lo;
      Mat<T>::split(v, hi, lo);
      *reinterpret_cast<u32x4*>(o) = hi;
      *reinterpret_cast<u32x4*>(o + ChunkRec<T>::kTl) = lo;
    } else {
      *reinterpret_cast<u32x4*>(o) = *reinterpret_cast<const u32x4*>(y);
    }
  }
}

// ------------------------------------------------------------------ the walk over the chunks

// A workgroup of NW waves walks one sequence of one value head; wave w keeps
// 16 columns of the state (dv), which need nothing from the other columns.
// The chunk's K, Q and record are shared through LDS, brought by DMA while
// the chunk before is worked on (STAGES = 2; the widest heads have room for
// one stage); the wave's own V comes ahead in registers.
template <typename T, int DK, int NW, int STAGES>
struct Walk {
  static constexpr int kK = 0, kQ = Panels<T>::bytes(DK), kRec = 2 * kQ;
  static constexpr int kStage = kRec + ChunkRec<T>::kBytes;
  static constexpr int kSmem = STAGES * kStage;
  static constexpr int kLoads = 2 * Panels<T>::loads(DK) + ChunkRec<T>::kBytes / 1024;
};

template <typename T> __device__ __forceinline__ float raw_load(__amdgpu_buffer_rsrc_t r, unsigned off);
template <> __device__ __forceinline__ float raw_load<bf16>(__amdgpu_buffer_rsrc_t r, unsigned off) {
  return __uint_as_float((unsigned)__builtin_amdgcn_raw_buffer_load_b16(r, off, 0, 0) << 16);
}
template <> __device__ __forceinline__ float raw_load<float>(__amdgpu_buffer_rsrc_t r, unsigned off) {
  return __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(r, off, 0, 0));
}

template <typename T, int DK, int NW, int STAGES>
__global__ __launch_bounds__(64 * NW) void k_delta_walk(DeltaArgs p, const char* rec) {
  using M = Mat<T>;
  using G = Walk<T, DK, NW, STAGES>;
  constexpr int ST = DK / 16, SS = DK / M::KB;       // state blocks, steps over dk
  constexpr int CS = kDC / M::KB;                    // steps over a chunk's tokens
  extern __shared__ __attribute__((aligned(16))) char smem[];
  const int parts = (p.dv + 16 * NW - 1) / (16 * NW);
  const int id = xcd_remap(blockIdx.x, gridDim.x);
  const int part = id % parts, h = (id / parts) % p.Hv, seq = id / parts / p.Hv;
  const int w = wave_id(), lane = lane_id(), m = lane & 15, g = lane >> 4;
  const int col0 = (part * NW + w) * 16, kh = h / (p.Hv / p.Hk);
  const SeqPlace sp = seq_place(p.seqs, seq);
  const int chunks = (sp.len + kDC - 1) / kDC;
  const unsigned kp = p.sk.t * sizeof(T), qp = p.sq.t * sizeof(T), vp = p.sv.t * sizeof(T);
  const unsigned row_bytes = p.dk * sizeof(T);
  const T* k0 = (const T*)p.k + sp.b * p.sk.b + kh * p.sk.h + sp.tok0 * p.sk.t;
  const T* q0 = (const T*)p.q + sp.b * p.sq.b + kh * p.sq.h + sp.tok0 * p.sq.t;
  const T* v0 = (const T*)p.v + sp.b * p.sv.b + h * p.sv.h + sp.tok0 * p.sv.t;
  T* o0 = (T*)p.O + sp.b * p.so.b + h * p.so.h + sp.tok0 * p.so.t;

  auto fetch = [&](int c, char* stage) {
    const int len = min(kDC, sp.len - c * kDC);
    const __amdgpu_buffer_rsrc_t rk = make_rsrc(k0 + (int64_t)c * kDC * p.sk.t, (uint64_t)kOOB);
    const __amdgpu_buffer_rsrc_t rq = make_rsrc(q0 + (int64_t)c * kDC * p.sq.t, (uint64_t)kOOB);
    const __amdgpu_buffer_rsrc_t rr =
        make_rsrc(rec + ((int64_t)(sp.slot0 + c) * p.Hv + h) * ChunkRec<T>::kBytes, ChunkRec<T>::kBytes);
    constexpr int NL = Panels<T>::loads(DK);
#pragma unroll
    for (int i = 0; i < (G::kLoads + NW - 1) / NW; ++i) {
      const int l = i * NW + w;
      if (l < NL)
        Panels<T>::load(rk, l, len, kp, row_bytes, stage + G::kK);
      else if (l < 2 * NL)
        Panels<T>::load(rq, l - NL, len, qp, row_bytes, stage + G::kQ);
      else if (l < G::kLoads)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rr, (lds_ptr_t)(stage + G::kRec + (l - 2 * NL) * 1024), 16,
                                                 (unsigned)((l - 2 * NL) * 1024 + lane * 16), 0, 0, 0);
    }
  };
  float v[16];
  auto fetch_v = [&](int c) {
    const int len = min(kDC, sp.len - c * kDC);
    const __amdgpu_buffer_rsrc_t rv = make_rsrc(v0 + (int64_t)c * kDC * p.sv.t, (uint64_t)kOOB);
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int i = M::row(t, g * 4 + r);
        v[t * 4 + r] = raw_load<T>(rv, i < len && col0 + m < p.dv ? i * vp + (col0 + m) * (unsigned)sizeof(T) : kOOB);
      }
  };

  if (chunks > 0) {
    fetch(0, smem);
    fetch_v(0);
  }
  // state block t, register r: dk = row(t, 4 g + r), dv = col0 + m
  f32x4 S[ST];
  const int64_t wbase = (((int64_t)seq * p.Hv + h) * p.dv + col0 + m) * p.dk;
#pragma unroll
  for (int t = 0; t < ST; ++t) {
    const int d = M::row(t, g * 4);
    S[t] = (f32x4){0.f, 0.f, 0.f, 0.f};
    if (p.W_init && d < p.dk && col0 + m < p.dv) S[t] = *reinterpret_cast<const f32x4*>(p.W_init + wbase + d);
  }

  for (int c = 0; c < chunks; ++c) {
    char* st = smem + (STAGES == 2 ? (c & 1) * G::kStage : 0);
    const int len = min(kDC, sp.len - c * kDC);
    __builtin_amdgcn_s_waitcnt(0x0f70);              // vmcnt(0): this chunk's loads
    __syncthreads();
    if (STAGES == 2 && c + 1 < chunks) fetch(c + 1, smem + ((c + 1) & 1) * G::kStage);
    const float* gate = reinterpret_cast<const float*>(st + G::kRec + ChunkRec<T>::kGate);

    u32x4 Sh[SS], Sl[SS];
#pragma unroll
    for (int s = 0; s < SS; ++s) M::split(S + s * M::TPS, Sh[s], Sl[s]);
    // V - exp(b) K S
    f32x4 e[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      f32x4 acc = {0.f, 0.f, 0.f, 0.f};
      const int r = M::row(t, m);
#pragma unroll
      for (int s = 0; s < SS; ++s) acc = mma_split<T>(Panels<T>::frag(st + G::kK, r, s, g), Sh[s], Sl[s], acc);
      const f32x4 ga = *reinterpret_cast<const f32x4*>(gate + M::row(t, g * 4));
#pragma unroll
      for (int i = 0; i < 4; ++i) e[t][i] = v[t * 4 + i] - ga[i] * acc[i];
    }
    if (c + 1 < chunks) fetch_v(c + 1);
    u32x4 Rh[CS], Rl[CS];
#pragma unroll
    for (int s = 0; s < CS; ++s) M::split(e + s * M::TPS, Rh[s], Rl[s]);
    // E = T (V - exp(b) K S)
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int s = 0; s < M::steps(t); ++s) {
        const char* f = st + G::kRec + M::tri(t, s) * 1024 + lane * 16;
        const u32x4 th = *reinterpret_cast<const u32x4*>(f);
        const u32x4 tl = M::kSplit ? *reinterpret_cast<const u32x4*>(f + ChunkRec<T>::kTl) : th;
        acc = mma_split2<T>(th, tl, Rh[s], Rl[s], acc);
      }
      e[t] = acc;
    }
    // O: the state's columns in the instruction's rows, tokens in its columns, so a lane has 4 columns of one token
    {
      u32x4 Eh[CS];
#pragma unroll
      for (int s = 0; s < CS; ++s) Eh[s] = M::frag(e + s * M::TPS);
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const int r = M::row(t, m);
        f32x4 o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < SS; ++s) o = M::mma(Sh[s], Panels<T>::frag(st + G::kQ, r, s, g), o);
        o *= p.scale * gate[r];
#pragma unroll
        for (int s = 0; s < M::steps(t); ++s)
          o = M::mma(Eh[s], *reinterpret_cast<const u32x4*>(st + G::kRec + ChunkRec<T>::kP + M::tri(t, s) * 1024 +
                                                           lane * 16), o);
        if (r < len && col0 + g * 4 < p.dv)
          store4(o0 + (int64_t)(c * kDC + r) * p.so.t + col0 + g * 4, o[0], o[1], o[2], o[3]);
      }
    }
    // S = exp(b_63) S + K^T (exp(b_63 - b) beta E)
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const int i = M::row(t, g * 4);
      e[t] *= *reinterpret_cast<const f32x4*>(gate + 64 + i) * *reinterpret_cast<const f32x4*>(gate + 128 + i);
    }
#pragma unroll
    for (int s = 0; s < CS; ++s) M::split(e + s * M::TPS, Rh[s], Rl[s]);
    const float decay = gate[63];
#pragma unroll
    for (int t = 0; t < ST; ++t) {
      S[t] *= decay;
#pragma unroll
      for (int s = 0; s < CS; ++s) S[t] = mma_split<T>(Panels<T>::frag_t(st + G::kK, t, s, lane), Rh[s], Rl[s], S[t]);
    }
    if (STAGES == 1 && c + 1 < chunks) {
      __syncthreads();
      fetch(c + 1, smem);
    }
  }
#pragma unroll
  for (int t = 0; t < ST; ++t) {
    const int d = M::row(t, g * 4);
    if (d < p.dk && col0 + m < p.dv) *reinterpret_cast<f32x4*>(p.W_final + wbase + d) = S[t];
  }
}

template <typename T, int DK, int NW>
hipError_t launch_walk(const DeltaArgs& a, const char* rec, int sequences, hipStream_t s) {
  constexpr int STAGES = 2 * Walk<T, DK, NW, 1>::kStage <= 160 * 1024 ? 2 : 1;
  using G = Walk<T, DK, NW, STAGES>;
  auto kern = k_delta_walk<T, DK, NW, STAGES>;
  static const hipError_t set =
      hipFuncSetAttribute((const void*)kern, hipFuncAttributeMaxDynamicSharedMemorySize, G::kSmem);
  if (set != hipSuccess) return set;
  const int64_t parts = (a.dv + 16 * NW - 1) / (16 * NW);
  kern<<<dim3((unsigned)(parts * a.Hv * sequences)), 64 * NW, G::kSmem, s>>>(a, rec);
  return hipGetLastError();
}

}  // namespace

template <typename T>
size_t delta_workspace_bytes(const DeltaArgs& a) {
  return (size_t)delta_slots(a.seqs, a.batch) * a.Hv * ChunkRec<T>::kBytes;
}

template <typename T>
hipError_t launch_delta(const DeltaArgs& a, hipStream_t s) {
  const int64_t slots = delta_slots(a.seqs, a.batch);
  if (slots > 0 && a.seqs.n > 0) {
    k_delta_chunks<T><<<dim3((unsigned)(slots * a.Hv)), kChunkThreads, 0, s>>>(a, a.ws);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const int sequences = a.seqs.starts ? a.seqs.num : a.batch;
  if (sequences == 0) return hipSuccess;
  if (a.dk <= 64) return launch_walk<T, 64, 2>(a, a.ws, sequences, s);
  if (a.dk <= 128) return launch_walk<T, 128, 2>(a, a.ws, sequences, s);
  return launch_walk<T, 256, 2>(a, a.ws, sequences, s);
}

template size_t delta_workspace_bytes<bf16>(const DeltaArgs&);
template size_t delta_workspace_bytes<float>(const DeltaArgs&);
template hipError_t launch_delta<bf16>(const DeltaArgs&, hipStream_t);
template hipError_t launch_delta<float>(const DeltaArgs&, hipStream_t);

}  // namespace ttt
