// Backward of the selective scan (gfx950).
//
// With scan.hpp's notation, S the state before a chunk, dS the gradient of the state behind it, du_j that of u_j = r_j x_j:
//   du_j = sum_{i >= j} (C_i . B_j) exp(b_i - b_j) dO_i + exp(b_63 - b_j) dS B_j,     dx_j = r_j du_j + D dO_j
//   W_ij = (dO_i . x_j) exp(b_i - b_j) r_j  (j <= i)
//   dC_i = sum over heads of  sum_{j <= i} W_ij B_j + exp(b_i) S^T dO_i
//   dB_j = sum over heads of  sum_{i >= j} W_ij C_i + exp(b_63 - b_j) dS^T u_j
// The gradient of token t's log decay is summed from the terms that pass it alone, so that none has to cancel:
//   dg_t = sum_{i >= t > j} W_ij (C_i . B_j) + sum_{i >= t} exp(b_i) dO_i . S C_i + sum_{j < t} exp(b_63 - b_j) u_j . dS B_j
//          + exp(b_63) <S, dS>
//   dr_t = x_t . du_t + A dg_t,  dA = sum_t r_t dg_t,  ddt_t = dr_t, with softplus times its derivative.
// The states S and, walking back, dS' = exp(b_63) dS + sum_i exp(b_i) dO_i C_i^T are kept for every chunk (scan_walk.hpp);
// what is local to a chunk is made for all chunks at once, a workgroup for a chunk and group, its heads one after the
// other, dB and dC staying in registers over them.  In bf16, states enter as three bf16 values (their fp32's 24 bits), the
// decayed products as two; no product of rounded values goes into dg: the pairs' sums are of fp32 results alone.
#include "scan_walk.hpp"

namespace ttt {
namespace {

// Rows of B or C that a chunk has: in LDS, or where that has no room (the widest fp32 states) in memory.
template <typename T, bool LDS> struct Features {
  const char* lds;
  const T* rows;
  int64_t pitch;
  int len, N;
  __device__ __forceinline__ u32x4 frag(const LaneAt<T>& L, int t, int s) const {
    if constexpr (LDS) return L.frag(lds, t, s);
    const int r = Mat<T>::row(t, lane_id() & 15), n = s * 16 + (lane_id() >> 4) * 4;
    return r < len && n < N ? *reinterpret_cast<const u32x4*>(rows + r * pitch + n) : (u32x4){0, 0, 0, 0};
  }
  __device__ __forceinline__ u32x4 cols(const LaneAt<T>& L, int t, int s) const {
    if constexpr (LDS) return L.cols(lds, t, s);
    const int n = t * 16 + (lane_id() & 15), r = s * 16 + (lane_id() >> 4) * 4;
    u32x4 o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = r + i < len && n < N ? __float_as_uint((float)rows[(r + i) * pitch + n]) : 0u;
    return o;
  }
  __device__ __forceinline__ f32x4 at(const LaneAt<T>& L, int t, int ct) const {
    if constexpr (LDS) return L.at(lds, t, ct);
    const int r = Mat<T>::row(t, lane_id() & 15), n = ct * 16 + (lane_id() >> 4) * 4;
    return r < len && n < N ? load4(rows + r * pitch + n) : (f32x4){0.f, 0.f, 0.f, 0.f};
  }
};

// A head's block of 64 rows of P: x and dO of the chunk's tokens, and 64 columns of S and dS at a time.
constexpr int kBV = 64, kBN = 64;
template <typename T, int DN_, bool LDS_> struct GradShape {
  static constexpr int DN = DN_, NB = DN / kBN, KS = kBN / Mat<T>::KB;
  static constexpr bool LDS = LDS_;
  static constexpr int SP = Mat<T>::kSplit ? 3 : 1;          // planes of a state: their sum is it
  static constexpr int kB = LDS ? tile_bytes<T>(DN) : 0, kS = tile_bytes<T>(kBN), kX = tile_bytes<T>(kBV);
  static constexpr int kM = tile_bytes<T>(kDC);           // a 64 x 64 matrix (bf16: and what its rounding left)
  static constexpr int kMs = kM * (Mat<T>::kSplit ? 2 : 1);
  // x, dO and the gates come by DMA, where LDS has room for it while the block before is worked on.
  static constexpr int XB = 2 * kB + 2 * SP * kS + 4 * kX + kMs <= kMaxLds - 12 * 1024 ? 2 : 1;
  static constexpr int oS = 2 * kB, oX = oS + 2 * SP * kS, oM = oX + 2 * XB * kX, kSmem = oM + kMs;
};

// x summed over the four lanes that hold a token.
template <typename F> __device__ __forceinline__ F token_sum(F x) {
  x += __shfl_xor(x, 16, 64);
  return x + __shfl_xor(x, 32, 64);
}
// x summed over the 16 lanes of a group.
template <int ROR> __device__ __forceinline__ float ror_add(float x) {
  return x + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x120 + ROR, 0xf, 0xf, true));
}
template <int ROR> __device__ __forceinline__ double ror_add(double x) {
  u32x2 w = __builtin_bit_cast(u32x2, x);
#pragma unroll
  for (int i = 0; i < 2; ++i) w[i] = (unsigned)__builtin_amdgcn_update_dpp(0, (int)w[i], 0x120 + ROR, 0xf, 0xf, true);
  return x + __builtin_bit_cast(double, w);
}
template <typename F> __device__ __forceinline__ F group_sum(F x) { return ror_add<1>(ror_add<2>(ror_add<4>(ror_add<8>(x)))); }
__device__ __forceinline__ float dot4(f32x4 a, f32x4 b) { return a[0] * b[0] + a[1] * b[1] + a[2] * b[2] + a[3] * b[3]; }
// Keeps the instructions of a phase together: reads drawn ahead over phases cost registers, and what is then spilled waits
// for the loads under way.
__device__ __forceinline__ void phase() { __builtin_amdgcn_sched_barrier(0); }
// 16 bytes at `base` + off, zero for off >= kOOB.
__device__ __forceinline__ u32x4 load_or_zero(__amdgpu_buffer_rsrc_t rs, unsigned off) {
  return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, off, 0, 0));
}

// 8 fp32 values of a row of a state block to its planes: each the 8 leading bits of what the ones before left, 24 in all.
template <typename T, int SP>
__device__ __forceinline__ void put_planes(f32x4 a, f32x4 b, char* plane, int stride, int r, int c8) {
  if constexpr (sizeof(T) == 2) {
    char* at = plane + r * 128 + ((c8 ^ row_swz(r)) << 4);
    unsigned v[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = __float_as_uint(a[i]);
      v[4 + i] = __float_as_uint(b[i]);
    }
#pragma unroll
    for (int k = 0; k < SP; ++k) {
      u32x4 w;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        w[i] = __builtin_amdgcn_perm(v[2 * i + 1], v[2 * i], 0x07060302);
        if (k + 1 < SP) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const unsigned u = v[2 * i + j];
            v[2 * i + j] = __float_as_uint(__uint_as_float(u) - __uint_as_float(u & 0xffff0000u));
          }
        }
      }
      *reinterpret_cast<u32x4*>(at + k * stride) = w;
    }
  } else {
    char* at = plane + (c8 >> 2) * kPanel64 + r * 128;
    *reinterpret_cast<f32x4*>(at + (((c8 & 3) * 2 ^ row_swz(r)) << 4)) = a;
    *reinterpret_cast<f32x4*>(at + (((c8 & 3) * 2 + 1 ^ row_swz(r)) << 4)) = b;
  }
}

// What the gradients of a chunk's rates are made of, for one head: with Z_ij = (C_i . B_j) (dO_i . x_j) exp(b_i - b_j),
// by token: sums of Z_ij r_j over j < i (by steps of j), of Z_ij over i > j (by blocks of i), Z_ii and dO_i . x_i; C_i . S^T
// dO_i and B_j . dS^T x_j by blocks of N; and <S, dS> by waves.  The sums of Z are fp64: a decay gets the difference of
// the rows' and columns' sums up to its token, in which all but the pairs about it have to cancel (in fp32 what was left of
// them, the same for all tokens that follow, made dA and the bias's gradient of fast heads off by 4e-6).
template <typename T> struct TokenSums {
  double rows[kDC / Mat<T>::KB][kDC], cols[4][kDC];
  float diag[2][kDC], dots[8][kDC], ss[8], pad[8];
};

// One workgroup of 8 waves per chunk slot and group, its heads one after the other; where several share them, each leaves its
// fp32 part of dB and dC.
//   waves 0-3  S^T dO and dC, waves 4-7  dS^T x and dB: block w & 3 of every 64 features of N, all tokens
//   du         blocks 2 (w & 1) and the next of P, tokens row(w >> 1, .)
//   C B^T, dO x^T and their decayed forms by fragments, a wave one (fp32: two); they go to LDS once for all waves
// States come as fp32, the next block's loads under way while one is worked on, and are cut into planes on their way to
// LDS; sums that go into ddt are of all three planes, dx of two.  4 x 4,096 tokens x 32 heads of 64 x 128 in bf16: 268 us at the
// least under a trace, 2.2 TB/s; one workgroup a CU fits LDS, and its barriers leave the matrix cores busy for 16 % of the
// cycles, LDS for 30 %.
template <typename T, int DN, bool LDS>
__global__ __launch_bounds__(512, 2) void k_scan_grads(ScanGradArgs a) {
#if __HIP_DEVICE_COMPILE__
  using M = Mat<T>;
  using Z = GradShape<T, DN, LDS>;
  constexpr int NS = DN / M::KB, CS = kDC / M::KB, NB = Z::NB, KS = Z::KS, U = M::TPS, SP = Z::SP;
  constexpr int F = (M::kTri + 7) / 8, XB = Z::XB;           // F: fragments a wave
  constexpr int PB = U;                                      // blocks of P that are stored as one
  extern __shared__ __attribute__((aligned(16))) char smem[];
  __shared__ __attribute__((aligned(1024))) char kept[2][2048];   // of a head and the next (KeptGates)
  __shared__ TokenSums<T> sums;
  const ScanArgs& p = a.f;
  const int id = xcd_remap(blockIdx.x, gridDim.x);
  const int share = id % a.parts, grp = id / a.parts % p.G, slot = id / a.parts / p.G, shared = p.H / p.G;
  const int head0 = grp * shared + share * a.heads, last = min(head0 + a.heads, (grp + 1) * shared);
  const ChunkPlace c = chunk_place(p.seqs, slot);
  if (c.len <= 0) return;
  const int tid = threadIdx.x, wave = wave_id(), side = wave >> 2, nt = wave & 3, lane = lane_id(), m = lane & 15, g = lane >> 4;
  const int P = p.P, N = p.N, len = c.len;
  const int64_t size = (int64_t)P * N;
  const Features<T, LDS> B{smem, (const T*)p.B + c.b * p.sB.b + grp * p.sB.h + c.tok0 * p.sB.t, p.sB.t, len, N};
  const Features<T, LDS> C{smem + Z::kB, (const T*)p.C + c.b * p.sC.b + grp * p.sC.h + c.tok0 * p.sC.t, p.sC.t, len, N};
  if constexpr (LDS) {
    TileLoader<T, DN, 8>(p.sB.t * sizeof(T), N * sizeof(T)).issue(B.rows, len, smem);
    TileLoader<T, DN, 8>(p.sC.t * sizeof(T), N * sizeof(T)).issue(C.rows, len, smem + Z::kB);
  }
  const LaneAt<T> L(lane);
  const Split<T> split(lane);
  char *const Sp = smem + Z::oS, *const Dp = Sp + SP * Z::kS, *const Mp = smem + Z::oM;

  // The workgroup's heads of the group, from the first on.
  const float *S = a.S + ((int64_t)slot * p.H + head0) * size, *dS = a.dS + ((int64_t)slot * p.H + head0) * size;
  const T* x = (const T*)p.x + c.b * p.sx.b + head0 * p.sx.h + c.tok0 * p.sx.t;
  const T* y = (const T*)a.dO + c.b * a.sdO.b + head0 * a.sdO.h + c.tok0 * a.sdO.t;
  const char* gates = (const char*)(a.gates + (int64_t)slot * p.H + head0);
  T* dx = (T*)a.dx + c.b * a.sdx.b + head0 * a.sdx.h + c.tok0 * a.sdx.t;
  char* to = a.sums + ((int64_t)slot * p.H + head0) * sizeof(TokenSums<T>);

  const int dtile = wave >> 1, dtok = M::row(dtile, m), dblock = 2 * (wave & 1);   // du's tokens and blocks of P

  // What is on its way: 8 columns of a row of S and dS.
  const int row8 = tid >> 3, col8 = (tid & 7) * 8;
  const unsigned soff = (unsigned)(row8 * N + col8) * 4u;
  const unsigned dxoff = dtok < len ? (unsigned)dtok * (unsigned)(a.sdx.t * sizeof(T)) : kOOB;
  u32x4 ns[2], nd[2];
  const TileLoader<T, kBV, 8> xload(p.sx.t * sizeof(T), kBV * sizeof(T)), yload(a.sdO.t * sizeof(T), kBV * sizeof(T));
  auto load_states = [&](const float* s, const float* d, int p0, int n0) __attribute__((always_inline)) {
    const unsigned off = p0 + row8 < P && n0 + col8 < N ? soff : kOOB;
    const __amdgpu_buffer_rsrc_t rs = rows_rsrc(s + (int64_t)p0 * N + n0), rd = rows_rsrc(d + (int64_t)p0 * N + n0);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      ns[k] = load_or_zero(rs, off + 16 * k);
      nd[k] = load_or_zero(rd, off + 16 * k);
    }
  };
  auto load_rows = [&](const T* xh, const T* yh, int p0, char* to) __attribute__((always_inline)) {
    if (p0 + kBV <= P) {
      xload.issue(xh + p0, len, to);
      yload.issue(yh + p0, len, to + Z::kX);
    } else {
      TileLoader<T, kBV, 8>(p.sx.t * sizeof(T), (P - p0) * sizeof(T)).issue(xh + p0, len, to);
      TileLoader<T, kBV, 8>(a.sdO.t * sizeof(T), (P - p0) * sizeof(T)).issue(yh + p0, len, to + Z::kX);
    }
  };
  auto load_gates = [&](const char* from, char* to) __attribute__((always_inline)) {
    if (wave < 2)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(make_rsrc(from, sizeof(KeptGates)), (lds_ptr_t)(to + wave * 1024), 16,
                                               (unsigned)tid * 16u, 0, 0, 0);
  };
  int turn = 0, hturn = 0;                                   // blocks of P, heads
  load_rows(x, y, 0, smem + Z::oX);
  load_gates(gates, kept[0]);
  load_states(S, dS, 0, 0);
  if constexpr (LDS) {
    wait_vm<0>();
    __syncthreads();
  }
  // C_i . B_j, token i = row(t, m), j = row(s U + u, 4 g + 0..3)
  f32x4 G[F][U];
  int ft[F], fs[F];
#pragma unroll
  for (int k = 0; k < F; ++k) {
    tri_place<T>(min(wave + 8 * k, M::kTri - 1), &ft[k], &fs[k]);
#pragma unroll
    for (int u = 0; u < U; ++u) G[k][u] = (f32x4){0.f, 0.f, 0.f, 0.f};
    if (wave + 8 * k < M::kTri)
#pragma unroll
      for (int n = 0; n < NS; ++n) {
        if (past<T, kBV>(n * M::KB, N)) break;
        const u32x4 f = C.frag(L, ft[k], n);
#pragma unroll
        for (int u = 0; u < U; ++u) G[k][u] = M::mma(B.frag(L, fs[k] * U + u, n), f, G[k][u]);
      }
  }
  f32x4 acc[NB][4];                                          // dC or dB: block nt of every 64 of N, tokens row(t, m)
#pragma unroll
  for (int n = 0; n < NB; ++n)
#pragma unroll
    for (int t = 0; t < 4; ++t) acc[n][t] = (f32x4){0.f, 0.f, 0.f, 0.f};
  const char *const state = side ? Dp : Sp;
  const Features<T, LDS> own = side ? B : C, cross = side ? C : B;

  for (int h = head0; h < last; ++h) {
    const float D = p.D ? p.D[h] : 0.f;
    const KeptGates& gate = *reinterpret_cast<const KeptGates*>(kept[hturn]);
    const Gates& q = gate.g;
    const float* const scales = side ? q.w : q.eb;
    f32x4 V[F][U], E[F][U];                                  // dO_i . x_j; exp(b_i - b_j), 0 for j > i
#pragma unroll
    for (int k = 0; k < F; ++k)
#pragma unroll
      for (int u = 0; u < U; ++u) V[k][u] = (f32x4){0.f, 0.f, 0.f, 0.f};
    float ss = 0.f, dot[4] = {0.f, 0.f, 0.f, 0.f};           // <S, dS>; C_i . S^T dO_i or B_j . dS^T x_j
    for (int p0 = 0; p0 < P; p0 += kBV) {
      const bool more = p0 + kBV < P, next = more || h + 1 < last;
      char *const Xp = smem + Z::oX + turn * 2 * Z::kX, *const Yp = Xp + Z::kX;
      const char* const other = side ? Xp : Yp;
      f32x4 du[2];
      du[0] = du[1] = (f32x4){0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        const int n0 = nb * kBN;
        if (NB > 2 && n0 >= N) continue;
        f32x4 s2[2], d2[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          s2[k] = __builtin_bit_cast(f32x4, ns[k]);
          d2[k] = __builtin_bit_cast(f32x4, nd[k]);
          ss += dot4(s2[k], d2[k]);
        }
        put_planes<T, SP>(s2[0], s2[1], Sp, Z::kS, row8, tid & 7);
        put_planes<T, SP>(d2[0], d2[1], Dp, Z::kS, row8, tid & 7);
        if (nb == 0) wait_vm<0>();                           // x, dO and the gates
        __syncthreads();
        if (nb + 1 < NB && (NB <= 2 || n0 + kBN < N)) {
          load_states(S, dS, p0, n0 + kBN);
        } else if (next) {
          if (XB == 2) {
            load_rows(more ? x : x + p.sx.h, more ? y : y + a.sdO.h, more ? p0 + kBV : 0, smem + Z::oX + (turn ^ 1) * 2 * Z::kX);
            if (!more) load_gates(gates + sizeof(KeptGates), kept[hturn ^ 1]);
          }
          load_states(more ? S : S + size, more ? dS : dS + size, more ? p0 + kBV : 0, 0);
        }
        phase();
        if (nb == 0) {
#pragma unroll
          for (int k = 0; k < F; ++k) {
            if (wave + 8 * k >= M::kTri) continue;
            int i = M::row(ft[k], m);
            asm volatile("" : "+v"(i));                    // (what follows from it is made again, not kept in masks)
#pragma unroll
            for (int v = 0; v < KS; ++v) {
              if (past<T, kBV>(v * M::KB, P - p0)) break;
              const u32x4 f = L.frag(Yp, ft[k], v);
#pragma unroll
              for (int u = 0; u < U; ++u) V[k][u] = M::mma(L.frag(Xp, fs[k] * U + u, v), f, V[k][u]);
            }
            if (p0 == 0) {                                   // (C_i . B_j) exp(b_i - b_j)
              const float ih = q.hi[i], il = q.lo[i];
              f32x4 w[U];
#pragma unroll
              for (int u = 0; u < U; ++u) {
                const int j = M::row(fs[k] * U + u, 4 * g);
                const f32x4 jh = *reinterpret_cast<const f32x4*>(q.hi + j), jl = *reinterpret_cast<const f32x4*>(q.lo + j);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  E[k][u][e] = j + e <= i ? exp2_hw((ih - jh[e]) + (il - jl[e])) : 0.f;
                  w[u][e] = G[k][u][e] * E[k][u][e];
                }
              }
              u32x4 hi, lo;
              split.two(w, hi, lo);
              char* f = L.place(Mp, ft[k], fs[k]);
              *reinterpret_cast<u32x4*>(f) = hi;
              if (M::kSplit) *reinterpret_cast<u32x4*>(f + Z::kM) = lo;
            }
          }
        }
        phase();
        // S^T dO (dS^T x), four independent sums
        if (!past<T, kBV>(n0 + nt * 16, N)) {
          f32x4 o[4];
#pragma unroll
          for (int t = 0; t < 4; ++t) o[t] = (f32x4){0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int s = 0; s < KS; ++s) {
            if (past<T, kBV>(s * M::KB, P - p0)) break;
            u32x4 f[SP], b[4];
#pragma unroll
            for (int z = 0; z < SP; ++z) f[z] = L.cols(state + z * Z::kS, nt, s);
#pragma unroll
            for (int t = 0; t < 4; ++t) b[t] = L.frag(other, t, s);
#pragma unroll
            for (int z = SP - 1; z >= 0; --z)
#pragma unroll
              for (int t = 0; t < 4; ++t) o[t] = M::mma(f[z], b[t], o[t]);
          }
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            dot[t] += dot4(o[t], own.at(L, t, 4 * nb + nt));
            acc[nb][t] += scales[M::row(t, m)] * o[t];
          }
        }
        phase();
        // dS B
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          if (past<T, kBV>(n0 + s * M::KB, N)) break;
          const u32x4 b = B.frag(L, dtile, nb * KS + s);
#pragma unroll
          for (int k = 0; k < 2; ++k)
            if (!past<T, kBV>((dblock + k) * 16, P - p0))
#pragma unroll
              for (int z = (SP > 1 ? 1 : 0); z >= 0; --z)
                du[k] = M::mma(L.frag(Dp + z * Z::kS, dblock + k, s), b, du[k]);
        }
        __syncthreads();                                     // the planes have been read, (C B^T exp) is there
      }
      // dx: of the tokens behind in the chunk, and of the state behind it
      {
        const float f = gate.rest[dtok], r = q.r[dtok];
#pragma unroll
        for (int k = 0; k < 2; ++k) du[k] *= f;
#pragma unroll
        for (int s = 0; s < CS; ++s) {
          if (s < M::first(dtile)) continue;
          const u32x4 hi = L.cols_row(Mp, dtile, s);
          u32x4 lo;
          if constexpr (M::kSplit) lo = L.cols_row(Mp + Z::kM, dtile, s);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            if (past<T, kBV>((dblock + k) * 16, P - p0)) continue;
            const u32x4 o = L.cols_row(Yp, dblock + k, s);
            if constexpr (M::kSplit) du[k] = M::mma(o, lo, du[k]);
            du[k] = M::mma(o, hi, du[k]);
          }
        }
        const __amdgpu_buffer_rsrc_t rs = rows_rsrc(dx + p0);
#pragma unroll
        for (int k = 0; k < 2; k += PB) {
          const int pp = M::row(dblock + k, 4 * g);
          f32x4 v[PB];
#pragma unroll
          for (int e = 0; e < PB; ++e) v[e] = r * du[k + e] + D * L.at_row(Yp, dtile, dblock + k + e);
          // (outside of the rows and of P: nothing is written)
          const unsigned off = p0 + pp < P ? dxoff + pp * (unsigned)sizeof(T) : kOOB;
          __builtin_amdgcn_raw_buffer_store_b128(M::frag(v), rs, off, 0, 0);
        }
      }
      __syncthreads();                                       // x, dO and (C B^T exp) have been read
      if (XB == 1 && next) {
        load_rows(more ? x : x + p.sx.h, more ? y : y + a.sdO.h, more ? p0 + kBV : 0, smem + Z::oX);
        if (!more) load_gates(gates + sizeof(KeptGates), kept[hturn ^ 1]);
      }
      turn ^= XB - 1;
    }
    // W to LDS, and the sums of W_ij (C_i . B_j) / r_j over rows and columns
#pragma unroll
    for (int k = 0; k < F; ++k) {
      if (wave + 8 * k >= M::kTri) continue;
      const int t = ft[k], s = fs[k];
      int i = M::row(t, m);
      asm volatile("" : "+v"(i));
      f32x4 w[U];
      double rs = 0.0;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int j = M::row(s * U + u, 4 * g);
        const f32x4 r = *reinterpret_cast<const f32x4*>(q.r + j);
        double cs[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float v = V[k][u][e] * E[k][u][e], z = v * G[k][u][e];
          w[u][e] = v * r[e];
          if (j + e == i) {
            sums.diag[0][i] = z;
            sums.diag[1][i] = V[k][u][e];
          }
          const double below = j + e < i ? z : 0.f;
          rs += below * r[e];
          cs[e] = group_sum(below);
        }
        if (m == 0)
#pragma unroll
          for (int e = 0; e < 4; ++e) sums.cols[t][j + e] = cs[e];
      }
      rs = token_sum(rs);
      if (g == 0) sums.rows[s][i] = rs;
      u32x4 hi, lo;
      split.two(w, hi, lo);
      char* f = L.place(Mp, t, s);
      *reinterpret_cast<u32x4*>(f) = hi;
      if (M::kSplit) *reinterpret_cast<u32x4*>(f + Z::kM) = lo;
    }
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const float d = token_sum(dot[t]);
      if (g == 0) sums.dots[wave][M::row(t, m)] = d;
    }
    ss = token_sum(group_sum(ss));
    if (lane == 0) sums.ss[wave] = ss;
    __syncthreads();
    // what a token has of the chunk's other tokens
    auto others = [&](auto back) __attribute__((always_inline)) {
      constexpr bool BACK = decltype(back)::value;
#pragma unroll
      for (int s = 0; s < CS; ++s) {
        u32x4 f[NB];
#pragma unroll
        for (int n = 0; n < NB; ++n)
          if (NB <= 2 || n * kBN < N) f[n] = cross.cols(L, 4 * n + nt, s);
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          if (BACK ? s < M::first(t) : s >= M::steps(t)) continue;
          const u32x4 hi = BACK ? L.cols_row(Mp, t, s) : L.frag(Mp, t, s);
          u32x4 lo;
          if constexpr (M::kSplit)
            lo = BACK ? L.cols_row(Mp + Z::kM, t, s) : L.frag(Mp + Z::kM, t, s);
#pragma unroll
          for (int n = 0; n < NB; ++n) {
            if (NB > 2 && n * kBN >= N) continue;
            if constexpr (M::kSplit) acc[n][t] = M::mma(f[n], lo, acc[n][t]);
            acc[n][t] = M::mma(f[n], hi, acc[n][t]);
          }
        }
      }
    };
    if (side) others(std::true_type()); else others(std::false_type());
    if (tid < (int)sizeof(sums) / 16) reinterpret_cast<u32x4*>(to)[tid] = reinterpret_cast<const u32x4*>(&sums)[tid];
    to += sizeof(sums);
    S += size;
    dS += size;
    x += p.sx.h;
    y += a.sdO.h;
    gates += sizeof(KeptGates);
    hturn ^= 1;
    dx += a.sdx.h;
    __syncthreads();                                         // W and the sums have been read
  }
  if (a.parts > 1) {
    float* out = a.shares + (((int64_t)id * 2 + side) * kDC) * N;
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const int i = M::row(t, m), col = n * kBN + nt * 16 + 4 * g;
        if (i < len && col < N) *reinterpret_cast<f32x4*>(out + i * N + col) = acc[n][t];
      }
    return;
  }
  T* out = side ? (T*)a.dB + c.b * a.sdB.b + grp * a.sdB.h + c.tok0 * a.sdB.t
                : (T*)a.dC + c.b * a.sdC.b + grp * a.sdC.h + c.tok0 * a.sdC.t;
  const int64_t pitch = side ? a.sdB.t : a.sdC.t;
#pragma unroll
  for (int n = 0; n < NB; ++n)
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const int i = M::row(t, m), col = n * kBN + nt * 16 + 4 * g;
      if (i < len && col < N) store4(out + i * pitch + col, acc[n][t][0], acc[n][t][1], acc[n][t][2], acc[n][t][3]);
    }
#endif
}

// The rates' gradients from their sums: a wave for each chunk slot and head, a lane for each token.  Its parts of dA, dD
// and ddt_bias go to part.
template <typename T>
__global__ __launch_bounds__(256) void k_scan_rates(ScanGradArgs a, int64_t chunk_heads) {
  using M = Mat<T>;
  const ScanArgs& p = a.f;
  const int64_t sh = (int64_t)blockIdx.x * 4 + wave_id();
  if (sh >= chunk_heads) return;
  const int slot = (int)(sh / p.H), h = (int)(sh % p.H), lane = lane_id();
  const ChunkPlace c = chunk_place(p.seqs, slot);
  f32x4 part = {0.f, 0.f, 0.f, 0.f};
  if (c.len > 0) {
    const TokenSums<T>& s = reinterpret_cast<const TokenSums<T>*>(a.sums)[sh];
    const KeptGates& q = a.gates[sh];
    double rsum = 0.0, csum = 0.0;
#pragma unroll
    for (int k = 0; k < kDC / M::KB; ++k) rsum += lane >= k * M::KB ? s.rows[k][lane] : 0.0;
#pragma unroll
    for (int t = 0; t < 4; ++t) csum += lane / M::KB < M::steps(t) ? s.cols[t][lane] : 0.0;
    const float r = q.g.r[lane];
    double so = 0.0, us = 0.0, all = 0.0;                    // dO . S C, x . dS B, <S, dS>
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      so += s.dots[i][lane];
      us += s.dots[4 + i][lane];
    }
    us *= q.rest[lane];
#pragma unroll
    for (int i = 0; i < 8; ++i) all += s.ss[i];
    double R = csum * r - rsum, z = us * r, y = q.g.eb[lane] * so;
    const double r0 = R, z0 = z;
#pragma unroll
    for (int i = 1; i < 64; i <<= 1) {
      const double up = __shfl_up(R, i, 64), uz = __shfl_up(z, i, 64), dy = __shfl_down(y, i, 64);
      if (lane >= i) {
        R += up;
        z += uz;
      }
      if (lane + i < 64) y += dy;
    }
    // pairs that token t's decay lies between: those of t - 1, less row t - 1's, and column t - 1's
    const double dg = (R - r0) + (z - z0) + y + q.g.eb[kDC - 1] * all;
    const bool in = lane < c.len;
    const double ddt = in ? (us + csum + s.diag[0][lane] + p.A[h] * dg) * q.slope[lane] : 0.0;
    if (in) a.ddt[c.b * a.sddt.b + h * a.sddt.h + (c.tok0 + lane) * a.sddt.t] = (float)ddt;
    double sa = in ? dg * r : 0.0, sb = ddt, sd = s.diag[1][lane];
#pragma unroll
    for (int i = 1; i < 64; i <<= 1) {
      sa += __shfl_xor(sa, i, 64);
      sb += __shfl_xor(sb, i, 64);
      sd += __shfl_xor(sd, i, 64);
    }
    part = (f32x4){(float)sa, (float)sd, (float)sb, 0.f};
  }
  if (lane == 0) *reinterpret_cast<f32x4*>(a.part + sh * 4) = part;
}

// dA, dD, ddt_bias: the chunks' parts, in a fixed order.
__global__ __launch_bounds__(256) void k_scan_grad_sum(const float* __restrict__ part, int64_t slots, int H,
                                                       float* __restrict__ dA, float* __restrict__ dD, float* __restrict__ db) {
  __shared__ double sum[3][4];
  const int h = blockIdx.x, lane = lane_id(), w = wave_id();
  double s[3] = {0.0, 0.0, 0.0};
  for (int64_t i = threadIdx.x; i < slots; i += 256) {
    const f32x4 v = *reinterpret_cast<const f32x4*>(part + (i * H + h) * 4);
#pragma unroll
    for (int k = 0; k < 3; ++k) s[k] += v[k];
  }
#pragma unroll
  for (int k = 0; k < 3; ++k) {
#pragma unroll
    for (int i = 1; i < 64; i <<= 1) s[k] += __shfl_xor(s[k], i, 64);
    if (lane == 0) sum[k][w] = s[k];
  }
  __syncthreads();
  if (threadIdx.x < 3) {
    const double* v = sum[threadIdx.x];
    float* o = threadIdx.x == 0 ? dA : threadIdx.x == 1 ? dD : db;
    if (o) o[h] = (float)(v[0] + v[1] + v[2] + v[3]);
  }
}

// dB and dC of a chunk and group from its workgroups' shares, in their order.
template <typename T>
__global__ __launch_bounds__(256) void k_scan_share_sum(ScanGradArgs a) {
  const ScanArgs& p = a.f;
  const int side = blockIdx.x & 1, unit = blockIdx.x >> 1, grp = unit % p.G, slot = unit / p.G, N = p.N;
  const ChunkPlace c = chunk_place(p.seqs, slot);
  T* out = side ? (T*)a.dB + c.b * a.sdB.b + grp * a.sdB.h + c.tok0 * a.sdB.t
                : (T*)a.dC + c.b * a.sdC.b + grp * a.sdC.h + c.tok0 * a.sdC.t;
  const int64_t pitch = side ? a.sdB.t : a.sdC.t;
  const float* in = a.shares + (((int64_t)unit * a.parts * 2 + side) * kDC) * N;
  for (int e = threadIdx.x * 4; e < c.len * N; e += 1024) {
    f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int k = 0; k < a.parts; ++k) v += *reinterpret_cast<const f32x4*>(in + (int64_t)k * 2 * kDC * N + e);
    store4(out + e / N * pitch + e % N, v[0], v[1], v[2], v[3]);
  }
}

template <typename T, int DN, bool LDS>
hipError_t launch_grads(const ScanGradArgs& a, int64_t chunks, hipStream_t s) {
  using Z = GradShape<T, DN, LDS>;
  static_assert(Z::kSmem + 11 * 1024 <= kMaxLds, "LDS");
  k_scan_grads<T, DN, LDS><<<dim3((unsigned)(chunks * a.f.G * a.parts)), 512, Z::kSmem, s>>>(a);
  if (a.parts > 1) {
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    k_scan_share_sum<T><<<dim3((unsigned)(chunks * a.f.G * 2)), 256, 0, s>>>(a);
  }
  return hipGetLastError();
}

// Regions of the workspace, in bytes, multiples of 16.
struct GradSpace {
  int seg;
  int parts, heads;
  int64_t slots, chunks, keep, gates, tokens, sums, decays, part, shares;
  int64_t total() const { return 2 * keep + gates + tokens + 2 * sums + 2 * decays + part + shares; }
};
template <typename T>
GradSpace grad_space(const ScanArgs& a) {
  GradSpace g;
  // both directions' walks run at once: half a round each (4 x 4,096 tokens x 32 heads: 256 485 us, 384 499 us, 512 505 us)
  g.seg = scan_seg<T>(a, 256, 128);
  g.slots = seg_slots(a.seqs, a.batch, g.seg);
  g.chunks = delta_slots(a.seqs, a.batch);
  const int64_t cuts = seg_cuts(a.seqs, a.batch, g.seg);
  g.gates = g.chunks * a.H * sizeof(KeptGates);
  g.tokens = g.chunks * a.H * sizeof(TokenSums<T>);
  g.keep = g.chunks * a.H * a.P * a.N * 4;
  g.sums = cuts * a.H * a.P * a.N * 4;
  g.decays = (cuts * a.H * 4 + 15) / 16 * 16;
  g.part = g.chunks * a.H * 16;
  // The heads of a group are dealt to as many workgroups as take least, by rounds of one a CU: `once` heads' time for what
  // each does once, `join` for the sum of the shares (fitted).  32 heads of 64 x 128 in one group, 300 tokens: bf16 241 -> 79
  // us, fp32 598 -> 100 us; 16 in two, 4,000 tokens: 114 -> 102, 236 -> 185; 64 in eight, 3,000 tokens, two workgroups for one:
  // bf16 223 -> 231 (not taken), fp32 524 -> 492.
  const double once = sizeof(T) == 2 ? 1.5 : 0.5, join = sizeof(T) == 2 ? 2.5 : 0.5;
  const int64_t units = std::max<int64_t>(g.chunks * a.G, 1);
  const int shared = a.H / a.G;
  double least = 0.0;
  for (int parts = 1; parts <= shared && (parts == 1 || units * parts <= 1024); ++parts) {   // shares of 512 KB N at most
    const int heads = (shared + parts - 1) / parts;
    const double cost = (double)((units * parts + 255) / 256) * (heads + once) + (parts > 1 ? join : 0.0);
    if (parts == 1 || cost < least) {
      least = cost;
      g.heads = heads;
      g.parts = (shared + heads - 1) / heads;
    }
  }
  g.shares = g.parts > 1 ? g.chunks * a.G * g.parts * 2 * kDC * a.N * 4 : 0;
  return g;
}

}  // namespace

template <typename T>
size_t scan_grad_workspace_bytes(const ScanArgs& a) {
  return (size_t)grad_space<T>(a).total();
}

template <typename T>
hipError_t launch_scan_grad(const ScanGradArgs& in, hipStream_t s) {
  ScanGradArgs a = in;
  const ScanArgs& f = a.f;
  const GradSpace g = grad_space<T>(f);
  const int64_t sequences = f.seqs.starts ? f.seqs.num : f.batch;
  char* at = f.ws;
  auto take = [&](int64_t bytes) {
    char* p = at;
    at += bytes;
    return p;
  };
  a.S = (float*)take(g.keep);
  a.dS = (float*)take(g.keep);
  a.gates = (KeptGates*)take(g.gates);
  a.sums = take(g.tokens);
  const bool cut = g.sums > 0;
  StateWalk one{f.x, f.B, f.sx, f.sB, f.S_init, nullptr, cut ? (float*)take(g.sums) : nullptr,
                cut ? (float*)take(g.decays) : nullptr, a.S, a.gates, false};
  StateWalk two{a.dO, f.C, a.sdO, f.sC, a.dS_final, a.dS_init, cut ? (float*)take(g.sums) : nullptr,
                cut ? (float*)take(g.decays) : nullptr, a.dS, nullptr, true};
  a.part = (float*)take(g.part);
  a.shares = (float*)take(g.shares);
  a.parts = g.parts;
  a.heads = g.heads;
  const int64_t join = sequences * f.H * (((int64_t)f.P * f.N / 4 + 255) / 256);
  if (sequences > 0) {
    hipError_t e = with_scan<T>(f.P, f.N, f.H / f.G, [&](auto dn, auto hw, auto pw) {
      constexpr int DN = decltype(dn)::value, HW = decltype(hw)::value, PW = decltype(pw)::value;
      hipError_t e;
      if (cut && (e = launch_states<T, DN, HW, PW, false>(f, one, &two, g.seg, g.slots, s)) != hipSuccess) return e;
      if (cut || (a.dS_init && (f.seqs.starts || f.seqs.n == 0))) {   // segments, or sequences without tokens
        k_scan_join<<<dim3((unsigned)(2 * join)), 256, 0, s>>>(f, one, nullptr, two, a.dS_init, g.seg, (int)join);
        if ((e = hipGetLastError()) != hipSuccess) return e;
      }
      if (g.chunks == 0 || f.seqs.n == 0) return hipSuccess;
      return launch_states<T, DN, HW, PW, true>(f, one, &two, g.seg, g.slots, s);
    });
    if (e != hipSuccess) return e;
  }
  const int64_t chunks = f.seqs.n > 0 ? g.chunks : 0;
  if (chunks > 0) {
    hipError_t e;
    if (f.N <= 64)
      e = launch_grads<T, 64, true>(a, chunks, s);
    else if (f.N <= 128)
      e = launch_grads<T, 128, true>(a, chunks, s);
    else
      e = launch_grads<T, 256, sizeof(T) == 2>(a, chunks, s);
    if (e != hipSuccess) return e;
    k_scan_rates<T><<<dim3((unsigned)((chunks * f.H + 3) / 4)), 256, 0, s>>>(a, chunks * f.H);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  k_scan_grad_sum<<<dim3((unsigned)f.H), 256, 0, s>>>(a.part, chunks, f.H, a.dA, a.dD, a.ddt_bias);
  return hipGetLastError();
}

#define TTT_SCAN_GRAD(T)                                        \
  template size_t scan_grad_workspace_bytes<T>(const ScanArgs&); \
  template hipError_t launch_scan_grad<T>(const ScanGradArgs&, hipStream_t);
TTT_SCAN_GRAD(bf16)
TTT_SCAN_GRAD(float)

}  // namespace ttt
