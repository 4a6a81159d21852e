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
// other, dB and dC staying in registers over them.  In bf16 kept states and all fp32 operands are pairs of bf16 values.
#include "scan_walk.hpp"

namespace ttt {
namespace {

// Rows of B or C that a chunk has: in LDS, or where that has no room (the widest fp32 states) in memory.
template <typename T, bool LDS> struct Features {
  const char* lds;
  const T* rows;
  int64_t pitch;
  int len, N;
  __device__ __forceinline__ u32x4 frag(int r, int s, int g) const {
    if constexpr (LDS) return Panels<T>::frag(lds, r, s, g);
    const int n = s * 16 + g * 4;
    return r < len && n < N ? *reinterpret_cast<const u32x4*>(rows + r * pitch + n) : (u32x4){0, 0, 0, 0};
  }
  __device__ __forceinline__ u32x4 frag_t(int tile, int s, int lane) const {
    if constexpr (LDS) return Panels<T>::frag_t(lds, tile, s, lane);
    const int n = tile * 16 + (lane & 15), r = s * 16 + (lane >> 4) * 4;
    u32x4 o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = r + i < len && n < N ? __float_as_uint((float)rows[(r + i) * pitch + n]) : 0u;
    return o;
  }
  __device__ __forceinline__ f32x4 at4(int r, int n) const {
    if constexpr (LDS) return load4((const T*)(lds + Panels<T>::at(r, n)));
    return r < len && n < N ? load4(rows + r * pitch + n) : (f32x4){0.f, 0.f, 0.f, 0.f};
  }
};

// BV: rows of P that are in LDS at a time.
template <typename T, int DN_, int BV_, bool LDS_> struct GradShape {
  static constexpr int DN = DN_, BV = BV_;
  static constexpr bool LDS = LDS_;
  using Rows = Panels<T, BV>;                                // of S and dS
  static constexpr int BVX = BV * (int)sizeof(T) < 128 ? 128 / (int)sizeof(T) : BV;
  static constexpr int SP = Mat<T>::kSplit ? 2 : 1;
  static constexpr int kB = LDS ? Panels<T>::bytes(DN) : 0, kS = Rows::bytes(DN), kX = Panels<T>::bytes(BVX);
  static constexpr int oS = 2 * kB, oD = oS + SP * kS, oX = oD + SP * kS, oY = oX + kX, kSmem = oY + kX;
};

// x summed over the four lanes that hold a token.
__device__ __forceinline__ float token_sum(float x) {
  x += __shfl_xor(x, 16, 64);
  return x + __shfl_xor(x, 32, 64);
}
__device__ __forceinline__ float dot4(f32x4 a, f32x4 b) { return a[0] * b[0] + a[1] * b[1] + a[2] * b[2] + a[3] * b[3]; }

// One workgroup of 8 waves per chunk slot and group; waves w and w + 4 have the tokens row(w, .) as their products'
// columns and half of the features (of P and of N) each.
template <typename T, int DN, int BV, bool LDS>
__global__ __launch_bounds__(512, 2) void k_scan_grads(ScanGradArgs a) {
  using M = Mat<T>;
  using Z = GradShape<T, DN, BV, LDS>;
  using Rows = typename Z::Rows;
  constexpr int NS = DN / M::KB, CS = kDC / M::KB, VS = BV / M::KB, NTH = DN / 32, PT = BV / 32, U = M::TPS;
  constexpr int PB = U == 2 && PT == 2 ? 2 : 1;              // blocks of P that are stored as one
  extern __shared__ __attribute__((aligned(16))) char smem[];
  __shared__ Gates q;
  __shared__ float rest[kDC], rowsum[kDC], colsum[kDC], qsum[2][kDC], zsum[2][kDC], usum[2][kDC], wsum[8], diag[4];
  const ScanArgs& p = a.f;
  const int id = xcd_remap(blockIdx.x, gridDim.x);
  const int grp = id % p.G, slot = id / p.G, shared = p.H / p.G;
  const ChunkPlace c = chunk_place(p.seqs, slot);
  if (c.len <= 0) {                                          // nothing of the sums over tokens
    for (int i = threadIdx.x; i < 4 * shared; i += 512) a.part[((int64_t)slot * p.H + grp * shared) * 4 + i] = 0.f;
    return;
  }
  const int wave = wave_id(), t = wave & 3, hf = wave >> 2, lane = lane_id(), m = lane & 15, g = lane >> 4;
  const int tok = M::row(t, m);                              // this lane's token
  const int64_t size = (int64_t)p.P * p.N;
  const Features<T, LDS> B{smem, (const T*)p.B + c.b * p.sB.b + grp * p.sB.h + c.tok0 * p.sB.t, p.sB.t, c.len, p.N};
  const Features<T, LDS> C{smem + Z::kB, (const T*)p.C + c.b * p.sC.b + grp * p.sC.h + c.tok0 * p.sC.t, p.sC.t, c.len, p.N};
  if constexpr (LDS) {
    PanelLoader<T, DN, 8>(p.sB.t * sizeof(T), p.N * sizeof(T)).issue(B.rows, c.len, smem);
    PanelLoader<T, DN, 8>(p.sC.t * sizeof(T), p.N * sizeof(T)).issue(C.rows, c.len, smem + Z::kB);
    wait_vm<0>();
    __syncthreads();
  }
  const PanelLoader<T, DN, 8, BV> sload(p.N * sizeof(T), p.N * sizeof(T));
  char *const Sp = smem + Z::oS, *const Dp = smem + Z::oD, *const Xp = smem + Z::oX, *const Yp = smem + Z::oY;

  // C_i . B_j: the lane's token as i with j <= i in the rows, and as j with i >= j
  f32x4 gi[CS][U], gj[CS][U];
#pragma unroll
  for (int s = 0; s < CS; ++s)
#pragma unroll
    for (int u = 0; u < U; ++u) {
      gi[s][u] = gj[s][u] = (f32x4){0.f, 0.f, 0.f, 0.f};
      const int r = M::row(s * U + u, m);
#pragma unroll
      for (int ns = 0; ns < NS; ++ns) {
        if (ns * M::KB >= p.N) continue;
        if (s < M::steps(t)) gi[s][u] = M::mma(B.frag(r, ns, g), C.frag(tok, ns, g), gi[s][u]);
        if (s >= M::first(t)) gj[s][u] = M::mma(C.frag(r, ns, g), B.frag(tok, ns, g), gj[s][u]);
      }
    }
  f32x4 dC[NTH], dB[NTH];
#pragma unroll
  for (int k = 0; k < NTH; ++k) dC[k] = dB[k] = (f32x4){0.f, 0.f, 0.f, 0.f};

  for (int h = grp * shared; h < (grp + 1) * shared; ++h) {
    const int64_t sh = (int64_t)slot * p.H + h;
    const T *S = (const T*)(a.S + sh * kept_bytes(p.P, p.N)), *dS = (const T*)(a.dS + sh * kept_bytes(p.P, p.N));
    const T* x = (const T*)p.x + c.b * p.sx.b + h * p.sx.h + c.tok0 * p.sx.t;
    const T* y = (const T*)a.dO + c.b * a.sdO.b + h * a.sdO.h + c.tok0 * a.sdO.t;
    const float D = p.D ? p.D[h] : 0.f, A = p.A[h], bias = p.dt_bias ? p.dt_bias[h] : 0.f;
    const float dt = wave == 0 && lane < c.len ? p.dt[c.b * p.sdt.b + h * p.sdt.h + (c.tok0 + lane) * p.sdt.t] : 0.f;
    f32x4 so[NTH], sx[NTH], vi[CS][U], vj[CS][U];            // S^T dO, dS^T x; dO_i . x_j, token i, token j
    u32x4 mh[CS], ml[CS];                                    // (C_i . B_j) exp(b_i - b_j), token j
#pragma unroll
    for (int k = 0; k < NTH; ++k) so[k] = sx[k] = (f32x4){0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s = 0; s < CS; ++s)
#pragma unroll
      for (int u = 0; u < U; ++u) vi[s][u] = vj[s][u] = (f32x4){0.f, 0.f, 0.f, 0.f};
    float ss = 0.f, zs = 0.f, us = 0.f;                      // <S, dS>; x_j . dS B_j; x_j . du_j
    for (int p0 = 0; p0 < p.P; p0 += BV) {
      const int rows = min(BV, p.P - p0);
      __syncthreads();                                       // the block (and the head) before has been read
#pragma unroll
      for (int k = 0; k < Z::SP; ++k) {
        sload.issue(S + k * size + (int64_t)p0 * p.N, rows, Sp + k * Z::kS);
        sload.issue(dS + k * size + (int64_t)p0 * p.N, rows, Dp + k * Z::kS);
      }
      PanelLoader<T, Z::BVX, 8>(p.sx.t * sizeof(T), rows * sizeof(T)).issue(x + p0, c.len, Xp);
      PanelLoader<T, Z::BVX, 8>(a.sdO.t * sizeof(T), rows * sizeof(T)).issue(y + p0, c.len, Yp);
      if (p0 == 0 && wave == 0) make_gates(dt, A, bias, p.softplus, c.len, &q, rest);
      wait_vm<0>();
      __syncthreads();
      if (p0 == 0) {
        const float th = q.hi[tok], tl = q.lo[tok];
#pragma unroll
        for (int s = 0; s < CS; ++s) {
          if (s < M::first(t)) continue;
          f32x4 v[U];
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const int i = M::row(s * U + u, 4 * g);
            const f32x4 ih = *reinterpret_cast<const f32x4*>(q.hi + i), il = *reinterpret_cast<const f32x4*>(q.lo + i);
#pragma unroll
            for (int e = 0; e < 4; ++e)
              v[u][e] = i + e >= tok ? gj[s][u][e] * exp2_hw((ih[e] - th) + (il[e] - tl)) : 0.f;
          }
          M::split(v, mh[s], ml[s]);
        }
      }
      u32x4 fx[VS], fy[VS];                                  // x, dO of the lane's token
#pragma unroll
      for (int s = 0; s < VS; ++s) {
        fx[s] = Panels<T>::frag(Xp, tok, s, g);
        fy[s] = Panels<T>::frag(Yp, tok, s, g);
      }
#pragma unroll
      for (int s = 0; s < CS; ++s)
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int r = M::row(s * U + u, m);
#pragma unroll
          for (int v = 0; v < VS; ++v) {
            if (s < M::steps(t)) vi[s][u] = M::mma(Panels<T>::frag(Xp, r, v, g), fy[v], vi[s][u]);
            if (s >= M::first(t)) vj[s][u] = M::mma(Panels<T>::frag(Yp, r, v, g), fx[v], vj[s][u]);
          }
        }
#pragma unroll
      for (int k = 0; k < NTH; ++k) {
        const int n = hf * NTH + k;
        if (n / U * M::KB >= p.N) continue;
#pragma unroll
        for (int v = 0; v < VS; ++v)
#pragma unroll
          for (int z = Z::SP - 1; z >= 0; --z) {
            so[k] = M::mma(Rows::frag_t(Sp + z * Z::kS, n, v, lane), fy[v], so[k]);
            sx[k] = M::mma(Rows::frag_t(Dp + z * Z::kS, n, v, lane), fx[v], sx[k]);
          }
      }
      // du of the lane's token, rows of P
      const float f = rest[tok], r = q.r[tok];
      f32x4 du[PT];
#pragma unroll
      for (int k = 0; k < PT; ++k) {
        const int pt = hf * PT + k, row = M::row(pt, m);
        du[k] = (f32x4){0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int ns = 0; ns < NS; ++ns) {
          if (ns * M::KB >= p.N) continue;
          const u32x4 b = B.frag(tok, ns, g);
#pragma unroll
          for (int z = Z::SP - 1; z >= 0; --z) du[k] = M::mma(Rows::frag(Dp + z * Z::kS, row, ns, g), b, du[k]);
        }
        du[k] *= f;
        const f32x4 xt = load4((const T*)(Xp + Panels<T>::at(tok, M::row(pt, 4 * g))));
        zs += dot4(du[k], xt);
#pragma unroll
        for (int s = 0; s < CS; ++s) {
          if (s < M::first(t)) continue;
          const u32x4 o = Panels<T>::frag_t(Yp, pt, s, lane);
          if (M::kSplit) du[k] = M::mma(o, ml[s], du[k]);
          du[k] = M::mma(o, mh[s], du[k]);
        }
        us += dot4(du[k], xt);
      }
      if (tok < c.len) {
        T* o = (T*)a.dx + c.b * a.sdx.b + h * a.sdx.h + (int64_t)(c.tok0 + tok) * a.sdx.t + p0;
#pragma unroll
        for (int k = 0; k < PT; k += PB) {
          const int pp = M::row(hf * PT + k, 4 * g);
          if (pp >= rows) continue;
          f32x4 v[PB];
#pragma unroll
          for (int e = 0; e < PB; ++e) v[e] = r * du[k + e] + D * load4((const T*)(Yp + Panels<T>::at(tok, pp + 4 * e)));
          if constexpr (PB == 2)
            *reinterpret_cast<u32x4*>(o + pp) = M::frag(v);
          else
            store4(o + pp, v[0][0], v[0][1], v[0][2], v[0][3]);
        }
      }
      // rows past the block's are zero in LDS; the same slots of all panels hold the same element
      for (int at = threadIdx.x * 16; at < Z::kS; at += 512 * 16) {
        const u32x4 s0 = *reinterpret_cast<const u32x4*>(Sp + at), d0 = *reinterpret_cast<const u32x4*>(Dp + at);
        if constexpr (M::kSplit) {
          float u[8], v[8], u1[8], v1[8];
          unpack8(s0, u);
          unpack8(d0, v);
          unpack8(*reinterpret_cast<const u32x4*>(Sp + Z::kS + at), u1);
          unpack8(*reinterpret_cast<const u32x4*>(Dp + Z::kS + at), v1);
#pragma unroll
          for (int j = 0; j < 8; ++j) ss += (u[j] + u1[j]) * (v[j] + v1[j]);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) ss += __uint_as_float(s0[j]) * __uint_as_float(d0[j]);
        }
      }
    }
    // W and the tokens' products with it
    const float th = q.hi[tok], tl = q.lo[tok], tr = q.r[tok], eb = q.eb[tok], wt = q.w[tok];
    float rs = 0.f, cs = 0.f, trace = 0.f, qs = 0.f;
#pragma unroll
    for (int s = 0; s < CS; ++s) {
      if (s < M::steps(t)) {
        f32x4 v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int j = M::row(s * U + u, 4 * g);
          const f32x4 jh = *reinterpret_cast<const f32x4*>(q.hi + j), jl = *reinterpret_cast<const f32x4*>(q.lo + j),
                      jr = *reinterpret_cast<const f32x4*>(q.r + j);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            v[u][e] = j + e <= tok ? vi[s][u][e] * exp2_hw((th - jh[e]) + (tl - jl[e])) * jr[e] : 0.f;
            if (j + e < tok) rs += v[u][e] * gi[s][u][e];
            if (j + e == tok) trace += vi[s][u][e];
          }
        }
        u32x4 hi, lo;
        M::split(v, hi, lo);
#pragma unroll
        for (int k = 0; k < NTH; ++k) {
          const int n = hf * NTH + k;
          if (n / U * M::KB >= p.N) continue;
          const u32x4 b = B.frag_t(n, s, lane);
          if (M::kSplit) dC[k] = M::mma(b, lo, dC[k]);
          dC[k] = M::mma(b, hi, dC[k]);
        }
      }
      if (s >= M::first(t)) {
        f32x4 v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int i = M::row(s * U + u, 4 * g);
          const f32x4 ih = *reinterpret_cast<const f32x4*>(q.hi + i), il = *reinterpret_cast<const f32x4*>(q.lo + i);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            v[u][e] = i + e >= tok ? vj[s][u][e] * exp2_hw((ih[e] - th) + (il[e] - tl)) * tr : 0.f;
            if (i + e > tok) cs += v[u][e] * gj[s][u][e];
          }
        }
        u32x4 hi, lo;
        M::split(v, hi, lo);
#pragma unroll
        for (int k = 0; k < NTH; ++k) {
          const int n = hf * NTH + k;
          if (n / U * M::KB >= p.N) continue;
          const u32x4 b = C.frag_t(n, s, lane);
          if (M::kSplit) dB[k] = M::mma(b, lo, dB[k]);
          dB[k] = M::mma(b, hi, dB[k]);
        }
      }
    }
#pragma unroll
    for (int k = 0; k < NTH; ++k) {
      const int n = M::row(hf * NTH + k, 4 * g);
      if ((hf * NTH + k) / U * M::KB >= p.N) continue;
      qs += dot4(so[k], C.at4(tok, n));
      dC[k] += eb * so[k];
      dB[k] += wt * sx[k];
    }
    rs = token_sum(rs);
    cs = token_sum(cs);
    qs = token_sum(qs) * eb;
    zs = token_sum(zs) * tr;
    us = token_sum(us);
    trace = token_sum(trace);
#pragma unroll
    for (int i = 1; i < 16; i <<= 1) trace += __shfl_xor(trace, i, 64);
#pragma unroll
    for (int i = 1; i < 64; i <<= 1) ss += __shfl_xor(ss, i, 64);
    if (g == 0) {
      if (hf == 0) {
        rowsum[tok] = rs;
        colsum[tok] = cs;
      }
      qsum[hf][tok] = qs;
      zsum[hf][tok] = zs;
      usum[hf][tok] = us;
    }
    if (lane == 0) {
      wsum[wave] = ss;
      if (hf == 0) diag[t] = trace;
    }
    __syncthreads();
    if (wave == 0) {                                         // lane: token
      double R = (double)colsum[lane] - rowsum[lane], zq = zsum[0][lane] + zsum[1][lane], qq = qsum[0][lane] + qsum[1][lane];
      const double r0 = R, z0 = zq;
#pragma unroll
      for (int i = 1; i < 64; i <<= 1) {
        const double up = __shfl_up(R, i, 64), uz = __shfl_up(zq, i, 64), dq = __shfl_down(qq, i, 64);
        if (lane >= i) {
          R += up;
          zq += uz;
        }
        if (lane + i < 64) qq += dq;
      }
      float dots = 0.f, tr4 = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) dots += wsum[i];
#pragma unroll
      for (int i = 0; i < 4; ++i) tr4 += diag[i];
      // pairs that token t's decay lies between: those of t - 1, less row t - 1's, and column t - 1's
      const float dg = (float)((R - r0) + (zq - z0) + qq) + q.eb[kDC - 1] * dots;
      const float raw = dt + bias, slope = p.softplus ? 1.f / (1.f + expf(-raw)) : 1.f;
      const bool in = lane < c.len;
      const float ddt = in ? (usum[0][lane] + usum[1][lane] + A * dg) * slope : 0.f;
      if (in) a.ddt[c.b * a.sddt.b + h * a.sddt.h + (c.tok0 + lane) * a.sddt.t] = ddt;
      double sa = in ? (double)dg * q.r[lane] : 0.0, sb = ddt;
#pragma unroll
      for (int i = 1; i < 64; i <<= 1) {
        sa += __shfl_xor(sa, i, 64);
        sb += __shfl_xor(sb, i, 64);
      }
      if (lane == 0) *reinterpret_cast<f32x4*>(a.part + sh * 4) = (f32x4){(float)sa, tr4, (float)sb, 0.f};
    }
  }
  if (tok < c.len) {
    T* oC = (T*)a.dC + c.b * a.sdC.b + grp * a.sdC.h + (int64_t)(c.tok0 + tok) * a.sdC.t;
    T* oB = (T*)a.dB + c.b * a.sdB.b + grp * a.sdB.h + (int64_t)(c.tok0 + tok) * a.sdB.t;
#pragma unroll
    for (int k = 0; k < NTH; k += U) {
      const int n = M::row(hf * NTH + k, 4 * g);
      if (n >= p.N) continue;
      *reinterpret_cast<u32x4*>(oC + n) = M::frag(&dC[k]);
      *reinterpret_cast<u32x4*>(oB + n) = M::frag(&dB[k]);
    }
  }
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

template <typename T, int DN, int BV, bool LDS>
hipError_t launch_grads(const ScanGradArgs& a, int64_t chunks, hipStream_t s) {
  using Z = GradShape<T, DN, BV, LDS>;
  static_assert(Z::kSmem + 5 * 1024 <= kMaxLds, "LDS");
  k_scan_grads<T, DN, BV, LDS><<<dim3((unsigned)(chunks * a.f.G)), 512, Z::kSmem, s>>>(a);
  return hipGetLastError();
}

// Regions of the workspace, in bytes, multiples of 16.
struct GradSpace {
  int seg;
  int64_t slots, chunks, keep, sums, decays, part;
  int64_t total() const { return 2 * keep + 2 * sums + 2 * decays + part; }
};
template <typename T>
GradSpace grad_space(const ScanArgs& a) {
  GradSpace g;
  g.seg = scan_seg<T>(a);
  g.slots = seg_slots(a.seqs, a.batch, g.seg);
  g.chunks = delta_slots(a.seqs, a.batch);
  const bool cut = g.seg < a.seqs.n;
  g.keep = g.chunks * a.H * kept_bytes(a.P, a.N);
  g.sums = cut ? g.slots * a.H * a.P * a.N * 4 : 0;
  g.decays = cut ? (g.slots * a.H * 4 + 15) / 16 * 16 : 0;
  g.part = g.chunks * a.H * 16;
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
  a.S = take(g.keep);
  a.dS = take(g.keep);
  const bool cut = g.sums > 0;
  StateWalk one{f.x, f.B, f.sx, f.sB, f.S_init, nullptr, cut ? (float*)take(g.sums) : nullptr,
                cut ? (float*)take(g.decays) : nullptr, a.S, false};
  StateWalk two{a.dO, f.C, a.sdO, f.sC, a.dS_final, a.dS_init, cut ? (float*)take(g.sums) : nullptr,
                cut ? (float*)take(g.decays) : nullptr, a.dS, true};
  a.part = (float*)take(g.part);
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
    constexpr bool wide = sizeof(T) == 2;
    hipError_t e;
    if (f.N <= 64)
      e = launch_grads<T, 64, wide ? 64 : 32, true>(a, chunks, s);
    else if (f.N <= 128)
      e = launch_grads<T, 128, wide ? 64 : 32, true>(a, chunks, s);
    else
      e = launch_grads<T, 256, 32, wide>(a, chunks, s);
    if (e != hipSuccess) return e;
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
