// The selective scan over whole sequences for gfx950; the mathematics and the operands are in scan.hpp.
#include "scan_walk.hpp"

namespace ttt {
namespace {

// The walk over a segment's chunks with outputs.  sums: every cut's and head's [P, N] state, or null: sequences are one
// segment.  A chunk's turn:
//   C B^T by fragments, decayed for each head (D on its diagonal, so that D x comes with the product), to LDS
//   S C from the state's two parts, then S' with x and B: B and C have been read, the next chunk's come
//   the decayed C B^T times x, the outputs packed; they are stored in the next turn, behind its barrier, so that no wait
//   for loads waits for them
// Bound by the chain of a chunk on two waves a SIMD (registers): 65,536 tokens x 64 heads of 64 x 128 in bf16 take 72 % of
// the call's time (traced: 523 us at the least), the matrix cores busy for 47 % of its cycles; a block of columns less a wave
// and four waves a SIMD spill and take 1,469 us.
template <typename T, int DN, int HW, int PW>
__global__ __launch_bounds__(64 * HW * PW, 2) void k_scan(ScanArgs a, int seg, int slots, const float* sums) {
#if __HIP_DEVICE_COMPILE__
  using Z = ScanShape<T, DN, HW, PW>;
  using M = Mat<T>;
  constexpr int CT = Z::CT, NT = Z::NT, NS = Z::NS, CS = Z::CS, W = Z::W, U = M::TPS;
  constexpr int PB = CT == 2 && U == 2 ? 2 : 1, CB = CT / PB;  // blocks of P that are stored as one; of those
  constexpr int FW = (M::kTri + W - 1) / W;                // fragments of C B^T a wave makes: w, w + W, ..
  // Where that gives some waves one more than the others, those E fragments are dealt out by heads: a wave makes W + w % E
  // for the heads with its w / E (of W / E).
  constexpr int E = M::kTri - W, Q = E > 0 && E < W ? W / E : 1;
  constexpr bool kDealt = Q > 1;
  extern __shared__ __attribute__((aligned(16))) char smem[];
  __shared__ Gates gates[2][HW];
  char *const Bp = smem, *const Cp = Bp + Z::kB, *const Xp = Cp + Z::kB, *const Mp = Xp + HW * Z::kX;
  const int shared = a.H / a.G, parts = (a.P + Z::cols - 1) / Z::cols;
  ScanPlace at;
  if (!scan_place(blockIdx.x, slots, a.G, shared, parts, HW, &at)) return;
  const SegPlace sp = seg_place(a.seqs, seg, at.slot);
  if (sp.len <= 0) return;
  const int w = wave_id(), hw = w / PW, pw = w % PW, lane = lane_id(), m = lane & 15, g = lane >> 4;
  const bool mine = at.head0 + hw < shared;                // a head of the group
  const int h = at.group * shared + min(at.head0 + hw, shared - 1);
  const int p0 = at.part * Z::cols, tile0 = (p0 >> 4) + pw * CT;
  const bool busy = mine && tile0 * 16 < a.P;              // rows of its state
  const int64_t size = (int64_t)a.P * a.N;

  const LaneAt<T> L(lane);
  const Split<T> split(lane);
  StateRows<T, CT, NT> S;
  S.zero();
  if (busy) {
    if (!sp.first)
      S.load(sums + ((int64_t)(sp.cut - 1) * a.H + h) * size, tile0, a.P, a.N);
    else if (a.S_init)
      S.load(a.S_init + ((int64_t)sp.seq * a.H + h) * size, tile0, a.P, a.N);
  }

  const TileLoader<T, DN, W> bload(a.sB.t * sizeof(T), a.N * sizeof(T)), cload(a.sC.t * sizeof(T), a.N * sizeof(T));
  const TileLoader<T, Z::DX, PW> xload(a.sx.t * sizeof(T), min(a.P - p0, Z::cols) * sizeof(T));
  const T* B = (const T*)a.B + sp.b * a.sB.b + at.group * a.sB.h + sp.tok0 * a.sB.t;
  const T* C = (const T*)a.C + sp.b * a.sC.b + at.group * a.sC.h + sp.tok0 * a.sC.t;
  const T* x = (const T*)a.x + sp.b * a.sx.b + h * a.sx.h + sp.tok0 * a.sx.t + p0;
  T* O = (T*)a.O + sp.b * a.sO.b + h * a.sO.h + sp.tok0 * a.sO.t;
  char *const Xh = Xp + hw * Z::kX, *const Mh = Mp + hw * Z::kM;
  // the heads' gates are made by the last waves, which have fewer fragments
  const int gw = w - (W - HW), gh = at.group * shared + min(at.head0 + max(gw, 0), shared - 1);
  const float* dt = a.dt + sp.b * a.sdt.b + gh * a.sdt.h + sp.tok0 * a.sdt.t;
  const float A = a.A[gh], bias = a.dt_bias ? a.dt_bias[gh] : 0.f;
  const unsigned pitch = (unsigned)(a.sO.t * sizeof(T));
  float D[HW];
#pragma unroll
  for (int i = 0; i < HW; ++i) D[i] = a.D ? a.D[at.group * shared + min(at.head0 + i, shared - 1)] : 0.f;
  float dt_next = 0.f;
  if (gw >= 0 && lane < sp.len) dt_next = dt[lane * a.sdt.t];
  auto make = [&](int t, int turn) __attribute__((always_inline)) {
    if (gw < 0) return;
    const LaneGates v = make_gates(dt_next, A, bias, a.softplus, min(kDC, sp.len - t));
    put_gates<T>(v, &gates[turn][gw]);
    if (t + kDC + lane < sp.len) dt_next = dt[(t + kDC + lane) * a.sdt.t];
  };
  u32x4 out[CB][4];                                        // O of the chunk before, of token row(t, m)
  auto store = [&](int t0) __attribute__((always_inline)) {
    const __amdgpu_buffer_rsrc_t rs = rows_rsrc(O + t0 * a.sO.t);
    const int len = min(kDC, sp.len - t0);
#pragma unroll
    for (int c = 0; c < CB; ++c) {
      const int p = state_row<T, CT>(tile0 + c * PB, 4 * g);
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const int i = M::row(t, m);
        const unsigned off = p < a.P && i < len ? i * pitch + p * (unsigned)sizeof(T) : kOOB;
        if constexpr (PB == U)
          __builtin_amdgcn_raw_buffer_store_b128(out[c][t], rs, off, 0, 0);
        else
          __builtin_amdgcn_raw_buffer_store_b64((u32x2){out[c][t][0], out[c][t][1]}, rs, off, 0, 0);
      }
    }
  };

  bload.issue(B, min(kDC, sp.len), Bp);
  cload.issue(C, min(kDC, sp.len), Cp);
  if (mine) xload.issue(x, min(kDC, sp.len), Xh);
  make(0, 0);
  int turn = 0;
  for (int t0 = 0; t0 < sp.len; t0 += kDC, turn ^= 1) {
    const int next = t0 + kDC, nlen = min(kDC, sp.len - next);
    wait_vm<0>();
    __syncthreads();                                       // the chunk and its gates are there
    if (busy && t0 > 0) store(t0 - kDC);
    u32x4 xf[CS][CT];
#pragma unroll
    for (int s = 0; s < CS; ++s)
#pragma unroll
      for (int c = 0; c < CT; ++c) xf[s][c] = state_cols<T, CT>(L, Xh, pw * CT + c, s);
    auto fragment = [&](int k) { return kDealt && k > 0 ? W + w % E : w + k * W; };
    // C B^T of a fragment's tokens row(t, .) and those before them; all of a wave's fragments at once
    auto decayed = [&](auto count) __attribute__((always_inline)) {
      constexpr int NF = decltype(count)::value;
      int ft[NF], fs[NF], fi[NF];
      f32x4 d[NF][U];
#pragma unroll
      for (int k = 0; k < NF; ++k) {
        tri_place<T>(fragment(k), &ft[k], &fs[k]);
        fi[k] = M::row(ft[k], m);
#pragma unroll
        for (int u = 0; u < U; ++u) d[k][u] = (f32x4){0.f, 0.f, 0.f, 0.f};
      }
#pragma unroll
      for (int ns = 0; ns < NS; ++ns) {
        if (past<T, DN>(ns * M::KB, a.N)) break;
#pragma unroll
        for (int k = 0; k < NF; ++k) {
          const u32x4 c = L.frag(Cp, ft[k], ns);
#pragma unroll
          for (int u = 0; u < U; ++u) d[k][u] = M::mma(L.frag(Bp, fs[k] * U + u, ns), c, d[k][u]);
        }
      }
#pragma unroll
      for (int hd = 0; hd < HW; ++hd) {
        const Gates& q = gates[turn][hd];
        const bool parts = two_part_gates<T>(q);
#pragma unroll
        for (int k = 0; k < NF; ++k) {
          if (kDealt && k > 0 && hd % Q != w / E) continue;
          const int i = fi[k];
          const float bh = q.hi[i];
          int behind = i - M::row(fs[k] * U, 4 * g);       // tokens of the lane's row of d before i
          asm volatile("" : "+v"(behind));                 // (compared again for every chunk, not kept in masks)
          f32x4 v[U];
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const int j = M::row(fs[k] * U + u, 4 * g);
            const f32x4 jh = *reinterpret_cast<const f32x4*>(q.hi + j), jr = *reinterpret_cast<const f32x4*>(q.r + j);
            f32x4 x;
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = bh - jh[e];
            if (parts) {
              const f32x4 jl = *reinterpret_cast<const f32x4*>(q.lo + j);
              const float bl = q.lo[i];
#pragma unroll
              for (int e = 0; e < 4; ++e) x[e] += bl - jl[e];
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float z = d[k][u][e] * exp2_hw(x[e]) * jr[e];
              v[u][e] = 4 * u + e < behind ? z : 4 * u + e == behind ? z + D[hd] : 0.f;
            }
          }
          u32x4 hi, lo;
          split.two(v, hi, lo);
          char* to = Mp + hd * Z::kM + fragment(k) * 1024 + lane * 16;
          *reinterpret_cast<u32x4*>(to) = hi;
          if (M::kSplit) *reinterpret_cast<u32x4*>(to + M::kTri * 1024) = lo;
        }
      }
    };
    if (kDealt ? w / E < HW : M::kTri % W == 0 || w < M::kTri % W)
      decayed(std::integral_constant<int, FW>());
    else if constexpr (FW > 1)
      decayed(std::integral_constant<int, FW - 1>());
    __syncthreads();                                       // it is there, x has been read
    if (mine && next < sp.len) xload.issue(x + next * a.sx.t, nlen, Xh);
    const Gates& q = gates[turn][hw];
    f32x4 o[CT][4];
    __builtin_amdgcn_s_setprio(1);                         // the products before the other waves' decays: 3 %
    if (busy) {
      if (t0 == 0 && sp.first && q.eb[0] == 0.f) S.zero(); // emptied by its first token: S_init is not looked at
#pragma unroll
      for (int c = 0; c < CT; ++c)
#pragma unroll
        for (int t = 0; t < 4; ++t) o[c][t] = (f32x4){0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int ns = 0; ns < NS; ++ns) {
        if (past<T, DN>(ns * M::KB, a.N)) break;
        u32x4 hi[CT], lo[CT];
#pragma unroll
        for (int c = 0; c < CT; ++c) split.two(&S.s[c][ns * U], hi[c], lo[c]);
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const u32x4 f = L.halves(Cp, t, ns);
#pragma unroll
          for (int c = 0; c < CT; ++c) {
            if (M::kSplit) o[c][t] = M::mma(lo[c], f, o[c][t]);
            o[c][t] = M::mma(hi[c], f, o[c][t]);
          }
        }
      }
      S.decay(q.eb[kDC - 1]);
#pragma unroll
      for (int s = 0; s < CS; ++s) S.add(L, split, xf[s], Bp, s, q.w + s * M::KB + g * (M::KB / 4), a.N);
    }
    __builtin_amdgcn_s_setprio(0);
    __syncthreads();                                       // B and C have been read
    if (next < sp.len) {
      bload.issue(B + next * a.sB.t, nlen, Bp);
      cload.issue(C + next * a.sC.t, nlen, Cp);
      make(next, turn ^ 1);
    }
    if (busy) {
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const float e = q.eb[M::row(t, m)];
#pragma unroll
        for (int c = 0; c < CT; ++c) o[c][t] *= e;
#pragma unroll
        for (int s = 0; s < CS; ++s) {
          if (s >= M::steps(t)) continue;
          const char* f = Mh + M::tri(t, s) * 1024 + lane * 16;
          const u32x4 hi = *reinterpret_cast<const u32x4*>(f);
          if constexpr (M::kSplit) {
            const u32x4 lo = *reinterpret_cast<const u32x4*>(f + M::kTri * 1024);
#pragma unroll
            for (int c = 0; c < CT; ++c) o[c][t] = M::mma(xf[s][c], lo, o[c][t]);
          }
#pragma unroll
          for (int c = 0; c < CT; ++c) o[c][t] = M::mma(xf[s][c], hi, o[c][t]);
        }
        // p = row(tile0 + c, 4 g + 0..3) of token row(t, m): bf16 pairs of blocks are 8 together
#pragma unroll
        for (int c = 0; c < CB; ++c) {
          if constexpr (PB == U) {
            f32x4 v[PB];
#pragma unroll
            for (int k = 0; k < PB; ++k) v[k] = o[c * PB + k][t];
            out[c][t] = M::frag(v);
          } else {                                         // one block of bf16: 4 together
            out[c][t] = (u32x4){pack2_bf16(o[c][t][0], o[c][t][1]), pack2_bf16(o[c][t][2], o[c][t][3]), 0, 0};
          }
        }
      }
    }
  }
  if (busy) {
    store((sp.len - 1) / kDC * kDC);
    if (sp.last) S.store(a.S_final + ((int64_t)sp.seq * a.H + h) * size, tile0, a.P, a.N);
  }
#endif
}

template <typename T, int DN, int HW, int PW>
hipError_t launch(const ScanArgs& a, int seg, int64_t slots, const float* sums, hipStream_t s) {
  using Z = ScanShape<T, DN, HW, PW>;
  constexpr int smem = 2 * Z::kB + HW * (Z::kX + Z::kM);
  static_assert(smem + 2 * (int)sizeof(Gates) * HW <= kMaxLds, "LDS");
  const int64_t shared = a.H / a.G;
  const int64_t per = (shared + HW - 1) / HW * ((a.P + Z::cols - 1) / Z::cols);
  k_scan<T, DN, HW, PW><<<dim3((unsigned)scan_grid(slots * a.G, per)), 64 * HW * PW, smem, s>>>(a, seg, (int)slots, sums);
  return hipGetLastError();
}

// 512 workgroups are on the chip at once: one round of them, by the tokens in all (the ends of packed sequences come on top:
// 12 prompts of 16,456 tokens have 576; longer segments for them gained for one long prompt and lost for equal ones).
// 65,536 tokens x 64 heads: 384 860 us, 512 707 us, 768 794 us, 1024 745 us.  Whole sequences save the pass over the
// segments' sums: 8 x 64 heads, 256 workgroups, take 91 us for 1,024 tokens each (in two segments 109 us) and 341 us for
// 4,096 (284 us), 12 x 64 heads 425 us for 4,096 (490 us).
template <typename T>
int forward_seg(const ScanArgs& a) {
  return scan_seg<T>(a, 512, a.seqs.n < 2048 ? 256 : 384);
}

}  // namespace

template <typename T>
size_t scan_workspace_bytes(const ScanArgs& a) {
  const int seg = forward_seg<T>(a);
  if (seg >= a.seqs.n) return 0;
  const int64_t sh = seg_cuts(a.seqs, a.batch, seg) * a.H;
  return (size_t)sh * a.P * a.N * 4 + (size_t)((sh * 4 + 15) / 16 * 16);
}

template <typename T>
hipError_t launch_scan(const ScanArgs& a, hipStream_t s) {
  const int seg = forward_seg<T>(a);
  const int64_t slots = seg_slots(a.seqs, a.batch, seg), sequences = a.seqs.starts ? a.seqs.num : a.batch;
  if (sequences == 0) return hipSuccess;
  const int64_t join = sequences * a.H * (((int64_t)a.P * a.N / 4 + 255) / 256);
  StateWalk k{};
  k.rows = a.x;
  k.cols = a.B;
  k.srows = a.sx;
  k.scols = a.sB;
  k.start = a.S_init;
  if (seg < a.seqs.n) {
    k.sums = (float*)a.ws;
    k.decays = k.sums + seg_cuts(a.seqs, a.batch, seg) * a.H * a.P * a.N;
  }
  return with_scan<T>(a.P, a.N, a.H / a.G, [&](auto dn, auto hw, auto pw) {
    constexpr int DN = decltype(dn)::value, HW = decltype(hw)::value, PW = decltype(pw)::value;
    hipError_t e;
    if (k.sums && (e = launch_states<T, DN, HW, PW, false>(a, k, nullptr, seg, slots, s)) != hipSuccess) return e;
    if (k.sums || a.seqs.starts || a.seqs.n == 0) {        // sequences of segments, or some without tokens
      k_scan_join<<<dim3((unsigned)join), 256, 0, s>>>(a, k, a.S_final, k, nullptr, seg, (int)join);
      if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    if (a.seqs.n == 0) return hipSuccess;
    return launch<T, DN, HW, PW>(a, seg, slots, k.sums, s);
  });
}

#define TTT_SCAN(T)                                                  \
  template size_t scan_workspace_bytes<T>(const ScanArgs&);          \
  template hipError_t launch_scan<T>(const ScanArgs&, hipStream_t);
TTT_SCAN(bf16)
TTT_SCAN(float)

}  // namespace ttt
