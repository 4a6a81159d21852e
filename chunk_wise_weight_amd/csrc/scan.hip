// The selective scan over whole sequences for gfx950; the mathematics and the operands are in scan.hpp.
#include "scan_walk.hpp"

namespace ttt {
namespace {

// The walk over a segment's chunks with outputs.  sums: every slot's and head's [P, N] state before the segment, or
// null: sequences are one segment.
template <typename T, int DN, int HW, int PW>
__global__ __launch_bounds__(64 * HW * PW, 2) void k_scan(ScanArgs a, int seg, int slots, const float* sums) {
  using Z = ScanShape<T, DN, HW, PW>;
  using M = Mat<T>;
  constexpr int CT = Z::CT, NT = Z::NT, NS = Z::NS, CS = Z::CS, W = Z::W;
  extern __shared__ __attribute__((aligned(16))) char smem[];
  __shared__ Gates gates[HW];
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
  const int64_t sh = (int64_t)at.slot * a.H + h, size = (int64_t)a.P * a.N;

  LaneAt<T> L(lane);
  L.keep();
  StateRows<T, CT, NT> S;
  S.zero();
  if (mine) {
    if (sums)
      S.load(sums + sh * size, tile0, a.P, a.N);
    else if (a.S_init)
      S.load(a.S_init + ((int64_t)sp.seq * a.H + h) * size, tile0, a.P, a.N);
  }

  const PanelLoader<T, DN, W> bload(a.sB.t * sizeof(T), a.N * sizeof(T)), cload(a.sC.t * sizeof(T), a.N * sizeof(T));
  const PanelLoader<T, Z::DX, PW> xload(a.sx.t * sizeof(T), min(a.P - p0, Z::cols) * sizeof(T));
  const T* B = (const T*)a.B + sp.b * a.sB.b + at.group * a.sB.h + sp.tok0 * a.sB.t;
  const T* C = (const T*)a.C + sp.b * a.sC.b + at.group * a.sC.h + sp.tok0 * a.sC.t;
  const T* x = (const T*)a.x + sp.b * a.sx.b + h * a.sx.h + sp.tok0 * a.sx.t + p0;
  T* O = (T*)a.O + sp.b * a.sO.b + h * a.sO.h + sp.tok0 * a.sO.t;
  char *const Xh = Xp + hw * Z::kX, *const Mh = Mp + hw * Z::kM;
  // the gates of head head0 + w are made by wave w
  const int gh = at.group * shared + min(at.head0 + w, shared - 1);
  const float* dt = a.dt + sp.b * a.sdt.b + gh * a.sdt.h + sp.tok0 * a.sdt.t;
  const float A = a.A[gh], bias = a.dt_bias ? a.dt_bias[gh] : 0.f, D = a.D ? a.D[h] : 0.f;
  float dt_next = 0.f;
  if (w < HW && lane < sp.len) dt_next = dt[lane * a.sdt.t];

  for (int t0 = 0; t0 < sp.len; t0 += kDC) {
    const int len = min(kDC, sp.len - t0);
    if (t0 > 0) __syncthreads();                           // the chunk before has been read
    bload.issue(B + t0 * a.sB.t, len, Bp);
    cload.issue(C + t0 * a.sC.t, len, Cp);
    if (mine) xload.issue(x + t0 * a.sx.t, len, Xh);
    if (w < HW) {
      make_gates(dt_next, A, bias, a.softplus, len, &gates[w]);
      if (t0 + kDC + lane < sp.len) dt_next = dt[(t0 + kDC + lane) * a.sdt.t];
    }
    wait_vm<0>();
    __syncthreads();
    {
      // C B^T once for the workgroup's heads, by fragments (t, s) of tokens row(t, .) and those before them
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int s = 0; s < CS; ++s) {
          if (s >= M::steps(t) || M::tri(t, s) % W != w) continue;
          const int i = M::row(t, m);
          f32x4 d[M::TPS];
#pragma unroll
          for (int u = 0; u < M::TPS; ++u) d[u] = (f32x4){0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int ns = 0; ns < NS; ++ns) {
            if (NS > 128 / M::KB && ns % (64 / M::KB) == 0 && ns * M::KB >= a.N) break;
            const u32x4 c = L.frag(Cp, t, ns);
#pragma unroll
            for (int u = 0; u < M::TPS; ++u) d[u] = M::mma(L.frag(Bp, s * M::TPS + u, ns), c, d[u]);
          }
          for (int k = 0; k < HW; ++k) {
            const Gates& q = gates[k];
            const float bh = q.hi[i], bl = q.lo[i];
            f32x4 v[M::TPS];
#pragma unroll
            for (int u = 0; u < M::TPS; ++u) {
              const int j = M::row(s * M::TPS + u, 4 * g);
              const f32x4 jh = *reinterpret_cast<const f32x4*>(q.hi + j), jl = *reinterpret_cast<const f32x4*>(q.lo + j),
                          jr = *reinterpret_cast<const f32x4*>(q.r + j);
#pragma unroll
              for (int e = 0; e < 4; ++e)
                v[u][e] = j + e <= i ? d[u][e] * exp2_hw((bh - jh[e]) + (bl - jl[e])) * jr[e] : 0.f;
            }
            u32x4 hi, lo;
            M::split(v, hi, lo);
            char* f = Mp + k * Z::kM + M::tri(t, s) * 1024 + lane * 16;
            *reinterpret_cast<u32x4*>(f) = hi;
            if (M::kSplit) *reinterpret_cast<u32x4*>(f + M::kTri * 1024) = lo;
          }
        }
      __syncthreads();
    }
    if (!mine) continue;
    const Gates& q = gates[hw];
    if (t0 == 0 && sp.first && q.eb[0] == 0.f) S.zero();   // emptied by its first token: S_init is not looked at
    u32x4 xf[CS][CT];
#pragma unroll
    for (int c = 0; c < CT; ++c)
#pragma unroll
      for (int s = 0; s < CS; ++s) xf[s][c] = L.frag_t(Xh, pw * CT + c, s);
    {
      f32x4 o[CT][4];
#pragma unroll
      for (int c = 0; c < CT; ++c)
#pragma unroll
        for (int t = 0; t < 4; ++t) o[c][t] = (f32x4){0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int ns = 0; ns < NS; ++ns) {
        if (NS > 128 / M::KB && ns % (64 / M::KB) == 0 && ns * M::KB >= a.N) break;
        {
          u32x4 sh_[CT], sl[CT];
#pragma unroll
          for (int c = 0; c < CT; ++c) M::split(&S.s[c][ns * M::TPS], sh_[c], sl[c]);
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            const u32x4 f = L.frag(Cp, t, ns);
#pragma unroll
            for (int c = 0; c < CT; ++c) {
              if (M::kSplit) o[c][t] = M::mma(sl[c], f, o[c][t]);
              o[c][t] = M::mma(sh_[c], f, o[c][t]);
            }
          }
        }
      }
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
      }
      // o[c][t]: p = row(tile0 + c, 4 g + 0..3) of token row(t, m); a pair of blocks has 8 of bf16 together
      constexpr int PB = CT == 2 && M::TPS == 2 ? 2 : 1;   // blocks that are stored as one
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const int i = M::row(t, m);
        if (i >= len) continue;
        T* out = O + (t0 + i) * a.sO.t;
#pragma unroll
        for (int c = 0; c < CT; c += PB) {
          const int p = M::row(tile0 + c, 4 * g);
          if (p >= a.P) continue;
          f32x4 v[PB];
#pragma unroll
          for (int k = 0; k < PB; ++k) {
            v[k] = o[c + k][t];
            if (a.D) v[k] += D * L.at4(Xh, t, pw * CT + c + k);
          }
          if constexpr (PB == 2)
            *reinterpret_cast<u32x4*>(out + p) = M::frag(v);
          else
            store4(out + p, v[0][0], v[0][1], v[0][2], v[0][3]);
        }
      }
    }
    S.decay(q.eb[kDC - 1]);
#pragma unroll
    for (int s = 0; s < CS; ++s) S.add(L, xf[s], Bp, s, q.w + s * M::KB + g * (M::KB / 4), a.N);
  }
  if (mine && sp.last) S.store(a.S_final + ((int64_t)sp.seq * a.H + h) * size, tile0, a.P, a.N);
}

template <typename T, int DN, int HW, int PW>
hipError_t launch(const ScanArgs& a, int seg, int64_t slots, const float* sums, hipStream_t s) {
  using Z = ScanShape<T, DN, HW, PW>;
  constexpr int smem = 2 * Z::kB + HW * (Z::kX + Z::kM);
  static_assert(smem + (int)sizeof(Gates) * HW <= kMaxLds, "LDS");
  const int64_t shared = a.H / a.G;
  const int64_t per = (shared + HW - 1) / HW * ((a.P + Z::cols - 1) / Z::cols);
  k_scan<T, DN, HW, PW><<<dim3((unsigned)walk_blocks(slots * a.G, per)), 64 * HW * PW, smem, s>>>(a, seg, (int)slots, sums);
  return hipGetLastError();
}

}  // namespace

template <typename T>
int64_t scan_blocks(const ScanArgs& a) {
  return (seg_slots(a.seqs, a.batch, scan_seg<T>(a)) + 8) * scan_per_slot<T>(a);
}

template <typename T>
size_t scan_workspace_bytes(const ScanArgs& a) {
  const int seg = scan_seg<T>(a);
  if (seg >= a.seqs.n) return 0;
  const int64_t sh = seg_slots(a.seqs, a.batch, seg) * a.H;
  return (size_t)sh * a.P * a.N * 4 + (size_t)((sh * 4 + 15) / 16 * 16);
}

template <typename T>
hipError_t launch_scan(const ScanArgs& a, hipStream_t s) {
  const int seg = scan_seg<T>(a);
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
    k.decays = k.sums + slots * a.H * a.P * a.N;
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
  template int64_t scan_blocks<T>(const ScanArgs&);                  \
  template size_t scan_workspace_bytes<T>(const ScanArgs&);          \
  template hipError_t launch_scan<T>(const ScanArgs&, hipStream_t);
TTT_SCAN(bf16)
TTT_SCAN(float)

}  // namespace ttt
