// The selective scan over whole sequences for gfx950; the mathematics and the operands are in scan.hpp.
#include "scan.hpp"

namespace ttt {
namespace {

constexpr int kMaxLds = 160 * 1024;

// Which (segment slot, group, heads, part of P) a workgroup has: those that read the same B and C go to one XCD.
struct ScanPlace {
  int slot, group, head0, part;       // head0: first head, within the group
};
__device__ __forceinline__ bool scan_place(int bid, int slots, int G, int heads, int parts, int HW, ScanPlace* o) {
  const int per = (heads + HW - 1) / HW * parts, unit = bid / 8 / per * 8 + (bid & 7), j = bid / 8 % per;
  if (unit >= slots * G) return false;
  *o = {unit / G, unit % G, j / parts * HW, j % parts};
  return true;
}

// Work of a segment: its walk over the chunks with outputs (OUT), or only its state from zero.
// sums: every slot's and head's [P, N] states and, behind them, decays.
template <typename T, int DN, int HW, int PW, bool OUT>
__global__ __launch_bounds__(64 * HW * PW, 2) void k_scan(ScanArgs a, int seg, int slots, float* sums, float* decays) {
  using Z = ScanShape<T, DN, HW, PW>;
  using M = Mat<T>;
  constexpr int CT = Z::CT, NT = Z::NT, NS = Z::NS, CS = Z::CS, W = Z::W;
  extern __shared__ __attribute__((aligned(16))) char smem[];
  __shared__ Gates gates[HW];
  char *const Bp = smem, *const Cp = Bp + Z::kB, *const Xp = Cp + (OUT ? Z::kB : 0), *const Mp = Xp + HW * Z::kX;
  const int shared = a.H / a.G, parts = (a.P + Z::cols - 1) / Z::cols;
  ScanPlace at;
  if (!scan_place(blockIdx.x, slots, a.G, shared, parts, HW, &at)) return;
  const SegPlace sp = seg_place(a.seqs, seg, at.slot);
  if (sp.len <= 0 || (!OUT && sp.last)) return;
  const int w = wave_id(), hw = w / PW, pw = w % PW, lane = lane_id(), m = lane & 15, g = lane >> 4;
  const bool mine = at.head0 + hw < shared;                // a head of the group
  const int h = at.group * shared + min(at.head0 + hw, shared - 1);
  const int p0 = at.part * Z::cols, tile0 = (p0 >> 4) + pw * CT;
  const int64_t sh = (int64_t)at.slot * a.H + h, size = (int64_t)a.P * a.N;

  StateRows<T, CT, NT> S;
  S.zero();
  if (OUT && mine) {
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
  double total = 0.0;
  if (w < HW && lane < sp.len) dt_next = dt[lane * a.sdt.t];

  for (int t0 = 0; t0 < sp.len; t0 += kDC) {
    const int len = min(kDC, sp.len - t0);
    if (t0 > 0) __syncthreads();                           // the chunk before has been read
    bload.issue(B + t0 * a.sB.t, len, Bp);
    if (OUT) cload.issue(C + t0 * a.sC.t, len, Cp);
    if (mine) xload.issue(x + t0 * a.sx.t, len, Xh);
    if (w < HW) {
      total += make_gates(dt_next, A, bias, a.softplus, len, &gates[w]);
      if (t0 + kDC + lane < sp.len) dt_next = dt[(t0 + kDC + lane) * a.sdt.t];
    }
    wait_vm<0>();
    __syncthreads();
    if constexpr (OUT) {
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
            if (ns * M::KB < a.N) {
              const u32x4 c = Panels<T>::frag(Cp, i, ns, g);
#pragma unroll
              for (int u = 0; u < M::TPS; ++u)
                d[u] = M::mma(Panels<T>::frag(Bp, M::row(s * M::TPS + u, m), ns, g), c, d[u]);
            }
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
    if (OUT && t0 == 0 && sp.first && q.eb[0] == 0.f) S.zero();   // emptied by its first token: S_init is not looked at
    u32x4 xf[CT][CS];
#pragma unroll
    for (int c = 0; c < CT; ++c)
#pragma unroll
      for (int s = 0; s < CS; ++s) xf[c][s] = Panels<T>::frag_t(Xh, pw * CT + c, s, lane);
    if constexpr (OUT) {
      f32x4 o[CT][4];
#pragma unroll
      for (int c = 0; c < CT; ++c)
#pragma unroll
        for (int t = 0; t < 4; ++t) o[c][t] = (f32x4){0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int ns = 0; ns < NS; ++ns) {
        if (ns * M::KB < a.N) {
          u32x4 sh_[CT], sl[CT];
#pragma unroll
          for (int c = 0; c < CT; ++c) M::split(&S.s[c][ns * M::TPS], sh_[c], sl[c]);
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            const u32x4 f = Panels<T>::frag(Cp, M::row(t, m), ns, g);
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
            for (int c = 0; c < CT; ++c) o[c][t] = M::mma(xf[c][s], lo, o[c][t]);
          }
#pragma unroll
          for (int c = 0; c < CT; ++c) o[c][t] = M::mma(xf[c][s], hi, o[c][t]);
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
            if (a.D) v[k] += D * load4((const T*)(Xh + Panels<T>::at(i, p + 4 * k - p0)));
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
    for (int s = 0; s < CS; ++s) {
      // (made for both blocks of P at once, so that an operand of B is read once)
      const float* weights = q.w + s * M::KB + g * (M::KB / 4);
      if constexpr (CT == 2) {
        const Scaled<T> u0(xf[0][s], weights), u1(xf[1][s], weights);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          if (t / M::TPS * M::KB < a.N) {
            const u32x4 f = Panels<T>::frag_t(Bp, t, s, lane);
            S.s[0][t] = u0.mma(f, S.s[0][t]);
            S.s[1][t] = u1.mma(f, S.s[1][t]);
          }
        }
      } else {
        const Scaled<T> u0(xf[0][s], weights);
#pragma unroll
        for (int t = 0; t < NT; ++t)
          if (t / M::TPS * M::KB < a.N) S.s[0][t] = u0.mma(Panels<T>::frag_t(Bp, t, s, lane), S.s[0][t]);
      }
    }
  }
  if (OUT) {
    if (mine && sp.last && a.S_final) S.store(a.S_final + ((int64_t)sp.seq * a.H + h) * size, tile0, a.P, a.N);
  } else {
    if (mine) S.store(sums + sh * size, tile0, a.P, a.N);
    // (heads past the group's repeat the last one's)
    if (w < HW && lane == 0 && at.part == 0) decays[(int64_t)at.slot * a.H + gh] = exp2_hw((float)total);
  }
}

// The state before every segment from the segments' own: a thread has 4 elements of a sequence's and head's state.
// Sequences without tokens: their last state is their first.
__global__ __launch_bounds__(256) void k_scan_join(ScanArgs a, int seg, float* sums, const float* decays) {
  const int64_t size = (int64_t)a.P * a.N;
  const int blocks = (int)((size / 4 + 255) / 256), s = blockIdx.x / blocks / a.H, h = blockIdx.x / blocks % a.H;
  const int64_t e = ((int64_t)(blockIdx.x % blocks) * 256 + threadIdx.x) * 4;
  if (e >= size) return;
  const SeqSlots q = seq_slots(a.seqs, seg, s);
  f32x4 S = {0.f, 0.f, 0.f, 0.f};
  if (a.S_init) S = *reinterpret_cast<const f32x4*>(a.S_init + ((int64_t)s * a.H + h) * size + e);
  for (int c = 0; c < q.count; ++c) {
    const int64_t sh = (int64_t)(q.first + c) * a.H + h;
    f32x4* at = reinterpret_cast<f32x4*>(sums + sh * size + e);
    const f32x4 own = *at;                                 // the last segment's is not made
    *at = S;
    if (c + 1 < q.count) {
      const float d = decays[sh];
      S = d == 0.f ? own : S * d + own;
    }
  }
  if (q.count == 0) *reinterpret_cast<f32x4*>(a.S_final + ((int64_t)s * a.H + h) * size + e) = S;
}

// Sequences without tokens where no segments are joined.
__global__ __launch_bounds__(256) void k_scan_empty(ScanArgs a) {
  const int64_t size = (int64_t)a.P * a.N;
  const int blocks = (int)((size / 4 + 255) / 256), s = blockIdx.x / blocks / a.H, h = blockIdx.x / blocks % a.H;
  const int64_t e = ((int64_t)(blockIdx.x % blocks) * 256 + threadIdx.x) * 4;
  if (e >= size || seq_slots(a.seqs, kDC, s).count > 0) return;
  const int64_t o = ((int64_t)s * a.H + h) * size + e;
  *reinterpret_cast<f32x4*>(a.S_final + o) =
      a.S_init ? *reinterpret_cast<const f32x4*>(a.S_init + o) : (f32x4){0.f, 0.f, 0.f, 0.f};
}

// The variant for heads of P and N, `shared` of them to a group: DN, HW, PW.
template <typename T, typename F>
hipError_t with_scan(int P, int N, int shared, F f) {
  using std::integral_constant;
  auto pick = [&](auto dn) {
    using I1 = integral_constant<int, 1>;
    using I2 = integral_constant<int, 2>;
    using I4 = integral_constant<int, 4>;
    if constexpr (decltype(dn)::value <= 128) {
      if (P <= 32 && shared > 2) return f(dn, I4(), I1());
      if (P <= 64) return shared > 1 ? f(dn, I2(), I2()) : f(dn, I1(), I2());
    }
    return f(dn, I1(), I4());
  };
  if (N <= 64) return pick(integral_constant<int, 64>());
  if (N <= 128) return pick(integral_constant<int, 128>());
  return pick(integral_constant<int, 256>());
}

// Workgroups of a segment slot.
template <typename T>
int64_t scan_per_slot(const ScanArgs& a) {
  int64_t per = 0;
  const int shared = a.H / a.G;
  (void)with_scan<T>(a.P, a.N, shared, [&](auto dn, auto hw, auto pw) {
    using Z = ScanShape<T, decltype(dn)::value, decltype(hw)::value, decltype(pw)::value>;
    per = (int64_t)a.G * ((shared + Z::HW - 1) / Z::HW) * ((a.P + Z::cols - 1) / Z::cols);
    return hipSuccess;
  });
  return per;
}

// Tokens of a segment: as many as leave the chip some workgroups a CU, whole sequences where those do that.
constexpr int64_t kFill = 1024, kLeastSeg = 256;
template <typename T>
int scan_seg(const ScanArgs& a) {
  const int64_t n = std::max(a.seqs.n, 1), whole = (n + kDC - 1) / kDC * kDC, per = scan_per_slot<T>(a);
  if (!a.seqs.starts && a.batch * per >= kFill / 2) return (int)whole;
  const int64_t tokens = a.seqs.starts ? n : n * a.batch;
  const int64_t seg = std::max(kLeastSeg, (tokens * per / kFill + kDC - 1) / kDC * kDC);
  return (int)std::min(seg, whole);
}

template <typename T, int DN, int HW, int PW, bool OUT>
hipError_t launch(const ScanArgs& a, int seg, int64_t slots, float* sums, float* decays, hipStream_t s) {
  using Z = ScanShape<T, DN, HW, PW>;
  constexpr int smem = (OUT ? 2 : 1) * Z::kB + HW * Z::kX + (OUT ? HW * Z::kM : 0);
  static_assert(smem + (int)sizeof(Gates) * HW <= kMaxLds, "LDS");
  const int64_t shared = a.H / a.G;
  const int64_t per = (shared + HW - 1) / HW * ((a.P + Z::cols - 1) / Z::cols);
  k_scan<T, DN, HW, PW, OUT><<<dim3((unsigned)walk_blocks(slots * a.G, per)), 64 * HW * PW, smem, s>>>(a, seg, (int)slots,
                                                                                                       sums, decays);
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
  float *sums = nullptr, *decays = nullptr;
  if (seg < a.seqs.n) {
    sums = (float*)a.ws;
    decays = sums + slots * a.H * a.P * a.N;
  }
  return with_scan<T>(a.P, a.N, a.H / a.G, [&](auto dn, auto hw, auto pw) {
    constexpr int DN = decltype(dn)::value, HW = decltype(hw)::value, PW = decltype(pw)::value;
    hipError_t e;
    if (sums) {
      if ((e = launch<T, DN, HW, PW, false>(a, seg, slots, sums, decays, s)) != hipSuccess) return e;
      k_scan_join<<<dim3((unsigned)join), 256, 0, s>>>(a, seg, sums, decays);
      if ((e = hipGetLastError()) != hipSuccess) return e;
    } else if (a.seqs.starts || a.seqs.n == 0) {
      k_scan_empty<<<dim3((unsigned)join), 256, 0, s>>>(a);
      if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    if (a.seqs.n == 0) return hipSuccess;
    return launch<T, DN, HW, PW, true>(a, seg, slots, sums, decays, s);
  });
}

#define TTT_SCAN(T)                                                  \
  template int64_t scan_blocks<T>(const ScanArgs&);                  \
  template size_t scan_workspace_bytes<T>(const ScanArgs&);          \
  template hipError_t launch_scan<T>(const ScanArgs&, hipStream_t);
TTT_SCAN(bf16)
TTT_SCAN(float)

}  // namespace ttt
