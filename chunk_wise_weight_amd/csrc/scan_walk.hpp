// The walks over a sequence's states that the selective scan's forward and backward pass share (gfx950); the
// mathematics and the operands are in scan.hpp.
#pragma once
#include <algorithm>

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

// What a walk over states works on: forward S from B, x and exp(b_63 - b) r, or back dS from C, dO and exp(b).
struct StateWalk {
  const void *rows, *cols;            // x or dO [b, H, n, P]; B or C [b, G, n, N]
  DeltaStrides srows, scols;
  const float* start;                 // S_init or dS_final [sequences, H, P, N], or null: zero
  float* end;                         // dS_init (back) [sequences, H, P, N], or null
  float *sums, *decays;               // of segment slots and heads [P, N], 1; null: sequences are one segment
  float* keep;                        // of chunk slots and heads: the state before the chunk (back: after it)
  KeptGates* gates;                   // of chunk slots and heads, or null
  bool back;
};

// First chunk slot of a sequence (delta.hpp).
__device__ __forceinline__ int chunk_slot0(const DeltaSeqs& q, int s) {
  return q.starts ? seq_start(q, s) / kDC + s : s * ((q.n + kDC - 1) / kDC);
}
__device__ __forceinline__ int seq_first(const DeltaSeqs& q, int s) { return q.starts ? seq_start(q, s) : 0; }

// The state of a segment: from zero, for the join (KEEP false), or before every chunk, kept for the gradients.
template <typename T, int DN, int HW, int PW, bool KEEP>
__device__ __forceinline__ void walk_segment(const ScanArgs& a, const StateWalk& k, int seg, int slots, int bid, char* smem,
                                             Gates* gates) {
  using Z = ScanShape<T, DN, HW, PW>;
  using M = Mat<T>;
  constexpr int CT = Z::CT, NT = Z::NT, CS = Z::CS, W = Z::W;
  char *const Bp = smem, *const Xp = Bp + Z::kB;
  const int shared = a.H / a.G, parts = (a.P + Z::cols - 1) / Z::cols;
  ScanPlace at;
  if (!scan_place(bid, slots, a.G, shared, parts, HW, &at)) return;
  const SegPlace sp = seg_place(a.seqs, seg, at.slot);
  if (sp.len <= 0 || (!KEEP && (k.back ? sp.first : sp.last))) return;
  const int w = wave_id(), hw = w / PW, pw = w % PW, lane = lane_id(), g = lane >> 4;
  const bool mine = at.head0 + hw < shared;                // a head of the group
  const int h = at.group * shared + min(at.head0 + hw, shared - 1);
  const int p0 = at.part * Z::cols, tile0 = (p0 >> 4) + pw * CT;
  const int64_t sh = (int64_t)at.slot * a.H + h, size = (int64_t)a.P * a.N;
  LaneAt<T> L(lane);
  L.keep();
  StateRows<T, CT, NT> S;
  S.zero();
  if (KEEP && mine) {
    if (k.sums)
      S.load(k.sums + sh * size, tile0, a.P, a.N);
    else if (k.start)
      S.load(k.start + ((int64_t)sp.seq * a.H + h) * size, tile0, a.P, a.N);
  }
  const PanelLoader<T, DN, W> bload(k.scols.t * sizeof(T), a.N * sizeof(T));
  const PanelLoader<T, Z::DX, PW> xload(k.srows.t * sizeof(T), min(a.P - p0, Z::cols) * sizeof(T));
  const T* B = (const T*)k.cols + sp.b * k.scols.b + at.group * k.scols.h + sp.tok0 * k.scols.t;
  const T* x = (const T*)k.rows + sp.b * k.srows.b + h * k.srows.h + sp.tok0 * k.srows.t + p0;
  char* const Xh = Xp + hw * Z::kX;
  // the gates of head head0 + w are made by wave w
  const int gh = at.group * shared + min(at.head0 + w, shared - 1);
  const float* dt = a.dt + sp.b * a.sdt.b + gh * a.sdt.h + sp.tok0 * a.sdt.t;
  const float A = a.A[gh], bias = a.dt_bias ? a.dt_bias[gh] : 0.f;
  const int chunks = (sp.len + kDC - 1) / kDC, step = k.back ? -kDC : kDC;
  const int slot0 = chunk_slot0(a.seqs, sp.seq) + (sp.tok0 - seq_first(a.seqs, sp.seq)) / kDC;
  int t0 = k.back ? (chunks - 1) * kDC : 0;
  float dt_next = 0.f;
  double total = 0.0;
  if (w < HW && t0 + lane < sp.len) dt_next = dt[(t0 + lane) * a.sdt.t];

  for (int i = 0; i < chunks; ++i, t0 += step) {
    const int len = min(kDC, sp.len - t0);
    if (i > 0) __syncthreads();                            // the chunk before has been read
    bload.issue(B + t0 * k.scols.t, len, Bp);
    if (mine) xload.issue(x + t0 * k.srows.t, len, Xh);
    if (w < HW) {
      const LaneGates v = make_gates(dt_next, A, bias, a.softplus, len, &gates[w]);
      total += v.sum;
      if (KEEP && k.gates && at.part == 0) {               // (heads past the group's repeat the last one's)
        KeptGates* o = k.gates + (int64_t)(slot0 + t0 / kDC) * a.H + gh;
        o->g.hi[lane] = v.hi;
        o->g.lo[lane] = v.lo;
        o->g.eb[lane] = v.eb;
        o->g.r[lane] = v.r;
        o->g.w[lane] = v.w;
        o->rest[lane] = v.rest;
        o->slope[lane] = a.softplus ? 1.f / (1.f + expf(-(dt_next + bias))) : 1.f;
      }
      if (i + 1 < chunks && t0 + step + lane < sp.len) dt_next = dt[(t0 + step + lane) * a.sdt.t];
    }
    wait_vm<0>();
    __syncthreads();
    if (!mine) continue;
    const Gates& q = gates[hw];
    if constexpr (KEEP) {
      if (!k.back && sp.first && i == 0 && q.eb[0] == 0.f) S.zero();   // emptied by its first token
      S.store(k.keep + ((int64_t)(slot0 + t0 / kDC) * a.H + h) * size, tile0, a.P, a.N);
    }
    S.decay(q.eb[kDC - 1]);
    const float* weights = (k.back ? q.eb : q.w) + g * (M::KB / 4);
#pragma unroll
    for (int s = 0; s < CS; ++s) {
      u32x4 xf[CT];
#pragma unroll
      for (int c = 0; c < CT; ++c) xf[c] = L.frag_t(Xh, pw * CT + c, s);
      S.add(L, xf, Bp, s, weights + s * M::KB, a.N);
    }
  }
  if (!mine) {
    // (heads past the group's: nothing is theirs)
  } else if (!KEEP) {
    S.store(k.sums + sh * size, tile0, a.P, a.N);
  } else if (k.back && sp.first && k.end) {
    S.store(k.end + ((int64_t)sp.seq * a.H + h) * size, tile0, a.P, a.N);
  }
  // (waves of heads past the group's repeat the last one's)
  if (!KEEP && w < HW && lane == 0 && at.part == 0) k.decays[(int64_t)at.slot * a.H + gh] = exp2_hw((float)total);
}

// Walks of one or two directions: the first `half` workgroups take `one`, the others `two`.
template <typename T, int DN, int HW, int PW, bool KEEP>
__global__ __launch_bounds__(64 * HW * PW, 2) void k_scan_states(ScanArgs a, StateWalk one, StateWalk two, int seg, int slots,
                                                                 int half) {
  extern __shared__ __attribute__((aligned(16))) char smem[];
  __shared__ Gates gates[HW];
  const bool second = (int)blockIdx.x >= half;
  walk_segment<T, DN, HW, PW, KEEP>(a, second ? two : one, seg, slots, second ? blockIdx.x - half : blockIdx.x, smem, gates);
}

template <typename T, int DN, int HW, int PW, bool KEEP>
hipError_t launch_states(const ScanArgs& a, const StateWalk& one, const StateWalk* two, int seg, int64_t slots, hipStream_t s) {
  using Z = ScanShape<T, DN, HW, PW>;
  constexpr int smem = Z::kB + HW * Z::kX;
  static_assert(smem + (int)sizeof(Gates) * HW <= kMaxLds, "LDS");
  const int64_t shared = a.H / a.G;
  const int64_t half = walk_blocks(slots * a.G, (shared + HW - 1) / HW * ((a.P + Z::cols - 1) / Z::cols));
  k_scan_states<T, DN, HW, PW, KEEP><<<dim3((unsigned)(two ? 2 * half : half)), 64 * HW * PW, smem, s>>>(
      a, one, two ? *two : one, seg, (int)slots, (int)half);
  return hipGetLastError();
}

// The state before (back: after) every segment from the segments' own: a thread has 4 elements of a sequence's and
// head's state.  Sequences without tokens: their `empty` state is their first.
__device__ __forceinline__ void join_segments(const ScanArgs& a, const StateWalk& k, float* empty, int seg, int bid) {
  const int64_t size = (int64_t)a.P * a.N;
  const int blocks = (int)((size / 4 + 255) / 256), s = bid / blocks / a.H, h = bid / blocks % a.H;
  const int64_t e = ((int64_t)(bid % blocks) * 256 + threadIdx.x) * 4;
  if (e >= size) return;
  const SeqSlots q = seq_slots(a.seqs, seg, s);
  const int64_t o = ((int64_t)s * a.H + h) * size + e;
  f32x4 S = {0.f, 0.f, 0.f, 0.f};
  if (k.start) S = *reinterpret_cast<const f32x4*>(k.start + o);
  if (k.sums)
    for (int i = 0; i < q.count; ++i) {
      const int64_t sh = (int64_t)(q.first + (k.back ? q.count - 1 - i : i)) * a.H + h;
      f32x4* at = reinterpret_cast<f32x4*>(k.sums + sh * size + e);
      const f32x4 own = *at;                               // the last one's is not made
      *at = S;
      if (i + 1 < q.count) {
        const float d = k.decays[sh];
        S = d == 0.f ? own : S * d + own;
      }
    }
  if (q.count == 0 && empty) *reinterpret_cast<f32x4*>(empty + o) = S;
}
__global__ __launch_bounds__(256) void k_scan_join(ScanArgs a, StateWalk one, float* empty1, StateWalk two, float* empty2,
                                                   int seg, int half) {
  const bool second = (int)blockIdx.x >= half;
  join_segments(a, second ? two : one, second ? empty2 : empty1, seg, second ? blockIdx.x - half : blockIdx.x);
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

}  // namespace
}  // namespace ttt
