// The walks over a sequence's states that the selective scan's forward and backward pass share (gfx950); the
// mathematics and the operands are in scan.hpp.
#pragma once
#include <algorithm>

#include "scan.hpp"

namespace ttt {
namespace {

constexpr int kMaxLds = 160 * 1024;

// Which (segment slot, group, heads, part of P) a workgroup has.  Up to 4 that read the same B and C go to one
// XCD: all of them would leave the XCDs unevenly filled where sequences differ (12 packed prompts, 32 heads of one group: all
// 16 132 us, 8 167 us, 4 126 us, 2 131 us; equal segments of 64 heads: 662, 656, 661, 670 us).
struct ScanPlace {
  int slot, group, head0, part;       // head0: first head, within the group
};
inline __host__ __device__ int scan_near(int per) { return per % 4 == 0 ? 4 : per % 2 == 0 ? 2 : 1; }
__device__ __forceinline__ bool scan_place(int bid, int slots, int G, int heads, int parts, int HW, ScanPlace* o) {
  const int per = (heads + HW - 1) / HW * parts, near = scan_near(per);
  const int at = (bid / 8 / near * 8 + (bid & 7)) * near + bid / 8 % near, unit = at / per, j = at % per;
  if (unit >= slots * G) return false;
  *o = {unit / G, unit % G, j / parts * HW, j % parts};
  return true;
}

inline int64_t scan_grid(int64_t units, int64_t per) {
  const int near = scan_near((int)per);
  return walk_blocks(units * (per / near), near);
}

// What a walk over states works on: forward S from B, x and exp(b_63 - b) r, or back dS from C, dO and exp(b).
struct StateWalk {
  const void *rows, *cols;            // x or dO [b, H, n, P]; B or C [b, G, n, N]
  DeltaStrides srows, scols;
  const float* start;                 // S_init or dS_final [sequences, H, P, N], or null: zero
  float* end;                         // dS_init (back) [sequences, H, P, N], or null
  float *sums, *decays;               // of cuts and heads [P, N], 1; null: sequences are one segment
  float* keep;                        // of chunk slots and heads: the state before the chunk (back: after it)
  KeptGates* gates;                   // of chunk slots and heads, or null
  bool back;
};

// First chunk slot of a sequence (delta.hpp).
__device__ __forceinline__ int chunk_slot0(const DeltaSeqs& q, int s) {
  return q.starts ? seq_start(q, s) / kDC + s : s * ((q.n + kDC - 1) / kDC);
}
__device__ __forceinline__ int seq_first(const DeltaSeqs& q, int s) { return q.starts ? seq_start(q, s) : 0; }

// What a workgroup of a walk over states has in hand.
template <typename T, int DN, int HW, int PW, int CT_> struct StateWalker {
  using Z = ScanShape<T, DN, HW, PW, CT_>;
  using M = Mat<T>;
  static constexpr int CT = Z::CT, NT = Z::NT, CS = Z::CS, W = Z::W;
  static constexpr int kStage = Z::kB + HW * Z::kX;
  // Two stages, the next chunk coming while one is worked on; one, where LDS has no room for more.
  static constexpr int kStages = 2 * kStage + 2 * (int)sizeof(Gates) * HW <= kMaxLds ? 2 : 1;
  const ScanArgs& a;
  const StateWalk& k;
  ScanPlace at;
  SegPlace sp;
  int w, hw, pw, lane, h, gh, tile0, chunks;
  bool mine, busy;                                           // a head of the group; rows of its state
  TileLoader<T, DN, W> cload;
  TileLoader<T, Z::DX, PW> rload;
  const T *cols, *rows;
  const float* dt;
  float A, bias;
  char* smem;
  __device__ __forceinline__ StateWalker(const ScanArgs& a_, const StateWalk& k_, const ScanPlace& at_, const SegPlace& sp_,
                                         char* smem_)
      : a(a_), k(k_), at(at_), sp(sp_), w(wave_id()), hw(w / PW), pw(w % PW), lane(lane_id()),
        cload(k_.scols.t * sizeof(T), a_.N * sizeof(T)),
        rload(k_.srows.t * sizeof(T), min(a_.P - at_.part * Z::cols, Z::cols) * sizeof(T)), smem(smem_) {
    const int shared = a.H / a.G, p0 = at.part * Z::cols;
    mine = at.head0 + hw < shared;
    h = at.group * shared + min(at.head0 + hw, shared - 1);
    gh = at.group * shared + min(at.head0 + w, shared - 1);  // the gates of head head0 + w are made by wave w
    tile0 = (p0 >> 4) + pw * CT;
    busy = mine && tile0 * 16 < a.P;
    chunks = (sp.len + kDC - 1) / kDC;
    cols = (const T*)k.cols + sp.b * k.scols.b + at.group * k.scols.h + sp.tok0 * k.scols.t;
    rows = (const T*)k.rows + sp.b * k.srows.b + h * k.srows.h + sp.tok0 * k.srows.t + p0;
    dt = a.dt + sp.b * a.sdt.b + gh * a.sdt.h + sp.tok0 * a.sdt.t;
    A = a.A[gh];
    bias = a.dt_bias ? a.dt_bias[gh] : 0.f;
  }
  __device__ __forceinline__ int len(int t0) const { return min(kDC, sp.len - t0); }
  __device__ __forceinline__ void load(int t0, int stage) const {
    char* s = smem + stage * (kStages - 1) * kStage;
    cload.issue(cols + t0 * k.scols.t, len(t0), s);
    if (mine) rload.issue(rows + t0 * k.srows.t, len(t0), s + Z::kB + hw * Z::kX);
  }
  __device__ __forceinline__ float load_dt(int t0) const {
    return w < HW && t0 >= 0 && t0 + lane < sp.len ? dt[(t0 + lane) * a.sdt.t] : 0.f;
  }
  // += the chunk in a stage, tokens weighted
  __device__ __forceinline__ void add(StateRows<T, CT, NT>& S, const LaneAt<T>& L, const Split<T>& split, int stage,
                                      const float* weights) const {
    const char *s = smem + stage * (kStages - 1) * kStage, *x = s + Z::kB + hw * Z::kX;
#pragma unroll
    for (int st = 0; st < CS; ++st) {
      u32x4 xf[CT];
#pragma unroll
      for (int c = 0; c < CT; ++c) xf[c] = state_cols<T, CT>(L, x, pw * CT + c, st);
      S.add(L, split, xf, s, st, weights + (lane >> 4) * (M::KB / 4) + st * M::KB, a.N);
    }
  }
};

// The state of a segment from zero, for the join (65,536 tokens x 64 heads of 64 x 128 in bf16: 26 % of the call's time,
// traced 190 us at the least, matrix cores busy for 31 % of its cycles; with two blocks of 16 columns a wave 234 us).  The
// chunks go by from the segment's far end (forward walks: the last one first), their weights decayed by what lies between,
// so that the state itself need not be, and none is read whose weights are zero in fp32.
template <typename T, int DN, int HW, int PW, int CT>
__device__ __forceinline__ void sum_segment(const ScanArgs& a, const StateWalk& k, int seg, int slots, int bid, char* smem) {
  using K = StateWalker<T, DN, HW, PW, CT>;
  __shared__ float weights[2][HW][kDC];
  __shared__ int live[2][HW];
  ScanPlace at;
  if (!scan_place(bid, slots, a.G, a.H / a.G, (a.P + K::Z::cols - 1) / K::Z::cols, HW, &at)) return;
  const SegPlace sp = seg_place(a.seqs, seg, at.slot);
  if (sp.len <= 0 || (k.back ? sp.first : sp.last)) return;
  const K q(a, k, at, sp, smem);
  const LaneAt<T> L(q.lane);
  const Split<T> split(q.lane);
  StateRows<T, K::CT, K::NT> S;
  S.zero();
  const int step = k.back ? kDC : -kDC, end = k.back ? q.chunks * kDC : -kDC;
  int t0 = k.back ? 0 : (q.chunks - 1) * kDC, stage = 0;
  double F = 0.0;                                            // log decays between the chunk and the segment's end
  constexpr double kNone = -150.0;                           // base 2: nothing of fp32 is left
  float dt_next = q.load_dt(t0);
  auto gates = [&](int t, int st) __attribute__((always_inline)) {   // of the chunk at t, by wave w those of head w
    if (q.w >= HW) return;
    const LaneGates v = make_gates(dt_next, q.A, q.bias, a.softplus, q.len(t));
    dt_next = q.load_dt(t + step);
    weights[st][q.w][q.lane] = k.back ? exp2_hw((float)(F + v.b)) : v.r * exp2_hw((float)(F + v.sum - v.b));
    if (q.lane == 0) live[st][q.w] = F > kNone;
    F += v.sum;
  };
  q.load(t0, 0);
  gates(t0, 0);
  for (; t0 != end; t0 += step) {
    wait_vm<0>();
    __syncthreads();                                         // the stage is there, the other one has been read
    bool any = false;
#pragma unroll
    for (int i = 0; i < HW; ++i) any |= live[stage][i] != 0;
    if (!any) break;
    if (t0 + step != end) {
      if (K::kStages == 2) q.load(t0 + step, stage ^ 1);
      gates(t0 + step, stage ^ 1);
    }
    if (q.busy) q.add(S, L, split, stage, weights[stage][q.hw]);
    if (K::kStages == 1 && t0 + step != end) {
      __syncthreads();
      q.load(t0 + step, 0);
    }
    stage ^= 1;
  }
  const int64_t size = (int64_t)a.P * a.N;
  const int64_t cut = k.back ? sp.cut - 1 : sp.cut;          // at its end in the walk's direction
  if (q.busy) S.store(k.sums + (cut * a.H + q.h) * size, q.tile0, a.P, a.N);
  // (heads past the group's repeat the last one's; after a break F is below kNone and stays there)
  if (q.w < HW && q.lane == 0 && at.part == 0) k.decays[cut * a.H + q.gh] = exp2_hw((float)F);
}

// The states before (back: after) every chunk, kept for the gradients.  Bound by their stores: 4 x 4,096 tokens x 32 heads of
// 64 x 128 both ways 147 us at the least under a trace, 3.6 TB/s.
template <typename T, int DN, int HW, int PW, int CT>
__device__ __forceinline__ void keep_segment(const ScanArgs& a, const StateWalk& k, int seg, int slots, int bid, char* smem) {
  using K = StateWalker<T, DN, HW, PW, CT>;
  __shared__ Gates gates[2][HW];
  ScanPlace at;
  if (!scan_place(bid, slots, a.G, a.H / a.G, (a.P + K::Z::cols - 1) / K::Z::cols, HW, &at)) return;
  const SegPlace sp = seg_place(a.seqs, seg, at.slot);
  if (sp.len <= 0) return;
  const K q(a, k, at, sp, smem);
  const int64_t size = (int64_t)a.P * a.N;
  const LaneAt<T> L(q.lane);
  const Split<T> split(q.lane);
  StateRows<T, K::CT, K::NT> S;
  S.zero();
  if (q.busy) {
    if (!(k.back ? sp.last : sp.first))
      S.load(k.sums + ((int64_t)(k.back ? sp.cut : sp.cut - 1) * a.H + q.h) * size, q.tile0, a.P, a.N);
    else if (k.start)
      S.load(k.start + ((int64_t)sp.seq * a.H + q.h) * size, q.tile0, a.P, a.N);
  }
  const int slot0 = chunk_slot0(a.seqs, sp.seq) + (sp.tok0 - seq_first(a.seqs, sp.seq)) / kDC;
  const int step = k.back ? -kDC : kDC, end = k.back ? -kDC : q.chunks * kDC;
  int t0 = k.back ? (q.chunks - 1) * kDC : 0, stage = 0;
  float dt_next = q.load_dt(t0);
  auto make = [&](int t, int st) __attribute__((always_inline)) {   // gates of the chunk at t, by wave w those of head w
    if (q.w >= HW) return;
    const LaneGates v = make_gates(dt_next, q.A, q.bias, a.softplus, q.len(t));
    Gates* o = &gates[st][q.w];
    const float eb = exp2_hw((float)v.b), rest = exp2_hw((float)(v.sum - v.b));
    o->eb[q.lane] = eb;
    o->w[q.lane] = v.r * rest;
    if (k.gates && at.part == 0) {                           // (heads past the group's repeat the last one's)
      KeptGates* to = k.gates + (int64_t)(slot0 + t / kDC) * a.H + q.gh;
      two_parts(v.b, &to->g.hi[q.lane], &to->g.lo[q.lane]);
      to->g.eb[q.lane] = eb;
      to->g.r[q.lane] = v.r;
      to->g.w[q.lane] = v.r * rest;
      to->rest[q.lane] = rest;
      to->slope[q.lane] = scan_rate_slope(dt_next, q.bias, a.softplus);
    }
    dt_next = q.load_dt(t + step);
  };
  q.load(t0, 0);
  make(t0, 0);
  for (; t0 != end; t0 += step) {
    wait_vm<0>();
    __syncthreads();                                         // the stage is there, the other one has been read
    const Gates& g = gates[stage][q.hw];
    if (q.busy) {
      if (!k.back && sp.first && t0 == 0 && g.eb[0] == 0.f) S.zero();   // emptied by its first token
      S.store(k.keep + ((int64_t)(slot0 + t0 / kDC) * a.H + q.h) * size, q.tile0, a.P, a.N);
    }
    if (t0 + step != end) {
      if (K::kStages == 2) q.load(t0 + step, stage ^ 1);
      make(t0 + step, stage ^ 1);
    }
    if (q.busy) {
      S.decay(g.eb[kDC - 1]);
      q.add(S, L, split, stage, k.back ? g.eb : g.w);
    }
    if (K::kStages == 1 && t0 + step != end) {
      __syncthreads();
      q.load(t0 + step, 0);
    }
    stage ^= 1;
  }
  if (q.busy && k.back && sp.first && k.end)
    S.store(k.end + ((int64_t)sp.seq * a.H + q.h) * size, q.tile0, a.P, a.N);
}

// Walks of one or two directions: the first `half` workgroups take `one`, the others `two`.
template <typename T, int DN, int HW, int PW, int CT, bool KEEP>
__global__ __launch_bounds__(64 * HW * PW, KEEP ? 2 : 4) void k_scan_states(ScanArgs a, StateWalk one, StateWalk two, int seg, int slots,
                                                                 int half) {
#if __HIP_DEVICE_COMPILE__
  extern __shared__ __attribute__((aligned(16))) char smem[];
  const bool second = (int)blockIdx.x >= half;
  const StateWalk& k = second ? two : one;
  const int bid = second ? blockIdx.x - half : blockIdx.x;
  if constexpr (KEEP)
    keep_segment<T, DN, HW, PW, CT>(a, k, seg, slots, bid, smem);
  else
    sum_segment<T, DN, HW, PW, CT>(a, k, seg, slots, bid, smem);
#endif
}

// PW: the outputs' walk's, whose waves have kBlocks each.
template <typename T, int DN, int HW, int PW_, bool KEEP>
hipError_t launch_states(const ScanArgs& a, const StateWalk& one, const StateWalk* two, int seg, int64_t slots, hipStream_t s) {
  constexpr int CT = KEEP ? kBlocks<T, DN> : 1, PW = PW_ * kBlocks<T, DN> / CT;
  using Z = ScanShape<T, DN, HW, PW, CT>;
  using K = StateWalker<T, DN, HW, PW, CT>;
  constexpr int smem = K::kStages * K::kStage;
  static_assert(smem + 2 * (int)sizeof(Gates) * HW <= kMaxLds, "LDS");
  const int64_t shared = a.H / a.G;
  const int64_t half = scan_grid(slots * a.G, (shared + HW - 1) / HW * ((a.P + Z::cols - 1) / Z::cols));
  k_scan_states<T, DN, HW, PW, CT, KEEP><<<dim3((unsigned)(two ? 2 * half : half)), 64 * HW * PW, smem, s>>>(
      a, one, two ? *two : one, seg, (int)slots, (int)half);
  return hipGetLastError();
}

// The state at every cut from the segments' own: a thread has 4 elements of a sequence's and head's state.  A cut's place
// holds the sum of the segment that ends there (in the walk's direction) and then the state that the next one begins with;
// a sequence's first begins with `start`.  Sequences without tokens: their `empty` state is that.
__device__ __forceinline__ void join_segments(const ScanArgs& a, const StateWalk& k, float* empty, int seg, int bid) {
  const int64_t size = (int64_t)a.P * a.N;
  const int blocks = (int)((size / 4 + 255) / 256), s = bid / blocks / a.H, h = bid / blocks % a.H;
  const int64_t e = ((int64_t)(bid % blocks) * 256 + threadIdx.x) * 4;
  const SeqCuts q = seq_cuts(a.seqs, seg, s);
  const int cuts = q.count - 1;
  if (e >= size || (q.count == 0 ? empty == nullptr : cuts == 0)) return;
  const int64_t o = ((int64_t)s * a.H + h) * size + e;
  f32x4 S = {0.f, 0.f, 0.f, 0.f};
  if (k.start) S = *reinterpret_cast<const f32x4*>(k.start + o);
  if (q.count == 0) {
    *reinterpret_cast<f32x4*>(empty + o) = S;
    return;
  }
  constexpr int U = 4;                                       // cuts whose loads are under way at once
  for (int i0 = 0; i0 < cuts; i0 += U) {
    f32x4 own[U];
    float d[U];
    auto place = [&](int i) { return (int64_t)(q.first + (k.back ? cuts - 1 - i : i)) * a.H + h; };
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (i0 + u < cuts) {
        own[u] = *reinterpret_cast<const f32x4*>(k.sums + place(i0 + u) * size + e);
        d[u] = k.decays[place(i0 + u)];
      }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (i0 + u < cuts) {
        S = d[u] == 0.f ? own[u] : S * d[u] + own[u];
        *reinterpret_cast<f32x4*>(k.sums + place(i0 + u) * size + e) = S;
      }
  }
}
__global__ __launch_bounds__(256) void k_scan_join(ScanArgs a, StateWalk one, float* empty1, StateWalk two, float* empty2,
                                                   int seg, int half) {
  const bool second = (int)blockIdx.x >= half;
  join_segments(a, second ? two : one, second ? empty2 : empty1, seg, second ? blockIdx.x - half : blockIdx.x);
}

// The variant for heads of P and N, `shared` of them to a group: DN, HW, PW.  Heads of a group in one workgroup read B and C
// and make C B^T once: 16,384 tokens, 64 heads of 64 x 128 over 8 groups in bf16, two heads 183 us, one 247 us (fp32, 4,096
// tokens, 201, 246 us).  Four heads of up to 32 x 128: fp32 116 us, two 179 us; bf16 169 us, two 136 us: its waves without
// rows of P help with C B^T.
template <typename T, typename F>
hipError_t with_scan(int P, int N, int shared, F f) {
  using std::integral_constant;
  auto pick = [&](auto dn) {
    using I1 = integral_constant<int, 1>;
    using I2 = integral_constant<int, 2>;
    using I4 = integral_constant<int, 4>;
    if constexpr (decltype(dn)::value <= 128) {
      constexpr int kWide = 4 / kBlocks<T, decltype(dn)::value>;     // waves of 64 columns
      using W = integral_constant<int, kWide>;
      if constexpr (sizeof(T) == 4)
        if (P <= 32 && shared > 2) return f(dn, I4(), integral_constant<int, kWide / 2>());
      if (P <= 64) return shared > 1 ? f(dn, I2(), W()) : f(dn, I1(), W());
      return f(dn, I1(), integral_constant<int, 2 * kWide>());
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

// Tokens of a segment: as many as give the chip `fill` workgroups, or, where those are fewer than 256, up to 256 that still
// give half of it; whole sequences where those are `whole` or more, or one segment would be.  (Shorter than 256, bf16 / fp32,
// us: 4 heads, 5 sequences of 1177 tokens 42 -> 29 / 91 -> 41; 16 heads, 4,000 tokens 50 -> 44 / 97 -> 69; where 256 fills half
// of the chip it stays better, 64 heads, 2,000 tokens 56, with 128 58 / 106, with 128 124.)
template <typename T>
int scan_seg(const ScanArgs& a, int64_t fill, int64_t whole) {
  constexpr int64_t kShort = 256;
  const int64_t n = std::max(a.seqs.n, 1), all = (n + kDC - 1) / kDC * kDC, per = scan_per_slot<T>(a);
  if (all <= kShort || (!a.seqs.starts && a.batch * per >= whole)) return (int)all;
  const int64_t tokens = a.seqs.starts ? n : n * a.batch;
  const int64_t even = tokens * per / fill, seg = std::max(even, std::min(kShort, 2 * even));
  return (int)std::min(std::max<int64_t>((seg + kDC - 1) / kDC, 1) * kDC, all);
}

}  // namespace
}  // namespace ttt
