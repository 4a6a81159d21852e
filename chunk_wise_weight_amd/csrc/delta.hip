// The gated delta rule over whole sequences, forward (gfx950).
#include <algorithm>

#include "delta_walk.hpp"

namespace ttt {
namespace {

template <typename T, int DK, int NW, int STAGES, int OUT, bool QLDS>
__global__ __launch_bounds__((Walk<T, DK, NW, STAGES, OUT, QLDS>::kThreads)) void k_delta_walk(DeltaArgs p, const char* rec,
                                                                                               int sequences) {
  WalkPlace at;
  if (!walk_place(blockIdx.x, sequences, p.Hk, p.Hv / p.Hk, (p.dv + 16 * NW - 1) / (16 * NW), &at)) return;
  const SeqPlace sp = seq_place(p.seqs, at.seq);
  const int w = wave_id();
  if (w < 2)
    walk_loads<T, DK, NW, STAGES, OUT, QLDS>(p, 1 << w, rec, at, sp);
  else if (w < 2 + NW)
    walk_states<T, DK, NW, STAGES, OUT, QLDS>(p, w - 2, nullptr, nullptr, at, sp);
  else if constexpr (OUT == kHelped)
    walk_outputs<T, DK, NW, STAGES, QLDS>(p, rec, w - 2 - NW, at, sp);
}

constexpr int kMaxLds = 160 * 1024;

template <typename T, int DK, int NW, int STAGES, int OUT, bool QLDS>
hipError_t launch_walk(const DeltaArgs& a, int sequences, hipStream_t s) {
  using G = Walk<T, DK, NW, STAGES, OUT, QLDS>;
  static_assert(G::kSmem <= kMaxLds, "one stage has to fit");
  auto kern = k_delta_walk<T, DK, NW, STAGES, OUT, QLDS>;
  const int64_t blocks = walk_blocks((int64_t)sequences * a.Hk, a.Hv / a.Hk * ((a.dv + 16 * NW - 1) / (16 * NW)));
  kern<<<dim3((unsigned)blocks), G::kThreads, G::kSmem, s>>>(a, a.ws, sequences);
  return hipGetLastError();
}

// Whether the state waves make O themselves.  A chunk takes a helped walk less
// time than a walk of its own, but the latter's workgroup has 64 columns of the
// state instead of 32.  LDS has room for one workgroup a CU, so rows of equal
// length take as many rounds as there are times 256 workgroups; packed
// sequences take their longest's time at least, and otherwise their chunks'
// over 256 CUs.  Microseconds a chunk where the chip is full, helped / own: bf16
// heads of up to 128 (kernels of 128) 1.9 / 2.65, of up to 64 1.55 / 2.05, fp32
// of up to 64 3.35 / 5.5.  Both forms, rows x tokens, heads k x v (us, 32 value
// heads but where said):
//   bf16 128 x 128  1 x 16K 422 / 617   4 x 4K 244 / 174   8 x 2K 247 / 186, 8 heads 57 / 81, 48 heads 374 / 258
//   bf16 64 x 64    1 x 16K 298 / 413   4 x 4K  99 / 113   8 x 2K 102 /  68, 8 heads 36 / 55, 48 heads 163 / 138
//   bf16 96 x 96    1 x 16K 451 / 593   4 x 4K 236 / 166   8 x 2K 201 / 167, 8 heads 51 / 79, 48 heads 298 / 246
//   fp32 64 x 64    1 x 16K 805 / 1269  4 x 4K 212 / 334   8 x 2K 216 / 178, 8 heads 103 / 163, 48 heads 321 / 339
// 12 packed prompts, 16 heads of 128, the longest 6007 of 16456 tokens: 150 / 236.
// The lengths of packed sequences are known on the device only: the longest is
// taken for four times the mean.
template <typename T, int DK>
inline bool own_outputs(const DeltaArgs& a, int sequences) {
  constexpr double kHelpedUs = sizeof(T) == 4 ? 3.35 : DK == 64 ? 1.55 : 1.9;
  constexpr double kOwnUs = sizeof(T) == 4 ? 5.5 : DK == 64 ? 2.05 : 2.65;
  const double row = (a.seqs.n + kDC - 1) / kDC;                          // chunks of a row
  const double longest = std::min(row, 4 * row / std::max(sequences, 1));  // packed: of a sequence, taken for
  auto time = [&](int columns, double chunk) {
    const int64_t parts = (int64_t)a.Hv * ((a.dv + columns - 1) / columns);
    if (a.seqs.starts) return std::max(longest, row * parts / 256.0) * chunk;
    return (double)((sequences * parts + 255) / 256) * row * chunk;
  };
  return time(64, kOwnUs) < time(32, kHelpedUs);
}

template <typename T, int DK>
hipError_t launch_walks(const DeltaArgs& a, int sequences, hipStream_t s) {
  constexpr int NW = Walk<T, DK, 2, 1, kHelped, false>::kSmem <= kMaxLds ? 2 : 1;
  constexpr bool QLDS = Walk<T, DK, NW, 2, kHelped, true>::kSmem <= kMaxLds;
  constexpr int STAGES = Walk<T, DK, NW, 2, kHelped, QLDS>::kSmem <= kMaxLds ? 2 : 1;
  if constexpr (Walk<T, DK, 4, 2, kOwn, true>::kSmem <= kMaxLds)
    if (own_outputs<T, DK>(a, sequences))
      return launch_walk<T, DK, 4, 2, kOwn, true>(a, sequences, s);
  return launch_walk<T, DK, NW, STAGES, kHelped, QLDS>(a, sequences, s);
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
    k_delta_chunks<T, false><<<dim3((unsigned)(slots * a.Hv)), kChunkThreads, 0, s>>>(a, a.ws, nullptr);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const int sequences = a.seqs.starts ? a.seqs.num : a.batch;
  if (sequences == 0) return hipSuccess;
  if (a.dk <= 64) return launch_walks<T, 64>(a, sequences, s);
  if (a.dk <= 128) return launch_walks<T, 128>(a, sequences, s);
  return launch_walks<T, 256>(a, sequences, s);
}

template size_t delta_workspace_bytes<bf16>(const DeltaArgs&);
template size_t delta_workspace_bytes<float>(const DeltaArgs&);
template hipError_t launch_delta<bf16>(const DeltaArgs&, hipStream_t);
template hipError_t launch_delta<float>(const DeltaArgs&, hipStream_t);

}  // namespace ttt
