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

// Whether the state waves make O themselves.  A chunk takes a helped walk about
// 1.4 us and a walk of its own 2.2 us (dk = 128, bf16), but the latter's
// workgroup has 64 columns of the state instead of 32; a walk cannot end
// before its longest chain, nor the launch before its workgroups have gone
// over the 256 CUs.  One call, dk = dv = 128, 32 value heads, helped / own: 1 x
// 64K tokens 2.20 / 3.4 ms, 8 x 8K 1.41 / 1.11 ms, 32 x 2K 1.44 / 1.11 ms; 12
// packed prompts, 16 heads, the longest 6007 of 16456 tokens 0.22 / 0.30 ms.
// The lengths of packed sequences are known on the device only: the longest is
// taken for four times the mean.
inline bool own_outputs(const DeltaArgs& a, int sequences) {
  const double all = (double)a.batch * ((a.seqs.n + kDC - 1) / kDC);      // chunks of all rows
  const double mean = all / std::max(sequences, 1), longest = a.seqs.starts ? std::min(all, 4 * mean) : mean;
  auto time = [&](int columns, double chunk) {
    return std::max(longest, all * a.Hv * ((a.dv + columns - 1) / columns) / 256.0) * chunk;
  };
  return time(64, 2.2) < time(32, 1.4);
}

template <typename T, int DK>
hipError_t launch_walks(const DeltaArgs& a, int sequences, hipStream_t s) {
  constexpr int NW = Walk<T, DK, 2, 1, kHelped, false>::kSmem <= kMaxLds ? 2 : 1;
  constexpr bool QLDS = Walk<T, DK, NW, 2, kHelped, true>::kSmem <= kMaxLds;
  constexpr int STAGES = Walk<T, DK, NW, 2, kHelped, QLDS>::kSmem <= kMaxLds ? 2 : 1;
  if constexpr (Walk<T, DK, 4, 2, kOwn, true>::kSmem <= kMaxLds)
    if (own_outputs(a, sequences))
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
