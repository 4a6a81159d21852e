// The gated delta rule over whole sequences, forward (gfx950).
#include "delta_walk.hpp"

namespace ttt {
namespace {

template <typename T, int DK, int NW, int STAGES, bool QLDS>
__global__ __launch_bounds__(64 * (1 + 2 * NW)) void k_delta_walk(DeltaArgs p, const char* rec, int sequences) {
  WalkPlace at;
  if (!walk_place(blockIdx.x, sequences, p.Hk, p.Hv / p.Hk, (p.dv + 16 * NW - 1) / (16 * NW), &at)) return;
  const SeqPlace sp = seq_place(p.seqs, at.seq);
  const int w = wave_id();
  if (w == 0)
    walk_loads<T, DK, NW, STAGES, true, QLDS>(p, rec, at, sp);
  else if (w <= NW)
    walk_states<T, DK, NW, STAGES, true, QLDS>(p, w - 1, nullptr, nullptr, at, sp);
  else
    walk_outputs<T, DK, NW, STAGES, QLDS>(p, rec, w - 1 - NW, at, sp);
}

template <typename T, int DK, int NW>
hipError_t launch_walk(const DeltaArgs& a, int sequences, hipStream_t s) {
  constexpr int kMax = 160 * 1024;
  constexpr bool QLDS = Walk<T, DK, NW, 2, true, true>::kSmem <= kMax;
  constexpr int STAGES = Walk<T, DK, NW, 2, true, QLDS>::kSmem <= kMax ? 2 : 1;
  using G = Walk<T, DK, NW, STAGES, true, QLDS>;
  static_assert(G::kSmem <= kMax, "one stage has to fit");
  auto kern = k_delta_walk<T, DK, NW, STAGES, QLDS>;
  static const hipError_t set =
      hipFuncSetAttribute((const void*)kern, hipFuncAttributeMaxDynamicSharedMemorySize, G::kSmem);
  if (set != hipSuccess) return set;
  const int64_t blocks = walk_blocks((int64_t)sequences * a.Hk, a.Hv / a.Hk * ((a.dv + 16 * NW - 1) / (16 * NW)));
  kern<<<dim3((unsigned)blocks), G::kThreads, G::kSmem, s>>>(a, a.ws, sequences);
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
    k_delta_chunks<T, false><<<dim3((unsigned)(slots * a.Hv)), kChunkThreads, 0, s>>>(a, a.ws, nullptr);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const int sequences = a.seqs.starts ? a.seqs.num : a.batch;
  if (sequences == 0) return hipSuccess;
  if (a.dk <= 64) return launch_walk<T, 64, 2>(a, sequences, s);
  if (a.dk <= 128) return launch_walk<T, 128, 2>(a, sequences, s);
  return launch_walk<T, 256, sizeof(T) == 2 ? 2 : 1>(a, sequences, s);
}

template size_t delta_workspace_bytes<bf16>(const DeltaArgs&);
template size_t delta_workspace_bytes<float>(const DeltaArgs&);
template hipError_t launch_delta<bf16>(const DeltaArgs&, hipStream_t);
template hipError_t launch_delta<float>(const DeltaArgs&, hipStream_t);

}  // namespace ttt
