// The gated delta rule over whole sequences, forward (gfx950).
#include "delta_walk.hpp"

namespace ttt {
namespace {

template <typename T, int DK, int NW, int STAGES>
__global__ __launch_bounds__(128 * NW) __attribute__((amdgpu_waves_per_eu(1, 1))) void k_delta_walk(DeltaArgs p, const char* rec) {
  extern __shared__ __attribute__((aligned(16))) char smem[];
  const int parts = (p.dv + 16 * NW - 1) / (16 * NW);
  const int id = xcd_remap(blockIdx.x, gridDim.x);
  const int part = id % parts, h = (id / parts) % p.Hv, seq = id / parts / p.Hv;
  const SeqPlace sp = seq_place(p.seqs, seq);
  if (wave_id() < NW)
    walk_states<T, DK, NW, STAGES, true>(p, rec, nullptr, nullptr, part, h, seq, sp, smem);
  else if (sp.len > 0)
    walk_outputs<T, DK, NW, STAGES>(p, rec, part, h, sp, smem);
}

template <typename T, int DK, int NW>
hipError_t launch_walk(const DeltaArgs& a, int sequences, hipStream_t s) {
  constexpr int STAGES = Walk<T, DK, NW, 2, true>::kSmem <= 160 * 1024 ? 2 : 1;
  using G = Walk<T, DK, NW, STAGES, true>;
  static_assert(G::kSmem <= 160 * 1024, "one stage has to fit");
  auto kern = k_delta_walk<T, DK, NW, STAGES>;
  static const hipError_t set =
      hipFuncSetAttribute((const void*)kern, hipFuncAttributeMaxDynamicSharedMemorySize, G::kSmem);
  if (set != hipSuccess) return set;
  const int64_t parts = (a.dv + 16 * NW - 1) / (16 * NW);
  kern<<<dim3((unsigned)(parts * a.Hv * sequences)), G::kThreads, G::kSmem, s>>>(a, a.ws);
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
