// What the norms' kernels share (gfx950): rows of elements in vectors,
// sums over the threads of a row, the variant for a row's width, and the
// columns' sums of their backward passes.  How the threads hold a row is in
// norm.hip.
#pragma once
#include <algorithm>

#include "common.hpp"

namespace ttt {
namespace {

constexpr int kNormThreads = 256;

// VEC consecutive elements as they are stored (bf16 stays packed until used).
template <typename T, int VEC> struct Pack;
template <> struct Pack<bf16, 8> { u32x4 w; };
template <> struct Pack<bf16, 4> { u32x2 w; };
template <> struct Pack<float, 4> { f32x4 w; };

__device__ __forceinline__ void widen(const Pack<bf16, 8>& p, float* o) { unpack8(p.w, o); }
__device__ __forceinline__ void widen(const Pack<bf16, 4>& p, float* o) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    o[2 * i] = __uint_as_float(p.w[i] << 16);
    o[2 * i + 1] = __uint_as_float(p.w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void widen(const Pack<float, 4>& p, float* o) {
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = p.w[i];
}

__device__ __forceinline__ void narrow(const float* o, Pack<bf16, 8>& p) {
#pragma unroll
  for (int i = 0; i < 4; ++i) p.w[i] = pack2_bf16(o[2 * i], o[2 * i + 1]);
}
__device__ __forceinline__ void narrow(const float* o, Pack<bf16, 4>& p) {
  p.w = (u32x2){pack2_bf16(o[0], o[1]), pack2_bf16(o[2], o[3])};
}
__device__ __forceinline__ void narrow(const float* o, Pack<float, 4>& p) { p.w = (f32x4){o[0], o[1], o[2], o[3]}; }

// `left` elements remain from p to the row's end (RAG; else they are VEC or more); those past it are zero.  STREAM:
// what passes by is not kept in the caches.
template <typename T, int VEC, bool RAG, bool STREAM = false>
__device__ __forceinline__ Pack<T, VEC> load_pack(const T* p, int left) {
  if constexpr (STREAM && !RAG) {
    const auto* at = reinterpret_cast<const Pack<T, VEC>*>(p);
    return {__builtin_nontemporal_load(&at->w)};
  }
  if constexpr (!RAG) return *reinterpret_cast<const Pack<T, VEC>*>(p);
  Pack<T, VEC> o;
  if (left >= VEC) {
    __builtin_memcpy(&o, p, sizeof(o));
  } else {
    T e[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) e[j] = j < left ? p[j] : (T)0.f;
    __builtin_memcpy(&o, e, sizeof(o));
  }
  return o;
}
template <typename T, int VEC, bool RAG, bool STREAM = false>
__device__ __forceinline__ void store_pack(T* p, const Pack<T, VEC>& v, int left) {
  if constexpr (STREAM && !RAG) {
    __builtin_nontemporal_store(v.w, &reinterpret_cast<Pack<T, VEC>*>(p)->w);
  } else if constexpr (!RAG) {
    *reinterpret_cast<Pack<T, VEC>*>(p) = v;
  } else if (left >= VEC) {
    __builtin_memcpy(p, &v, sizeof(v));
  } else {
    T e[VEC];
    __builtin_memcpy(e, &v, sizeof(v));
#pragma unroll
    for (int j = 0; j < VEC; ++j)
      if (j < left) p[j] = e[j];
  }
}

// Sums of N values over the threads of a row, given to all of them.  Where a
// workgroup has the row (TPR = 0) the waves' sums meet in `red`; `turn`
// alternates between its two halves, so that one barrier a sum is enough.
template <int TPR, int N>
__device__ __forceinline__ void row_sum(float (&v)[N], float* red, int& turn) {
#pragma unroll
  for (int m = (TPR > 0 && TPR < 64 ? TPR : 64) / 2; m > 0; m >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor(v[i], m, 64);
  if constexpr (TPR == 0) {
    const int waves = blockDim.x >> 6;
    float* half = red + turn * (N * 16);
    turn ^= 1;
    if ((threadIdx.x & 63) == 0)
#pragma unroll
      for (int i = 0; i < N; ++i) half[i * 16 + (threadIdx.x >> 6)] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      v[i] = 0.f;
      for (int w = 0; w < waves; ++w) v[i] += half[i * 16 + w];
    }
  }
}

// dw[c], db[c] = the sums, of type S, of part[0..G)[.][c] (gridDim.y 1: dw alone): a workgroup
// takes 16 columns of one of the two, its 64 rows of threads every 64th block each (narrow columns
// of many rows, so that few blocks' sums are read one after the other also
// where d is small), joined in LDS in a fixed order.
template <typename S>
__global__ __launch_bounds__(1024) void k_norm_grad_sum(const S* __restrict__ part, int G, int d,
                                                        float* __restrict__ dw, float* __restrict__ db) {
  __shared__ S sum[64][16];
  const int j = threadIdx.x & 15, k = threadIdx.x >> 4, c = blockIdx.x * 16 + j, q = blockIdx.y;
  float* out = q == 0 ? dw : db;
  if (out == nullptr) return;
  S a = 0;
  if (c < d) {
#pragma unroll 4
    for (int g = k; g < G; g += 64) a += part[((int64_t)g * gridDim.y + q) * d + c];
  }
  sum[k][j] = a;
  __syncthreads();
  if (k == 0 && c < d) {
    a = 0;
#pragma unroll
    for (int i = 0; i < 64; ++i) a += sum[i][j];
    out[c] = (float)a;
  }
}

// The variant for rows of d elements.
struct NormPlan {
  bool rag;
  int tpr, threads, nv;           // threads: of a workgroup; tpr 0: all of them share a row
};
// A wave has rows of up to 64 `most` vectors: forward 8, backward 2.  Measured
// (bf16, us; a wave a row / a workgroup a row): forward 131072 x 2560 296 /
// 411, 32768 x 1024 fp32 46 / 57; backward 131072 x 2560 545 / 396, 16384 x
// 4096 153 / 103.  The forward pass has nothing to wait for but its loads, which
// a wave's own registers keep under way; the backward's three rows of registers
// leave too few waves for that.
template <typename T>
NormPlan norm_plan(int d, int most) {
  constexpr int V = Vec<T>::V;
  NormPlan p;
  p.rag = d % V != 0;
  const int units = (d + V - 1) / V;
  p.threads = kNormThreads;
  p.nv = 1;
  if (units <= 16) {
    p.tpr = 16;
  } else if (units <= 64 * most) {
    p.tpr = 64;
    p.nv = (units + 63) / 64;
  } else {
    p.tpr = 0;
    p.nv = (units + 1023) / 1024;
    p.threads = (units + 64 * p.nv - 1) / (64 * p.nv) * 64;
  }
  return p;
}

// Counts of vectors a thread that have a kernel: the next larger one serves.
template <typename T, typename F>
hipError_t with_plan(const NormPlan& p, F f) {
  using std::integral_constant;
  auto with_tpr = [&](auto rag, auto nv) {
    constexpr int NV = decltype(nv)::value;
    if (p.tpr == 0) return f(rag, integral_constant<int, 0>(), nv);
    if constexpr (NV <= 8) {
      if (p.tpr == 64) return f(rag, integral_constant<int, 64>(), nv);
    }
    if constexpr (NV == 1) {
      if (p.tpr == 16) return f(rag, integral_constant<int, 16>(), nv);
    }
    return hipErrorInvalidValue;
  };
  auto go = [&](auto rag) {
    switch (p.nv) {
      case 1: return with_tpr(rag, integral_constant<int, 1>());
      case 2: return with_tpr(rag, integral_constant<int, 2>());
      case 3: return with_tpr(rag, integral_constant<int, 3>());
      case 4: return with_tpr(rag, integral_constant<int, 4>());
      case 5: return with_tpr(rag, integral_constant<int, 5>());
      case 6: return with_tpr(rag, integral_constant<int, 6>());
      case 7:
      case 8: return with_tpr(rag, integral_constant<int, 8>());
      default:                    // fp32 rows of more than 32768
        if constexpr (sizeof(T) == 4) return with_tpr(rag, integral_constant<int, 16>());
        return hipErrorInvalidValue;
    }
  };
  return p.rag ? go(std::true_type()) : go(std::false_type());
}

}  // namespace
}  // namespace ttt
