// Root-mean-square norm of x + residual, forward (in 8 bits too) and backward, for gfx950.
//
//   forward   h = x + residual, rounded to their type,  y = h r w,  r = 1 / sqrt(mean(h^2) + eps)
//   in 8 bits q = e4m3(y / s),  s = max(max |y| / 448, 2^-126) over the row or a group of its columns (y / s as a division
//             rounds it: y times 1 / s falls on the other side of a border between two codes once in 10^5)
//   backward  n = h r, a = dY w:  dx = r (a - n mean(a n)) + dH,  dw = sum_rows dY n
//
// Rows lie in registers as in the layer norm (norm.hip): read once, summed, written once, bound by HBM.  Sums,
// scales and y are fp32; h is rounded before it is squared, so that the norm is of the sum as it is kept and the
// backward pass, which reads it, has the same n.  A group's largest |y| is found among the few lanes that hold its
// columns, a row's among all of its threads.  131,072 x 2560 with residual, bf16 to e4m3 with 128 columns a scale: 433 us,
// 5.5 TB/s; backward of 4,099 x 1001 in fp32 with dH: 17 us, 3.9 TB/s, and 4 us for the weight's sums; of 131,072 x 2560 in
// bf16: 515 us, 5.2 TB/s.
#include "launch.hpp"
#include "norm.hpp"

namespace ttt {
namespace {

constexpr float kE4m3Max = 448.f, kMinScale = 0x1p-126f;
// From this scale on the remainder of a quotient that e4m3 tells from zero (2^-10 and more, 2^-24 of that left) is no
// subnormal.
constexpr float kFullScale = 0x1p-90f;

// The largest of v over the threads of a row, given to all of them; `red` and `turn` as for row_sum.
template <int TPR>
__device__ __forceinline__ float row_max(float v, float* red, int& turn) {
#pragma unroll
  for (int m = (TPR > 0 && TPR < 64 ? TPR : 64) / 2; m > 0; m >>= 1) v = fmaxf(v, __shfl_xor(v, m, 64));
  if constexpr (TPR == 0) {
    float* half = red + turn * 16;
    turn ^= 1;
    if ((threadIdx.x & 63) == 0) half[threadIdx.x >> 6] = v;
    __syncthreads();
    const int waves = blockDim.x >> 6;
    v = 0.f;
    for (int w = 0; w < waves; ++w) v = fmaxf(v, half[w]);
  }
  return v;
}

// Four values to e4m3 (round to nearest even).
__device__ __forceinline__ unsigned pack4_e4m3(float a, float b, float c, float d) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return (unsigned)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
}

// VEC e4m3 values of a row: RAG rows start at any byte and end inside a vector.
template <int VEC, bool RAG, bool STREAM>
__device__ __forceinline__ void store_e4m3(uint8_t* p, const float* v, int left) {
  unsigned w[VEC / 4];
#pragma unroll
  for (int j = 0; j < VEC / 4; ++j) w[j] = pack4_e4m3(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
  if constexpr (!RAG) {
    using W = std::conditional_t<VEC == 8, u32x2, unsigned>;
    W all;
    __builtin_memcpy(&all, w, VEC);
    if constexpr (STREAM)
      __builtin_nontemporal_store(all, reinterpret_cast<W*>(p));
    else
      *reinterpret_cast<W*>(p) = all;
  } else if (left >= VEC) {
    __builtin_memcpy(p, w, VEC);
  } else {
#pragma unroll
    for (int j = 0; j < VEC; ++j)
      if (j < left) p[j] = (uint8_t)(w[j / 4] >> (8 * (j & 3)));
  }
}

// lanes: those that hold a group of columns (a power of two), 0: the scale is the row's.  Four waves a SIMD
// for rows of up to 5 vectors a thread (bf16 to e4m3, 131,072 x 2560: 433 us with 4 of 130 registers spilled, 443 with three
// waves and none).
template <typename T, bool RAG, int TPR, int NV, bool OUT8, bool STREAM>
__global__ __launch_bounds__(TPR == 0 ? 1024 : kNormThreads, NV <= 5 ? 4 : 1) void k_rms(
    const T* __restrict__ x, const T* __restrict__ res, const T* __restrict__ weight, T* __restrict__ ho,
    void* __restrict__ yo, float* __restrict__ rstd, float* __restrict__ scale, int64_t rows, int d, float eps, int lanes) {
  constexpr int VEC = Vec<T>::V;
  const int tpr = TPR ? TPR : (int)blockDim.x, rpb = TPR ? kNormThreads / TPR : 1;
  __shared__ float red[TPR ? 1 : 2 * 16];
  const int t = threadIdx.x % tpr;
  int turn = 0;
  // one turn of this loop, unless there are more rows than a grid may have workgroups
  for (int64_t row = (int64_t)blockIdx.x * rpb + threadIdx.x / tpr; row < rows; row += (int64_t)gridDim.x * rpb) {
    Pack<T, VEC> raw[NV], more[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = (i * tpr + t) * VEC;
      if (e < d) {
        raw[i] = load_pack<T, VEC, RAG, STREAM>(x + row * d + e, d - e);
        if (res) more[i] = load_pack<T, VEC, RAG, STREAM>(res + row * d + e, d - e);
      }
    }
    float v[NV][VEC], s[1] = {0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = (i * tpr + t) * VEC;
      if (e < d) {
        widen(raw[i], v[i]);
        if (res) {
          float o[VEC];
          widen(more[i], o);
#pragma unroll
          for (int j = 0; j < VEC; ++j) v[i][j] += o[j];
          Pack<T, VEC> h;
          narrow(v[i], h);
          store_pack<T, VEC, RAG, STREAM>(ho + row * d + e, h, d - e);
          widen(h, v[i]);
        }
#pragma unroll
        for (int j = 0; j < VEC; ++j) s[0] += v[i][j] * v[i][j];   // elements past the row's end are zero
      }
    }
    row_sum<TPR>(s, red, turn);
    const float r = 1.0f / sqrtf(s[0] / (float)d + eps);
    if (t == 0) rstd[row] = r;
    float most[OUT8 ? NV : 1], all = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = (i * tpr + t) * VEC;
      if (OUT8) most[i] = 0.f;
      if (e < d) {
        float w[VEC];
        if (weight) {
          widen(load_pack<T, VEC, RAG>(weight + e, d - e), w);
        } else {
#pragma unroll
          for (int j = 0; j < VEC; ++j) w[j] = 1.f;
        }
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          v[i][j] = v[i][j] * r * w[j];
          if (OUT8) most[i] = fmaxf(most[i], fabsf(v[i][j]));
        }
        if constexpr (OUT8) {
          all = fmaxf(all, most[i]);
        } else {
          Pack<T, VEC> o;
          narrow(v[i], o);
          store_pack<T, VEC, RAG, STREAM>((T*)yo + row * d + e, o, d - e);
        }
      }
    }
    if constexpr (OUT8) {
      const int cols = lanes * VEC, groups = lanes ? (d + cols - 1) / cols : 1;
      if (lanes == 0) all = row_max<TPR>(all, red, turn);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int e = (i * tpr + t) * VEC;
        float a = all;
        if (lanes) {
          a = most[i];
          for (int m = lanes >> 1; m > 0; m >>= 1) a = fmaxf(a, __shfl_xor(a, m, 64));
        }
        const float sc = fmaxf(a / kE4m3Max, kMinScale), inv = 1.0f / sc;
        if (e < d) {
          if (lanes ? t % lanes == 0 : i == 0 && t == 0) scale[row * groups + (lanes ? e / cols : 0)] = sc;
          // y / sc as a division rounds it: what y inv leaves of y, times inv, puts it right
          if (sc >= kFullScale) {
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
              const float q = v[i][j] * inv;
              v[i][j] = fmaf(fmaf(-q, sc, v[i][j]), inv, q);
            }
          } else {
#pragma unroll
            for (int j = 0; j < VEC; ++j) v[i][j] /= sc;
          }
          store_e4m3<VEC, RAG, STREAM>((uint8_t*)yo + row * d + e, v[i], d - e);
        }
      }
    }
  }
}

// As the layer norm's backward pass: each workgroup takes rows, the next one's loads under way while this one's sums
// are made, and keeps the sums of its columns' dY n in registers; part[blockIdx.x][d] is added up in block order by
// k_norm_grad_sum: no atomics, the same bits every run.  Sums over rows are fp64
// throughout: of terms of either sign off by 4e-8, with fp32 sums by 2e-7 (4,099 x 1001 fp32: 23.0 us in place of 21.5,
// 131,072 x 2560 bf16: 516 in place of 514).
template <typename T, bool RAG, int TPR, int NV>
__global__ __launch_bounds__(TPR == 0 ? 1024 : kNormThreads) void k_rms_grad(
    const T* __restrict__ h, const T* __restrict__ weight, const T* __restrict__ dy, const float* __restrict__ rstd,
    const T* __restrict__ dh, T* __restrict__ dx, double* __restrict__ part, int64_t rows, int d) {
  constexpr int VEC = Vec<T>::V, RPB = TPR ? kNormThreads / TPR : 1;
  const int tpr = TPR ? TPR : (int)blockDim.x;
  __shared__ float red[TPR ? 1 : 2 * 16];
  __shared__ double cols[RPB > 1 ? TPR * VEC * RPB : 1];       // one vector's sums of every row slot
  const int t = threadIdx.x % tpr, slot = threadIdx.x / tpr;
  int turn = 0;
  float w[NV][VEC];
  double dw[NV][VEC];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = (i * tpr + t) * VEC;
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      w[i][j] = 1.f;
      dw[i][j] = 0.0;
    }
    if (weight && e < d) widen(load_pack<T, VEC, RAG>(weight + e, d - e), w[i]);
  }
  struct Row {
    Pack<T, VEC> h[NV], g[NV], u[NV];
    float r;
  };
  auto load = [&](int64_t row, Row& o) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = (i * tpr + t) * VEC;
      if (e < d) {
        o.h[i] = load_pack<T, VEC, RAG>(h + row * d + e, d - e);
        o.g[i] = load_pack<T, VEC, RAG>(dy + row * d + e, d - e);
        if (dh) o.u[i] = load_pack<T, VEC, RAG>(dh + row * d + e, d - e);
      }
    }
    o.r = rstd[row];
  };
  const int64_t step = (int64_t)gridDim.x * RPB;
  int64_t row = (int64_t)blockIdx.x * RPB + slot;
  Row now, next;
  constexpr bool AHEAD = NV == 1 || (NV == 2 && TPR != 0);   // where registers allow it
  if (AHEAD && row < rows) load(row, now);
  for (; row < rows; row += step) {
    if (!AHEAD) load(row, now);
    if (AHEAD && row + step < rows) load(row + step, next);
    float s[1] = {0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if ((i * tpr + t) * VEC < d) {
        float hv[VEC], gv[VEC];
        widen(now.h[i], hv);
        widen(now.g[i], gv);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const float n = hv[j] * now.r;
          s[0] += gv[j] * w[i][j] * n;
          dw[i][j] += gv[j] * n;
        }
      }
    }
    row_sum<TPR>(s, red, turn);
    const float mean = s[0] / (float)d;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = (i * tpr + t) * VEC;
      if (e < d) {
        float hv[VEC], gv[VEC], o[VEC];
        widen(now.h[i], hv);
        widen(now.g[i], gv);
#pragma unroll
        for (int j = 0; j < VEC; ++j) o[j] = now.r * (gv[j] * w[i][j] - hv[j] * now.r * mean);
        if (dh) {
          float u[VEC];
          widen(now.u[i], u);
#pragma unroll
          for (int j = 0; j < VEC; ++j) o[j] += u[j];
        }
        Pack<T, VEC> p;
        narrow(o, p);
        store_pack<T, VEC, RAG>(dx + row * d + e, p, d - e);
      }
    }
    if (AHEAD) now = next;
  }
  double* pw = part + (int64_t)blockIdx.x * d;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = (i * tpr + t) * VEC;
    if constexpr (RPB > 1) {
      __syncthreads();
#pragma unroll
      for (int j = 0; j < VEC; ++j) cols[(slot * VEC + j) * TPR + t] = dw[i][j];
      __syncthreads();
      if (slot == 0 && e < d)
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          double a = 0.0;
          for (int k = 0; k < RPB; ++k) a += cols[(k * VEC + j) * TPR + t];
          if (!RAG || e + j < d) pw[e + j] = a;
        }
    } else if (e < d) {
#pragma unroll
      for (int j = 0; j < VEC; ++j)
        if (!RAG || e + j < d) pw[e + j] = dw[i][j];
    }
  }
}

}  // namespace

template <typename T>
hipError_t launch_rms(const RmsArgs& a, hipStream_t s) {
  const NormPlan p = norm_plan<T>(a.d, 8);
  const int rpb = p.tpr ? p.threads / p.tpr : 1;
  const int64_t grid = std::min<int64_t>((a.rows + rpb - 1) / rpb, 1 << 21);
  // lanes of a group: never more than have a row
  const int lanes = a.group ? std::min(a.group / Vec<T>::V, p.tpr ? p.tpr : 64) : 0;
  return with_plan<T>(p, [&](auto rag, auto tpr, auto nv) {
    auto go = [&](auto out8, auto streams) {
      k_rms<T, decltype(rag)::value, decltype(tpr)::value, decltype(nv)::value, decltype(out8)::value,
            decltype(streams)::value><<<dim3((unsigned)grid), p.threads, 0, s>>>(
          (const T*)a.x, (const T*)a.residual, (const T*)a.weight, (T*)a.h, a.y, a.rstd, a.scale, a.rows, a.d, a.eps, lanes);
      return hipGetLastError();
    };
    // x, the residual and h, and y
    const int64_t bytes = a.rows * a.d * ((a.residual ? 3 : 1) * (int)sizeof(T) + (a.scale ? 1 : (int)sizeof(T)));
    if constexpr (!decltype(rag)::value)
      if (bytes > kStreamBytes)
        return a.scale ? go(std::true_type(), std::true_type()) : go(std::false_type(), std::true_type());
    return a.scale ? go(std::true_type(), std::false_type()) : go(std::false_type(), std::false_type());
  });
}

// Workgroups of the backward pass: as the layer norm's.
template <typename T>
int rms_grad_blocks(int64_t rows, int d) {
  const NormPlan p = norm_plan<T>(d, 2);
  const int64_t rpb = p.tpr ? p.threads / p.tpr : 1;
  return (int)std::min<int64_t>((rows + rpb - 1) / rpb, p.tpr ? 1280 : p.threads > 512 ? 512 : 768);
}

template <typename T>
hipError_t launch_rms_grad(const RmsGradArgs& a, hipStream_t s) {
  const NormPlan p = norm_plan<T>(a.d, 2);
  const int G = rms_grad_blocks<T>(a.rows, a.d);
  if (G > 0) {
    hipError_t e = with_plan<T>(p, [&](auto rag, auto tpr, auto nv) {
      k_rms_grad<T, decltype(rag)::value, decltype(tpr)::value, decltype(nv)::value>
          <<<dim3((unsigned)G), p.threads, 0, s>>>((const T*)a.h, (const T*)a.weight, (const T*)a.dy, a.rstd,
                                                   (const T*)a.dh, (T*)a.dx, a.part, a.rows, a.d);
      return hipGetLastError();
    });
    if (e != hipSuccess) return e;
  }
  if (a.dweight == nullptr) return hipSuccess;
  k_norm_grad_sum<double><<<dim3((unsigned)((a.d + 15) / 16), 1), 1024, 0, s>>>(a.part, G, a.d, a.dweight, nullptr);
  return hipGetLastError();
}

#define TTT_RMS(T)                                                     \
  template hipError_t launch_rms<T>(const RmsArgs&, hipStream_t);      \
  template int rms_grad_blocks<T>(int64_t, int);                       \
  template hipError_t launch_rms_grad<T>(const RmsGradArgs&, hipStream_t);
TTT_RMS(bf16)
TTT_RMS(float)

}  // namespace ttt
