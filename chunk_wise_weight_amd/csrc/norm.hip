// Layer norm over the last index, forward and backward, for gfx950.
//
//   forward   y = (x - mean) rstd w + b,  rstd = 1 / sqrt(mean((x - mean)^2) + eps)
//   backward  h = (x - mean) rstd, a = dY w:
//             dx = rstd (a - mean(a) - h mean(a h)),  dw = sum_rows dY h,  db = sum_rows dY
//
// Both passes are bound by HBM: a row is read once, held in registers between
// the statistics and the output (the variance is the second of two passes over
// the registers, so a large common offset costs no digits), and written once.
// TPR threads share a row, each holding NV vectors of VEC elements; vector i
// of thread t starts at element (i TPR + t) VEC, so a wave's loads are
// contiguous.  Rows of up to 64 x 8 vectors belong to one wave or a part of
// one: no barrier, and a workgroup works on 4 rows or more.  VEC = 16 bytes
// where the row length keeps every row 16-byte aligned, else 1.
#include <algorithm>

#include "common.hpp"
#include "launch.hpp"

namespace ttt {
namespace {

constexpr int kNormThreads = 256;

// VEC consecutive elements as they are stored (bf16 stays packed until used).
template <typename T, int VEC> struct Pack;
template <> struct Pack<bf16, 8> { u32x4 w; };
template <> struct Pack<float, 4> { f32x4 w; };
template <> struct Pack<bf16, 1> { bf16 w; };
template <> struct Pack<float, 1> { float w; };

__device__ __forceinline__ void widen(const Pack<bf16, 8>& p, float* o) { unpack8(p.w, o); }
__device__ __forceinline__ void widen(const Pack<float, 4>& p, float* o) {
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = p.w[i];
}
__device__ __forceinline__ void widen(const Pack<bf16, 1>& p, float* o) { o[0] = to_f32(p.w); }
__device__ __forceinline__ void widen(const Pack<float, 1>& p, float* o) { o[0] = p.w; }

__device__ __forceinline__ void narrow(const float* o, Pack<bf16, 8>& p) {
#pragma unroll
  for (int i = 0; i < 4; ++i) p.w[i] = pack2_bf16(o[2 * i], o[2 * i + 1]);
}
__device__ __forceinline__ void narrow(const float* o, Pack<float, 4>& p) { p.w = (f32x4){o[0], o[1], o[2], o[3]}; }
__device__ __forceinline__ void narrow(const float* o, Pack<bf16, 1>& p) { p.w = from_f32<bf16>(o[0]); }
__device__ __forceinline__ void narrow(const float* o, Pack<float, 1>& p) { p.w = o[0]; }

template <typename T, int VEC>
__device__ __forceinline__ Pack<T, VEC> load_pack(const T* p) {
  return *reinterpret_cast<const Pack<T, VEC>*>(p);
}
template <typename T, int VEC>
__device__ __forceinline__ void store_pack(T* p, const Pack<T, VEC>& v) {
  *reinterpret_cast<Pack<T, VEC>*>(p) = v;
}

// Sums of N values over the TPR threads of a row, given to all of them.  Above
// one wave the waves' sums meet in `red`; `turn` alternates between its two
// halves, so that one barrier a sum is enough.
template <int TPR, int N>
__device__ __forceinline__ void row_sum(float (&v)[N], float* red, int& turn) {
#pragma unroll
  for (int m = (TPR < 64 ? TPR : 64) / 2; m > 0; m >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor(v[i], m, 64);
  if constexpr (TPR > 64) {
    constexpr int W = TPR / 64;
    float* half = red + turn * (N * W);
    turn ^= 1;
    if ((threadIdx.x & 63) == 0)
#pragma unroll
      for (int i = 0; i < N; ++i) half[i * W + (threadIdx.x >> 6)] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      v[i] = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) v[i] += half[i * W + w];
    }
  }
}

template <typename T, int VEC, int TPR, int NV>
__global__ __launch_bounds__(TPR > kNormThreads ? TPR : kNormThreads) void k_norm(
    const T* __restrict__ x, const T* __restrict__ weight, const T* __restrict__ bias, T* __restrict__ y,
    float* __restrict__ mean, float* __restrict__ rstd, int64_t rows, int d, float eps) {
  constexpr int BT = TPR > kNormThreads ? TPR : kNormThreads, RPB = BT / TPR;
  __shared__ float red[TPR > 64 ? 2 * (TPR / 64) : 1];
  const int t = threadIdx.x % TPR;
  int turn = 0;
  // one turn of this loop, unless there are more rows than a grid may have workgroups
  for (int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR; row < rows; row += (int64_t)gridDim.x * RPB) {
    const T* xr = x + row * d;
    Pack<T, VEC> raw[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = (i * TPR + t) * VEC;
      if (e < d) raw[i] = load_pack<T, VEC>(xr + e);
    }
    float v[NV][VEC];
    float s[1] = {0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if ((i * TPR + t) * VEC < d) {
        widen(raw[i], v[i]);
#pragma unroll
        for (int j = 0; j < VEC; ++j) s[0] += v[i][j];
      }
    }
    row_sum<TPR>(s, red, turn);
    const float mu = s[0] / (float)d;
    s[0] = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if ((i * TPR + t) * VEC < d) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          v[i][j] -= mu;
          s[0] += v[i][j] * v[i][j];
        }
      }
    }
    row_sum<TPR>(s, red, turn);
    const float r = 1.0f / sqrtf(s[0] / (float)d + eps);
    if (t == 0) {
      mean[row] = mu;
      rstd[row] = r;
    }
    T* yr = y + row * d;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = (i * TPR + t) * VEC;
      if (e < d) {
        float w[VEC], b[VEC];
        if (weight) {
          widen(load_pack<T, VEC>(weight + e), w);
        } else {
#pragma unroll
          for (int j = 0; j < VEC; ++j) w[j] = 1.f;
        }
        if (bias) {
          widen(load_pack<T, VEC>(bias + e), b);
        } else {
#pragma unroll
          for (int j = 0; j < VEC; ++j) b[j] = 0.f;
        }
#pragma unroll
        for (int j = 0; j < VEC; ++j) v[i][j] = v[i][j] * r * w[j] + b[j];
        Pack<T, VEC> o;
        narrow(v[i], o);
        store_pack<T, VEC>(yr + e, o);
      }
    }
  }
}

// Each workgroup takes rows blockIdx.x RPB + i, stepping by gridDim.x RPB, and
// keeps the sums of its columns' dY h and dY in registers; the RPB row slots'
// sums meet in LDS at the end and go to part[blockIdx.x][2][d], which
// k_norm_grad_sum adds up in block order: no atomics, the same bits every run.
template <typename T, int VEC, int TPR, int NV>
__global__ __launch_bounds__(TPR > kNormThreads ? TPR : kNormThreads) void k_norm_grad(
    const T* __restrict__ x, const T* __restrict__ weight, const T* __restrict__ dy, const float* __restrict__ mean,
    const float* __restrict__ rstd, T* __restrict__ dx, float* __restrict__ part, int64_t rows, int d, bool want_db) {
  constexpr int BT = TPR > kNormThreads ? TPR : kNormThreads, RPB = BT / TPR;
  __shared__ float red[TPR > 64 ? 4 * (TPR / 64) : 1];
  // sums of the row slots: one slot's columns at a time
  __shared__ float cols[RPB > 1 ? TPR * VEC * RPB : 1];
  const int t = threadIdx.x % TPR, slot = threadIdx.x / TPR;
  int turn = 0;
  float w[NV][VEC], dw[NV][VEC], db[NV][VEC];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = (i * TPR + t) * VEC;
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      w[i][j] = 1.f;
      dw[i][j] = db[i][j] = 0.f;
    }
    if (weight && e < d) widen(load_pack<T, VEC>(weight + e), w[i]);
  }
  const int64_t step = (int64_t)gridDim.x * RPB;
  for (int64_t row = (int64_t)blockIdx.x * RPB + slot; row < rows; row += step) {
    const T* xr = x + row * d;
    const T* gr = dy + row * d;
    Pack<T, VEC> px[NV], pg[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = (i * TPR + t) * VEC;
      if (e < d) {
        px[i] = load_pack<T, VEC>(xr + e);
        pg[i] = load_pack<T, VEC>(gr + e);
      }
    }
    const float mu = mean[row], r = rstd[row];
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if ((i * TPR + t) * VEC < d) {
        float xv[VEC], gv[VEC];
        widen(px[i], xv);
        widen(pg[i], gv);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const float h = (xv[j] - mu) * r, a = gv[j] * w[i][j];
          s[0] += a;
          s[1] += a * h;
          dw[i][j] += gv[j] * h;
          db[i][j] += gv[j];
        }
      }
    }
    row_sum<TPR>(s, red, turn);
    const float ma = s[0] / (float)d, mah = s[1] / (float)d;
    T* dr = dx + row * d;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = (i * TPR + t) * VEC;
      if (e < d) {
        float xv[VEC], gv[VEC], o[VEC];
        widen(px[i], xv);
        widen(pg[i], gv);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const float h = (xv[j] - mu) * r;
          o[j] = r * (gv[j] * w[i][j] - ma - h * mah);
        }
        Pack<T, VEC> p;
        narrow(o, p);
        store_pack<T, VEC>(dr + e, p);
      }
    }
  }
  float* pw = part + (int64_t)blockIdx.x * 2 * d;
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    if (q == 1 && !want_db) break;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = (i * TPR + t) * VEC;
      float* mine = q == 0 ? dw[i] : db[i];
      if constexpr (RPB > 1) {
        __syncthreads();
#pragma unroll
        for (int j = 0; j < VEC; ++j) cols[(slot * VEC + j) * TPR + t] = mine[j];
        __syncthreads();
        if (slot == 0 && e < d)
#pragma unroll
          for (int j = 0; j < VEC; ++j) {
            float a = 0.f;
            for (int k = 0; k < RPB; ++k) a += cols[(k * VEC + j) * TPR + t];
            pw[(int64_t)q * d + e + j] = a;
          }
      } else if (e < d) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) pw[(int64_t)q * d + e + j] = mine[j];
      }
    }
  }
}

// dw[c], db[c] = the sums of part[0..G)[.][c]: a workgroup takes 64 columns of
// one of the two, its 16 rows of threads every 16th block each, joined in LDS.
__global__ __launch_bounds__(1024) void k_norm_grad_sum(const float* __restrict__ part, int G, int d,
                                                        float* __restrict__ dw, float* __restrict__ db) {
  __shared__ float sum[16][64];
  const int c = blockIdx.x * 64 + (threadIdx.x & 63), k = threadIdx.x >> 6, q = blockIdx.y;
  float* out = q == 0 ? dw : db;
  if (out == nullptr) return;
  float a = 0.f;
  if (c < d)
    for (int g = k; g < G; g += 16) a += part[((int64_t)g * 2 + q) * d + c];
  sum[k][threadIdx.x & 63] = a;
  __syncthreads();
  if (k == 0 && c < d) {
    a = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) a += sum[i][threadIdx.x & 63];
    out[c] = a;
  }
}

// The variant for rows of d elements: the fewest threads a row (16, 64, 256,
// 1024) that hold it in at most 8 vectors each (64 single elements).
struct NormPlan {
  bool vec;
  int tpr, nv;
};
template <typename T>
NormPlan norm_plan(int d) {
  constexpr int V = Vec<T>::V;
  NormPlan p;
  p.vec = d % V == 0;
  const int units = p.vec ? d / V : d;
  const int most = p.vec ? 8 : 16;
  p.tpr = units <= 16 ? 16 : units <= 64 * most ? 64 : units <= 256 * most ? 256 : 1024;
  p.nv = (units + p.tpr - 1) / p.tpr;
  return p;
}

// Counts of vectors a thread that have a kernel: the next larger one serves.
template <bool VECTORS, typename F>
hipError_t with_nv(int nv, F f) {
  if constexpr (VECTORS) {
    switch (nv) {
      case 1: return f(std::integral_constant<int, 1>());
      case 2: return f(std::integral_constant<int, 2>());
      case 3: return f(std::integral_constant<int, 3>());
      case 4: return f(std::integral_constant<int, 4>());
      case 5: return f(std::integral_constant<int, 5>());
      case 6: return f(std::integral_constant<int, 6>());
      case 7:
      case 8: return f(std::integral_constant<int, 8>());
      default: return f(std::integral_constant<int, 16>());   // fp32 rows of more than 32768
    }
  } else {
    if (nv <= 4) return f(std::integral_constant<int, 4>());
    if (nv <= 16) return f(std::integral_constant<int, 16>());
    return f(std::integral_constant<int, 64>());
  }
}

template <typename T, typename F>
hipError_t with_plan(const NormPlan& p, F f) {
  auto tpr = [&](auto vec) {
    constexpr int VEC = decltype(vec)::value;
    return with_nv<(VEC > 1)>(p.nv, [&](auto nv) {
      constexpr int NV = decltype(nv)::value;
      if constexpr (VEC > 1 ? NV == 1 : NV == 4) {
        if (p.tpr == 16) return f(vec, std::integral_constant<int, 16>(), nv);
      }
      if constexpr (NV <= (VEC > 1 ? 8 : 16)) {
        if (p.tpr == 64) return f(vec, std::integral_constant<int, 64>(), nv);
        if (p.tpr == 256) return f(vec, std::integral_constant<int, 256>(), nv);
      }
      if constexpr (NV == 16 && VEC == 8) return hipErrorInvalidValue;    // 1024 x 8 x 8 is the widest row
      else return f(vec, std::integral_constant<int, 1024>(), nv);
    });
  };
  if (p.vec) return tpr(std::integral_constant<int, Vec<T>::V>());
  return tpr(std::integral_constant<int, 1>());
}

}  // namespace

template <typename T>
hipError_t launch_norm(const T* x, const T* w, const T* b, T* y, float* mean, float* rstd, int64_t rows, int d,
                       float eps, hipStream_t s) {
  const NormPlan p = norm_plan<T>(d);
  return with_plan<T>(p, [&](auto vec, auto tpr, auto nv) {
    constexpr int VEC = decltype(vec)::value, TPR = decltype(tpr)::value, NV = decltype(nv)::value;
    constexpr int BT = TPR > kNormThreads ? TPR : kNormThreads, RPB = BT / TPR;
    const int64_t grid = std::min<int64_t>((rows + RPB - 1) / RPB, 1 << 21);
    k_norm<T, VEC, TPR, NV><<<dim3((unsigned)grid), BT, 0, s>>>(x, w, b, y, mean, rstd, rows, d, eps);
    return hipGetLastError();
  });
}

// Workgroups of the backward pass: enough to fill the 256 CUs, and no more
// than 4 a CU, so that the partial sums (8 d bytes a workgroup) stay small.
template <typename T>
int norm_grad_blocks(int64_t rows, int d) {
  const NormPlan p = norm_plan<T>(d);
  const int64_t rpb = std::max(kNormThreads, p.tpr) / p.tpr;
  return (int)std::min<int64_t>((rows + rpb - 1) / rpb, p.tpr == 1024 ? 512 : 1024);
}

template <typename T>
hipError_t launch_norm_grad(const T* x, const T* w, const T* dy, const float* mean, const float* rstd, T* dx,
                            float* dw, float* db, float* part, int64_t rows, int d, hipStream_t s) {
  const NormPlan p = norm_plan<T>(d);
  const int G = norm_grad_blocks<T>(rows, d);
  if (G > 0) {
    hipError_t e = with_plan<T>(p, [&](auto vec, auto tpr, auto nv) {
      constexpr int VEC = decltype(vec)::value, TPR = decltype(tpr)::value, NV = decltype(nv)::value;
      constexpr int BT = TPR > kNormThreads ? TPR : kNormThreads;
      k_norm_grad<T, VEC, TPR, NV><<<dim3((unsigned)G), BT, 0, s>>>(x, w, dy, mean, rstd, dx, part, rows, d,
                                                                   db != nullptr);
      return hipGetLastError();
    });
    if (e != hipSuccess) return e;
  }
  if (dw == nullptr && db == nullptr) return hipSuccess;
  k_norm_grad_sum<<<dim3((unsigned)((d + 63) / 64), 2), 1024, 0, s>>>(part, G, d, dw, db);
  return hipGetLastError();
}

#define TTT_NORM(T)                                                                                               \
  template hipError_t launch_norm<T>(const T*, const T*, const T*, T*, float*, float*, int64_t, int, float,       \
                                     hipStream_t);                                                                \
  template int norm_grad_blocks<T>(int64_t, int);                                                                 \
  template hipError_t launch_norm_grad<T>(const T*, const T*, const T*, const float*, const float*, T*, float*,   \
                                          float*, float*, int64_t, int, hipStream_t);
TTT_NORM(bf16)
TTT_NORM(float)

}  // namespace ttt
