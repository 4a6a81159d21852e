// Layer norm over the last index, forward and backward, for gfx950.
//
//   forward   y = (x - mean) rstd w + b,  rstd = 1 / sqrt(mean((x - mean)^2) + eps)
//   backward  h = (x - mean) rstd, a = dY w:
//             dx = rstd (a - mean(a) - h mean(a h)),  dw = sum_rows dY h,  db = sum_rows dY
//
// Both passes are bound by HBM: a row is read once, held in registers between
// the statistics and the output (the variance is the second of two passes over
// the registers, so a large common offset is not squared; the mean itself is
// fp32, so y is off by some 2^-24 of the offset over the row's spread), and
// written once.
// TPR threads share a row, each holding NV vectors of VEC elements; vector i
// of thread t starts at element (i TPR + t) VEC, so a wave's loads are
// contiguous.  Narrower rows (norm_plan) belong to one wave or a quarter of
// one: no barrier, and a workgroup works on 4 rows or more.  Wider rows have a
// workgroup of as many waves as they fill (TPR = 0: its size, up to 1024), one
// vector a thread while that reaches.  VEC = 16 bytes.  RAG: row lengths that
// are no multiple of it: rows then start at any element, so the vectors are
// read and written without alignment, and a row's last one element by element.  Forward 131072 x 2560 bf16: 280
// us, 4.8 TB/s; backward 32768 x 2560: 106 us, 524288 x 128: 81 us, 5 TB/s.  fp32
// 32768 x 1024: forward 44 us, backward 96 us (4.2 TB/s); 16384 x 2560, wider than
// a wave's rows: 99 and 100 us (3.4 and 5.0 TB/s).
#include "launch.hpp"
#include "norm.hpp"

namespace ttt {
namespace {

template <typename T, bool RAG, int TPR, int NV>
__global__ __launch_bounds__(TPR == 0 ? 1024 : kNormThreads) void k_norm(
    const T* __restrict__ x, const T* __restrict__ weight, const T* __restrict__ bias, T* __restrict__ y,
    float* __restrict__ mean, float* __restrict__ rstd, int64_t rows, int d, float eps) {
  constexpr int VEC = Vec<T>::V;
  const int tpr = TPR ? TPR : (int)blockDim.x, rpb = TPR ? kNormThreads / TPR : 1;
  __shared__ float red[TPR ? 1 : 2 * 16];
  const int t = threadIdx.x % tpr;
  int turn = 0;
  // one turn of this loop, unless there are more rows than a grid may have workgroups
  for (int64_t row = (int64_t)blockIdx.x * rpb + threadIdx.x / tpr; row < rows; row += (int64_t)gridDim.x * rpb) {
    const T* xr = x + row * d;
    Pack<T, VEC> raw[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = (i * tpr + t) * VEC;
      if (e < d) raw[i] = load_pack<T, VEC, RAG>(xr + e, d - e);
    }
    float v[NV][VEC];
    float s[1] = {0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if ((i * tpr + t) * VEC < d) {
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
      if ((i * tpr + t) * VEC < d) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          v[i][j] = !RAG || (i * tpr + t) * VEC + j < d ? v[i][j] - mu : 0.f;
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
      const int e = (i * tpr + t) * VEC;
      if (e < d) {
        float w[VEC], b[VEC];
        if (weight) {
          widen(load_pack<T, VEC, RAG>(weight + e, d - e), w);
        } else {
#pragma unroll
          for (int j = 0; j < VEC; ++j) w[j] = 1.f;
        }
        if (bias) {
          widen(load_pack<T, VEC, RAG>(bias + e, d - e), b);
        } else {
#pragma unroll
          for (int j = 0; j < VEC; ++j) b[j] = 0.f;
        }
#pragma unroll
        for (int j = 0; j < VEC; ++j) v[i][j] = v[i][j] * r * w[j] + b[j];
        Pack<T, VEC> o;
        narrow(v[i], o);
        store_pack<T, VEC, RAG>(yr + e, o, d - e);
      }
    }
  }
}

// Each workgroup takes rows blockIdx.x rpb + i, stepping by gridDim.x rpb, the
// next row's loads under way while this one's sums are made, and keeps the sums
// of its columns' dY h and dY in registers; its rows' sums meet in LDS at the
// end and go to part[blockIdx.x][2][d], which k_norm_grad_sum adds up in block
// order: no atomics, the same bits every run.
template <typename T, bool RAG, int TPR, int NV>
__global__ __launch_bounds__(TPR == 0 ? 1024 : kNormThreads) void k_norm_grad(
    const T* __restrict__ x, const T* __restrict__ weight, const T* __restrict__ dy, const float* __restrict__ mean,
    const float* __restrict__ rstd, T* __restrict__ dx, float* __restrict__ part, int64_t rows, int d, bool want_db) {
  constexpr int VEC = Vec<T>::V, RPB = TPR ? kNormThreads / TPR : 1;
  const int tpr = TPR ? TPR : (int)blockDim.x;
  __shared__ float red[TPR ? 1 : 4 * 16];
  __shared__ float cols[RPB > 1 ? TPR * VEC * RPB : 1];       // one vector's sums of every row slot
  const int t = threadIdx.x % tpr, slot = threadIdx.x / tpr;
  int turn = 0;
  float w[NV][VEC], dw[NV][VEC], db[NV][VEC];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = (i * tpr + t) * VEC;
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      w[i][j] = 1.f;
      dw[i][j] = db[i][j] = 0.f;
    }
    if (weight && e < d) widen(load_pack<T, VEC, RAG>(weight + e, d - e), w[i]);
  }
  struct Row {
    Pack<T, VEC> x[NV], g[NV];
    float mu, r;
  };
  auto load = [&](int64_t row, Row& o) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = (i * tpr + t) * VEC;
      if (e < d) {
        o.x[i] = load_pack<T, VEC, RAG>(x + row * d + e, d - e);
        o.g[i] = load_pack<T, VEC, RAG>(dy + row * d + e, d - e);
      }
    }
    o.mu = mean[row];
    o.r = rstd[row];
  };
  const int64_t step = (int64_t)gridDim.x * RPB;
  int64_t row = (int64_t)blockIdx.x * RPB + slot;
  Row now, next;
  constexpr bool AHEAD = NV <= 2;                 // where registers allow it
  if (AHEAD && row < rows) load(row, now);
  for (; row < rows; row += step) {
    if (!AHEAD) load(row, now);
    if (AHEAD && row + step < rows) load(row + step, next);
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if ((i * tpr + t) * VEC < d) {
        float xv[VEC], gv[VEC];
        widen(now.x[i], xv);
        widen(now.g[i], gv);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const float h = (xv[j] - now.mu) * now.r, a = gv[j] * w[i][j];
          s[0] += a;
          s[1] += a * h;
          dw[i][j] += gv[j] * h;
          db[i][j] += gv[j];
        }
      }
    }
    row_sum<TPR>(s, red, turn);
    const float ma = s[0] / (float)d, mah = s[1] / (float)d;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = (i * tpr + t) * VEC;
      if (e < d) {
        float xv[VEC], gv[VEC], o[VEC];
        widen(now.x[i], xv);
        widen(now.g[i], gv);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const float h = (xv[j] - now.mu) * now.r;
          o[j] = now.r * (gv[j] * w[i][j] - ma - h * mah);
        }
        Pack<T, VEC> p;
        narrow(o, p);
        store_pack<T, VEC, RAG>(dx + row * d + e, p, d - e);
      }
    }
    if (AHEAD) now = next;
  }
  float* pw = part + (int64_t)blockIdx.x * 2 * d;
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    if (q == 1 && !want_db) break;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = (i * tpr + t) * VEC;
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
            if (!RAG || e + j < d) pw[(int64_t)q * d + e + j] = a;
          }
      } else if (e < d) {
#pragma unroll
        for (int j = 0; j < VEC; ++j)
          if (!RAG || e + j < d) pw[(int64_t)q * d + e + j] = mine[j];
      }
    }
  }
}

}  // namespace

template <typename T>
hipError_t launch_norm(const T* x, const T* w, const T* b, T* y, float* mean, float* rstd, int64_t rows, int d,
                       float eps, hipStream_t s) {
  const NormPlan p = norm_plan<T>(d, 8);
  const int rpb = p.tpr ? p.threads / p.tpr : 1;
  const int64_t grid = std::min<int64_t>((rows + rpb - 1) / rpb, 1 << 21);
  return with_plan<T>(p, [&](auto rag, auto tpr, auto nv) {
    k_norm<T, decltype(rag)::value, decltype(tpr)::value, decltype(nv)::value>
        <<<dim3((unsigned)grid), p.threads, 0, s>>>(x, w, b, y, mean, rstd, rows, d, eps);
    return hipGetLastError();
  });
}

// Workgroups of the backward pass: enough to keep the 256 CUs' loads under
// way, and few enough that the partial sums (8 d bytes a workgroup, written and
// read) stay small beside the rows.
template <typename T>
int norm_grad_blocks(int64_t rows, int d) {
  const NormPlan p = norm_plan<T>(d, 2);
  const int64_t rpb = p.tpr ? p.threads / p.tpr : 1;
  return (int)std::min<int64_t>((rows + rpb - 1) / rpb, p.tpr ? 1280 : p.threads > 512 ? 512 : 768);
}

template <typename T>
hipError_t launch_norm_grad(const T* x, const T* w, const T* dy, const float* mean, const float* rstd, T* dx,
                            float* dw, float* db, float* part, int64_t rows, int d, hipStream_t s) {
  const NormPlan p = norm_plan<T>(d, 2);
  const int G = norm_grad_blocks<T>(rows, d);
  if (G > 0) {
    hipError_t e = with_plan<T>(p, [&](auto rag, auto tpr, auto nv) {
      k_norm_grad<T, decltype(rag)::value, decltype(tpr)::value, decltype(nv)::value>
          <<<dim3((unsigned)G), p.threads, 0, s>>>(x, w, dy, mean, rstd, dx, part, rows, d, db != nullptr);
      return hipGetLastError();
    });
    if (e != hipSuccess) return e;
  }
  if (dw == nullptr && db == nullptr) return hipSuccess;
  k_norm_grad_sum<float><<<dim3((unsigned)((d + 15) / 16), 2), 1024, 0, s>>>(part, G, d, dw, db);
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
