// One token of the selective scan for every row of a serving batch (gfx950).
//
// Per row, head and row p of the state S [P, N], with r the rate and a = exp(A r):
//   S_p <- a S_p + (r x_p) B,   o_p = S_p . C + D x_p
// The state's rows are independent, so a workgroup takes some rows of one head's state, all loads of them in flight
// before the first use, and needs no LDS: S_p . C is summed over the LPR lanes that hold a row.  All sums are fp32, as
// is the state: bound by HBM, 8 bytes a state element (256 rows x 64 heads x 64 x 128: 184 us, 5.7 TB/s; 205 us without
// the streaming form).
#include "scan_rate.hpp"
#include "slots.hpp"
#include "launch.hpp"

namespace ttt {
namespace {

constexpr int kStepWaves = 4;

template <int LPR>
__device__ __forceinline__ float lanes_sum(float x) {
#pragma unroll
  for (int m = LPR / 2; m > 0; m >>= 1) x += __shfl_xor(x, m, 64);
  return x;
}

// LPR lanes hold a state row (4 elements each, N <= 4 LPR); a wave holds 64 / LPR rows at a time and takes IT such groups.
template <typename T, int LPR, int IT, bool STREAM>
__global__ __launch_bounds__(64 * kStepWaves) void k_scan_step(ScanStepArgs p) {
  constexpr int RPW = 64 / LPR;                 // state rows of a wave at a time
  constexpr int ROWS = RPW * IT * kStepWaves;   // state rows of a workgroup
  const int parts = (p.P + ROWS - 1) / ROWS;
  const int part = blockIdx.x % parts, h = (blockIdx.x / parts) % p.H;
  int r = blockIdx.x / parts / p.H;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = (lane % LPR) * 4;               // first of this lane's 4 elements
  const bool in = c < p.N;
  const int j0 = part * ROWS + wave * (RPW * IT) + lane / LPR;
  const int64_t slot = p.slots ? (int64_t)p.slots[r] : (int64_t)r;
  if (slot < 0 || slot >= p.pool) {             // a padding row: no state, its output is zero
    if (lane % LPR == 0)
#pragma unroll
      for (int i = 0; i < IT; ++i)
        if (j0 + i * RPW < p.P) ((T*)p.O)[((int64_t)r * p.H + h) * p.P + j0 + i * RPW] = from_f32<T>(0.f);
    return;
  }
  float* S = p.S + (slot * p.H + h) * (int64_t)p.P * p.N + c;
  f32x4 s[IT];
#pragma unroll
  for (int i = 0; i < IT; ++i) {
    const int j = j0 + i * RPW;
    s[i] = (f32x4){0.f, 0.f, 0.f, 0.f};
    const f32x4* at = reinterpret_cast<const f32x4*>(S + (int64_t)j * p.N);
    if (in && j < p.P) s[i] = STREAM ? __builtin_nontemporal_load(at) : *at;
  }
  // Rows that name the same state take it one after the other, in row order: the first of them carries it through all.
  if (p.slots && next_row(p.slots, r, 0, (int)slot) < r) return;
  const int grp = h / (p.H / p.G);
  const float A = p.A[h], D = p.D ? p.D[h] : 0.f, bias = p.dt_bias ? p.dt_bias[h] : 0.f;
  do {
    const int64_t bc = ((int64_t)r * p.G + grp) * p.N + c, rh = (int64_t)r * p.H + h;
    f32x4 b = {0.f, 0.f, 0.f, 0.f}, q = b;
    if (in) {
      b = load4((const T*)p.B + bc);
      q = load4((const T*)p.C + bc);
    }
    const T* x = (const T*)p.x + rh * p.P;
    T* o = (T*)p.O + rh * p.P;
    float xj[IT];
#pragma unroll
    for (int i = 0; i < IT; ++i) xj[i] = j0 + i * RPW < p.P ? to_f32(x[j0 + i * RPW]) : 0.f;
    const float rate = scan_rate(p.dt[rh], bias, p.softplus), a = exp_neg(A * rate);
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      s[i] = a == 0.f ? (f32x4){0.f, 0.f, 0.f, 0.f} : s[i] * a;   // an emptied state also loses what is not finite
      s[i] += rate * xj[i] * b;
      const float y = lanes_sum<LPR>(s[i][0] * q[0] + s[i][1] * q[1] + s[i][2] * q[2] + s[i][3] * q[3]);
      if (lane % LPR == 0 && j0 + i * RPW < p.P) o[j0 + i * RPW] = from_f32<T>(y + D * xj[i]);
    }
    r = p.slots ? next_row(p.slots, p.rows, r + 1, (int)slot) : p.rows;
  } while (r < p.rows);
#pragma unroll
  for (int i = 0; i < IT; ++i) {
    const int j = j0 + i * RPW;
    f32x4* at = reinterpret_cast<f32x4*>(S + (int64_t)j * p.N);
    if (in && j < p.P) {
      if constexpr (STREAM)
        __builtin_nontemporal_store(s[i], at);
      else
        *at = s[i];
    }
  }
}

template <typename T, int LPR, int IT>
hipError_t launch(const ScanStepArgs& a, hipStream_t s) {
  constexpr int ROWS = 64 / LPR * IT * kStepWaves;
  const int64_t parts = (a.P + ROWS - 1) / ROWS;
  const dim3 grid((unsigned)(parts * a.H * a.rows));
  if (a.rows * (int64_t)a.H * a.P * a.N * 4 > kStreamBytes)
    k_scan_step<T, LPR, IT, true><<<grid, 64 * kStepWaves, 0, s>>>(a);
  else
    k_scan_step<T, LPR, IT, false><<<grid, 64 * kStepWaves, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace

template <typename T>
hipError_t launch_scan_step(const ScanStepArgs& a, hipStream_t s) {
  if (a.N <= 16) return launch<T, 4, 2>(a, s);
  if (a.N <= 32) return launch<T, 8, 4>(a, s);
  if (a.N <= 64) return launch<T, 16, 4>(a, s);
  if (a.N <= 128) return launch<T, 32, 4>(a, s);
  return launch<T, 64, 4>(a, s);
}

template hipError_t launch_scan_step<bf16>(const ScanStepArgs&, hipStream_t);
template hipError_t launch_scan_step<float>(const ScanStepArgs&, hipStream_t);

}  // namespace ttt
