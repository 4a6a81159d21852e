// One token of the gated delta rule for every row of a serving batch (gfx950).
//
// Per row, value head and state row j of W [dv, dk]:
//   u_j = beta (v_j - a W_j.k),  W_j <- a W_j + u_j k,  o_j = scale W_j.q,  a = exp(g)
// The state rows are independent, so a workgroup takes some rows of one head's
// state, all loads of them in flight before the first use, and needs no LDS:
// W_j.k and the old W_j.q are summed over the LPR lanes that hold a row, and
// the new row's product with q is a W_j.q + u_j k.q, so the state is read once
// and written once.  All sums are fp32, as is the state: bound by HBM, 8 bytes
// a state element.  256 rows of 32 heads of 128 x 128: 207 us, 5.2 TB/s.
//
// Named states (slots): every workgroup looks through all rows' slots for
// others of its state, work that grows with the rows' square: 256 rows of 32
// heads of 128 210 us instead of 204, 1024 rows 858 instead of 813, 4096 rows
// 3.76 ms instead of 3.37; 16384 rows of 8 heads of 64 1.72 ms instead of 0.78.
// Hence the limit of 65536 rows.
#include "common.hpp"
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

// The first position >= from of `slot` in slots[0, rows), or rows: blocks of 512 that do not hold it are passed over at
// two loads a lane (4096 rows of 32 heads: 3.76 ms; all of them by 64 slots a time 6.17), the rest goes by 64.
__device__ __forceinline__ int next_row(const int32_t* slots, int rows, int from, int slot) {
  const int lane = threadIdx.x & 63;
  int at = from;
  for (; at + 512 <= rows; at += 512) {
    int4 s[2];
    bool in = false;
#pragma unroll
    for (int i = 0; i < 2; ++i) __builtin_memcpy(&s[i], slots + at + i * 256 + lane * 4, 16);
#pragma unroll
    for (int i = 0; i < 2; ++i) in |= s[i].x == slot | s[i].y == slot | s[i].z == slot | s[i].w == slot;
    if (__ballot(in)) break;
  }
  for (; at < rows; at += 64) {
    const unsigned long long hit = __ballot(at + lane < rows && slots[at + lane < rows ? at + lane : from] == slot);
    if (hit) return at + __builtin_ctzll(hit);
  }
  return rows;
}

// LPR lanes hold a state row (4 elements each, dk <= 4 LPR); a wave holds 64 /
// LPR rows at a time and takes IT such groups.
template <typename T, int LPR, int IT>
__global__ __launch_bounds__(64 * kStepWaves) void k_delta_step(DeltaStepArgs p) {
  constexpr int RPW = 64 / LPR;                 // state rows of a wave at a time
  constexpr int ROWS = RPW * IT * kStepWaves;   // state rows of a workgroup
  const int parts = (p.dv + ROWS - 1) / ROWS;
  const int part = blockIdx.x % parts, h = (blockIdx.x / parts) % p.Hv;
  int r = blockIdx.x / parts / p.Hv;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = (lane % LPR) * 4;               // first of this lane's 4 elements
  const bool in = c < p.dk;
  const int j0 = part * ROWS + wave * (RPW * IT) + lane / LPR;
  const int64_t slot = p.slots ? (int64_t)p.slots[r] : (int64_t)r;
  if (slot < 0 || slot >= p.pool) {             // a padding row: no state, its output is zero
    if (lane % LPR == 0)
#pragma unroll
      for (int i = 0; i < IT; ++i)
        if (j0 + i * RPW < p.dv) ((T*)p.O)[((int64_t)r * p.Hv + h) * p.dv + j0 + i * RPW] = from_f32<T>(0.f);
    return;
  }
  float* W = p.W + (slot * p.Hv + h) * (int64_t)p.dv * p.dk + c;
  f32x4 w[IT];
#pragma unroll
  for (int i = 0; i < IT; ++i) {
    const int j = j0 + i * RPW;
    w[i] = in && j < p.dv ? *reinterpret_cast<const f32x4*>(W + (int64_t)j * p.dk) : (f32x4){0.f, 0.f, 0.f, 0.f};
  }
  // Rows that name the same state take it one after the other, in row order:
  // the first of them carries it through all.
  if (p.slots && next_row(p.slots, r, 0, (int)slot) < r) return;
  const int kh = h / (p.Hv / p.Hk);
  do {
    const int64_t qk = ((int64_t)r * p.Hk + kh) * p.dk + c, rh = (int64_t)r * p.Hv + h;
    f32x4 q = {0.f, 0.f, 0.f, 0.f}, k = q;
    if (in) {
      q = load4((const T*)p.q + qk);
      k = load4((const T*)p.k + qk);
    }
    const float a = __expf(p.g[rh]), beta = p.beta[rh];
    const T* v = (const T*)p.v + rh * p.dv;
    T* o = (T*)p.O + rh * p.dv;
    float vj[IT];
#pragma unroll
    for (int i = 0; i < IT; ++i) vj[i] = j0 + i * RPW < p.dv ? to_f32(v[j0 + i * RPW]) : 0.f;
    const float kq = lanes_sum<LPR>(k[0] * q[0] + k[1] * q[1] + k[2] * q[2] + k[3] * q[3]);
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      w[i] = a == 0.f ? (f32x4){0.f, 0.f, 0.f, 0.f} : w[i] * a;   // a reset also clears what is not finite
      const float wk = lanes_sum<LPR>(w[i][0] * k[0] + w[i][1] * k[1] + w[i][2] * k[2] + w[i][3] * k[3]);
      const float wq = lanes_sum<LPR>(w[i][0] * q[0] + w[i][1] * q[1] + w[i][2] * q[2] + w[i][3] * q[3]);
      const float u = beta * (vj[i] - wk);
      w[i] += u * k;
      if (lane % LPR == 0 && j0 + i * RPW < p.dv) o[j0 + i * RPW] = from_f32<T>(p.scale * (wq + u * kq));
    }
    r = p.slots ? next_row(p.slots, p.rows, r + 1, (int)slot) : p.rows;
  } while (r < p.rows);
#pragma unroll
  for (int i = 0; i < IT; ++i) {
    const int j = j0 + i * RPW;
    if (in && j < p.dv) *reinterpret_cast<f32x4*>(W + (int64_t)j * p.dk) = w[i];
  }
}

template <typename T, int LPR, int IT>
hipError_t launch(const DeltaStepArgs& a, hipStream_t s) {
  constexpr int ROWS = 64 / LPR * IT * kStepWaves;
  const int64_t parts = (a.dv + ROWS - 1) / ROWS;
  k_delta_step<T, LPR, IT><<<dim3((unsigned)(parts * a.Hv * a.rows)), 64 * kStepWaves, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace

template <typename T>
hipError_t launch_delta_step(const DeltaStepArgs& a, hipStream_t s) {
  if (a.dk <= 64) return launch<T, 16, 4>(a, s);
  if (a.dk <= 128) return launch<T, 32, 4>(a, s);
  return launch<T, 64, 4>(a, s);
}

template hipError_t launch_delta_step<bf16>(const DeltaStepArgs&, hipStream_t);
template hipError_t launch_delta_step<float>(const DeltaStepArgs&, hipStream_t);

}  // namespace ttt
