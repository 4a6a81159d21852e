// C ABI of the gated delta rule and of layer norm: argument validation
// (complete before any device work), workspace sizes and dispatch.
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include <hip/hip_runtime.h>

#include "launch.hpp"
#include "ttt.h"

namespace {

using ttt::bf16;

inline bool aligned(const void* p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
inline bool ok_ptr(const void* p, size_t a = 16) { return p != nullptr && aligned(p, a); }
inline int dev(hipError_t e) { return e == hipSuccess ? TTT_OK : TTT_ERR_DEVICE; }
inline bool ok_dtype(int t) { return t == TTT_F32 || t == TTT_BF16; }
inline int64_t esize(int t) { return t == TTT_BF16 ? 2 : 4; }

// A grid has fewer than 2^32 threads.  kMaxBlocks holds workgroups of 256 (chunk and step kernels) to that; a
// forward walk's, of up to 384, are at most half as many.
constexpr int64_t kMaxThreads = ((int64_t)1 << 32) - 1, kMaxBlocks = kMaxThreads / 256;
constexpr int64_t kMaxDim = 256, kMaxVDim = 4096, kMaxTokenStride = (int64_t)1 << 22;
constexpr int64_t kMaxNamedRows = 65536;     // of a step with slots: each workgroup looks through all of them

int check_heads(int64_t Hk, int64_t Hv, int64_t dk, int64_t dv) {
  if (Hk <= 0 || Hv <= 0 || dk <= 0 || dv <= 0 || Hv % Hk) return TTT_ERR_SHAPE;
  if (dk % 8 || dv % 8 || dk > kMaxDim || dv > kMaxVDim || Hv > 65536) return TTT_ERR_UNSUPPORTED;
  return TTT_OK;
}

// Chunk slots; num_seqs < 0: one sequence a batch row.
int64_t slots_of(const ttt_delta_shape* s, int64_t num_seqs) {
  if (num_seqs >= 0) return num_seqs > 0 ? s->seq_len / 64 + num_seqs : 0;
  return s->batch * ((s->seq_len + 63) / 64);
}

int check_delta(const ttt_delta_shape* s, int dtype, int64_t num_seqs) {
  if (s == nullptr) return TTT_ERR_ARG;
  if (!ok_dtype(dtype)) return TTT_ERR_DTYPE;
  if (s->batch < 0 || s->seq_len < 0) return TTT_ERR_SHAPE;
  if (int st = check_heads(s->k_heads, s->v_heads, s->k_dim, s->v_dim)) return st;
  const bool packed = num_seqs >= 0;
  if (packed && s->batch != 1) return TTT_ERR_SHAPE;
  const int64_t lim = (int64_t)1 << 30, seqs = packed ? num_seqs : s->batch;
  if (s->seq_len > lim || seqs > lim || (!packed && s->batch * s->seq_len > lim)) return TTT_ERR_UNSUPPORTED;
  const int64_t slots = slots_of(s, num_seqs);
  // a walk's grid: key heads in eights (and twice that in the backward pass)
  if (slots * s->v_heads > kMaxBlocks || 2 * (seqs + 8) * s->v_heads * ((s->v_dim + 15) / 16) > kMaxBlocks)
    return TTT_ERR_UNSUPPORTED;
  return TTT_OK;
}

int64_t sequences(const ttt_delta_shape* s, int64_t num_seqs) { return num_seqs >= 0 ? num_seqs : s->batch; }

// What the backward pass takes less of: its walks have 320 threads, half of the workgroups going back, and the
// chunk-local kernel 512 a chunk slot and key head.
int check_delta_backward(const ttt_delta_shape* s, int dtype, int64_t num_seqs) {
  const int64_t columns = s->k_dim <= 128 || dtype == TTT_BF16 ? 64 : 32;
  const int64_t per = s->v_heads / s->k_heads * ((s->v_dim + columns - 1) / columns);
  const int64_t walks = 2 * ((sequences(s, num_seqs) * s->k_heads + 7) / 8 * 8) * per;
  const int64_t chunks = slots_of(s, num_seqs) * s->k_heads;
  return walks * 320 > kMaxThreads || chunks * 512 > kMaxThreads ? TTT_ERR_UNSUPPORTED : TTT_OK;
}

// Strides of a [B, H, n, d] tensor: given ones, or contiguous.  unit: elements of 16 bytes (1 for gates).
bool take_strides(const ttt_delta_strides* in, int64_t H, int64_t n, int64_t d, int64_t unit, ttt::DeltaStrides* out) {
  if (in == nullptr) {
    *out = {H * n * d, n * d, d};
    return true;
  }
  if (in->batch < 0 || in->head < 0 || in->token < 0 || in->batch % unit || in->head % unit || in->token % unit ||
      in->token > kMaxTokenStride)
    return false;
  *out = {in->batch, in->head, in->token};
  return true;
}

// The same of a tensor that is written: no two of its elements may lie at one place.
bool take_out_strides(const ttt_delta_strides* in, int64_t B, int64_t H, int64_t n, int64_t d, int64_t unit,
                      ttt::DeltaStrides* out) {
  if (!take_strides(in, H, n, d, unit, out)) return false;
  if (in == nullptr || B == 0 || n == 0) return true;
  struct {
    int64_t stride, count;
  } at[3] = {{out->b, B}, {out->h, H}, {out->t, n}};
  std::sort(at, at + 3, [](const auto& x, const auto& y) { return x.stride < y.stride; });
  int64_t reach = d;                  // elements that lie within one stride of the next index
  for (const auto& x : at) {
    if (x.count == 1) continue;
    if (x.stride < reach || x.stride > INT64_MAX / x.count) return false;
    reach = x.stride * x.count;
  }
  return true;
}

ttt::DeltaArgs sizes(const ttt_delta_shape* s, int64_t num_seqs) {
  ttt::DeltaArgs a{};
  a.batch = (int)s->batch;
  a.Hk = (int)s->k_heads;
  a.Hv = (int)s->v_heads;
  a.dk = (int)s->k_dim;
  a.dv = (int)s->v_dim;
  // packed rows are told from others by their starts: any address serves where only sizes are asked for
  static const int32_t some = 0;
  a.seqs = {num_seqs >= 0 ? &some : nullptr, (int)std::max<int64_t>(num_seqs, 0), (int)s->seq_len};
  return a;
}

size_t forward_bytes(const ttt_delta_shape* s, int dtype, int64_t num_seqs) {
  const ttt::DeltaArgs a = sizes(s, num_seqs);
  return dtype == TTT_BF16 ? ttt::delta_workspace_bytes<bf16>(a) : ttt::delta_workspace_bytes<float>(a);
}

// What the forward and the backward call take alike, checked and put into *a.
int take_inputs(const ttt_delta_shape* s, int dtype, float scale, const void* q, const void* k, const void* v,
                const float* g, const float* beta, const ttt_delta_options* opt, ttt::DeltaArgs* a) {
  static const ttt_delta_options none{};
  if (opt == nullptr) opt = &none;
  const int64_t num = opt->seq_starts ? opt->num_seqs : -1;
  if (opt->seq_starts && (num < 0 || !aligned(opt->seq_starts, 4))) return TTT_ERR_ARG;
  if (int st = check_delta(s, dtype, num)) return st;
  if (!isfinite(scale)) return TTT_ERR_ARG;
  *a = sizes(s, num);
  a->seqs.starts = opt->seq_starts;
  const ttt_delta_layout* l = opt->layout;
  const int64_t n = s->seq_len, u = 16 / esize(dtype);
  if (!take_strides(l ? &l->q : nullptr, s->k_heads, n, s->k_dim, u, &a->sq) ||
      !take_strides(l ? &l->k : nullptr, s->k_heads, n, s->k_dim, u, &a->sk) ||
      !take_strides(l ? &l->v : nullptr, s->v_heads, n, s->v_dim, u, &a->sv) ||
      !take_strides(l ? &l->g : nullptr, s->v_heads, n, 1, 1, &a->sg) ||
      !take_strides(l ? &l->beta : nullptr, s->v_heads, n, 1, 1, &a->sbeta))
    return TTT_ERR_ARG;
  if (s->batch * n > 0 && (!ok_ptr(q) || !ok_ptr(k) || !ok_ptr(v) || !ok_ptr(g, 4) || !ok_ptr(beta, 4)))
    return TTT_ERR_ARG;
  if (!aligned(opt->W_init, 16)) return TTT_ERR_ARG;
  a->q = q;
  a->k = k;
  a->v = v;
  a->g = g;
  a->beta = beta;
  a->W_init = opt->W_init;
  a->scale = scale;
  return TTT_OK;
}

int check_norm(int64_t rows, int64_t dim, int dtype) {
  if (!ok_dtype(dtype)) return TTT_ERR_DTYPE;
  if (rows < 0 || dim <= 0) return TTT_ERR_SHAPE;
  if (dim > 65536 || rows > ((int64_t)1 << 40)) return TTT_ERR_UNSUPPORTED;
  return TTT_OK;
}

// Rows of whole 16-byte vectors are read as aligned ones; others need their elements' alignment only.
size_t norm_align(int64_t dim, int dtype) { return dim * esize(dtype) % 16 ? (size_t)esize(dtype) : 16; }

}  // namespace

extern "C" {

int ttt_gated_delta_workspace_bytes(const ttt_delta_shape* shape, int dtype, int64_t num_seqs, size_t* bytes) {
  if (bytes == nullptr) return TTT_ERR_ARG;
  if (int st = check_delta(shape, dtype, num_seqs)) return st;
  *bytes = forward_bytes(shape, dtype, num_seqs);
  return TTT_OK;
}

int ttt_gated_delta(const ttt_delta_shape* shape, int dtype, float scale, const void* q, const void* k, const void* v,
                    const float* g, const float* beta, const ttt_delta_options* options, void* O, float* W_final,
                    void* workspace, size_t workspace_bytes, void* stream) {
  ttt::DeltaArgs a;
  if (int st = take_inputs(shape, dtype, scale, q, k, v, g, beta, options, &a)) return st;
  const int64_t num = a.seqs.starts ? a.seqs.num : -1;
  if (!take_out_strides(options && options->layout ? &options->layout->O : nullptr, shape->batch, shape->v_heads,
                        shape->seq_len, shape->v_dim, 16 / esize(dtype), &a.so))
    return TTT_ERR_ARG;
  if (sequences(shape, num) > 0 && !ok_ptr(W_final)) return TTT_ERR_ARG;
  if (shape->batch * shape->seq_len > 0 && !ok_ptr(O)) return TTT_ERR_ARG;
  const size_t need = forward_bytes(shape, dtype, num);
  if (need > 0 && (!ok_ptr(workspace) || workspace_bytes < need)) return TTT_ERR_WORKSPACE;
  a.O = O;
  a.W_final = W_final;
  a.ws = (char*)workspace;
  hipStream_t s = (hipStream_t)stream;
  return dev(dtype == TTT_BF16 ? ttt::launch_delta<bf16>(a, s) : ttt::launch_delta<float>(a, s));
}

int ttt_gated_delta_backward_workspace_bytes(const ttt_delta_shape* shape, int dtype, int64_t num_seqs,
                                             size_t* bytes) {
  if (bytes == nullptr) return TTT_ERR_ARG;
  if (int st = check_delta(shape, dtype, num_seqs)) return st;
  if (int st = check_delta_backward(shape, dtype, num_seqs)) return st;
  const ttt::DeltaArgs a = sizes(shape, num_seqs);
  *bytes = dtype == TTT_BF16 ? ttt::delta_grad_workspace_bytes<bf16>(a) : ttt::delta_grad_workspace_bytes<float>(a);
  return TTT_OK;
}

int ttt_gated_delta_backward(const ttt_delta_shape* shape, int dtype, float scale, const void* q, const void* k,
                             const void* v, const float* g, const float* beta, const void* dO, const float* dW_final,
                             const ttt_delta_options* options, const ttt_delta_grad_layout* grad_layout, void* dq,
                             void* dk, void* dv, void* dg, void* dbeta, float* dW_init, void* workspace,
                             size_t workspace_bytes, void* stream) {
  ttt::DeltaGradArgs a{};
  if (int st = take_inputs(shape, dtype, scale, q, k, v, g, beta, options, &a.f)) return st;
  const int64_t num = a.f.seqs.starts ? a.f.seqs.num : -1;
  const ttt_delta_grad_layout* l = grad_layout;
  const int64_t B = shape->batch, n = shape->seq_len, u = 16 / esize(dtype), Hk = shape->k_heads, Hv = shape->v_heads;
  if (!take_strides(l ? &l->dO : nullptr, Hv, n, shape->v_dim, u, &a.sdo) ||
      !take_out_strides(l ? &l->dq : nullptr, B, Hk, n, shape->k_dim, u, &a.sdq) ||
      !take_out_strides(l ? &l->dk : nullptr, B, Hk, n, shape->k_dim, u, &a.sdk) ||
      !take_out_strides(l ? &l->dv : nullptr, B, Hv, n, shape->v_dim, u, &a.sdv) ||
      !take_out_strides(l ? &l->dg : nullptr, B, Hv, n, 1, 1, &a.sdg) ||
      !take_out_strides(l ? &l->dbeta : nullptr, B, Hv, n, 1, 1, &a.sdbeta))
    return TTT_ERR_ARG;
  a.gates_f32 = l && l->gates_f32;
  const size_t gate = a.gates_f32 ? 4 : esize(dtype);
  if (B * n > 0 && (!ok_ptr(dO) || !ok_ptr(dq) || !ok_ptr(dk) || !ok_ptr(dv) || !ok_ptr(dg, gate) ||
                    !ok_ptr(dbeta, gate)))
    return TTT_ERR_ARG;
  if (!aligned(dW_final, 16) || !aligned(dW_init, 16)) return TTT_ERR_ARG;
  size_t need = 0;
  if (int st = ttt_gated_delta_backward_workspace_bytes(shape, dtype, num, &need)) return st;
  if (need > 0 && (!ok_ptr(workspace) || workspace_bytes < need)) return TTT_ERR_WORKSPACE;
  a.f.ws = (char*)workspace;
  a.dO = dO;
  a.dW_final = dW_final;
  a.dq = dq;
  a.dk = dk;
  a.dv = dv;
  a.dg = dg;
  a.dbeta = dbeta;
  a.dW_init = dW_init;
  hipStream_t s = (hipStream_t)stream;
  return dev(dtype == TTT_BF16 ? ttt::launch_delta_grad<bf16>(a, s) : ttt::launch_delta_grad<float>(a, s));
}

int ttt_gated_delta_step(const ttt_delta_step_shape* shape, int dtype, float scale, const void* q, const void* k,
                         const void* v, const float* g, const float* beta, float* W, const int32_t* slots, void* O,
                         void* stream) {
  if (shape == nullptr) return TTT_ERR_ARG;
  if (!ok_dtype(dtype)) return TTT_ERR_DTYPE;
  if (shape->rows < 0 || shape->states < 0) return TTT_ERR_SHAPE;
  if (int st = check_heads(shape->k_heads, shape->v_heads, shape->k_dim, shape->v_dim)) return st;
  if (shape->states > INT32_MAX || shape->rows > INT32_MAX ||
      shape->rows * shape->v_heads * ((shape->v_dim + 15) / 16) > kMaxBlocks)
    return TTT_ERR_UNSUPPORTED;
  if (slots != nullptr && shape->rows > kMaxNamedRows) return TTT_ERR_UNSUPPORTED;
  if (slots == nullptr && shape->rows > shape->states) return TTT_ERR_SHAPE;
  if (!isfinite(scale)) return TTT_ERR_ARG;
  if (shape->rows == 0) return TTT_OK;
  if (!ok_ptr(q) || !ok_ptr(k) || !ok_ptr(v) || !ok_ptr(g, 4) || !ok_ptr(beta, 4) || !ok_ptr(O) || !aligned(slots, 4) ||
      (shape->states > 0 && !ok_ptr(W)))
    return TTT_ERR_ARG;
  ttt::DeltaStepArgs a{(int)shape->rows, (int)shape->k_heads, (int)shape->v_heads, (int)shape->k_dim,
                       (int)shape->v_dim, shape->states, q, k, v, g, beta, W, slots, O, scale};
  hipStream_t s = (hipStream_t)stream;
  return dev(dtype == TTT_BF16 ? ttt::launch_delta_step<bf16>(a, s) : ttt::launch_delta_step<float>(a, s));
}

int ttt_layer_norm(int64_t rows, int64_t dim, int dtype, float eps, const void* x, const void* weight,
                   const void* bias, void* y, float* mean, float* rstd, void* stream) {
  if (int st = check_norm(rows, dim, dtype)) return st;
  if (!isfinite(eps) || eps < 0.f) return TTT_ERR_ARG;
  if (rows == 0) return TTT_OK;
  const size_t al = norm_align(dim, dtype);
  if (!ok_ptr(x, al) || !ok_ptr(y, al) || !ok_ptr(mean, 4) || !ok_ptr(rstd, 4) || !aligned(weight, al) ||
      !aligned(bias, al))
    return TTT_ERR_ARG;
  hipStream_t s = (hipStream_t)stream;
  if (dtype == TTT_BF16)
    return dev(ttt::launch_norm<bf16>((const bf16*)x, (const bf16*)weight, (const bf16*)bias, (bf16*)y, mean, rstd,
                                      rows, (int)dim, eps, s));
  return dev(ttt::launch_norm<float>((const float*)x, (const float*)weight, (const float*)bias, (float*)y, mean, rstd,
                                     rows, (int)dim, eps, s));
}

int ttt_layer_norm_backward_workspace_bytes(int64_t rows, int64_t dim, int dtype, size_t* bytes) {
  if (bytes == nullptr) return TTT_ERR_ARG;
  if (int st = check_norm(rows, dim, dtype)) return st;
  const int G = dtype == TTT_BF16 ? ttt::norm_grad_blocks<bf16>(rows, (int)dim)
                                  : ttt::norm_grad_blocks<float>(rows, (int)dim);
  *bytes = (size_t)G * 2 * dim * sizeof(float);
  return TTT_OK;
}

int ttt_layer_norm_backward(int64_t rows, int64_t dim, int dtype, const void* x, const void* weight, const void* dy,
                            const float* mean, const float* rstd, void* dx, float* dweight, float* dbias,
                            void* workspace, size_t workspace_bytes, void* stream) {
  size_t need = 0;
  if (int st = ttt_layer_norm_backward_workspace_bytes(rows, dim, dtype, &need)) return st;
  const size_t al = norm_align(dim, dtype);
  if (rows > 0 && (!ok_ptr(x, al) || !ok_ptr(dy, al) || !ok_ptr(dx, al) || !ok_ptr(mean, 4) || !ok_ptr(rstd, 4)))
    return TTT_ERR_ARG;
  if (!aligned(weight, al) || !aligned(dweight, 4) || !aligned(dbias, 4)) return TTT_ERR_ARG;
  if (need > 0 && (!ok_ptr(workspace) || workspace_bytes < need)) return TTT_ERR_WORKSPACE;
  hipStream_t s = (hipStream_t)stream;
  if (dtype == TTT_BF16)
    return dev(ttt::launch_norm_grad<bf16>((const bf16*)x, (const bf16*)weight, (const bf16*)dy, mean, rstd, (bf16*)dx,
                                           dweight, dbias, (float*)workspace, rows, (int)dim, s));
  return dev(ttt::launch_norm_grad<float>((const float*)x, (const float*)weight, (const float*)dy, mean, rstd,
                                          (float*)dx, dweight, dbias, (float*)workspace, rows, (int)dim, s));
}

}  // extern "C"
