// C ABI of the selective scan, the short convolution and the root-mean-square norm: argument validation (complete before
// any device work), workspace sizes and dispatch.
#include "api_util.hpp"

namespace {

using ttt::bf16;

constexpr int64_t kMaxState = 256, kMaxHeadDim = 4096, kMaxTaps = 8, kMaxChannels = (int64_t)1 << 20;

int check_scan_heads(int64_t H, int64_t G, int64_t P, int64_t N) {
  if (H <= 0 || G <= 0 || P <= 0 || N <= 0 || H % G) return TTT_ERR_SHAPE;
  if (P % 8 || N % 8 || N > kMaxState || P > kMaxHeadDim || H > 65536) return TTT_ERR_UNSUPPORTED;
  return TTT_OK;
}

int check_conv(int64_t batch, int64_t n, int64_t d, int64_t K, int dtype) {
  if (!ok_dtype(dtype)) return TTT_ERR_DTYPE;
  if (batch < 0 || n < 0 || d <= 0 || K <= 0) return TTT_ERR_SHAPE;
  const int64_t lim = (int64_t)1 << 30;
  if (K > kMaxTaps || d > kMaxChannels || n > lim || batch > lim || batch * n > lim) return TTT_ERR_UNSUPPORTED;
  return TTT_OK;
}

int check_conv(const ttt_conv_shape* s, int dtype, int64_t num_seqs) {
  if (s == nullptr) return TTT_ERR_ARG;
  if (int st = check_conv(s->batch, s->seq_len, s->dim, s->taps, dtype)) return st;
  if (num_seqs >= 0 && s->batch != 1) return TTT_ERR_SHAPE;
  if (num_seqs > (int64_t)1 << 30) return TTT_ERR_UNSUPPORTED;
  return TTT_OK;
}

ttt::ConvArgs conv_sizes(const ttt_conv_shape* s, int64_t num_seqs) {
  ttt::ConvArgs a{};
  a.batch = (int)s->batch;
  a.d = (int)s->dim;
  a.K = (int)s->taps;
  // packed rows are told from others by their starts: any address serves where only sizes are asked for
  static const int32_t some = 0;
  a.seqs = {num_seqs >= 0 ? &some : nullptr, (int)std::max<int64_t>(num_seqs, 0), (int)s->seq_len};
  return a;
}

int64_t conv_launch_blocks(const ttt::ConvArgs& a, int dtype, bool grad) {
  return dtype == TTT_BF16 ? ttt::conv_blocks<bf16>(a, grad) : ttt::conv_blocks<float>(a, grad);
}

// A [B, n, d] tensor's strides, given or contiguous; rows of any alignment of their elements.
bool take_rows(const ttt_row_strides* in, int64_t B, int64_t n, int64_t d, bool out, ttt::DeltaStrides* o) {
  if (in == nullptr) {
    *o = {n * d, 0, d};
    return true;
  }
  const int64_t most = (int64_t)1 << 40;
  if (in->batch < 0 || in->token < 0 || in->batch > most || in->token > most) return false;
  *o = {in->batch, 0, in->token};
  if (!out || B == 0 || n == 0) return true;
  const int64_t b = in->batch, t = in->token;
  if (n > 1 && t < d) return false;
  if (B > 1 && (b < d || (n > 1 && (b >= t ? b < t * n : t < b * B)))) return false;
  return true;
}

// Whether a tensor's rows are whole 16-byte vectors at 16-byte addresses.
bool whole_rows(const void* p, const ttt::DeltaStrides& s, int64_t es) {
  return aligned(p, 16) && s.b * es % 16 == 0 && s.t * es % 16 == 0;
}

// What the forward and the backward call take alike, checked and put into *a.
int take_conv(const ttt_conv_shape* s, int dtype, const void* x, const void* w, const ttt_conv_options* opt,
              ttt::ConvArgs* a) {
  static const ttt_conv_options none{};
  if (opt == nullptr) opt = &none;
  const int64_t num = opt->seq_starts ? opt->num_seqs : -1;
  if (opt->seq_starts && (num < 0 || !aligned(opt->seq_starts, 4))) return TTT_ERR_ARG;
  if (int st = check_conv(s, dtype, num)) return st;
  *a = conv_sizes(s, num);
  a->seqs.starts = opt->seq_starts;
  const size_t es = esize(dtype);
  if (!take_rows(opt->layout ? &opt->layout->x : nullptr, s->batch, s->seq_len, s->dim, false, &a->sx)) return TTT_ERR_ARG;
  if (s->batch * s->seq_len > 0 && !ok_ptr(x, es)) return TTT_ERR_ARG;
  if (!ok_ptr(w, es) || !aligned(opt->bias, es) || !aligned(opt->x_init, es)) return TTT_ERR_ARG;
  a->x = x;
  a->w = w;
  a->bias = opt->bias;
  a->silu = opt->silu != 0;
  a->x_init = s->taps > 1 ? opt->x_init : nullptr;
  a->rag = s->dim * es % 16 || !whole_rows(x, a->sx, es) || !aligned(w, 16) || !aligned(opt->bias, 16) ||
           !aligned(opt->x_init, 16);
  return TTT_OK;
}

int64_t scan_sequences(const ttt_scan_shape* s, int64_t num_seqs) { return num_seqs >= 0 ? num_seqs : s->batch; }

ttt::ScanArgs scan_sizes(const ttt_scan_shape* s, int64_t num_seqs) {
  ttt::ScanArgs a{};
  a.batch = (int)s->batch;
  a.H = (int)s->heads;
  a.G = (int)s->groups;
  a.P = (int)s->head_dim;
  a.N = (int)s->state;
  static const int32_t some = 0;
  a.seqs = {num_seqs >= 0 ? &some : nullptr, (int)std::max<int64_t>(num_seqs, 0), (int)s->seq_len};
  return a;
}

// At least the workgroups, of up to 512, of a walk's or a gradient's launch: no segment is shorter than a chunk, none
// takes fewer heads or more than 64 rows of P less than one (the 8 are scan_place's rounding).
int64_t scan_walks(const ttt_scan_shape* s, int64_t num_seqs) {
  const int64_t chunks = num_seqs >= 0 ? s->seq_len / 64 + num_seqs : s->batch * ((s->seq_len + 63) / 64);
  return (chunks + 8) * s->heads * ((s->head_dim + 63) / 64);
}
// The join's workgroups: the states' elements by 1024.
int64_t scan_states(const ttt_scan_shape* s, int64_t num_seqs) {
  return scan_sequences(s, num_seqs) * s->heads * ((s->head_dim * s->state + 1023) / 1024);
}

int check_scan(const ttt_scan_shape* s, int dtype, int64_t num_seqs) {
  if (s == nullptr) return TTT_ERR_ARG;
  if (!ok_dtype(dtype)) return TTT_ERR_DTYPE;
  if (s->batch < 0 || s->seq_len < 0) return TTT_ERR_SHAPE;
  if (int st = check_scan_heads(s->heads, s->groups, s->head_dim, s->state)) return st;
  if (num_seqs >= 0 && s->batch != 1) return TTT_ERR_SHAPE;
  const int64_t lim = (int64_t)1 << 30, seqs = scan_sequences(s, num_seqs);
  if (s->seq_len > lim || seqs > lim || (num_seqs < 0 && s->batch * s->seq_len > lim)) return TTT_ERR_UNSUPPORTED;
  if (scan_walks(s, num_seqs) > kMaxBlocks / 2 || scan_states(s, num_seqs) > kMaxBlocks) return TTT_ERR_UNSUPPORTED;
  return TTT_OK;
}

// What the backward pass takes less of: walks and joins in both directions at once.
int check_scan_backward(const ttt_scan_shape* s, int64_t num_seqs) {
  if (scan_walks(s, num_seqs) > kMaxBlocks / 4 || scan_states(s, num_seqs) > kMaxBlocks / 2) return TTT_ERR_UNSUPPORTED;
  return TTT_OK;
}

size_t scan_bytes(const ttt_scan_shape* s, int dtype, int64_t num_seqs) {
  const ttt::ScanArgs a = scan_sizes(s, num_seqs);
  return dtype == TTT_BF16 ? ttt::scan_workspace_bytes<bf16>(a) : ttt::scan_workspace_bytes<float>(a);
}

// What the forward and the backward call take alike, checked and put into *a.
int take_scan(const ttt_scan_shape* s, int dtype, const void* x, const float* dt, const float* A, const void* B,
              const void* C, const ttt_scan_options* opt, ttt::ScanArgs* a) {
  static const ttt_scan_options none{};
  if (opt == nullptr) opt = &none;
  const int64_t num = opt->seq_starts ? opt->num_seqs : -1;
  if (opt->seq_starts && (num < 0 || !aligned(opt->seq_starts, 4))) return TTT_ERR_ARG;
  if (int st = check_scan(s, dtype, num)) return st;
  *a = scan_sizes(s, num);
  a->seqs.starts = opt->seq_starts;
  const ttt_scan_layout* l = opt->layout;
  const int64_t n = s->seq_len, u = 16 / esize(dtype);
  if (!take_strides(l ? &l->x : nullptr, s->heads, n, s->head_dim, u, &a->sx) ||
      !take_strides(l ? &l->dt : nullptr, s->heads, n, 1, 1, &a->sdt) ||
      !take_strides(l ? &l->B : nullptr, s->groups, n, s->state, u, &a->sB) ||
      !take_strides(l ? &l->C : nullptr, s->groups, n, s->state, u, &a->sC))
    return TTT_ERR_ARG;
  if (!ok_ptr(A, 4) || !aligned(opt->D, 4) || !aligned(opt->dt_bias, 4) || !aligned(opt->S_init, 16)) return TTT_ERR_ARG;
  if (s->batch * n > 0 && (!ok_ptr(x) || !ok_ptr(dt, 4) || !ok_ptr(B) || !ok_ptr(C))) return TTT_ERR_ARG;
  a->x = x;
  a->dt = dt;
  a->A = A;
  a->B = B;
  a->C = C;
  a->D = opt->D;
  a->dt_bias = opt->dt_bias;
  a->softplus = opt->softplus != 0;
  a->S_init = opt->S_init;
  return TTT_OK;
}

int64_t conv_sequences(const ttt::ConvArgs& a) { return a.seqs.starts ? a.seqs.num : a.batch; }

}  // namespace

extern "C" {

int ttt_short_conv(const ttt_conv_shape* shape, int dtype, const void* x, const void* conv_w,
                   const ttt_conv_options* options, void* y, void* x_final, void* stream) {
  ttt::ConvArgs a;
  if (int st = take_conv(shape, dtype, x, conv_w, options, &a)) return st;
  const size_t es = esize(dtype);
  if (!take_rows(options && options->layout ? &options->layout->y : nullptr, shape->batch, shape->seq_len, shape->dim,
                 true, &a.sy))
    return TTT_ERR_ARG;
  if (shape->batch * shape->seq_len > 0 && !ok_ptr(y, es)) return TTT_ERR_ARG;
  if (conv_sequences(a) > 0 && shape->taps > 1 && !ok_ptr(x_final, es)) return TTT_ERR_ARG;
  if (conv_launch_blocks(a, dtype, false) > kMaxBlocks) return TTT_ERR_UNSUPPORTED;
  a.Y = y;
  a.x_final = x_final;
  a.rag = a.rag || !whole_rows(y, a.sy, es) || !aligned(x_final, 16);
  hipStream_t s = (hipStream_t)stream;
  return dev(dtype == TTT_BF16 ? ttt::launch_conv<bf16>(a, s) : ttt::launch_conv<float>(a, s));
}

int ttt_short_conv_backward_workspace_bytes(const ttt_conv_shape* shape, int dtype, int64_t num_seqs, size_t* bytes) {
  if (bytes == nullptr) return TTT_ERR_ARG;
  if (int st = check_conv(shape, dtype, num_seqs)) return st;
  const ttt::ConvArgs a = conv_sizes(shape, num_seqs);
  if (conv_launch_blocks(a, dtype, true) > kMaxBlocks) return TTT_ERR_UNSUPPORTED;
  const int64_t parts = dtype == TTT_BF16 ? ttt::conv_grad_parts<bf16>(a) : ttt::conv_grad_parts<float>(a);
  *bytes = (size_t)parts * (shape->taps + 1) * shape->dim * sizeof(float);
  return TTT_OK;
}

int ttt_short_conv_backward(const ttt_conv_shape* shape, int dtype, const void* x, const void* conv_w, const void* dy,
                            const void* dx_final, const ttt_conv_options* options,
                            const ttt_conv_grad_layout* grad_layout, void* dx, float* dconv_w, float* dbias,
                            void* dx_init, void* workspace, size_t workspace_bytes, void* stream) {
  ttt::ConvGradArgs a{};
  if (int st = take_conv(shape, dtype, x, conv_w, options, &a.f)) return st;
  const size_t es = esize(dtype);
  const int64_t B = shape->batch, n = shape->seq_len, d = shape->dim;
  if (!take_rows(grad_layout ? &grad_layout->dy : nullptr, B, n, d, false, &a.sdy) ||
      !take_rows(grad_layout ? &grad_layout->dx : nullptr, B, n, d, true, &a.sdx))
    return TTT_ERR_ARG;
  if (B * n > 0 && (!ok_ptr(dy, es) || !ok_ptr(dx, es))) return TTT_ERR_ARG;
  if (!ok_ptr(dconv_w, 4) || !aligned(dbias, 4) || !aligned(dx_final, es) || !aligned(dx_init, es)) return TTT_ERR_ARG;
  size_t need = 0;
  if (int st = ttt_short_conv_backward_workspace_bytes(shape, dtype, a.f.seqs.starts ? a.f.seqs.num : -1, &need)) return st;
  if (need > 0 && (!ok_ptr(workspace) || workspace_bytes < need)) return TTT_ERR_WORKSPACE;
  a.dY = dy;
  a.dx_final = shape->taps > 1 ? dx_final : nullptr;
  a.dx = dx;
  a.dx_init = dx_init;
  a.dw = dconv_w;
  a.dbias = dbias;
  a.part = (float*)workspace;
  a.f.rag = a.f.rag || !whole_rows(dy, a.sdy, es) || !whole_rows(dx, a.sdx, es) || !aligned(dx_final, 16) ||
            !aligned(dx_init, 16);
  hipStream_t s = (hipStream_t)stream;
  return dev(dtype == TTT_BF16 ? ttt::launch_conv_grad<bf16>(a, s) : ttt::launch_conv_grad<float>(a, s));
}

int ttt_short_conv_step(int64_t rows, int64_t states, int64_t dim, int64_t taps, int dtype, int silu, const void* x,
                        const void* conv_w, const void* bias, void* halo, const int32_t* slots, void* y, void* stream) {
  if (int st = check_conv(rows, 1, dim, taps, dtype)) return st;
  if (states < 0) return TTT_ERR_SHAPE;
  if (states > INT32_MAX || rows * ((dim + 1023) / 1024) > kMaxBlocks) return TTT_ERR_UNSUPPORTED;
  if (slots != nullptr && rows > kMaxNamedRows) return TTT_ERR_UNSUPPORTED;
  if (slots == nullptr && rows > states) return TTT_ERR_SHAPE;
  if (rows == 0) return TTT_OK;
  const size_t es = esize(dtype);
  if (!ok_ptr(x, es) || !ok_ptr(conv_w, es) || !aligned(bias, es) || !ok_ptr(y, es) || !aligned(slots, 4) ||
      !aligned(halo, es) || (states > 0 && taps > 1 && halo == nullptr))
    return TTT_ERR_ARG;
  const bool rag = dim * es % 16 || !aligned(x, 16) || !aligned(conv_w, 16) || !aligned(bias, 16) || !aligned(halo, 16) ||
                   !aligned(y, 16);
  ttt::ConvStepArgs a{(int)rows, (int)dim, (int)taps, silu != 0, rag, states, x, conv_w, bias, halo, slots, y};
  hipStream_t s = (hipStream_t)stream;
  return dev(dtype == TTT_BF16 ? ttt::launch_conv_step<bf16>(a, s) : ttt::launch_conv_step<float>(a, s));
}

int ttt_selective_scan_workspace_bytes(const ttt_scan_shape* shape, int dtype, int64_t num_seqs, size_t* bytes) {
  if (bytes == nullptr) return TTT_ERR_ARG;
  if (int st = check_scan(shape, dtype, num_seqs)) return st;
  *bytes = scan_bytes(shape, dtype, num_seqs);
  return TTT_OK;
}

int ttt_selective_scan(const ttt_scan_shape* shape, int dtype, const void* x, const float* dt, const float* A,
                       const void* B, const void* C, const ttt_scan_options* options, void* O, float* S_final,
                       void* workspace, size_t workspace_bytes, void* stream) {
  ttt::ScanArgs a;
  if (int st = take_scan(shape, dtype, x, dt, A, B, C, options, &a)) return st;
  const int64_t num = a.seqs.starts ? a.seqs.num : -1;
  if (!take_out_strides(options && options->layout ? &options->layout->O : nullptr, shape->batch, shape->heads,
                        shape->seq_len, shape->head_dim, 16 / esize(dtype), &a.sO))
    return TTT_ERR_ARG;
  if (scan_sequences(shape, num) > 0 && !ok_ptr(S_final)) return TTT_ERR_ARG;
  if (shape->batch * shape->seq_len > 0 && !ok_ptr(O)) return TTT_ERR_ARG;
  const size_t need = scan_bytes(shape, dtype, num);
  if (need > 0 && (!ok_ptr(workspace) || workspace_bytes < need)) return TTT_ERR_WORKSPACE;
  a.O = O;
  a.S_final = S_final;
  a.ws = (char*)workspace;
  hipStream_t s = (hipStream_t)stream;
  return dev(dtype == TTT_BF16 ? ttt::launch_scan<bf16>(a, s) : ttt::launch_scan<float>(a, s));
}

int ttt_selective_scan_backward_workspace_bytes(const ttt_scan_shape* shape, int dtype, int64_t num_seqs, size_t* bytes) {
  if (bytes == nullptr) return TTT_ERR_ARG;
  if (int st = check_scan(shape, dtype, num_seqs)) return st;
  if (int st = check_scan_backward(shape, num_seqs)) return st;
  const ttt::ScanArgs a = scan_sizes(shape, num_seqs);
  *bytes = dtype == TTT_BF16 ? ttt::scan_grad_workspace_bytes<bf16>(a) : ttt::scan_grad_workspace_bytes<float>(a);
  return TTT_OK;
}

int ttt_selective_scan_backward(const ttt_scan_shape* shape, int dtype, const void* x, const float* dt, const float* A,
                                const void* B, const void* C, const void* dO, const float* dS_final,
                                const ttt_scan_options* options, const ttt_scan_grad_layout* grad_layout, void* dx,
                                float* ddt, float* dA, void* dB, void* dC, float* dD, float* ddt_bias, float* dS_init,
                                void* workspace, size_t workspace_bytes, void* stream) {
  ttt::ScanGradArgs a{};
  if (int st = take_scan(shape, dtype, x, dt, A, B, C, options, &a.f)) return st;
  const int64_t num = a.f.seqs.starts ? a.f.seqs.num : -1;
  const ttt_scan_grad_layout* l = grad_layout;
  const int64_t b = shape->batch, n = shape->seq_len, u = 16 / esize(dtype), H = shape->heads, G = shape->groups;
  if (!take_strides(l ? &l->dO : nullptr, H, n, shape->head_dim, u, &a.sdO) ||
      !take_out_strides(l ? &l->dx : nullptr, b, H, n, shape->head_dim, u, &a.sdx) ||
      !take_out_strides(l ? &l->ddt : nullptr, b, H, n, 1, 1, &a.sddt) ||
      !take_out_strides(l ? &l->dB : nullptr, b, G, n, shape->state, u, &a.sdB) ||
      !take_out_strides(l ? &l->dC : nullptr, b, G, n, shape->state, u, &a.sdC))
    return TTT_ERR_ARG;
  if (b * n > 0 && (!ok_ptr(dO) || !ok_ptr(dx) || !ok_ptr(ddt, 4) || !ok_ptr(dB) || !ok_ptr(dC))) return TTT_ERR_ARG;
  if (!ok_ptr(dA, 4) || !aligned(dD, 4) || !aligned(ddt_bias, 4) || !aligned(dS_final, 16) || !aligned(dS_init, 16))
    return TTT_ERR_ARG;
  size_t need = 0;
  if (int st = ttt_selective_scan_backward_workspace_bytes(shape, dtype, num, &need)) return st;
  if (need > 0 && (!ok_ptr(workspace) || workspace_bytes < need)) return TTT_ERR_WORKSPACE;
  a.f.ws = (char*)workspace;
  a.dO = dO;
  a.dS_final = dS_final;
  a.dx = dx;
  a.ddt = ddt;
  a.dA = dA;
  a.dB = dB;
  a.dC = dC;
  a.dD = dD;
  a.ddt_bias = ddt_bias;
  a.dS_init = dS_init;
  hipStream_t s = (hipStream_t)stream;
  return dev(dtype == TTT_BF16 ? ttt::launch_scan_grad<bf16>(a, s) : ttt::launch_scan_grad<float>(a, s));
}

int ttt_selective_scan_step(const ttt_scan_step_shape* shape, int dtype, const void* x, const float* dt, const float* A,
                            const void* B, const void* C, const float* D, const float* dt_bias, int softplus, float* S,
                            const int32_t* slots, void* O, void* stream) {
  if (shape == nullptr) return TTT_ERR_ARG;
  if (!ok_dtype(dtype)) return TTT_ERR_DTYPE;
  if (shape->rows < 0 || shape->states < 0) return TTT_ERR_SHAPE;
  if (int st = check_scan_heads(shape->heads, shape->groups, shape->head_dim, shape->state)) return st;
  if (shape->states > INT32_MAX || shape->rows > INT32_MAX ||
      shape->rows * shape->heads * ((shape->head_dim + 7) / 8) > kMaxBlocks)
    return TTT_ERR_UNSUPPORTED;
  if (slots != nullptr && shape->rows > kMaxNamedRows) return TTT_ERR_UNSUPPORTED;
  if (slots == nullptr && shape->rows > shape->states) return TTT_ERR_SHAPE;
  if (shape->rows == 0) return TTT_OK;
  if (!ok_ptr(x) || !ok_ptr(dt, 4) || !ok_ptr(A, 4) || !ok_ptr(B) || !ok_ptr(C) || !aligned(D, 4) ||
      !aligned(dt_bias, 4) || !ok_ptr(O) || !aligned(slots, 4) || !aligned(S, 16) || (shape->states > 0 && S == nullptr))
    return TTT_ERR_ARG;
  ttt::ScanStepArgs a{(int)shape->rows, (int)shape->heads, (int)shape->groups, (int)shape->head_dim, (int)shape->state,
                      softplus != 0,    shape->states,     x,                  B,                    C,
                      dt,               A,                 D,                  dt_bias,              S,
                      slots,            O};
  hipStream_t s = (hipStream_t)stream;
  return dev(dtype == TTT_BF16 ? ttt::launch_scan_step<bf16>(a, s) : ttt::launch_scan_step<float>(a, s));
}

int ttt_rms_norm(int64_t rows, int64_t dim, int dtype, float eps, const void* x, const void* residual, const void* weight,
                 void* h, void* y, float* rstd, float* scale, int64_t group, void* stream) {
  if (int st = check_norm(rows, dim, dtype)) return st;
  if (!isfinite(eps) || eps < 0.f) return TTT_ERR_ARG;
  if (group != 0 && group != 32 && group != 64 && group != 128) return TTT_ERR_ARG;
  if (rows == 0) return TTT_OK;
  if (group != 0 && scale == nullptr) return TTT_ERR_ARG;
  const size_t al = norm_align(dim, dtype);
  if (!ok_ptr(x, al) || !aligned(residual, al) || !aligned(weight, al) || !ok_ptr(rstd, 4) || !aligned(scale, 4) ||
      (residual && !ok_ptr(h, al)) || !ok_ptr(y, scale == nullptr ? al : al == 16 ? 16 : 1))
    return TTT_ERR_ARG;
  ttt::RmsArgs a{rows, (int)dim, (int)group, eps, x, residual, weight, h, y, rstd, scale};
  hipStream_t s = (hipStream_t)stream;
  return dev(dtype == TTT_BF16 ? ttt::launch_rms<bf16>(a, s) : ttt::launch_rms<float>(a, s));
}

int ttt_rms_norm_backward_workspace_bytes(int64_t rows, int64_t dim, int dtype, size_t* bytes) {
  if (bytes == nullptr) return TTT_ERR_ARG;
  if (int st = check_norm(rows, dim, dtype)) return st;
  const int G = dtype == TTT_BF16 ? ttt::rms_grad_blocks<bf16>(rows, (int)dim) : ttt::rms_grad_blocks<float>(rows, (int)dim);
  *bytes = (size_t)G * dim * sizeof(double);
  return TTT_OK;
}

int ttt_rms_norm_backward(int64_t rows, int64_t dim, int dtype, const void* h, const void* weight, const void* dy,
                          const float* rstd, const void* dh, void* dx, float* dweight, void* workspace,
                          size_t workspace_bytes, void* stream) {
  size_t need = 0;
  if (int st = ttt_rms_norm_backward_workspace_bytes(rows, dim, dtype, &need)) return st;
  const size_t al = norm_align(dim, dtype);
  if (rows > 0 && (!ok_ptr(h, al) || !ok_ptr(dy, al) || !ok_ptr(dx, al) || !ok_ptr(rstd, 4))) return TTT_ERR_ARG;
  if (!aligned(weight, al) || !aligned(dh, al) || !aligned(dweight, 4)) return TTT_ERR_ARG;
  if (need > 0 && (!ok_ptr(workspace) || workspace_bytes < need)) return TTT_ERR_WORKSPACE;
  ttt::RmsGradArgs a{rows, (int)dim, h, weight, dy, dh, rstd, dx, dweight, (double*)workspace};
  hipStream_t s = (hipStream_t)stream;
  return dev(dtype == TTT_BF16 ? ttt::launch_rms_grad<bf16>(a, s) : ttt::launch_rms_grad<float>(a, s));
}

}  // extern "C"
