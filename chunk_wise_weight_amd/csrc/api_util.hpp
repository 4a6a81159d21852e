// What the C entry points of the token-wise operators share: checks of pointers, types and strides.
#pragma once
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include <hip/hip_runtime.h>

#include "launch.hpp"
#include "ttt.h"

namespace {

inline bool aligned(const void* p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
inline bool ok_ptr(const void* p, size_t a = 16) { return p != nullptr && aligned(p, a); }
inline int dev(hipError_t e) { return e == hipSuccess ? TTT_OK : TTT_ERR_DEVICE; }
inline bool ok_dtype(int t) { return t == TTT_F32 || t == TTT_BF16; }
inline int64_t esize(int t) { return t == TTT_BF16 ? 2 : 4; }

// A grid has fewer than 2^32 threads.
constexpr int64_t kMaxThreads = ((int64_t)1 << 32) - 1, kMaxBlocks = kMaxThreads / 256;
constexpr int64_t kMaxTokenStride = (int64_t)1 << 22;
constexpr int64_t kMaxNamedRows = 65536;     // of a step with slots: each workgroup looks through all of them

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

int check_norm(int64_t rows, int64_t dim, int dtype) {
  if (!ok_dtype(dtype)) return TTT_ERR_DTYPE;
  if (rows < 0 || dim <= 0) return TTT_ERR_SHAPE;
  if (dim > 65536 || rows > ((int64_t)1 << 40)) return TTT_ERR_UNSUPPORTED;
  return TTT_OK;
}

// Rows of whole 16-byte vectors are read as aligned ones; others need their elements' alignment only.
size_t norm_align(int64_t dim, int dtype) { return dim * esize(dtype) % 16 ? (size_t)esize(dtype) : 16; }

}  // namespace
