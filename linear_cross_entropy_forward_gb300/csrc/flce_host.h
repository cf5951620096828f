// Host helpers shared by the library's entry points.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/flce.h"

namespace flce {

// FLCE_OK and the current device's SM count, or FLCE_ERR_DEVICE / FLCE_ERR_CUDA.
int require_device(int* sms);

// The error word of a workspace header, read behind the work on `st` (synchronises).
int read_status(const void* workspace, cudaStream_t st);

// Upstream gradients formed inside flce_forward_backward: after the per-token loss and
// entropy of rows [n0, n0 + rows) are on the stream, `mid` enqueues the work that fills
// g_loss and g_entropy for those rows; `end` follows the last rows' mid.
struct GradHook {
  void* ctx;
  int (*mid)(void* ctx, int64_t n0, int64_t rows, int64_t chunks, cudaStream_t st);
  int (*end)(void* ctx, int64_t chunks, cudaStream_t st);
  // called once the workspace header is clear
  void (*begin)(void* ctx, uint32_t* err);
};

// flce_forward_backward, with a hook or (NULL) given gradients.
int forward_backward(const flce_params* p, const void* hidden, const void* weight,
                     const int64_t* labels, const float* g_loss, const float* g_entropy,
                     float* loss, float* entropy, float* lse, float* ez, void* dhidden,
                     void* dweight, void* workspace, size_t ws_bytes, void* stream,
                     const GradHook* hook);

// Token chunks flce_forward_backward takes.
int64_t fused_chunks(const flce_params* p);

// Tensor map over a row-major [outer, inner] bf16 array (rows row_elems long) with boxes of
// box_inner x box_outer, 128-byte swizzle, zeros out of bounds.
bool tensor_map(CUtensorMap* map, const void* base, int64_t inner, int64_t outer,
                int64_t row_elems, int box_inner, int box_outer);

// A stream beside `st` (one per thread and device) that waits for the work on it so far; side_join
// makes `st` wait for the work on that stream.
int side_fork(cudaStream_t st, cudaStream_t* side);
int side_join(cudaStream_t st);

}  // namespace flce
