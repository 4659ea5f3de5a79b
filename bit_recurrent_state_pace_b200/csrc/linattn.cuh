// Linear attention with a fixed decay for each head: what its kernels share.
#pragma once

#include "pace_internal.cuh"

namespace pace {

// One walk of the recurrence over every sequence.  The forward operator and
// each of the three gradients are such walks with the tensors' parts changed:
//   forward  o :  query q,  key k, value v,  forwards, state S
//   gradient dq:  query do, key v, value k,  forwards, state S^T
//   gradient dv:  query k,  key q, value do, backwards, state X (the gradient of S)
//   gradient dk:  query v,  key do, value q, backwards, state X^T
// Forwards:  S <- a S + value key^T, out = S query.
// Backwards, from the last token on: D = S + value key^T, out = D query, S <- a D.
struct LinWalk {
  const void* query;
  const void* key;
  const void* value;
  void* out;
  int64_t query_stride, key_stride, value_stride, out_stride;   // elements from row to row
  const float* S_in;        // or NULL: zeros
  float* S_out;             // or NULL
  int32_t back;             // 1: from the last token to the first
  int32_t swap;             // 1: the states lie transposed in memory ([key][value])
};

constexpr int kLinMaxWalks = 3;

struct LinArgs {
  int32_t N, H, D, io, walks;
  int32_t total;            // rows of the packed tensors
  int32_t max_len;
  const int32_t* cu;        // or NULL: sequence n is rows [n max_len, (n + 1) max_len)
  const float* log_decay;
  uint32_t* flags;          // or NULL
  LinWalk walk[kLinMaxWalks];
};

// Rows [begin, end) of sequence n, inside [0, total] whatever cu holds.
__device__ __forceinline__ void seq_rows(const LinArgs& a, int n, int* begin, int* end) {
  if (a.cu) {
    const int b = a.cu[n], e = a.cu[n + 1];
    *begin = b < 0 ? 0 : (b > a.total ? a.total : b);
    *end = e > a.total ? a.total : e;
    if (*end < *begin) *end = *begin;
  } else {
    *begin = n * a.max_len;
    *end = *begin + a.max_len;
  }
}

// exp(g n) for n >= 0 tokens; g is held above -1000 so that g = -inf gives 1
// for n = 0 and 0 beyond (a NaN stays one).
__device__ __forceinline__ float clamp_log_decay(float g) { return g < -1000.f ? -1000.f : g; }
__device__ __forceinline__ float decay_pow(float g, int n) { return expf(g * (float)n); }

// Lets `kernel` have `bytes` of dynamic shared memory, on the first call for a device (`done` is the caller's own, one
// for each kernel; calls at the same time set the same thing).
template <class K>
inline cudaError_t allow_shared(K kernel, int bytes, bool (&done)[64]) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 0 && dev < 64 && done[dev]) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && dev >= 0 && dev < 64) done[dev] = true;
  return e;
}

cudaError_t launch_linattn_stream(const LinArgs& a, cudaStream_t st);
cudaError_t launch_linattn_step(float* S, const void* q, const void* k, const void* v, const float* log_decay, void* o,
                                int64_t qs, int64_t ks, int64_t vs, int64_t os, int N, int H, int D, int io,
                                cudaStream_t st);

// pace_qk_norm_rotate: one side (queries or keys)
struct NormSide {
  const void* x;
  const void* dy;           // backward: gradient of the output, rows packed
  void* y;                  // output, or dx
  const float* w;           // or NULL
  float* dw;                // or NULL
  int64_t x_stride, y_stride;
  int32_t heads;
  float scale;
};

struct NormArgs {
  int32_t tokens, D, rot, interleaved, io;
  float inv_n, eps;         // 1 / n of the mean
  const int32_t* pos;
  const float* inv_freq;
  NormSide side[2];         // queries, keys
  float* partial;           // [blocks][2][D], backward with weight gradients
};

size_t qk_norm_partial_bytes(int64_t tokens, int D);
cudaError_t launch_qk_norm(const NormArgs& a, cudaStream_t st);
cudaError_t launch_qk_norm_backward(const NormArgs& a, cudaStream_t st);

}  // namespace pace
