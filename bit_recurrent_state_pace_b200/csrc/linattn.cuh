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

// How every sequence is cut into stretches that run side by side where sequences and heads alone would leave SMs idle:
// stretch s is its chunks (of kLinChunk tokens) [s per, (s + 1) per), the last one what is left.  A first pass over all
// but the last gives each one's own contribution to the state, the chain kernel turns those into the states before each
// stretch, and the stretches then run from these.
constexpr int kLinChunk = 64;
struct LinSplit {
  int32_t stretches;        // at most, for one sequence
  int32_t per;              // chunks a stretch
};
// Stretches of a sequence of `len` tokens (one for an empty one).
__device__ __forceinline__ int stretches_of(const LinSplit& sp, int len) {
  const int nc = (int)(((int64_t)len + kLinChunk - 1) / kLinChunk), ns = (nc + sp.per - 1) / sp.per;
  return ns < 1 ? 1 : (ns > sp.stretches ? sp.stretches : ns);
}
// The stretches' states: ws[walk][n][h][stretch][D][D], fp32, in the walk's own order of rows.
__device__ __forceinline__ int64_t stretch_index(const LinArgs& a, const LinSplit& sp, int w, int n, int h, int seg) {
  return (((int64_t)w * a.N + n) * a.H + h) * sp.stretches + seg;
}
// `items` run side by side uncut and `fill` of them fill the SMs.  Stretches of `least` chunks at least; fewer than `few`
// of them are not worth the first pass.
inline LinSplit lin_split(int64_t items, int64_t max_len, int64_t fill, int least, int few) {
  const int64_t chunks = (max_len + kLinChunk - 1) / kLinChunk;
  LinSplit sp;
  sp.stretches = 1;
  sp.per = (int32_t)(chunks < 1 ? 1 : chunks);
  int64_t n = fill / items;
  if (n > chunks / least) n = chunks / least;
  if (n < few) return sp;
  sp.per = (int32_t)((chunks + n - 1) / n);
  sp.stretches = (int32_t)((chunks + sp.per - 1) / sp.per);
  return sp;
}

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

// The walk token by token; ws: of sp.stretches > 1.
LinSplit linattn_stream_split(int64_t heads, int64_t max_len, int walks, int D);
cudaError_t launch_linattn_stream(const LinArgs& a, const LinSplit& sp, float* ws, cudaStream_t st);
cudaError_t launch_linattn_chain(const LinArgs& a, const LinSplit& sp, float* ws, cudaStream_t st);
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

size_t qk_norm_partial_bytes(int D);
cudaError_t launch_qk_norm(const NormArgs& a, cudaStream_t st);
cudaError_t launch_qk_norm_backward(const NormArgs& a, cudaStream_t st);

}  // namespace pace
