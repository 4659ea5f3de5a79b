// Host side of the linear-attention and query/key-norm entry points:
// argument checks, workspace layout, launches.  Nothing here throws.
#include <cmath>
#include <string.h>

#include "linattn_tc.cuh"

namespace {

inline cudaStream_t as_stream(void* s) { return reinterpret_cast<cudaStream_t>(s); }

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline pace_status from_cuda(cudaError_t e) {
  if (e == cudaSuccess) return PACE_OK;
  (void)cudaGetLastError();  // clear a non-sticky error so later calls start clean
  return PACE_ERR_CUDA;
}

// Row stride in elements: 0 stands for packed rows of `width` elements; others hold a whole row and leave every
// offset inside 63 bits.
inline bool stride_ok(int64_t given, int64_t width, int64_t* out) {
  *out = given == 0 ? width : given;
  return *out >= width && *out <= ((int64_t)1 << 30);
}

struct LinShape {
  int64_t qs, ks, vs, os;
  size_t esz;
};

pace_status check_lin(const pace_linattn_desc* d, LinShape* s, bool tokens) {
  if (!d) return PACE_ERR_INVALID_ARG;
  if (d->num_seqs < 1 || d->num_heads < 1 || d->num_heads > PACE_MAX_HEADS) return PACE_ERR_INVALID_ARG;
  if (d->d_k < 1 || d->d_v < 1) return PACE_ERR_INVALID_ARG;
  if (d->io_dtype != PACE_IO_BF16 && d->io_dtype != PACE_IO_F32) return PACE_ERR_INVALID_ARG;
  if (tokens && (d->total_tokens < 0 || d->max_len < 0)) return PACE_ERR_INVALID_ARG;
  const int64_t w = (int64_t)d->num_heads * d->d_k;
  if (d->d_k != d->d_v) return PACE_ERR_UNSUPPORTED;
  if (d->d_k != 32 && d->d_k != 64 && d->d_k != 128) return PACE_ERR_UNSUPPORTED;
  if (!stride_ok(d->q_stride, w, &s->qs) || !stride_ok(d->k_stride, w, &s->ks) || !stride_ok(d->v_stride, w, &s->vs) ||
      !stride_ok(d->o_stride, w, &s->os))
    return PACE_ERR_INVALID_ARG;
  if (tokens && (d->total_tokens > 0x7fffffffll || d->max_len > 0x7fffffffll)) return PACE_ERR_UNSUPPORTED;
  if ((int64_t)d->num_seqs * d->num_heads > (0x7fffffffll >> 4)) return PACE_ERR_UNSUPPORTED;   // grid sizes
  s->esz = (size_t)pace::io_size(d->io_dtype);
  return PACE_OK;
}

// io tensors and states; `need` says whether NULL is refused
inline bool io_ok(const void* p, size_t esz, bool need) { return p ? aligned(p, esz) : !need; }
inline bool state_ok(const float* p) { return aligned(p, 16); }

pace::LinArgs lin_args(const pace_linattn_desc* d, const float* log_decay, const int32_t* cu, uint32_t* flags) {
  pace::LinArgs a;
  memset(&a, 0, sizeof a);
  a.N = d->num_seqs;
  a.H = d->num_heads;
  a.D = d->d_k;
  a.io = d->io_dtype;
  a.total = (int32_t)d->total_tokens;
  a.max_len = (int32_t)d->max_len;
  a.cu = cu;
  a.log_decay = log_decay;
  a.flags = flags;
  return a;
}

// A tensor's bytes: `rows` of `width`, `stride` apart (width <= stride where there are several).
struct Bytes {
  const void* p;
  int64_t width, stride, rows;
};
inline Bytes io_bytes(const void* p, int64_t elements, int64_t stride, int64_t rows, size_t esz) {
  return Bytes{p, elements * (int64_t)esz, stride * (int64_t)esz, rows};
}
inline Bytes state_bytes(const float* p, const pace_linattn_desc* d) {
  const int64_t n = (int64_t)d->num_seqs * d->num_heads * d->d_k * d->d_v * 4;
  return Bytes{p, n, n, 1};
}
inline Bytes vector_bytes(const float* p, int n) { return Bytes{p, 4 * (int64_t)n, 4 * (int64_t)n, 1}; }

// Whether a byte of row i of a, at i stride, is one of row j of b: -width_b < (b - a) + t stride < width_a for a t = j - i.
bool rows_meet(const Bytes& a, const Bytes& b, int64_t stride) {
  const __int128 at = (__int128)(intptr_t)b.p - (intptr_t)a.p;
  auto floor_div = [&](__int128 x) { return x >= 0 ? x / stride : -((-x + stride - 1) / stride); };
  __int128 low = floor_div(-b.width - at) + 1, high = floor_div(a.width - 1 - at);
  if (low < 1 - (__int128)a.rows) low = 1 - (__int128)a.rows;
  if (high > b.rows - 1) high = b.rows - 1;
  return low <= high;
}
// Whether two tensors share memory: exact for rows at one stride (parts of one wider row do not, where their columns
// differ) or where one of them is a single row; of rows at two strides only the first ones are looked for in the other
// tensor.
bool overlap(const Bytes& a, const Bytes& b) {
  if (!a.p || !b.p || a.rows <= 0 || b.rows <= 0 || a.width <= 0 || b.width <= 0) return false;
  auto behind = [](const Bytes& x) { return (__int128)(intptr_t)x.p + (__int128)(x.rows - 1) * x.stride + x.width; };
  if (behind(a) <= (intptr_t)b.p || behind(b) <= (intptr_t)a.p) return false;
  if (a.rows == 1 || a.stride == b.stride) return rows_meet(a, b, b.stride);
  if (b.rows == 1) return rows_meet(a, b, a.stride);
  Bytes a0 = a, b0 = b;
  a0.rows = b0.rows = 1;
  return rows_meet(a0, b, b.stride) || rows_meet(a, b0, a.stride);
}
// Outputs do not overlap inputs or one another: rows of a head or sequence are read by several blocks, in any order.
bool apart(const Bytes* outs, int n_out, const Bytes* ins, int n_in) {
  for (int i = 0; i < n_out; ++i) {
    for (int j = 0; j < n_in; ++j)
      if (overlap(outs[i], ins[j])) return false;
    for (int j = 0; j < i; ++j)
      if (overlap(outs[i], outs[j])) return false;
  }
  return true;
}
// ... or are the very input, row for row
inline bool same_rows(const Bytes& a, const Bytes& b) { return a.p == b.p && (a.stride == b.stride || a.rows <= 1); }

// Walks over all sequences, on the tensor cores where their shapes allow.  The workspace depends on the desc alone: where
// alignment keeps a shape that the tensor cores would take off them, the sequences are not cut.
inline bool tc_shape(const pace_linattn_desc* d) { return d->io_dtype == PACE_IO_BF16 && d->d_k >= 64; }
inline pace::LinSplit split_of(const pace_linattn_desc* d, int walks) {
  const int64_t heads = (int64_t)d->num_seqs * d->num_heads;
  return tc_shape(d) ? pace::linattn_tc_split(heads, d->max_len, walks)
                     : pace::linattn_stream_split(heads, d->max_len, walks, d->d_k);
}
inline size_t stretch_bytes(const pace_linattn_desc* d, int walks) {
  const pace::LinSplit sp = split_of(d, walks);
  if (sp.stretches <= 1) return 0;
  return (size_t)walks * d->num_seqs * d->num_heads * sp.stretches * d->d_k * d->d_k * sizeof(float);
}
pace_status run_walks(const pace_linattn_desc* d, const pace::LinArgs& a, void* ws, cudaStream_t st) {
  const pace::LinSplit sp = split_of(d, a.walks);
  float* states = reinterpret_cast<float*>(ws);
  const bool tc = pace::linattn_tc_takes(a);
  if (tc_shape(d) && !tc) {
    pace::LinSplit whole = sp;
    whole.stretches = 1;
    return from_cuda(pace::launch_linattn_stream(a, whole, nullptr, st));
  }
  if (sp.stretches > 1 && !ws) return PACE_ERR_INVALID_ARG;
  return from_cuda(tc ? pace::launch_linattn_tc(a, sp, states, st) : pace::launch_linattn_stream(a, sp, states, st));
}

struct NormShape { int64_t qs, ks, qo, ko; size_t esz; };

pace_status check_norm(const pace_qk_norm_desc* d, NormShape* s) {
  if (!d) return PACE_ERR_INVALID_ARG;
  if (d->num_tokens < 0 || d->num_q_heads < 0 || d->num_k_heads < 0 || d->num_q_heads > PACE_MAX_HEADS ||
      d->num_k_heads > PACE_MAX_HEADS || d->num_q_heads + d->num_k_heads == 0)
    return PACE_ERR_INVALID_ARG;
  if (d->head_dim < 1 || d->rotary_dim < 0 || d->rotary_dim > d->head_dim || d->rotary_dim % 2) return PACE_ERR_INVALID_ARG;
  if (d->interleaved != 0 && d->interleaved != 1) return PACE_ERR_INVALID_ARG;
  if (d->norm != PACE_NORM_L2 && d->norm != PACE_NORM_RMS) return PACE_ERR_INVALID_ARG;
  if (d->io_dtype != PACE_IO_BF16 && d->io_dtype != PACE_IO_F32) return PACE_ERR_INVALID_ARG;
  if (!(d->eps > 0.f) || !std::isfinite(d->eps) || !std::isfinite(d->q_scale)) return PACE_ERR_INVALID_ARG;
  const int64_t wq = (int64_t)d->num_q_heads * d->head_dim, wk = (int64_t)d->num_k_heads * d->head_dim;
  if (!stride_ok(d->q_stride, wq, &s->qs) || !stride_ok(d->k_stride, wk, &s->ks) ||
      !stride_ok(d->q_out_stride, wq, &s->qo) || !stride_ok(d->k_out_stride, wk, &s->ko))
    return PACE_ERR_INVALID_ARG;
  if (d->head_dim % 8 || d->head_dim > 256 || d->num_tokens > 0x7fffffffll) return PACE_ERR_UNSUPPORTED;
  s->esz = (size_t)pace::io_size(d->io_dtype);
  return PACE_OK;
}

pace_status norm_args(const pace_qk_norm_desc* d, const NormShape& s, const void* q, const void* k, const float* wq,
                      const float* wk, const int32_t* pos, const float* inv, void* qo, void* ko, pace::NormArgs* a) {
  const bool any = d->num_tokens > 0;
  if (!io_ok(q, s.esz, any && d->num_q_heads) || !io_ok(qo, s.esz, any && d->num_q_heads) ||
      !io_ok(k, s.esz, any && d->num_k_heads) || !io_ok(ko, s.esz, any && d->num_k_heads))
    return PACE_ERR_INVALID_ARG;
  if (d->rotary_dim && (!inv || (any && !pos))) return PACE_ERR_INVALID_ARG;
  if (!aligned(wq, 4) || !aligned(wk, 4) || !aligned(pos, 4) || !aligned(inv, 4)) return PACE_ERR_INVALID_ARG;
  memset(a, 0, sizeof *a);
  a->tokens = (int32_t)d->num_tokens;
  a->D = d->head_dim;
  a->rot = d->rotary_dim;
  a->interleaved = d->interleaved;
  a->io = d->io_dtype;
  a->inv_n = d->norm == PACE_NORM_RMS ? 1.f / (float)d->head_dim : 1.f;
  a->eps = d->eps;
  a->pos = pos;
  a->inv_freq = inv;
  a->side[0] = pace::NormSide{q, nullptr, qo, wq, nullptr, s.qs, s.qo, d->num_q_heads, d->q_scale};
  a->side[1] = pace::NormSide{k, nullptr, ko, wk, nullptr, s.ks, s.ko, d->num_k_heads, 1.f};
  return PACE_OK;
}

}  // namespace

extern "C" {

pace_status pace_linattn_workspace_bytes(const pace_linattn_desc* desc, int32_t backward, size_t* bytes) {
  LinShape s;
  if (!bytes || (backward != 0 && backward != 1)) return PACE_ERR_INVALID_ARG;
  const pace_status st = check_lin(desc, &s, true);
  if (st != PACE_OK) return st;
  *bytes = stretch_bytes(desc, backward ? 3 : 1);
  return PACE_OK;
}

pace_status pace_linattn_forward(const pace_linattn_desc* desc, const void* q, const void* k, const void* v,
                                 const float* log_decay, const int32_t* cu_seqlens, const float* S0, void* o,
                                 float* ST, void* d_workspace, uint32_t* d_flags, void* stream) {
  LinShape s;
  const pace_status st = check_lin(desc, &s, true);
  if (st != PACE_OK) return st;
  if (!cu_seqlens && desc->total_tokens != (int64_t)desc->num_seqs * desc->max_len) return PACE_ERR_INVALID_ARG;
  const bool any = desc->total_tokens > 0;
  if (!io_ok(q, s.esz, any) || !io_ok(k, s.esz, any) || !io_ok(v, s.esz, any) || !io_ok(o, s.esz, any))
    return PACE_ERR_INVALID_ARG;
  if (!log_decay || !aligned(log_decay, 4) || !aligned(cu_seqlens, 4) || !state_ok(S0) || !state_ok(ST) ||
      !aligned(d_flags, 4) || !aligned(d_workspace, 256))
    return PACE_ERR_INVALID_ARG;
  const int64_t w = (int64_t)desc->num_heads * desc->d_k, rows = desc->total_tokens;
  const Bytes outs[2] = {io_bytes(o, w, s.os, rows, s.esz), state_bytes(ST, desc)};
  const Bytes ins[4] = {io_bytes(q, w, s.qs, rows, s.esz), io_bytes(k, w, s.ks, rows, s.esz), io_bytes(v, w, s.vs, rows, s.esz),
                        state_bytes(ST == S0 ? nullptr : S0, desc)};
  if (!apart(outs, 2, ins, 4)) return PACE_ERR_INVALID_ARG;
  pace::LinArgs a = lin_args(desc, log_decay, cu_seqlens, d_flags);
  a.walks = 1;
  a.walk[0] = pace::LinWalk{q, k, v, o, s.qs, s.ks, s.vs, s.os, S0, ST, 0, 0};
  return run_walks(desc, a, d_workspace, as_stream(stream));
}

pace_status pace_linattn_backward(const pace_linattn_desc* desc, const void* q, const void* k, const void* v,
                                  const float* log_decay, const int32_t* cu_seqlens, const float* S0,
                                  const void* d_o, const float* dST, void* dq, void* dk, void* dv, float* dS0,
                                  void* d_workspace, uint32_t* d_flags, void* stream) {
  LinShape s;
  const pace_status st = check_lin(desc, &s, true);
  if (st != PACE_OK) return st;
  if (!cu_seqlens && desc->total_tokens != (int64_t)desc->num_seqs * desc->max_len) return PACE_ERR_INVALID_ARG;
  const bool any = desc->total_tokens > 0;
  if (!io_ok(q, s.esz, any) || !io_ok(k, s.esz, any) || !io_ok(v, s.esz, any) || !io_ok(d_o, s.esz, any) ||
      !io_ok(dq, s.esz, any) || !io_ok(dk, s.esz, any) || !io_ok(dv, s.esz, any))
    return PACE_ERR_INVALID_ARG;
  if (!log_decay || !aligned(log_decay, 4) || !aligned(cu_seqlens, 4) || !state_ok(S0) || !state_ok(dST) ||
      !state_ok(dS0) || !aligned(d_flags, 4) || !aligned(d_workspace, 256))
    return PACE_ERR_INVALID_ARG;
  const int64_t w = (int64_t)desc->num_heads * desc->d_k, rows = desc->total_tokens;
  const Bytes outs[4] = {io_bytes(dq, w, s.qs, rows, s.esz), io_bytes(dk, w, s.ks, rows, s.esz),
                         io_bytes(dv, w, s.vs, rows, s.esz), state_bytes(dS0, desc)};
  const Bytes ins[6] = {io_bytes(q, w, s.qs, rows, s.esz), io_bytes(k, w, s.ks, rows, s.esz), io_bytes(v, w, s.vs, rows, s.esz),
                        io_bytes(d_o, w, s.os, rows, s.esz), state_bytes(S0, desc), state_bytes(dST, desc)};
  if (!apart(outs, 4, ins, 6)) return PACE_ERR_INVALID_ARG;
  pace::LinArgs a = lin_args(desc, log_decay, cu_seqlens, d_flags);
  a.walks = 3;
  a.walk[0] = pace::LinWalk{k, q, d_o, dv, s.ks, s.qs, s.os, s.vs, dST, dS0, 1, 0};
  a.walk[1] = pace::LinWalk{v, d_o, q, dk, s.vs, s.os, s.qs, s.ks, dST, nullptr, 1, 1};
  a.walk[2] = pace::LinWalk{d_o, v, k, dq, s.os, s.vs, s.ks, s.qs, S0, nullptr, 0, 1};
  return run_walks(desc, a, d_workspace, as_stream(stream));
}

pace_status pace_debug_linattn_wait(uint32_t wait_tries, uint32_t extra_tx_bytes) {
  if (wait_tries == 0 && extra_tx_bytes == 0) {
    pace::linattn_tc_debug(0, 0);
    return PACE_OK;
  }
  if (wait_tries < 100 || wait_tries > pace::ltc::kWaitTries || (extra_tx_bytes != 0 && extra_tx_bytes != 16))
    return PACE_ERR_INVALID_ARG;
  if (extra_tx_bytes && wait_tries > 1000) return PACE_ERR_INVALID_ARG;
  pace::linattn_tc_debug(wait_tries, extra_tx_bytes);
  return PACE_OK;
}

pace_status pace_linattn_step(const pace_linattn_desc* desc, float* S, const void* q, const void* k, const void* v,
                              const float* log_decay, void* o, void* stream) {
  LinShape s;
  const pace_status st = check_lin(desc, &s, false);
  if (st != PACE_OK) return st;
  if (!S || !state_ok(S) || !log_decay || !aligned(log_decay, 4) || !io_ok(q, s.esz, true) || !io_ok(k, s.esz, true) ||
      !io_ok(v, s.esz, true) || !io_ok(o, s.esz, true))
    return PACE_ERR_INVALID_ARG;
  const int64_t w = (int64_t)desc->num_heads * desc->d_k, rows = desc->num_seqs;
  const Bytes outs[2] = {io_bytes(o, w, s.os, rows, s.esz), state_bytes(S, desc)};
  const Bytes ins[3] = {io_bytes(q, w, s.qs, rows, s.esz), io_bytes(k, w, s.ks, rows, s.esz), io_bytes(v, w, s.vs, rows, s.esz)};
  if (!apart(outs, 2, ins, 3)) return PACE_ERR_INVALID_ARG;
  return from_cuda(pace::launch_linattn_step(S, q, k, v, log_decay, o, s.qs, s.ks, s.vs, s.os, desc->num_seqs,
                                             desc->num_heads, desc->d_k, desc->io_dtype, as_stream(stream)));
}

pace_status pace_qk_norm_rotate(const pace_qk_norm_desc* desc, const void* q, const void* k, const float* q_weight,
                                const float* k_weight, const int32_t* positions, const float* inv_freq, void* q_out,
                                void* k_out, void* stream) {
  NormShape s;
  pace::NormArgs a;
  pace_status st = check_norm(desc, &s);
  if (st == PACE_OK) st = norm_args(desc, s, q, k, q_weight, k_weight, positions, inv_freq, q_out, k_out, &a);
  if (st != PACE_OK) return st;
  const int64_t wq = (int64_t)desc->num_q_heads * desc->head_dim, wk = (int64_t)desc->num_k_heads * desc->head_dim;
  const int64_t rows = desc->num_tokens;
  const Bytes outs[2] = {io_bytes(q_out, wq, s.qo, rows, s.esz), io_bytes(k_out, wk, s.ko, rows, s.esz)};
  const Bytes ins[2] = {io_bytes(q, wq, s.qs, rows, s.esz), io_bytes(k, wk, s.ks, rows, s.esz)};
  for (int i = 0; i < 2; ++i)
    if ((overlap(outs[i], ins[i]) && !same_rows(outs[i], ins[i])) || overlap(outs[i], ins[1 - i])) return PACE_ERR_INVALID_ARG;
  if (overlap(outs[0], outs[1])) return PACE_ERR_INVALID_ARG;
  return from_cuda(pace::launch_qk_norm(a, as_stream(stream)));
}

pace_status pace_qk_norm_workspace_bytes(const pace_qk_norm_desc* desc, size_t* bytes) {
  NormShape s;
  if (!bytes) return PACE_ERR_INVALID_ARG;
  const pace_status st = check_norm(desc, &s);
  if (st != PACE_OK) return st;
  *bytes = pace::qk_norm_partial_bytes(desc->head_dim);
  return PACE_OK;
}

pace_status pace_qk_norm_rotate_backward(const pace_qk_norm_desc* desc, const void* q, const void* k,
                                         const float* q_weight, const float* k_weight, const int32_t* positions,
                                         const float* inv_freq, const void* d_q_out, const void* d_k_out, void* dq,
                                         void* dk, float* dq_weight, float* dk_weight, void* d_workspace,
                                         void* stream) {
  NormShape s;
  pace::NormArgs a;
  pace_status st = check_norm(desc, &s);
  if (st == PACE_OK) st = norm_args(desc, s, q, k, q_weight, k_weight, positions, inv_freq, dq, dk, &a);
  if (st != PACE_OK) return st;
  const bool any = desc->num_tokens > 0;
  if (!io_ok(d_q_out, s.esz, any && desc->num_q_heads) || !io_ok(d_k_out, s.esz, any && desc->num_k_heads))
    return PACE_ERR_INVALID_ARG;
  const int64_t wq = (int64_t)desc->num_q_heads * desc->head_dim, wk = (int64_t)desc->num_k_heads * desc->head_dim;
  const int64_t rows = desc->num_tokens;
  const Bytes outs[2] = {io_bytes(dq, wq, s.qo, rows, s.esz), io_bytes(dk, wk, s.ko, rows, s.esz)};
  const Bytes ins[2] = {io_bytes(q, wq, s.qs, rows, s.esz), io_bytes(k, wk, s.ks, rows, s.esz)};
  const Bytes grads[2] = {io_bytes(d_q_out, wq, wq, rows, s.esz), io_bytes(d_k_out, wk, wk, rows, s.esz)};
  for (int i = 0; i < 2; ++i) {
    if (overlap(outs[i], ins[1 - i]) || overlap(outs[i], grads[1 - i])) return PACE_ERR_INVALID_ARG;
    if (overlap(outs[i], ins[i]) && !same_rows(outs[i], ins[i])) return PACE_ERR_INVALID_ARG;
    if (overlap(outs[i], grads[i]) && !same_rows(outs[i], grads[i])) return PACE_ERR_INVALID_ARG;
  }
  if (overlap(outs[0], outs[1])) return PACE_ERR_INVALID_ARG;
  if (overlap(vector_bytes(dq_weight, desc->head_dim), vector_bytes(dk_weight, desc->head_dim))) return PACE_ERR_INVALID_ARG;
  if (!aligned(dq_weight, 4) || !aligned(dk_weight, 4)) return PACE_ERR_INVALID_ARG;
  if ((dq_weight || dk_weight) && (!d_workspace || !aligned(d_workspace, 256))) return PACE_ERR_INVALID_ARG;
  a.side[0].dy = d_q_out;
  a.side[1].dy = d_k_out;
  a.side[0].dw = dq_weight;
  a.side[1].dw = dk_weight;
  a.partial = reinterpret_cast<float*>(d_workspace);
  return from_cuda(pace::launch_qk_norm_backward(a, as_stream(stream)));
}

}  // extern "C"
