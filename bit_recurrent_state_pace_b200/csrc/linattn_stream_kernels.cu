// Linear attention with a fixed decay for each head, token by token: the
// walk that is right for every type, size and alignment (linattn.cuh), and
// the recurrent step of single tokens.
//
//   forwards:  S <- a S + v k^T, o = S q;   backwards: D = S + v k^T, o = D q, S <- a D.
#include "linattn.cuh"

namespace pace {

namespace {

constexpr unsigned FULL = 0xffffffffu;

// ---- the walk ------------------------------------------------------------------
// A block walks one sequence and head for 32 rows of S.  Four threads share a
// row; a thread holds the columns 4 (c + 4 e) .. + 3 of it in registers, so that
// the four threads' reads of a key or query are 64 contiguous bytes.  The state
// never leaves the registers; tokens come through shared memory, TT at a time,
// the next ones being loaded while these are used.
constexpr int kWalkThreads = 128, kRows = 32, TT = 16;

template <int D, bool BF16>
__global__ void __launch_bounds__(kWalkThreads) linattn_walk_kernel(const __grid_constant__ LinArgs a) {
  constexpr int V4 = D / 16;                         // float4 groups of a thread
  constexpr int QKN = TT * D / kWalkThreads, VN = TT * kRows / kWalkThreads;
  __shared__ __align__(16) float qs[TT][D], ks[TT][D];
  __shared__ float vs[TT][kRows], os[TT][kRows];
  const int tid = threadIdx.x, row = tid >> 2, c = tid & 3;
  constexpr int SL = D / kRows;                      // row slices of a state
  const int slice = blockIdx.x % SL;
  const int rest = blockIdx.x / SL;
  const int h = rest % a.H, n = rest / a.H;
  const LinWalk& w = a.walk[blockIdx.y];
  int begin, end;
  seq_rows(a, n, &begin, &end);
  const int len = end - begin;
  const float al = expf(clamp_log_decay(a.log_decay[h]));
  const size_t st0 = ((size_t)n * a.H + h) * D * D;
  const int i = slice * kRows + row;                 // this thread's row of S
  float2 S[V4 * 2];
#pragma unroll
  for (int e = 0; e < V4; ++e) {
    float x[4] = {0.f, 0.f, 0.f, 0.f};
    if (w.S_in) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int col = 4 * (c + 4 * e) + j;
        x[j] = w.S_in[st0 + (w.swap ? (size_t)col * D + i : (size_t)i * D + col)];
      }
    }
    S[2 * e] = make_float2(x[0], x[1]);
    S[2 * e + 1] = make_float2(x[2], x[3]);
  }
  const size_t hd = (size_t)h * D;
  float nq[QKN], nk[QKN], nv[VN];
  auto fetch = [&](int t0) {                         // tokens t0 .. t0 + TT - 1 in walking order
#pragma unroll
    for (int e = 0; e < QKN; ++e) {
      const int x = tid + e * kWalkThreads, t = t0 + x / D, j = x % D;
      const bool in = t < len;
      const size_t r = (size_t)(w.back ? end - 1 - t : begin + t);
      nq[e] = in ? load_io(w.query, r * w.query_stride + hd + j, BF16 ? PACE_IO_BF16 : PACE_IO_F32) : 0.f;
      nk[e] = in ? load_io(w.key, r * w.key_stride + hd + j, BF16 ? PACE_IO_BF16 : PACE_IO_F32) : 0.f;
    }
#pragma unroll
    for (int e = 0; e < VN; ++e) {
      const int x = tid + e * kWalkThreads, t = t0 + x / kRows, j = x % kRows;
      const size_t r = (size_t)(w.back ? end - 1 - t : begin + t);
      nv[e] = t < len ? load_io(w.value, r * w.value_stride + hd + slice * kRows + j, BF16 ? PACE_IO_BF16 : PACE_IO_F32) : 0.f;
    }
  };
  fetch(0);
  for (int t0 = 0; t0 < len; t0 += TT) {
#pragma unroll
    for (int e = 0; e < QKN; ++e) {
      const int x = tid + e * kWalkThreads;
      (&qs[0][0])[x] = nq[e];
      (&ks[0][0])[x] = nk[e];
    }
#pragma unroll
    for (int e = 0; e < VN; ++e) (&vs[0][0])[tid + e * kWalkThreads] = nv[e];
    __syncthreads();
    if (t0 + TT < len) fetch(t0 + TT);
    const int m = min(TT, len - t0);
    for (int t = 0; t < m; ++t) {
      const float v = vs[t][row];
      const float2 v2 = make_float2(v, v), a2 = make_float2(al, al);
      float2 acc = make_float2(0.f, 0.f), acc1 = make_float2(0.f, 0.f);
#pragma unroll
      for (int e = 0; e < V4; ++e) {
        const float4 kk = *reinterpret_cast<const float4*>(&ks[t][4 * (c + 4 * e)]);
        const float4 qq = *reinterpret_cast<const float4*>(&qs[t][4 * (c + 4 * e)]);
        float2 x0 = S[2 * e], x1 = S[2 * e + 1];
        if (!w.back) {
          x0 = __fmul2_rn(x0, a2);
          x1 = __fmul2_rn(x1, a2);
        }
        x0 = __ffma2_rn(v2, make_float2(kk.x, kk.y), x0);
        x1 = __ffma2_rn(v2, make_float2(kk.z, kk.w), x1);
        acc = __ffma2_rn(x0, make_float2(qq.x, qq.y), acc);
        acc1 = __ffma2_rn(x1, make_float2(qq.z, qq.w), acc1);
        if (w.back) {
          x0 = __fmul2_rn(x0, a2);
          x1 = __fmul2_rn(x1, a2);
        }
        S[2 * e] = x0;
        S[2 * e + 1] = x1;
      }
      float s = (acc.x + acc.y) + (acc1.x + acc1.y);
      s += __shfl_xor_sync(FULL, s, 1);
      s += __shfl_xor_sync(FULL, s, 2);
      if (c == 0) os[t][row] = s;
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < VN; ++e) {
      const int x = tid + e * kWalkThreads, t = x / kRows, j = x % kRows;
      if (t < m) {
        const size_t r = (size_t)(w.back ? end - 1 - (t0 + t) : begin + t0 + t);
        const size_t at = r * w.out_stride + hd + slice * kRows + j;
        if (BF16) reinterpret_cast<uint16_t*>(w.out)[at] = float_to_bf16_bits_rn(os[t][j]);
        else reinterpret_cast<float*>(w.out)[at] = os[t][j];
      }
    }
    __syncthreads();
  }
  if (w.S_out) {
#pragma unroll
    for (int e = 0; e < V4; ++e) {
      const float x[4] = {S[2 * e].x, S[2 * e].y, S[2 * e + 1].x, S[2 * e + 1].y};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int col = 4 * (c + 4 * e) + j;
        w.S_out[st0 + (w.swap ? (size_t)col * D + i : (size_t)i * D + col)] = x[j];
      }
    }
  }
}

template <int D>
cudaError_t walk(const LinArgs& a, cudaStream_t st) {
  const int64_t blocks = (int64_t)a.N * a.H * (D / kRows);
  if (blocks > 0x7fffffffll) return cudaErrorInvalidValue;
  const dim3 grid((unsigned)blocks, (unsigned)a.walks);
  if (a.io == PACE_IO_BF16) linattn_walk_kernel<D, true><<<grid, kWalkThreads, 0, st>>>(a);
  else linattn_walk_kernel<D, false><<<grid, kWalkThreads, 0, st>>>(a);
  return cudaGetLastError();
}

// ---- one token --------------------------------------------------------------------
// S is read and written once: 8 d^2 bytes a head, all else is small.  A warp
// takes RPW rows of one state; LPR lanes read a row in 16-byte pieces, so a
// warp's load is 512 contiguous bytes and RPW * D / 128 of them are in flight.
constexpr int kStepThreads = 128, RPW = 8;

template <int D, bool BF16>
__global__ void __launch_bounds__(kStepThreads)
    linattn_step_kernel(float* __restrict__ S, const void* __restrict__ q, const void* __restrict__ k,
                        const void* __restrict__ v, const float* __restrict__ log_decay, void* __restrict__ o,
                        int64_t qs, int64_t ks, int64_t vs, int64_t os, int H) {
  constexpr int LPR = D / 4, RPL = 32 / LPR, NL = RPW / RPL;    // lanes a row, rows a load, loads
  constexpr int IO = BF16 ? PACE_IO_BF16 : PACE_IO_F32;
  constexpr int WPH = D / RPW;                                  // warps a head
  const int lane = threadIdx.x & 31;
  const int64_t gw = (int64_t)blockIdx.x * (kStepThreads / 32) + (threadIdx.x >> 5);
  const int64_t head = gw / WPH;                                // n H + h
  const int r0 = (int)(gw % WPH) * RPW;
  const int64_t n = head / H;
  const int h = (int)(head % H);
  float4* base = reinterpret_cast<float4*>(S + (size_t)head * D * D + (size_t)r0 * D);
  float4 x[NL];
#pragma unroll
  for (int e = 0; e < NL; ++e) x[e] = base[e * 32 + lane];
  const float al = expf(clamp_log_decay(log_decay[h]));
  const int c = lane % LPR, rr = lane / LPR;
  float kk[4], qq[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    kk[j] = load_io(k, (size_t)(n * ks) + (size_t)h * D + 4 * c + j, IO);
    qq[j] = load_io(q, (size_t)(n * qs) + (size_t)h * D + 4 * c + j, IO);
  }
  float s[NL];
#pragma unroll
  for (int e = 0; e < NL; ++e) {
    const float vv = load_io(v, (size_t)(n * vs) + (size_t)h * D + r0 + e * RPL + rr, IO);
    x[e].x = fmaf(al, x[e].x, vv * kk[0]);
    x[e].y = fmaf(al, x[e].y, vv * kk[1]);
    x[e].z = fmaf(al, x[e].z, vv * kk[2]);
    x[e].w = fmaf(al, x[e].w, vv * kk[3]);
    base[e * 32 + lane] = x[e];
    s[e] = fmaf(x[e].x, qq[0], x[e].y * qq[1]) + fmaf(x[e].z, qq[2], x[e].w * qq[3]);
  }
#pragma unroll
  for (int e = 0; e < NL; ++e) {
#pragma unroll
    for (int off = LPR / 2; off; off >>= 1) s[e] += __shfl_xor_sync(FULL, s[e], off);
    if (c == 0) {
      const size_t at = (size_t)(n * os) + (size_t)h * D + r0 + e * RPL + rr;
      if (BF16) reinterpret_cast<uint16_t*>(o)[at] = float_to_bf16_bits_rn(s[e]);
      else reinterpret_cast<float*>(o)[at] = s[e];
    }
  }
}

template <int D>
cudaError_t step(float* S, const void* q, const void* k, const void* v, const float* g, void* o, int64_t qs, int64_t ks,
                 int64_t vs, int64_t os, int N, int H, int io, cudaStream_t st) {
  const int64_t blocks = (int64_t)N * H * (D / RPW) / (kStepThreads / 32);   // D / RPW is a multiple of 4
  if (blocks > 0x7fffffffll) return cudaErrorInvalidValue;
  if (io == PACE_IO_BF16)
    linattn_step_kernel<D, true><<<(unsigned)blocks, kStepThreads, 0, st>>>(S, q, k, v, g, o, qs, ks, vs, os, H);
  else
    linattn_step_kernel<D, false><<<(unsigned)blocks, kStepThreads, 0, st>>>(S, q, k, v, g, o, qs, ks, vs, os, H);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_linattn_stream(const LinArgs& a, cudaStream_t st) {
  switch (a.D) {
    case 32: return walk<32>(a, st);
    case 64: return walk<64>(a, st);
    case 128: return walk<128>(a, st);
  }
  return cudaErrorInvalidValue;
}

cudaError_t launch_linattn_step(float* S, const void* q, const void* k, const void* v, const float* log_decay, void* o,
                                int64_t qs, int64_t ks, int64_t vs, int64_t os, int N, int H, int D, int io,
                                cudaStream_t st) {
  switch (D) {
    case 32: return step<32>(S, q, k, v, log_decay, o, qs, ks, vs, os, N, H, io, st);
    case 64: return step<64>(S, q, k, v, log_decay, o, qs, ks, vs, os, N, H, io, st);
    case 128: return step<128>(S, q, k, v, log_decay, o, qs, ks, vs, os, N, H, io, st);
  }
  return cudaErrorInvalidValue;
}

}  // namespace pace
