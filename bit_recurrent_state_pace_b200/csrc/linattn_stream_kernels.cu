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
// A block walks one sequence and head for 32 rows of S, which never leave the
// registers: sixteen threads hold four rows, D / 16 columns of them each, so
// that a token costs a thread 8 D / 32 packed products for a few loads of its
// key, query and value from shared memory.  Tokens come there TT at a time,
// the next ones being loaded while these are used; the outputs of four tokens
// and four rows are summed over the sixteen threads together.
//
// Within TT tokens S is kept without its decay: token t adds value / A^p key^T
// (p tokens of decay so far) and reads A^p S query, and the decay of all TT is
// applied once, in 48 bits -- a product each token would cost half as much
// again and, by a fixed rounding of A, several 1e-6 of a state that remembers
// hundreds of tokens.  Heads that forget faster than A^-TT can hold (g < -3)
// take the product each token.
constexpr int kWalkThreads = 128, kRows = 32, TT = 16;

template <int D>
struct WalkSmem {
  float q[TT][D], k[TT][D];
  float v[TT][kRows], o[TT][kRows];
  float up[TT + 1], down[TT + 1], down_lo[TT + 1];   // A^-p, A^p and the rest of A^p
};

template <int D, bool BACK, bool FAST>
__device__ __forceinline__ void walk_tokens(WalkSmem<D>& sm, float2 (&S)[4][D / 32], int m, int rg, int c, float al) {
  constexpr int CP = D / 32;                         // column pairs of a thread
  constexpr int W = CP < 2 ? 1 : 2;                  // pairs a load
  const float2 a2 = make_float2(al, al);
  for (int t0 = 0; t0 < m; t0 += 4) {
    float acc[4][4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int t = t0 + u;                          // tokens from m on hold zeros
      const float4 v4 = *reinterpret_cast<const float4*>(&sm.v[t][4 * rg]);
      const float v[4] = {v4.x, v4.y, v4.z, v4.w};
      float2 k2[CP], q2[CP];
#pragma unroll
      for (int e = 0; e < CP; e += W) {
        const int col = 2 * W * c + 32 * e;
        if (W == 2) {
          const float4 kk = *reinterpret_cast<const float4*>(&sm.k[t][col]);
          const float4 qq = *reinterpret_cast<const float4*>(&sm.q[t][col]);
          k2[e] = make_float2(kk.x, kk.y), k2[e + W - 1] = make_float2(kk.z, kk.w);
          q2[e] = make_float2(qq.x, qq.y), q2[e + W - 1] = make_float2(qq.z, qq.w);
        } else {
          k2[e] = *reinterpret_cast<const float2*>(&sm.k[t][col]);
          q2[e] = *reinterpret_cast<const float2*>(&sm.q[t][col]);
        }
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float2 v2 = make_float2(v[r], v[r]);
        float2 s = make_float2(0.f, 0.f);
#pragma unroll
        for (int e = 0; e < CP; ++e) {
          float2 x = S[r][e];
          if (FAST && !BACK && t < m) x = __fmul2_rn(x, a2);
          x = __ffma2_rn(v2, k2[e], x);
          s = __ffma2_rn(x, q2[e], s);
          if (FAST && BACK && t < m) x = __fmul2_rn(x, a2);
          S[r][e] = x;
        }
        acc[u][r] = s.x + s.y;
      }
    }
    // sums over the 16 threads: each step halves the values a thread keeps; thread c ends with token c / 4, row c % 4
    float h8[8], h4[4], h2[2];
    const bool b3 = c & 8, b2 = c & 4, b1 = c & 2, b0 = c & 1;
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      const float lo = acc[x >> 2][x & 3], hi = acc[2 + (x >> 2)][x & 3];
      h8[x] = (b3 ? hi : lo) + __shfl_xor_sync(FULL, b3 ? lo : hi, 8);
    }
#pragma unroll
    for (int x = 0; x < 4; ++x) h4[x] = (b2 ? h8[4 + x] : h8[x]) + __shfl_xor_sync(FULL, b2 ? h8[x] : h8[4 + x], 4);
#pragma unroll
    for (int x = 0; x < 2; ++x) h2[x] = (b1 ? h4[2 + x] : h4[x]) + __shfl_xor_sync(FULL, b1 ? h4[x] : h4[2 + x], 2);
    const float o = (b0 ? h2[1] : h2[0]) + __shfl_xor_sync(FULL, b0 ? h2[0] : h2[1], 1);
    const int t = t0 + (c >> 2);
    sm.o[t][4 * rg + (c & 3)] = FAST ? o : o * sm.down[BACK ? t : t + 1];
  }
}

template <int D, bool BF16>
__global__ void __launch_bounds__(kWalkThreads) linattn_walk_kernel(const __grid_constant__ LinArgs a) {
  constexpr int CP = D / 32, W = CP < 2 ? 1 : 2;
  constexpr int QKN = TT * D / kWalkThreads, VN = TT * kRows / kWalkThreads;
  constexpr int IO = BF16 ? PACE_IO_BF16 : PACE_IO_F32;
  __shared__ __align__(16) WalkSmem<D> sm;
  const int tid = threadIdx.x, rg = tid >> 4, c = tid & 15;
  constexpr int SL = D / kRows;                      // row slices of a state
  const int slice = blockIdx.x % SL;
  const int rest = blockIdx.x / SL;
  const int h = rest % a.H, n = rest / a.H;
  const LinWalk& w = a.walk[blockIdx.y];
  int begin, end;
  seq_rows(a, n, &begin, &end);
  const int len = end - begin;
  const float g = clamp_log_decay(a.log_decay[h]), al = expf(g);
  const bool fast = !(g >= -3.f);
  if (tid <= TT) {
    const double d = exp((double)g * tid);
    sm.down[tid] = (float)d;
    sm.down_lo[tid] = (float)(d - (double)(float)d);
    sm.up[tid] = fast ? 1.f : (float)exp(-(double)g * tid);
  }
  const size_t st0 = ((size_t)n * a.H + h) * D * D;
  float2 S[4][CP];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int i = slice * kRows + 4 * rg + r;
#pragma unroll
    for (int e = 0; e < CP; ++e) {
      const int col = 2 * W * c + 32 * (e / W) * W + 2 * (e % W);
      S[r][e] = make_float2(0.f, 0.f);
      if (w.S_in) {
        S[r][e].x = w.S_in[st0 + (w.swap ? (size_t)col * D + i : (size_t)i * D + col)];
        S[r][e].y = w.S_in[st0 + (w.swap ? (size_t)(col + 1) * D + i : (size_t)i * D + col + 1)];
      }
    }
  }
  const size_t hd = (size_t)h * D;
  float nq[QKN], nk[QKN], nv[VN];
  auto fetch = [&](int t0) {                         // tokens t0 .. t0 + TT - 1 in walking order
#pragma unroll
    for (int e = 0; e < QKN; ++e) {
      const int x = tid + e * kWalkThreads, t = t0 + x / D, j = x % D;
      const bool in = t < len;
      const size_t r = (size_t)(w.back ? end - 1 - t : begin + t);
      nq[e] = in ? load_io(w.query, r * w.query_stride + hd + j, IO) : 0.f;
      nk[e] = in ? load_io(w.key, r * w.key_stride + hd + j, IO) : 0.f;
    }
#pragma unroll
    for (int e = 0; e < VN; ++e) {
      const int x = tid + e * kWalkThreads, t = t0 + x / kRows, j = x % kRows;
      const size_t r = (size_t)(w.back ? end - 1 - t : begin + t);
      nv[e] = t < len ? load_io(w.value, r * w.value_stride + hd + slice * kRows + j, IO) : 0.f;
    }
  };
  fetch(0);
  __syncthreads();                                   // the tables
  for (int t0 = 0; t0 < len; t0 += TT) {
#pragma unroll
    for (int e = 0; e < QKN; ++e) {
      const int x = tid + e * kWalkThreads;
      (&sm.q[0][0])[x] = nq[e];
      (&sm.k[0][0])[x] = nk[e];
    }
#pragma unroll
    for (int e = 0; e < VN; ++e) {
      const int x = tid + e * kWalkThreads, t = x / kRows;
      (&sm.v[0][0])[x] = nv[e] * sm.up[w.back ? t : t + 1];
    }
    __syncthreads();
    if (t0 + TT < len) fetch(t0 + TT);
    const int m = min(TT, len - t0);
    if (fast) {
      if (w.back) walk_tokens<D, true, true>(sm, S, m, rg, c, al);
      else walk_tokens<D, false, true>(sm, S, m, rg, c, al);
    } else {
      if (w.back) walk_tokens<D, true, false>(sm, S, m, rg, c, al);
      else walk_tokens<D, false, false>(sm, S, m, rg, c, al);
      const float2 hi = make_float2(sm.down[m], sm.down[m]), lo = make_float2(sm.down_lo[m], sm.down_lo[m]);
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int e = 0; e < CP; ++e) S[r][e] = __ffma2_rn(S[r][e], hi, __fmul2_rn(S[r][e], lo));
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < VN; ++e) {
      const int x = tid + e * kWalkThreads, t = x / kRows, j = x % kRows;
      if (t < m) {
        const size_t r = (size_t)(w.back ? end - 1 - (t0 + t) : begin + t0 + t);
        const size_t at = r * w.out_stride + hd + slice * kRows + j;
        if (BF16) reinterpret_cast<uint16_t*>(w.out)[at] = float_to_bf16_bits_rn(sm.o[t][j]);
        else reinterpret_cast<float*>(w.out)[at] = sm.o[t][j];
      }
    }
  }
  if (w.S_out) {
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int i = slice * kRows + 4 * rg + r;
#pragma unroll
      for (int e = 0; e < CP; ++e) {
        const int col = 2 * W * c + 32 * (e / W) * W + 2 * (e % W);
        w.S_out[st0 + (w.swap ? (size_t)col * D + i : (size_t)i * D + col)] = S[r][e].x;
        w.S_out[st0 + (w.swap ? (size_t)(col + 1) * D + i : (size_t)i * D + col + 1)] = S[r][e].y;
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
