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
// hundreds of tokens.  Heads that forget fast (g < -1) take the product each
// token: their memory is short, and A^-TT is then below 9e6 for the others, so
// that it is only for products value key^T above 1e31 that S could overflow.
//
// 8 sequences x 16 heads, 1000 tokens, d = 64, fp32: 124 us; 16 x 32 heads, 512 tokens: 177 us, where reads of shared
// memory and shuffles keep L1 85 % busy (the packed products have 29 % of their pipe's instruction slots, two each); with
// fewer heads it is latency.
constexpr int kWalkThreads = 128, kRows = 32, TT = 16;

template <int D>
struct WalkSmem {
  float q[TT][D], k[TT][D];
  float v[TT][kRows], o[TT][kRows];
  float up[TT + 1], down[TT + 1], down_lo[TT + 1];   // A^-p, A^p and the rest of A^p
};

template <int D, bool BACK, bool FAST, bool STATE_ONLY>
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
          const float4 qq = STATE_ONLY ? kk : *reinterpret_cast<const float4*>(&sm.q[t][col]);
          k2[e] = make_float2(kk.x, kk.y), k2[e + W - 1] = make_float2(kk.z, kk.w);
          q2[e] = make_float2(qq.x, qq.y), q2[e + W - 1] = make_float2(qq.z, qq.w);
        } else {
          k2[e] = *reinterpret_cast<const float2*>(&sm.k[t][col]);
          q2[e] = STATE_ONLY ? k2[e] : *reinterpret_cast<const float2*>(&sm.q[t][col]);
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
          if (!STATE_ONLY) s = __ffma2_rn(x, q2[e], s);
          if (FAST && BACK && t < m) x = __fmul2_rn(x, a2);
          S[r][e] = x;
        }
        acc[u][r] = s.x + s.y;
      }
    }
    if (STATE_ONLY) continue;
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

template <bool BF16>
__device__ __forceinline__ float4 load4(const void* p, size_t at, bool vec) {
  constexpr int IO = BF16 ? PACE_IO_BF16 : PACE_IO_F32;
  if (!vec) return make_float4(load_io(p, at, IO), load_io(p, at + 1, IO), load_io(p, at + 2, IO), load_io(p, at + 3, IO));
  if (!BF16) return *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(p) + at);
  const uint2 x = *reinterpret_cast<const uint2*>(reinterpret_cast<const uint16_t*>(p) + at);
  return make_float4(__uint_as_float(x.x << 16), __uint_as_float(x.x & 0xffff0000u), __uint_as_float(x.y << 16),
                     __uint_as_float(x.y & 0xffff0000u));
}
template <bool BF16>
__device__ __forceinline__ void store4(void* p, size_t at, float4 x, bool vec) {
  if (BF16) {
    uint16_t* to = reinterpret_cast<uint16_t*>(p) + at;
    const uint16_t b[4] = {float_to_bf16_bits_rn(x.x), float_to_bf16_bits_rn(x.y), float_to_bf16_bits_rn(x.z), float_to_bf16_bits_rn(x.w)};
    if (vec) *reinterpret_cast<uint2*>(to) = make_uint2(b[0] | (uint32_t)b[1] << 16, b[2] | (uint32_t)b[3] << 16);
    else to[0] = b[0], to[1] = b[1], to[2] = b[2], to[3] = b[3];
  } else {
    float* to = reinterpret_cast<float*>(p) + at;
    if (vec) *reinterpret_cast<float4*>(to) = x;
    else to[0] = x.x, to[1] = x.y, to[2] = x.z, to[3] = x.w;
  }
}

// `vec`: every row starts on a boundary of four elements, so that four go in one access.  STATE_ONLY: the contribution
// of each stretch to the state, from zeros into ws.
template <int D, bool BF16, bool STATE_ONLY>
__global__ void __launch_bounds__(kWalkThreads, D == 128 ? 1 : 0)      // (d = 128: 155 registers, not 216, 12 % faster)
    linattn_walk_kernel(const __grid_constant__ LinArgs a, const LinSplit sp, float* ws, bool vec) {
  constexpr int CP = D / 32, W = CP < 2 ? 1 : 2;
  constexpr int QKN = TT * D / kWalkThreads / 4;     // pieces of four elements a thread loads
  static_assert(TT * kRows == 4 * kWalkThreads, "one piece of the values and outputs a thread");
  __shared__ __align__(16) WalkSmem<D> sm;
  const int tid = threadIdx.x, rg = tid >> 4, c = tid & 15;
  constexpr int SL = D / kRows;                      // row slices of a state
  const int slice = blockIdx.x % SL;
  const int head = blockIdx.x / SL;                  // n H + h
  const int h = head % a.H, n = head / a.H, seg = blockIdx.z;
  const LinWalk& w = a.walk[blockIdx.y];
  int begin, end;
  seq_rows(a, n, &begin, &end);
  const int nseg = stretches_of(sp, end - begin), last = w.back ? 0 : nseg - 1;   // the stretch a walk ends with
  if (seg >= nseg || (STATE_ONLY && seg == last)) return;
  if (seg < nseg - 1) end = begin + (seg + 1) * sp.per * kLinChunk;
  begin += seg * sp.per * kLinChunk;
  const int len = end - begin;
  const float g = clamp_log_decay(a.log_decay[h]), al = expf(g);
  const bool fast = !(g >= -1.f);
  if (tid <= TT) {
    const double d = exp((double)g * tid);
    sm.down[tid] = (float)d;
    sm.down_lo[tid] = (float)(d - (double)(float)d);
    sm.up[tid] = fast ? 1.f : (float)exp(-(double)g * tid);
  }
  // the state before: the caller's, or the chain's, which lie as the walk wants them
  const size_t st0 = (size_t)head * D * D;
  float* const stretch = nseg > 1 ? ws + (size_t)stretch_index(a, sp, blockIdx.y, n, h, seg) * D * D : nullptr;
  const float* S_in = STATE_ONLY ? nullptr : (stretch ? stretch : w.S_in ? w.S_in + st0 : nullptr);
  float* S_out = STATE_ONLY ? stretch : (w.S_out && seg == last ? w.S_out + st0 : nullptr);
  const bool swap_in = w.swap && !stretch, swap_out = w.swap && !STATE_ONLY;
  float2 S[4][CP];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int i = slice * kRows + 4 * rg + r;
#pragma unroll
    for (int e = 0; e < CP; ++e) {
      const int col = 2 * W * c + 32 * (e / W) * W + 2 * (e % W);
      S[r][e] = make_float2(0.f, 0.f);
      if (S_in) {
        S[r][e].x = S_in[swap_in ? (size_t)col * D + i : (size_t)i * D + col];
        S[r][e].y = S_in[swap_in ? (size_t)(col + 1) * D + i : (size_t)i * D + col + 1];
      }
    }
  }
  const size_t hd = (size_t)h * D;
  float4 nq[QKN], nk[QKN], nv;
  const int vt = tid / (kRows / 4), vj = tid % (kRows / 4) * 4;    // this thread's piece of the values and outputs
  auto row_of = [&](int t) { return (size_t)(w.back ? end - 1 - t : begin + t); };
  auto fetch = [&](int t0) {                         // tokens t0 .. t0 + TT - 1 in walking order
    const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int e = 0; e < QKN; ++e) {
      const int x = 4 * (tid + e * kWalkThreads), t = t0 + x / D, j = x % D;
      const size_t r = row_of(t);
      nq[e] = nk[e] = zero;
      if (t < len) {
        if (!STATE_ONLY) nq[e] = load4<BF16>(w.query, r * w.query_stride + hd + j, vec);
        nk[e] = load4<BF16>(w.key, r * w.key_stride + hd + j, vec);
      }
    }
    nv = t0 + vt < len ? load4<BF16>(w.value, row_of(t0 + vt) * w.value_stride + hd + slice * kRows + vj, vec) : zero;
  };
  fetch(0);
  __syncthreads();                                   // the tables
  for (int t0 = 0; t0 < len; t0 += TT) {
#pragma unroll
    for (int e = 0; e < QKN; ++e) {
      const int x = 4 * (tid + e * kWalkThreads);
      if (!STATE_ONLY) *reinterpret_cast<float4*>(&sm.q[0][0] + x) = nq[e];
      *reinterpret_cast<float4*>(&sm.k[0][0] + x) = nk[e];
    }
    const float up = sm.up[w.back ? vt : vt + 1];
    *reinterpret_cast<float4*>(&sm.v[vt][vj]) = make_float4(nv.x * up, nv.y * up, nv.z * up, nv.w * up);
    __syncthreads();
    if (t0 + TT < len) fetch(t0 + TT);
    const int m = min(TT, len - t0);
    if (fast) {
      if (w.back) walk_tokens<D, true, true, STATE_ONLY>(sm, S, m, rg, c, al);
      else walk_tokens<D, false, true, STATE_ONLY>(sm, S, m, rg, c, al);
    } else {
      if (w.back) walk_tokens<D, true, false, STATE_ONLY>(sm, S, m, rg, c, al);
      else walk_tokens<D, false, false, STATE_ONLY>(sm, S, m, rg, c, al);
      const float2 hi = make_float2(sm.down[m], sm.down[m]), lo = make_float2(sm.down_lo[m], sm.down_lo[m]);
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int e = 0; e < CP; ++e) S[r][e] = __ffma2_rn(S[r][e], hi, __fmul2_rn(S[r][e], lo));
    }
    __syncthreads();
    if (!STATE_ONLY && vt < m)
      store4<BF16>(w.out, row_of(t0 + vt) * w.out_stride + hd + slice * kRows + vj, *reinterpret_cast<const float4*>(&sm.o[vt][vj]), vec);
  }
  if (S_out) {
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int i = slice * kRows + 4 * rg + r;
#pragma unroll
      for (int e = 0; e < CP; ++e) {
        const int col = 2 * W * c + 32 * (e / W) * W + 2 * (e % W);
        S_out[swap_out ? (size_t)col * D + i : (size_t)i * D + col] = S[r][e].x;
        S_out[swap_out ? (size_t)(col + 1) * D + i : (size_t)i * D + col + 1] = S[r][e].y;
      }
    }
  }
}

// ---- chaining the stretches ----------------------------------------------------------
// ws[s] (stretch s's own contribution) -> the state before stretch s, in the walk's order:
//   run = S_in;  for s in order: (ws[s], run) = (run, A^tokens(s) run + ws[s]).
// A thread chains four elements, the next stretches' loads in flight; with four times the elements and no loads ahead it
// took 131 us where this takes 8 (9 stretches of 32 heads, d = 128).
constexpr int kChainAhead = 4;
template <int D>
__global__ void __launch_bounds__(256)
    linattn_chain_kernel(const __grid_constant__ LinArgs a, const LinSplit sp, float* states) {
  __shared__ float decay[2];
  const int wi = blockIdx.x % a.walks, head = blockIdx.x / a.walks, h = head % a.H, n = head / a.H;
  int begin, end;
  seq_rows(a, n, &begin, &end);
  const int ns = stretches_of(sp, end - begin);
  if (ns <= 1) return;
  const LinWalk& w = a.walk[wi];
  if (threadIdx.x < 2) {
    // every stretch but the sequence's last one is `per` chunks long
    const double full = (double)sp.per * kLinChunk, tokens = threadIdx.x ? (end - begin) - (ns - 1) * full : full;
    decay[threadIdx.x] = (float)exp((double)clamp_log_decay(a.log_decay[h]) * tokens);
  }
  __syncthreads();
  const int y = (blockIdx.y * 256 + threadIdx.x) * 4;
  float* ws = states + (size_t)stretch_index(a, sp, wi, n, h, 0) * D * D + y;
  const size_t st0 = (size_t)head * D * D;
  auto at = [&](int k) { return reinterpret_cast<float4*>(ws + (size_t)(w.back ? ns - 1 - k : k) * D * D); };
  float4 run = make_float4(0.f, 0.f, 0.f, 0.f), own[kChainAhead];
#pragma unroll
  for (int k = 0; k < kChainAhead; ++k)
    if (k + 1 < ns) own[k] = *at(k);
  if (w.S_in) {
    if (w.swap) {
      const int i = y / D, j = y % D;
      run = make_float4(w.S_in[st0 + (size_t)j * D + i], w.S_in[st0 + (size_t)(j + 1) * D + i],
                        w.S_in[st0 + (size_t)(j + 2) * D + i], w.S_in[st0 + (size_t)(j + 3) * D + i]);
    } else {
      run = *reinterpret_cast<const float4*>(w.S_in + st0 + y);
    }
  }
  for (int k0 = 0; k0 < ns; k0 += kChainAhead) {
#pragma unroll
    for (int u = 0; u < kChainAhead; ++u) {
      const int k = k0 + u;
      if (k >= ns) break;
      const float4 o = own[u];
      if (k + kChainAhead + 1 < ns) own[u] = *at(k + kChainAhead);
      *at(k) = run;
      const float al = decay[(w.back ? ns - 1 - k : k) == ns - 1];
      if (k + 1 < ns) run = make_float4(fmaf(al, run.x, o.x), fmaf(al, run.y, o.y), fmaf(al, run.z, o.z), fmaf(al, run.w, o.w));
    }
  }
}

template <int D, bool BF16>
cudaError_t walk(const LinArgs& a, const LinSplit& sp, float* ws, cudaStream_t st) {
  const int64_t blocks = (int64_t)a.N * a.H * (D / kRows);
  if (blocks > 0x7fffffffll || sp.stretches > 65535) return cudaErrorInvalidValue;
  const size_t four = BF16 ? 8 : 16;
  bool vec = true;
  for (int i = 0; i < a.walks; ++i) {
    const LinWalk& w = a.walk[i];
    vec = vec && ((uintptr_t)w.query | (uintptr_t)w.key | (uintptr_t)w.value | (uintptr_t)w.out) % four == 0 &&
          (w.query_stride | w.key_stride | w.value_stride | w.out_stride) % 4 == 0;
  }
  const dim3 grid((unsigned)blocks, (unsigned)a.walks, (unsigned)sp.stretches);
  if (sp.stretches > 1) {
    linattn_walk_kernel<D, BF16, true><<<grid, kWalkThreads, 0, st>>>(a, sp, ws, vec);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || (e = launch_linattn_chain(a, sp, ws, st)) != cudaSuccess) return e;
  }
  linattn_walk_kernel<D, BF16, false><<<grid, kWalkThreads, 0, st>>>(a, sp, ws, vec);
  return cudaGetLastError();
}

// ---- one token --------------------------------------------------------------------
// S is read and written once: 8 d^2 bytes a head, all else is small.  A warp
// takes RPW rows of one state; LPR lanes read a row in 16-byte pieces, so a
// warp's load is 512 contiguous bytes and RPW * D / 128 of them are in flight.
// 256 sequences x 48 heads, d = 128: 246 us, the copy's bandwidth.
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

LinSplit linattn_stream_split(int64_t heads, int64_t max_len, int walks, int D) {
  // The first pass has no queries and no sums over threads, but it and the chain come on top.
  const int64_t items = heads * walks * (D / kRows);
  if (D == 128) {
    // Three rounds of the 3 blocks an SM holds, so that the last one's idle SMs weigh little, but a sequence in no more than
    // 148 stretches (the chain).  fp32, us, against one and a third rounds, as before / one round / uncut: 8 heads x 4096
    // tokens 129 / 142 / 128 / 486, their gradients 324 / 341 / 368 / 488; 48 heads 611 / 716 / 668 / 716; 16 heads x 1024
    // tokens 73 / 78 / 82 / 126.  It gained with 192 blocks (those 48 heads) and lost from 220 on (55 heads x 2048 tokens: 361
    // uncut, 371 cut; 4 x 16 heads: 361, 407; gradients of 32 heads x 4096 tokens: 973, 1150).
    const int64_t fill = 148 * (items < 9 ? items : 9);
    return lin_split(items, max_len, items <= 200 ? fill : 0, 1, 4);
  }
  // As many blocks as the SMs hold at once by their registers.  Cutting gained from four stretches on (16 heads, 256 tokens,
  // d = 64: 25 -> 16 us; 8 x 32 heads, 2048 tokens, d = 32, bf16: 266 -> 181 us).
  return lin_split(items, max_len, 148 * (D == 32 ? 7 : 5), 1, 4);
}

cudaError_t launch_linattn_stream(const LinArgs& a, const LinSplit& sp, float* ws, cudaStream_t st) {
  const bool b = a.io == PACE_IO_BF16;
  switch (a.D) {
    case 32: return b ? walk<32, true>(a, sp, ws, st) : walk<32, false>(a, sp, ws, st);
    case 64: return b ? walk<64, true>(a, sp, ws, st) : walk<64, false>(a, sp, ws, st);
    case 128: return b ? walk<128, true>(a, sp, ws, st) : walk<128, false>(a, sp, ws, st);
  }
  return cudaErrorInvalidValue;
}

cudaError_t launch_linattn_chain(const LinArgs& a, const LinSplit& sp, float* ws, cudaStream_t st) {
  const dim3 grid((unsigned)((int64_t)a.N * a.H * a.walks), (unsigned)(a.D * a.D / 1024));
  switch (a.D) {
    case 32: linattn_chain_kernel<32><<<grid, 256, 0, st>>>(a, sp, ws); break;
    case 64: linattn_chain_kernel<64><<<grid, 256, 0, st>>>(a, sp, ws); break;
    case 128: linattn_chain_kernel<128><<<grid, 256, 0, st>>>(a, sp, ws); break;
    default: return cudaErrorInvalidValue;
  }
  return cudaGetLastError();
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
