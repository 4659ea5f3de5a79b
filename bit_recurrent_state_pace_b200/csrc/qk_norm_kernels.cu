// Queries and keys normalised for each head and turned by their position, and
// the gradients of that, one pass over the data each.
//
//   y = s R(pos) (w * x r),  r = (sum x^2 / n + eps)^(-1/2)
//   u = s R(-pos) dy,  dw = sum u * x^,  h = u * w,  dx = r (h - x^ (x^ . h) / n),  x^ = x r
//
// Memory-bound: 2 (3 in the backward pass) times the tensors' bytes.  The rows
// of all tokens, each token's queries before its keys, are one list; a block
// of 256 threads takes a stretch of it.  A row is held by L lanes of one warp,
// 8 elements (one 16-byte load in bf16) each, so a warp's loads are full lines
// and both sums are shuffles; a thread has U rows' loads in flight.  Angles
// are computed once for each token of the stretch, into shared memory, while
// the loads fly: pos * inv_freq / 2 pi in fp64, whose fraction alone goes on
// in fp32, so that far positions lose nothing.
#include "linattn.cuh"

namespace pace {

namespace {

constexpr unsigned FULL = 0xffffffffu;
constexpr int kThreads = 256;
constexpr int kMaxBackBlocks = 148 * 4;

// lanes that hold a row: the power of two that gives each at most 8 elements
inline int lanes_of(int D) {
  int L = 1;
  while (8 * L < D) L *= 2;
  return L;
}

struct Row {
  bool in;          // there is such a row and this lane holds a part of it
  int side, head, ltok;
  size_t tok;
};

template <bool BF16, bool VEC>
__device__ __forceinline__ void load8(const void* p, size_t at, float (&x)[8]) {
  if (BF16) {
    if (VEC) {
      const uint4 u = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(p) + at);
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x[2 * j] = __uint_as_float(w[j] << 16);
        x[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = load_io(p, at + j, PACE_IO_BF16);
    }
  } else {
    const float* f = reinterpret_cast<const float*>(p) + at;
    if (VEC) {
      const float4 a = *reinterpret_cast<const float4*>(f), b = *reinterpret_cast<const float4*>(f + 4);
      x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = f[j];
    }
  }
}

template <bool BF16, bool VEC>
__device__ __forceinline__ void store8(void* p, size_t at, const float (&x)[8]) {
  if (BF16) {
    uint16_t* b = reinterpret_cast<uint16_t*>(p) + at;
    if (VEC) {
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * j], x[2 * j + 1]);
        w[j] = *reinterpret_cast<const uint32_t*>(&h);
      }
      *reinterpret_cast<uint4*>(b) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) b[j] = float_to_bf16_bits_rn(x[j]);
    }
  } else {
    float* f = reinterpret_cast<float*>(p) + at;
    if (VEC) {
      *reinterpret_cast<float4*>(f) = make_float4(x[0], x[1], x[2], x[3]);
      *reinterpret_cast<float4*>(f + 4) = make_float4(x[4], x[5], x[6], x[7]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = x[j];
    }
  }
}

__device__ __forceinline__ float row_sum(float s, int L) {
  for (int off = L >> 1; off; off >>= 1) s += __shfl_xor_sync(FULL, s, off);
  return s;
}

// cos and sin of every pair's angle for the `ntok` tokens from tok0 on: tab[ltok][pair]
__device__ __forceinline__ void angle_table(const NormArgs& a, float2* tab, size_t tok0, int ntok) {
  const int half = a.rot >> 1;
  for (int e = threadIdx.x; e < ntok * half; e += kThreads) {
    const int lt = e / half, i = e - lt * half;
    if (tok0 + lt < (size_t)a.tokens) {
      const double turns = (double)a.pos[tok0 + lt] * (double)a.inv_freq[i] * 0.15915494309189533577;
      const float f = (float)(turns - rint(turns));
      float s, c;
      sincospif(2.f * f, &s, &c);
      tab[e] = make_float2(c, s);
    }
  }
}

// Turns the row held by the lanes of this group by `sgn` times its angles.  c: the lane's place in its row.
// Half-split pairs lie rotary_dim / 2 apart: whole lanes apart where that is a multiple of 8, and come by
// shuffles; else through shared memory.
__device__ __forceinline__ void turn8(const NormArgs& a, float (&y)[8], const float2* t, float sgn, int c, int L, float* xch) {
  const int col = 8 * c, half = a.rot >> 1;
  if (a.interleaved) {
    if (col < a.rot) {
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        if (col + j < a.rot) {
          const float2 cs = t[(col + j) >> 1];
          const float s = sgn * cs.y, u = y[j], v = y[j + 1];
          y[j] = u * cs.x - v * s;
          y[j + 1] = v * cs.x + u * s;
        }
      }
    }
    return;
  }
  if ((half & 7) == 0) {
    const int lane = threadIdx.x & 31, hl = half >> 3, base = lane - c;
    const int from = c < hl ? c + hl : (c < 2 * hl ? c - hl : c);
    const float flip = c < hl ? -sgn : sgn;
    const bool on = c < 2 * hl;
    const int i0 = c < hl ? col : col - half;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float o = __shfl_sync(FULL, y[j], base + from);
      if (on) {
        const float2 cs = t[i0 + j];
        y[j] = y[j] * cs.x + o * (flip * cs.y);
      }
    }
    return;
  }
  float* mine = xch + (size_t)(threadIdx.x - c) * 8;    // the row, 8 L floats
#pragma unroll
  for (int j = 0; j < 8; ++j) mine[col + j] = y[j];
  __syncwarp();
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int x = col + j;
    if (x < half) {
      const float2 cs = t[x];
      y[j] = y[j] * cs.x - mine[x + half] * (sgn * cs.y);
    } else if (x < a.rot) {
      const float2 cs = t[x - half];
      y[j] = y[j] * cs.x + mine[x - half] * (sgn * cs.y);
    }
  }
  __syncwarp();
}

// Row `first + off` of the list, first being row r0 of token tok0.
__device__ __forceinline__ Row locate(const NormArgs& a, int64_t first, int64_t rows, size_t tok0, int r0, int R, int off, int c) {
  Row r;
  const int x = r0 + off;
  r.ltok = x / R;
  int head = x - r.ltok * R;
  r.side = head >= a.side[0].heads ? 1 : 0;
  r.head = r.side ? head - a.side[0].heads : head;
  r.tok = tok0 + r.ltok;
  r.in = first + off < rows && 8 * c < a.D;
  return r;
}

template <bool BF16, bool VEC, int U>
__global__ void __launch_bounds__(kThreads) qk_norm_kernel(const __grid_constant__ NormArgs a, int L) {
  extern __shared__ float2 tab[];
  float* xch = nullptr;
  const int c = threadIdx.x & (L - 1), slot = threadIdx.x / L, slots = kThreads / L;
  const int R = a.side[0].heads + a.side[1].heads;
  const int64_t rows = (int64_t)a.tokens * R, first = (int64_t)blockIdx.x * (slots * U);
  const size_t tok0 = (size_t)(first / R);
  const int r0 = (int)(first - (int64_t)tok0 * R);
  Row row[U];
  float x[U][8];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    row[u] = locate(a, first, rows, tok0, r0, R, u * slots + slot, c);
    const NormSide& s = a.side[row[u].side];
    if (row[u].in) load8<BF16, VEC>(s.x, row[u].tok * s.x_stride + (size_t)row[u].head * a.D + 8 * c, x[u]);
    else {
#pragma unroll
      for (int j = 0; j < 8; ++j) x[u][j] = 0.f;
    }
  }
  if (a.rot) {
    const int ntok = (r0 + slots * U - 1) / R + 1;
    angle_table(a, tab, tok0, ntok);
    xch = reinterpret_cast<float*>(tab + (size_t)ntok * (a.rot >> 1));
    __syncthreads();
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const NormSide& s = a.side[row[u].side];
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = fmaf(x[u][j], x[u][j], ss);
    ss = row_sum(ss, L);
    const float r = rsqrtf(fmaf(ss, a.inv_n, a.eps));
    if (s.w && row[u].in) {
      float w[8];
      load8<false, false>(s.w, 8 * c, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) x[u][j] = x[u][j] * r * w[j];
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) x[u][j] *= r;
    }
    if (a.rot) turn8(a, x[u], tab + (size_t)row[u].ltok * (a.rot >> 1), 1.f, c, L, xch);
#pragma unroll
    for (int j = 0; j < 8; ++j) x[u][j] *= s.scale;
    if (row[u].in) store8<BF16, VEC>(s.y, row[u].tok * s.y_stride + (size_t)row[u].head * a.D + 8 * c, x[u]);
  }
}

template <bool BF16, bool VEC, int U, bool DW>
__global__ void __launch_bounds__(kThreads) qk_norm_backward_kernel(const __grid_constant__ NormArgs a, int L, int64_t tiles) {
  extern __shared__ float2 tab[];
  const int c = threadIdx.x & (L - 1), slot = threadIdx.x / L, slots = kThreads / L;
  const int R = a.side[0].heads + a.side[1].heads;
  const int64_t rows = (int64_t)a.tokens * R;
  const int maxtok = a.rot ? (R - 1 + slots * U - 1) / R + 1 : 0;
  float* xch = reinterpret_cast<float*>(tab + (size_t)maxtok * (a.rot >> 1));
  float dw[2][8];
#pragma unroll
  for (int j = 0; j < 8; ++j) dw[0][j] = dw[1][j] = 0.f;
  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int64_t first = tile * (slots * U);
    const size_t tok0 = (size_t)(first / R);
    const int r0 = (int)(first - (int64_t)tok0 * R);
    Row row[U];
    float x[U][8], g[U][8];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      row[u] = locate(a, first, rows, tok0, r0, R, u * slots + slot, c);
      const NormSide& s = a.side[row[u].side];
      if (row[u].in) {
        load8<BF16, VEC>(s.x, row[u].tok * s.x_stride + (size_t)row[u].head * a.D + 8 * c, x[u]);
        load8<BF16, VEC>(s.dy, (row[u].tok * s.heads + row[u].head) * a.D + 8 * c, g[u]);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[u][j] = g[u][j] = 0.f;
      }
    }
    if (a.rot) {
      if (tile != (int64_t)blockIdx.x) __syncthreads();      // the last tile's table is done with
      angle_table(a, tab, tok0, (r0 + slots * U - 1) / R + 1);
      __syncthreads();
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const NormSide& s = a.side[row[u].side];
      if (a.rot) turn8(a, g[u], tab + (size_t)row[u].ltok * (a.rot >> 1), -1.f, c, L, xch);
      float ss = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = fmaf(x[u][j], x[u][j], ss);
      ss = row_sum(ss, L);
      const float r = rsqrtf(fmaf(ss, a.inv_n, a.eps));
      float w[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = 1.f;
      if (s.w && row[u].in) load8<false, false>(s.w, 8 * c, w);
      float dot = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        x[u][j] *= r;                                         // x^
        g[u][j] *= s.scale;                                   // u
        if (DW) {
          const float t = x[u][j] * g[u][j];
          if (row[u].in) {
            if (row[u].side) dw[1][j] += t;
            else dw[0][j] += t;
          }
        }
        g[u][j] *= w[j];                                      // h
        dot = fmaf(x[u][j], g[u][j], dot);
      }
      dot = row_sum(dot, L) * a.inv_n;
#pragma unroll
      for (int j = 0; j < 8; ++j) g[u][j] = r * (g[u][j] - x[u][j] * dot);
      if (row[u].in) store8<BF16, VEC>(s.y, row[u].tok * s.y_stride + (size_t)row[u].head * a.D + 8 * c, g[u]);
    }
  }
  if (DW) {
    // this block's sums: over its row slots, in the order of the slots
    __shared__ float red[kThreads * 8];
    for (int side = 0; side < 2; ++side) {
      __syncthreads();
#pragma unroll
      for (int j = 0; j < 8; ++j) red[threadIdx.x * 8 + j] = dw[side][j];
      __syncthreads();
      for (int col = threadIdx.x; col < a.D; col += kThreads) {
        float s = 0.f;
        for (int k = 0; k < slots; ++k) s += red[k * L * 8 + col];
        a.partial[((size_t)blockIdx.x * 2 + side) * a.D + col] = s;
      }
    }
  }
}

// Sums the blocks' partial sums of 32 columns of one side: 8 threads a column, each a stretch of the blocks in
// order, then the 8 in order.
__global__ void __launch_bounds__(256) qk_norm_reduce_kernel(const float* __restrict__ partial, int blocks, int D,
                                                             float* dwq, float* dwk) {
  __shared__ float red[8][32];
  const int side = blockIdx.y, col = blockIdx.x * 32 + (threadIdx.x & 31), k = threadIdx.x >> 5;
  float* dw = side ? dwk : dwq;
  if (!dw) return;
  float s = 0.f;
  const int per = (blocks + 7) / 8, b1 = min(blocks, (k + 1) * per);
  if (col < D)
    for (int b = k * per; b < b1; ++b) s += partial[((size_t)b * 2 + side) * D + col];
  red[k][threadIdx.x & 31] = s;
  __syncthreads();
  if (k == 0 && col < D) {
    for (int e = 1; e < 8; ++e) s += red[e][threadIdx.x & 31];
    dw[col] = s;
  }
}

bool aligned16(const NormArgs& a, bool back) {
  const size_t e = a.io == PACE_IO_BF16 ? 2 : 4;
  for (const NormSide& s : a.side) {
    if (!s.heads) continue;
    if (((uintptr_t)s.x | (uintptr_t)s.y | (back ? (uintptr_t)s.dy : 0)) % 16) return false;
    if ((s.x_stride * e) % 16 || (s.y_stride * e) % 16) return false;
  }
  return true;
}

// tokens that a stretch of `rows` rows can touch
size_t table_bytes(const NormArgs& a, int rows, bool exchange) {
  const int R = a.side[0].heads + a.side[1].heads;
  const size_t ntok = a.rot ? (size_t)(R - 1 + rows - 1) / R + 1 : 0;
  return ntok * (a.rot / 2) * sizeof(float2) + (exchange ? kThreads * 8 * sizeof(float) : 0);
}

inline bool needs_exchange(const NormArgs& a) { return a.rot && !a.interleaved && (a.rot / 2) % 8 != 0; }

template <bool BF16, bool VEC, int U>
cudaError_t forward(const NormArgs& a, int64_t rows, int L, cudaStream_t st) {
  const int per = kThreads / L * U;
  const int64_t blocks = (rows + per - 1) / per;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidValue;
  qk_norm_kernel<BF16, VEC, U><<<(unsigned)blocks, kThreads, table_bytes(a, per, needs_exchange(a)), st>>>(a, L);
  return cudaGetLastError();
}

template <bool BF16, bool VEC>
cudaError_t backward(const NormArgs& a, int64_t rows, int L, cudaStream_t st) {
  constexpr int U = 2;
  const int per = kThreads / L * U;
  const int64_t tiles = (rows + per - 1) / per;
  const int blocks = (int)(tiles < kMaxBackBlocks ? tiles : kMaxBackBlocks);
  const size_t smem = table_bytes(a, per, needs_exchange(a));
  const bool dw = a.side[0].dw || a.side[1].dw;
  if (dw) qk_norm_backward_kernel<BF16, VEC, U, true><<<blocks, kThreads, smem, st>>>(a, L, tiles);
  else qk_norm_backward_kernel<BF16, VEC, U, false><<<blocks, kThreads, smem, st>>>(a, L, tiles);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !dw) return e;
  qk_norm_reduce_kernel<<<dim3((a.D + 31) / 32, 2), 256, 0, st>>>(a.partial, blocks, a.D, a.side[0].dw, a.side[1].dw);
  return cudaGetLastError();
}

}  // namespace

size_t qk_norm_partial_bytes(int64_t, int D) { return (size_t)kMaxBackBlocks * 2 * D * sizeof(float); }

cudaError_t launch_qk_norm(const NormArgs& a, cudaStream_t st) {
  const int64_t rows = (int64_t)a.tokens * (a.side[0].heads + a.side[1].heads);
  if (rows == 0) return cudaSuccess;
  const int L = lanes_of(a.D);
  const bool vec = aligned16(a, false), bf = a.io == PACE_IO_BF16;
  // few rows: one a thread, so that they spread over the SMs
  const bool few = rows * L / kThreads < 148 * 8;
  if (few) {
    if (bf) return vec ? forward<true, true, 1>(a, rows, L, st) : forward<true, false, 1>(a, rows, L, st);
    return vec ? forward<false, true, 1>(a, rows, L, st) : forward<false, false, 1>(a, rows, L, st);
  }
  if (bf) return vec ? forward<true, true, 4>(a, rows, L, st) : forward<true, false, 4>(a, rows, L, st);
  return vec ? forward<false, true, 4>(a, rows, L, st) : forward<false, false, 4>(a, rows, L, st);
}

cudaError_t launch_qk_norm_backward(const NormArgs& a, cudaStream_t st) {
  const int64_t rows = (int64_t)a.tokens * (a.side[0].heads + a.side[1].heads);
  if (rows == 0) {
    for (const NormSide& s : a.side) {
      if (!s.dw) continue;
      const cudaError_t e = cudaMemsetAsync(s.dw, 0, sizeof(float) * a.D, st);
      if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
  }
  const int L = lanes_of(a.D);
  const bool vec = aligned16(a, true), bf = a.io == PACE_IO_BF16;
  if (bf) return vec ? backward<true, true>(a, rows, L, st) : backward<true, false>(a, rows, L, st);
  return vec ? backward<false, true>(a, rows, L, st) : backward<false, false>(a, rows, L, st);
}

}  // namespace pace
