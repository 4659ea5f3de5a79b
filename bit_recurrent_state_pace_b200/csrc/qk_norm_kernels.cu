// Queries and keys normalised for each head and turned by their position, and
// the gradients of that, one pass over the data each.
//
//   y = s R(pos) (w * x r),  r = (sum x^2 / n + eps)^(-1/2)
//   u = s R(-pos) dy,  dw = sum u * x^,  h = u * w,  dx = r (h - x^ (x^ . h) / n),  x^ = x r
//
// Memory-bound: 2 (3 in the backward pass) times the tensors' bytes.  A row (one head of one token) is held by L lanes
// of one warp, 8 elements (one 16-byte load in bf16) each, so a warp's loads are full lines and both sums are shuffles.
// A block walks over tiles -- some tokens with all their heads, or a part of one token's -- with the next tile's loads
// in flight and its tokens' angles being computed while it works on one: a thread keeps its columns, so the weights stay
// in registers.  The angle pos * inv_freq / 2 pi is taken in fp64 and only its fraction goes on in fp32: far positions
// lose nothing, and each token's angles are computed once for all its heads.
#include "linattn.cuh"

namespace pace {

namespace {

constexpr unsigned FULL = 0xffffffffu;
constexpr int kThreads = 256;
constexpr int kSms = 148;                  // B200
constexpr int kBlocks = kSms * 2;          // resident: two of 256 threads an SM

// lanes that hold a row: the power of two that gives each at most 8 elements
inline int lanes_of(int D) {
  int L = 1;
  while (8 * L < D) L *= 2;
  return L;
}

// How the rows are cut into tiles.
struct NormTiles {
  int32_t L, R;             // lanes a row, rows a token
  uint32_t magic;           // ceil(2^32 / R): x / R = umulhi(x, magic) for x < 2^16 (R > 1)
  int32_t tokens, passes;   // tokens a tile; tiles that share them
  int64_t tiles;
};

// One row's eight elements of this lane, as they lie in memory.
template <bool BF16>
struct Raw {
  uint32_t w[BF16 ? 4 : 8];
};

template <bool BF16, bool VEC>
__device__ __forceinline__ Raw<BF16> load_raw(const void* p, size_t at) {
  Raw<BF16> r;
  if (VEC) {
    const uint4* q = reinterpret_cast<const uint4*>(reinterpret_cast<const uint8_t*>(p) + at * (BF16 ? 2 : 4));
    const uint4 a = q[0];
    r.w[0] = a.x, r.w[1] = a.y, r.w[2] = a.z, r.w[3] = a.w;
    if (!BF16) {
      const uint4 b = q[1];
      r.w[BF16 ? 0 : 4] = b.x, r.w[BF16 ? 1 : 5] = b.y, r.w[BF16 ? 2 : 6] = b.z, r.w[BF16 ? 3 : 7] = b.w;
    }
  } else if (BF16) {
    const uint16_t* q = reinterpret_cast<const uint16_t*>(p) + at;
#pragma unroll
    for (int j = 0; j < 4; ++j) r.w[j] = (uint32_t)q[2 * j] | ((uint32_t)q[2 * j + 1] << 16);
  } else {
    const uint32_t* q = reinterpret_cast<const uint32_t*>(p) + at;
#pragma unroll
    for (int j = 0; j < (BF16 ? 4 : 8); ++j) r.w[j] = q[j];
  }
  return r;
}

template <bool BF16>
__device__ __forceinline__ Raw<BF16> zero_raw() {
  Raw<BF16> r;
#pragma unroll
  for (int j = 0; j < (BF16 ? 4 : 8); ++j) r.w[j] = 0u;
  return r;
}

template <bool BF16>
__device__ __forceinline__ void unpack(const Raw<BF16>& r, float2 (&x)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (BF16) x[j] = make_float2(__uint_as_float(r.w[j] << 16), __uint_as_float(r.w[j] & 0xffff0000u));
    else x[j] = make_float2(__uint_as_float(r.w[BF16 ? 0 : 2 * j]), __uint_as_float(r.w[BF16 ? 0 : 2 * j + 1]));
  }
}

template <bool BF16, bool VEC>
__device__ __forceinline__ void store8(void* p, size_t at, const float2 (&x)[4]) {
  if (BF16) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const __nv_bfloat162 h = __float22bfloat162_rn(x[j]);
      w[j] = *reinterpret_cast<const uint32_t*>(&h);
    }
    uint16_t* b = reinterpret_cast<uint16_t*>(p) + at;
    if (VEC) {
      *reinterpret_cast<uint4*>(b) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) b[j] = (uint16_t)(w[j >> 1] >> (16 * (j & 1)));
    }
  } else {
    float* f = reinterpret_cast<float*>(p) + at;
    if (VEC) {
      *reinterpret_cast<float4*>(f) = make_float4(x[0].x, x[0].y, x[1].x, x[1].y);
      *reinterpret_cast<float4*>(f + 4) = make_float4(x[2].x, x[2].y, x[3].x, x[3].y);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) f[2 * j] = x[j].x, f[2 * j + 1] = x[j].y;
    }
  }
}

__device__ __forceinline__ float row_sum(float s, int L) {
  for (int off = L >> 1; off; off >>= 1) s += __shfl_xor_sync(FULL, s, off);
  return s;
}
__device__ __forceinline__ float dot8(const float2 (&a)[4], const float2 (&b)[4]) {
  float2 s = __fmul2_rn(a[0], b[0]);
#pragma unroll
  for (int j = 1; j < 4; ++j) s = __ffma2_rn(a[j], b[j], s);
  return s.x + s.y;
}

// How the rotation's pairs lie: in one lane (interleaved), half a row of whole lanes apart, or otherwise apart.
enum Pairs { PAIRS_NONE, PAIRS_LANE, PAIRS_LANES, PAIRS_ANY };
__host__ __device__ inline Pairs pairs_of(const NormArgs& a) {
  if (!a.rot) return PAIRS_NONE;
  if (a.interleaved) return a.rot % 8 == 0 ? PAIRS_LANE : PAIRS_ANY;
  return a.rot % 16 == 0 ? PAIRS_LANES : PAIRS_ANY;
}
// Place of pair i in a token's table.  A lane reads its 4 or 8 pairs two at a time; a step's reads of all lanes lie side
// by side.
__device__ __forceinline__ int pair_place(Pairs p, int half, int i) {
  if (p == PAIRS_LANE) return (((i & 3) >> 1) * (half >> 2) + (i >> 2)) * 2 + (i & 1);
  if (p == PAIRS_LANES) return (((i & 7) >> 1) * (half >> 3) + (i >> 3)) * 2 + (i & 1);
  return i;
}

// cos and sin of every pair's angle for `ntok` tokens from tok0 on: tab[token][place]
__device__ __forceinline__ void angle_table(const NormArgs& a, Pairs p, float2* tab, int64_t tok0, int ntok) {
  const int half = a.rot >> 1;
  for (int e = threadIdx.x; e < ntok * half; e += kThreads) {
    const int lt = e / half, i = e - lt * half;
    float2 cs = make_float2(1.f, 0.f);               // behind the last token: rows of zeros, turned by nothing
    if (tok0 + lt < a.tokens) {
      const double turns = (double)a.pos[tok0 + lt] * (double)a.inv_freq[i] * 0.15915494309189533577;
      sincospif(2.f * (float)(turns - rint(turns)), &cs.y, &cs.x);
    }
    tab[lt * half + pair_place(p, half, i)] = cs;
  }
}

// Turns the row held by the lanes of this group by `sgn` times its angles.  c: the lane's place in its row; xch: shared
// memory of 8 floats a thread, for pairs that lie anyhow.
__device__ __forceinline__ void turn8(const NormArgs& a, Pairs p, float2 (&y)[4], const float2* t, float sgn, int c, float* xch) {
  const int col = 8 * c, half = a.rot >> 1;
  if (p == PAIRS_LANE) {
    if (col < a.rot) {
      const float4* t4 = reinterpret_cast<const float4*>(t) + c;
      const int step = half >> 2;
#pragma unroll
      for (int j = 0; j < 4; j += 2) {
        const float4 cs = t4[(j >> 1) * step];
        const float s0 = sgn * cs.y, s1 = sgn * cs.w;
        y[j] = make_float2(y[j].x * cs.x - y[j].y * s0, y[j].y * cs.x + y[j].x * s0);
        y[j + 1] = make_float2(y[j + 1].x * cs.z - y[j + 1].y * s1, y[j + 1].y * cs.z + y[j + 1].x * s1);
      }
    }
  } else if (p == PAIRS_LANES) {
    const int lane = threadIdx.x & 31, hl = half >> 3, base = lane - c;
    const bool low = c < hl, on = c < 2 * hl;
    const int mate = low ? c + hl : (on ? c - hl : c);
    const float flip = low ? -sgn : sgn;
    const float4* t4 = reinterpret_cast<const float4*>(t) + (low ? c : (on ? c - hl : 0));
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float ox = __shfl_sync(FULL, y[j].x, base + mate), oy = __shfl_sync(FULL, y[j].y, base + mate);
      const float4 cs = t4[j * hl];
      if (on) y[j] = make_float2(y[j].x * cs.x + ox * (flip * cs.y), y[j].y * cs.z + oy * (flip * cs.w));
    }
  } else {
    float* mine = xch + (size_t)(threadIdx.x - c) * 8;    // the row, 8 L floats
#pragma unroll
    for (int j = 0; j < 4; ++j) mine[col + 2 * j] = y[j].x, mine[col + 2 * j + 1] = y[j].y;
    __syncwarp();
    float z[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int x = col + j;
      z[j] = mine[col + j];
      if (x < a.rot) {
        const int i = a.interleaved ? x >> 1 : (x < half ? x : x - half);
        const bool first = a.interleaved ? !(x & 1) : x < half;
        const float other = mine[a.interleaved ? x ^ 1 : (first ? x + half : x - half)];
        const float2 cs = t[i];
        z[j] = z[j] * cs.x + other * ((first ? -sgn : sgn) * cs.y);
      }
    }
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] = make_float2(z[2 * j], z[2 * j + 1]);
  }
}

// Where row x of a tile lies.
struct Row {
  bool in;                  // there is such a row and this lane holds a part of it
  int side, head, ltok;
  int64_t tok;
};
__device__ __forceinline__ Row locate(const NormArgs& a, const NormTiles& n, int64_t tok0, int x, int c) {
  Row r;
  r.ltok = n.R > 1 ? (int)__umulhi((uint32_t)x, n.magic) : x;
  const int row = x - r.ltok * n.R;
  r.side = row >= a.side[0].heads;
  r.head = r.side ? row - a.side[0].heads : row;
  r.tok = tok0 + r.ltok;
  r.in = r.ltok < n.tokens && r.tok < a.tokens && 8 * c < a.D;
  if (r.ltok >= n.tokens) r.ltok = n.tokens - 1;
  return r;
}

// BACK 0: the operator; 1: its gradient; 2: with the weights' gradients.  U rows a thread and tile.
template <bool BF16, bool VEC, int U, int BACK>
__global__ void __launch_bounds__(kThreads, 2) qk_norm_kernel(const __grid_constant__ NormArgs a, const __grid_constant__ NormTiles n) {
  extern __shared__ __align__(16) float2 shared[];
  const Pairs pairs = pairs_of(a);
  const int L = n.L, c = threadIdx.x & (L - 1), slots = kThreads / L, slot = threadIdx.x / L;
  const int tab_size = n.tokens * (a.rot >> 1) + ((n.tokens * (a.rot >> 1)) & 1);
  float2* tab[2] = {shared, shared + tab_size};
  float* xch = reinterpret_cast<float*>(shared + 2 * tab_size);
  float2 w[2][4];
#pragma unroll
  for (int s = 0; s < 2; ++s)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      w[s][j] = make_float2(1.f, 1.f);
      if (a.side[s].w && 8 * c < a.D) w[s][j] = make_float2(a.side[s].w[8 * c + 2 * j], a.side[s].w[8 * c + 2 * j + 1]);
    }
  float2 dw[2][4];
  if (BACK == 2) {
#pragma unroll
    for (int j = 0; j < 4; ++j) dw[0][j] = dw[1][j] = make_float2(0.f, 0.f);
  }
  auto first_token = [&](int64_t tile, int* x0) {
    const int64_t group = n.passes > 1 ? tile / n.passes : tile;
    *x0 = (int)(tile - group * n.passes) * (slots * U) + slot;
    return group * n.tokens;
  };
  Raw<BF16> nx[U], ng[BACK ? U : 1];
  auto fetch = [&](int64_t tile) {
    int x0;
    const int64_t tok0 = first_token(tile, &x0);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const Row r = locate(a, n, tok0, x0 + u * slots, c);
      const NormSide& s = a.side[r.side];
      nx[u] = zero_raw<BF16>();
      if (BACK) ng[BACK ? u : 0] = zero_raw<BF16>();
      if (r.in) {
        nx[u] = load_raw<BF16, VEC>(s.x, (size_t)(r.tok * s.x_stride) + (size_t)r.head * a.D + 8 * c);
        if (BACK) ng[BACK ? u : 0] = load_raw<BF16, VEC>(s.dy, (size_t)(r.tok * s.heads + r.head) * a.D + 8 * c);
      }
    }
    return tok0;
  };
  int64_t tile = blockIdx.x;
  int64_t tok0 = fetch(tile);
  int cur = 0;
  if (pairs != PAIRS_NONE) {
    angle_table(a, pairs, tab[0], tok0, n.tokens);
    __syncthreads();
  }
  for (; tile < n.tiles; tile += gridDim.x, cur ^= 1) {
    Raw<BF16> rx[U], rg[BACK ? U : 1];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      rx[u] = nx[u];
      if (BACK) rg[BACK ? u : 0] = ng[BACK ? u : 0];
    }
    int x0;
    tok0 = first_token(tile, &x0);
    const bool more = tile + gridDim.x < n.tiles;
    if (more) {
      const int64_t next = fetch(tile + gridDim.x);
      if (pairs != PAIRS_NONE) angle_table(a, pairs, tab[cur ^ 1], next, n.tokens);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const Row r = locate(a, n, tok0, x0 + u * slots, c);
      const NormSide& s = a.side[r.side];
      const float2* t = tab[cur] + r.ltok * (a.rot >> 1);
      const size_t at = (size_t)(r.tok * s.y_stride) + (size_t)r.head * a.D + 8 * c;
      float2 x[4], ww[4];
      unpack<BF16>(rx[u], x);
#pragma unroll
      for (int j = 0; j < 4; ++j) ww[j] = r.side ? w[1][j] : w[0][j];
      const float rr = rsqrtf(fmaf(row_sum(dot8(x, x), L), a.inv_n, a.eps));
      if (!BACK) {
        const float2 f = make_float2(rr * s.scale, rr * s.scale);
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = __fmul2_rn(__fmul2_rn(x[j], f), ww[j]);
        if (pairs != PAIRS_NONE) turn8(a, pairs, x, t, 1.f, c, xch);
        if (r.in) store8<BF16, VEC>(s.y, at, x);
      } else {
        float2 g[4];
        unpack<BF16>(rg[BACK ? u : 0], g);
        if (pairs != PAIRS_NONE) turn8(a, pairs, g, t, -1.f, c, xch);
        const float2 r2 = make_float2(rr, rr), sc = make_float2(s.scale, s.scale);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          x[j] = __fmul2_rn(x[j], r2);                          // x^
          g[j] = __fmul2_rn(g[j], sc);                          // u
          if (BACK == 2) {
            const float2 z = make_float2(0.f, 0.f);
            const float2 keep = r.in ? x[j] : z;
            dw[0][j] = __ffma2_rn(r.side ? z : keep, g[j], dw[0][j]);
            dw[1][j] = __ffma2_rn(r.side ? keep : z, g[j], dw[1][j]);
          }
          g[j] = __fmul2_rn(g[j], ww[j]);                       // h
        }
        const float d = row_sum(dot8(x, g), L) * -a.inv_n;
        const float2 d2 = make_float2(d, d);
#pragma unroll
        for (int j = 0; j < 4; ++j) g[j] = __fmul2_rn(r2, __ffma2_rn(x[j], d2, g[j]));
        if (r.in) store8<BF16, VEC>(s.y, at, g);
      }
    }
    if (pairs != PAIRS_NONE && more) __syncthreads();           // the next table is whole, this one is done with
  }
  if (BACK == 2) {
    // this block's sums over its row slots, in the order of the slots
    __shared__ float2 red[kThreads * 4];
    for (int side = 0; side < 2; ++side) {
      __syncthreads();
#pragma unroll
      for (int j = 0; j < 4; ++j) red[threadIdx.x * 4 + j] = dw[side][j];
      __syncthreads();
      for (int col = threadIdx.x; col < a.D; col += kThreads) {
        float s = 0.f;
        for (int k = 0; k < slots; ++k) s += reinterpret_cast<const float*>(red)[k * L * 8 + col];
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

// Tiles of `per` rows: as many whole tokens as fit, or a part of one.
NormTiles tiles_of(const NormArgs& a, int per) {
  NormTiles n;
  n.L = lanes_of(a.D);
  n.R = a.side[0].heads + a.side[1].heads;
  n.magic = n.R > 1 ? (uint32_t)((((uint64_t)1 << 32) + n.R - 1) / n.R) : 0;
  n.tokens = per >= n.R ? per / n.R : 1;
  n.passes = per >= n.R ? 1 : (n.R + per - 1) / per;
  n.tiles = ((int64_t)a.tokens + n.tokens - 1) / n.tokens * n.passes;
  return n;
}

size_t shared_bytes(const NormArgs& a, const NormTiles& n) {
  const size_t t = (size_t)n.tokens * (a.rot / 2);
  return 2 * (t + (t & 1)) * sizeof(float2) + (pairs_of(a) == PAIRS_ANY ? kThreads * 8 * sizeof(float) : 0);
}

template <bool BF16, bool VEC, int U, int BACK>
cudaError_t launch_u(const NormArgs& a, cudaStream_t st, int* blocks_out) {
  const NormTiles n = tiles_of(a, kThreads / lanes_of(a.D) * U);
  const size_t smem = shared_bytes(a, n);
  const int64_t most = kBlocks;
  const int blocks = (int)(n.tiles < most ? n.tiles : most);
  if (blocks_out) *blocks_out = blocks;
  if (smem > 48 * 1024) {          // small heads in fp32 rows of one token each: tables of 32 KB and more
    const cudaError_t e = cudaFuncSetAttribute(qk_norm_kernel<BF16, VEC, U, BACK>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  qk_norm_kernel<BF16, VEC, U, BACK><<<blocks, kThreads, smem, st>>>(a, n);
  return cudaGetLastError();
}

// U rows a thread where that still gives every SM some blocks, else one.
template <bool BF16, bool VEC, int BACK>
cudaError_t launch_t(const NormArgs& a, int64_t rows, cudaStream_t st, int* blocks) {
  constexpr int U = BACK ? (BF16 ? 2 : 1) : (BF16 ? 4 : 2);
  if (U == 1 || rows * lanes_of(a.D) / (kThreads * U) < 2 * kSms) return launch_u<BF16, VEC, 1, BACK>(a, st, blocks);
  return launch_u<BF16, VEC, U, BACK>(a, st, blocks);
}

template <int BACK>
cudaError_t launch(const NormArgs& a, int64_t rows, cudaStream_t st, int* blocks) {
  const bool vec = aligned16(a, BACK != 0);
  if (a.io == PACE_IO_BF16)
    return vec ? launch_t<true, true, BACK>(a, rows, st, blocks) : launch_t<true, false, BACK>(a, rows, st, blocks);
  return vec ? launch_t<false, true, BACK>(a, rows, st, blocks) : launch_t<false, false, BACK>(a, rows, st, blocks);
}

}  // namespace

size_t qk_norm_partial_bytes(int64_t, int D) { return (size_t)kBlocks * 2 * D * sizeof(float); }

cudaError_t launch_qk_norm(const NormArgs& a, cudaStream_t st) {
  const int64_t rows = (int64_t)a.tokens * (a.side[0].heads + a.side[1].heads);
  return rows == 0 ? cudaSuccess : launch<0>(a, rows, st, nullptr);
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
  if (!a.side[0].dw && !a.side[1].dw) return launch<1>(a, rows, st, nullptr);
  int blocks = 0;
  const cudaError_t e = launch<2>(a, rows, st, &blocks);
  if (e != cudaSuccess) return e;
  qk_norm_reduce_kernel<<<dim3((a.D + 31) / 32, 2), 256, 0, st>>>(a.partial, blocks, a.D, a.side[0].dw, a.side[1].dw);
  return cudaGetLastError();
}

}  // namespace pace
