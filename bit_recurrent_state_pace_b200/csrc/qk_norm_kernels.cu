// Queries and keys normalised for each head and turned by their position, and
// the gradients of that, one pass over the data each.
//
//   y = s R(pos) (w * x r),  r = (sum x^2 / n + eps)^(-1/2)
//   u = s R(-pos) dy,  dw = sum u * x^,  h = u * w,  dx = r (h - x^ (x^ . h) / n),  x^ = x r
//
// Memory-bound: 2 (3 in the backward pass) times the tensors' bytes, so what counts beside enough loads in flight is the
// number of instructions a row.  A row (one head of one token) is held by L lanes of a warp, 8 elements (one 16-byte load
// in bf16) each, so a warp's loads are full lines and both sums are shuffles.  A warp takes a token (or, where there are
// few, a part of one) and goes through its queries, then its keys, U rows a lane at a time with the next ones' loads in
// flight (asynchronous copies to shared memory: four batches, where registers held one): a lane keeps its columns, so the
// weights, and the token's cosines and sines, stay in registers.  The angle pos * inv_freq / 2 pi is taken in fp64 and
// only its fraction goes on in fp32: far positions lose nothing.
//
// Blocks with one table of angles for their tokens, rows in a flat list, took 174 instructions a row (this: about 80) and
// waited at a barrier for the table.
//
// 32768 tokens x 40 heads, d = 128, bf16: 128 us, 0.79 of the measured copy; gradients of 16384 x 64 heads with weights:
// 178 us, 0.69 (two rows in for one out, two sums a row, fewer rows in flight).
#include "linattn.cuh"

namespace pace {

namespace {

constexpr unsigned FULL = 0xffffffffu;
constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kSms = 148;                  // B200
constexpr int kBlocks = kSms * 2;          // resident: two an SM
constexpr int kMaxD = 256;
constexpr int kStages = 4;

// lanes that hold a row: the power of two that gives each at most 8 elements
inline int lanes_of(int D) {
  int L = 1;
  while (8 * L < D) L *= 2;
  return L;
}

// One row's eight elements of this lane, as they lie in memory.
template <bool BF16>
struct Raw {
  uint32_t w[BF16 ? 4 : 8];
};

// A lane's eight elements of a row into its own place of shared memory (16 bytes a thread and step of kThreads), by
// asynchronous copies where the addresses allow; zeros where there is no such row.
template <bool BF16, bool VEC>
__device__ __forceinline__ void copy_in(uint4* to, const uint8_t* p, bool in) {
  if (VEC) {
#pragma unroll
    for (int h = 0; h < (BF16 ? 1 : 2); ++h)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(to + h * kThreads)),
                   "l"(p + 16 * h), "r"(in ? 16 : 0)
                   : "memory");
  } else {
    uint32_t w[BF16 ? 4 : 8];
#pragma unroll
    for (int j = 0; j < (BF16 ? 4 : 8); ++j) {
      w[j] = 0u;
      if (!in) continue;
      if (BF16) {
        const uint16_t* q = reinterpret_cast<const uint16_t*>(p) + 2 * j;
        w[j] = (uint32_t)q[0] | ((uint32_t)q[1] << 16);
      } else {
        w[j] = reinterpret_cast<const uint32_t*>(p)[j];
      }
    }
#pragma unroll
    for (int h = 0; h < (BF16 ? 1 : 2); ++h) to[h * kThreads] = make_uint4(w[4 * h], w[4 * h + 1], w[4 * h + 2], w[4 * h + 3]);
  }
}
template <bool BF16>
__device__ __forceinline__ Raw<BF16> copied(const uint4* from) {
  Raw<BF16> r;
#pragma unroll
  for (int h = 0; h < (BF16 ? 1 : 2); ++h) {
    const uint4 v = from[h * kThreads];
    r.w[4 * h] = v.x, r.w[4 * h + 1] = v.y, r.w[4 * h + 2] = v.z, r.w[4 * h + 3] = v.w;
  }
  return r;
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

template <bool BF16>
__device__ __forceinline__ void unpack(const Raw<BF16>& r, float2 (&x)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (BF16) x[j] = make_float2(__uint_as_float(r.w[j] << 16), __uint_as_float(r.w[j] & 0xffff0000u));
    else x[j] = make_float2(__uint_as_float(r.w[BF16 ? 0 : 2 * j]), __uint_as_float(r.w[BF16 ? 0 : 2 * j + 1]));
  }
}

template <bool BF16, bool VEC>
__device__ __forceinline__ void store8(uint8_t* p, const float2 (&x)[4]) {
  if (BF16) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const __nv_bfloat162 h = __float22bfloat162_rn(x[j]);
      w[j] = *reinterpret_cast<const uint32_t*>(&h);
    }
    uint16_t* b = reinterpret_cast<uint16_t*>(p);
    if (VEC) {
      *reinterpret_cast<uint4*>(b) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) b[j] = (uint16_t)(w[j >> 1] >> (16 * (j & 1)));
    }
  } else {
    float* f = reinterpret_cast<float*>(p);
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
#pragma unroll
  for (int off = 16; off; off >>= 1)
    if (off < L) s += __shfl_xor_sync(FULL, s, off);
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
// Place of pair i in the token's table.  A lane reads its 4 or 8 pairs two at a time; a step's reads of all lanes lie
// side by side.
__device__ __forceinline__ int pair_place(Pairs p, int half, int i) {
  if (p == PAIRS_LANE) return (((i & 3) >> 1) * (half >> 2) + (i >> 2)) * 2 + (i & 1);
  if (p == PAIRS_LANES) return (((i & 7) >> 1) * (half >> 3) + (i >> 3)) * 2 + (i & 1);
  return i;
}

// A token's turn as this lane applies it: y[j] -> y[j] * c[j] + (its mates) * s[j], the signs and channels that are not
// turned (c = 1, s = 0) in c and s.
struct Turn {
  float2 c[4], s[4];
  int mate;                // PAIRS_LANES: the lane that holds the mates
};

// cos and sin of every pair's angle at position `pos`, by the whole warp: into its table, from there into `turn`.  sgn: -1
// turns back.  turns: inv_freq / 2 pi.
__device__ __forceinline__ void set_turn(const NormArgs& a, Pairs p, Turn& t, float2* tab, const double* turns, int pos,
                                         float sgn, int c, int lane) {
  const int half = a.rot >> 1;
  __syncwarp();
  for (int i = lane; i < half; i += 32) {
    const double x = (double)pos * turns[i];
    float s, co;
    sincospif(2.f * (float)(x - rint(x)), &s, &co);
    tab[pair_place(p, half, i)] = make_float2(co, sgn * s);
  }
  __syncwarp();
  if (p == PAIRS_ANY) return;
#pragma unroll
  for (int j = 0; j < 4; ++j) t.c[j] = make_float2(1.f, 1.f), t.s[j] = make_float2(0.f, 0.f);
  const float4* t4 = reinterpret_cast<const float4*>(tab);
  if (p == PAIRS_LANE) {
    if (8 * c < a.rot) {
#pragma unroll
      for (int j = 0; j < 4; j += 2) {
        const float4 v = t4[(j >> 1) * (half >> 2) + c];
        t.c[j] = make_float2(v.x, v.x), t.c[j + 1] = make_float2(v.z, v.z);
        t.s[j] = make_float2(-v.y, v.y), t.s[j + 1] = make_float2(-v.w, v.w);
      }
    }
  } else {
    const int hl = half >> 3;
    const bool low = c < hl, on = c < 2 * hl;
    t.mate = (lane - c) + (low ? c + hl : (on ? c - hl : c));
    if (on) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float4 v = t4[j * hl + (low ? c : c - hl)];
        t.c[j] = make_float2(v.x, v.z);
        t.s[j] = low ? make_float2(-v.y, -v.w) : make_float2(v.y, v.w);
      }
    }
  }
}

// xch: shared memory of 8 floats a lane, for pairs that lie anyhow.
__device__ __forceinline__ void turn8(const NormArgs& a, Pairs p, float2 (&y)[4], const Turn& t, const float2* tab, int c, int lane,
                                      float* xch) {
  if (p == PAIRS_LANE) {
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] = __ffma2_rn(make_float2(y[j].y, y[j].x), t.s[j], __fmul2_rn(y[j], t.c[j]));
  } else if (p == PAIRS_LANES) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 o = make_float2(__shfl_sync(FULL, y[j].x, t.mate), __shfl_sync(FULL, y[j].y, t.mate));
      y[j] = __ffma2_rn(o, t.s[j], __fmul2_rn(y[j], t.c[j]));
    }
  } else {
    const int col = 8 * c, half = a.rot >> 1;
    float* mine = xch + (size_t)(lane - c) * 8;           // the row, 8 L floats
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
        const float2 cs = tab[i];
        z[j] = z[j] * cs.x + other * (first ? -cs.y : cs.y);
      }
    }
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] = make_float2(z[2 * j], z[2 * j + 1]);
  }
}

// How the work is cut: units of one token and one of `parts` equal shares of its batches.
struct NormUnits {
  int32_t L;                // lanes a row
  int32_t batches[2];       // of a token's queries, of its keys: U rows a lane each
  int32_t parts, share;     // batches a part
  int64_t units;
};

// BACK 0: the operator; 1: its gradient; 2: with the weights' gradients.  U rows a lane and batch.  LL: lanes a row (0:
// as `n` says).
template <bool BF16, bool VEC, int LL, int U, int BACK>
__global__ void __launch_bounds__(kThreads, 2) qk_norm_kernel(const __grid_constant__ NormArgs a, const __grid_constant__ NormUnits n) {
  constexpr int E = BF16 ? 2 : 4;
  __shared__ double turns[kMaxD / 2];
  __shared__ __align__(16) float2 tabs[kWarps][kMaxD / 2];
  __shared__ float xch[kWarps][256];
  const Pairs pairs = pairs_of(a);
  const int L = LL ? LL : n.L, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = lane & (L - 1), sub = lane / L, RPI = 32 / L;
  for (int i = threadIdx.x; i < a.rot / 2; i += kThreads) turns[i] = (double)a.inv_freq[i] * 0.15915494309189533577;
  __syncthreads();
  const bool held = 8 * c < a.D;
  float2 dw[2][4];
  if (BACK == 2) {
#pragma unroll
    for (int j = 0; j < 4; ++j) dw[0][j] = dw[1][j] = make_float2(0.f, 0.f);
  }
  // a batch: rows RPI (U b + u) + sub of one side of one token
  struct Batch {
    int64_t unit;
    int tok, side, b, left;          // left: batches of the unit from this one on
  };
  auto begin = [&](Batch& x) {       // the first batch of x.unit
    const int64_t tok = n.parts > 1 ? x.unit / n.parts : x.unit;
    int b = (int)(x.unit - tok * n.parts) * n.share;
    x.tok = (int)tok;
    x.left = min(n.share, n.batches[0] + n.batches[1] - b);
    x.side = b >= n.batches[0];
    x.b = x.side ? b - n.batches[0] : b;
  };
  const int64_t warps = (int64_t)gridDim.x * kWarps;
  auto advance = [&](Batch& x) {     // false behind the last
    if (--x.left > 0) {
      if (++x.b == (x.side ? n.batches[1] : n.batches[0])) {
        x.b = 0;
        x.side = 1;
      }
      return true;
    }
    x.unit += warps;
    if (x.unit >= n.units) return false;
    begin(x);
    return x.left > 0;
  };
  // batches on their way: kStages - 1 ahead of the one worked on.  A lane reads what it copied itself, so that nothing
  // but its own copies is waited for.
  extern __shared__ __align__(16) uint4 staged[];
  constexpr int kRow = BF16 ? 1 : 2, kStage = (BACK ? 2 : 1) * U * kRow * kThreads;       // in 16 bytes
  auto fetch = [&](const Batch& x, int stage) {
    uint4* to = staged + stage * kStage + threadIdx.x;
    const NormSide& s = a.side[x.side];
    const uint8_t* px = reinterpret_cast<const uint8_t*>(s.x) + (x.tok * s.x_stride + 8 * c) * E;
    const uint8_t* pg = reinterpret_cast<const uint8_t*>(s.dy) + ((int64_t)x.tok * s.heads * a.D + 8 * c) * E;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int row = RPI * (U * x.b + u) + sub;
      const bool in = row < s.heads && held;
      copy_in<BF16, VEC>(to + u * kRow * kThreads, px + row * a.D * E, in);
      if (BACK) copy_in<BF16, VEC>(to + (U + u) * kRow * kThreads, pg + row * a.D * E, in);
    }
    return pairs != PAIRS_NONE ? a.pos[x.tok] : 0;
  };
  Batch cur, ahead;
  cur.unit = (int64_t)blockIdx.x * kWarps + warp;
  bool more = cur.unit < n.units;
  if (more) {
    begin(cur);
    more = cur.left > 0;
  }
  ahead = cur;
  bool to_fetch = more;
  int pos[kStages - 1];              // positions of the batches on their way
#pragma unroll
  for (int k = 0; k < kStages - 1; ++k) {
    pos[k] = 0;
    if (to_fetch) {
      pos[k] = fetch(ahead, k);
      to_fetch = advance(ahead);
    }
    copies_commit();
  }
  int stage = 0;
  Turn turn;
  int turned = -1, weighted = -1;    // the token of `turn`, the side of `w`
  float2 w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) w[j] = make_float2(1.f, 1.f);
  while (more) {
    const Batch now = cur;
    copies_wait<kStages - 2>();
    const int at = pos[0];
#pragma unroll
    for (int k = 0; k + 2 < kStages; ++k) pos[k] = pos[k + 1];
    if (to_fetch) {                  // into the stage worked on last
      pos[kStages - 2] = fetch(ahead, stage == 0 ? kStages - 1 : stage - 1);
      to_fetch = advance(ahead);
    }
    copies_commit();
    const uint4* from = staged + stage * kStage + threadIdx.x;
    stage = stage + 1 == kStages ? 0 : stage + 1;
    more = advance(cur);
    const NormSide& s = a.side[now.side];
    if (pairs != PAIRS_NONE && now.tok != turned) {
      set_turn(a, pairs, turn, tabs[warp], turns, at, BACK ? -1.f : 1.f, c, lane);
      turned = now.tok;
    }
    if (now.side != weighted) {
      weighted = now.side;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        w[j] = s.w && held ? make_float2(s.w[8 * c + 2 * j], s.w[8 * c + 2 * j + 1]) : make_float2(1.f, 1.f);
    }
    uint8_t* py = reinterpret_cast<uint8_t*>(s.y) + (now.tok * s.y_stride + 8 * c) * E;
    const float scale = s.scale;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int row = RPI * (U * now.b + u) + sub;
      const bool in = row < s.heads && held;
      float2 x[4];
      unpack<BF16>(copied<BF16>(from + u * kRow * kThreads), x);
      const float rr = rsqrtf(fmaf(row_sum(dot8(x, x), L), a.inv_n, a.eps));
      if (!BACK) {
        const float2 f = make_float2(rr * scale, rr * scale);
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = __fmul2_rn(__fmul2_rn(x[j], f), w[j]);
        if (pairs != PAIRS_NONE) turn8(a, pairs, x, turn, tabs[warp], c, lane, xch[warp]);
        if (in) store8<BF16, VEC>(py + row * a.D * E, x);
      } else {
        float2 g[4];
        unpack<BF16>(copied<BF16>(from + (U + u) * kRow * kThreads), g);
        if (pairs != PAIRS_NONE) turn8(a, pairs, g, turn, tabs[warp], c, lane, xch[warp]);
        const float2 r2 = make_float2(rr, rr), sc = make_float2(scale, scale);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          x[j] = __fmul2_rn(x[j], r2);                          // x^
          g[j] = __fmul2_rn(g[j], sc);                          // u
        }
        if (BACK == 2) {                                        // rows that are not there are zeros
          if (now.side) {
#pragma unroll
            for (int j = 0; j < 4; ++j) dw[1][j] = __ffma2_rn(x[j], g[j], dw[1][j]);
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) dw[0][j] = __ffma2_rn(x[j], g[j], dw[0][j]);
          }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) g[j] = __fmul2_rn(g[j], w[j]);      // h
        const float d = row_sum(dot8(x, g), L) * -a.inv_n;
        const float2 d2 = make_float2(d, d);
#pragma unroll
        for (int j = 0; j < 4; ++j) g[j] = __fmul2_rn(r2, __ffma2_rn(x[j], d2, g[j]));
        if (in) store8<BF16, VEC>(py + row * a.D * E, g);
      }
    }
  }
  if (BACK == 2) {
    // this block's sums over its rows, in the order of the warps and of the rows a warp holds
    __shared__ float2 red[kThreads * 4];
    for (int side = 0; side < 2; ++side) {
      __syncthreads();
#pragma unroll
      for (int j = 0; j < 4; ++j) red[threadIdx.x * 4 + j] = dw[side][j];
      __syncthreads();
      for (int col = threadIdx.x; col < a.D; col += kThreads) {
        float sum = 0.f;
        for (int k = 0; k < kWarps * RPI; ++k) sum += reinterpret_cast<const float*>(red)[k * L * 8 + col];
        a.partial[((size_t)blockIdx.x * 2 + side) * a.D + col] = sum;
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

template <bool BF16, bool VEC, int LL, int BACK>
cudaError_t launch_l(const NormArgs& a, cudaStream_t st, int* blocks_out) {
  constexpr int U = BACK ? (BF16 ? 2 : 1) : (BF16 ? 4 : 2);
  NormUnits n;
  n.L = lanes_of(a.D);
  const int per = 32 / n.L * U;
  n.batches[0] = (a.side[0].heads + per - 1) / per;
  n.batches[1] = (a.side[1].heads + per - 1) / per;
  const int all = n.batches[0] + n.batches[1];
  // a token a warp; in parts where that leaves warps without work
  const int64_t warps = (int64_t)kBlocks * kWarps;
  int64_t parts = a.tokens >= warps ? 1 : warps / a.tokens;
  if (parts > all) parts = all;
  n.share = (int32_t)((all + parts - 1) / parts);
  n.parts = (all + n.share - 1) / n.share;
  n.units = (int64_t)a.tokens * n.parts;
  const int64_t need = (n.units + kWarps - 1) / kWarps;
  const int blocks = (int)(need < kBlocks ? need : kBlocks);
  if (blocks_out) *blocks_out = blocks;
  const int smem = kStages * (BACK ? 2 : 1) * U * (BF16 ? 1 : 2) * kThreads * 16;
  static bool allowed[64];
  const cudaError_t e = allow_shared(qk_norm_kernel<BF16, VEC, LL, U, BACK>, smem, allowed);
  if (e != cudaSuccess) return e;
  qk_norm_kernel<BF16, VEC, LL, U, BACK><<<blocks, kThreads, smem, st>>>(a, n);
  return cudaGetLastError();
}

template <bool BF16, bool VEC, int BACK>
cudaError_t launch_t(const NormArgs& a, cudaStream_t st, int* blocks) {
  if constexpr (VEC) {
    switch (lanes_of(a.D)) {
      case 8: return launch_l<BF16, VEC, 8, BACK>(a, st, blocks);
      case 16: return launch_l<BF16, VEC, 16, BACK>(a, st, blocks);
      case 32: return launch_l<BF16, VEC, 32, BACK>(a, st, blocks);
    }
  }
  return launch_l<BF16, VEC, 0, BACK>(a, st, blocks);
}

template <int BACK>
cudaError_t launch(const NormArgs& a, cudaStream_t st, int* blocks) {
  const bool vec = aligned16(a, BACK != 0);
  if (a.io == PACE_IO_BF16)
    return vec ? launch_t<true, true, BACK>(a, st, blocks) : launch_t<true, false, BACK>(a, st, blocks);
  return vec ? launch_t<false, true, BACK>(a, st, blocks) : launch_t<false, false, BACK>(a, st, blocks);
}

}  // namespace

size_t qk_norm_partial_bytes(int D) { return (size_t)kBlocks * 2 * D * sizeof(float); }

cudaError_t launch_qk_norm(const NormArgs& a, cudaStream_t st) {
  const int64_t rows = (int64_t)a.tokens * (a.side[0].heads + a.side[1].heads);
  return rows == 0 ? cudaSuccess : launch<0>(a, st, nullptr);
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
  if (!a.side[0].dw && !a.side[1].dw) return launch<1>(a, st, nullptr);
  int blocks = 0;
  const cudaError_t e = launch<2>(a, st, &blocks);
  if (e != cudaSuccess) return e;
  qk_norm_reduce_kernel<<<dim3((a.D + 31) / 32, 2), 256, 0, st>>>(a.partial, blocks, a.D, a.side[0].dw, a.side[1].dw);
  return cudaGetLastError();
}

}  // namespace pace
