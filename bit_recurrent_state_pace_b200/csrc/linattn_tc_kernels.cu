// Linear attention with a fixed decay for each head in chunked form on the
// fifth-generation tensor cores (tcgen05, TMEM), bf16, d = 64 or 128.
//
// A walk (linattn.cuh) takes a sequence in chunks of C = 64 tokens.  With A =
// exp(g), chunk rows i, j = 0..r-1 and S the state before the chunk,
//   forwards:   out_i = sum_{j <= i} A^(i-j) (query_i . key_j) value_j + A^(i+1) S query_i
//               S <- A^r S + sum_j A^(r-1-j) value_j key_j^T
//   backwards:  out_i = sum_{j >= i} A^(j-i) (query_i . key_j) value_j + A^(r-1-i) S query_i
//               S <- A^r S + sum_j A^(j+1) value_j key_j^T
// which is four products a chunk, transposed so that the value channels lie
// on the 128 TMEM lanes:
//   SC  [i, j]  = Q K^T                        (lanes i)
//   OI  [e, i]  = bf16(S) Q^T                  A in TMEM
//   OP  [e, i]  = V^T P,  P = bf16(mask A^|i-j| SC)   A in TMEM, P in shared memory
//   U   [e, c]  = (V A^..)^T K                 A in TMEM in three bf16 parts, K read MN-major
// out^T = OP + A^.. OI, and S stays in registers in fp32.
//
// Roundings: P and the copy of S that multiplies the query are bf16, once for
// each term (2^-9 of it, the size of the output's own rounding).  The value
// times its decay is split into three bf16 parts (24 bits), so that the
// states, which are fp32 outputs and run over the whole sequence, are summed
// from exact products of 24 bits; two parts left 2.7e-6 of the state.
//
// One persistent CTA of 16 warps per SM:
//  * warp 0: loads the chunks' tiles by TMA, three chunks ahead;
//  * warp 1: issues the products.  SC of the next chunk goes before OP and U of
//    this one, so that P is made while U runs;
//  * warps 4-7: P from SC, then the value's raw and decayed parts into TMEM;
//  * warps 8-15: the state (half of the key channels each four) and the output
//    (half of the tokens each four).
// Traffic is each input once and each output once; 128 d + 10 d^2 / ... products
// a token keep the tensor pipe about half busy, so memory bounds it.
//
// Sequences too few to fill the SMs are cut into stretches: the same kernel
// without outputs gives each stretch's own contribution to the state, a small
// one chains them, and the stretches then run from their true states.
#include <type_traits>

#include "linattn_tc.cuh"

namespace pace {

namespace {

constexpr unsigned FULL = 0xffffffffu;
constexpr int C = 64;                 // tokens a chunk
constexpr int NST = 3;                // staged chunks
constexpr int kTcThreads = 512;
constexpr int kSms = 148;             // B200

// TMEM columns
constexpr uint32_t T_SC = 0, T_OI = 64, T_OP = 128, T_U = 192, T_S = 320, T_VR = 384, T_V = 416;

struct LinMaps { CUtensorMap m[4]; };

struct LinTc {
  LinArgs a;
  int32_t map_q[kLinMaxWalks], map_k[kLinMaxWalks], map_v[kLinMaxWalks];
  LinSplit split;
  float* ws;               // [walks][N][H][stretches][D][D]: each stretch's state
  int32_t items;
};

template <int D>
struct alignas(1024) LinSmem {
  static constexpr int TILE = C * D * 2;                 // D / 64 blocks of 64 rows of 128 bytes
  uint8_t stage[NST][3][TILE];                           // query | key | value
  uint8_t p[C * 128];                                    // P[i][j], 128-byte swizzle
  uint16_t o[2][2][C / 2][D];                            // [buffer][half of the tokens]
  float pw1[2][2 * C];                                   // warps 4-7: A^n at [n], two items alternate
  float pw2[2][2][C + 8];                                // warps 8-11, 12-15: A^n; [C + 4 ..] hi, lo of A^C and A^tail
  uint64_t full[NST], empty[NST];
  uint64_t sc_full, p_full, v_full, s_full, u_full, op_full, o_empty, drain;
  uint32_t taddr;
  int abort;
};

__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, uint32_t* flags, int* abort) {
  if (mbar_try_wait(bar, parity)) return true;
  if (tc::mbar_wait_sleep(bar, parity, flags)) return true;
  *reinterpret_cast<volatile int*>(abort) = 1;
  return false;
}
__device__ __forceinline__ bool aborted(const int* abort) { return *reinterpret_cast<const volatile int*>(abort) != 0; }

// Work item: one walk of one stretch of one sequence and head.
struct Item {
  int w, n, h, seg, begin, len, c0, c1;     // rows [begin, begin + len) of the sequence, chunks [c0, c1)
  int nseg;                                 // stretches of this sequence
  bool on;                                  // there is something to do
  __device__ __forceinline__ int chunks() const { return c1 - c0; }
  __device__ __forceinline__ int rows(int c) const { return min(C, len - c * C); }
};

template <bool STATE_ONLY>
__device__ __forceinline__ Item item_of(const LinTc& t, int x) {
  Item it;
  it.w = x % t.a.walks;
  x /= t.a.walks;
  it.seg = x % t.split.stretches;
  x /= t.split.stretches;
  it.h = x % t.a.H;
  it.n = x / t.a.H;
  int end;
  seq_rows(t.a, it.n, &it.begin, &end);
  it.len = end - it.begin;
  const int nc = (it.len + C - 1) / C;
  int ns = (nc + t.split.per - 1) / t.split.per;
  it.nseg = ns < 1 ? 1 : (ns > t.split.stretches ? t.split.stretches : ns);
  it.on = it.seg < it.nseg;
  // the stretch that a walk ends with hands its state to no other
  if (STATE_ONLY) it.on = it.on && it.seg != (t.a.walk[it.w].back ? 0 : it.nseg - 1);
  it.c0 = it.seg * t.split.per;
  it.c1 = it.seg == it.nseg - 1 ? nc : it.c0 + t.split.per;
  if (!it.on) it.c0 = it.c1 = 0;
  return it;
}
__device__ __forceinline__ float* stretch_state(const LinTc& t, const Item& it) {
  return t.ws + (((size_t)it.w * t.a.N + it.n) * t.a.H + it.h) * t.split.stretches * t.a.D * t.a.D +
         (size_t)it.seg * t.a.D * t.a.D;
}
// k-th chunk of an item in its walk's order
__device__ __forceinline__ int chunk_at(const Item& it, bool back, int k) { return back ? it.c1 - 1 - k : it.c0 + k; }

// ---- loads ---------------------------------------------------------------------
template <int D, bool STATE_ONLY>
__device__ void load_role(const LinTc& t, const LinMaps& maps, LinSmem<D>& sm) {
  using SM = LinSmem<D>;
  int k = 0;
  bool ok = true;
  for (int x = blockIdx.x; x < t.items && ok; x += gridDim.x) {
    const Item it = item_of<STATE_ONLY>(t, x);
    const bool back = t.a.walk[it.w].back;
    const CUtensorMap* mp[3] = {&maps.m[t.map_q[it.w]], &maps.m[t.map_k[it.w]], &maps.m[t.map_v[it.w]]};
    for (int c = 0; c < it.chunks(); ++c, ++k) {
      const int s = k % NST, r = k / NST;
      if (r > 0 && !wait_bar(&sm.empty[s], (uint32_t)((r - 1) & 1), t.a.flags, &sm.abort)) { ok = false; break; }
      if (aborted(&sm.abort)) { ok = false; break; }
      const int row = it.begin + chunk_at(it, back, c) * C;
      constexpr int first = STATE_ONLY ? 1 : 0;
      mbar_arrive_expect_tx(&sm.full[s], (3 - first) * SM::TILE);
#pragma unroll
      for (int m = first; m < 3; ++m)
#pragma unroll
        for (int b = 0; b < D / 64; ++b)
          ltc::tensor_load_2d(smem_addr(&sm.stage[s][m][b * C * 128]), mp[m], it.h * D + 64 * b, row, &sm.full[s]);
    }
  }
  if (!ok) {      // gave up: nothing of ours may land after the block has left
    for (int j = max(0, k - NST); j < k; ++j)
      tc::mbar_wait_sleep(&sm.full[j % NST], (uint32_t)((j / NST) & 1), t.a.flags);
  }
}

// ---- products --------------------------------------------------------------------
template <int D, bool STATE_ONLY>
__device__ void mma_role(const LinTc& t, LinSmem<D>& sm, uint32_t tm) {
  using SM = LinSmem<D>;
  constexpr uint32_t id_n64 = ltc::idesc_bf16(128, C, 0), id_u = ltc::idesc_bf16(128, D, 1);
  // this CTA's chunks, over all its items
  int total = 0;
  for (int x = blockIdx.x; x < t.items; x += gridDim.x) total += item_of<STATE_ONLY>(t, x).chunks();
  auto scores = [&](int k) {
    const uint32_t q = smem_addr(sm.stage[k % NST][0]), kk = smem_addr(sm.stage[k % NST][1]);
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
      const uint32_t at = (ks >> 2) * (C * 128) + (ks & 3) * 32u;
      // the product has 128 rows; the tile's 64 are followed by others of the stage, whose lanes nobody reads
      tc::mma_f16(tm + T_SC, tc::smem_desc(q + at, 16, 1024, tc::kSwizzle128),
                  tc::smem_desc(kk + at, 16, 1024, tc::kSwizzle128), id_n64, ks > 0);
    }
    tc::commit(&sm.sc_full);
  };
  bool ok = true;
  if (!STATE_ONLY && total > 0) {
    ok = wait_bar(&sm.full[0], 0, t.a.flags, &sm.abort);
    if (ok) scores(0);
  }
  for (int k = 0; k < total && ok; ++k) {
    const int s = k % NST;
    const uint32_t par = (uint32_t)(k & 1);
    const uint32_t q = smem_addr(sm.stage[s][0]), kk = smem_addr(sm.stage[s][1]);
    // the state before the chunk is in TMEM (and the last chunk's U has been read)
    if (!wait_bar(&sm.s_full, par, t.a.flags, &sm.abort)) break;
    if (!STATE_ONLY) {
      if (k > 0 && !wait_bar(&sm.o_empty, par ^ 1u, t.a.flags, &sm.abort)) break;
      tc::fence_after_sync();
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks)
        ltc::mma_bf16_ta(tm + T_OI, tm + T_S + 8u * ks,
                         tc::smem_desc(q + (ks >> 2) * (C * 128) + (ks & 3) * 32u, 16, 1024, tc::kSwizzle128), id_n64, ks > 0);
      if (!wait_bar(&sm.p_full, par, t.a.flags, &sm.abort)) break;
      if (k + 1 < total) {
        if (!wait_bar(&sm.full[(k + 1) % NST], (uint32_t)(((k + 1) / NST) & 1), t.a.flags, &sm.abort)) break;
        tc::fence_after_sync();
        scores(k + 1);
      }
    }
    if (!wait_bar(&sm.v_full, par, t.a.flags, &sm.abort)) break;
    tc::fence_after_sync();
    if (!STATE_ONLY) {
#pragma unroll
      for (int ks = 0; ks < C / 16; ++ks)
        ltc::mma_bf16_ta(tm + T_OP, tm + T_VR + 8u * ks,
                         tc::smem_desc(smem_addr(sm.p) + ks * 32u, 16, 1024, tc::kSwizzle128), id_n64, ks > 0);
      tc::commit(&sm.op_full);
    }
#pragma unroll
    for (int part = 0; part < 3; ++part)
#pragma unroll
      for (int ks = 0; ks < C / 16; ++ks)
        ltc::mma_bf16_ta(tm + T_U, tm + T_V + 32u * part + 8u * ks,
                         tc::smem_desc(kk + ks * 2048u, C * 128, 1024, tc::kSwizzle128), id_u, part + ks > 0);
    tc::commit(&sm.u_full);
    tc::commit(&sm.empty[s]);
  }
  // every product issued has completed before TMEM is released
  tc::commit(&sm.drain);
  tc::mbar_wait_sleep(&sm.drain, 0, t.a.flags);
}

// ---- P and the value's parts -------------------------------------------------------
// The value tile, transposed into TMEM lanes: raw, and times its decay in three bf16 parts.
template <int D, bool TAIL>
__device__ __forceinline__ void value_parts(const uint8_t* tile, const float* w, int step, int r, uint32_t tm, int e) {
  // element (token i, channel e): block e / 64, row i, 16-byte piece (e % 64) / 8 exchanged by the row's low bits
  const uint8_t* base = tile + (e >> 6) * (C * 128) + (e & 7) * 2;
  const int piece = (e & 63) >> 3;
  const uint32_t lane_addr = tm + ((uint32_t)(e & ~31) << 16);
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    uint32_t raw[16], hi[16], mid[16], lo[16];
#pragma unroll
    for (int x = 0; x < 16; ++x) {
      const int i = 32 * half + 2 * x;
      uint32_t u0 = *reinterpret_cast<const uint16_t*>(base + i * 128 + ((piece ^ (i & 7)) << 4));
      uint32_t u1 = *reinterpret_cast<const uint16_t*>(base + (i + 1) * 128 + ((piece ^ ((i + 1) & 7)) << 4));
      if (TAIL) {       // rows behind the sequence's end are somebody else's
        if (i >= r) u0 = 0;
        if (i + 1 >= r) u1 = 0;
      }
      raw[x] = u0 | (u1 << 16);
      float x0 = __uint_as_float(u0 << 16), x1 = __uint_as_float(u1 << 16);
      const float w0 = TAIL ? (i < r ? w[i * step] : 0.f) : w[i * step];
      const float w1 = TAIL ? (i + 1 < r ? w[(i + 1) * step] : 0.f) : w[(i + 1) * step];
      x0 *= w0;
      x1 *= w1;
      hi[x] = ltc::pack_bf16(x0, x1);
      x0 -= ltc::bf16_lo(hi[x]);
      x1 -= ltc::bf16_hi(hi[x]);
      mid[x] = ltc::pack_bf16(x0, x1);
      x0 -= ltc::bf16_lo(mid[x]);
      x1 -= ltc::bf16_hi(mid[x]);
      lo[x] = ltc::pack_bf16(x0, x1);
    }
    ltc::st_32x32b_x16(lane_addr + T_VR + 16u * half, raw);
    ltc::st_32x32b_x16(lane_addr + T_V + 16u * half, hi);
    ltc::st_32x32b_x16(lane_addr + T_V + 32u + 16u * half, mid);
    ltc::st_32x32b_x16(lane_addr + T_V + 64u + 16u * half, lo);
  }
}

template <int D, bool STATE_ONLY>
__device__ void value_role(const LinTc& t, LinSmem<D>& sm, uint32_t tm, int warp, int lane) {
  using SM = LinSmem<D>;
  const int qd = warp & 3, e = 32 * qd + lane, tid = e;      // e: TMEM lane: value channel, and row i of SC
  int k = 0, n_item = 0;
  bool ok = true;
  for (int x = blockIdx.x; x < t.items; x += gridDim.x) {
    const Item it = item_of<STATE_ONLY>(t, x);
    if (it.chunks() == 0) continue;
    const bool back = t.a.walk[it.w].back;
    float* pw = sm.pw1[n_item & 1];
    ++n_item;
    const float g = clamp_log_decay(t.a.log_decay[it.h]);
    if (tid <= C) pw[tid] = decay_pow(g, tid);
    if (tc::named_sync_any(1, 128, !ok)) return;
    for (int c = 0; c < it.chunks() && ok; ++c, ++k) {
      const int s = k % NST, r = it.rows(chunk_at(it, back, c));
      const uint32_t par = (uint32_t)(k & 1);
      if (!STATE_ONLY && qd < 2) {
        // P: rows i on lanes 0..63
        ok = wait_bar(&sm.sc_full, par, t.a.flags, &sm.abort);
        if (ok && k > 0) ok = wait_bar(&sm.op_full, par ^ 1u, t.a.flags, &sm.abort);    // the last P has been used
        if (!__all_sync(FULL, ok)) { ok = false; break; }
        tc::fence_after_sync();
        uint8_t* row = sm.p + e * 128;
#pragma unroll
        for (int j0 = 0; j0 < C; j0 += 16) {
          uint32_t sc[16], p2[8];
          tc::ld_32x32b_x16(tm + ((uint32_t)(32 * qd) << 16) + T_SC + j0, sc);
          tc::wait_ld();
#pragma unroll
          for (int j = 0; j < 16; j += 2) {
            float v[2];
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const int age = back ? j0 + j + y - e : e - (j0 + j + y);
              const bool in = age >= 0 && j0 + j + y < r;
              v[y] = in ? __uint_as_float(sc[j + y]) * pw[age & 63] : 0.f;
            }
            p2[j >> 1] = ltc::pack_bf16(v[0], v[1]);
          }
          const int ch = j0 >> 3;
          *reinterpret_cast<uint4*>(row + ((ch ^ (e & 7)) << 4)) = make_uint4(p2[0], p2[1], p2[2], p2[3]);
          *reinterpret_cast<uint4*>(row + (((ch + 1) ^ (e & 7)) << 4)) = make_uint4(p2[4], p2[5], p2[6], p2[7]);
        }
        fence_proxy_async_smem();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&sm.p_full);
      }
      ok = wait_bar(&sm.full[s], (uint32_t)((k / NST) & 1), t.a.flags, &sm.abort);
      if (ok && k > 0) ok = wait_bar(&sm.u_full, par ^ 1u, t.a.flags, &sm.abort);       // the last parts have been used
      if (!__all_sync(FULL, ok)) { ok = false; break; }
      tc::fence_after_sync();
      if (r < C) {
        // keys behind the sequence's end: zeros, for their products with zero values must be zero
        uint8_t* kt = sm.stage[s][1];
        for (int y = tid; y < (C - r) * (D / 8); y += 128) {
          const int row = r + y / (D / 8), ch = y % (D / 8);
          *reinterpret_cast<uint4*>(kt + (ch >> 3) * (C * 128) + row * 128 + (ch & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();
      }
      if (32 * qd < D) {
        // decay of row i: forwards A^(r-1-i), backwards A^(i+1)
        const float* w = back ? pw + 1 : pw + r - 1;
        if (r < C) value_parts<D, true>(sm.stage[s][2], w, back ? 1 : -1, r, tm, e);
        else if (back) value_parts<D, false>(sm.stage[s][2], w, 1, r, tm, e);
        else value_parts<D, false>(sm.stage[s][2], w, -1, r, tm, e);
        ltc::wait_st();
      }
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) {
        tc::mbar_arrive(&sm.v_full);
        tc::mbar_arrive(&sm.empty[s]);
      }
    }
  }
}

// ---- state and output ---------------------------------------------------------------
template <int D>
__device__ __forceinline__ void state_to_tmem(const float (&S)[D / 2], uint32_t at) {
#pragma unroll
  for (int b = 0; b < D / 64; ++b) {
    uint32_t u[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) u[j] = ltc::pack_bf16(S[32 * b + 2 * j], S[32 * b + 2 * j + 1]);
    ltc::st_32x32b_x16(at + 16u * b, u);
  }
  ltc::wait_st();
}

template <int D, bool STATE_ONLY>
__device__ void state_role(const LinTc& t, LinSmem<D>& sm, uint32_t tm, int warp, int lane) {
  constexpr int HC = D / 2;                                  // key channels of a thread
  const int qd = warp & 3, half = (warp - 8) >> 2, e = 32 * qd + lane, tid = e;
  const bool mine = 32 * qd < D;                             // lanes beyond d hold nothing
  const uint32_t lane_addr = tm + ((uint32_t)(32 * qd) << 16);
  const int bar_id = 2 + half;
  int k = 0, n_item = 0;
  bool ok = true;
  float S[HC];
  for (int x = blockIdx.x; x < t.items; x += gridDim.x) {
    const Item it = item_of<STATE_ONLY>(t, x);
    if (!it.on) continue;
    const LinWalk& w = t.a.walk[it.w];
    const bool back = w.back;
    const size_t st0 = ((size_t)it.n * t.a.H + it.h) * D * D;
    const float* in = STATE_ONLY ? nullptr : (it.nseg > 1 ? stretch_state(t, it) : (w.S_in ? w.S_in + st0 : nullptr));
    const bool in_swap = it.nseg > 1 ? false : w.swap != 0;
    float* out = STATE_ONLY ? stretch_state(t, it)
                            : (w.S_out && it.seg == (back ? 0 : it.nseg - 1) ? w.S_out + st0 : nullptr);
    const bool out_swap = !STATE_ONLY && w.swap != 0;
    // tables of the decay
    float* pw = sm.pw2[n_item & 1][half];
    ++n_item;
    const float g = clamp_log_decay(t.a.log_decay[it.h]);
    if (tid < C) pw[tid] = decay_pow(g, tid + (back ? 0 : 1));        // forwards A^(i+1); backwards A^i
    if (tid >= 96 && tid < 98 && it.chunks() > 0) {
      // A^rows of a full chunk and of the last one, 48 bits: the state is multiplied by them all along
      const double a = exp((double)g * (tid == 96 ? C : it.rows(it.c1 - 1)));
      pw[C + 4 + 2 * (tid - 96)] = (float)a;
      pw[C + 5 + 2 * (tid - 96)] = (float)(a - (double)(float)a);
    }
    if (mine) {
      if (in && in_swap) {
#pragma unroll
        for (int j = 0; j < HC; ++j) S[j] = in[(size_t)(HC * half + j) * D + e];
      } else if (in) {
#pragma unroll
        for (int j = 0; j < HC; j += 4)
          *reinterpret_cast<float4*>(&S[j]) = *reinterpret_cast<const float4*>(in + (size_t)e * D + HC * half + j);
      } else {
#pragma unroll
        for (int j = 0; j < HC; ++j) S[j] = 0.f;
      }
    }
    if (tc::named_sync_any(bar_id, 128, !ok)) return;
    for (int c = 0; c < it.chunks(); ++c, ++k) {
      const int ch = chunk_at(it, back, c), r = it.rows(ch);
      const uint32_t par = (uint32_t)(k & 1);
      if (c == 0) {
        // the state before the first chunk; the products of the chunk before have been waited for
        if (!STATE_ONLY && mine) state_to_tmem<D>(S, lane_addr + T_S + (HC / 2) * half);
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&sm.s_full);
      }
      ok = __all_sync(FULL, wait_bar(&sm.u_full, par, t.a.flags, &sm.abort));
      if (ok) {
        tc::fence_after_sync();
        const float ah = pw[C + 4 + (r < C ? 2 : 0)], al = pw[C + 5 + (r < C ? 2 : 0)];
        if (mine) {
          const float2 h2 = make_float2(ah, ah), l2 = make_float2(al, al);
#pragma unroll
          for (int j0 = 0; j0 < HC; j0 += 16) {
            uint32_t u[16];
            tc::ld_32x32b_x16(lane_addr + T_U + HC * half + j0, u);
            tc::wait_ld();
#pragma unroll
            for (int j = 0; j < 16; j += 2) {
              const float2 s2 = make_float2(S[j0 + j], S[j0 + j + 1]);
              const float2 n2 = __ffma2_rn(s2, h2, __ffma2_rn(s2, l2, make_float2(__uint_as_float(u[j]), __uint_as_float(u[j + 1]))));
              S[j0 + j] = n2.x;
              S[j0 + j + 1] = n2.y;
            }
          }
        }
        if (c + 1 < it.chunks()) {
          if (!STATE_ONLY && mine) state_to_tmem<D>(S, lane_addr + T_S + (HC / 2) * half);
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&sm.s_full);
        }
      }
      if (STATE_ONLY) {
        if (tc::named_sync_any(bar_id, 128, !ok)) return;
        continue;
      }
      // the output: tokens 32 half .. + 31 of the chunk
      if (ok) ok = __all_sync(FULL, wait_bar(&sm.op_full, par, t.a.flags, &sm.abort));
      uint16_t(*os)[D] = sm.o[k & 1][half];
      if (ok) {
        tc::fence_after_sync();
        if (mine) {
#pragma unroll
          for (int i0 = 0; i0 < 32; i0 += 16) {
            uint32_t oi[16], op[16];
            tc::ld_32x32b_x16(lane_addr + T_OI + 32 * half + i0, oi);
            tc::ld_32x32b_x16(lane_addr + T_OP + 32 * half + i0, op);
            tc::wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const int tok = 32 * half + i0 + i;
              const float wt = back ? pw[max(r - 1 - tok, 0)] : pw[tok];
              os[i0 + i][e] = float_to_bf16_bits_rn(fmaf(wt, __uint_as_float(oi[i]), __uint_as_float(op[i])));
            }
          }
        }
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&sm.o_empty);
      }
      if (tc::named_sync_any(bar_id, 128, !ok)) return;
      constexpr int PR = D / 8;                              // 16-byte pieces a row
#pragma unroll
      for (int y = tid; y < 32 * PR; y += 128) {
        const int i = y / PR, ch16 = y % PR, tok = 32 * half + i;
        if (tok < r) {
          uint16_t* dst = reinterpret_cast<uint16_t*>(w.out) + (size_t)(it.begin + ch * C + tok) * w.out_stride + it.h * D + 8 * ch16;
          *reinterpret_cast<uint4*>(dst) = *reinterpret_cast<const uint4*>(&os[i][8 * ch16]);
        }
      }
    }
    if (out && mine) {
      if (out_swap) {
#pragma unroll
        for (int j = 0; j < HC; ++j) out[(size_t)(HC * half + j) * D + e] = S[j];
      } else {
#pragma unroll
        for (int j = 0; j < HC; j += 4)
          *reinterpret_cast<float4*>(out + (size_t)e * D + HC * half + j) = *reinterpret_cast<const float4*>(&S[j]);
      }
    }
  }
}

template <int D, bool STATE_ONLY>
__global__ void __launch_bounds__(kTcThreads, 1)
    linattn_tc_kernel(const __grid_constant__ LinTc t, const __grid_constant__ LinMaps maps) {
  using SM = LinSmem<D>;
  extern __shared__ uint8_t smem_raw[];
  SM& sm = *reinterpret_cast<SM*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int s = 0; s < NST; ++s) {
      mbar_init(&sm.full[s], 1);
      mbar_init(&sm.empty[s], 5);              // the products, and the four warps that read the values
    }
    mbar_init(&sm.sc_full, 1);
    mbar_init(&sm.p_full, 2);
    mbar_init(&sm.v_full, 4);
    mbar_init(&sm.s_full, 8);
    mbar_init(&sm.u_full, 1);
    mbar_init(&sm.op_full, 1);
    mbar_init(&sm.o_empty, 8);
    mbar_init(&sm.drain, 1);
    sm.abort = 0;
    fence_mbar_init();
  }
  if (warp == 1) tc::tmem_alloc(&sm.taddr, 512);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tm = sm.taddr;
  if (warp == 0) {
    if (lane == 0) load_role<D, STATE_ONLY>(t, maps, sm);
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0) mma_role<D, STATE_ONLY>(t, sm, tm);
    __syncwarp();
  } else if (warp >= 8) {
    state_role<D, STATE_ONLY>(t, sm, tm, warp, lane);
  } else if (warp >= 4) {
    value_role<D, STATE_ONLY>(t, sm, tm, warp, lane);
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == 1) tc::tmem_free(tm, 512);
}

// ---- chaining the stretches ----------------------------------------------------------
// ws[s] (stretch s's own contribution) -> the state before stretch s, in the walk's order:
//   run = S_in;  for s in order: (ws[s], run) = (run, A^tokens(s) run + ws[s]).
template <int D>
__global__ void __launch_bounds__(256) linattn_chain_kernel(const __grid_constant__ LinTc t) {
  const int x = blockIdx.x;
  Item it;
  it.w = x % t.a.walks;
  it.h = (x / t.a.walks) % t.a.H;
  it.n = x / t.a.walks / t.a.H;
  it.seg = 0;
  int end;
  seq_rows(t.a, it.n, &it.begin, &end);
  it.len = end - it.begin;
  const int nc = (it.len + C - 1) / C;
  const int ns = min((nc + t.split.per - 1) / t.split.per, t.split.stretches);
  if (ns <= 1) return;
  const LinWalk& w = t.a.walk[it.w];
  const double g = (double)clamp_log_decay(t.a.log_decay[it.h]);
  float* ws = stretch_state(t, it);
  const size_t st0 = ((size_t)it.n * t.a.H + it.h) * D * D;
  // every stretch between the ends of a walk is `per` chunks long; the last one of the sequence may differ
  const float a_full = (float)exp(g * (double)t.split.per * C);
  const float a_last = (float)exp(g * (double)(it.len - (ns - 1) * t.split.per * C));
  for (int y = (blockIdx.y * 256 + threadIdx.x) * 4; y < D * D; y += gridDim.y * 256 * 4) {
    float4 run = make_float4(0.f, 0.f, 0.f, 0.f);
    if (w.S_in) {
      if (w.swap) {
        const int i = y / D, j = y % D;
        run = make_float4(w.S_in[st0 + (size_t)j * D + i], w.S_in[st0 + (size_t)(j + 1) * D + i],
                          w.S_in[st0 + (size_t)(j + 2) * D + i], w.S_in[st0 + (size_t)(j + 3) * D + i]);
      } else {
        run = *reinterpret_cast<const float4*>(w.S_in + st0 + y);
      }
    }
    for (int k = 0; k < ns; ++k) {
      const int s = w.back ? ns - 1 - k : k;
      float4* at = reinterpret_cast<float4*>(ws + (size_t)s * D * D + y);
      if (k + 1 < ns) {
        const float4 own = *at;
        *at = run;
        const float a = s == ns - 1 ? a_last : a_full;
        run = make_float4(fmaf(a, run.x, own.x), fmaf(a, run.y, own.y), fmaf(a, run.z, own.z), fmaf(a, run.w, own.w));
      } else {
        *at = run;
      }
    }
  }
}

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
  static EncodeFn encode = nullptr;
  if (!encode) {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &fn, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess || !fn) {
      (void)cudaGetLastError();
      return nullptr;
    }
    encode = reinterpret_cast<EncodeFn>(fn);
  }
  return encode;
}

// rows of `width` bf16, `stride` elements apart, in boxes of 64 rows of 64 elements
bool make_map(CUtensorMap* m, const void* p, int64_t width, int64_t stride, int64_t rows) {
  EncodeFn encode = encode_fn();
  if (!encode) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)width, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)stride * 2};
  const cuuint32_t box[2] = {64, (cuuint32_t)C};
  const cuuint32_t estr[2] = {1, 1};
  return encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(p), dims, strides, box, estr,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
cudaError_t launch_tc(const LinTc& t0, const LinMaps& maps, cudaStream_t st) {
  LinTc t = t0;
  const size_t smem = sizeof(LinSmem<D>) + 1024;
  static_assert(sizeof(LinSmem<D>) + 1024 <= 232448, "shared memory");
  cudaError_t e = cudaFuncSetAttribute(linattn_tc_kernel<D, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  const unsigned blocks = (unsigned)(t.items < kSms ? t.items : kSms);
  if (t.split.stretches > 1) {
    e = cudaFuncSetAttribute(linattn_tc_kernel<D, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    linattn_tc_kernel<D, true><<<blocks, kTcThreads, smem, st>>>(t, maps);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    linattn_chain_kernel<D><<<dim3((unsigned)(t.a.N * t.a.H * t.a.walks), D == 128 ? 4 : 1), 256, 0, st>>>(t);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  linattn_tc_kernel<D, false><<<blocks, kTcThreads, smem, st>>>(t, maps);
  return cudaGetLastError();
}

}  // namespace

LinSplit linattn_tc_split(int64_t heads, int64_t max_len, int walks) {
  LinSplit sp;
  sp.stretches = 1;
  const int64_t chunks = (max_len + C - 1) / C, items = heads * walks;
  sp.per = (int32_t)(chunks < 1 ? 1 : chunks);
  if (items >= kSms || chunks < 16) return sp;
  // stretches of 8 chunks at least, two rounds of the SMs at most
  int64_t n = 2 * kSms / items;
  if (n > chunks / 8) n = chunks / 8;
  if (n < 2) return sp;
  sp.per = (int32_t)((chunks + n - 1) / n);
  sp.stretches = (int32_t)((chunks + sp.per - 1) / sp.per);
  return sp;
}

bool linattn_tc_takes(const LinArgs& a) {
  if (a.io != PACE_IO_BF16 || (a.D != 64 && a.D != 128) || a.total == 0) return false;
  for (int w = 0; w < a.walks; ++w) {
    const LinWalk& k = a.walk[w];
    if (((uintptr_t)k.query | (uintptr_t)k.key | (uintptr_t)k.value | (uintptr_t)k.out) % 16) return false;
    if ((k.query_stride | k.key_stride | k.value_stride | k.out_stride) % 8) return false;
  }
  return true;
}

cudaError_t launch_linattn_tc(const LinArgs& a, const LinSplit& sp, float* ws, cudaStream_t st) {
  LinTc t;
  LinMaps maps;
  t.a = a;
  t.split = sp;
  t.ws = ws;
  const int64_t items = (int64_t)a.N * a.H * a.walks * sp.stretches;
  if (items > 0x7fffffffll) return cudaErrorInvalidValue;
  t.items = (int32_t)items;
  // the tensors of all walks, each mapped once
  struct Seen { const void* p; int64_t stride; } seen[4];
  int n = 0;
  auto index = [&](const void* p, int64_t stride) {
    for (int i = 0; i < n; ++i)
      if (seen[i].p == p && seen[i].stride == stride) return i;
    if (n == 4 || !make_map(&maps.m[n], p, (int64_t)a.H * a.D, stride, a.total)) return -1;
    seen[n] = Seen{p, stride};
    return n++;
  };
  for (int w = 0; w < a.walks; ++w) {
    t.map_q[w] = index(a.walk[w].query, a.walk[w].query_stride);
    t.map_k[w] = index(a.walk[w].key, a.walk[w].key_stride);
    t.map_v[w] = index(a.walk[w].value, a.walk[w].value_stride);
    if (t.map_q[w] < 0 || t.map_k[w] < 0 || t.map_v[w] < 0) return cudaErrorInvalidValue;
  }
  return a.D == 128 ? launch_tc<128>(t, maps, st) : launch_tc<64>(t, maps, st);
}

}  // namespace pace
