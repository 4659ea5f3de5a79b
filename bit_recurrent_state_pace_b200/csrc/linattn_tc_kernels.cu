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
//   OP  [e, i]  = V^T P,  P = mask A^|i-j| SC  V read MN-major, P in two bf16 parts
//   U   [e, c]  = (V A^..)^T K                 A in TMEM in three bf16 parts, K read MN-major
// out^T = OP + A^.. OI, and S stays in registers in fp32.
//
// Roundings: the copy of S that multiplies the query is bf16 (2^-9 of each term, the size of the output's own
// rounding).  P is split into two bf16 parts (16 bits): rounded to one, short prompts came 1.5 times as far from the
// exact outputs as those rounded once.  The value times its decay is split into three (24 bits), so that the states,
// which are fp32 outputs and run over the whole sequence, are summed from exact products of 24 bits; two parts would
// leave about 2e-6 of the state, and are taken in a backward pass without dS0 (a third of U's products and of the split).
//
// One persistent CTA of 28 warps per SM, each group of four (a TMEM lane quadrant each) with one job, so that their
// latencies overlap:
//  * warp 0: loads the chunks' tiles by TMA, two chunks ahead; warp 2: the states;
//  * warp 1 issues U, warp 3 SC, OI and OP: by one warp, every product waited for the slowest of the others' operands;
//  * warps 4-11: the value's decayed parts into TMEM, half of the tokens each four;
//  * warps 12-15: P from SC;  warps 16-19: the output, stored by TMA;
//  * warps 20-27: the state, half of the key channels each four.
//
// Sequences too few to fill the SMs are cut into stretches: the same kernel
// without outputs gives each stretch's own contribution to the state, a small
// one chains them, and the stretches then run from their true states.
//
// Gradients of 8 x 32 heads, 4096 tokens, d = 128: 857 us (0.33 of the measured copy); 64 prompts of 1 to 1021 tokens, 32
// heads, with states: 228 us (0.42); one of 32768 tokens, 32 heads: 478 us (0.34).  In the steady state a chunk takes 4200
// cycles (d = 64: 3400), of a backward pass 3600 (3400), and the tensor pipe is active for 30 % of them; the rest is what
// the groups wait for one another and, a fifth of it, for instructions: the loops fill the instruction cache, so that code
// costs time even where it is not run.  Loops of seconds over long sequences draw 990 W, which holds the SM clock at 1.55 to
// 1.8 GHz (the ragged prompts 950 W, at the full clock).
#include <atomic>

#include "linattn_tc.cuh"

namespace pace {

namespace {

constexpr unsigned FULL = 0xffffffffu;
constexpr int C = 64;                 // tokens a chunk
constexpr int NST = 3;                // staged chunks
constexpr int kTcThreads = 896;
constexpr int kSms = 148;             // B200
constexpr int kMaxSorted = 512;       // sequences that are put in order (more come out even anyway)

// TMEM columns.  All 512 are allocated, so the allocation begins at column 0.
constexpr uint32_t T_SC = 0, T_OI = 64, T_OP = 128, T_S = 320;
// U and the value's parts: one buffer each, or two where only states are wanted and there is room
template <bool STATE_ONLY>
__device__ __forceinline__ uint32_t t_u(int k) { return STATE_ONLY ? 128u * (k & 1) : 192u; }
template <bool STATE_ONLY>
__device__ __forceinline__ uint32_t t_v(int k) { return STATE_ONLY ? 256u + 96u * (k & 1) : 384u; }
// Chunk k's phase of a barrier kept for each buffer, and whether an earlier chunk had the buffer.
template <bool STATE_ONLY>
__device__ __forceinline__ int buffer_of(int k) { return STATE_ONLY ? (k & 1) : 0; }
template <bool STATE_ONLY>
__device__ __forceinline__ uint32_t phase_of(int k) { return (uint32_t)((STATE_ONLY ? k >> 1 : k) & 1); }
template <bool STATE_ONLY>
__device__ __forceinline__ bool used_before(int k) { return k >= (STATE_ONLY ? 2 : 1); }

struct LinMaps {
  CUtensorMap in[4], out[kLinMaxWalks];              // the packed tensors
  CUtensorMap s_in[kLinMaxWalks], s_out[kLinMaxWalks], ws;   // states: rows of D fp32
};

struct LinTc {
  LinArgs a;
  int32_t map_q[kLinMaxWalks], map_k[kLinMaxWalks], map_v[kLinMaxWalks];
  LinSplit split;
  float* ws;               // [walks][N][H][stretches][D][D]: each stretch's state
  int32_t items;           // (n, h, stretch, walk)
  uint32_t tries;          // tests of a wait
  uint32_t extra_tx;       // 0; 16: the first loads' barrier of block 0 waits for more than they bring (debug)
};

template <int D>
struct alignas(1024) LinSmem {
  static constexpr int TILE = C * D * 2;                 // D / 64 blocks of 64 rows of 128 bytes
  uint8_t stage[NST][3][TILE];                           // query | key | value
  uint8_t p[2][C * 128];                                 // P[i][j] in two bf16 parts, 128-byte swizzle
  static constexpr int STATE = D * D * 2;                // half of a state (D / 2 key channels)
  uint8_t st[STATE];                                     // states on their way in and out: rows of 128 bytes, swizzled
  uint8_t o[4][C * 64];                                  // outputs on their way: 64 rows of 32 channels for each lane quadrant
  // tables of the decay, of two items in turn, each group of warps its own:
  uint2 wv[2][2][2][C / 4];                              // warps 4-7, 8-11: decay of their tokens' values in the state behind
                                                         // a full chunk, and behind the sequence's last one (zeros beyond
                                                         // it): two tokens an entry, as value_parts wants them
  float pz[2][2 * C + 8];                                // warps 12-15: A^n at [C + n], zeros below
  float wo[2][2][C];                                     // warps 16-19: of the state in a token's output, as wv
  uint64_t full[NST], empty[NST];
  uint64_t sc_full, sc_empty, p_full, v_full[2], s_full, u_full[2], u_empty[2], op_full, o_empty, st_full[2], st_done[2], drain[2];
  int chunks[kMaxSorted];                                // of each sequence
  uint16_t order[kMaxSorted];                            // sequences, the longest first
  uint32_t taddr;
  int bad;                                               // a wait gave up
  uint32_t tries;                                        // tests of a wait
};

template <class SM>
__device__ __forceinline__ bool wait_all(const SM& sm, uint64_t* bar, uint32_t parity) {
  return __all_sync(FULL, ltc::wait_tries(sm, bar, parity)) != 0;
}
template <int D>
__device__ __forceinline__ void gave_up(const LinTc& t, LinSmem<D>& sm) {
  *reinterpret_cast<volatile int*>(&sm.bad) = 1;
  if (t.a.flags) atomicOr(t.a.flags, PACE_FLAG_TIMEOUT);
}

// Work item: one walk of one stretch of one sequence and head.
struct Item {
  int w, n, h, seg, begin, len, c0, c1;     // rows [begin, begin + len) of the sequence, chunks [c0, c1)
  int nseg;                                 // stretches of this sequence
  bool on;                                  // there is something to do
  __device__ __forceinline__ int chunks() const { return c1 - c0; }
  __device__ __forceinline__ int rows(int c) const { return min(C, len - c * C); }
};

// The k-th item of this block (order_sequences says which those are), for k < item_rounds.
__device__ __forceinline__ int item_rounds(const LinTc& t) { return (t.items + (int)gridDim.x - 1) / (int)gridDim.x; }
template <bool STATE_ONLY>
__device__ __forceinline__ Item item_of(const LinTc& t, const uint16_t* order, int k) {
  int x = k * (int)gridDim.x + (int)(t.a.cu && (k & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
  Item it;
  const bool there = x < t.items;
  if (!there) x = 0;
  it.w = x % t.a.walks;
  x /= t.a.walks;
  it.seg = x % t.split.stretches;
  x /= t.split.stretches;
  it.h = x % t.a.H;
  it.n = x / t.a.H;
  if (t.a.cu && t.a.N <= kMaxSorted) it.n = order[it.n];
  int end;
  seq_rows(t.a, it.n, &it.begin, &end);
  it.len = end - it.begin;
  const int nc = (it.len + C - 1) / C;
  it.nseg = stretches_of(t.split, it.len);
  it.on = there && it.seg < it.nseg;
  // the stretch that a walk ends with hands its state to no other
  if (STATE_ONLY) it.on = it.on && it.seg != (t.a.walk[it.w].back ? 0 : it.nseg - 1);
  it.c0 = it.seg * t.split.per;
  it.c1 = it.seg == it.nseg - 1 ? nc : it.c0 + t.split.per;
  if (!it.on) it.c0 = it.c1 = 0;
  return it;
}

// What an item begins from and leaves: a state of ws, of the walk's tensors (transposed or not), or none.
struct StateIo {
  bool in, out, in_swap, out_swap;
};
template <bool STATE_ONLY>
__device__ __forceinline__ StateIo state_io(const LinTc& t, const Item& it) {
  const LinWalk& w = t.a.walk[it.w];
  StateIo io;
  const bool cut = it.nseg > 1;
  io.in = !STATE_ONLY && (cut || w.S_in);
  io.in_swap = !cut && w.swap;
  io.out = STATE_ONLY || (w.S_out && it.seg == (w.back ? 0 : it.nseg - 1));
  io.out_swap = !STATE_ONLY && w.swap;
  return io;
}
// The state's place in shared memory is exchanged in one go (the last item's state out, this one's in) where both lie
// alike; else the one leaves before the other comes.
__device__ __forceinline__ bool two_rounds(const StateIo& last, const StateIo& now) {
  return last.out && now.in && last.out_swap != now.in_swap;
}
// k-th chunk of an item in its walk's order
__device__ __forceinline__ int chunk_at(const Item& it, bool back, int k) { return back ? it.c1 - 1 - k : it.c0 + k; }

// ---- which items a block takes ------------------------------------------------------
// The items -- sequence, head, stretch, walk -- are dealt to the blocks in turn: the heads of a sequence run at the same
// time, so that their parts of a token's row are read together, and so do the three walks of a backward pass over a
// head, which read the same tensors.  (A block that keeps to one walk took 7 % longer.)  Where lengths differ the longest
// sequences go first, back and forth, and the blocks' sums come out about even: in the order given, 64 prompts of 1 to
// 1021 tokens kept some blocks busy twice as long as the mean; contiguous shares of equal cost were a fifth slower than
// that.
template <int D>
__device__ void order_sequences(const LinTc& t, LinSmem<D>& sm) {
  if (!t.a.cu || t.a.N > kMaxSorted) return;
  for (int n = threadIdx.x; n < t.a.N; n += kTcThreads) {
    int begin, end;
    seq_rows(t.a, n, &begin, &end);
    sm.chunks[n] = (end - begin + C - 1) / C;
  }
  __syncthreads();
  for (int n = threadIdx.x; n < t.a.N; n += kTcThreads) {
    const int own = sm.chunks[n];
    int rank = 0;
    for (int m = 0; m < t.a.N; ++m) {
      const int c = sm.chunks[m];
      rank += c > own || (c == own && m < n);
    }
    sm.order[rank] = (uint16_t)n;
  }
}

// ---- loads ---------------------------------------------------------------------
template <int D, bool STATE_ONLY>
__device__ void load_role(const LinTc& t, const LinMaps& maps, LinSmem<D>& sm) {
  using SM = LinSmem<D>;
  int k = 0;
  bool ok = true;
  for (int i = 0; i < item_rounds(t) && ok; ++i) {
    const Item it = item_of<STATE_ONLY>(t, sm.order, i);
    const bool back = t.a.walk[it.w].back;
    const CUtensorMap* mp[3] = {&maps.in[t.map_q[it.w]], &maps.in[t.map_k[it.w]], &maps.in[t.map_v[it.w]]};
    for (int c = 0; c < it.chunks(); ++c, ++k) {
      const int s = k % NST, r = k / NST;
      if (r > 0 && !ltc::wait_tries(sm, &sm.empty[s], (uint32_t)((r - 1) & 1))) { ok = false; break; }
      const int row = it.begin + chunk_at(it, back, c) * C;
      constexpr int first = STATE_ONLY ? 1 : 0;
      mbar_arrive_expect_tx(&sm.full[s], (3 - first) * SM::TILE + (k == 0 && blockIdx.x == 0 ? t.extra_tx : 0u));
#pragma unroll
      for (int m = first; m < 3; ++m)
#pragma unroll
        for (int b = 0; b < D / 64; ++b)
          ltc::tensor_load_2d(smem_addr(&sm.stage[s][m][b * C * 128]), mp[m], it.h * D + 64 * b, row, &sm.full[s]);
    }
  }
  if (!ok) gave_up(t, sm);
  // nothing may land after the block has left, though nobody waits for it
  for (int j = max(0, k - NST); j < k; ++j) ltc::wait_tries(sm, &sm.full[j % NST], (uint32_t)((j / NST) & 1));
}

// ---- states ---------------------------------------------------------------------
// One place in shared memory serves the states of all items, a half (the key channels of one group of the state's warps)
// at a time: a half is loaded into it as soon as the one before has left, the warps exchange it for theirs, and theirs
// goes out.  The next item's first half is there long before its use.  Each round: (load or not) -> st_full -> the
// exchange -> st_done -> (store or not).  By the state's own threads, row by row, reading and writing a state took
// 14,000 cycles of an item.
template <int D, bool STATE_ONLY>
__device__ void state_io_role(const LinTc& t, const LinMaps& maps, LinSmem<D>& sm) {
  uint32_t round[2] = {0, 0};
  bool ok = true;
  // half of a state as its tensor map's boxes: 32 columns by D rows, or (transposed) by D / 2 rows
  auto load = [&](const Item& it, int half, bool in, bool swap) {
    if (!in) {
      tc::mbar_arrive(&sm.st_full[half]);
      return;
    }
    const CUtensorMap* m = it.nseg > 1 ? &maps.ws : &maps.s_in[it.w];
    const int row = (it.nseg > 1 ? (int)stretch_index(t.a, t.split, it.w, it.n, it.h, it.seg) : it.n * t.a.H + it.h) * D;
    mbar_arrive_expect_tx(&sm.st_full[half], LinSmem<D>::STATE);
    const int boxes = swap ? D / 32 : D / 64, bytes = swap ? D * 64 : D * 128;
    for (int b = 0; b < boxes; ++b)
      ltc::tensor_load_2d(smem_addr(sm.st) + b * bytes, m, 32 * b + (swap ? 0 : D / 2 * half), row + (swap ? D / 2 * half : 0),
                          &sm.st_full[half]);
  };
  auto done = [&](const Item& it, int half, bool out, bool swap) {
    // the state's warps come to it when they have walked the item: as many budgets as it has chunks, and one
    const uint32_t par = round[half]++ & 1u;
    bool there = ltc::wait_tries(sm, &sm.st_done[half], par);
    for (int c = it.chunks(); !there && c > 0 && !*reinterpret_cast<volatile int*>(&sm.bad); --c)
      there = ltc::wait_tries(sm, &sm.st_done[half], par);
    if (!there) return false;
    if (out) {
      const CUtensorMap* m = STATE_ONLY ? &maps.ws : &maps.s_out[it.w];
      const int row = (STATE_ONLY ? (int)stretch_index(t.a, t.split, it.w, it.n, it.h, it.seg) : it.n * t.a.H + it.h) * D;
      const int boxes = swap ? D / 32 : D / 64, bytes = swap ? D * 64 : D * 128;
      for (int b = 0; b < boxes; ++b)
        tc::tensor_store_2d(m, smem_addr(sm.st) + b * bytes, 32 * b + (swap ? 0 : D / 2 * half), row + (swap ? D / 2 * half : 0));
      tc::bulk_commit_group();
      tc::bulk_wait_read_all();
    }
    return true;
  };
  Item last = {};
  StateIo last_io = {false, false, false, false};
  for (int i = 0; i < item_rounds(t) && ok; ++i) {
    const Item it = item_of<STATE_ONLY>(t, sm.order, i);
    if (!it.on) continue;
    const StateIo io = state_io<STATE_ONLY>(t, it);
    const bool two = two_rounds(last_io, io);
    for (int half = 0; half < 2 && ok; ++half) {
      if (two) {
        load(last, half, false, false);
        ok = done(last, half, true, last_io.out_swap);
        if (!ok) break;
      }
      load(it, half, io.in, io.in_swap);
      ok = done(last, half, !two && last_io.out, last_io.out_swap);
    }
    last = it;
    last_io = io;
  }
  for (int half = 0; half < 2 && ok && last_io.out; ++half) {
    load(last, half, false, false);
    ok = done(last, half, true, last_io.out_swap);
  }
  if (!ok) {
    gave_up(t, sm);
    // nothing of ours may land after the block has left: a round that gave up had its load before it
    for (int half = 0; half < 2; ++half)
      if (round[half]) ltc::wait_tries(sm, &sm.st_full[half], (round[half] - 1) & 1u);
  }
  tc::bulk_wait_all();
}

// ---- products --------------------------------------------------------------------
// This CTA's chunks, over all its items.
template <int D, bool STATE_ONLY>
__device__ __forceinline__ int chunks_of_block(const LinTc& t, const LinSmem<D>& sm) {
  int total = 0;
#pragma unroll 1
  for (int i = 0; i < item_rounds(t); ++i) total += item_of<STATE_ONLY>(t, sm.order, i).chunks();
  return total;
}
// every product that the calling warp issued has completed (TMEM is released after that)
template <int D>
__device__ __forceinline__ void drain(LinSmem<D>& sm, int which) {
  if (ltc::elect_one()) tc::commit(&sm.drain[which]);
  __syncwarp();
  ltc::wait_tries(sm, &sm.drain[which], 0);
}

// Warp 1: U of each chunk, as soon as the value's parts are there and the last U has been read.
template <int D, int PARTS, bool STATE_ONLY>
__device__ void update_role(const LinTc& t, LinSmem<D>& sm, int total) {
  using SM = LinSmem<D>;
  constexpr uint32_t id_u = ltc::idesc_bf16(128, D, 0, 1);
  // descriptors of stage 0; a tile or step further is its bytes / 16 more
  const uint64_t kt0 = tc::smem_desc(smem_addr(sm.stage[0][1]), C * 128, 1024, tc::kSwizzle128);
  constexpr uint32_t kStage = 3 * SM::TILE / 16;
  bool ok = true;
  int s = 0;
  for (int k = 0; k < total; ++k) {
    const int b = buffer_of<STATE_ONLY>(k);
    const uint32_t par = phase_of<STATE_ONLY>(k);
    if (!(ok = wait_all(sm, &sm.v_full[b], par))) break;
    if (used_before<STATE_ONLY>(k) && !(ok = wait_all(sm, &sm.u_empty[b], par ^ 1u))) break;
    tc::fence_after_sync();
    if (ltc::elect_one()) {
#pragma unroll 1
      for (int part = 0; part < PARTS; ++part)
#pragma unroll
        for (int ks = 0; ks < C / 16; ++ks)
          ltc::mma_ts(t_u<STATE_ONLY>(k), t_v<STATE_ONLY>(k) + 32u * part + 8u * ks, kt0 + (kStage * s + 128u * ks), id_u, part + ks > 0);
      tc::commit(&sm.u_full[b]);
      tc::commit(&sm.empty[s]);
    }
    __syncwarp();
    s = s + 1 == NST ? 0 : s + 1;
  }
  if (!ok) gave_up(t, sm);
  drain<D>(sm, 0);
}

// Warp 3: SC of the next chunk as soon as this one's has been read, then this one's OI and OP.
template <int D>
__device__ void output_mma_role(const LinTc& t, LinSmem<D>& sm, int total) {
  using SM = LinSmem<D>;
  constexpr uint32_t id_sc = ltc::idesc_bf16(C, C, 0, 0), id_oi = ltc::idesc_bf16(128, C, 0, 0), id_op = ltc::idesc_bf16(128, C, 1, 0);
  const uint64_t q0 = tc::smem_desc(smem_addr(sm.stage[0][0]), 16, 1024, tc::kSwizzle128);
  const uint64_t k0 = tc::smem_desc(smem_addr(sm.stage[0][1]), 16, 1024, tc::kSwizzle128);
  // the value as A has 128 rows; for d = 64 its one block of channels twice, the upper lanes are not read
  const uint64_t vt0 = tc::smem_desc(smem_addr(sm.stage[0][2]), D == 128 ? C * 128 : 0, 1024, tc::kSwizzle128);
  const uint64_t p0 = tc::smem_desc(smem_addr(sm.p), 16, 1024, tc::kSwizzle128);
  constexpr uint32_t kStage = 3 * SM::TILE / 16;
  auto scores = [&](int s) {
    if (ltc::elect_one()) {
#pragma unroll 1
      for (int b = 0; b < D / 64; ++b) {
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
          const uint32_t at = kStage * s + b * (C * 8) + ks * 2u;
          tc::mma_f16(T_SC, q0 + at, k0 + at, id_sc, b + ks > 0);
        }
      }
      tc::commit(&sm.sc_full);
    }
    __syncwarp();
  };
  bool ok = true;
  if (total > 0) {
    ok = wait_all(sm, &sm.full[0], 0);
    if (ok) scores(0);
  }
  int s = 0, turn = 0;                       // stage of chunk k and how often the stages went round
  for (int k = 0; k < total && ok; ++k) {
    const uint32_t par = (uint32_t)(k & 1);
    const int sn = s + 1 == NST ? 0 : s + 1, turn_n = s + 1 == NST ? turn + 1 : turn;
    if (k + 1 < total) {
      if (!(ok = wait_all(sm, &sm.sc_empty, par))) break;
      if (!(ok = wait_all(sm, &sm.full[sn], (uint32_t)(turn_n & 1)))) break;
      tc::fence_after_sync();
      scores(sn);
    }
    // the state before the chunk is in TMEM, and the last chunk's output has been read
    if (!(ok = wait_all(sm, &sm.s_full, par))) break;
    if (k > 0 && !(ok = wait_all(sm, &sm.o_empty, par ^ 1u))) break;
    tc::fence_after_sync();
    if (ltc::elect_one()) {
#pragma unroll 1
      for (int b = 0; b < D / 64; ++b)
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
          ltc::mma_ts(T_OI, T_S + 32u * b + 8u * ks, q0 + (kStage * s + b * (C * 8) + ks * 2u), id_oi, b + ks > 0);
    }
    __syncwarp();
    // P of this chunk, and zeros in its values behind the sequence's end
    if (!(ok = wait_all(sm, &sm.p_full, par))) break;
    tc::fence_after_sync();
    if (ltc::elect_one()) {
#pragma unroll 1
      for (int b = 0; b < 2; ++b)            // the parts of P one behind the other
#pragma unroll
        for (int ks = 0; ks < C / 16; ++ks)
          tc::mma_f16(T_OP, vt0 + (kStage * s + 128u * ks), p0 + b * (C * 8) + 2u * ks, id_op, b + ks > 0);
      tc::commit(&sm.op_full);
      tc::commit(&sm.empty[s]);
    }
    __syncwarp();
    s = sn;
    turn = turn_n;
  }
  if (!ok) gave_up(t, sm);
  drain<D>(sm, 1);
}

// ---- P, the value's parts, the output -------------------------------------------------
// Rows 16 qd .. + 15 of P from the scores x (this warp's 16 TMEM lanes as 16x256b fragments): times their decay, in two
// bf16 parts, x[2 c + ..] the upper ones of column block c (rows g, g + 8) and x[16 + 2 c + ..] the rest.  pz:
// &sm.pz[..][C], A^n at [n] and zeros below; sgn: 1 forwards, -1 backwards.
__device__ __forceinline__ void make_p(uint32_t (&x)[32], const float* pz, int sgn, int r, int qd, int lane) {
  const int g = lane >> 2, q = lane & 3;
  if (r < C) {                                   // scores of keys behind the sequence's end may be anything
#pragma unroll
    for (int y = 0; y < 32; ++y)
      if (8 * (y >> 2) + 2 * q + (y & 1) >= r) x[y] = 0u;
  }
  // age of (row 16 qd + g, column 8 c + 2 q): sgn (base - 8 c); the next column's is sgn less, and the row 8 below has
  // the age of the column block before
  const float* at = pz + sgn * (16 * qd + g - 2 * q + 8);
  float2 w0 = make_float2(at[0], at[-sgn]);
  uint32_t hi[16], lo[16];
  auto split = [](float2 v, uint32_t* h, uint32_t* l) {
    *h = ltc::pack_bf16(v.x, v.y);
    *l = ltc::pack_bf16(v.x - ltc::bf16_lo(*h), v.y - ltc::bf16_hi(*h));
  };
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    at -= 8 * sgn;
    const float2 w1 = make_float2(at[0], at[-sgn]);
    split(__fmul2_rn(make_float2(__uint_as_float(x[4 * c]), __uint_as_float(x[4 * c + 1])), w1), &hi[2 * c], &lo[2 * c]);
    split(__fmul2_rn(make_float2(__uint_as_float(x[4 * c + 2]), __uint_as_float(x[4 * c + 3])), w0), &hi[2 * c + 1], &lo[2 * c + 1]);
    w0 = w1;
  }
#pragma unroll
  for (int y = 0; y < 16; ++y) {
    x[y] = hi[y];
    x[16 + y] = lo[y];
    asm volatile("" : "+r"(x[y]), "+r"(x[16 + y]));      // made here, not behind the wait that follows
  }
}

// Tokens 32 th .. + 31 of the value tile, times their decay, transposed for TMEM lanes 32 qd .. + 31 (channels), two
// tokens a word, in PARTS bf16 parts.  v[part][16 channels of h][..]: words of token groups 0..3, channels g and g + 8.
//
// Three parts: the product in fp32 (wv: the two tokens' decays), cut off, not rounded: 8 bits each of its 24, so that
// their sum is the product.
//
// Two parts, all in packed bf16 (wv: both decays' first 8 bits w1, the next w2): x w1 = hi + r exactly (the rest of a
// rounded product fits bf16 and a fused multiply-add gives it), and mid = x w2 + r holds the product to 2^-17.  That is
// a third of the instructions; for three parts it would be as many as in fp32, with more registers (all spilled: 64
// ragged prompts 228 -> 276 us).
template <int PARTS>
__device__ __forceinline__ void value_parts(uint32_t (&v)[PARTS][2][8], uint32_t tile, const uint2* wv, int r, int th, int qd,
                                            int lane) {
  const int q = lane & 3;
  // lane's row address of an ldmatrix: matrix lane / 8 = (channels + 8 (m & 1), tokens + 8 (m >> 1)), row lane % 8
  const int m = lane >> 3, tt = lane & 7;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int ch = 32 * qd + 16 * h + 8 * (m & 1);
    const uint32_t at = tile + (ch >> 6) * (C * 128) + (32 * th + 8 * (m >> 1) + tt) * 128 + ((((ch & 63) >> 3) ^ tt) << 4);
    ltc::ldsm_x4_trans(at, v[0][h][0], v[0][h][1], v[0][h][2], v[0][h][3]);
    ltc::ldsm_x4_trans(at + 2048, v[0][h][4], v[0][h][5], v[0][h][6], v[0][h][7]);
  }
  if (r < C) {                                 // rows behind the sequence's end are somebody else's
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        const int i = 32 * th + 8 * (x >> 1) + 2 * q;
        v[0][h][x] = i >= r ? 0u : (i + 1 >= r ? v[0][h][x] & 0xffffu : v[0][h][x]);
      }
  }
  using B2 = __nv_bfloat162;
  auto b2 = [](uint32_t u) { return *reinterpret_cast<const B2*>(&u); };
  auto u32 = [](B2 b) { return *reinterpret_cast<const uint32_t*>(&b); };
  const float2 minus = make_float2(-1.f, -1.f);
#pragma unroll
  for (int x = 0; x < 8; ++x) {                // tokens 8 (x >> 1) + 2 q, + 1
    const uint2 w = wv[4 * (x >> 1) + q];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t e = v[0][h][x];
      if (PARTS == 2) {
        const B2 hi = __hmul2_rn(b2(e), b2(w.x));
        v[0][h][x] = u32(hi);
        v[1][h][x] = u32(__hfma2(b2(e), b2(w.y), __hfma2(b2(e), b2(w.x), __hneg2(hi))));
      } else {
        float2 p = __fmul2_rn(make_float2(ltc::bf16_lo(e), ltc::bf16_hi(e)),
                              make_float2(__uint_as_float(w.x), __uint_as_float(w.y)));
#pragma unroll
        for (int part = 0; part < PARTS; ++part) {
          const uint32_t a0 = __float_as_uint(p.x), a1 = __float_as_uint(p.y);
          v[part][h][x] = ltc::upper_halves(a0, a1);
          if (part + 1 < PARTS)
            p = __ffma2_rn(make_float2(__uint_as_float(a0 & 0xffff0000u), __uint_as_float(a1 & 0xffff0000u)), minus, p);
        }
      }
    }
  }
}

// The output of a chunk, the 32 channels of this warp's lanes: OP + weight * OI, in 64 rows of 64 bytes of shared memory
// whose 16-byte pieces are exchanged as a 64-byte swizzled tensor store wants them.  Sixteen tokens at a time; `read` is
// called when all accumulators have been read.
template <class F>
__device__ __forceinline__ void make_out(uint8_t* os, const float* wo, int qd, int lane, F read) {
  const int q = lane & 3, tok = 8 * (lane >> 4) + (lane & 7);       // tok: the row whose address this lane gives
  uint32_t oi[2][8], op[2][8];
  auto load = [&](int grp) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {                                   // 16 channels: g and g + 8; two tokens each of two blocks
      const uint32_t at = ((uint32_t)(32 * qd + 16 * h) << 16) + 16 * grp;
      ltc::ld_16x256b_x2(at + T_OI, oi[h]);
      ltc::ld_16x256b_x2(at + T_OP, op[h]);
    }
  };
#pragma unroll 1
  for (int grp = 0; grp < 4; ++grp) {
    load(grp);
    const float2 w0 = *reinterpret_cast<const float2*>(&wo[16 * grp + 2 * q]);
    const float2 w1 = *reinterpret_cast<const float2*>(&wo[16 * grp + 8 + 2 * q]);
    tc::wait_ld();
    if (grp == 3) read();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t m[4];
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const float2 v = __ffma2_rn(make_float2(__uint_as_float(oi[h][2 * y]), __uint_as_float(oi[h][2 * y + 1])), y < 2 ? w0 : w1,
                                    make_float2(__uint_as_float(op[h][2 * y]), __uint_as_float(op[h][2 * y + 1])));
        m[y] = ltc::pack_bf16(v.x, v.y);
      }
      // matrices: (channels + 0, block 0), (+ 8, 0), (+ 0, 1), (+ 8, 1); rows are tokens
      const int piece = 2 * h + ((lane >> 3) & 1);
      ltc::stsm_x4_trans(smem_addr(os) + (16 * grp + tok) * 64 + ((piece ^ ((tok >> 1) & 3)) << 4), m[0], m[1], m[2], m[3]);
    }
  }
}

// What the state's part of token i's output is multiplied by: forwards A^(i + 1), backwards A^(rows - 1 - i); of a full
// chunk, or (tail) of the sequence's last.
__device__ __forceinline__ void out_weights(float* wo, int i, const LinTc& t, const Item& it, int tail) {
  const int rows = tail ? it.rows(it.c1 - 1) : C;
  wo[i] = decay_pow(clamp_log_decay(t.a.log_decay[it.h]), t.a.walk[it.w].back ? max(rows - 1 - i, 0) : i + 1);
}

// Rows r .. of a tile, by `threads` threads.
template <int D>
__device__ __forceinline__ void zero_rows(uint8_t* tile, int r, int thread, int threads) {
  for (int y = thread; y < (C - r) * (D / 8); y += threads) {
    const int row = r + y / (D / 8), piece = y % (D / 8);
    *reinterpret_cast<uint4*>(tile + (piece >> 3) * (C * 128) + row * 128 + (piece & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
  }
}

// Warps 4-7 (th = 0) and 8-11 (th = 1): half of the tokens' value parts each.  They are made while U of the chunk before
// runs and stored when it is done.
template <int D, int PARTS, bool STATE_ONLY>
__device__ void value_role(const LinTc& t, LinSmem<D>& sm, int warp, int lane) {
  const int qd = warp & 3, th = (warp - 4) >> 2, tid = 32 * qd + lane;
  int k = 0, n_item = 0, s = 0;
  uint32_t turn = 0;                             // parity of stage s
  bool ok = true;
  for (int i = 0; i < item_rounds(t); ++i) {
    const Item it = item_of<STATE_ONLY>(t, sm.order, i);
    if (it.chunks() == 0) continue;
    const bool back = t.a.walk[it.w].back;
    uint2(*wv)[C / 4] = sm.wv[n_item & 1][th];
    ++n_item;
    if (tid < C / 2) {
      // forwards A^(rows - 1 - i), backwards A^(i + 1)
      const float g = clamp_log_decay(t.a.log_decay[it.h]);
      const int tail = tid >> 4, rows = tail ? it.rows(it.c1 - 1) : C;
      float w[2];
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int i = 32 * th + 2 * (tid & 15) + y;
        w[y] = i < rows ? decay_pow(g, back ? i + 1 : rows - 1 - i) : 0.f;
      }
      uint2 e = make_uint2(__float_as_uint(w[0]), __float_as_uint(w[1]));
      if (PARTS == 2) {
        e.x = ltc::pack_bf16(w[0], w[1]);
        e.y = ltc::pack_bf16(w[0] - ltc::bf16_lo(e.x), w[1] - ltc::bf16_hi(e.x));
      }
      wv[tail][tid & 15] = e;
    }
    if (tc::named_sync_any(1 + th, 128, !ok)) break;
    for (int c = 0; c < it.chunks(); ++c, ++k) {
      const int r = it.rows(chunk_at(it, back, c));
      if (!(ok = wait_all(sm, &sm.full[s], turn))) break;
      uint32_t v[PARTS][2][8];
      if (32 * qd < D) value_parts<PARTS>(v, smem_addr(sm.stage[s][2]), wv[r < C], r, th, qd, lane);
      if (r < C) {
        // keys behind the sequence's end: zeros, for products of theirs with zeros must be zero
        zero_rows<D>(sm.stage[s][1], r, tid + 128 * th, 256);
        fence_proxy_async_smem();
      }
      const int b = buffer_of<STATE_ONLY>(k);
      // the parts that were there have been used
      if (used_before<STATE_ONLY>(k) && !(ok = wait_all(sm, &sm.u_full[b], phase_of<STATE_ONLY>(k) ^ 1u))) break;
      tc::fence_after_sync();
      if (32 * qd < D) {
#pragma unroll
        for (int part = 0; part < PARTS; ++part) {
#pragma unroll
          for (int h = 0; h < 2; ++h)
            ltc::st_16x128b_x4(((uint32_t)(32 * qd + 16 * h) << 16) + t_v<STATE_ONLY>(k) + 32u * part + 16u * th,
                               v[part][h]);
        }
        ltc::wait_st();
      }
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) {
        tc::mbar_arrive(&sm.v_full[b]);
        tc::mbar_arrive(&sm.empty[s]);
      }
      if (++s == NST) {
        s = 0;
        turn ^= 1u;
      }
    }
  }
  if (!ok) gave_up(t, sm);
}

// Warps 12-15: P from the scores.
template <int D>
__device__ void score_role(const LinTc& t, LinSmem<D>& sm, int warp, int lane) {
  const int qd = warp & 3, tid = 32 * qd + lane;
  int k = 0, n_item = 0;
  bool ok = true;
  for (int i = 0; i < item_rounds(t); ++i) {
    const Item it = item_of<false>(t, sm.order, i);
    if (it.chunks() == 0) continue;
    const bool back = t.a.walk[it.w].back;
    float* pz = sm.pz[n_item & 1];
    ++n_item;
    pz[tid] = tid < C ? 0.f : decay_pow(clamp_log_decay(t.a.log_decay[it.h]), tid - C);
    if (tid < 8) pz[2 * C + tid] = 0.f;
    if (tc::named_sync_any(3, 128, !ok)) break;
    for (int c = 0; c < it.chunks(); ++c, ++k) {
      if (!(ok = wait_all(sm, &sm.sc_full, (uint32_t)(k & 1)))) break;
      tc::fence_after_sync();
      uint32_t x[32];
      tc::ld_16x256b_x8(((uint32_t)(32 * qd) << 16) + T_SC, x);
      tc::wait_ld();
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&sm.sc_empty);
      const int r = it.rows(chunk_at(it, back, c));
      if (r < C) zero_rows<D>(sm.stage[k % NST][2], r, tid, 128);      // values behind the sequence's end, as the keys
      make_p(x, pz + C, back ? -1 : 1, r, qd, lane);
      if (k > 0 && !(ok = wait_all(sm, &sm.op_full, (uint32_t)((k - 1) & 1)))) break;     // the last P has been used
      tc::fence_after_sync();
      // matrices: (rows 0-7, block y), (rows 8-15, block y), (rows 0-7, block y + 1), (rows 8-15, block y + 1)
      const uint32_t row = 16 * qd + (lane & 15), to = smem_addr(sm.p) + row * 128;
#pragma unroll
      for (int y = 0; y < 8; y += 2) {
        const uint32_t piece = ((y + (lane >> 4)) ^ (row & 7)) << 4;
        ltc::stsm_x4(to + piece, x[2 * y], x[2 * y + 1], x[2 * y + 2], x[2 * y + 3]);
        ltc::stsm_x4(to + C * 128 + piece, x[16 + 2 * y], x[17 + 2 * y], x[18 + 2 * y], x[19 + 2 * y]);
      }
      fence_proxy_async_smem();
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&sm.p_full);
    }
  }
  if (!ok) gave_up(t, sm);
}

// Warps 16-19: the outputs.
template <int D>
__device__ void out_role(const LinTc& t, const LinMaps& maps, LinSmem<D>& sm, int warp, int lane) {
  const int qd = warp & 3, tid = 32 * qd + lane;
  int k = 0, n_item = 0;
  bool ok = true;
  uint8_t* os = sm.o[qd];
  for (int i = 0; i < item_rounds(t); ++i) {
    const Item it = item_of<false>(t, sm.order, i);
    if (it.chunks() == 0) continue;
    const LinWalk& w = t.a.walk[it.w];
    float(*wo)[C] = sm.wo[n_item & 1];
    ++n_item;
    out_weights(wo[tid >> 6], tid & 63, t, it, tid >> 6);
    if (tc::named_sync_any(4, 128, !ok)) break;
    for (int c = 0; c < it.chunks(); ++c, ++k) {
      const int ch = chunk_at(it, w.back, c), r = it.rows(ch), row = it.begin + ch * C;
      if (lane == 0) tc::bulk_wait_read_all();     // the last tile's store has left the buffer
      if (!(ok = wait_all(sm, &sm.op_full, (uint32_t)(k & 1)))) break;
      tc::fence_after_sync();
      auto read = [&] {
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&sm.o_empty);
      };
      if (32 * qd >= D) {
        read();
        continue;
      }
      make_out(os, wo[r < C], qd, lane, read);
      fence_proxy_async_smem();
      __syncwarp();
      if (r == C) {
        if (lane == 0) {
          tc::tensor_store_2d(&maps.out[it.w], smem_addr(os), it.h * D + 32 * qd, row);
          tc::bulk_commit_group();
        }
      } else {
        // the rows behind the end are not ours
        for (int y = lane; y < r * 4; y += 32) {
          const int j = y >> 2, piece = y & 3;
          uint16_t* dst = reinterpret_cast<uint16_t*>(w.out) + (size_t)(row + j) * w.out_stride + it.h * D + 32 * qd + 8 * piece;
          *reinterpret_cast<uint4*>(dst) = *reinterpret_cast<const uint4*>(os + j * 64 + ((piece ^ ((j >> 1) & 3)) << 4));
        }
        __syncwarp();
      }
    }
  }
  if (lane == 0) tc::bulk_wait_all();
  if (!ok) gave_up(t, sm);
}

// ---- state ---------------------------------------------------------------------------
// What `rows` tokens leave of the state.  Half of it or more: S + m S, m = A^rows - 1, which keeps what a product with
// A^rows, rounded to 24 bits, would lose chunk after chunk.  Less: the product m S, m = A^rows, off by 2^-24 of what is
// left, where A^rows - 1, rounded, would be off by 2^-25 of what was there (1 % of what g = -0.2 leaves of a chunk).
struct Fade {
  float m;
  bool rest;
};
__device__ __forceinline__ Fade fade_of(float g, int rows) {
  const float p = g * (float)rows;
  const bool rest = p > -0.6931f;
  return {rest ? expm1f(p) : expf(p), rest};
}

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

// This thread's part of the state (row e of its half of the key channels) exchanged for what lies in shared memory.  Both ways
// in every case: where one is not wanted, what is read is not used, or what is written not stored; a choice made this code,
// unrolled over the registers that hold the state, a third of the kernel's (training gradients 878 us, so 783).
// Rows of 128 bytes whose 16-byte pieces are exchanged by the row's low bits: the lanes of a row-wise access fall in
// distinct banks, as those of a column-wise one (`swap`: the state lies transposed) do anyway.
template <int D>
__device__ __forceinline__ void exchange_state(float (&S)[D / 2], uint8_t* st, int e, bool swap) {
  constexpr int HC = D / 2;
  if (!swap) {
    uint8_t* row = st + e * 128;
#pragma unroll
    for (int j = 0; j < HC; j += 4) {
      float4* at = reinterpret_cast<float4*>(row + (j / 32) * (D * 128) + ((((j % 32) / 4) ^ (e & 7)) << 4));
      const float4 x = *at;
      *at = make_float4(S[j], S[j + 1], S[j + 2], S[j + 3]);
      S[j] = x.x, S[j + 1] = x.y, S[j + 2] = x.z, S[j + 3] = x.w;
    }
  } else {
    uint8_t* col = st + (e >> 5) * (D * 64) + (e & 3) * 4;
    const int piece = (e & 31) >> 2;
#pragma unroll
    for (int j = 0; j < HC; ++j) {
      float* at = reinterpret_cast<float*>(col + j * 128 + ((piece ^ (j & 7)) << 4));
      const float x = *at;
      *at = S[j];
      S[j] = x;
    }
  }
}

template <int D, bool STATE_ONLY>
__device__ void state_role(const LinTc& t, LinSmem<D>& sm, int warp, int lane) {
  constexpr int HC = D / 2;                                  // key channels of a thread
  const int qd = warp & 3, half = (warp - 20) >> 2, e = 32 * qd + lane;
  const bool mine = 32 * qd < D;                             // lanes beyond d hold nothing
  const uint32_t lane_addr = (uint32_t)(32 * qd) << 16;
  int k = 0;
  uint32_t round = 0;
  bool ok = true;
  float S[HC];
  StateIo last_io = {false, false, false, false};
#pragma unroll
  for (int j = 0; j < HC; ++j) S[j] = 0.f;
  // one round more than there are items: the last one's state goes out
#pragma unroll 1
  for (int i = 0; i <= item_rounds(t); ++i) {
    const bool end = i == item_rounds(t);
    if (end && !last_io.out) break;
    const Item it = item_of<STATE_ONLY>(t, sm.order, i);
    if (!it.on && !end) continue;
    StateIo io = {false, false, false, false};
    if (!end) io = state_io<STATE_ONLY>(t, it);
    const bool back = t.a.walk[it.w].back, two = two_rounds(last_io, io);
#pragma unroll 1
    for (int turn = two ? 0 : 1; turn < 2; ++turn) {
      if (!(ok = wait_all(sm, &sm.st_full[half], round++ & 1u))) break;
      if (mine && (io.in || last_io.out)) exchange_state<D>(S, sm.st, e, turn && io.in ? io.in_swap : last_io.out_swap);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&sm.st_done[half]);
    }
    if (end || !ok) break;
    last_io = io;
    if (!io.in) {
#pragma unroll
      for (int j = 0; j < HC; ++j) S[j] = 0.f;
    }
    const float g = clamp_log_decay(t.a.log_decay[it.h]);
    const Fade full = fade_of(g, C);
    for (int c = 0; c < it.chunks(); ++c, ++k) {
      const int ch = chunk_at(it, back, c), r = it.rows(ch);
      const uint32_t par = (uint32_t)(k & 1);
      if (c == 0 && !STATE_ONLY) {
        // the state before the first chunk; the last item's products have been waited for
        if (mine) state_to_tmem<D>(S, lane_addr + T_S + (HC / 2) * half);
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&sm.s_full);
      }
      if (mine) {        // while U runs
        const Fade f = r < C ? fade_of(g, r) : full;
        const float2 m2 = make_float2(f.m, f.m);
        if (f.rest) {
#pragma unroll
          for (int j = 0; j < HC; j += 2) {
            const float2 s2 = make_float2(S[j], S[j + 1]), n2 = __ffma2_rn(s2, m2, s2);
            S[j] = n2.x;
            S[j + 1] = n2.y;
          }
        } else {
#pragma unroll
          for (int j = 0; j < HC; j += 2) {
            const float2 n2 = __fmul2_rn(make_float2(S[j], S[j + 1]), m2);
            S[j] = n2.x;
            S[j + 1] = n2.y;
          }
        }
#pragma unroll
        for (int j = 0; j < HC; ++j) asm volatile("" : "+f"(S[j]));
      }
      if (!(ok = wait_all(sm, &sm.u_full[buffer_of<STATE_ONLY>(k)], phase_of<STATE_ONLY>(k)))) break;
      tc::fence_after_sync();
#pragma unroll
      for (int j0 = 0; j0 < HC; j0 += 16) {
        uint32_t u[16];
        if (mine) {
          tc::ld_32x32b_x16(lane_addr + t_u<STATE_ONLY>(k) + HC * half + j0, u);
          tc::wait_ld();
        }
        if (j0 + 16 == HC) {         // U may be written again
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&sm.u_empty[buffer_of<STATE_ONLY>(k)]);
        }
        if (mine) {
#pragma unroll
          for (int j = 0; j < 16; j += 2) {
            const float2 n2 = __fadd2_rn(make_float2(S[j0 + j], S[j0 + j + 1]),
                                         make_float2(__uint_as_float(u[j]), __uint_as_float(u[j + 1])));
            S[j0 + j] = n2.x;
            S[j0 + j + 1] = n2.y;
          }
        }
      }
      if (STATE_ONLY) continue;
      if (!(ok = wait_all(sm, &sm.op_full, par))) break;          // the last copy has been used
      tc::fence_after_sync();
      if (c + 1 < it.chunks()) {
        if (mine) state_to_tmem<D>(S, lane_addr + T_S + (HC / 2) * half);
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&sm.s_full);
      }
    }
    if (!ok) break;
  }
  if (!ok) gave_up(t, sm);
}

// A block in which a wait gave up leaves NaN in all that its items were to write, so that nobody takes what lies there for
// results (a stretch's state hands them on to the stretches behind it).  Threads 0 .. 255 of the state's warps, when every
// store of the block has completed.  (Rolled loops: the kernel is short of room for instructions.)
template <int D, bool STATE_ONLY>
__device__ void spoil(const LinTc& t, const LinSmem<D>& sm, int thread) {
#pragma unroll 1
  for (int i = 0; i < item_rounds(t); ++i) {
    const Item it = item_of<STATE_ONLY>(t, sm.order, i);
    if (!it.on) continue;
    const LinWalk& w = t.a.walk[it.w];
    if (!STATE_ONLY) {
      const int r0 = it.begin + it.c0 * C, rows = min(it.len - it.c0 * C, (it.c1 - it.c0) * C);
#pragma unroll 1
      for (int64_t x = thread; x < (int64_t)rows * (D / 8); x += 256) {
        uint16_t* dst = reinterpret_cast<uint16_t*>(w.out) + (r0 + x / (D / 8)) * w.out_stride + it.h * D + 8 * (x % (D / 8));
        *reinterpret_cast<uint4*>(dst) = make_uint4(0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu);
      }
    }
    if (state_io<STATE_ONLY>(t, it).out) {
      float* S = STATE_ONLY ? t.ws + stretch_index(t.a, t.split, it.w, it.n, it.h, it.seg) * (D * D)
                            : w.S_out + ((int64_t)it.n * t.a.H + it.h) * (D * D);
#pragma unroll 1
      for (int x = thread; x < D * D; x += 256) S[x] = __int_as_float(0x7fffffff);
    }
  }
}

template <int D, int PARTS, bool STATE_ONLY>
__global__ void __launch_bounds__(kTcThreads, 1)
    linattn_tc_kernel(const __grid_constant__ LinTc t, const __grid_constant__ LinMaps maps) {
  using SM = LinSmem<D>;
  extern __shared__ uint8_t smem_raw[];
  SM& sm = *reinterpret_cast<SM*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int s = 0; s < NST; ++s) {
      mbar_init(&sm.full[s], 1);
      mbar_init(&sm.empty[s], STATE_ONLY ? 9 : 10);     // the products' warps, and the eight that read the values
    }
    mbar_init(&sm.sc_full, 1);
    mbar_init(&sm.p_full, 4);
    mbar_init(&sm.s_full, 8);
    for (int b = 0; b < 2; ++b) {
      mbar_init(&sm.v_full[b], 8);
      mbar_init(&sm.u_full[b], 1);
      mbar_init(&sm.u_empty[b], 8);
    }
    mbar_init(&sm.op_full, 1);
    mbar_init(&sm.o_empty, 4);
    for (int h = 0; h < 2; ++h) {
      mbar_init(&sm.st_full[h], 1);
      mbar_init(&sm.st_done[h], 4);
    }
    mbar_init(&sm.drain[0], 1);
    mbar_init(&sm.drain[1], 1);
    mbar_init(&sm.sc_empty, 4);
    sm.bad = 0;
    sm.tries = t.tries;
    fence_mbar_init();
  }
  if (warp == 1) tc::tmem_alloc(&sm.taddr, 512);
  order_sequences<D>(t, sm);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  // registers: 896 threads x 72 at launch hold 128 x (40 + 72 + 72 + 64 + 48 + 104 + 104)
  if (warp < 4) {
    ltc::regs_down<40>();
    if (warp == 0) {
      if (lane == 0) load_role<D, STATE_ONLY>(t, maps, sm);
      __syncwarp();
    } else if (warp == 1) {
      update_role<D, PARTS, STATE_ONLY>(t, sm, chunks_of_block<D, STATE_ONLY>(t, sm));
    } else if (warp == 2) {
      if (lane == 0) state_io_role<D, STATE_ONLY>(t, maps, sm);
      __syncwarp();
    } else if (!STATE_ONLY) {
      output_mma_role<D>(t, sm, chunks_of_block<D, STATE_ONLY>(t, sm));
    }
    tc::named_sync(5, kTcThreads);
  } else if (warp < 12) {
    value_role<D, PARTS, STATE_ONLY>(t, sm, warp, lane);
    tc::named_sync(5, kTcThreads);
  } else if (warp < 16) {
    ltc::regs_down<64>();
    if (!STATE_ONLY) score_role<D>(t, sm, warp, lane);
    tc::named_sync(5, kTcThreads);
  } else if (warp < 20) {
    ltc::regs_down<48>();
    if (!STATE_ONLY) out_role<D>(t, maps, sm, warp, lane);
    tc::named_sync(5, kTcThreads);
  } else {
    ltc::regs_up<104>();
    state_role<D, STATE_ONLY>(t, sm, warp, lane);
    tc::named_sync(5, kTcThreads);           // every role is through, its stores completed
    if (*reinterpret_cast<volatile int*>(&sm.bad)) spoil<D, STATE_ONLY>(t, sm, tid - 640);
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == 1) tc::tmem_free(sm.taddr, 512);
}

// ---- launch ----------------------------------------------------------------------------
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

// rows of `width` bf16, `stride` elements apart, in boxes of `high` rows of `inner` (64 or 32) elements
bool make_map(CUtensorMap* m, const void* p, int64_t width, int64_t stride, int64_t rows, int inner, int high) {
  EncodeFn encode = encode_fn();
  if (!encode) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)width, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)stride * 2};
  const cuuint32_t box[2] = {(cuuint32_t)inner, (cuuint32_t)high};
  const cuuint32_t estr[2] = {1, 1};
  return encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(p), dims, strides, box, estr,
                CU_TENSOR_MAP_INTERLEAVE_NONE, inner == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// states: `count` of D rows of D fp32, in boxes of 32 columns by D rows, or (transposed) by D / 2
bool make_state_map(CUtensorMap* m, const void* p, int D, int64_t count, bool swap) {
  EncodeFn encode = encode_fn();
  if (!encode) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)D, (cuuint64_t)(count * D)};
  const cuuint64_t strides[1] = {(cuuint64_t)D * 4};
  const cuuint32_t box[2] = {32, (cuuint32_t)(swap ? D / 2 : D)};
  const cuuint32_t estr[2] = {1, 1};
  return encode(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, const_cast<void*>(p), dims, strides, box, estr,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int PARTS>
cudaError_t launch_tc(const LinTc& t0, const LinMaps& maps, cudaStream_t st) {
  LinTc t = t0;
  const size_t smem = sizeof(LinSmem<D>) + 1024;
  static_assert(sizeof(LinSmem<D>) + 1024 <= 232448, "shared memory");
  static bool allowed[2][64];
  cudaError_t e = allow_shared(linattn_tc_kernel<D, PARTS, false>, (int)smem, allowed[0]);
  if (e != cudaSuccess) return e;
  const unsigned blocks = (unsigned)(t.items < kSms ? t.items : kSms);
  if (t.split.stretches > 1) {
    e = allow_shared(linattn_tc_kernel<D, PARTS, true>, (int)smem, allowed[1]);
    if (e != cudaSuccess) return e;
    linattn_tc_kernel<D, PARTS, true><<<blocks, kTcThreads, smem, st>>>(t, maps);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    if ((e = launch_linattn_chain(t.a, t.split, t.ws, st)) != cudaSuccess) return e;
  }
  linattn_tc_kernel<D, PARTS, false><<<blocks, kTcThreads, smem, st>>>(t, maps);
  return cudaGetLastError();
}

}  // namespace

LinSplit linattn_tc_split(int64_t heads, int64_t max_len, int walks) {
  const int64_t items = heads * walks;
  // stretches of 8 chunks at least, two rounds of the SMs at most
  return lin_split(items, max_len, items >= kSms ? 0 : 2 * kSms, 8, 2);
}

bool linattn_tc_takes(const LinArgs& a) {
  if (a.io != PACE_IO_BF16 || (a.D != 64 && a.D != 128) || a.total == 0) return false;
  // rows of the states, as a tensor load's coordinate
  if ((int64_t)a.N * a.H * a.D > 0x7fffffffll) return false;
  for (int w = 0; w < a.walks; ++w) {
    const LinWalk& k = a.walk[w];
    if (((uintptr_t)k.query | (uintptr_t)k.key | (uintptr_t)k.value | (uintptr_t)k.out) % 16) return false;
    if ((k.query_stride | k.key_stride | k.value_stride | k.out_stride) % 8) return false;
  }
  return true;
}

static std::atomic<uint32_t> g_wait_tries{ltc::kWaitTries}, g_extra_tx{0};
void linattn_tc_debug(uint32_t wait_tries, uint32_t extra_tx) {
  g_wait_tries = wait_tries ? wait_tries : ltc::kWaitTries;
  g_extra_tx = extra_tx;
}

cudaError_t launch_linattn_tc(const LinArgs& a, const LinSplit& sp, float* ws, cudaStream_t st) {
  LinTc t;
  t.tries = g_wait_tries;
  t.extra_tx = g_extra_tx;
  LinMaps maps;
  t.a = a;
  t.split = sp;
  t.ws = ws;
  const int64_t items = (int64_t)a.N * a.H * sp.stretches;
  if (items * a.walks > 0x7fff0000ll) return cudaErrorInvalidValue;
  t.items = (int32_t)(items * a.walks);
  // the tensors of all walks, each mapped once
  struct Seen { const void* p; int64_t stride; } seen[4];
  int n = 0;
  auto index = [&](const void* p, int64_t stride) {
    for (int i = 0; i < n; ++i)
      if (seen[i].p == p && seen[i].stride == stride) return i;
    if (n == 4 || !make_map(&maps.in[n], p, (int64_t)a.H * a.D, stride, a.total, 64, C)) return -1;
    seen[n] = Seen{p, stride};
    return n++;
  };
  for (int w = 0; w < a.walks; ++w) {
    t.map_q[w] = index(a.walk[w].query, a.walk[w].query_stride);
    t.map_k[w] = index(a.walk[w].key, a.walk[w].key_stride);
    t.map_v[w] = index(a.walk[w].value, a.walk[w].value_stride);
    if (t.map_q[w] < 0 || t.map_k[w] < 0 || t.map_v[w] < 0) return cudaErrorInvalidValue;
    if (!make_map(&maps.out[w], a.walk[w].out, (int64_t)a.H * a.D, a.walk[w].out_stride, a.total, 32, C)) return cudaErrorInvalidValue;
  }
  for (int w = 0; w < a.walks; ++w) {
    if (a.walk[w].S_in && !make_state_map(&maps.s_in[w], a.walk[w].S_in, a.D, (int64_t)a.N * a.H, a.walk[w].swap)) return cudaErrorInvalidValue;
    if (a.walk[w].S_out && !make_state_map(&maps.s_out[w], a.walk[w].S_out, a.D, (int64_t)a.N * a.H, a.walk[w].swap)) return cudaErrorInvalidValue;
  }
  if (sp.stretches > 1 && !make_state_map(&maps.ws, ws, a.D, items * a.walks, false)) return cudaErrorInvalidValue;
  // gradients without dS0 are bf16 all; the forward operator's outputs do not depend on whether ST is wanted
  const bool two = a.walks > 1 && !a.walk[0].S_out && !a.walk[1].S_out && !a.walk[2].S_out;
  if (two) return a.D == 128 ? launch_tc<128, 2>(t, maps, st) : launch_tc<64, 2>(t, maps, st);
  return a.D == 128 ? launch_tc<128, 3>(t, maps, st) : launch_tc<64, 3>(t, maps, st);
}

}  // namespace pace
