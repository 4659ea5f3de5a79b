// What the tensor-memory kernel of the linear attention needs beside tc.cuh:
// bf16 products with the A operand in TMEM, TMEM stores, 2-D tensor loads.
#pragma once

#include "linattn.cuh"
#include "tc.cuh"

namespace pace {
namespace ltc {

// Instruction descriptor: bf16 x bf16 -> f32, M x N, each operand K-major (0) or MN-major (1).
__host__ __device__ constexpr uint32_t idesc_bf16(int M, int N, int a_mn, int b_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) | ((uint32_t)(N >> 3) << 17) |
         ((uint32_t)(M >> 4) << 24);
}

// D[tmem] (+)= A * B with A in TMEM, issued by one thread.  A: row r in lane r, two bf16 of the contraction a column.
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
      : "memory");
}
// One thread of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
  return r != 0;
}

// 32x32b.x16: thread t of the warp writes lane (base + t), 16 consecutive columns.
__device__ __forceinline__ void st_32x32b_x16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// 16x256b.x2: lanes base..base+15, 16 columns; thread (g = t/4, q = t%4) gets, for column block c (8
// columns), r[4c], r[4c + 1] = lane g, columns 8c + 2q, + 1; r[4c + 2], r[4c + 3] = the same of lane g + 8.
__device__ __forceinline__ void ld_16x256b_x2(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}
// 16x128b.x4: lanes base..base+15, 16 columns; thread (g = t/4, q = t%4) writes, for column block c (4 columns),
// r[2c] = lane g, column 4c + q; r[2c + 1] = the same of lane g + 8.
__device__ __forceinline__ void st_16x128b_x4(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
// Wait for phase `parity` of `bar`; false after kWaitTries tests (or the debug limit).  The first test is
// one without a time limit, which costs 52 cycles where the phase is complete (133 with one); a later one suspends the
// thread for at most 10 us, so that giving up takes 2 s at most and, should no test suspend, still some milliseconds: far
// above what a chunk takes, which is what a wait of this kernel may last (the one that lasts an item has a budget for each
// of its chunks).
constexpr uint32_t kWaitTries = 200000;
// sm.tries: that number, in shared memory, so that a phase that is complete costs no more than its test.
template <class SM>
__device__ __forceinline__ bool wait_tries(const SM& sm, uint64_t* bar, uint32_t parity) {
  uint32_t left;
  asm volatile(
      "{\n .reg .pred p, z;\n mov.u32 %0, 1;\n"
      " mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n @p bra DONE_%=;\n"
      " ld.shared.u32 %0, [%3+%4];\n"
      "WAIT_%=:\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %5;\n @p bra DONE_%=;\n"
      " sub.u32 %0, %0, 1;\n setp.ne.u32 z, %0, 0;\n @z bra WAIT_%=;\nDONE_%=:\n}\n"
      : "=&r"(left)
      : "r"(smem_addr(bar)), "r"(parity), "r"(smem_addr(&sm)), "n"(offsetof(SM, tries)), "r"(10000u)
      : "memory");
  return left != 0;
}
// Four 8 x 8 matrices of 16-bit elements, transposed; threads 8m .. 8m + 7 give the row addresses of matrix m.
// Loaded: thread (g, q) gets in r[m] the elements [row 2q][column g] (low half) and [row 2q + 1][column g].
__device__ __forceinline__ void ldsm_x4_trans(uint32_t row_addr, uint32_t& r0, uint32_t& r1, uint32_t& r2, uint32_t& r3) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
               : "r"(row_addr)
               : "memory");
}
// Stored: thread (g, q)'s r[m] holds [row g][columns 2q, 2q + 1], or (trans) [rows 2q, 2q + 1][column g].
__device__ __forceinline__ void stsm_x4(uint32_t row_addr, uint32_t r0, uint32_t r1, uint32_t r2, uint32_t r3) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(row_addr), "r"(r0), "r"(r1),
               "r"(r2), "r"(r3)
               : "memory");
}
__device__ __forceinline__ void stsm_x4_trans(uint32_t row_addr, uint32_t r0, uint32_t r1, uint32_t r2, uint32_t r3) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(row_addr), "r"(r0),
               "r"(r1), "r"(r2), "r"(r3)
               : "memory");
}
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Box at (x, y) of a 2-D map into shared memory, completed on `bar` (no multicast).
__device__ __forceinline__ void tensor_load_2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
      "l"(map), "r"(smem_addr(bar)), "r"(x), "r"(y)
      : "memory");
}
// A warpgroup's share of the block's registers.
template <int N>
__device__ __forceinline__ void regs_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void regs_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// the upper halves of two words: lo's below, hi's above
__device__ __forceinline__ uint32_t upper_halves(uint32_t lo, uint32_t hi) { return __byte_perm(lo, hi, 0x7632); }
__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

}  // namespace ltc

LinSplit linattn_tc_split(int64_t heads, int64_t max_len, int walks);
bool linattn_tc_takes(const LinArgs& a);
cudaError_t launch_linattn_tc(const LinArgs& a, const LinSplit& sp, float* ws, cudaStream_t st);
void linattn_tc_debug(uint32_t wait_tries, uint32_t extra_tx);     // 0, 0: the defaults

}  // namespace pace
