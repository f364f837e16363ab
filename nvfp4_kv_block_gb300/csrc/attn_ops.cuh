// Device helpers of the attention kernels over NVFP4 pages on tcgen05 (tree_attn.cu,
// prefill.cu): waits of a whole warp, matrix instructions with P in tensor memory, packed
// fp32 arithmetic, and the conversion of codes to FP8 and f16 operands.
#pragma once

#include <cuda_bf16.h>

#include "common.cuh"

namespace msa {

__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(r));
  return r != 0;
}
// Waits (the whole warp) for the phase with the given parity: as mbar_wait, bounded in
// time and given up when another role has, but short in code (there are thirty of them).
__device__ __forceinline__ bool twait(uint32_t bar, uint32_t parity, const WaitCtl& w) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  const unsigned long long t0 = globaltimer_ns();
  for (;;) {
#pragma unroll 1
    for (int i = 0; i < 16; ++i)
      if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    if (__any_sync(0xffffffffu, *w.abort || globaltimer_ns() - t0 > w.limit_ns)) {
      *w.abort = 1;
      return false;
    }
  }
}
// One poll without mbar_try_wait's hint.
__device__ __forceinline__ bool mbar_poll(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// Waits as twait does, without the hint: a hand-over between two warps takes 112 cycles, 142 with it.  (A poll
// answers each lane for itself; a vote at every poll keeps the warp together.  Lanes that poll alone and vote once
// at the end need 170.)
__device__ __forceinline__ bool swait(uint32_t bar, uint32_t parity, const WaitCtl& w) {
  if (__all_sync(0xffffffffu, mbar_poll(bar, parity))) return true;
  const unsigned long long t0 = globaltimer_ns();
  for (;;) {
#pragma unroll 1
    for (int i = 0; i < 64; ++i)
      if (__all_sync(0xffffffffu, mbar_poll(bar, parity))) return true;
    if (__any_sync(0xffffffffu, *w.abort || globaltimer_ns() - t0 > w.limit_ns)) {
      *w.abort = 1;
      return false;
    }
  }
}
__device__ __forceinline__ void tmem_st_x16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
      ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// kind::f16 with A in tensor memory (row m in lane m, two f16 per column), B in shared memory.
__device__ __forceinline__ void umma_f16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
// Shared memory by 32-bit address (every access in program order).
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds_u8(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void sts128(uint32_t a, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
template <int N>
__device__ __forceinline__ void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
__device__ __forceinline__ uint64_t pair64(uint32_t a, uint32_t b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint2 split64(uint64_t x) {
  uint2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=r"(r.x), "=r"(r.y) : "l"(x));
  return r;
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
// OR of a predicate over the threads of a named barrier (all of them wait).
__device__ __forceinline__ bool barrier_or(int id, int nthreads, bool pred) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n bar.red.or.pred q, %2, %3, p;\n"
      " selp.u32 %0, 1, 0, q;\n}"
      : "=r"(r)
      : "r"((uint32_t)pred), "r"(id), "r"(nthreads)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// One code word (8 channels) -> 8 f16 values v8 2^-8, through the scale's table:
// hi = E4M3 magnitude bits >> 1, lo = their last bit << 7, per E2M1 magnitude.
__device__ __forceinline__ uint4 dequant8_f16(uint32_t w, uint4 t) {
  const uint32_t m = w & 0x77777777u, m2 = m >> 16;
  const uint32_t h0 = prmt(t.x, t.y, m) | (w & 0x80808080u);
  const uint32_t h1 = prmt(t.x, t.y, m2) | ((w << 4) & 0x80808080u);
  const uint32_t l0 = prmt(t.z, t.w, m), l1 = prmt(t.z, t.w, m2);
  return make_uint4(prmt(l0, h0, 0x5140u), prmt(l0, h0, 0x7362u), prmt(l1, h1, 0x5140u), prmt(l1, h1, 0x7362u));
}

// Tables of scale byte sb (0 .. 127): K's E4M3 bytes of the eight magnitudes, V's halves for
// dequant8_f16, each in as many copies as lanes read it from banks of their own.
template <int kKCopies, int kVCopies>
__device__ __forceinline__ void convert_tables(int sb, uint2* kt, uint4* vt) {
  const float mags[8] = {0.f, 0.5f, 1.f, 1.5f, 2.f, 3.f, 4.f, 6.f};
  // (0x7F is no number and never written: it counts as zero)
  const float s = sb == 127 ? 0.f : e4m3_to_f32((uint32_t)sb);
  uint32_t k[2] = {0, 0}, hi[2] = {0, 0}, lo[2] = {0, 0};
#pragma unroll
  for (int m = 0; m < 8; ++m) {
    const uint32_t e = f32_to_e4m3(mags[m] * s);
    k[m >> 2] |= e << (8 * (m & 3));
    hi[m >> 2] |= (e >> 1) << (8 * (m & 3));
    lo[m >> 2] |= ((e & 1) << 7) << (8 * (m & 3));
  }
#pragma unroll
  for (int c = 0; c < kKCopies; ++c) kt[sb * kKCopies + c] = make_uint2(k[0], k[1]);
#pragma unroll
  for (int c = 0; c < kVCopies; ++c) vt[sb * kVCopies + c] = make_uint4(hi[0], hi[1], lo[0], lo[1]);
}

__device__ __forceinline__ uint32_t pack16(float a, float b, bool f16) {
  if (f16) return cvt_f16x2_f32(b, a);
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

}  // namespace msa
