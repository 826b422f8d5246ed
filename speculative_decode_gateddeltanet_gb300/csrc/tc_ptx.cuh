// The 5th-generation tensor cores, TMA and mbarriers as the attention kernels use them: PTX by name, waits that are bounded
// by time, operand layouts and tensor maps of paged pools.
#pragma once
#include <cuda.h>

#include "attn_common.cuh"

namespace gdnattn {

constexpr int kTcRows = 128;  // M of every product
#ifndef GDN_WAIT_LIMIT_NS
#define GDN_WAIT_LIMIT_NS 500000000ull
#endif
constexpr unsigned long long kWaitNs = GDN_WAIT_LIMIT_NS;

__device__ __forceinline__ uint32_t smem_addr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

__device__ __forceinline__ void bar_init(uint32_t bar, int count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
// one arrival for the warp, behind all its lanes' work (32 arrivals on one word are 32 shared-memory atomics in a row)
__device__ __forceinline__ void warp_arrive(uint32_t bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) bar_arrive(bar);
}
__device__ __forceinline__ void bar_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
// One try suspends the warp for up to a millisecond: a poll is a shared-memory access, and warps that poll at full
// speed take that bandwidth from the MMA's operands.
__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\tselp.b32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity), "r"(1000000u)
      : "memory");
  return ok;
}
__device__ __forceinline__ unsigned long long now_ns() {
  unsigned long long t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}

// false when the wait ran out or another role gave up
__device__ __forceinline__ bool bar_wait_slow(uint32_t bar, uint32_t parity, volatile int* gave_up) {
  const unsigned long long end = now_ns() + kWaitNs;
  while (!bar_try(bar, parity)) {
    if (*gave_up) return false;
    if (now_ns() > end) {
      *gave_up = 1;
      return false;
    }
  }
  return true;
}
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, volatile int* gave_up) {
  if (bar_try(bar, parity)) return true;
  return bar_wait_slow(bar, parity, gave_up);
}

// the same for a whole warp: all lanes go on, or none (one lane's try and a shuffle of its outcome: 432 -> 484 us for a
// step of prompt chunks; a branch of each lane's own before the vote: 432, not 427)
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* gave_up) {
  if (__all_sync(kFull, bar_try(bar, parity))) return true;
  return __all_sync(kFull, bar_wait_slow(bar, parity, gave_up));
}

__device__ __forceinline__ void tma_box(const CUtensorMap* map, uint32_t dst, uint32_t bar, int col, int token, int head, int page) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(map), "r"(col), "r"(token), "r"(head), "r"(page), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void tma_page(const CUtensorMap* map, uint32_t dst, uint32_t bar, int group, int number) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %2, %2, %3, %4}], [%5];" ::"r"(dst),
      "l"(map), "r"(0), "r"(group), "r"(number), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
// The two products' steps.  The operand descriptors are taken as their low words (address and leading stride, what
// changes from step to step) and a constant high word: the issuing thread has 64 clocks per step, and 64-bit arithmetic
// on whole descriptors took longer than that.
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t hi, uint32_t idesc, uint32_t add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tsetp.ne.b32 p, %5, 0;\n\tmov.b64 a, {%1, %3};\n\tmov.b64 b, {%2, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n\t}" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "r"(add)
      : "memory");
}
// mma_ss with the operands' high words apart
__device__ __forceinline__ void mma_two(uint32_t d, uint32_t a_lo, uint32_t a_hi, uint32_t b_lo, uint32_t b_hi, uint32_t idesc, uint32_t add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tsetp.ne.b32 p, %6, 0;\n\tmov.b64 a, {%1, %2};\n\tmov.b64 b, {%3, %4};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, p;\n\t}" ::"r"(d),
      "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(add)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t hi, uint32_t idesc, uint32_t add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\tsetp.ne.b32 p, %5, 0;\n\tmov.b64 b, {%2, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b_lo), "r"(hi), "r"(idesc), "r"(add)
      : "memory");
}

#define GDN_R4(r, i) "=r"(r[i]), "=r"(r[i + 1]), "=r"(r[i + 2]), "=r"(r[i + 3])
#define GDN_W4(r, i) "r"(r[i]), "r"(r[i + 1]), "r"(r[i + 2]), "r"(r[i + 3])
// 32 columns of this thread's TMEM lane
__device__ __forceinline__ void tmem_load(uint32_t (&r)[32], uint32_t at) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : GDN_R4(r, 0), GDN_R4(r, 4), GDN_R4(r, 8), GDN_R4(r, 12), GDN_R4(r, 16), GDN_R4(r, 20), GDN_R4(r, 24), GDN_R4(r, 28)
      : "r"(at));
}
__device__ __forceinline__ void tmem_store(uint32_t at, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(at),
      GDN_W4(r, 0), GDN_W4(r, 4), GDN_W4(r, 8), GDN_W4(r, 12), GDN_W4(r, 16), GDN_W4(r, 20), GDN_W4(r, 24), GDN_W4(r, 28)
      : "memory");
}
__device__ __forceinline__ void tmem_store(uint32_t at, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(at),
      GDN_W4(r, 0), GDN_W4(r, 4), GDN_W4(r, 8), GDN_W4(r, 12)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_load() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
// after the wait, for each load: nothing reads the registers ahead of it
#define GDN_RW4(r, i) "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3])
__device__ __forceinline__ void tmem_loaded(uint32_t (&r)[32]) {
  asm volatile(""
               : GDN_RW4(r, 0), GDN_RW4(r, 4), GDN_RW4(r, 8), GDN_RW4(r, 12), GDN_RW4(r, 16), GDN_RW4(r, 20), GDN_RW4(r, 24), GDN_RW4(r, 28));
}
__device__ __forceinline__ void tmem_wait_store() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// shared-memory operand descriptor, 128-byte swizzle: start address and leading stride in 16-byte units (low word);
// groups of eight rows 1024 bytes apart, version 1 (high word)
__device__ __forceinline__ uint32_t operand_lo(uint32_t addr, uint32_t lead) { return addr >> 4 | (lead >> 4) << 16; }
constexpr uint32_t kOperandHi = 1024 >> 4 | 1u << 14 | 2u << 29;
// bf16 x bf16 -> 32-bit, M = 128; transpose_b: B's N is its contiguous dimension
__host__ __device__ constexpr uint32_t instruction(int n, bool transpose_b) {
  return 1u << 4 | 1u << 7 | 1u << 10 | (transpose_b ? 1u << 16 : 0) | (uint32_t)(n >> 3) << 17 | (uint32_t)(kTcRows >> 4) << 24;
}

// two 32-bit numbers as one operand: half the instructions of the softmax's multiply-adds and sums (8192 tokens at d = 64
// 401 -> 367 us, prompt chunks at d = 128 440 -> 431)
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 halves(uint64_t x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                              CUtensorMapFloatOOBfill);

// looked up once; null where there is no driver
inline EncodeFn encoder() {
  static const EncodeFn fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult found;
    const bool ok = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) == cudaSuccess &&
                    found == cudaDriverEntryPointSuccess;
    return ok ? reinterpret_cast<EncodeFn>(f) : nullptr;
  }();
  return fn;
}

inline bool make_map(CUtensorMap* map, const Params& p, const void* base, int64_t token, int64_t head, int64_t page, int box) {
  const EncodeFn encode = encoder();
  if (!encode) return false;
  const cuuint64_t dims[4] = {(cuuint64_t)p.d, (cuuint64_t)p.page_size, (cuuint64_t)p.H_kv, (cuuint64_t)p.n_pages};
  // the stride of a dimension of one entry is never used, but must be a valid one
  const cuuint64_t strides[3] = {(cuuint64_t)token * 2, (cuuint64_t)(p.H_kv > 1 ? head : token) * 2,
                                 (cuuint64_t)(p.n_pages > 1 ? page : token) * 2};
  const cuuint32_t box_dims[4] = {64, (cuuint32_t)box, 1, 1}, steps[4] = {1, 1, 1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box_dims, steps,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// How a pool's pages are copied whole: its rows as [64][8][d / 64][page_size / 8][page and head], so that one instruction copies
// a page's tokens of a head, or `box` of them, to [group of eight][chunk of 64][8 tokens][128 bytes].
struct PageMap {
  int per_page;  // (page, head) is number page * per_page + head; 0: a page is no whole number of heads long, or the numbers
                 // pass 32 bits, and `map` is make_map's with boxes of eight tokens
  int outside;   // a number outside the map
};
inline bool make_page_map(CUtensorMap* map, PageMap* m, const Params& p, const void* base, int64_t token, int64_t head, int64_t page, int box) {
  const EncodeFn encode = encoder();
  *m = {0, 0};
  // the stride of a dimension of one entry is never used, but must be a valid one
  const int64_t number = p.H_kv > 1 ? head : p.n_pages > 1 ? page : token;
  if (encode && number > 0 && (p.n_pages == 1 || page % number == 0)) {
    const int64_t per_page = p.n_pages > 1 ? page / number : p.H_kv;
    if (per_page >= 1 && per_page <= INT32_MAX / p.n_pages - 1) {
      const int64_t numbers = (p.n_pages - 1) * per_page + p.H_kv;
      const cuuint64_t dims[5] = {64, 8, (cuuint64_t)p.d / 64, (cuuint64_t)p.page_size / 8, (cuuint64_t)numbers};
      const cuuint64_t strides[4] = {(cuuint64_t)token * 2, 128, (cuuint64_t)token * 16, (cuuint64_t)number * 2};
      const cuuint32_t box_dims[5] = {64, 8, (cuuint32_t)p.d / 64, (cuuint32_t)box / 8, 1}, steps[5] = {1, 1, 1, 1, 1};
      if (encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void*>(base), dims, strides, box_dims, steps,
                 CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                 CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS) {
        *m = {(int)per_page, (int)numbers};
        return true;
      }
    }
  }
  return make_map(map, p, base, token, head, page, 8);
}
// `box` tokens of a page and head to `to`, by one lane; outside the pool: zeros
template <int kD>
__device__ __forceinline__ void copy_page(const CUtensorMap* map, const PageMap& m, uint32_t to, uint32_t bar, int box, int token, int head, int page,
                                          int n_pages) {
  const bool good = (unsigned)page < (unsigned)n_pages;
  if (m.per_page > 0) {
    tma_page(map, to, bar, token / 8, good ? page * m.per_page + head : m.outside);
  } else {
    for (int i = 0; i < box / 8 * (kD / 64); ++i)
      tma_box(map, to + i * 1024, bar, i % (kD / 64) * 64, token + i / (kD / 64) * 8, head, good ? page : n_pages);
  }
}
// the high word of such a tile's descriptor
template <int kD>
__host__ __device__ constexpr uint32_t page_tile_hi() {
  return (kD / 64) * 1024 >> 4 | 1u << 14 | 2u << 29;
}

}  // namespace gdnattn
