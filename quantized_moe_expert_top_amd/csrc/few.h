// Int8 products of up to 16 rows, bound by the bytes of the weights: what the layer's and
// the dense product's kernels share.
//
// One block per CU holds the codes of all rows in LDS. Each of its waves streams weight
// rows, 16 at a time, through a ring of its own in LDS, 128 bytes of k of every row a step,
// D steps ahead: a wave load takes 8 rows x 128 bytes, whole cache lines, and nothing waits
// for other waves. (Loads straight into operand registers, 16 rows x 64 bytes each, streamed
// 235 MB at 4.0 TB/s where this reaches 5.9.) v_mfma_i32_16x16x64 multiplies the 16 weight
// rows with up to 16 rows of codes; int32 sums are exact.
#pragma once
#include "quant.h"

namespace moe {

constexpr int kFewTokens = 16;    // rows of codes of one MFMA operand
constexpr int kFewThreads = 512, kFewWaves = kFewThreads / kWave;
constexpr int kFewBlocks = 256;   // one per CU
constexpr int kFewStep = 128;     // bytes of k of each row a step
constexpr int kFewSlot = 16 * kFewStep;

// A barrier for what is written to LDS by instructions; __syncthreads would wait for the
// rings' loads too.
__device__ __forceinline__ void few_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }
// Writes to LDS while ring loads are in flight. The compiler cannot tell them from those
// loads' own writes, and would wait for every load before each; few_barrier waits for these.
__device__ __forceinline__ uint32_t few_lds_at(const void* p) {
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) const void*)p));
}
__device__ __forceinline__ void few_put4(void* p, uint32_t v) {
  asm volatile("ds_write_b32 %0, %1" ::"v"(few_lds_at(p)), "v"(v) : "memory");
}
__device__ __forceinline__ void few_put8(void* p, uint2 v) {
  asm volatile("ds_write_b64 %0, %1" ::"v"(few_lds_at(p)), "v"(__builtin_bit_cast(uint64_t, v)) : "memory");
}
__device__ __forceinline__ void few_put16(void* p, i32x4_t v) {
  asm volatile("ds_write_b128 %0, %1" ::"v"(few_lds_at(p)), "v"(v) : "memory");
}
__device__ __forceinline__ void few_max(uint32_t* p, uint32_t v) {
  asm volatile("ds_max_u32 %0, %1" ::"v"(few_lds_at(p)), "v"(v) : "memory");
}
// An MFMA's result that inline assembly reads next. The compiler places the wait states
// between an MFMA and the instructions it knows, but not before an asm block: the product
// of 16x16x64 codes has 4 passes and its result may be read 8 wait states later, which the
// branch and the address before the first such read do not fill. Once a tile, 16 of them.
__device__ __forceinline__ void few_settle(i32x4_t& acc) { asm volatile("s_nop 15" : "+v"(acc)); }
__device__ __forceinline__ void few_add(int* p, int v) {
  asm volatile("ds_add_u32 %0, %1" ::"v"(few_lds_at(p)), "v"(v) : "memory");
}
// Rows of values [rows, K] to codes in LDS (`stride` bytes a row) and scales by a whole
// block, in two phases: get() requests this thread's chunks of 8 values and amax() adds to
// the rows' maxima in LDS; after a barrier put() writes the codes. Every chunk stays in
// registers, so rows * K is at most kFewValues.
constexpr int kFewChunks = 4, kFewValues = kFewChunks * 8 * kFewThreads;
template <class T, bool F32>
struct FewRows {
  Row8<T, F32> v[kFewChunks];
  uint32_t inv;   // division by the chunks of a row, exact below 2^16
  __device__ __forceinline__ int row_of(int c) const { return __umulhi(c, inv); }
  __device__ __forceinline__ void get(const void* x, int rows, int K) {
    const int C = K / 8, total = rows * C;
    inv = 0xFFFFFFFFu / C + 1;
    // all of them, for the compiler to count: past the end the last chunk again
#pragma unroll
    for (int i = 0; i < kFewChunks; ++i)
      v[i].load(x, static_cast<size_t>(min(static_cast<int>(threadIdx.x) + i * kFewThreads, total - 1)) * 8);
  }
  __device__ __forceinline__ void amax(int rows, int K, uint32_t* m) {
    const int total = rows * (K / 8);
#pragma unroll
    for (int i = 0; i < kFewChunks; ++i) {
      if (i * kFewThreads >= total) break;
      const int c = threadIdx.x + i * kFewThreads, r = row_of(min(c, total - 1));
      const uint32_t a = amax8(v[i], 0);   // past the end: the last chunk again
      const int r0 = __builtin_amdgcn_readfirstlane(r);
      if (__ballot(r != r0) == 0) {
        const uint32_t w = wave_max_u32(a);
        if ((threadIdx.x & (kWave - 1)) == 0) few_max(&m[r0], w);
      } else {
        few_max(&m[r], a);
      }
    }
  }
  __device__ __forceinline__ void put(int rows, int K, const uint32_t* m, uint8_t* to, int stride, float* scale) {
    const int C = K / 8, total = rows * C;
#pragma unroll
    for (int i = 0; i < kFewChunks; ++i) {
      const int c = threadIdx.x + i * kFewThreads;
      if (i * kFewThreads >= total) break;
      if (c >= total) continue;
      const int r = row_of(c);
      float f[8];
      v[i].values(f);
      few_put8(to + r * stride + (c - r * C) * 8, codes8(f, row_scale(m[r])));
    }
    if (static_cast<int>(threadIdx.x) < rows)
      few_put4(&scale[threadIdx.x], __float_as_uint(row_scale(m[threadIdx.x]).s));
  }
};
// The same where the codes are there already: get() requests the first of them, put() copies
// all.
struct FewCodes {
  static constexpr int kBatch = 4;
  uint4 v[kBatch];   // 16 codes each
  float scale;
  __device__ __forceinline__ void batch(const int8_t* q, int c0, int total) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i) v[i] = ld16(q + static_cast<size_t>(min(c0 + i * kFewThreads, total - 1)) * 16);
  }
  __device__ __forceinline__ void get(const int8_t* q, const float* q_scale, int rows, int K) {
    batch(q, threadIdx.x, rows * (K / 16));
    scale = q_scale[min(static_cast<int>(threadIdx.x), rows - 1)];
  }
  __device__ __forceinline__ void put(const int8_t* q, int rows, int K, uint8_t* to, int stride, float* s_scale) {
    const int C = K / 16, total = rows * C;
    const uint32_t inv = 0xFFFFFFFFu / C + (C > 1);   // C 1: every chunk a row
    auto write = [&](int c0) {
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int c = c0 + i * kFewThreads;
        if (c >= total) break;
        const int r = C > 1 ? __umulhi(c, inv) : c;
        few_put16(to + r * stride + (c - r * C) * 16, __builtin_bit_cast(i32x4_t, v[i]));
      }
    };
    write(threadIdx.x);
    for (int c0 = kBatch * kFewThreads; c0 < total; c0 += kBatch * kFewThreads) {
      batch(q, c0 + threadIdx.x, total);
      write(c0 + threadIdx.x);
    }
    if (static_cast<int>(threadIdx.x) < rows) few_put4(&s_scale[threadIdx.x], __float_as_uint(scale));
  }
};

// Ring slot: a load's lane fills 16 bytes, row lane / 8 of its 8, chunk lane % 8 of the row's
// 128 bytes, which holds chunk (lane % 8) ^ (row % 8) of the step, so that the operand reads
// (16 rows at one chunk) fall in distinct banks.
__device__ __forceinline__ int few_chunk(int lane) { return (lane & 7) ^ (lane >> 3); }
// The two loads of a step: rows 0 to 7 from rs0 at off0, rows 8 to 15 from rs1 at off1.
// Always two, so that they can be counted: where `in` is false they read nothing (zeros).
__device__ __forceinline__ void few_issue(uint8_t* slot, const __amdgpu_buffer_rsrc_t& rs0, uint32_t off0,
                                          const __amdgpu_buffer_rsrc_t& rs1, uint32_t off1, bool in) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(rs0, (lds_void_t*)slot, 16, in ? off0 : kMMPastEnd, 0, 0, 2);
  __builtin_amdgcn_raw_ptr_buffer_load_lds(rs1, (lds_void_t*)(slot + 1024), 16, in ? off1 : kMMPastEnd, 0, 0, 2);
}
// At most the loads of the last N steps are in flight. Loads return in order, so other
// vector memory operations in between only make the wait longer.
template <int N>
__device__ __forceinline__ void few_wait() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(2 * N) : "memory");
}
// A step's weight operands from the ring.
__device__ __forceinline__ void few_read(const uint8_t* slot, i32x4_t& w0, i32x4_t& w1) {
  const int lane = threadIdx.x & (kWave - 1), l16 = lane & 15, kg = lane >> 4;
  const uint8_t* at = slot + l16 * kFewStep;
  w0 = *reinterpret_cast<const i32x4_t*>(at + ((kg ^ (l16 & 7)) * 16));
  w1 = *reinterpret_cast<const i32x4_t*>(at + (((4 + kg) ^ (l16 & 7)) * 16));
}

}  // namespace moe
