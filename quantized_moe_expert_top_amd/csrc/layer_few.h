// The W8A8 layer for a few tokens (moe_layer_w8a8), bound by the bytes of the picked
// experts' weights: two kernels, gate/up and down with the combine, and before each a small
// one where its codes are more than its blocks make in time (layer_w8a8_plan). One token of
// 7168 x 2048, 8 experts: gate/up 40 us, 235 MB at 5.9 TB/s, down 24 us, 117 MB at 4.9; two
// tokens of 2048 x 768: 13.2 us for 47 MB and 9.8 for 24, which by themselves stream in 8 and
// 4; the rest is the launch, the picks, the codes and the rings' first loads, one after
// another.
#pragma once
#include "../../include/moe.h"
#include "few.h"
#include "launch_int8.h"
#include "norm_rows.h"

namespace moe {

constexpr int kFewMaxR = kFewTokens * MOE_MAX_TOPK;

// What the gate/up kernel found about the picks, for the down kernel: few_table's list.
struct FewRecord {
  int n_act;
  uint16_t act[kFewMaxR], beg[kFewMaxR + 2], sorted[kFewMaxR];
  __device__ __forceinline__ void put(int n, int R, const uint16_t* s_act, const uint16_t* s_beg, const uint16_t* s_sorted) {
    const int f = threadIdx.x;
    if (f < R) {
      act[f] = s_act[f];   // past n: unused
      beg[f] = s_beg[f];
      sorted[f] = s_sorted[f];
    }
    if (f == 0) {
      n_act = n;
      beg[n] = static_cast<uint16_t>(R);
    }
  }
  __device__ __forceinline__ void get(int R, uint16_t* s_act, uint16_t* s_beg, uint16_t* s_sorted) const {
    const int f = threadIdx.x;
    if (f < R) {
      s_act[f] = act[f];
      s_beg[f] = beg[f];
      s_sorted[f] = sorted[f];
    }
    if (f == 0) s_beg[R] = static_cast<uint16_t>(R);
  }
};

struct FewArgs {
  const float* logits;
  const void* x;
  const int8_t* xq;        // CODES: codes of x and of h, and their scales
  const float* xs;
  const int8_t* hq;
  const float* hs;
  const int8_t* w13;
  const float* s13;
  const int8_t* w2;
  const float* s2;
  const void* residual;    // or NULL
  int* ids;
  float* w;
  int* offsets;            // or NULL
  FewRecord* record;
  float* h;                // [T k, I], by slot
  void* out;
  int T, H, I, E, k;
};

__device__ __forceinline__ void few_clear(int* count) { count[threadIdx.x] = count[threadIdx.x + kFewThreads] = 0; }
// The picked experts in ascending order: expert act[i] has the slots sorted[beg[i]] to
// sorted[beg[i + 1]], in an order that depends on timing (here it only says which column of
// a product a slot takes); count[e] is beg of expert e. offsets, where given: moe_permute's.
// Returns the number of experts. ids in LDS and few_clear(count), both behind a barrier;
// count: 1024 words of LDS that nothing else uses. All threads, also for the few slots that a wave could order by itself:
// one slot after another that took 2 us more at 32 slots and 4 at 64.
__device__ __forceinline__ int few_table(const int* ids, int R, int* count, uint16_t* act, uint16_t* beg, uint16_t* sorted,
                                         int* offsets, int E) {
  const int f = threadIdx.x;
  static_assert(MOE_MAX_EXPERTS == 2 * kFewThreads && kFewMaxR <= kFewThreads, "a thread's experts and slots");
  __shared__ int tot[kFewWaves];
  const int id = f < R ? ids[f] : 0;
  const int place = f < R ? atomicAdd(&count[id], 1) : 0;
  __syncthreads();
  const int c0 = count[2 * f], c1 = count[2 * f + 1];
  // experts in the high half, slots in the low one
  int total;
  int at = block_excl_scan<kFewThreads>(((c0 > 0) + (c1 > 0)) << 16 | (c0 + c1), tot, total);
  if (offsets) {
    if (2 * f < E) offsets[2 * f] = at & 0xFFFF;
    if (2 * f + 1 < E) offsets[2 * f + 1] = (at & 0xFFFF) + c0;
    if (f == 0) offsets[E] = R;
  }
  auto enter = [&](int e, int c) {
    if (c > 0) {
      act[at >> 16] = e;
      beg[at >> 16] = at & 0xFFFF;
      count[e] = at & 0xFFFF;
      at += 1 << 16 | c;
    }
  };
  enter(2 * f, c0);
  enter(2 * f + 1, c1);
  if (f == 0) beg[total >> 16] = R;
  __syncthreads();
  if (f < R) sorted[count[id] + place] = f;
  __syncthreads();
  return total >> 16;
}

// Eight scales at each of two uniform addresses, by scalar loads: a vector load's wait
// would be one for all loads of the ring.
typedef __attribute__((__vector_size__(8 * sizeof(float)))) float f32x8_t;
__device__ __forceinline__ const float* few_uniform(const float* p) {
  const uint64_t v = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v)),
                 hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v >> 32));
  return reinterpret_cast<const float*>(static_cast<uint64_t>(hi) << 32 | lo);
}
__device__ __forceinline__ void few_scales(const float* p, const float* q, f32x8_t& a, f32x8_t& b) {
  p = few_uniform(p);
  q = few_uniform(q);
  asm volatile("s_load_dwordx8 %0, %2, 0x0\n\ts_load_dwordx8 %1, %3, 0x0\n\ts_waitcnt lgkmcnt(0)"
               : "=&s"(a), "=&s"(b) : "s"(p), "s"(q) : "memory");
}

// KIND 0: gate/up. Unit: 8 gate rows and the 8 matching up rows of one expert; h[f] =
// silu(g) u of token f / k. Every block routes the tokens and makes the codes of x itself
// (once per CU); block 0 writes the picks.
// CODES: the codes of the rows (of x, of h) are there, and the picks; for more values than
// a CU makes in the time of a launch.
// KIND 1: down. A block owns tiles of 8 output columns for all picked experts and keeps
// their y in LDS, so that it can take the combine too. Unit: the 8 weight rows of two
// experts; a lane half's columns are the one's slots, the other half's the other's.
template <int KIND, bool CODES, class T, bool OUT32, int S, int D>
__global__ __launch_bounds__(kFewThreads, 2) void layer_few_kernel(const FewArgs a) {
  extern __shared__ __attribute__((aligned(16))) uint8_t few_lds[];   // ring, codes, y
  __shared__ int s_ids[kFewMaxR];
  __shared__ uint16_t s_sorted[kFewMaxR], s_act[kFewMaxR], s_beg[kFewMaxR + 1];
  __shared__ float s_w[kFewMaxR];
  constexpr int kRows = KIND == 0 ? kFewTokens : kFewMaxR;
  __shared__ float s_scale[kRows];
  __shared__ uint32_t s_amax[kRows];
  const int tid = threadIdx.x, lane = tid & (kWave - 1);
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l16 = lane & 15, kg = lane >> 4;
  const int R = a.T * a.k;
  const int K = KIND == 0 ? a.H : a.I, rows = KIND == 0 ? a.T : R, stride = K + 16;
  uint8_t* ring = few_lds + wv * (D * kFewSlot);
  uint8_t* codes = few_lds + kFewWaves * D * kFewSlot;
  float* s_y = reinterpret_cast<float*>(codes + static_cast<size_t>(rows) * stride);   // KIND 1

  // rows first: loads return in order, so that these are not waited for behind the ring's
  FewRows<T, KIND == 1> made;
  FewCodes copied;
  if constexpr (!CODES) {
    made.get(KIND == 0 ? a.x : a.h, rows, K);
    if (tid < rows) s_amax[tid] = 0;
  } else if (KIND == 1) {
    copied.get(a.hq, a.hs, rows, K);
  }
  int n_act;
  if constexpr (KIND == 0) {
    int* count = reinterpret_cast<int*>(few_lds);   // the rings are not in use yet
    few_clear(count);
    if constexpr (CODES) {
      if (tid < R) s_ids[tid] = a.ids[tid];
      copied.get(a.xq, a.xs, rows, K);
      copied.put(a.xq, rows, K, codes, stride, s_scale);
    } else {
      few_barrier();   // s_amax is cleared
      if (wv < a.T)
        wave_topk<S>(a.logits + static_cast<size_t>(wv) * a.E, a.E, a.k, s_ids + wv * a.k, s_w + wv * a.k);
      made.amax(rows, K, s_amax);
    }
    few_barrier();
    n_act = few_table(s_ids, R, count, s_act, s_beg, s_sorted,
                      blockIdx.x == 0 ? a.offsets : nullptr, a.E);
    if (blockIdx.x == 0) {
      if (!CODES && tid < R) {
        a.ids[tid] = s_ids[tid];
        a.w[tid] = s_w[tid];
      }
      a.record->put(n_act, R, s_act, s_beg, s_sorted);
    }
  } else {
    n_act = a.record->n_act;
    if (tid < R) s_w[tid] = a.w[tid];
    a.record->get(R, s_act, s_beg, s_sorted);
    few_barrier();
  }
  n_act = __builtin_amdgcn_readfirstlane(n_act);

  // units of this wave: i-th of the block where i % waves is the wave
  const int steps = (K + kFewStep - 1) / kFewStep;
  const int pairs = (n_act + 1) / 2;
  const int tiles = (KIND == 0 ? a.I : a.H) / 8;
  const int b = blockIdx.x;
  // KIND 0: units b, b + blocks, ... of n_act x tiles; KIND 1: tiles b, b + blocks, ...,
  // `pairs` units each
  const int mine = KIND == 0 ? (n_act * tiles - b + kFewBlocks - 1) / kFewBlocks
                             : (tiles - b + kFewBlocks - 1) / kFewBlocks * pairs;
  const int count = (mine - wv + kFewWaves - 1) / kFewWaves;   // may be <= 0
  const int total = count > 0 ? count * steps : 0;
  struct Unit {
    int tile, a0, a1;   // indices into s_act; a1 -1: none
  };
  auto unit = [&](int j) {
    const int i = wv + j * kFewWaves;
    Unit u;
    if (KIND == 0) {
      const int g = b + i * kFewBlocks;
      u.a0 = u.a1 = g / tiles;
      u.tile = g - u.a0 * tiles;
    } else {
      const int t = i / pairs, p = i - t * pairs;
      u.tile = b + t * kFewBlocks;
      u.a0 = 2 * p;
      u.a1 = 2 * p + 1 < n_act ? 2 * p + 1 : -1;
    }
    return u;
  };

  const int N = KIND == 0 ? 2 * a.I : a.H;
  const int8_t* W = KIND == 0 ? a.w13 : a.w2;
  const int lrow = lane >> 3, chunk = few_chunk(lane);
  // issue cursor
  int iu = 0, is = 0;
  uint32_t off0 = 0, off1 = 0;
  __amdgpu_buffer_rsrc_t rs0 = buffer_rsrc(W, 0), rs1 = rs0;
  auto enter = [&](int j) {
    const Unit u = unit(j);
    const int e0 = __builtin_amdgcn_readfirstlane(s_act[u.a0]);
    const size_t each = static_cast<size_t>(N) * K;
    rs0 = buffer_rsrc(W + e0 * each, static_cast<uint32_t>(each));
    if (KIND == 0) {
      rs1 = rs0;
      // ring rows 4 q + {0, 1} are gate rows 2 q + {0, 1}, 4 q + {2, 3} the matching up
      // rows, so that a lane ends with both of an output
      const int r0 = u.tile * 8 + (lrow >> 2) * 2 + (lrow & 1) + (lrow & 2 ? a.I : 0);
      off0 = __umul24(r0, K) + chunk * 16;
      off1 = off0 + 4u * K;
    } else {
      const int e1 = u.a1 < 0 ? -1 : __builtin_amdgcn_readfirstlane(s_act[u.a1]);
      rs1 = buffer_rsrc(W + (e1 < 0 ? 0 : e1) * each, e1 < 0 ? 0u : static_cast<uint32_t>(each));
      off0 = off1 = __umul24(u.tile * 8 + lrow, K) + chunk * 16;
    }
  };
  auto issue = [&](int slot) {
    const int k0 = is * kFewStep;
    few_issue(ring + slot * kFewSlot, rs0, off0 + k0, rs1, off1 + k0, iu < count && k0 + chunk * 16 < K);
    if (++is == steps) {
      is = 0;
      if (++iu < count) enter(iu);
    }
  };
  // not the whole ring before the codes are made: loads waiting to be issued would hold that
  // up (layers of 1 to 8 tokens 1 to 2% slower with all of it or half of it)
  constexpr int kFirst = CODES ? D : D / 4 * 3;
  // Issued by every wave, whether it has units or not: the compiler counts them.
  if (total > 0) enter(0);
#pragma unroll
  for (int d = 0; d < kFirst; ++d) issue(d);
  if constexpr (!CODES) {
    if (KIND == 1) {
      made.amax(rows, K, s_amax);
      few_barrier();
    }
    made.put(rows, K, s_amax, codes, stride, s_scale);
#pragma unroll
    for (int d = kFirst; d < D; ++d) issue(d);
    few_barrier();
  } else if (KIND == 1) {
    copied.put(a.hq, rows, K, codes, stride, s_scale);
    few_barrier();
  }

  int st = 0, ju = 0;   // consume cursor
  Unit u = {};
  const uint8_t *x0 = codes, *x1 = codes;
  bool two = false;
  i32x4_t acc0 = {0, 0, 0, 0}, acc1 = acc0;
  int m_lane = 0, slot0 = 0, slot1 = 0;   // this lane's slots, and how many its expert has
  f32x8_t c0, c1;   // the unit's scales: gate and up, or the two experts'
  auto begin = [&](int j) {
    u = unit(j);
    const int e0 = __builtin_amdgcn_readfirstlane(s_act[u.a0]);
    if (KIND == 0) {
      const float* at = a.s13 + static_cast<size_t>(e0) * N + u.tile * 8;
      few_scales(at, at + a.I, c0, c1);
    } else {
      const int e1 = __builtin_amdgcn_readfirstlane(s_act[u.a1 < 0 ? u.a0 : u.a1]);
      few_scales(a.s2 + static_cast<size_t>(e0) * N + u.tile * 8, a.s2 + static_cast<size_t>(e1) * N + u.tile * 8, c0, c1);
    }
    const int ai = KIND == 0 ? u.a0 : (l16 < 8 ? u.a0 : u.a1);
    const int c = KIND == 0 ? l16 : l16 & 7;
    const int lo = ai < 0 ? 0 : s_beg[ai], M = ai < 0 ? 0 : s_beg[ai + 1] - lo;
    m_lane = M;
    slot0 = s_sorted[lo + max(min(c, M - 1), 0)];
    slot1 = KIND == 0 ? slot0 : s_sorted[lo + max(min(c + 8, M - 1), 0)];
    x0 = codes + (KIND == 0 ? slot0 / a.k : slot0) * stride;
    x1 = codes + slot1 * stride;
    two = KIND == 1 && __ballot(M > 8) != 0;
    acc0 = acc1 = i32x4_t{0, 0, 0, 0};
  };
  auto finish = [&]() {
    if constexpr (KIND == 0) {
      float g0 = c0[0], g1 = c0[1], p0 = c1[0], p1 = c1[1];
#pragma unroll
      for (int q = 1; q < 4; ++q) {
        g0 = kg == q ? c0[2 * q] : g0;
        g1 = kg == q ? c0[2 * q + 1] : g1;
        p0 = kg == q ? c1[2 * q] : p0;
        p1 = kg == q ? c1[2 * q + 1] : p1;
      }
      if (l16 < m_lane) {
        const float xs = s_scale[slot0 / a.k];
        const float za = static_cast<float>(acc0[0]) * xs * g0, zb = static_cast<float>(acc0[1]) * xs * g1;
        const float ua = static_cast<float>(acc0[2]) * xs * p0, ub = static_cast<float>(acc0[3]) * xs * p1;
        *reinterpret_cast<float2*>(a.h + static_cast<size_t>(slot0) * a.I + u.tile * 8 + kg * 2) =
            make_float2(silu_f32<true>(za) * ua, silu_f32<true>(zb) * ub);
      }
    } else {
      float s[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float lo = l16 < 8 ? c0[i] : c1[i], hi = l16 < 8 ? c0[4 + i] : c1[4 + i];
        s[i] = kg & 1 ? hi : lo;
      }
      if ((kg >> 1) == (l16 >> 3)) {
        float* to = s_y + static_cast<size_t>(u.tile / kFewBlocks) * R * 8 + (kg & 1) * 4;
        auto put = [&](const i32x4_t& acc, int slot) {
          const float hs = s_scale[slot];
          const f32x4_t v = {static_cast<float>(acc[0]) * hs * s[0], static_cast<float>(acc[1]) * hs * s[1],
                             static_cast<float>(acc[2]) * hs * s[2], static_cast<float>(acc[3]) * hs * s[3]};
          few_put16(to + slot * 8, __builtin_bit_cast(i32x4_t, v));
        };
        if ((l16 & 7) < m_lane) put(acc0, slot0);
        if ((l16 & 7) + 8 < m_lane) put(acc1, slot1);
      }
    }
  };
  for (int i = 0, slot = 0; i < total; ++i) {
    if (st == 0) begin(ju);
    few_wait<D - 1>();
    i32x4_t w0, w1;
    few_read(ring + slot * kFewSlot, w0, w1);
    // past k the weights are zeros, and any codes will do
    const int k0 = min(st * kFewStep + kg * 16, K - 16), k1 = min(st * kFewStep + 64 + kg * 16, K - 16);
    const i32x4_t a0 = *reinterpret_cast<const i32x4_t*>(x0 + k0), a1 = *reinterpret_cast<const i32x4_t*>(x0 + k1);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // the slot is read
    issue(slot);
    acc0 = __builtin_amdgcn_mfma_i32_16x16x64_i8(w0, a0, acc0, 0, 0, 0);
    acc0 = __builtin_amdgcn_mfma_i32_16x16x64_i8(w1, a1, acc0, 0, 0, 0);
    if (KIND == 1 && two) {
      acc1 = __builtin_amdgcn_mfma_i32_16x16x64_i8(w0, *reinterpret_cast<const i32x4_t*>(x1 + k0), acc1, 0, 0, 0);
      acc1 = __builtin_amdgcn_mfma_i32_16x16x64_i8(w1, *reinterpret_cast<const i32x4_t*>(x1 + k1), acc1, 0, 0, 0);
    }
    slot = slot + 1 == D ? 0 : slot + 1;
    if (++st == steps) {
      finish();
      st = 0;
      ++ju;
    }
  }
  // no load to LDS outlives the block
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  if constexpr (KIND == 1) {
    few_barrier();
    // out[t] = residual[t] + sum_j w[t, j] y[t k + j], in increasing j
    const int my_tiles = (tiles - b + kFewBlocks - 1) / kFewBlocks;
    for (int i = tid; i < my_tiles * a.T; i += kFewThreads) {
      const int tl = i / a.T, t = i - tl * a.T;
      const size_t at = static_cast<size_t>(t) * a.H + (b + tl * kFewBlocks) * 8;
      float res[8], o[8] = {0, 0, 0, 0, 0, 0, 0, 0};
      if (a.residual) row_load8<T>(a.residual, at, OUT32, res);
      for (int j = 0; j < a.k; ++j) {
        const float* y = s_y + (static_cast<size_t>(tl) * R + t * a.k + j) * 8;
        const float wj = s_w[t * a.k + j];
#pragma unroll
        for (int x = 0; x < 8; ++x) o[x] += wj * y[x];
      }
      if (a.residual)
#pragma unroll
        for (int x = 0; x < 8; ++x) o[x] += res[x];
      row_store8<T>(a.out, at, OUT32, o);
    }
  }
}

// Picks and codes of the tokens, for CODES: a block makes a token's codes, or routes four
// tokens.
template <class T, int S>
__global__ __launch_bounds__(256) void layer_route_kernel(const FewArgs a, int8_t* xq, float* xs) {
  __shared__ uint32_t red[4];
  const int lane = threadIdx.x & (kWave - 1), wv = threadIdx.x >> 6;
  if (static_cast<int>(blockIdx.x) >= a.T) {
    const int t = (blockIdx.x - a.T) * 4 + wv;
    if (t < a.T)
      wave_topk<S>(a.logits + static_cast<size_t>(t) * a.E, a.E, a.k, a.ids + t * a.k, a.w + t * a.k);
    return;
  }
  const int C = a.H / 8;
  const size_t row = static_cast<size_t>(blockIdx.x) * a.H;
  constexpr int NC = 8;   // H <= 16384
  Row8<T, false> v[NC];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < NC; ++i)
    if (i * 256 < C) v[i].load(a.x, row + min(static_cast<int>(threadIdx.x) + i * 256, C - 1) * 8);
#pragma unroll
  for (int i = 0; i < NC; ++i)
    if (i * 256 < C) m = amax8(v[i], m);
  m = wave_max_u32(m);
  if (lane == 0) red[wv] = m;
  __syncthreads();
  const RowScale s = row_scale(max_u32(max_u32(red[0], red[1]), max_u32(red[2], red[3])));
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = threadIdx.x + i * 256;
    if (c >= C) continue;
    float f[8];
    v[i].values(f);
    *reinterpret_cast<uint2*>(xq + row + c * 8) = codes8(f, s);
  }
  if (threadIdx.x == 0) xs[blockIdx.x] = s.s;
}

}  // namespace moe
