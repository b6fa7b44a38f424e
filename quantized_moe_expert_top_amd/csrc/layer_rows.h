// The W8A8 layer for some tens of tokens (moe_layer_w8a8), where the codes of all rows no
// longer fit in LDS beside the rings: gate/up and down products of up to 512 picks, bound
// by the bytes of the picked experts' weights.
//
// As in layer_few.h one block per CU streams units of 16 weight rows through its waves'
// rings (few.h); here the unit's rows of codes come through the ring too, 128 bytes of k of
// each a step, from L2. A unit takes 16 rows of one expert: an expert with more has several,
// which read its weights again. 64 tokens of 2048 x 768, 8 of 128 experts: gate/up 62 us, 341
// MB at 5.5 TB/s; down 33 us, 171 MB at 5.1.
#pragma once
#include "layer_few.h"

namespace moe {

constexpr int kRowsDepth = 4, kRowsSlot = 2 * kFewSlot;

// The groups of up to 16 picks of one expert: e, its first place in `sorted`, its picks.
struct RowsRecord {
  int groups;
  int e[kFewMaxR], lo[kFewMaxR], n[kFewMaxR];
  uint16_t sorted[kFewMaxR];
};
struct RowsArgs {
  const int8_t* q;       // KIND 0: codes of x [T, H]; KIND 1: of h by slot [T k, I]
  const float* q_scale;
  const int8_t* w;       // [E, N, K]
  const float* w_scale;  // [E, N]
  const int* ids;        // [T k]
  float* out;            // h by slot, or y by slot
  int* offsets;          // KIND 0: [E + 1] or NULL
  RowsRecord* record;    // KIND 0: written, KIND 1: read
  int rows, R, K, width, E, k;   // rows of q; columns of out
};

template <int KIND>
__global__ __launch_bounds__(kFewThreads, 2) void layer_rows_kernel(const RowsArgs a) {
  extern __shared__ __attribute__((aligned(16))) uint8_t few_lds[];   // rings
  __shared__ int s_e[kFewMaxR], s_lo[kFewMaxR], s_n[kFewMaxR];
  __shared__ uint16_t s_sorted[kFewMaxR];
  __shared__ float s_scale[kFewMaxR];
  constexpr int D = kRowsDepth;
  const int tid = threadIdx.x, lane = tid & (kWave - 1);
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l16 = lane & 15, kg = lane >> 4;
  const int R = a.R, K = a.K;
  uint8_t* ring = few_lds + wv * (D * kRowsSlot);

  if (tid < a.rows) s_scale[tid] = a.q_scale[tid];
  int groups;
  if constexpr (KIND == 0) {
    // scratch in the rings, which are not in use yet
    int* s_ids = reinterpret_cast<int*>(few_lds);
    int* s_count = s_ids + kFewMaxR;
    uint16_t* s_act = reinterpret_cast<uint16_t*>(s_count + MOE_MAX_EXPERTS);
    uint16_t* s_beg = s_act + kFewMaxR;
    __shared__ int tot[kFewWaves];
    few_clear(s_count);
    if (tid < R) s_ids[tid] = a.ids[tid];
    __syncthreads();
    const int n_act = few_table(s_ids, R, s_count, s_act, s_beg, s_sorted,
                                blockIdx.x == 0 ? a.offsets : nullptr, a.E);
    // the same order in every block, ascending: an expert's groups go to several of them
    int start = 0, rank = 0;
    if (tid < R) {
      const int id = s_ids[tid];
      start = s_count[id];
      for (int p = start; p < R && s_ids[s_sorted[p]] == id; ++p) rank += s_sorted[p] < tid;
    }
    __syncthreads();
    if (tid < R) s_sorted[start + rank] = static_cast<uint16_t>(tid);
    __syncthreads();
    const int lo = tid < n_act ? s_beg[tid] : 0, n = tid < n_act ? s_beg[tid + 1] - lo : 0;
    int at = block_excl_scan<kFewThreads>((n + 15) / 16, tot, groups);
    for (int i = 0; i < n; i += 16, ++at) {
      s_e[at] = s_act[tid];
      s_lo[at] = lo + i;
      s_n[at] = min(16, n - i);
    }
    __syncthreads();
    if (blockIdx.x == 0) {
      if (tid < R) {
        a.record->e[tid] = s_e[tid];   // past the groups: unused
        a.record->lo[tid] = s_lo[tid];
        a.record->n[tid] = s_n[tid];
        a.record->sorted[tid] = s_sorted[tid];
      }
      if (tid == 0) a.record->groups = groups;
    }
  } else {
    groups = a.record->groups;
    if (tid < R) {
      s_e[tid] = a.record->e[tid];
      s_lo[tid] = a.record->lo[tid];
      s_n[tid] = a.record->n[tid];
      s_sorted[tid] = a.record->sorted[tid];
    }
    __syncthreads();
  }
  groups = __builtin_amdgcn_readfirstlane(groups);

  const int steps = (K + kFewStep - 1) / kFewStep;
  const int cols = KIND == 0 ? 8 : 16, tiles = a.width / cols;
  const int b = blockIdx.x;
  const int mine = (groups * tiles - b + kFewBlocks - 1) / kFewBlocks;
  const int count = (mine - wv + kFewWaves - 1) / kFewWaves;   // may be <= 0
  const int total = count > 0 ? count * steps : 0;
  struct Unit {
    int tile, g;
  };
  auto unit = [&](int j) {
    const int i = b + (wv + j * kFewWaves) * kFewBlocks;
    Unit u;
    u.g = i / tiles;
    u.tile = i - u.g * tiles;
    return u;
  };
  const int N = KIND == 0 ? 2 * a.width : a.width;
  const size_t each = static_cast<size_t>(N) * K;
  const __amdgpu_buffer_rsrc_t x_rs = buffer_rsrc(a.q, static_cast<uint32_t>(a.rows) * K);
  const int lrow = lane >> 3, chunk = few_chunk(lane);
  int iu = 0, is = 0;   // issue cursor
  uint32_t off0 = 0, off1 = 0, x0 = kMMPastEnd, x1 = kMMPastEnd;
  __amdgpu_buffer_rsrc_t rs = buffer_rsrc(a.w, 0);
  auto enter = [&](int j) {
    const Unit u = unit(j);
    const int e = __builtin_amdgcn_readfirstlane(s_e[u.g]);
    rs = buffer_rsrc(a.w + e * each, static_cast<uint32_t>(each));
    // gate/up: ring rows 4 q + {0, 1} are gate rows 2 q + {0, 1}, 4 q + {2, 3} the matching up rows
    const int r0 = KIND == 0 ? u.tile * 8 + (lrow >> 2) * 2 + (lrow & 1) + (lrow & 2 ? a.width : 0) : u.tile * 16 + lrow;
    off0 = __umul24(r0, K) + chunk * 16;
    off1 = off0 + (KIND == 0 ? 4u : 8u) * K;
    const int lo = s_lo[u.g], n = s_n[u.g];
    const int f0 = s_sorted[lo + min(lrow, n - 1)], f1 = s_sorted[lo + min(lrow + 8, n - 1)];
    x0 = lrow < n ? static_cast<uint32_t>(KIND == 0 ? f0 / a.k : f0) * K + chunk * 16 : kMMPastEnd;
    x1 = lrow + 8 < n ? static_cast<uint32_t>(KIND == 0 ? f1 / a.k : f1) * K + chunk * 16 : kMMPastEnd;
  };
  // always four loads, so that they can be counted
  auto issue = [&](int slot) {
    const int k0 = is * kFewStep;
    const bool in = iu < count && k0 + chunk * 16 < K;
    uint8_t* to = ring + slot * kRowsSlot;
    few_issue(to, rs, off0 + k0, rs, off1 + k0, in);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(x_rs, (lds_void_t*)(to + kFewSlot), 16,
                                             in && x0 != kMMPastEnd ? x0 + k0 : kMMPastEnd, 0, 0, 0);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(x_rs, (lds_void_t*)(to + kFewSlot + 1024), 16,
                                             in && x1 != kMMPastEnd ? x1 + k0 : kMMPastEnd, 0, 0, 0);
    if (++is == steps) {
      is = 0;
      if (++iu < count) enter(iu);
    }
  };
  if (total > 0) enter(0);
#pragma unroll
  for (int d = 0; d < D; ++d) issue(d);

  Unit u = {};
  int n = 0, f = 0;   // picks of the unit, this lane's
  f32x8_t c0, c1;     // the unit's weight scales: gate and up, or columns 0 to 7 and 8 to 15
  i32x4_t acc = {0, 0, 0, 0};
  auto begin = [&](int j) {
    u = unit(j);
    const int e = __builtin_amdgcn_readfirstlane(s_e[u.g]);
    const float* at = a.w_scale + static_cast<size_t>(e) * N + u.tile * cols;
    few_scales(at, at + (KIND == 0 ? a.width : 8), c0, c1);
    n = s_n[u.g];
    f = s_sorted[s_lo[u.g] + min(l16, n - 1)];
    acc = i32x4_t{0, 0, 0, 0};
  };
  auto finish = [&]() {
    if (l16 >= n) return;
    const float xs = s_scale[KIND == 0 ? f / a.k : f];
    if constexpr (KIND == 0) {
      float g0 = c0[0], g1 = c0[1], p0 = c1[0], p1 = c1[1];
#pragma unroll
      for (int q = 1; q < 4; ++q) {
        g0 = kg == q ? c0[2 * q] : g0;
        g1 = kg == q ? c0[2 * q + 1] : g1;
        p0 = kg == q ? c1[2 * q] : p0;
        p1 = kg == q ? c1[2 * q + 1] : p1;
      }
      const float za = static_cast<float>(acc[0]) * xs * g0, zb = static_cast<float>(acc[1]) * xs * g1;
      const float ua = static_cast<float>(acc[2]) * xs * p0, ub = static_cast<float>(acc[3]) * xs * p1;
      *reinterpret_cast<float2*>(a.out + static_cast<size_t>(f) * a.width + u.tile * 8 + kg * 2) =
          make_float2(silu_f32<true>(za) * ua, silu_f32<true>(zb) * ub);
    } else {
      f32x4_t v;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float lo = kg & 1 ? c0[4 + i] : c0[i], hi = kg & 1 ? c1[4 + i] : c1[i];
        v[i] = static_cast<float>(acc[i]) * xs * (kg & 2 ? hi : lo);
      }
      *reinterpret_cast<f32x4_t*>(a.out + static_cast<size_t>(f) * a.width + u.tile * 16 + kg * 4) = v;
    }
  };
  for (int i = 0, slot = 0, st = 0, ju = 0; i < total; ++i) {
    if (st == 0) begin(ju);
    few_wait<2 * (D - 1)>();   // four loads a step
    i32x4_t w0, w1, q0, q1;
    few_read(ring + slot * kRowsSlot, w0, w1);
    few_read(ring + slot * kRowsSlot + kFewSlot, q0, q1);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // the slot is read
    issue(slot);
    acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(w0, q0, acc, 0, 0, 0);
    acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(w1, q1, acc, 0, 0, 0);
    slot = slot + 1 == D ? 0 : slot + 1;
    if (++st == steps) {
      finish();
      st = 0;
      ++ju;
    }
  }
  // no load to LDS outlives the block
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}

}  // namespace moe
