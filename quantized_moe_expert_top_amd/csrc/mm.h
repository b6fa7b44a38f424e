// bf16 / fp16 tile products of the block operators (moe_block.h): device code
// shared by the forward (NT), row-gradient (NN) and weight-gradient (TN) kernels.
//
//   C[m][n] = sum_k A(m, k) B(n, k), float32 accumulators, C row-major
//
//            C              A(m, k)                B(n, k)             contraction k
//   NT   z = x W^T      x [row m][k], rows      W [n][k]             K
//                       optionally gathered
//   NN   dx = dz W      dz [row m][k]           W [k][n]             N (W's rows)
//   TN   dW = dz^T x    dz [row k][m]           x [row k][n], rows   the rows of an expert
//                                               optionally gathered
//
// An operand whose contraction index is contiguous in memory ("K-major") is
// staged as tile rows of BK values and read from LDS 16 bytes (8 k) per lane.
// One whose output index is contiguous ("M-major") is staged as BK rows of tile
// columns and read with ds_read_b64_tr_b16, which transposes on the way: per 16
// lanes it reads 4 k rows of 16 columns and hands lane i column i, 4 k values.
// Both give lane (l32, hf) of a 16-k step the k values 8 hf + [0, 8) of row or
// column l32, so any two operands agree.
//
// Both stagings are direct loads to LDS (buffer_load_dwordx4 ... lds): 64 lanes
// fill 64 consecutive 16-byte slots, and the source address of each slot is
// free, so slots are swizzled for the reads at no cost. Loads past a buffer
// resource's end return zeros: rows past an expert's block, columns past the
// matrix and k past the contraction are never read from memory.
#pragma once
#include <type_traits>

#include "common.h"

namespace moe {

typedef __attribute__((__vector_size__(8 * sizeof(_Float16)))) _Float16 f16x8_t;
typedef __attribute__((__vector_size__(2 * sizeof(_Float16)))) _Float16 f16x2_t;
typedef __attribute__((__vector_size__(4 * sizeof(short)))) short s16x4_t;
typedef __attribute__((address_space(3))) s16x4_t lds_s16x4_t;

typedef __attribute__((__vector_size__(2 * sizeof(int)))) int i32x2_t;
typedef i32x4_t frag_t;   // 8 values of one operand

struct bf16_tag {};
struct fp16_tag {};

template <class T>
__device__ __forceinline__ f32x16_t mfma16(frag_t a, frag_t b, f32x16_t c) {
  if constexpr (__is_same(T, bf16_tag))
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a),
                                                   __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8_t, a),
                                                  __builtin_bit_cast(f16x8_t, b), c, 0, 0, 0);
}

// two floats -> two values of T, round to nearest even (fp16: past the largest
// value to infinity)
template <class T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (__is_same(T, bf16_tag)) {
    return pack_bf16x2(lo, hi);
  } else {
    const f16x2_t v = {(_Float16)lo, (_Float16)hi};
    return __builtin_bit_cast(uint32_t, v);
  }
}
template <class T>
__device__ __forceinline__ void unpack2(uint32_t w, float& lo, float& hi) {
  if constexpr (__is_same(T, bf16_tag)) {
    lo = bf16lo(w);
    hi = bf16hi(w);
  } else {
    const f16x2_t v = __builtin_bit_cast(f16x2_t, w);
    lo = (float)v[0];
    hi = (float)v[1];
  }
}

// Activations and their derivatives in float32. `u` below is 2^-24; the hardware's
// exp2 and reciprocal are within 2 u. EXACT, for results that are stored as float32:
// within 18 u of the value itself over the whole range. Otherwise the exponential is
// one exp2, whose argument's rounding makes e^x off by |x| u: up to 2^-16 of a result
// in an activation's far tail, which the rounding to 16 bits (2^-12 or 2^-9) hides.
// 8192 x 4096 x 1024 to bf16: silu 82 us, gelu 93, SwiGLU 69; 88, 98 and 72 EXACT.
// Results whose exponential is below 2^-126 become 0 (|silu| < 1.1e-36).
//
// EXACT: exp(x + lo), x <= 0, |lo| small, within 3.2 u: exp2(t), t = x log2 e rounded,
// times 1 + d with d = x - t ln 2 + lo, what t's rounding left out. Held at -104,
// where the result is 0, so that an infinite x gives no infinity minus infinity.
__device__ __forceinline__ float exp_neg_f32(float x, float lo = 0.0f) {
  x = __builtin_fmaxf(x, -104.0f);
  const float t = x * 1.4426950408889634f;
  float d = __builtin_fmaf(t, -0.693147182464599609375f, x);   // ln 2 to 24 bits,
  d = __builtin_fmaf(t, 1.904654323148236e-9f, d) + lo;        // and the rest of it
  const float e = __builtin_amdgcn_exp2f(t);
  return __builtin_fmaf(e, d, e);
}
// s = 1 / (1 + e^-z) and c = 1 - s. EXACT: both through e^-|z|, so that neither
// overflows and neither is a difference; each within 7.2 u.
template <bool EXACT>
__device__ __forceinline__ void sigmoid2_f32(float z, float& s, float& c) {
  if constexpr (EXACT) {
    const float e = exp_neg_f32(-__builtin_fabsf(z)), r = __builtin_amdgcn_rcpf(1.0f + e), er = e * r;
    s = z < 0.0f ? er : r;
    c = z < 0.0f ? r : er;
  } else {
    s = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-z * 1.4426950408889634f));
    c = 1.0f - s;
  }
}
template <bool EXACT>
__device__ __forceinline__ float silu_f32(float z) {
  float s, c;
  sigmoid2_f32<EXACT>(z, s, c);
  return z * s;
}
// The Gaussian cdf, and e = exp(-z^2 / 2): with s = |z| the tail is
// cdf(-s) = erfc(s / sqrt 2) / 2 = e t P(t), t = 1 / (1 + 0.325 s), P of degree 9 by
// least relative error (1.4 u); relative to the tail, so nothing cancels for
// negative z. EXACT: s^2 goes into the exponential with its rounding error; within
// 17 u in all (t's 3 u count 2.5 times through t P, Horner's steps 2.9 u, e 3.2 u).
// The library's erfc takes some hundred instructions (8192 x 4096 x 1024 with it:
// 157 us).
template <bool EXACT>
__device__ __forceinline__ float normal_cdf_f32(float z, float& e) {
  float s = __builtin_fabsf(z);
  if constexpr (EXACT) s = __builtin_fminf(s, 16.0f);   // e is 0 from there on
  const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.325f, s, 1.0f)), q = s * s;
  if constexpr (EXACT) e = exp_neg_f32(-0.5f * q, -0.5f * __builtin_fmaf(s, s, -q));
  else e = __builtin_amdgcn_exp2f(-0.72134752044448170f * q);
  float p = -0.0211383961f;
  p = __builtin_fmaf(p, t, 0.091305308f);
  p = __builtin_fmaf(p, t, -0.129665121f);
  p = __builtin_fmaf(p, t, 0.0433723368f);
  p = __builtin_fmaf(p, t, -0.00181293103f);
  p = __builtin_fmaf(p, t, 0.0542199835f);
  p = __builtin_fmaf(p, t, 0.0884514824f);
  p = __builtin_fmaf(p, t, 0.115954153f);
  p = __builtin_fmaf(p, t, 0.129656926f);
  p = __builtin_fmaf(p, t, 0.12965624f);
  const float tail = p * t * e;
  return z >= 0.0f ? 1.0f - tail : tail;
}
template <bool EXACT>
__device__ __forceinline__ float act_f32(float z, int act) {
  if (act == 1) return z > 0.0f ? z : (z != z ? z : 0.0f);   // relu; NaN stays
  if (act == 2) return silu_f32<EXACT>(z);
  float e;
  if (act == 3) return z * normal_cdf_f32<EXACT>(z, e);   // gelu
  return z;
}
template <bool EXACT>
__device__ __forceinline__ float act_grad_f32(float z, int act) {
  if (act == 1) return z > 0.0f ? 1.0f : (z != z ? z : 0.0f);
  if (act == 2) {
    float s, c;
    sigmoid2_f32<EXACT>(z, s, c);
    return s * __builtin_fmaf(z, c, 1.0f);
  }
  if (act == 3) {   // cdf + z pdf
    float e;
    const float cdf = normal_cdf_f32<EXACT>(z, e);
    return __builtin_fmaf(z * 0.39894228040143268f, e, cdf);
  }
  return 1.0f;
}

// Gradients of y = silu(g) u in g and u. dy multiplies last: dy g or dy u may leave
// float32's range (and infinity times silu = 0 be NaN) where the gradient does not.
template <bool EXACT>
__device__ __forceinline__ void swiglu_grad_f32(float dy, float g, float u, float& dg, float& du) {
  float s, c;
  sigmoid2_f32<EXACT>(g, s, c);
  du = dy * (g * s);
  dg = dy * (u * (s * __builtin_fmaf(g, c, 1.0f)));
}

typedef __attribute__((__vector_size__(4 * sizeof(float)))) float f32x4_t;
__device__ __forceinline__ void mm_area8(const float* p, float (&v)[8]) {
  const f32x4_t a = reinterpret_cast<const f32x4_t*>(p)[0], b = reinterpret_cast<const f32x4_t*>(p)[1];
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    v[t] = a[t];
    v[4 + t] = b[t];
  }
}
template <class T>
__device__ __forceinline__ void mm_add8(const uint4& w, float (&v)[8]) {
  const uint32_t d[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    float lo, hi;
    unpack2<T>(d[t], lo, hi);
    v[2 * t] += lo;
    v[2 * t + 1] += hi;
  }
}
// Stores of results, 16 bytes at `off` of a resource over the tile's rows.
// `stream` (uniform): with the non-temporal hint (aux 2), which sends them on to
// memory at once. Left to the L2s, a round of tiles fills them with dirty lines
// and the next round's stores wait for their eviction: weight gradients of 128
// experts x 1536 x 2048 from 32768 rows 420 -> 315 us, from 4096 rows 207 ->
// 160 us. (Two plain stores that differ in the hint alone would be merged into
// one without it.)
__device__ __forceinline__ void mm_put16(i32x4_t w, __amdgpu_buffer_rsrc_t rs, uint32_t off,
                                         bool stream) {
  if (stream) __builtin_amdgcn_raw_buffer_store_b128(w, rs, off, 0, 2);
  else __builtin_amdgcn_raw_buffer_store_b128(w, rs, off, 0, 0);
}
template <class T>
__device__ __forceinline__ i32x4_t mm_pack8(const float (&v)[8]) {
  return i32x4_t{static_cast<int>(pack2<T>(v[0], v[1])), static_cast<int>(pack2<T>(v[2], v[3])),
                 static_cast<int>(pack2<T>(v[4], v[5])), static_cast<int>(pack2<T>(v[6], v[7]))};
}

enum { kModeNT = 0, kModeNN = 1, kModeTN = 2 };
constexpr int kActSwiglu = 4;

struct MMArgs {
  const void* A;
  const void* B;
  const int* offsets;    // [E + 1]; NULL: one block of all rows
  const int* slot;       // gather of the rows of x (NT: A, TN: B), or NULL
  const void* bias;      // [n], or NULL (NT)
  const void* residual;  // like C, or NULL (NT)
  void* z;               // [rows][N] of T, or NULL (NT)
  void* C;
  int rows;              // grouped rows
  int x_rows;            // rows of x under a gather
  int topk;
  int E;
  int mdim;              // TN: rows of C (NT, NN: rows of the groups)
  int ndim;              // columns of C before the activation
  int kdim;              // NT, NN: contraction length
  int act;
  int c_f32;             // C is float32 (else T)
  int stream_out;        // C and z are past what the caches can keep
  int splits;            // parts of the contraction, each to its own C (TN; NN without offsets)
  int nt;                // n tiles
  int mt;                // TN: m tiles
  int xm;                // TN: m slices of an expert's tiles over the XCDs (1, 2, 4, 8), or 0
};

// Geometry of a block: BM x BN of C, WM x WN waves, K in stages of BK, STAGES of
// them rotating through LDS, WPE waves per SIMD (as blocks allow).
template <int BM_, int BN_, int WM_, int WN_, int BK_, int STAGES_, int WPE_>
struct MMGeom {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, BK = BK_, STAGES = STAGES_;
  static constexpr int WPE = WPE_;
  static constexpr int kThreads = WM * WN * kWave;
  static constexpr int MI = BM / WM / 32, NJ = BN / WN / 32;   // 32 x 32 subtiles per wave
  static constexpr int kASlots = BM * BK / 8, kBSlots = BN * BK / 8;   // 16-byte slots
  static constexpr int kAPer = kASlots / kThreads, kBPer = kBSlots / kThreads;
  static constexpr int kStageBytes = (kASlots + kBSlots) * 16;
  static constexpr int kAreaBytes = WM * WN * 32 * (BN / WN + 4) * 4;   // epilogue
  static constexpr int kLds = STAGES * kStageBytes > kAreaBytes ? STAGES * kStageBytes : kAreaBytes;
  static constexpr int kLoads = kAPer + kBPer;                 // per thread and stage
  static_assert(kASlots % kThreads == 0 && kBSlots % kThreads == 0, "slots split evenly");
  static_assert(kAPer >= 1 && kAPer <= 8 && kBPer >= 1 && kBPer <= 8, "slot arrays hold eight");
  static_assert(MI >= 1 && MI <= 4 && NJ >= 1 && NJ <= 4, "accumulator array holds 4 x 4");
  static_assert(BK == 32 || BK == 64, "K-major rows of a stage: whole cache lines at 64");
  static_assert(STAGES >= 2 && STAGES <= 5, "waits below");
};

// K-major tile, rows of BK values = CPR chunks of 16 bytes: chunk c of row r sits
// at slot r * CPR + (c ^ swz), so 16 consecutive rows read at one chunk fall in
// distinct banks.
template <int CPR>
__device__ __forceinline__ int kmajor_swz(int row) { return (row / (16 / CPR)) & (CPR - 1); }
// M-major tile, BK rows of COLS values: a transposing read takes 4 consecutive k
// rows at two neighbouring 16-column groups (32 bytes each); the chunk index is
// XORed so that these eight fall in distinct banks.
template <int COLS>
__device__ __forceinline__ int mmajor_swz(int k) {
  if (COLS >= 128) return (k & 3) << 2;
  if (COLS == 64) return ((k >> 1) & 1) << 2;
  return 0;
}

// At most N of this wave's loads to LDS in flight and all its LDS reads done,
// then the barrier.
template <int N>
__device__ __forceinline__ void mm_wait_barrier() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}
template <int LPS, int MAXL>
__device__ __forceinline__ void mm_wait_stage(int later) {
  if constexpr (MAXL >= 4) { if (later >= 4) { mm_wait_barrier<4 * LPS>(); return; } }
  if constexpr (MAXL >= 3) { if (later == 3) { mm_wait_barrier<3 * LPS>(); return; } }
  if constexpr (MAXL >= 2) { if (later == 2) { mm_wait_barrier<2 * LPS>(); return; } }
  if constexpr (MAXL >= 1) { if (later == 1) { mm_wait_barrier<LPS>(); return; } }
  mm_wait_barrier<0>();
}

// Order of the instructions since the last scheduling barrier: READS LDS reads
// and LOADS loads spread over the first of MFMAS multiplies.
template <int READS, int LOADS, int MFMAS>
__device__ __forceinline__ void mm_interleave() {
  constexpr int kSlots = MFMAS > 2 ? MFMAS - 2 : 1;   // the last two cover the reads' latency
  constexpr int R = (READS + kSlots - 1) / kSlots, L = (LOADS + kSlots - 1) / kSlots;
#pragma unroll
  for (int m = 0; m < MFMAS; ++m) {
    if (m * R < READS) __builtin_amdgcn_sched_group_barrier(0x100, R, 0);
    if (m * L < LOADS) __builtin_amdgcn_sched_group_barrier(0x020, L, 0);
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
  }
  __builtin_amdgcn_sched_barrier(0);
}

constexpr uint32_t kMMPastEnd = 0x80000000u;   // at or past the end of every resource here

// Whether a launch of `tiles` blocks (rounded up to eight, see mm_find_tile) fits:
// under 2^32 threads, so under 2^26 tiles.
inline bool mm_fits(long long tiles, int threads) {
  return (tiles + 7) / 8 * 8 * threads < (1LL << 32);
}
constexpr int kMMSegRows = 1024;               // TN gather: source rows held in LDS at a time
constexpr int kMMGroupM = 8;                   // m tiles walked together over all n tiles

// Tile of a row-grouped product (NT, NN). Tiles are ordered expert by expert;
// inside an expert, groups of kMMGroupM m tiles walk the n tiles together. Each
// XCD (block % 8) takes a contiguous run of that order, so that the tiles
// it holds at one time share W strips and x rows in its L2. Offsets are clamped
// to [0, rows] and a block's end to its start, so that values outside the
// contract cannot lead out of the buffers. Returns false for a block without a tile.
// Counts are unsigned: an expert's tiles stay under 2^31 for any offsets, but where
// blocks overlap (outside the contract) their sum may wrap, so that a block finds
// several experts, or none. Each of the four values it reads is one that some expert
// wrote, and the tile is checked against them.
struct MMTile {
  int e, nt, p0, p1;   // rows [p0, p1), at most BM of them
};
__device__ __forceinline__ i32x2_t tr_read(const lds_s16x4_t* __restrict__ p) {
  return __builtin_bit_cast(i32x2_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t*)p));
}

template <int BM, int NTHR>
__device__ __forceinline__ bool mm_find_tile(const int* __restrict__ offsets, int rows, int E,
                                             int NT, int* sm, uint32_t bid, MMTile& t) {
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wv = tid >> 6;
  int e = 0, mtiles = 0, beg = 0, end = 0;
  uint32_t local = 0;
  if (offsets == nullptr) {
    mtiles = (rows + BM - 1) / BM;
    const uint32_t total = static_cast<uint32_t>(mtiles) * NT, chunk = (total + 7) / 8;
    local = (bid & 7) * chunk + (bid >> 3);
    if ((bid >> 3) >= chunk || local >= total) return false;
    end = rows;
  } else {
    constexpr int kPer = 1024 / NTHR > 0 ? 1024 / NTHR : 1;   // E <= 1024
    const int ept = (E + NTHR - 1) / NTHR;
    int* out = sm + NTHR / kWave;
    int b[kPer], n[kPer];
    uint32_t cnt[kPer], sum = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int ei = tid * ept + i;
      int lo = 0, hi = 0;
      uint32_t c = 0;
      if (i < ept && ei < E) {
        lo = min(max(offsets[ei], 0), rows);
        hi = min(max(offsets[ei + 1], lo), rows);
        c = static_cast<uint32_t>((hi - lo + BM - 1) / BM) * NT;
      }
      cnt[i] = c;
      b[i] = lo;
      n[i] = hi;
      sum += c;
    }
    uint32_t incl = sum;
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
      const uint32_t o = __shfl_up(incl, d, kWave);
      if (lane >= d) incl += o;
    }
    if (lane == kWave - 1) sm[wv] = static_cast<int>(incl);
    if (tid == 0) out[0] = -1;
    __syncthreads();
    uint32_t before = 0, total = 0;
#pragma unroll
    for (int i = 0; i < NTHR / kWave; ++i) {
      const uint32_t s = sm[i];
      if (i < wv) before += s;
      total += s;
    }
    const uint32_t chunk = total / 8 + (total % 8 != 0);
    const uint32_t tau = (bid & 7) * chunk + (bid >> 3);
    if ((bid >> 3) >= chunk || tau >= total) return false;   // uniform
    uint32_t start = before + incl - sum;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      if (tau - start < cnt[i]) {
        out[0] = tid * ept + i;
        out[1] = static_cast<int>(tau - start);
        out[2] = b[i];
        out[3] = n[i];
      }
      start += cnt[i];
    }
    __syncthreads();
    e = __builtin_amdgcn_readfirstlane(out[0]);
    local = __builtin_amdgcn_readfirstlane(out[1]);
    beg = __builtin_amdgcn_readfirstlane(out[2]);
    end = __builtin_amdgcn_readfirstlane(out[3]);
    if (e < 0 || beg >= end) return false;
    mtiles = (end - beg + BM - 1) / BM;
    if (local >= static_cast<uint32_t>(mtiles) * NT) return false;
  }
  const int per = kMMGroupM * NT, g = static_cast<int>(local) / per,
            r = static_cast<int>(local) - g * per;
  const int gm = min(kMMGroupM, mtiles - g * kMMGroupM);
  t.e = e;
  t.nt = r / gm;
  t.p0 = beg + (g * kMMGroupM + r % gm) * BM;
  t.p1 = min(end, t.p0 + BM);
  return true;
}

// One tile: block `bid` of a grid of its mode's tiles.
template <class T, int MODE, class G>
__device__ __forceinline__ void mm_tile(const uint8_t* __restrict__ Ab,
                                        const uint8_t* __restrict__ Bb, const MMArgs& a,
                                        uint32_t bid) {
  constexpr int BM = G::BM, BN = G::BN, BK = G::BK, NTHR = G::kThreads, STAGES = G::STAGES;
  constexpr int MI = G::MI, NJ = G::NJ, CPR = BK / 8, KS = BK / 16;
  constexpr int RW = BM / G::WM, CW = BN / G::WN;   // tile rows / columns per wave
  constexpr bool kAK = MODE != kModeTN;             // A is K-major
  constexpr bool kBK = MODE == kModeNT;             // B is K-major
  extern __shared__ __attribute__((aligned(16))) uint8_t mm_lds[];   // G::kLds
  __shared__ int row_src[MODE == kModeTN ? kMMSegRows : BM];
  __shared__ int sm_tile[NTHR / kWave + 4];

  const int tid = threadIdx.x, lane = tid & (kWave - 1), wv = tid >> 6;
  const int l32 = lane & 31, hf = lane >> 5, l16 = lane & 15;
  const int wm = wv / G::WN, wn = wv % G::WN;
  const bool swiglu = MODE == kModeNT && a.act == kActSwiglu;   // uniform

  // ---- the tile
  int e = 0, m0 = 0, n0 = 0;        // expert, first C row and column of the tile
  int mrows = 0;                    // rows of C in the tile
  int k_begin = 0, k_end = 0;       // what is contracted over (TN: rows)
  int split = 0;
  if constexpr (MODE == kModeTN) {
    int es, mi, ni;
    if (a.xm > 0) {
      // several experts: every XCD takes a rectangle of each expert's tiles (xm
      // slices of m by 8 / xm of n), so that experts with many rows load all XCDs
      // alike (128 x 1536 x 2048 from 32768 rows, 8 to 1513 per expert: 308 us, 300
      // with 256 each; runs of whole experts per XCD: 394 and 314)
      const int xcd = bid & 7, l0 = bid >> 3;
      const int xn = 8 / a.xm, tm = (a.mt + a.xm - 1) / a.xm, tn = (a.nt + xn - 1) / xn;
      es = l0 / (tm * tn);
      const int l = l0 - es * tm * tn;
      mi = (xcd % a.xm) * tm + l % tm;
      ni = (xcd / a.xm) * tn + l / tm;
      if (es >= a.E * a.splits || mi >= a.mt || ni >= a.nt) return;
    } else {
      const int total = a.E * a.splits * a.mt * a.nt, chunk = (total + 7) / 8;
      int tau = (bid & 7) * chunk + (bid >> 3);
      if (static_cast<int>(bid >> 3) >= chunk || tau >= total) return;
      const int per_e = a.mt * a.nt;
      es = tau / per_e;
      tau -= es * per_e;
      const int per = kMMGroupM * a.nt, g = tau / per, r = tau - g * per;
      const int gm = min(kMMGroupM, a.mt - g * kMMGroupM);
      ni = r / gm;
      mi = g * kMMGroupM + r % gm;
    }
    e = es / a.splits;
    split = es % a.splits;
    n0 = ni * BN;
    m0 = mi * BM;
    mrows = min(BM, a.mdim - m0);
    int lo = 0, hi = a.rows;
    if (a.offsets) {
      lo = min(max(a.offsets[e], 0), a.rows);
      hi = min(max(a.offsets[e + 1], lo), a.rows);
    }
    // equal parts of whole stages
    const int part = ((hi - lo + a.splits - 1) / a.splits + BK - 1) / BK * BK;
    k_begin = __builtin_amdgcn_readfirstlane(min(lo + split * part, hi));
    k_end = __builtin_amdgcn_readfirstlane(min(k_begin + part, hi));
  } else {
    MMTile t;
    const int nts = MODE == kModeNN ? a.nt * a.splits : a.nt;   // a part's tiles: more columns
    if (!mm_find_tile<BM, NTHR>(a.offsets, a.rows, a.E, nts, sm_tile, bid, t)) return;
    if constexpr (MODE == kModeNN) {
      split = __builtin_amdgcn_readfirstlane(t.nt / a.nt);
      t.nt -= split * a.nt;
      const int part = ((a.kdim + a.splits - 1) / a.splits + BK - 1) / BK * BK;
      k_begin = min(split * part, a.kdim);
      k_end = min(k_begin + part, a.kdim);
    } else {
      k_end = a.kdim;
    }
    e = t.e;
    m0 = t.p0;
    mrows = t.p1 - t.p0;
    n0 = t.nt * (swiglu ? BN / 2 : BN);
  }
  const int half_n = a.ndim / 2;
  // W row of the NT tile's B row j. SwiGLU: a wave's first CW/2 rows are gate
  // rows and its last CW/2 the matching up rows, so both halves of an output
  // meet in one lane. -1: past the matrix.
  auto b_row = [&](int j) -> int {
    if (swiglu) {
      const int w = j / CW, c = j % CW, h = c / (CW / 2);
      const int col = n0 + w * (CW / 2) + c % (CW / 2);
      return col < half_n ? h * half_n + col : -1;
    }
    return n0 + j < a.ndim ? n0 + j : -1;
  };

  // ---- operand addresses
  const size_t esz = 2;
  const bool gather = a.slot != nullptr;
  if constexpr (MODE == kModeNT) {
    if (gather) {
      for (int r = tid; r < BM; r += NTHR)
        row_src[r] = r < mrows ? min(max(a.slot[m0 + r] / a.topk, 0), a.x_rows - 1) : -1;
      __syncthreads();
    }
  }
  uint32_t aoff[8], boff[8], akc[8], bkc[8];
  const uint32_t kb = static_cast<uint32_t>(a.kdim) * 2, nb = static_cast<uint32_t>(a.ndim) * 2,
                 mb = static_cast<uint32_t>(a.mdim) * 2;
#pragma unroll
  for (int v = 0; v < G::kAPer; ++v) {
    const int s = tid + NTHR * v;
    if constexpr (kAK) {
      const int row = s / CPR, c = (s % CPR) ^ kmajor_swz<CPR>(row);
      int src = row < mrows ? row : -1;
      if (MODE == kModeNT && gather) src = row_src[row];
      aoff[v] = src < 0 ? kMMPastEnd : static_cast<uint32_t>(src) * kb + c * 16;
      akc[v] = c * 8;
    } else {
      constexpr int CT = BM / 8;
      const int k = s / CT, c = (s % CT) ^ mmajor_swz<BM>(k);
      aoff[v] = m0 + c * 8 < a.mdim ? static_cast<uint32_t>(k) * mb + (m0 + c * 8) * 2 : kMMPastEnd;
      akc[v] = k;
    }
  }
#pragma unroll
  for (int v = 0; v < G::kBPer; ++v) {
    const int s = tid + NTHR * v;
    if constexpr (kBK) {
      const int row = s / CPR, c = (s % CPR) ^ kmajor_swz<CPR>(row);
      const int src = b_row(row);
      boff[v] = src < 0 ? kMMPastEnd : static_cast<uint32_t>(src) * kb + c * 16;
      bkc[v] = c * 8;
    } else {
      constexpr int CT = BN / 8;
      const int k = s / CT, c = (s % CT) ^ mmajor_swz<BN>(k);
      const bool in = n0 + c * 8 < a.ndim;
      boff[v] = in ? static_cast<uint32_t>(k) * nb + (n0 + c * 8) * 2 : kMMPastEnd;
      if (MODE == kModeTN && gather) boff[v] = in ? (n0 + c * 8) * 2 : kMMPastEnd;
      bkc[v] = k;
    }
  }
  const int klen = k_end - k_begin;
  const int steps = (klen + BK - 1) / BK;
  const int wvu = __builtin_amdgcn_readfirstlane(wv);
  const uint8_t* wexp = Bb + static_cast<size_t>(e) * a.kdim * a.ndim * esz;   // NT, NN: W_e

  // Resources whose extent does not move with k
  const uint32_t x_bytes = MODE == kModeNT && gather ? static_cast<uint32_t>(a.x_rows) * kb
                                                     : static_cast<uint32_t>(mrows) * kb - k_begin * 2;
  const __amdgpu_buffer_rsrc_t a_fix = buffer_rsrc(
      MODE == kModeNT && gather ? Ab : Ab + static_cast<size_t>(m0) * kb + (kAK ? k_begin * 2 : 0),
      kAK ? x_bytes : 0);
  const __amdgpu_buffer_rsrc_t b_fix =
      buffer_rsrc(kBK ? wexp : Bb, kBK ? static_cast<uint32_t>(a.ndim) * kb
                                       : MODE == kModeTN && gather
                                             ? static_cast<uint32_t>(a.x_rows) * nb
                                             : 0);

  // TN gather: the source rows of the next stage's loads, read from LDS a stage
  // ahead (past the segment's last stage: unused, held in bounds)
  int srow[8];
  auto read_sources = [&](int st) {
#pragma unroll
    for (int v = 0; v < G::kBPer; ++v) srow[v] = row_src[min(st * BK + static_cast<int>(bkc[v]), kMMSegRows - 1)];
  };

  // Loads of stage st (its buffer: st % STAGES). M-major operands move the
  // resource itself: its end is the last row of the contraction, so rows past
  // it read as zeros.
  auto issue = [&](int st, int seg0) {
    uint8_t* base = mm_lds + (st % STAGES) * G::kStageBytes + wvu * kWave * 16;
    const int k0 = (seg0 + st) * BK;
    const uint32_t left = static_cast<uint32_t>(min(BK, klen - k0));
    if constexpr (kAK) {
#pragma unroll
      for (int v = 0; v < G::kAPer; ++v)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            a_fix, (lds_void_t*)(base + NTHR * v * 16), 16,
            akc[v] < left ? aoff[v] : kMMPastEnd, k0 * 2, 0, 0);
    } else {
      const __amdgpu_buffer_rsrc_t rs =
          buffer_rsrc(Ab + static_cast<size_t>(k_begin + k0) * mb, left * mb);
#pragma unroll
      for (int v = 0; v < G::kAPer; ++v)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void_t*)(base + NTHR * v * 16), 16,
                                                 aoff[v], 0, 0, 0);
    }
    if constexpr (kBK) {
#pragma unroll
      for (int v = 0; v < G::kBPer; ++v)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            b_fix, (lds_void_t*)(base + (G::kASlots + NTHR * v) * 16), 16,
            bkc[v] < left ? boff[v] : kMMPastEnd, k0 * 2, 0, 0);
    } else if (MODE == kModeTN && gather) {
#pragma unroll
      for (int v = 0; v < G::kBPer; ++v) {
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            b_fix, (lds_void_t*)(base + (G::kASlots + NTHR * v) * 16), 16,
            srow[v] < 0 || boff[v] == kMMPastEnd
                ? kMMPastEnd : static_cast<uint32_t>(srow[v]) * nb + boff[v], 0, 0, 0);
      }
      read_sources(st + 1);
    } else {
      const __amdgpu_buffer_rsrc_t rs =
          buffer_rsrc((MODE == kModeTN ? Bb : wexp) + static_cast<size_t>(k_begin + k0) * nb,
                      left * nb);
#pragma unroll
      for (int v = 0; v < G::kBPer; ++v)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            rs, (lds_void_t*)(base + (G::kASlots + NTHR * v) * 16), 16, boff[v], 0, 0, 0);
    }
  };

  f32x16_t acc[4][4];   // MI x NJ used (fixed: captured by a lambda)
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;

  // operand fragment of 16-k step ks at tile row / column `at` (a multiple of 32)
  auto kmajor_frag = [&](const uint8_t* tile, int at, int ks) -> frag_t {
    const int row = at + l32;
    return *reinterpret_cast<const frag_t*>(
        tile + (row * CPR + ((2 * ks + hf) ^ kmajor_swz<CPR>(row))) * 16);
  };
  auto mmajor_frag = [&](const uint8_t* tile, int at, int ks, auto cols) -> frag_t {
    constexpr int COLS = decltype(cols)::value;
    const int k = 16 * ks + 8 * hf + (l16 >> 2);
    const int c = (at + (lane & 16)) / 8 + ((l16 & 3) >> 1);
    const uint8_t* p = tile + (k * (COLS / 8) + (c ^ mmajor_swz<COLS>(k))) * 16 + (l16 & 1) * 8;
    const i32x2_t l2 = tr_read((const lds_s16x4_t*)(p));
    const i32x2_t h2 = tr_read((const lds_s16x4_t*)(p + 4 * COLS * 2));
    return frag_t{l2[0], l2[1], h2[0], h2[1]};
  };
  // fragments of 16-k step ks of the stage at `base`
  auto read_frags = [&](const uint8_t* base, int ks, frag_t (&fa)[4], frag_t (&fb)[4]) {
    const uint8_t* bt = base + G::kASlots * 16;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      if constexpr (kBK) fb[j] = kmajor_frag(bt, wn * CW + j * 32, ks);
      else fb[j] = mmajor_frag(bt, wn * CW + j * 32, ks, std::integral_constant<int, BN>{});
    }
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      if constexpr (kAK) fa[i] = kmajor_frag(base, wm * RW + i * 32, ks);
      else fa[i] = mmajor_frag(base, wm * RW + i * 32, ks, std::integral_constant<int, BM>{});
    }
  };
  // C^T subtiles: a lane ends with 4 consecutive columns n of one row m
  auto multiply = [&](const frag_t (&fa)[4], const frag_t (&fb)[4], auto from, auto to) {
#pragma unroll
    for (int i = decltype(from)::value; i < decltype(to)::value; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j) acc[i][j] = mfma16<T>(fb[j], fa[i], acc[i][j]);
  };
  constexpr std::integral_constant<int, 0> c0{};
  constexpr std::integral_constant<int, MI / 2> c1{};
  constexpr std::integral_constant<int, MI> c2{};
  // LDS reads of one step's fragments, spread over its multiplies
  constexpr int kReads = NJ * (kBK ? 1 : 2) + MI * (kAK ? 1 : 2);
  // a wave whose rows all lie past the tile's last row has nothing to compute
  const bool live = __builtin_amdgcn_readfirstlane(wm) * RW < mrows;

  // Pipeline: the fragments of a 16-k step are read from LDS while the step
  // before it multiplies, across stages too. The one barrier of a stage stands
  // in the middle of its last step: there every wave holds that step's fragments
  // in registers, so the stage's buffer is free for stage st + STAGES, and the
  // first fragments of stage st + 1 (landed by then) can be read; the multiplies
  // issued before it run on while the waves gather. sched_group_barrier keeps
  // LDS reads (0x100), loads (0x020) and MFMAs (0x008) interleaved in that order:
  // left alone, the compiler sinks each read to its use.
  auto run = [&](auto livec, int ns, int seg0) {
    constexpr bool LIVE = decltype(livec)::value;
    frag_t fa[2][4], fb[2][4];
#pragma unroll
    for (int st = 0; st < STAGES; ++st)
      if (st < ns) issue(st, seg0);
    mm_wait_stage<G::kLoads, STAGES - 1>(min(STAGES - 1, ns - 1));
    if constexpr (LIVE) read_frags(mm_lds, 0, fa[0], fb[0]);
    auto stage = [&](int st, auto mainc) {
      constexpr bool MAIN = decltype(mainc)::value;   // stage st + STAGES exists
      const uint8_t* base = mm_lds + (st % STAGES) * G::kStageBytes;
      if constexpr (LIVE) {
#pragma unroll
        for (int ks = 0; ks < KS - 1; ++ks) {
          read_frags(base, ks + 1, fa[(ks + 1) & 1], fb[(ks + 1) & 1]);
          multiply(fa[ks & 1], fb[ks & 1], c0, c2);
          mm_interleave<kReads, 0, MI * NJ>();
        }
        multiply(fa[1], fb[1], c0, c1);
        __builtin_amdgcn_sched_barrier(0);
      }
      if (MAIN || st + 1 < ns) {
        if constexpr (MAIN && STAGES >= 2) mm_wait_barrier<(STAGES - 2) * G::kLoads>();
        else mm_wait_stage<G::kLoads, STAGES - 2>(min(STAGES - 2, ns - 2 - st));
        if constexpr (MAIN) issue(st + STAGES, seg0);
        if constexpr (LIVE) read_frags(mm_lds + ((st + 1) % STAGES) * G::kStageBytes, 0, fa[0], fb[0]);
      }
      if constexpr (LIVE) {
        multiply(fa[1], fb[1], c1, c2);
        mm_interleave<kReads, MAIN ? G::kLoads : 0, (MI - MI / 2) * NJ>();
      }
    };
    int st = 0;
    for (; st + STAGES < ns; ++st) stage(st, std::true_type{});
    for (; st < ns; ++st) stage(st, std::false_type{});
  };

  // ---- where the results go
  const int out_w = swiglu ? half_n : a.ndim;
  const int wcols = swiglu ? CW / 2 : CW;        // output columns of the wave
  const size_t crow = static_cast<size_t>(m0) +
                      (MODE == kModeTN   ? (static_cast<size_t>(e) * a.splits + split) * a.mdim
                       : MODE == kModeNN ? static_cast<size_t>(split) * a.rows
                                         : 0);
  const int col0 = n0 + wn * wcols;
  const int per_row = wcols / 8;                 // lanes per row
  // what is added to 8 columns of a row (NT), as it is stored
  struct Added {
    uint4 bias, bias_up, res, res_hi;   // bias_up: SwiGLU; res_hi: float32
  };
  auto load_added = [&](int row, int col, Added& v) {
    if (a.bias) {
      v.bias = ld16(static_cast<const uint16_t*>(a.bias) + col);
      if (swiglu) v.bias_up = ld16(static_cast<const uint16_t*>(a.bias) + half_n + col);
    }
    if (a.residual) {
      const size_t at = (crow + row) * out_w + col;
      if (a.c_f32) {
        v.res = ld16(static_cast<const float*>(a.residual) + at);
        v.res_hi = ld16(static_cast<const float*>(a.residual) + at + 4);
      } else {
        v.res = ld16(static_cast<const uint16_t*>(a.residual) + at);
      }
    }
  };
  auto load_piece = [&](int i, int it, Added& v) {   // piece `it` of 32 rows i
    const int r = it / per_row, row = wm * RW + i * 32 + r, col = col0 + (it - r * per_row) * 8;
    if (r < 32 && row < mrows && col < out_w) load_added(row, col, v);
  };
  // Waves of one subtile: both of their row pieces are requested here, ahead of the
  // products; otherwise the epilogue requests each a piece ahead.
  constexpr bool kAhead = MODE == kModeNT && MI * NJ == 1;
  Added ahead[2];
  if constexpr (kAhead) {
    load_piece(0, lane, ahead[0]);
    load_piece(0, lane + kWave, ahead[1]);
  }

  constexpr int kSegSteps = kMMSegRows / BK;
  const int seg_len = MODE == kModeTN && gather ? kSegSteps : steps;
  for (int seg0 = 0; seg0 < steps; seg0 += seg_len) {
    const int ns = min(seg_len, steps - seg0);
    if constexpr (MODE == kModeTN) {
      if (gather) {
        __syncthreads();   // the last segment's reads of row_src and of the stages are done
        for (int r = tid; r < ns * BK; r += NTHR) {
          const int p = k_begin + seg0 * BK + r;
          row_src[r] = p < k_end ? min(max(a.slot[p] / a.topk, 0), a.x_rows - 1) : -1;
        }
        __syncthreads();
        read_sources(0);
      }
    }
    if (live) run(std::true_type{}, ns, seg0);
    else run(std::false_type{}, ns, seg0);
  }

  // ---- epilogue. Lane (l32, hf) holds row l32 and columns 8q + 4hf + [0, 4) of
  // each 32 x 32 subtile. 32 rows of a wave's columns at a time pass through a
  // float32 area of LDS that is the wave's own, from where 8 columns of a row go
  // to a lane: whole row pieces are read and written (bias, residual, z, C), and
  // the activation's code stands once instead of once per accumulator.
  __syncthreads();   // the stages are read
  if (!live) return;
  constexpr int kRowF = CW + 4;   // floats per row of the area; + 4: banks
  float* area = reinterpret_cast<float*>(mm_lds) + wvu * 32 * kRowF;
  const bool stream = a.stream_out != 0;
  // rows of C and z: at most 256 of 2^20 values, so 32-bit offsets
  const uint32_t cbytes = static_cast<uint32_t>(out_w) * (a.c_f32 ? 4 : 2);
  const __amdgpu_buffer_rsrc_t c_rs =
      buffer_rsrc(static_cast<uint8_t*>(a.C) + crow * cbytes, mrows * cbytes);
  const __amdgpu_buffer_rsrc_t z_rs =
      buffer_rsrc(static_cast<uint8_t*>(a.z) + (MODE == kModeNT && a.z ? crow * nb : 0),
                  MODE == kModeNT && a.z ? mrows * nb : 0);
  if constexpr (MODE == kModeNT && !kAhead) load_piece(0, lane, ahead[0]);
  for (int i = 0; i < MI; ++i) {
#pragma unroll
    for (int x = 0; x < MI; ++x)
      if (x == i) {
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q)
            *reinterpret_cast<f32x4_t*>(area + l32 * kRowF + j * 32 + q * 8 + hf * 4) =
                f32x4_t{acc[x][j][q * 4], acc[x][j][q * 4 + 1], acc[x][j][q * 4 + 2],
                        acc[x][j][q * 4 + 3]};
      }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    auto piece = [&](int it, const Added& add, auto addedc) {
      constexpr bool ADDED = decltype(addedc)::value;   // a bias or a residual
      const int r = it / per_row, c = (it - r * per_row) * 8;
      const int row = wm * RW + i * 32 + r, col = col0 + c;
      if (row >= mrows || col >= out_w) return;
      float v[8];
      mm_area8(area + r * kRowF + c, v);
      if constexpr (MODE == kModeNT) {
        if (ADDED && a.bias) mm_add8<T>(add.bias, v);
        const uint32_t zoff = (static_cast<uint32_t>(row) * a.ndim + col) * 2;
        if (a.z) {
          mm_put16(mm_pack8<T>(v), z_rs, zoff, stream);
        }
        if (swiglu) {
          float u[8];
          mm_area8(area + r * kRowF + CW / 2 + c, u);
          if (ADDED && a.bias) mm_add8<T>(add.bias_up, u);
          if (a.z) mm_put16(mm_pack8<T>(u), z_rs, zoff + half_n * 2, stream);
          auto gated = [&](auto exact) {
#pragma unroll
            for (int t = 0; t < 8; ++t) v[t] = silu_f32<decltype(exact)::value>(v[t]) * u[t];
          };
          if (a.c_f32) gated(std::true_type{});
          else gated(std::false_type{});
        } else if (a.act != 0) {
          auto activated = [&](auto exact) {
#pragma unroll
            for (int t = 0; t < 8; ++t) v[t] = act_f32<decltype(exact)::value>(v[t], a.act);
          };
          if (a.c_f32) activated(std::true_type{});
          else activated(std::false_type{});
        }
      }
      if (MODE == kModeNT && ADDED && a.residual) {
        if (a.c_f32) {
          const f32x4_t lo = __builtin_bit_cast(f32x4_t, add.res),
                        hi = __builtin_bit_cast(f32x4_t, add.res_hi);
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            v[t] += lo[t];
            v[4 + t] += hi[t];
          }
        } else {
          mm_add8<T>(add.res, v);
        }
      }
      const uint32_t coff = (static_cast<uint32_t>(row) * out_w + col) * (a.c_f32 ? 4 : 2);
      if (a.c_f32) {
        mm_put16(__builtin_bit_cast(i32x4_t, f32x4_t{v[0], v[1], v[2], v[3]}), c_rs, coff, stream);
        mm_put16(__builtin_bit_cast(i32x4_t, f32x4_t{v[4], v[5], v[6], v[7]}), c_rs, coff + 16, stream);
      } else {
        mm_put16(mm_pack8<T>(v), c_rs, coff, stream);
      }
    };
    if constexpr (kAhead) {
      static_assert(CW == 32, "two pieces per lane");
      piece(lane, ahead[0], std::true_type{});
      if (!swiglu) piece(lane + kWave, ahead[1], std::true_type{});
    } else if (MODE == kModeNT && (a.bias || a.residual)) {
      for (int it = lane; it < 32 * per_row; it += kWave) {
        const bool last = it + kWave >= 32 * per_row;
        ahead[1] = ahead[0];
        if (!last || i + 1 < MI) load_piece(last ? i + 1 : i, last ? lane : it + kWave, ahead[0]);
        piece(it, ahead[1], std::true_type{});
      }
    } else {
      // a loop of its own: a wait for `ahead` would be one for the stores before it
      // (32768 x 2048 x 768 to float32 230 us in one loop, 223 in two)
      for (int it = lane; it < 32 * per_row; it += kWave) piece(it, ahead[1], std::false_type{});
    }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  }
}

template <class T, int MODE, class G>
__global__ __launch_bounds__(G::kThreads, G::WPE) void mm_kernel(
    const uint8_t* __restrict__ Ab, const uint8_t* __restrict__ Bb, const MMArgs a) {
  mm_tile<T, MODE, G>(Ab, Bb, a, blockIdx.x);
}

}  // namespace moe
