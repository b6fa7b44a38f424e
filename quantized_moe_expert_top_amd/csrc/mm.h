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

struct bf16_tag {};
struct fp16_tag {};

template <class T>
__device__ __forceinline__ f32x16_t mfma16(uint4 a, uint4 b, f32x16_t c) {
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

// Activations and their derivatives in float32. The exponential and reciprocal
// are the hardware's (about 1 ulp); silu(z) for z below about -88 is -0 through
// a zero reciprocal.
__device__ __forceinline__ float sigmoid_f32(float z) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-z * 1.4426950408889634f));
}
__device__ __forceinline__ float act_f32(float z, int act) {
  if (act == 1) return z > 0.0f ? z : (z != z ? z : 0.0f);   // relu; NaN stays
  if (act == 2) return z * sigmoid_f32(z);
  // gelu as z/2 erfc(-z / sqrt 2): no cancellation for negative z
  if (act == 3) return 0.5f * z * erfcf(-0.70710678118654752f * z);
  return z;
}
__device__ __forceinline__ float act_grad_f32(float z, int act) {
  if (act == 1) return z > 0.0f ? 1.0f : (z != z ? z : 0.0f);
  if (act == 2) {
    const float s = sigmoid_f32(z);
    return s * (1.0f + z * (1.0f - s));
  }
  if (act == 3)   // cdf + z pdf
    return 0.5f * erfcf(-0.70710678118654752f * z) +
           z * 0.39894228040143268f * __builtin_amdgcn_exp2f(-0.72134752044448170f * z * z);
  return 1.0f;
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
  int splits;            // TN: parts of an expert's rows, each to its own C
  int nt;                // n tiles
  int mt;                // TN: m tiles
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
  static constexpr int kLds = STAGES * kStageBytes;
  static constexpr int kLoads = kAPer + kBPer;                 // per thread and stage
  static_assert(kASlots % kThreads == 0 && kBSlots % kThreads == 0, "slots split evenly");
  static_assert(kAPer >= 1 && kAPer <= 8 && kBPer >= 1 && kBPer <= 8, "slot arrays hold eight");
  static_assert(MI >= 1 && MI <= 4 && NJ >= 1 && NJ <= 4, "accumulator array holds 4 x 4");
  static_assert(BK == 32 || BK == 64, "swizzles below");
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

template <int N>
__device__ __forceinline__ void mm_wait_barrier() {
  // s_waitcnt vmcnt(N), then the barrier: the immediate carries the count
  asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(N) : "memory");
}
template <int LPS, int MAXL>
__device__ __forceinline__ void mm_wait_stage(int later) {
  if constexpr (MAXL >= 3) { if (later >= 3) { mm_wait_barrier<3 * LPS>(); return; } }
  if constexpr (MAXL >= 2) { if (later == 2) { mm_wait_barrier<2 * LPS>(); return; } }
  if constexpr (MAXL >= 1) { if (later == 1) { mm_wait_barrier<LPS>(); return; } }
  mm_wait_barrier<0>();
}

constexpr uint32_t kMMPastEnd = 0x80000000u;   // at or past the end of every resource here
constexpr int kMMSegRows = 2048;               // TN gather: source rows held in LDS at a time
constexpr int kMMGroupM = 8;                   // m tiles walked together over all n tiles

// Tile of a row-grouped product (NT, NN). Tiles are ordered expert by expert;
// inside an expert, groups of kMMGroupM m tiles walk the n tiles together. Each
// XCD (blockIdx % 8) takes a contiguous run of that order, so that the tiles
// it holds at one time share W strips and x rows in its L2. Offsets are clamped
// to [0, rows] and a block's end to its start, so that values outside the
// contract cannot lead out of the buffers. Returns false for a block without a tile.
struct MMTile {
  int e, nt, p0, p1;   // rows [p0, p1), at most BM of them
};
template <int BM, int NTHR>
__device__ __forceinline__ bool mm_find_tile(const int* __restrict__ offsets, int rows, int E,
                                             int NT, int* sm, MMTile& t) {
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wv = tid >> 6;
  int e = 0, local = 0, mtiles = 0, beg = 0, end = 0;
  if (offsets == nullptr) {
    mtiles = (rows + BM - 1) / BM;
    const int total = mtiles * NT, chunk = (total + 7) / 8;
    local = (blockIdx.x & 7) * chunk + (blockIdx.x >> 3);
    if (static_cast<int>(blockIdx.x >> 3) >= chunk || local >= total) return false;
    end = rows;
  } else {
    constexpr int kPer = 1024 / NTHR > 0 ? 1024 / NTHR : 1;   // E <= 1024
    const int ept = (E + NTHR - 1) / NTHR;
    int cnt[kPer], b[kPer], n[kPer], sum = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int ei = tid * ept + i;
      int c = 0, lo = 0, hi = 0;
      if (i < ept && ei < E) {
        lo = min(max(offsets[ei], 0), rows);
        hi = min(max(offsets[ei + 1], lo), rows);
        c = (hi - lo + BM - 1) / BM * NT;
      }
      cnt[i] = c;
      b[i] = lo;
      n[i] = hi;
      sum += c;
    }
    int incl = sum;
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
      const int o = __shfl_up(incl, d, kWave);
      if (lane >= d) incl += o;
    }
    if (lane == kWave - 1) sm[wv] = incl;
    __syncthreads();
    int before = 0, total = 0;
#pragma unroll
    for (int i = 0; i < NTHR / kWave; ++i) {
      const int s = sm[i];
      if (i < wv) before += s;
      total += s;
    }
    const int chunk = (total + 7) / 8;
    const int tau = (blockIdx.x & 7) * chunk + (blockIdx.x >> 3);
    if (static_cast<int>(blockIdx.x >> 3) >= chunk || tau >= total) return false;   // uniform
    int start = before + incl - sum;
    int* out = sm + NTHR / kWave;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      if (tau >= start && tau < start + cnt[i]) {
        out[0] = tid * ept + i;
        out[1] = tau - start;
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
    mtiles = (end - beg + BM - 1) / BM;
  }
  const int per = kMMGroupM * NT, g = local / per, r = local - g * per;
  const int gm = min(kMMGroupM, mtiles - g * kMMGroupM);
  t.e = e;
  t.nt = r / gm;
  t.p0 = beg + (g * kMMGroupM + r % gm) * BM;
  t.p1 = min(end, t.p0 + BM);
  return true;
}

template <class T, int MODE, class G>
__global__ __launch_bounds__(G::kThreads, G::WPE) void mm_kernel(const MMArgs a) {
  constexpr int BM = G::BM, BN = G::BN, BK = G::BK, NTHR = G::kThreads, STAGES = G::STAGES;
  constexpr int MI = G::MI, NJ = G::NJ, CPR = BK / 8;
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
  int k_begin = 0, k_end = 0;       // TN: rows contracted over
  int split = 0;
  if constexpr (MODE == kModeTN) {
    const int total = a.E * a.splits * a.mt * a.nt, chunk = (total + 7) / 8;
    int tau = (blockIdx.x & 7) * chunk + (blockIdx.x >> 3);
    if (static_cast<int>(blockIdx.x >> 3) >= chunk || tau >= total) return;
    const int per_e = a.mt * a.nt;
    const int es = tau / per_e;
    tau -= es * per_e;
    e = es / a.splits;
    split = es % a.splits;
    const int per = kMMGroupM * a.nt, g = tau / per, r = tau - g * per;
    const int gm = min(kMMGroupM, a.mt - g * kMMGroupM);
    n0 = (r / gm) * BN;
    m0 = (g * kMMGroupM + r % gm) * BM;
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
    if (!mm_find_tile<BM, NTHR>(a.offsets, a.rows, a.E, a.nt, sm_tile, t)) return;
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
  const uint8_t* Ab = static_cast<const uint8_t*>(a.A);
  const uint8_t* Bb = static_cast<const uint8_t*>(a.B);
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
  const int klen = MODE == kModeTN ? k_end - k_begin : a.kdim;
  const int steps = (klen + BK - 1) / BK;
  const int wvu = __builtin_amdgcn_readfirstlane(wv);
  const uint8_t* wexp = Bb + static_cast<size_t>(e) * a.kdim * a.ndim * esz;   // NT, NN: W_e

  // Resources whose extent does not move with k
  const uint32_t x_bytes = MODE == kModeNT && gather ? static_cast<uint32_t>(a.x_rows) * kb
                                                     : static_cast<uint32_t>(mrows) * kb;
  const __amdgpu_buffer_rsrc_t a_fix = buffer_rsrc(
      MODE == kModeNT && gather ? Ab : Ab + static_cast<size_t>(m0) * kb, kAK ? x_bytes : 0);
  const __amdgpu_buffer_rsrc_t b_fix =
      buffer_rsrc(kBK ? wexp : Bb, kBK ? static_cast<uint32_t>(a.ndim) * kb
                                       : MODE == kModeTN && gather
                                             ? static_cast<uint32_t>(a.x_rows) * nb
                                             : 0);

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
        const int src = row_src[st * BK + bkc[v]];
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            b_fix, (lds_void_t*)(base + (G::kASlots + NTHR * v) * 16), 16,
            src < 0 || boff[v] == kMMPastEnd ? kMMPastEnd
                                             : static_cast<uint32_t>(src) * nb + boff[v], 0, 0, 0);
      }
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
  auto kmajor_frag = [&](const uint8_t* tile, int at, int ks) -> uint4 {
    const int row = at + l32;
    return *reinterpret_cast<const uint4*>(
        tile + (row * CPR + ((2 * ks + hf) ^ kmajor_swz<CPR>(row))) * 16);
  };
  auto mmajor_frag = [&](const uint8_t* tile, int at, int ks, auto cols) -> uint4 {
    constexpr int COLS = decltype(cols)::value;
    const int k = 16 * ks + 8 * hf + (l16 >> 2);
    const int c = (at + (lane & 16)) / 8 + ((l16 & 3) >> 1);
    const uint8_t* p = tile + (k * (COLS / 8) + (c ^ mmajor_swz<COLS>(k))) * 16 + (l16 & 1) * 8;
    const s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t*)(p));
    const s16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t*)(p + 4 * COLS * 2));
    const uint2 l2 = __builtin_bit_cast(uint2, lo), h2 = __builtin_bit_cast(uint2, hi);
    return make_uint4(l2.x, l2.y, h2.x, h2.y);
  };
  auto compute = [&](const uint8_t* base) {
    const uint8_t* at = base;
    const uint8_t* bt = base + G::kASlots * 16;
#pragma unroll
    for (int ks = 0; ks < BK / 16; ++ks) {
      uint4 fa[MI], fb[NJ];
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        if constexpr (kAK) fa[i] = kmajor_frag(at, wm * RW + i * 32, ks);
        else fa[i] = mmajor_frag(at, wm * RW + i * 32, ks, std::integral_constant<int, BM>{});
      }
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        if constexpr (kBK) fb[j] = kmajor_frag(bt, wn * CW + j * 32, ks);
        else fb[j] = mmajor_frag(bt, wn * CW + j * 32, ks, std::integral_constant<int, BN>{});
      }
      // C^T subtiles: a lane ends with 4 consecutive columns n of one row m
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j) acc[i][j] = mfma16<T>(fb[j], fa[i], acc[i][j]);
    }
  };
  // a wave whose rows all lie past the tile's last row has nothing to compute
  const bool live = __builtin_amdgcn_readfirstlane(wm) * RW < mrows;

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
      }
    }
#pragma unroll
    for (int st = 0; st < STAGES - 1; ++st)
      if (st < ns) issue(st, seg0);
    for (int st = 0; st < ns; ++st) {
      // stage st has landed once at most the later stages' loads are in flight;
      // the barrier also ends every wave's reads of the buffer issued next
      mm_wait_stage<G::kLoads, STAGES - 2>(min(STAGES - 2, ns - 1 - st));
      if (st + STAGES - 1 < ns) issue(st + STAGES - 1, seg0);
      if (live) compute(mm_lds + (st % STAGES) * G::kStageBytes);
    }
  }
  if (!live) return;

  // ---- epilogue: lane (l32, hf) holds row l32 and columns 8q + 4hf + [0, 4) of
  // each 32 x 32 subtile
  const int out_w = swiglu ? half_n : a.ndim;
  const int nj_out = swiglu ? NJ / 2 : NJ;
#pragma unroll
  for (int i = 0; i < MI; ++i) {
    const int row = wm * RW + i * 32 + l32;
    if (row >= mrows) continue;
    const size_t p = static_cast<size_t>(m0) + row;
    size_t cp = p;
    if (MODE == kModeTN)
      cp = (static_cast<size_t>(e) * a.splits + split) * a.mdim + p;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      if (j >= nj_out) continue;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int col = n0 + (swiglu ? wn * (CW / 2) : wn * CW) + j * 32 + q * 8 + hf * 4;
        if (col >= out_w) continue;
        float v[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) v[t] = acc[i][j][q * 4 + t];
        if constexpr (MODE == kModeNT) {
          if (a.bias) {
            const uint2 bw = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(a.bias) + col);
            float b[4];
            unpack2<T>(bw.x, b[0], b[1]);
            unpack2<T>(bw.y, b[2], b[3]);
#pragma unroll
            for (int t = 0; t < 4; ++t) v[t] += b[t];
          }
          uint16_t* zrow = static_cast<uint16_t*>(a.z);
          if (zrow) {
            zrow += p * a.ndim;
            *reinterpret_cast<uint2*>(zrow + col) = make_uint2(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]));
          }
          if (swiglu) {
            if constexpr (NJ >= 2) {
              float u[4];
#pragma unroll
              for (int t = 0; t < 4; ++t) u[t] = acc[i][(j + NJ / 2) % NJ][q * 4 + t];
              if (a.bias) {
                const uint2 bw = *reinterpret_cast<const uint2*>(
                    static_cast<const uint16_t*>(a.bias) + half_n + col);
                float b[4];
                unpack2<T>(bw.x, b[0], b[1]);
                unpack2<T>(bw.y, b[2], b[3]);
#pragma unroll
                for (int t = 0; t < 4; ++t) u[t] += b[t];
              }
              if (zrow)
                *reinterpret_cast<uint2*>(zrow + half_n + col) =
                    make_uint2(pack2<T>(u[0], u[1]), pack2<T>(u[2], u[3]));
#pragma unroll
              for (int t = 0; t < 4; ++t) v[t] = act_f32(v[t], 2) * u[t];
            }
          } else {
#pragma unroll
            for (int t = 0; t < 4; ++t) v[t] = act_f32(v[t], a.act);
          }
        }
        const size_t at = cp * out_w + col;
        if (MODE == kModeNT && a.residual) {
          if (a.c_f32) {
            const float4 r4 = *reinterpret_cast<const float4*>(static_cast<const float*>(a.residual) + at);
            v[0] += r4.x;
            v[1] += r4.y;
            v[2] += r4.z;
            v[3] += r4.w;
          } else {
            const uint2 rw = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(a.residual) + at);
            float r[4];
            unpack2<T>(rw.x, r[0], r[1]);
            unpack2<T>(rw.y, r[2], r[3]);
#pragma unroll
            for (int t = 0; t < 4; ++t) v[t] += r[t];
          }
        }
        if (a.c_f32)
          *reinterpret_cast<float4*>(static_cast<float*>(a.C) + at) = make_float4(v[0], v[1], v[2], v[3]);
        else
          *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.C) + at) =
              make_uint2(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]));
      }
    }
  }
}

}  // namespace moe
