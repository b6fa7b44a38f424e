// Passes beside the gradient products: dz = act'(z) dy with the bias gradient's
// partial sums, and sums of float32 parts.
#include "launch_block.h"
#include "mm.h"
#include "part_sum.h"

namespace moe {
namespace {

template <class T>
__device__ __forceinline__ void load8(const void* p, size_t at, bool f32, float (&v)[8]) {
  if (f32) {
    const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + at);
    const float4 a = q[0], b = q[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
    const uint4 w = ld16(static_cast<const uint16_t*>(p) + at);
    unpack2<T>(w.x, v[0], v[1]);
    unpack2<T>(w.y, v[2], v[3]);
    unpack2<T>(w.z, v[4], v[5]);
    unpack2<T>(w.w, v[6], v[7]);
  }
}
template <class T>
__device__ __forceinline__ void store8(void* p, size_t at, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + at) =
      make_uint4(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]), pack2<T>(v[4], v[5]),
                 pack2<T>(v[6], v[7]));
}

// A block takes 512 columns of dy (8 per thread) and a strip of rows, four at a
// time; bound by the bytes of dy, z and dz. The column sums stay in registers
// over the strip and are joined in LDS in a fixed order. EXACT (see mm.h): the sums,
// where the bias gradient is float32; dz is the other form's always, so that dx and dw
// are the same bits whether a bias gradient is asked for or not.
constexpr int kDzCols = 512;

// dz is stored in the operands' type: the matrix instructions take 16-bit operands,
// and two parts of it would double both products. Its half step adds to that of the
// results (relative 2-norm of dx and dW: bf16 0.00166 with a float32 dz, 0.00235;
// fp16 0.00021, 0.00029); the bias sums take it unrounded.
template <class T, bool SWIGLU, bool EXACT>
__global__ __launch_bounds__(256) void dz_kernel(const void* __restrict__ dy, int dy_f32,
                                                 const void* __restrict__ z,
                                                 int rows, int N, int act, int strip_rows,
                                                 int col_blocks, void* __restrict__ dz,
                                                 float* __restrict__ part) {
  constexpr int S = SWIGLU ? 2 : 1;
  __shared__ float red[3][S][kDzCols];
  const int No = SWIGLU ? N / 2 : N;
  const int cb = blockIdx.x % col_blocks, strip = blockIdx.x / col_blocks;
  const int tx = threadIdx.x & 63, ty = threadIdx.x >> 6;
  const int col = cb * kDzCols + tx * 8;
  // 64-bit: the last strip's end may pass 2^31
  const long long r0 = static_cast<long long>(strip) * strip_rows;
  const long long r1 = min(r0 + strip_rows, static_cast<long long>(rows));
  float sum[S][8];
#pragma unroll
  for (int s = 0; s < S; ++s)
#pragma unroll
    for (int i = 0; i < 8; ++i) sum[s][i] = 0.0f;
  if (col < No) {
#pragma unroll 2
    for (long long r = r0 + ty; r < r1; r += 4) {
      float d[8], g[8], e[8], du[8], eu[8];   // dz; EXACT: e, what the sums take
      load8<T>(dy, r * No + col, dy_f32, d);
      if (SWIGLU) {
        float u[8];
        load8<T>(z, r * N + col, false, g);
        load8<T>(z, r * N + No + col, false, u);
        if (EXACT)
#pragma unroll
          for (int i = 0; i < 8; ++i) swiglu_grad_f32<true>(d[i], g[i], u[i], e[i], eu[i]);
        if (!EXACT || dz)
#pragma unroll
          for (int i = 0; i < 8; ++i) swiglu_grad_f32<false>(d[i], g[i], u[i], d[i], du[i]);
        if (dz) {
          store8<T>(dz, r * N + col, d);
          store8<T>(dz, r * N + No + col, du);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[S - 1][i] += EXACT ? eu[i] : du[i];
      } else {
        if (act != 0) {   // EXACT: it is not 0
          load8<T>(z, r * N + col, false, g);
          if (EXACT)
#pragma unroll
            for (int i = 0; i < 8; ++i) e[i] = d[i] * act_grad_f32<true>(g[i], act);
          if (!EXACT || dz)
#pragma unroll
            for (int i = 0; i < 8; ++i) d[i] *= act_grad_f32<false>(g[i], act);
        }
        if (dz) store8<T>(dz, r * N + col, d);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) sum[0][i] += EXACT ? e[i] : d[i];
    }
  }
  if (ty > 0)
#pragma unroll
    for (int s = 0; s < S; ++s)
#pragma unroll
      for (int i = 0; i < 8; ++i) red[ty - 1][s][tx * 8 + i] = sum[s][i];
  __syncthreads();
  if (ty == 0 && col < No)
#pragma unroll
    for (int s = 0; s < S; ++s)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float v = sum[s][i];
#pragma unroll
        for (int y = 0; y < 3; ++y) v += red[y][s][tx * 8 + i];
        part[static_cast<size_t>(strip) * N + s * No + col + i] = v;
      }
}

// The same without column sums: 8 values of dy per thread and step, every row
// piece its own thread (a block of columns per row strip leaves a quarter of the
// threads idle at 768 columns: 32768 x 768 SwiGLU 68 us).
template <class T, bool SWIGLU>
__global__ __launch_bounds__(256) void dz_flat_kernel(const void* __restrict__ dy, int dy_f32,
                                                      const void* __restrict__ z,
                                                      const int* __restrict__ offsets, int E,
                                                      int rows, int N, int act,
                                                      void* __restrict__ dz) {
  const int No = SWIGLU ? N / 2 : N;
  const uint32_t per_row = static_cast<uint32_t>(No) / 8;
  long long lo = 0, hi = rows;
  if (offsets) {
    lo = min(max(offsets[0], 0), rows);
    hi = min(max(offsets[E], static_cast<int>(lo)), rows);
  }
  const long long total = (hi - lo) * per_row, step = static_cast<long long>(gridDim.x) * 256;
#pragma unroll 2
  for (long long i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x; i < total; i += step) {
    // a 32-bit division wherever the index allows it
    const long long rr = total <= 0xffffffffLL
                             ? static_cast<long long>(static_cast<uint32_t>(i) / per_row)
                             : i / per_row;
    const size_t r = static_cast<size_t>(lo + rr);
    const int col = static_cast<int>(i - rr * per_row) * 8;
    float d[8], g[8];
    load8<T>(dy, r * No + col, dy_f32, d);
    if (SWIGLU) {
      float u[8], du[8];
      load8<T>(z, r * N + col, false, g);
      load8<T>(z, r * N + No + col, false, u);
#pragma unroll
      for (int x = 0; x < 8; ++x) swiglu_grad_f32<false>(d[x], g[x], u[x], d[x], du[x]);
      store8<T>(dz, r * N + col, d);
      store8<T>(dz, r * N + No + col, du);
    } else {
      if (act != 0) {
        load8<T>(z, r * N + col, false, g);
#pragma unroll
        for (int x = 0; x < 8; ++x) d[x] *= act_grad_f32<false>(g[x], act);
      }
      store8<T>(dz, r * N + col, d);
    }
  }
}

__device__ __forceinline__ void sum_splits_block(const SplitSum& a, uint32_t bid, uint32_t blocks) {
  const long long n4 = a.n / 4, total4 = n4 * a.E;
  for (long long i = static_cast<long long>(bid) * 256 + threadIdx.x; i < total4;
       i += static_cast<long long>(blocks) * 256) {
    const long long e = i / n4, c = i - e * n4;
    const float4* p = reinterpret_cast<const float4*>(a.part) + e * a.splits * n4 + c;
    float4 v = p[0];
#pragma unroll 4
    for (int s = 1; s < a.splits; ++s) {
      const float4 w = p[s * n4];
      v.x += w.x;
      v.y += w.y;
      v.z += w.z;
      v.w += w.w;
    }
    if (a.out_type == 2) {
      reinterpret_cast<float4*>(a.out)[i] = v;
    } else if (a.out_type == 0) {
      reinterpret_cast<uint2*>(a.out)[i] = make_uint2(pack2<bf16_tag>(v.x, v.y), pack2<bf16_tag>(v.z, v.w));
    } else {
      reinterpret_cast<uint2*>(a.out)[i] = make_uint2(pack2<fp16_tag>(v.x, v.y), pack2<fp16_tag>(v.z, v.w));
    }
  }
}

// One launch for all sums of a call: a launch of a few us each would cost more
// than the sums.
__global__ __launch_bounds__(256) void sums_kernel(const SplitSum a, const SplitSum b,
                                                   const PartSum c, uint32_t a_blocks,
                                                   uint32_t b_blocks) {
  if (blockIdx.x < a_blocks) sum_splits_block(a, blockIdx.x, a_blocks);
  else if (blockIdx.x < a_blocks + b_blocks) sum_splits_block(b, blockIdx.x - a_blocks, b_blocks);
  else sum_parts_block(c, blockIdx.x - a_blocks - b_blocks);
}

// Rows of a strip: as many strips as fill the chip (about 768 blocks of 512
// columns: 4093 x 1536 9 us, 23 us with 192 blocks), and no more, since their sums
// are read again.
int most_strips(int No) {
  const int cb = (No + kDzCols - 1) / kDzCols;
  return cb >= 768 ? 1 : 768 / cb;
}
int strip_rows_of(int rows, int No) {
  const int strips = most_strips(No);
  const int r = static_cast<int>((static_cast<long long>(rows) + strips - 1) / strips);
  return r < 8 ? 8 : (r + 3) / 4 * 4;
}

}  // namespace

int dz_strips(int rows, int N, int act) {
  const int sr = strip_rows_of(rows, act == kActSwiglu ? N / 2 : N);
  return static_cast<int>((static_cast<long long>(rows) + sr - 1) / sr);
}

int dz_most_strips(int rows, int N, int act) {
  const int s = most_strips(act == kActSwiglu ? N / 2 : N);
  const int all = static_cast<int>((static_cast<long long>(rows) + 7) / 8);
  return all < s ? all : s;
}

hipError_t launch_dz(const void* dy, bool dy_f32, const void* z, const int* offsets, int E,
                     int rows, int N, int act, bool fp16, void* dz, float* part, bool part_f32,
                     hipStream_t s) {
  if (rows == 0) return hipSuccess;
  const int No = act == kActSwiglu ? N / 2 : N;
  const int cb = (No + kDzCols - 1) / kDzCols;
  const int sr = strip_rows_of(rows, No);
  const dim3 grid(static_cast<unsigned>(dz_strips(rows, N, act)) * cb), block(256);
  const int f = dy_f32;
  if (part == nullptr) {
    const long long n = (static_cast<long long>(rows) * (No / 8) + 511) / 512;
    const dim3 flat(static_cast<unsigned>(n < 65536 ? n : 65536));
    if (act == kActSwiglu) {
      if (fp16) dz_flat_kernel<fp16_tag, true><<<flat, block, 0, s>>>(dy, f, z, offsets, E, rows, N, act, dz);
      else dz_flat_kernel<bf16_tag, true><<<flat, block, 0, s>>>(dy, f, z, offsets, E, rows, N, act, dz);
    } else {
      if (fp16) dz_flat_kernel<fp16_tag, false><<<flat, block, 0, s>>>(dy, f, z, offsets, E, rows, N, act, dz);
      else dz_flat_kernel<bf16_tag, false><<<flat, block, 0, s>>>(dy, f, z, offsets, E, rows, N, act, dz);
    }
    return hipGetLastError();
  }
  auto run = [&](auto tag, auto swiglu, auto exact) {
    dz_kernel<decltype(tag), decltype(swiglu)::value, decltype(exact)::value>
        <<<grid, block, 0, s>>>(dy, f, z, rows, N, act, sr, cb, dz, part);
  };
  auto typed = [&](auto tag) {
    if (act == kActSwiglu) {
      if (part_f32) run(tag, std::true_type{}, std::true_type{});
      else run(tag, std::true_type{}, std::false_type{});
    } else if (part_f32 && act != 0) {
      run(tag, std::false_type{}, std::true_type{});
    } else {
      run(tag, std::false_type{}, std::false_type{});
    }
  };
  if (fp16) typed(fp16_tag{});
  else typed(bf16_tag{});
  return hipGetLastError();
}

hipError_t launch_sums(const SplitSum& a, const SplitSum& b, const PartSum& c, hipStream_t s) {
  auto blocks = [](const SplitSum& v) -> uint32_t {
    const long long n = v.out ? (v.n / 4 * v.E + 255) / 256 : 0;
    return static_cast<uint32_t>(n < 4096 ? n : 4096);
  };
  const uint32_t ab = blocks(a), bb = blocks(b), grid = ab + bb + sum_parts_blocks(c);
  if (grid == 0) return hipSuccess;
  sums_kernel<<<grid, 256, 0, s>>>(a, b, c, ab, bb);
  return hipGetLastError();
}

}  // namespace moe
