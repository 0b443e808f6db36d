// 8-bit block quantisation and the elementwise passes of the Muon step.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "bcjr_tc.cuh"

namespace bcjr {
namespace quant {

enum InType { IN_F32 = 0, IN_F16 = 1, IN_BF16 = 2 };

template <int T>
struct In;
template <>
struct In<IN_F32> {
  using type = float;
  static __device__ __forceinline__ float get(float v) { return v; }
  static __device__ __forceinline__ void get4(const float* p, float (&v)[4]) {
    const float4 u = *reinterpret_cast<const float4*>(p);
    v[0] = u.x; v[1] = u.y; v[2] = u.z; v[3] = u.w;
  }
};
template <>
struct In<IN_F16> {
  using type = __half;
  static __device__ __forceinline__ float get(__half v) { return __half2float(v); }
  static __device__ __forceinline__ void get4(const __half* p, float (&v)[4]) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&u.x));
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&u.y));
    v[0] = a.x; v[1] = a.y; v[2] = b.x; v[3] = b.y;
  }
};
template <>
struct In<IN_BF16> {
  using type = __nv_bfloat16;
  static __device__ __forceinline__ float get(__nv_bfloat16 v) { return __bfloat162float(v); }
  static __device__ __forceinline__ void get4(const __nv_bfloat16* p, float (&v)[4]) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    v[0] = __uint_as_float(u.x << 16); v[1] = __uint_as_float(u.x & 0xFFFF0000u);
    v[2] = __uint_as_float(u.y << 16); v[3] = __uint_as_float(u.y & 0xFFFF0000u);
  }
};

struct QuantParams {
  const void* x;
  const float* minus;          // or null
  uint8_t *q, *s, *qt, *st;    // q and s, or qt and st, may be null
  int64_t ld_x, ld_minus, ld_q, ld_s, ld_qt, ld_st;
  int rows, cols, tiles_c;
  int vec;                     // rows of x (and minus) start on 4-element boundaries
  int tiles;
};

constexpr int kThreads = 512;
constexpr int kTile = 128;
constexpr int kRows = 8;       // rows of a warp

// Exponent of the block's scale from the largest |x| as fp32 bits: the least
// e >= -127 with |x| <= FMAX 2^e, FMAX = 0.875 * 2^TOP (448 or 57344), 0 for a
// block of zeros, as the byte e + 127; 255 (NaN) if a value is not finite.
// |x| = 1.m 2^(E - 127) fits 0.875 2^(TOP + e) if 1.m <= 1.75 and E - 126 <= TOP + e.
template <int TOP>
__device__ __forceinline__ uint32_t scale_byte(uint32_t bits) {
  if (bits >= 0x7F800000u) return 255u;
  if (bits == 0) return 127u;
  const int e = (int)(bits >> 23) - 126 - TOP + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return (uint32_t)(max(e, -127) + 127);
}
// 2^-e, exact (e >= -127 and e <= 128 - TOP), NaN for the byte 255.
__device__ __forceinline__ float scale_factor(uint32_t byte) {
  return byte == 255u ? __uint_as_float(0x7FFFFFFFu) : __uint_as_float((254u - byte) << 23);
}

template <bool E5M2>
__device__ __forceinline__ uint32_t codes2(float lo, float hi) {
  uint16_t r;
  if (E5M2) asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  else asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
template <bool E5M2>
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
  return codes2<E5M2>(a, b) | (codes2<E5M2>(c, d) << 16);
}

// Asynchronous copy of up to N bytes (8 or 16) to shared memory, zeros behind them.
template <int N>
__device__ __forceinline__ void copy_async(void* dst, const void* src, int bytes) {
  const uint32_t d = static_cast<uint32_t>(__cvta_generic_to_shared(dst));
  if (N == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d), "l"(src), "r"(bytes) : "memory");
  else asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(d), "l"(src), "r"(bytes) : "memory");
}

// One block takes one 128 x 128 tile of x: warp w the rows 8 w .. 8 w + 7,
// lane l the columns 4 l .. 4 l + 3, so a tile is read once, in 16-byte loads
// that are all in flight at once, and stays in registers for both layouts.  The
// largest |x| of a row is one warp reduction on the fp32 bits (for values that
// are not negative their order is the numbers' order, NaN above all); those of
// the columns, or of the tile, meet in shared memory.  The codes of x^T go
// through shared memory as words of four rows, word index xor (column / 4), so
// that neither side has bank conflicts.
// Blocks take tiles in turn.  PIPE: the next tile's values are on their way into
// shared memory (cp.async, each thread fetching just what it will read, so no
// barrier guards them) while this one is worked on and stored.
// ROW_BLOCKS: one scale for each row (or column) and 128 values; else one for the tile.
// 8192 x 8192 fp32 minus fp32 to both layouts: 105 to 113 us, 6.0 to 6.4 TB/s of the
// measured 6.57 (without PIPE 148 us: between a tile's loads and its stores its SM
// asked for nothing).  4003 x 2048 bf16 to both: 12 us, a tile's own latency twice.
template <int T, bool E5M2, bool ROW_BLOCKS, bool PIPE>
__global__ void __launch_bounds__(kThreads, 2) quantise_kernel(const QuantParams p) {
  constexpr int TOP = E5M2 ? 16 : 9;
  using X = typename In<T>::type;
  constexpr int kBytes = 4 * (int)sizeof(X);
  extern __shared__ __align__(16) uint8_t fetched[];   // PIPE: [8 rows][512 threads] of 4 values of x, then of minus
  __shared__ alignas(16) uint32_t most[16][kTile];
  __shared__ uint32_t words[kTile][32];
  tc::launch_dependents();
  tc::wait_for_earlier();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint8_t* mine = fetched + threadIdx.x * kBytes;
  uint8_t* mine_minus = fetched + kRows * kThreads * kBytes + threadIdx.x * 16;
  auto fetch = [&](int tile) {
    const int r0 = tile / p.tiles_c * kTile + warp * kRows, c = tile % p.tiles_c * kTile + 4 * lane;
    const int n = max(0, min(4, p.cols - c));        // values of a row
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const bool some = r0 + i < p.rows && n > 0;
      const X* x = static_cast<const X*>(p.x) + (some ? (int64_t)(r0 + i) * p.ld_x + c : 0);
      copy_async<kBytes>(mine + i * kThreads * kBytes, x, some ? n * (int)sizeof(X) : 0);
    }
    if (p.minus != nullptr) {
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const bool some = r0 + i < p.rows && n > 0;
        const float* m = p.minus + (some ? (int64_t)(r0 + i) * p.ld_minus + c : 0);
        copy_async<16>(mine_minus + i * kThreads * 16, m, some ? 4 * n : 0);
      }
    }
  };
  if (PIPE) fetch(blockIdx.x);
  for (int tile = blockIdx.x; tile < p.tiles; tile += gridDim.x) {
    const int tr = tile / p.tiles_c, tc = tile % p.tiles_c;
    const int r0 = tr * kTile + warp * kRows, c0 = tc * kTile, c = c0 + 4 * lane;
    const int live = min(kRows, p.rows - r0);            // rows of this warp, may be <= 0
    float v[kRows][4];
    if (PIPE) {
      asm volatile("cp.async.wait_all;" ::: "memory");
#pragma unroll
      for (int i = 0; i < kRows; ++i) In<T>::get4(reinterpret_cast<const X*>(mine + i * kThreads * kBytes), v[i]);
      if (p.minus != nullptr) {
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
          float u[4];
          In<IN_F32>::get4(reinterpret_cast<const float*>(mine_minus + i * kThreads * 16), u);
#pragma unroll
          for (int j = 0; j < 4; ++j) v[i][j] = __fsub_rn(v[i][j], u[j]);
        }
      }
      if (tile + (int)gridDim.x < p.tiles) fetch(tile + gridDim.x);
    } else {
      const X* x = static_cast<const X*>(p.x) + (int64_t)r0 * p.ld_x + c;
      const bool whole = live == kRows && c + 4 <= p.cols && p.vec;
      if (whole) {
#pragma unroll
        for (int i = 0; i < kRows; ++i) In<T>::get4(x + (int64_t)i * p.ld_x, v[i]);
      } else {
#pragma unroll
        for (int i = 0; i < kRows; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            v[i][j] = (i < live && c + j < p.cols) ? In<T>::get(x[(int64_t)i * p.ld_x + j]) : 0.f;
      }
      if (p.minus != nullptr) {
        const float* m = p.minus + (int64_t)r0 * p.ld_minus + c;
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
          float u[4] = {0.f, 0.f, 0.f, 0.f};
          if (whole) {
            In<IN_F32>::get4(m + (int64_t)i * p.ld_minus, u);
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (i < live && c + j < p.cols) u[j] = m[(int64_t)i * p.ld_minus + j];
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) v[i][j] = __fsub_rn(v[i][j], u[j]);
        }
      }
    }

    uint32_t col[4] = {0, 0, 0, 0};
    uint32_t rowb[kRows];                                 // row scales as bytes
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      uint32_t b[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        b[j] = __float_as_uint(v[i][j]) & 0x7FFFFFFFu;
        col[j] = max(col[j], b[j]);
      }
      if (ROW_BLOCKS && p.q != nullptr)
        rowb[i] = scale_byte<TOP>(__reduce_max_sync(0xFFFFFFFFu, max(max(b[0], b[1]), max(b[2], b[3]))));
    }
    uint32_t tile_byte = 0;
    if (!ROW_BLOCKS) {
      const uint32_t m = __reduce_max_sync(0xFFFFFFFFu, max(max(col[0], col[1]), max(col[2], col[3])));
      if (lane == 0) most[warp][0] = m;
      __syncthreads();
      uint32_t a = 0;
#pragma unroll
      for (int w = 0; w < 16; ++w) a = max(a, most[w][0]);
      tile_byte = scale_byte<TOP>(a);
#pragma unroll
      for (int i = 0; i < kRows; ++i) rowb[i] = tile_byte;
    }

    if (p.q != nullptr) {
      if (ROW_BLOCKS) {
        if (lane == 0) {
#pragma unroll
          for (int i = 0; i < kRows; ++i)
            if (i < live) p.s[(int64_t)(r0 + i) * p.ld_s + tc] = (uint8_t)rowb[i];
        }
      } else if (threadIdx.x == 0) {
        p.s[(int64_t)tr * p.ld_s + tc] = (uint8_t)tile_byte;
      }
      uint8_t* q = p.q + (int64_t)r0 * p.ld_q + c;
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        if (i >= live) break;
        const float f = scale_factor(rowb[i]);
        const uint32_t w = codes4<E5M2>(v[i][0] * f, v[i][1] * f, v[i][2] * f, v[i][3] * f);
        if (c + 4 <= p.cols) {
          *reinterpret_cast<uint32_t*>(q + (int64_t)i * p.ld_q) = w;
        } else {
#pragma unroll
          for (int j = 0; j < 3; ++j)
            if (c + j < p.cols) q[(int64_t)i * p.ld_q + j] = (uint8_t)(w >> (8 * j));
        }
      }
    }

    if (p.qt != nullptr) {
      uint32_t colb[4];
      if (ROW_BLOCKS) {
        *reinterpret_cast<uint4*>(&most[warp][4 * lane]) = make_uint4(col[0], col[1], col[2], col[3]);
        __syncthreads();
        if (threadIdx.x < kTile) {
          uint32_t a = 0;
#pragma unroll
          for (int w = 0; w < 16; ++w) a = max(a, most[w][threadIdx.x]);
          a = scale_byte<TOP>(a);
          most[0][threadIdx.x] = a;    // its own column's: nobody else reads it before the barrier
          if (c0 + (int)threadIdx.x < p.cols) p.st[(int64_t)(c0 + threadIdx.x) * p.ld_st + tr] = (uint8_t)a;
        }
        __syncthreads();
        const uint4 b = *reinterpret_cast<const uint4*>(&most[0][4 * lane]);
        colb[0] = b.x; colb[1] = b.y; colb[2] = b.z; colb[3] = b.w;
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) colb[j] = tile_byte;
        if (threadIdx.x == 0) p.st[(int64_t)tc * p.ld_st + tr] = (uint8_t)tile_byte;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float f = scale_factor(colb[j]);
#pragma unroll
        for (int i = 0; i < kRows; i += 4)
          words[4 * lane + j][(warp * (kRows / 4) + i / 4) ^ lane] = codes4<E5M2>(v[i][j] * f, v[i + 1][j] * f, v[i + 2][j] * f, v[i + 3][j] * f);
      }
      __syncthreads();
      const int r = tr * kTile + 4 * lane;             // four rows of x, now columns
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const int cl = warp * kRows + i;
        if (c0 + cl >= p.cols) break;
        const uint32_t w = words[cl][lane ^ (cl >> 2)];
        uint8_t* q = p.qt + (int64_t)(c0 + cl) * p.ld_qt + r;
        if (r + 4 <= p.rows) {
          *reinterpret_cast<uint32_t*>(q) = w;
        } else {
#pragma unroll
          for (int j = 0; j < 3; ++j)
            if (r + j < p.rows) q[j] = (uint8_t)(w >> (8 * j));
        }
      }
    }
    __syncthreads();   // the next tile's sums and words
  }
}

// ------------------------------------------------------------ Muon's elementwise passes

constexpr int kUpdateThreads = 256;
constexpr int kSpan = 512;        // columns that a warp takes at a time

struct UpdateParams {
  const void* g;
  float* momentum;         // or null: the update is g itself
  double* partial;         // [batch][parts]
  __half* x;               // [batch][planes][rows][ld_x]
  int64_t ld_g, batch_g, ld_m, ld_x, batch_x;
  int rows, cols, parts;
  int vec;                 // rows of g and momentum start on 4-element boundaries
  int planes;              // 2: what the rounding of the first plane left in a second
  int64_t plane_x;
  float mu;
  int nesterov;
  float eps, scale;
  __half* squares;         // or null: planes of `count` square matrices [batch][cleared][side][ld_s], see norm_kernel
  int64_t ld_s, plane_s, batch_s, next_s;   // next_s: from one square matrix to the next
  int side, count, cleared;
};

// u = g + mu momentum (nesterov) or momentum, from the momentum already updated.
__device__ __forceinline__ float update_of(const UpdateParams& p, float g, float m) {
  return p.nesterov ? fmaf(p.mu, m, g) : m;
}

// Both passes read g (and the momentum) once: a warp takes 512 columns of a row at
// a time, 16 values a lane in four 4-element loads that are in flight together.
template <int T>
__device__ __forceinline__ void load_span(const UpdateParams& p, const typename In<T>::type* g, const float* m, int c,
                                          float (&u)[16], float (&mv)[16]) {
  if (c + kSpan - 4 * (int)(threadIdx.x & 31) <= p.cols && p.vec) {
#pragma unroll
    for (int j = 0; j < 4; ++j) In<T>::get4(g + c + 128 * j, *reinterpret_cast<float(*)[4]>(&u[4 * j]));
    if (m != nullptr) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float4 q = __ldcg(reinterpret_cast<const float4*>(m + c + 128 * j));
        mv[4 * j] = q.x; mv[4 * j + 1] = q.y; mv[4 * j + 2] = q.z; mv[4 * j + 3] = q.w;
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const int at = c + 128 * (j / 4) + j % 4;
      u[j] = at < p.cols ? In<T>::get(g[at]) : 0.f;
      mv[j] = m != nullptr && at < p.cols ? __ldcg(m + at) : 0.f;
    }
  }
}

// First pass: updates the momentum (in place) and leaves each block's sum of squares of u.  It also clears the blocks of
// 256 on the diagonals of the square matrices' second (and third) planes, of which only the diagonals are ever written.
template <int T>
__global__ void __launch_bounds__(kUpdateThreads) norm_kernel(const UpdateParams p) {
  using X = typename In<T>::type;
  __shared__ double part[8];
  tc::launch_dependents();
  tc::wait_for_earlier();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int spans = (p.cols + kSpan - 1) / kSpan;
  const X* g = static_cast<const X*>(p.g) + blockIdx.y * p.batch_g;
  if (p.squares != nullptr) {
    // groups of eight: 32 of a row (fewer at the end: ld_s is a multiple of 8)
    for (int i = blockIdx.x * kUpdateThreads + threadIdx.x; i < p.count * p.cleared * p.side * 32; i += gridDim.x * kUpdateThreads) {
      const int row = i / 32, r = row % p.side, c = (r & ~255) + 8 * (i % 32), plane = row / p.side;
      __half* to = p.squares + plane / p.cleared * p.next_s + plane % p.cleared * p.plane_s + blockIdx.y * p.batch_s + (int64_t)r * p.ld_s + c;
      if (c < p.ld_s) *reinterpret_cast<uint4*>(to) = make_uint4(0, 0, 0, 0);
    }
  }
  double sum = 0.0;
  for (int i = blockIdx.x * 8 + warp; i < p.rows * spans; i += gridDim.x * 8) {
    const int r = i / spans, c = (i - r * spans) * kSpan + 4 * lane;
    float u[16], m[16];
    float* mp = p.momentum == nullptr ? nullptr : p.momentum + (int64_t)r * p.ld_m;
    load_span<T>(p, g + (int64_t)r * p.ld_g, mp, c, u, m);
    if (mp != nullptr) {
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        m[j] = fmaf(p.mu, m[j], u[j]);
        u[j] = update_of(p, u[j], m[j]);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int at = c + 128 * j;
        if (at + 4 <= p.cols && p.vec) {
          *reinterpret_cast<float4*>(mp + at) = make_float4(m[4 * j], m[4 * j + 1], m[4 * j + 2], m[4 * j + 3]);
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (at + k < p.cols) mp[at + k] = m[4 * j + k];
        }
      }
    }
    // in fp64: squares of fp32 values neither overflow nor vanish, and nothing is lost to a long sum
#pragma unroll
    for (int j = 0; j < 16; ++j) sum = fma((double)u[j], (double)u[j], sum);
  }
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
  if (lane == 0) part[warp] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < 8; ++w) sum += part[w];
    p.partial[(int64_t)blockIdx.y * p.parts + blockIdx.x] = sum;
  }
}

// Second pass: X_0 = u / (|u| + eps), scaled, as fp16.  From the last row to the first: what
// the first pass touched last is still in L2.
template <int T>
__global__ void __launch_bounds__(kUpdateThreads) start_kernel(const UpdateParams p) {
  using X = typename In<T>::type;
  __shared__ double part[8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  tc::launch_dependents();
  tc::wait_for_earlier();
  // every block adds up all parts in the same order
  double sum = 0.0;
  for (int i = threadIdx.x; i < p.parts; i += kUpdateThreads) sum += __ldcg(p.partial + (int64_t)blockIdx.y * p.parts + i);
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
  if (lane == 0) part[warp] = sum;
  __syncthreads();
  sum = 0.0;
  for (int w = 0; w < 8; ++w) sum += part[w];
  // the factor as a power of two and the rest, since it may lie outside fp32's range (a multiplication by a power of
  // two rounds nothing unless the result underflows)
  const double factor = (double)p.scale / (sqrt(sum) + (double)p.eps);
  const int e = factor > 0.0 && factor < 1e300 ? ilogb(factor) / 2 : 0;
  const float f2 = (float)ldexp(1.0, e), f = (float)ldexp(factor, -e);
  const int spans = (p.cols + kSpan - 1) / kSpan;
  const X* g = static_cast<const X*>(p.g) + blockIdx.y * p.batch_g;
  __half* x = p.x + blockIdx.y * p.batch_x;
  for (int i = blockIdx.x * 8 + warp; i < p.rows * spans; i += gridDim.x * 8) {
    const int at_row = i / spans, r = p.rows - 1 - at_row, c = (i - at_row * spans) * kSpan + 4 * lane;
    float u[16], m[16];
    const float* mp = p.momentum == nullptr ? nullptr : p.momentum + (int64_t)r * p.ld_m;
    load_span<T>(p, g + (int64_t)r * p.ld_g, mp, c, u, m);
    __half* o = x + (int64_t)r * p.ld_x;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int at = c + 128 * j;
      if (at >= p.cols) break;
      alignas(8) __half h[4], l[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float v = (mp == nullptr ? u[4 * j + k] : update_of(p, u[4 * j + k], m[4 * j + k])) * f2 * f;
        h[k] = __float2half_rn(v);
        l[k] = __float2half_rn(v - __half2float(h[k]));
      }
      if (p.planes > 1) *reinterpret_cast<uint2*>(o + p.plane_x + at) = *reinterpret_cast<const uint2*>(l);
      // rows of x have room for whole groups of 8
      *reinterpret_cast<uint2*>(o + at) = *reinterpret_cast<const uint2*>(h);
    }
  }
}

}  // namespace quant
}  // namespace bcjr
