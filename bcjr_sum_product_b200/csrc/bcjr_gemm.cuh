// Tensor-core matrix products of the layer-wise QAT operators (sm_100a).
//
//   D[r][c] = sum_k R[r][k] C[c][k]
//
// R is the side of the tensor-memory lanes, C the side of its columns.  Every
// result is stored row-major with r along the row, so that the 32 lanes of a
// warp write neighbouring values: the product y = a b^T takes R = b, C = a.
//
// Two kinds of operands:
//   F16  fp16 values (the Newton-Schulz iterates), each operand contiguous
//        along k (K-major) or along r or c (MN-major), so that no transposed
//        copy of an iterate is ever made;
//   MX   8-bit values contiguous along k with one power-of-two scale for each
//        row (or 128 rows) and 128 values of k.  The scales go into the
//        product itself (tcgen05 kind::mxf8f6f4 with block scales, which takes
//        them for every 32 values of k: the same byte four times), so the sum
//        over all of k stays in tensor memory in fp32 and nothing is rescaled
//        outside it.
//
// Two kernels:
//   tile_kernel  one block, one 128 x BN tile, with k split over a cluster
//                where there are few tiles: for small products;
//   pair_kernel  persistent pairs of blocks, 256 x BN tiles, sums of one tile
//                read out while the next is computed: for large ones.
// Both fill a ring of shared-memory stages by TMA (128 bytes of k each,
// 128-byte swizzle) from one thread and issue the products from another.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "bcjr_tc.cuh"

namespace bcjr {
namespace gemm {

// First error recorded by a kernel here (a status code of the C interface).
__device__ int g_dense_error = 0;
constexpr int kErrTimeout = 4;

enum Kind { F16 = 0, MX = 1 };
enum Epilogue {
  OUT = 0,    // out = alpha D
  GRAM = 1,   // P = D, symmetric, both halves stored (also a product of two polynomials of one P)
  POLY = 2,   // B = a I + b P + c D, symmetric, both halves stored
  ITER = 3,   // X' = D
  LAST = 4,   // out = D
  STEP = 5    // w = keep w - rate D
};
enum OutType { OUT_F32 = 0, OUT_F16 = 1, OUT_BF16 = 2 };

// Iterates and the square matrices are kept as fp16(2^12 x), one plane of 11 bits, and
// what its rounding left as a second one (22 bits in all).  With 2^12, |x| <= 16 stays
// finite, and values are rounded to 11 bits down to 2^-26 instead of 2^-14 (the entries
// of a large matrix of norm 1 are that small).
//
// Which second planes a product needs for a result of 8 bits:
//   X in B X: it.  A rounding E of X is added to X, puts a share of |E| into
//     directions where X has next to nothing, and every step multiplies those by up to
//     a = 3.4445 (485 times in five).  With one plane a result of rank 1 is off by 15 %,
//     of rank 8 by 4 %.  With 512 rows or more B's diagonal is enough of B for it: where X
//     has little, B is a I, and what the rest of B would make of the second plane lies
//     among directions that X has, is not amplified and gets less with more rows (rank 1 to
//     m / 4, m = 512: 1.5e-3 of the result instead of 1.1e-3; 256: 2.5e-3).
//   X in X X^T: none.  It would change P by less than P's own rounding.
//   P and B: the diagonal.  Roundings of B multiply X, so their errors stay in proportion
//     to each direction and average out over a row, as do those of P, which only enters B.
//     Not so a diagonal's: P and B may be nearly constant there (then their roundings all
//     go one way), and a I next to a product that nearly cancels it makes an error of half
//     a step of a (rank 1, 1536 x 6145, two steps at once: 1 %).  Of the second
//     planes' blocks of 256 on the diagonal, zeros but for it, a product takes those of
//     its tile's own rows: one to four blocks of k more.
// So held, a result is within 1.6e-3 of the exact iteration in the 2-norm whatever its
// singular values (half of that for updates of full rank).  For results of more than
// 8 bits, and for matrices of few rows, every product takes all second planes:
// R0 C0 + R0 C1 + R1 C0.
constexpr float kIterScale = 4096.f;

// Which part of an operand's or a result's second plane counts.  ACROSS: all of it, but multiplied by the other operand's
// diagonal alone (of its first plane), which that keeps as a third plane.
enum Second { NONE = 0, DIAGONAL = 1, ALL = 2, ACROSS = 3 };

struct Params {
  int rows, cols, k;         // extents of r, c, k
  int tiles_r;               // tiles along r
  int tiles;                 // tiles of one matrix
  int batch;
  int splits;                // blocks of one tile (the cluster of tile_kernel)
  int second_r, second_c;    // Second, of the operands
  int planes_r, planes_c;    // of one matrix of the batch, one after the other in the operands' maps' third dimension
  int band;                  // pair_kernel: tiles along r of a band
  // MX
  const uint8_t* sr;         // scales of R: sr[(r >> shift_r) * ld_sr + k / 128]
  const uint8_t* sc;
  int64_t ld_sr, ld_sc;
  int shift_r, shift_c;      // 0: one scale for each row, 7: for 128 rows
  int fmt_r, fmt_c;          // 0: e4m3, 1: e5m2
  // epilogue
  void* out;
  const __half* x;           // P (POLY), laid out as D
  int64_t ld_out, ld_x;
  int64_t batch_out, batch_x;
  int64_t plane_out, plane_x;   // from one plane to the other
  int second_out;               // Second, of the result and of x
  int third_out;                // the result's diagonal as a third plane too (second_out DIAGONAL)
  int out_type;
  float fa, fb, fc;          // OUT: alpha; POLY: a, b, c
  float keep, rate;          // STEP
  int nofill;                // tests: the last block of a cluster fetches one stage and no more, so that waits run out
};

constexpr int kRowsTile = 128;                      // rows of a block's tile
constexpr int kStageBytesR = kRowsTile * 128;

template <int T>
__device__ __forceinline__ void store_one(void* out, int64_t i, float v) {
  if (T == OUT_F32) static_cast<float*>(out)[i] = v;
  else if (T == OUT_F16) static_cast<__half*>(out)[i] = __float2half_rn(v);
  else static_cast<__nv_bfloat16*>(out)[i] = __float2bfloat16_rn(v);
}
template <int T, int W>
__device__ __forceinline__ void store_columns(void* out, int64_t at, int64_t ld, int n, const float (&v)[W]) {
#pragma unroll
  for (int i = 0; i < W; ++i) {
    if (i < n) store_one<T>(out, at, v[i]);
    at += ld;
  }
}

// Whether the diagonal passes through columns c0..c0+W-1 of the warp's rows.
template <int W>
__device__ __forceinline__ bool on_diagonal(int r, int c0) {
  return c0 < (r & ~31) + 32 && c0 + W > (r & ~31);
}

// What the end of W columns of a row reads, loaded ahead: W entries of row r of P
// (symmetric, so they lie side by side; ld_x is a multiple of 8), and what rounding took
// from all of them or from the diagonal's.
template <int W>
struct Ahead {
  uint4 h[W / 8], l[W / 8];
  __half diagonal;
};
template <int EPI, int W>
__device__ __forceinline__ void load_ahead(const Params& p, int64_t batch, int r, int c0, Ahead<W>& a) {
  if (EPI == POLY && r < p.rows) {
    const __half* x = p.x + batch * p.batch_x + (int64_t)r * p.ld_x;
#pragma unroll
    for (int i = 0; i < W / 8; ++i) {
      const bool in = c0 + 8 * i < p.cols;
      a.h[i] = in ? __ldcg(reinterpret_cast<const uint4*>(x + c0 + 8 * i)) : make_uint4(0, 0, 0, 0);
      a.l[i] = in && p.second_out == ALL ? __ldcg(reinterpret_cast<const uint4*>(x + p.plane_x + c0 + 8 * i)) : make_uint4(0, 0, 0, 0);
    }
    a.diagonal = p.second_out != ALL && on_diagonal<W>(r, c0) ? __ldcg(x + p.plane_x + r) : __float2half_rn(0.f);
  }
}

// Stores columns c0..c0+W-1 (as far as they exist) of row r.
template <int EPI, int W>
__device__ __forceinline__ void finish(const Params& p, int64_t batch, int r, int c0, bool mirror, const Ahead<W>& a,
                                       float (&v)[W]) {
  constexpr bool SQUARE = EPI == GRAM || EPI == POLY;
  if (!SQUARE && EPI != ITER && r >= p.rows) return;   // (the others' lanes exchange values below)
  const int n = p.cols - c0;
  const int64_t at = batch * p.batch_out + (int64_t)c0 * p.ld_out + r;
  const float unit = EPI == OUT ? p.fa : EPI == LAST ? 1.f / (kIterScale * kIterScale) : 1.f / kIterScale;
#pragma unroll
  for (int i = 0; i < W; ++i) v[i] *= unit;
  if constexpr (EPI == OUT || EPI == LAST) {
    if (p.out_type == OUT_F32) store_columns<OUT_F32, W>(p.out, at, p.ld_out, n, v);
    else if (p.out_type == OUT_F16) store_columns<OUT_F16, W>(p.out, at, p.ld_out, n, v);
    else store_columns<OUT_BF16, W>(p.out, at, p.ld_out, n, v);
  } else if constexpr (SQUARE || EPI == ITER) {
    const bool diagonal = SQUARE && on_diagonal<W>(r, c0);
    if constexpr (EPI == POLY) {
      const __half *x = reinterpret_cast<const __half*>(a.h), *l = reinterpret_cast<const __half*>(a.l);
#pragma unroll
      for (int i = 0; i < W; ++i) v[i] = fmaf(p.fb, __half2float(x[i]) + __half2float(l[i]), p.fc * v[i]);
      if (diagonal) {
        const float add = fmaf(p.fa, kIterScale, p.fb * __half2float(a.diagonal));
        // (as a sum of products with 0 and 1: a selection becomes an index into local memory)
#pragma unroll
        for (int i = 0; i < W; ++i) v[i] = fmaf(i == r - c0 ? 1.f : 0.f, add, v[i]);
      }
    }
    alignas(16) __half h[W];
#pragma unroll
    for (int i = 0; i < W; ++i) h[i] = __float2half_rn(v[i]);
    __half* out = static_cast<__half*>(p.out) + batch * p.batch_out;
    // the row's own values, side by side: 16-byte aligned; whole groups of 8 stay inside the row's room (ld_out is the
    // columns rounded up to 8)
    auto reflect = [&](const __half(&u)[W], __half* to) {
      if (SQUARE && mirror && r < p.rows) {
#pragma unroll
        for (int j = 0; j < W / 8; ++j)
          if (8 * j < n) reinterpret_cast<uint4*>(to + (int64_t)r * p.ld_out + c0)[j] = reinterpret_cast<const uint4*>(u)[j];
      }
    };
    reflect(h, out);
    if (p.second_out == ALL) {
      // Neighbouring lanes exchange halves: the even one stores both lanes' values, the odd one both lanes' second
      // planes, 4 bytes each, so two planes take as many stores as one (behind an odd number of rows there is room).
      alignas(16) __half l[W];
      const bool odd = r & 1;
      uint32_t* to = reinterpret_cast<uint32_t*>(out + (odd ? p.plane_out : 0) + (int64_t)c0 * p.ld_out + (r & ~1));
#pragma unroll
      for (int i = 0; i < W; ++i) {
        l[i] = __float2half_rn(v[i] - __half2float(h[i]));
        const uint32_t own = (uint32_t)__half_as_ushort(h[i]) | ((uint32_t)__half_as_ushort(l[i]) << 16);
        const uint32_t other = __shfl_xor_sync(0xFFFFFFFFu, own, 1);
        if (i < n && (r & ~1) < p.rows) *to = odd ? __byte_perm(other, own, 0x7632) : __byte_perm(own, other, 0x5410);
        to += p.ld_out / 2;
      }
      reflect(l, out + p.plane_out);
    } else if (r < p.rows) {
      __half* to = out + (int64_t)c0 * p.ld_out + r;
#pragma unroll
      for (int i = 0; i < W; ++i) {
        if (i < n) *to = h[i];
        to += p.ld_out;
      }
      if (diagonal && (unsigned)(r - c0) < (unsigned)min(W, n)) {
        float left = 0.f, first = 0.f;
#pragma unroll
        for (int i = 0; i < W; ++i) {
          left = i == r - c0 ? v[i] - __half2float(h[i]) : left;
          first = i == r - c0 ? __half2float(h[i]) : first;
        }
        __half* at = out + p.plane_out + (int64_t)r * p.ld_out + r;
        *at = __float2half_rn(left);
        if (p.third_out) at[p.plane_out] = __float2half_rn(first);
      }
    }
  } else {   // STEP
    float* w = static_cast<float*>(p.out) + at;
    float wv[W];
#pragma unroll
    for (int i = 0; i < W; ++i) wv[i] = i < n ? w[(int64_t)i * p.ld_out] : 0.f;
#pragma unroll
    for (int i = 0; i < W; ++i) v[i] = fmaf(-p.rate * (1.f / kIterScale), v[i], p.keep * wv[i]);
    store_columns<OUT_F32, W>(p.out, at, p.ld_out, n, v);
  }
}

// One 32-bit word of four scale bytes (k blocks 4 g .. 4 g + 3) of row `row`; rows and
// blocks that do not exist give 1 (their codes are read as zero).
__device__ __forceinline__ uint32_t scale_word(const uint8_t* s, int64_t ld, int shift, int row, int rows, int g, int blocks) {
  uint32_t w = 0x7F7F7F7Fu;
  if (row < rows) {
    const uint8_t* q = s + (int64_t)(row >> shift) * ld + 4 * g;
    const int n = blocks - 4 * g;                     // may be <= 0
    if (n >= 4 && (reinterpret_cast<uintptr_t>(q) & 3) == 0) {
      w = *reinterpret_cast<const uint32_t*>(q);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < n) w = (w & ~(0xFFu << (8 * i))) | ((uint32_t)q[i] << (8 * i));
    }
  }
  return w;
}

// The same for k blocks 16 g .. 16 g + 15, in one load where the row allows it.
__device__ __forceinline__ uint4 scale_words(const uint8_t* s, int64_t ld, int shift, int row, int rows, int g, int blocks) {
  if (row < rows && 16 * g + 16 <= blocks) {
    const uint8_t* q = s + (int64_t)(row >> shift) * ld + 16 * g;
    if ((reinterpret_cast<uintptr_t>(q) & 15) == 0) return *reinterpret_cast<const uint4*>(q);
  }
  uint4 w;
  w.x = scale_word(s, ld, shift, row, rows, 4 * g, blocks);
  w.y = scale_word(s, ld, shift, row, rows, 4 * g + 1, blocks);
  w.z = scale_word(s, ld, shift, row, rows, 4 * g + 2, blocks);
  w.w = scale_word(s, ld, shift, row, rows, 4 * g + 3, blocks);
  return w;
}

// The blocks of k of a tile at row r0 and column c0 (of the pair's whole tile): all of k; then again, for what counts of
// C's second plane; then of R's.  On the diagonal, that is where k is one of the tile's own columns or rows, across
// where it is on the other operand's.
template <int KIND, int TR, int TC>
struct Blocks {
  int all, first_c, in_c, first_r, in_r;
  __device__ __forceinline__ Blocks(const Params& p, int blocks, int r0, int c0) : all(blocks), first_c(0), in_c(0), first_r(0), in_r(0) {
    if (KIND == MX) return;
    if (p.second_c == DIAGONAL) {
      first_c = c0 / 64;
      in_c = min(TC / 64, blocks - first_c);
    } else if (p.second_c == ACROSS) {
      first_c = r0 / 64;
      in_c = min(TR / 64, blocks - first_c);
    } else if (p.second_c == ALL) {
      in_c = blocks;
    }
    if (p.second_r == DIAGONAL) {
      first_r = r0 / 64;
      in_r = min(TR / 64, blocks - first_r);
    } else if (p.second_r == ACROSS) {
      first_r = c0 / 64;
      in_r = min(TC / 64, blocks - first_r);
    } else if (p.second_r == ALL) {
      in_r = blocks;
    }
  }
  __device__ __forceinline__ int total() const { return all + in_c + in_r; }
  // The first value of k of block kb, the third coordinates of R and C in their maps.
  __device__ __forceinline__ void place(const Params& p, int kb, int batch, int* k, int* zr, int* zc) const {
    *zr = batch * p.planes_r;
    *zc = batch * p.planes_c;
    int b = kb;
    if (KIND == F16 && kb >= all) {
      b = kb - all;
      if (b < in_c) {
        b += first_c;
        *zc += 1;
        if (p.second_c == ACROSS) *zr += 2;
      } else {
        b += first_r - in_c;
        *zr += 1;
        if (p.second_r == ACROSS) *zc += 2;
      }
    }
    *k = b * (KIND == MX ? 128 : 64);
  }
};

// Tile t of a symmetric product of TR-row and TC-column tiles: row tile j has the
// (j + 1) TR / TC column tiles up to its diagonal block.
template <int TR, int TC>
__device__ __forceinline__ void symmetric_tile(int t, int* tr, int* tc, bool* mirror) {
  constexpr int q = TR / TC;
  static_assert(q * TC == TR, "column tiles divide the row tiles");
  int j = (int)((sqrtf(8.f * (float)(t / q) + 1.f) - 1.f) * 0.5f);
  while (q * (j + 1) * (j + 2) / 2 <= t) ++j;
  while (q * j * (j + 1) / 2 > t) --j;
  *tr = j;
  *tc = t - q * j * (j + 1) / 2;
  *mirror = *tc < j * q;
}

// The products of one stage: four instructions of 32 bytes of k.
template <int CG, int KIND, bool R_MN, bool C_MN>
__device__ __forceinline__ void stage_products(uint32_t acc, uint32_t a, uint32_t b, uint32_t idesc, uint32_t ts, bool add) {
  const uint64_t da0 = tc::desc_sw128(a, R_MN ? 8192 : 0), db0 = tc::desc_sw128(b, C_MN ? 8192 : 0);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // 32 bytes along K, or 16 rows of 128 bytes where K runs over the rows
    const uint64_t da = da0 + i * (R_MN ? 128 : 2), db = db0 + i * (C_MN ? 128 : 2);
    if (KIND == MX) tc::mma_mx<CG>(acc, da, db, idesc, ts, ts + 4, add || i > 0);
    else tc::mma_f16<CG>(acc, da, db, idesc, add || i > 0);
  }
}

// ------------------------------------------------------------ small products

constexpr int kTileThreads = 576;
// Blocks on an SM that the registers must leave room for.  Two (56 registers) for what runs in more blocks than there
// are SMs.  64-column tiles of symmetric products seldom do and are faster with 87 or 96 registers (512 x 2048: 118 us
// against 124; 16 of 333 x 130: 111 against 119; products with X in one block an SM: 120); 128 columns of a polynomial
// in 56 spill (256 of 128 x 256: 276 us against 259), so the compiler chooses (76).
__host__ __device__ constexpr int tile_blocks(int bn, int epi) {
  return bn < 128 && (epi == GRAM || epi == POLY) ? 1 : epi == POLY ? 0 : 2;
}

template <int KIND, int BN>
struct TileShape {
  static constexpr int kStageBytes = kStageBytesR + BN * 128;
  static constexpr int kStages = BN <= 64 ? 4 : 3;             // two blocks fit an SM
  static constexpr int kScaleStages = 2;                       // MX: rings of 512 values of k
  static constexpr int kScaleBytes = KIND == MX ? 1024 : 0;
  static constexpr int kScaleCols = KIND == MX ? 8 : 0;
  static constexpr int kUsedCols = BN + kScaleStages * kScaleCols;
  static constexpr int kTmemCols = kUsedCols <= 32 ? 32 : kUsedCols <= 64 ? 64 : kUsedCols <= 128 ? 128 : 256;
  static constexpr int kRing = kStages * kStageBytes;
  static constexpr int kSmem = 1024 + kRing + kScaleStages * kScaleBytes + 256;
  static_assert(kRowsTile * BN * 4 <= kRing, "the sums of a cluster's blocks fit the ring");
};

// One block computes one 128 x BN tile over its share of k.  Warp 0 fills the
// stages, one thread of warp 1 issues the products, warps 2 to 5 bring the
// scales (MX), and warps 2 to 17 read the sums and store them, eight columns at a
// time in a loop that is not unrolled: each block runs it once, and fetching
// straight-line code for 64 columns took longer than the stores (about 3 us).  Where there
// are too few tiles for the GPU's SMs, a cluster of blocks splits k: each sends its
// sums of a unit of columns to the block that finishes it, which adds them up in
// the order of the ranks, so the result does not depend on timing.  What bounds it
// is latency, not a pipe: of the 6 us of a product of 512 x 512 x 2048 the first
// copy takes 0.8, eight stages 1.7 (64 bytes a clock and SM from L2), the exchange
// 2.0, the stores 0.9.  One token through 8192 x 2048 (17 MB): 6.5 us, 2.6 TB/s of L2
// (calls in a row on the same operands); 11.6 us, 1.5 TB/s, from HBM.
template <int KIND, int BN, bool R_MN, bool C_MN, int EPI>
__global__ void __launch_bounds__(kTileThreads, tile_blocks(BN, EPI)) tile_kernel(const __grid_constant__ CUtensorMap map_r,
                                                             const __grid_constant__ CUtensorMap map_c, const Params p) {
  using S = TileShape<KIND, BN>;
  constexpr bool SYM = EPI == GRAM || EPI == POLY;
  constexpr int kElems = KIND == MX ? 128 : 64;     // values of k in a stage
  constexpr int kUnits = BN / 8;
  static_assert(BN <= 128, "");
  static_assert(KIND == F16 || (!R_MN && !C_MN), "8-bit operands are K-major");
  static_assert(!C_MN || BN >= 64, "an MN-major box is 64 wide");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t ring = tc::smem_addr(smem);
  const uint32_t scales = ring + S::kRing;
  const uint32_t ctl = scales + S::kScaleStages * S::kScaleBytes;
  const uint32_t full = ctl, empty = full + 8 * S::kStages, sfull = empty + 8 * S::kStages,
                 sempty = sfull + 8 * S::kScaleStages, done = sempty + 8 * S::kScaleStages, slot = done + 8;
  volatile uint32_t* slot_p = reinterpret_cast<volatile uint32_t*>(smem + (slot - ring));
  volatile int* fail = reinterpret_cast<volatile int*>(smem + (slot + 4 - ring));

  tc::launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tile = blockIdx.x / p.splits, rank = blockIdx.x % p.splits, batch = blockIdx.z;
  int tr, tcn;
  bool mirror = false;
  if constexpr (SYM) {
    symmetric_tile<kRowsTile, BN>(tile, &tr, &tcn, &mirror);
  } else {
    tr = tile % p.tiles_r;
    tcn = tile / p.tiles_r;
  }
  const int r0 = tr * kRowsTile, c0 = tcn * BN;
  const int blocks = (p.k + kElems - 1) / kElems;
  const Blocks<KIND, kRowsTile, BN> order(p, blocks, r0, c0);
  const int total = order.total();
  const int kb0 = (int)((int64_t)total * rank / p.splits), kb1 = (int)((int64_t)total * (rank + 1) / p.splits);

  if (threadIdx.x == 0) {
    tc::prefetch_map(&map_r);
    tc::prefetch_map(&map_c);
    for (int i = 0; i < S::kStages; ++i) {
      tc::mbar_init(full + 8 * i, 1);
      tc::mbar_init(empty + 8 * i, 1);
    }
    for (int i = 0; i < S::kScaleStages; ++i) {
      tc::mbar_init(sfull + 8 * i, 128);
      tc::mbar_init(sempty + 8 * i, 1);
    }
    tc::mbar_init(done, 1);
    *fail = 0;
    tc::mbar_init_fence();
  }
  if (warp == 1) tc::tmem_alloc<1, S::kTmemCols>(slot);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  tc::wait_for_earlier();
  const uint32_t acc = *slot_p;
  const uint32_t tscale = acc + BN;
  auto gave_up = [&]() {
    *fail = 1;
    atomicCAS(&g_dense_error, 0, kErrTimeout);
  };
  // the columns whose sums this warp finishes: units of eight, one in 4 * splits
  const int row = r0 + 32 * (warp & 3) + lane;
  const int unit0 = rank + p.splits * ((warp - 2) >> 2), step = 4 * p.splits;
  Ahead<8> ahead;

  if (warp == 0) {
    if (lane == 0) {
      int issued = 0;
      for (int kb = kb0; kb < kb1; ++kb) {
        const int s = issued % S::kStages;
        if (p.nofill && rank + 1 == p.splits && issued > 0) break;
        if (!tc::mbar_wait(empty + 8 * s, ((issued / S::kStages) & 1) ^ 1)) {
          gave_up();
          break;
        }
        const uint32_t dst = ring + s * S::kStageBytes, bar = full + 8 * s;
        tc::mbar_expect(bar, S::kStageBytes);
        int k, zr, zc;
        order.place(p, kb, batch, &k, &zr, &zc);
        if (R_MN) {
          tc::tma_load3(dst, &map_r, r0, k, zr, bar);
          tc::tma_load3(dst + 8192, &map_r, r0 + 64, k, zr, bar);
        } else {
          tc::tma_load3(dst, &map_r, k, r0, zr, bar);
        }
        if (C_MN) {
#pragma unroll
          for (int i = 0; i < BN / 64; ++i)
            tc::tma_load3(dst + kStageBytesR + 8192 * i, &map_c, c0 + 64 * i, k, zc, bar);
        } else {
          tc::tma_load3(dst + kStageBytesR, &map_c, k, c0, zc, bar);
        }
        ++issued;
      }
      // no copy is in flight when the block leaves (the products waited for them unless something gave up)
      for (int i = issued > S::kStages ? issued - S::kStages : 0; i < issued; ++i)
        tc::mbar_wait(full + 8 * (i % S::kStages), (i / S::kStages) & 1);
    }
  } else if (warp == 1) {
    const uint32_t idesc = KIND == MX ? tc::idesc_mx(128, BN, p.fmt_r, p.fmt_c) : tc::idesc_f16(128, BN, R_MN, C_MN);
    int it = 0, group = -1, groups = 0;
    uint32_t ts = 0;
    bool ok = true;
    for (int kb = kb0; kb < kb1; ++kb, ++it) {
      const int s = it % S::kStages;
      ok = __all_sync(0xFFFFFFFFu, tc::mbar_wait(full + 8 * s, (it / S::kStages) & 1));
      if (!ok) break;
      if (KIND == MX && group != kb / 4) {
        group = kb / 4;
        const int ss = groups % S::kScaleStages;
        ok = __all_sync(0xFFFFFFFFu, tc::mbar_wait(sfull + 8 * ss, (groups / S::kScaleStages) & 1));
        if (!ok) break;
        ++groups;
        tc::fence_after();
        ts = tscale + ss * S::kScaleCols;
        if (tc::elect_one()) {
          tc::copy_scales<1>(ts, tc::desc_scales(scales + ss * S::kScaleBytes));
          tc::copy_scales<1>(ts + 4, tc::desc_scales(scales + ss * S::kScaleBytes + 512));
        }
        __syncwarp();
      }
      tc::fence_after();
      if (tc::elect_one()) {
        const uint32_t a = ring + s * S::kStageBytes;
        stage_products<1, KIND, R_MN, C_MN>(acc, a, a + kStageBytesR, KIND == MX ? tc::idesc_mx_id(idesc, kb & 3) : idesc,
                                            ts, it > 0);
        tc::commit<1>(empty + 8 * s);
        if (KIND == MX && ((kb & 3) == 3 || kb + 1 == kb1)) tc::commit<1>(sempty + 8 * ((groups - 1) % S::kScaleStages));
      }
      __syncwarp();
    }
    if (!ok) gave_up();
    if (tc::elect_one()) tc::commit<1>(done);
    __syncwarp();
  } else {
    const int t = threadIdx.x - 64;   // 0..511
    bool ok = true;
    if (KIND == MX && t < 128) {
      const int g1 = kb1 > kb0 ? (kb1 - 1) / 4 + 1 : kb0 / 4;
      int n = 0;
      for (int g = kb0 / 4; g < g1; ++g, ++n) {
        const int ss = n % S::kScaleStages;
        const uint32_t wr = scale_word(p.sr, p.ld_sr, p.shift_r, r0 + t, p.rows, g, blocks);
        const uint32_t wc = scale_word(p.sc, p.ld_sc, p.shift_c, t < BN ? c0 + t : p.cols, p.cols, g, blocks);
        ok = tc::mbar_wait(sempty + 8 * ss, ((n / S::kScaleStages) & 1) ^ 1);
        if (!ok) break;
        uint8_t* dst = smem + (scales - ring) + ss * S::kScaleBytes + (t & 31) * 16 + (t >> 5) * 4;
        *reinterpret_cast<uint32_t*>(dst) = wr;
        *reinterpret_cast<uint32_t*>(dst + 512) = wc;
        tc::fence_async_shared();
        tc::mbar_arrive(sfull + 8 * ss);
      }
    }
    if (unit0 < kUnits) load_ahead<EPI, 8>(p, batch, row, c0 + 8 * unit0, ahead);
    ok = ok && tc::mbar_wait(done, 0);
    if (!ok) gave_up();
  }
  __syncwarp();
  __syncthreads();
  tc::fence_after();

  // The sums: lane r of the warp's quarter, eight columns at a time.
  const bool some = kb1 > kb0;
  const uint32_t sums = acc + ((uint32_t)(32 * (warp & 3)) << 16);
  const int rl = 32 * (warp & 3) + lane;
  // Unit u is finished by rank u % splits; its sums from rank s lie over the stages of that block (no
  // copy is in flight there after the first cluster barrier) as [u / splits][s][two halves][128 rows] float4.
  if (p.splits > 1) {
    tc::cluster_sync();
    // the sums of a block that gave up are incomplete: none of the cluster's may be stored
    if (threadIdx.x < p.splits && *fail != 0) tc::st_cluster(tc::map_rank(slot + 4, threadIdx.x), 1);
    if (warp >= 2) {
#pragma unroll 2
      for (int u = (warp - 2) >> 2; u < kUnits; u += 4) {
        uint32_t w[8];
        if (some) {
          tc::tmem_ld8(sums + 8 * u, w);
          tc::tmem_wait_ld8(w);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) w[i] = 0;
        }
        const uint32_t to = tc::map_rank(ring + (((u / p.splits) * p.splits + rank) * 256 + rl) * 16, u % p.splits);
        tc::st_cluster4(to, w[0], w[1], w[2], w[3]);
        tc::st_cluster4(to + 128 * 16, w[4], w[5], w[6], w[7]);
      }
    }
    tc::cluster_sync();
  }
  if (warp >= 2 && *fail == 0) {
#pragma unroll 1
    for (int u = unit0; u < kUnits; u += step) {
      const int c = c0 + 8 * u;
      if (c >= p.cols) break;
      float v[8];
      if (p.splits == 1) {
        uint32_t w[8];
        if (some) {
          tc::tmem_ld8(sums + 8 * u, w);
          tc::tmem_wait_ld8(w);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = some ? __uint_as_float(w[i]) : 0.f;
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = 0.f;
        const float4* from = reinterpret_cast<const float4*>(smem) + (u / p.splits) * p.splits * 256 + rl;
#pragma unroll 4
        for (int s = 0; s < p.splits; ++s) {
          const float4 f = from[256 * s], g = from[256 * s + 128];
          v[0] += f.x; v[1] += f.y; v[2] += f.z; v[3] += f.w;
          v[4] += g.x; v[5] += g.y; v[6] += g.z; v[7] += g.w;
        }
      }
      const Ahead<8> now = ahead;
      if (u + step < kUnits) load_ahead<EPI, 8>(p, batch, row, c + 8 * step, ahead);
      finish<EPI, 8>(p, batch, row, c, mirror, now, v);
    }
  }
  tc::fence_before();
  __syncthreads();
  if (warp == 1) {
    tc::fence_after();
    tc::tmem_dealloc<1, S::kTmemCols>(acc);
  }
}

// ------------------------------------------------------------ large products

constexpr int kPairThreads = 384;

template <int KIND, int BN>
struct PairShape {
  static constexpr int kSub = 2;                                // 128-byte blocks of k in a stage
  static constexpr int kSubBytes = kStageBytesR + BN / 2 * 128;  // a block of the pair brings half of the columns
  static constexpr int kStageBytes = kSub * kSubBytes;
  static constexpr int kStages = (200 * 1024) / kStageBytes;
  static constexpr int kScaleStages = 2;
  static constexpr int kScaleBytes = KIND == MX ? 512 + 512 * ((BN + 127) / 128) : 0;
  static constexpr int kScaleCols = KIND == MX ? 4 + 4 * ((BN + 127) / 128) : 0;
  static constexpr int kSets = 2 * BN + kScaleStages * kScaleCols <= 512 ? 2 : 1;   // sets of sums
  static constexpr int kTmemCols = 512;
  static constexpr int kSmem = 1024 + kStages * kStageBytes + kScaleStages * kScaleBytes + 512;
  static_assert(kStages >= 3, "the scales' waits need three stages");
  static_assert(BN % 32 == 0 && kSubBytes % 1024 == 0, "");
};

// Pairs of blocks (clusters of two, one block on each SM) take 256 x BN tiles in
// turn.  Of each stage a block brings the 128 rows of R that its own tensor
// memory sums up and half of the columns of C; one thread of the first block
// issues the products for both (cta_group::2), so each byte of C is read from
// shared memory by both SMs but copied there once: per SM 16 KB + 64 BN bytes
// for 256 x BN x 128 bytes' worth of products, against 16 KB + 128 BN of a
// block on its own, which would ask for more than the L2 delivers.  The sums
// alternate between two halves of tensor memory, and warps 4 to 11 store one
// tile while the next is computed.  Warps 2 and 3 bring the scales.  A stage holds
// two blocks of k, since every commit (the hand-back of a stage) makes the tensor
// cores pause: about 0.13 us each, measured.  8-bit 8192 x 8192 x 2048: 120 us in a
// row, 2.29 PFLOP/s (145 us with inputs and outputs that L2 does not hold).  No unit is
// at its limit: the tensor pipe is active 61 % of the time, L2 delivers 9.8 TB/s (43 % of
// its throughput, a third of the SMs' way to it).  The rest is waiting: eight commits a
// tile and sixteen tiles (17 us), the stores on the operands' way (without them 106 us),
// the first stages of each tile, and a clock of 1.6 GHz under the power limit.
// fp16 256 x 256 tiles: 0.29 us for 64 values of k, the tensor cores' own rate 0.27.
template <int KIND, int BN, bool R_MN, bool C_MN, int EPI>
__global__ void __launch_bounds__(kPairThreads, 1) pair_kernel(const __grid_constant__ CUtensorMap map_r,
                                                                const __grid_constant__ CUtensorMap map_c, const Params p) {
  using S = PairShape<KIND, BN>;
  constexpr bool SYM = EPI == GRAM || EPI == POLY;
  constexpr int kElems = KIND == MX ? 128 : 64;
  constexpr int kHalf = BN / 2;
  static_assert(KIND == F16 || (!R_MN && !C_MN), "8-bit operands are K-major");
  static_assert(!C_MN || kHalf % 64 == 0, "an MN-major box is 64 wide");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t ring = tc::smem_addr(smem);
  const uint32_t scales = ring + S::kStages * S::kStageBytes;
  const uint32_t ctl = scales + S::kScaleStages * S::kScaleBytes;
  const uint32_t full = ctl, empty = full + 8 * S::kStages, sfull = empty + 8 * S::kStages,
                 accfull = sfull + 8 * S::kScaleStages, accempty = accfull + 16, ended = accempty + 16, slot = ended + 8;
  volatile uint32_t* slot_p = reinterpret_cast<volatile uint32_t*>(smem + (slot - ring));
  volatile int* fail = reinterpret_cast<volatile int*>(smem + (slot + 4 - ring));

  tc::launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = tc::cluster_rank();
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const int all = p.tiles * p.batch;
  const int blocks = (p.k + kElems - 1) / kElems;   // > 0
  using Order = Blocks<KIND, 2 * kRowsTile, BN>;

  if (threadIdx.x == 0) {
    tc::prefetch_map(&map_r);
    tc::prefetch_map(&map_c);
    for (int i = 0; i < S::kStages; ++i) {
      tc::mbar_init(full + 8 * i, 1);
      tc::mbar_init(empty + 8 * i, 1);
    }
    for (int i = 0; i < S::kScaleStages; ++i) tc::mbar_init(sfull + 8 * i, 4);   // two warps of each block
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(accfull + 8 * i, 1);
      tc::mbar_init(accempty + 8 * i, 16);  // eight warps of each block
    }
    tc::mbar_init(ended, 1);
    *fail = 0;
    tc::mbar_init_fence();
  }
  if (warp == 1) tc::tmem_alloc<2, S::kTmemCols>(slot);
  tc::fence_before();
  __syncthreads();
  tc::cluster_sync();
  tc::fence_after();
  tc::wait_for_earlier();
  const uint32_t acc = *slot_p;
  const uint32_t tscale = acc + S::kSets * BN;
  auto gave_up = [&]() {
    *fail = 1;
    atomicCAS(&g_dense_error, 0, kErrTimeout);
  };
  auto place = [&](int tile, int* r0, int* c0, int* batch, bool* mirror) {
    const int b = tile / p.tiles, t = tile - b * p.tiles;
    int tr, tcn;
    *mirror = false;
    if constexpr (SYM) {
      symmetric_tile<2 * kRowsTile, BN>(t, &tr, &tcn, mirror);
    } else {
      // bands of `band` tiles along r, column by column: the pairs that run together share rows and columns
      const int tiles_c = p.tiles / p.tiles_r, band = t / (p.band * tiles_c), in = t - band * p.band * tiles_c;
      const int high = min(p.band, p.tiles_r - band * p.band);
      tcn = in / high;
      tr = band * p.band + in - tcn * high;
    }
    *r0 = tr * 2 * kRowsTile + (int)rank * kRowsTile;
    *c0 = tcn * BN;
    *batch = b;
  };

  if (warp == 0) {
    if (lane == 0) {
      int it = 0;
      bool ok = true;
      for (int tile = pair; tile < all && ok; tile += pairs) {
        int r0, c0, batch;
        bool mirror;
        place(tile, &r0, &c0, &batch, &mirror);
        const int ch = c0 + (int)rank * kHalf;
        const Order order(p, blocks, r0 - (int)rank * kRowsTile, c0);
        const int total = order.total();
        for (int kb = 0; kb < total; kb += S::kSub, ++it) {
          const int s = it % S::kStages, n = min(S::kSub, total - kb);
          if (p.nofill && rank == 1 && it > 0) break;
          ok = tc::mbar_wait(empty + 8 * s, ((it / S::kStages) & 1) ^ 1);
          if (!ok) break;
          const uint32_t bar = tc::map_rank(full + 8 * s, 0);
          if (rank == 0) tc::mbar_expect(full + 8 * s, 2 * n * S::kSubBytes);   // both blocks' bytes
          for (int j = 0; j < n; ++j) {
            const uint32_t dst = ring + s * S::kStageBytes + j * S::kSubBytes;
            int k, zr, zc;
            order.place(p, kb + j, batch, &k, &zr, &zc);
            if (R_MN) {
              tc::tma_load3_pair(dst, &map_r, r0, k, zr, bar);
              tc::tma_load3_pair(dst + 8192, &map_r, r0 + 64, k, zr, bar);
            } else {
              tc::tma_load3_pair(dst, &map_r, k, r0, zr, bar);
            }
            if (C_MN) {
#pragma unroll
              for (int i = 0; i < kHalf / 64; ++i)
                tc::tma_load3_pair(dst + kStageBytesR + 8192 * i, &map_c, ch + 64 * i, k, zc, bar);
            } else {
              tc::tma_load3_pair(dst + kStageBytesR, &map_c, k, ch, zc, bar);
            }
          }
        }
      }
      if (!ok) gave_up();
      // no copy is in flight when the blocks leave: both blocks' complete on the first one's barriers,
      // and the second does not leave before the first
      if (rank == 0)
        for (int i = it > S::kStages ? it - S::kStages : 0; i < it; ++i)
          tc::mbar_wait(full + 8 * (i % S::kStages), (i / S::kStages) & 1);
    }
  } else if (warp == 1) {
    if (rank == 0) {
      const uint32_t idesc = KIND == MX ? tc::idesc_mx(256, BN, p.fmt_r, p.fmt_c) : tc::idesc_f16(256, BN, R_MN, C_MN);
      int it = 0, groups = 0, n = 0;
      uint32_t ts = 0;
      bool ok = true;
      for (int tile = pair; tile < all && ok; tile += pairs, ++n) {
        const int set = n % S::kSets;
        ok = __all_sync(0xFFFFFFFFu, tc::mbar_wait_cluster(accempty + 8 * set, ((n / S::kSets) & 1) ^ 1));
        if (!ok) break;
        tc::fence_after();
        const uint32_t d = acc + set * BN;
        int r0, c0, batch;
        bool mirror;
        place(tile, &r0, &c0, &batch, &mirror);
        const int total = Order(p, blocks, r0, c0).total();
        for (int kb = 0; kb < total; kb += S::kSub, ++it) {
          const int s = it % S::kStages;
          ok = __all_sync(0xFFFFFFFFu, tc::mbar_wait(full + 8 * s, (it / S::kStages) & 1));
          if (!ok) break;
          if (KIND == MX && (kb & 3) == 0) {
            const int ss = groups % S::kScaleStages;
            ok = __all_sync(0xFFFFFFFFu, tc::mbar_wait_cluster(sfull + 8 * ss, (groups / S::kScaleStages) & 1));
            if (!ok) break;
            ++groups;
            ts = tscale + ss * S::kScaleCols;
            const uint32_t src = scales + ss * S::kScaleBytes;
            tc::fence_after();
            if (tc::elect_one()) {
              tc::copy_scales<2>(ts, tc::desc_scales(src));
#pragma unroll
              for (int i = 0; i < (BN + 127) / 128; ++i)
                tc::copy_scales<2>(ts + 4 + 4 * i, tc::desc_scales(src + 512 + 512 * i));
            }
            __syncwarp();
          } else {
            tc::fence_after();
          }
          if (tc::elect_one()) {
#pragma unroll
            for (int j = 0; j < S::kSub; ++j) {
              if (kb + j < total) {
                const uint32_t a = ring + s * S::kStageBytes + j * S::kSubBytes;
                stage_products<2, KIND, R_MN, C_MN>(d, a, a + kStageBytesR,
                                                    KIND == MX ? tc::idesc_mx_id(idesc, (kb + j) & 3) : idesc, ts, kb + j > 0);
              }
            }
            tc::commit<2>(empty + 8 * s);
          }
          __syncwarp();
        }
        if (ok && tc::elect_one()) tc::commit<2>(accfull + 8 * set);
        __syncwarp();
      }
      if (!ok) {
        gave_up();
        // what was issued ends before the blocks leave; the tile's sums are incomplete, so both blocks' readers wait in vain
        if (tc::elect_one()) tc::commit_pair_here(ended);
        tc::mbar_wait(ended, 0);
      }
    }
  } else if (warp < 4) {
    if (KIND == MX) {
      const int t = threadIdx.x - 64;   // 0..63
      const uint32_t peer_full = tc::map_rank(sfull, 0);
      constexpr int kWords = 2 + 2 * ((BN + 127) / 128);
      int n = 0, stage = 0;              // groups and stages so far
      int last1 = -1, last2 = -1;        // last stages of the last two groups
      bool ok = true;
      for (int tile = pair; tile < all && ok; tile += pairs) {
        int r0, c0, batch;
        bool mirror;
        place(tile, &r0, &c0, &batch, &mirror);
        uint4 w[kWords];
        for (int g = 0; 4 * g < blocks; ++g, ++n) {
          const int ss = n % S::kScaleStages;
          if ((g & 3) == 0) {
            // 16 bytes of a row at once: single words of 350 rows kept the load path of the SM busy enough to slow
            // the copies (8-bit 8192 x 8192 x 2048: 124 us; 114 with no loads of scales at all)
#pragma unroll
            for (int i = 0; i < 2; ++i)
              w[i] = scale_words(p.sr, p.ld_sr, p.shift_r, r0 + t + 64 * i, p.rows, g / 4, blocks);
#pragma unroll
            for (int i = 2; i < kWords; ++i) {
              const int c = t + 64 * (i - 2);
              w[i] = scale_words(p.sc, p.ld_sc, p.shift_c, c < BN ? c0 + c : p.cols, p.cols, g / 4, blocks);
            }
          } else {
#pragma unroll
            for (int i = 0; i < kWords; ++i) w[i] = make_uint4(w[i].y, w[i].z, w[i].w, 0);
          }
          // The slot is free once the stages of the group before last have been used up, which their own
          // barriers tell (a commit for the slot alone would cost the tensor cores another pause).  Stage
          // last2 + kStages belongs to this group or a later one, so that barrier is at most one phase ahead.
          ok = last2 < 0 || tc::mbar_wait(empty + 8 * (last2 % S::kStages), (last2 / S::kStages) & 1);
          ok = __all_sync(0xFFFFFFFFu, ok);
          if (!ok) break;
          last2 = last1;
          stage += min(2, (blocks - 4 * g + S::kSub - 1) / S::kSub);
          last1 = stage - 1;
          uint8_t* dst = smem + (scales - ring) + ss * S::kScaleBytes;
#pragma unroll
          for (int i = 0; i < kWords; ++i) {
            const int x = t + 64 * (i & 1);
            *reinterpret_cast<uint32_t*>(dst + 512 * (i >> 1) + (x & 31) * 16 + (x >> 5) * 4) = w[i].x;
          }
          tc::fence_async_shared();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive_cluster(peer_full + 8 * ss);
        }
      }
      if (!ok) gave_up();
    }
  } else {
    // eight warps: two for each quarter of the lanes, in turn on groups of 16 columns; the next
    // group's sums (and what else its end reads) are loaded while this one is stored
    const uint32_t sums = acc + ((uint32_t)(32 * (warp & 3)) << 16);
    const int first = (warp - 4) >> 2;
    int n = 0;
    bool ok = true;
    for (int tile = pair; tile < all && ok; tile += pairs, ++n) {
      int r0, c0, batch;
      bool mirror;
      place(tile, &r0, &c0, &batch, &mirror);
      const int set = n % S::kSets, row = r0 + 32 * (warp & 3) + lane;
      Ahead<16> ahead;
      uint32_t u[16];
      load_ahead<EPI, 16>(p, batch, row, c0 + 16 * first, ahead);
      ok = tc::mbar_wait(accfull + 8 * set, (n / S::kSets) & 1);
      ok = __all_sync(0xFFFFFFFFu, ok && *fail == 0);
      if (!ok) break;
      tc::fence_after();
      tc::tmem_ld16(sums + set * BN + 16 * first, u);
#pragma unroll 1
      for (int c = 16 * first; c < BN; c += 32) {
        if (c0 + c >= p.cols) break;
        tc::tmem_wait_ld(u);
        float v[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) v[k] = __uint_as_float(u[k]);
        const Ahead<16> now = ahead;
        if (c + 32 < BN) {
          tc::tmem_ld16(sums + set * BN + c + 32, u);
          load_ahead<EPI, 16>(p, batch, row, c0 + c + 32, ahead);
        }
        finish<EPI, 16>(p, batch, row, c0 + c, mirror, now, v);
      }
      tc::tmem_drain_ld();
      tc::fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive_cluster(tc::map_rank(accempty + 8 * set, 0));
    }
    if (!ok) gave_up();
  }
  __syncwarp();
  __syncthreads();
  tc::fence_before();
  tc::cluster_sync();
  if (warp == 1) {
    tc::fence_after();
    tc::tmem_dealloc<2, S::kTmemCols>(acc);
  }
}

}  // namespace gemm
}  // namespace bcjr
