// Tensor-core matrix products of the layer-wise QAT operators (sm_100a).
//
//   D[r][c] = sum_k R[r][k] C[c][k]
//
// R is the side of 128 tensor-memory lanes, C the side of its columns.  Every
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
// One block computes one 128 x BN tile over its share of k.  Warp 0 fills a
// ring of shared-memory stages by TMA (128 bytes of k each, 128-byte swizzle),
// one thread of warp 1 issues the products, warps 2 to 5 bring the scales (MX)
// and then read the sums.  Where there are too few tiles for the GPU's 148
// SMs, a cluster of blocks splits k: each leaves its sums in shared memory and
// adds up its share of the columns over the cluster, in the order of the
// ranks, so the result does not depend on timing.
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
  GRAM = 1,   // P = D, symmetric, both halves stored
  POLY = 2,   // B = b P + c D, symmetric, both halves stored
  ITER = 3,   // X' = a X + D
  LAST = 4,   // out = a X + D
  STEP = 5    // w = keep w - rate (a X + D)
};
enum OutType { OUT_F32 = 0, OUT_F16 = 1, OUT_BF16 = 2 };

// The iterates are kept as fp16(2^12 x): |x| <= 16 stays finite, and values are
// rounded to 11 bits down to 2^-26 instead of 2^-14 (the entries of a large
// matrix of norm 1 are that small).
constexpr float kIterScale = 4096.f;

struct Params {
  int rows, cols, k;         // extents of r, c, k
  int tiles_r;               // tiles along r
  int splits;                // blocks of one tile (the cluster)
  // MX
  const uint8_t* sr;         // scales of R: sr[(r >> shift_r) * ld_sr + k / 128]
  const uint8_t* sc;
  int64_t ld_sr, ld_sc;
  int shift_r, shift_c;      // 0: one scale for each row, 7: for 128 rows
  int fmt_r, fmt_c;          // 0: e4m3, 1: e5m2
  // epilogue
  void* out;
  const __half* x;           // P (POLY) or X (ITER, LAST, STEP), laid out as D
  int64_t ld_out, ld_x;
  int64_t batch_out, batch_x;
  int out_type;
  float fa, fb;              // OUT: alpha; POLY: c and b; ITER, LAST, STEP: 1 and a
  float keep, rate;          // STEP
};

constexpr int kThreads = 192;
constexpr int kRowsTile = 128;
constexpr int kStageBytesR = kRowsTile * 128;

template <int KIND, int BN>
struct Shape {
  static constexpr int kStageBytes = kStageBytesR + BN * 128;
  // as many stages as fit beside one another: two blocks on an SM up to 128 columns
  static constexpr int kStages = BN <= 128 ? (BN <= 64 ? 4 : 3) : 4;
  static constexpr int kScaleStages = 2;                       // MX: rings of 512 values of k
  static constexpr int kScaleBytes = KIND == MX ? 512 + 512 * ((BN + 127) / 128) : 0;
  static constexpr int kScaleCols = KIND == MX ? 4 + 4 * ((BN + 127) / 128) : 0;
  static constexpr int kUsedCols = BN + kScaleStages * kScaleCols;
  static constexpr int kTmemCols = kUsedCols <= 32 ? 32 : kUsedCols <= 64 ? 64 : kUsedCols <= 128 ? 128 : kUsedCols <= 256 ? 256 : 512;
  static constexpr int kDumpBytes = kRowsTile * BN * 4;        // sums left for the cluster, over the stages
  static constexpr int kRing = kStages * kStageBytes > kDumpBytes ? kStages * kStageBytes : kDumpBytes;
  static constexpr int kSmem = 1024 + kRing + kScaleStages * kScaleBytes + 256;
};

template <int T>
__device__ __forceinline__ void store_one(void* out, int64_t i, float v) {
  if (T == OUT_F32) static_cast<float*>(out)[i] = v;
  else if (T == OUT_F16) static_cast<__half*>(out)[i] = __float2half_rn(v);
  else static_cast<__nv_bfloat16*>(out)[i] = __float2bfloat16_rn(v);
}

// Stores 16 columns c0..c0+15 of row r (of which `n` exist).
template <int EPI>
__device__ __forceinline__ void finish16(const Params& p, int64_t batch, int r, int c0, int n, bool mirror,
                                         const float (&v)[16]) {
  if (r >= p.rows) return;
  if (EPI == OUT) {
    const int64_t at = (int64_t)c0 * p.ld_out + r;
#define BCJR_STORE(T)                                                                      \
  _Pragma("unroll") for (int i = 0; i < 16; ++i) if (i < n)                                \
      store_one<T>(p.out, at + (int64_t)i * p.ld_out, p.fa * v[i]);
    if (p.out_type == OUT_F32) { BCJR_STORE(OUT_F32) }
    else if (p.out_type == OUT_F16) { BCJR_STORE(OUT_F16) }
    else { BCJR_STORE(OUT_BF16) }
#undef BCJR_STORE
    return;
  }
  float y[16];
  if (EPI == GRAM) {
#pragma unroll
    for (int i = 0; i < 16; ++i) y[i] = v[i] * (1.f / kIterScale);
  } else {
    const __half* x = p.x + batch * p.batch_x + (int64_t)c0 * p.ld_x + r;
    float xv[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) xv[i] = i < n ? __half2float(x[(int64_t)i * p.ld_x]) : 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) y[i] = fmaf(p.fb, xv[i], p.fa * (1.f / kIterScale) * v[i]);
  }
  if (EPI == GRAM || EPI == POLY || EPI == ITER) {
    __half h[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) h[i] = __float2half_rn(y[i]);
    __half* o = static_cast<__half*>(p.out) + batch * p.batch_out;
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (i < n) o[(int64_t)(c0 + i) * p.ld_out + r] = h[i];
    if (EPI != ITER && mirror) {
      __half* m = o + (int64_t)r * p.ld_out + c0;   // ld_out and c0 are multiples of 8
      if (n == 16) {
        reinterpret_cast<uint4*>(m)[0] = reinterpret_cast<const uint4*>(h)[0];
        reinterpret_cast<uint4*>(m)[1] = reinterpret_cast<const uint4*>(h)[1];
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (i < n) m[i] = h[i];
      }
    }
  } else if (EPI == LAST) {
    const int64_t at = batch * p.batch_out + (int64_t)c0 * p.ld_out + r;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      if (i < n) {
        if (p.out_type == OUT_F16) store_one<OUT_F16>(p.out, at + (int64_t)i * p.ld_out, y[i] * (1.f / kIterScale));
        else store_one<OUT_BF16>(p.out, at + (int64_t)i * p.ld_out, y[i] * (1.f / kIterScale));
      }
    }
  } else {   // STEP
    float* w = static_cast<float*>(p.out) + (int64_t)c0 * p.ld_out + r;
    float wv[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) wv[i] = i < n ? w[(int64_t)i * p.ld_out] : 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (i < n) w[(int64_t)i * p.ld_out] = fmaf(-p.rate * (1.f / kIterScale), y[i], p.keep * wv[i]);
  }
}

// One 32-bit word of four scale bytes (k blocks 4 g .. 4 g + 3) of row `row`; rows and
// blocks that do not exist give 1 (their codes are read as zero).
__device__ __forceinline__ uint32_t scale_word(const uint8_t* s, int64_t ld, int shift, int row, int rows, int g, int blocks) {
  uint32_t w = 0x7F7F7F7Fu;
  if (row < rows) {
    const uint8_t* q = s + (int64_t)(row >> shift) * ld + 4 * g;
    const int n = blocks - 4 * g;
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

template <int KIND, int BN, bool R_MN, bool C_MN, int EPI>
__global__ void __launch_bounds__(kThreads) tile_kernel(const __grid_constant__ CUtensorMap map_r,
                                                         const __grid_constant__ CUtensorMap map_c, const Params p) {
  using S = Shape<KIND, BN>;
  constexpr bool SYM = EPI == GRAM || EPI == POLY;
  constexpr int kElems = KIND == MX ? 128 : 64;     // values of k in a stage
  static_assert(!SYM || BN <= 128, "symmetric tiles divide 128");
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

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tile = blockIdx.x / p.splits, rank = blockIdx.x % p.splits, batch = blockIdx.z;
  int tr, tcn;
  bool mirror = false;
  if (SYM) {   // row tile j has (j + 1) q column tiles
    constexpr int q = 128 / (BN < 128 ? BN : 128);
    int j = (int)((sqrtf(8.f * (float)(tile / q) + 1.f) - 1.f) * 0.5f);
    while (q * (j + 1) * (j + 2) / 2 <= tile) ++j;
    while (q * j * (j + 1) / 2 > tile) --j;
    tr = j;
    tcn = tile - q * j * (j + 1) / 2;
    mirror = tcn < j * q;
  } else {
    tr = tile % p.tiles_r;
    tcn = tile / p.tiles_r;
  }
  const int r0 = tr * kRowsTile, c0 = tcn * BN;
  const int blocks = (p.k + kElems - 1) / kElems;
  const int kb0 = (int)((int64_t)blocks * rank / p.splits), kb1 = (int)((int64_t)blocks * (rank + 1) / p.splits);

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
  if (warp == 1) tc::tmem_alloc<S::kTmemCols>(slot);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t acc = *slot_p;
  const uint32_t tscale = acc + BN;
  auto gave_up = [&]() {
    *fail = 1;
    atomicCAS(&g_dense_error, 0, kErrTimeout);
  };

  if (warp == 0) {
    if (lane == 0) {
      int issued = 0;
      for (int kb = kb0; kb < kb1; ++kb) {
        const int s = issued % S::kStages;
        if (!tc::mbar_wait(empty + 8 * s, ((issued / S::kStages) & 1) ^ 1)) {
          gave_up();
          break;
        }
        const uint32_t dst = ring + s * S::kStageBytes, bar = full + 8 * s;
        tc::mbar_expect(bar, S::kStageBytes);
        if (R_MN) {
          tc::tma_load3(dst, &map_r, r0, kb * kElems, batch, bar);
          tc::tma_load3(dst + 8192, &map_r, r0 + 64, kb * kElems, batch, bar);
        } else {
          tc::tma_load3(dst, &map_r, kb * kElems, r0, batch, bar);
        }
        if (C_MN) {
#pragma unroll
          for (int i = 0; i < BN / 64; ++i)
            tc::tma_load3(dst + kStageBytesR + 8192 * i, &map_c, c0 + 64 * i, kb * kElems, batch, bar);
        } else {
          tc::tma_load3(dst + kStageBytesR, &map_c, kb * kElems, c0, batch, bar);
        }
        ++issued;
      }
      // no copy is in flight when the block leaves (the products waited for them unless something gave up)
      for (int i = issued > S::kStages ? issued - S::kStages : 0; i < issued; ++i)
        tc::mbar_wait(full + 8 * (i % S::kStages), (i / S::kStages) & 1);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      const uint32_t idesc = KIND == MX ? tc::idesc_mx(128, BN, p.fmt_r, p.fmt_c) : tc::idesc_f16(128, BN, R_MN, C_MN);
      int it = 0, group = -1, groups = 0;
      bool add = false, ok = true;
      for (int kb = kb0; kb < kb1 && ok; ++kb, ++it) {
        const int s = it % S::kStages;
        ok = tc::mbar_wait(full + 8 * s, (it / S::kStages) & 1);
        if (!ok) break;
        uint32_t ts = 0;
        if (KIND == MX) {
          const int ss = (groups - (group == kb / 4 ? 1 : 0)) % S::kScaleStages;
          ts = tscale + ss * S::kScaleCols;
          if (group != kb / 4) {
            group = kb / 4;
            ok = tc::mbar_wait(sfull + 8 * ss, (groups / S::kScaleStages) & 1);
            if (!ok) break;
            ++groups;
            tc::fence_after();
            const uint32_t src = scales + ss * S::kScaleBytes;
            tc::copy_scales(ts, tc::desc_scales(src));
#pragma unroll
            for (int i = 0; i < (BN + 127) / 128; ++i) tc::copy_scales(ts + 4 + 4 * i, tc::desc_scales(src + 512 + 512 * i));
          }
        }
        tc::fence_after();
        const uint32_t a = ring + s * S::kStageBytes, b = a + kStageBytesR;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          // 32 bytes along K, or 16 rows of 128 bytes where K runs over the rows
          const uint64_t da = tc::desc_sw128(a + i * (R_MN ? 2048 : 32), R_MN ? 8192 : 0);
          const uint64_t db = tc::desc_sw128(b + i * (C_MN ? 2048 : 32), C_MN ? 8192 : 0);
          if (KIND == MX) tc::mma_mx(acc, da, db, tc::idesc_mx_id(idesc, kb & 3), ts, ts + 4, add);
          else tc::mma_f16(acc, da, db, idesc, add);
          add = true;
        }
        tc::commit(empty + 8 * s);
        if (KIND == MX && ((kb & 3) == 3 || kb + 1 == kb1)) tc::commit(sempty + 8 * ((groups - 1) % S::kScaleStages));
      }
      if (!ok) gave_up();
      tc::commit(done);
    }
  } else {
    const int t = threadIdx.x - 64;   // 0..127
    bool ok = true;
    if (KIND == MX) {
      const int g1 = kb1 > kb0 ? (kb1 - 1) / 4 + 1 : kb0 / 4;
      int n = 0;
      for (int g = kb0 / 4; g < g1 && ok; ++g, ++n) {
        const int ss = n % S::kScaleStages;
        const uint32_t wr = scale_word(p.sr, p.ld_sr, p.shift_r, r0 + t, p.rows, g, blocks);
        uint32_t wc[(BN + 127) / 128];
#pragma unroll
        for (int i = 0; i < (BN + 127) / 128; ++i) {
          const int c = 128 * i + t;
          wc[i] = scale_word(p.sc, p.ld_sc, p.shift_c, c < BN ? c0 + c : p.cols, p.cols, g, blocks);
        }
        ok = tc::mbar_wait(sempty + 8 * ss, ((n / S::kScaleStages) & 1) ^ 1);
        if (!ok) break;
        uint8_t* dst = smem + (scales - ring) + ss * S::kScaleBytes + (t & 31) * 16 + (t >> 5) * 4;
        *reinterpret_cast<uint32_t*>(dst) = wr;
#pragma unroll
        for (int i = 0; i < (BN + 127) / 128; ++i) *reinterpret_cast<uint32_t*>(dst + 512 + 512 * i) = wc[i];
        tc::fence_async_shared();
        tc::mbar_arrive(sfull + 8 * ss);
      }
    }
    ok = ok && tc::mbar_wait(done, 0);
    if (!ok) gave_up();
  }
  __syncwarp();
  __syncthreads();
  tc::fence_after();

  // The sums: lane r of the warp's quarter, 16 columns at a time.
  const bool usable = *fail == 0;
  if (p.splits == 1) {
    if (warp >= 2 && usable) {
      const int q = warp & 3, r = r0 + 32 * q + lane;
      const uint32_t t = acc + ((uint32_t)(32 * q) << 16);
#pragma unroll
      for (int j = 0; j < BN; j += 16) {
        if (c0 + j >= p.cols) break;
        uint32_t u[16];
        float v[16];
        if (kb1 > kb0) {
          tc::tmem_ld16(t + j, u);
          tc::tmem_wait_ld(u);
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = kb1 > kb0 ? __uint_as_float(u[i]) : 0.f;
        finish16<EPI>(p, batch, r, c0 + j, min(16, p.cols - c0 - j), mirror, v);
      }
    }
  } else {
    float* dump = reinterpret_cast<float*>(smem);   // [BN][128], over the stages: no copy is in flight
    if (warp >= 2) {
      const int q = warp & 3;
      const uint32_t t = acc + ((uint32_t)(32 * q) << 16);
#pragma unroll
      for (int j = 0; j < BN; j += 16) {
        uint32_t u[16];
        if (kb1 > kb0) {
          tc::tmem_ld16(t + j, u);
          tc::tmem_wait_ld(u);
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) dump[(j + i) * 128 + 32 * q + lane] = kb1 > kb0 ? __uint_as_float(u[i]) : 0.f;
      }
    }
    tc::cluster_sync();
    if (warp >= 2 && usable) {
      const int rl = 32 * (warp & 3) + lane;
      const int groups = BN / 16;
      for (int g = rank; g < groups; g += p.splits) {
        if (c0 + 16 * g >= p.cols) break;
        float v[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = 0.f;
        for (int s = 0; s < p.splits; ++s) {
          const uint32_t src = tc::map_rank(ring, s) + ((16 * g) * 128 + rl) * 4;
#pragma unroll
          for (int i = 0; i < 16; ++i) v[i] += tc::ld_cluster(src + i * 512);
        }
        finish16<EPI>(p, batch, r0 + rl, c0 + 16 * g, min(16, p.cols - c0 - 16 * g), mirror, v);
      }
    }
    tc::cluster_sync();
  }
  tc::fence_before();
  __syncthreads();
  if (warp == 1) {
    tc::fence_after();
    tc::tmem_dealloc<S::kTmemCols>(acc);
  }
}

}  // namespace gemm
}  // namespace bcjr
