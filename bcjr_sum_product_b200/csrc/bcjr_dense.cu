// Host side of the layer-wise QAT operators declared in include/bcjr.h: 8-bit
// block quantisation, the block-scaled product, Newton-Schulz orthogonalisation
// and the Muon step.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstdlib>
#include <mutex>

#include <cuda.h>
#include <cuda_runtime.h>

#include "bcjr.h"
#include "bcjr_gemm.cuh"
#include "bcjr_host.h"
#include "bcjr_quant.cuh"

namespace bcjr {
namespace host {

int take_dense_error(int* flag) {
  int zero = 0;
  if (cudaMemcpyFromSymbol(flag, gemm::g_dense_error, sizeof(int)) != cudaSuccess) return BCJR_ERR_CUDA;
  if (*flag != 0 && cudaMemcpyToSymbol(gemm::g_dense_error, &zero, sizeof(int)) != cudaSuccess) return BCJR_ERR_CUDA;
  return BCJR_OK;
}

}  // namespace host
}  // namespace bcjr

namespace {

using namespace bcjr::host;
namespace G = bcjr::gemm;
namespace Q = bcjr::quant;

static_assert(G::kErrTimeout == BCJR_ERR_TIMEOUT, "device and host status codes agree");
static_assert((int)G::OUT_F32 == BCJR_F32 && (int)G::OUT_F16 == BCJR_F16 && (int)G::OUT_BF16 == BCJR_BF16, "output types");
static_assert((int)Q::IN_F32 == BCJR_F32 && (int)Q::IN_F16 == BCJR_F16 && (int)Q::IN_BF16 == BCJR_BF16, "input types");

constexpr int64_t kMaxExtent = (int64_t)1 << 30;
constexpr int64_t kMaxMatrix = 65536;   // orthogonalise: rows and columns
constexpr int64_t kMaxBatch = 32767;    // two planes each, along a grid dimension
constexpr int kMaxSteps = 64;

// A device or managed pointer of the current device, aligned to `align` bytes.
int check_ptr(const void* p, size_t align) {
  if (p == nullptr || reinterpret_cast<uintptr_t>(p) % align != 0) return BCJR_ERR_INVALID_ARG;
  cudaPointerAttributes a;
  int dev = 0;
  if (cudaPointerGetAttributes(&a, p) != cudaSuccess || cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return BCJR_ERR_INVALID_ARG;
  }
  if (a.type == cudaMemoryTypeManaged) return BCJR_OK;
  return a.type == cudaMemoryTypeDevice && a.device == dev ? BCJR_OK : BCJR_ERR_INVALID_ARG;
}

bool is_wide(int t) { return t == BCJR_F32 || t == BCJR_F16 || t == BCJR_BF16; }
bool is_8bit(int t) { return t == BCJR_E4M3 || t == BCJR_E5M2; }
size_t size_of(int t) { return t == BCJR_F32 ? 4 : is_8bit(t) ? 1 : 2; }
int64_t up(int64_t n, int64_t m) { return (n + m - 1) / m * m; }
int64_t parts(int64_t n, int64_t m) { return (n + m - 1) / m; }

int sm_count(int* n) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    cudaGetLastError();
    return BCJR_ERR_CUDA;
  }
  return BCJR_OK;
}

// cuTensorMapEncodeTiled through the runtime (the library does not link against the driver).
using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeFn encode_fn() {
  static std::mutex mu;
  static EncodeFn fn = nullptr;
  std::lock_guard<std::mutex> lk(mu);
  if (fn == nullptr) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult st;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &st) == cudaSuccess &&
        st == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeFn>(p);
    else
      cudaGetLastError();
  }
  return fn;
}

// One operand of a product: [batch][outer][inner], rows of `ld` elements.
struct Operand {
  const void* p;
  int64_t inner, outer, ld, batch, batch_stride;
};

// Copies of 128 bytes (inner) x `box` rows, 128-byte swizzle, zeros outside.
int make_map(CUtensorMap* map, const Operand& o, int elem, int box) {
  EncodeFn fn = encode_fn();
  if (fn == nullptr) return BCJR_ERR_CUDA;
  const cuuint64_t dims[3] = {(cuuint64_t)o.inner, (cuuint64_t)o.outer, (cuuint64_t)o.batch};
  const int64_t row = o.outer > 1 ? o.ld * elem : up(o.inner * elem, 16);
  const cuuint64_t strides[2] = {(cuuint64_t)row, (cuuint64_t)(o.batch > 1 ? o.batch_stride * elem : row * o.outer)};
  const cuuint32_t boxes[3] = {(cuuint32_t)(128 / elem), (cuuint32_t)box, 1};
  const cuuint32_t ones[3] = {1, 1, 1};
  const CUresult r = fn(map, elem == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
                        const_cast<void*>(o.p), dims, strides, boxes, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? BCJR_OK : BCJR_ERR_CUDA;
}

// cudaFuncSetAttribute once for each kernel and device.
int allow_smem(const void* kern, std::atomic<uint64_t>* done, int smem) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return BCJR_ERR_CUDA;
  }
  const uint64_t bit = (uint64_t)1 << (dev & 63);
  if (dev < 64 && (done->load(std::memory_order_relaxed) & bit)) return BCJR_OK;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) {
    cudaGetLastError();
    return BCJR_ERR_CUDA;
  }
  if (dev < 64) done->fetch_or(bit, std::memory_order_relaxed);
  return BCJR_OK;
}

// BCJR_DENSE_TEST_NOFILL=1 (tests only): products stop fetching, so that their bounded waits run out and they report
// BCJR_ERR_TIMEOUT.
bool test_nofill() {
  const char* e = std::getenv("BCJR_DENSE_TEST_NOFILL");
  return e && e[0] == '1';
}

// Dependent launch: this kernel's set-up may overlap the end of the kernel before it on
// the stream, where that one allows it (the library's own do); it waits for that one
// before it touches memory.
template <class Kern>
int launch(Kern kern, int64_t grid, int64_t batch, int threads, int smem, int cluster, const CUtensorMap& mr,
           const CUtensorMap& mc, G::Params p, cudaStream_t st) {
  if (grid > INT32_MAX) return BCJR_ERR_UNSUPPORTED;
  p.nofill = test_nofill() ? 1 : 0;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid, 1, (unsigned)batch);
  cfg.blockDim = dim3((unsigned)threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  if (cudaLaunchKernelEx(&cfg, kern, mr, mc, p) != cudaSuccess) {
    cudaGetLastError();
    return BCJR_ERR_CUDA;
  }
  counted_launch();
  return BCJR_OK;
}

template <int KIND, int BN, bool R_MN, bool C_MN, int EPI>
int launch_tile(const Operand& r, const Operand& c, const G::Params& p, cudaStream_t st) {
  using S = G::TileShape<KIND, BN>;
  constexpr int elem = KIND == G::MX ? 1 : 2;
  static std::atomic<uint64_t> done{0};
  CUtensorMap mr, mc;
  int rc;
  if ((rc = make_map(&mr, r, elem, R_MN ? 64 : G::kRowsTile)) || (rc = make_map(&mc, c, elem, C_MN ? 64 : BN))) return rc;
  auto kern = G::tile_kernel<KIND, BN, R_MN, C_MN, EPI>;
  if ((rc = allow_smem(reinterpret_cast<const void*>(kern), &done, S::kSmem))) return rc;
  return launch(kern, (int64_t)p.tiles * p.splits, p.batch, G::kTileThreads, S::kSmem, p.splits, mr, mc, p, st);
}

template <int KIND, int BN, bool R_MN, bool C_MN, int EPI>
int launch_pair(const Operand& r, const Operand& c, const G::Params& p, int nsm, cudaStream_t st) {
  using S = G::PairShape<KIND, BN>;
  constexpr int elem = KIND == G::MX ? 1 : 2;
  static std::atomic<uint64_t> done{0};
  CUtensorMap mr, mc;
  int rc;
  if ((rc = make_map(&mr, r, elem, R_MN ? 64 : G::kRowsTile)) || (rc = make_map(&mc, c, elem, C_MN ? 64 : BN / 2))) return rc;
  auto kern = G::pair_kernel<KIND, BN, R_MN, C_MN, EPI>;
  if ((rc = allow_smem(reinterpret_cast<const void*>(kern), &done, S::kSmem))) return rc;
  const int64_t pairs = std::min<int64_t>((int64_t)p.tiles * p.batch, nsm / 2);
  // The pairs that run together work on neighbouring columns of all of R, which then has to stay in
  // L2 (126 MB); a larger R, second plane included, is taken in bands of 16 tiles (8-bit 8192 x 8192 x 8192: 492 -> 446
  // us; fp16 orthogonalisation of 2048 x 8192, X in two planes of 34 MB: 1475 -> 1435; 8-bit with k = 2048, where R is 16
  // MB, bands cost 3 %).
  G::Params pb = p;
  const int64_t bytes = r.inner * r.outer * elem * (p.second_r == G::ALL ? 2 : 1);
  pb.band = bytes > ((int64_t)48 << 20) ? std::min(p.tiles_r, 16) : p.tiles_r;
  return launch(kern, 2 * pairs, 1, G::kPairThreads, S::kSmem, 2, mr, mc, pb, st);
}

// Blocks of one tile: as many (1, 2, 4 or 8) as the tiles leave room for, each with at least four stages of k.  Exchanging
// the sums costs about 2 us, a stage 0.2.  Updates of 128 x 4096: 143 us unsplit, 95 in up to eight; 512 x 2048: 138 and
// 118; two blocks on an SM instead of one would make the latter slower again (with one plane 105 us against 89).
int splits_for(int64_t tiles, int64_t stages, int nsm) {
  int s = 1;
  while (s < 8 && tiles * s * 2 <= nsm && stages >= s * 8) s *= 2;
  return s;
}

// ------------------------------------------------------------ 8-bit product

template <int BN>
int matmul_tile(const Operand& r, const Operand& c, G::Params p, int nsm, cudaStream_t st) {
  const int64_t tiles = parts(p.rows, G::kRowsTile) * parts(p.cols, BN);
  if (tiles * 8 > INT32_MAX) return BCJR_ERR_UNSUPPORTED;
  p.tiles_r = (int)parts(p.rows, G::kRowsTile);
  p.tiles = (int)tiles;
  p.splits = splits_for(tiles, parts(p.k, 128), nsm);
  return launch_tile<G::MX, BN, false, false, G::OUT>(r, c, p, st);
}
template <int BN>
int matmul_pair(const Operand& r, const Operand& c, G::Params p, int nsm, cudaStream_t st) {
  const int64_t tiles = parts(p.rows, 2 * G::kRowsTile) * parts(p.cols, BN);
  if (tiles > INT32_MAX / 2) return BCJR_ERR_UNSUPPORTED;
  p.tiles_r = (int)parts(p.rows, 2 * G::kRowsTile);
  p.tiles = (int)tiles;
  return launch_pair<G::MX, BN, false, false, G::OUT>(r, c, p, nsm, st);
}

int run_matmul(const Operand& r, const Operand& c, G::Params p, cudaStream_t st) {
  int nsm = 0;
  if (int rc = sm_count(&nsm)) return rc;
  p.batch = p.planes_r = p.planes_c = 1;
  if (p.cols <= 16) return matmul_tile<16>(r, c, p, nsm, st);
  if (p.cols <= 32) return matmul_tile<32>(r, c, p, nsm, st);
  if (p.cols <= 64) return matmul_tile<64>(r, c, p, nsm, st);
  // More columns: the kernel and tile width whose estimated time in us is least.  The estimates are fitted to measured
  // times (100 to 8192 x 512 to 8192 x 512 to 8192); what they choose is within a tenth of the best of the five almost
  // everywhere.  For pairs: rounds over the GPU, each of `block` for 128 values of k and `end`, but at least as long as
  // its stores (256 columns leave room for one set of sums only, whose stores overlap nothing).  For single blocks: rounds
  // of two blocks an SM, `block` shared by the blocks of an SM, and the exchange of sums where k is split.
  // 8192 x 8192 x 2048: pairs of 128 / 224 / 256 columns 160 / 122 / 132 us; 2048 x 2048 x 8192: 44 / 49 / 32;
  // 400 x 2048 x 512: single blocks of 64 / 128 columns 5.7 / 6.6, pairs 8.6 / 10.8 / 11.4; 200 x 2048 x 8192: 16.4 / 12.8,
  // pairs 23 / 28 / 29.
  const int64_t pairs = nsm / 2, rows2 = parts(p.rows, 256), rows = parts(p.rows, 128), blocks = parts(p.k, 128);
  const auto pair = [&](int width, double block, double end, double stores) {
    return 4.0 + (double)parts(rows2 * parts(p.cols, width), pairs) * std::max(blocks * block + end, stores);
  };
  const auto single = [&](int width, double begin, double block, double exchange) {
    const int64_t tiles = rows * parts(p.cols, width);
    const int s = splits_for(tiles, blocks, nsm);
    return begin * (double)parts(tiles * s, 2 * nsm) + std::max(1.0, (double)(tiles * s) / nsm) * (double)parts(blocks, s) * block +
           (s > 1 ? exchange : 0.0);
  };
  const double cost[5] = {single(64, 5.3, 0.30, 1.4), single(128, 5.8, 0.38, 3.5), pair(128, 0.33, 0.4, 2.9),
                          pair(224, 0.435, 0.6, 4.6), pair(256, 0.45, 3.5, 0.0)};
  switch (std::min_element(cost, cost + 5) - cost) {
    case 0: return matmul_tile<64>(r, c, p, nsm, st);
    case 1: return matmul_tile<128>(r, c, p, nsm, st);
    case 2: return matmul_pair<128>(r, c, p, nsm, st);
    case 3: return matmul_pair<224>(r, c, p, nsm, st);
    default: return matmul_pair<256>(r, c, p, nsm, st);
  }
}

// ------------------------------------------------------------ Newton-Schulz

constexpr float kMuonCoeffs[3] = {3.4445f, -4.7750f, 2.0315f};

// The coefficients of each step, and the largest |a + b t + c t^2| that it can reach, by which it can amplify what an
// earlier one left in X.
struct Steps {
  int count;
  float co[3 * kMaxSteps], reach[kMaxSteps];
};

// The iterates and polynomials are kept in fp16 with headroom for entries up to
// 16; the singular values of u / |u| lie in [0, 1].  False if, sampled over the
// interval that each step can reach, the coefficients drive a singular value
// above 2 or |a + b t + c t^2| above 8.  (Muon's own are known: a + b t + c t^2 is
// largest at t = 0.  Sampling them took 3.5 us of every call.)
bool take_steps(const float* co, int steps, Steps* out) {
  out->count = steps;
  if (co == nullptr) {
    for (int i = 0; i < 3 * steps; ++i) out->co[i] = kMuonCoeffs[i % 3];
    for (int s = 0; s < steps; ++s) out->reach[s] = kMuonCoeffs[0];
    return true;
  }
  double top = 1.0;
  for (int s = 0; s < steps; ++s) {
    const double a = out->co[3 * s] = co[3 * s], b = out->co[3 * s + 1] = co[3 * s + 1], c = out->co[3 * s + 2] = co[3 * s + 2];
    double most = 0.0, inner = 0.0;
    for (int i = 0; i <= 256; ++i) {
      const double x = top * i / 256.0, t = x * x;
      most = std::max(most, std::fabs(x * (a + t * (b + t * c))));
      inner = std::max(inner, std::fabs(a + t * (b + t * c)));
    }
    if (!(most <= 2.0) || !(inner <= 8.0)) return false;
    out->reach[s] = (float)inner;
    top = most;
  }
  return true;
}

struct Shape2 {
  int64_t batch, rows, cols;
};

int check_iteration(const Shape2& sh, int steps, const float* coeffs, float eps, Steps* it) {
  if (sh.batch < 0 || sh.rows < 0 || sh.cols < 0) return BCJR_ERR_INVALID_ARG;
  if (steps < 1 || !(eps >= 0.f) || !std::isfinite(eps)) return BCJR_ERR_INVALID_ARG;
  if (steps > kMaxSteps || sh.rows > kMaxMatrix || sh.cols > kMaxMatrix || sh.batch > kMaxBatch) return BCJR_ERR_UNSUPPORTED;
  return take_steps(coeffs, steps, it) ? BCJR_OK : BCJR_ERR_INVALID_ARG;
}

// Stages of k of one product of iterates, but for those of a diagonal.
int64_t stages_of(const G::Params& p) {
  return parts(p.k, 64) * (1 + (p.second_r == G::ALL) + (p.second_c == G::ALL));
}

// Symmetric products x y^T: P = X X^T (or X^T X), B = a I + b P + c P^2, and products of such matrices with one
// another (polynomials of one matrix commute), tiles up to the diagonal.
template <int BN, int EPI, bool MN>
int sym_tile(const Operand& x, const Operand& y, G::Params p, int nsm, cudaStream_t st) {
  const int64_t t = parts(p.rows, G::kRowsTile);
  p.tiles = (int)((G::kRowsTile / BN) * t * (t + 1) / 2);
  p.splits = splits_for((int64_t)p.tiles * p.batch, stages_of(p), nsm);
  return launch_tile<G::F16, BN, MN, MN, EPI>(x, y, p, st);
}
template <int BN, int EPI, bool MN>
int sym_pair(const Operand& x, const Operand& y, G::Params p, int nsm, cudaStream_t st) {
  const int64_t t = parts(p.rows, 2 * G::kRowsTile);
  p.tiles_r = (int)t;
  p.tiles = (int)((2 * G::kRowsTile / BN) * t * (t + 1) / 2);
  return launch_pair<G::F16, BN, MN, MN, EPI>(x, y, p, nsm, st);
}
// Pairs of SMs (tiles of 256 rows) where they have a quarter of the GPU's SMs' number of tiles to work on: from half of
// that on 1024^2 takes 165 us instead of 127, with twice of it 2048^2 takes 339 instead of 272.  Never for matrices of at
// most 128 rows, where half of every such tile is empty: 256 of 128 x 256 take 257 us in single blocks and 415 in pairs,
// 1000 of 32 x 96 345 and 707; from 129 rows on pairs win (64 of 256 x 512: 237 us against 281).  Single blocks take 64
// columns where those fill two blocks an SM at most, else 128 (256 of 128 x 256: 257 us against 306; 1000 of 32 x 96:
// 345 against 495).
template <int EPI, bool MN>
int run_sym(const Operand& x, const Operand& y, const G::Params& p, int nsm, cudaStream_t st) {
  const int64_t t = parts(p.rows, G::kRowsTile), t2 = parts(p.rows, 2 * G::kRowsTile);
  if (p.rows > G::kRowsTile && t2 * (t2 + 1) * p.batch * 4 >= nsm) return sym_pair<128, EPI, MN>(x, y, p, nsm, st);
  if (t * (t + 1) * p.batch <= 2 * nsm) return sym_tile<64, EPI, MN>(x, y, p, nsm, st);
  return sym_tile<128, EPI, MN>(x, y, p, nsm, st);
}

// X' = B X (or X B).
template <int BN, int EPI, bool R_MN>
int iter_tile(const Operand& r, const Operand& c, G::Params p, int nsm, cudaStream_t st) {
  p.tiles_r = (int)parts(p.rows, G::kRowsTile);
  p.tiles = (int)(p.tiles_r * parts(p.cols, BN));
  p.splits = splits_for((int64_t)p.tiles * p.batch, stages_of(p), nsm);
  return launch_tile<G::F16, BN, R_MN, false, EPI>(r, c, p, st);
}
template <int BN, int EPI, bool R_MN>
int iter_pair(const Operand& r, const Operand& c, G::Params p, int nsm, cudaStream_t st) {
  p.tiles_r = (int)parts(p.rows, 2 * G::kRowsTile);
  p.tiles = (int)(p.tiles_r * parts(p.cols, BN));
  return launch_pair<G::F16, BN, R_MN, false, EPI>(r, c, p, nsm, st);
}
// As for the symmetric products: pairs from a quarter (from an eighth 1024 x 2048 takes 168 us instead of 143, from a half
// 2048^2 275 instead of 272), and not for 128 rows or fewer (64 of 128 x 128: 91 us against 155).  Single blocks take 64
// columns up to two blocks an SM (16 of 333 x 130: 119 us, up to one block an SM 136), else 128 (300 of 96 x 40: 209 us
// against 219).
template <int EPI, bool R_MN>
int run_iter(const Operand& r, const Operand& c, const G::Params& p, int nsm, cudaStream_t st) {
  const int64_t t = parts(p.rows, G::kRowsTile), t2 = parts(p.rows, 2 * G::kRowsTile);
  if (p.rows > G::kRowsTile && t2 * parts(p.cols, 256) * p.batch * 4 >= nsm)
    return iter_pair<256, EPI, R_MN>(r, c, p, nsm, st);
  // (one wide matrix that is not for pairs never has more tiles than that)
  if constexpr (!(EPI == G::STEP && R_MN))
    if (p.cols > 64 && t * parts(p.cols, 64) * p.batch > 2 * nsm) return iter_tile<128, EPI, R_MN>(r, c, p, nsm, st);
  return iter_tile<64, EPI, R_MN>(r, c, p, nsm, st);
}

// Whether the first two steps are worth doing at once: with B1 = B(P1), P2 = B1 P1 B1 and B2 = B(P2), X <- (B2 B1) X takes
// one Gram matrix of X and one product with X instead of two, for three more products of the shorter
// side's size (1536 x 6145: 456 us against 494; 8192 x 2048: 650 against 720).  Estimated from measured times: 5 us for
// each product's beginning and end, and 1.3, 1.6 and 0.9 PFLOP/s for Gram matrices (whole flops), products with X and
// small symmetric products.
// Only the first two, and from 512 rows on.  A rounding N of P turns a direction of eigenvalue t into others by
// |N u| (f(t) - f(0)) / t, with f = B2 B1 from 11.9 at t = 0 to 0.5 at t = 1.  |N u| is about 2^-12 t sqrt(rank / m), and
// at first t is at most 1 / rank: next to nothing (512 rows or more: as one step at a time; 16 x 3652: 2.3e-3 against
// 1.1e-3).  Later every t is near 1: the last two steps at once made results of rank 256 of 1536 x 6145 wrong by 6e-3.
bool worth_pairing(const Shape2& sh) {
  if (std::min(sh.rows, sh.cols) < 512) return false;
  const double m = (double)std::min(sh.rows, sh.cols), n = (double)std::max(sh.rows, sh.cols), b = (double)sh.batch;
  const double saved = 10.0 + 1e6 * b * m * m * n * (1 / 1.3e15 + 2 / 1.6e15);
  return saved > 1.1 * 3.0 * (5.0 + 1e6 * b * m * m * m / 0.9e15);
}

template <int T>
int launch_update(const Q::UpdateParams& u, int64_t batch, cudaStream_t st) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)u.parts, (unsigned)batch, 1);
  cfg.blockDim = dim3(Q::kUpdateThreads, 1, 1);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, Q::norm_kernel<T>, u);
  if (e == cudaSuccess) e = cudaLaunchKernelEx(&cfg, Q::start_kernel<T>, u);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return BCJR_ERR_CUDA;
  }
  counted_launch(2);
  return BCJR_OK;
}

// The whole iteration; `last` holds the epilogue of the last product (out, its layout and type, the weights'
// factors) and says which by `epi`.  `precise`: every product with all second planes, for a result of more than 8 bits.
// So are matrices of fewer than 32 rows (or columns), too few for roundings to average out (2 x 5 otherwise up to 1e-2, 8 x 8
// 4e-3, 32 x 32 1.4e-3): they have one block of k, so it is a stage or two more.  Not the Gram matrix of a long one, where
// X's roundings average out along the other side (1024: 2^-11 / 55).
int run_newton_schulz(const Shape2& sh, Q::UpdateParams u, int g_type, const Steps& it, int epi, bool precise, const G::Params& last,
                      cudaStream_t st) {
  const int steps = it.count;
  int nsm = 0;
  if (int rc = sm_count(&nsm)) return rc;
  const bool tall = sh.rows > sh.cols;
  const int64_t m = std::min(sh.rows, sh.cols);
  const int64_t ld_x = up(sh.cols, 8), ld_p = up(m, 8);
  const int64_t nx = sh.rows * ld_x, np = m * ld_p;
  // warps take 512 columns of a row at a time; enough blocks of eight warps for every SM four times over
  const int64_t items = sh.rows * parts(sh.cols, Q::kSpan);
  u.parts = (int)std::max<int64_t>(1, std::min<int64_t>(parts(items, 8), parts(8 * nsm, sh.batch)));
  const bool pairing = steps > 1 && worth_pairing(sh);
  // The product with X_s reads its second plane unless what one plane leaves out can grow at most four times in the steps
  // that are left (Muon's last step: 3.4): a result of rank 1, 512 x 512, is off by 0.9e-3 with both planes in all five
  // steps, 1.4e-3 in all but the last, 2.9e-3 in all but the last two, 0.15 in none.
  const bool all = precise || m < 32, gram_all = precise || (all && std::max(sh.rows, sh.cols) < 1024);
  bool both[kMaxSteps];
  double gain = 1.0;
  for (int s = steps - 1; s >= 0; --s) {
    gain *= it.reach[s];
    both[s] = all || gain > 4.0;
  }
  const bool across = !all && m >= 512;   // see kIterScale
  const int sq_planes = across ? 3 : 2;
  const G::Second squares = all ? G::ALL : G::DIAGONAL;
  __half *x0, *x1, *pp, *bb, *tt;
  const int64_t next = up(sh.batch * sq_planes * np, 128);   // from one square matrix to the next
  double* partial;
  auto layout = [&](Arena& ar) {
    partial = ar.take<double>((size_t)(sh.batch * u.parts));
    for (__half** x : {&x0, &x1}) *x = ar.take<__half>((size_t)(sh.batch * 2 * nx));
    pp = ar.take<__half>((size_t)((pairing ? 3 : 2) * next));
    bb = pp + next;
    tt = bb + next;   // where steps are paired
  };
  Arena sizing;
  layout(sizing);
  void* mem = nullptr;
  if (int rc = scratch_alloc(&mem, sizing.off, st)) return rc;
  Arena ar;
  ar.base = static_cast<char*>(mem);
  layout(ar);

  u.partial = partial;
  u.x = x0;
  u.ld_x = ld_x;
  u.batch_x = 2 * nx;
  u.plane_x = nx;
  u.planes = both[0] ? 2 : 1;
  if (!all) {
    u.squares = pp + np;
    u.ld_s = ld_p;
    u.plane_s = np;
    u.batch_s = sq_planes * np;
    u.next_s = next;
    u.cleared = sq_planes - 1;
    u.side = (int)m;
    u.count = pairing ? 3 : 2;
  }
  u.rows = (int)sh.rows;
  u.cols = (int)sh.cols;
  u.scale = G::kIterScale;
  u.vec = u.ld_g % 4 == 0 && (sh.batch == 1 || u.batch_g % 4 == 0) &&
          reinterpret_cast<uintptr_t>(u.g) % (4 * size_of(g_type)) == 0 &&
          (u.momentum == nullptr || (u.ld_m % 4 == 0 && reinterpret_cast<uintptr_t>(u.momentum) % 16 == 0));
  int rc = g_type == BCJR_F32   ? launch_update<Q::IN_F32>(u, sh.batch, st)
           : g_type == BCJR_F16 ? launch_update<Q::IN_F16>(u, sh.batch, st)
                                : launch_update<Q::IN_BF16>(u, sh.batch, st);
  G::Params p{};
  p.rows = p.cols = (int)m;
  p.batch = (int)sh.batch;
  p.planes_r = p.planes_c = sq_planes;
  p.ld_out = p.ld_x = ld_p;
  p.batch_out = p.batch_x = sq_planes * np;
  p.plane_out = p.plane_x = np;
  p.second_out = squares;
  p.third_out = across ? 1 : 0;
  const auto square = [&](const __half* q) { return Operand{q, m, m, ld_p, sh.batch * sq_planes, np}; };
  // out = B(x) with the coefficients of step s; out = x y
  const auto polynomial = [&](__half* out, const __half* x, int s) {
    G::Params q = p;
    q.k = (int)m;
    q.second_r = q.second_c = squares;
    q.out = out;
    q.x = x;
    q.fa = it.co[3 * s];
    q.fb = it.co[3 * s + 1];
    q.fc = it.co[3 * s + 2];
    return run_sym<G::POLY, false>(square(x), square(x), q, nsm, st);
  };
  const auto product = [&](__half* out, const __half* x, const __half* y) {
    G::Params q = p;
    q.k = (int)m;
    q.second_r = q.second_c = squares;
    q.out = out;
    return run_sym<G::GRAM, false>(square(x), square(y), q, nsm, st);
  };
  for (int s = 0; s < steps && rc == BCJR_OK;) {
    const bool two = pairing && s == 0 && it.reach[0] * it.reach[1] <= 15.f;   // their product stays within fp16's headroom
    // X along its rows (inner = columns): the Gram matrix of the shorter side
    // sums over the columns (wide, K-major) or over the rows (tall, MN-major)
    const Operand x{x0, sh.cols, sh.rows, ld_x, sh.batch * 2, nx};
    G::Params gram = p;
    gram.k = (int)(tall ? sh.rows : sh.cols);
    gram.planes_r = gram.planes_c = 2;
    gram.second_r = gram.second_c = gram_all ? G::ALL : G::NONE;
    gram.out = pp;
    rc = tall ? run_sym<G::GRAM, true>(x, x, gram, nsm, st) : run_sym<G::GRAM, false>(x, x, gram, nsm, st);
    if (rc || (rc = polynomial(bb, pp, s))) break;
    if (two && ((rc = product(tt, bb, pp)) || (rc = product(pp, tt, bb)) || (rc = polynomial(tt, pp, s + 1)) ||
                (rc = product(pp, tt, bb))))
      break;
    const G::Second second = !both[s] ? G::NONE : across ? G::ACROSS : G::ALL;
    s += two ? 2 : 1;
    // wide: D[r = column][c = row] = sum_k X[k][r] B[c][k]; tall: sum_k B[r][k] X[c][k]
    const Operand poly = square(two ? pp : bb);
    const bool end = s == steps;
    G::Params q = end ? last : G::Params{};
    q.rows = (int)sh.cols;
    q.cols = (int)sh.rows;
    q.k = (int)m;
    q.batch = (int)sh.batch;
    (tall ? q.planes_r : q.planes_c) = sq_planes;
    (tall ? q.planes_c : q.planes_r) = 2;
    (tall ? q.second_r : q.second_c) = squares;
    (tall ? q.second_c : q.second_r) = second;
    if (!end) {
      q.out = x1;
      q.ld_out = ld_x;
      q.batch_out = 2 * nx;
      q.plane_out = nx;
      q.second_out = both[s] ? G::ALL : G::NONE;
    }
#define BCJR_ITER(E) (tall ? run_iter<E, false>(poly, x, q, nsm, st) : run_iter<E, true>(x, poly, q, nsm, st))
    rc = !end ? BCJR_ITER(G::ITER) : epi == G::STEP ? BCJR_ITER(G::STEP) : BCJR_ITER(G::LAST);
#undef BCJR_ITER
    std::swap(x0, x1);
  }
  if (cudaFreeAsync(mem, st) != cudaSuccess && rc == BCJR_OK) rc = BCJR_ERR_CUDA;
  return rc;
}

template <int T, bool PIPE>
int launch_quantise(const Q::QuantParams& p, bool e5m2, bool row_blocks, int grid, cudaStream_t st) {
  static std::atomic<uint64_t> done[4];
  void (*kern)(Q::QuantParams) =
      e5m2 ? (row_blocks ? Q::quantise_kernel<T, true, true, PIPE> : Q::quantise_kernel<T, true, false, PIPE>)
           : (row_blocks ? Q::quantise_kernel<T, false, true, PIPE> : Q::quantise_kernel<T, false, false, PIPE>);
  const int values = Q::kRows * Q::kThreads * 4;
  const int smem = PIPE ? values * (T == Q::IN_F32 ? 4 : 2) + (p.minus != nullptr ? values * 4 : 0) : 0;
  if (PIPE) {
    const int most = values * (T == Q::IN_F32 ? 8 : 6);
    if (int rc = allow_smem(reinterpret_cast<const void*>(kern), &done[2 * e5m2 + row_blocks], most)) return rc;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid, 1, 1);
  cfg.blockDim = dim3(Q::kThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kern, p) != cudaSuccess) {
    cudaGetLastError();
    return BCJR_ERR_CUDA;
  }
  counted_launch();
  return BCJR_OK;
}

// From four rounds of tiles on, blocks stay (two to an SM, or one where both x and minus, 96 to
// 128 KB of a tile, are fetched ahead) and fetch ahead.
template <int T>
int run_quantise(Q::QuantParams p, bool e5m2, bool row_blocks, int nsm, cudaStream_t st) {
  if (p.vec && p.tiles > 4 * nsm)
    return launch_quantise<T, true>(p, e5m2, row_blocks, p.minus != nullptr ? nsm : 2 * nsm, st);
  return launch_quantise<T, false>(p, e5m2, row_blocks, p.tiles, st);
}

}  // namespace

extern "C" {

int bcjr_fp8_quantise(const void* x, int x_type, int64_t rows, int64_t cols, int64_t ld_x, const float* minus,
                      int64_t ld_minus, int q_type, int block_rows, void* q, int64_t ld_q, void* scale,
                      int64_t ld_scale, void* qt, int64_t ld_qt, void* scale_t, int64_t ld_scale_t, void* stream) {
  if (rows < 0 || cols < 0 || !is_wide(x_type) || !is_8bit(q_type)) return BCJR_ERR_INVALID_ARG;
  if (block_rows != 1 && block_rows != 128) return BCJR_ERR_INVALID_ARG;
  if ((q == nullptr) != (scale == nullptr) || (qt == nullptr) != (scale_t == nullptr)) return BCJR_ERR_INVALID_ARG;
  if (rows > kMaxExtent || cols > kMaxExtent) return BCJR_ERR_UNSUPPORTED;
  if (rows == 0 || cols == 0) return BCJR_OK;
  if (q == nullptr && qt == nullptr) return BCJR_ERR_INVALID_ARG;
  const int64_t tiles_r = parts(rows, 128), tiles_c = parts(cols, 128);
  if (ld_x < cols || (minus != nullptr && ld_minus < cols)) return BCJR_ERR_INVALID_ARG;
  if (q != nullptr && (ld_q < cols || ld_q % 16 != 0 || ld_scale < tiles_c)) return BCJR_ERR_INVALID_ARG;
  if (qt != nullptr && (ld_qt < rows || ld_qt % 16 != 0 || ld_scale_t < tiles_r)) return BCJR_ERR_INVALID_ARG;
  if (tiles_r * tiles_c > INT32_MAX) return BCJR_ERR_UNSUPPORTED;
  int rc;
  if ((rc = check_ptr(x, size_of(x_type)))) return rc;
  if (minus != nullptr && (rc = check_ptr(minus, 4))) return rc;
  if (q != nullptr && ((rc = check_ptr(q, 16)) || (rc = check_ptr(scale, 1)))) return rc;
  if (qt != nullptr && ((rc = check_ptr(qt, 16)) || (rc = check_ptr(scale_t, 1)))) return rc;
  Q::QuantParams p{};
  p.x = x; p.minus = minus;
  p.q = static_cast<uint8_t*>(q); p.s = static_cast<uint8_t*>(scale);
  p.qt = static_cast<uint8_t*>(qt); p.st = static_cast<uint8_t*>(scale_t);
  p.ld_x = ld_x; p.ld_minus = ld_minus; p.ld_q = ld_q; p.ld_s = ld_scale; p.ld_qt = ld_qt; p.ld_st = ld_scale_t;
  p.rows = (int)rows; p.cols = (int)cols; p.tiles_c = (int)tiles_c;
  p.vec = ld_x % 4 == 0 && reinterpret_cast<uintptr_t>(x) % (4 * size_of(x_type)) == 0 &&
          (minus == nullptr || (ld_minus % 4 == 0 && reinterpret_cast<uintptr_t>(minus) % 16 == 0));
  int nsm = 0;
  if ((rc = sm_count(&nsm))) return rc;
  p.tiles = (int)(tiles_r * tiles_c);
  const bool e5m2 = q_type == BCJR_E5M2;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (x_type == BCJR_F32) return run_quantise<Q::IN_F32>(p, e5m2, block_rows == 1, nsm, st);
  if (x_type == BCJR_F16) return run_quantise<Q::IN_F16>(p, e5m2, block_rows == 1, nsm, st);
  return run_quantise<Q::IN_BF16>(p, e5m2, block_rows == 1, nsm, st);
}

int bcjr_fp8_matmul(const void* a, int a_type, int64_t ld_a, const void* scale_a, int64_t ld_scale_a, int a_block_rows,
                    const void* b, int b_type, int64_t ld_b, const void* scale_b, int64_t ld_scale_b, int b_block_rows,
                    int64_t M, int64_t N, int64_t K, float alpha, void* out, int out_type, int64_t ld_out,
                    void* stream) {
  if (M < 0 || N < 0 || K < 0 || !is_8bit(a_type) || !is_8bit(b_type) || !is_wide(out_type)) return BCJR_ERR_INVALID_ARG;
  if ((a_block_rows != 1 && a_block_rows != 128) || (b_block_rows != 1 && b_block_rows != 128)) return BCJR_ERR_INVALID_ARG;
  if (!std::isfinite(alpha)) return BCJR_ERR_INVALID_ARG;
  if (M > kMaxExtent || N > kMaxExtent || K > kMaxExtent) return BCJR_ERR_UNSUPPORTED;
  if (M == 0 || N == 0) return BCJR_OK;
  if (ld_out < N) return BCJR_ERR_INVALID_ARG;
  int rc;
  if ((rc = check_ptr(out, size_of(out_type)))) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (K == 0)
    return cudaMemset2DAsync(out, (size_t)ld_out * size_of(out_type), 0, (size_t)N * size_of(out_type), (size_t)M, st) == cudaSuccess
               ? BCJR_OK
               : BCJR_ERR_CUDA;
  const int64_t kb = parts(K, 128);
  if (ld_a < K || ld_a % 16 != 0 || ld_b < K || ld_b % 16 != 0 || ld_scale_a < kb || ld_scale_b < kb) return BCJR_ERR_INVALID_ARG;
  if ((rc = check_ptr(a, 16)) || (rc = check_ptr(b, 16)) || (rc = check_ptr(scale_a, 1)) || (rc = check_ptr(scale_b, 1)))
    return rc;
  // r (the lanes) runs along the rows of out
  const Operand r{b, K, N, ld_b, 1, 0}, c{a, K, M, ld_a, 1, 0};
  G::Params p{};
  p.rows = (int)N; p.cols = (int)M; p.k = (int)K;
  p.sr = static_cast<const uint8_t*>(scale_b); p.sc = static_cast<const uint8_t*>(scale_a);
  p.ld_sr = ld_scale_b; p.ld_sc = ld_scale_a;
  p.shift_r = b_block_rows == 128 ? 7 : 0; p.shift_c = a_block_rows == 128 ? 7 : 0;
  p.fmt_r = b_type == BCJR_E5M2 ? 1 : 0; p.fmt_c = a_type == BCJR_E5M2 ? 1 : 0;
  p.out = out; p.ld_out = ld_out; p.out_type = out_type; p.fa = alpha;
  return run_matmul(r, c, p, st);
}

int bcjr_orthogonalise(const void* g, int g_type, int64_t batch, int64_t rows, int64_t cols, int64_t ld_g,
                       int64_t batch_stride_g, int steps, const float* coeffs, float eps, void* out, int out_type,
                       int64_t ld_out, int64_t batch_stride_out, void* stream) {
  const Shape2 sh{batch, rows, cols};
  Steps it;
  int rc = check_iteration(sh, steps, coeffs, eps, &it);
  if (rc) return rc;
  if (!is_wide(g_type) || (out_type != BCJR_F16 && out_type != BCJR_BF16)) return BCJR_ERR_INVALID_ARG;
  if (batch == 0 || rows == 0 || cols == 0) return BCJR_OK;
  if (ld_g < cols || ld_out < cols) return BCJR_ERR_INVALID_ARG;
  if (batch > 1 && (batch_stride_g < 0 || batch_stride_out < (rows - 1) * ld_out + cols)) return BCJR_ERR_INVALID_ARG;
  if ((rc = check_ptr(g, size_of(g_type))) || (rc = check_ptr(out, 2))) return rc;
  Q::UpdateParams u{};
  u.g = g; u.ld_g = ld_g; u.batch_g = batch_stride_g; u.eps = eps;
  G::Params last{};
  last.out = out; last.ld_out = ld_out; last.batch_out = batch_stride_out; last.out_type = out_type;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return run_newton_schulz(sh, u, g_type, it, G::LAST, out_type != BCJR_BF16, last, st);
}

int bcjr_muon_step(float* w, int64_t ld_w, const void* grad, int grad_type, int64_t ld_grad, float* momentum,
                   int64_t ld_momentum, int64_t rows, int64_t cols, float lr, float mu, int nesterov,
                   float weight_decay, float scale, int steps, const float* coeffs, float eps, void* stream) {
  const Shape2 sh{1, rows, cols};
  Steps it;
  int rc = check_iteration(sh, steps, coeffs, eps, &it);
  if (rc) return rc;
  if (!is_wide(grad_type)) return BCJR_ERR_INVALID_ARG;
  if (!std::isfinite(lr) || !std::isfinite(mu) || !std::isfinite(weight_decay) || !std::isfinite(scale)) return BCJR_ERR_INVALID_ARG;
  if (rows == 0 || cols == 0) return BCJR_OK;
  if (ld_w < cols || ld_grad < cols || ld_momentum < cols) return BCJR_ERR_INVALID_ARG;
  if ((rc = check_ptr(w, 4)) || (rc = check_ptr(grad, size_of(grad_type))) || (rc = check_ptr(momentum, 4))) return rc;
  Q::UpdateParams u{};
  u.g = grad; u.ld_g = ld_grad; u.momentum = momentum; u.ld_m = ld_momentum;
  u.mu = mu; u.nesterov = nesterov ? 1 : 0; u.eps = eps;
  G::Params last{};
  last.out = w; last.ld_out = ld_w;
  last.keep = (float)(1.0 - (double)lr * (double)weight_decay);
  last.rate = (float)((double)lr * (double)scale);
  return run_newton_schulz(sh, u, grad_type, it, G::STEP, false, last, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
