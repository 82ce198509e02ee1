// Host side of the products with packed weights (bsq_packed_linear).
#include <algorithm>

#include "host_common.h"
#include "host_regions.h"
#include "packed_linear.cuh"
#include "packed_many.cuh"

namespace {

using namespace bsq;

// Blocks that the GPU's 152 SMs hold at a time in clusters of 1 to 8, with one and with two per SM (as reported for these kernels: clusters
// lie within a GPU processing cluster, whose SMs they may not divide).
constexpr int kResident[9] = {0, 152, 152, 138, 144, 140, 138, 105, 120}, kResidentTwo[9] = {0, 304, 304, 291, 296, 290, 276, 266, 288};

// The figures of both sides beside the rules here are of three sets of inputs in turn, part of which stays in L2 with the smaller sizes.
//
// How the kernel for few tokens is laid out: sets of 32 rows per block (1 or 4), pieces of K per block and of its tokens at a time.
//
// The cost is fitted to 1, 2, 4, 8 and 16 tokens with 1 and 4 sets and 1 to 8 blocks along K (10240 x 7168, 7168 x 8192, 4096 x 4096
// NVFP4, 4096 x 8192, 2048 x 16384 and 256 x 7168 MXFP8, 1000 x 2912 MXFP4): a call takes about 5 us and 0.043 us for each unit that the
// fullest SM has, where a unit is a piece of 32 rows, its tokens count 0.23 each, a further segment of tokens 60, a block for which the SM has
// no room at first 85, a sum over a cluster 12, and a block that is alone on its SM a tenth more.  Both sides, in us:
//   1 token, 10240 x 7168: 4 sets and 5 blocks along K 11.8, 1 set and one block 12.6, two 14.0; 4096 x 4096: 1 set and one block 4.3, 4 and 4 5.1
//   8 tokens, 10240 x 7168: 4 sets and 3 blocks 15.2, 7 blocks 18.2, 1 set 35; 2048 x 16384 MXFP8: 4 sets and 6 blocks 14.4, 8 14.9, 4 22.0
//   16 tokens, 7168 x 8192: 4 sets and 5 blocks 15.7, 8 20.9, 1 set 34.9; 256 x 7168 MXFP8: 1 set and 8 blocks 6.2, 4 sets 8.4
struct PlPlan {
  int sets, per_rank, segment, ranks, smem;
};
PlPlan plan_linear(const PlArgs& a, int cols_of_piece, int token_tile) {
  const int toks = a.tokens;  // at most token_tile
  constexpr int kBlockMost = 227 * 1024, kOverhead = 2 * 1024;  // static shared memory and what the system takes, per block
  const int bands = static_cast<int>(ceil_div(a.rows, 128));
  const int token_bytes = cols_of_piece * 2;  // of a piece
  PlPlan best{};
  double least = 0;
  for (int sets = 1; sets <= 4; sets += 3) {
    const int split = kPlWarps / sets, step = split * cols_of_piece % 256 == 0 ? split : 2 * split;  // a segment: a multiple of 256 columns
    const int room = 113 * 1024 - kOverhead - kPlRing;  // for tokens, with two blocks per SM
    const int most = std::max(step, (room / toks - 64) / (step * token_bytes) * step);
    int last = 0;
    for (int r = 1; r <= 8; ++r) {
      const int share = ((a.pieces + r - 1) / r + split - 1) & -split;  // split and step are powers of two
      if (share == last) continue;
      last = share;
      const int ranks = (a.pieces + share - 1) / share, blocks = bands * (4 / sets) * ranks;
      const int segment = std::min(most, (share + step - 1) & -step), more = segment < share ? (share - 1) / segment : 0;
      const int smem = std::max(kPlRing + toks * (segment * token_bytes + 64), kPlWarps * token_tile * 32 * 4);
      const int resident = std::min(token_tile == 8 ? 3 : 2, kBlockMost / (smem + kOverhead));
      const double n = blocks <= kResident[ranks] ? 1.1 : blocks <= kResidentTwo[ranks] ? 2.0 : static_cast<double>((2 * blocks - 1) / kResidentTwo[ranks] + 1);
      const double cost = n * (sets * share + 0.23 / 128 * (share * toks * cols_of_piece) + 60.0 * more) + 85.0 * std::max(0.0, n - resident) +
                          (ranks > 1 ? 12.0 : 0.0);
      if (best.sets == 0 || cost < least) {
        least = cost;
        best = {sets, share, segment, ranks, smem};
      }
    }
  }
  return best;
}

template <int FMT, bool F16, int NT, int RT>
bsq_status launch_linear(PlArgs& a, const PlPlan& plan, const HostDevice& d, cudaStream_t st) {
  auto kernel = packed_linear_kernel<FMT, F16, NT, RT>;
  a.per_rank = plan.per_rank;
  a.segment = plan.segment;
  const int64_t row_tiles = ceil_div(a.rows, 128) * 4 / RT;
  const int ranks = plan.ranks, smem = plan.smem;
  if (bsq_status s = allow_smem(reinterpret_cast<const void*>(kernel), 227 * 1024 - 2048, d.index); s != BSQ_OK) return s;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ranks, static_cast<unsigned>(row_tiles));
  cfg.blockDim = dim3(kPlThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ranks;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, a) == cudaSuccess ? BSQ_OK : BSQ_ERR_CUDA;
}

bool linear_map(CUtensorMap* map, CUtensorMapDataType type, const void* ptr, int64_t inner, int64_t rows, int64_t stride_bytes,
                uint32_t box_inner, uint32_t box_rows, CUtensorMapSwizzle swizzle) {
  auto enc = encode_tiled();
  if (!enc) return false;
  const cuuint64_t dim[2] = {static_cast<cuuint64_t>(inner), static_cast<cuuint64_t>(rows)};
  const cuuint64_t stride[1] = {static_cast<cuuint64_t>(stride_bytes)};
  const cuuint32_t box[2] = {box_inner, box_rows}, ones[2] = {1, 1};
  return enc(map, type, 2, const_cast<void*>(ptr), dim, stride, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int kPmSmem = 227 * 1024 - 2048;  // dynamic shared memory at most: one block per SM

// How the work of the kernel for many tokens is split: tokens of a tile, tiles, blocks along K and their share of it.
struct PmPlan {
  int tokens_tile, token_tiles, row_tiles, ranks, share;
  int64_t tiles;
  double cost;
};
PmPlan plan_many(const PlArgs& p, int mt, int sm_count) {
  PmPlan a{};
  const int most = 256 / mt;
  a.row_tiles = static_cast<int>(ceil_div(p.rows, 128 * mt));
  // tokens of a tile: those with which the last wave of tiles ends first, a tile costing its tokens and about 128 more (2048 tokens, 10240 rows
  // 168 us, with tiles of 256 177; 300 tokens 56 and 64)
  a.token_tiles = static_cast<int>(ceil_div(p.tokens, most));
  int64_t least = INT64_MAX;
  for (int64_t t = a.token_tiles, n = 0; t <= 2 * ceil_div(p.tokens, most); ++t) {
    n = ceil_div(ceil_div(p.tokens, t), 16) * 16;
    const int64_t tiles = a.row_tiles * ceil_div(p.tokens, n), cost = ceil_div(tiles, sm_count) * (n + 128);
    if (tiles >= sm_count ? cost < least : least == INT64_MAX) {
      least = cost;
      a.tokens_tile = static_cast<int>(n);
      a.token_tiles = static_cast<int>(ceil_div(p.tokens, n));
    }
  }
  const int64_t units = ceil_div(p.cols, 128);
  a.tiles = static_cast<int64_t>(a.row_tiles) * a.token_tiles;
  // blocks of a cluster, which share K: the number that ends first, where a block costs its 128 columns' worth and about eight more, and
  // clusters are held by as many SMs as have room for whole ones.  64 tokens, 7168 x 8192, two tiles: 1 to 8 blocks 56, 34, 26, 22, 20,
  // 34, 33, 31 us (5 are taken); 300 tokens 39, 49, 58, 64, 63, 71, 102, 97 (1)
  int64_t best = INT64_MAX;
  for (int r = 1; r <= 8 && (r == 1 || a.tiles < 2 * sm_count); ++r) {
    const int64_t share = ceil_div(units, r), waves = ceil_div(a.tiles * r, kResident[r]);
    if (ceil_div(units, share) == r && waves * (share + 8) < best) {
      best = waves * (share + 8);
      a.ranks = r;
      a.share = static_cast<int>(share);
      // with up to 128 tokens, in us: as measured for 17 to 128 tokens of 7168 x 8192, 16384 x 7168 and 1024 x 8192 NVFP4
      a.cost = waves * (mt == 2 ? 5.0 + 0.055 * p.tokens + 0.9 * share : 5.2 + 0.015 * p.tokens + 0.47 * share);
    }
  }
  return a;
}

template <int FMT, bool F16, int MT>
bsq_status launch_many(const PlArgs& p, const PmPlan& plan, const HostDevice& d, cudaStream_t st) {
  using F = PmFmt<FMT>;
  auto kernel = packed_many_kernel<FMT, F16, MT>;
  const int64_t tiles = plan.tiles;
  if (tiles >= (int64_t(1) << 31)) return BSQ_ERR_SHAPE;
  PmArgs a{};
  a.p = p;
  a.err = d.error_word;
  a.tokens_tile = plan.tokens_tile;
  a.row_tiles = plan.row_tiles;
  a.token_tiles = plan.token_tiles;
  a.share = plan.share;
  const int ranks = plan.ranks;
  a.x_bytes = a.tokens_tile * 128;
  a.w_bytes = static_cast<int>(ceil_div(MT * (F::kTileBytes + F::kAtoms * 512), 1024) * 1024);
  // as many steps as tensor memory holds weights of, four at least, if their tokens leave room for three stages of weights
  const int room = kPmSmem - 1024, d_cols = MT == 1 ? 256 : a.tokens_tile <= 64 ? 128 : 256;
  a.depth = std::min((512 - d_cols) / (32 * MT), std::max(4, (room - 3 * a.w_bytes) / a.x_bytes));
  a.w_stages = std::min(6, (room - a.depth * a.x_bytes) / a.w_bytes);
  // more than half of the SM's memory, and the sums of a cluster's block
  const int smem = std::max({1024 + a.w_stages * a.w_bytes + a.depth * a.x_bytes, 120 * 1024,
                             ranks > 1 ? 1024 + (a.tokens_tile + ranks) * 128 * MT * 4 : 0});
  CUtensorMap mw, mx;
  if (!linear_map(&mw, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.w, p.row_bytes, p.rows, p.row_bytes, 128, 128, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !linear_map(&mx, CU_TENSOR_MAP_DATA_TYPE_UINT16, p.x, p.cols, p.tokens, p.ld_x * 2, 64, a.tokens_tile, CU_TENSOR_MAP_SWIZZLE_128B))
    return BSQ_ERR_CUDA;
  if (bsq_status s = allow_smem(reinterpret_cast<const void*>(kernel), kPmSmem, d.index); s != BSQ_OK) return s;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ranks > 1 ? tiles : std::min<int64_t>(tiles, d.sm_count)), ranks);
  cfg.blockDim = dim3(kPmThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 1;
  attr[1].val.clusterDim.y = ranks;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, mw, mx, a) == cudaSuccess ? BSQ_OK : BSQ_ERR_CUDA;
}

template <int FMT, bool F16>
bsq_status launch_linear_tokens(PlArgs& a, const HostDevice& d, cudaStream_t st) {
  // The weights' stream up to 16 tokens, tensor memory beyond.  10240 x 7168 NVFP4: 16 tokens 23.4 us against 22.5, 24 tokens 38.8 against
  // 22.8; 16384 x 7168: 16 tokens 28.5, 17 tokens with the other kernel 30.3; 1024 x 2048 5.1 and 6.4; 256 x 7168 6.2 and 8.6; 7168 x 8192, from
  // DRAM, 16.7 and 19.3.
  if (a.tokens <= 8) {
    const PlPlan p = plan_linear(a, PlFmt<FMT>::kCols, 8);
    return p.sets == 1 ? launch_linear<FMT, F16, 1, 1>(a, p, d, st) : launch_linear<FMT, F16, 1, 4>(a, p, d, st);
  }
  if (a.tokens <= 16) {
    const PlPlan p = plan_linear(a, PlFmt<FMT>::kCols, 16);
    return p.sets == 1 ? launch_linear<FMT, F16, 2, 1>(a, p, d, st) : launch_linear<FMT, F16, 2, 4>(a, p, d, st);
  }
  // one or two tiles of rows per block.  Two halve the blocks, and so the sums that blocks along K exchange, and share the tokens' columns:
  // 64 tokens, 7168 x 8192 20.0 us against 22.4, 24 tokens 17.3 and 21.0; with too few rows to fill the GPU one is better: 64 tokens,
  // 1024 x 8192 10.2 us against 13.9.  Beyond 128 tokens one tile takes twice as many of them: 192 tokens 26.8 and 36.5.  The cost's constants are
  // of NVFP4; with MX weights (20, 32, 64 and 128 tokens of seven sizes) it names the slower one for 128 tokens of 7168 x 8192, by 5 and 6 %
  // (MXFP4 22.7 and 21.6 us, MXFP8 26.2 and 24.7), for 64 of 16384 x 7168 MXFP8 by 2 %, and the faster one elsewhere.
  const PmPlan one = plan_many(a, 1, d.sm_count);
  if (a.tokens <= 128) {
    const PmPlan two = plan_many(a, 2, d.sm_count);
    if (two.cost < one.cost) return launch_many<FMT, F16, 2>(a, two, d, st);
  }
  return launch_many<FMT, F16, 1>(a, one, d, st);
}

}  // namespace

extern "C" int32_t bsq_packed_linear(int32_t fmt, int32_t dtype, const void* x, int64_t tokens, int64_t cols, int64_t ld_x, const void* w,
                                     const void* w_scales5d, int64_t rows, const float* w_sf, const void* add, int64_t ld_add,
                                     int32_t out_dtype, void* out, int64_t ld_out, void* stream) {
  if (!fmt_ok(fmt) || (dtype != BSQ_BF16 && dtype != BSQ_F16) || (out_dtype != dtype && out_dtype != BSQ_F32)) return BSQ_ERR_VALUE;
  if (tokens < 0 || rows < 0 || tokens > (1 << 20) || rows > (1 << 20) || cols < 32 || cols % 32 != 0 || cols > (1 << 20) ||
      (tokens > 1 && (ld_x < cols || ld_out < rows)) || ld_x < 0 || ld_out < 0 || ld_add < 0 || ld_x >= (int64_t(1) << 31) ||
      ld_out >= (int64_t(1) << 31) || ld_add >= (int64_t(1) << 31) || (add && ld_add != 0 && tokens > 1 && ld_add < rows))
    return BSQ_ERR_SHAPE;
  if (tokens == 0 || rows == 0) return BSQ_OK;
  if (!x || !w || !w_scales5d || !out || (fmt == BSQ_NVFP4 && !w_sf)) return BSQ_ERR_NULL;
  const int elem = out_dtype == BSQ_F32 ? 4 : 2;
  if (!aligned(x, 16) || ld_x % 8 != 0 || !aligned(w, 16) || !aligned(w_scales5d, 16) || !aligned(w_sf, 4) || !aligned(add, elem) ||
      !aligned(out, elem))
    return BSQ_ERR_ALIGN;
  const auto rows_of = [&](const void* at, int64_t width, int64_t step) { return HostRegion{at, width, {step ? tokens : 1, 1}, {step, 0}}; };
  const HostRegion of_out = rows_of(out, rows * elem, ld_out * elem);
  if (regions_overlap(rows_of(x, cols * 2, ld_x * 2), of_out)) return BSQ_ERR_VALUE;
  if (!(add == out && (tokens == 1 || ld_add == ld_out)) && regions_overlap(rows_of(add, rows * elem, ld_add * elem), of_out)) return BSQ_ERR_VALUE;
  HostDevice d;
  if (bsq_status s = host_device(&d); s != BSQ_OK) return s;
  PlArgs a{};
  a.x = static_cast<const uint16_t*>(x);
  a.ld_x = ld_x;
  a.w = static_cast<const uint8_t*>(w);
  a.scales = static_cast<const uint8_t*>(w_scales5d);
  a.sf = w_sf;
  a.add = add;
  a.ld_add = ld_add;
  a.out = out;
  a.ld_out = ld_out;
  a.rows = rows;
  a.tokens = static_cast<int>(tokens);
  a.cols = static_cast<int>(cols);
  a.row_bytes = row_bytes_of(fmt, cols);
  a.pieces = static_cast<int>(ceil_div(a.row_bytes, 64));
  a.k_atoms = static_cast<int>(ceil_div(cols, atom_cols_of(fmt)));
  a.out_f32 = out_dtype == BSQ_F32;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool f16 = dtype == BSQ_F16;
  switch (fmt) {
    case BSQ_NVFP4: return f16 ? launch_linear_tokens<kNVFP4, true>(a, d, st) : launch_linear_tokens<kNVFP4, false>(a, d, st);
    case BSQ_MXFP4: return f16 ? launch_linear_tokens<kMXFP4, true>(a, d, st) : launch_linear_tokens<kMXFP4, false>(a, d, st);
    default: return f16 ? launch_linear_tokens<kMXFP8, true>(a, d, st) : launch_linear_tokens<kMXFP8, false>(a, d, st);
  }
}
