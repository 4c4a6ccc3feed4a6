// mxfp4_product.cu -- products of rows of microscaled 4-bit numbers: a model's
// output head, out[n, v] = sum over k of a[n, k] w[v, k].
//
// The fifth-generation tensor cores multiply such numbers with their scales
// (kind::mxf4, 64 columns an instruction) into float32 accumulators in tensor
// memory.  The head's rows are the instruction's 128 rows and the tokens its
// columns (16 to 256): one token then costs no more than the weights' bytes,
// and an accumulator's lanes are consecutive logits.  An output is the sum of
// the same instructions' results over k in the same order whatever the number
// of tokens, their place in the batch or the tile's width, and no tile is split
// along k: a row's logits do not depend on the batch it came in.
//
// A block per SM walks tiles of 128 head rows by up to 256 tokens (tokens
// fastest, so that neighbours share the head's rows in L2).  With more than 128
// tokens two blocks work as a pair (cta_group::2): on 256 head rows, each with its own
// 128 and half of the tokens in shared memory, so that a token's codes cross from
// L2 once for 256 rows.  One thread copies
// stages of 256 columns (TMA, 128-byte swizzle; scales by bulk copies) through a
// ring in shared memory, one copies the scales on to tensor memory and issues
// the products, and eight warps take the accumulators: each keeps half of a
// row's columns in registers, so that the next tile's products start as soon as
// tensor memory is read, while the logits are still being rounded and stored.
// Measured, 131072 head rows of 4096 columns: one token 53 us (5.4 TB/s of codes and
// scales; memory's copy rate would take 43), 256 tokens 70 us (54), 4096 tokens 776 us
// by itself (5.7 PFLOP/s; the tensor pipe is busy 78% of the time) and 916 us again and
// again, under the power limit.  Single blocks took 922 us, pairs without the
// exchange of logits 916.  (At 168 registers the wide forms keep a few values in local memory:
// 92 bytes in 16 bits, 56 in float32.)
#include <type_traits>

#include <cuda.h>

#include "cluster.cuh"
#include "mxfp4.cuh"
#include "logits_common.cuh"
#include "rans_common.cuh"
#include "rans_internal.h"

namespace rb {
namespace {

constexpr int kHeadRows = 128;                  // of a tile
constexpr int kMostTokens = 256;
constexpr int kStageCols = 256;                 // 128 bytes of codes a row
constexpr int kStageBytes = kStageCols / 2;
constexpr int kStepCols = 64;                   // of one instruction
constexpr int kMaxStages = 12;
constexpr int kEpilogueWarps = 8;
constexpr int kProductThreads = 128 + 32 * kEpilogueWarps;
constexpr int kStoreTokens = 16;                // that change places at a time
constexpr int kPitch = kHeadRows + 4;           // of their rows there
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kScaleCol = 256;             // scales behind the accumulators
constexpr uint32_t kScaleCols = 24;             // of one stage: 8 of the head, 16 of the tokens

struct ProductShape {
  int32_t tokens, head_rows;  // n, V
  int32_t box;                // tokens of a stage's tile (a multiple of 16)
  int32_t token_tiles, tiles;
  int32_t steps;              // of 64 columns
  int32_t groups;             // of 128 columns
  int32_t stages;             // of the ring
  int32_t wait;               // the tokens come from the kernel before
  ProductLimits limits;
};

// Descriptors of shared memory: the upper half is the layout's, the lower one the
// address in units of 16 bytes.
constexpr uint32_t kSwizzledDesc = 1024 >> 4 | 1u << 14 | 2u << 29;  // 8 rows of 128 bytes, swizzled
constexpr uint32_t kPlainDesc = 128 >> 4 | 1u << 14;                 // 8 rows of 16 bytes
__device__ __forceinline__ uint32_t desc_of(uint32_t addr) { return (addr & 0x3ffff) >> 4; }
// 4-bit floats with scales of an exponent's byte, rows along k on both sides.
__device__ __forceinline__ uint32_t instruction(int head_rows, int tokens, int scale_byte) {
  return (uint32_t)scale_byte << 4 | 1u << 7 | 1u << 10 | (uint32_t)(tokens >> 3) << 17 |
         1u << 23 | (uint32_t)(head_rows >> 4) << 24 | (uint32_t)scale_byte << 29;
}
template <bool PAIR>
__device__ __forceinline__ void multiply(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc,
                                         uint32_t sfa, uint32_t sfb, bool add) {
#define RB_MULTIPLY(GROUP)                                                                     \
  asm volatile(                                                                                \
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tsetp.ne.u32 p, %6, 0;\n\t"                     \
      "mov.b64 a, {%1, %7};\n\tmov.b64 b, {%2, %7};\n\t"                                       \
      "tcgen05.mma.cta_group::" GROUP                                                          \
      ".kind::mxf4.block_scale.scale_vec::2X [%0], a, b, %3, [%4], [%5], p;\n\t}" ::"r"(d),    \
      "r"(a), "r"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"((uint32_t)add), "n"(kSwizzledDesc)   \
      : "memory")
  if constexpr (PAIR) RB_MULTIPLY("2");
  else RB_MULTIPLY("1");
#undef RB_MULTIPLY
}
template <bool PAIR>
__device__ __forceinline__ void copy_scales(uint32_t to, uint32_t from) {
#define RB_COPY(GROUP)                                                             \
  asm volatile("{\n\t.reg .b64 d;\n\tmov.b64 d, {%1, %2};\n\t"                     \
               "tcgen05.cp.cta_group::" GROUP ".32x128b.warpx4 [%0], d;\n\t}" ::"r"(to), \
               "r"(from), "n"(kPlainDesc)                                          \
               : "memory")
  if constexpr (PAIR) RB_COPY("2");
  else RB_COPY("1");
#undef RB_COPY
}
// Arrives when the products issued so far are done; of a pair, at both blocks'.
template <bool PAIR>
__device__ __forceinline__ void commit(uint32_t bar) {
  if constexpr (PAIR)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
        "[%0], %1;" ::"r"(bar),
        "h"((uint16_t)3)
        : "memory");
  else
    asm volatile(
        "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
        : "memory");
}
// Arrives at one in this block alone.
template <bool PAIR>
__device__ __forceinline__ void commit_here(uint32_t bar) {
  if constexpr (PAIR)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
        : "memory");
  else
    commit<false>(bar);
}
// The four warps of a half of the accumulators.
__device__ __forceinline__ void meet(int half) {
  asm volatile("bar.sync %0, 128;" ::"r"(1 + half) : "memory");
}
// A barrier in this block or in another one of the cluster.  Relaxed: nothing in memory
// goes with it (a release would wait for the logits' stores).
__device__ __forceinline__ void arrive_at(uint32_t bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool try_wait_cluster(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity), "r"(1000u)
      : "memory");
  return ok != 0;
}
// A tile into this block's memory, announced at a barrier of either of the pair.
__device__ __forceinline__ void load_2d_pair(uint32_t dst, const CUtensorMap *map, int x, int y,
                                             uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void load_2d(uint32_t dst, const CUtensorMap *map, int x, int y,
                                        uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void load_bulk(uint32_t dst, const void *src, uint32_t bytes,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
          "r"(dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}
// One lane of a converged warp.  What only one thread issues stands behind this, in
// code that the whole warp runs: behind `lane == 0`, where the compiler cannot tell
// that its operands are the warp's, every copy and product cost over 100 cycles.
__device__ __forceinline__ bool elected() {
  uint32_t yes;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(yes));
  return yes != 0;
}
// Columns of a warp's 32 accumulator lanes, 16 or 8.
__device__ __forceinline__ void load_columns16(float *v, uint32_t at) {
  uint32_t *u = reinterpret_cast<uint32_t *>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15}, [%16];"
      : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]),
        "=r"(u[7]), "=r"(u[8]), "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]),
        "=r"(u[14]), "=r"(u[15])
      : "r"(at));
}
__device__ __forceinline__ void load_columns(float *v, uint32_t at) {
  uint32_t *u = reinterpret_cast<uint32_t *>(v);
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]),
                 "=r"(u[6]), "=r"(u[7])
               : "r"(at));
}

template <typename O>
struct __align__(4 * sizeof(O)) Four {
  uint32_t x[sizeof(O)];
};
// The tensor maps of a product.
struct ProductMaps {
  CUtensorMap head, tokens;               // codes
  CUtensorMap head_scales, token_scales;  // of a pair
};

// SHORT: waits and copies are limited by the call (always, for float32; to the others a
// limit that is not a constant costs registers: 907 us for 868 for the corpus, where
// float32 with a constant takes 287 us for 250 for 4096 x 50021 x 1024).
// HALF: most columns that an epilogue warp keeps.  PAIR: two blocks on 256 head rows;
// the first of them issues the products, and all copies are announced at its barriers.
template <typename O, int HALF, bool PAIR, bool SHORT>
__global__ void __launch_bounds__(kProductThreads, 1)
    product_kernel(const __grid_constant__ ProductMaps maps, const uint8_t *head_scales,
                   const uint8_t *token_scales, O *out, int64_t out_stride, ProductShape sh,
                   int32_t *status) {
  extern __shared__ unsigned char smem_raw[];
  __shared__ __align__(8) uint64_t full_bar[kMaxStages], empty_bar[kMaxStages], done_bar, free_bar,
      last_bar;
  __shared__ uint32_t tmem_base;
  __shared__ volatile int dead;  // a wait gave up
  const int tid = threadIdx.x, lane = tid & 31, wid = __shfl_sync(kFull, tid >> 5, 0);
  const int rank = PAIR ? (int)cluster_rank() : 0;
  const int first_tile = PAIR ? (int)blockIdx.x >> 1 : (int)blockIdx.x;
  const int tile_step = PAIR ? (int)gridDim.x >> 1 : (int)gridDim.x;
  constexpr int kRows = PAIR ? 2 * kHeadRows : kHeadRows;
  const uint32_t smem = (smem_addr(smem_raw) + 1023u) & ~1023u;
  const uint32_t token_bytes = (uint32_t)(PAIR ? kMostTokens / 2 : sh.box) * kStageBytes;
  const int row_tiles = (sh.box + kMxTileRows - 1) / kMxTileRows;
  const uint32_t at_tokens = kHeadRows * kStageBytes, at_head_scales = at_tokens + token_bytes;
  const uint32_t at_token_scales = at_head_scales + 2 * kMxTileBytes;
  const uint32_t stage_bytes = at_token_scales + (uint32_t)row_tiles * 2 * kMxTileBytes;
  const int per_tile = (sh.steps + 3) / 4;  // stages of a tile
  // tokens of a tile as the products take them: a pair's halves are a multiple of 16
  auto width_of = [&](int left) {
    const int n = min(left, kMostTokens);
    return PAIR ? (n + 31) & ~31 : min(sh.box, (n + 15) & ~15);
  };

  if (wid == 1) {
    if (lane == 0) {
      for (int i = 0; i < sh.stages; ++i) {
        tma::mbar_init(smem_addr(&full_bar[i]), 2);  // the head's side, the tokens'
        tma::mbar_init(smem_addr(&empty_bar[i]), 1);
      }
      tma::mbar_init(smem_addr(&done_bar), 1);
      tma::mbar_init(smem_addr(&last_bar), 1);
      tma::mbar_init(smem_addr(&free_bar), PAIR ? 2 * kEpilogueWarps : kEpilogueWarps);
      dead = 0;
      tma::fence_mbar_init();
      tma::fence_proxy_async();
    }
  } else if (wid == 3) {
    if constexpr (PAIR) {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                       smem_addr(&tmem_base)),
                   "n"(kTmemCols)
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
      asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                       smem_addr(&tmem_base)),
                   "n"(kTmemCols)
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  }
  __syncthreads();
  if constexpr (PAIR) {  // the other block's barriers are there
    cluster_arrive();
    cluster_wait();
  }
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = tmem_base;
  // A barrier's address in the block that issues the products.
  auto leader = [&](const uint64_t *bar) {
    return PAIR ? peer_address(bar, 0) : smem_addr(bar);
  };
  // A warp's wait: until another gave up, or for its own share.
  // (Only what the other block's threads arrive at is waited for at the cluster's scope,
  // whose fences cost more than a stage.)
  constexpr bool kLimited = SHORT || sizeof(O) == 4;
  const uint32_t tries = kLimited ? sh.limits.tries : ProductLimits::kTries;
  auto wait = [&](uint64_t *bar, uint32_t parity, bool cluster = false) {
    const uint32_t b = smem_addr(bar);
    for (uint32_t i = 0; i < tries; ++i) {
      if (__all_sync(kFull, cluster ? try_wait_cluster(b, parity) : mbar_try_wait(b, parity)))
        return true;
      if (__any_sync(kFull, dead)) return false;
    }
    if (lane == 0) {
      dead = 1;
      if (status) report(status, RANS_ERR_TIMEOUT, -1);
    }
    __syncwarp();
    return false;
  };

  if (wid == 0 || wid == 2) {
    // ------------------------------------------------------- the copies --
    // one warp for the head's, one for the tokens'.  (A stage's place is counted up: a
    // division took longer than the stage's products.)
    if (wid == 2 && sh.wait) asm volatile("griddepcontrol.wait;" ::: "memory");
    int tile = first_tile, kb = 0, stage = 0;
    uint32_t lap = 0;
    bool ok = true;
    int mt = tile / sh.token_tiles, nt = tile - mt * sh.token_tiles;
    uint32_t left = wid == 2 && kLimited ? sh.limits.token_stages : ~0u;
    while (tile < sh.tiles && left-- != 0) {
      if (lap > 0) {
        ok = wait(&empty_bar[stage], (lap - 1) & 1);
        if (!ok) break;
      }
      const uint32_t bar = leader(&full_bar[stage]), s = smem + stage * stage_bytes;
      const int row = mt * kRows + rank * kHeadRows;
      if constexpr (PAIR) {
        // Scales as tiles of 1024 bytes, zeros past the last.  The first block expects
        // what both copy: the other's may be there before that, but not before the
        // stage's last use, which its own wait has seen.
        if (elected()) {
          if (wid == 0) {
            if (rank == 0) tma::arrive_expect(smem_addr(&full_bar[stage]), 2 * (at_tokens + 2 * kMxTileBytes));
            load_2d_pair(s, &maps.head, kb * kStageBytes, row, bar);
            load_2d_pair(s + at_head_scales, &maps.head_scales, kb * (2 * kMxTileBytes / 4),
                         row / kMxTileRows, bar);
          } else {
            const int n0 = nt * kMostTokens;
            const int half = width_of(sh.tokens - n0) / 2;
            if (rank == 0)
              tma::arrive_expect(smem_addr(&full_bar[stage]),
                                 2 * (token_bytes + (uint32_t)row_tiles * 2 * kMxTileBytes));
            load_2d_pair(s + at_tokens, &maps.tokens, kb * kStageBytes, n0 + rank * half, bar);
            for (int h = 0; h < row_tiles; ++h)
              load_2d_pair(s + at_token_scales + h * 2 * kMxTileBytes, &maps.token_scales,
                           kb * (2 * kMxTileBytes / 4), n0 / kMxTileRows + h, bar);
          }
        }
      } else {
        const uint32_t bytes = (uint32_t)min(2, sh.groups - 2 * kb) * kMxTileBytes;
        if (elected()) {
          if (wid == 0) {
            tma::arrive_expect(bar, at_tokens + bytes);
            load_2d(s, &maps.head, kb * kStageBytes, row, bar);
            load_bulk(s + at_head_scales,
                      head_scales + ((int64_t)mt * sh.groups + 2 * kb) * kMxTileBytes, bytes, bar);
          } else {
            const int first = nt * (kMostTokens / kMxTileRows);
            const bool two = row_tiles > 1 && (first + 1) * kMxTileRows < sh.tokens;
            tma::arrive_expect(bar, token_bytes + (two ? 2 * bytes : bytes));
            load_2d(s + at_tokens, &maps.tokens, kb * kStageBytes, nt * kMostTokens, bar);
            const uint8_t *scales =
                token_scales + ((int64_t)first * sh.groups + 2 * kb) * kMxTileBytes;
            load_bulk(s + at_token_scales, scales, bytes, bar);
            if (two)
              load_bulk(s + at_token_scales + 2 * kMxTileBytes,
                        scales + (int64_t)sh.groups * kMxTileBytes, bytes, bar);
          }
        }
      }
      __syncwarp();
      if (++stage == sh.stages) {
        stage = 0;
        ++lap;
      }
      if (++kb == per_tile) {
        kb = 0;
        tile += tile_step;
        mt = tile / sh.token_tiles;
        nt = tile - mt * sh.token_tiles;
      }
    }
    if (!ok && rank == 0) {
      // copies in flight write to this block's memory: they end first (as far as all
      // warps have issued theirs)
      for (int i = 0; i < sh.stages; ++i)
        tma::wait_bounded(smem_addr(&full_bar[i]), (i < stage ? lap : lap - 1) & 1,
                          min(tries, 1u << 18));
    }
  } else if (wid == 1 && rank == 0) {
    // ----------------------------------------------------- the products --
    int stage = 0, n_tile = 0;
    uint32_t lap = 0, odd = 0;
    bool ok = true;
    for (int tile = first_tile; tile < sh.tiles; tile += tile_step, ++n_tile) {
      const int width = width_of(sh.tokens - tile % sh.token_tiles * kMostTokens);
      const uint32_t idesc0 = instruction(kRows, width, 0), idesc2 = instruction(kRows, width, 2);
      ok = n_tile == 0 || wait(&free_bar, (uint32_t)(n_tile - 1) & 1, PAIR);
      if (!ok) break;
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      for (int kb = 0; kb < per_tile; ++kb) {
        ok = wait(&full_bar[stage], lap & 1);
        if (!ok) break;
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        const uint32_t s = smem + stage * stage_bytes;
        const uint32_t sf = tmem + kScaleCol + odd * kScaleCols;
        const int groups = min(2, sh.groups - 2 * kb), steps = min(4, sh.steps - 4 * kb);
        if (elected()) {
          const uint32_t a = desc_of(s), b = desc_of(s + at_tokens);
          const uint32_t fa = desc_of(s + at_head_scales), fb = desc_of(s + at_token_scales);
          // a whole stage as constants, the last one of a row by its sizes; 64 columns
          // are 32 bytes, 2 in units of a descriptor, a tile of scales 32
          auto work = [&](int groups, int steps) {
#pragma unroll
            for (int g = 0; g < 2; ++g)
              if (g < groups) {
                copy_scales<PAIR>(sf + 4 * g, fa + 32 * g);
                copy_scales<PAIR>(sf + 8 + 8 * g, fb + 32 * g);
                if (width > kMxTileRows) copy_scales<PAIR>(sf + 12 + 8 * g, fb + 64 + 32 * g);
              }
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (j < steps)
                multiply<PAIR>(tmem, a + 2 * j, b + 2 * j, j & 1 ? idesc2 : idesc0,
                               sf + 4 * (j >> 1), sf + 8 + 8 * (j >> 1), j > 0 || kb > 0);
          };
          if (steps == 4) work(2, 4);
          else work(groups, steps);
          commit<PAIR>(smem_addr(&empty_bar[stage]));
          if (kb == per_tile - 1) commit<PAIR>(smem_addr(&done_bar));
        }
        __syncwarp();
        odd ^= 1;
        if (++stage == sh.stages) {
          stage = 0;
          ++lap;
        }
      }
      if (!ok) break;
    }
    if (!ok) {
      // products in flight: a last commit follows them (at a barrier of its own: nobody
      // is to take it for a tile's)
      if (elected()) commit_here<PAIR>(smem_addr(&last_bar));
      tma::wait_bounded(smem_addr(&last_bar), 0, tries);
    }
  } else if (wid >= 4) {
    // --------------------------------------------------- the accumulators --
    const int quarter = wid & 3, half = (wid - 4) >> 2;
    const uint32_t freed = leader(&free_bar);
    unsigned char *exchange = smem_raw + (smem - smem_addr(smem_raw)) + sh.stages * stage_bytes;
    int n_tile = 0, turn = 0;
    int tile = first_tile;
    for (; tile < sh.tiles; tile += tile_step, ++n_tile) {
      const int mt = tile / sh.token_tiles, n0 = tile % sh.token_tiles * kMostTokens;
      const int left = sh.tokens - n0, width = width_of(left);
      const int c0 = half * (width / 2);
      const int count = min(width / 2, left - c0);  // columns of this warp that are tokens
      if (!wait(&done_bar, (uint32_t)n_tile & 1)) break;
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      float v[HALF];
      const uint32_t from = tmem + ((uint32_t)quarter << 21) + c0;
#pragma unroll
      for (int i = 0; i < HALF; i += 16) {
        if (i + 8 < count) load_columns16(v + i, from + i);
        else if (i < count) load_columns(v + i, from + i);
      }
      asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
      // (nothing is computed from the registers before that)
#pragma unroll
      for (int i = 0; i < HALF; ++i) asm volatile("" : "+f"(v[i]));
      asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
      __syncwarp();
      if (lane == 0) {
        if constexpr (PAIR) arrive_at(freed);
        else arrive(freed);
      }
      const int row0 = mt * kRows + rank * kHeadRows, row = quarter * 32 + lane;
      O *o = out + (int64_t)(n0 + c0) * out_stride + row0;
      if constexpr (HALF < kStoreTokens * 2) {
        if (row0 + row < sh.head_rows) {
#pragma unroll
          for (int i = 0; i < HALF; ++i)
            if (i < count) o[i * out_stride + row] = float_logit<O>(v[i]);
        }
      } else {
        // A lane has one logit of many tokens; 16 tokens at a time change places in shared
        // memory, so that a store takes a token's 128 logits, four a lane.  (Stored as they
        // come, two bytes a lane, they took longer than the products.)  Rows of the
        // result that do not start on a multiple of four lie shifted by as much there, so
        // that whole fours go to aligned places; the four logits left at the two ends go
        // singly.
        const int valid = min(kHeadRows, sh.head_rows - row0);
        const int past0 = (int)((reinterpret_cast<uintptr_t>(o) / sizeof(O)) & 3);
        const int skew = (int)(out_stride & 3);  // from one token to the next
        int at[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) at[i] = row + ((past0 + i * skew) & 3);
        // (a warp's tokens are four apart: their rows are shifted alike)
        const int past = (past0 + quarter * skew) & 3;
        const int edge = lane < 4 - past ? lane : kHeadRows - 4 + lane;
        const O *from = reinterpret_cast<const O *>(exchange) + quarter * kPitch;
        O *to = o + quarter * out_stride;
        const int64_t four = 4 * out_stride;
        // A form for what a result allows, so that little code is run: whole fours; fours
        // between edges; any part of a row.
        auto pieces = [&](auto form) {
          constexpr int FORM = decltype(form)::value;
#pragma unroll
          for (int p = 0; p < HALF; p += kStoreTokens) {
            if (p >= count) break;
            const int shift = (half * 2 + turn) * kStoreTokens * kPitch;
            O *buf = reinterpret_cast<O *>(exchange) + shift;
#pragma unroll
            for (int i = 0; i < kStoreTokens; ++i)
              buf[i * kPitch + at[i & 3]] = float_logit<O>(v[p + i]);
            meet(half);
            const O *f = from + shift;
            if constexpr (FORM == 0) {
              Four<O> x[kStoreTokens / 4];
#pragma unroll
              for (int i = 0; i < kStoreTokens / 4; ++i)
                x[i] = *reinterpret_cast<const Four<O> *>(f + 4 * i * kPitch + 4 * lane);
#pragma unroll
              for (int i = 0; i < kStoreTokens / 4; ++i, to += four)
                *reinterpret_cast<Four<O> *>(to + 4 * lane) = x[i];
            } else {
              const int rows = min(kStoreTokens / 4, (count - p - quarter + 3) >> 2);
              if constexpr (FORM == 1) {
                Four<O> x[kStoreTokens / 4];
                O one[kStoreTokens / 4];
#pragma unroll
                for (int i = 0; i < kStoreTokens / 4; ++i) {
                  x[i] = *reinterpret_cast<const Four<O> *>(f + 4 * i * kPitch + 4 * lane);
                  one[i] = f[4 * i * kPitch + past + (edge & (kHeadRows - 1))];
                }
#pragma unroll
                for (int i = 0; i < kStoreTokens / 4; ++i, to += four)
                  if (i < rows) {
                    if (past == 0 || lane > 0)
                      *reinterpret_cast<Four<O> *>(to + 4 * lane - past) = x[i];
                    if (past && lane < 4) to[edge] = one[i];
                  }
              } else {
#pragma unroll 1
                for (int i = 0; i < kStoreTokens / 4; ++i, to += four)
                  for (int e = lane; e < valid && i < rows; e += 32)
                    to[e] = f[4 * i * kPitch + past + e];
              }
            }
            turn ^= 1;
          }
        };
        if (valid < kHeadRows) pieces(std::integral_constant<int, 2>());
        else if (past0 != 0 || skew != 0 || count % kStoreTokens != 0)
          pieces(std::integral_constant<int, 1>());
        else pieces(std::integral_constant<int, 0>());
      }
    }
    // Where a wait gave up: a half's four warps meet for every piece of a tile, and those
    // that saw the tile done would wait for ever for one that had left.  It meets them
    // in all that is left.
    if constexpr (HALF >= kStoreTokens * 2)
      for (; tile < sh.tiles; tile += tile_step) {
        const int left = sh.tokens - tile % sh.token_tiles * kMostTokens, width = width_of(left);
        const int count = min(width / 2, left - half * (width / 2));
        for (int p = 0; p < count; p += kStoreTokens) meet(half);
      }
  }
  __syncwarp();
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  if constexpr (PAIR) {  // nothing reaches into a block that has left
    cluster_arrive();
    cluster_wait();
  }
  if (wid == 3) {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    if constexpr (PAIR)
      asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                   "n"(kTmemCols));
    else
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                   "n"(kTmemCols));
  }
}

template <typename O, int HALF, bool PAIR, bool SHORT>
int launch_t(const ProductMaps &maps, const rans_mxfp4 &a, const rans_mxfp4 &w, void *out,
             int64_t stride, const ProductShape &sh, uint32_t smem, int32_t *status, int blocks,
             cudaStream_t st) {
  auto kern = product_kernel<O, HALF, PAIR, SHORT>;
  if (ensure_dyn_smem((const void *)kern, smem) != cudaSuccess) return RANS_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(kProductThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  unsigned n = 0;
  if (PAIR) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = 2;
    attr[n].val.clusterDim.y = attr[n].val.clusterDim.z = 1;
    ++n;
  }
  if (sh.wait) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n].val.programmaticStreamSerializationAllowed = 1;
    ++n;
  }
  cfg.attrs = attr;
  cfg.numAttrs = n;
  const cudaError_t e =
      cudaLaunchKernelEx(&cfg, kern, maps, (const uint8_t *)w.scales, (const uint8_t *)a.scales,
                         static_cast<O *>(out), stride, sh, status);
  return e == cudaSuccess ? RANS_OK : RANS_ERR_CUDA;
}

template <typename O, bool SHORT = false>
int launch_o(const ProductMaps &maps, const rans_mxfp4 &a, const rans_mxfp4 &w, void *out,
             int64_t stride, const ProductShape &sh, bool pair, uint32_t smem, int32_t *status,
             int blocks, cudaStream_t st) {
  auto go = [&](auto half, auto two) {
    return launch_t<O, decltype(half)::value, decltype(two)::value, SHORT>(
        maps, a, w, out, stride, sh, smem, status, blocks, st);
  };
  if (pair) return go(std::integral_constant<int, 128>(), std::true_type());
  if (sh.box <= 32) return go(std::integral_constant<int, 16>(), std::false_type());
  if (sh.box <= 128) return go(std::integral_constant<int, 64>(), std::false_type());
  return go(std::integral_constant<int, 128>(), std::false_type());
}

}  // namespace

int launch_mxfp4_product(const rans_mxfp4 &a, const rans_mxfp4 &w, void *out, int dtype,
                         int64_t stride, int32_t *status, bool follows,
                         const ProductLimits &limits, cudaStream_t st) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return RANS_ERR_CUDA;
  const int sms = num_sms(dev);
  // pairs where there are tokens to share and head rows for all of them
  const bool pair = a.rows > kMostTokens / 2 && w.rows >= (int64_t)kHeadRows * sms;
  const int rows = pair ? 2 * kHeadRows : kHeadRows;
  ProductShape sh;
  sh.tokens = (int32_t)a.rows;
  sh.head_rows = (int32_t)w.rows;
  sh.box = pair || a.rows >= kMostTokens ? kMostTokens : (int32_t)((a.rows + 15) & ~15);
  sh.token_tiles = (int32_t)((a.rows + kMostTokens - 1) / kMostTokens);
  const int64_t tiles = (int64_t)sh.token_tiles * ((w.rows + rows - 1) / rows);
  sh.steps = (int32_t)((w.cols + kStepCols - 1) / kStepCols);
  sh.groups = mx_groups(w.cols);
  // a block's stages are counted in 31 bits
  if (tiles * ((sh.steps + 3) / 4) > 0x3fffffff) return RANS_ERR_ARG;
  sh.tiles = (int32_t)tiles;
  sh.wait = follows ? 1 : 0;
  sh.limits = limits;
  const int box = pair ? kMostTokens / 2 : sh.box;  // tokens in a block's memory
  const uint32_t stage = kHeadRows * kStageBytes + (uint32_t)box * kStageBytes +
                         2 * kMxTileBytes * (1 + (uint32_t)(sh.box + kMxTileRows - 1) / kMxTileRows);
  // both halves' logits changing places, two buffers each
  const uint32_t exchange =
      sh.box <= 32 ? 0 : 4u * kStoreTokens * kPitch * (dtype == RANS_LOGITS_F32 ? 4u : 2u);
  const uint32_t room = (uint32_t)smem_optin(dev) - 2048 - exchange;  // its static part, alignment
  sh.stages = (int32_t)(room / stage < (uint32_t)kMaxStages ? room / stage : kMaxStages);
  if (sh.stages < 2) return RANS_ERR_CUDA;
  ProductMaps maps;
  const uint64_t row = (uint64_t)mx_row_bytes(w.cols);
  int e = encode_rows_map(&maps.head, w.codes, row, (uint64_t)w.rows, kHeadRows);
  if (!e) e = encode_rows_map(&maps.tokens, a.codes, row, (uint64_t)a.rows, (uint32_t)box);
  if (!e && pair) {
    const uint64_t width = (uint64_t)sh.groups * (kMxTileBytes / 4);
    auto scale_tiles = [](int64_t n) { return (uint64_t)((n + kMxTileRows - 1) / kMxTileRows); };
    e = encode_words_map(&maps.head_scales, w.scales, width, scale_tiles(w.rows),
                         2 * kMxTileBytes / 4);
    if (!e)
      e = encode_words_map(&maps.token_scales, a.scales, width, scale_tiles(a.rows),
                           2 * kMxTileBytes / 4);
  }
  if (e) return e;
  const uint32_t smem = stage * (uint32_t)sh.stages + 1024 + exchange;
  const int most = pair ? sms / 2 : sms;
  const int blocks = (sh.tiles < most ? sh.tiles : most) * (pair ? 2 : 1);
  switch (dtype) {
    case RANS_LOGITS_F32:
      return launch_o<float>(maps, a, w, out, stride, sh, pair, smem, status, blocks, st);
    case RANS_LOGITS_F16:
      return launch_o<__half>(maps, a, w, out, stride, sh, pair, smem, status, blocks, st);
    default:
      if (!limits.none())
        return launch_o<__nv_bfloat16, true>(maps, a, w, out, stride, sh, pair, smem, status,
                                             blocks, st);
      return launch_o<__nv_bfloat16>(maps, a, w, out, stride, sh, pair, smem, status, blocks, st);
  }
}

}  // namespace rb
