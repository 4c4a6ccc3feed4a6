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
// fastest, so that neighbours share the head's rows in L2).  One thread copies
// stages of 256 columns (TMA, 128-byte swizzle; scales by bulk copies) through a
// ring in shared memory, one copies the scales on to tensor memory and issues
// the products, and eight warps take the accumulators: each keeps half of a
// row's columns in registers, so that the next tile's products start as soon as
// tensor memory is read, while the logits are still being rounded and stored.
#include <cuda.h>

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
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kScaleCol = 256;             // scales behind the accumulators
constexpr uint32_t kScaleCols = 24;             // of one stage: 8 of the head, 16 of the tokens
constexpr uint32_t kTries = 1u << 21;           // of a bounded wait, about 1 us each

struct ProductShape {
  int32_t tokens, head_rows;  // n, V
  int32_t box;                // tokens of a stage's tile (a multiple of 16)
  int32_t token_tiles, tiles;
  int32_t steps;              // of 64 columns
  int32_t groups;             // of 128 columns
  int32_t stages;             // of the ring
  int32_t wait;               // the tokens come from the kernel before
};

// Descriptors of shared memory: the upper half is the layout's, the lower one the
// address in units of 16 bytes.
constexpr uint32_t kSwizzledDesc = 1024 >> 4 | 1u << 14 | 2u << 29;  // 8 rows of 128 bytes, swizzled
constexpr uint32_t kPlainDesc = 128 >> 4 | 1u << 14;                 // 8 rows of 16 bytes
__device__ __forceinline__ uint32_t desc_of(uint32_t addr) { return (addr & 0x3ffff) >> 4; }
// 4-bit floats with scales of an exponent's byte, rows along k on both sides.
__device__ __forceinline__ uint32_t instruction(int tokens, int scale_byte) {
  return (uint32_t)scale_byte << 4 | 1u << 7 | 1u << 10 | (uint32_t)(tokens >> 3) << 17 |
         1u << 23 | (uint32_t)(kHeadRows >> 4) << 24 | (uint32_t)scale_byte << 29;
}
__device__ __forceinline__ void multiply(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc,
                                         uint32_t sfa, uint32_t sfb, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tsetp.ne.u32 p, %6, 0;\n\t"
      "mov.b64 a, {%1, %7};\n\tmov.b64 b, {%2, %7};\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], a, b, %3, [%4], [%5], "
      "p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"((uint32_t)add), "n"(kSwizzledDesc)
      : "memory");
}
__device__ __forceinline__ void copy_scales(uint32_t to, uint32_t from) {
  asm volatile(
      "{\n\t.reg .b64 d;\n\tmov.b64 d, {%1, %2};\n\t"
      "tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], d;\n\t}" ::"r"(to),
      "r"(from), "n"(kPlainDesc)
      : "memory");
}
__device__ __forceinline__ void commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                   bar)
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
// Eight columns of a warp's 32 accumulator lanes.
__device__ __forceinline__ void load_columns(float *v, uint32_t at) {
  uint32_t *u = reinterpret_cast<uint32_t *>(v);
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]),
                 "=r"(u[6]), "=r"(u[7])
               : "r"(at));
}

// HALF: most columns that an epilogue warp keeps.
template <typename O, int HALF>
__global__ void __launch_bounds__(kProductThreads, 1)
    product_kernel(const __grid_constant__ CUtensorMap head_map,
                   const __grid_constant__ CUtensorMap token_map, const uint8_t *head_scales,
                   const uint8_t *token_scales, O *out, int64_t out_stride, ProductShape sh,
                   int32_t *status) {
  extern __shared__ unsigned char smem_raw[];
  __shared__ __align__(8) uint64_t full_bar[kMaxStages], empty_bar[kMaxStages], done_bar, free_bar;
  __shared__ uint32_t tmem_base;
  __shared__ volatile int dead;  // a wait gave up
  const int tid = threadIdx.x, lane = tid & 31, wid = __shfl_sync(kFull, tid >> 5, 0);
  const uint32_t smem = (smem_addr(smem_raw) + 1023u) & ~1023u;
  const uint32_t token_bytes = (uint32_t)sh.box * kStageBytes;
  const int row_tiles = (sh.box + kMxTileRows - 1) / kMxTileRows;
  const uint32_t at_tokens = kHeadRows * kStageBytes, at_head_scales = at_tokens + token_bytes;
  const uint32_t at_token_scales = at_head_scales + 2 * kMxTileBytes;
  const uint32_t stage_bytes = at_token_scales + (uint32_t)row_tiles * 2 * kMxTileBytes;
  const int per_tile = (sh.steps + 3) / 4;  // stages of a tile

  if (wid == 0) {
    if (lane == 0) {
      asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&head_map)) : "memory");
      asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&token_map)) : "memory");
    }
  } else if (wid == 1) {
    if (lane == 0) {
      for (int i = 0; i < sh.stages; ++i) {
        tma::mbar_init(smem_addr(&full_bar[i]), 2);  // the head's side, the tokens'
        tma::mbar_init(smem_addr(&empty_bar[i]), 1);
      }
      tma::mbar_init(smem_addr(&done_bar), 1);
      tma::mbar_init(smem_addr(&free_bar), kEpilogueWarps);
      dead = 0;
      tma::fence_mbar_init();
      tma::fence_proxy_async();
    }
  } else if (wid == 3) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_addr(&tmem_base)),
                 "n"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  }
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = tmem_base;
  // A warp's wait: until another gave up, or for its own share.
  auto wait = [&](uint64_t *bar, uint32_t parity) {
    const uint32_t b = smem_addr(bar);
    for (uint32_t i = 0; i < kTries; ++i) {
      if (__all_sync(kFull, mbar_try_wait(b, parity))) return true;
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
    int tile = (int)blockIdx.x, kb = 0, stage = 0;
    uint32_t lap = 0;
    bool ok = true;
    int mt = tile / sh.token_tiles, nt = tile - mt * sh.token_tiles;
    while (tile < sh.tiles) {
      if (lap > 0) {
        ok = wait(&empty_bar[stage], (lap - 1) & 1);
        if (!ok) break;
      }
      const uint32_t bar = smem_addr(&full_bar[stage]), s = smem + stage * stage_bytes;
      const uint32_t bytes = (uint32_t)min(2, sh.groups - 2 * kb) * kMxTileBytes;
      if (elected()) {
        if (wid == 0) {
          tma::arrive_expect(bar, at_tokens + bytes);
          load_2d(s, &head_map, kb * kStageBytes, mt * kHeadRows, bar);
          load_bulk(s + at_head_scales,
                    head_scales + ((int64_t)mt * sh.groups + 2 * kb) * kMxTileBytes, bytes, bar);
        } else {
          const int first = nt * (kMostTokens / kMxTileRows);
          const bool two = row_tiles > 1 && (first + 1) * kMxTileRows < sh.tokens;
          tma::arrive_expect(bar, token_bytes + (two ? 2 * bytes : bytes));
          load_2d(s + at_tokens, &token_map, kb * kStageBytes, nt * kMostTokens, bar);
          const uint8_t *scales = token_scales + ((int64_t)first * sh.groups + 2 * kb) * kMxTileBytes;
          load_bulk(s + at_token_scales, scales, bytes, bar);
          if (two)
            load_bulk(s + at_token_scales + 2 * kMxTileBytes,
                      scales + (int64_t)sh.groups * kMxTileBytes, bytes, bar);
        }
      }
      __syncwarp();
      if (++stage == sh.stages) {
        stage = 0;
        ++lap;
      }
      if (++kb == per_tile) {
        kb = 0;
        tile += (int)gridDim.x;
        mt = tile / sh.token_tiles;
        nt = tile - mt * sh.token_tiles;
      }
    }
    if (!ok) {
      // copies in flight write to this block's memory: they end first (as far as both
      // warps have issued theirs)
      for (int i = 0; i < sh.stages; ++i)
        tma::wait_bounded(smem_addr(&full_bar[i]), (i < stage ? lap : lap - 1) & 1, 1u << 18);
    }
  } else if (wid == 1) {
    // ----------------------------------------------------- the products --
    int stage = 0, n_tile = 0;
    uint32_t lap = 0, odd = 0;
    bool ok = true;
    for (int tile = (int)blockIdx.x; tile < sh.tiles; tile += (int)gridDim.x, ++n_tile) {
      const int left = sh.tokens - tile % sh.token_tiles * kMostTokens;
      const int width = min(sh.box, (left + 15) & ~15);
      const uint32_t idesc0 = instruction(width, 0), idesc2 = instruction(width, 2);
      ok = n_tile == 0 || wait(&free_bar, (uint32_t)(n_tile - 1) & 1);
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
                copy_scales(sf + 4 * g, fa + 32 * g);
                copy_scales(sf + 8 + 8 * g, fb + 32 * g);
                if (width > kMxTileRows) copy_scales(sf + 12 + 8 * g, fb + 64 + 32 * g);
              }
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (j < steps)
                multiply(tmem, a + 2 * j, b + 2 * j, j & 1 ? idesc2 : idesc0, sf + 4 * (j >> 1),
                         sf + 8 + 8 * (j >> 1), j > 0 || kb > 0);
          };
          if (steps == 4) work(2, 4);
          else work(groups, steps);
          commit(smem_addr(&empty_bar[stage]));
          if (kb == per_tile - 1) commit(smem_addr(&done_bar));
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
      // products in flight: a last commit follows them
      if (elected()) commit(smem_addr(&done_bar));
      tma::wait_bounded(smem_addr(&done_bar), (uint32_t)n_tile & 1, 1u << 21);
    }
  } else if (wid >= 4) {
    // --------------------------------------------------- the accumulators --
    const int quarter = wid & 3, half = (wid - 4) >> 2;
    int n_tile = 0;
    for (int tile = (int)blockIdx.x; tile < sh.tiles; tile += (int)gridDim.x, ++n_tile) {
      const int mt = tile / sh.token_tiles, n0 = tile % sh.token_tiles * kMostTokens;
      const int left = sh.tokens - n0, width = min(sh.box, (left + 15) & ~15);
      const int c0 = half * (width / 2);
      const int count = min(width / 2, left - c0);  // columns of this warp that are tokens
      if (!wait(&done_bar, (uint32_t)n_tile & 1)) break;
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      float v[HALF];
#pragma unroll
      for (int i = 0; i < HALF; i += 8)
        if (i < count) load_columns(v + i, tmem + ((uint32_t)quarter << 21) + c0 + i);
      asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
      // (nothing is computed from the registers before that)
#pragma unroll
      for (int i = 0; i < HALF; ++i) asm volatile("" : "+f"(v[i]));
      asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
      __syncwarp();
      if (lane == 0) arrive(smem_addr(&free_bar));
      const int row = mt * kHeadRows + quarter * 32 + lane;
      if (row < sh.head_rows) {
        O *o = out + (int64_t)(n0 + c0) * out_stride + row;
#pragma unroll
        for (int i = 0; i < HALF; ++i)
          if (i < count) o[i * out_stride] = float_logit<O>(v[i]);
      }
    }
  }
  __syncwarp();
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  if (wid == 3) {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "n"(kTmemCols));
  }
}

template <typename O, int HALF>
int launch_t(const CUtensorMap &hm, const CUtensorMap &tm, const rans_mxfp4 &a,
             const rans_mxfp4 &w, void *out, int64_t stride, const ProductShape &sh,
             uint32_t smem, int32_t *status, int sms, cudaStream_t st) {
  auto kern = product_kernel<O, HALF>;
  if (ensure_dyn_smem((const void *)kern, smem) != cudaSuccess) return RANS_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(sh.tiles < sms ? sh.tiles : sms));
  cfg.blockDim = dim3(kProductThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = sh.wait ? 1 : 0;
  const cudaError_t e =
      cudaLaunchKernelEx(&cfg, kern, hm, tm, (const uint8_t *)w.scales, (const uint8_t *)a.scales,
                         static_cast<O *>(out), stride, sh, status);
  return e == cudaSuccess ? RANS_OK : RANS_ERR_CUDA;
}

template <typename O>
int launch_o(const CUtensorMap &hm, const CUtensorMap &tm, const rans_mxfp4 &a,
             const rans_mxfp4 &w, void *out, int64_t stride, const ProductShape &sh,
             uint32_t smem, int32_t *status, int sms, cudaStream_t st) {
  if (sh.box <= 32) return launch_t<O, 16>(hm, tm, a, w, out, stride, sh, smem, status, sms, st);
  if (sh.box <= 128) return launch_t<O, 64>(hm, tm, a, w, out, stride, sh, smem, status, sms, st);
  return launch_t<O, 128>(hm, tm, a, w, out, stride, sh, smem, status, sms, st);
}

}  // namespace

int launch_mxfp4_product(const rans_mxfp4 &a, const rans_mxfp4 &w, void *out, int dtype,
                         int64_t stride, int32_t *status, bool follows, cudaStream_t st) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return RANS_ERR_CUDA;
  ProductShape sh;
  sh.tokens = (int32_t)a.rows;
  sh.head_rows = (int32_t)w.rows;
  sh.box = a.rows >= kMostTokens ? kMostTokens : (int32_t)((a.rows + 15) & ~15);
  sh.token_tiles = (sh.tokens + kMostTokens - 1) / kMostTokens;
  const int64_t tiles = (int64_t)sh.token_tiles * ((w.rows + kHeadRows - 1) / kHeadRows);
  sh.steps = (int32_t)((w.cols + kStepCols - 1) / kStepCols);
  sh.groups = mx_groups(w.cols);
  // a block's stages are counted in 31 bits
  if (tiles * ((sh.steps + 3) / 4) > 0x3fffffff) return RANS_ERR_ARG;
  sh.tiles = (int32_t)tiles;
  sh.wait = follows ? 1 : 0;
  const uint32_t stage = kHeadRows * kStageBytes + (uint32_t)sh.box * kStageBytes +
                         2 * kMxTileBytes * (1 + (uint32_t)(sh.box + kMxTileRows - 1) / kMxTileRows);
  const uint32_t room = (uint32_t)smem_optin(dev) - 2048;  // its static part, alignment
  sh.stages = (int32_t)(room / stage < (uint32_t)kMaxStages ? room / stage : kMaxStages);
  if (sh.stages < 2) return RANS_ERR_CUDA;
  CUtensorMap hm, tm;
  const uint64_t row = (uint64_t)mx_row_bytes(w.cols);
  int e = encode_rows_map(&hm, w.codes, row, (uint64_t)w.rows, kStageBytes, kHeadRows);
  if (!e) e = encode_rows_map(&tm, a.codes, row, (uint64_t)a.rows, kStageBytes, (uint32_t)sh.box);
  if (e) return e;
  const uint32_t smem = stage * (uint32_t)sh.stages + 1024;
  const int sms = num_sms(dev);
  switch (dtype) {
    case RANS_LOGITS_F32:
      return launch_o<float>(hm, tm, a, w, out, stride, sh, smem, status, sms, st);
    case RANS_LOGITS_F16:
      return launch_o<__half>(hm, tm, a, w, out, stride, sh, smem, status, sms, st);
    default:
      return launch_o<__nv_bfloat16>(hm, tm, a, w, out, stride, sh, smem, status, sms, st);
  }
}

}  // namespace rb
