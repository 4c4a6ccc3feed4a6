// api.cu -- the extern "C" entry points of librans_b200: argument checks,
// chunking geometry, workspace layout and launch order.  Every coding step
// runs in the kernels of tables.cu, encode.cu and decode.cu; logits.cu,
// tokens.cu and distill.cu hold those of tokens under a model's logits.
#include <cstring>
#include <mutex>
#include <utility>
#include <vector>

#include <nvtx3/nvToolsExt.h>

#include "rans_common.cuh"
#include "rans_internal.h"

#define RANS_API extern "C" __attribute__((visibility("default")))

namespace rb {

int num_sms(int device) {
  static int cache[128] = {0};
  if (device < 0 || device >= 128) return 1;
  if (cache[device] == 0) {
    int v = 0;
    cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, device);
    cache[device] = v > 0 ? v : 1;
  }
  return cache[device];
}

int smem_optin(int device) {
  static int cache[128] = {0};
  if (device < 0 || device >= 128) return 0;
  if (cache[device] == 0) {
    int v = 0;
    cudaDeviceGetAttribute(&v, cudaDevAttrMaxSharedMemoryPerBlockOptin, device);
    cache[device] = v;
  }
  return cache[device];
}

// Launch set-up answers cached per (kernel, device): the dynamic shared
// memory limit already set, and resident blocks per SM for a (threads,
// shared memory) pair, so a coding call repeats no runtime query.
namespace {
struct SmemEntry {
  const void *fn;
  int dev;
  uint32_t bytes;
};
struct OccEntry {
  const void *fn;
  int dev, threads;
  uint32_t smem;
  int blocks;
};
std::mutex g_launch_mutex;
std::vector<SmemEntry> g_smem_set;
std::vector<OccEntry> g_occ;
std::vector<std::pair<const void *, int>> g_cluster_set;
}  // namespace

cudaError_t ensure_dyn_smem(const void *fn, uint32_t bytes) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lock(g_launch_mutex);
  for (SmemEntry &x : g_smem_set)
    if (x.fn == fn && x.dev == dev) {
      if (x.bytes >= bytes) return cudaSuccess;
      e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
      if (e == cudaSuccess) x.bytes = bytes;
      return e;
    }
  e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e == cudaSuccess) g_smem_set.push_back({fn, dev, bytes});
  return e;
}

cudaError_t ensure_cluster(const void *fn) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lock(g_launch_mutex);
  for (const auto &x : g_cluster_set)
    if (x.first == fn && x.second == dev) return cudaSuccess;
  e = cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess) {
    try {
      g_cluster_set.push_back({fn, dev});
    } catch (...) {  // no memory to remember it: set again next time
    }
  }
  return e;
}

cudaError_t blocks_per_sm(int *out, const void *fn, int threads, uint32_t smem) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lock(g_launch_mutex);
  for (const OccEntry &x : g_occ)
    if (x.fn == fn && x.dev == dev && x.threads == threads && x.smem == smem) {
      *out = x.blocks;
      return cudaSuccess;
    }
  e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(out, fn, threads, (size_t)smem);
  if (e == cudaSuccess && g_occ.size() < 4096) g_occ.push_back({fn, dev, threads, smem, *out});
  return e;
}

}  // namespace rb

namespace {

using rb::Geom;

// An NVTX range around an entry point, so that traces show the library's
// calls (no cost beyond a call when no tool is attached).
struct NvtxRange {
  explicit NvtxRange(const char *name) { nvtxRangePushA(name); }
  ~NvtxRange() { nvtxRangePop(); }
};

constexpr uint64_t kWsHeader = 256;

uint64_t align256(uint64_t v) { return (v + 255) & ~uint64_t(255); }

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

bool is_pow2(int64_t v) { return v > 0 && (v & (v - 1)) == 0; }

int make_geom(const rans_chunking *ch, int64_t n, Geom &g) {
  if (ch == nullptr || n < 0) return RANS_ERR_ARG;
  if (ch->interleave != 1 && ch->interleave != 2 && ch->interleave != 4 && ch->interleave != 8 &&
      ch->interleave != 32)
    return RANS_ERR_ARG;
  if (!is_pow2(ch->index_block)) return RANS_ERR_ARG;
  const int base_fmt = ch->format & ~RANS_FMT_ALIAS;
  const bool alias = (ch->format & RANS_FMT_ALIAS) != 0;
  if (base_fmt != RANS_FMT_RANS64 && base_fmt != RANS_FMT_RANS32_16) return RANS_ERR_ARG;
  if (alias && ch->interleave == 32) return RANS_ERR_ARG;  // no 32-way alias coder
  std::memset(&g, 0, sizeof(g));
  g.kind = ch->kind;
  g.fmt = base_fmt;
  g.alias = alias ? 1 : 0;
  g.W = ch->interleave;
  g.n = n;
  int ib = 0;
  while ((int64_t(1) << ib) < ch->index_block) ++ib;
  g.ib_shift = ib;
  g.slot_extra = 16ull * (uint64_t)g.W + 16ull;
  int64_t max_n = 0;
  switch (ch->kind) {
    case RANS_CHUNK_CONTIG:
      if (ch->n_streams < 1) return RANS_ERR_ARG;
      g.S = ch->n_streams;
      g.per = cdiv(n, g.S);
      max_n = g.per;
      if (g.per >= (int64_t(1) << 31) - 64) return RANS_ERR_ARG;
      break;
    case RANS_CHUNK_EXPLICIT:
      if (ch->n_streams < 0 || (ch->n_streams > 0 && ch->stream_starts == nullptr))
        return RANS_ERR_ARG;
      g.S = ch->n_streams;
      g.starts = ch->stream_starts;
      break;
    case RANS_CHUNK_TILED: {
      const int64_t B = ch->shape[0], C = ch->shape[1], H = ch->shape[2], W = ch->shape[3];
      if (B < 0 || C < 1 || H < 1 || W < 1) return RANS_ERR_ARG;
      if (ch->group < 1 || ch->tile_h < 1 || ch->tile_w < 1) return RANS_ERR_ARG;
      if (B * C * H * W != n) return RANS_ERR_ARG;
      g.C = C;
      g.H = H;
      g.Wd = W;
      g.cg = ch->group;
      g.th = ch->tile_h;
      g.tw = ch->tile_w;
      g.ng = cdiv(C, g.cg);
      g.nty = cdiv(H, g.th);
      g.ntx = cdiv(W, g.tw);
      g.S = B * g.ng * g.nty * g.ntx;
      max_n = (g.cg < C ? g.cg : C) * (g.th < H ? g.th : H) * (g.tw < W ? g.tw : W);
      if (C * H * W >= (int64_t(1) << 31) - 64) return RANS_ERR_ARG;
      {
        // tile classes (last group?, last tile row?, last tile column?), largest first
        const int64_t full[3] = {C % g.cg ? g.ng - 1 : g.ng, H % g.th ? g.nty - 1 : g.nty,
                                 W % g.tw ? g.ntx - 1 : g.ntx};
        const int64_t part[3] = {C % g.cg ? 1 : 0, H % g.th ? 1 : 0, W % g.tw ? 1 : 0};
        const int64_t fsz[3] = {g.cg, g.th, g.tw};
        const int64_t psz[3] = {C % g.cg, H % g.th, W % g.tw};
        int64_t size[8], count[8];
        int bits[8], nc = 0;
        for (int b = 0; b < 8; ++b) {
          int64_t cnt = B, sz = 1;
          for (int d = 0; d < 3; ++d) {
            cnt *= (b >> d & 1) ? part[d] : full[d];
            sz *= (b >> d & 1) ? psz[d] : fsz[d];
          }
          if (cnt == 0) continue;
          int at = nc++;
          while (at > 0 && size[at - 1] < sz) {  // stable insertion, larger first
            size[at] = size[at - 1];
            count[at] = count[at - 1];
            bits[at] = bits[at - 1];
            --at;
          }
          size[at] = sz;
          count[at] = cnt;
          bits[at] = b;
        }
        g.nclass = nc;
        int64_t run = 0;
        for (int i = 0; i < nc; ++i) {
          g.cls_start[i] = run;
          g.cls_bits[i] = bits[i];
          run += count[i];
        }
        if (run != g.S) return RANS_ERR_ARG;
      }
      break;
    }
    default:
      return RANS_ERR_ARG;
  }
  g.slot_bytes = rb::pad16(8ull * (uint64_t)max_n + g.slot_extra);
  return RANS_OK;
}

uint64_t lens_bytes(const Geom &g) { return align256(8ull * (uint64_t)g.S); }

uint64_t scratch_bytes(const Geom &g) {
  if (g.kind == RANS_CHUNK_EXPLICIT) return align256(8ull * (uint64_t)g.n + g.slot_extra * g.S);
  return align256(g.slot_bytes * (uint64_t)g.S);
}

uint64_t enc_ws_bytes(const Geom &g) { return kWsHeader + lens_bytes(g) + scratch_bytes(g); }

bool tables_usable(const rans_tables *t) {
  if (t == nullptr || t->blob == nullptr || t->K < 1) return false;
  if (t->precision < 1 || t->precision > 16) return false;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev != t->device) return false;
  return true;
}

// RANS64 codes rows of precision 16, RANS32_16 rows of precision <= 15;
// alias coding needs the alias tables.
bool format_fits(const Geom &g, const rans_tables *t) {
  if (g.alias && t->alias == nullptr) return false;
  return g.fmt == RANS_FMT_RANS64 ? t->precision == 16 : t->precision <= 15;
}

// Bytes of the format's stream word.
uint64_t word_bytes(const Geom &g) { return g.fmt == RANS_FMT_RANS32_16 ? 2 : 4; }

cudaStream_t as_stream(void *s) { return static_cast<cudaStream_t>(s); }

}  // namespace

RANS_API const char *rans_status_string(int status) {
  switch (status) {
    case RANS_OK: return "ok";
    case RANS_ERR_ARG: return "invalid argument";
    case RANS_ERR_INDEX: return "index, token or stream id out of range, or named twice";
    case RANS_ERR_ZERO_FREQ: return "symbol or token maps to a bucket of width 0";
    case RANS_ERR_RANGE: return "value out of range (escape raw value, interval, logit)";
    case RANS_ERR_CAPACITY: return "buffer too small";
    case RANS_ERR_CORRUPT: return "stream truncated, too long or inconsistent";
    case RANS_ERR_CUDA: return "CUDA runtime call failed";
    case RANS_ERR_TABLE: return "malformed CDF row or pmf";
    case RANS_ERR_TIMEOUT: return "bounded device wait gave up";
    default: return "unknown status";
  }
}

RANS_API int rans_version(void) { return 200; }

RANS_API int rans_gaussian_lengths(const float *scales, int32_t K, double tail_mass,
                                   int32_t *cdf_lengths, int32_t *offsets, void *stream) {
  if (K < 1 || !scales || !cdf_lengths || !offsets) return RANS_ERR_ARG;
  if (!(tail_mass > 0.0) || !(tail_mass < 1.0)) return RANS_ERR_ARG;
  return rb::launch_gaussian_lengths(scales, K, tail_mass, cdf_lengths, offsets,
                                     as_stream(stream));
}

RANS_API int rans_build_cdfs_from_scales(const float *scales, int32_t K, double tail_mass,
                                         int32_t precision, int32_t *cdfs, int32_t Lmax,
                                         int32_t *cdf_lengths, int32_t *offsets, void *stream) {
  NvtxRange nvtx_("rans_build_cdfs_from_scales");
  if (K < 1 || Lmax < 3 || !scales || !cdfs || !cdf_lengths || !offsets) return RANS_ERR_ARG;
  if (!(tail_mass > 0.0) || !(tail_mass < 1.0)) return RANS_ERR_ARG;
  if (precision < 1 || precision > 16) return RANS_ERR_ARG;
  return rb::launch_gaussian_rows(scales, K, tail_mass, precision, cdfs, Lmax, cdf_lengths,
                                  offsets, as_stream(stream));
}

RANS_API int rans_build_cdfs_from_pmfs(const float *pmfs, int32_t K, int32_t pmf_stride,
                                       const int32_t *pmf_lengths, const float *tail_mass,
                                       int32_t precision, int32_t *cdfs, int32_t Lmax,
                                       int32_t *cdf_lengths, void *stream) {
  NvtxRange nvtx_("rans_build_cdfs_from_pmfs");
  if (K < 1 || pmf_stride < 1 || Lmax < 2 || !pmfs || !pmf_lengths || !tail_mass || !cdfs ||
      !cdf_lengths)
    return RANS_ERR_ARG;
  if (precision < 1 || precision > 16) return RANS_ERR_ARG;
  return rb::launch_pmf_rows(pmfs, K, pmf_stride, pmf_lengths, tail_mass, precision, cdfs,
                             Lmax, cdf_lengths, as_stream(stream));
}

RANS_API uint64_t rans_tables_bytes(int32_t K, int32_t Lmax) {
  return rb::tables_bytes_bound(K, Lmax);
}

RANS_API int rans_tables_prepare(const int32_t *cdfs, int32_t K, int32_t Lmax,
                                 const int32_t *cdf_lengths, const int32_t *offsets,
                                 int32_t precision, void *blob, uint64_t blob_bytes,
                                 rans_tables *out, void *stream) {
  NvtxRange nvtx_("rans_tables_prepare");
  if (K < 1 || Lmax < 2 || Lmax > 65537 || !cdfs || !cdf_lengths || !offsets || !blob || !out)
    return RANS_ERR_ARG;
  if (precision < 1 || precision > 16) return RANS_ERR_ARG;
  return rb::prepare_tables(cdfs, K, Lmax, cdf_lengths, offsets, precision, blob, blob_bytes,
                            out, as_stream(stream));
}

RANS_API int rans_tables_refresh(const int32_t *cdfs, int32_t K, int32_t Lmax,
                                 const int32_t *cdf_lengths, const int32_t *offsets,
                                 const rans_tables *tables, void *stream) {
  NvtxRange nvtx_("rans_tables_refresh");
  if (!tables_usable(tables) || K != tables->K || Lmax < 2 || !cdfs || !cdf_lengths || !offsets)
    return RANS_ERR_ARG;
  return rb::refresh_tables(cdfs, K, Lmax, cdf_lengths, offsets, *tables, as_stream(stream));
}

RANS_API int rans_tables_refresh_from_scales(const float *scales, int32_t K, double tail_mass,
                                             int32_t *cdfs, int32_t Lmax, int32_t *cdf_lengths,
                                             int32_t *offsets, const rans_tables *tables,
                                             void *stream) {
  NvtxRange nvtx_("rans_tables_refresh_from_scales");
  if (!tables_usable(tables) || K != tables->K || Lmax < 3 || !scales || !cdfs ||
      !cdf_lengths || !offsets)
    return RANS_ERR_ARG;
  if (!(tail_mass > 0.0) || !(tail_mass < 1.0)) return RANS_ERR_ARG;
  return rb::refresh_tables_from_scales(scales, K, tail_mass, cdfs, Lmax, cdf_lengths, offsets,
                                        *tables, as_stream(stream));
}

RANS_API uint64_t rans_alias_bytes(const rans_tables *tables) {
  if (!tables || tables->K < 1 || tables->precision < 1 || tables->precision > 16) return 0;
  return ((8ull * (uint64_t)tables->n_buckets + 255) & ~255ull) +
         2ull * (uint64_t)tables->K * (1ull << tables->precision);
}

RANS_API int rans_alias_prepare(const int32_t *cdfs, int32_t K, int32_t Lmax,
                                const int32_t *cdf_lengths, rans_tables *tables, void *alias,
                                uint64_t alias_bytes, void *stream) {
  NvtxRange nvtx_("rans_alias_prepare");
  if (!tables_usable(tables) || K != tables->K || Lmax < 2 || !cdfs || !cdf_lengths || !alias)
    return RANS_ERR_ARG;
  return rb::prepare_alias(cdfs, K, Lmax, cdf_lengths, *tables, alias, alias_bytes,
                           as_stream(stream));
}

RANS_API int64_t rans_num_streams(const rans_chunking *chunking, int64_t n) {
  Geom g;
  int st = make_geom(chunking, n, g);
  return st ? st : g.S;
}

RANS_API uint64_t rans_encode_workspace_bytes(const rans_chunking *chunking, int64_t n) {
  Geom g;
  if (make_geom(chunking, n, g)) return 0;
  return enc_ws_bytes(g);
}

RANS_API uint64_t rans_decode_workspace_bytes(const rans_chunking *chunking, int64_t n) {
  Geom g;
  if (make_geom(chunking, n, g)) return 0;
  return kWsHeader;
}

RANS_API uint64_t rans_max_compressed_bytes(const rans_chunking *chunking, int64_t n) {
  Geom g;
  if (make_geom(chunking, n, g)) return 0;
  return 8ull * (uint64_t)n + g.slot_extra * (uint64_t)g.S;
}

RANS_API int rans_encode_with_indexes(const void *symbols, int32_t sym_dtype,
                                      const int32_t *indexes, int64_t n,
                                      const rans_tables *tables, const rans_chunking *chunking,
                                      uint8_t *out, uint64_t out_capacity,
                                      uint64_t *stream_offsets, void *workspace,
                                      uint64_t workspace_bytes, void *stream) {
  NvtxRange nvtx_("rans_encode_with_indexes");
  if (!tables_usable(tables)) return RANS_ERR_ARG;
  if (n > 0 && (!symbols || !indexes)) return RANS_ERR_ARG;
  if (!stream_offsets || !workspace || (out_capacity > 0 && !out)) return RANS_ERR_ARG;
  if (sym_dtype != RANS_SYM_INT32 && sym_dtype != RANS_SYM_UINT8 && sym_dtype != RANS_SYM_INT16)
    return RANS_ERR_ARG;
  if ((reinterpret_cast<uintptr_t>(workspace) & 255) != 0) return RANS_ERR_ARG;
  Geom g;
  int st = make_geom(chunking, n, g);
  if (st) return st;
  if (!format_fits(g, tables)) return RANS_ERR_ARG;
  if (workspace_bytes < enc_ws_bytes(g)) return RANS_ERR_CAPACITY;
  cudaStream_t s = as_stream(stream);
  char *ws = reinterpret_cast<char *>(workspace);
  int32_t *status = reinterpret_cast<int32_t *>(ws);
  uint64_t *lens = reinterpret_cast<uint64_t *>(ws + kWsHeader);
  char *scratch = ws + kWsHeader + lens_bytes(g);
  if (cudaMemsetAsync(ws, 0, kWsHeader + 8ull * (uint64_t)g.S, s) != cudaSuccess)
    return RANS_ERR_CUDA;
  if (g.S > 0) {
    st = rb::launch_encode(symbols, sym_dtype, indexes, *tables, g, scratch, lens, status, s);
    if (st) return st;
  }
  return rb::launch_compact(g, scratch, lens, out, out_capacity, stream_offsets, status, s);
}

RANS_API int rans_decode_with_indexes(const uint8_t *in, uint64_t in_bytes,
                                      const uint64_t *stream_offsets, const int32_t *indexes,
                                      int64_t n, const rans_tables *tables,
                                      const rans_chunking *chunking, void *symbols_out,
                                      int32_t sym_dtype, void *workspace,
                                      uint64_t workspace_bytes, void *stream) {
  NvtxRange nvtx_("rans_decode_with_indexes");
  if (!tables_usable(tables)) return RANS_ERR_ARG;
  if (n > 0 && (!symbols_out || !indexes)) return RANS_ERR_ARG;
  if (!stream_offsets || !workspace || (in_bytes > 0 && !in)) return RANS_ERR_ARG;
  if (sym_dtype != RANS_SYM_INT32 && sym_dtype != RANS_SYM_UINT8 && sym_dtype != RANS_SYM_INT16)
    return RANS_ERR_ARG;
  if ((reinterpret_cast<uintptr_t>(workspace) & 255) != 0) return RANS_ERR_ARG;
  Geom g;
  int st = make_geom(chunking, n, g);
  if (st) return st;
  if (!format_fits(g, tables)) return RANS_ERR_ARG;
  if ((reinterpret_cast<uintptr_t>(in) & (word_bytes(g) - 1)) != 0) return RANS_ERR_ARG;
  if (workspace_bytes < kWsHeader) return RANS_ERR_CAPACITY;
  cudaStream_t s = as_stream(stream);
  int32_t *status = reinterpret_cast<int32_t *>(workspace);
  if (cudaMemsetAsync(workspace, 0, kWsHeader, s) != cudaSuccess) return RANS_ERR_CUDA;
  if (g.S == 0) return RANS_OK;
  return rb::launch_decode(in, in_bytes, stream_offsets, indexes, *tables, g, symbols_out,
                           sym_dtype, status, s);
}

// ---- float latents ------------------------------------------------------

RANS_API int rans_build_indexes(const float *scales, int64_t n, const float *scale_table,
                                int32_t K, float scale_bound, int32_t *indexes, void *stream) {
  NvtxRange nvtx_("rans_build_indexes");
  if (n < 0 || K < 1 || (n > 0 && (!scales || !scale_table || !indexes))) return RANS_ERR_ARG;
  return rb::launch_build_indexes(scales, n, scale_table, K, scale_bound, indexes,
                                  as_stream(stream));
}

// The float entry points take one scale per element (index_block 1) and a
// scale table with one entry per table row.
static int float_args(const rans_tables *tables, const rans_chunking *chunking,
                      int32_t table_len) {
  if (!tables_usable(tables) || !chunking) return RANS_ERR_ARG;
  if (table_len != tables->K || chunking->index_block != 1) return RANS_ERR_ARG;
  if (chunking->format != RANS_FMT_RANS64 || tables->precision != 16) return RANS_ERR_ARG;
  if (chunking->interleave != 1 && chunking->interleave != 32) return RANS_ERR_ARG;
  return RANS_OK;
}

RANS_API int rans_encode_from_scales(const float *y, const float *means, const float *scales,
                                     int64_t n, const float *scale_table, int32_t table_len,
                                     float scale_bound, const rans_tables *tables,
                                     const rans_chunking *chunking, uint8_t *out,
                                     uint64_t out_capacity, uint64_t *stream_offsets,
                                     void *workspace, uint64_t workspace_bytes, void *stream) {
  NvtxRange nvtx_("rans_encode_from_scales");
  int st = float_args(tables, chunking, table_len);
  if (st) return st;
  if (n > 0 && (!y || !scales || !scale_table)) return RANS_ERR_ARG;
  if (!stream_offsets || !workspace || (out_capacity > 0 && !out)) return RANS_ERR_ARG;
  if ((reinterpret_cast<uintptr_t>(workspace) & 255) != 0) return RANS_ERR_ARG;
  Geom g;
  st = make_geom(chunking, n, g);
  if (st) return st;
  if (workspace_bytes < enc_ws_bytes(g)) return RANS_ERR_CAPACITY;
  cudaStream_t s = as_stream(stream);
  char *ws = reinterpret_cast<char *>(workspace);
  int32_t *status = reinterpret_cast<int32_t *>(ws);
  uint64_t *lens = reinterpret_cast<uint64_t *>(ws + kWsHeader);
  char *scratch = ws + kWsHeader + lens_bytes(g);
  if (cudaMemsetAsync(ws, 0, kWsHeader + 8ull * (uint64_t)g.S, s) != cudaSuccess)
    return RANS_ERR_CUDA;
  if (g.S > 0) {
    st = rb::launch_encode_float(y, means, scales, scale_table, scale_bound, *tables, g,
                                 scratch, lens, status, s);
    if (st) return st;
  }
  return rb::launch_compact(g, scratch, lens, out, out_capacity, stream_offsets, status, s);
}

RANS_API int rans_decode_to_values(const uint8_t *in, uint64_t in_bytes,
                                   const uint64_t *stream_offsets, const float *scales,
                                   const float *means, int64_t n, const float *scale_table,
                                   int32_t table_len, float scale_bound,
                                   const rans_tables *tables, const rans_chunking *chunking,
                                   float *values, void *workspace, uint64_t workspace_bytes,
                                   void *stream) {
  NvtxRange nvtx_("rans_decode_to_values");
  int st = float_args(tables, chunking, table_len);
  if (st) return st;
  if (n > 0 && (!values || !scales || !scale_table)) return RANS_ERR_ARG;
  if (!stream_offsets || !workspace || (in_bytes > 0 && !in)) return RANS_ERR_ARG;
  if ((reinterpret_cast<uintptr_t>(workspace) & 255) != 0) return RANS_ERR_ARG;
  if ((reinterpret_cast<uintptr_t>(in) & 3) != 0) return RANS_ERR_ARG;
  Geom g;
  st = make_geom(chunking, n, g);
  if (st) return st;
  if (workspace_bytes < kWsHeader) return RANS_ERR_CAPACITY;
  cudaStream_t s = as_stream(stream);
  int32_t *status = reinterpret_cast<int32_t *>(workspace);
  if (cudaMemsetAsync(workspace, 0, kWsHeader, s) != cudaSuccess) return RANS_ERR_CUDA;
  if (g.S == 0) return RANS_OK;
  return rb::launch_decode_float(in, in_bytes, stream_offsets, scales, means, scale_table,
                                 scale_bound, *tables, g, values, status, s);
}

// ---- tokens under a model's logits --------------------------------------

namespace {

// Bytes per element of a logits type, 0 for none.
int logits_bytes(int32_t dtype) {
  return dtype == RANS_LOGITS_F32 ? 4 : dtype == RANS_LOGITS_F16 || dtype == RANS_LOGITS_BF16 ? 2
                                                                                             : 0;
}

bool aligned_to(const void *p, uint64_t bytes) {
  return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0;
}

// Whether all of these lie as their type has to (an absent one does): a kernel's
// access to one that does not would end the caller's context.
template <typename... T>
bool natural(const T *...p) {
  return (aligned_to(p, sizeof(T)) && ...);
}

int check_logits(const rans_logits *in) {
  if (!in || in->rows < 0 || in->vocab < 1 || in->vocab > RANS_MAX_VOCAB) return RANS_ERR_ARG;
  const int e = logits_bytes(in->dtype);
  if (e == 0) return RANS_ERR_ARG;
  if (in->rows > 1 && in->row_stride < in->vocab) return RANS_ERR_ARG;
  if (in->rows > 0 && (!in->data || !aligned_to(in->data, (uint64_t)e))) return RANS_ERR_ARG;
  return RANS_OK;
}

bool finite(float x) { return x - x == 0.0f; }

// The adjustment of a call in `out`: the caller's, checked, or a neutral one.
int check_adjust(const rans_adjust *a, int32_t vocab, rans_adjust &out) {
  if (!a) {
    std::memset(&out, 0, sizeof(out));
    out.repetition = 1.0f;
    out.inv_temperature = 1.0f;
    return RANS_OK;
  }
  out = *a;
  if (!a->params &&
      (!(a->repetition > 0.0f) || !finite(a->repetition) || !(a->inv_temperature > 0.0f) ||
       !finite(a->inv_temperature) || !finite(a->frequency) || !finite(a->presence)))
    return RANS_ERR_ARG;
  if (a->history && (!a->history_begin || !a->history_end || a->history_len < 0))
    return RANS_ERR_ARG;
  if (a->bias_ids && (!a->bias_values || !a->bias_begin || !a->bias_end || a->bias_len < 0))
    return RANS_ERR_ARG;
  if (a->mask && a->mask_stride != 0 && a->mask_stride < (vocab + 31) / 32) return RANS_ERR_ARG;
  if (!natural(a->params, a->history, a->history_begin, a->history_end, a->bias_ids,
               a->bias_values, a->bias_begin, a->bias_end, a->mask))
    return RANS_ERR_ARG;
  return RANS_OK;
}

int check_status_word(const void *status) {
  return status && aligned_to(status, 256) ? RANS_OK : RANS_ERR_ARG;
}

int check_streams(const uint8_t *in, uint64_t in_bytes, const uint64_t *offsets, int64_t S) {
  if (S < 0 || (S > 0 && !offsets) || !natural(offsets)) return RANS_ERR_ARG;
  if ((in_bytes > 0 && !in) || !aligned_to(in, 4)) return RANS_ERR_ARG;
  return RANS_OK;
}

int check_distill(const rans_logits *in, const int32_t *ids, const float *lp, int32_t K,
                  float inv_temperature) {
  const int st = check_logits(in);
  if (st) return st;
  if (K < 1 || K > RANS_MAX_TOP) return RANS_ERR_ARG;
  if (!(inv_temperature > 0.0f) || !finite(inv_temperature)) return RANS_ERR_ARG;
  if (in->rows > 0 && (!ids || !lp)) return RANS_ERR_ARG;
  if (!natural(ids, lp)) return RANS_ERR_ARG;
  return RANS_OK;
}

// Whether two arrays share memory (an absent one shares none).
bool overlap(const void *a, uint64_t na, const void *b, uint64_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && x < y + nb && y < x + na;
}

// A result of the logits' shape: its rows, and what it may share with them.
int check_result(const rans_logits *in, const void *out, int32_t dtype, int64_t stride) {
  const int e = logits_bytes(dtype);
  if (e == 0) return RANS_ERR_ARG;
  if (in->rows == 0) return RANS_OK;
  if (!out || !aligned_to(out, (uint64_t)e)) return RANS_ERR_ARG;
  if (in->rows > 1 && stride < in->vocab) return RANS_ERR_ARG;
  const uintptr_t a = reinterpret_cast<uintptr_t>(in->data), b = reinterpret_cast<uintptr_t>(out);
  const uint64_t ein = (uint64_t)logits_bytes(in->dtype);
  const uint64_t la = ((uint64_t)(in->rows - 1) * (uint64_t)in->row_stride + in->vocab) * ein;
  const uint64_t lb = ((uint64_t)(in->rows - 1) * (uint64_t)stride + in->vocab) * (uint64_t)e;
  if (a < b + lb && b < a + la) {
    // the same rows, or interleaved ones of one buffer
    if (dtype != in->dtype || (in->rows > 1 && stride != in->row_stride)) return RANS_ERR_ARG;
    if (a == b) return RANS_OK;
    if (in->rows == 1) return RANS_ERR_ARG;
    const uint64_t d = a < b ? b - a : a - b, row = (uint64_t)stride * ein;
    const uint64_t off = d % row, len = (uint64_t)in->vocab * ein;
    if (off < len || row - off < len) return RANS_ERR_ARG;
  }
  return RANS_OK;
}

// Whether an array lies on any of a result's rows (between them it may).
bool on_rows(const void *p, uint64_t bytes, const rans_logits *in, const void *out,
             int64_t stride) {
  const uint64_t e = (uint64_t)logits_bytes(in->dtype), len = (uint64_t)in->vocab * e;
  const uint64_t step = (uint64_t)stride * e;
  if (!overlap(p, bytes, out, (in->rows > 1 ? (uint64_t)(in->rows - 1) * step : 0) + len))
    return false;
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(out);
  if (in->rows == 1 || a < b) return true;
  const uint64_t off = (a - b) % step;
  return off < len || off + bytes > step;
}

// A distillation reads its lists more than once, and from several blocks: no
// result may lie on them, nor on what else is read, nor on another result.
// (losses may be the weights: every block has read its row's before.)
int check_distill_memory(const rans_logits *in, const int32_t *ids, const float *lp, int32_t K,
                         const float *weights, const float *losses, const float *stats,
                         bool stats_written, const void *grad, int64_t stride) {
  const uint64_t row = 4ull * (uint64_t)in->rows, list = row * (uint64_t)K, st = 8 * row;
  auto on_grad = [&](const void *p, uint64_t bytes) {
    return p && grad && on_rows(p, bytes, in, grad, stride);
  };
  auto on_stats = [&](const void *p, uint64_t bytes) {
    return stats_written && overlap(p, bytes, stats, st);
  };
  auto on_losses = [&](const void *p, uint64_t bytes) { return overlap(p, bytes, losses, row); };
  auto on_logits = [&](const void *p, uint64_t bytes) {
    return p && on_rows(p, bytes, in, in->data, in->row_stride);
  };
  if (on_grad(ids, list) || on_stats(ids, list) || on_losses(ids, list) || on_grad(lp, list) ||
      on_stats(lp, list) || on_losses(lp, list))
    return RANS_ERR_ARG;
  if (on_grad(weights, row) || on_stats(weights, row) ||
      (weights != losses && on_losses(weights, row)))
    return RANS_ERR_ARG;
  if (on_grad(losses, row) || on_stats(losses, row) || on_logits(losses, row) ||
      on_grad(stats, st) || (stats_written && on_logits(stats, st)))
    return RANS_ERR_ARG;
  return RANS_OK;
}

}  // namespace

RANS_API int rans_adjust_logits(const rans_logits *logits, const rans_adjust *adjust, void *out,
                                int32_t out_dtype, int64_t out_stride, void *stream) {
  NvtxRange nvtx_("rans_adjust_logits");
  rans_adjust a;
  int st = check_logits(logits);
  if (!st) st = check_adjust(adjust, logits->vocab, a);
  if (!st) st = check_result(logits, out, out_dtype, out_stride);
  if (st || logits->rows == 0) return st;
  return rb::launch_adjust(*logits, a, out, out_dtype, out_stride, as_stream(stream));
}

RANS_API int rans_token_intervals(const rans_logits *logits, const rans_adjust *adjust,
                                  const int32_t *tokens, uint32_t *starts, uint32_t *freqs,
                                  void *status, void *stream) {
  NvtxRange nvtx_("rans_token_intervals");
  rans_adjust a;
  int st = check_logits(logits);
  if (!st) st = check_adjust(adjust, logits->vocab, a);
  if (!st) st = check_status_word(status);
  if (st) return st;
  if (logits->rows == 0) return RANS_OK;
  if (!tokens || !starts || !freqs || !natural(tokens, starts, freqs)) return RANS_ERR_ARG;
  // a row's blocks read its token while others may be done with theirs
  const uint64_t bytes = 4ull * (uint64_t)logits->rows;
  if (overlap(tokens, bytes, starts, bytes) || overlap(tokens, bytes, freqs, bytes) ||
      overlap(starts, bytes, freqs, bytes) || overlap(status, 256, tokens, bytes))
    return RANS_ERR_ARG;
  return rb::launch_token_intervals(*logits, a, tokens, starts, freqs,
                                    static_cast<int32_t *>(status), as_stream(stream));
}

RANS_API int rans_encode_intervals(const uint32_t *starts, const uint32_t *freqs, int64_t n,
                                   const rans_chunking *chunking, uint8_t *out,
                                   uint64_t out_capacity, uint64_t *stream_offsets,
                                   void *workspace, uint64_t workspace_bytes, void *stream) {
  NvtxRange nvtx_("rans_encode_intervals");
  if (n > 0 && (!starts || !freqs)) return RANS_ERR_ARG;
  if (!stream_offsets || !workspace || (out_capacity > 0 && !out)) return RANS_ERR_ARG;
  if (!aligned_to(workspace, 256) || !aligned_to(out, 4)) return RANS_ERR_ARG;
  if (!natural(starts, freqs, stream_offsets)) return RANS_ERR_ARG;
  Geom g;
  int st = make_geom(chunking, n, g);
  if (st) return st;
  if (g.kind != RANS_CHUNK_CONTIG && g.kind != RANS_CHUNK_EXPLICIT) return RANS_ERR_ARG;
  if (g.kind == RANS_CHUNK_EXPLICIT && !natural(g.starts)) return RANS_ERR_ARG;
  if (g.W != 1 || g.ib_shift != 0 || g.fmt != RANS_FMT_RANS64 || g.alias) return RANS_ERR_ARG;
  if (workspace_bytes < enc_ws_bytes(g)) return RANS_ERR_CAPACITY;
  return rb::launch_encode_intervals(starts, freqs, g, reinterpret_cast<char *>(workspace),
                                     kWsHeader, lens_bytes(g), out, out_capacity, stream_offsets,
                                     as_stream(stream));
}

RANS_API int rans_token_states(const uint8_t *in, uint64_t in_bytes,
                               const uint64_t *stream_offsets, int64_t S, uint64_t *states,
                               void *status, void *stream) {
  NvtxRange nvtx_("rans_token_states");
  int st = check_streams(in, in_bytes, stream_offsets, S);
  if (!st) st = check_status_word(status);
  if (st) return st;
  if (S == 0) return RANS_OK;
  if (!states || !natural(states)) return RANS_ERR_ARG;
  return rb::launch_token_states(in, in_bytes, stream_offsets, S, states,
                                 static_cast<int32_t *>(status), as_stream(stream));
}

RANS_API int rans_decode_tokens(const rans_logits *logits, const rans_adjust *adjust,
                                const uint8_t *in, uint64_t in_bytes,
                                const uint64_t *stream_offsets, int64_t S,
                                const int32_t *stream_ids, const uint64_t *states_in,
                                uint64_t *states_out, int32_t *tokens, void *status,
                                void *stream) {
  NvtxRange nvtx_("rans_decode_tokens");
  rans_adjust a;
  int st = check_logits(logits);
  if (!st) st = check_adjust(adjust, logits->vocab, a);
  if (!st) st = check_streams(in, in_bytes, stream_offsets, S);
  if (!st) st = check_status_word(status);
  if (st) return st;
  if (!stream_ids && logits->rows > S) return RANS_ERR_ARG;
  if (logits->rows == 0) return RANS_OK;
  if (!states_in || !states_out || !tokens || !stream_offsets) return RANS_ERR_ARG;
  if (!natural(stream_ids, states_in, states_out, tokens)) return RANS_ERR_ARG;
  const uint64_t row_bytes = 4ull * (uint64_t)logits->rows, state_bytes = 16ull * (uint64_t)S;
  if ((states_in != states_out && overlap(states_in, state_bytes, states_out, state_bytes)) ||
      overlap(tokens, row_bytes, stream_ids, row_bytes) ||
      overlap(tokens, row_bytes, states_in, state_bytes) ||
      overlap(tokens, row_bytes, states_out, state_bytes) ||
      overlap(states_out, state_bytes, stream_ids, row_bytes) ||
      overlap(status, 256, stream_ids, row_bytes) || overlap(status, 256, states_in, state_bytes))
    return RANS_ERR_ARG;
  return rb::launch_decode_tokens(*logits, a, in, in_bytes, stream_offsets, S, stream_ids,
                                  states_in, states_out, tokens, static_cast<int32_t *>(status),
                                  as_stream(stream));
}

RANS_API int rans_token_states_finish(const uint64_t *stream_offsets, int64_t S,
                                      const uint64_t *states, void *status, void *stream) {
  NvtxRange nvtx_("rans_token_states_finish");
  if (S < 0 || (S > 0 && (!stream_offsets || !states))) return RANS_ERR_ARG;
  if (!natural(stream_offsets, states)) return RANS_ERR_ARG;
  const int st = check_status_word(status);
  if (st || S == 0) return st;
  return rb::launch_token_finish(stream_offsets, S, states, static_cast<int32_t *>(status),
                                 as_stream(stream));
}

RANS_API int rans_distill_forward(const rans_logits *logits, const int32_t *ids,
                                  const float *logprobs, int32_t K, float inv_temperature,
                                  int32_t tail, float *losses, float *stats, void *status,
                                  void *stream) {
  NvtxRange nvtx_("rans_distill_forward");
  int st = check_distill(logits, ids, logprobs, K, inv_temperature);
  if (!st) st = check_status_word(status);
  if (st || logits->rows == 0) return st;
  if (!losses || !stats || !aligned_to(stats, 16) || !natural(losses)) return RANS_ERR_ARG;
  if (check_distill_memory(logits, ids, logprobs, K, nullptr, losses, stats, true, nullptr, 0))
    return RANS_ERR_ARG;
  return rb::launch_distill_forward(*logits, ids, logprobs, K, inv_temperature, tail, losses,
                                    stats, static_cast<int32_t *>(status), as_stream(stream));
}

RANS_API int rans_distill_backward(const rans_logits *logits, const int32_t *ids,
                                   const float *logprobs, int32_t K, float inv_temperature,
                                   const float *stats, const float *grad_losses, void *grad,
                                   int64_t grad_stride, void *stream) {
  NvtxRange nvtx_("rans_distill_backward");
  int st = check_distill(logits, ids, logprobs, K, inv_temperature);
  if (!st) st = check_result(logits, grad, logits->dtype, grad_stride);
  if (st || logits->rows == 0) return st;
  if (!stats || !aligned_to(stats, 16) || !grad_losses || !natural(grad_losses))
    return RANS_ERR_ARG;
  if (check_distill_memory(logits, ids, logprobs, K, grad_losses, nullptr, stats, false, grad,
                           grad_stride))
    return RANS_ERR_ARG;
  return rb::launch_distill_backward(*logits, ids, logprobs, K, inv_temperature, stats,
                                     grad_losses, grad, grad_stride, as_stream(stream));
}

RANS_API int rans_distill(const rans_logits *logits, const int32_t *ids, const float *logprobs,
                          int32_t K, float inv_temperature, int32_t tail,
                          const float *grad_losses, float *losses, void *grad,
                          int64_t grad_stride, void *status, void *stream) {
  NvtxRange nvtx_("rans_distill");
  int st = check_distill(logits, ids, logprobs, K, inv_temperature);
  if (!st) st = check_result(logits, grad, logits->dtype, grad_stride);
  if (!st) st = check_status_word(status);
  if (st || logits->rows == 0) return st;
  if (!losses || !grad_losses || !natural(losses, grad_losses)) return RANS_ERR_ARG;
  if (check_distill_memory(logits, ids, logprobs, K, grad_losses, losses, nullptr, false, grad,
                           grad_stride))
    return RANS_ERR_ARG;
  return rb::launch_distill(*logits, ids, logprobs, K, inv_temperature, tail, grad_losses, losses,
                            grad, grad_stride, static_cast<int32_t *>(status),
                            as_stream(stream));
}

RANS_API int rans_get_status(void *workspace, void *stream) {
  if (!workspace) return RANS_ERR_ARG;
  cudaStream_t s = as_stream(stream);
  rb::StatusWord sw;
  if (cudaMemcpyAsync(&sw, workspace, sizeof(sw), cudaMemcpyDeviceToHost, s) != cudaSuccess ||
      cudaStreamSynchronize(s) != cudaSuccess)
    return RANS_ERR_CUDA;
  if (sw.code != 0) {
    if (cudaMemsetAsync(workspace, 0, sizeof(sw), s) != cudaSuccess ||
        cudaStreamSynchronize(s) != cudaSuccess)
      return RANS_ERR_CUDA;
  }
  return sw.code;
}

RANS_API int rans_debug_divide(const uint64_t *x, const uint32_t *f, int64_t n, uint64_t *q,
                               uint32_t *r, void *stream) {
  if (n < 0 || (n > 0 && (!x || !f || !q || !r))) return RANS_ERR_ARG;
  return rb::launch_debug_divide(x, f, n, q, r, as_stream(stream));
}
