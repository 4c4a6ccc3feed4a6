// beam_states.cu -- what follows a selection: a search's own bookkeeping
// (rans_beam_advance) and the model's states (rans_reorder_states).
//
// States are moved in place: a thread takes the same bytes of all beams of a
// text, loads what moves and then stores it, so any map of parents (cycles too)
// is right without a second buffer, and only moving beams' live positions are
// read and written.  Bound by memory.
#include "logits_common.cuh"
#include "rans_common.cuh"
#include "rans_internal.h"

namespace rb {
namespace {

constexpr int kMoveThreads = 256;
constexpr int kStatesPerLaunch = 56;  // their descriptions are a launch's arguments

struct Moves {
  rans_state state[kStatesPerLaunch];
  int64_t first[kStatesPerLaunch + 1];  // blocks of a text before each state's
  int32_t chunks[kStatesPerLaunch];     // blocks of a segment
  int32_t bytes[kStatesPerLaunch];      // of an access: 16, 8, 4, 2 or 1
  int32_t n;
};
static_assert(sizeof(Moves) < 4096 - 64, "arguments of a launch");

template <typename V, int MOST>
__device__ __forceinline__ void move_bytes(char *at, int64_t row_stride, const int2 *moves,
                                           int n_moves, int64_t bytes, int64_t from) {
  // whole accesses, then single bytes of the last one
  const int64_t i = from + (int64_t)threadIdx.x * sizeof(V);
  if (i + (int64_t)sizeof(V) <= bytes) {
    V v[MOST];
#pragma unroll
    for (int m = 0; m < MOST; ++m)
      if (m < n_moves) v[m] = *reinterpret_cast<const V *>(at + moves[m].x * row_stride + i);
#pragma unroll
    for (int m = 0; m < MOST; ++m)
      if (m < n_moves) *reinterpret_cast<V *>(at + moves[m].y * row_stride + i) = v[m];
  } else {
    for (int64_t j = i; j < bytes; ++j) {
      char v[MOST];
#pragma unroll
      for (int m = 0; m < MOST; ++m)
        if (m < n_moves) v[m] = at[moves[m].x * row_stride + j];
#pragma unroll
      for (int m = 0; m < MOST; ++m)
        if (m < n_moves) at[moves[m].y * row_stride + j] = v[m];
    }
  }
}

template <int MOST>
__global__ void __launch_bounds__(kMoveThreads)
    reorder_kernel(const __grid_constant__ Moves mv, int beams, const int32_t *parents,
                   const int32_t *lengths, int32_t *status) {
  __shared__ int2 moves[RANS_MAX_BEAMS];
  __shared__ int n_moves;
  const int64_t per_text = mv.first[mv.n];
  const int64_t t = blockIdx.x / per_text, unit = blockIdx.x - t * per_text;
  int k = 0;
  while (unit >= mv.first[k + 1]) ++k;
  const rans_state &s = mv.state[k];
  const int64_t seg = (unit - mv.first[k]) / mv.chunks[k];
  const int64_t chunk = unit - mv.first[k] - seg * mv.chunks[k];
  int64_t live = s.positions;
  if (lengths) live = min(live, (int64_t)max(lengths[t], 0));
  const int64_t bytes = live * s.position_bytes, from = chunk * kMoveThreads * mv.bytes[k];
  if (threadIdx.x < 32) {
    int at = 0;
    for (int b0 = 0; b0 < beams; b0 += 32) {
      const int b = b0 + (int)threadIdx.x;
      const int p = b < beams ? parents[t * beams + b] : -1;
      const bool off = p < -1 || p >= beams, go = p >= 0 && !off && p != b;
      if (off && unit == 0 && status) report(status, RANS_ERR_INDEX, t * beams + b);
      const uint32_t all = __ballot_sync(0xffffffffu, go);
      if (go) moves[at + __popc(all & ((1u << (threadIdx.x & 31)) - 1u))] = make_int2(p, b);
      at += __popc(all);
    }
    if (threadIdx.x == 0) n_moves = at;
  }
  __syncthreads();
  const int n = n_moves;
  if (n == 0 || from >= bytes) return;
  char *at = static_cast<char *>(s.data) + t * beams * s.row_stride + seg * s.segment_stride;
  switch (mv.bytes[k]) {
    case 16:
      if constexpr (MOST <= 32) move_bytes<uint4, MOST>(at, s.row_stride, moves, n, bytes, from);
      break;
    case 8: move_bytes<uint2, MOST>(at, s.row_stride, moves, n, bytes, from); break;
    case 4: move_bytes<uint32_t, MOST>(at, s.row_stride, moves, n, bytes, from); break;
    case 2: move_bytes<uint16_t, MOST>(at, s.row_stride, moves, n, bytes, from); break;
    default: move_bytes<uint8_t, MOST>(at, s.row_stride, moves, n, bytes, from);
  }
}

// The widest access that a state's addresses allow.
int access_bytes(const rans_state &s, int most) {
  uint64_t x = reinterpret_cast<uintptr_t>(s.data) | (uint64_t)s.row_stride;
  if (s.segments > 1) x |= (uint64_t)s.segment_stride;
  int w = most;
  while (x & (uint64_t)(w - 1)) w >>= 1;
  return w;
}

// ------------------------------------------------------------- bookkeeping --
constexpr int kAdvanceThreads = 128;

__device__ __forceinline__ float penalised(float score, int length, float penalty) {
  return penalty == 0.0f ? score : score / powf((float)length, penalty);
}

// One block per text.  One thread goes through the candidates, best first; the
// block then copies token histories.
__global__ void __launch_bounds__(kAdvanceThreads)
    beam_advance_kernel(const float *scores, const int32_t *tokens, const int32_t *parents,
                        int count, rans_beams s) {
  __shared__ int source[RANS_MAX_BEAMS];  // of each slot, or -1
  __shared__ int ended[RANS_MAX_BEAMS];   // parent of what ends in each place, or -1
  __shared__ int32_t token[RANS_MAX_BEAMS], last[RANS_MAX_BEAMS];
  __shared__ float score[RANS_MAX_BEAMS], pool[RANS_MAX_BEAMS];
  __shared__ int late[RANS_MAX_BEAMS];    // candidates whose parent's slot is taken
  __shared__ bool stop;
  const int tid = threadIdx.x, K = s.beams;
  const int64_t t = blockIdx.x;
  const int length = s.lengths[t];
  if (length < 0 || length >= s.capacity) {
    // full: nothing changes, nothing moves
    for (int b = tid; b < K; b += kAdvanceThreads) s.parents[t * K + b] = b;
    return;
  }
  for (int b = tid; b < K; b += kAdvanceThreads) {
    source[b] = ended[b] = -1;
    pool[b] = s.done_scores[t * K + b];
  }
  __syncthreads();
  if (tid == 0) {
    int kept = 0, n_late = 0, n_done = s.done_counts[t];
    float best = kNegInf;
    for (int j = 0; j < count && kept < K; ++j) {
      const float v = scores[t * count + j];
      const int32_t tok = tokens[t * count + j];
      const int p = parents[t * count + j];
      if (tok < 0 || p < 0 || p >= K || !(v > kNegInf)) break;
      bool end = false;
      for (int i = 0; i < s.n_ends; ++i) end |= s.ends[i] == tok;
      if (end) {
        if (j >= K) continue;  // as good a beam goes on instead
        const float w = penalised(v, length + 1, s.length_penalty);
        int at = n_done;
        if (n_done >= K) {  // the worst makes room, the last of equals
          at = 0;
          for (int i = 1; i < K; ++i)
            if (pool[i] <= pool[at]) at = i;
          if (!(w > pool[at])) continue;
        } else {
          ++n_done;
        }
        pool[at] = w;
        ended[at] = p;
        last[at] = tok;
        continue;
      }
      if (kept == 0) best = v;
      ++kept;
      if (source[p] < 0) {
        source[p] = p;
        token[p] = tok;
        score[p] = v;
      } else {
        late[n_late++] = j;
      }
    }
    // whoever finds its parent's slot taken moves to one that nobody goes on in
    for (int i = 0, b = 0; i < n_late; ++i, ++b) {
      while (source[b] >= 0) ++b;  // (kept <= K: there is one)
      const int j = late[i];
      source[b] = parents[t * count + j];
      token[b] = tokens[t * count + j];
      score[b] = scores[t * count + j];
    }
    // The search of a text is over when its beams are dead, or its places are
    // full and no beam can still reach the worst of them.
    bool over = kept == 0;
    if (n_done >= K) {
      float worst = pool[0];
      for (int i = 1; i < K; ++i) worst = fminf(worst, pool[i]);
      const int reach = s.length_penalty > 0.0f ? s.capacity : length + 1;
      over |= s.early || !(penalised(best, reach, s.length_penalty) > worst);
    }
    s.done_counts[t] = n_done;
    stop = over;
  }
  __syncthreads();
  const bool over = stop;
  // what has ended, before its beams' rows are written to
  for (int b = 0; b < K; ++b) {
    const int p = ended[b];
    if (p < 0) continue;
    const int32_t *from = s.history + (t * K + p) * s.capacity;
    int32_t *to = s.done_tokens + (t * K + b) * s.capacity;
    for (int i = tid; i < length; i += kAdvanceThreads) to[i] = from[i];
    if (tid == 0) {
      to[length] = last[b];
      s.done_lengths[t * K + b] = length + 1;
      s.done_scores[t * K + b] = pool[b];
    }
  }
  __syncthreads();
  for (int b = 0; b < K; ++b) {
    const int p = source[b];
    int32_t *to = s.history + (t * K + b) * s.capacity;
    // (a beam with a child that moved has one that stayed: its row is not written)
    if (p >= 0 && p != b) {
      const int32_t *from = s.history + (t * K + p) * s.capacity;
      for (int i = tid; i < length; i += kAdvanceThreads) to[i] = from[i];
    }
    if (tid == 0) {
      const int32_t tok = p >= 0 ? token[b] : s.pad;
      to[length] = tok;
      s.tokens[t * K + b] = tok;
      s.parents[t * K + b] = p >= 0 ? p : b;
      s.scores[t * K + b] = p >= 0 && !over ? score[b] : kNegInf;
    }
  }
  __syncthreads();
  if (tid == 0) {
    s.lengths[t] = length + 1;
    s.over[t] = over ? 1 : 0;
  }
  for (int b = tid; b < K; b += kAdvanceThreads)
    s.window_end[t * K + b] = (t * K + b) * s.capacity + length + 1;
}

template <int MOST>
int launch_moves(const Moves &mv, int64_t texts, int beams, const int32_t *parents,
                 const int32_t *lengths, int32_t *status, cudaStream_t st) {
  const int64_t per_text = mv.first[mv.n];
  if (per_text == 0) return RANS_OK;
  if (texts > 0x7fffffff / per_text) return RANS_ERR_ARG;
  reorder_kernel<MOST><<<(unsigned)(texts * per_text), kMoveThreads, 0, st>>>(mv, beams, parents,
                                                                              lengths, status);
  return cudaGetLastError() == cudaSuccess ? RANS_OK : RANS_ERR_CUDA;
}

}  // namespace

int launch_reorder_states(const rans_state *states, int32_t n, int64_t texts, int beams,
                          const int32_t *parents, const int32_t *lengths, int32_t *status,
                          cudaStream_t st) {
  for (int32_t i0 = 0; i0 < n; i0 += kStatesPerLaunch) {
    Moves mv;
    mv.n = n - i0 < kStatesPerLaunch ? n - i0 : kStatesPerLaunch;
    mv.first[0] = 0;
    for (int32_t i = 0; i < mv.n; ++i) {
      const rans_state &s = states[i0 + i];
      mv.state[i] = s;
      // (64 beams: 8 bytes each, which fit a thread's registers)
      mv.bytes[i] = access_bytes(s, beams > 32 ? 8 : 16);
      const int64_t chunk = (int64_t)kMoveThreads * mv.bytes[i];
      const int64_t chunks = (s.positions * s.position_bytes + chunk - 1) / chunk;
      if (chunks > 0x7fffffff) return RANS_ERR_ARG;
      mv.chunks[i] = (int32_t)chunks;
      mv.first[i + 1] = mv.first[i] + chunks * s.segments;
      if (mv.first[i + 1] > 0x7fffffff) return RANS_ERR_ARG;
    }
    int e;
    if (beams <= 4) e = launch_moves<4>(mv, texts, beams, parents, lengths, status, st);
    else if (beams <= 8) e = launch_moves<8>(mv, texts, beams, parents, lengths, status, st);
    else if (beams <= 16) e = launch_moves<16>(mv, texts, beams, parents, lengths, status, st);
    else if (beams <= 32) e = launch_moves<32>(mv, texts, beams, parents, lengths, status, st);
    else e = launch_moves<64>(mv, texts, beams, parents, lengths, status, st);
    if (e) return e;
  }
  return RANS_OK;
}

int launch_beam_advance(const float *scores, const int32_t *tokens, const int32_t *parents,
                        int count, const rans_beams &s, cudaStream_t st) {
  if (s.texts > 0x7fffffff) return RANS_ERR_ARG;
  beam_advance_kernel<<<(unsigned)s.texts, kAdvanceThreads, 0, st>>>(scores, tokens, parents, count,
                                                                     s);
  return cudaGetLastError() == cudaSuccess ? RANS_OK : RANS_ERR_CUDA;
}

}  // namespace rb
