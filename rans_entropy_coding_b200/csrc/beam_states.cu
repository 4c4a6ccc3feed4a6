// beam_states.cu -- what follows a selection: a search's own bookkeeping
// (rans_beam_advance) and the model's states (rans_reorder_states).
//
// States are moved in place: a thread takes the same bytes of all beams of a
// text, so what it moves is its own, and only moving beams' live positions are read
// and written.  Where no source moves itself, as in a search's own maps, beams
// are moved a few at a time; bound by memory.  In any other map (chains, cycles) a thread
// loads all that moves before it stores any: up to 16 beams as words of 8 bytes in
// registers, more, or rows off 8 bytes, as 64 words under the same limit of registers,
// most of which then lie in local memory (696 bytes stored and 1512 loaded a thread, as
// compiled).  Measured, 1.07 GB moved where half of 32 x 8 beams' states move: 322 us; all
// of them in cycles (2.1 GB): 1.07 ms; cycles of 32 beams 4.4 ms; rows off 4 bytes, byte by
// byte, 9 to 20 ms.
#include "logits_common.cuh"
#include "rans_common.cuh"
#include "rans_internal.h"

namespace rb {
namespace {

constexpr int kMoveThreads = 256;
constexpr int kMoveSteps = 4;         // accesses of a thread in a beam's row
constexpr int kStatesPerLaunch = 56;  // their descriptions are a launch's arguments

struct Moves {
  rans_state state[kStatesPerLaunch];
  int64_t first[kStatesPerLaunch + 1];  // blocks of a text before each state's
  int32_t chunks[kStatesPerLaunch];     // blocks of a segment
  int32_t bytes[kStatesPerLaunch];      // of an access: 16, 8, 4, 2 or 1
  int32_t n;
};
static_assert(sizeof(Moves) < 4096 - 64, "arguments of a launch");

// Moves the bytes from .. to - 1 of a piece of `bytes`, G beams' accesses at a time in
// registers (G >= n_moves: all of them before any is stored).
template <typename V, int G>
__device__ __forceinline__ void move_bytes(char *at, int64_t row_stride, const int2 *moves,
                                           int n_moves, int64_t bytes, int64_t from, int64_t to) {
  const int64_t end = min(bytes, to);
  for (int64_t i = from + (int64_t)threadIdx.x * sizeof(V); i < end;
       i += (int64_t)kMoveThreads * sizeof(V)) {
    if (i + (int64_t)sizeof(V) <= bytes) {
      for (int m0 = 0; m0 < n_moves; m0 += G) {
        V v[G];
#pragma unroll
        for (int m = 0; m < G; ++m)
          if (m0 + m < n_moves)
            v[m] = *reinterpret_cast<const V *>(at + moves[m0 + m].x * row_stride + i);
#pragma unroll
        for (int m = 0; m < G; ++m)
          if (m0 + m < n_moves) *reinterpret_cast<V *>(at + moves[m0 + m].y * row_stride + i) = v[m];
      }
    } else {  // the last access of a piece that it does not fill
      for (int64_t k = i; k < bytes; ++k)
        for (int m0 = 0; m0 < n_moves; m0 += G) {
          char v[G];
#pragma unroll
          for (int m = 0; m < G; ++m)
            if (m0 + m < n_moves) v[m] = at[moves[m0 + m].x * row_stride + k];
#pragma unroll
          for (int m = 0; m < G; ++m)
            if (m0 + m < n_moves) at[moves[m0 + m].y * row_stride + k] = v[m];
        }
    }
  }
}

// A whole block's share where no source moves: two beams' kMoveSteps accesses in
// flight per thread.  Measured, 32 texts of 8 beams, 1.4 GB to read and write: 214 us
// (6.4 TB/s); single accesses of four beams at a time 320 us, of all beams 255 us.
template <typename V>
__device__ __forceinline__ void move_block(char *at, int64_t row_stride, const int2 *moves,
                                           int n_moves, int64_t from) {
  constexpr int64_t kStep = (int64_t)kMoveThreads * sizeof(V);
  at += from + (int64_t)threadIdx.x * sizeof(V);
  for (int m = 0; m < n_moves; m += 2) {
    const int2 a = moves[m], b = moves[min(m + 1, n_moves - 1)];
    const char *pa = at + a.x * row_stride, *pb = at + b.x * row_stride;
    V v[2][kMoveSteps];
#pragma unroll
    for (int u = 0; u < kMoveSteps; ++u) v[0][u] = *reinterpret_cast<const V *>(pa + u * kStep);
    if (m + 1 < n_moves) {
#pragma unroll
      for (int u = 0; u < kMoveSteps; ++u) v[1][u] = *reinterpret_cast<const V *>(pb + u * kStep);
    }
    char *qa = at + a.y * row_stride, *qb = at + b.y * row_stride;
#pragma unroll
    for (int u = 0; u < kMoveSteps; ++u) *reinterpret_cast<V *>(qa + u * kStep) = v[0][u];
    if (m + 1 < n_moves) {
#pragma unroll
      for (int u = 0; u < kMoveSteps; ++u) *reinterpret_cast<V *>(qb + u * kStep) = v[1][u];
    }
  }
}

__global__ void __launch_bounds__(kMoveThreads, 4)
    reorder_kernel(const __grid_constant__ Moves mv, int beams, const int32_t *parents,
                   const int32_t *lengths, int32_t *status) {
  __shared__ int2 moves[RANS_MAX_BEAMS];
  __shared__ int n_moves;
  __shared__ bool chained;  // a source moves itself
  const int64_t per_text = mv.first[mv.n];
  const int64_t t = blockIdx.x / per_text, unit = blockIdx.x - t * per_text;
  int k = 0;
  while (unit >= mv.first[k + 1]) ++k;
  const rans_state &s = mv.state[k];
  const int64_t seg = (unit - mv.first[k]) / mv.chunks[k];
  const int64_t chunk = unit - mv.first[k] - seg * mv.chunks[k];
  int64_t live = s.positions;
  if (lengths) live = min(live, (int64_t)max(lengths[t], 0));
  const int64_t bytes = live * s.position_bytes, from = chunk * kMoveThreads * kMoveSteps * mv.bytes[k];
  if (threadIdx.x < 32) {
    int at = 0;
    unsigned long long sources = 0, targets = 0;
    for (int b0 = 0; b0 < beams; b0 += 32) {
      const int b = b0 + (int)threadIdx.x;
      const int p = b < beams ? parents[t * beams + b] : -1;
      const bool off = p < -1 || p >= beams, go = p >= 0 && !off && p != b;
      if (off && unit == 0 && status) report(status, RANS_ERR_INDEX, t * beams + b);
      const uint32_t all = __ballot_sync(0xffffffffu, go);
      if (go) {
        moves[at + __popc(all & ((1u << (threadIdx.x & 31)) - 1u))] = make_int2(p, b);
        sources |= 1ull << p;
      }
      targets |= (unsigned long long)all << b0;
      at += __popc(all);
    }
    const bool hit = __any_sync(0xffffffffu, (sources & targets) != 0);
    if (threadIdx.x == 0) {
      n_moves = at;
      chained = hit;
    }
  }
  __syncthreads();
  const int n = n_moves, width = mv.bytes[k];
  if (n == 0 || from >= bytes) return;
  char *at = static_cast<char *>(s.data) + t * beams * s.row_stride + seg * s.segment_stride;
  const int64_t to = from + (int64_t)kMoveThreads * kMoveSteps * width;
  if (!chained) {
    if (width == 16 && to <= bytes) return move_block<uint4>(at, s.row_stride, moves, n, from);
    switch (width) {
      case 16: return move_bytes<uint4, 4>(at, s.row_stride, moves, n, bytes, from, to);
      case 8: return move_bytes<uint2, 4>(at, s.row_stride, moves, n, bytes, from, to);
      case 4: return move_bytes<uint32_t, 4>(at, s.row_stride, moves, n, bytes, from, to);
      case 2: return move_bytes<uint16_t, 4>(at, s.row_stride, moves, n, bytes, from, to);
      default: return move_bytes<uint8_t, 4>(at, s.row_stride, moves, n, bytes, from, to);
    }
  }
  if (width >= 8 && n <= 16)
    move_bytes<uint2, 16>(at, s.row_stride, moves, n, bytes, from, to);
  else if (width >= 4)
    move_bytes<uint32_t, RANS_MAX_BEAMS>(at, s.row_stride, moves, n, bytes, from, to);
  else
    move_bytes<uint8_t, RANS_MAX_BEAMS>(at, s.row_stride, moves, n, bytes, from, to);
}

// The widest access that a state's addresses allow.
int access_bytes(const rans_state &s) {
  uint64_t x = reinterpret_cast<uintptr_t>(s.data) | (uint64_t)s.row_stride;
  if (s.segments > 1) x |= (uint64_t)s.segment_stride;
  int w = 16;
  while (x & (uint64_t)(w - 1)) w >>= 1;
  return w;
}

// ------------------------------------------------------------- bookkeeping --
constexpr int kAdvanceThreads = 128;

__device__ __forceinline__ float penalised(float score, int length, float penalty) {
  return penalty == 0.0f ? score : score / powf((float)length, penalty);
}

// One block per text.  One thread goes through the candidates, best first; the
// block then copies token histories.  Measured in a graph, behind a fill of the lengths,
// 512 tokens a beam: 1 text of 4 beams 6 us, 32 of 8 10 us (7 ends: 11), 256 of 8 11 us, 32
// of 64 56 us.  Bound by that thread's chain of reads, with many beams by the histories,
// row after row.
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

}  // namespace

namespace {

// The next states' moves as one launch has them, of a text; how many there are, or an
// error.
int plan_moves(const rans_state *states, int32_t n, int64_t texts, Moves &mv) {
  mv.n = n < kStatesPerLaunch ? n : kStatesPerLaunch;
  mv.first[0] = 0;
  for (int32_t i = 0; i < mv.n; ++i) {
    const rans_state &s = states[i];
    mv.state[i] = s;
    mv.bytes[i] = access_bytes(s);
    const int64_t chunk = (int64_t)kMoveThreads * kMoveSteps * mv.bytes[i];
    const int64_t chunks = (s.positions * s.position_bytes + chunk - 1) / chunk;
    if (chunks > 0x7fffffff) return RANS_ERR_ARG;
    mv.chunks[i] = (int32_t)chunks;
    mv.first[i + 1] = mv.first[i] + chunks * s.segments;
    if (mv.first[i + 1] > 0x7fffffff) return RANS_ERR_ARG;
  }
  if (mv.first[mv.n] > 0 && texts > 0x7fffffff / mv.first[mv.n]) return RANS_ERR_ARG;
  return mv.n;
}

}  // namespace

int check_reorder_states(const rans_state *states, int32_t n, int64_t texts) {
  Moves mv;
  for (int32_t i = 0; i < n; i += mv.n) {
    const int e = plan_moves(states + i, n - i, texts, mv);
    if (e < 0) return e;
  }
  return RANS_OK;
}

int launch_reorder_states(const rans_state *states, int32_t n, int64_t texts, int beams,
                          const int32_t *parents, const int32_t *lengths, int32_t *status,
                          cudaStream_t st) {
  // (what the second launch would refuse, the first must not have moved)
  const int bad = n > kStatesPerLaunch ? check_reorder_states(states, n, texts) : RANS_OK;
  if (bad) return bad;
  Moves mv;
  for (int32_t i = 0; i < n; i += mv.n) {
    const int e = plan_moves(states + i, n - i, texts, mv);
    if (e < 0) return e;
    const int64_t per_text = mv.first[mv.n];
    if (per_text == 0) continue;
    reorder_kernel<<<(unsigned)(texts * per_text), kMoveThreads, 0, st>>>(mv, beams, parents,
                                                                          lengths, status);
    if (cudaGetLastError() != cudaSuccess) return RANS_ERR_CUDA;
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
