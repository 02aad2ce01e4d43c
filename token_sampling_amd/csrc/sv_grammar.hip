// sv_grammar.hip -- byte automata over the vocabulary: the masks of states
// (sv_grammar_masks) and the states along tokens (sv_grammar_advance).
//
// A state s takes a byte c to next[s][classes[c]]; a token is the walk over its
// bytes.  -1 stands for "no grammar" (and for a refused byte within a walk).
#include <type_traits>

#include "sv_common.hpp"

namespace sv {
namespace {

constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / kWave;
constexpr int kHeld = 16;  // bytes of a token that a lane holds

struct GrammarArgs {
  sv_grammar g;
  sv_vocab v;
};

// The automaton as the walks see it: each byte is a column, step(s, column) the
// place after it.  Column stay() leaves every place (a token's end), column
// refused() leads to the dead place from everywhere, as does a byte whose class
// or next state lies outside the table; the dead place is never left.
//
// In LDS: rows of n_classes + 2 columns, the last row the dead place's, each
// entry the start of the row it leads to, so that a step is an addition and a
// 16-bit read.
template <int kEntries>
struct Table {
  const uint16_t* t;
  int classes, dead_;
  static __host__ __device__ bool fits(const sv_grammar& g) {
    return (int64_t)(g.n_states + 1ll) * (g.n_classes + 2) <= kEntries;
  }
  __device__ Table(const sv_grammar& g, uint16_t* lds) : t(lds) {
    classes = g.n_classes;
    const int width = classes + 2;
    dead_ = g.n_states * width;
    int s = threadIdx.x / width, c = threadIdx.x % width;
    for (int i = threadIdx.x; i < dead_ + width; i += kThreads) {
      int to = s;  // stay
      if (c < classes && s < g.n_states) to = g.next[s * classes + c];
      if (to < 0 || to > g.n_states || c > classes) to = g.n_states;
      lds[i] = (uint16_t)(to * width);
      s += kThreads / width;
      c += kThreads % width;
      if (c >= width) {
        c -= width;
        ++s;
      }
    }
  }
  __device__ int stay() const { return classes; }
  __device__ int refused() const { return classes + 1; }
  __device__ int dead() const { return dead_; }
  __device__ int at(int state) const { return state * (classes + 2); }
  __device__ int state(int place) const { return place / (classes + 2); }
  __device__ int step(int s, int column) const { return t[s + column]; }
};
// In global memory, for automata that do not fit: places are states.
template <>
struct Table<0> {
  const int32_t* next;
  int states, classes;
  __device__ Table(const sv_grammar& g, uint16_t*)
      : next(g.next), states(g.n_states), classes(g.n_classes) {}
  __device__ int stay() const { return classes; }
  __device__ int refused() const { return classes + 1; }
  __device__ int dead() const { return -1; }
  __device__ int at(int state) const { return state; }
  __device__ int state(int place) const { return place; }
  __device__ int step(int s, int column) const {
    if (s < 0 || column == classes) return s;
    const int to = column > classes ? -1 : next[(int64_t)s * classes + column];
    return to >= 0 && to < states ? to : -1;
  }
};

// Calls f(0), f(1), .. f(N - 1), each with its constant, until one returns false
// (a loop around wave-wide votes is not unrolled, and an array that it indexes
// would go to memory).
template <int N, int K = 0, typename F>
__device__ inline void until(F&& f) {
  if constexpr (K < N)
    if (f(std::integral_constant<int, K>())) until<N, K + 1>(f);
}

// A token as a lane holds it: the columns of its first bytes, two to a word,
// filled up with stay().
struct Token {
  int lo, len;  // its bytes; len = 0 for a token without any
  bool end;     // it ends a text
  uint32_t columns[kHeld / 2];
};

template <typename TableT>
__device__ inline Token token_of(const sv_vocab& v, const TableT& table, const uint16_t* column,
                                 int id) {
  Token t;
  t.lo = 0;
  t.len = 0;
  t.end = false;
  if (id >= 0 && id < v.V) {
    const int lo = v.offsets[id], hi = v.offsets[id + 1];
    t.lo = lo < 0 ? 0 : lo;
    t.len = (hi > v.n_bytes ? v.n_bytes : hi) - t.lo;
    t.len = t.len < 0 ? 0 : t.len;
    for (int i = 0; i < v.n_end; ++i) t.end |= v.end[i] == id;
    if (t.end) t.len = 0;
  }
  uint8_t x[kHeld] = {};
  if (t.len > 0) {
    if (t.lo + kHeld <= v.n_bytes) {
      __builtin_memcpy(x, v.bytes + t.lo, kHeld);
    } else {
#pragma unroll
      for (int k = 0; k < kHeld; ++k)
        if (k < t.len) x[k] = v.bytes[t.lo + k];
    }
  }
#pragma unroll
  for (int k = 0; k < kHeld; k += 2) {
    const uint32_t c0 = k < t.len ? column[x[k]] : table.stay();
    const uint32_t c1 = k + 1 < t.len ? column[x[k + 1]] : table.stay();
    t.columns[k / 2] = c0 | c1 << 16;
  }
  return t;
}

template <typename TableT>
__device__ inline void columns_of(const sv_grammar& g, const TableT& table, uint16_t* column) {
  if (threadIdx.x < 256) {
    const int c = g.classes[threadIdx.x];
    column[threadIdx.x] = (uint16_t)(c < g.n_classes ? c : table.refused());
  }
}

// Masks of states k0 .. k0 + kStates - 1 over 1024 tokens: a unit of work.  Each
// lane holds one token and takes it through kAbreast states at a time, whose
// lookups overlap; a wave stops where none of its tokens goes on.  The ballots
// are gathered in LDS and stored 128 bytes a state.
constexpr int kStates = 64;
#ifndef SV_ABREAST
#define SV_ABREAST 4
#endif
constexpr int kAbreast = SV_ABREAST;
static_assert(kStates % kAbreast == 0, "groups of states end with a unit");
template <int kEntries>
__global__ __launch_bounds__(kThreads) void k_masks(GrammarArgs a, const int32_t* states, int n,
                                                    int chunk, uint32_t* bits) {
  __shared__ uint16_t lds[kEntries ? kEntries : 1];
  __shared__ uint16_t column[256];
  __shared__ uint64_t rows[kStates][kWaves];
  __shared__ int32_t begin[kStates];  // the unit's states, -1 where every token is allowed
  __shared__ bool accepts[kStates];
  const Table<kEntries> table(a.g, lds);
  columns_of(a.g, table, column);
  __syncthreads();
  const int lane = __lane_id();
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int W = (a.v.V + 31) / 32;
  const int chunks = (n + chunk - 1) / chunk, tiles = (a.v.V + kThreads - 1) / kThreads;
  const int64_t units = (int64_t)tiles * chunks;
  // a workgroup's units are neighbours: mostly the same tokens
  const int64_t each = (units + gridDim.x - 1) / gridDim.x;
  const int64_t u1 = (blockIdx.x + 1) * each < units ? (blockIdx.x + 1) * each : units;
  int tile = -1, longest = 0;
  Token t = {};
  uint64_t valid = 0, ends = 0;
  for (int64_t u = blockIdx.x * each; u < u1; ++u) {
    if (tile != (int)(u / chunks)) {
      tile = (int)(u / chunks);
      const int id = tile * kThreads + (int)threadIdx.x;
      t = token_of(a.v, table, column, id);
      valid = __ballot(id < a.v.V);
      ends = __ballot(t.end);
      longest = wave_reduce(t.len, OpMax());
    }
    const int k0 = (int)(u % chunks) * chunk;
    const int count = n - k0 < chunk ? n - k0 : chunk;
    if (threadIdx.x < kStates) {
      const int state = threadIdx.x < count ? states[k0 + threadIdx.x] : -1;
      const bool in = state >= 0 && state < a.g.n_states;
      begin[threadIdx.x] = in ? state : -1;
      accepts[threadIdx.x] = in && a.g.accept[state] != 0;
    }
    __syncthreads();
    for (int j0 = 0; j0 < count; j0 += kAbreast) {
      int start[kAbreast], s[kAbreast];
#pragma unroll
      for (int q = 0; q < kAbreast; ++q) {
        start[q] = __builtin_amdgcn_readfirstlane(begin[j0 + q]);
        s[q] = start[q] >= 0 ? table.at(start[q]) : table.dead();
      }
      until<kHeld>([&](auto k) {
        const int c = k % 2 ? t.columns[k / 2] >> 16 : t.columns[k / 2] & 0xFFFF;
        bool live = false;
#pragma unroll
        for (int q = 0; q < kAbreast; ++q) {
          s[q] = table.step(s[q], c);
          live |= s[q] != table.dead();
        }
        return __any(live && k + 1 < t.len) != 0;
      });
      if (longest > kHeld) {
        for (int k = kHeld; k < t.len; ++k) {
          const int c = column[a.v.bytes[t.lo + k]];
          bool live = false;
#pragma unroll
          for (int q = 0; q < kAbreast; ++q) {
            s[q] = table.step(s[q], c);
            live |= s[q] != table.dead();
          }
          if (!live) break;
        }
      }
#pragma unroll
      for (int q = 0; q < kAbreast; ++q) {
        uint64_t m = __ballot(s[q] != table.dead() && t.len > 0);
        if (ends != 0 && accepts[j0 + q]) m |= ends;
        if (start[q] < 0) m = valid;
        if (lane == 0 && j0 + q < count) rows[j0 + q][wave] = m;
      }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < count * kWaves * 2; i += kThreads) {
      const int j = i / (kWaves * 2), w = tile * (kThreads / 32) + i % (kWaves * 2);
      if (w < W) bits[(size_t)(k0 + j) * W + w] = ((const uint32_t*)rows[j])[i % (kWaves * 2)];
    }
    __syncthreads();
  }
}

// A session's tokens: a wave holds 64 of them, one a lane, and walks them one
// after another, every lane alike; the chain of lookups is what it waits for.
template <int kEntries>
__global__ __launch_bounds__(kThreads) void k_advance(GrammarArgs a, const int32_t* states,
                                                      const int32_t* tokens, const int32_t* lens,
                                                      int B, int L, int32_t* out, int32_t* last) {
  __shared__ uint16_t lds[kEntries ? kEntries : 1];
  __shared__ uint16_t column[256];
  const Table<kEntries> table(a.g, lds);
  columns_of(a.g, table, column);
  __syncthreads();
  const int lane = __lane_id();
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int b = blockIdx.x * kWaves + wave;
  if (b >= B) return;
  const int from = states[b];
  const bool in = from >= 0 && from < a.g.n_states;
  int s = in ? table.at(from) : table.dead();
  int n = lens ? lens[b] : L;
  n = n < 0 ? 0 : n > L ? L : n;
  out += (size_t)b * (L + 1);
  if (lane == 0) out[0] = in ? from : -1;
  for (int i0 = 0; i0 < L; i0 += kWave) {
    const int held = n - i0 < kWave ? n - i0 : kWave;  // may be 0 or less
    const Token t =
        token_of(a.v, table, column, lane < held ? tokens[(size_t)b * L + i0 + lane] : -1);
    int mine = table.dead();
    for (int i = 0; i < held && s != table.dead(); ++i) {
      const int len = lane_read(t.len, i);
      if (len == 0) {
        s = table.dead();
        break;
      }
      until<kHeld>([&](auto k) {
        const uint32_t c = lane_read(t.columns[k / 2], i);
        s = table.step(s, k % 2 ? c >> 16 : c & 0xFFFF);
        return k + 1 < len;
      });
      if (len > kHeld) {
        const int lo = lane_read(t.lo, i);
        for (int k = kHeld; k < len && s != table.dead(); ++k)
          s = table.step(s, column[a.v.bytes[lo + k]]);
      }
      s = __builtin_amdgcn_readfirstlane(s);
      if (lane == i) mine = s;
    }
    if (i0 + lane < L) out[i0 + lane + 1] = mine == table.dead() ? -1 : table.state(mine);
  }
  if (last && lane == 0) last[b] = s == table.dead() ? -1 : table.state(s);
}

// Calls f with the LDS table size for g, 0 where none holds it.
template <typename F>
void by_size(const sv_grammar& g, F f) {
  if (Table<8192>::fits(g)) f(std::integral_constant<int, 8192>());
  else if (Table<32768>::fits(g)) f(std::integral_constant<int, 32768>());
  else if (Table<65536>::fits(g)) f(std::integral_constant<int, 65536>());
  else f(std::integral_constant<int, 0>());
}

bool grammar_ok(const sv_grammar* g, const sv_vocab* v) {
  if (!g || !g->next || !g->classes || !g->accept || g->n_states < 1 || g->n_classes < 1 ||
      g->n_classes > 256)
    return false;
  if (!v || !v->offsets || v->n_bytes < 0 || (v->n_bytes > 0 && !v->bytes) || v->n_end < 0 ||
      v->n_end > SV_STOP_MAX || (v->n_end > 0 && !v->end) || v->V < 1 || v->V > SV_V_MAX)
    return false;
  return true;
}

}  // namespace
}  // namespace sv

extern "C" int sv_grammar_masks(const sv_grammar* grammar, const sv_vocab* vocab,
                                const int32_t* states, int32_t n, uint32_t* bits, void* stream) {
  using namespace sv;
  if (!grammar_ok(grammar, vocab) || !states || !bits || n < 1) return SV_ERR_ARG;
  GrammarArgs a = {*grammar, *vocab};
  (void)hipGetLastError();
  by_size(*grammar, [&](auto entries) {
    constexpr int kEntries = decltype(entries)::value;
    // units of up to kStates states for every workgroup that the card holds
    const int64_t tiles = (vocab->V + kThreads - 1) / kThreads;
    const int64_t places = kEntries > 32768 ? 256 : 512;
    int64_t chunk = (n * tiles + places - 1) / places;
    chunk = chunk < kAbreast ? kAbreast : chunk > kStates ? kStates : chunk;
    const int64_t units = tiles * ((n + chunk - 1) / chunk);
    hipLaunchKernelGGL(k_masks<kEntries>, dim3((unsigned)(units < places ? units : places)),
                       dim3(kThreads), 0, (hipStream_t)stream, a, states, n, (int)chunk, bits);
  });
  return hipGetLastError() == hipSuccess ? SV_OK : SV_ERR_DEVICE;
}

extern "C" int sv_grammar_advance(const sv_grammar* grammar, const sv_vocab* vocab,
                                  const int32_t* states, const int32_t* tokens,
                                  const int32_t* lens, int32_t B, int32_t L, int32_t* out_states,
                                  int32_t* last, void* stream) {
  using namespace sv;
  if (!grammar_ok(grammar, vocab) || !states || !out_states || B < 1 || B > SV_B_MAX || L < 0 ||
      L > SV_M_MAX + 1 || (L > 0 && !tokens))
    return SV_ERR_ARG;
  GrammarArgs a = {*grammar, *vocab};
  (void)hipGetLastError();
  by_size(*grammar, [&](auto entries) {
    hipLaunchKernelGGL(k_advance<decltype(entries)::value>, dim3((B + kWaves - 1) / kWaves),
                       dim3(kThreads), 0, (hipStream_t)stream, a, states, tokens, lens, B, L,
                       out_states, last);
  });
  return hipGetLastError() == hipSuccess ? SV_OK : SV_ERR_DEVICE;
}
