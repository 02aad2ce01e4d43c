// sv_grammar.hip -- byte automata over the vocabulary: the masks of states
// (sv_grammar_masks) and the states along tokens (sv_grammar_advance).
//
// A state s takes a byte c to next[s][classes[c]]; a token is the walk over its
// bytes.  -1 stands for "no grammar" (and for a refused byte within a walk).
#include <limits.h>

#include <type_traits>

#include "sv_common.hpp"

namespace sv {
namespace {

constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / kWave;
constexpr int kHeld = 16;  // first bytes of a token that are held
constexpr int kMostEntries = 57344;  // of a table in LDS: 112 KB, and 48 KB for the tokens

struct GrammarArgs {
  sv_grammar g;
  sv_vocab v;
};

// The automaton as the walks see it: step(s, column) is the place after place s
// and a byte of the column (class); the dead place, after a byte that is
// refused, is never left.
//
// In LDS: each entry is the start of the row it leads to, so that a step is an
// addition and a 16-bit read; the dead place's row follows the states'.  With
// kEnd there is one column more, end(), which stands for the end of a token and
// leads from every state's place to the done place, the last row: places below
// dead() are those of walks that go on.
template <int kEntries, bool kEnd>
struct Table {
  const uint16_t* t;
  int width, dead_;
  static bool fits(const sv_grammar& g) {
    return g.n_classes < 256 && (g.n_states + (int64_t)2) * (g.n_classes + 1) <= kEntries;
  }
  __device__ Table(const sv_grammar& g, uint16_t* lds) : t(lds) {
    const int classes = g.n_classes, total = g.n_states * classes;
    width = classes + (kEnd ? 1 : 0);
    dead_ = g.n_states * width;
    // entry i of next, in row s and column c, is entry i + s here with kEnd; 16
    // bytes of them a load, all loads of a pass before the first is used
    const bool pieces = (uintptr_t)g.next % 16 == 0;
    const int whole = pieces ? total / 4 : 0;
    constexpr int kAhead = 4;
    int s = 4 * threadIdx.x / classes, c = 4 * threadIdx.x % classes;
    const int ds = 4 * kThreads / classes, dc = 4 * kThreads % classes;
    auto put = [&](int i, int row, int to) {
      lds[i + (kEnd ? row : 0)] = (uint16_t)(to >= 0 && to < g.n_states ? to * width : dead_);
    };
    for (int p0 = threadIdx.x; p0 < whole; p0 += kThreads * kAhead) {
      int4 to[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int p = p0 + k * kThreads;
        to[k] = ((const int4*)g.next)[p < whole ? p : p0];
      }
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int i = 4 * (p0 + k * kThreads);
        if (i < 4 * whole) {
          int row = s, col = c;
          auto next_column = [&] {
            if (++col == classes) {
              col = 0;
              ++row;
            }
          };
          put(i, row, to[k].x);
          next_column();
          put(i + 1, row, to[k].y);
          next_column();
          put(i + 2, row, to[k].z);
          next_column();
          put(i + 3, row, to[k].w);
        }
        s += ds;
        c += dc;
        if (c >= classes) {
          c -= classes;
          ++s;
        }
      }
    }
    for (int i = 4 * whole + threadIdx.x; i < total; i += kThreads) put(i, i / classes, g.next[i]);
    if (threadIdx.x < (unsigned)width) lds[dead_ + threadIdx.x] = (uint16_t)dead_;
    if constexpr (kEnd) {
      const int done = dead_ + width;
      for (int r = threadIdx.x; r < g.n_states; r += kThreads)
        lds[r * width + classes] = (uint16_t)done;
      if (threadIdx.x < (unsigned)width) lds[done + threadIdx.x] = (uint16_t)done;
    }
  }
  __device__ int dead() const { return dead_; }
  __device__ int end() const { return width - 1; }
  __device__ int at(int state) const { return state * width; }
  __device__ int state(int place) const { return place / width; }
  __device__ int step(int s, int column) const { return t[s + column]; }
};
// In global memory, for automata that do not fit: places are states.
template <bool kEnd>
struct Table<0, kEnd> {
  const int32_t* next;
  int states, classes;
  __device__ Table(const sv_grammar& g, uint16_t*)
      : next(g.next), states(g.n_states), classes(g.n_classes) {}
  __device__ int dead() const { return -1; }
  __device__ int end() const { return 0; }  // walks stop by the token's length here
  __device__ int at(int state) const { return state; }
  __device__ int state(int place) const { return place; }
  __device__ int step(int s, int column) const {
    const int to = next[(int64_t)max(s, 0) * classes + column];
    return s >= 0 && to >= 0 && to < states ? to : -1;
  }
};

// A byte's column, kRefused for a class outside the table.
constexpr int kRefused = 0xFFFF;
__device__ inline void columns_of(const sv_grammar& g, uint16_t* column) {
  if (threadIdx.x < 256) {
    const int c = g.classes[threadIdx.x];
    column[threadIdx.x] = (uint16_t)(c < g.n_classes ? c : kRefused);
  }
}

// Calls f(0), f(1), .. f(N - 1), each with its constant, until one returns false
// (a loop around wave-wide votes is not unrolled, and an array that it indexes
// would go to memory).
template <int N, int K = 0, typename F>
__device__ inline void until(F&& f) {
  if constexpr (K < N)
    if (f(std::integral_constant<int, K>())) until<N, K + 1>(f);
}

// A token and its first bytes.
struct Token {
  int lo, len;  // its bytes; len = 0 for a token without any, or that ends a text
  bool end;     // it ends a text
  uint8_t bytes[kHeld];
};

// bytes[at] .. and up to kHeld - 1 more, n of them at least where there are so many.
__device__ inline void held_bytes(const sv_vocab& v, int at, int n, uint8_t (&x)[kHeld]) {
  if (v.n_bytes - at >= kHeld) {
    __builtin_memcpy(x, v.bytes + at, kHeld);
  } else {
#pragma unroll
    for (int k = 0; k < kHeld; ++k) x[k] = k < n ? v.bytes[at + k] : 0;
  }
}

// An offset, kept within the bytes.
__device__ inline int offset_of(const sv_vocab& v, int i) {
  return min(max(v.offsets[i], 0), v.n_bytes);
}

__device__ inline Token token_of(const sv_vocab& v, int id) {
  Token t = {};
  if (id >= 0 && id < v.V) {
    t.lo = offset_of(v, id);
    t.len = max(offset_of(v, id + 1) - t.lo, 0);
    for (int i = 0; i < v.n_end; ++i) t.end |= v.end[i] == id;
    if (t.end) t.len = 0;
  }
  if (t.len > 0) held_bytes(v, t.lo, t.len, t.bytes);
  return t;
}

// Masks of states over a tile of kTile tokens, which a workgroup holds in LDS
// with the automaton, its tokens ordered by their first column.
//
// A state of a grammar mostly goes on from one byte in a hundred, so nearly all
// walks would end at their first byte.  A wave takes one state at a time and
// walks the tokens of the columns alone that the state goes on from, runs of
// neighbouring columns together, 64 tokens abreast; those that are allowed set
// their bit in the wave's words in LDS, which then go out whole.  Waves take
// states as they become free, since some (inside a string) allow most tokens.
//
// 1500 states of an automaton of 1474 by 37, V=128256: 65 us, 24 MB written.
// Vector instructions issue in half of the time (218 of them, 94 scalar and 50
// LDS instructions a state and tile); the waves, 4 on a SIMD, wait in 54% of
// their cycles, by the code mostly for LDS lookups one after another.  With the
// table in global memory (1799 to 7322 states by 37) 97 us.  20 states, V=32000:
// 12.6 us, the table's and the tokens' loads and one state that allows most of a
// tile.  Steps: a lane for each token and state,
// the table in global memory, 803 us; in LDS, four states abreast, 309; tokens by
// first column within 1024, a wave's states tested together, 186; this order with
// a test of each token's length in each step, 115; the end() column instead, 66.
// Tokens longer than kHeld bytes have a run of their own: finished one by one
// inside the others', they took as long as all the rest.
constexpr int kTile = 2048;
constexpr int kStates = 512;  // states that a workgroup has at hand
constexpr int kAbreast = 4;   // 64s of tokens whose lookups overlap (2: 71, 8: 65 us of then 65)
template <int kEntries, int kParts>
__global__ __launch_bounds__(kThreads) void k_masks(GrammarArgs a, const int32_t* states, int n,
                                                    int part, uint32_t* bits) {
  constexpr int kWords = kTile / 32, kEach = kTile / kThreads, kPart = kTile / kParts;
  static_assert(kWords == kWave, "a word a lane");
  __shared__ uint16_t lds[kEntries ? kEntries : 1];
  __shared__ uint16_t column[256];
  __shared__ __attribute__((aligned(16))) uint8_t columns[kTile][kHeld];
  __shared__ uint16_t places[kTile];  // in the tile
  __shared__ uint8_t lens[kEntries ? 1 : kTile];  // kHeld for longer ones; for walks without end()
  __shared__ uint32_t words[kWaves][kWords];
  __shared__ uint32_t ends[kWords];  // the tile's end tokens
  constexpr int kLong = 256, kNone = 257;  // after the columns
  __shared__ uint32_t begins[kParts][kNone + 1];  // where each column's tokens begin
  __shared__ int32_t from_state[kStates];  // states in work, -1 where every token is allowed
  __shared__ bool accepts[kStates];
  __shared__ int next;  // the first that no wave has taken
  const int lane = __lane_id();
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int W = (a.v.V + 31) / 32, tile = blockIdx.x;
  int k0 = blockIdx.y * part;
  const int k1 = n - k0 < part ? n : k0 + part;
  // the tokens' loads go ahead of the table's
  int len[kEach];
  uint8_t held[kEach][kHeld];
  {
    int lo[kEach];
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      const int id = min(tile * kTile + e * kThreads + (int)threadIdx.x, a.v.V - 1);
      lo[e] = offset_of(a.v, id);
      len[e] = offset_of(a.v, id + 1);
    }
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      len[e] -= lo[e];
      if (tile * kTile + e * kThreads + (int)threadIdx.x >= a.v.V) len[e] = 0;
      if (len[e] > 0) held_bytes(a.v, lo[e], len[e], held[e]);
    }
  }
  const Table<kEntries, true> table(a.g, lds);
  columns_of(a.g, column);
  for (int i = threadIdx.x; i < kParts * (kNone + 1); i += kThreads) (&begins[0][0])[i] = 0;
  if (threadIdx.x < kWords) ends[threadIdx.x] = 0;
  __syncthreads();

  // the tile's tokens by first column, then the long ones, then those that
  // nothing allows (no bytes, or one that every state refuses)
  {
    if (threadIdx.x < (unsigned)a.v.n_end) {
      const int i = a.v.end[threadIdx.x] - tile * kTile;
      if (i >= 0 && i < kTile && i + tile * kTile < a.v.V) atomicOr(ends + i / 32, 1u << (i % 32));
    }
    int first[kEach];
    uint32_t rank[kEach];
    __syncthreads();
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      const int i = e * kThreads + (int)threadIdx.x;
      if ((ends[i / 32] >> (i % 32)) & 1) len[e] = 0;
#pragma unroll
      for (int k = 0; k < kHeld; ++k) {
        const int c = k < len[e] ? column[held[e][k]] : table.end();
        held[e][k] = (uint8_t)c;
        if (c == kRefused) len[e] = 0;
      }
      first[e] = len[e] > kHeld ? kLong : len[e] > 0 ? held[e][0] : kNone;
      rank[e] = atomicAdd(&begins[i / kPart][first[e]], 1u);
    }
    __syncthreads();
    if (wave < kParts) {
      uint32_t* begin = begins[wave];
      uint32_t before = wave * kPart;
      for (int c0 = 0; c0 <= kNone; c0 += kWave) {
        const uint32_t x = c0 + lane <= kNone ? begin[c0 + lane] : 0;
        const uint32_t upto = wave_incl_scan(x);
        if (c0 + lane <= kNone) begin[c0 + lane] = before + upto - x;
        before += lane_read(upto, kWave - 1);
      }
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      const int i = e * kThreads + (int)threadIdx.x;
      const int p = begins[i / kPart][first[e]] + rank[e];
      places[p] = (uint16_t)i;
      if constexpr (!kEntries) lens[p] = (uint8_t)min(len[e], kHeld);
      __builtin_memcpy(__builtin_assume_aligned(columns[p], 16), held[e], kHeld);
    }
    __syncthreads();
  }

  uint32_t* mine = words[wave];

  // N times 64 tokens from p on, those before p1, from state place from on
  auto walk = [&](int from, int p, int p1, auto abreast, auto tails) {
    constexpr int N = decltype(abreast)::value;
    constexpr bool kTails = decltype(tails)::value;  // tokens longer than kHeld
    int place[N], s[N];
    [[maybe_unused]] int len[N];
    uint32_t c[N][kHeld / 4];
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int q = min(p + j * kWave + lane, p1 - 1);
      __builtin_memcpy(c[j], __builtin_assume_aligned(columns[q], 16), kHeld);
      place[j] = places[q];
      if constexpr (!kEntries) len[j] = lens[q];
      s[j] = p + j * kWave + lane < p1 ? from : table.dead();
    }
    until<kHeld>([&](auto k) {
      bool live = false;
      int least = INT_MAX;
#pragma unroll
      for (int j = 0; j < N; ++j) {
        // (a branch here would keep the lookups from overlapping)
        const int to = table.step(s[j], (c[j][k / 4] >> (8 * (k % 4))) & 0xFF);
        if constexpr (kEntries) {
          s[j] = to;
          least = min(least, to);
        } else {
          s[j] = k < len[j] ? to : s[j];
          live |= k + 1 < len[j] && s[j] != table.dead();
        }
      }
      if constexpr (kEntries) live = least < table.dead();
      return __any(live) != 0;
    });
#pragma unroll
    for (int j = 0; j < N; ++j) {
      if (kTails && s[j] != table.dead()) {
        const int id = tile * kTile + place[j];
        const int at = offset_of(a.v, id), end = offset_of(a.v, id + 1);
        for (int b = at + kHeld; b < end && s[j] != table.dead(); b += kHeld) {
          uint8_t y[kHeld];
          int then[kHeld];
          held_bytes(a.v, b, end - b, y);
#pragma unroll
          for (int k = 0; k < kHeld; ++k) then[k] = column[y[k]];
#pragma unroll
          for (int k = 0; k < kHeld; ++k) {
            const int to = table.step(s[j], then[k] == kRefused ? 0 : then[k]);
            if (k < end - b) s[j] = then[k] == kRefused ? table.dead() : to;
          }
        }
      }
      if (s[j] != table.dead()) atomicOr(mine + place[j] / 32, 1u << (place[j] % 32));
    }
  };

  for (; k0 < k1; k0 += kStates) {
    const int count = min(k1 - k0, kStates);
    __syncthreads();
    if (threadIdx.x < (unsigned)count) {
      const int state = states[k0 + threadIdx.x];
      const bool in = state >= 0 && state < a.g.n_states;
      from_state[threadIdx.x] = in ? state : -1;
      accepts[threadIdx.x] = in && a.g.accept[state] != 0;
    }
    if (threadIdx.x == 0) next = 0;
    __syncthreads();
    for (;;) {
      int k = 0;
      if (lane == 0) k = atomicAdd(&next, 1);
      k = __builtin_amdgcn_readfirstlane(k);
      if (k >= count * kParts) break;
      const uint32_t* begin = begins[k % kParts];
      const int word = k % kParts * (kWords / kParts) + lane;  // the lane's, within the tile
      const int w = tile * kWords + word, left = a.v.V - w * 32;  // tokens from it on
      k /= kParts;
      const int state = __builtin_amdgcn_readfirstlane(from_state[k]);
      uint32_t x = left < 32 ? (1u << max(left, 0)) - 1 : ~0u;
      if (state >= 0) {
        const int from = table.at(state);
        mine[lane] = 0;
        for (int c0 = 0; c0 < a.g.n_classes; c0 += kWave) {
          uint64_t on = __ballot(c0 + lane < a.g.n_classes &&
                                 table.step(from, c0 + lane) != table.dead());
          while (on != 0) {
            const int lo = __builtin_ctzll(on);
            const uint64_t rest = ~(on >> lo);
            const int run = rest != 0 ? __builtin_ctzll(rest) : kWave - lo;
            on = lo + run < kWave ? on & (~0ull << (lo + run)) : 0;
            int p = __builtin_amdgcn_readfirstlane(begin[c0 + lo]);
            const int p1 = __builtin_amdgcn_readfirstlane(begin[c0 + lo + run]);
            for (; p1 - p > kWave; p += kAbreast * kWave)
              walk(from, p, p1, std::integral_constant<int, kAbreast>(), std::false_type());
            if (p < p1) walk(from, p, p1, std::integral_constant<int, 1>(), std::false_type());
          }
        }
        const int tails = __builtin_amdgcn_readfirstlane(begin[kNone]);
        for (int p = __builtin_amdgcn_readfirstlane(begin[kLong]); p < tails; p += kWave)
          walk(from, p, tails, std::integral_constant<int, 1>(), std::true_type());
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        if (lane < kWords / kParts) x = mine[word] | (accepts[k] ? ends[word] : 0);
      }
      if (lane < kWords / kParts && w < W) bits[(size_t)(k0 + k) * W + w] = x;
    }
  }
}

// A session's tokens: a wave holds 64 of them, one a lane, and walks them one
// after another, every lane alike; the chain of lookups is what it waits for.
// 8 drafts of 256 sessions: 8.6 us, of which 4 to bring a table of 109 KB to
// LDS; 64 drafts of 1024 sessions, up to 400 bytes each: 18.7 us.  Automata that
// do not fit take 7.3 and 28 us (nothing to bring, lookups slower).  One lane a
// session with the table in global memory took 16 and 103 us.
template <int kEntries>
__global__ __launch_bounds__(kThreads) void k_walk(GrammarArgs a, const int32_t* states,
                                                   const int32_t* tokens, const int32_t* lens,
                                                   int B, int L, int32_t* out, int32_t* last) {
  __shared__ uint16_t lds[kEntries ? kEntries : 1];
  __shared__ uint16_t column[256];
  const int lane = __lane_id();
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int b = blockIdx.x * kWaves + wave;
  // the tokens' loads go ahead of the table's
  int from = -1, n = 0;
  Token t = {};
  if (b < B) {
    from = states[b];
    n = lens ? lens[b] : L;
    n = n < 0 ? 0 : n > L ? L : n;
    t = token_of(a.v, lane < n ? tokens[(size_t)b * L + lane] : -1);
  }
  const Table<kEntries, false> table(a.g, lds);
  columns_of(a.g, column);
  __syncthreads();
  if (b >= B) return;
  const bool in = from >= 0 && from < a.g.n_states;
  int s = in ? table.at(from) : table.dead();
  out += (size_t)b * (L + 1);
  if (lane == 0) out[0] = in ? from : -1;
  for (int i0 = 0; i0 < L; i0 += kWave) {
    const int held = n - i0 < kWave ? n - i0 : kWave;  // may be 0 or less
    if (i0 > 0) t = token_of(a.v, lane < held ? tokens[(size_t)b * L + i0 + lane] : -1);
    // its first bytes' columns, two to a word; a token with a byte that every
    // state refuses counts as one without bytes
    uint32_t columns[kHeld / 2];
    bool refused = false;
#pragma unroll
    for (int k = 0; k < kHeld; k += 2) {
      const uint32_t c0 = column[t.bytes[k]], c1 = column[t.bytes[k + 1]];
      refused |= (k < t.len && c0 == kRefused) || (k + 1 < t.len && c1 == kRefused);
      columns[k / 2] = c0 | c1 << 16;
    }
    if (refused) t.len = 0;
    int mine = table.dead();
    for (int i = 0; i < held && s != table.dead(); ++i) {
      const int len = lane_read(t.len, i);
      if (len == 0) {
        s = table.dead();
        break;
      }
      until<kHeld>([&](auto k) {
        const uint32_t c = lane_read(columns[k / 2], i);
        s = table.step(s, k % 2 ? c >> 16 : c & 0xFFFF);
        return k + 1 < len;
      });
      if (len > kHeld) {
        const int lo = lane_read(t.lo, i);
        for (int k0 = kHeld; k0 < len && s != table.dead(); k0 += kWave) {
          // the next 64 bytes' columns, one a lane
          const int c = k0 + lane < len ? column[a.v.bytes[lo + k0 + lane]] : kRefused;
          for (int k = 0; k < kWave && k0 + k < len; ++k) {
            const int next = lane_read(c, k);
            s = next == kRefused ? table.dead() : table.step(s, next);
          }
        }
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
  if (Table<8192, true>::fits(g)) f(std::integral_constant<int, 8192>());
  else if (Table<kMostEntries, true>::fits(g)) f(std::integral_constant<int, kMostEntries>());
  else f(std::integral_constant<int, 0>());
}

bool grammar_ok(const sv_grammar* g, const sv_vocab* v) {
  if (!g || !g->next || !g->classes || !g->accept || g->n_states < 1 || g->n_classes < 1 ||
      g->n_classes > 256)
    return false;
  if (!v || !v->offsets || v->n_bytes < 0 || v->n_bytes > SV_ENTRIES_MAX || (v->n_bytes > 0 && !v->bytes) || v->n_end < 0 ||
      v->n_end > SV_STOP_MAX || (v->n_end > 0 && !v->end) || v->V < 1 || v->V > SV_V_MAX)
    return false;
  return true;
}

}  // namespace
}  // namespace sv

extern "C" int sv_grammar_masks(const sv_grammar* grammar, const sv_vocab* vocab,
                                const int32_t* states, int32_t n, uint32_t* bits, void* stream) {
  using namespace sv;
  if (!grammar_ok(grammar, vocab) || !states || !bits || n < 1 || n > SV_ENTRIES_MAX)
    return SV_ERR_ARG;
  GrammarArgs a = {*grammar, *vocab};
  (void)hipGetLastError();
  by_size(*grammar, [&](auto entries) {
    constexpr int kEntries = decltype(entries)::value;
    // each tile's states go to as many workgroups as fill the card, of a few
    // states a wave
    const int64_t tiles = (vocab->V + kTile - 1) / kTile, places = kEntries > 8192 ? 256 : 512;
    auto launch = [&](auto tile_parts) {
      constexpr int kParts = decltype(tile_parts)::value;
      int64_t parts = places > tiles ? places / tiles : 1;
      const int64_t most = ((int64_t)n * kParts + kWaves - 1) / kWaves;
      parts = parts < most ? parts : most;
      const int64_t part = (n + parts - 1) / parts;
      const dim3 grid((unsigned)tiles, (unsigned)((n + part - 1) / part));
      hipLaunchKernelGGL((k_masks<kEntries, kParts>), grid, dim3(kThreads), 0, (hipStream_t)stream,
                         a, states, n, (int)part, bits);
    };
    // few units: a quarter of a tile each, so that the longest, a state that allows
    // most tokens, ends sooner (V=32000: 24.4 against 27.0 us for 400 states of 60
    // members' objects, 37.1 against 32.8 for 1000; 12.7 against 16.3 for 20)
    if (n * tiles <= 8192) launch(std::integral_constant<int, 4>());
    else launch(std::integral_constant<int, 1>());
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
    hipLaunchKernelGGL(k_walk<decltype(entries)::value>, dim3((B + kWaves - 1) / kWaves),
                       dim3(kThreads), 0, (hipStream_t)stream, a, states, tokens, lens, B, L,
                       out_states, last);
  });
  return hipGetLastError() == hipSuccess ? SV_OK : SV_ERR_DEVICE;
}
