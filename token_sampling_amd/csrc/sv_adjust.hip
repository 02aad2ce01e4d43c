// sv_adjust.hip -- sv_adjust_logits: penalties for repeated tokens, biases and
// vocabulary masks on a round's logits, in one pass.
//
// For token v of row r of a session with count c (stored output count plus how
// often v is among the drafted tokens before the row):
//   z = v seen ? (z > 0 ? z / rep : z * rep) : z
//   z = z - freq * c - (c > 0 ? pres : 0) + bias(v)
//   z = mask bit clear ? -inf : z
// in binary32, rounded once to the logits' type; as z * f + t, with f the rounded
// 1 / rep or rep, and t the bias less the penalties (3 roundings of 2^-24 of the
// terms' magnitudes at most).
#include <limits.h>
#include <math.h>

#include <type_traits>

#include "sv_common.hpp"

namespace sv {
namespace {

// Waves to fill the card with, half its places (B=64, R=5, V=32000: 12.5 us, with
// 8192 14.2; B=64, R=65, V=1300: 18.2 and 17.7).
constexpr int64_t kWantedWaves = 4096;
// Most rows of a wave that streams them: longer ones end late (192 sessions of up
// to 17 rows, V=151935: 184 us, uncut 191, by 6 rows 191; 32 sessions of 65 rows,
// V=128256: 177, uncut 193).  Even rows cut in two set up twice, and gain or lose
// little by it: 10, 12, 14, 16 rows of 256 sessions, V=128256, take 191, 218, 257,
// 289 us, uncut 195, 218, 263, 295; of 1024 sessions, V=32000, 194, 228, 267, 285,
// uncut 187, 225, 267, 290 (each +-2% from run to run).
constexpr int kMostRows = 9;
constexpr int kGridY = 32768;           // sessions of a launch
constexpr int kXcds = 8;
constexpr int kBatch = 4;               // logits of a lane in flight, in place
constexpr int kTurns = 4;               // turns over a tile's listed tokens whose reads overlap

__device__ uint32_t nothing[4];  // where a vector that is not needed comes from

struct AdjustArgs {
  const void* logits;
  int64_t in_session, in_row;
  void* out;
  int64_t out_session, out_row;
  const int32_t* tokens;
  const int32_t* m;
  const sv_penalties* pen;
  const int32_t* counts;
  const uint32_t* seen;
  const int32_t* slots;
  int32_t n_slots;
  const int32_t* bias_off;
  const int32_t* bias_id;
  const float* bias_val;
  int32_t n_bias;
  const uint32_t* mask_bits;
  const int32_t* mask_rows;
  int32_t n_masks;
  int32_t B, M, R, V, W;
  int32_t chunk;  // rows of a unit of work
  int32_t b0;     // the launch's first session
  int32_t* status;
};

typedef unsigned int u32x4 __attribute__((ext_vector_type(4), may_alias));
// a vector at any logit's address
typedef unsigned int u32x4_any __attribute__((ext_vector_type(4), aligned(2), may_alias));
__device__ inline u32x4 load16(const void* p) {
  return __builtin_nontemporal_load((const u32x4_any*)p);
}
__device__ inline void store16(void* p, u32x4 v) {
  __builtin_nontemporal_store((u32x4_any)v, (u32x4_any*)p);
}

// A lane's share of a row: one 16-byte vector per group, 8 bf16 or 4 binary32
// logits, 64 lanes side by side.
template <typename T>
struct Lanes {
  static constexpr int kE = 16 / (int)sizeof(T);  // logits of a vector
  static constexpr int kGroup = kWave * kE;       // logits of a group
};

// Groups of a tile, which holds kSize * 512 logits.
template <typename T>
constexpr int groups(int size) {
  return size * (int)sizeof(T) / 2;
}

__device__ inline void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// What a wave knows of its session; every lane of the wave takes part.
struct Session {
  int32_t status;
  int m, slot;
  int32_t token;      // lane i: x_{i+1}, -1 past m
  int32_t mask_row;   // lane r: the mask of row r
  int32_t mask_row64; // row 64's
  int bias_lo, bias_hi;
  float repetition, frequency, presence;
};

// All of a session's controls come with three loads that do not wait for each
// other: lane by lane the single values, the drafted tokens, the rows' masks.
__device__ inline Session session_of(const AdjustArgs& a, int b) {
  const int lane = __lane_id();
  const int32_t* p = nullptr;
  if (lane == 0 && a.m) p = a.m + b;
  if (lane == 1 && a.slots) p = a.slots + b;
  if (lane >= 2 && lane < 6 && a.pen) p = (const int32_t*)(a.pen + b) + (lane - 2);
  if (lane >= 6 && lane < 8 && a.bias_off) p = a.bias_off + b + (lane - 6);
  if (lane == 8 && a.mask_rows && a.R > kWave) p = a.mask_rows + (size_t)b * a.R + kWave;
  int32_t value = 0, token = -1, mask_row = -1;
  if (p) value = *p;
  if (a.pen && lane < a.M) token = a.tokens[(size_t)b * a.M + lane];
  if (a.mask_rows && lane < a.R) mask_row = a.mask_rows[(size_t)b * a.R + lane];

  Session s;
  s.m = a.m ? lane_read(value, 0) : a.M;
  s.slot = a.counts == nullptr ? -1 : a.slots ? lane_read(value, 1) : b;
  s.repetition = a.pen ? __builtin_bit_cast(float, lane_read(value, 2)) : 1.f;
  s.frequency = __builtin_bit_cast(float, lane_read(value, 3));
  s.presence = __builtin_bit_cast(float, lane_read(value, 4));
  s.bias_lo = lane_read(value, 6);
  s.bias_hi = lane_read(value, 7);
  const int rows = s.m + (a.R - a.M);
  s.mask_row = lane < rows ? mask_row : -1;
  s.mask_row64 = a.mask_rows && rows > kWave ? lane_read(value, 8) : -1;
  s.token = lane < s.m ? token : -1;
  // a reciprocal of a repetition within these bounds is a normal number
  const bool bad =
      !(s.repetition >= 0x1p-64f && s.repetition <= 0x1p64f) || !isfinite(s.frequency) ||
      !isfinite(s.presence) || (a.pen && lane_read(value, 5) != 0) || s.slot < -1 ||
      (a.counts != nullptr && s.slot >= a.n_slots) || s.bias_lo < 0 || s.bias_hi < s.bias_lo ||
      s.bias_hi > a.n_bias || s.mask_row < -1 || (a.mask_rows && s.mask_row >= a.n_masks) ||
      s.mask_row64 < -1 || (a.mask_rows && s.mask_row64 >= a.n_masks);
  const bool bad_token = a.pen && lane < s.m && (token < 0 || token >= a.V);
  s.status = s.m < 0 || s.m > a.M ? SV_S_LIMIT
             : __any(bad)         ? SV_S_BAD_CONTROL
             : __any(bad_token)   ? SV_S_BAD_PROPOSAL
                                  : 0;
  return s;
}

// Narrows ascending ids[lo, hi) to a range with every id of [v, v + n): 64
// probes, which tell the entries before the last probe below v and after the
// first one not below v + n, as often as that halves the range.
__device__ inline void narrow(const int32_t* ids, int& lo, int& hi, int v, int n) {
  while (hi - lo > kWave) {
    const int step = (hi - lo + kWave - 1) / kWave;
    const int64_t at = lo + (int64_t)__lane_id() * step;
    const int id = at < hi ? ids[at] : INT_MAX;
    const int below = __popcll(__ballot(id < v)), upto = __popcll(__ballot(id < v + n));
    const int64_t end = lo + (int64_t)upto * step;
    const int was = hi - lo;
    if (below > 0) lo += (below - 1) * step + 1;
    if (end < hi) hi = (int)end;
    if (hi - lo > was / 2) return;
  }
}

// All ones where bit i of bits is set, else zeros.
__device__ inline uint32_t spread(uint32_t bits, int i) {
  return (uint32_t)__builtin_amdgcn_sbfe((int)bits, i, 1);
}

// Word d of a vector's selection: the elements whose bits are set.
__device__ inline uint32_t select_word(uint32_t bits, int d, __bf16) {
  return (spread(bits, 2 * d) & 0xFFFFu) | (spread(bits, 2 * d + 1) & 0xFFFF0000u);
}
__device__ inline uint32_t select_word(uint32_t bits, int d, float) { return spread(bits, d); }

// A logit's bits, zero-extended, and its value: the wait for the load comes with
// the second.
__device__ inline uint32_t load_bits(const __bf16* p) { return *(const uint16_t*)p; }
__device__ inline uint32_t load_bits(const float* p) { return *(const uint32_t*)p; }
__device__ inline float from_bits(uint32_t x, __bf16) { return __builtin_bit_cast(float, x << 16); }
__device__ inline float from_bits(uint32_t x, float) { return __builtin_bit_cast(float, x); }

template <typename T>
constexpr uint32_t kMinusInf = sizeof(T) == 2 ? 0xFF80FF80u : 0xFF800000u;

// What a token without a bias has for one: -0, which leaves every logit as it is (+0
// would make a logit of -0 another).
constexpr float kNoBias = -0.f;

// What a token's logit gets added: its bias, less its penalties at count c.
__device__ inline float term_of(const Session& s, float bias, int c) {
  return c > 0 ? bias - fmaf(s.frequency, (float)c, s.presence) : bias;
}

// A touched token of a tile, 16 bits: its place in the tile and
constexpr uint32_t kPlace = 0x0FFF;
constexpr uint32_t kRep = 0x1000;   // seen: the repetition penalty applies
constexpr uint32_t kHad = 0x2000;   // output before: its presence is counted
constexpr uint32_t kOn = 0x4000;    // a rule changes it (not yet, for a drafted token ahead)
constexpr uint32_t kBias = 0x8000;  // it has a bias

// One wave, a workgroup of its own, works on kTile neighbouring tokens of one
// session, row after row.  What the rows share is set up once, in LDS: the list
// of the tokens that the history, a bias or a drafted token touches, and an
// additive term for each.  Then the rows stream in 16-byte vectors; vectors that
// hold listed tokens pass through LDS, where one lane a listed token changes it,
// and vectors with an empty mask are not read.  In place, the vectors that change
// move; where the call has no masks, listed tokens alone, lanes spread over tokens
// and rows.
//
// What bounds it.  Out of place, HBM: 159 to 165 us at B=256, M=8, V=128256 bf16 with
// every rule, where half the masks leave a few tokens (0.58 GB written, 0.16 to
// 0.6 GB read); 61 us for one binary32 row of 256 sessions at V=129280 (277 MB,
// 4.5 TB/s).  In place, the same 256 sessions without masks take 98 us for 0.18
// GB in scattered 64-byte pieces; two vectors a lane, which also halve the waves
// in flight, or more rows of a lane's in flight do not shorten it.  Its waves, 8 on
// a SIMD, wait in 69% of their cycles: for the chain of their setup or for the
// pieces, which the counters do not tell apart.  In place with masks, 180 us for
// 706 MB.  Small batches, the chain of dependent loads (controls; history bits,
// masks, biases; counts; logits), 5 us.
// Why so.
//  - Lanes that each work out their own vector's changes take 200 vector
//    instructions a row and tile against 60 here; in place they were the bound.
//  - All of a session's controls come with three loads, and everything that
//    hangs on them alone with the next few: one after another, they made a wave
//    wait 13 us.
//  - Workgroups of four waves hold their LDS until the last one ends: 230 us
//    where single waves took 202.
//  - Loads and stores are non-temporal, since a row is met once: 202 to 188 us,
//    and the acceptance step that reads the rows next is 15% faster too.
//  - The next row's vectors and the mask of the row after it are on the way while
//    a row is worked on, with no load passed over, so that the compiler's waits
//    are for single loads: 188 to 159 us.
// Scalar registers run out in the kernels of two vectors (4 spilled to lanes of a
// vector register without masks, 13 with them) and in place with masks (10).
template <typename T, int kSize, bool kInPlace, bool kMasks>
__global__ __launch_bounds__(kWave) void k_adjust(AdjustArgs a) {
  using L = Lanes<T>;
  constexpr int G = groups<T>(kSize), E = L::kE, kTile = G * L::kGroup;
  constexpr uint32_t kAll = (1u << E) - 1;  // one vector's tokens
  constexpr uint32_t kFull = G * E == 32 ? ~0u : (1u << (G * E)) - 1;
  static_assert(G * E <= 32 && kTile <= (int)kPlace + 1, "a lane's tokens fit one word");
  constexpr bool kVectors = !kInPlace || kMasks;  // whole vectors move
  __shared__ __attribute__((aligned(16))) T raw[kTile];
  __shared__ float term[kTile];
  __shared__ uint16_t list[kTile];
  __shared__ uint32_t bits[kTile / 32];
  const int lane = __lane_id();
  int tile = blockIdx.x;
  if constexpr (kSize == 2) {
    // uneven rows: neighbouring tiles to one XCD (workgroups go to them in turn),
    // whose L2 then has the lines that they share (197 to 191 us for 192 sessions
    // of up to 17 rows, V=151935; even rows lose 2% by it)
    const int nth = tile % kXcds, each = gridDim.x / kXcds, over = gridDim.x % kXcds;
    tile = nth * each + min(nth, over) + tile / kXcds;
  }
  const int v0 = tile * kTile;
  const int first = lane * E;   // a lane's vectors start at first + g * kGroup
  const int left = a.V - v0;    // tokens from the tile's start to the row's end
  const int chunk = blockIdx.z;
  uint32_t within = 0;  // a lane's tokens that the row has
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const int n = left - g * L::kGroup - first;
    within |= (n >= E ? kAll : n > 0 ? (1u << n) - 1 : 0u) << (g * E);
  }

  const int b = a.b0 + blockIdx.y;
  const Session s = session_of(a, b);
  if (a.status && tile == 0 && chunk == 0 && lane == 0) a.status[b] = s.status;
  const int rows = s.status == 0 ? s.m + (a.R - a.M) : a.R;
  const int r0 = chunk * a.chunk, r1 = r0 + a.chunk < rows ? r0 + a.chunk : rows;
  if (r0 >= r1) return;
  const T* in = (const T*)a.logits + b * a.in_session + v0;
  T* out = (T*)a.out + b * a.out_session + v0;
  if (s.status != 0) {
    for (int r = r0; r < r1; ++r)
      for (int i = lane; i < kTile && i < left; i += kWave)
        out[r * a.out_row + i] = (T)__builtin_nanf("");
    return;
  }

  // A lane's bits of a bit row over the vocabulary: the bytes that hold them,
  // and those packed vector by vector, none past the row's end.
  struct Bytes {
    uint32_t of[G];
  };
  auto bytes_of = [&](const uint32_t* words) {
    Bytes y;
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const int v = v0 + g * L::kGroup + first;
      y.of[g] = ((const uint8_t*)words)[(v < a.V ? v : a.V - 1) / 8];
    }
    return y;
  };
  auto packed = [&](const Bytes& y) {
    uint32_t w = 0;
#pragma unroll
    for (int g = 0; g < G; ++g) w |= ((y.of[g] >> (first % 8)) & kAll) << (g * E);
    return w & within;
  };
  auto mask_row = [&](int r) {
    if (!kMasks || r >= r1) return -1;
    return r < kWave ? lane_read(s.mask_row, r) : s.mask_row64;
  };
  auto mask_of = [&](int k) {
    return k < 0 ? kFull : packed(bytes_of(a.mask_bits + (size_t)k * a.W));
  };
  auto load = [&](int r, uint32_t mk, uint32_t needed, u32x4 (&x)[G]) {
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const int i = g * L::kGroup + first;
      x[g] = u32x4{0, 0, 0, 0};
      if (((mk >> (g * E)) & kAll) != 0 && ((needed >> (g * E)) & kAll) != 0 && i < left) {
        const T* p = in + r * a.in_row + i;
        if (i + E <= left) {
          x[g] = load16(p);
        } else {
          T t[E];
#pragma unroll
          for (int k = 0; k < E; ++k) t[k] = i + k < left ? p[k] : T(0);
          __builtin_memcpy(&x[g], t, 16);
        }
      }
    }
  };

  // The same for a tile that the row has all of, rows past the last included:
  // vectors that are not needed come from nothing, so that every lane loads.
  [[maybe_unused]] auto load_whole = [&](int r, uint32_t mk, uint32_t needed, u32x4 (&x)[G]) {
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const bool wanted = r < r1 && ((mk >> (g * E)) & kAll) != 0 &&
                          ((needed >> (g * E)) & kAll) != 0;
      x[g] = load16(wanted ? in + r * a.in_row + g * L::kGroup + first : (const T*)nothing);
    }
  };
  // A row's mask bytes on the way.
  struct Ahead {
    bool masked;
    Bytes bytes;
  };
  [[maybe_unused]] auto mask_ahead = [&](int r) {
    Ahead h = {};
    if constexpr (kMasks) {
      const int k = mask_row(r);
      h.masked = k >= 0;
      const uint8_t* row = h.masked ? (const uint8_t*)(a.mask_bits + (size_t)k * a.W) + v0 / 8
                                    : (const uint8_t*)nothing;
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const int i = g * L::kGroup + first;
        h.bytes.of[g] = row[h.masked && i < left ? i / 8 : 0];
      }
    }
    return h;
  };
  [[maybe_unused]] auto ahead_of = [&](const Ahead& h) { return h.masked ? packed(h.bytes) : kFull; };

  // ---- what the rows share; loads first
  Bytes prompt = {}, output = {}, mask = {};
  if (s.slot >= 0) {
    const uint32_t* seen = a.seen + (size_t)s.slot * 2 * a.W;
    prompt = bytes_of(seen);
    output = bytes_of(seen + a.W);
  }
  const int mask0 = mask_row(r0);
  if (mask0 >= 0) mask = bytes_of(a.mask_bits + (size_t)mask0 * a.W);
  int bias_lo = s.bias_lo, bias_hi = s.bias_hi;
  narrow(a.bias_id, bias_lo, bias_hi, v0, kTile);
  int32_t id = -1;
  float bias = 0.f;
  if (bias_lo + lane < bias_hi) {
    id = a.bias_id[bias_lo + lane];
    bias = a.bias_val[bias_lo + lane];
  }
  u32x4 x[G];
  [[maybe_unused]] Ahead ahead = {};
  if constexpr (!kInPlace) ahead = mask_ahead(r0 + 1);
  uint32_t mk = mask0 < 0 ? kFull : packed(mask);
  if constexpr (!kInPlace) {
    if (left >= kTile) load_whole(r0, mk, kFull, x);
    else load(r0, mk, kFull, x);
  }

  const uint32_t had = packed(output), rep = packed(prompt) | had;
  // drafted tokens of this tile that rows before r1 meet
  const uint64_t mine = __ballot(s.token >= v0 && s.token - v0 < kTile && lane < r1 - 1);
  uint32_t biased = 0, any = rep;
  auto here = [&](int v) { return v >= v0 && v < a.V && v - v0 < kTile; };
  if (mine != 0 || __any(here(id)) || bias_hi - bias_lo > kWave) {
    for (int w = lane; w < kTile / 32; w += kWave) bits[w] = 0;
    wave_sync();
    for (int e = bias_lo + lane; e < bias_hi; e += kWave) {
      if (e != bias_lo + lane) {
        id = a.bias_id[e];
        bias = a.bias_val[e];
      }
      if (here(id)) {
        atomicOr(bits + (id - v0) / 32, 1u << ((id - v0) % 32));
        term[id - v0] = bias;
      }
    }
    wave_sync();
    auto noted = [&] {
      uint32_t w = 0;
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const int i = g * L::kGroup + first;
        w |= ((bits[i / 32] >> (i % 32)) & kAll) << (g * E);
      }
      return w;
    };
    biased = noted();
    wave_sync();
    if ((mine >> lane) & 1) atomicOr(bits + (s.token - v0) / 32, 1u << ((s.token - v0) % 32));
    wave_sync();
    any |= noted();
  }
  // those before the first row count from the start: 16 bits a token, in raw
  const uint64_t early = r0 < kWave ? mine & ~(~0ull << r0) : mine;
  typedef uint16_t u16_alias __attribute__((may_alias));
  typedef uint32_t u32_alias __attribute__((may_alias));
  const u16_alias* early_count = (const u16_alias*)raw;
  if (early != 0) {
    for (int w = lane; w < kTile / 2; w += kWave) ((u32_alias*)raw)[w] = 0;
    wave_sync();
    if ((early >> lane) & 1)
      atomicAdd((u32_alias*)raw + (s.token - v0) / 2, 1u << (16 * ((s.token - v0) % 2)));
    wave_sync();
  }
  const int count = __popc(any);
  const int upto = wave_incl_scan(count);
  const int listed = lane_read(upto, kWave - 1);
  const int base = upto - count;  // the list has a lane's tokens from here on, in order
  if (listed > 0) {
    int at = base;
    for (uint32_t w = any; w != 0; w &= w - 1) {
      const int k = __builtin_ctz(w);
      const uint32_t bit = 1u << k;
      uint32_t e = (k / E) * L::kGroup + first + k % E;
      if (rep & bit) e |= kRep | kOn;
      if (had & bit) e |= kHad;
      if (biased & bit) e |= kBias | kOn;
      list[at++] = (uint16_t)e;
    }
    wave_sync();
    for (int j = lane; j < listed; j += kWave) {
      uint32_t e = list[j];
      const int i = e & kPlace;
      float t = e & kBias ? term[i] : kNoBias;
      int c = e & kHad ? a.counts[(size_t)s.slot * a.V + v0 + i] : 0;
      if (early != 0) {
        const int more = early_count[i];
        c += more;
        if (more > 0) {
          e |= kRep | kHad | kOn;
          list[j] = (uint16_t)e;
        }
      }
      term[i] = term_of(s, t, c);
    }
    wave_sync();
  }

  // ---- the rows
  const uint64_t masked = __ballot(s.mask_row >= 0);
  const float up = s.repetition, down = 1.f / s.repetition;
  auto changed = [&](float z, uint32_t e, float t) {
    const float f = z > 0.f ? down : up;
    return (e & kRep ? z * f : z) + t;
  };
  auto meet = [&](int d) {  // drafted token d counts from here on
    const int v = lane_read(s.token, d), place = v - v0;
    const int owner = place % L::kGroup / E, k = place / L::kGroup * E + place % E;
    const int j = lane_read(base, owner) + __popc(lane_read(any, owner) & ((1u << k) - 1));
    // the term anew from the count, so that a row's result does not depend on
    // the row its wave began with
    int c = __popcll(__ballot(s.token == v && lane <= d));
    if ((lane_read(had, owner) >> k) & 1) c += a.counts[(size_t)s.slot * a.V + v];
    float t = kNoBias;
    const uint32_t e = list[j];
    if (e & kBias)
      for (int i = bias_lo + lane; i < bias_hi; i += kWave)
        if (a.bias_id[i] == v) t = a.bias_val[i];
    t = wave_reduce(t, OpAdd());
    wave_sync();
    term[place] = term_of(s, t, c);  // every lane the same
    list[j] = (uint16_t)(e | kRep | kHad | kOn);
    wave_sync();
  };

  // Row r from its vectors y: the listed tokens, the mask, and out it goes.  kWhole:
  // the row has all of the tile's tokens.
  auto finish = [&](int r, uint32_t mk, u32x4 (&y)[G], auto whole) {
    constexpr bool kWhole = decltype(whole)::value;
    if (listed > 0) {
#pragma unroll
      for (int g = 0; g < G; ++g)
        if ((any >> (g * E)) & kAll) *(u32x4*)(raw + g * L::kGroup + first) = y[g];
      wave_sync();
      auto turn = [&](int j0, auto turns) {  // whose reads go out together
        constexpr int N = decltype(turns)::value;
        uint32_t e[N];
        float t[N], z[N];
#pragma unroll
        for (int q = 0; q < N; ++q) {
          const int j = j0 + q * kWave + lane;
          e[q] = j < listed ? list[j] : 0;
        }
#pragma unroll
        for (int q = 0; q < N; ++q) {
          t[q] = term[e[q] & kPlace];
          z[q] = (float)raw[e[q] & kPlace];
        }
#pragma unroll
        for (int q = 0; q < N; ++q)
          if (e[q] & kOn) raw[e[q] & kPlace] = (T)changed(z[q], e[q], t[q]);
      };
      int j0 = 0;
      for (; listed - j0 > kWave; j0 += kTurns * kWave)
        turn(j0, std::integral_constant<int, kTurns>());
      if (j0 < listed) turn(j0, std::integral_constant<int, 1>());
      wave_sync();
#pragma unroll
      for (int g = 0; g < G; ++g)
        if ((any >> (g * E)) & kAll) y[g] = *(const u32x4*)(raw + g * L::kGroup + first);
    }
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const int i = g * L::kGroup + first;
      const uint32_t ok = (mk >> (g * E)) & kAll;
      if ((!kWhole && i >= left) || (kInPlace && ((any >> (g * E)) & kAll) == 0 && ok == kAll)) continue;
      if (ok != kAll) {
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          const uint32_t sel = select_word(ok, d, T(0)), w = y[g][d];
          y[g][d] = (w & sel) | (kMinusInf<T> & ~sel);
        }
      }
      T* p = out + r * a.out_row + i;
      if (kWhole || i + E <= left) {
        store16(p, y[g]);
      } else {
        T t[E];
        __builtin_memcpy(t, &y[g], 16);
#pragma unroll
        for (int k = 0; k < E; ++k)
          if (i + k < left) p[k] = t[k];
      }
    }
  };

  // the vectors of a row that move: in place, those that change (any has a bit
  // for each listed token)
  [[maybe_unused]] auto moved = [&](uint32_t ok) { return kInPlace ? any | (ok ^ kFull) : kFull; };
  if constexpr (kVectors) {
    if (left >= kTile) {
      // two rows in turn, the next one's loads on the way while one is worked on;
      // no load or store is passed over, so that each wait is for its own
      if constexpr (kInPlace) {
        ahead = mask_ahead(r0 + 1);
        load_whole(r0, mk, moved(mk), x);
      }
      __builtin_amdgcn_s_waitcnt(0);
      auto half = [&](int r, u32x4 (&x0)[G], uint32_t m0, u32x4 (&x1)[G], uint32_t& m1) {
        if (r > r0 && ((mine >> (r - 1)) & 1)) meet(r - 1);
        m1 = ahead_of(ahead);
        ahead = mask_ahead(r + 2);
        load_whole(r + 1, m1, moved(m1), x1);
        finish(r, m0, x0, std::true_type());
      };
      u32x4 x1[G];
      uint32_t m1;
      for (int r = r0;;) {
        half(r, x, mk, x1, m1);
        if (++r >= r1) break;
        half(r, x1, m1, x, mk);
        if (++r >= r1) break;
      }
      return;
    }
  }
  for (int r = r0; r < r1;) {
    if (r > r0 && ((mine >> (r - 1)) & 1)) meet(r - 1);
    if (!kVectors || (kInPlace && mask_row(r) < 0)) {
      // rows alike: up to the next that meets a token of this tile or has a mask
      int n = r1 - r;
      const uint64_t met = r < kWave ? mine >> r : 0, held = r < kWave ? masked >> r : 0;
      if (met != 0) n = min(n, __builtin_ctzll(met) + 1);
      if (held != 0) n = min(n, __builtin_ctzll(held));
      if (s.mask_row64 >= 0) n = min(n, kWave - r);
      // lanes: 2^p listed tokens by 64 / 2^p rows
      const int p = listed > 32 ? 6 : listed > 1 ? 32 - __builtin_clz(listed - 1) : 0;
      const int step = kWave >> p;
      for (int j = lane & ((1 << p) - 1); j < listed; j += kWave) {
        const uint32_t e = list[j];
        const int i = e & kPlace;
        const float t = term[i];
        if (!(e & kOn)) continue;
        for (int q0 = lane >> p; q0 < n; q0 += kBatch * step) {
          uint32_t z[kBatch];
#pragma unroll
          for (int k = 0; k < kBatch; ++k)
            z[k] = load_bits(in + (r + min(q0 + k * step, n - 1)) * a.in_row + i);
#pragma unroll
          for (int k = 0; k < kBatch; ++k)
            if (q0 + k * step < n)
              out[(r + q0 + k * step) * a.out_row + i] = (T)changed(from_bits(z[k], T(0)), e, t);
        }
      }
      r += n;
      continue;
    }
    if constexpr (kVectors) {
      const uint32_t next = mask_of(mask_row(r + 1));
      if constexpr (kInPlace) {
        mk = mask_of(mask_row(r));
        load(r, mk, moved(mk), x);
      }
      u32x4 y[G];
#pragma unroll
      for (int g = 0; g < G; ++g) y[g] = x[g];
      if constexpr (!kInPlace) {
        if (r + 1 < r1) load(r + 1, next, kFull, x);
      }
      finish(r, mk, y, std::false_type());
      mk = next;
      ++r;
    }
  }
}

template <typename T, int kSize, bool kInPlace, bool kMasks>
void launch(AdjustArgs a, hipStream_t st) {
  constexpr int kTile = groups<T>(kSize) * Lanes<T>::kGroup;
  const int64_t tiles = (a.V + kTile - 1) / kTile;
  // rows go to several waves where a wave per tile would leave the card idle; half
  // as many where rows move their listed tokens alone and the setup is most of the
  // work
  const int64_t wanted = kInPlace && !kMasks ? kWantedWaves / 2 : kWantedWaves;
  int64_t chunks = (wanted + tiles * a.B - 1) / (tiles * a.B);
  if (!kInPlace || kMasks) {
    const int64_t least = (a.R + kMostRows - 1) / kMostRows;
    chunks = chunks > least ? chunks : least;
  }
  chunks = chunks < a.R ? chunks : a.R;
  a.chunk = (int)((a.R + chunks - 1) / chunks);
  chunks = (a.R + a.chunk - 1) / a.chunk;
  for (a.b0 = 0; a.b0 < a.B; a.b0 += kGridY) {
    const dim3 grid((unsigned)tiles, a.B - a.b0 < kGridY ? a.B - a.b0 : kGridY, (unsigned)chunks);
    hipLaunchKernelGGL((k_adjust<T, kSize, kInPlace, kMasks>), grid, dim3(kWave), 0, st, a);
  }
}

// One vector of a row per lane, or two.  One lets twice the waves share the LDS:
// 52.0 against 56.1 us at B=128, R=17, V=32000 and 165 against 174 us at
// V=128256 (bf16, penalties and masks).  Where rows start off a 16-byte
// boundary every tile's ends share cache lines with its neighbours', and two
// vectors have half as many ends: 186 against 202 us for 9 rows of 256 sessions,
// V=128255, in bf16 with every rule, 47 against 54 for one row; in binary32,
// though its kernel has 3 to 4 waves a SIMD, 361 against 379 and 64 against 71.
template <typename T>
void launch(const AdjustArgs& a, hipStream_t st) {
  constexpr int E = Lanes<T>::kE;
  const bool even = (uintptr_t)a.logits % 16 == 0 && (uintptr_t)a.out % 16 == 0 &&
                    a.in_session % E == 0 && a.in_row % E == 0 && a.out_session % E == 0 &&
                    a.out_row % E == 0;
  const bool many = (int64_t)a.B * a.V > 2 * kWantedWaves * Lanes<T>::kGroup;
  if (a.out == a.logits) {
    if (a.mask_rows) launch<T, 1, true, true>(a, st);
    else launch<T, 1, true, false>(a, st);
  } else if (many && !even) {
    if (a.mask_rows) launch<T, 2, false, true>(a, st);
    else launch<T, 2, false, false>(a, st);
  } else {
    if (a.mask_rows) launch<T, 1, false, true>(a, st);
    else launch<T, 1, false, false>(a, st);
  }
}

// Whether no two of the B * R rows of V logits share one: in place, each is written
// by waves of its own.  Rows dr apart within their sessions come nearest where
// the sessions' distance is just below dr * row_stride, or just above it.
bool rows_apart(int64_t session_stride, int64_t row_stride, int B, int R, int V) {
  if (B > 1 && session_stride < V) return false;
  for (int dr = 1; dr < R; ++dr) {
    const int64_t x = dr * row_stride;
    const int64_t db = B == 1 ? 0 : x / session_stride < B ? x / session_stride : B - 1;
    if (x - db * session_stride < V) return false;
    if (db + 1 < B && (db + 1) * session_stride - x < V) return false;
  }
  return true;
}

}  // namespace
}  // namespace sv

extern "C" int sv_adjust_logits(const void* logits, int64_t session_stride, int64_t row_stride,
                                int32_t dtype, const int32_t* draft_tokens, const int32_t* m,
                                const sv_penalties* penalties, const sv_history* history,
                                const int32_t* slots, const sv_bias* bias, const sv_masks* masks,
                                int32_t B, int32_t M, int32_t R, int32_t V, void* out,
                                int32_t* status, void* stream) {
  using namespace sv;
  if (!logits || !out || (dtype != SV_BF16 && dtype != SV_FP32)) return SV_ERR_ARG;
  if (B < 1 || B > SV_B_MAX || M < 0 || M > SV_M_MAX || R < 1 || (R != M && R != M + 1) || V < 1 ||
      V > SV_V_MAX)
    return SV_ERR_ARG;
  // element offsets stay within a signed 64-bit index
  if (session_stride < 0 || row_stride < 0 || session_stride > (int64_t)1 << 40 ||
      row_stride > (int64_t)1 << 40)
    return SV_ERR_ARG;
  if (out == logits && !rows_apart(session_stride, row_stride, B, R, V)) return SV_ERR_ARG;
  if (M > 0 && penalties && !draft_tokens) return SV_ERR_ARG;
  if (history && (!history->counts || !history->seen || history->n_slots < 1 ||
                  (!slots && history->n_slots < B)))
    return SV_ERR_ARG;
  if (bias && (!bias->offsets || bias->n < 0 || bias->n > SV_ENTRIES_MAX || (bias->n > 0 && (!bias->ids || !bias->values))))
    return SV_ERR_ARG;
  if (masks && (!masks->bits || !masks->rows || masks->n_masks < 1)) return SV_ERR_ARG;
  AdjustArgs a = {};
  a.logits = logits;
  a.in_session = session_stride;
  a.in_row = row_stride;
  a.out = out;
  const bool in_place = out == logits;
  a.out_session = in_place ? session_stride : (int64_t)R * V;
  a.out_row = in_place ? row_stride : V;
  a.tokens = draft_tokens;
  a.m = m;
  a.pen = penalties;
  if (history && penalties) {
    a.counts = history->counts;
    a.seen = history->seen;
    a.n_slots = history->n_slots;
    a.slots = slots;
  }
  if (bias) {
    a.bias_off = bias->offsets;
    a.bias_id = bias->ids;
    a.bias_val = bias->values;
    a.n_bias = bias->n;
  }
  if (masks) {
    a.mask_bits = masks->bits;
    a.mask_rows = masks->rows;
    a.n_masks = masks->n_masks;
  }
  a.B = B;
  a.M = M;
  a.R = R;
  a.V = V;
  a.W = (V + 31) / 32;
  a.status = status;
  (void)hipGetLastError();
  if (dtype == SV_BF16) launch<__bf16>(a, (hipStream_t)stream);
  else launch<float>(a, (hipStream_t)stream);
  return hipGetLastError() == hipSuccess ? SV_OK : SV_ERR_DEVICE;
}
