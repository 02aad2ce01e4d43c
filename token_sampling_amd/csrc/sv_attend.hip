// sv_attend.hip -- sv_cache_attention: attention of a round's rows over the paged
// cache, after a plan (sv_plan.hip).
//
// With scores z_t = scale * q . k_t and running largest score m, sum l and values o,
// a tile of keys t turns them into
//   m' = max(m, max z_t),  l' = l 2^(m - m') + sum 2^(z_t - m'),
//   o' = o 2^(m - m') + sum 2^(z_t - m') v_t     (scores times log2 e)
// and partial results join the same way, so keys may be split at will.
#include "sv_attend.hpp"

namespace sv {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

struct Bf {
  typedef __bf16 vec8 __attribute__((ext_vector_type(8)));
  typedef __bf16 vec2 __attribute__((ext_vector_type(2)));
  static constexpr uint32_t kExp = 0x7F80u;  // exponent of infinities and NaN
  static constexpr float kLift = 0.0f;       // see kSlack
  __device__ static inline float value(uint32_t bits) { return __uint_as_float(bits << 16); }
  __device__ static inline f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(vec8, a),
                                                   __builtin_bit_cast(vec8, b), c, 0, 0, 0);
  }
};
struct Hf {
  typedef _Float16 vec8 __attribute__((ext_vector_type(8)));
  typedef _Float16 vec2 __attribute__((ext_vector_type(2)));
  static constexpr uint32_t kExp = 0x7C00u;
  static constexpr float kLift = 7.0f;
  __device__ static inline float value(uint32_t bits) { return (float)__builtin_bit_cast(_Float16, (uint16_t)bits); }
  __device__ static inline f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(vec8, a),
                                                  __builtin_bit_cast(vec8, b), c, 0, 0, 0);
  }
};
template <typename E>
__device__ inline uint32_t pack2(float x, float y) {  // to nearest, ties to even
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{x, y}, typename E::vec2));
}

struct AttendArgs {
  CacheView c;
  AttendPlan p;
  const char* q;
  int64_t q_session, q_row, q_head;
  char* out;
  float* part_o;      // partial results: [places][head_dim]
  float* part_ml;     // [places][2]
  int64_t cuts[2];    // where the places by piece begin, of each line
  int32_t rows[2];    // of a set at most
  float scale;        // times log2 e
  int64_t base;       // the layer's first element
  int32_t G, B, R;
};

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;

// A set's row j: where its query and output stand (-1: no such row), and the keys
// that it sees (those before lim).
struct Row {
  int64_t q, out;
  int lim;
};
__device__ inline Row row_at(const AttendArgs& a, const AttendSet& set, int head, int j) {
  if (j >= set.n) return Row{-1, -1, 0};
  const int jj = set.j0 + j, row = a.p.row_of[set.t0 + jj / a.G];
  const int b = row / a.R, r = row % a.R, hq = head * a.G + jj % a.G;
  return Row{b * a.q_session + r * a.q_row + hq * a.q_head,
             ((int64_t)row * (a.G * a.c.n_kv) + hq) * a.c.head_dim, set.base + r + 1};
}

// Four dimensions of a whole result.
template <typename E>
__device__ inline void put4(char* out, f32x4 x, float norm) {
  uint2 y;
  y.x = pack2<E>(x[0] * norm, x[1] * norm);
  y.y = pack2<E>(x[2] * norm, x[3] * norm);
  *(uint2*)out = y;
}

// Where a piece of a line goes on.
struct Cursor {
  int64_t x, end;
  int s, head, blk, sets, piece;
};
// The first row's place among the partial results.
__device__ inline int64_t by_row(const AttendArgs& a, const AttendSet& set, int head) {
  return ((int64_t)set.kind * a.c.n_kv + head) * a.B * a.R * a.G + (int64_t)set.t0 * a.G + set.j0;
}
__device__ inline int64_t by_piece(const AttendArgs& a, int line, int piece) {
  return a.cuts[line] + (int64_t)piece * a.rows[line];
}
__device__ inline int64_t place(const AttendArgs& a, int line, const AttendSet& set, const Cursor& at) {
  return at.blk == 0 ? by_row(a, set, at.head) : by_piece(a, line, at.piece);
}
constexpr int kXcds = 8;
__device__ inline bool begin(const AttendArgs& a, int line, Cursor& at) {
  const int64_t total = a.p.head->total[line], piece = a.p.head->piece[line];
  at.piece = blockIdx.x % kXcds * (kPieces[line] / kXcds) + blockIdx.x / kXcds;
  at.sets = a.p.head->sets[line];
  at.x = at.piece * piece;
  at.end = min(at.x + piece, total);
  if (at.x >= at.end) return false;
  const int4 start = a.p.starts[line][at.piece];
  at.s = start.x, at.head = start.y, at.blk = start.z;
  return true;
}
__device__ inline void advance(Cursor& at, int blocks) {
  at.x += blocks;
  at.blk = 0;
  if (++at.s == at.sets) at.s = 0, ++at.head;
}

// Scores of 32 keys' keys against 16 rows, a lane its row's: keys 8 g .. 8 g + 7.
template <typename E, int kC>
__device__ inline void score(const u32x4 (&kf)[kC], const u32x4 (&q)[kC], f32x4& z) {
  z = f32x4{0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < kC; ++i) z = E::mfma(kf[i], q[i], z);
}

// Scores become weights: 2^(z * scale - m), with m a value near the row's largest
// score so far.  m follows the largest only where a score's weight exceeds what that one
// had by 2^kSlack, which after the first tiles hardly happens: the lanes need not agree on
// a tile's largest, and what is summed is seldom multiplied.  The largest score's weight
// lies between 2^kLift and 2^(kLift + kSlack).  That costs no digits in binary32 or
// bfloat16, whose exponents reach far enough with a kLift of 0.  Halves end at 2^16 and
// have fewer digits below 2^-14, so kLift is 7 there: a key's weight is off by half its last
// digit or 2^-32 of the largest, and 131072 keys together by 2^-15 at most (without the
// lift 2^-25 and 2^-8: they would be lost from the values but not from the sum).  Whether m
// has to follow is asked of the weight's own exponent, rounded as the weight's is: z * scale
// and m + kReach are rounded otherwise, and from scores of 2^24 on, whose last digit is
// worth 2, a weight would pass 2^16 unnoticed.  m itself is off by half its last digit,
// which is harmless up to scores of 2^28 (bfloat16 2^31).
constexpr float kSlack = 8.0f;
template <typename E>
constexpr float kReach = E::kLift + kSlack;
constexpr float kLowest = -3.402823466e38f;  // m of a row that has seen nothing
// Hidden scores are -inf; true where a row's m has to follow.
template <typename E, bool kEdge, int NT>
__device__ inline bool look_up(f32x4 (&z)[NT][2], float (&top)[NT], float scale, int key, const int (&lim)[NT],
                               const float (&m)[NT]) {
  bool far = false;
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    if (kEdge) {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (key + e >= lim[t]) z[t][e / 4][e % 4] = -INFINITY;
    }
    top[t] = z[t][0][0];
#pragma unroll
    for (int e = 1; e < 8; ++e) top[t] = fmaxf(top[t], z[t][e / 4][e % 4]);
    far |= fmaf(top[t], scale, -m[t]) > kReach<E>;
  }
  return __any(far);
}
template <typename E, int NT, int kN>
__device__ inline void follow(const float (&top)[NT], float scale, float (&m)[NT], float (&l)[NT],
                              f32x4 (&o)[NT][kN]) {
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    float now = fmaxf(top[t], lane_xor<16>(top[t]));
    now = fmaxf(m[t], fmaf(fmaxf(now, lane_xor<32>(now)), scale, -E::kLift));
    const float keep = __builtin_amdgcn_exp2f(m[t] - now);
    m[t] = now;
    l[t] *= keep;
#pragma unroll
    for (int i = 0; i < kN; ++i) o[t][i] *= keep;
  }
}
// The weights, and their sums.
template <typename E, int NT>
__device__ inline void powers(const f32x4 (&z)[NT][2], u32x4 (&w)[NT], float (&sum)[NT], float scale,
                              const float (&m)[NT]) {
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    float p[8];
    sum[t] = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      p[e] = __builtin_amdgcn_exp2f(fmaf(z[t][e / 4][e % 4], scale, -m[t]));
      sum[t] += p[e];
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) w[t][e] = pack2<E>(p[2 * e], p[2 * e + 1]);
  }
}
template <typename E, bool kEdge, int NT, int kN>
__device__ inline void weigh(f32x4 (&z)[NT][2], u32x4 (&w)[NT], float scale, int key, const int (&lim)[NT],
                             float (&m)[NT], float (&l)[NT], f32x4 (&o)[NT][kN]) {
  float top[NT], sum[NT];
  if (look_up<E, kEdge>(z, top, scale, key, lim, m)) follow<E>(top, scale, m, l, o);
  powers<E>(z, w, sum, scale, m);
#pragma unroll
  for (int t = 0; t < NT; ++t) l[t] += sum[t];
}

// Values of 32 keys meet the weights, 16 dimensions at a time; values(i) has them.
template <typename E, int NT, int kN, typename V>
__device__ inline void mix(const V& values, const u32x4 (&w)[NT], f32x4 (&o)[NT][kN]) {
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    const u32x4 vf = values(i);
#pragma unroll
    for (int t = 0; t < NT; ++t) o[t][i] = E::mfma(vf, w[t], o[t][i]);
  }
}
// The same where some rows do not see all keys: what lies behind the last key (never
// written for this session) counts as 0.  False, and nothing done, where a value is
// not finite: times a weight of 0 it would reach rows that do not see it.
template <typename E, int NT, int kN, typename V>
__device__ inline bool mix_edge(const V& values, const u32x4 (&w)[NT], int key, int key1, f32x4 (&o)[NT][kN]) {
  const int g = threadIdx.x % kWave / 16;
  u32x4 there;
#pragma unroll
  for (int e = 0; e < 4; ++e)
    there[e] = (key + g * 8 + 2 * e < key1 ? 0x0000FFFFu : 0u) | (key + g * 8 + 2 * e + 1 < key1 ? 0xFFFF0000u : 0u);
  bool odd = false;
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    const u32x4 vf = values(i) & there;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      odd |= (vf[e] & E::kExp) == E::kExp || (vf[e] >> 16 & E::kExp) == E::kExp;
  }
  if (__any(odd)) return false;
  mix<E>([&](int i) { return values(i) & there; }, w, o);
  return true;
}
// Then: key by key, for the rows that see it, out of the values' 16-bit elements.
template <typename E, int NT, int kN>
__device__ inline void mix_slowly(const uint16_t* values, const u32x4 (&w)[NT], int key, int key1,
                                  const int (&lim)[NT], f32x4 (&o)[NT][kN]) {
  const int lane = threadIdx.x % kWave, col = lane % 16, g = lane / 16;
#pragma unroll 1
  for (int k = 0; k < 32 && key + k < key1; ++k) {
    float p[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const uint32_t two = k & 4 ? (k & 2 ? w[t][3] : w[t][2]) : (k & 2 ? w[t][1] : w[t][0]);
      uint32_t there = (uint32_t)__shfl((int)two, k / 8 * 16 + col);
      pin(there);
      p[t] = E::value(there >> (16 * (k & 1)) & 0xFFFFu);
    }
    const uint16_t* at = values + (k / 8 * 16 + g * 4) * 8 + k % 8;
#pragma unroll
    for (int i = 0; i < kN; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float v = E::value(at[i * 512 + e * 8]);
#pragma unroll
        for (int t = 0; t < NT; ++t) o[t][i][e] = key + k < lim[t] ? fmaf(p[t], v, o[t][i][e]) : o[t][i][e];
      }
  }
}

struct Yes { static constexpr bool value = true; };
struct No { static constexpr bool value = false; };

// A stretch of a set's keys, for one key head: where the pages' parts of it stand.
struct Stretch {
  const int32_t* list;
  int64_t base;  // of the layer and head
  int lo, hi;
  __device__ int page(const CacheView& c, int key) const {
    return key < hi ? min((uint32_t)list[key >> c.shift], (uint32_t)(c.n_pages - 1)) : 0;
  }
  // bytes from a plane's start to the 32 keys from `key` on, which lie in `page`
  __device__ int64_t at(const CacheView& c, int page, int key) const {
    return 2 * (base + page * c.page_elems() + (int64_t)(key & (c.page() - 1)) * c.head_dim);
  }
};
__device__ inline Stretch stretch(const AttendArgs& a, const AttendSet& set, int head, int blk, int cnt) {
  return Stretch{a.c.table + (int64_t)set.slot * a.c.max_pages, a.base + head * a.c.head_elems(),
                 set.key0 + blk * kBlock, min(set.key0 + (blk + cnt) * kBlock, set.key1)};
}

// A narrow set: the waves take the tiles of 32 keys in turn, each for all of its up to
// NT * 16 rows, with the next tile's keys and values on the way into registers, and
// join at the end.
template <int D, int NT>
struct Meet {
  f32x4 o[kWaves][D / 16][kWave];
  float m[kWaves][NT * 16], l[kWaves][NT * 16];
};
template <typename E, int D, int NT, int kMax>
__device__ inline void narrow_set(const AttendArgs& a, const AttendSet& set, const Cursor& at, int cnt,
                                  Meet<D, kMax>& red) {
  constexpr int kC = D / 32, kN = D / 16;
  const CacheView& c = a.c;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), lane = threadIdx.x % kWave;
  const int col = lane % 16, g = lane / 16;
  const Stretch keys = stretch(a, set, at.head, at.blk, cnt);
  u32x4 kf[2][kC], vf[kN];
  const auto bring_keys = [&](int page, int key) {
    const u32x4* p = (const u32x4*)(c.k + keys.at(c, page, key)) + lane;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < kC; ++i) kf[h][i] = p[(h * kC + i) * kWave];
  };
  const auto bring_values = [&](int page, int key) {
    const u32x4* p = (const u32x4*)(c.v + keys.at(c, page, key)) + lane;
#pragma unroll
    for (int i = 0; i < kN; ++i) vf[i] = p[i * kWave];
  };
  constexpr int kStep = kWaves * 32;
  int key = keys.lo + wave * 32;
  int page = keys.page(c, key), next = keys.page(c, key + kStep);
  if (key < keys.hi) {
    bring_keys(page, key);
    bring_values(page, key);
  }
  u32x4 q[NT][kC];
  int lim[NT];
  f32x4 o[NT][kN];
  float m[NT], l[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const Row row = row_at(a, set, at.head, t * 16 + col);
    lim[t] = row.lim;
#pragma unroll
    for (int i = 0; i < kC; ++i)
      q[t][i] = row.q >= 0 ? *(const u32x4*)(a.q + 2 * (row.q + i * 32 + g * 8)) : u32x4{0, 0, 0, 0};
    m[t] = kLowest, l[t] = 0;
#pragma unroll
    for (int i = 0; i < kN; ++i) o[t][i] = f32x4{0, 0, 0, 0};
  }
  // the tiles that every row sees whole, then the others: a loop each, so that the
  // first has the registers to itself
  const auto pass = [&](auto edge, int end) {
    for (; key < end; key += kStep) {
      const bool more = key + kStep < keys.hi;
      f32x4 z[NT][2];
      u32x4 w[NT];
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int h = 0; h < 2; ++h) score<E>(kf[h], q[t], z[t][h]);
      if (more) bring_keys(next, key + kStep);
      weigh<E, decltype(edge)::value>(z, w, a.scale, key + g * 8, lim, m, l, o);
      const auto values = [&](int i) { return vf[i]; };
      if constexpr (!decltype(edge)::value)
        mix<E>(values, w, o);
      else if (!mix_edge<E>(values, w, key, set.key1, o))
        mix_slowly<E>((const uint16_t*)(c.v + keys.at(c, page, key)), w, key, set.key1, lim, o);
      if (more) bring_values(next, key + kStep);
      page = next;
      next = keys.page(c, key + 2 * kStep);
    }
  };
  pass(No{}, min(keys.hi, set.base - 30));  // key + 32 <= base + 1
  pass(Yes{}, keys.hi);
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    l[t] += lane_xor<16>(l[t]);
    l[t] += lane_xor<32>(l[t]);
    pin(l[t]);
    if (lane < 16) {
      red.m[wave][t * 16 + lane] = m[t];
      red.l[wave][t * 16 + lane] = l[t];
    }
  }
  __syncthreads();
  const int64_t part = place(a, kNarrow, set, at);
  const bool whole = set.alone && cnt == set.blocks();
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int j = t * 16 + col;
    float top = kLowest, sum = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) top = fmaxf(top, red.m[w][j]);
#pragma unroll
    for (int w = 0; w < kWaves; ++w) sum += red.l[w][j] * __builtin_amdgcn_exp2f(red.m[w][j] - top);
    const float mine = __builtin_amdgcn_exp2f(m[t] - top);
#pragma unroll
    for (int i = 0; i < kN; ++i) red.o[wave][i][lane] = o[t][i] * mine;
    __syncthreads();
    if (j < set.n) {
      const float norm = 1.0f / sum;
      char* out = a.out + 2 * (whole ? row_at(a, set, at.head, j).out : 0);
#pragma unroll
      for (int i0 = 0; i0 < (kN + kWaves - 1) / kWaves; ++i0) {
        const int i = i0 * kWaves + wave;
        if (i >= kN) break;
        f32x4 all = red.o[0][i][lane];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) all += red.o[w][i][lane];
        if (whole) put4<E>(out + 2 * (i * 16 + g * 4), all, norm);
        else *(f32x4*)(a.part_o + (part + j) * D + i * 16 + g * 4) = all;
      }
      if (!whole && wave == 0 && g == 0)
        *(f32x2*)(a.part_ml + (part + j) * 2) = f32x2{top, sum};
    }
    __syncthreads();
  }
}

// A workgroup goes over a piece of the narrow line, set by set.  256 sessions of up to
// 4096 tokens, 9 rows, 8 heads of 128 (36 rows a set): 2.5 GB in 455 us, 5.6 TB/s;
// two sessions of 131072 tokens 195 us, 5.5 TB/s.  What bounds it there are the loads
// in flight: a wave a SIMD with 16 to 32 KiB under way (48 rows take more than half of
// the registers).  Sets of a few blocks are bound by their chains of loads: 239
// sessions of 300 keys 113 us.
template <typename E, int D, int NT>
__global__ __launch_bounds__(kThreads) void k_attend(AttendArgs a) {
  __shared__ Meet<D, NT> red;
  Cursor at;
  if (!begin(a, kNarrow, at)) return;
  while (at.x < at.end) {
    const AttendSet set = a.p.sets[kNarrow][at.s];
    const int cnt = (int)min((int64_t)(set.blocks() - at.blk), at.end - at.x);
    if (NT == 1 || set.n <= 16) narrow_set<E, D, 1, NT>(a, set, at, cnt, red);
    else if (NT == 2 || set.n <= 32) narrow_set<E, D, NT < 2 ? NT : 2, NT>(a, set, at, cnt, red);
    else if (set.n <= 48) narrow_set<E, D, NT < 3 ? NT : 3, NT>(a, set, at, cnt, red);
    else narrow_set<E, D, NT, NT>(a, set, at, cnt, red);
    advance(at, cnt);
  }
}

// The wide sets' inner loop: one tile's values meet its weights w while the next tile's
// scores are taken and become weights, in an order laid down here step by step (the
// compiler would put the products and the exponentials one after the other): eight
// steps a row tile, in each a product or two of the matrix unit and an eighth of the
// vector unit's work for the row tile whose scores are ready.
template <typename E, int kC, int kN, int NT>
__device__ inline void in_turn(const u32x4 (*keys)[kWave], const u32x4 (*values)[kWave], const u32x4 (&q)[NT][kC],
                               u32x4 (&w)[NT], f32x4 (&o)[NT][kN], f32x4 (&z)[NT][2], float (&top)[NT],
                               float (&sum)[NT], float scale, const float (&m)[NT]) {
  const int lane = threadIdx.x % kWave;
  float before[NT];
  u32x4 w_next[NT];
  const auto weigh_one = [&](int t, int e) {  // score e of row tile t
    const float x = z[t][e / 4][e % 4], p = __builtin_amdgcn_exp2f(fmaf(x, scale, -m[t]));
    top[t] = e ? fmaxf(top[t], x) : x;
    sum[t] = e ? sum[t] + p : p;
    if (e % 2) w_next[t][e / 2] = pack2<E>(before[t], p);
    else before[t] = p;
  };
  constexpr int kAhead = 2;
  u32x4 kf[2 * kC], vf[kN];  // a few of each live
#pragma unroll
  for (int t = 0; t < NT; ++t) z[t][0] = z[t][1] = f32x4{0, 0, 0, 0};
#pragma unroll
  for (int j = 0; j < kAhead; ++j) kf[j] = keys[j % 2 * kC + j / 2][lane];
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int j = 0; j < 2 * kC; ++j) {
    const int n = j + kAhead;
    if (n < 2 * kC) kf[n] = keys[n % 2 * kC + n / 2][lane];
    else if (n - 2 * kC < kAhead) vf[n - 2 * kC] = values[n - 2 * kC][lane];
#pragma unroll
    for (int t = 0; t < NT; ++t) z[t][j % 2] = E::mfma(kf[j], q[t][j / 2], z[t][j % 2]);
    __builtin_amdgcn_sched_barrier(0);
  }
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    if (i + kAhead < kN) vf[i + kAhead] = values[i + kAhead][lane];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      o[t][i] = E::mfma(vf[i], w[t], o[t][i]);
#pragma unroll
      for (int e = i * 8 / kN; e < (i + 1) * 8 / kN; ++e) weigh_one(t, e);
    }
    __builtin_amdgcn_sched_barrier(0);
  }
  // here, not where they turn out to be needed
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    asm volatile("" : "+v"(w_next[t]), "+v"(sum[t]));
    w[t] = w_next[t];
  }
}

// A workgroup goes over a piece of the wide line: its waves share the set's tiles of
// 16 rows, NT each, and tiles of 32 keys and values stand in a ring in LDS, brought
// there past the registers two tiles ahead.  Two workgroups a CU, so that one's products
// run under the other's exponentials: that bounds NT, by 256 registers.  4780 rows a
// head over 8192 shared keys, 8 heads of 128: 1.6e11 operations in 200 us, 0.8 PFLOP/s,
// where a large library product reaches 1.2.  The matrix unit is busy in 37% of the
// cycles and the vector unit in 42%; without the loads it would take 173 us.  Tried and
// left: NT = 3 (230 us, and 520 with registers spilled: a spilled value's load waits
// for the tiles on their way), one workgroup a CU with NT = 4 (227 us).
__device__ inline void to_lds(const char* from, void* to) {  // 16 bytes a lane, side by side
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)from,
                                   (__attribute__((address_space(3))) void*)to, 16, 0, 0);
}
template <typename E, int D, int NT>
__global__ __launch_bounds__(kThreads, D > 128 ? 1 : 2) void k_attend_wide(AttendArgs a) {
  constexpr int kC = D / 32, kN = D / 16, kF = 2 * kC + kN;  // KiB of 32 keys
  constexpr int kRing = 4;                                   // tiles of 32 keys
  __shared__ u32x4 tile[kRing][kF][kWave];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), lane = threadIdx.x % kWave;
  const int col = lane % 16, g = lane / 16;
  const CacheView& c = a.c;
  const int no_limit[NT] = {};
  Cursor at;
  if (!begin(a, kWide, at)) return;
  while (at.x < at.end) {
    const AttendSet set = a.p.sets[kWide][at.s];
    const int cnt = (int)min((int64_t)(set.blocks() - at.blk), at.end - at.x);
    const Stretch keys = stretch(a, set, at.head, at.blk, cnt);
    const int tiles = (keys.hi - keys.lo + 31) / 32;
    int page = keys.page(c, keys.lo);  // of the tile to bring next
    const auto bring = [&](int i) {
      if (i >= tiles) return;
      const int64_t from = keys.at(c, page, keys.lo + 32 * i) + lane * 16;
      page = keys.page(c, keys.lo + 32 * i + 32);
      static_assert(kF % kWaves == 0, "a tile in equal parts");
#pragma unroll
      for (int k = 0; k < kF / kWaves; ++k) {
        const int f = k * kWaves + wave;
        to_lds(f < 2 * kC ? c.k + from + f * 1024 : c.v + from + (f - 2 * kC) * 1024, &tile[i % kRing][f][0]);
      }
    };
    const auto arrived = [&](bool all) {  // the tiles but the last one on its way, for every wave
      if (all) asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      else asm volatile("s_waitcnt vmcnt(%0)" ::"n"(kF / kWaves) : "memory");
      __syncthreads();
    };
    __syncthreads();  // the last set's tiles are done with
#pragma unroll
    for (int i = 0; i < kRing - 1; ++i) bring(i);
    u32x4 q[NT][kC];
    f32x4 o[NT][kN];
    float m[NT], l[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const Row row = row_at(a, set, at.head, (t * kWaves + wave) * 16 + col);
#pragma unroll
      for (int i = 0; i < kC; ++i)
        q[t][i] = row.q >= 0 ? *(const u32x4*)(a.q + 2 * (row.q + i * 32 + g * 8)) : u32x4{0, 0, 0, 0};
      m[t] = kLowest, l[t] = 0;
#pragma unroll
      for (int i = 0; i < kN; ++i) o[t][i] = f32x4{0, 0, 0, 0};
    }
    // one tile's values and the next one's scores and weights go side by side; where a
    // row's m has to follow, which is rare, the inner loop is left for it
    u32x4 w[NT];
    f32x4 z[NT][2];
    float top[NT], sum[NT];  // of the tile whose weights are in w: not yet in l
    arrived(true);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      u32x4 kf[kC];
#pragma unroll
      for (int j = 0; j < kC; ++j) kf[j] = tile[0][h * kC + j][lane];
#pragma unroll
      for (int t = 0; t < NT; ++t) score<E>(kf, q[t], z[t][h]);
    }
    look_up<E, false>(z, top, a.scale, 0, no_limit, m);
    bool far = true;
    for (int i = 0;;) {
      if (far) {
        follow<E>(top, a.scale, m, l, o);
        powers<E>(z, w, sum, a.scale, m);
      }
      if (i + 1 == tiles) break;
      do {
        arrived(i + 2 >= tiles);
        bring(i + kRing - 1);  // in place of the tile before this one
#pragma unroll
        for (int t = 0; t < NT; ++t) l[t] += sum[t];
        in_turn<E>(&tile[(i + 1) % kRing][0], &tile[i % kRing][2 * kC], q, w, o, z, top, sum, a.scale, m);
        far = false;
#pragma unroll
        for (int t = 0; t < NT; ++t) far |= fmaf(top[t], a.scale, -m[t]) > kReach<E>;
        far = __any(far);
        ++i;
      } while (!far && i + 1 < tiles);
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) l[t] += sum[t];
    const u32x4(*last)[kWave] = &tile[(tiles - 1) % kRing][2 * kC];
    mix<E>([&](int j) { return last[j][lane]; }, w, o);
    const int64_t part = place(a, kWide, set, at);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      l[t] += lane_xor<16>(l[t]);
      l[t] += lane_xor<32>(l[t]);
      pin(l[t]);
      const int j = (t * kWaves + wave) * 16 + col;
      if (j >= set.n) continue;
#pragma unroll
      for (int i = 0; i < kN; ++i)
        *(f32x4*)(a.part_o + (part + j) * D + i * 16 + g * 4) = o[t][i];
      if (g == 0) *(f32x2*)(a.part_ml + (part + j) * 2) = f32x2{m[t], l[t]};
    }
    advance(at, cnt);
  }
}

// x / piece, in 32 bits where the whole line fits them: the quotient is on the way
// of every row.
__device__ inline int piece_of(int64_t x, int64_t total, int64_t piece) {
  return total >> 32 ? (int)(x / piece) : (int)((uint32_t)x / (uint32_t)piece);
}

// Joins the partial results of every row.  A lane has 8 dimensions of a row and head, a
// wave some heads of a row, side by side; parts are loaded four at a time, as what they
// wait for is memory (eight: 12 against 14 us for 640 rows of 32 parts, but 23 against
// 19 for 38000 rows of two or three, whose waves then have too many registers).  NaN
// where the session failed.
template <int D>
struct Join {
  static constexpr int kLanes = D == 96 ? 16 : D / 8;         // of a row and head
  static constexpr int kHeads = kWaves * kWave / kLanes;      // of a workgroup
};
template <typename E, int D>
__global__ __launch_bounds__(kThreads) void k_join(AttendArgs a) {
  constexpr int kLanes = Join<D>::kLanes, kStep = 4;
  const CacheView& c = a.c;
  const int b = blockIdx.x / a.R, r = blockIdx.x % a.R;
  const int heads = a.G * c.n_kv, hq = blockIdx.y * Join<D>::kHeads + threadIdx.x / kLanes;
  const int d = threadIdx.x % kLanes * 8;
  const AttendSession ss = a.p.sess[b];
  const AttendHead lines = *a.p.head;
  if (hq >= heads || d >= D || (ss.status == 0 && r >= ss.n)) return;
  f32x4 o[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
  float m = kLowest, l = ss.status == 0 ? 0 : NAN;
  if (ss.status == 0) {
    const int head = hq / a.G;
#pragma unroll
    for (int level = 0; level < kKinds; ++level) {
      if (ss.first[level] < 0) continue;
      const int first = ss.first[level] / 2, line = ss.first[level] % 2;
      const AttendSet& set = a.p.sets[line][first];
      // a session's own sets begin with its first row, a run's with the run's
      const int j = (ss.t0 + r - set.t0) * a.G + hq % a.G, nth = j / set.per, row = j - nth * set.per;
      const int nb = set.blocks();
      const int64_t blocks = line ? lines.blocks[1] : lines.blocks[0];
      const int64_t total = line ? lines.total[1] : lines.total[0];
      const int64_t piece = line ? lines.piece[1] : lines.piece[0];
      const int64_t x = head * blocks + set.cum + (int64_t)nth * nb;
      const int p0 = piece_of(x, total, piece), n = piece_of(x + nb - 1, total, piece) - p0 + 1;
      if (n == 1 && set.alone) return;
      // the first part's place by row (set is the first over its keys, j the row from there),
      // the others' by piece
      const int rows = line ? a.rows[1] : a.rows[0];
      const int64_t at0 = by_row(a, set, head) + j, at1 = (line ? a.cuts[1] : a.cuts[0]) + (int64_t)p0 * rows + row;
      const auto take = [&](int k0) {
        f32x2 ml[kStep];
        f32x4 y[kStep][2];
#pragma unroll
        for (int k = 0; k < kStep; ++k) {
          const int nth_part = min(k0 + k, n - 1);
          const int64_t at = nth_part == 0 ? at0 : at1 + (int64_t)nth_part * rows;
          ml[k] = *(const f32x2*)(a.part_ml + at * 2);
          y[k][0] = *(const f32x4*)(a.part_o + at * D + d);
          y[k][1] = *(const f32x4*)(a.part_o + at * D + d + 4);
        }
        float now = m;
#pragma unroll
        for (int k = 0; k < kStep; ++k) now = fmaxf(now, ml[k][0]);
        const float old = __builtin_amdgcn_exp2f(m - now);
        m = now;
        l *= old, o[0] *= old, o[1] *= old;
#pragma unroll
        for (int k = 0; k < kStep; ++k) {
          const float w = __builtin_amdgcn_exp2f(ml[k][0] - now);
          if (k0 + k < n) l += ml[k][1] * w, o[0] += y[k][0] * w, o[1] += y[k][1] * w;
        }
      };
      for (int k0 = 0; k0 < n; k0 += kStep) take(k0);
    }
  }
  const float norm = 1.0f / l;
  char* out = a.out + 2 * (((int64_t)blockIdx.x * heads + hq) * D + d);
  *(u32x4*)out = u32x4{pack2<E>(o[0][0] * norm, o[0][1] * norm), pack2<E>(o[0][2] * norm, o[0][3] * norm),
                       pack2<E>(o[1][0] * norm, o[1][1] * norm), pack2<E>(o[1][2] * norm, o[1][3] * norm)};
}

template <typename E, int D>
void launch(const AttendArgs& a, hipStream_t st) {
  if (may_be_wide((int64_t)a.R * a.G, a.c.n_kv, D, a.B, (int64_t)a.c.max_pages << a.c.shift))
    hipLaunchKernelGGL((k_attend_wide<E, D, wide_tiles(D)>), dim3(kPieces[kWide]), dim3(kThreads), 0, st, a);
  const auto narrow = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3(kPieces[kNarrow]), dim3(kThreads), 0, st, a);
  };
  if constexpr (D > 128) {
    narrow(k_attend<E, D, 1>);
  } else {
    switch (a.rows[kNarrow]) {
      case 16: narrow(k_attend<E, D, 1>); break;
      case 32: narrow(k_attend<E, D, 2>); break;
      case 48: narrow(k_attend<E, D, 3>); break;
      default: narrow(k_attend<E, D, 4>);
    }
  }
  const unsigned gy = (a.G * a.c.n_kv + Join<D>::kHeads - 1) / Join<D>::kHeads;
  hipLaunchKernelGGL((k_join<E, D>), dim3(a.B * a.R, gy), dim3(kThreads), 0, st, a);
}
template <typename E>
void launch_dim(const AttendArgs& a, hipStream_t st) {
  switch (a.c.head_dim) {
    case 64: return launch<E, 64>(a, st);
    case 96: return launch<E, 96>(a, st);
    case 128: return launch<E, 128>(a, st);
    default: return launch<E, 256>(a, st);
  }
}

bool stride_ok(int64_t s) { return s >= 0 && s % 8 == 0 && s <= ((int64_t)1 << 40); }

// Places for partial results: one a row and head for each kind of sets that can occur,
// and a set's rows for each piece of a line.
struct Parts {
  int64_t by_row, places;
  size_t bytes;
};
Parts parts_of(const sv_cache* c, int32_t B, int32_t R, int32_t G) {
  const int64_t rows = (int64_t)R * G, most = (int64_t)c->max_pages * c->page;
  const int narrow = narrow_rows(rows, c->head_dim);
  const int kinds = 1 + (rows > narrow) + (may_share(c->n_kv, c->head_dim, B, most) ? 2 : 0);
  Parts p;
  p.by_row = (int64_t)kinds * c->n_kv * B * rows;
  p.places = p.by_row + (int64_t)kPieces[kNarrow] * narrow;
  if (may_be_wide(rows, c->n_kv, c->head_dim, B, most)) p.places += (int64_t)kPieces[kWide] * wide_rows(c->head_dim);
  p.bytes = (size_t)p.places * (c->head_dim + 2) * 4;
  return p;
}

}  // namespace
}  // namespace sv

extern "C" size_t sv_cache_attention_bytes(const sv_cache* cache, int32_t n_heads, int32_t B,
                                           int32_t R) {
  using namespace sv;
  if (sv_cache_plan_bytes(cache, n_heads, B, R) == 0) return 0;
  const int G = n_heads / cache->n_kv;
  return parts_of(cache, B, R, G).bytes;
}

extern "C" int sv_cache_attention(const sv_cache* cache, int32_t layer, const void* q,
                                  int64_t q_session, int64_t q_row, int64_t q_head, float scale,
                                  const void* plan, int32_t n_heads, int32_t B, int32_t R,
                                  void* out, void* workspace, size_t workspace_bytes, void* stream) {
  using namespace sv;
  const size_t need = sv_cache_attention_bytes(cache, n_heads, B, R);
  if (need == 0 || layer < 0 || layer >= cache->n_layers || !q || !plan || !out || !workspace)
    return SV_ERR_ARG;
  if (((uintptr_t)q | (uintptr_t)plan | (uintptr_t)out | (uintptr_t)workspace) % 16 != 0)
    return SV_ERR_ARG;
  if (!stride_ok(q_session) || !stride_ok(q_row) || !stride_ok(q_head)) return SV_ERR_ARG;
  const float in_twos = scale * 1.44269504088896340736f;  // of powers of two
  if (!(in_twos > 0) || !(in_twos < INFINITY)) return SV_ERR_ARG;
  if (workspace_bytes < need) return SV_ERR_WORKSPACE;
  const int G = n_heads / cache->n_kv;
  const PlanSizes z = plan_sizes(B, R, G, cache->head_dim);
  const Parts parts = parts_of(cache, B, R, G);
  const int32_t narrow = narrow_rows((int64_t)R * G, cache->head_dim);
  float* part = (float*)workspace;
  AttendArgs a = {view_of(cache), plan_of(z, (void*)plan), (const char*)q, q_session, q_row, q_head, (char*)out,
                  part, part + parts.places * cache->head_dim,
                  {parts.by_row, parts.by_row + (int64_t)kPieces[kNarrow] * narrow},
                  {narrow, wide_rows(cache->head_dim)}, in_twos, 0, G, B, R};
  a.base = layer * a.c.layer_elems();
  hipStream_t st = (hipStream_t)stream;
  (void)hipGetLastError();
  if (cache->dtype == SV_BF16) launch_dim<Bf>(a, st);
  else launch_dim<Hf>(a, st);
  return hipGetLastError() == hipSuccess ? SV_OK : SV_ERR_DEVICE;
}
