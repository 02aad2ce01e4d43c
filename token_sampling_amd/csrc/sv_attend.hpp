// sv_attend.hpp -- the plan of a round's attention (sv_cache_plan), as the
// attention's kernels read it.
//
// A set is a number of query rows (a row here is a round's row and a query head of
// the set's key head) that go over the same keys: one session's rows over the keys
// that it has alone, or rows of neighbouring sessions over keys that they share.
// Where they fit one wave's registers the set is narrow: the waves of a workgroup
// take its keys in turn, and what counts is the bytes that arrive.  Else it is
// wide: the waves take its rows, and share the keys in LDS; every row of a wide set
// sees all of its keys, what rows see in part is left to narrow ones.  Keys are counted in
// blocks of kBlock.  The narrow sets' blocks stand in one line, the first key head's,
// then the second's and so on, the wide sets' in another; a line is cut into equal
// pieces, a piece a workgroup.  A piece leaves a partial result (largest score, sum,
// weighted values) for every set and head that it touches, and where a set and head lie
// in one piece and nothing else belongs to their rows, the result itself.  A row is in at
// most one set of a kind (below), so the partial result of a set's first blocks has its
// place by kind, head and row; what a piece finds of a set that began in the one before,
// one at most, has its place by the piece.
// An XCD has neighbouring pieces (its workgroups are every eighth): sets of many rows
// over the same keys go over a head's keys in one L2.
#pragma once

#include "sv_cache.hpp"

namespace sv {

constexpr int kBlock = 128;     // keys
constexpr int kNarrow = 0, kWide = 1;
constexpr int kPieces[2] = {512, 512};  // of a line: two workgroups a CU
constexpr int kFar = 1 << 30;   // no limit on keys

struct AttendSet {
  int32_t t0;    // the first of the rows' places in row_of
  int32_t j0;    // the set's first row (of round rows times heads) from there
  int32_t n;     // rows
  int32_t key0, key1;
  int32_t slot;  // whose list of pages
  int32_t base;  // round row r sees the keys before base + r + 1; kFar: all
  int32_t alone; // nothing else belongs to these rows
  int64_t cum;   // blocks of the sets before
  int32_t per;   // rows of each but the last set over the same keys
  int32_t kind;  // the place of its kind among the partial results
  __host__ __device__ int blocks() const { return (key1 - key0 + kBlock - 1) / kBlock; }
};
static_assert(sizeof(AttendSet) == 48, "AttendSet layout");

// A session's rows stand in the sets from first[0] (its run's shared keys), first[1]
// (its run's in that run), first[2] (its own keys that all its rows see, where these
// are many) and first[3] (its other keys) on: 2 * set + line, -1: none.  Of partial
// results only the kinds that can occur have places: first[3]'s, then first[2]'s, then
// first[0]'s and first[1]'s.
constexpr int kKinds = 4;
struct AttendSession {
  int32_t status, n, t0;  // rows in use, their first place in row_of
  int32_t first[kKinds];
  int32_t pad;
};

struct AttendHead {
  int64_t blocks[2], total[2], piece[2];  // of all sets, of all sets and heads, of a piece
  int32_t sets[2];
};

struct AttendPlan {
  AttendHead* head;
  AttendSession* sess;   // [B]
  int4* starts[2];       // a piece: set, key head, block; of pieces that begin before total
  int32_t* shared;       // [B]: keys shared with the session before
  int32_t* row_of;       // [B * R]: session * R + round row
  AttendSet* sets[2];
};

// Rows of a narrow set at most, by the rows that a round brings a key head, and of a
// wide one.  Up to 64 rows a session's keys go into one narrow set, all of whose rows
// have to fit a wave's registers: 64 sessions of 8192 tokens, 8 heads, 64 rows, take 218
// us so and 320 as wide sets with heads of 64, 292 and 336 with heads of 96; with heads
// of 128 the registers spill (133 of them, 472 bytes a lane) and neither wins, 430 and
// 420.  What is left of a wide set's session, the keys that not all rows see, goes in
// sets of 48.  Heads of 256 leave room for 16 rows only (32 in registers: 399 against
// 391 us for 16 rows, 449 against 446 for 32).
inline int narrow_rows(int64_t rows, int head_dim) {
  if (rows <= 16 || head_dim > 128) return 16;
  if (rows <= 32) return 32;
  return rows > 48 && rows <= 64 ? 64 : 48;
}
constexpr int wide_tiles(int head_dim) {  // tiles of 16 rows of each of four waves, in 256 registers
  return head_dim > 128 ? 1 : head_dim > 64 ? 2 : 3;
}
inline int wide_rows(int head_dim) { return 64 * wide_tiles(head_dim); }

// Keys that n neighbours share are worth sets of their own from so many on.  Read by each
// session they come from caches mostly, and a row's further part and the wide sets'
// start cost some 20 us.  Keys at which both sides were measured to take the same time, for
// one row and for 9 rows a session, 4 query heads a key head, layers in turn; in brackets the
// rule, which does not ask for the rows:
//               8 heads of 128      16 of 128           8 of 64               1 of 64
//      4        12600 9100 (8789)   2600 3700 (4394)    16300 20900 (17578)   -
//     16        6200 5200 (8789)    3300 3000 (4394)    14300 5600 (17578)    -
//     64        2900 3300 (2746)    1600 1800 (1373)    4900 2900 (5493)      36800 11900 (43945)
//    256        870 1050 (1255)     <512 650 (627)      1060 <1024 (2511)     10300 3400 (20089)
//   1024        <512 610 (1255)     <512 540 (627)      <1024 <1024 (2511)    2400 1600 (20089)
// (8192 keys of 8 heads of 128, 9 rows: 39 us apart and 41 shared, 79 and 69, 171 and 127,
// 659 and 415, 2667 and 1591.)  Where it is off it mostly shares too late, most so for
// many sessions of few small heads: 1024 of one head of 64, one row, 16384 keys, take 180 us
// where 58 would do.  n counts places, also those without a session or rows this round: 140
// places of which 4 have rows share from 1255 keys on, where 4 would from 8789 (4 sessions
// behind 4096 keys: 22 us shared, 17 apart).
__host__ __device__ inline int worth(int n_kv, int head_dim, int n) {
  return 180000000 / (n_kv * head_dim * (n < 20 ? 20 : n > 140 ? 140 : n));
}
// Whether B sessions of `most` tokens can share enough.
inline bool may_share(int n_kv, int head_dim, int B, int64_t most) {
  return B > 1 && most >= worth(n_kv, head_dim, B);
}
// Whether a plan can hold wide sets: rows too many for a narrow one, or shared keys.
// Where it cannot, their kernel is not launched.
inline bool may_be_wide(int64_t rows, int n_kv, int head_dim, int B, int64_t most) {
  return rows > narrow_rows(rows, head_dim) || may_share(n_kv, head_dim, B, most);
}

struct PlanSizes {
  int64_t sets[2], bytes, sess, starts, shared, row_of, set_at[2];
};
inline PlanSizes plan_sizes(int32_t B, int32_t R, int32_t G, int32_t head_dim) {
  PlanSizes z;
  const int64_t rows = (int64_t)R * G, wide = wide_rows(head_dim);
  const int64_t runs = 2 * ((int64_t)B / 2 + 1);  // of two sessions or more, on two levels
  const int64_t narrow = narrow_rows(rows, head_dim);
  z.sets[kNarrow] = B * ((rows + narrow - 1) / narrow) + runs;
  z.sets[kWide] = 2 * ((B * rows + wide - 1) / wide) + runs;
  if (rows > narrow) z.sets[kWide] += B * ((rows + wide - 1) / wide);
  int64_t at = 256;
  const auto take = [&at](int64_t n) {
    const int64_t here = at;
    at = (at + n + 255) / 256 * 256;
    return here;
  };
  z.sess = take((int64_t)B * sizeof(AttendSession));
  z.starts = take((kPieces[0] + kPieces[1]) * sizeof(int4));
  z.shared = take((int64_t)B * 4);
  z.row_of = take((int64_t)B * R * 4);
  for (int line = 0; line < 2; ++line) z.set_at[line] = take(z.sets[line] * sizeof(AttendSet));
  z.bytes = at;
  return z;
}
inline AttendPlan plan_of(const PlanSizes& z, void* p) {
  char* c = (char*)p;
  int4* starts = (int4*)(c + z.starts);
  return AttendPlan{(AttendHead*)c, (AttendSession*)(c + z.sess), {starts, starts + kPieces[0]},
                    (int32_t*)(c + z.shared), (int32_t*)(c + z.row_of),
                    {(AttendSet*)(c + z.set_at[0]), (AttendSet*)(c + z.set_at[1])}};
}

}  // namespace sv
