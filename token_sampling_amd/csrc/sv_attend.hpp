// sv_attend.hpp -- the plan of a round's attention (sv_cache_plan), as the
// attention's kernels read it.
//
// A set is up to kRows query rows (a row here is a round's row and a query head
// of the set's key head) that go over the same keys: a block of one session's
// rows over the keys that it has alone, or of the rows of neighbouring sessions
// over keys that they share.  Keys are counted in blocks of kBlock.  The sets'
// blocks, for every key head, stand in one line, which is cut into equal pieces, a
// piece a workgroup: piece i leaves a partial result (largest score, sum, weighted
// values) for every set and head that it touches, in slot set * n_kv + head + i, and
// where a set and head lie in one piece and nothing else belongs to their rows, the
// result itself.
#pragma once

#include "sv_cache.hpp"

namespace sv {

constexpr int kBlock = 128;       // keys
constexpr int kPieces = 512;      // workgroups: two a CU
constexpr int kFar = 1 << 30;     // no limit on keys

struct AttendSet {
  int32_t t0;    // the first of the rows' places in row_of
  int32_t j0;    // the set's first row (of round rows times heads) from there
  int32_t n;     // rows
  int32_t key0, key1;
  int32_t slot;  // whose list of pages
  int32_t base;  // round row r sees the keys before base + r + 1; kFar: all
  int32_t alone; // nothing else belongs to these rows
  int64_t cum;   // blocks of the sets before
  int64_t pad;
  __host__ __device__ int blocks() const { return (key1 - key0 + kBlock - 1) / kBlock; }
};
static_assert(sizeof(AttendSet) == 48, "AttendSet layout");

struct AttendSession {
  int32_t status, n, t0;    // rows in use, their first place in row_of
  int32_t leaf;             // the first set over the keys of its own; -1: no rows
  int32_t node[2];          // the first sets over shared keys, -1: none
  int32_t pad[2];
};

struct AttendHead {
  int64_t total, piece;  // blocks of all sets and heads, of a piece
  int32_t n_sets, pad[3];
};

struct AttendPlan {
  AttendHead* head;
  AttendSession* sess;  // [B]
  int4* starts;         // [kPieces]: set, key head, block; of pieces that begin before total
  int32_t* shared;      // [B]: keys shared with the session before
  int32_t* row_of;      // [B * R]: session * R + round row
  AttendSet* sets;
};

// Query rows of a set.
inline int rows_of_set(int64_t rows, int head_dim) {
  if (rows <= 16) return 16;
  if (rows <= 32 || head_dim > 128) return 32;
  return 64;
}

struct PlanSizes {
  int64_t sets, bytes, sess, starts, shared, row_of, set_at;
};
inline PlanSizes plan_sizes(int32_t B, int32_t R, int32_t G, int32_t per) {
  PlanSizes z;
  // a session's own, and on two levels those of its run of sessions
  z.sets = (int64_t)B * (((int64_t)R * G + per - 1) / per) +
           2 * (((int64_t)B * R * G + per - 1) / per + B / 2 + 1);
  int64_t at = 256;
  const auto take = [&at](int64_t n) {
    const int64_t here = at;
    at = (at + n + 255) / 256 * 256;
    return here;
  };
  z.sess = take((int64_t)B * sizeof(AttendSession));
  z.starts = take(kPieces * sizeof(int4));
  z.shared = take((int64_t)B * 4);
  z.row_of = take((int64_t)B * R * 4);
  z.set_at = take(z.sets * sizeof(AttendSet));
  z.bytes = at;
  return z;
}
inline AttendPlan plan_of(const PlanSizes& z, void* p) {
  char* c = (char*)p;
  return AttendPlan{(AttendHead*)c, (AttendSession*)(c + z.sess), (int4*)(c + z.starts),
                    (int32_t*)(c + z.shared), (int32_t*)(c + z.row_of), (AttendSet*)(c + z.set_at)};
}

}  // namespace sv
