// sv_plan.hip -- sv_cache_plan: which keys and rows of a round's attention go
// together, and where its line of work is cut.
#include "sv_attend.hpp"

namespace sv {
namespace {

constexpr int kOne = 1024;
constexpr int kPer = SV_CACHE_B_MAX / kOne;
constexpr int kNone = 0x7FFFFFFF;

struct PlanArgs {
  CacheView c;
  AttendPlan p;
  const int32_t *slots, *rows;
  int32_t* status;
  int32_t G, B, R, per;  // query heads a key head; rows of a set
  int32_t least;         // keys shared that are worth a set of their own
};

__device__ inline int place_of(const PlanArgs& a, int b) { return a.slots ? a.slots[b] : b; }

// A workgroup a session: the keys in leading pages that it has in common with the
// session before it, in whole blocks (and pages, which are powers of two like them).
constexpr int kShared = 256;
__global__ __launch_bounds__(kShared) void k_shared(PlanArgs a) {
  __shared__ int first;
  const CacheView& c = a.c;
  const int b = blockIdx.x, h = place_of(a, b);
  int keys = 0;
  if (h < 0 || h >= c.n_slots) {
    keys = kNone;  // no session: the run goes on behind it
  } else {
    int q = b - 1;
    while (q >= 0 && (place_of(a, q) < 0 || place_of(a, q) >= c.n_slots)) --q;
    if (q >= 0) {
      const int g = place_of(a, q);
      const int len = min(max(c.lens[h], 0), max(c.lens[g], 0));
      const int held = min(min(c.held[h], c.held[g]), c.max_pages);
      const int n = min(len >> c.shift, held);
      const int32_t *x = c.table + (int64_t)h * c.max_pages, *y = c.table + (int64_t)g * c.max_pages;
      if (threadIdx.x == 0) first = n;
      __syncthreads();
      for (int base = 0; base < n; base += kShared) {
        const int i = base + threadIdx.x;
        const bool differ = i < n && x[i] != y[i];
        if (differ) atomicMin(&first, i);
        if (__syncthreads_or(differ)) break;
      }
      __syncthreads();
      const int whole = max(kBlock, c.page());
      keys = (int)(((int64_t)first << c.shift) / whole * whole);
      if (keys < a.least) keys = 0;
    }
  }
  if (threadIdx.x == 0) a.p.shared[b] = keys;
}

__global__ __launch_bounds__(kOne) void k_plan(PlanArgs a) {
  // by session
  __shared__ int32_t t_at[SV_CACHE_B_MAX + 1], set_at[SV_CACHE_B_MAX];
  __shared__ int64_t cum_at[SV_CACHE_B_MAX];
  // by run, of both levels: first session, shared keys
  __shared__ int32_t first[2][SV_CACHE_B_MAX + 1], depth[2][SV_CACHE_B_MAX];
  __shared__ int64_t smem[kOne / kWave];
  const CacheView& c = a.c;
  const int tid = threadIdx.x;
  int st[kPer], n[kPer], len[kPer], slot[kPer], run[2][kPer], shared[kPer];

  // the sessions' rows
  int64_t rows_all = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    if (i * kOne >= a.B) break;
    const int b = i * kOne + tid;
    st[i] = n[i] = len[i] = 0, slot[i] = -1, shared[i] = kNone;
    if (b < a.B) {
      const int h = place_of(a, b);
      const int rows = a.rows ? a.rows[b] : a.R;
      shared[i] = a.p.shared[b];
      if (h < -1 || h >= c.n_slots) {
        st[i] = SV_S_BAD_CACHE;
      } else if (h >= 0) {
        if (rows < 0 || rows > a.R) {
          st[i] = SV_S_LIMIT;
        } else if (rows > 0) {
          // the rows' positions must lie in pages of the session's own
          const int64_t at = c.lens[h], end = at + rows;
          const int held = min(c.held[h], c.max_pages);
          bool ok = at >= 0 && end <= (int64_t)held << c.shift;
          for (int64_t p = at >> c.shift; ok && p <= (end - 1) >> c.shift; ++p) {
            const int page = c.table[(int64_t)h * c.max_pages + p];
            ok = page >= 0 && page < c.n_pages && c.refs[page] == 1;
          }
          if (ok) {
            n[i] = rows, len[i] = (int)at, slot[i] = h;
          } else {
            st[i] = SV_S_BAD_CACHE;
          }
        }
      }
    }
    int64_t total;
    const int64_t t = rows_all + block_incl_scan<kOne, int64_t>(n[i], smem, total) - n[i];
    if (b < a.B) t_at[b] = (int)t;
    for (int r = 0; r < n[i]; ++r) a.p.row_of[t + r] = b * a.R + r;
    rows_all += total;
  }
  if (tid == 0) t_at[a.B] = (int)rows_all;

  // runs of sessions that share their first keys; in them, runs that share more
  int runs[2];
#pragma unroll
  for (int level = 0; level < 2; ++level) {
    int64_t before = 0;
    for (int i = tid; i < a.B; i += kOne) depth[level][i] = kNone;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      if (i * kOne >= a.B) break;
      const int b = i * kOne + tid;
      int least = 1;
      if (level == 1 && b < a.B) {
        const int d = depth[0][run[0][i]];
        least = (d == kNone ? 0 : d) + a.least;
      }
      const bool starts = b < a.B && (b == 0 || shared[i] < least || (level == 1 && first[0][run[0][i]] == b));
      int64_t total;
      run[level][i] = (int)(before + block_incl_scan<kOne, int64_t>(starts, smem, total)) - 1;
      if (starts) first[level][run[level][i]] = b;
      else if (b < a.B) atomicMin(&depth[level][run[level][i]], shared[i]);
      before += total;
    }
    runs[level] = (int)before;
    if (tid == 0) first[level][runs[level]] = a.B;
    __syncthreads();
  }

  // the sets of every session: its runs' where they begin with it, then its own
  int own[kPer], key0[kPer], k1[kPer], d1[kPer], d2[kPer], n1[kPer], n2[kPer];
  int64_t sets_all = 0, cum_all = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    if (i * kOne >= a.B) break;
    const int b = i * kOne + tid;
    own[i] = key0[i] = d1[i] = d2[i] = n1[i] = n2[i] = k1[i] = 0;
    if (b < a.B) {
      const int r1 = run[0][i], r2 = run[1][i];
      d1[i] = depth[0][r1] == kNone ? 0 : depth[0][r1];
      d2[i] = depth[1][r2] == kNone ? d1[i] : depth[1][r2];
      const int64_t rows1 = (int64_t)(t_at[first[0][r1 + 1]] - t_at[first[0][r1]]) * a.G;
      const int64_t rows2 = (int64_t)(t_at[first[1][r2 + 1]] - t_at[first[1][r2]]) * a.G;
      if (d1[i] > 0) n1[i] = (int)((rows1 + a.per - 1) / a.per);
      if (d2[i] > d1[i]) n2[i] = (int)((rows2 + a.per - 1) / a.per);
      key0[i] = d2[i], k1[i] = len[i] + n[i];
      if (n[i] > 0) own[i] = (int)(((int64_t)n[i] * a.G + a.per - 1) / a.per);
    }
    const int at1 = b < a.B && first[0][run[0][i]] == b ? n1[i] : 0;
    const int at2 = b < a.B && first[1][run[1][i]] == b ? n2[i] : 0;
    const int64_t sets = (int64_t)at1 + at2 + own[i];
    const int64_t blocks = (int64_t)at1 * (d1[i] / kBlock) + (int64_t)at2 * ((d2[i] - d1[i]) / kBlock) +
                           (int64_t)own[i] * ((k1[i] - key0[i] + kBlock - 1) / kBlock);
    int64_t total;
    const int64_t s = sets_all + block_incl_scan<kOne, int64_t>(sets, smem, total) - sets;
    sets_all += total;
    const int64_t cum = cum_all + block_incl_scan<kOne, int64_t>(blocks, smem, total) - blocks;
    cum_all += total;
    if (b < a.B) {
      set_at[b] = (int)s;
      cum_at[b] = cum;
    }
  }
  __syncthreads();
  // written by a wave a session
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    if (i * kOne >= a.B) break;
    const int b = i * kOne + tid;
    if (b < a.B) {
      const int f1 = first[0][run[0][i]], f2 = first[1][run[1][i]];
      const bool begins1 = f1 == b, begins2 = f2 == b;
      int s = set_at[b];
      int64_t cum = cum_at[b];
      if (begins1 && n1[i] > 0) {
        const int rows = (t_at[first[0][run[0][i] + 1]] - t_at[b]) * a.G;
        // a run's pages are in the list of any of its sessions that has rows
        for (int k = 0; k < n1[i]; ++k, ++s, cum += d1[i] / kBlock)
          a.p.sets[s] = AttendSet{t_at[b], k * a.per, min(a.per, rows - k * a.per), 0, d1[i], -1,
                                  kFar, 0, cum, 0};
      }
      if (begins2 && n2[i] > 0) {
        const int rows = (t_at[first[1][run[1][i] + 1]] - t_at[b]) * a.G;
        for (int k = 0; k < n2[i]; ++k, ++s, cum += (d2[i] - d1[i]) / kBlock)
          a.p.sets[s] = AttendSet{t_at[b], k * a.per, min(a.per, rows - k * a.per), d1[i], d2[i], -1,
                                  kFar, 0, cum, 0};
      }
      const int leaf = s;
      const int blocks = (k1[i] - key0[i] + kBlock - 1) / kBlock;
      for (int k = 0; k < own[i]; ++k, ++s, cum += blocks)
        a.p.sets[s] = AttendSet{t_at[b], k * a.per, min(a.per, n[i] * a.G - k * a.per), key0[i], k1[i],
                                slot[i], len[i], d2[i] == 0, cum, 0};
      const int s1 = set_at[f1];
      const int s2 = set_at[f2] + (first[0][run[0][i]] == f2 ? n1[i] : 0);
      a.p.sess[b] = AttendSession{st[i], n[i], t_at[b], n[i] > 0 ? leaf : -1,
                                  {n[i] > 0 && n1[i] > 0 ? s1 : -1, n[i] > 0 && n2[i] > 0 ? s2 : -1},
                                  {0, 0}};
      if (a.status) a.status[b] = st[i];
    }
  }
  __syncthreads();
  // a run's list of pages: that of the session of its first row
  for (int64_t s = tid; s < sets_all; s += kOne)
    if (a.p.sets[s].slot < 0) a.p.sets[s].slot = place_of(a, a.p.row_of[a.p.sets[s].t0] / a.R);
  const int64_t total = cum_all * c.n_kv;
  const int64_t piece = (total + kPieces - 1) / kPieces;
  if (tid == 0) *a.p.head = AttendHead{total, piece, (int32_t)sets_all, {0, 0, 0}};
  for (int i = tid; i < kPieces; i += kOne) {
    const int64_t x = i * piece;
    if (x >= total) continue;
    int64_t lo = 0, hi = sets_all - 1;
    while (lo < hi) {
      const int64_t mid = (lo + hi + 1) / 2;
      if (a.p.sets[mid].cum * c.n_kv <= x) lo = mid;
      else hi = mid - 1;
    }
    const AttendSet& set = a.p.sets[lo];
    const int64_t in = x - set.cum * c.n_kv;
    a.p.starts[i] = make_int4((int)lo, (int)(in / set.blocks()), (int)(in % set.blocks()), 0);
  }
}

bool sizes_ok(const sv_cache* c, int32_t n_heads, int32_t B, int32_t R) {
  return cache_ok(c) && n_heads >= 1 && n_heads <= 1024 && n_heads % c->n_kv == 0 && B >= 1 &&
         B <= SV_CACHE_B_MAX && R >= 1 && R <= SV_M_MAX + 1;
}

}  // namespace
}  // namespace sv

extern "C" size_t sv_cache_plan_bytes(const sv_cache* cache, int32_t n_heads, int32_t B, int32_t R) {
  using namespace sv;
  if (!sizes_ok(cache, n_heads, B, R)) return 0;
  const int G = n_heads / cache->n_kv;
  return (size_t)plan_sizes(B, R, G, rows_of_set((int64_t)R * G, cache->head_dim)).bytes;
}

extern "C" int sv_cache_plan(const sv_cache* cache, const int32_t* slots, const int32_t* rows,
                             int32_t n_heads, int32_t B, int32_t R, int32_t* status, void* plan,
                             size_t plan_bytes, void* stream) {
  using namespace sv;
  if (!sizes_ok(cache, n_heads, B, R) || !sessions_ok(cache, slots, B) || !plan) return SV_ERR_ARG;
  if ((uintptr_t)plan % 16 != 0) return SV_ERR_ARG;
  const int G = n_heads / cache->n_kv;
  const int per = rows_of_set((int64_t)R * G, cache->head_dim);
  const PlanSizes z = plan_sizes(B, R, G, per);
  if (plan_bytes < (size_t)z.bytes) return SV_ERR_WORKSPACE;
  hipStream_t st = (hipStream_t)stream;
  (void)hipGetLastError();
  const PlanArgs a = {view_of(cache), plan_of(z, plan), slots, rows, status, G, B, R, per, 256};
  hipLaunchKernelGGL(k_shared, dim3(B), dim3(kShared), 0, st, a);
  hipLaunchKernelGGL(k_plan, dim3(1), dim3(kOne), 0, st, a);
  return hipGetLastError() == hipSuccess ? SV_OK : SV_ERR_DEVICE;
}
