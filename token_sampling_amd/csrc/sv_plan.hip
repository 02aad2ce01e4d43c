// sv_plan.hip -- sv_cache_plan: which keys and rows of a round's attention go
// together, and where its line of work is cut.
#include "sv_attend.hpp"

namespace sv {
namespace {

constexpr int kOne = 1024;
constexpr int kNone = 0x7FFFFFFF;

struct PlanArgs {
  CacheView c;
  AttendPlan p;
  const int32_t *slots, *rows;
  int32_t* status;
  int32_t G, B, R;       // query heads a key head
  int32_t narrow, wide;  // rows of a set
  int32_t pieces[2];
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
    }
  }
  if (threadIdx.x == 0) a.p.shared[b] = keys;
}

// Rows over the same keys as sets of a line: the number of sets, equal but for the
// last, in whole tiles of 16 rows.
struct Cut {
  int line, n, per;
};
__device__ inline Cut cut_rows(const PlanArgs& a, int64_t rows) {
  if (rows <= a.narrow) return Cut{kNarrow, rows > 0, a.narrow};
  const int n = (int)((rows + a.wide - 1) / a.wide);
  return Cut{kWide, n, (int)((rows + n - 1) / n + 15) / 16 * 16};
}

// The keys of a session's own, behind the `from` that it shares: where those end that
// go into wide sets (whole blocks that all rows see, where the rows are many).
__device__ inline int clear_end(const PlanArgs& a, int rows, int len, int from) {
  return (int64_t)rows * a.G > a.narrow ? max(from, len / kBlock * kBlock) : from;
}

// One workgroup, kPer sessions a thread.  12 us for one session, 25 for 1024: chains of
// dependent loads and a dozen barriers, once a round for all layers.  With four sessions a
// thread 540 registers spill; with k_shared 56 us for 1025 sessions, 74 for 2048, 132 for
// 4096.
template <int kPer>
__global__ __launch_bounds__(kOne) void k_plan(PlanArgs a) {
  // by session: the first row's place; in each line the first set, and the blocks
  // before it
  __shared__ int32_t t_at[SV_CACHE_B_MAX + 1], set_at[2][SV_CACHE_B_MAX + 1];
  __shared__ int64_t cum_at[SV_CACHE_B_MAX];
  // by run, of both levels: first session, shared keys
  __shared__ int32_t first[2][SV_CACHE_B_MAX + 1], depth[2][SV_CACHE_B_MAX];
  __shared__ int64_t smem[kOne / kWave];
  const CacheView& c = a.c;
  const int tid = threadIdx.x;
  const int many = (int64_t)a.R * a.G > a.narrow;  // whether sets of the third kind can occur
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
          // the rows' positions must lie in pages of the session's own: at most
          // four, looked up side by side
          static_assert((SV_M_MAX + 1 + 30) / 32 + 1 <= 4, "pages of a round's rows");
          const int64_t at = c.lens[h], end = at + rows;
          const int held = min(c.held[h], c.max_pages);
          bool ok = at >= 0 && end <= (int64_t)held << c.shift;
          if (ok) {
            const int32_t* list = c.table + (int64_t)h * c.max_pages;
            const int p0 = (int)(at >> c.shift), p1 = (int)((end - 1) >> c.shift);
            int page[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) page[k] = list[min(p0 + k, p1)];
#pragma unroll
            for (int k = 0; k < 4; ++k)
              ok = ok & (page[k] >= 0) & (page[k] < c.n_pages) &
                   (c.refs[min(max(page[k], 0), c.n_pages - 1)] == 1);
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
    rows_all += total;
  }
  if (tid == 0) t_at[a.B] = (int)rows_all;
  __syncthreads();
  for (int b = tid / kWave; b < a.B; b += kOne / kWave)  // a wave a session
    for (int r = tid % kWave; r < t_at[b + 1] - t_at[b]; r += kWave) a.p.row_of[t_at[b] + r] = b * a.R + r;

  // runs of sessions that share their first keys; in them, runs that share more
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
        least = (d == kNone ? 0 : d) + kBlock;
      }
      const bool starts = b < a.B && (b == 0 || shared[i] < least || (level == 1 && first[0][run[0][i]] == b));
      int64_t total;
      run[level][i] = (int)(before + block_incl_scan<kOne, int64_t>(starts, smem, total)) - 1;
      if (starts) first[level][run[level][i]] = b;
      else if (b < a.B) atomicMin(&depth[level][run[level][i]], shared[i]);
      before += total;
    }
    if (tid == 0) first[level][before] = a.B;
    __syncthreads();
  }

  // every session's sets: its runs' where they begin with it, then its own
  Cut cut[kKinds][kPer];
  int key[kKinds][kPer];  // where their keys end
  int64_t cum[2][kPer], sets_all[2] = {0, 0}, cum_all[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    if (i * kOne >= a.B) break;
    const int b = i * kOne + tid;
    int64_t sets[2] = {0, 0}, blocks[2] = {0, 0};
#pragma unroll
    for (int k = 0; k < kKinds; ++k) cut[k][i] = Cut{0, 0, 16}, key[k][i] = 0;
    if (b < a.B) {
      int from = 0;
#pragma unroll
      for (int k = 0; k < kKinds; ++k) {
        bool begins = true;
        if (k < 2) {
          const int r = run[k][i];
          int d = depth[k][r];
          if (d == kNone || d - from < worth(c.n_kv, c.head_dim, first[k][r + 1] - first[k][r])) d = from;
          key[k][i] = d;
          if (d > from) cut[k][i] = cut_rows(a, (int64_t)(t_at[first[k][r + 1]] - t_at[first[k][r]]) * a.G);
          begins = first[k][r] == b;
        } else if (k == 2) {
          key[k][i] = clear_end(a, n[i], len[i], from);
          if (key[k][i] > from) cut[k][i] = cut_rows(a, (int64_t)n[i] * a.G);
        } else {
          key[k][i] = len[i] + n[i];
          cut[k][i] = Cut{kNarrow, (n[i] * a.G + a.narrow - 1) / a.narrow, a.narrow};
        }
        if (begins && cut[k][i].n > 0) {
          const int64_t nb = (key[k][i] - from + kBlock - 1) / kBlock;
          const bool wide = cut[k][i].line == kWide;  // no array is indexed: it would leave the registers
          sets[0] += wide ? 0 : cut[k][i].n, sets[1] += wide ? cut[k][i].n : 0;
          blocks[0] += wide ? 0 : cut[k][i].n * nb, blocks[1] += wide ? cut[k][i].n * nb : 0;
        }
        from = key[k][i];
      }
    }
#pragma unroll
    for (int line = 0; line < 2; ++line) {
      int64_t total;
      const int64_t s = sets_all[line] + block_incl_scan<kOne, int64_t>(sets[line], smem, total) - sets[line];
      sets_all[line] += total;
      cum[line][i] = cum_all[line] + block_incl_scan<kOne, int64_t>(blocks[line], smem, total) - blocks[line];
      cum_all[line] += total;
      if (b < a.B) set_at[line][b] = (int)s;
    }
  }
  if (tid < 2) set_at[tid][a.B] = (int)sets_all[tid];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    if (i * kOne >= a.B) break;
    const int b = i * kOne + tid;
    if (b >= a.B) continue;
    AttendSession ss = {st[i], n[i], t_at[b], {-1, -1, -1, -1}, 0};
    int s[2] = {set_at[0][b], set_at[1][b]};
    int64_t x[2] = {cum[0][i], cum[1][i]};
    int from = 0;
#pragma unroll
    for (int k = 0; k < kKinds; ++k) {
      const Cut& cc = cut[k][i];
      const int f = k < 2 ? first[k][run[k][i]] : b;
      if (cc.n > 0) {
        if (f == b) {
          const int rows = k < 2 ? (t_at[first[k][run[k][i] + 1]] - t_at[b]) * a.G : n[i] * a.G;
          // a run's list of pages: that of the session of its first row
          const int list = k < 2 ? place_of(a, a.p.row_of[t_at[b]] / a.R) : slot[i];
          const int nb = (key[k][i] - from + kBlock - 1) / kBlock;
          int at = cc.line ? s[1] : s[0];
          int64_t y = cc.line ? x[1] : x[0];
          if (n[i] > 0 || k < 2) ss.first[k] = 2 * at + cc.line;
          AttendSet* sets = cc.line ? a.p.sets[1] : a.p.sets[0];
          for (int q = 0; q < cc.n; ++q, ++at, y += nb)
            sets[at] = AttendSet{t_at[b], q * cc.per, min(cc.per, rows - q * cc.per), from,
                                 key[k][i], list, k < 3 ? kFar : len[i], k == 3 && from == 0, y, cc.per,
                                 k < 2 ? many + 1 + k : 3 - k};
          if (cc.line) s[1] = at, x[1] = y;
          else s[0] = at, x[0] = y;
        } else {
          // behind the sets that session f has in this line for a run of the level above
          int at = cc.line ? set_at[1][f] : set_at[0][f];
          if (k == 1 && first[0][run[0][i]] == f && cut[0][i].n > 0 && cut[0][i].line == cc.line)
            at += cut[0][i].n;
          ss.first[k] = 2 * at + cc.line;
        }
      }
      from = key[k][i];
    }
    if (n[i] == 0) ss.first[0] = ss.first[1] = -1;
    a.p.sess[b] = ss;
    if (a.status) a.status[b] = st[i];
  }

  // where each line's pieces begin
#pragma unroll
  for (int line = 0; line < 2; ++line) {
    const int64_t total = cum_all[line] * c.n_kv;
    const int64_t piece = (total + a.pieces[line] - 1) / a.pieces[line];
    if (tid == 0) {
      a.p.head->total[line] = total;
      a.p.head->piece[line] = piece;
      a.p.head->blocks[line] = cum_all[line];
      a.p.head->sets[line] = (int)sets_all[line];
    }
    if (total == 0) continue;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      if (i * kOne >= a.B) break;
      if (i * kOne + tid < a.B) cum_at[i * kOne + tid] = cum[line][i];
    }
    __syncthreads();
    const int64_t x = tid * piece;
    if (tid < a.pieces[line] && x < total) {
      const int64_t head = x / cum_all[line], y = x - head * cum_all[line];
      int lo = 0, hi = a.B - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (cum_at[mid] <= y) lo = mid;
        else hi = mid - 1;
      }
      const AttendSet* sets = a.p.sets[line];
      hi = set_at[line][lo + 1] - 1, lo = set_at[line][lo];
      while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (sets[mid].cum <= y) lo = mid;
        else hi = mid - 1;
      }
      a.p.starts[line][tid] = make_int4(lo, (int)head, (int)(y - sets[lo].cum), 0);
    }
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
  return (size_t)plan_sizes(B, R, G, cache->head_dim).bytes;
}

extern "C" int sv_cache_plan(const sv_cache* cache, const int32_t* slots, const int32_t* rows,
                             int32_t n_heads, int32_t B, int32_t R, int32_t* status, void* plan,
                             size_t plan_bytes, void* stream) {
  using namespace sv;
  if (!sizes_ok(cache, n_heads, B, R) || !sessions_ok(cache, slots, B) || !plan) return SV_ERR_ARG;
  if ((uintptr_t)plan % 16 != 0) return SV_ERR_ARG;
  const int G = n_heads / cache->n_kv;
  const PlanSizes z = plan_sizes(B, R, G, cache->head_dim);
  if (plan_bytes < (size_t)z.bytes) return SV_ERR_WORKSPACE;
  hipStream_t st = (hipStream_t)stream;
  (void)hipGetLastError();
  const PlanArgs a = {view_of(cache), plan_of(z, plan), slots, rows, status, G, B, R,
                      narrow_rows((int64_t)R * G, cache->head_dim), wide_rows(cache->head_dim),
                      {kPieces[0], kPieces[1]}};
  hipLaunchKernelGGL(k_shared, dim3(B), dim3(kShared), 0, st, a);
  if (B <= kOne) hipLaunchKernelGGL(k_plan<1>, dim3(1), dim3(kOne), 0, st, a);
  else hipLaunchKernelGGL(k_plan<SV_CACHE_B_MAX / kOne>, dim3(1), dim3(kOne), 0, st, a);
  return hipGetLastError() == hipSuccess ? SV_OK : SV_ERR_DEVICE;
}
