// sv_cache.hip -- the pages of the cache: sv_cache_reserve, sv_cache_keep,
// sv_cache_fork, sv_cache_compact, and sv_cache_write.
//
// Which pages are free is what refs says (0), nothing else is kept, so the free
// pages' order is that of their numbers and the calls' results are functions of
// the state alone: adds on refs commute, and pages are handed out by prefix sums.
#include "sv_cache.hpp"

namespace sv {
namespace {

constexpr int kOne = 1024;                          // threads of the single workgroups
constexpr int kTile = 32 * kOne;                    // pages looked at together

struct Pair {
  int32_t src, dst, blocks, pad;  // pages, and how many blocks of 32 tokens
};

// The workspace of reserve and compact.
struct Scratch {
  int32_t* n_pairs;  // [1]
  Pair* pairs;       // reserve: [B]; compact: [n_pages / 2]
  int32_t* list;     // [n_pages] free pages in order
  int32_t* map;      // [n_pages]
};
size_t scratch_bytes(const sv_cache* c, int32_t B) {
  const size_t pairs = (size_t)(c->n_pages / 2 > B ? c->n_pages / 2 : B);
  return 256 + pairs * sizeof(Pair) + 2 * (size_t)c->n_pages * sizeof(int32_t);
}
Scratch scratch_of(const sv_cache* c, int32_t B, void* ws) {
  const size_t pairs = (size_t)(c->n_pages / 2 > B ? c->n_pages / 2 : B);
  Scratch s;
  s.n_pairs = (int32_t*)ws;
  s.pairs = (Pair*)((char*)ws + 256);
  s.list = (int32_t*)(s.pairs + pairs);
  s.map = s.list + c->n_pages;
  return s;
}

// Bit k: page p0 + k is free (want_free) or in use, of the 32 pages from p0.
__device__ inline uint32_t pages_word(const int32_t* refs, int p0, int n_pages, bool want_free) {
  uint32_t bits = 0;
  if (p0 + 32 <= n_pages) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const u32x4 r = *(const u32x4*)(refs + p0 + 4 * i);
#pragma unroll
      for (int j = 0; j < 4; ++j) bits |= (uint32_t)((r[j] == 0) == want_free) << (4 * i + j);
    }
  } else {
    for (int i = 0; p0 + i < n_pages && i < 32; ++i)
      bits |= (uint32_t)((refs[p0 + i] == 0) == want_free) << i;
  }
  return bits;
}

// The lowest pages that are free (or in use), in order, from page `from` on and
// before `to`, at most n of them, into list; returns how many there were.
__device__ inline int64_t list_pages(const int32_t* refs, int from, int to, int n_pages, bool want_free,
                                     int64_t n, int32_t* list, int64_t* smem) {
  int64_t found = 0;
  for (int base = from / 32 * 32; base < to && found < n; base += kTile) {
    const int p0 = base + 32 * (int)threadIdx.x;
    uint32_t bits = p0 < to ? pages_word(refs, p0, n_pages, want_free) : 0;
    if (p0 < from) bits &= p0 + 32 <= from ? 0u : ~0u << (from - p0);
    if (p0 < to && to - p0 < 32) bits &= (1u << (to - p0)) - 1;
    int64_t total;
    const int cnt = __popc(bits);
    int64_t at = found + block_incl_scan<kOne, int64_t>(cnt, smem, total) - cnt;
    for (; bits && at < n; bits &= bits - 1, ++at) list[at] = p0 + __ffs(bits) - 1;
    found += total;
  }
  return found < n ? found : n;
}

struct ReserveArgs {
  CacheView c;
  Scratch s;
  const int32_t *slots, *add;
  int32_t* status;
  int32_t B;
};

// One workgroup, kPer sessions a thread: what the sessions want, the free pages, and
// who gets which.  13 us for 1024 sessions in a pool of 194000 pages, 8 in a small one: a
// chain of dependent loads, and 32768 pages' refs at a time until enough are found.  With
// four sessions a thread 88 registers spill; that and k_copy without a pair take 8 us for
// 2048 sessions that want no pages and 16 for 4096 (1024: 6).
template <int kPer>
__global__ __launch_bounds__(kOne) void k_reserve(ReserveArgs a) {
  __shared__ uint32_t seen[SV_CACHE_SLOTS_MAX / 32], twice[SV_CACHE_SLOTS_MAX / 32];
  __shared__ int64_t smem[kOne / kWave];
  __shared__ int32_t n_long, n_pairs, longs[kOne];
  const CacheView& c = a.c;
  const int tid = threadIdx.x;
  if (a.slots) {
    for (int i = tid; i < (c.n_slots + 31) / 32; i += kOne) seen[i] = twice[i] = 0;
    __syncthreads();
    for (int b = tid; b < a.B; b += kOne) {
      const int h = a.slots[b];
      if (h < 0 || h >= c.n_slots) continue;
      const uint32_t bit = 1u << (h % 32);
      if (atomicOr(seen + h / 32, bit) & bit) atomicOr(twice + h / 32, bit);
    }
  }
  if (tid == 0) n_pairs = 0;
  __syncthreads();
  int st[kPer], slot[kPer], len[kPer], held[kPer], more[kPer], old[kPer];
  int64_t first[kPer], want_all = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    if (i * kOne >= a.B) break;
    const int b = i * kOne + tid;
    st[i] = 0, slot[i] = -1, len[i] = held[i] = more[i] = 0, old[i] = -1;
    if (b < a.B) {
      const int h = a.slots ? a.slots[b] : b;
      const int add = a.add[b];
      if (h < -1 || h >= c.n_slots || (h >= 0 && a.slots && (twice[h / 32] >> (h % 32) & 1))) {
        st[i] = SV_S_BAD_CACHE;
      } else if (h >= 0) {
        len[i] = max(c.lens[h], 0), held[i] = min(max(c.held[h], 0), c.max_pages);
        const int64_t all = ((int64_t)len[i] + add + c.page() - 1) >> c.shift;
        if (add < 0 || all > c.max_pages) {
          st[i] = SV_S_LIMIT;
        } else {
          slot[i] = h;
          more[i] = all > held[i] ? (int)all - held[i] : 0;
          const int last = len[i] >> c.shift;
          if (add > 0 && last < held[i]) {
            const int p = c.table[(int64_t)h * c.max_pages + last];
            if (p >= 0 && p < c.n_pages && c.refs[p] > 1) old[i] = p;
          }
        }
      }
    }
    const int want = more[i] + (old[i] >= 0);
    int64_t total;
    first[i] = want_all + block_incl_scan<kOne, int64_t>(want, smem, total) - want;
    want_all += total;
  }
  const int64_t got =
      list_pages(c.refs, 0, c.n_pages, c.n_pages, true, want_all < c.n_pages ? want_all : c.n_pages,
                 a.s.list, smem);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    if (i * kOne >= a.B) break;
    const int b = i * kOne + tid;
    if (tid == 0) n_long = 0;
    __syncthreads();
    const int want = more[i] + (old[i] >= 0);
    if (slot[i] >= 0 && want > 0) {
      if (first[i] + want > got) {
        st[i] = SV_S_NO_PAGES;
      } else {
        int32_t* row = c.table + (int64_t)slot[i] * c.max_pages;
        int64_t at = first[i];
        if (old[i] >= 0) {
          const int p = a.s.list[at++], last = len[i] >> c.shift;
          row[last] = p;
          c.refs[p] = 1;
          atomicSub(c.refs + old[i], 1);
          const int part = len[i] & (c.page() - 1);
          if (part) a.s.pairs[atomicAdd(&n_pairs, 1)] = Pair{old[i], p, (part + 31) / 32, 0};
        }
        c.held[slot[i]] = held[i] + more[i];
        if (more[i] <= 8) {
          for (int j = 0; j < more[i]; ++j) {
            const int p = a.s.list[at + j];
            row[held[i] + j] = p;
            c.refs[p] = 1;
          }
        } else {
          longs[atomicAdd(&n_long, 1)] = tid;
        }
      }
    }
    if (b < a.B && a.status) a.status[b] = st[i];
    __syncthreads();
    // sessions that get many pages (prompts): the workgroup takes them one by one
    const int n_longs = n_long;
    for (int k = 0; k < n_longs; ++k) {
      __shared__ int64_t s_row, s_at;
      __shared__ int32_t s_n;
      if (tid == longs[k]) {
        s_row = (int64_t)slot[i] * c.max_pages + held[i];
        s_at = first[i] + (old[i] >= 0);
        s_n = more[i];
      }
      __syncthreads();
      for (int j = tid; j < s_n; j += kOne) {
        const int p = a.s.list[s_at + j];
        c.table[s_row + j] = p;
        c.refs[p] = 1;
      }
      __syncthreads();
    }
  }
  if (tid == 0) *a.s.n_pairs = n_pairs;
}

struct CopyArgs {
  CacheView c;
  const int32_t* n_pairs;
  const Pair* pairs;
  const int32_t* map;  // compact: the lists' pages to rename, else null
  const int32_t* used;
};

// Pages (or their first blocks) of every layer, a unit a layer and a plane of a pair:
// 40000 copies of 128 KiB, 6.4 GB read and written, take 1315 us (4.9 TB/s, what a large
// copy reaches); without a pair, the grid's 3.8 us.  Then the lists' entries are renamed
// where pages have moved.
constexpr int kCopy = 256;
__global__ __launch_bounds__(kCopy) void k_copy(CopyArgs a) {
  const CacheView& c = a.c;
  const int per = 2 * c.n_layers;
  const int64_t units = (int64_t)*a.n_pairs * per;
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const Pair p = a.pairs[u / per];
    const int layer = (int)(u % per) >> 1;
    char* pool = u % per & 1 ? c.v : c.k;
    const int64_t base = layer * c.layer_elems();
    const u32x4* src = (const u32x4*)(pool + 2 * (base + p.src * c.page_elems()));
    u32x4* dst = (u32x4*)(pool + 2 * (base + p.dst * c.page_elems()));
    const int part = p.blocks * 4 * c.head_dim;             // 16-byte vectors of a head
    const int head = (int)(c.head_elems() / 8);             // of a head's part of a page
    const int n = part * c.n_kv;
    for (int i = threadIdx.x; i < n; i += kCopy) {
      const int at = part == head ? i : i / part * head + i % part;
      dst[at] = src[at];
    }
  }
  if (a.map) {
    const int n_used = *a.used;
    for (int h = blockIdx.x; h < c.n_slots; h += gridDim.x) {
      int32_t* row = c.table + (int64_t)h * c.max_pages;
      const int held = min(c.held[h], c.max_pages);
      for (int i = threadIdx.x; i < held; i += kCopy) {
        const int p = row[i];
        if (p >= n_used && p < c.n_pages) row[i] = a.map[p];
      }
    }
  }
}

// One workgroup: U = the pages in use, the free ones before U, the used ones from U on.
struct CompactArgs {
  CacheView c;
  Scratch s;
  int32_t *used, *moved;
};
__global__ __launch_bounds__(kOne) void k_compact(CompactArgs a) {
  __shared__ int64_t smem[kOne / kWave];
  const CacheView& c = a.c;
  int64_t cnt = 0;
  for (int base = 0; base < c.n_pages; base += kTile) {
    const int p0 = base + 32 * (int)threadIdx.x;
    if (p0 < c.n_pages) cnt += __popc(pages_word(c.refs, p0, c.n_pages, false));
  }
  int64_t total;
  block_incl_scan<kOne, int64_t>(cnt, smem, total);
  const int U = (int)total;
  const int holes = (int)list_pages(c.refs, 0, U, c.n_pages, true, c.n_pages, a.s.list, smem);
  // as many used pages behind U; their list stands behind the holes'
  list_pages(c.refs, U, c.n_pages, c.n_pages, false, holes, a.s.list + holes, smem);
  __syncthreads();
  if (a.moved)
    for (int p = threadIdx.x; p < c.n_pages; p += kOne) a.moved[p] = c.refs[p] != 0 ? p : -1;
  __syncthreads();
  for (int i = threadIdx.x; i < holes; i += kOne) {
    const int to = a.s.list[i], from = a.s.list[holes + i];
    a.s.pairs[i] = Pair{from, to, c.page() / 32, 0};
    a.s.map[from] = to;
    c.refs[to] = c.refs[from];
    c.refs[from] = 0;
    if (a.moved) a.moved[from] = to;
  }
  if (threadIdx.x == 0) {
    *a.s.n_pairs = holes;
    *a.used = U;
  }
}

struct KeepArgs {
  CacheView c;
  const int32_t *slots, *count;
  int32_t* status;
  int32_t absolute, B;
};

// Whether x stands in the n values of list at another place than i; a wave's question.
__device__ inline bool listed_again(const int32_t* list, int n, int x, int i) {
  bool again = false;
  for (int j = threadIdx.x % kWave; j < n; j += kWave) again |= list[j] == x && j != i;
  return __any(again);
}

// A wave a session; 4.7 us for 1024 of them.
__global__ __launch_bounds__(kWave) void k_keep(KeepArgs a) {
  const CacheView& c = a.c;
  const int b = blockIdx.x;
  const int h = a.slots ? a.slots[b] : b;
  int st = 0;
  if (h < -1 || h >= c.n_slots || (h >= 0 && a.slots && listed_again(a.slots, a.B, h, b))) {
    st = SV_S_BAD_CACHE;
  } else if (h >= 0) {
    const int held = min(max(c.held[h], 0), c.max_pages);
    const int64_t count = a.count[b], len = a.absolute ? count : count + c.lens[h];
    if (count < 0 || len < 0 || len > (int64_t)held << c.shift) {
      st = SV_S_LIMIT;
    } else {
      const int stay = (int)((len + c.page() - 1) >> c.shift);
      int32_t* row = c.table + (int64_t)h * c.max_pages;
      for (int i = stay + (int)threadIdx.x; i < held; i += kWave) {
        const int p = row[i];
        row[i] = -1;
        if (p >= 0 && p < c.n_pages) atomicSub(c.refs + p, 1);
      }
      if (threadIdx.x == 0) {
        c.lens[h] = (int)len;
        c.held[h] = stay < held ? stay : held;
      }
    }
  }
  if (threadIdx.x == 0 && a.status) a.status[b] = st;
}

struct ForkArgs {
  CacheView c;
  const int32_t *src, *dst;
  int32_t* status;
  int32_t n;
};
constexpr int kFork = 256;
__global__ __launch_bounds__(kFork) void k_fork(ForkArgs a) {
  const CacheView& c = a.c;
  const int i = blockIdx.x;
  const int from = a.src[i], to = a.dst[i];
  int st = 0;
  if (from != -1 && to != -1) {
    // No other place may write this one's slots: every wave asks for itself, and
    // slots that pass are read by this workgroup while nobody writes them.
    if (from < 0 || from >= c.n_slots || to < 0 || to >= c.n_slots ||
        listed_again(a.dst, a.n, to, i) || listed_again(a.dst, a.n, from, -1) || c.held[to] != 0) {
      st = SV_S_BAD_CACHE;
    } else {
      __syncthreads();  // every wave has seen held[to] before it changes
      const int len = max(c.lens[from], 0);
      const int64_t need = ((int64_t)len + c.page() - 1) >> c.shift;
      const int n = (int)min(need, (int64_t)min(max(c.held[from], 0), c.max_pages));
      const int32_t* row = c.table + (int64_t)from * c.max_pages;
      int32_t* out = c.table + (int64_t)to * c.max_pages;
      for (int j = threadIdx.x; j < n; j += kFork) {
        const int p = row[j];
        out[j] = p;
        if (p >= 0 && p < c.n_pages) atomicAdd(c.refs + p, 1);
      }
      if (threadIdx.x == 0) {
        c.lens[to] = len;
        c.held[to] = n;
      }
    }
  }
  if (threadIdx.x == 0 && a.status) a.status[i] = st;
}

// ------------------------------------------------------------------- writing rows
struct WriteArgs {
  CacheView c;
  const char *k, *v;
  int64_t k_session, k_row, k_head, v_session, v_row, v_head;
  const int32_t *slots, *rows, *offsets;
  int64_t base;  // the layer's first element
  int32_t B, R, octets;
};
constexpr int kWrite = 256;

// A thread takes 8 dimensions of a head of the up to 8 rows whose positions share an
// octet of a page: the keys of each are a 16-byte piece as it comes, the values are
// turned in registers into 8 pieces of 8 tokens.  A wave's 512 pieces then change
// places in LDS, so that it stores them as they lie in the page, keys 64 bytes and
// values 1 KiB side by side (48 prompts of up to 5000 tokens, 8 heads of 128: 983 MB
// in 201 us, 4.9 TB/s, what a large copy reaches; stored as they come 345 us).  Pieces
// of an octet that the rows fill in part are read and written back: a round of 256
// sessions takes 8.5 us, its chain of lookups and a launch.
__device__ inline int64_t shfl64(int64_t x, int lane) {
  const uint32_t lo = __shfl((int)(uint32_t)x, lane), hi = __shfl((int)(uint32_t)(x >> 32), lane);
  return (int64_t)((uint64_t)hi << 32 | lo);
}
__global__ __launch_bounds__(kWrite) void k_write(WriteArgs a) {
  __shared__ u32x4 pieces[kWrite / kWave][kWave * 8];
  const CacheView& c = a.c;
  const int lane = threadIdx.x % kWave;
  u32x4* mine = pieces[threadIdx.x / kWave];
  const int groups = c.n_kv * (c.head_dim / 8);
  const int64_t all = (int64_t)a.octets * (a.offsets ? 1 : a.B) * groups;
  // whole waves go round, as they work together
  const int64_t step = (int64_t)gridDim.x * kWrite, waves_end = (all + kWave - 1) / kWave * kWave;
  for (int64_t w = (int64_t)blockIdx.x * kWrite + threadIdx.x; w < waves_end; w += step) {
    const int64_t item = w / groups;
    const int dg = (int)(w % groups), head = dg / (c.head_dim / 8), d = dg % (c.head_dim / 8) * 8;
    int b = 0, n = 0, lo = 0, octet = 0;
    if (w < all && a.offsets) {
      // session b's octets are the items from offsets[b] / 8 + 2 b on
      int left = 0, right = a.B - 1;
      while (left < right) {
        const int mid = (left + right + 1) / 2;
        if (min(max(a.offsets[mid], 0), a.R) / 8 + 2 * (int64_t)mid <= item) left = mid;
        else right = mid - 1;
      }
      b = left;
      lo = min(max(a.offsets[b], 0), a.R);
      n = min(max(a.offsets[b + 1], 0), a.R) - lo;
      octet = (int)(item - (lo / 8 + 2 * (int64_t)b));
    } else if (w < all) {
      b = (int)(item / a.octets);
      octet = (int)(item % a.octets);
      n = a.rows ? min(max(a.rows[b], 0), a.R) : a.R;
    }
    // items before the first session's (offsets[0] rows belong to none) have octet < 0
    const int h = n > 0 && octet >= 0 ? (a.slots ? a.slots[b] : b) : -1;
    const bool some = h >= 0 && h < c.n_slots;
    const int64_t len = some ? c.lens[h] : 0;
    const int64_t pos = (len / 8 + octet) * 8;  // the octet's first position
    const int e0 = some && pos < len ? (int)(len - pos) : 0;
    const int e1 = some && len >= 0 ? (int)min((int64_t)8, len + n - pos) : 0;
    // the rows, which do not wait for the page
    const int64_t row0 = lo + pos - len;  // row of element 0 of the octet (may lie before the rows)
    const char* kp = a.k + 2 * (b * a.k_session + row0 * a.k_row + head * a.k_head + d);
    const char* vp = a.v + 2 * (b * a.v_session + row0 * a.v_row + head * a.v_head + d);
    u32x4 kr[8], vr[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const bool in = e >= e0 && e < e1;
      kr[e] = in ? *(const u32x4*)(kp + 2 * e * a.k_row) : u32x4{0, 0, 0, 0};
      vr[e] = in ? *(const u32x4*)(vp + 2 * e * a.v_row) : u32x4{0, 0, 0, 0};
    }
    int page = -1;
    if (e1 > e0 && pos >> c.shift < min(c.held[h], c.max_pages)) {
      page = c.table[(int64_t)h * c.max_pages + (pos >> c.shift)];
      if (page < 0 || page >= c.n_pages || c.refs[page] != 1) page = -1;
    }
    const int u = (int)(pos & (c.page() - 1));
    const int64_t at = a.base + max(page, 0) * c.page_elems() + head * c.head_elems();
    const int64_t k_at = 2 * (at + key_at(u, d, c.head_dim)), v_at = 2 * (at + value_at(u, d, c.head_dim));
    const int span = page < 0 ? 0 : e0 | e1 << 4;  // 0: stores nothing
    // keys: four tokens of 16 threads at a time; of a thread's pieces the one of token e
    // stands at place e ^ lane % 8, so that neither side meets in one bank
#pragma unroll
    for (int e = 0; e < 8; ++e) mine[lane * 8 + (e ^ lane % 8)] = kr[e];
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int from = i / 2 * 16 + lane / 4, e = i % 2 * 4 + lane % 4;
      int64_t to = shfl64(k_at, from);
      int sp = __shfl(span, from);
      pin(to), pin(sp);
      const u32x4 x = mine[from * 8 + (e ^ from % 8)];
      if (e >= (sp & 15) && e < sp >> 4)
        *(u32x4*)(c.k + to + 2 * ((e / 4) * (c.head_dim / 32) * 512 + e % 4 * 8)) = x;
    }
    __builtin_amdgcn_wave_barrier();
    // values
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      u32x4 x;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t x0 = vr[2 * e][j / 2], x1 = vr[2 * e + 1][j / 2];
        x[e] = j % 2 ? x0 >> 16 | (x1 & 0xFFFF0000u) : (x0 & 0xFFFFu) | x1 << 16;
      }
      mine[lane * 8 + (j ^ lane % 8)] = x;
    }
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int from = i * 8 + lane / 8, j = lane % 8;
      int64_t to = shfl64(v_at, from);
      int sp = __shfl(span, from);
      pin(to), pin(sp);
      u32x4* out = (u32x4*)(c.v + to + 16 * j);
      const int f0 = sp & 15, f1 = sp >> 4;
      u32x4 x = mine[from * 8 + (j ^ from % 8)];
      if (f1 <= f0) continue;
      if (f0 > 0 || f1 < 8) {
        const u32x4 old = *out;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t mask = (2 * e >= f0 && 2 * e < f1 ? 0xFFFFu : 0u) |
                                (2 * e + 1 >= f0 && 2 * e + 1 < f1 ? 0xFFFF0000u : 0u);
          x[e] = (x[e] & mask) | (old[e] & ~mask);
        }
      }
      *out = x;
    }
    __builtin_amdgcn_wave_barrier();
  }
}

bool stride_ok(int64_t s) { return s >= 0 && s % 8 == 0 && s <= ((int64_t)1 << 40); }

}  // namespace
}  // namespace sv

extern "C" size_t sv_cache_workspace_bytes(const sv_cache* cache, int32_t B) {
  if (!sv::cache_ok(cache) || B < 1 || B > SV_CACHE_B_MAX) return 0;
  return sv::scratch_bytes(cache, B);
}

extern "C" int sv_cache_reserve(const sv_cache* cache, const int32_t* slots, const int32_t* add,
                                int32_t B, int32_t* status, void* workspace,
                                size_t workspace_bytes, void* stream) {
  using namespace sv;
  if (!cache_ok(cache) || !add || !workspace || !sessions_ok(cache, slots, B)) return SV_ERR_ARG;
  if ((uintptr_t)workspace % 16 != 0) return SV_ERR_ARG;
  if (workspace_bytes < scratch_bytes(cache, B)) return SV_ERR_WORKSPACE;
  hipStream_t st = (hipStream_t)stream;
  (void)hipGetLastError();
  const Scratch s = scratch_of(cache, B, workspace);
  const ReserveArgs a = {view_of(cache), s, slots, add, status, B};
  if (B <= kOne) hipLaunchKernelGGL(k_reserve<1>, dim3(1), dim3(kOne), 0, st, a);
  else hipLaunchKernelGGL(k_reserve<SV_CACHE_B_MAX / kOne>, dim3(1), dim3(kOne), 0, st, a);
  const CopyArgs p = {a.c, s.n_pairs, s.pairs, nullptr, nullptr};
  const int64_t units = (int64_t)B * 2 * cache->n_layers;
  hipLaunchKernelGGL(k_copy, dim3((unsigned)(units < 2048 ? units : 2048)), dim3(kCopy), 0, st, p);
  return hipGetLastError() == hipSuccess ? SV_OK : SV_ERR_DEVICE;
}

extern "C" int sv_cache_keep(const sv_cache* cache, const int32_t* slots, const int32_t* count,
                             int32_t absolute, int32_t B, int32_t* status, void* stream) {
  using namespace sv;
  if (!cache_ok(cache) || !count || !sessions_ok(cache, slots, B)) return SV_ERR_ARG;
  (void)hipGetLastError();
  const KeepArgs a = {view_of(cache), slots, count, status, absolute, B};
  hipLaunchKernelGGL(k_keep, dim3(B), dim3(kWave), 0, (hipStream_t)stream, a);
  return hipGetLastError() == hipSuccess ? SV_OK : SV_ERR_DEVICE;
}

extern "C" int sv_cache_fork(const sv_cache* cache, const int32_t* src, const int32_t* dst,
                             int32_t n, int32_t* status, void* stream) {
  using namespace sv;
  if (!cache_ok(cache) || !src || !dst || n < 1 || n > SV_CACHE_B_MAX) return SV_ERR_ARG;
  (void)hipGetLastError();
  const ForkArgs a = {view_of(cache), src, dst, status, n};
  hipLaunchKernelGGL(k_fork, dim3(n), dim3(kFork), 0, (hipStream_t)stream, a);
  return hipGetLastError() == hipSuccess ? SV_OK : SV_ERR_DEVICE;
}

extern "C" int sv_cache_compact(const sv_cache* cache, int32_t* used, int32_t* moved,
                                void* workspace, size_t workspace_bytes, void* stream) {
  using namespace sv;
  if (!cache_ok(cache) || !used || !workspace || (uintptr_t)workspace % 16 != 0) return SV_ERR_ARG;
  if (workspace_bytes < scratch_bytes(cache, 1)) return SV_ERR_WORKSPACE;
  hipStream_t st = (hipStream_t)stream;
  (void)hipGetLastError();
  const Scratch s = scratch_of(cache, 1, workspace);
  const CompactArgs a = {view_of(cache), s, used, moved};
  hipLaunchKernelGGL(k_compact, dim3(1), dim3(kOne), 0, st, a);
  const CopyArgs p = {a.c, s.n_pairs, s.pairs, s.map, used};
  hipLaunchKernelGGL(k_copy, dim3(2048), dim3(kCopy), 0, st, p);
  return hipGetLastError() == hipSuccess ? SV_OK : SV_ERR_DEVICE;
}

extern "C" int sv_cache_write(const sv_cache* cache, int32_t layer, const sv_rows* from,
                              const int32_t* slots, const int32_t* rows, const int32_t* offsets,
                              int32_t B, int32_t R, void* stream) {
  using namespace sv;
  if (!cache_ok(cache) || layer < 0 || layer >= cache->n_layers || !sessions_ok(cache, slots, B))
    return SV_ERR_ARG;
  if (!from || R < 0 || (R > 0 && (!from->k || !from->v)) || (rows && offsets)) return SV_ERR_ARG;
  if (((uintptr_t)from->k | (uintptr_t)from->v) % 16 != 0) return SV_ERR_ARG;
  if (!stride_ok(from->k_session) || !stride_ok(from->k_row) || !stride_ok(from->k_head) ||
      !stride_ok(from->v_session) || !stride_ok(from->v_row) || !stride_ok(from->v_head))
    return SV_ERR_ARG;
  if (R == 0) return SV_OK;
  WriteArgs a = {view_of(cache), (const char*)from->k, (const char*)from->v, from->k_session,
                 from->k_row, from->k_head, from->v_session, from->v_row, from->v_head, slots,
                 rows, offsets, 0, B, R, 0};
  a.base = layer * a.c.layer_elems();
  if (offsets) a.k_session = a.v_session = 0;
  // octets that n rows touch, wherever they begin: (n + 14) / 8 at most; in a line
  // a session's share of R / 8 + 2 B items holds as many
  a.octets = offsets ? R / 8 + 2 * B : (int)(((int64_t)R + 14) / 8);
  const int64_t all = (int64_t)a.octets * (offsets ? 1 : B) * cache->n_kv * (cache->head_dim / 8);
  const int64_t grid = (all + kWrite - 1) / kWrite;
  (void)hipGetLastError();
  hipLaunchKernelGGL(k_write, dim3((unsigned)(grid < (1 << 20) ? grid : 1 << 20)), dim3(kWrite), 0,
                     (hipStream_t)stream, a);
  return hipGetLastError() == hipSuccess ? SV_OK : SV_ERR_DEVICE;
}
