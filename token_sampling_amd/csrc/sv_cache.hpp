// sv_cache.hpp -- what the cache's kernels share: the host's checks of sv_cache,
// and the places of a page's elements.
#pragma once

#include "sv_common.hpp"

namespace sv {

typedef unsigned int u32x4 __attribute__((ext_vector_type(4), may_alias));

// The cache as the kernels take it.
struct CacheView {
  char *k, *v;
  int32_t *table, *lens, *held, *refs;
  int32_t n_layers, n_pages, n_kv, shift, head_dim, n_slots, max_pages;  // page = 1 << shift
  __host__ __device__ int page() const { return 1 << shift; }
  // elements of a head's part of a page, of a page, and of a layer
  __host__ __device__ int64_t head_elems() const { return (int64_t)head_dim << shift; }
  __host__ __device__ int64_t page_elems() const { return head_elems() * n_kv; }
  __host__ __device__ int64_t layer_elems() const { return page_elems() * n_pages; }
};

inline bool cache_ok(const sv_cache* c) {
  if (!c || !c->k || !c->v || !c->table || !c->lens || !c->held || !c->refs) return false;
  if (((uintptr_t)c->k | (uintptr_t)c->v | (uintptr_t)c->refs) % 16 != 0) return false;
  if (c->dtype != SV_BF16 && c->dtype != SV_FP16) return false;
  if (c->page != 32 && c->page != 64 && c->page != 128 && c->page != 256) return false;
  if (c->head_dim != 64 && c->head_dim != 96 && c->head_dim != 128 && c->head_dim != 256) return false;
  if (c->n_layers < 1 || c->n_layers > 4096 || c->n_kv < 1 || c->n_kv > 1024) return false;
  if (c->n_pages < 1 || c->n_pages > SV_CACHE_PAGES_MAX) return false;
  if (c->max_pages < 1 || c->max_pages > SV_CACHE_PAGES_MAX) return false;
  return c->n_slots >= 1 && c->n_slots <= SV_CACHE_SLOTS_MAX;
}

inline CacheView view_of(const sv_cache* c) {
  const int shift = c->page == 32 ? 5 : c->page == 64 ? 6 : c->page == 128 ? 7 : 8;
  return CacheView{(char*)c->k, (char*)c->v, c->table, c->lens, c->held, c->refs, c->n_layers,
                   c->n_pages, c->n_kv, shift, c->head_dim, c->n_slots, c->max_pages};
}

// B sessions on slots, or on slot b.
inline bool sessions_ok(const sv_cache* c, const int32_t* slots, int32_t B) {
  return B >= 1 && B <= SV_CACHE_B_MAX && (slots || B <= c->n_slots);
}

// A page's elements stand as the 16x16x32 matrix instructions read them: 64
// lanes with 8 elements of 16 bits each, 1 KiB that a wave loads as it lies.
// Keys are that instruction's left operand with 16 keys in its rows and 32
// dimensions in its depth; values are the left operand with 16 dimensions in its
// rows and 32 keys in its depth.  Lane (g, m) = g * 16 + m then holds values of the
// keys 8 g .. 8 g + 7, and so that the scores come out with the same keys in the
// same lane, row m of the first (second) product over keys is key m / 4 * 8 + m %
// 4 (+ 4): the weights need no exchange between the two products.
// Elements from the start of a head's part of the page; u a token of the page.
__device__ inline int key_at(int u, int d, int head_dim) {
  const int t = u % 32, row = t / 8 * 4 + t % 4, half = t / 4 % 2;
  return ((u / 32 * 2 + half) * (head_dim / 32) + d / 32) * 512 + (d / 8 % 4 * 16 + row) * 8 + d % 8;
}
__device__ inline int value_at(int u, int d, int head_dim) {
  const int t = u % 32;
  return (u / 32 * (head_dim / 16) + d / 16) * 512 + (t / 8 * 16 + d % 16) * 8 + t % 8;
}

// Keeps x's computation where it stands, in every lane: what comes from other lanes must
// not be fetched under a branch that only some lanes take.
template <typename T>
__device__ inline void pin(T& x) {
  asm volatile("" : "+v"(x));
}

// Inclusive prefix sum over a workgroup of NT threads, and its total.
template <int NT, typename T>
__device__ inline T block_incl_scan(T v, T* smem, T& total) {
  const int wave = threadIdx.x / kWave;
  v = wave_incl_scan(v);
  __syncthreads();
  if (threadIdx.x % kWave == kWave - 1) smem[wave] = v;
  __syncthreads();
  T before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < NT / kWave; ++w) {
    if (w < wave) before += smem[w];
    all += smem[w];
  }
  total = all;
  return v + before;
}

}  // namespace sv
