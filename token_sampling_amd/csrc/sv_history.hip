// sv_history.hip -- sv_count_tokens: notes prompt tokens and committed tokens
// in the history that sv_adjust_logits' penalties read.
//
// A token is an add on its count and an or on its bit; whole numbers, so the
// order of the atomics does not matter.  The committed tokens of 256 sessions
// take 2.3 us in a graph, a launch and four dependent loads.  64 prompts of up to
// 32768 tokens, V=128256, take 13 us: 7.6 to empty their slots (35 MB written,
// 4.6 TB/s), 5 to note 1e6 tokens.  The kernel and its workgroups go by the mean
// length, so a line with one long session among short ones is slow: 102400
// tokens of 256 sessions take 5.9 us in equal parts (prompts; outputs 9.7) and
// 110 (147) where one session has 100000 of them, which fits two workgroups of
// k_count_few; a call of its own takes it in 3.8 (8.8).
#include "sv_common.hpp"

namespace sv {
namespace {

typedef unsigned int u32x4 __attribute__((ext_vector_type(4), may_alias));
constexpr int kThreads = 256;
constexpr int kGridZ = 32768;  // sessions of a launch
// Up to so many tokens a session, k_count_few: prompts of 400 tokens take 2.7
// against 3.1 us (16 sessions), of 800 3.3 against 3.2, of 8000 15 against 4.4;
// outputs, whose counts k_count_many gathers over 8 ranges of ids at V=128256,
// 6.7 against 6.9 us at 2000 and 23 against 9.4 at 8000.
constexpr int kFewPrompt = 512, kFewOutput = 2048;

struct CountArgs {
  int32_t* counts;
  uint32_t* seen;
  const int32_t* slots;
  const int32_t* tokens;
  const int32_t* offsets;
  const int32_t* lens;
  int32_t n_slots, B, L, V, W, plane;
  int32_t b0;  // the launch's first session
};

__device__ inline int slot_of(const CountArgs& a, int b) {
  const int s = a.slots ? a.slots[b] : b;
  return s >= 0 && s < a.n_slots ? s : -1;
}

// The tokens [lo, hi) of session b.
__device__ inline void span_of(const CountArgs& a, int b, int64_t& lo, int64_t& hi) {
  if (a.offsets) {
    lo = a.offsets[b];
    hi = a.offsets[b + 1];
    lo = lo < 0 ? 0 : lo;
    hi = hi > a.L ? a.L : hi;
  } else {
    int n = a.lens ? a.lens[b] : a.L;
    n = n < 0 ? 0 : n > a.L ? a.L : n;
    lo = (int64_t)b * a.L;
    hi = lo + n;
  }
}

// Empties a row, 16 bytes a store between its first and last 16-byte boundary.
__device__ inline void clear_row(uint32_t* row, int n, int at, int step) {
  const int head = (int)((16 - (uintptr_t)row % 16) % 16 / 4);
  const int body = n > head ? (n - head) / 4 : 0;
  if (at < head && at < n) row[at] = 0;
  for (int i = at; i < body; i += step) *(u32x4*)(row + head + 4 * i) = u32x4{0, 0, 0, 0};
  for (int i = head + 4 * body + at; i < n; i += step) row[i] = 0;
}
__global__ __launch_bounds__(kThreads) void k_clear(CountArgs a) {
  for (int b = blockIdx.y; b < a.B; b += gridDim.y) {
    const int slot = slot_of(a, b);
    if (slot < 0) continue;
    const int at = blockIdx.x * kThreads + threadIdx.x, step = gridDim.x * kThreads;
    clear_row((uint32_t*)a.counts + (size_t)slot * a.V, a.V, at, step);
    clear_row(a.seen + (size_t)slot * 2 * a.W, 2 * a.W, at, step);
  }
}

// A few tokens a session (a round's): one atomic or two a token.
__global__ __launch_bounds__(kThreads) void k_count_few(CountArgs a) {
  for (int b = blockIdx.y; b < a.B; b += gridDim.y) {
    const int slot = slot_of(a, b);
    if (slot < 0) continue;
    int64_t lo, hi;
    span_of(a, b, lo, hi);
    int32_t* counts = a.counts + (size_t)slot * a.V;
    uint32_t* seen = a.seen + ((size_t)slot * 2 + a.plane) * a.W;
    for (int64_t i = lo + blockIdx.x * kThreads + threadIdx.x; i < hi;
         i += (int64_t)gridDim.x * kThreads) {
      const int t = a.tokens[i];
      if (t < 0 || t >= a.V) continue;
      if (a.plane) atomicAdd(counts + t, 1);
      atomicOr(seen + t / 32, 1u << (t % 32));
    }
  }
}

// Many tokens a session (prompts, resumed outputs): a workgroup gathers kPart
// tokens in LDS, over a range of ids, and then updates what came up once.  The
// frequent tokens of a text (a few percent of it each) would queue at their
// words' atomics otherwise.
constexpr int kManyThreads = 1024;
constexpr int kPart = 8192;
template <int kPlane>
__global__ __launch_bounds__(kManyThreads) void k_count_many(CountArgs a) {
  constexpr int kRange = kPlane ? 1 << 14 : 1 << 18;     // ids of a workgroup
  constexpr int kWords = kPlane ? kRange : kRange / 32;  // counts, or bits
  __shared__ uint32_t lds[kWords];
  const int b = a.b0 + blockIdx.z, v0 = blockIdx.y * kRange;
  const int slot = slot_of(a, b);
  if (slot < 0) return;
  int64_t lo, hi;
  span_of(a, b, lo, hi);
  lo += (int64_t)blockIdx.x * kPart;
  if (lo >= hi) return;
  const int ids = a.V - v0 < kRange ? a.V - v0 : kRange;
  const int words = kPlane ? ids : (ids + 31) / 32;
  for (int w = threadIdx.x; w < words; w += kManyThreads) lds[w] = 0;
  __syncthreads();
  for (; lo < hi; lo += (int64_t)gridDim.x * kPart) {
    const int n = hi - lo < kPart ? (int)(hi - lo) : kPart;
    int32_t t[kPart / kManyThreads];
#pragma unroll
    for (int k = 0; k < kPart / kManyThreads; ++k)
      t[k] = a.tokens[lo + min(k * kManyThreads + (int)threadIdx.x, n - 1)];
#pragma unroll
    for (int k = 0; k < kPart / kManyThreads; ++k) {
      if (k * kManyThreads + (int)threadIdx.x >= n || t[k] < v0 || t[k] - v0 >= ids) continue;
      if (kPlane) atomicAdd(lds + (t[k] - v0), 1u);
      else atomicOr(lds + (t[k] - v0) / 32, 1u << (t[k] % 32));
    }
  }
  __syncthreads();
  uint32_t* seen = a.seen + ((size_t)slot * 2 + kPlane) * a.W + v0 / 32;
  for (int w0 = 0; w0 < words; w0 += kManyThreads) {
    const int w = w0 + threadIdx.x;
    const uint32_t x = w < words ? lds[w] : 0;
    if (kPlane) {
      if (x != 0) atomicAdd(a.counts + (size_t)slot * a.V + v0 + w, (int)x);
      const uint64_t came = __ballot(x != 0);
      const uint32_t half = threadIdx.x & 32 ? (uint32_t)(came >> 32) : (uint32_t)came;
      if (threadIdx.x % 32 == 0 && half != 0) atomicOr(seen + w / 32, half);
    } else if (x != 0) {
      atomicOr(seen + w, x);
    }
  }
}

template <int kPlane>
void launch_many(CountArgs a, int64_t mean, hipStream_t st) {
  constexpr int kRange = kPlane ? 1 << 14 : 1 << 18;
  // workgroups for a session of the mean length, twice as many where lengths
  // are not known here; longer ones take more turns
  const int64_t parts = (mean * (a.offsets ? 2 : 1) + kPart - 1) / kPart;
  for (a.b0 = 0; a.b0 < a.B; a.b0 += kGridZ) {
    const dim3 grid((unsigned)(parts < 16 ? parts : 16), (a.V + kRange - 1) / kRange,
                    a.B - a.b0 < kGridZ ? a.B - a.b0 : kGridZ);
    hipLaunchKernelGGL(k_count_many<kPlane>, grid, dim3(kManyThreads), 0, st, a);
  }
}

}  // namespace
}  // namespace sv

extern "C" int sv_count_tokens(const sv_history* history, const int32_t* slots,
                               const int32_t* tokens, const int32_t* offsets, const int32_t* lens,
                               int32_t B, int32_t L, int32_t V, int32_t plane, int32_t clear,
                               void* stream) {
  using namespace sv;
  if (!history || !history->counts || !history->seen || history->n_slots < 1) return SV_ERR_ARG;
  if (B < 1 || B > SV_B_MAX || L < 0 || V < 1 || V > SV_V_MAX) return SV_ERR_ARG;
  if (plane != 0 && plane != 1) return SV_ERR_ARG;
  if ((L > 0 && !tokens) || (offsets && lens) || (!slots && history->n_slots < B))
    return SV_ERR_ARG;
  CountArgs a = {history->counts, history->seen, slots, tokens, offsets, lens,
                 history->n_slots, B, L, V, (V + 31) / 32, plane, 0};
  hipStream_t st = (hipStream_t)stream;
  (void)hipGetLastError();
  const unsigned gy = B < 32768 ? B : 32768;
  if (clear) {
    // about 16 KB a workgroup
    const unsigned gx = (unsigned)((V + 4095) / 4096);
    hipLaunchKernelGGL(k_clear, dim3(gx, gy), dim3(kThreads), 0, st, a);
  }
  // tokens of a session: L, or on average in a line
  const int64_t mean = offsets ? ((int64_t)L + B - 1) / B : L;
  if (mean > (plane ? kFewOutput : kFewPrompt)) {
    if (plane) launch_many<1>(a, mean, st);
    else launch_many<0>(a, mean, st);
  } else if (L > 0) {
    const unsigned gx = (unsigned)((mean + kThreads - 1) / kThreads);
    hipLaunchKernelGGL(k_count_few, dim3(gx, gy), dim3(kThreads), 0, st, a);
  }
  return hipGetLastError() == hipSuccess ? SV_OK : SV_ERR_DEVICE;
}
