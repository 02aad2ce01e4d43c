// sv_history.hip -- sv_count_tokens: notes prompt tokens and committed tokens
// in the history that sv_adjust_logits' penalties read.
#include "sv_common.hpp"

namespace sv {
namespace {

constexpr int kThreads = 256;

struct CountArgs {
  int32_t* counts;
  uint32_t* seen;
  const int32_t* slots;
  const int32_t* tokens;
  const int32_t* offsets;
  const int32_t* lens;
  int32_t n_slots, B, L, V, W, plane;
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

__global__ __launch_bounds__(kThreads) void k_clear(CountArgs a) {
  for (int b = blockIdx.y; b < a.B; b += gridDim.y) {
    const int slot = slot_of(a, b);
    if (slot < 0) continue;
    int32_t* counts = a.counts + (size_t)slot * a.V;
    uint32_t* seen = a.seen + (size_t)slot * 2 * a.W;
    const int step = gridDim.x * kThreads;
    for (int v = blockIdx.x * kThreads + threadIdx.x; v < a.V; v += step) counts[v] = 0;
    for (int w = blockIdx.x * kThreads + threadIdx.x; w < 2 * a.W; w += step) seen[w] = 0;
  }
}

__global__ __launch_bounds__(kThreads) void k_count(CountArgs a) {
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
                 history->n_slots, B, L, V, (V + 31) / 32, plane};
  hipStream_t st = (hipStream_t)stream;
  (void)hipGetLastError();
  const unsigned gy = B < 32768 ? B : 32768;
  if (clear) hipLaunchKernelGGL(k_clear, dim3(16, gy), dim3(kThreads), 0, st, a);
  if (L > 0) {
    const unsigned gx = L <= kThreads ? 1 : 8;
    hipLaunchKernelGGL(k_count, dim3(gx, gy), dim3(kThreads), 0, st, a);
  }
  return hipGetLastError() == hipSuccess ? SV_OK : SV_ERR_DEVICE;
}
