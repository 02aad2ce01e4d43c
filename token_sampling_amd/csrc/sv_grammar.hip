// sv_grammar.hip -- byte automata over the vocabulary: the masks of states
// (sv_grammar_masks) and the states along tokens (sv_grammar_advance).
//
// A state s takes a byte c to next[s][classes[c]]; a token is the walk over its
// bytes.  -1 stands for "no grammar" (and for a refused byte within a walk).
#include "sv_common.hpp"

namespace sv {
namespace {

constexpr int kThreads = 256;

struct GrammarArgs {
  sv_grammar g;
  sv_vocab v;
};

__device__ inline int step(const sv_grammar& g, int s, uint8_t byte) {
  const int c = g.classes[byte];
  if (c >= g.n_classes) return -1;
  const int to = g.next[(int64_t)s * g.n_classes + c];
  return to >= 0 && to < g.n_states ? to : -1;
}

// The bytes [lo, hi) of token t, kept within the array.
__device__ inline void bytes_of(const sv_vocab& v, int t, int& lo, int& hi) {
  lo = v.offsets[t];
  hi = v.offsets[t + 1];
  lo = lo < 0 ? 0 : lo;
  hi = hi > v.n_bytes ? v.n_bytes : hi;
}

__device__ inline bool is_end(const sv_vocab& v, int t) {
  bool e = false;
  for (int i = 0; i < v.n_end; ++i) e |= v.end[i] == t;
  return e;
}

__global__ __launch_bounds__(kThreads) void k_masks(GrammarArgs a, const int32_t* states, int n,
                                                    uint32_t* bits) {
  const int W = (a.v.V + 31) / 32;
  const int v = blockIdx.x * kThreads + threadIdx.x;
  for (int k = blockIdx.y; k < n; k += gridDim.y) {
    const int s0 = states[k];
    bool ok = false;
    if (v < a.v.V) {
      if (s0 < 0 || s0 >= a.g.n_states) {
        ok = true;
      } else if (is_end(a.v, v)) {
        ok = a.g.accept[s0] != 0;
      } else {
        int lo, hi, s = s0;
        bytes_of(a.v, v, lo, hi);
        ok = lo < hi;
        for (; lo < hi && s >= 0; ++lo) s = step(a.g, s, a.v.bytes[lo]);
        ok = ok && s >= 0;
      }
    }
    const uint64_t m = __ballot(ok);
    const int lane = threadIdx.x % kWave, w = v / 32;
    if (lane % 32 == 0 && w < W)
      bits[(size_t)k * W + w] = lane ? (uint32_t)(m >> 32) : (uint32_t)m;
  }
}

__global__ __launch_bounds__(kWave) void k_advance(GrammarArgs a, const int32_t* states,
                                                   const int32_t* tokens, const int32_t* lens,
                                                   int B, int L, int32_t* out, int32_t* last) {
  const int b = blockIdx.x * kWave + threadIdx.x;
  if (b >= B) return;
  int s = states[b];
  if (s >= a.g.n_states || s < 0) s = -1;
  int n = lens ? lens[b] : L;
  n = n < 0 ? 0 : n > L ? L : n;
  out += (size_t)b * (L + 1);
  out[0] = s;
  for (int i = 0; i < n; ++i) {
    const int t = tokens[(size_t)b * L + i];
    if (s >= 0) {
      int lo = 0, hi = 0;
      if (t >= 0 && t < a.v.V && !is_end(a.v, t)) bytes_of(a.v, t, lo, hi);
      if (lo >= hi) s = -1;
      for (; lo < hi && s >= 0; ++lo) s = step(a.g, s, a.v.bytes[lo]);
    }
    out[i + 1] = s;
  }
  for (int i = n; i < L; ++i) out[i + 1] = -1;
  if (last) last[b] = s;
}

bool grammar_ok(const sv_grammar* g, const sv_vocab* v) {
  if (!g || !g->next || !g->classes || !g->accept || g->n_states < 1 || g->n_classes < 1 ||
      g->n_classes > 256)
    return false;
  if (!v || !v->offsets || v->n_bytes < 0 || (v->n_bytes > 0 && !v->bytes) || v->n_end < 0 ||
      v->n_end > SV_STOP_MAX || (v->n_end > 0 && !v->end) || v->V < 1 || v->V > SV_V_MAX)
    return false;
  return true;
}

}  // namespace
}  // namespace sv

extern "C" int sv_grammar_masks(const sv_grammar* grammar, const sv_vocab* vocab,
                                const int32_t* states, int32_t n, uint32_t* bits, void* stream) {
  using namespace sv;
  if (!grammar_ok(grammar, vocab) || !states || !bits || n < 1) return SV_ERR_ARG;
  GrammarArgs a = {*grammar, *vocab};
  const unsigned gx = (vocab->V + kThreads - 1) / kThreads;
  (void)hipGetLastError();
  hipLaunchKernelGGL(k_masks, dim3(gx, n < 4096 ? n : 4096), dim3(kThreads), 0,
                     (hipStream_t)stream, a, states, n, bits);
  return hipGetLastError() == hipSuccess ? SV_OK : SV_ERR_DEVICE;
}

extern "C" int sv_grammar_advance(const sv_grammar* grammar, const sv_vocab* vocab,
                                  const int32_t* states, const int32_t* tokens,
                                  const int32_t* lens, int32_t B, int32_t L, int32_t* out_states,
                                  int32_t* last, void* stream) {
  using namespace sv;
  if (!grammar_ok(grammar, vocab) || !states || !out_states || B < 1 || B > SV_B_MAX || L < 0 ||
      L > SV_M_MAX + 1 || (L > 0 && !tokens))
    return SV_ERR_ARG;
  GrammarArgs a = {*grammar, *vocab};
  (void)hipGetLastError();
  hipLaunchKernelGGL(k_advance, dim3((B + kWave - 1) / kWave), dim3(kWave), 0,
                     (hipStream_t)stream, a, states, tokens, lens, B, L, out_states, last);
  return hipGetLastError() == hipSuccess ? SV_OK : SV_ERR_DEVICE;
}
