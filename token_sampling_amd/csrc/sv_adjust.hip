// sv_adjust.hip -- sv_adjust_logits: penalties for repeated tokens, biases and
// vocabulary masks on a round's logits, in one pass.
//
// For token v of row r of a session with count c (stored output count plus how
// often v is among the drafted tokens before the row):
//   z = v seen ? (z > 0 ? z / rep : z * rep) : z
//   z = z - freq * c - (c > 0 ? pres : 0) + bias(v)
//   z = mask bit clear ? -inf : z
// in binary32, rounded once to the logits' type.
#include <math.h>

#include "sv_common.hpp"

namespace sv {
namespace {

constexpr int kThreads = 256;
constexpr int kTile = 2048;  // tokens of one unit of work

struct AdjustArgs {
  const void* logits;
  int64_t in_session, in_row;
  void* out;
  int64_t out_session, out_row;
  const int32_t* tokens;
  const int32_t* m;
  const sv_penalties* pen;
  const int32_t* counts;
  const uint32_t* seen;
  const int32_t* slots;
  int32_t n_slots;
  const int32_t* bias_off;
  const int32_t* bias_id;
  const float* bias_val;
  int32_t n_bias;
  const uint32_t* mask_bits;
  const int32_t* mask_rows;
  int32_t n_masks;
  int32_t B, M, R, V, W, n_tiles;
  int32_t* status;
};

__device__ inline float load_f32(const float* p) { return *p; }
__device__ inline float load_f32(const __bf16* p) { return (float)*p; }

// A session's status and its used rows; every lane of the wave takes part.
__device__ inline int32_t session_check(const AdjustArgs& a, int b, int& m, int& slot) {
  const int lane = __lane_id();
  m = a.m ? a.m[b] : a.M;
  if (m < 0 || m > a.M) return SV_S_LIMIT;
  bool bad = false;
  slot = -1;
  if (a.pen) {
    const sv_penalties p = a.pen[b];
    bad |= !(p.repetition > 0.f) || !isfinite(p.repetition) || !isfinite(p.frequency) ||
           !isfinite(p.presence) || p.reserved != 0;
    if (a.counts) {
      slot = a.slots ? a.slots[b] : b;
      bad |= slot < -1 || slot >= a.n_slots;
    }
  }
  if (a.bias_off) {
    const int lo = a.bias_off[b], hi = a.bias_off[b + 1];
    bad |= lo < 0 || hi < lo || hi > a.n_bias;
  }
  if (a.mask_rows) {
    const int rows = m + (a.R - a.M);
    for (int r = lane; r < rows; r += kWave) {
      const int k = a.mask_rows[(size_t)b * a.R + r];
      bad |= k < -1 || k >= a.n_masks;
    }
  }
  if (__any(bad)) return SV_S_BAD_CONTROL;
  if (a.pen && lane < m) {
    const int t = a.tokens[(size_t)b * a.M + lane];
    bad = t < 0 || t >= a.V;
  }
  return __any(bad) ? SV_S_BAD_PROPOSAL : 0;
}

template <typename T>
__global__ __launch_bounds__(kThreads) void k_adjust(AdjustArgs a) {
  const int64_t units = (int64_t)a.B * a.n_tiles;
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int b = (int)(u / a.n_tiles), tile = (int)(u % a.n_tiles);
    const T* in = (const T*)a.logits + b * a.in_session;
    T* out = (T*)a.out + b * a.out_session;
    const bool in_place = (const void*)a.out == a.logits;
    int m, slot;
    const int32_t status = session_check(a, b, m, slot);
    if (tile == 0 && threadIdx.x == 0 && a.status) a.status[b] = status;
    const int rows = status == 0 ? m + (a.R - a.M) : a.R;
    const int v0 = tile * kTile, v1 = v0 + kTile < a.V ? v0 + kTile : a.V;
    sv_penalties p = {1.f, 0.f, 0.f, 0};
    if (a.pen && status == 0) p = a.pen[b];
    for (int r = 0; r < rows; ++r) {
      const int mask = status == 0 && a.mask_rows ? a.mask_rows[(size_t)b * a.R + r] : -1;
      for (int v = v0 + threadIdx.x; v < v1; v += kThreads) {
        if (status != 0) {
          out[r * a.out_row + v] = (T)__builtin_nanf("");
          continue;
        }
        const T raw = in[r * a.in_row + v];
        float z = load_f32(&raw);
        bool changed = false;
        if (a.pen) {
          int c = 0;
          bool seen = false;
          if (slot >= 0) {
            const uint32_t* s = a.seen + (size_t)slot * 2 * a.W + v / 32;
            seen = (s[0] >> (v % 32)) & 1;
            if ((s[a.W] >> (v % 32)) & 1) c = a.counts[(size_t)slot * a.V + v];
          }
          for (int j = 0; j < r; ++j) c += a.tokens[(size_t)b * a.M + j] == v;
          if (seen || c > 0) {
            changed = true;
            z = z > 0.f ? z / p.repetition : z * p.repetition;
            z = z - p.frequency * (float)c;
            if (c > 0) z -= p.presence;
          }
        }
        if (a.bias_off) {
          int lo = a.bias_off[b], hi = a.bias_off[b + 1];
          const int end = hi;
          while (lo < hi) {
            const int mid = lo + (hi - lo) / 2;
            if (a.bias_id[mid] < v) lo = mid + 1; else hi = mid;
          }
          if (lo < end && a.bias_id[lo] == v) {
            changed = true;
            z += a.bias_val[lo];
          }
        }
        if (mask >= 0 && !((a.mask_bits[(size_t)mask * a.W + v / 32] >> (v % 32)) & 1)) {
          changed = true;
          z = -__builtin_inff();
        }
        if (changed) out[r * a.out_row + v] = (T)z;
        else if (!in_place) out[r * a.out_row + v] = raw;
      }
    }
  }
}

}  // namespace
}  // namespace sv

extern "C" int sv_adjust_logits(const void* logits, int64_t session_stride, int64_t row_stride,
                                int32_t dtype, const int32_t* draft_tokens, const int32_t* m,
                                const sv_penalties* penalties, const sv_history* history,
                                const int32_t* slots, const sv_bias* bias, const sv_masks* masks,
                                int32_t B, int32_t M, int32_t R, int32_t V, void* out,
                                int32_t* status, void* stream) {
  using namespace sv;
  if (!logits || !out || (dtype != SV_BF16 && dtype != SV_FP32)) return SV_ERR_ARG;
  if (B < 1 || B > SV_B_MAX || M < 0 || M > SV_M_MAX || R < 1 || (R != M && R != M + 1) || V < 1 ||
      V > SV_V_MAX)
    return SV_ERR_ARG;
  // element offsets stay within a signed 64-bit index
  if (session_stride < 0 || row_stride < 0 || session_stride > (int64_t)1 << 40 ||
      row_stride > (int64_t)1 << 40)
    return SV_ERR_ARG;
  if (M > 0 && penalties && !draft_tokens) return SV_ERR_ARG;
  if (history && (!history->counts || !history->seen || history->n_slots < 1 ||
                  (!slots && history->n_slots < B)))
    return SV_ERR_ARG;
  if (bias && (!bias->offsets || bias->n < 0 || (bias->n > 0 && (!bias->ids || !bias->values))))
    return SV_ERR_ARG;
  if (masks && (!masks->bits || !masks->rows || masks->n_masks < 1)) return SV_ERR_ARG;
  AdjustArgs a = {};
  a.logits = logits;
  a.in_session = session_stride;
  a.in_row = row_stride;
  a.out = out;
  const bool in_place = out == logits;
  a.out_session = in_place ? session_stride : (int64_t)R * V;
  a.out_row = in_place ? row_stride : V;
  a.tokens = draft_tokens;
  a.m = m;
  a.pen = penalties;
  if (history && penalties) {
    a.counts = history->counts;
    a.seen = history->seen;
    a.n_slots = history->n_slots;
    a.slots = slots;
  }
  if (bias) {
    a.bias_off = bias->offsets;
    a.bias_id = bias->ids;
    a.bias_val = bias->values;
    a.n_bias = bias->n;
  }
  if (masks) {
    a.mask_bits = masks->bits;
    a.mask_rows = masks->rows;
    a.n_masks = masks->n_masks;
  }
  a.B = B;
  a.M = M;
  a.R = R;
  a.V = V;
  a.W = (V + 31) / 32;
  a.n_tiles = (V + kTile - 1) / kTile;
  a.status = status;
  const int64_t units = (int64_t)B * a.n_tiles;
  const unsigned grid = (unsigned)(units < 65536 * 16 ? units : 65536 * 16);
  hipStream_t st = (hipStream_t)stream;
  (void)hipGetLastError();
  if (dtype == SV_BF16)
    hipLaunchKernelGGL(k_adjust<__bf16>, dim3(grid), dim3(kThreads), 0, st, a);
  else
    hipLaunchKernelGGL(k_adjust<float>, dim3(grid), dim3(kThreads), 0, st, a);
  return hipGetLastError() == hipSuccess ? SV_OK : SV_ERR_DEVICE;
}
