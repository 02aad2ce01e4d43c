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

constexpr int kWaves = 4;  // per workgroup; each works by itself
constexpr int64_t kWantedWaves = 8192;   // two for each place of a wave in the card's SIMDs
constexpr int64_t kMaxGroups = 1 << 22;  // keeps the launch's work-items within 32 bits
#ifndef SV_ADJUST_GROUPS
#define SV_ADJUST_GROUPS 2
#endif

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
  int32_t B, M, R, V, W, n_tiles, n_chunks, chunk;
  int32_t* status;
};

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
struct __attribute__((packed, aligned(2))) Vec16b {
  u32x4 v;
};

// A lane's share of a row: one 16-byte vector per group, 8 bf16 or 4 binary32
// logits, 64 lanes side by side.
template <typename T>
struct Lanes {
  static constexpr int kE = 16 / (int)sizeof(T);  // logits of a vector
  static constexpr int kGroup = kWave * kE;       // logits of a group
};

__device__ inline void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// What a wave knows of its session; every lane of the wave takes part.
struct Session {
  int32_t status;
  int m, slot;
  int32_t token;      // lane i: x_{i+1}, -1 past m
  int32_t mask_row;   // lane r: the mask of row r
  int32_t mask_row64; // row 64's
  int bias_lo, bias_hi;
  sv_penalties pen;
};

__device__ inline Session session_of(const AdjustArgs& a, int b) {
  const int lane = __lane_id();
  Session s;
  s.status = 0;
  s.slot = -1;
  s.token = -1;
  s.mask_row = s.mask_row64 = -1;
  s.bias_lo = s.bias_hi = 0;
  s.pen = {1.f, 0.f, 0.f, 0};
  s.m = a.m ? a.m[b] : a.M;
  if (s.m < 0 || s.m > a.M) {
    s.status = SV_S_LIMIT;
    return s;
  }
  const int rows = s.m + (a.R - a.M);
  bool bad = false, bad_token = false;
  if (a.pen) {
    if (lane < s.m) {
      s.token = a.tokens[(size_t)b * a.M + lane];
      bad_token = s.token < 0 || s.token >= a.V;
    }
    const sv_penalties p = a.pen[b];
    // within these bounds the reciprocal is a normal number
    bad |= !(p.repetition >= 0x1p-64f && p.repetition <= 0x1p64f) || !isfinite(p.frequency) ||
           !isfinite(p.presence) || p.reserved != 0;
    if (a.counts) {
      s.slot = a.slots ? a.slots[b] : b;
      bad |= s.slot < -1 || s.slot >= a.n_slots;
    }
    s.pen = p;
  }
  if (a.bias_off) {
    s.bias_lo = a.bias_off[b];
    s.bias_hi = a.bias_off[b + 1];
    bad |= s.bias_lo < 0 || s.bias_hi < s.bias_lo || s.bias_hi > a.n_bias;
  }
  if (a.mask_rows) {
    const int32_t* k = a.mask_rows + (size_t)b * a.R;
    if (lane < rows) s.mask_row = k[lane];
    if (rows > kWave) s.mask_row64 = k[kWave];
    bad |= s.mask_row < -1 || s.mask_row >= a.n_masks || s.mask_row64 < -1 ||
           s.mask_row64 >= a.n_masks;
  }
  s.status = __any(bad) ? SV_S_BAD_CONTROL : __any(bad_token) ? SV_S_BAD_PROPOSAL : 0;
  return s;
}

// The first entry of ids[lo, hi) that is not below v, found by the wave: 64
// probes a step.
__device__ inline int lower_bound(const int32_t* ids, int lo, int hi, int v) {
  const int lane = __lane_id();
  while (lo < hi) {
    const int step = (hi - lo + kWave - 1) / kWave;
    const int64_t at = (int64_t)lo + (int64_t)lane * step;
    // probes are ascending: those below v come first
    const int below = __popcll(__ballot(at < hi && ids[at] < v));
    if (step == 1) return lo + below;
    if (below == 0) return lo;
    const int64_t end = (int64_t)lo + (int64_t)below * step;
    lo = lo + (below - 1) * step + 1;
    hi = end < hi ? (int)end : hi;
  }
  return lo;
}

__device__ inline float widen(const u32x4& x, int i, __bf16) {
  const uint32_t w = x[i / 2];
  return __builtin_bit_cast(float, i % 2 ? w & 0xFFFF0000u : w << 16);
}
__device__ inline float widen(const u32x4& x, int i, float) {
  const uint32_t w = x[i];
  return __builtin_bit_cast(float, w);
}

// All ones where bit i of bits is set, else zeros.
__device__ inline uint32_t spread(uint32_t bits, int i) {
  return (uint32_t)__builtin_amdgcn_sbfe((int)bits, i, 1);
}

// Word d of a vector's selection: the elements whose bits are set.
__device__ inline uint32_t select_word(uint32_t bits, int d, __bf16) {
  return (spread(bits, 2 * d) & 0xFFFFu) | (spread(bits, 2 * d + 1) & 0xFFFF0000u);
}
__device__ inline uint32_t select_word(uint32_t bits, int d, float) { return spread(bits, d); }

__device__ inline uint32_t round_word(const float* z, int d, __bf16) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  const bf16x2 h = {(__bf16)z[2 * d], (__bf16)z[2 * d + 1]};
  return __builtin_bit_cast(uint32_t, h);
}
__device__ inline uint32_t round_word(const float* z, int d, float) {
  return __builtin_bit_cast(uint32_t, z[d]);
}

template <typename T>
constexpr uint32_t kMinusInf = sizeof(T) == 2 ? 0xFF80FF80u : 0xFF800000u;

// One wave works on one unit: kTile neighbouring tokens of one session, row
// after row.  What the rows share is set up once: an additive term for each
// token that the history, a bias or a drafted token touches (in LDS, the
// wave's own), and three bits a token in registers: rep (seen, the repetition
// penalty applies), had (output, so no presence any more) and hot (the token
// changes).  Row r then adds what x_r changes, which only the tiles holding
// x_r do, and streams: a vector without hot tokens and with a full mask is a
// copy (in place: not touched), one with an empty mask is not read.
template <typename T, int G, bool kInPlace>
__global__ __launch_bounds__(kWaves* kWave) void k_adjust(AdjustArgs a) {
  using L = Lanes<T>;
  constexpr int E = L::kE, kTile = G * L::kGroup;
  constexpr uint32_t kAll = (1u << E) - 1;
  static_assert(G * E <= 32, "a lane's tokens fit one word");
  __shared__ __attribute__((aligned(16))) float lds_term[kWaves][kTile];
  __shared__ uint32_t lds_bits[kWaves][kTile / 32];
  const int lane = __lane_id();
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  float* term = lds_term[wave];
  uint32_t* bits = lds_bits[wave];
  const int64_t units = (int64_t)a.B * a.n_tiles * a.n_chunks;
  const T nil = T(0);

  for (int64_t u0 = (int64_t)blockIdx.x * kWaves; u0 < units; u0 += (int64_t)gridDim.x * kWaves) {
    const int64_t u = u0 + wave;
    if (u >= units) break;
    const int tile = (int)(u % a.n_tiles);
    const int64_t bc = u / a.n_tiles;
    const int b = (int)(bc / a.n_chunks), chunk = (int)(bc % a.n_chunks);
    const int v0 = tile * kTile;
    const Session s = session_of(a, b);
    if (a.status && tile == 0 && chunk == 0 && lane == 0) a.status[b] = s.status;
    const int rows = s.status == 0 ? s.m + (a.R - a.M) : a.R;
    const int r0 = chunk * a.chunk, r1 = r0 + a.chunk < rows ? r0 + a.chunk : rows;
    if (r0 >= r1) continue;
    const T* in = (const T*)a.logits + b * a.in_session + v0;
    T* out = (T*)a.out + b * a.out_session + v0;

    // a lane's vectors: tokens v0 + first + g * kGroup ...
    const int first = lane * E;
    const int left = a.V - v0;  // tokens from the tile's start to the row's end
    if (s.status != 0) {
      for (int r = r0; r < r1; ++r)
        for (int i = lane; i < kTile && i < left; i += kWave)
          out[r * a.out_row + i] = (T)__builtin_nanf("");
      continue;
    }

    // ---- what the rows share
    uint32_t rep = 0, had = 0, hot = 0;
    // drafted tokens of this tile that rows before r1 meet
    const uint64_t mine =
        __ballot(s.token >= v0 && s.token - v0 < kTile && lane < r1 - 1);
    const uint32_t* seen = a.seen;
    if (s.slot >= 0) {
      seen += (size_t)s.slot * 2 * a.W;
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const int v = v0 + g * L::kGroup + first;
        if (v < a.V) {
          const uint32_t p = ((const uint8_t*)seen)[v / 8] >> (v % 8);
          const uint32_t o = ((const uint8_t*)(seen + a.W))[v / 8] >> (v % 8);
          rep |= ((p | o) & kAll) << (g * E);
          had |= (o & kAll) << (g * E);
        }
      }
    }
    int bias_lo = 0, bias_hi = 0;
    if (s.bias_lo < s.bias_hi) {
      bias_lo = lower_bound(a.bias_id, s.bias_lo, s.bias_hi, v0);
      bias_hi = lower_bound(a.bias_id, bias_lo, s.bias_hi, v0 + kTile);
    }
    hot = rep;
    uint32_t groups = hot;  // tokens whose vectors need terms
    if (mine != 0 || bias_lo < bias_hi) {
      if (lane < kTile / 32) bits[lane] = 0;
      wave_sync();
      for (int e = bias_lo + lane; e < bias_hi; e += kWave) {
        const int i = a.bias_id[e] - v0;
        if (i >= 0 && i < kTile) atomicOr(bits + i / 32, 1u << (i % 32));
      }
      wave_sync();
      uint32_t biased = 0;
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const int i = g * L::kGroup + first;
        biased |= ((bits[i / 32] >> (i % 32)) & kAll) << (g * E);
      }
      hot |= biased;
      wave_sync();
      if ((mine >> lane) & 1) atomicOr(bits + (s.token - v0) / 32, 1u << ((s.token - v0) % 32));
      wave_sync();
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const int i = g * L::kGroup + first;
        groups |= ((bits[i / 32] >> (i % 32)) & kAll) << (g * E);
      }
      groups |= hot;
    }
    if (__any(groups != 0)) {
#pragma unroll
      for (int g = 0; g < G; ++g) {
        if (((groups >> (g * E)) & kAll) == 0) continue;
        const int i = g * L::kGroup + first, v = v0 + i;
        const uint32_t o = (had >> (g * E)) & kAll;
        float t[E];
#pragma unroll
        for (int k = 0; k < E; ++k) t[k] = 0.f;
        if (o != 0) {
          int32_t c[E];
          const int32_t* row = a.counts + (size_t)s.slot * a.V + v;
          if (v + E <= a.V) {
            __builtin_memcpy(c, row, sizeof(c));
          } else {
#pragma unroll
            for (int k = 0; k < E; ++k) c[k] = v + k < a.V ? row[k] : 0;
          }
#pragma unroll
          for (int k = 0; k < E; ++k)
            if ((o >> k) & 1 && c[k] > 0) t[k] = -(s.pen.frequency * (float)c[k] + s.pen.presence);
        }
#pragma unroll
        for (int k = 0; k < E; k += 4) *(f32x4*)(term + i + k) = f32x4{t[k], t[k + 1], t[k + 2], t[k + 3]};
      }
      wave_sync();
      for (int e = bias_lo + lane; e < bias_hi; e += kWave) {
        const int i = a.bias_id[e] - v0;
        if (i >= 0 && i < kTile) term[i] += a.bias_val[e];
      }
      wave_sync();
    }

    // ---- the rows
    const float up = s.pen.repetition, down = 1.f / s.pen.repetition;
    auto meet = [&](int j) {  // drafted token j counts from here on
      const int i = lane_read(s.token, j) - v0;
      const int g = i / L::kGroup;
      if (lane == (i % L::kGroup) / E) {
        const uint32_t bit = 1u << (g * E + i % E);
        term[i] -= had & bit ? s.pen.frequency : s.pen.frequency + s.pen.presence;
        had |= bit;
        rep |= bit;
        hot |= bit;
      }
      wave_sync();
    };
    for (int j = 0; j < r0; ++j)
      if ((mine >> j) & 1) meet(j);

    auto mask_of = [&](int r, uint32_t (&mk)[G]) {
#pragma unroll
      for (int g = 0; g < G; ++g) mk[g] = kAll;
      if (a.mask_rows == nullptr || r >= r1) return;
      const int k = r < kWave ? lane_read(s.mask_row, r) : s.mask_row64;
      if (k < 0) return;
      const uint8_t* row = (const uint8_t*)(a.mask_bits + (size_t)k * a.W);
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const int v = v0 + g * L::kGroup + first;
        if (v < a.V) mk[g] = ((uint32_t)row[v / 8] >> (v % 8)) & kAll;
      }
    };
    uint32_t mk[G];
    mask_of(r0, mk);
    for (int r = r0; r < r1; ++r) {
      if (r > r0 && ((mine >> (r - 1)) & 1)) meet(r - 1);
      u32x4 x[G];
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const int i = g * L::kGroup + first;
        const uint32_t h = (hot >> (g * E)) & kAll;
        x[g] = u32x4{0, 0, 0, 0};
        if (mk[g] != 0 && i < left && (!kInPlace || h != 0 || mk[g] != kAll)) {
          const T* p = in + r * a.in_row + i;
          if (i + E <= left) {
            x[g] = ((const Vec16b*)p)->v;
          } else {
            T t[E];
#pragma unroll
            for (int k = 0; k < E; ++k) t[k] = i + k < left ? p[k] : nil;
            __builtin_memcpy(&x[g], t, 16);
          }
        }
      }
      uint32_t next[G];
      mask_of(r + 1, next);
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const int i = g * L::kGroup + first;
        const uint32_t h = (hot >> (g * E)) & kAll;
        if (i < left && (!kInPlace || h != 0 || mk[g] != kAll)) {
          if (h != 0) {
            float z[E];
#pragma unroll
            for (int k = 0; k < E; k += 4) {
              const f32x4 t = *(const f32x4*)(term + i + k);
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                const float y = widen(x[g], k + q, nil);
                const float f = y > 0.f ? down : up;
                z[k + q] = ((rep >> (g * E + k + q)) & 1 ? y * f : y) + t[q];
              }
            }
#pragma unroll
            for (int d = 0; d < 4; ++d) {
              const uint32_t sel = select_word(h, d, nil);
              const uint32_t w = x[g][d];
              x[g][d] = (round_word(z, d, nil) & sel) | (w & ~sel);
            }
          }
          if (mk[g] != kAll) {
#pragma unroll
            for (int d = 0; d < 4; ++d) {
              const uint32_t sel = select_word(mk[g], d, nil);
              const uint32_t w = x[g][d];
              x[g][d] = (w & sel) | (kMinusInf<T> & ~sel);
            }
          }
          T* p = out + r * a.out_row + i;
          if (i + E <= left) {
            ((Vec16b*)p)->v = x[g];
          } else {
            T t[E];
            __builtin_memcpy(t, &x[g], 16);
#pragma unroll
            for (int k = 0; k < E; ++k)
              if (i + k < left) p[k] = t[k];
          }
        }
        mk[g] = next[g];
      }
    }
  }
}

template <typename T, bool kInPlace>
void launch(AdjustArgs a, hipStream_t st) {
  constexpr int G = SV_ADJUST_GROUPS * (int)sizeof(T) / 2, kTile = G * Lanes<T>::kGroup;
  a.n_tiles = (a.V + kTile - 1) / kTile;
  // rows go to several waves where a wave per tile would leave the card idle
  const int64_t tiles = (int64_t)a.B * a.n_tiles;
  int64_t chunks = (kWantedWaves + tiles - 1) / tiles;
  chunks = chunks < a.R ? chunks : a.R;
  a.chunk = (int)((a.R + chunks - 1) / chunks);
  a.n_chunks = (a.R + a.chunk - 1) / a.chunk;
  const int64_t groups = (tiles * a.n_chunks + kWaves - 1) / kWaves;
  const unsigned grid = (unsigned)(groups < kMaxGroups ? groups : kMaxGroups);
  hipLaunchKernelGGL((k_adjust<T, G, kInPlace>), dim3(grid), dim3(kWaves * kWave), 0, st, a);
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
  a.status = status;
  (void)hipGetLastError();
  if (dtype == SV_BF16) {
    if (in_place) launch<__bf16, true>(a, (hipStream_t)stream);
    else launch<__bf16, false>(a, (hipStream_t)stream);
  } else {
    if (in_place) launch<float, true>(a, (hipStream_t)stream);
    else launch<float, false>(a, (hipStream_t)stream);
  }
  return hipGetLastError() == hipSuccess ? SV_OK : SV_ERR_DEVICE;
}
