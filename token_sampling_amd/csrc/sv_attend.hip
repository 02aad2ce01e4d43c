// sv_attend.hip -- sv_cache_attention: attention of a round's rows over the paged
// cache, after a plan (sv_plan.hip).
//
// With scores z_t = scale * q . k_t and running largest score m, sum l and values o,
// a tile of keys t turns them into
//   m' = max(m, max z_t),  l' = l 2^(m - m') + sum 2^(z_t - m'),
//   o' = o 2^(m - m') + sum 2^(z_t - m') v_t     (scores times log2 e)
// and partial results join the same way, so keys may be split at will.
#include "sv_attend.hpp"

namespace sv {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

struct Bf {
  typedef __bf16 vec8 __attribute__((ext_vector_type(8)));
  typedef __bf16 vec2 __attribute__((ext_vector_type(2)));
  static constexpr uint32_t kExp = 0x7F80u;  // exponent of infinities and NaN
  __device__ static inline f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(vec8, a),
                                                   __builtin_bit_cast(vec8, b), c, 0, 0, 0);
  }
};
struct Hf {
  typedef _Float16 vec8 __attribute__((ext_vector_type(8)));
  typedef _Float16 vec2 __attribute__((ext_vector_type(2)));
  static constexpr uint32_t kExp = 0x7C00u;
  __device__ static inline f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(vec8, a),
                                                  __builtin_bit_cast(vec8, b), c, 0, 0, 0);
  }
};
template <typename E>
__device__ inline uint32_t pack2(float x, float y) {  // to nearest, ties to even
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{x, y}, typename E::vec2));
}

struct AttendArgs {
  CacheView c;
  AttendPlan p;
  const char* q;
  int64_t q_session, q_row, q_head;
  char* out;
  float* part_o;   // [slots][per][head_dim]
  float* part_ml;  // [slots][per][2]
  float scale;     // times log2 e
  int64_t base;    // the layer's first element
  int32_t G, B, R, per;
};

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;

// A workgroup goes over a piece of the line, set by set: its waves take the tiles of
// 32 keys in turn, each for all rows of the set, and join at the set's end.
template <typename E, int D, int NT>
__global__ __launch_bounds__(kThreads) void k_attend(AttendArgs a) {
  constexpr int kC = D / 32, kN = D / 16;
  __shared__ f32x4 red[kWaves][kN][kWave];
  __shared__ float red_m[kWaves][NT * 16], red_l[kWaves][NT * 16];
  const int tid = threadIdx.x, wave = tid / kWave, lane = tid % kWave;
  const int col = lane % 16, g = lane / 16;
  const CacheView& c = a.c;
  const int64_t total = a.p.head->total, piece = a.p.head->piece;
  int64_t x = blockIdx.x * piece;
  const int64_t x_end = min(x + piece, total);
  if (x >= x_end) return;
  const int4 start = a.p.starts[blockIdx.x];
  int s = start.x, head = start.y, blk = start.z;
  while (x < x_end) {
    const AttendSet set = a.p.sets[s];
    const int nb = set.blocks();
    const int cnt = (int)min((int64_t)(nb - blk), x_end - x);
    // ---- the set's rows
    u32x4 q[NT][kC];
    int lim[NT];  // a row sees the keys before it
    int64_t out_at[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int j = t * 16 + col;
      lim[t] = 0;
      out_at[t] = -1;
      int64_t at = -1;
      if (j < set.n) {
        const int jj = set.j0 + j, place = set.t0 + jj / a.G, row = a.p.row_of[place];
        const int b = row / a.R, r = row % a.R, hq = head * a.G + jj % a.G;
        at = b * a.q_session + r * a.q_row + hq * a.q_head;
        lim[t] = set.base + r + 1;
        out_at[t] = ((int64_t)row * (a.G * c.n_kv) + hq) * D;
      }
#pragma unroll
      for (int i = 0; i < kC; ++i)
        q[t][i] = at >= 0 ? *(const u32x4*)(a.q + 2 * (at + i * 32 + g * 8)) : u32x4{0, 0, 0, 0};
    }
    f32x4 o[NT][kN];
    float m[NT], l[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      m[t] = -INFINITY, l[t] = 0;
#pragma unroll
      for (int i = 0; i < kN; ++i) o[t][i] = f32x4{0, 0, 0, 0};
    }
    // ---- its keys
    const int32_t* list = c.table + (int64_t)set.slot * c.max_pages;
    const int lo = set.key0 + blk * kBlock, hi = min(set.key0 + (blk + cnt) * kBlock, set.key1);
    for (int key = lo + wave * 32; key < hi; key += kWaves * 32) {
      const uint32_t page = min((uint32_t)list[key >> c.shift], (uint32_t)(c.n_pages - 1));
      const int64_t at = a.base + page * c.page_elems() + head * c.head_elems() +
                         (int64_t)(key & (c.page() - 1)) * D;
      const u32x4* kp = (const u32x4*)(c.k + 2 * at) + lane;
      const u32x4* vp = (const u32x4*)(c.v + 2 * at) + lane;
      u32x4 kf[2][kC], vf[kN];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < kC; ++i) kf[h][i] = kp[(h * kC + i) * kWave];
#pragma unroll
      for (int i = 0; i < kN; ++i) vf[i] = vp[i * kWave];
      const bool edge = key + 32 > set.base + 1;  // some row does not see all keys
      bool odd = false;                           // values that are not finite
      if (edge) {
        // nothing behind the last key has been written for this session
#pragma unroll
        for (int i = 0; i < kN; ++i)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            if (key + g * 8 + e >= set.key1) vf[i][e / 2] &= e % 2 ? 0x0000FFFFu : 0xFFFF0000u;
            odd |= (vf[i][e / 2] >> (16 * (e % 2)) & E::kExp) == E::kExp;
          }
        odd = __any(odd);
      }
      u32x4 w[NT];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        f32x4 z[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          z[h] = f32x4{0, 0, 0, 0};
#pragma unroll
          for (int i = 0; i < kC; ++i) z[h] = E::mfma(kf[h][i], q[t][i], z[h]);
        }
        if (edge) {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (key + g * 8 + e >= lim[t]) z[e / 4][e % 4] = -INFINITY;
        }
        float top = z[0][0];
#pragma unroll
        for (int e = 1; e < 8; ++e) top = fmaxf(top, z[e / 4][e % 4]);
        top = fmaxf(top, lane_xor<16>(top));
        top = fmaxf(top, lane_xor<32>(top));
        const float now = fmaxf(m[t], top * a.scale);
        const float use = now == -INFINITY ? 0.0f : now;  // a row that has seen nothing
        const float keep = __builtin_amdgcn_exp2f(m[t] - use);
        m[t] = now;
        float p[8], sum = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          p[e] = __builtin_amdgcn_exp2f(fmaf(z[e / 4][e % 4], a.scale, -use));
          sum += p[e];
        }
        l[t] = l[t] * keep + sum;
#pragma unroll
        for (int i = 0; i < kN; ++i) o[t][i] *= keep;
#pragma unroll
        for (int e = 0; e < 4; ++e) w[t][e] = pack2<E>(p[2 * e], p[2 * e + 1]);
      }
      if (!odd) {
#pragma unroll
        for (int i = 0; i < kN; ++i)
#pragma unroll
          for (int t = 0; t < NT; ++t) o[t][i] = E::mfma(vf[i], w[t], o[t][i]);
      } else {
        // key by key, so that a value that is not finite reaches only rows that see it
        for (int u = 0; u < 32; ++u) {
#pragma unroll
          for (int i = 0; i < kN; ++i) {
            u32x4 one;
#pragma unroll
            for (int e = 0; e < 4; ++e)
              one[e] = vf[i][e] & ((g * 8 + 2 * e == u ? 0x0000FFFFu : 0u) |
                                   (g * 8 + 2 * e + 1 == u ? 0xFFFF0000u : 0u));
#pragma unroll
            for (int t = 0; t < NT; ++t) {
              const f32x4 with = E::mfma(one, w[t], o[t][i]);
              if (key + u < lim[t]) o[t][i] = with;
            }
          }
        }
      }
    }
    // ---- the waves' results joined
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      l[t] += lane_xor<16>(l[t]);
      l[t] += lane_xor<32>(l[t]);
      if (lane < 16) {
        red_m[wave][t * 16 + lane] = m[t];
        red_l[wave][t * 16 + lane] = l[t];
      }
    }
    __syncthreads();
    const int64_t part = (int64_t)s * c.n_kv + head + blockIdx.x;
    const bool whole = set.alone && cnt == nb;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int j = t * 16 + col;
      float top = -INFINITY, sum = 0;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) top = fmaxf(top, red_m[w][j]);
      const float use = top == -INFINITY ? 0.0f : top;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) sum += red_l[w][j] * __builtin_amdgcn_exp2f(red_m[w][j] - use);
      const float mine = __builtin_amdgcn_exp2f(m[t] - use);
#pragma unroll
      for (int i = 0; i < kN; ++i) red[wave][i][lane] = o[t][i] * mine;
      __syncthreads();
      if (j < set.n) {
        const float norm = 1.0f / sum;
#pragma unroll
        for (int i0 = 0; i0 < (kN + kWaves - 1) / kWaves; ++i0) {
          const int i = i0 * kWaves + wave;
          if (i >= kN) break;
          f32x4 all = red[0][i][lane];
#pragma unroll
          for (int w = 1; w < kWaves; ++w) all += red[w][i][lane];
          if (whole) {
            uint2 y;
            y.x = pack2<E>(all[0] * norm, all[1] * norm);
            y.y = pack2<E>(all[2] * norm, all[3] * norm);
            *(uint2*)(a.out + 2 * (out_at[t] + i * 16 + g * 4)) = y;
          } else {
            *(f32x4*)(a.part_o + (part * a.per + j) * D + i * 16 + g * 4) = all;
          }
        }
        if (!whole && wave == 0 && g == 0)
          *(f32x2*)(a.part_ml + (part * a.per + j) * 2) = f32x2{top, sum};
      }
      __syncthreads();
    }
    x += cnt;
    blk = 0;
    if (++head == c.n_kv) head = 0, ++s;
  }
}

// Joins the partial results of every row; a wave a row and head.  NaN where the
// session failed.
template <typename E, int D>
__global__ __launch_bounds__(kThreads) void k_join(AttendArgs a) {
  constexpr int kVec = D % 128 == 0 ? D / 64 : D == 96 ? 2 : 1;  // elements a lane
  const int lane = threadIdx.x % kWave;
  const CacheView& c = a.c;
  const int b = blockIdx.x / a.R, r = blockIdx.x % a.R;
  const AttendSession ss = a.p.sess[b];
  const int heads = a.G * c.n_kv;
  if (ss.status == 0 && r >= ss.n) return;
  const int64_t total = a.p.head->total, piece = a.p.head->piece;
  (void)total;
  for (int hq = threadIdx.x / kWave + blockIdx.y * kWaves; hq < heads; hq += kWaves * gridDim.y) {
    char* out = a.out + 2 * (((int64_t)blockIdx.x * heads + hq) * D + lane * kVec);
    float o[kVec], m = -INFINITY, l = 0;
#pragma unroll
    for (int i = 0; i < kVec; ++i) o[i] = 0;
    bool done = false;
    if (ss.status == 0) {
#pragma unroll
      for (int level = 0; level < 3; ++level) {
        const int first = level < 2 ? ss.node[level] : ss.leaf;
        if (first < 0) continue;
        const int j = (ss.t0 + r - a.p.sets[first].t0) * a.G + hq % a.G;
        const int s = first + j / a.per, row = j % a.per, head = hq / a.G;
        const AttendSet& set = a.p.sets[s];
        const int nb = set.blocks();
        const int64_t x = set.cum * c.n_kv + (int64_t)head * nb;
        const int p0 = (int)(x / piece), p1 = (int)((x + nb - 1) / piece);
        if (set.alone && p0 == p1) done = true;
        if (done) break;
        for (int p = p0; p <= p1; ++p) {
          const int64_t at = ((int64_t)s * c.n_kv + head + p) * a.per + row;
          const f32x2 ml = *(const f32x2*)(a.part_ml + at * 2);
          const float now = fmaxf(m, ml[0]), use = now == -INFINITY ? 0.0f : now;
          const float old = __builtin_amdgcn_exp2f(m - use), add = __builtin_amdgcn_exp2f(ml[0] - use);
          m = now;
          l = l * old + ml[1] * add;
          if (lane * kVec < D) {
            const float* y = a.part_o + at * D + lane * kVec;
#pragma unroll
            for (int i = 0; i < kVec; ++i) o[i] = o[i] * old + y[i] * add;
          }
        }
      }
    } else {
      l = NAN;
    }
    if (done || lane * kVec >= D) continue;
    const float norm = 1.0f / l;
    if constexpr (kVec == 1) {
      *(uint16_t*)out = (uint16_t)pack2<E>(o[0] * norm, 0);
    } else {
#pragma unroll
      for (int i = 0; i < kVec; i += 2) *(uint32_t*)(out + 2 * i) = pack2<E>(o[i] * norm, o[i + 1] * norm);
    }
  }
}

template <typename E, int D>
void launch(const AttendArgs& a, hipStream_t st) {
  if (a.per == 16)
    hipLaunchKernelGGL((k_attend<E, D, 1>), dim3(kPieces), dim3(kThreads), 0, st, a);
  else if (a.per == 32)
    hipLaunchKernelGGL((k_attend<E, D, 2>), dim3(kPieces), dim3(kThreads), 0, st, a);
  else if constexpr (D <= 128)
    hipLaunchKernelGGL((k_attend<E, D, 4>), dim3(kPieces), dim3(kThreads), 0, st, a);
  const int heads = a.G * a.c.n_kv;
  const unsigned gy = (heads + 8 * kWaves - 1) / (8 * kWaves);
  hipLaunchKernelGGL((k_join<E, D>), dim3(a.B * a.R, gy), dim3(kThreads), 0, st, a);
}
template <typename E>
void launch_dim(const AttendArgs& a, hipStream_t st) {
  switch (a.c.head_dim) {
    case 64: return launch<E, 64>(a, st);
    case 96: return launch<E, 96>(a, st);
    case 128: return launch<E, 128>(a, st);
    default: return launch<E, 256>(a, st);
  }
}

bool stride_ok(int64_t s) { return s >= 0 && s % 8 == 0 && s <= ((int64_t)1 << 40); }

// Slots for partial results: one a set and head, and one for every cut.
int64_t slots_of(const sv_cache* c, int64_t sets) { return sets * c->n_kv + kPieces; }

}  // namespace
}  // namespace sv

extern "C" size_t sv_cache_attention_bytes(const sv_cache* cache, int32_t n_heads, int32_t B,
                                           int32_t R) {
  using namespace sv;
  if (sv_cache_plan_bytes(cache, n_heads, B, R) == 0) return 0;
  const int G = n_heads / cache->n_kv, per = rows_of_set((int64_t)R * G, cache->head_dim);
  const int64_t slots = slots_of(cache, plan_sizes(B, R, G, per).sets);
  return (size_t)(slots * per * (cache->head_dim + 2) * 4);
}

extern "C" int sv_cache_attention(const sv_cache* cache, int32_t layer, const void* q,
                                  int64_t q_session, int64_t q_row, int64_t q_head, float scale,
                                  const void* plan, int32_t n_heads, int32_t B, int32_t R,
                                  void* out, void* workspace, size_t workspace_bytes, void* stream) {
  using namespace sv;
  const size_t need = sv_cache_attention_bytes(cache, n_heads, B, R);
  if (need == 0 || layer < 0 || layer >= cache->n_layers || !q || !plan || !out || !workspace)
    return SV_ERR_ARG;
  if (((uintptr_t)q | (uintptr_t)plan | (uintptr_t)out | (uintptr_t)workspace) % 16 != 0)
    return SV_ERR_ARG;
  if (!stride_ok(q_session) || !stride_ok(q_row) || !stride_ok(q_head)) return SV_ERR_ARG;
  if (!(scale > 0) || !(scale < INFINITY)) return SV_ERR_ARG;
  if (workspace_bytes < need) return SV_ERR_WORKSPACE;
  const int G = n_heads / cache->n_kv, per = rows_of_set((int64_t)R * G, cache->head_dim);
  const PlanSizes z = plan_sizes(B, R, G, per);
  AttendArgs a = {view_of(cache), plan_of(z, (void*)plan), (const char*)q, q_session, q_row, q_head,
                  (char*)out, (float*)workspace, nullptr, scale * 1.44269504088896340736f, 0, G, B,
                  R, per};
  a.part_ml = a.part_o + slots_of(cache, z.sets) * per * cache->head_dim;
  a.base = layer * a.c.layer_elems();
  hipStream_t st = (hipStream_t)stream;
  (void)hipGetLastError();
  if (cache->dtype == SV_BF16) launch_dim<Bf>(a, st);
  else launch_dim<Hf>(a, st);
  return hipGetLastError() == hipSuccess ? SV_OK : SV_ERR_DEVICE;
}
