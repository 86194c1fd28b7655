// Attention of drafted tokens over the selected blocks, the cache's tail and
// their ancestors (fp32 caches), split over the units of a kv group, and the
// join of the splits.
//
//   o_i = softmax(scale q_i K + bias) V over the kept blocks (bias log g),
//   the tail and the path (bias 0, or log g of block c0 for the keys that a
//   path has moved into it; left out when the token does not keep c0).
//
// k_tree_attn_simt: one CTA per (32 rows, kv group, split), rows being the
// group's heads x drafted tokens. Every unit (64 keys) is read once per CTA;
// a warp owns four rows and keeps their running maximum, sum and output in
// registers. fp32 FMAs bound it: the copy of a unit's keys runs under the
// softmax and P V of the unit before, that of its values under Q K and the
// softmax, in one buffer each (at d 128 a second pair would halve the CTAs
// of an SM). Against both copied before the unit's arithmetic, us a call at d
// 128, top-k 31, random trees, contiguous: one sequence of 16300, 32/8 heads, 24
// tokens 104.3 -> 96.4; two of 3000, 8/2 heads, 20 tokens 50.6 -> 47.7; one of
// 8000, 32/8 heads, 8 tokens 68.5 -> 64.5; splits of one unit each are unchanged.
#include <math.h>

#include "common.cuh"
#include "kernels.h"
#include "ptx.cuh"
#include "tree.cuh"

namespace sas {

__device__ uint32_t g_tree_attn_err = 0;

namespace {
constexpr int TA_THREADS = 256;
constexpr int TA_ROWS = 32;  // rows of a CTA
constexpr int TA_WROWS = TA_ROWS / (TA_THREADS / 32);
constexpr float LOG2E = 1.4426950408889634f;
}  // namespace

template <int D>
__global__ void __launch_bounds__(TA_THREADS) k_tree_attn_simt(TreeArgs a, TreeWs w) {
  constexpr int LD = D + 4, E = D / 32;
  extern __shared__ __align__(16) float sm_f[];
  float* qs = sm_f;                 // [32][D]
  float* ks = qs + TA_ROWS * D;     // [64][LD]
  float* vs = ks + SAS_BLOCK * LD;  // [64][D]
  uint32_t* bits = reinterpret_cast<uint32_t*>(vs + SAS_BLOCK * D);
  __shared__ TreeShared tree;
  __shared__ int warp_s[TA_THREADS / 32];
  __shared__ int start_s;
  const int r = blockIdx.y, b = blockIdx.z, tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const int split = blockIdx.x % a.ns, tile = blockIdx.x / a.ns;
  const int G = a.Hq / a.Hkv;
  const size_t group = (size_t)b * a.Hkv + r;
  // without selection this kernel is the call's first: it waits before anything
  // else
  if (a.topk == 0) grid_dep_wait();
  grid_dep_launch();
  const bool report = a.topk == 0 && blockIdx.x == 0 && r == 0;  // else the selection does
  const TreeSeq s = tree_load(a, b, tree, report ? &g_tree_attn_err : nullptr);
  const int rows = G * s.nt, row0 = tile * TA_ROWS;
  if (row0 >= rows) {
    grid_dep_wait();
    return;
  }
  const unsigned long long early_tok = tree_early(tree);
  const float* q = static_cast<const float*>(a.q);
  for (int e = tid; e < TA_ROWS * D / 4; e += TA_THREADS) {
    const int i = e / (D / 4), row = min(row0 + i, rows - 1), c = (e % (D / 4)) * 4;
    cp_async16(qs + i * D + c,
               q + (((size_t)b * a.Hq + r * G + row / s.nt) * a.T + row % s.nt) * D + c,
               row0 + i < rows);
  }
  grid_dep_wait();
  int u0, u1;
  const int nu = tree_units<TA_THREADS>(a, w.ubits + group * a.words, bits, warp_s, &start_s,
                                        split, u0, u1);
  float m[TA_WROWS], l[TA_WROWS], acc[TA_WROWS][E];
  TreeRow info[TA_WROWS];
  int tok[TA_WROWS];
#pragma unroll
  for (int i = 0; i < TA_WROWS; ++i) {
    const int row = row0 + wid * TA_WROWS + i;
    m[i] = -1e30f;
    l[i] = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[i][e] = 0.f;
    tok[i] = row < rows ? row % s.nt : 0;
    info[i] = tree_row(a, w, s, group, tok[i], tree.anc[tok[i]]);
  }
  const float c1 = a.scale * LOG2E;
  // A unit's keys: where they lie and how many there are (0: none, no tail).
  struct Unit {
    const float *k, *v;
    int nk, blk;
  };
  auto unit = [&](int u, int blk) -> Unit {
    Unit x;
    x.nk = SAS_BLOCK;
    x.blk = blk;
    if (u > nu) {
      x.nk = s.nt;
      x.k = static_cast<const float*>(a.kd) + group * a.T * D;
      x.v = static_cast<const float*>(a.vd) + group * a.T * D;
      return x;
    }
    if (u < nu)
      x.blk = u == u0 ? start_s : tree_next(bits, a.words, blk + 1);
    else
      x.nk = s.tail;
    int place = x.nk > 0 ? tree_place(a, b, u < nu ? x.blk : s.c0, &g_tree_attn_err) : 0;
    if (place < 0) place = x.nk = 0;  // its page is outside the pool
    const size_t at = tree_block_row(a, b, r, place) * D;
    x.k = static_cast<const float*>(a.kc) + at;
    x.v = static_cast<const float*>(a.vc) + at;
    return x;
  };
  auto load = [&](float* dst, int ld, const float* src, int nk) {
#pragma unroll 4
    for (int e = tid; e < SAS_BLOCK * D / 4; e += TA_THREADS) {
      const int row = e / (D / 4), c = (e % (D / 4)) * 4;
      cp_async16(dst + row * ld + c, src + (size_t)min(row, nk - 1) * D + c, row < nk);
    }
  };
  // K of a unit is loaded under P V of the one before it, V under Q K: copies
  // in groups, K and V in turn (an empty group where there is none)
  int u = u0;
  Unit cur = {};
  if (u < u1) {
    cur = unit(u, -1);
    if (cur.nk == 0 && ++u < u1) cur = unit(u, cur.blk);
  }
  if (u < u1) load(ks, LD, cur.k, cur.nk);
  cp_async_commit();
  if (u < u1) load(vs, D, cur.v, cur.nk);
  cp_async_commit();
  while (u < u1) {
    const int nk = cur.nk, blk = cur.blk;
    cp_async_wait_group<1>();  // K
    __syncthreads();
    float z[TA_WROWS][2], p[TA_WROWS][2];
#pragma unroll
    for (int i = 0; i < TA_WROWS; ++i) z[i][0] = z[i][1] = 0.f;
#pragma unroll 4
    for (int c = 0; c < D; c += 4) {
      const float4 k0 = *reinterpret_cast<const float4*>(ks + lane * LD + c);
      const float4 k1 = *reinterpret_cast<const float4*>(ks + (lane + 32) * LD + c);
#pragma unroll
      for (int i = 0; i < TA_WROWS; ++i) {
        const float4 x = *reinterpret_cast<const float4*>(qs + (wid * TA_WROWS + i) * D + c);
        z[i][0] = fmaf(x.x, k0.x, fmaf(x.y, k0.y, fmaf(x.z, k0.z, fmaf(x.w, k0.w, z[i][0]))));
        z[i][1] = fmaf(x.x, k1.x, fmaf(x.y, k1.y, fmaf(x.z, k1.z, fmaf(x.w, k1.w, z[i][1]))));
      }
    }
    int next = u + 1;
    Unit nx = {};
    if (next < u1) {
      nx = unit(next, blk);
      if (nx.nk == 0 && ++next < u1) nx = unit(next, nx.blk);
    }
    __syncthreads();  // K has been read
    if (next < u1) load(ks, LD, nx.k, nx.nk);
    cp_async_commit();
#pragma unroll
    for (int i = 0; i < TA_WROWS; ++i) {
      const int row = row0 + wid * TA_WROWS + i;
      float bias[2] = {-INFINITY, -INFINITY};
      if (row < rows) {
        if (u < nu) {
          const float sc = __ldcg(w.scores + (group * a.T + tok[i]) * tree_stride(a.N / SAS_BLOCK) + blk);
          bias[0] = bias[1] = tree_bias(info[i], sc, blk, a.gated) * LOG2E;
        } else {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int j = lane + 32 * h;
            if (u == nu) {
              if (j < nk) bias[h] = info[i].tail_bias * LOG2E;
            } else if (j < nk && (tree.anc[tok[i]] >> j & 1ull)) {
              bias[h] = early_tok >> j & 1ull ? info[i].tail_bias * LOG2E : 0.f;
            }
          }
        }
      }
      // a masked key's logit is -inf whatever its product was
      const float z0 = bias[0] == -INFINITY ? -INFINITY : fmaf(z[i][0], c1, bias[0]);
      const float z1 = bias[1] == -INFINITY ? -INFINITY : fmaf(z[i][1], c1, bias[1]);
      const float mx = warp_max(fmaxf(z0, z1));
      p[i][0] = p[i][1] = 0.f;
      if (!(mx > -INFINITY) && !__any_sync(0xffffffffu, z0 != z0 || z1 != z1)) continue;
      const float mn = fmaxf(m[i], mx), alpha = exp2f(m[i] - mn);
      p[i][0] = exp2f(z0 - mn);
      p[i][1] = exp2f(z1 - mn);
      m[i] = mn;
      l[i] = l[i] * alpha + warp_sum(p[i][0] + p[i][1]);
#pragma unroll
      for (int e = 0; e < E; ++e) acc[i][e] *= alpha;
    }
    // O += P V: a key's values are read once for the warp's rows
    cp_async_wait_group<1>();  // V
    __syncthreads();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll 4
      for (int j = 0; j < 32; ++j) {
        float v[E];
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = vs[(32 * h + j) * D + lane * E + e];
#pragma unroll
        for (int i = 0; i < TA_WROWS; ++i) {
          const float pj = __shfl_sync(0xffffffffu, p[i][h], j);
          if (pj != 0.f) {  // a masked key's value is not touched
#pragma unroll
            for (int e = 0; e < E; ++e) acc[i][e] = fmaf(pj, v[e], acc[i][e]);
          }
        }
      }
    }
    __syncthreads();  // V has been read
    u = next;
    cur = nx;
    if (u < u1) load(vs, D, cur.v, cur.nk);
    cp_async_commit();
  }
  cp_async_wait();  // no copy in flight, also without a unit
#pragma unroll
  for (int i = 0; i < TA_WROWS; ++i) {
    const int row = row0 + wid * TA_WROWS + i;
    if (row >= rows) continue;
    const size_t at = (group * a.ns + split) * (size_t)(G * a.T) + row;
    if (lane == 0) w.ml[at] = make_float2(m[i], l[i]);
    if (l[i] != 0.f) {
      float* out = w.part + ((group * a.ns + split) * (size_t)(G * a.T)) * D + (size_t)row * 4 +
                   tree_part_at(lane * E, (size_t)G * a.T);
      if constexpr (E == 4)
        *reinterpret_cast<float4*>(out) = make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
      else
        *reinterpret_cast<float2*>(out) = make_float2(acc[i][0], acc[i][1]);
    }
  }
}

// Four values through L2, zeros when !on: a predicated load, so that several go
// out together.
__device__ __forceinline__ float4 load_if(const float* p, bool on) {
  float4 v;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.u32 p, %5, 0;\n\t"
      "mov.f32 %0, 0f00000000;\n\tmov.f32 %1, 0f00000000;\n\t"
      "mov.f32 %2, 0f00000000;\n\tmov.f32 %3, 0f00000000;\n\t"
      "@p ld.global.cg.v4.f32 {%0, %1, %2, %3}, [%4];\n\t}"
      : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
      : "l"(p), "r"((uint32_t)on)
      : "memory");
  return v;
}

// Joins the splits: o = sum_s 2^(m_s - M) o_s / sum_s 2^(m_s - M) l_s. One CTA
// per 8 / PARTS rows: a warp turns a row's maxima and sums into one factor per
// split (lane s); thread (row, four columns, part) adds every
// PARTS-th split's partial output, four in flight, and the parts meet in shared
// memory. A split that saw none of a row's keys has l = 0, and its partial
// output is not read. Two rows or more side by side make every access a full
// 32-byte sector. Latency bounds it: two dependent reads.
template <typename T, int D, int PARTS>
__global__ void __launch_bounds__(8 * D / 4) k_tree_join(TreeArgs a, TreeWs w) {
  constexpr int ROWS = 8 / PARTS, PER = D / 4, WARPS = 8 * PER / 32;
  __shared__ float fs[ROWS][32];
  __shared__ float4 part[PARTS > 1 ? PARTS - 1 : 1][ROWS * PER];
  const int b = blockIdx.z, r = blockIdx.y, lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const int G = a.Hq / a.Hkv, row0 = blockIdx.x * ROWS;
  int n, nt;
  tree_lengths(a, b, n, nt);
  grid_dep_wait();
  const int rows = G * nt;
  if (row0 >= rows) return;
  const size_t group = (size_t)b * a.Hkv + r, R = (size_t)G * a.T;
  for (int i = wid; i < ROWS; i += WARPS) {
    float2 ml = make_float2(-1e30f, 0.f);
    if (lane < a.ns && row0 + i < rows) ml = __ldcg(w.ml + (group * a.ns + lane) * R + row0 + i);
    const bool seen = ml.y != 0.f;
    const float M = warp_max(seen ? ml.x : -INFINITY);
    const float f = seen ? exp2f(ml.x - M) : 0.f;
    const float L = warp_sum(seen ? ml.y * f : 0.f);
    fs[i][lane] = seen ? f / L : -1.f;  // -1: not read
  }
  __syncthreads();
  const int e = threadIdx.x % (ROWS * PER), p = threadIdx.x / (ROWS * PER);
  const int i = e % ROWS, c4 = e / ROWS, row = row0 + i;
  const float* src = w.part + group * a.ns * R * D + ((size_t)c4 * R + row) * 4;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s0 = p; s0 < a.ns; s0 += 4 * PARTS) {
    float4 x[4];
    float g[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int s = s0 + PARTS * k;
      g[k] = s < a.ns ? fs[i][s] : -1.f;
      x[k] = load_if(src + s * R * D, !(g[k] < 0.f));
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      acc.x = fmaf(x[k].x, g[k], acc.x);
      acc.y = fmaf(x[k].y, g[k], acc.y);
      acc.z = fmaf(x[k].z, g[k], acc.z);
      acc.w = fmaf(x[k].w, g[k], acc.w);
    }
  }
  if constexpr (PARTS > 1) {
    if (p > 0) part[p - 1][e] = acc;
    __syncthreads();
    if (p > 0) return;
#pragma unroll
    for (int k = 0; k < PARTS - 1; ++k) {
      const float4 y = part[k][e];
      acc.x += y.x;
      acc.y += y.y;
      acc.z += y.z;
      acc.w += y.w;
    }
  }
  if (row >= rows) return;
  T* o = static_cast<T*>(a.o) +
         (((size_t)b * a.Hq + r * G + row / nt) * a.T + row % nt) * D + c4 * 4;
  if constexpr (sizeof(T) == 2) {
    const __nv_bfloat162 lo = __floats2bfloat162_rn(acc.x, acc.y);
    const __nv_bfloat162 hi = __floats2bfloat162_rn(acc.z, acc.w);
    *reinterpret_cast<uint2*>(o) = make_uint2(*reinterpret_cast<const uint32_t*>(&lo),
                                              *reinterpret_cast<const uint32_t*>(&hi));
  } else {
    *reinterpret_cast<float4*>(o) = acc;
  }
}

// ------------------------------------------------------------------ host
// Parts of a row's splits: four where there are many splits, which then means
// few rows; one thread adds up to eight.
template <typename T, int D>
static cudaError_t launch_join(const TreeArgs& a, const TreeWs& w, cudaStream_t st) {
  const int rows = a.Hq / a.Hkv * a.T;
  if (a.ns > 8)
    return tree_launch(k_tree_join<T, D, 4>, dim3((rows + 1) / 2, a.Hkv, a.B), 8 * D / 4, 0, st, a, w);
  return tree_launch(k_tree_join<T, D, 1>, dim3((rows + 7) / 8, a.Hkv, a.B), 8 * D / 4, 0, st, a, w);
}

cudaError_t launch_tree_join(const TreeArgs& a, const TreeWs& w, int bf16, int d,
                             cudaStream_t st) {
  if (bf16)
    return d == 128 ? launch_join<__nv_bfloat16, 128>(a, w, st)
                    : launch_join<__nv_bfloat16, 64>(a, w, st);
  return d == 128 ? launch_join<float, 128>(a, w, st) : launch_join<float, 64>(a, w, st);
}

template <int D>
static cudaError_t launch_simt(const TreeArgs& a, const TreeWs& w, cudaStream_t st) {
  const size_t smem =
      (size_t)(TA_ROWS * D + SAS_BLOCK * (D + 4) + SAS_BLOCK * D + a.words) * sizeof(float);
  cudaError_t e = ensure_smem(k_tree_attn_simt<D>, smem);
  if (e != cudaSuccess) return e;
  const int rows = a.Hq / a.Hkv * a.T, tiles = (rows + TA_ROWS - 1) / TA_ROWS;
  e = tree_launch(k_tree_attn_simt<D>, dim3(tiles * a.ns, a.Hkv, a.B), TA_THREADS, smem, st, a, w);
  return e != cudaSuccess ? e : launch_tree_join(a, w, 0, D, st);
}

cudaError_t launch_tree_attn_simt(const TreeArgs& a, const TreeWs& w, int d, cudaStream_t st) {
  return d == 128 ? launch_simt<128>(a, w, st) : launch_simt<64>(a, w, st);
}

// Splits of a kv group's units: as many as one wave of two CTAs an SM holds (a
// second, shorter wave costs another start: 8 x 128K 62 us a call, 69 with
// twice the splits, 83 with one CTA an SM), and no more than the units that the
// tokens can select. How many they do select is not known here, and splits
// without a unit still cost the join: at most 20 (64K, 4 tokens, some 20 units:
// 20.1 us a call, 22.2 with 32 splits, 22.0 with 8), or 24 of the fp32 kernel,
// whose units take longer (20 tokens over 46 blocks: 51 us with 24 splits, 62
// with 20). Even two units are split: a unit of one CTA costs as much as the
// join. The cap was set where units are few; a call with one kv head and many
// selected units would use the 32 splits that the join takes at most (one
// sequence of 128K, 64 tokens, top-k 127: 37.0 us with 32, 44.1 as it is; top-k
// 63 31.1 and 33.2; 4 tokens, top-k 15 18.3 and 18.5).
int tree_splits(int B, int Hq, int Hkv, int T, int N, int topk, int bf16) {
  const int tile = bf16 ? 128 : TA_ROWS;
  const long long tiles = ((long long)(Hq / Hkv) * T + tile - 1) / tile;
  const long long ctas = tiles * Hkv * B;
  long long units = (long long)T * topk;
  if (units > N / SAS_BLOCK) units = N / SAS_BLOCK;
  long long ns = 2 * 148 / ctas;
  if (ns > units + 2) ns = units + 2;
  const int most = bf16 ? 20 : 24;
  if (ns > most) ns = most;
  return ns < 1 ? 1 : (int)ns;
}

uint32_t* tree_attn_error_word() {
  void* p = nullptr;
  cudaGetSymbolAddress(&p, g_tree_attn_err);
  return static_cast<uint32_t*>(p);
}

}  // namespace sas
