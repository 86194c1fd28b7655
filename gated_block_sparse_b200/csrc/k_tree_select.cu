// Block selection of drafted tokens: scores over the cached block summaries,
// then gate and Top-K of every token's own row.
//
//   s_im = scale qbar_i . ksum_m, qbar_i the mean of the group's heads at
//   token i, m < c0; for a token whose path has filled the tail's block, also
//   s_i,c0 with the mean of that block's 64 keys (rounded to the summaries'
//   type); log g = s - LSE(s); the topk best, ties to the lower block.
//
// k_tree_scores: one CTA per (64 summaries, kv group, sequence) reads its
// summaries once for all T tokens. k_tree_select: one CTA per row.
#include <math.h>

#include "common.cuh"
#include "kernels.h"
#include "ptx.cuh"
#include "tree.cuh"

namespace sas {

__device__ uint32_t g_tree_select_err = 0;

namespace {
constexpr int TS_THREADS = 256;
constexpr int TS_BLOCKS = 64;  // summaries of a CTA
}

template <typename T, typename S, int D>
__global__ void __launch_bounds__(TS_THREADS) k_tree_scores(TreeArgs a, TreeWs w) {
  constexpr int LD = D + 4;
  extern __shared__ __align__(16) float sm_f[];
  float* ks = sm_f;                  // [64][LD]
  float* qb = sm_f + TS_BLOCKS * LD;  // [64][LD]
  const int r = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
  const int m0 = blockIdx.x * TS_BLOCKS, G = a.Hq / a.Hkv, C = a.N / SAS_BLOCK;
  const size_t group = (size_t)b * a.Hkv + r;
  if (tid < TS_BLOCKS / 32) {
    const int word = m0 / 32 + tid;
    if (word < a.words) w.ubits[group * a.words + word] = 0u;
  }
  const TreeSeq s = tree_seq(a, b, nullptr);
  if (m0 >= s.c0 || s.nt == 0) return;
  constexpr int VS = Vec16<S>::N, VT = Vec16<T>::N;
  for (int e = tid; e < TS_BLOCKS * (D / VS); e += TS_THREADS) {
    const int row = e / (D / VS), c = (e % (D / VS)) * VS, m = m0 + row;
    float x[VS];
#pragma unroll
    for (int i = 0; i < VS; ++i) x[i] = 0.f;
    if (m < s.c0) {
      const size_t at = a.table ? (size_t)tree_page(a, b, m, &g_tree_select_err) * a.Hkv + r
                                : group * C + m;
      Vec16<S>::load_nc(static_cast<const S*>(a.ksum) + at * D + c, x);
    }
#pragma unroll
    for (int i = 0; i < VS; ++i) ks[row * LD + c + i] = x[i];
  }
  const float inv_g = 1.0f / (float)G;
  for (int e = tid; e < TREE_MAX * (D / VT); e += TS_THREADS) {
    const int row = e / (D / VT), c = (e % (D / VT)) * VT;
    float x[VT];
#pragma unroll
    for (int i = 0; i < VT; ++i) x[i] = 0.f;
    if (row < s.nt)
      for (int g = 0; g < G; ++g) {
        float y[VT];
        Vec16<T>::load_nc(static_cast<const T*>(a.q) +
                              (((size_t)b * a.Hq + r * G + g) * a.T + row) * D + c, y);
#pragma unroll
        for (int i = 0; i < VT; ++i) x[i] += y[i];
      }
#pragma unroll
    for (int i = 0; i < VT; ++i) qb[row * LD + c + i] = x[i] * inv_g;
  }
  __syncthreads();
  // 4 x 4 scores a thread: tokens ti + 16 i, blocks tj + 16 j
  const int tj = tid & 15, ti = tid >> 4;
  if (ti >= s.nt) return;
  float acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
#pragma unroll 4
  for (int c = 0; c < D; c += 4) {
    float4 x[4], y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[i] = *reinterpret_cast<const float4*>(qb + (ti + 16 * i) * LD + c);
      y[i] = *reinterpret_cast<const float4*>(ks + (tj + 16 * i) * LD + c);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        acc[i][j] = fmaf(x[i].x, y[j].x, acc[i][j]);
        acc[i][j] = fmaf(x[i].y, y[j].y, acc[i][j]);
        acc[i][j] = fmaf(x[i].z, y[j].z, acc[i][j]);
        acc[i][j] = fmaf(x[i].w, y[j].w, acc[i][j]);
      }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int t = ti + 16 * i, m = m0 + tj + 16 * j;
      if (t < s.nt && m < s.c0) w.scores[(group * a.T + t) * C + m] = acc[i][j] * a.scale + 0.f;
    }
}

namespace {
constexpr int SEL_THREADS = 256;
}

__device__ __forceinline__ float block_sum(float v, float* red) {
  v = warp_sum(v);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float t = 0.f;
#pragma unroll
  for (int i = 0; i < SEL_THREADS / 32; ++i) t += red[i];
  __syncthreads();
  return t;
}
__device__ __forceinline__ float block_max(float v, float* red) {
  v = warp_max(v);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float t = red[0];
#pragma unroll
  for (int i = 1; i < SEL_THREADS / 32; ++i) t = fmaxf(t, red[i]);
  __syncthreads();
  return t;
}

template <typename T, typename S, int D>
__global__ void __launch_bounds__(SEL_THREADS) k_tree_select(TreeArgs a, TreeWs w) {
  extern __shared__ __align__(16) uint32_t keys[];  // (C_i) keys, thread t owns [t n, t n + n)
  __shared__ TreeShared tree;
  __shared__ float red[SEL_THREADS / 32];
  __shared__ uint32_t scan[SEL_THREADS / 32];
  __shared__ float part[SEL_THREADS];
  __shared__ int last_s;
  const int i = blockIdx.x, r = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
  if (tid == 0) last_s = -1;
  const int C = a.N / SAS_BLOCK, G = a.Hq / a.Hkv;
  const size_t group = (size_t)b * a.Hkv + r, row = group * a.T + i;
  const TreeSeq s = tree_seq(a, b, (i == 0 && r == 0) ? &g_tree_select_err : nullptr);
  if (i >= s.nt) return;
  tree_masks(a, b, s.nt, tree, (i == 0 && r == 0) ? &g_tree_select_err : nullptr);
  const unsigned long long anc = tree.anc[i];
  const int depth = tree_depth(anc);
  const bool crossed = s.tail + depth >= SAS_BLOCK;
  const int Ci = s.c0 + (crossed ? 1 : 0);
  const int kk = min(a.topk, Ci);
  float virt = 0.f;
  if (crossed) {
    // mean key of the tail's block as this path fills it: thread (half, column)
    // sums every second key, tail keys first, then the path's in their order
    constexpr int P = SEL_THREADS / D;
    const int c = tid % D, p = tid / D;
    const T* kc = static_cast<const T*>(a.kc);
    const T* kd = static_cast<const T*>(a.kd) + group * a.T * D;
    float sum = 0.f;
    if (s.tail > 0) {
      const size_t base = tree_block_row(a, b, r, s.c0, &g_tree_select_err);
      for (int j = p; j < s.tail; j += P) sum += to_f(kc[(base + j) * D + c]);
    }
    unsigned long long rest = anc;
    for (int n = 0; n < SAS_BLOCK - s.tail; ++n) {
      const int j = __ffsll((long long)rest) - 1;
      rest &= rest - 1;
      if ((n % P) == p) sum += to_f(kd[(size_t)j * D + c]);
    }
    part[tid] = sum;
    __syncthreads();
    float dot = 0.f;
    if (tid < D) {
      float mean = 0.f;
#pragma unroll
      for (int k = 0; k < P; ++k) mean += part[k * D + tid];
      mean = to_f(from_f<S>(mean * (1.0f / SAS_BLOCK)));
      float qb = 0.f;
      for (int g = 0; g < G; ++g)
        qb += to_f(static_cast<const T*>(a.q)[(((size_t)b * a.Hq + r * G + g) * a.T + i) * D + tid]);
      dot = qb * (1.0f / (float)G) * mean;
    }
    virt = block_sum(dot, red) * a.scale;
  }
  // each thread owns a stretch of n (odd: no bank conflicts) blocks
  const int n = ((Ci + SEL_THREADS - 1) / SEL_THREADS) | 1;
  const float* sc = w.scores + row * C;
  float mx = -INFINITY;
  for (int m = tid; m < Ci; m += SEL_THREADS) {
    const float v = m < s.c0 ? sc[m] : virt;
    keys[m] = score_key(v);
    mx = fmaxf(mx, v);
  }
  mx = block_max(mx, red);
  const int lo = min(tid * n, Ci), hi = min(lo + n, Ci);
  float sum = 0.f;
  for (int m = lo; m < hi; ++m) sum += expf(score_of(keys[m]) - mx);
  const float lse = mx + logf(block_sum(sum, red));
  // k-th largest key by bits, from the top: the largest th with at least kk keys >= th
  uint32_t th = 0;
  if (kk > 0) {
    for (int bit = 31; bit >= 0; --bit) {
      const uint32_t cand = th | (1u << bit);
      int c = 0;
      for (int m = lo; m < hi; ++m) c += keys[m] >= cand;
      c = (int)block_sum((float)c, red);
      if (c >= kk) th = cand;
    }
  }
  // keys above th are kept; of those equal to it the first ones, in block order
  uint32_t above = 0, equal = 0;
  for (int m = lo; m < hi; ++m) {
    above += keys[m] > th;
    equal += keys[m] == th;
  }
  uint32_t v = (above << 16) | equal;  // both below 2^16
  const int lane = tid & 31, wid = tid >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += y;
  }
  if (lane == 31) scan[wid] = v;
  __syncthreads();
  uint32_t before = v - ((above << 16) | equal), all = 0;
#pragma unroll
  for (int k = 0; k < SEL_THREADS / 32; ++k) {
    before += k < wid ? scan[k] : 0u;
    all += scan[k];
  }
  const int take = kk - (int)(all >> 16);  // of the keys equal to th
  int eq = (int)(before & 0xffffu);
  int at = (int)(before >> 16) + min(eq, take);
  if (kk > 0)
    for (int m = lo; m < hi; ++m) {
      const uint32_t key = keys[m];
      const bool keep = key > th || (key == th && eq < take);
      eq += key == th;
      if (key == th && eq == take) last_s = m;
      if (keep && at < kk) {
        if (a.idx_out) a.idx_out[row * a.topk + at] = m;
        if (m < s.c0) atomicOr(&w.ubits[group * a.words + (m >> 5)], 1u << (m & 31));
        ++at;
      }
    }
  if (a.idx_out)
    for (int p = kk + tid; p < a.topk; p += SEL_THREADS) a.idx_out[row * a.topk + p] = -1;
  __syncthreads();
  if (tid == 0) {
    TreeRow t;
    t.lse = lse;
    t.th = kk > 0 ? th : 0xffffffffu;
    t.last = last_s;
    t.tail_bias = 0.f;
    if (crossed) t.tail_bias = kk > 0 ? tree_bias(t, virt, s.c0, a.gated) : -INFINITY;
    w.rows[row] = t;
  }
}

// ------------------------------------------------------------------ host
template <typename T, typename S, int D>
static cudaError_t launch_typed(const TreeArgs& a, const TreeWs& w, cudaStream_t st) {
  const int C = a.N / SAS_BLOCK;
  const size_t smem = (size_t)(TS_BLOCKS + TREE_MAX) * (D + 4) * sizeof(float);
  cudaError_t e = ensure_smem(k_tree_scores<T, S, D>, smem);
  if (e != cudaSuccess) return e;
  const size_t ksm = (size_t)(C + 1) * sizeof(uint32_t);
  e = ensure_smem(k_tree_select<T, S, D>, ksm);
  if (e != cudaSuccess) return e;
  k_tree_scores<T, S, D><<<dim3((C + TS_BLOCKS - 1) / TS_BLOCKS, a.Hkv, a.B), TS_THREADS, smem,
                           st>>>(a, w);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  k_tree_select<T, S, D><<<dim3(a.T, a.Hkv, a.B), SEL_THREADS, ksm, st>>>(a, w);
  return cudaGetLastError();
}

cudaError_t launch_tree_select(const TreeArgs& a, const TreeWs& w, int bf16, int sum_bf16, int d,
                               cudaStream_t st) {
#define SAS_TREE(T, S)                                    \
  return d == 128 ? launch_typed<T, S, 128>(a, w, st) \
                  : launch_typed<T, S, 64>(a, w, st)
  if (bf16) {
    if (sum_bf16) SAS_TREE(__nv_bfloat16, __nv_bfloat16);
    SAS_TREE(__nv_bfloat16, float);
  }
  if (sum_bf16) SAS_TREE(float, __nv_bfloat16);
  SAS_TREE(float, float);
#undef SAS_TREE
}

// Workspace: bitmap, rows, scores, maxima and sums, partial outputs, each from
// a 256-byte boundary.
static size_t tree_carve(int B, int Hq, int Hkv, int T, int N, int d, int topk, int ns,
                         unsigned char* base, TreeWs* w) {
  const size_t groups = (size_t)B * Hkv, C = N / SAS_BLOCK, words = (C + 31) / 32;
  const size_t rows = groups * T, parts = groups * ns * (size_t)(Hq / Hkv) * T;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += (bytes + 255) & ~(size_t)255;
    return base ? base + here : nullptr;
  };
  TreeWs t;
  t.ubits = reinterpret_cast<uint32_t*>(take(topk > 0 ? groups * words * 4 : 0));
  t.rows = reinterpret_cast<TreeRow*>(take(topk > 0 ? rows * sizeof(TreeRow) : 0));
  t.scores = reinterpret_cast<float*>(take(topk > 0 ? rows * C * 4 : 0));
  t.ml = reinterpret_cast<float2*>(take(parts * sizeof(float2)));
  t.part = reinterpret_cast<float*>(take(parts * d * 4));
  if (w) *w = t;
  return at;
}

size_t tree_ws_bytes(int B, int Hq, int Hkv, int T, int N, int d, int topk, int bf16) {
  return tree_carve(B, Hq, Hkv, T, N, d, topk, tree_splits(B, Hq, Hkv, T, N, topk, bf16), nullptr,
                    nullptr);
}

cudaError_t launch_tree(TreeArgs a, int bf16, int sum_bf16, int d, void* ws, cudaStream_t st) {
  TreeWs w;
  a.words = (a.N / SAS_BLOCK + 31) / 32;
  a.ns = tree_splits(a.B, a.Hq, a.Hkv, a.T, a.N, a.topk, bf16);
  tree_carve(a.B, a.Hq, a.Hkv, a.T, a.N, d, a.topk, a.ns, static_cast<unsigned char*>(ws), &w);
  if (a.topk > 0) {
    cudaError_t e = launch_tree_select(a, w, bf16, sum_bf16, d, st);
    if (e != cudaSuccess) return e;
  }
  return bf16 ? launch_tree_attn_tc(a, w, d, st) : launch_tree_attn_simt(a, w, d, st);
}

uint32_t* tree_select_error_word() {
  void* p = nullptr;
  cudaGetSymbolAddress(&p, g_tree_select_err);
  return static_cast<uint32_t*>(p);
}

}  // namespace sas
