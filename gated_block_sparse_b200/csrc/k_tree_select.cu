// Block selection of drafted tokens: scores over the cached block summaries,
// then gate and Top-K of every token's own row.
//
//   s_im = scale qbar_i . ksum_m, qbar_i the mean of the group's heads at
//   token i, m < c0; for a token whose path has filled the tail's block, also
//   s_i,c0 with the mean of that block's 64 keys (rounded to the summaries'
//   type); log g = s - LSE(s); the topk best, ties to the lower block.
//
// k_tree_scores reads every summary once for all T tokens. The products are
// tensor-core work (T x C x d multiply-adds: fp32 FMAs would take 14 us at
// 512K and T = 64, where the summaries' bytes take 5), but the order of the
// blocks needs fp32: each factor is split into two tf32 parts, x = hi + lo + e
// with |e| <= 2^-22 |x|, and hi hi + hi lo + lo hi is accumulated in fp32
// (bf16 summaries are tf32 values: one part). What is dropped is 2^-22 of a
// product, below the fp32 accumulation's own rounding.
// k_tree_select: one CTA per row.
#include <math.h>

#include "common.cuh"
#include "kernels.h"
#include "ptx.cuh"
#include "tree.cuh"

namespace sas {

__device__ uint32_t g_tree_select_err = 0;

namespace {

constexpr int TS_THREADS = 128;
constexpr int TS_BLOCKS = 16 * (TS_THREADS / 32);  // summaries of a pass: 16 a warp

// D += A B, m16n8k8: A[row][k], B[k][col] in tf32 (row-major, column-major
// fragments), D in fp32.
__device__ __forceinline__ void mma_tf32(float (&c)[4], const float (&a)[4], float b0, float b1) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(__float_as_uint(a[0])), "r"(__float_as_uint(a[1])), "r"(__float_as_uint(a[2])),
        "r"(__float_as_uint(a[3])), "r"(__float_as_uint(b0)), "r"(__float_as_uint(b1)));
}

// The leading 11 significant bits of x (a tf32 value), and of what is left.
__device__ __forceinline__ float tf32_hi(float x) {
  return __uint_as_float(__float_as_uint(x) & 0xffffe000u);
}

// Four consecutive summary elements as loaded.
template <typename S> struct Raw;
template <> struct Raw<float> {
  float4 v;
  __device__ __forceinline__ void load(const float* p) {
    v = __ldg(reinterpret_cast<const float4*>(p));
  }
  __device__ __forceinline__ float get(int i) const {
    return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
  }
};
template <> struct Raw<__nv_bfloat16> {
  uint2 v;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    v = __ldg(reinterpret_cast<const uint2*>(p));
  }
  __device__ __forceinline__ float get(int i) const {
    const uint32_t w = i < 2 ? v.x : v.y;
    return __uint_as_float((i & 1) ? (w & 0xffff0000u) : (w << 16));
  }
};

}  // namespace

// One CTA per (stretch of summaries, kv group, sequence). A warp multiplies 16
// summaries (rows of A, straight from global memory) with all tokens (columns
// of B, in shared memory, split once). The order of the k index inside a group
// of 16 is free as long as A and B share it: lane c of a quad takes elements
// 4c .. 4c + 3, one 16-byte load, as k = c and c + 4 of two steps. Rows of
// shared memory are D + 16 floats apart, so that those loads meet no bank twice.
template <typename T, typename S, int D>
__global__ void __launch_bounds__(TS_THREADS, 3) k_tree_scores(TreeArgs a, TreeWs w, int stretch) {
  constexpr int LD = D + 16, VT = Vec16<T>::N, KG = D / 16;
  constexpr bool SPLIT = sizeof(S) == 4;
  extern __shared__ __align__(16) float sm_f[];
  const int T8 = (a.T + 7) & ~7;
  float* qh = sm_f;            // [T8][LD]
  float* ql = sm_f + T8 * LD;  // [T8][LD]
  const int r = blockIdx.y, b = blockIdx.z, tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const int G = a.Hq / a.Hkv, C = a.N / SAS_BLOCK;
  const int m_lo = blockIdx.x * stretch;
  const size_t group = (size_t)b * a.Hkv + r;
  grid_dep_wait();
  grid_dep_launch();
  for (int i = m_lo / 32 + tid; i < min((m_lo + stretch) / 32, a.words); i += TS_THREADS)
    w.ubits[group * a.words + i] = 0u;
  const int n = __ldg(a.lens + b), ntk = a.ntok ? __ldg(a.ntok + b) : a.T;
  const int c0 = min(max(n, 0), a.N) / SAS_BLOCK, nt = min(max(ntk, 0), a.T);
  const int m_hi = min(m_lo + stretch, c0);
  if (m_lo >= m_hi || nt == 0) return;
  // A of a pass: rows quad and quad + 8 of the warp's 16 (a row past the end
  // reads the last one), loaded a pass ahead
  const int quad = lane >> 2, c = lane & 3, ntiles = (nt + 7) >> 3;
  const S* sums = static_cast<const S*>(a.ksum) + 4 * c;
  auto row_at = [&](int m) -> size_t {
    m = min(m, m_hi - 1);
    return (a.table ? (size_t)tree_page(a, b, m, &g_tree_select_err) * a.Hkv + r : group * C + m) * D;
  };
  Raw<S> x[2][KG];
  size_t at[2];
  int m0 = m_lo + wid * 16;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    at[h] = row_at(m0 + quad + 8 * h);
#pragma unroll
    for (int g = 0; g < KG; ++g) x[h][g].load(sums + at[h] + 16 * g);
    at[h] = row_at(m0 + TS_BLOCKS + quad + 8 * h);
  }
  const float inv_g = 1.0f / (float)G;
#pragma unroll 2
  for (int e = tid; e < T8 * (D / VT); e += TS_THREADS) {
    const int row = e / (D / VT), col = (e % (D / VT)) * VT;
    float s[VT];
#pragma unroll
    for (int i = 0; i < VT; ++i) s[i] = 0.f;
    if (row < nt) {
      const T* q = static_cast<const T*>(a.q) + (((size_t)b * a.Hq + r * G) * a.T + row) * D + col;
#pragma unroll 4
      for (int g = 0; g < G; ++g) {
        float y[VT];
        Vec16<T>::load_nc(q + (size_t)g * a.T * D, y);
#pragma unroll
        for (int i = 0; i < VT; ++i) s[i] += y[i];
      }
    }
#pragma unroll
    for (int i = 0; i < VT; i += 4) {
      float4 h, l;
      const float m[4] = {s[i] * inv_g, s[i + 1] * inv_g, s[i + 2] * inv_g, s[i + 3] * inv_g};
      h = make_float4(tf32_hi(m[0]), tf32_hi(m[1]), tf32_hi(m[2]), tf32_hi(m[3]));
      l = make_float4(tf32_hi(m[0] - h.x), tf32_hi(m[1] - h.y), tf32_hi(m[2] - h.z),
                      tf32_hi(m[3] - h.w));
      *reinterpret_cast<float4*>(qh + row * LD + col + i) = h;
      *reinterpret_cast<float4*>(ql + row * LD + col + i) = l;
    }
  }
  __syncthreads();
  const int CS = tree_stride(C);
  float* out = w.scores + group * a.T * CS;
  for (; m0 < m_hi; m0 += TS_BLOCKS) {
    float acc[TREE_MAX / 8][4];
#pragma unroll
    for (int j = 0; j < TREE_MAX / 8; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[j][i] = 0.f;
    const bool more = m0 + TS_BLOCKS < m_hi;
#pragma unroll
    for (int g = 0; g < KG; ++g) {
      float hi[2][4], lo[2][4];  // of the two k steps of this group
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // fragment i: row half i & 1, k half i >> 1
          const float v = x[i & 1][g].get(2 * k + (i >> 1));
          hi[k][i] = SPLIT ? tf32_hi(v) : v;
          lo[k][i] = SPLIT ? tf32_hi(v - hi[k][i]) : 0.f;
        }
      if (more) {  // this group's registers take the next pass's values
#pragma unroll
        for (int h = 0; h < 2; ++h) x[h][g].load(sums + at[h] + 16 * g);
      }
      // four token tiles at a time: consecutive MMAs go to different sums
#pragma unroll
      for (int j0 = 0; j0 < TREE_MAX / 8; j0 += 4) {
        if (j0 >= ntiles) break;
        float4 bh[4], bl[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (j0 + j < ntiles) {
            const int o = (8 * (j0 + j) + quad) * LD + 16 * g + 4 * c;
            bh[j] = *reinterpret_cast<const float4*>(qh + o);
            bl[j] = *reinterpret_cast<const float4*>(ql + o);
          }
#define SAS_EACH(A, X, Y)              \
  _Pragma("unroll") for (int j = 0; j < 4; ++j) if (j0 + j < ntiles) \
      mma_tf32(acc[j0 + j], A, X, Y)
        SAS_EACH(hi[0], bl[j].x, bl[j].y);
        SAS_EACH(hi[1], bl[j].z, bl[j].w);
        if (SPLIT) {
          SAS_EACH(lo[0], bh[j].x, bh[j].y);
          SAS_EACH(lo[1], bh[j].z, bh[j].w);
        }
        SAS_EACH(hi[0], bh[j].x, bh[j].y);
        SAS_EACH(hi[1], bh[j].z, bh[j].w);
#undef SAS_EACH
      }
    }
    if (more) {
#pragma unroll
      for (int h = 0; h < 2; ++h) at[h] = row_at(m0 + 2 * TS_BLOCKS + quad + 8 * h);
    }
    float* o = out + (size_t)(2 * c) * CS + m0 + quad;
#pragma unroll
    for (int j = 0; j < TREE_MAX / 8; ++j) {
      if (j < ntiles) {
#pragma unroll
        for (int i = 0; i < 4; ++i)  // row quad + 8 (i >> 1), column 2 c + (i & 1)
          if (8 * j + 2 * c + (i & 1) < nt && m0 + quad + 8 * (i >> 1) < m_hi)
            o[(size_t)(8 * j + (i & 1)) * CS + 8 * (i >> 1)] = acc[j][i] * a.scale + 0.f;
      }
    }
  }
}

namespace {
constexpr int SEL_THREADS = 256;
constexpr int SEL_WARPS = SEL_THREADS / 32;
constexpr int SEL_LIST = 512;  // candidates ranked by counting
constexpr float LOG2E = 1.4426950408889634f;
}  // namespace

__device__ __forceinline__ float block_sum(float v, float* red) {
  v = warp_sum(v);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float t = 0.f;
#pragma unroll
  for (int i = 0; i < SEL_WARPS; ++i) t += red[i];
  __syncthreads();
  return t;
}

// The kk-th best of n keys and the last block that is kept at that key, for
// sets with more equal or near-equal keys than the list holds: the threshold
// bit by bit, then the keys equal to it in block order. Every thread owns the
// stretch [lo, hi). Returns through th and last (shared).
__device__ __noinline__ void select_by_bits(const uint32_t* keys, int lo, int hi, int kk,
                                            uint32_t* scan, uint32_t* th_s, int* last_s) {
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  uint32_t th = 0;
  for (int bit = 31; bit >= 0; --bit) {
    const uint32_t cand = th | (1u << bit);
    uint32_t c = 0;
    for (int m = lo; m < hi; ++m) c += keys[m] >= cand;
    c = __reduce_add_sync(0xffffffffu, c);
    if (lane == 0) scan[wid] = c;
    __syncthreads();
    c = 0;
#pragma unroll
    for (int i = 0; i < SEL_WARPS; ++i) c += scan[i];
    if (c >= (uint32_t)kk) th = cand;
    __syncthreads();
  }
  uint32_t above = 0, equal = 0;
  for (int m = lo; m < hi; ++m) {
    above += keys[m] > th;
    equal += keys[m] == th;
  }
  uint32_t v = (above << 16) | equal;  // both below 2^16
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += y;
  }
  if (lane == 31) scan[wid] = v;
  __syncthreads();
  uint32_t before = v - ((above << 16) | equal), all = 0;
#pragma unroll
  for (int i = 0; i < SEL_WARPS; ++i) {
    before += i < wid ? scan[i] : 0u;
    all += scan[i];
  }
  const int take = kk - (int)(all >> 16);  // of the keys equal to th
  int eq = (int)(before & 0xffffu);
  for (int m = lo; m < hi; ++m)
    if (keys[m] == th && ++eq == take) *last_s = m;
  if (tid == 0) *th_s = th;
  __syncthreads();
}

template <typename T, typename S, int D>
__global__ void __launch_bounds__(SEL_THREADS) k_tree_select(TreeArgs a, TreeWs w) {
  extern __shared__ __align__(16) float vals[];  // C_i scores
  __shared__ TreeShared tree;
  __shared__ float red[SEL_WARPS];
  __shared__ uint32_t scan[SEL_WARPS];
  __shared__ float part[SEL_THREADS];
  __shared__ __align__(16) unsigned long long list[SEL_LIST];
  __shared__ int kept[128];
  __shared__ int cnt_s, last_s;
  __shared__ uint32_t th_s;
  const int i = blockIdx.x, r = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
  const int lane = tid & 31, wid = tid >> 5;
  grid_dep_launch();
  const int C = a.N / SAS_BLOCK, G = a.Hq / a.Hkv;
  const size_t group = (size_t)b * a.Hkv + r, row = group * a.T + i;
  const TreeSeq s = tree_load(a, b, tree, (i == 0 && r == 0) ? &g_tree_select_err : nullptr);
  if (i >= s.nt) {
    grid_dep_wait();
    return;
  }
  const unsigned long long anc = tree.anc[i];
  const bool crossed = s.tail + tree_depth(anc) >= SAS_BLOCK;
  const int Ci = s.c0 + (crossed ? 1 : 0);
  const int kk = min(a.topk, Ci);
  float virt = 0.f;
  if (crossed) {
    // mean key of the tail's block as this path fills it: thread (part, column)
    // sums every P-th key, the tail's first, then the path's in their order
    constexpr int P = SEL_THREADS / D;
    const int c = tid % D, p = tid / D;
    const T* kc = static_cast<const T*>(a.kc);
    const T* kd = static_cast<const T*>(a.kd) + group * a.T * D;
    float sum = 0.f;
    if (s.tail > 0) {
      const size_t base = tree_block_row(a, b, r, s.c0, &g_tree_select_err);
#pragma unroll 8
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
  if (tid == 0) {
    cnt_s = 0;
    last_s = -1;
    th_s = 0xffffffffu;
  }
  grid_dep_wait();
  // Scores: four at a time into shared memory, with the thread's maximum; the
  // tail's block last.
  const float* sc = w.scores + row * tree_stride(C);
  float mx = -INFINITY;
#pragma unroll 4
  for (int m = 4 * tid; m < s.c0; m += 4 * SEL_THREADS) {
    float4 v = __ldcg(reinterpret_cast<const float4*>(sc + m));
    if (m + 1 >= s.c0) v.y = -INFINITY;
    if (m + 2 >= s.c0) v.z = -INFINITY;
    if (m + 3 >= s.c0) v.w = -INFINITY;
    *reinterpret_cast<float4*>(vals + m) = v;
    mx = fmaxf(mx, fmaxf(fmaxf(v.x, v.y), fmaxf(v.z, v.w)));
  }
  const uint32_t best = mx > -INFINITY ? score_key(mx) : 0u;  // a subset's keys bound the set's
  mx = warp_max(mx);
  if (lane == 0) red[wid] = mx;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < SEL_WARPS; ++k) mx = fmaxf(mx, red[k]);
  if (crossed) {
    mx = fmaxf(mx, virt);
    if (tid == 0) vals[s.c0] = virt;
  }
  // A lower bound of the kk-th best key: that of the threads' own best ones (a
  // subset), by its upper 16 bits.
  uint32_t bound = 0;
#pragma unroll 1
  for (int bit = 31; bit >= 16; --bit) {
    const uint32_t cand = bound | (1u << bit);
    if (__syncthreads_count(best >= cand) >= kk) bound = cand;
  }
  // The sum of the gate's softmax, and the list of the keys at or above the bound.
  float sum = 0.f;
  for (int m0 = 0; m0 < Ci; m0 += 4 * SEL_THREADS) {
    const int m = m0 + 4 * tid;
    float v[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
    if (m + 4 <= Ci) {
      const float4 x = *reinterpret_cast<const float4*>(vals + m);
      v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (m + k < Ci) v[k] = vals[m + k];
    }
    int n = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      sum += exp2f((v[k] - mx) * LOG2E);
      n += m + k < Ci && score_key(v[k]) >= bound;
    }
    if (n > 0) {
      int at = atomicAdd(&cnt_s, n);  // the list's order does not matter: keys are ranked below
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t key = score_key(v[k]);
        if (m + k < Ci && key >= bound && at < SEL_LIST)
          list[at++] = ((unsigned long long)key << 32) | (0xffffffffu - (uint32_t)(m + k));
      }
    }
  }
  const float lse = mx + logf(block_sum(sum, red));  // its barriers also close the list
  const int n = cnt_s;
  if (kk > 0 && n <= SEL_LIST) {
    // unique keys: a candidate's rank is the number of larger ones
    for (int e = tid; e < n; e += SEL_THREADS) {
      const unsigned long long key = list[e];
      const int rank = count_above(list, n, key);
      if (rank < kk) {
        const int m = key_block(key);
        kept[rank] = m;
        if (m < s.c0) atomicOr(&w.ubits[group * a.words + (m >> 5)], 1u << (m & 31));
        if (rank == kk - 1) {
          th_s = (uint32_t)(key >> 32);
          last_s = m;
        }
      }
    }
    __syncthreads();
    if (a.idx_out && tid < kk) {  // ascending: a block's place is the number of smaller ones
      const int m = kept[tid];
      int at = 0;
      for (int e = 0; e < kk; ++e) at += kept[e] < m;
      a.idx_out[row * a.topk + at] = m;
    }
  } else if (kk > 0) {
    const int per = ((Ci + SEL_THREADS - 1) / SEL_THREADS) | 1;  // odd: no bank conflicts
    const int lo = min(tid * per, Ci), hi = min(lo + per, Ci);
    uint32_t* keys = reinterpret_cast<uint32_t*>(vals);
    for (int m = tid; m < Ci; m += SEL_THREADS) keys[m] = score_key(vals[m]);
    __syncthreads();
    select_by_bits(keys, lo, hi, kk, scan, &th_s, &last_s);
    const uint32_t th = th_s;
    const int last = last_s;
    // places by counting the kept blocks of the earlier threads
    uint32_t mine = 0;
    for (int m = lo; m < hi; ++m) mine += keys[m] > th || (keys[m] == th && m <= last);
    uint32_t v = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += y;
    }
    if (lane == 31) scan[wid] = v;
    __syncthreads();
    int at = (int)(v - mine);
    for (int k = 0; k < wid; ++k) at += scan[k];
    for (int m = lo; m < hi; ++m)
      if ((keys[m] > th || (keys[m] == th && m <= last)) && at < kk) {
        if (a.idx_out) a.idx_out[row * a.topk + at] = m;
        if (m < s.c0) atomicOr(&w.ubits[group * a.words + (m >> 5)], 1u << (m & 31));
        ++at;
      }
  }
  if (a.idx_out)
    for (int p = kk + tid; p < a.topk; p += SEL_THREADS) a.idx_out[row * a.topk + p] = -1;
  if (tid == 0) {
    TreeRow t;
    t.lse = lse;
    t.th = th_s;
    t.last = last_s;
    t.tail_bias = 0.f;
    if (crossed) t.tail_bias = kk > 0 ? tree_bias(t, virt, s.c0, a.gated) : -INFINITY;
    w.rows[row] = t;
  }
}

// ------------------------------------------------------------------ host
template <typename T, typename S, int D>
static cudaError_t launch_typed(const TreeArgs& a, const TreeWs& w, cudaStream_t st) {
  const int C = a.N / SAS_BLOCK, T8 = (a.T + 7) & ~7;
  const size_t smem = (size_t)2 * T8 * (D + 16) * sizeof(float);
  cudaError_t e = ensure_smem(k_tree_scores<T, S, D>, smem);
  if (e != cudaSuccess) return e;
  const size_t ksm = (size_t)(tree_stride(C) + 4) * sizeof(float);
  e = ensure_smem(k_tree_select<T, S, D>, ksm);
  if (e != cudaSuccess) return e;
  // summaries of a CTA: whole passes, and one wave of the CTAs that an SM holds
  // (three by registers, fewer by shared memory)
  const long long groups = (long long)a.B * a.Hkv;
  const long long room = 148 * (smem > 75 * 1024 ? 2 : 3);
  long long per_group = room / groups;
  if (per_group < 1) per_group = 1;
  long long stretch = (C + per_group - 1) / per_group;
  stretch = (stretch + TS_BLOCKS - 1) / TS_BLOCKS * TS_BLOCKS;
  e = tree_launch(k_tree_scores<T, S, D>, dim3((unsigned)((C + stretch - 1) / stretch), a.Hkv, a.B),
                  TS_THREADS, smem, st, a, w, (int)stretch);
  if (e != cudaSuccess) return e;
  return tree_launch(k_tree_select<T, S, D>, dim3(a.T, a.Hkv, a.B), SEL_THREADS, ksm, st, a, w);
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
  t.scores = reinterpret_cast<float*>(take(topk > 0 ? rows * tree_stride((int)C) * 4 : 0));
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
