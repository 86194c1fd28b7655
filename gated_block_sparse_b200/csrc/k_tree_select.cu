// Block selection of drafted tokens: gate and Top-K of every token's own row
// of scores (k_tree_scores.cu).
//
//   log g = s - LSE(s) over the row's C_i blocks; the topk best are kept, ties
//   to the lower block. A token whose path has filled the tail's block also
//   scores that block, s_i,c0 = scale qbar_i . mean of its 64 keys (rounded to
//   the summaries' type).
//
// k_tree_select: one CTA per row. The row's scores go into shared memory once;
// the threads' maxima bound the topk-th score, the few scores above the bound
// are ranked by counting, and the gate's sum is taken on the way. What it leaves
// is one 16-byte record a row and one bit a block: the attention reads a row's
// score of a block and the record, and no list is searched or sorted. Latency
// bounds it (ncu, the kernel alone: 64K, 4 tokens 5.3 us; 512K, 64 tokens, 512
// rows of 8191 scores 15.7 us; its prologue overlaps the scores in a call).
#include <math.h>

#include "common.cuh"
#include "kernels.h"
#include "ptx.cuh"
#include "tree.cuh"

namespace sas {

__device__ uint32_t g_tree_select_err = 0;

namespace {
constexpr int SEL_LIST = 512;  // candidates ranked by counting
constexpr float LOG2E = 1.4426950408889634f;
}  // namespace

template <int THREADS>
__device__ __forceinline__ float block_sum(float v, float* red) {
  v = warp_sum(v);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float t = 0.f;
#pragma unroll
  for (int i = 0; i < THREADS / 32; ++i) t += red[i];
  __syncthreads();
  return t;
}

// The kk-th best of n keys and the last block that is kept at that key, for
// sets with more equal or near-equal keys than the list holds: the threshold
// bit by bit, then the keys equal to it in block order. Every thread owns the
// stretch [lo, hi). Returns through th and last (shared).
template <int THREADS>
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
    for (int i = 0; i < THREADS / 32; ++i) c += scan[i];
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
  for (int i = 0; i < THREADS / 32; ++i) {
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

template <typename T, typename S, int D, int THREADS>
__global__ void __launch_bounds__(THREADS) k_tree_select(TreeArgs a, TreeWs w) {
  constexpr int SEL_WARPS = THREADS / 32, SEL_BUCKETS = THREADS;  // a bucket a thread
  extern __shared__ __align__(16) float vals[];  // C_i scores
  __shared__ TreeShared tree;
  __shared__ float red[SEL_WARPS];
  __shared__ uint32_t scan[SEL_WARPS];
  __shared__ float part[THREADS * 8];  // at most 8 columns of a key a thread
  __shared__ int path[SAS_BLOCK];
  __shared__ float red2[SEL_WARPS];
  __shared__ int hist[SEL_BUCKETS];
  __shared__ __align__(16) unsigned long long list[SEL_LIST];
  __shared__ __align__(16) int kept[128];
  __shared__ int cnt_s, last_s, bucket_s, many_s;
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
  bool tail_in = true;  // the tail's page lies in the pool
  if (crossed) {
    const int place = s.tail > 0 ? tree_place(a, b, s.c0, &g_tree_select_err) : 0;
    tail_in = place >= 0;
    // Mean key of the tail's block as this path fills it: the tail's keys, then
    // the path's first ones. Thread (group, piece) sums every GRP-th key of one
    // 16-byte piece, all its loads in flight; the groups meet in shared memory.
    constexpr int VT = Vec16<T>::N, PIECES = D / VT, GRP = THREADS / PIECES;
    const int pc = (tid % PIECES) * VT, g = tid / PIECES;
    if (tid < TREE_MAX && (anc >> tid & 1ull)) {
      const int at = s.tail + __popcll(anc & ((1ull << tid) - 1ull));
      if (at < SAS_BLOCK) path[at] = tid;
    }
    __syncthreads();
    const T* kc = static_cast<const T*>(a.kc) +
                  (s.tail > 0 && tail_in ? tree_block_row(a, b, r, place) * D : 0);
    const T* kd = static_cast<const T*>(a.kd) + group * a.T * D;
    float sum[VT];
#pragma unroll
    for (int e = 0; e < VT; ++e) sum[e] = 0.f;
#pragma unroll
    for (int k = 0; k < SAS_BLOCK / GRP; ++k) {
      const int j = g + k * GRP;
      float y[VT];
      load_cg((j < s.tail ? kc + (size_t)j * D : kd + (size_t)path[j] * D) + pc, y);
#pragma unroll
      for (int e = 0; e < VT; ++e) sum[e] += y[e];
    }
#pragma unroll
    for (int e = 0; e < VT; ++e) part[g * D + pc + e] = sum[e];
    __syncthreads();
    float dot = 0.f;
    if (tid < D) {
      float qb = 0.f;
#pragma unroll 4
      for (int h = 0; h < G; ++h)
        qb += to_f(__ldcg(static_cast<const T*>(a.q) +
                          (((size_t)b * a.Hq + r * G + h) * a.T + i) * D + tid));
      float mean = 0.f;
#pragma unroll
      for (int k = 0; k < GRP; ++k) mean += part[k * D + tid];
      mean = to_f(from_f<S>(mean * (1.0f / SAS_BLOCK)));
      dot = qb * (1.0f / (float)G) * mean;
    }
    virt = block_sum<THREADS>(dot, red) * a.scale;
    if (!tail_in) virt = -INFINITY;
  }
  if (tid == 0) {
    cnt_s = 0;
    last_s = -1;
    th_s = 0xffffffffu;
  }
  hist[tid] = 0;
  if (tid < 128) kept[tid] = 0x7fffffff;
  grid_dep_wait();
  // Scores: four at a time into shared memory, with the thread's maximum; the
  // tail's block last.
  const float* sc = w.scores + row * tree_stride(C);
  float mx = -INFINITY;
#pragma unroll 4
  for (int m = 4 * tid; m < s.c0; m += 4 * THREADS) {
    float4 v = __ldcg(reinterpret_cast<const float4*>(sc + m));
    if (m + 1 >= s.c0) v.y = -INFINITY;
    if (m + 2 >= s.c0) v.z = -INFINITY;
    if (m + 3 >= s.c0) v.w = -INFINITY;
    *reinterpret_cast<float4*>(vals + m) = v;
    mx = fmaxf(mx, fmaxf(fmaxf(v.x, v.y), fmaxf(v.z, v.w)));
  }
  // A lower bound of the kk-th best score: that of the threads' own maxima (a
  // subset), by buckets of equal width between the least and the largest of
  // them. bucket() never decreases, so every score of the kk best lies in the
  // bound's bucket or above; a score that is not finite does too.
  const float best = mx;
  float mn = mx > -INFINITY ? mx : INFINITY;
  mx = warp_max(mx);
  mn = -warp_max(-mn);
  if (lane == 0) {
    red[wid] = mx;
    red2[wid] = mn;
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < SEL_WARPS; ++k) {
    mx = fmaxf(mx, red[k]);
    mn = fminf(mn, red2[k]);
  }
  if (crossed) {
    if (tid == 0) vals[s.c0] = virt;
  }
  // A few scores far above the rest leave the rest in few buckets: a bound whose
  // bucket holds many of the maxima is sought again inside that bucket (any
  // map that never decreases will do).
  float width = (mx - mn) * (1.0f / SEL_BUCKETS), inv_w = 0.f;
  auto bucket = [&](float v) { return fminf((v - mn) * inv_w, (float)(SEL_BUCKETS - 1)); };
  for (int pass = 0;; ++pass) {
    inv_w = width > 1e-30f && width < INFINITY ? 1.0f / width : 0.f;
    if (best > -INFINITY) atomicAdd(&hist[(int)fmaxf(bucket(best), 0.f)], 1);
    __syncthreads();
    if (wid == 0) {  // lane l: buckets 8 l .. 8 l + 7, counted from the top
      constexpr int PER = SEL_BUCKETS / 32;
      int c[PER], own = 0;
#pragma unroll
      for (int k = 0; k < PER; ++k) own += c[k] = hist[lane * PER + k];
      int above = own;  // of this lane and the higher ones
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_down_sync(0xffffffffu, above, o);
        if (lane + o < 32) above += y;
      }
      if (lane == 0) {  // fewer maxima than kk: every score is a candidate
        bucket_s = 0;
        many_s = 0;
      }
      __syncwarp();
      int run = above - own;
      if (run < kk && above >= kk) {
#pragma unroll
        for (int k = PER - 1; k >= 0; --k) {
          const int before = run;
          run += c[k];
          if (before < kk && run >= kk) {
            bucket_s = lane * PER + k;
            many_s = c[k] > 32;
          }
        }
      }
    }
    __syncthreads();
    if (!many_s || pass == 2 || inv_w == 0.f) break;
    mn += (float)bucket_s * width;
    width *= 1.0f / SEL_BUCKETS;
    hist[tid] = 0;
    __syncthreads();
  }
  if (crossed) mx = fmaxf(mx, virt);
  const float bound = bucket_s > 0 ? (float)bucket_s : -INFINITY;
  // The sum of the gate's softmax, and the list of the keys at or above the bound.
  float sum = 0.f;
  for (int m0 = 0; m0 < Ci; m0 += 4 * THREADS) {
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
      n += m + k < Ci && !(bucket(v[k]) < bound);
    }
    if (n > 0) {
      int at = atomicAdd(&cnt_s, n);  // the list's order does not matter: keys are ranked below
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (m + k < Ci && !(bucket(v[k]) < bound) && at < SEL_LIST)
          list[at++] = cand_key(v[k] + 0.f, m + k);
      }
    }
  }
  const float lse = mx + logf(block_sum<THREADS>(sum, red));  // its barriers also close the list
  const int n = cnt_s;
  // A kept block is one of the attention's units unless its page lies outside the
  // pool; its score is then -inf (only such a one is looked up again).
  auto is_unit = [&](int m, uint32_t key) {
    return m < s.c0 && (key != score_key(-INFINITY) || tree_place(a, b, m, nullptr) >= 0);
  };
  if (kk > 0 && n <= SEL_LIST) {
    // unique keys: a candidate's rank is the number of larger ones
    for (int e = tid; e < n; e += THREADS) {
      const unsigned long long key = list[e];
      const int rank = count_above(list, n, key);
      if (rank < kk) {
        const int m = key_block(key);
        kept[rank] = m;
        if (is_unit(m, (uint32_t)(key >> 32)))
          atomicOr(&w.ubits[group * a.words + (m >> 5)], 1u << (m & 31));
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
#pragma unroll 4
      for (int e = 0; e < kk; e += 4) {  // behind the last: no block's number
        const int4 o = *reinterpret_cast<const int4*>(kept + e);
        at += (o.x < m) + (o.y < m) + (o.z < m) + (o.w < m);
      }
      a.idx_out[row * a.topk + at] = m;
    }
  } else if (kk > 0) {
    const int per = ((Ci + THREADS - 1) / THREADS) | 1;  // odd: no bank conflicts
    const int lo = min(tid * per, Ci), hi = min(lo + per, Ci);
    uint32_t* keys = reinterpret_cast<uint32_t*>(vals);
    for (int m = tid; m < Ci; m += THREADS) keys[m] = score_key(vals[m]);
    __syncthreads();
    select_by_bits<THREADS>(keys, lo, hi, kk, scan, &th_s, &last_s);
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
        if (is_unit(m, keys[m])) atomicOr(&w.ubits[group * a.words + (m >> 5)], 1u << (m & 31));
        ++at;
      }
  }
  if (a.idx_out)
    for (int p = kk + tid; p < a.topk; p += THREADS) a.idx_out[row * a.topk + p] = -1;
  if (tid == 0) {
    TreeRow t;
    t.lse = lse;
    t.th = th_s;
    t.last = last_s;
    t.tail_bias = 0.f;
    if (crossed) t.tail_bias = kk > 0 && tail_in ? tree_bias(t, virt, s.c0, a.gated) : -INFINITY;
    w.rows[row] = t;
  }
}

// ------------------------------------------------------------------ host
template <typename T, typename S, int D, int THREADS>
static cudaError_t launch_threads(const TreeArgs& a, const TreeWs& w, cudaStream_t st) {
  const size_t smem = (size_t)(tree_stride(a.N / SAS_BLOCK) + 4) * sizeof(float);
  cudaError_t e = ensure_smem(k_tree_select<T, S, D, THREADS>, smem);
  if (e != cudaSuccess) return e;
  return tree_launch(k_tree_select<T, S, D, THREADS>, dim3(a.T, a.Hkv, a.B), THREADS, smem, st, a, w);
}

// Threads of a row: 128 up to 256 blocks, where the rows that fit an SM count for
// more than each row's time (four sequences of 120 tokens, 32 drafted: 25 us a
// call, 30 with 256); 256 beyond.
template <typename T, typename S, int D>
static cudaError_t launch_typed(const TreeArgs& a, const TreeWs& w, cudaStream_t st) {
  return a.N / SAS_BLOCK <= 256 ? launch_threads<T, S, D, 128>(a, w, st)
                                 : launch_threads<T, S, D, 256>(a, w, st);
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
    cudaError_t e = launch_tree_scores(a, w, bf16, sum_bf16, d, st);
    if (e != cudaSuccess) return e;
    e = launch_tree_select(a, w, bf16, sum_bf16, d, st);
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
