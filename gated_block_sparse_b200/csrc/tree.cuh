// A tree of drafted tokens beside a cache: what its kernels share.
//
// Sequence b has lens[b] = n cached tokens and up to T <= 64 drafted ones with
// a parent each (-1: the last cached token). Token i sits at position
// n + depth_i and sees the cache and its ancestors, itself included, exactly
// as if the path from the root to it had been appended to the cache:
//   C_i = (n + depth_i) / 64 history blocks, c0 = n / 64 of them whole in the
//   cache. A path that fills the block of the cache's tail (its
//   n - 64 c0 < 64 last tokens) makes it history block c0 of that token, with
//   a summary of its own: the mean of the tail's keys and of the path's keys
//   up to it. A path has at most 64 tokens, so it fills at most that one.
#pragma once

#include <math.h>

#include "common.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace sas {

constexpr int TREE_MAX = 64;  // drafted tokens of a sequence: one 64-bit mask a token

// The tree of one sequence, in shared memory.
struct TreeShared {
  unsigned long long anc[TREE_MAX];  // ancestors of token i, i included
  int up[TREE_MAX];
  uint32_t early[2];  // tokens whose key lies inside the tail's block
};

struct TreeSeq {
  int n;      // cached tokens
  int nt;     // drafted tokens
  int c0;     // whole blocks of the cache
  int tail;   // cached tokens past them
};

__device__ __forceinline__ int tree_depth(unsigned long long anc) { return __popcll(anc) - 1; }

// Cached and drafted tokens of sequence b: none drafted (the sequence is left
// out) when a length lies outside the buffers.
__device__ __forceinline__ bool tree_lengths(const TreeArgs& a, int b, int& n, int& nt) {
  n = __ldcg(a.lens + b);
  nt = a.ntok ? __ldcg(a.ntok + b) : a.T;
  if (n >= 0 && n <= a.N && nt >= 0 && nt <= a.T) return true;
  n = nt = 0;
  return false;
}

// Lengths and ancestor masks of sequence b, by pointer jumping: after round e
// a token's mask holds its 2^(e+1) nearest ancestors. The three loads go out
// together. A sequence with a length outside the buffers has no tokens, a
// parent that is not below its child is read as -1; both are reported when err
// is given. All threads of the block (at least TREE_MAX) call it; it ends with
// a barrier. No parents: a chain.
__device__ __forceinline__ TreeSeq tree_load(const TreeArgs& a, int b, TreeShared& t,
                                             uint32_t* err) {
  const int i = threadIdx.x;
  TreeSeq s;
  const bool fit = tree_lengths(a, b, s.n, s.nt);
  int p = i - 1;
  if (a.parents && i < a.T) p = __ldcg(a.parents + (size_t)b * a.T + i);
  s.c0 = s.n / SAS_BLOCK;
  s.tail = s.n - s.c0 * SAS_BLOCK;
  if (err && i == 0 && !fit) atomicOr(err, kErrBadIndex);
  unsigned long long m = 0;
  if (i < TREE_MAX) {
    if (i >= s.nt) p = -1;
    if (p < -1 || p >= i) {
      if (err) atomicOr(err, kErrBadIndex);
      p = -1;
    }
    m = a.parents ? 1ull << i : ~0ull >> (63 - i);
    if (!a.parents) p = -1;
    t.anc[i] = m;
    t.up[i] = p;
  }
  while (__syncthreads_or(p >= 0 && i < TREE_MAX)) {  // at most 6 rounds for 64 tokens
    if (i < TREE_MAX && p >= 0) {
      m |= t.anc[p];
      p = t.up[p];
    }
    __syncthreads();
    if (i < TREE_MAX) {
      t.anc[i] = m;
      t.up[i] = p;
    }
  }
  if (i < TREE_MAX) {
    const uint32_t e = __ballot_sync(0xffffffffu, i < s.nt && s.tail + tree_depth(m) < SAS_BLOCK);
    if ((i & 31) == 0) t.early[i >> 5] = e;
  }
  __syncthreads();
  return s;
}

__device__ __forceinline__ unsigned long long tree_early(const TreeShared& t) {
  return ((unsigned long long)t.early[1] << 32) | t.early[0];
}

// Where logical block m of sequence b lies: its page, or m itself in a
// contiguous cache. -1 for an id outside the pool, which is reported: the block
// is left out. The scores give it -inf and the selection keeps it out of the
// units, so the attention meets it in the tail alone.
__device__ __forceinline__ bool tree_page_ok(const TreeArgs& a, int page) {
  return !a.table || (page >= 0 && page < a.npages);
}
__device__ __forceinline__ int tree_place(const TreeArgs& a, int b, int m, uint32_t* err) {
  if (!a.table) return m;
  const int p = __ldcg(a.table + (size_t)b * (a.N / SAS_BLOCK) + m);
  if (tree_page_ok(a, p)) return p;
  if (err) atomicOr(err, kErrBadIndex);
  return -1;
}

// First row of the block at `place` (>= 0) of head r, in rows of the cache.
__device__ __forceinline__ size_t tree_block_row(const TreeArgs& a, int b, int r, int place) {
  if (a.table) return ((size_t)place * a.Hkv + r) * SAS_BLOCK;
  return ((size_t)b * a.Hkv + r) * a.N + (size_t)place * SAS_BLOCK;
}

// Order bits of a score of either zero (exact ties are equal).
__device__ __forceinline__ uint32_t score_key(float s) { return order_bits(s + 0.f); }

// What selection leaves of a row (sequence, kv group, drafted token): with
// the scores themselves it says which blocks the row keeps and their gates,
// so no list has to be searched and nothing is written per block.
struct __align__(16) TreeRow {
  float lse;        // log sum exp of the row's scores
  uint32_t th;      // key of the lowest kept score
  int last;         // the kept blocks of that score are those up to this one
  float tail_bias;  // log g of block c0 (-inf: not kept; 0: not yet filled)
};

// Bias of history block m: log g, or -inf when the row does not keep it.
__device__ __forceinline__ float tree_bias(const TreeRow& t, float score, int m, int gated) {
  const uint32_t key = score_key(score);
  const bool keep = key > t.th || (key == t.th && m <= t.last);
  return keep ? (gated ? score - t.lse : 0.f) : -INFINITY;
}

// Scores of a row: C of them, rows 16 bytes aligned.
__host__ __device__ __forceinline__ int tree_stride(int C) { return (C + 3) & ~3; }

// Workspace of one call.
struct TreeWs {
  float* scores;    // [row][tree_stride(N / 64)]
  TreeRow* rows;    // [row]
  uint32_t* ubits;  // [group][words]: blocks that some token selected
  float* part;      // [group][split][d / 4][G T][4]: outputs before the division
  float2* ml;       // [group][split][G T]: running maximum (log2 units) and sum
};

// The call's kernels overlap by programmatic dependent launch: each one's
// first part (lengths, tree, queries, tiles of the caller's tensors) runs while
// the one before it drains; grid_dep_wait() stands before the first access to
// the workspace. The first kernel waits before anything else and only then
// lets the next one start, so what the caller's earlier work wrote is complete
// for all of them. A kernel that starts while another runs may find old lines in
// its SM's L1, so everything that may have changed since the last call (the
// caller's tensors and the workspace) is read through L2: __ldcg, cp.async.cg
// and TMA.
template <typename... Params, typename... Args>
inline cudaError_t tree_launch(void (*kern)(Params...), dim3 grid, int threads, size_t smem,
                               cudaStream_t st, Args... args) {
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t c = {};
  c.gridDim = grid;
  c.blockDim = dim3(threads);
  c.dynamicSmemBytes = smem;
  c.stream = st;
  c.attrs = at;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, kern, static_cast<Params>(args)...);
}

// A 16-byte vector through L2, as fp32 values.
template <typename T>
__device__ __forceinline__ void load_cg(const T* p, float* out) {
  const uint4 v = __ldcg(reinterpret_cast<const uint4*>(p));
  Vec16<T>::load(reinterpret_cast<const T*>(&v), out);
}

// 16 bytes from global to shared memory without a register, zeros when !full.
__device__ __forceinline__ void cp_async16(void* dst, const void* src, bool full) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src),
               "r"(full ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
// Until at most N of this thread's latest groups are in flight.
template <int N>
__device__ __forceinline__ void cp_async_wait_group() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// Column c of a row's partial output, from the row's first four columns: the
// rows of a warp write 16-byte pieces side by side.
__device__ __forceinline__ size_t tree_part_at(int c, size_t R) {
  return (size_t)(c >> 2) * R * 4 + (c & 3);
}

cudaError_t launch_tree_scores(const TreeArgs& a, const TreeWs& w, int bf16, int sum_bf16, int d,
                               cudaStream_t st);
cudaError_t launch_tree_select(const TreeArgs& a, const TreeWs& w, int bf16, int sum_bf16, int d,
                               cudaStream_t st);
cudaError_t launch_tree_attn_simt(const TreeArgs& a, const TreeWs& w, int d, cudaStream_t st);
cudaError_t launch_tree_attn_tc(const TreeArgs& a, const TreeWs& w, int d, cudaStream_t st);
cudaError_t launch_tree_join(const TreeArgs& a, const TreeWs& w, int bf16, int d,
                             cudaStream_t st);

// The row of token i; without selection (topk 0) it keeps no block, and none
// of the tail's once its path has filled that block.
__device__ __forceinline__ TreeRow tree_row(const TreeArgs& a, const TreeWs& w, const TreeSeq& s,
                                            size_t group, int i, unsigned long long anc) {
  if (a.topk > 0) {
    const float4 x = __ldcg(reinterpret_cast<const float4*>(w.rows + group * a.T + i));
    TreeRow t;
    t.lse = x.x;
    t.th = __float_as_uint(x.y);
    t.last = __float_as_int(x.z);
    t.tail_bias = x.w;
    return t;
  }
  TreeRow t;
  t.lse = 0.f;
  t.th = 0xffffffffu;
  t.last = -1;
  t.tail_bias = s.tail + tree_depth(anc) >= SAS_BLOCK ? -INFINITY : 0.f;
  return t;
}

// Offset of 16-byte piece p of row `row` in a K-major bf16 tile of `nrows`
// rows under the 128-byte swizzle: 64-column chunks one after the other, rows
// of 128 bytes, the piece's index within the row xor (row mod 8).
__device__ __forceinline__ uint32_t sw_off(int row, int p, int nrows) {
  return (uint32_t)((p >> 3) * nrows * 128 + row * 128 + (((p & 7) ^ (row & 7)) << 4));
}

// The units of one split of a (sequence, kv group): the blocks that some
// token selected, ascending, then the tail (unit nu) and the drafted tokens
// (unit nu + 1). A split takes units [u0, u1) of the nu + 2. `bits` gets the
// group's block bitmap; *start the block of unit u0 (when u0 < nu). All
// THREADS threads of the block call it; it ends with a barrier.
template <int THREADS>
__device__ __forceinline__ int tree_units(const TreeArgs& a, const uint32_t* __restrict__ ubits,
                                          uint32_t* bits, int* warp_s, int* start, int split,
                                          int& u0, int& u1) {
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  int nu = 0;
  if (a.topk > 0) {
    const int per = (a.words + THREADS - 1) / THREADS;
    const int lo = min(tid * per, a.words), hi = min(lo + per, a.words);
    int c = 0;
    for (int i = lo; i < hi; ++i) {
      bits[i] = __ldcg(ubits + i);
      c += __popc(bits[i]);
    }
    int v = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += y;
    }
    if (lane == 31) warp_s[wid] = v;
    __syncthreads();
    int before = v - c;
#pragma unroll
    for (int i = 0; i < THREADS / 32; ++i) {
      before += i < wid ? warp_s[i] : 0;
      nu += warp_s[i];
    }
    u0 = (nu + 2) * split / a.ns;
    if (before <= u0 && u0 < before + c) {  // unit u0 is among this thread's blocks
      int left = u0 - before;
      for (int i = lo; i < hi; ++i) {
        uint32_t word = bits[i];
        const int pc = __popc(word);
        if (left < pc) {
          for (; left > 0; --left) word &= word - 1;
          *start = i * 32 + __ffs(word) - 1;
          break;
        }
        left -= pc;
      }
    }
  }
  __syncthreads();
  u0 = (nu + 2) * split / a.ns;
  u1 = (nu + 2) * (split + 1) / a.ns;
  return nu;
}

// Smallest selected block >= from; -1 past the end.
__device__ __forceinline__ int tree_next(const uint32_t* bits, int words, int from) {
  for (int i = from >> 5; i < words; ++i) {
    const uint32_t word = bits[i] & (i == (from >> 5) ? ~0u << (from & 31) : ~0u);
    if (word) return i * 32 + __ffs(word) - 1;
  }
  return -1;
}

}  // namespace sas
