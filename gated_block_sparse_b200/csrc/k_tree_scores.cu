// Selector scores of drafted tokens over the cached block summaries, on the
// 5th-generation tensor cores:
//   s_im = scale qbar_i . ksum_m for every token i and whole block m < c0,
// qbar_i the mean of the group's heads at token i.
//
// The order of the blocks needs fp32, so the factors are split into bf16
// parts, x = h + m + l with |m| <= 2^-8 |x| and |l| <= 2^-16 |x| (each part the
// nearest bf16 of what the earlier ones leave; the rest is below 2^-24 |x|).
// fp32 summaries take the six products h h, h m, m h, m m, h l, l h, bf16
// summaries (one part) the three with qbar's parts; the MMAs accumulate in
// fp32. What is dropped is below 2^-23 of a product, as an fp32 product rounds.
// A score that comes out inf or NaN is computed again by fp32 FMAs.
//
// One CTA per (stretch of summaries, kv group, sequence), in tiles of 128
// summaries: M = 128 blocks, K = d, and the three parts of qbar side by side
// along N (3 x 16 to 3 x 64 columns, added when they are read), since an MMA
// of few columns is bound by reading its A tile. h is multiplied by all three
// parts, m by the first two, l by the first. All threads
// bring a tile's rows into registers a tile ahead (rows of a paged cache lie
// anywhere), split them and store the parts as swizzled K-major tiles; one
// thread issues the MMAs; four warps read a token's scores of 32 consecutive
// blocks from TMEM and write them, 128 bytes a store. Every summary is read
// once. 512K, T = 64: 34 MB read, 17 MB of scores written in 19.5 us (ncu, the
// kernel alone, 2 us of it its start), where the reads take 5, the writes 3 and
// the MMAs 3: a CTA's loads, splits, MMAs and stores follow one another. 8 x
// 128K, T = 16, bf16 summaries, two CTAs an SM: 29 MB in 15 us. 64K, T = 4: 6 us,
// a chain of latencies. fp32 summaries of d = 128 in two steps of 64 columns, so
// that two CTAs share an SM: 512K, T = 64 65.0 us a call against 65.3 in one
// step, 8 x 128K, T = 16 81.2 against 82.5, but 512K, T = 4 32.7 against 29.5.
#include <math.h>

#include "common.cuh"
#include "kernels.h"
#include "ptx.cuh"
#include "tc.cuh"
#include "tree.cuh"

namespace sas {

__device__ uint32_t g_tree_scores_err = 0;

namespace {

constexpr int SC_THREADS = 256;
constexpr int SC_ROWS = 128;  // summaries of a tile

// 8 values as NP bf16 parts of 16 bytes, the nearest bf16 first.
template <int NP>
__device__ __forceinline__ void split_bf16(float (&x)[8], uint4 (&out)[NP]) {
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
      if (p + 1 < NP) {
        x[2 * i] -= __uint_as_float(w[i] << 16);
        x[2 * i + 1] -= __uint_as_float(w[i] & 0xffff0000u);
      }
    }
    out[p] = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// 8 consecutive summary elements as loaded.
template <typename S> struct Raw8;
template <> struct Raw8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = __ldcg(reinterpret_cast<const float4*>(p));
    b = __ldcg(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void nan() { a.x = a.y = a.z = a.w = b.x = b.y = b.z = b.w = NAN; }
  __device__ __forceinline__ void parts(uint4 (&out)[3]) const {
    float x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    split_bf16<3>(x, out);
  }
};
template <> struct Raw8<__nv_bfloat16> {
  uint4 a;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    a = __ldcg(reinterpret_cast<const uint4*>(p));
  }
  __device__ __forceinline__ void nan() { a.x = a.y = a.z = a.w = 0x7fff7fffu; }
  __device__ __forceinline__ void parts(uint4 (&out)[1]) const { out[0] = a; }
};

__host__ __device__ __forceinline__ int scores_cols(int T) { return (T + 15) & ~15; }

// The score of one (summary, token) by fp32 FMAs, for one that the split products
// made inf or NaN: a part of an infinity is NaN (inf - inf), as is its product
// with a part that is 0, and a finite value past the largest bf16 rounds to an
// infinite part. The mean query is the sum of its three parts in shared memory
// (its first part alone where that is not finite).
template <typename S, int D>
__device__ __forceinline__ float score_by_fma(const S* sum, const unsigned char* sb, int row, int NT) {
  float dot = 0.f;
#pragma unroll 2
  for (int p = 0; p < D / 8; ++p) {
    float q[8], m[8], l[8], x[8];
    auto part = [&](int k, float (&y)[8]) {
      Vec16<__nv_bfloat16>::load(
          reinterpret_cast<const __nv_bfloat16*>(sb + sw_off(k * NT + row, p, 3 * NT)), y);
    };
    part(0, q);
    part(1, m);
    part(2, l);
#pragma unroll
    for (int i = 0; i < 8 / Vec16<S>::N; ++i)
      load_cg(sum + p * 8 + i * Vec16<S>::N, x + i * Vec16<S>::N);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      dot = fmaf(fabsf(q[i]) < INFINITY ? q[i] + (m[i] + l[i]) : q[i], x[i], dot);
  }
  return dot;
}

// The scores of block m and the tokens t0 + i, i in `again`, which the MMAs left
// inf or NaN: by FMAs, or -inf where the block's page lies outside the pool.
template <typename S, int D>
__device__ __noinline__ void scores_again(const TreeArgs& a, float* scores, int b, int r, int m,
                                          int t0, uint32_t again, const unsigned char* sb) {
  const int C = a.N / SAS_BLOCK, place = tree_place(a, b, m, &g_tree_scores_err);
  const size_t group = (size_t)b * a.Hkv + r;
  const size_t row = a.table ? (size_t)max(place, 0) * a.Hkv + r : group * C + m;
  float* out = scores + (group * a.T + t0) * tree_stride(C) + m;
  for (; again; again &= again - 1) {
    const int t = __ffs(again) - 1;
    const float dot = score_by_fma<S, D>(static_cast<const S*>(a.ksum) + row * D, sb, t0 + t,
                                         scores_cols(a.T));
    out[(size_t)t * tree_stride(C)] = place < 0 ? -INFINITY : dot * a.scale + 0.f;
  }
}

// CTAs an SM: the 64 fp32 values that a thread loads ahead with D = 128 need
// more than the 128 registers of two (a spilled one would be waited for).
template <typename S, int D>
constexpr int scores_ctas() { return sizeof(S) * D > 256 ? 1 : 2; }

}  // namespace

// The arguments are grid constants, here and in the attention: a function that
// takes them by reference would have every thread copy them to its stack.
template <typename T, typename S, int D>
__global__ void __launch_bounds__(SC_THREADS, scores_ctas<S, D>())
    k_tree_scores(const __grid_constant__ TreeArgs a, const __grid_constant__ TreeWs w,
                  int stretch) {
  constexpr int NP = sizeof(S) == 4 ? 3 : 1;     // parts of a summary
  constexpr int PC = D / 8;                      // 16-byte pieces of a bf16 row
  constexpr int PER = SC_ROWS * PC / SC_THREADS; // pieces of a tile of a thread
  constexpr int BI = TREE_MAX * PC / SC_THREADS;
  constexpr uint32_t A_PART = SC_ROWS * D * 2;
  constexpr int VT = Vec16<T>::N;
  extern __shared__ __align__(1024) unsigned char sm[];  // parts of A, then parts of B
  __shared__ uint64_t bar;
  __shared__ uint32_t tmem_slot;
  uint32_t* err = &g_tree_scores_err;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int r = blockIdx.y, b = blockIdx.z, G = a.Hq / a.Hkv, C = a.N / SAS_BLOCK;
  const int NT = scores_cols(a.T);
  unsigned char* sb = sm + NP * A_PART;
  const size_t group = (size_t)b * a.Hkv + r;
  const int m_lo = blockIdx.x * stretch;
  grid_dep_wait();
  for (int i = m_lo / 32 + tid; i < min((m_lo + stretch) / 32, a.words); i += SC_THREADS)
    w.ubits[group * a.words + i] = 0u;
  int n, nt;
  tree_lengths(a, b, n, nt);
  const int c0 = n / SAS_BLOCK;
  const int m_hi = min(m_lo + stretch, c0);
  if (m_lo >= m_hi || nt == 0) return;
  if ((smem_u32(sm) & 1023u) != 0) {  // swizzled tiles need 1024-byte alignment
    if (tid == 0) atomicOr(err, kErrBadIndex);
    return;
  }
  if (tid == 0) {
    mbar_init(&bar, 1);
    fence_mbar_init();
  }
  if (warp == 0) {
    tc::tmem_alloc(&tmem_slot, 256);
    // Only now may the next kernels start: the attention's CTAs hold their TMEM
    // while they wait for this grid, so an allocation here after theirs would
    // wait for them and they for it.
    if (lane == 0) grid_dep_launch();
  }
  // Rows of a tile, a tile ahead; where they lie (row or page), one more. A row
  // past the end reads the last one.
  Raw8<S> x[PER];
  int at[PER];
  // A page outside the pool gives NaN scores, which the read-out turns to -inf.
  auto place_of = [&](int m) { return a.table ? __ldcg(a.table + (size_t)b * C + m) : m; };
  auto sum_row = [&](int place) -> size_t {
    return a.table ? (size_t)place * a.Hkv + r : group * C + place;
  };
  auto place_tile = [&](int m0) {
#pragma unroll
    for (int i = 0; i < PER; ++i)
      at[i] = place_of(min(m0 + tid / PC + i * (SC_THREADS / PC), m_hi - 1));
  };
  auto load_tile = [&] {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      if (tree_page_ok(a, at[i]))
        x[i].load(static_cast<const S*>(a.ksum) + sum_row(at[i]) * D + (tid % PC) * 8);
      else
        x[i].nan();
    }
  };
  place_tile(m_lo);
  // B: qbar in three parts side by side, zeros behind the last token; its loads
  // first, then those of the first tile of A, then the parts
  float s[BI][8];
#pragma unroll
  for (int e = 0; e < BI; ++e) {
    const int row = (tid + e * SC_THREADS) / PC, p = tid % PC;
#pragma unroll
    for (int i = 0; i < 8; ++i) s[e][i] = 0.f;
    if (row < nt) {
      const T* q = static_cast<const T*>(a.q) + (((size_t)b * a.Hq + r * G) * a.T + row) * D + p * 8;
#pragma unroll 4
      for (int g = 0; g < G; ++g) {
#pragma unroll
        for (int h = 0; h < 8 / VT; ++h) {
          float y[VT];
          load_cg(q + (size_t)g * a.T * D + h * VT, y);
#pragma unroll
          for (int i = 0; i < VT; ++i) s[e][h * VT + i] += y[i];
        }
      }
    }
  }
  load_tile();
  place_tile(m_lo + SC_ROWS);
  const float inv_g = 1.0f / (float)G;
#pragma unroll
  for (int e = 0; e < BI; ++e) {
    const int row = (tid + e * SC_THREADS) / PC, p = tid % PC;
    if (row >= NT) break;
    uint4 part[3];
#pragma unroll
    for (int i = 0; i < 8; ++i) s[e][i] *= inv_g;
    split_bf16<3>(s[e], part);
#pragma unroll
    for (int k = 0; k < 3; ++k)
      *reinterpret_cast<uint4*>(sb + sw_off(k * NT + row, p, 3 * NT)) = part[k];
  }
  const int CS = tree_stride(C);
  float* out = w.scores + group * a.T * CS;
  const uint64_t a_desc = tc::sw128_desc(smem_u32(sm), 16, 1024);
  const uint64_t b_desc = tc::sw128_desc(smem_u32(sb), 16, 1024);
  uint32_t tmem = 0;
  uint32_t phase = 0;
  for (int m0 = m_lo; m0 < m_hi; m0 += SC_ROWS) {
    // the previous tile's MMAs are done (waited on below), so A is free
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      uint4 part[NP];
      x[i].parts(part);
#pragma unroll
      for (int k = 0; k < NP; ++k)
        *reinterpret_cast<uint4*>(sm + k * A_PART +
                                  sw_off(tid / PC + i * (SC_THREADS / PC), tid % PC, SC_ROWS)) =
            part[k];
    }
    fence_proxy_async_smem();  // A and B are read by the tensor cores
    tc::fence_before_sync();   // and the previous tile's scores have been read
    __syncthreads();
    tc::fence_after_sync();
    tmem = tmem_slot;
    if (tid == 0) {
#pragma unroll 1
      for (int k = 0; k < NP; ++k) {
        const uint32_t idesc = tc::idesc_bf16(128, (3 - k) * NT, 0, 0);
        // a step along K moves a descriptor's address field (16-byte units) alone
        const uint64_t ad = a_desc + ((k * A_PART) >> 4);
        const uint32_t chunk = (uint32_t)(3 * NT) * 128;  // 64 columns of B
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {  // K in steps of 16 (32 bytes)
          const uint32_t c = ks >> 2, off = (ks & 3) * 32;
          tc::mma_bf16(tmem, ad + ((c * (SC_ROWS * 128) + off) >> 4),
                       b_desc + ((c * chunk + off) >> 4), idesc, (k > 0 || ks > 0) ? 1u : 0u);
        }
      }
      tc::commit(&bar);
    }
    // the next tile's rows, and the places of the one after
    if (m0 + SC_ROWS < m_hi) load_tile();
    place_tile(m0 + 2 * SC_ROWS);
    mbar_wait_data(&bar, phase, err);
    phase ^= 1;
    tc::fence_after_sync();
    // warp w: blocks 32 (w mod 4) .., tokens 32 (w / 4) ..
    const int m = m0 + 32 * (warp & 3) + lane, t0 = 32 * (warp >> 2);
    if (t0 < nt) {
      const uint32_t tm = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + t0;
      float v[32], y[32];
      tc::tmem_ld32(tm + 2 * NT, v);
      tc::tmem_ld32(tm + NT, y);
      tc::tmem_wait_ld();
#pragma unroll
      for (int t = 0; t < 32; ++t) v[t] += y[t];  // small parts first
      tc::tmem_ld32(tm, y);
      tc::tmem_wait_ld();
      float* o = out + (size_t)t0 * CS + m;
      uint32_t again = 0;  // tokens whose score is not finite
      if (m < m_hi) {
#pragma unroll
        for (int t = 0; t < 32; ++t) {
          if (t0 + t >= nt) break;
          const float s = (v[t] + y[t]) * a.scale + 0.f;
          if (!(fabsf(s) < INFINITY)) again |= 1u << t;
          *o = s;
          o += CS;
        }
      }
      if (again) scores_again<S, D>(a, w.scores, b, r, m, t0, again, sb);
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 0) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, 256);
  }
}

// ------------------------------------------------------------------ host
template <typename T, typename S, int D>
static cudaError_t launch_typed(const TreeArgs& a, const TreeWs& w, cudaStream_t st) {
  const int C = a.N / SAS_BLOCK;
  const size_t smem = (size_t)(sizeof(S) == 4 ? 3 : 1) * SC_ROWS * D * 2 +
                      (size_t)3 * scores_cols(a.T) * D * 2;
  cudaError_t e = ensure_smem(k_tree_scores<T, S, D>, smem);
  if (e != cudaSuccess) return e;
  // summaries of a CTA: whole tiles, and one wave of the CTAs that an SM holds
  const long long groups = (long long)a.B * a.Hkv;
  const long long room = 148 * scores_ctas<S, D>();
  long long per_group = room / groups;
  if (per_group < 1) per_group = 1;
  long long stretch = (C + per_group - 1) / per_group;
  stretch = (stretch + SC_ROWS - 1) / SC_ROWS * SC_ROWS;
  return tree_launch(k_tree_scores<T, S, D>,
                     dim3((unsigned)((C + stretch - 1) / stretch), a.Hkv, a.B), SC_THREADS, smem,
                     st, a, w, (int)stretch);
}

cudaError_t launch_tree_scores(const TreeArgs& a, const TreeWs& w, int bf16, int sum_bf16, int d,
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

uint32_t* tree_scores_error_word() {
  void* p = nullptr;
  cudaGetSymbolAddress(&p, g_tree_scores_err);
  return static_cast<uint32_t*>(p);
}

}  // namespace sas
