// Attention of drafted tokens on the 5th-generation tensor cores (bf16
// caches): the definition of k_tree_attn.cu, TMA-fed tcgen05 MMAs with TMEM
// accumulators.
//
// One CTA per (128 rows, kv group, split of its units); rows are the group's
// heads x drafted tokens, so one K/V tile serves them all. Even with few rows
// the tensor pipe is not the bound: an M = 128 unit (S = Q K^T, O += P V)
// takes about 740 cycles where an SM's share of HBM needs 1400 for its 32 KB.
//   warp 4     TMA producers: lane 0 K, lane 1 V of each history unit, each
//              into its own two-stage ring (a K slot is free once S is done,
//              a V slot once PV is done);
//   warp 5     one elected thread issues tcgen05.mma: S_j (M128 N64, two TMEM
//              buffers) and O += P_j V_j (A = P_j read from TMEM);
//   warps 0-3  softmax, thread i = row i = TMEM lane i; warps whose rows are
//              all past the end take no part.
// With at most 64 (32) rows the tile holds two (four) copies of them, and each
// copy's threads take the softmax of a half (quarter) of a unit's keys, with
// zeros in the rest of their P: the chain from S to P, which bounds a unit, is
// shorter, and the idle lanes do the work. The copies meet at the end, in
// shared memory.
// The tail and the drafted tokens, which end inside a tile, come first in
// their split: all threads write them into the ring's stages with zeros
// behind the last key (whatever the cache holds there, 0 * NaN would reach
// the sums). A value that is not finite in a block that only some rows keep
// would reach the others the same way; such a row shows up as a sum that is
// not finite, and its warp computes it again (repair_row).
// P goes to its MMA in two bf16 parts, the upper half of its fp32 bits and the
// rest rounded, which loses at most 2^-16 of a weight; one part loses 2^-8 and
// left the results a sixth to a third further from their 64-bit values than
// the rounding of the output alone. Everything else is fp32.
// About 100 KB of shared memory and 256 TMEM columns, so two CTAs an SM. In the
// loop a CTA takes 1.5 us a unit, 5.7 TB/s over all CTAs: HBM bounds 8 x 128K
// (125 MB of kept blocks, 42 us with the start, the last CTAs of uneven groups
// and the partial outputs), L2's way to the SMs 512K with T = 64 (two tiles of
// rows read the same 36 MB, 30 us). 64K, T = 4: 12 us, latencies. (ncu, the kernel
// alone; in a call its start overlaps the selection.) An L2 prefetch of the units
// ahead cost 5% instead (it delays the first loads).
#include <cuda.h>
#include <math.h>

#include "common.cuh"
#include "kernels.h"
#include "ptx.cuh"
#include "tc.cuh"
#include "tree.cuh"

namespace sas {

__device__ uint32_t g_tree_tc_err = 0;

namespace {

constexpr int TT_THREADS = 192;
constexpr float LOG2E = 1.4426950408889634f;
constexpr float RESCALE_LOG2 = 8.0f;  // lazy rescale threshold (log2 units)

template <int D>
struct Lay {
  static constexpr uint32_t TILE = 64 * D * 2;    // one K or V block
  static constexpr uint32_t Q = 0;
  static constexpr uint32_t KV = Q + 128 * D * 2;  // stage s: K, then V
  static constexpr uint32_t BAR = KV + 4 * TILE;
  static constexpr uint32_t BITS = BAR + 128;      // block bitmap
};

enum Bar {
  B_KF = 0, B_KE = 2, B_VF = 4, B_VE = 6, B_SF = 8, B_PF = 10, B_OD = 11, NBAR = 12
};
static_assert(NBAR * 8 + 4 <= 128, "barriers and the TMEM address fit their 128 bytes");

// Barrier 1 over the softmax and MMA warps (the TMA warp is not in it).
__device__ __forceinline__ void sync_but_tma() {
  asm volatile("bar.sync 1, %0;" ::"n"(TT_THREADS - 32) : "memory");
}

// 32 lanes x 16 consecutive 32-bit columns.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float* v) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
// n columns (16, 32 or 64) of this thread's lane.
template <int N>
__device__ __forceinline__ void tmem_row(uint32_t taddr, float (&z)[N]) {
  if constexpr (N == 16) {
    tmem_ld16(taddr, z);
  } else {
#pragma unroll
    for (int c = 0; c < N / 32; ++c) tc::tmem_ld32(taddr + 32 * c, reinterpret_cast<float(&)[32]>(z[32 * c]));
  }
  tc::tmem_wait_ld();
}

// What the repair of a row needs: the row and the split that it is computed for.
struct RowState {
  unsigned long long anc, early;
  TreeRow info;
  int tok;
};
struct SplitState {
  const uint32_t* bits;
  int b, r, nt, tail, c0, nu, u0, u1, start;
};

// One row again, over the units of this split, by a whole warp: only keys that
// the row sees are read, so what other rows' blocks hold does not matter. A lane
// takes two keys of a unit for q . k and D / 32 columns for p v. A visible key
// whose logit is NaN or +inf makes the row NaN, and the units behind it are not
// read; the tail and the drafted tokens, which many rows see, come first. About
// 5 us a row and unit: a NaN in a value of the tail, seen by every row, makes a
// call of 64K and 4 tokens 61 us (27 without, launched one by one), one of 512K
// and 64 tokens 1.6 ms (68); a NaN in its key 37 and 320 us. One thread a row
// took 0.9 and 21 ms.
template <int D>
__device__ __noinline__ float2 repair_row(const TreeArgs& a, const TreeWs& w, const SplitState& s,
                                          const RowState& rs, const __nv_bfloat16* q, float* out) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const size_t group = (size_t)s.b * a.Hkv + s.r, R = (size_t)(a.Hq / a.Hkv) * a.T;
  const __nv_bfloat16* kc = static_cast<const __nv_bfloat16*>(a.kc);
  const __nv_bfloat16* vc = static_cast<const __nv_bfloat16*>(a.vc);
  const float* sc = w.scores + (group * a.T + rs.tok) * tree_stride(a.N / SAS_BLOCK);
  float m = -1e30f, l = 0.f, acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  int blk = s.start - 1;
  const int special = s.u1 - max(s.u0, min(s.nu, s.u1));
  for (int i = 0; i < s.u1 - s.u0; ++i) {
    const int u = i < special ? s.u1 - special + i : s.u0 + i - special;
    const bool drafted = u > s.nu;
    size_t at = group * a.T;  // first row of the unit
    unsigned long long see = rs.anc, gate = rs.early;  // keys seen, those with the gate's bias
    float bias = rs.info.tail_bias;
    if (!drafted) {
      see = gate = ~0ull;
      if (u < s.nu) {
        blk = tree_next(s.bits, a.words, blk + 1);
        bias = tree_bias(rs.info, __ldcg(sc + blk), blk, a.gated);
      } else {
        see = (1ull << s.tail) - 1ull;
      }
    }
    if (bias == -INFINITY) see &= ~gate;
    if (see == 0ull) continue;
    if (!drafted)
      at = tree_block_row(a, s.b, s.r,
                          max(tree_place(a, s.b, u < s.nu ? blk : s.c0, nullptr), 0));
    const __nv_bfloat16* kp = (drafted ? static_cast<const __nv_bfloat16*>(a.kd) : kc) + at * D;
    const __nv_bfloat16* vp = (drafted ? static_cast<const __nv_bfloat16*>(a.vd) : vc) + at * D;
    float p[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int j = lane + 32 * h;
      p[h] = -INFINITY;
      if (see >> j & 1ull) {
        float z = 0.f;
#pragma unroll 8
        for (int c = 0; c < D; c += 8) {
          float x[8], y[8];
          load_cg(q + c, x);
          load_cg(kp + (size_t)j * D + c, y);
#pragma unroll
          for (int k = 0; k < 8; ++k) z = fmaf(x[k], y[k], z);
        }
        p[h] = (z * a.scale + (gate >> j & 1ull ? bias : 0.f)) * LOG2E;
      }
    }
    if (__any_sync(0xffffffffu, !(p[0] < INFINITY && p[1] < INFINITY))) {
      l = NAN;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] = NAN;
      break;
    }
    const float mx = warp_max(fmaxf(p[0], p[1]));
    if (mx == -INFINITY) continue;
    const float mn = fmaxf(m, mx), alpha = exp2f(m - mn);
    m = mn;
    p[0] = exp2f(p[0] - mn);
    p[1] = exp2f(p[1] - mn);
    l = l * alpha + warp_sum(p[0] + p[1]);
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = alpha == 0.f ? 0.f : acc[e] * alpha;  // not 0 * inf
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll 16
      for (int j = 0; j < 32; ++j) {
        const float pj = __shfl_sync(0xffffffffu, p[h], j);
        if (pj == 0.f) continue;  // not seen: not read
        const uint32_t* v =
            reinterpret_cast<const uint32_t*>(vp + (size_t)(32 * h + j) * D + lane * E);
#pragma unroll
        for (int e = 0; e < E; e += 2) {
          const uint32_t x = __ldcg(v + e / 2);
          acc[e] = fmaf(pj, __uint_as_float(x << 16), acc[e]);
          acc[e + 1] = fmaf(pj, __uint_as_float(x & 0xffff0000u), acc[e + 1]);
        }
      }
    }
  }
  out += tree_part_at(lane * E, R);
#pragma unroll
  for (int e = 0; e < E; ++e) out[e] = acc[e];
  return make_float2(m, l);
}

}  // namespace

template <int D, int COPIES>
__global__ void __launch_bounds__(TT_THREADS, 2)
    k_tree_attn_tc(const __grid_constant__ CUtensorMap kmap,
                   const __grid_constant__ CUtensorMap vmap, const __grid_constant__ TreeArgs a,
                   const __grid_constant__ TreeWs w) {
  using L = Lay<D>;
  constexpr int PC = D / 8;  // 16-byte pieces of a row
  constexpr int RT = 128 / COPIES, NC = 64 / COPIES;  // rows of a copy, keys of a thread
  extern __shared__ __align__(1024) unsigned char sm[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + L::BAR);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + L::BAR + NBAR * 8);
  uint32_t* bits = reinterpret_cast<uint32_t*>(sm + L::BITS);
  __shared__ TreeShared tree;
  __shared__ int warp_s[TT_THREADS / 32];
  __shared__ int start_s;
  uint32_t* err = &g_tree_tc_err;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int r = blockIdx.y, b = blockIdx.z;
  const int split = blockIdx.x % a.ns, tile = blockIdx.x / a.ns;
  const int G = a.Hq / a.Hkv;
  const size_t group = (size_t)b * a.Hkv + r;
  // without selection this kernel is the call's first: it waits before anything
  // else
  if (a.topk == 0) grid_dep_wait();
  grid_dep_launch();
  const bool report = a.topk == 0 && blockIdx.x == 0 && r == 0;  // else the selection does
  const TreeSeq s = tree_load(a, b, tree, report ? &g_tree_tc_err : nullptr);
  const int rows = G * s.nt, row0 = tile * RT;
  if (row0 >= rows) {
    grid_dep_wait();
    return;
  }
  if ((smem_u32(sm) & 1023u) != 0) {  // swizzled tiles need 1024-byte alignment
    if (tid == 0) atomicOr(err, kErrBadIndex);
    grid_dep_wait();
    return;
  }
  const int cw = min(RT / 32, (rows - row0 + 31) / 32);  // warps with rows, of a copy
  const int nwarp = COPIES * cw;
  const bool softmax = warp < 4 && warp % (RT / 32) < cw;
  if (tid == 0) {
    for (int i = 0; i < NBAR; ++i) mbar_init(&bars[i], i == B_PF ? nwarp : 1);
    fence_mbar_init();
  }
  if (warp == 5) tc::tmem_alloc(tmem_slot, 256);
  if (tid == 128) {
    tc::prefetch_map(&kmap);
    tc::prefetch_map(&vmap);
  }
  // Q: rows of the group's heads, zeros behind the last
  const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q);
  for (int e = warp == 5 ? 128 + lane : tid; warp != 4 && e < cw * 32 * PC;
       e += TT_THREADS - 32) {
    const int row = e / PC, p = e % PC, gr = min(row0 + row, rows - 1);
    const __nv_bfloat16* src =
        q + (((size_t)b * a.Hq + r * G + gr / s.nt) * a.T + gr % s.nt) * D + p * 8;
#pragma unroll
    for (int c = 0; c < COPIES; ++c)
      cp_async16(sm + L::Q + sw_off(c * RT + row, p, 128), src, row0 + row < rows);
  }
  grid_dep_wait();
  int u0, u1;
  const int nu = tree_units<TT_THREADS>(a, w.ubits + group * a.words, bits, warp_s, &start_s,
                                        split, u0, u1);
  // this split's units: the tail and the drafted tokens first, then history
  const bool has_tail = u0 <= nu && nu < u1 && s.tail > 0;
  const bool has_draft = u0 <= nu + 1 && nu + 1 < u1;
  const int nsp = (int)has_tail + (int)has_draft;
  const int nh = max(0, min(u1, nu) - u0), nunits = nsp + nh;
  const size_t R = (size_t)G * a.T, prow = (group * a.ns + split) * R + row0 + tid % RT;
  const int start = nh > 0 ? start_s : 0;
  int tail = s.tail;  // its keys that are read: none where its page is outside the pool
  if (warp == 4) {
    // ---------------------------------------------------------------- producer
    if (lane < 2) {
      const bool kl = lane == 0;
      const CUtensorMap* map = kl ? &kmap : &vmap;
      uint64_t* fullb = &bars[kl ? B_KF : B_VF];
      uint64_t* emptyb = &bars[kl ? B_KE : B_VE];
      int blk = start - 1;
      for (int j = nsp; j < nunits; ++j) {
        const int st = j & 1;
        if (j >= 2) mbar_wait_data(&emptyb[st], ((j >> 1) - 1) & 1, err);
        blk = tree_next(bits, a.words, blk + 1);
        int y = 64 * blk, z = (int)group;
        if (a.table) {
          z = max(tree_place(a, b, blk, err), 0) * a.Hkv + r;  // a unit's page is in the pool
          y = 0;
        }
        unsigned char* dst = sm + L::KV + st * 2 * L::TILE + (kl ? 0u : L::TILE);
        mbar_arrive_expect_tx(&fullb[st], L::TILE);
#pragma unroll
        for (int c = 0; c < D / 64; ++c)
          tc::tma_load_3d(dst + c * 8192, map, 64 * c, y, z, &fullb[st]);
      }
    }
  } else {
    // the units that end inside a tile
    const int t = warp == 5 ? 128 + lane : tid;
    for (int j = 0; j < nsp; ++j) {
      const bool is_tail = has_tail && j == 0;
      int nk = s.nt;
      const __nv_bfloat16 *kp, *vp;
      if (is_tail) {
        const int place = tree_place(a, b, s.c0, err);
        if (place < 0) tail = 0;
        nk = tail;
        const size_t at = tree_block_row(a, b, r, max(place, 0)) * D;
        kp = static_cast<const __nv_bfloat16*>(a.kc) + at;
        vp = static_cast<const __nv_bfloat16*>(a.vc) + at;
      } else {
        kp = static_cast<const __nv_bfloat16*>(a.kd) + group * a.T * D;
        vp = static_cast<const __nv_bfloat16*>(a.vd) + group * a.T * D;
      }
      unsigned char* st = sm + L::KV + j * 2 * L::TILE;
#pragma unroll 2
      for (int e = t; e < 64 * PC; e += TT_THREADS - 32) {
        const int row = e / PC, p = e % PC, from = max(min(row, nk - 1), 0);
        cp_async16(st + sw_off(row, p, 64), kp + (size_t)from * D + p * 8, row < nk);
        cp_async16(st + L::TILE + sw_off(row, p, 64), vp + (size_t)from * D + p * 8, row < nk);
      }
    }
    cp_async_wait();
    fence_proxy_async_smem();  // the tiles above are read by the tensor cores
    tc::fence_before_sync();
    sync_but_tma();
    tc::fence_after_sync();
  }
  const uint32_t tmem = *tmem_slot;
  const uint32_t tm_s[2] = {tmem, tmem + 64};
  const uint32_t tm_o = tmem + 128;
  if (nunits == 0) {  // more splits than units
    if (tid < RT && row0 + tid < rows) w.ml[prow] = make_float2(-1e30f, 0.f);
  } else if (warp == 5) {
    // ---------------------------------------------------------------- MMA issuer
    if (lane == 0) {
      constexpr uint32_t ID_QK = tc::idesc_bf16(128, 64, 0, 0);
      constexpr uint32_t ID_PV = tc::idesc_bf16(128, D, 0, 1);
      // a step along an operand moves its descriptor's address field (16-byte units)
      const uint64_t q_desc = tc::sw128_desc(smem_u32(sm + L::Q), 16, 1024);
      const uint64_t k_desc = tc::sw128_desc(smem_u32(sm + L::KV), 16, 1024);
      const uint64_t v_desc = tc::sw128_desc(smem_u32(sm + L::KV) + L::TILE, 8192, 1024);
      for (int j = 0; j < nsp; ++j) {  // written above
        mbar_arrive(&bars[B_KF + j]);
        mbar_arrive(&bars[B_VF + j]);
      }
      auto pv = [&](int j) {  // O += P_j V_j
        mbar_wait(&bars[B_PF], j & 1, err);
        mbar_wait_data(&bars[B_VF + (j & 1)], (j >> 1) & 1, err);
        tc::fence_after_sync();
        const uint64_t vd = v_desc + (((j & 1) * 2 * L::TILE) >> 4);
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) {  // P_j: its upper part, then its lower, 8 columns a step
          tc::mma_bf16_tmem_a(tm_o, tm_s[j & 1] + 8 * ks, vd + (((ks & 3) * 2048) >> 4),
                              ID_PV, (j > 0 || ks > 0) ? 1u : 0u);
        }
        tc::commit(&bars[B_OD]);
        tc::commit(&bars[B_VE + (j & 1)]);
      };
      for (int j = 0; j < nunits; ++j) {
        const int st = j & 1;
        mbar_wait_data(&bars[B_KF + st], (j >> 1) & 1, err);
        // S_j overwrites P_{j-2} (S_{j-2}'s buffer): PV_{j-2} must have read it
        if (j >= 2) mbar_wait(&bars[B_OD], (j - 2) & 1, err);
        tc::fence_after_sync();
        const uint64_t kd = k_desc + ((st * 2 * L::TILE) >> 4);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {  // K = D in steps of 16 (32 bytes)
          const uint32_t c = ks >> 2, off = (ks & 3) * 32;
          tc::mma_bf16(tm_s[st], q_desc + ((c * 16384 + off) >> 4), kd + ((c * 8192 + off) >> 4),
                       ID_QK, ks > 0 ? 1u : 0u);
        }
        tc::commit(&bars[B_SF + st]);
        tc::commit(&bars[B_KE + st]);
        if (j >= 1) pv(j - 1);
      }
      pv(nunits - 1);
    }
  } else if (softmax) {
    // ---------------------------------------------------------------- softmax
    const int copy = warp / (RT / 32), row = row0 + tid % RT;
    const int key0 = copy * NC;  // this thread's keys of a unit
    const bool valid = row < rows;
    const uint32_t lane_off = (uint32_t)(warp * 32) << 16;
    const float c1 = a.scale * LOG2E, inv_scale = 1.0f / a.scale;
    RowState rs;
    rs.tok = valid ? row % s.nt : 0;
    rs.anc = tree.anc[rs.tok];
    rs.early = tree_early(tree);
    rs.info = tree_row(a, w, s, group, rs.tok, rs.anc);
    const float* sc = w.scores + (group * a.T + rs.tok) * tree_stride(a.N / SAS_BLOCK);
    float m = -1e30f, l = 0.f;
    // history units' blocks and scores, loaded two units ahead
    int blk = start, blk1 = start;
    float score = 0.f, score1 = 0.f;
    if (nh > 0) score = __ldcg(sc + blk);
    if (nh > 1) {
      blk1 = tree_next(bits, a.words, blk + 1);
      score1 = __ldcg(sc + blk1);
    }
    for (int j = 0; j < nunits; ++j) {
      const int st = j & 1;
      float bias = 0.f;
      unsigned long long see = ~0ull;
      const bool special = j < nsp;
      const bool is_tail = has_tail && j == 0;
      if (special) {
        see = is_tail ? (1ull << tail) - 1ull : rs.anc;
        if (rs.info.tail_bias == -INFINITY) see &= is_tail ? 0ull : ~rs.early;
      } else {
        bias = tree_bias(rs.info, score, blk, a.gated) * LOG2E;
        blk = blk1;
        score = score1;
        if (j + 2 < nunits) {
          blk1 = tree_next(bits, a.words, blk1 + 1);
          score1 = __ldcg(sc + blk1);
        }
      }
      if (!valid) see = 0ull;
      see >>= key0;
      if (NC < 64) see &= (1ull << (NC & 63)) - 1ull;
      const bool dead = bias == -INFINITY || see == 0ull;  // the row sees none of these keys
      mbar_wait_data(&bars[B_SF + st], (j >> 1) & 1, err);
      tc::fence_after_sync();
      float z[NC];
      tmem_row<NC>(tm_s[st] + lane_off + key0, z);
      if (special) {
        // masked keys to -inf; keys that the path moved into the tail's block
        // get its gate, in units of the raw products
        const float g = rs.info.tail_bias == -INFINITY ? 0.f : rs.info.tail_bias * inv_scale;
        const unsigned long long gate = is_tail ? ~0ull : rs.early >> key0;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
          if (gate >> i & 1ull) z[i] += g;
          if (!(see >> i & 1ull)) z[i] = -INFINITY;
        }
      }
      float zm[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) zm[c] = fmaxf(z[2 * c], z[2 * c + 1]);
#pragma unroll
      for (int i = 8; i < NC; i += 8) {
#pragma unroll
        for (int c = 0; c < 4; ++c) zm[c] = tc::max3(zm[c], z[i + 2 * c], z[i + 2 * c + 1]);
      }
      // c1 > 0, so the maximum of z c1 + bias is that of z
      const float mx =
          dead ? -INFINITY : fmaxf(fmaxf(zm[0], zm[1]), fmaxf(zm[2], zm[3])) * c1 + bias;
      const float mnew = fmaxf(m, mx);
      const bool grow = (j == 0) || (mnew > m + RESCALE_LOG2);
      const float muse = grow ? mnew : m;
      const float off = bias - muse;
      float r0 = 0.f, r1 = 0.f;
      uint32_t pk[2][NC / 2];  // upper and lower parts of P, two keys a word
#pragma unroll
      for (int i = 0; i < NC / 2; ++i) {
        float a0, a1;
        tc::fma2c(a0, a1, z[2 * i], z[2 * i + 1], c1, off);
        const float p0 = tc::ex2(a0), p1 = tc::ex2(a1);
        tc::add2(r0, r1, p0, p1);
        const uint32_t w0 = __float_as_uint(p0), w1 = __float_as_uint(p1);
        pk[0][i] = __byte_perm(w0, w1, 0x7632);
        const __nv_bfloat162 h2 = __floats2bfloat162_rn(p0 - __uint_as_float(w0 & 0xffff0000u),
                                                        p1 - __uint_as_float(w1 & 0xffff0000u));
        pk[1][i] = *reinterpret_cast<const uint32_t*>(&h2);
      }
      float rsum = r0 + r1;
      if (dead) {  // whatever the products were, NaN included
        rsum = 0.f;
#pragma unroll
        for (int i = 0; i < NC / 2; ++i) pk[0][i] = pk[1][i] = 0u;
      }
      if (j > 0) {
        // PV_{j-1} done before O is rescaled. Waiting on every unit also keeps
        // this thread within one phase of the O-done barrier.
        mbar_wait_data(&bars[B_OD], (j - 1) & 1, err);
        tc::fence_after_sync();
        const float alpha = grow ? tc::ex2(m - muse) : 1.f;
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            float ov[32];
            tc::tmem_ld32(tm_o + lane_off + 32 * c, ov);
            tc::tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) ov[i] *= alpha;
            tc::tmem_st32(tm_o + lane_off + 32 * c, ov);
          }
          tc::tmem_wait_st();
        }
        l = l * alpha + rsum;
      } else {
        l = rsum;
      }
      m = muse;
      // P_j (two parts of 64 bf16, two per column) over S_j's buffer
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float pf[32];
#pragma unroll
        for (int i = 0; i < 32; ++i)  // zeros at the other copies' keys
          pf[i] = copy == i / (NC / 2) ? __uint_as_float(pk[h][i % (NC / 2)]) : 0.f;
        tc::tmem_st32(tm_s[st] + lane_off + 32 * h, pf);
      }
      tc::tmem_wait_st();
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[B_PF]);
    }
    // epilogue: the split's sums, and O before the division
    mbar_wait_data(&bars[B_OD], (nunits - 1) & 1, err);
    tc::fence_after_sync();
    float* out = w.part + (group * a.ns + split) * R * D + (size_t)row * 4;
    bool bad = !(fabsf(l) < INFINITY);
    if constexpr (COPIES == 1) {
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        float ov[32];
        tc::tmem_ld32(tm_o + lane_off + 32 * c, ov);
        tc::tmem_wait_ld();
        if (valid) {
#pragma unroll
          for (int i = 0; i < 32; ++i) bad |= !(fabsf(ov[i]) < INFINITY);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            *reinterpret_cast<float4*>(out + tree_part_at(32 * c + 4 * i, R)) =
                make_float4(ov[4 * i], ov[4 * i + 1], ov[4 * i + 2], ov[4 * i + 3]);
        }
      }
    } else {
      // The copies' O and sums through shared memory (every tile has been
      // read): rows side by side, four columns a piece; then each copy's
      // threads join D / COPIES columns of their row.
      float4* so = reinterpret_cast<float4*>(sm + L::KV);
      float4* sml = reinterpret_cast<float4*>(sm + L::Q);
      const int rr = tid % RT;
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        float ov[32];
        tc::tmem_ld32(tm_o + lane_off + 32 * c, ov);
        tc::tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 32; ++i) bad |= !(fabsf(ov[i]) < INFINITY);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          so[(copy * (D / 4) + 8 * c + i) * RT + rr] =
              make_float4(ov[4 * i], ov[4 * i + 1], ov[4 * i + 2], ov[4 * i + 3]);
      }
      sml[copy * RT + rr] = make_float4(m, l, bad ? 1.f : 0.f, 0.f);
      asm volatile("bar.sync 2, %0;" ::"r"(nwarp * 32) : "memory");
      float f[COPIES];
      float4 x[COPIES];
      m = -1e30f;
      bad = false;
#pragma unroll
      for (int k = 0; k < COPIES; ++k) {
        x[k] = sml[k * RT + rr];
        m = fmaxf(m, x[k].x);
        bad |= x[k].z != 0.f;
      }
      l = 0.f;
#pragma unroll
      for (int k = 0; k < COPIES; ++k) {
        f[k] = tc::ex2(x[k].x - m);
        l = fmaf(x[k].y, f[k], l);
      }
      if (valid && !bad) {
#pragma unroll
        for (int c = 0; c < D / 4 / COPIES; ++c) {
          const int c4 = copy * (D / 4 / COPIES) + c;
          float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int k = 0; k < COPIES; ++k) {
            const float4 v = so[(k * (D / 4) + c4) * RT + rr];
            y.x = fmaf(v.x, f[k], y.x);
            y.y = fmaf(v.y, f[k], y.y);
            y.z = fmaf(v.z, f[k], y.z);
            y.w = fmaf(v.w, f[k], y.w);
          }
          *reinterpret_cast<float4*>(out + tree_part_at(4 * c4, R)) = y;
        }
      }
    }
    if (valid && !bad && copy == 0) w.ml[prow] = make_float2(m, l);
    // Every copy's warp knows the bad rows; each takes every COPIES-th of them.
    const uint32_t again = __ballot_sync(0xffffffffu, valid && bad && lane % COPIES == copy);
    if (again) {
      __syncwarp();  // what a row's own thread wrote to `out` is overwritten
      const SplitState ss{bits, b, r, s.nt, tail, s.c0, nu, u0, u1, start};
      const size_t at = (group * a.ns + split) * R;
      for (uint32_t todo = again; todo; todo &= todo - 1) {
        const int row1 = row0 + (warp * 32 + __ffs(todo) - 1) % RT;
        RowState r1;
        r1.tok = row1 % s.nt;
        r1.anc = tree.anc[r1.tok];
        r1.early = rs.early;
        r1.info = tree_row(a, w, s, group, r1.tok, r1.anc);
        const float2 ml = repair_row<D>(
            a, w, ss, r1, q + (((size_t)b * a.Hq + r * G + row1 / s.nt) * a.T + r1.tok) * D,
            w.part + at * D + (size_t)row1 * 4);
        if (lane == 0) w.ml[at + row1] = ml;
      }
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 5) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, 256);
  }
}

// ------------------------------------------------------------------ host
template <int D, int COPIES>
static cudaError_t launch_tc(const TreeArgs& a, const TreeWs& w, cudaStream_t st) {
  CUtensorMap km, vm;
  const int rpp = a.table ? SAS_BLOCK : a.N, planes = (a.table ? a.npages : a.B) * a.Hkv;
  if (!make_tma_map_bf16_3d(&km, a.kc, D, rpp, planes) ||
      !make_tma_map_bf16_3d(&vm, a.vc, D, rpp, planes))
    return cudaErrorInvalidValue;
  const size_t smem = Lay<D>::BITS + (size_t)a.words * sizeof(uint32_t);
  cudaError_t e = ensure_smem(k_tree_attn_tc<D, COPIES>, smem);
  if (e != cudaSuccess) return e;
  const int rows = a.Hq / a.Hkv * a.T, rt = 128 / COPIES, tiles = (rows + rt - 1) / rt;
  e = tree_launch(k_tree_attn_tc<D, COPIES>, dim3(tiles * a.ns, a.Hkv, a.B), TT_THREADS, smem, st,
                  km, vm, a, w);
  if (e != cudaSuccess) return e;
  return launch_tree_join(a, w, 1, D, st);
}

// Copies of the rows in a tile: as many as fit.
template <int D>
static cudaError_t launch_rows(const TreeArgs& a, const TreeWs& w, cudaStream_t st) {
  const int rows = a.Hq / a.Hkv * a.T;
  if (rows <= 32) return launch_tc<D, 4>(a, w, st);
  return rows <= 64 ? launch_tc<D, 2>(a, w, st) : launch_tc<D, 1>(a, w, st);
}

cudaError_t launch_tree_attn_tc(const TreeArgs& a, const TreeWs& w, int d, cudaStream_t st) {
  return d == 128 ? launch_rows<128>(a, w, st) : launch_rows<64>(a, w, st);
}

uint32_t* tree_tc_error_word() {
  void* p = nullptr;
  cudaGetSymbolAddress(&p, g_tree_tc_err);
  return static_cast<uint32_t*>(p);
}

}  // namespace sas
