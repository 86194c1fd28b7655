// Block tables and slot maps from request lengths.
//
// Sequence b holds len tokens in ceil(len / 64) pages and receives n more. It
// needs ceil((len + n) / 64) - ceil(len / 64) new pages, taken from the list
// of free pages in the order of the sequences: its first one is at head plus
// the sum of the earlier needs. A sequence whose own numbers are impossible
// needs nothing and is refused; one whose pages end past the list is refused
// too, and its need still counts in the later sums, so every sequence finds
// its place by a prefix sum alone, whatever happened to the others.
//
// Latency bounds it: a decode step moves a few kilobytes (256 requests: 3.3 us;
// 64 prompts of up to 8192 tokens, 2 MB of slots: 3.3 us). Up to 16 tokens a
// sequence: one CTA, a thread per sequence, one scan. More: a grid of
// (sequence, 1024 tokens) CTAs that each sum the earlier needs themselves
// (two coalesced reads of the lengths), so no CTA waits for another. What that
// border costs, us for 256, 1024, 4096, 16384 and 65534 requests: the one CTA
// 3.3, 3.8, 9.6, 34 and 130 with one token, 6.4, 12, 46, 184 and 731 with 16;
// the grid 3.1, 4.4, 17, 129 and 1552 with 17, its sums quadratic in the requests.
#include "common.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace sas {

__device__ uint32_t g_pages_err = 0;

namespace {
constexpr int PG_THREADS = 256;   // grid form
constexpr int PG_ROWS = 1024;     // one-CTA form: sequences a pass
constexpr int PG_PER_THREAD = 4;  // slots a thread, one 16-byte store
}

// Pages that sequence (len, n) needs; false when its numbers are impossible.
__device__ __forceinline__ bool page_need(int len, int n, int T, int width, int& have, int& need) {
  have = need = 0;
  if (len < 0 || n < 0 || n > T || (long long)len + n > (long long)width * SAS_BLOCK) return false;
  have = (int)(((long long)len + SAS_BLOCK - 1) / SAS_BLOCK);
  need = (int)(((long long)len + n + SAS_BLOCK - 1) / SAS_BLOCK) - have;
  return true;
}

// Whether the need of a sequence whose earlier needs sum to `before` fits.
__device__ __forceinline__ bool page_fits(const PageMapArgs& a, int head, int before, int need) {
  return need == 0 || (head >= 0 && (long long)head + before + need <= a.nfree);
}

// Slot of token j of a sequence: its page is an earlier page of the table
// (the partly filled last one) or the one taken from the free list. An id
// outside the pool is reported and gives no slot.
__device__ __forceinline__ int slot_of(const PageMapArgs& a, int b, int len, int have, int first,
                                       int j) {
  const int p = len + j, m = p >> 6;
  const int page = m < have ? a.table[(size_t)b * a.width + m] : a.free_pages[first + m - have];
  if (page < 0 || page >= a.npages) {
    atomicOr(&g_pages_err, kErrBadIndex);
    return -1;
  }
  return page * SAS_BLOCK + (p & (SAS_BLOCK - 1));
}

// Inclusive sum over the block's threads; *total gets the sum of all.
template <int WARPS>
__device__ __forceinline__ int block_scan(int v, int* warp_sum_s, int* total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += y;
  }
  if (lane == 31) warp_sum_s[w] = v;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int i = 0; i < WARPS; ++i) {
    const int s = warp_sum_s[i];
    before += i < w ? s : 0;
    all += s;
  }
  __syncthreads();
  *total = all;
  return before + v;
}

// One CTA of THREADS threads, one per sequence: lengths, counts and head, and
// with SLOTS also slots and table. Every length is read by the thread that
// later writes it, so new_lens may be lens itself, and head_out free_head.
template <int THREADS, bool SLOTS>
__device__ __forceinline__ void page_rows(const PageMapArgs& a) {
  __shared__ int ws[THREADS / 32];
  __shared__ int granted_s;
  if (threadIdx.x == 0) granted_s = 0;
  const int head = a.free_head[0];
  if (threadIdx.x == 0 && (head < 0 || head > a.nfree)) atomicOr(&g_pages_err, kErrBadIndex);
  int carry = 0;
  for (int b0 = 0; b0 < a.B; b0 += THREADS) {
    const int b = b0 + (int)threadIdx.x;
    int len = 0, n = 0, have = 0, need = 0, total;
    bool ok = false;
    if (b < a.B) {
      len = a.lens[b];
      n = a.nnew[b];
      ok = page_need(len, n, a.T, a.width, have, need);
    }
    const int incl = block_scan<THREADS / 32>(need, ws, &total);
    const int before = carry + incl - need;
    carry += total;
    ok = ok && page_fits(a, head, before, need);
    if (b < a.B) {
      if (SLOTS) {
        for (int j = 0; j < a.T; ++j)
          a.slots[(size_t)b * a.T + j] =
              ok && j < n ? slot_of(a, b, len, have, head + before, j) : -1;
        if (ok)
          for (int i = 0; i < need; ++i)
            a.table[(size_t)b * a.width + have + i] = a.free_pages[head + before + i];
      }
      a.new_lens[b] = ok ? len + n : len;
      a.taken[b] = ok ? need : -1;
      if (ok && need) atomicAdd(&granted_s, need);  // a sum of integers: any order
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) a.head_out[0] = head + granted_s;
}

__global__ void __launch_bounds__(PG_ROWS) k_page_rows(PageMapArgs a) {
  page_rows<PG_ROWS, true>(a);
}
__global__ void __launch_bounds__(PG_ROWS) k_page_close(PageMapArgs a) {
  page_rows<PG_ROWS, false>(a);
}

// Row b of the grid: slots and table of sequence b. Row B, where the launch
// has one: the step's lengths, counts and head.
__global__ void __launch_bounds__(PG_THREADS) k_page_slots(PageMapArgs a) {
  __shared__ int ws[PG_THREADS / 32];
  const int b = blockIdx.y, tid = threadIdx.x;
  if (b == a.B) {
    if (blockIdx.x == 0) page_rows<PG_THREADS, false>(a);
    return;
  }
  const int head = a.free_head[0];
  int part = 0, before, have, need;
  for (int i = tid; i < b; i += PG_THREADS) {
    int h, nd;
    page_need(a.lens[i], a.nnew[i], a.T, a.width, h, nd);
    part += nd;
  }
  block_scan<PG_THREADS / 32>(part, ws, &before);
  const int len = a.lens[b], n = a.nnew[b];
  const bool ok = page_need(len, n, a.T, a.width, have, need) && page_fits(a, head, before, need);
  const int first = head + before;
  if (ok && blockIdx.x == 0)
    for (int i = tid; i < need; i += PG_THREADS)
      a.table[(size_t)b * a.width + have + i] = a.free_pages[first + i];
  const int j0 = ((int)blockIdx.x * PG_THREADS + tid) * PG_PER_THREAD;
  if (j0 >= a.T) return;
  int s[PG_PER_THREAD];
#pragma unroll
  for (int i = 0; i < PG_PER_THREAD; ++i)
    s[i] = ok && j0 + i < n ? slot_of(a, b, len, have, first, j0 + i) : -1;
  int32_t* out = a.slots + (size_t)b * a.T + j0;
  if (a.T % PG_PER_THREAD == 0) {
    *reinterpret_cast<int4*>(out) = make_int4(s[0], s[1], s[2], s[3]);
  } else {
#pragma unroll
    for (int i = 0; i < PG_PER_THREAD; ++i)
      if (j0 + i < a.T) out[i] = s[i];
  }
}

cudaError_t launch_page_map(const PageMapArgs& a, cudaStream_t st) {
  if (a.T <= 16 || a.B == 0) {
    k_page_rows<<<1, PG_ROWS, 0, st>>>(a);
    return cudaGetLastError();
  }
  // In place (lengths or head), the step is closed by a launch of its own,
  // after every CTA has read them.
  const bool in_place = a.new_lens == a.lens || a.head_out == a.free_head;
  const int per = PG_THREADS * PG_PER_THREAD;
  k_page_slots<<<dim3((a.T + per - 1) / per, a.B + !in_place), PG_THREADS, 0, st>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !in_place) return e;
  k_page_close<<<1, PG_ROWS, 0, st>>>(a);
  return cudaGetLastError();
}

uint32_t* pages_error_word() {
  void* p = nullptr;
  cudaGetSymbolAddress(&p, g_pages_err);
  return static_cast<uint32_t*>(p);
}

}  // namespace sas
