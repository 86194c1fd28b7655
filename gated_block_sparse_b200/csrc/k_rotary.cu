// Rotary positions of q and k, forward and backward, in one launch.
//
// A thread holds one unit (2 VN elements, VN pairs) of one token: it computes
// the unit's VN sines and cosines once and applies them to that unit of every
// head of its slice, of q and then of k. Memory bounds it: every element is
// read once and written once. q and k of 16384 tokens, 32 + 8 heads, d = 128,
// bf16, read from a fused projection: 335 MB in 55.6 us, 6 TB/s, where a plain
// copy of as many bytes takes 54 us; fp32 106 us. 64 tokens take 4.3 us, a launch's
// latency.
#include "common.cuh"
#include "kernels.h"
#include "ptx.cuh"
#include "rotary.cuh"

namespace sas {

__device__ uint32_t g_rotary_err = 0;

namespace {
constexpr int RT_THREADS = 256;
constexpr int RT_BATCH = 4;
}

// Depth of drafted token i: its number of ancestors. A parent is below its
// child, so each hop goes down and the walk ends; any other entry is
// reported and read as -1 (a child of the last cached token). Every thread walks
// its token's path, one dependent read a level, which suits drafted trees: a
// chain of 64 tokens costs 3 us over given positions, of 256 14 us, of 1024, the
// most that is taken, 58 us.
__device__ __forceinline__ int draft_depth(const int32_t* __restrict__ parents, int i,
                                           uint32_t* err) {
  int n = 0;
  while (true) {
    const int p = __ldg(parents + i);
    if (p < -1 || p >= i) {
      atomicOr(err, kErrBadIndex);
      return n;
    }
    if (p < 0) return n;
    ++n;
    i = p;
  }
}

template <typename T, int VN>
__global__ void __launch_bounds__(RT_THREADS) k_rotary(
    RotaryTensor q, RotaryTensor k, int N, int d, const float* __restrict__ inv_freq, int rot,
    int interleaved, float amp, int inverse, const int32_t* __restrict__ pos,
    const int32_t* __restrict__ start, const int32_t* __restrict__ parents, int hslice) {
  const int U = d / (2 * VN);
  const long long item = (long long)blockIdx.x * RT_THREADS + threadIdx.x;
  const int b = blockIdx.z;
  const int n = (int)(item / U), u = (int)(item % U);
  if (n >= N) return;
  int p;
  if (pos)
    p = __ldg(pos + (size_t)b * N + n);
  else
    p = (start ? __ldg(start + b) : 0) +
        (parents ? draft_depth(parents + (size_t)b * N, n, &g_rotary_err) : n);
  const bool turned = u < rot / (2 * VN);
  float c[VN], s[VN];
  if (turned) {
    UnitTurns<VN>(inv_freq, u).sincos(p, amp, c, s);
    if (inverse) {
#pragma unroll
      for (int i = 0; i < VN; ++i) s[i] = -s[i];
    }
  }
  int e0, e1;
  unit_offsets<VN>(u, rot, interleaved, e0, e1);
  const int h0 = blockIdx.y * hslice, h1 = min(h0 + hslice, q.H + k.H);
  // RT_BATCH heads at a time, all their loads before the first store (which may
  // overwrite the input: in place, a thread's own elements)
  for (int h = h0; h < h1; h += RT_BATCH) {
    Piece<T, VN> x0[RT_BATCH], x1[RT_BATCH];
#pragma unroll
    for (int i = 0; i < RT_BATCH; ++i) {
      if (h + i >= h1) break;
      const bool isq = h + i < q.H;
      const RotaryTensor& t = isq ? q : k;
      const T* x = static_cast<const T*>(t.x) + b * t.xs[0] + (h + i - (isq ? 0 : q.H)) * t.xs[1] +
                   n * t.xs[2];
      x0[i].load(x + e0);
      x1[i].load(x + e1);
    }
#pragma unroll
    for (int i = 0; i < RT_BATCH; ++i) {
      if (h + i >= h1) break;
      const bool isq = h + i < q.H;
      const RotaryTensor& t = isq ? q : k;
      T* y = static_cast<T*>(t.y) + b * t.ys[0] + (h + i - (isq ? 0 : q.H)) * t.ys[1] + n * t.ys[2];
      if (turned) {
        float v0[VN], v1[VN];
        x0[i].unpack(v0);
        x1[i].unpack(v1);
        rotate_unit<VN>(v0, v1, c, s, interleaved);
        x0[i].pack(v0);
        x1[i].pack(v1);
      }
      x0[i].store(y + e0);
      x1[i].store(y + e1);
    }
  }
}

template <typename T, int VN>
static cudaError_t launch(const RotaryTensor& q, const RotaryTensor& k, int B, int N, int d,
                          const float* inv_freq, int rot, int interleaved, float amp, int inverse,
                          const int32_t* pos, const int32_t* start, const int32_t* parents,
                          cudaStream_t st) {
  const long long items = (long long)N * (d / (2 * VN));
  const long long blocks = (items + RT_THREADS - 1) / RT_THREADS;
  const int H = q.H + k.H;
  // Heads per thread: as many as leave the grid about four blocks an SM (small
  // calls), but no more than two batches (q and k of 16K tokens, 40 heads: 55
  // us with 8 heads a thread, 58 with 20; the sines of a thread are then
  // computed five times over, beside the copies).
  const long long want = 148 * 4;
  long long slices = (want + blocks * B - 1) / (blocks * B);
  if (slices > H) slices = H;
  int hslice = (int)((H + slices - 1) / slices);
  if (hslice > 2 * RT_BATCH) hslice = 2 * RT_BATCH;
  dim3 grid((unsigned)blocks, (H + hslice - 1) / hslice, B);
  k_rotary<T, VN><<<grid, RT_THREADS, 0, st>>>(q, k, N, d, inv_freq, rot, interleaved, amp,
                                               inverse, pos, start, parents, hslice);
  return cudaGetLastError();
}

// Vectors fit when the rotated width and every stride are multiples of them
// (the base pointers are 16-byte aligned by the interface). Otherwise the whole
// call moves single elements, columns that are only copied too: 16K tokens, 32 + 8
// heads, bf16, rot 20 or 36 144 us, rot 32 or 48 57.
static bool strides_fit(const RotaryTensor& t, int vn) {
  if (t.H == 0) return true;
  for (int i = 0; i < 3; ++i)
    if (t.xs[i] % vn || t.ys[i] % vn) return false;
  return true;
}

cudaError_t launch_rotary(const RotaryTensor& q, const RotaryTensor& k, int bf16, int B, int N,
                          int d, const float* inv_freq, int rot, int interleaved, float amp,
                          int inverse, const int32_t* pos, const int32_t* start,
                          const int32_t* parents, cudaStream_t st) {
  const int vn = bf16 ? 8 : 4;
  const bool vec = rot % (2 * vn) == 0 && strides_fit(q, vn) && strides_fit(k, vn);
  if (bf16)
    return vec ? launch<__nv_bfloat16, 8>(q, k, B, N, d, inv_freq, rot, interleaved, amp, inverse,
                                          pos, start, parents, st)
               : launch<__nv_bfloat16, 1>(q, k, B, N, d, inv_freq, rot, interleaved, amp, inverse,
                                          pos, start, parents, st);
  return vec ? launch<float, 4>(q, k, B, N, d, inv_freq, rot, interleaved, amp, inverse, pos,
                                start, parents, st)
             : launch<float, 1>(q, k, B, N, d, inv_freq, rot, interleaved, amp, inverse, pos,
                                start, parents, st);
}

uint32_t* rotary_error_word() {
  void* p = nullptr;
  cudaGetSymbolAddress(&p, g_rotary_err);
  return static_cast<uint32_t*>(p);
}

}  // namespace sas
