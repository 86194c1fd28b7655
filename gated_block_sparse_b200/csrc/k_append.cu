// Cache write of new tokens: k rotated and written, v written, the summaries
// of the blocks that become complete, and q rotated beside them.
//
// One CTA per (sequence, 64-token block that receives tokens, slice of
// heads). Token j of sequence b has position lens[b] + j; its row of the
// cache is that position (contiguous) or its slot (64 page + row, pages of 64
// rows). A thread holds one unit (2 VN elements) of RPT rows of the block, so
// their sines and cosines are computed once and serve every head of the
// slice. When the block becomes complete the CTA has its new keys, as stored,
// in registers, reads the older ones, and reduces the 64 rows to the mean:
// no second pass over the cache. Memory bounds it: k and v are read and
// written once, and at most 63 older keys of a sequence are read again.
#include "common.cuh"
#include "kernels.h"
#include "ptx.cuh"
#include "rotary.cuh"

namespace sas {

__device__ uint32_t g_append_err = 0;

namespace {
constexpr int AP_THREADS = 256;
}

template <typename T, int VN, int D>
__global__ void __launch_bounds__(AP_THREADS) k_append(AppendArgs a) {
  constexpr int U = D / (2 * VN);            // units of a row
  constexpr int RG = AP_THREADS / U;         // rows that the CTA covers at once
  constexpr int RPT = SAS_BLOCK / RG;        // rows of a thread
  static_assert(AP_THREADS % U == 0 && SAS_BLOCK % RG == 0 && RPT >= 1, "rows divide evenly");
  __shared__ float red[RG][D];
  __shared__ int slot_s[SAS_BLOCK];
  __shared__ int src_s[SAS_BLOCK];
  const int b = blockIdx.z, tid = threadIdx.x;
  const int u = tid % U, g = tid / U;
  const int len = a.lens[b];
  int nt = a.ntok ? a.ntok[b] : a.T;
  if (len < 0 || nt < 0 || nt > a.T) {  // an impossible count: nothing is appended
    if (tid == 0 && blockIdx.x == 0 && blockIdx.y == 0) atomicOr(&g_append_err, kErrBadIndex);
    return;
  }
  const int off0 = len & (SAS_BLOCK - 1);
  const int jb = (int)blockIdx.x * SAS_BLOCK - off0;  // token of the block's row 0
  if (jb >= nt) return;
  // per row: the row of k and v that it takes (-1: none), and its place
  if (tid < SAS_BLOCK) {
    const int j = jb + tid;
    int src = -1, slot = -1;
    if (j >= 0 && j < nt) {
      src = j;
      if (a.rows) {
        src = a.rows[(size_t)b * a.T + j];
        if (src < 0 || src >= a.T) {
          atomicOr(&g_append_err, kErrBadIndex);
          src = -1;
        }
      }
      if (a.slots) {
        slot = a.slots[(size_t)b * a.T + j];
        if (slot >= 0 && (slot >> 6) >= a.npages) {
          atomicOr(&g_append_err, kErrBadIndex);
          slot = -1;
        }
      } else {
        const long long p = (long long)len + j;
        if (p < a.N)
          slot = (int)p;
        else
          atomicOr(&g_append_err, kErrBadIndex);
      }
      if (slot < 0) src = -1;
    }
    src_s[tid] = src;
    slot_s[tid] = slot;
  }
  __syncthreads();
  // The block is complete when its last row is new; its older rows then lie
  // in the page (or block) of that row. A page whose new rows are not all in
  // place (a skipped or foreign slot) keeps its summary.
  const int lslot = slot_s[SAS_BLOCK - 1];
  bool complete = a.ksum != nullptr && src_s[SAS_BLOCK - 1] >= 0;
  if (complete) {
    bool ok = true;
    if (tid < SAS_BLOCK && jb + tid >= 0)
      ok = src_s[tid] >= 0 && slot_s[tid] == lslot - (SAS_BLOCK - 1) + tid;
    complete = __syncthreads_and(ok && (lslot & (SAS_BLOCK - 1)) == SAS_BLOCK - 1);
  }
  float c[RPT][VN], s[RPT][VN];
  const bool turned = u < a.rot / (2 * VN);
  int e0, e1;
  unit_offsets<VN>(u, a.rot, a.interleaved, e0, e1);
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    const int j = jb + g + i * RG;
    if (turned && j >= 0 && j < nt) unit_sincos<VN>(a.inv_freq, u, len + j, a.amp, false, c[i], s[i]);
  }
  const int Hk = a.Hkv, Hall = Hk + (a.q ? a.Hq : 0);
  const int h0 = blockIdx.y * a.hslice, h1 = min(h0 + a.hslice, Hall);
  for (int h = h0; h < h1; ++h) {
    if (h >= Hk) {  // q: rotated only
      const T* q = static_cast<const T*>(a.q) + b * a.qs[0] + (h - Hk) * a.qs[1];
      T* y = static_cast<T*>(a.qo) + ((size_t)b * a.Hq + (h - Hk)) * a.T * D;
#pragma unroll
      for (int i = 0; i < RPT; ++i) {
        const int j = jb + g + i * RG;
        if (j < 0 || j >= nt) continue;
        float x0[VN], x1[VN];
        load_vec<T, VN>(q + j * a.qs[2] + e0, x0);
        load_vec<T, VN>(q + j * a.qs[2] + e1, x1);
        if (turned) rotate_unit<VN>(x0, x1, c[i], s[i], a.interleaved);
        store_vec<T, VN>(y + (size_t)j * D + e0, x0);
        store_vec<T, VN>(y + (size_t)j * D + e1, x1);
      }
      continue;
    }
    const T* k = static_cast<const T*>(a.k) + b * a.ks[0] + h * a.ks[1];
    const T* v = static_cast<const T*>(a.v) + b * a.vs[0] + h * a.vs[1];
    // row of the cache for a slot of this head
    auto place = [&](int slot) -> size_t {
      return a.slots ? (((size_t)(slot >> 6) * Hk + h) * SAS_BLOCK + (slot & 63)) * D
                     : (((size_t)b * Hk + h) * a.N + slot) * D;
    };
    T* kc = static_cast<T*>(a.kc);
    T* vc = static_cast<T*>(a.vc);
    float m0[VN], m1[VN];
#pragma unroll
    for (int i = 0; i < VN; ++i) m0[i] = m1[i] = 0.f;
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
      const int row = g + i * RG;
      const int src = src_s[row];
      float x0[VN], x1[VN];
      if (src >= 0) {
        T* ko = kc + place(slot_s[row]);
        T* vo = vc + place(slot_s[row]);
        float v0[VN], v1[VN];
        load_vec<T, VN>(k + src * a.ks[2] + e0, x0);
        load_vec<T, VN>(k + src * a.ks[2] + e1, x1);
        load_vec<T, VN>(v + src * a.vs[2] + e0, v0);
        load_vec<T, VN>(v + src * a.vs[2] + e1, v1);
        if (turned) rotate_unit<VN>(x0, x1, c[i], s[i], a.interleaved);
        store_vec<T, VN>(ko + e0, x0);
        store_vec<T, VN>(ko + e1, x1);
        store_vec<T, VN>(vo + e0, v0);
        store_vec<T, VN>(vo + e1, v1);
        if (complete) {  // the mean is that of the stored keys
#pragma unroll
          for (int w = 0; w < VN; ++w) {
            m0[w] += to_f(from_f<T>(x0[w]));
            m1[w] += to_f(from_f<T>(x1[w]));
          }
        }
      } else if (complete) {  // an older key of the block
        const T* ko = kc + place(lslot - (SAS_BLOCK - 1) + row);
        load_vec<T, VN>(ko + e0, x0);
        load_vec<T, VN>(ko + e1, x1);
#pragma unroll
        for (int w = 0; w < VN; ++w) {
          m0[w] += x0[w];
          m1[w] += x1[w];
        }
      }
    }
    if (complete) {
#pragma unroll
      for (int w = 0; w < VN; ++w) {
        red[g][e0 + w] = m0[w];
        red[g][e1 + w] = m1[w];
      }
      __syncthreads();
      if (tid < D) {
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < RG; ++i) sum += red[i][tid];
        sum *= 1.0f / SAS_BLOCK;
        const size_t at = a.slots ? ((size_t)(lslot >> 6) * Hk + h) * D + tid
                                  : (((size_t)b * Hk + h) * (a.N / SAS_BLOCK) + (lslot >> 6)) * D + tid;
        if (a.sum_bf16)
          static_cast<__nv_bfloat16*>(a.ksum)[at] = __float2bfloat16_rn(sum);
        else
          static_cast<float*>(a.ksum)[at] = sum;
      }
      __syncthreads();
    }
  }
}

template <typename T, int VN, int D>
static cudaError_t launch(AppendArgs a, cudaStream_t st) {
  const long long blocks = (a.T + SAS_BLOCK - 1) / SAS_BLOCK + 1;  // a start inside a block adds one
  const int H = a.Hkv + (a.q ? a.Hq : 0);
  long long slices = (148 * 4 + blocks * a.B - 1) / (blocks * a.B);
  if (slices > H) slices = H;
  a.hslice = (int)((H + slices - 1) / slices);
  dim3 grid((unsigned)blocks, (H + a.hslice - 1) / a.hslice, a.B);
  k_append<T, VN, D><<<grid, AP_THREADS, 0, st>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_append(const AppendArgs& a, int bf16, int d, cudaStream_t st) {
  const int vn = bf16 ? 8 : 4;
  bool vec = a.rot % (2 * vn) == 0;
  for (int i = 0; i < 3; ++i)
    vec = vec && a.ks[i] % vn == 0 && a.vs[i] % vn == 0 && (!a.q || a.qs[i] % vn == 0);
  if (bf16) {
    if (d == 128)
      return vec ? launch<__nv_bfloat16, 8, 128>(a, st) : launch<__nv_bfloat16, 1, 128>(a, st);
    return vec ? launch<__nv_bfloat16, 8, 64>(a, st) : launch<__nv_bfloat16, 1, 64>(a, st);
  }
  if (d == 128) return vec ? launch<float, 4, 128>(a, st) : launch<float, 1, 128>(a, st);
  return vec ? launch<float, 4, 64>(a, st) : launch<float, 1, 64>(a, st);
}

uint32_t* append_error_word() {
  void* p = nullptr;
  cudaGetSymbolAddress(&p, g_append_err);
  return static_cast<uint32_t*>(p);
}

}  // namespace sas
