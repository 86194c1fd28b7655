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
// no second pass over the cache. k and v are read and written once, and at most
// 63 older keys of a sequence are read again; the next head's rows are loaded
// while this one's are summed. Two prompts of 8192 tokens, 8 kv heads, d = 128,
// bf16: 134 MB in 29 us, 4.7 TB/s, bound by the latency of a block's heads (258
// blocks, two CTAs an SM by registers, one head's rows of k and v in flight); from
// a fused projection 30 us, in fp32 53. A rotated width of 32 takes 41 us, one off
// the vectors (20) 109: every element alone, v too. A decode step of 8 sequences
// with 32 query heads takes 5.0 us: lengths, slots and, where a block completes,
// its older keys are read one after the other.
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
__global__ void __launch_bounds__(AP_THREADS, 2) k_append(AppendArgs a) {
  constexpr int U = D / (2 * VN);            // units of a row
  constexpr int RG = AP_THREADS / U;         // rows that the CTA covers at once
  constexpr int RPT = SAS_BLOCK / RG;        // rows of a thread
  static_assert(AP_THREADS % U == 0 && SAS_BLOCK % RG == 0 && RPT >= 1, "rows divide evenly");
  __shared__ float red[2][RG][D];
  __shared__ int slot_s[SAS_BLOCK];
  __shared__ int src_s[SAS_BLOCK];
  const int b = blockIdx.z, tid = threadIdx.x;
  const int u = tid % U, g = tid / U;
  const int len = a.lens[b];
  int nt = a.ntok ? a.ntok[b] : a.T;
  // an impossible count, or positions past int32: nothing is appended
  if (len < 0 || nt < 0 || nt > a.T || len > 0x7fffffff - a.T) {
    if (tid == 0 && blockIdx.x == 0 && blockIdx.y == 0) atomicOr(&g_append_err, kErrBadIndex);
    return;
  }
  const int off0 = len & (SAS_BLOCK - 1);
  const int jb = (int)blockIdx.x * SAS_BLOCK - off0;  // token of the block's row 0
  if (jb >= (a.q ? a.T : nt)) return;  // q is rotated in all its rows
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
        if (slot < -1 || (slot >= 0 && (slot >> 6) >= a.npages)) {
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
  if (turned) {
    const UnitTurns<VN> turns(a.inv_freq, u);
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
      const int j = jb + g + i * RG;
      if (j >= 0 && j < a.T) turns.sincos(len + j, a.amp, c[i], s[i]);
    }
  }
  const int Hk = a.Hkv, Hall = Hk + (a.q ? a.Hq : 0);
  const int h0 = blockIdx.y * a.hslice, h1 = min(h0 + a.hslice, Hall);
  T* kc = static_cast<T*>(a.kc);
  T* vc = static_cast<T*>(a.vc);
  const int hk = jb < nt ? min(h1, Hk) : h0;
  // first element of a slot's row of head h
  auto place = [&](int h, int slot) -> size_t {
    return a.slots ? (((size_t)(slot >> 6) * Hk + h) * SAS_BLOCK + (slot & 63)) * D
                   : (((size_t)b * Hk + h) * a.N + slot) * D;
  };
  Piece<T, VN> k0[RPT], k1[RPT], v0[RPT], v1[RPT];
  auto load_head = [&](int h) {
    const T* k = static_cast<const T*>(a.k) + b * a.ks[0] + h * a.ks[1];
    const T* v = static_cast<const T*>(a.v) + b * a.vs[0] + h * a.vs[1];
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
      const int row = g + i * RG, src = src_s[row];
      if (src >= 0) {
        k0[i].load(k + src * a.ks[2] + e0);
        k1[i].load(k + src * a.ks[2] + e1);
        v0[i].load(v + src * a.vs[2] + e0);
        v1[i].load(v + src * a.vs[2] + e1);
      } else if (complete) {  // an older key of the block
        const T* ko = kc + place(h, lslot - (SAS_BLOCK - 1) + row);
        k0[i].load(ko + e0);
        k1[i].load(ko + e1);
      }
    }
  };
  if (h0 < hk) load_head(h0);
  for (int h = h0; h < hk; ++h) {
    float m0[VN], m1[VN];
#pragma unroll
    for (int i = 0; i < VN; ++i) m0[i] = m1[i] = 0.f;
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
      const int row = g + i * RG;
      const bool fresh = src_s[row] >= 0;
      if (!fresh && !complete) continue;
      float x0[VN], x1[VN];
      if (fresh) {
        if (turned) {
          k0[i].unpack(x0);
          k1[i].unpack(x1);
          rotate_unit<VN>(x0, x1, c[i], s[i], a.interleaved);
          k0[i].pack(x0);
          k1[i].pack(x1);
        }
        const size_t at = place(h, slot_s[row]);
        k0[i].store(kc + at + e0);
        k1[i].store(kc + at + e1);
        v0[i].store(vc + at + e0);  // v is moved as it is
        v1[i].store(vc + at + e1);
      }
      if (complete) {  // the mean is that of the stored keys
        k0[i].unpack(x0);
        k1[i].unpack(x1);
#pragma unroll
        for (int w = 0; w < VN; ++w) {
          m0[w] += x0[w];
          m1[w] += x1[w];
        }
      }
    }
    if (h + 1 < hk) load_head(h + 1);  // in flight under the sum
    if (complete) {
      float(*rs)[D] = red[(h - h0) & 1];  // two buffers: one barrier a head
#pragma unroll
      for (int w = 0; w < VN; ++w) {
        rs[g][e0 + w] = m0[w];
        rs[g][e1 + w] = m1[w];
      }
      __syncthreads();
      if (tid < D) {
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < RG; ++i) sum += rs[i][tid];
        sum *= 1.0f / SAS_BLOCK;
        const size_t at = a.slots ? ((size_t)(lslot >> 6) * Hk + h) * D + tid
                                  : (((size_t)b * Hk + h) * (a.N / SAS_BLOCK) + (lslot >> 6)) * D + tid;
        if (a.sum_bf16)
          static_cast<__nv_bfloat16*>(a.ksum)[at] = __float2bfloat16_rn(sum);
        else
          static_cast<float*>(a.ksum)[at] = sum;
      }
    }
  }
  // q: rotated only
  for (int h = max(h0, Hk); h < h1; ++h) {
    const T* q = static_cast<const T*>(a.q) + b * a.qs[0] + (h - Hk) * a.qs[1];
    T* y = static_cast<T*>(a.qo) + ((size_t)b * a.Hq + (h - Hk)) * a.T * D;
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
      const int j = jb + g + i * RG;
      if (j < 0 || j >= a.T) continue;
      k0[i].load(q + j * a.qs[2] + e0);
      k1[i].load(q + j * a.qs[2] + e1);
    }
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
      const int j = jb + g + i * RG;
      if (j < 0 || j >= a.T) continue;
      if (turned) {
        float x0[VN], x1[VN];
        k0[i].unpack(x0);
        k1[i].unpack(x1);
        rotate_unit<VN>(x0, x1, c[i], s[i], a.interleaved);
        k0[i].pack(x0);
        k1[i].pack(x1);
      }
      k0[i].store(y + (size_t)j * D + e0);
      k1[i].store(y + (size_t)j * D + e1);
    }
  }
}

template <typename T, int VN, int D>
static cudaError_t launch(AppendArgs a, cudaStream_t st) {
  const long long blocks = (a.T + SAS_BLOCK - 1) / SAS_BLOCK + 1;  // a start inside a block adds one
  const int H = a.Hkv + (a.q ? a.Hq : 0);
  // Heads of a CTA: all of them where the blocks fill the SMs (two prompts of
  // 8K tokens, 8 kv heads: 29 us, against 31 with 4 heads and 34 with 1: the
  // sines serve every head), else down to one (8 decode steps with q: 6.3 us,
  // against 9.5 with 3 heads, before the rows without a token skipped their sines).
  const long long ctas = blocks * a.B;
  long long slices = ctas >= 148 ? 1 : (148 * 8 + ctas - 1) / ctas;
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
