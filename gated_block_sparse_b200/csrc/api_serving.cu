// C ABI of the serving calls (declared in include/sas_serving.h): argument
// validation and launches. Host code only.
#include "../../include/sas_serving.h"

#include <algorithm>

#include "api_common.h"
#include "kernels.h"

using sas::aligned16;
using sas::check_common;
using sas::cuda_status;

namespace {

// Strides of a [B][H][N][d] tensor, from the caller's or contiguous.
void set_strides(long long (&out)[3], const int64_t* in, int H, int N, int d) {
  out[0] = in ? in[0] : (long long)H * N * d;
  out[1] = in ? in[1] : (long long)N * d;
  out[2] = in ? in[2] : d;
}

// Whether two ranges of memory share a byte.
struct Range {
  uintptr_t lo, hi;
  Range(const void* p, size_t bytes)
      : lo(reinterpret_cast<uintptr_t>(p)), hi(reinterpret_cast<uintptr_t>(p) + (p ? bytes : 0)) {}
  bool meets(const Range& o) const { return lo < o.hi && o.lo < hi; }
};

// Bytes from the first to behind the last row of a [B][H][N] array of rows of d.
size_t span_bytes(const long long (&s)[3], int B, int H, int N, int d, int es) {
  return (size_t)(s[0] * (B - 1) + s[1] * (H - 1) + s[2] * (N - 1) + d) * es;
}

// Dimensions of one element never use their stride, and no heads use none.
bool strides_ok(const long long (&s)[3], int B, int H, int N, long long least) {
  if (H == 0) return true;
  return (B <= 1 || s[0] >= least) && (H <= 1 || s[1] >= least) && (N <= 1 || s[2] >= least);
}

// A [B][H][N] array of rows of d elements: element strides, sizes.
struct Rows {
  const void* p;
  long long s[3];
  int n[3];
};

// Whether no two rows of the array share an element: with the strides in
// ascending order, each passes over the whole extent of the ones before. (Views
// that torch makes by slicing and transposing are all of that kind.)
bool rows_apart(const Rows& r, int d) {
  int order[3] = {0, 1, 2};
  std::sort(order, order + 3, [&](int i, int j) { return r.s[i] < r.s[j]; });
  long long extent = d;
  for (int i : order) {
    if (r.n[i] <= 1) continue;
    if (r.s[i] < extent) return false;
    extent += r.s[i] * (r.n[i] - 1);
  }
  return true;
}

bool same_strides(const Rows& x, const Rows& y) {
  for (int i = 0; i < 3; ++i)
    if (x.n[i] > 1 && y.n[i] > 1 && x.s[i] != y.s[i]) return false;
  return true;
}

// Whether a row of x shares an element with a row of y (rows_apart holds for y).
// Equal strides: whether the distance of their first elements is a sum of
// strides times differences of indices, and less than d; from the largest stride
// down, two multiples come into question each. Other strides: whether the ranges
// from first to last row meet.
bool rows_meet(const Rows& x, const Rows& y, int d, int es) {
  const Range rx(x.p, span_bytes(x.s, x.n[0], x.n[1], x.n[2], d, es));
  const Range ry(y.p, span_bytes(y.s, y.n[0], y.n[1], y.n[2], d, es));
  if (!rx.meets(ry)) return false;
  if (!same_strides(x, y)) return true;
  struct Dim {
    long long s;
    int lo, hi;  // index of x minus index of y
  } dim[3];
  int nd = 0;
  for (int i = 0; i < 3; ++i)
    if (x.n[i] > 1 || y.n[i] > 1)
      dim[nd++] = {x.n[i] > 1 ? x.s[i] : y.s[i], -(y.n[i] - 1), x.n[i] - 1};
  std::sort(dim, dim + nd, [](const Dim& a, const Dim& b) { return a.s > b.s; });
  const long long delta = ((long long)ry.lo - (long long)rx.lo) / es;
  for (int pick = 0; pick < 1 << nd; ++pick) {
    long long left = delta;
    bool fits = true;
    for (int i = 0; i < nd && fits; ++i) {
      if (dim[i].s <= 0) return true;
      long long k = left / dim[i].s - (left % dim[i].s < 0) + (pick >> i & 1);
      fits = k >= dim[i].lo && k <= dim[i].hi;
      left -= k * dim[i].s;
    }
    if (fits && left > -d && left < d) return true;
  }
  return false;
}

sas_status check_rotation(const float* inv_freq, int rot, int d, int interleaved,
                          float amplitude) {
  REQUIRE_PTR(inv_freq);
  REQUIRE(rot >= 2 && rot <= d && rot % 2 == 0, SAS_ERR_INVALID_ARG,
          "rot must be even and in [2, %d] (got %d)", d, rot);
  REQUIRE(interleaved == 0 || interleaved == 1, SAS_ERR_INVALID_ARG, "interleaved must be 0 or 1");
  REQUIRE(isfinite(amplitude), SAS_ERR_INVALID_ARG, "amplitude must be finite");
  return SAS_OK;
}

#define REQUIRE_OPT(p) \
  REQUIRE((p) == nullptr || aligned16(p), SAS_ERR_INVALID_ARG, "%s must be 16-byte aligned", #p)

}  // namespace

extern "C" {

sas_status sas_rotary(const void* q, const int64_t* q_strides, void* qo,
                      const int64_t* qo_strides, int Hq, const void* k, const int64_t* k_strides,
                      void* ko, const int64_t* ko_strides, int Hkv, sas_dtype dt, int B, int N,
                      int d, const float* inv_freq, int rot, int interleaved, float amplitude,
                      int inverse, const int32_t* pos, const int32_t* start,
                      const int32_t* parents, sas_stream_t stream) {
  sas::clear_error();
  sas_status s = check_common(dt, B, 1, 1, N, d, 0);
  if (s != SAS_OK) return s;
  REQUIRE(Hq >= 1 && Hkv >= 0, SAS_ERR_INVALID_ARG, "head counts: Hq >= 1, Hkv >= 0 (Hq=%d Hkv=%d)",
          Hq, Hkv);
  REQUIRE((Hkv == 0) == (k == nullptr), SAS_ERR_INVALID_ARG, "k goes with Hkv >= 1");
  REQUIRE(B <= 65535, SAS_ERR_UNSUPPORTED, "B must be <= 65535 (got %d)", B);
  REQUIRE(Hq + (long long)Hkv <= 65535, SAS_ERR_UNSUPPORTED, "at most 65535 heads");
  REQUIRE(inverse == 0 || inverse == 1, SAS_ERR_INVALID_ARG, "inverse must be 0 or 1");
  REQUIRE(pos == nullptr || (start == nullptr && parents == nullptr), SAS_ERR_INVALID_ARG,
          "pos excludes start and parents");
  // every thread walks its token's ancestors, so a long chain costs N squared
  REQUIRE(parents == nullptr || N <= 1024, SAS_ERR_UNSUPPORTED,
          "N must be <= 1024 with parents (got %d)", N);
  if (B == 0 || N == 0) return SAS_OK;
  s = check_rotation(inv_freq, rot, d, interleaved, amplitude);
  if (s != SAS_OK) return s;
  REQUIRE_PTR(q);
  REQUIRE_PTR(qo);
  if (k) {
    REQUIRE_PTR(k);
    REQUIRE_PTR(ko);
  }
  REQUIRE_OPT(pos);
  REQUIRE_OPT(start);
  REQUIRE_OPT(parents);
  sas::RotaryTensor tq{q, qo, Hq, {}, {}}, tk{k, ko, Hkv, {}, {}};
  set_strides(tq.xs, q_strides, Hq, N, d);
  set_strides(tq.ys, qo_strides, Hq, N, d);
  set_strides(tk.xs, k_strides, Hkv, N, d);
  set_strides(tk.ys, ko_strides, Hkv, N, d);
  REQUIRE(strides_ok(tq.xs, B, Hq, N, 0) && strides_ok(tk.xs, B, Hkv, N, 0), SAS_ERR_INVALID_ARG,
          "input strides must be >= 0");
  REQUIRE(strides_ok(tq.ys, B, Hq, N, d) && strides_ok(tk.ys, B, Hkv, N, d), SAS_ERR_INVALID_ARG,
          "output strides must be >= d (rows must not overlap)");
  const int es = dt == SAS_BF16 ? 2 : 4;
  auto rows = [&](const void* p, const long long (&st)[3], int H) {
    return Rows{p, {st[0], st[1], st[2]}, {B, H, N}};
  };
  const Rows in[2] = {rows(q, tq.xs, Hq), rows(k, tk.xs, Hkv)};
  const Rows out[2] = {rows(qo, tq.ys, Hq), rows(ko, tk.ys, Hkv)};
  for (int j = 0; j < (k ? 2 : 1); ++j)
    REQUIRE(rows_apart(out[j], d), SAS_ERR_INVALID_ARG, "output rows must not overlap");
  REQUIRE(!k || !rows_meet(out[0], out[1], d, es), SAS_ERR_INVALID_ARG,
          "qo and ko must not overlap");
  for (int i = 0; i < (k ? 2 : 1); ++i)
    for (int j = 0; j < (k ? 2 : 1); ++j) {
      const bool in_place = i == j && in[i].p == out[j].p && same_strides(in[i], out[j]);
      REQUIRE(in_place || !rows_meet(in[i], out[j], d, es), SAS_ERR_INVALID_ARG,
              "an output must be its input itself, with its strides, or lie apart from the inputs");
    }
  return cuda_status(sas::launch_rotary(tq, tk, dt == SAS_BF16, B, N, d, inv_freq, rot,
                                        interleaved, amplitude, inverse, pos, start, parents,
                                        (cudaStream_t)stream),
                     "sas_rotary launch");
}

sas_status sas_page_map(const int32_t* lens, const int32_t* nnew, int32_t* block_table,
                        const int32_t* free_pages, const int32_t* free_head, int B, int T,
                        int width, int npages, int nfree, int32_t* slots, int32_t* new_lens,
                        int32_t* taken, int32_t* head_out, sas_stream_t stream) {
  sas::clear_error();
  REQUIRE(B >= 0 && T >= 0 && width >= 0 && nfree >= 0, SAS_ERR_INVALID_ARG,
          "sizes must be >= 0 (B=%d T=%d width=%d nfree=%d)", B, T, width, nfree);
  REQUIRE(npages >= 0 && npages <= (1 << 25), SAS_ERR_UNSUPPORTED,
          "npages must be in [0, 2^25] (got %d)", npages);
  REQUIRE((long long)B * ((long long)T + 128) < (1ll << 31), SAS_ERR_UNSUPPORTED,
          "B (T + 128) must be below 2^31 (B=%d T=%d)", B, T);
  REQUIRE((long long)width * 64 < (1ll << 31), SAS_ERR_UNSUPPORTED,
          "64 width must be below 2^31 (width=%d)", width);
  REQUIRE(B <= 65534, SAS_ERR_UNSUPPORTED, "B must be <= 65534 (got %d)", B);
  if (B > 0) {
    REQUIRE_PTR(lens);
    REQUIRE_PTR(nnew);
    REQUIRE_PTR(new_lens);
    REQUIRE_PTR(taken);
    if (width > 0) REQUIRE_PTR(block_table);
    if (T > 0) REQUIRE_PTR(slots);
  }
  if (nfree > 0) REQUIRE_PTR(free_pages);
  REQUIRE_PTR(free_head);
  REQUIRE_PTR(head_out);
  // every array apart from the ones that are written, but for the two in place
  const struct {
    const char* name;
    Range r;
  } arrays[] = {{"slots", {slots, (size_t)B * T * 4}},
                {"new_lens", {new_lens, (size_t)B * 4}},
                {"taken", {taken, (size_t)B * 4}},
                {"head_out", {head_out, 4}},
                {"block_table", {block_table, (size_t)B * width * 4}},
                {"lens", {lens, (size_t)B * 4}},
                {"nnew", {nnew, (size_t)B * 4}},
                {"free_pages", {free_pages, (size_t)nfree * 4}},
                {"free_head", {free_head, 4}}};
  for (int i = 0; i < 5; ++i)
    for (int j = i + 1; j < 9; ++j) {
      const bool in_place = (i == 1 && j == 5 && new_lens == lens) ||
                            (i == 3 && j == 8 && head_out == free_head);
      REQUIRE(in_place || !arrays[i].r.meets(arrays[j].r), SAS_ERR_INVALID_ARG,
              "%s and %s must not overlap", arrays[i].name, arrays[j].name);
    }
  const sas::PageMapArgs a{lens,  nnew,     block_table, free_pages, free_head, slots, new_lens,
                           taken, head_out, B,           T,          width,     npages, nfree};
  return cuda_status(sas::launch_page_map(a, (cudaStream_t)stream), "sas_page_map launch");
}

sas_status sas_cache_append(const void* q, const int64_t* q_strides, void* qo, const void* k,
                            const int64_t* k_strides, const void* v, const int64_t* v_strides,
                            sas_dtype dt, int B, int Hq, int Hkv, int T, int d,
                            const int32_t* rows, const int32_t* lens, const int32_t* ntok,
                            const float* inv_freq, int rot, int interleaved, float amplitude,
                            const int32_t* slots, void* kc, void* vc, int N, int npages,
                            void* ksum, sas_dtype sum_dt, sas_stream_t stream) {
  sas::clear_error();
  sas_status s = check_common(dt, B, q ? Hq : Hkv, Hkv, T, d, 0);
  if (s != SAS_OK) return s;
  REQUIRE(sum_dt == SAS_F32 || sum_dt == SAS_BF16, SAS_ERR_INVALID_ARG,
          "summary dtype must be SAS_F32 or SAS_BF16");
  REQUIRE(B <= 65535, SAS_ERR_UNSUPPORTED, "B must be <= 65535 (got %d)", B);
  REQUIRE((q ? (long long)Hq : 0ll) + Hkv <= 65535, SAS_ERR_UNSUPPORTED, "at most 65535 heads");
  REQUIRE(q == nullptr || (inv_freq != nullptr && rows == nullptr), SAS_ERR_INVALID_ARG,
          "q needs inv_freq and no rows");
  REQUIRE(T <= (1 << 30), SAS_ERR_UNSUPPORTED, "T must be <= 2^30 (got %d)", T);
  if (slots)
    REQUIRE(npages >= 1 && npages <= (1 << 25), SAS_ERR_INVALID_ARG,
            "npages must be in [1, 2^25] (got %d)", npages);
  else
    REQUIRE(N >= 0 && N % 64 == 0, SAS_ERR_INVALID_ARG, "N must be a multiple of 64 (got %d)", N);
  if (B == 0 || T == 0) return SAS_OK;
  if (inv_freq) {
    s = check_rotation(inv_freq, rot, d, interleaved, amplitude);
    if (s != SAS_OK) return s;
  }
  REQUIRE_PTR(k);
  REQUIRE_PTR(v);
  REQUIRE_PTR(kc);
  REQUIRE_PTR(vc);
  REQUIRE_PTR(lens);
  if (q) {
    REQUIRE_PTR(q);
    REQUIRE_PTR(qo);
  }
  REQUIRE_OPT(rows);
  REQUIRE_OPT(ntok);
  REQUIRE_OPT(slots);
  REQUIRE_OPT(ksum);
  sas::AppendArgs a{};
  a.q = q; a.k = k; a.v = v;
  a.qo = qo; a.kc = kc; a.vc = vc; a.ksum = ksum;
  set_strides(a.qs, q_strides, Hq, T, d);
  set_strides(a.ks, k_strides, Hkv, T, d);
  set_strides(a.vs, v_strides, Hkv, T, d);
  REQUIRE(strides_ok(a.ks, B, Hkv, T, 0) && strides_ok(a.vs, B, Hkv, T, 0) &&
              (!q || strides_ok(a.qs, B, Hq, T, 0)),
          SAS_ERR_INVALID_ARG, "input strides must be >= 0");
  const int es = dt == SAS_BF16 ? 2 : 4;
  const size_t cache = (slots ? (size_t)npages * 64 : (size_t)B * N) * Hkv * d * es;
  const Range rk(k, span_bytes(a.ks, B, Hkv, T, d, es)), rv(v, span_bytes(a.vs, B, Hkv, T, d, es));
  const Range rkc(kc, cache), rvc(vc, cache);
  REQUIRE(!rkc.meets(rvc), SAS_ERR_INVALID_ARG, "kc and vc must not overlap");
  REQUIRE(!rk.meets(rkc) && !rk.meets(rvc) && !rv.meets(rkc) && !rv.meets(rvc),
          SAS_ERR_INVALID_ARG, "k and v must not lie in the cache (blocks are written in any order)");
  if (q) {
    const Range rq(q, span_bytes(a.qs, B, Hq, T, d, es)), rqo(qo, (size_t)B * Hq * T * d * es);
    const bool dense = (B <= 1 || a.qs[0] == (long long)Hq * T * d) &&
                       (Hq <= 1 || a.qs[1] == (long long)T * d) && (T <= 1 || a.qs[2] == d);
    REQUIRE((q == qo && dense) || !rq.meets(rqo), SAS_ERR_INVALID_ARG,
            "qo must be q itself (contiguous) or lie apart from it");
    REQUIRE(!rqo.meets(rk) && !rqo.meets(rv) && !rqo.meets(rkc) && !rqo.meets(rvc),
            SAS_ERR_INVALID_ARG, "qo must lie apart from k, v and the cache");
  }
  a.rows = rows; a.lens = lens; a.ntok = ntok; a.slots = slots;
  a.inv_freq = inv_freq;
  a.amp = amplitude;
  a.B = B; a.Hq = Hq; a.Hkv = Hkv; a.T = T; a.N = N; a.npages = npages;
  a.rot = inv_freq ? rot : 0;
  a.interleaved = interleaved;
  a.sum_bf16 = sum_dt == SAS_BF16;
  return cuda_status(sas::launch_append(a, dt == SAS_BF16, d, (cudaStream_t)stream),
                     "sas_cache_append launch");
}

static sas_status check_tree(sas_dtype dt, int B, int Hq, int Hkv, int T, int N, int d,
                             int topk) {
  sas_status s = check_common(dt, B, Hq, Hkv, N, d, topk);
  if (s != SAS_OK) return s;
  REQUIRE(T >= 1, SAS_ERR_INVALID_ARG, "T must be >= 1 (got %d)", T);
  REQUIRE(T <= 64, SAS_ERR_UNSUPPORTED, "at most 64 drafted tokens a sequence (got %d)", T);
  REQUIRE(N % 64 == 0 && N >= 64, SAS_ERR_INVALID_ARG, "N must be a positive multiple of 64");
  REQUIRE(N <= (1 << 20), SAS_ERR_UNSUPPORTED, "N must be <= 2^20 (got %d)", N);
  REQUIRE(B <= 65535, SAS_ERR_UNSUPPORTED, "B must be <= 65535 (got %d)", B);
  REQUIRE(Hkv <= 65535, SAS_ERR_UNSUPPORTED, "Hkv must be <= 65535 (got %d)", Hkv);
  return SAS_OK;
}

size_t sas_decode_tree_workspace_size(int B, int Hq, int Hkv, int T, int N, int d, int topk,
                                      sas_dtype dt) {
  if (B <= 0 || check_tree(dt, B, Hq, Hkv, T, N, d, topk) != SAS_OK) return 0;
  return sas::tree_ws_bytes(B, Hq, Hkv, T, N, d, topk, dt == SAS_BF16);
}

sas_status sas_decode_tree(const void* q, const void* kd, const void* vd, const void* kc,
                           const void* vc, sas_dtype dt, int B, int Hq, int Hkv, int T, int N,
                           int d, const int32_t* parents, const int32_t* ntok,
                           const int32_t* lens, const void* ksum, sas_dtype sum_dt,
                           const int32_t* block_table, int npages, int topk, int gated,
                           float scale, void* o, int32_t* idx_out, void* ws, size_t ws_bytes,
                           sas_stream_t stream) {
  sas::clear_error();
  sas_status s = check_tree(dt, B, Hq, Hkv, T, N, d, topk);
  if (s != SAS_OK) return s;
  REQUIRE(sum_dt == SAS_F32 || sum_dt == SAS_BF16, SAS_ERR_INVALID_ARG,
          "summary dtype must be SAS_F32 or SAS_BF16");
  REQUIRE(gated == 0 || gated == 1, SAS_ERR_INVALID_ARG, "gated must be 0 or 1");
  REQUIRE(block_table == nullptr || npages >= 1, SAS_ERR_INVALID_ARG,
          "npages must be >= 1 (got %d)", npages);
  if (B == 0) return SAS_OK;
  REQUIRE_PTR(q);
  REQUIRE_PTR(kd);
  REQUIRE_PTR(vd);
  REQUIRE_PTR(kc);
  REQUIRE_PTR(vc);
  REQUIRE_PTR(lens);
  REQUIRE_PTR(o);
  if (topk > 0) REQUIRE_PTR(ksum);
  REQUIRE_OPT(parents);
  REQUIRE_OPT(ntok);
  REQUIRE_OPT(block_table);
  REQUIRE_OPT(idx_out);
  const size_t need = sas_decode_tree_workspace_size(B, Hq, Hkv, T, N, d, topk, dt);
  REQUIRE(ws_bytes >= need, SAS_ERR_INVALID_ARG, "workspace too small: %zu < %zu", ws_bytes, need);
  REQUIRE_PTR(ws);
  sas::TreeArgs a{};
  a.q = q; a.kd = kd; a.vd = vd; a.kc = kc; a.vc = vc; a.ksum = ksum;
  a.parents = parents; a.ntok = ntok; a.lens = lens; a.table = block_table;
  a.o = o;
  a.idx_out = topk > 0 ? idx_out : nullptr;
  a.scale = sas::resolve_scale(scale, d);
  a.B = B; a.Hq = Hq; a.Hkv = Hkv; a.T = T; a.N = N; a.npages = npages;
  a.topk = topk; a.gated = gated;
  return cuda_status(sas::launch_tree(a, dt == SAS_BF16, sum_dt == SAS_BF16, d, ws,
                                      (cudaStream_t)stream),
                     "sas_decode_tree launch");
}

}  // extern "C"
