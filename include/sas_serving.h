/*
 * sas_serving.h -- the calls around the attention of sas.h: rotary positions,
 * page tables, the cache write and attention of drafted tokens (libsas.so,
 * CUDA kernels for sm_100a).
 *
 * A serving step with drafted tokens, over a paged cache:
 *   sas_rotary        q and k of the drafted tokens, at their tree positions
 *   sas_decode_tree   their attention over the cache and their ancestors
 *   sas_page_map      pages and slots for the tokens that were accepted
 *   sas_cache_append  their k and v into the pages, with the summaries of the
 *                     blocks that they complete
 * A plain decode step is sas_page_map, sas_cache_append (which rotates q
 * beside k) and sas_decode_paged; training rotates q and k with sas_rotary
 * before sas_select and sas_attn_fwd, and their gradients after sas_attn_bwd.
 *
 * The conventions of sas.h hold (device pointers of the caller, no allocation
 * and no synchronisation, 16-byte alignment, host-side checks before any
 * launch, calls may be captured in a CUDA graph). Numbers that live on the
 * device (lengths, parents, page ids, slots) cannot be checked on the host:
 * the kernels bound every one of them before they use it, report one that is
 * out of range through sas_device_status, and leave out what it named, as each
 * call says.
 */
#ifndef SAS_SERVING_H
#define SAS_SERVING_H

#include "sas.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Rotary positions of q and k in one launch, forward and backward. The pages
 * apply them inside the model that calls the attention (SAS close reading,
 * section 3.1); here they are a call of their own. Pair p of a head,
 * 0 <= p < rot/2, turns by theta = position * inv_freq[p]:
 *   y0 = A (x0 cos theta - x1 sin theta), y1 = A (x1 cos theta + x0 sin theta)
 * with (x0, x1) = elements (p, p + rot/2) of the head, or (2p, 2p + 1) when
 * interleaved = 1, and A = amplitude. Elements from rot on are passed through.
 * inverse = 1 turns by -theta: with the same A it is the transpose, so it
 * takes dy to dx. theta is exact to 4e-17 inv_freq + 6e-20 turns a position (no
 * fp32 product; 4e-11 turns at 2^20 positions and 1 radian a position); a long
 * context is set by inv_freq and A.
 *   q [B][Hq][N][d] (dt), k [B][Hkv][N][d] or NULL (with Hkv = 0), read
 *     through element strides {batch, head, token}; qo, ko likewise. A stride
 *     pointer (host memory, three values) of NULL means contiguous. Rows of d
 *     elements are contiguous. Input strides may be 0 (shared rows), output
 *     rows must not overlap; qo = q with equal strides rotates in place, any
 *     other overlap of an output with an input or with the other output is
 *     refused (by address; rows of one buffer may alternate if strides agree).
 *   inv_freq [rot/2] fp32, radians per position (an entry that is not finite
 *     turns its pair to NaN); rot even, 2 <= rot <= d
 *   pos [B][N] int32: the positions; or NULL, then position = start[b]
 *     (start [B] int32, NULL = 0) + n, or + the depth of token n when
 *     parents [B][N] int32 is given (the tree of sas_decode_tree: a parent is
 *     below its child, -1 has depth 0; another entry is reported and read
 *     as -1; N <= 1024 then, since every token walks up its path). Positions
 *     are int32: start + n has to stay below 2^31
 *   d in {64, 128}; B <= 65535
 */
sas_status sas_rotary(const void* q, const int64_t* q_strides, void* qo,
                      const int64_t* qo_strides, int Hq, const void* k, const int64_t* k_strides,
                      void* ko, const int64_t* ko_strides, int Hkv, sas_dtype dt, int B, int N,
                      int d, const float* inv_freq, int rot, int interleaved, float amplitude,
                      int inverse, const int32_t* pos, const int32_t* start,
                      const int32_t* parents, sas_stream_t stream);

/*
 * Block tables and slot maps from request lengths, for caches in pages of 64
 * tokens. Sequence b holds lens[b] tokens in its first ceil(lens[b]/64) table
 * entries and receives nnew[b] <= T more. The new pages it needs come from
 * free_pages[free_head ...], in the order of the sequences, into the next
 * entries of its row of the table; the others of the row are left as they
 * were.
 *   lens, nnew     [B] int32
 *   block_table    [B][width] int32, in and out
 *   free_pages     [nfree] int32; free_head [1] int32, how many are used up
 *   slots          [B][T] int32, out: 64 page + row of each new token, -1 from
 *                  token nnew[b] on
 *   new_lens       [B] int32, out: lens + nnew; may be lens itself
 *   taken          [B] int32, out: pages taken, -1 where refused
 *   head_out       [1] int32, out: free_head + all pages taken; may be
 *                  free_head itself
 * A sequence is refused, and keeps its length, table row and slots of -1, when
 * its pages would end past the list (the need of an earlier refused sequence
 * counts, so the order decides) or when its numbers are impossible (negative,
 * nnew > T, more than 64 width tokens). A page id outside [0, npages) is
 * written as listed, gives slots of -1 and is reported.
 *   npages <= 2^25; B <= 65534, B (T + 128) < 2^31. No workspace. No array that
 *   is written may overlap another, but for new_lens = lens and head_out =
 *   free_head (checked).
 */
sas_status sas_page_map(const int32_t* lens, const int32_t* nnew, int32_t* block_table,
                        const int32_t* free_pages, const int32_t* free_head, int B, int T,
                        int width, int npages, int nfree, int32_t* slots, int32_t* new_lens,
                        int32_t* taken, int32_t* head_out, sas_stream_t stream);

/*
 * Cache write of new tokens, with the summaries of the blocks they complete:
 * what sas_decode and sas_decode_paged expect of a cache. Token j of sequence
 * b, j < ntok[b], takes row j of k and v (or row rows[b][j]), has position
 * lens[b] + j, and
 *   its k, rotated at that position when inv_freq is given (as sas_rotary with
 *   rot, interleaved, amplitude), and its v are written to
 *     kc, vc [B][Hkv][N][d] at that position (slots NULL), or to
 *     kc, vc [npages][Hkv][64][d] at slots[b][j] (as sas_page_map writes them;
 *     -1 leaves the token out);
 *   when the last row of a 64-token block is written and ksum is given, the
 *   mean of the block's 64 stored keys goes to ksum [B][Hkv][N/64][d], or
 *   [npages][Hkv][d], of type sum_dt (summed in fp32 and rounded once, as
 *   sas_block_summary does, but in another order, which also depends on types
 *   and strides: the last bits may differ; a block with a token left out in
 *   this call keeps its summary);
 *   q [B][Hq][T][d], when given, is rotated at the same positions into
 *   qo [B][Hq][T][d] (contiguous), all its rows.
 *   k, v [B][Hkv][T][d] and q are read through element strides {batch, head,
 *     token} (host memory, NULL = contiguous), as in sas_rotary
 *   lens [B], the lengths before; ntok [B] or NULL (T everywhere); rows [B][T]
 *     or NULL (a row may be named twice). q needs inv_freq and no rows.
 *   N a multiple of 64 (0 with slots). A token past N, a row outside [0, T)
 *     or a slot below -1 or in a page past npages is left out and reported, as
 *     is a sequence with lens < 0 or ntok outside [0, T] (its rows of qo too),
 *     or with lens + T past 2^31 - 1. T <= 2^30.
 * Slots of two tokens must differ. k and v must not lie in the cache, nor qo in
 * anything but q (qo = q, contiguous, rotates in place): tokens are moved in any
 * order. Refused by their addresses. No workspace.
 */
sas_status sas_cache_append(const void* q, const int64_t* q_strides, void* qo, const void* k,
                            const int64_t* k_strides, const void* v, const int64_t* v_strides,
                            sas_dtype dt, int B, int Hq, int Hkv, int T, int d,
                            const int32_t* rows, const int32_t* lens, const int32_t* ntok,
                            const float* inv_freq, int rot, int interleaved, float amplitude,
                            const int32_t* slots, void* kc, void* vc, int N, int npages,
                            void* ksum, sas_dtype sum_dt, sas_stream_t stream);

/*
 * Decode of a tree of drafted tokens (SAS close reading, section 2.4, serving
 * path, for several query tokens a sequence). Drafted token i of sequence b
 * has parent parents[b][i] < i (-1: the last cached token), depth = number of
 * ancestors, position lens[b] + depth, and gets what sas_decode gives on a
 * cache with the path from the root to it appended, up to the rounding of fp32
 * sums in another order (scores that nearly tie may select another block): its
 * own Top-K row over
 * the (lens[b] + depth)/64 history blocks, gate, and attention over the kept
 * blocks, the current block's tokens and its ancestors. Where a path fills the
 * block of the cache's tail, that block is history for the tokens past it,
 * with the summary of its 64 keys (rounded to sum_dt).
 *   q [B][Hq][T][d], kd, vd [B][Hkv][T][d] (dt): the drafted tokens, 1 <= T <= 64
 *   kc, vc, ksum: the cache and its summaries (sum_dt), [B][Hkv][N][d] and
 *     [B][Hkv][N/64][d] (block_table NULL), or pools [npages][Hkv][64][d] and
 *     [npages][Hkv][d] with block_table [B][N/64]; cached rows from lens[b] on
 *     are not read into any result
 *   lens [B] int32, 0 <= lens[b] <= N: the cached tokens, the drafted ones not
 *     among them; summaries of all lens[b]/64 whole blocks are expected
 *   ntok [B] int32 or NULL: drafted tokens of each sequence (0 .. T)
 *   parents [B][T] int32 or NULL: a chain (parent i - 1)
 *   topk, gated, scale as sas_decode
 *   o [B][Hq][T][d] (dt); idx_out [B][Hkv][T][topk] int32 or NULL, logical
 *     blocks, ascending, -1 padded. Rows from ntok[b] on are left as they were.
 * Reported and left out: a sequence with lens outside [0, N] or ntok outside
 * [0, T] (all its rows stay as they were); a block whose page is outside
 * [0, npages) (unlike in sas_decode_paged, no other page is read in its place:
 * its score is -inf and none of its keys is attended to, also where it is the
 * partly filled last one, and where a path fills that, the path's keys in it
 * likewise; idx_out lists it where fewer than topk blocks score higher). A
 * parent that is not below its child is reported and read as -1.
 * N a positive multiple of 64, at most 2^20; at most 8 query heads a kv head.
 * Workspace: sas_decode_tree_workspace_size() bytes.
 */
size_t sas_decode_tree_workspace_size(int B, int Hq, int Hkv, int T, int N, int d, int topk,
                                      sas_dtype dt);
sas_status sas_decode_tree(const void* q, const void* kd, const void* vd, const void* kc,
                           const void* vc, sas_dtype dt, int B, int Hq, int Hkv, int T, int N,
                           int d, const int32_t* parents, const int32_t* ntok,
                           const int32_t* lens, const void* ksum, sas_dtype sum_dt,
                           const int32_t* block_table, int npages, int topk, int gated,
                           float scale, void* o, int32_t* idx_out, void* ws, size_t ws_bytes,
                           sas_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* SAS_SERVING_H */
