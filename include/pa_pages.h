/*
 * pa_pages.h — C ABI of the cache-page operators: handing out, sharing,
 * copying, taking back and compacting the pages (cache blocks) that the
 * block_table and slot_mapping of include/pa_latent.h name.
 *
 * The attention entry points read pages through block_table and write rows
 * through slot_mapping; they do not say where either comes from. These calls
 * keep that state on the device, so a serving loop never waits for the host:
 *
 *   block_table int32 [num_seqs, max_blocks_per_seq]  page of each logical
 *               block of a sequence (a row of the table), -1 where there is
 *               none. A row's pages are its first entries.
 *   past        int32 [num_seqs]    cached tokens of each sequence
 *   refcount    int32 [num_blocks]  rows that name a page; 0 = the page is free
 *   caches      any number of paged tensors (one per layer, or a key and a
 *               value cache per layer): page i of a cache is its bytes
 *               [i * page_bytes, (i + 1) * page_bytes), block_size rows of
 *               page_bytes / block_size bytes. All caches share the page ids.
 *
 * Every result is determined by the arguments alone: free pages are handed
 * out lowest id first, in the order of the call's sequences and positions,
 * whatever order the GPU works in.
 *
 * Conventions (pointers, streams, graphs, status codes, err_flags, no
 * allocation, no synchronisation) are those of pa_latent.h. The `caches`
 * array itself is host memory, read during the call. Every call but
 * pa_pages_free takes a workspace of pa_pages_workspace_size bytes, 256-byte
 * aligned, contents arbitrary, not shared with a call that may run at the
 * same time. Calls that touch the same table, refcounts or caches have to be
 * ordered by the caller (one stream, or events), as for any tensor.
 */
#ifndef PA_PAGES_H
#define PA_PAGES_H

#include "pa_latent.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Bits OR-ed into *err_flags, beside those of pa_latent.h. */
#define PA_DEVERR_POOL 0x100 /* no free page left for a sequence or a fork          */
#define PA_DEVERR_PAGE 0x200 /* a named page or sequence is out of range, named twice,
                                free where it has to be held, or held or shared where it
                                has to be free or private                             */

typedef struct pa_pages_params {
  int32_t num_blocks;         /* pages of every cache, 1..2^22; page ids are [0, num_blocks) */
  int32_t block_size;         /* rows per page: power of two >= 16                    */
  int32_t max_blocks_per_seq; /* columns of block_table                               */
  int32_t num_seqs;           /* rows of block_table and past, 1..2^22                */
} pa_pages_params;

/* One paged tensor: 16-byte aligned, page_bytes a positive multiple of
 * 16 * block_size (rows of 16 bytes or a multiple). */
typedef struct pa_pages_cache {
  void* data;
  int64_t page_bytes;
} pa_pages_cache;

pa_status pa_pages_validate(const pa_pages_params* p);

/* Workspace bytes any call with these parameters needs; 0 and an error
 * message for invalid parameters. */
size_t pa_pages_workspace_size(const pa_pages_params* p);

/*
 * Copies pages: cache[dst[i], 0:rows[i]] = cache[src[i], 0:rows[i]] for every
 * pair i and every cache.
 *   src, dst int32 [n]; rows int32 [n] in 0..block_size, or NULL for whole
 *   pages; n in 0..num_blocks.
 * The pairs are independent: a pair whose source is another pair's
 * destination, or whose destination an earlier pair names too, sets
 * PA_DEVERR_PAGE and is skipped, as is one with an index or row count out of
 * range. src[i] == dst[i] copies nothing.
 */
pa_status pa_pages_copy(const pa_pages_params* p, const pa_pages_cache* caches,
                        int32_t num_caches, const int32_t* src, const int32_t* dst,
                        const int32_t* rows, int32_t n, void* workspace, size_t workspace_bytes,
                        int32_t* err_flags, void* stream);

/*
 * Forks sequences: children[i] becomes a copy of parents[i]. The child's row
 * shares the parent's past / block_size full pages (their refcounts rise by
 * one); where past % block_size rows are left, it gets a free page of its own
 * with a copy of those rows in every cache. past[child] = past[parent].
 *   parents, children int32 [n], n in 0..num_seqs.
 * A parent may be forked any number of times in one call. Entry i is skipped
 * and sets PA_DEVERR_PAGE when an index is out of range, an earlier entry
 * names the same child, the child still holds a page, the parent is a child
 * of this call, or a page of the parent is out of range or free; it sets
 * PA_DEVERR_CONTEXT when past[parent] is negative or beyond its row, and
 * PA_DEVERR_POOL when no page is left for its last rows.
 * A beam step that permutes its own rows takes two sets of them: it forks the
 * rows of one set into the empty rows of the other, then frees the first set.
 */
pa_status pa_pages_fork(const pa_pages_params* p, const pa_pages_cache* caches,
                        int32_t num_caches, const int32_t* parents, const int32_t* children,
                        int32_t n, int32_t* block_table, int32_t* past, int32_t* refcount,
                        void* workspace, size_t workspace_bytes, int32_t* err_flags,
                        void* stream);

/*
 * Frees sequences: every page their rows name loses one reference (and is
 * free at 0), the rows become -1 and past 0. Freeing an empty row, or naming
 * a row twice, does nothing more. seqs int32 [n], n in 0..num_seqs.
 * PA_DEVERR_PAGE: a sequence or page out of range, or a page that is free
 * already.
 */
pa_status pa_pages_free(const pa_pages_params* p, const int32_t* seqs, int32_t n,
                        int32_t* block_table, int32_t* past, int32_t* refcount,
                        int32_t* err_flags, void* stream);

/*
 * Reserves the pages of the next tokens: sequence b is about to get
 * cumseq[b + 1] - cumseq[b] new tokens at positions past[b].. Each logical
 * block of those positions that has no page gets a free one, and
 * slot_mapping[t] = page * block_size + position % block_size for every
 * token t: what pa_latent_write, pa_separate_write and pa_diff_write take.
 * past stays as it is (a caller adds the new tokens once they are written).
 *   cumseq int32 [num_seqs + 1] as in pa_latent.h; slot_mapping int32
 *   [num_tokens].
 * A sequence gets all of its pages or none. It gets them while the needs of
 * the sequences up to it fit in the free pages; the others set PA_DEVERR_POOL
 * and their slots are -1, as are those of a sequence whose positions lie
 * outside its row (PA_DEVERR_CONTEXT), whose cumseq entries decrease or pass
 * num_tokens (PA_DEVERR_CUMSEQ), or that would write into a page that is out
 * of range, free or shared (PA_DEVERR_PAGE): those take no page and count for
 * no need. Tokens behind cumseq[num_seqs] get slot -1.
 */
pa_status pa_pages_reserve(const pa_pages_params* p, const int32_t* cumseq, int64_t num_tokens,
                           int32_t* block_table, const int32_t* past, int32_t* refcount,
                           int32_t* slot_mapping, void* workspace, size_t workspace_bytes,
                           int32_t* err_flags, void* stream);

/*
 * Compacts the pool: with L pages held, the k-th held page at or above L
 * moves to the k-th free page below L (its rows in every cache, its refcount
 * and every table entry that names it), so that the held pages are [0, L).
 *   live int32 [1] receives L (may be NULL).
 * A table entry that names a free page or none of the pool becomes -1 and
 * sets PA_DEVERR_PAGE.
 */
pa_status pa_pages_compact(const pa_pages_params* p, const pa_pages_cache* caches,
                           int32_t num_caches, int32_t* block_table, int32_t* refcount,
                           int32_t* live, void* workspace, size_t workspace_bytes,
                           int32_t* err_flags, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* PA_PAGES_H */
