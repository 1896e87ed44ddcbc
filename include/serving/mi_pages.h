/*
 * mi_pages — the pages of a paged cache on the device: rows of a block table
 * that fork, grow, end and are brought together, for gfx950 (MI355X).  Part of
 * libmi_topk.so.
 *
 * Row i of block_table (int32 [rows][block_table_cols], consecutive rows
 * block_table_stride entries apart) names the pages of one sequence: those of
 * its lengths[i] tokens are its first ceil(lengths[i] / block_size) entries.
 * refs[p] is the number of such entries that name page p; a page with none (0,
 * or less) is free.  A caller may count holders of its own besides.  Full pages
 * may be named by several rows; a row's last page, while it is not full, by that
 * row alone, since kv8_append() writes into it.  One table serves all layers
 * of a model: what is copied is a list of pairs (page, page to copy it to) that
 * pages_copy() works off for each layer's cache.
 *
 * Entries outside [0, num_pages) are pages that are not there: they are handed
 * on as they are and count nowhere.  Lengths count as between 0 and
 * block_table_cols * block_size.  The free pages are taken lowest first, by the
 * lower row first, so that results do not change from run to run.
 *
 * All pointers are device pointers owned by the caller; nothing is allocated or
 * synchronised, all work is enqueued on `stream`, and what the arrays hold is
 * read on the device only.  The workspace of pages_workspace() bytes, 16-byte
 * aligned, need not be cleared; calls that overlap in time need one each.
 * Status codes as in attention/mi_block_attention.h.
 */
#ifndef MI_PAGES_H
#define MI_PAGES_H

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

enum { MI_PAGES_FORK = 0, MI_PAGES_GROW = 1, MI_PAGES_COMPACT = 2 };

/*
 * pages_update(), by `op`:
 *
 * MI_PAGES_FORK: row i becomes a fork of what row parents[i] was before the
 * call, for all rows at once.  parents[i] == i leaves the row as it is; a parent
 * outside [0, rows) ends the row: its length is 0 and its pages are given up.  A
 * fork shares its parent's full pages.  The parent's last page, where it is not
 * full, stays with the parent's own row if that goes on, else with its first
 * fork; each other fork gets a free page (those that this call gives up are
 * free), and copies[i] = (the parent's page, that page), else (-1, -1).  If no
 * page is free copies[i] = (the parent's page, -1) and the row has its full
 * pages' tokens only.  Entries behind the last page of a row that changed are -1.
 *   given: parents int32 [rows]; out: copies int32 [rows][2].
 *
 * MI_PAGES_GROW: room for grow[i] more tokens (none if negative): lengths[i]
 * grows by that and the row gets the pages that it lacks.  A row whose table
 * has not the columns, or for which, with what the rows before it ask for, not
 * enough pages are free, stays as it is.  grown[i] receives by how many tokens
 * the row grew: grow[i] or 0.
 *   given: grow int32 [rows]; out: grown int32 [rows].
 *
 * MI_PAGES_COMPACT: with n pages in use, those from page n on move to the free
 * ones below it, the lowest to the lowest; refs and the rows' entries follow.
 * copies holds the moves in that order and (-1, -1) behind them.
 *   given: not looked at; out: copies int32 [num_pages / 2][2].
 */
typedef struct mi_pages_args {
  int32_t* block_table;
  int32_t* lengths;
  int32_t* refs;
  const int32_t* given;
  int32_t* out;
  void* workspace;
  uint64_t workspace_bytes;
  int64_t num_pages, block_table_stride;
  int32_t rows, block_table_cols, block_size, op;
} mi_pages_args;

uint64_t pages_workspace(const mi_pages_args* args);
int pages_update(const mi_pages_args* args, hipStream_t stream);

/*
 * Copies pages within one layer's 8-bit cache (attention/mi_kv8.h): codes,
 * scales and, where k_mean is not NULL, means.  copies int32 [num][2]: (page,
 * page to copy it to); a pair with an entry outside [0, num_pages) copies
 * nothing.  No page may be copied to twice, nor be copied both from and to.
 */
typedef struct mi_pages_copy_args {
  void* k_cache;
  void* v_cache;
  float* k_scale;
  float* v_scale;
  float* k_mean;
  const int32_t* copies;
  int64_t num, num_pages;
  int32_t kv_heads, dim, block_size;
} mi_pages_copy_args;

int pages_copy(const mi_pages_copy_args* args, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MI_PAGES_H */
