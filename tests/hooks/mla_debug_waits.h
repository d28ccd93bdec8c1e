/*
 * mla_debug_waits.h -- test hooks of the bounded waits that a warp of their own
 * watches (not part of the MLA operation, not in libmla.so).  In the library
 * of mla_debug.h, under the same conventions.
 */
#ifndef MLA_DEBUG_WAITS_H_
#define MLA_DEBUG_WAITS_H_

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* One CTA of four warps.  Warps 0 and 1 wait for a phase that is complete and,
 * if `stall`, for one that never will be; warp 2 then gets on for ten steps of
 * half of limit_ns (at most 1 s); warp 3 watches with that limit.  Warp w
 * writes out[4 w ..]: the nanoseconds until its waits, or its watch, ended;
 * those of its drains after them (warps 0 and 1: of the same two barriers);
 * 1 (the first barrier was there) + 2 (so was the second) + 4 (so it was to
 * the drain, or was not drained); the flag that ends the waits. */
int mla_debug_watched_waits(uint64_t* out, uint64_t limit_ns, int stall, void* stream);

/* mla_document_attention of rows and keys cu[0] .. cu[n_docs] of q [N, 64 * 192],
 * k [64, N, 192] and v [64, N, 128], without prefix or window, with a limit of
 * its waits: limit_ns without a key tile ends them (0: as soon as one is looked
 * at, before the first tile is done).  status: 16 KB, of which word 0 receives
 * the status; plan: 48 bytes for each 128 rows, for each document and once more;
 * first: int [n_docs]. */
int mla_debug_document_attention(const void* q, int N, const int* cu, const void* k, const void* v, int n_docs, void* out,
                                 uint32_t* status, void* plan, int* first, uint64_t limit_ns, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MLA_DEBUG_WAITS_H_ */
