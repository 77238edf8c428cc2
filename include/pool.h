/*
 * pool.h -- C ABI of libkda_fwd: slots of the state pools that serving steps read (gdn_step,
 * glr_step) copied, forked, freed and compacted on the device.
 *
 * A pool is a device array of `slots` slots of pool_ref.bytes bytes each, one behind the other; the
 * pools of one call (a model's layers) share their slot numbers. `used` is a device array of `slots`
 * bytes: 1 where a slot holds the state of a sequence, 0 where it is free. Free slots that these calls
 * leave are clear (all bytes zero), and a fork overwrites the slot that it takes.
 *
 * Conventions are kda_fwd.h's: nothing is allocated, nothing synchronises, no atomics; every index is
 * read on the device, so that calls can be captured in a graph. Index arrays and `used` must not
 * overlap each other or the pools. Host arrays (pools, sources) are read before the call returns. At
 * most 2^24 slots, 2^24 indices and slots of 2^39 bytes a call; pools need no alignment (16 bytes, and slots of a multiple of
 * 16 bytes, are faster).
 */
#ifndef POOL_H
#define POOL_H

#include <stddef.h>
#include <stdint.h>

#include "kda_fwd.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
    void *data;
    int64_t bytes;            /* of a slot */
} pool_ref;

/* Slot src[i] of the sources becomes slot dst[i] of the pools, for every i < n; src or dst NULL: i
   itself. sources: n_pools pointers to arrays of `source_slots` slots like the pools', or NULL for the
   pools themselves (then source_slots is ignored). A pair with an index outside [0, slots) is skipped.
   No destination may be named twice, nor be another pair's source in the same array (the copies race);
   a pair whose two indices are equal leaves its slot as it is. Sources do not overlap the pools. */
kda_status pool_copy(const pool_ref *pools, int32_t n_pools, int32_t slots, const void *const *sources,
                     int32_t source_slots, const int32_t *src, const int32_t *dst, int64_t n, void *stream);

/* Each i < n whose src[i] is in range (of the sources, as in pool_copy) takes a free slot, in order the
   lowest one left, which becomes used and a copy of slot src[i]; dst[i] is its number. dst[i] is -1
   where src[i] is out of range or no free slot is left; without sources, also where slot src[i] is free.
   src NULL: i itself, or without sources every i takes a slot and nothing is copied (n_pools may be 0).
   dst must not overlap src. */
kda_status pool_fork(const pool_ref *pools, int32_t n_pools, int32_t slots, const void *const *sources,
                     int32_t source_slots, uint8_t *used, const int32_t *src, int32_t *dst, int64_t n,
                     void *stream);

/* The slots that indices [n] name become free, and clear in every pool. An index may be named more than
   once or be out of range (skipped). */
kda_status pool_free(const pool_ref *pools, int32_t n_pools, int32_t slots, uint8_t *used, const int32_t *indices,
                     int64_t n, void *stream);

/* The used slots become slots 0 .. count - 1 of every pool: a used slot >= count moves to a free one
   below it (the i-th lowest of the former to the i-th lowest of the latter), and where it was is clear
   afterwards. indices [n] that name a moved slot are set to its new number, others stay. count: device
   int32 [1]. workspace: pool_compact_workspace_bytes(slots) bytes, 256-byte aligned. */
size_t pool_compact_workspace_bytes(int32_t slots);

kda_status pool_compact(const pool_ref *pools, int32_t n_pools, int32_t slots, uint8_t *used, int32_t *indices,
                        int64_t n, int32_t *count, void *workspace, size_t ws_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* POOL_H */
