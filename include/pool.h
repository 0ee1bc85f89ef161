/*
 * Pools of states -- slots taken, copied, forked, compacted and freed on the
 * device, for the pools that gdr_decode_step and glr_decode_step update in
 * place, in the same library.
 *
 * C ABI.  Plain pointers and sizes; no C++ or framework types cross it.
 *
 * A pool is n_slots rows of row_bytes bytes each, back to back in device
 * memory: pool p's slot j is the bytes base + j row_bytes.  A server has one
 * for each layer (and one more for whatever else a request carries, such as
 * the last tokens' window of a short convolution), all with the same slots:
 * request state j is slot j of every pool.  The calls take any number of
 * pools at once, of any element type.
 *
 * Which slots are taken is held in `used` [n_slots], one byte a slot, 0 for
 * a free one.  It lives in device memory and the calls read and update it on
 * their stream: a server can queue forks, frees and steps one after another
 * without asking the device which slots they got.  A recurrent state is
 * rewritten by its next token, so a fork is a copy; nothing is shared and
 * there is nothing to count.
 *
 * Ownership, errors and concurrency are those of kda.h: the caller owns
 * every buffer, nothing is allocated or synchronised, argument problems are
 * reported as a kda_status (kda_last_error has the message) before anything
 * is launched.  Slot numbers in device memory that lie outside the pool are
 * ignored as said at each call and never change the addresses touched.
 * Calls that touch the same pools, `used` or tables must be ordered by the
 * caller (one stream does).
 *
 * Sizes: 0 <= n_slots, n, n_table <= 2^24 each; 0 <= n_pools; 1 <= row_bytes <= 2^40;
 * n_slots row_bytes below 2^46.  Alignment: int32 arrays 4 bytes, pools 1.
 * (Rows are moved 16 bytes at a time where bases and row_bytes allow, else 4
 * or 1.)  Workspaces: 256 bytes.
 */
#ifndef POOL_H
#define POOL_H

#include "kda.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct pool_rows {
    void *base;       /* n_slots * row_bytes bytes of device memory */
    size_t row_bytes;
} pool_rows;

/*
 * pool_copy -- slot src[i] of each of `from` to slot dst[i] of its counterpart
 * in `to`, for i < n: states kept for later (a prompt's, at its end), or
 * brought back.  from[p] and to[p] have rows of one size; they may be the
 * same pools, or others with another number of slots.  A pair with a number
 * outside its pools is left out.  A destination named twice, or named as
 * another pair's source in the same pools, gets a mixture of the bytes it
 * could have; no other memory is touched.
 */
kda_status pool_copy(const pool_rows *from, const pool_rows *to, int32_t n_pools,
                     int32_t from_slots, int32_t to_slots, const int32_t *src, const int32_t *dst,
                     int32_t n, kda_stream_t stream);

/*
 * pool_alloc -- takes n free slots, lowest numbers first, for new requests:
 * slots[i] becomes the i-th lowest free slot, its rows are written with zeros
 * and it is marked as used; -1 where no free slot is left.
 */
kda_status pool_alloc(const pool_rows *pools, int32_t n_pools, uint8_t *used, int32_t n_slots,
                      int32_t n, int32_t *slots, kda_stream_t stream);

/*
 * pool_fork -- takes a free slot for a copy of each src[i]: dst[i] becomes the
 * lowest free slot that no earlier row got, its rows a copy of slot src[i]'s
 * in every pool, and it is marked as used.  The same source may be named any
 * number of times.  Where src[i] is no used slot (as at the call's start; any
 * number outside the pool counts as none), or no free slot is left, dst[i] is
 * -1 and nothing is copied.
 */
kda_status pool_fork(const pool_rows *pools, int32_t n_pools, uint8_t *used, int32_t n_slots,
                     const int32_t *src, int32_t n, int32_t *dst, kda_stream_t stream);

/*
 * pool_free -- marks slots[i], i < n, as free.  Numbers outside the pool and
 * slots that are free already are ignored; the rows keep their bytes until
 * they are taken again.
 */
kda_status pool_free(uint8_t *used, int32_t n_slots, const int32_t *slots, int32_t n,
                     kda_stream_t stream);

/*
 * pool_compact -- moves used slots to the front, so that the pool can be cut
 * down or the steps run over a shorter one.  With m used slots, those at m and
 * behind move, in order, into the free slots below m; used becomes 1 below m
 * and 0 behind.  remap [n_slots] gets each used slot's new number and -1 for a
 * free one; every entry of table [n_table] (NULL iff n_table is 0) that is a
 * slot number is rewritten through it (to -1 where it named a free slot), and
 * entries outside the pool stay.  The bytes of slots that end up free are
 * left as they were.  The workspace holds pool_compact_workspace_bytes bytes.
 */
size_t pool_compact_workspace_bytes(int32_t n_slots);
kda_status pool_compact(const pool_rows *pools, int32_t n_pools, uint8_t *used, int32_t n_slots,
                        int32_t *table, int64_t n_table, int32_t *remap, void *workspace,
                        size_t workspace_bytes, kda_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* POOL_H */
