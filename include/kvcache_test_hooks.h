/* Test hook of the windowed prompt attention, exported ONLY by the test build
 * (libdropkv_test_hooks.so, compiled with -DDROPKV_TEST_HOOKS: every wait gives
 * up after 10 ms); the product library does not export it.
 */
#ifndef KVCACHE_TEST_HOOKS_H
#define KVCACHE_TEST_HOOKS_H

#include "kvcache.h"

#ifdef __cplusplus
extern "C" {
#endif

/* From the next kvcache_window_attention on, CTA `cta` neither arms nor loads
 * its K/V pair number `pair` (counted over all its items): the pair's barrier
 * never completes, the waits for it run out, the CTA raises
 * DROPKV_FLAG_TIMEOUT, waits (with a limit) for its copies and MMAs in flight,
 * releases its tensor memory and returns; what it did not compute is not
 * written, and the other CTAs finish normally.  (-1, -1) switches the hook
 * off.  Host-synchronous; DROPKV_ERR_CUDA if the copy to the device fails. */
DROPKV_API dropkv_status kvcache_test_skip_window_pair(int32_t cta, int32_t pair);

#ifdef __cplusplus
}
#endif
#endif /* KVCACHE_TEST_HOOKS_H */
