/* Test hook of the shared attention, exported ONLY by the test build
 * (libdropkv_test_hooks.so, compiled with -DDROPKV_TEST_HOOKS: every wait gives
 * up after 10 ms); the product library does not export it.
 */
#ifndef KVCACHE_STEP_TEST_HOOKS_H
#define KVCACHE_STEP_TEST_HOOKS_H

#include "kvcache_step.h"

#ifdef __cplusplus
extern "C" {
#endif

/* From the next kvcache_shared_attention on, CTA `cta` of the shared tokens'
 * kernel neither arms nor makes its load number `load` (2 i: K's codes of its
 * tile i, 2 i + 1: V's): the waits for it run out, the CTA raises
 * DROPKV_FLAG_TIMEOUT, waits (with a limit) for its copies and MMAs in flight,
 * releases its tensor memory and returns; the rows of the heads it had tiles
 * of are undefined, the others are whole.  (-1, -1) switches the hook off.
 * Host-synchronous; DROPKV_ERR_CUDA if the copy to the device fails. */
DROPKV_API dropkv_status kvcache_test_skip_shared_load(int32_t cta, int32_t load);

#ifdef __cplusplus
}
#endif
#endif /* KVCACHE_STEP_TEST_HOOKS_H */
