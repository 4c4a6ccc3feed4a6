/*
 * rans_b200_debug.h -- test hooks of librans_b200 (not needed to code).
 *
 * They exercise the library's device-side failure handling without faulting
 * the GPU; the tests call them through the same C ABI as the coders.
 */
#ifndef RANS_B200_DEBUG_H
#define RANS_B200_DEBUG_H

#include <stdint.h>

#include "rans_b200.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Runs the bounded wait of the shared-memory table staging (an mbarrier
 * try-wait with a suspend hint, limited to `limit` tries) on a barrier that
 * expects 16 bytes no copy will deliver, so the wait gives up: the kernel
 * records RANS_ERR_TIMEOUT in the status word of `workspace` (device, >= 256
 * bytes, 256-byte aligned; read it with rans_get_status) and returns,
 * leaving the context usable.  limit must be in [1, 2^21].  Asynchronous.
 */
int rans_debug_wait_timeout(void *workspace, uint32_t limit, void *stream);

/*
 * rans_mxfp4_product whose blocks copy no more than `stages` stages (256 columns
 * each) of the tokens' numbers and wait `limit` tries in place of 2^21: blocks that
 * need more of them give up, record RANS_ERR_TIMEOUT in `status` (required) and return
 * after the copies and products in flight; the context stays usable.  The result is
 * undefined then.  limit must be in [1000, 2^21], out_dtype float32 or bfloat16.
 * Asynchronous.
 */
int rans_debug_product_timeout(const rans_mxfp4 *a, const rans_mxfp4 *head, void *out,
                               int32_t out_dtype, int64_t out_stride, void *status,
                               uint32_t stages, uint32_t limit, void *stream);

#ifdef __cplusplus
}
#endif

#endif
