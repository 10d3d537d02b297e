// api_checks.hpp -- argument checks and the launch report that the entry
// points share (api.hip, api_block.hip).
#pragma once

#include <stdint.h>
#include <stdio.h>

#include "rx.h"
#include "rx_internal.hpp"

namespace rx {
namespace {

constexpr size_t kMaxCount = (size_t)1 << 38;  // elements per buffer

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
bool aligned4(const void* p) { return ((uintptr_t)p & 3u) == 0; }
bool hp_type(rx_dtype_t t) { return t == RX_FP32 || t == RX_BF16; }
bool fp8_type(rx_dtype_t t) { return t == RX_FP8_E4M3 || t == RX_FP8_E5M2; }
bool valid_block(int b) { return b >= 32 && b <= 1024 && (b & (b - 1)) == 0; }

// A failed launch is always reported on stderr with the HIP error's name.
rx_status_t launched(hipError_t e)
{
    if (e == hipSuccess)
        return RX_OK;
    fprintf(stderr, "librx: launch failed: %s (%s)\n", hipGetErrorName(e), hipGetErrorString(e));
    return RX_ERR_HIP;
}

// Shared checks of a source-pointer array: NULL array / entries, alignment.
rx_status_t check_ptrs(const void* const* p, int n, bool align16)
{
    if (!p)
        return RX_ERR_NULL;
    for (int j = 0; j < n; ++j)
        if (!p[j])
            return RX_ERR_NULL;
    for (int j = 0; j < n; ++j)
        if (align16 ? !aligned16(p[j]) : !aligned4(p[j]))
            return RX_ERR_ALIGN;
    return RX_OK;
}

}  // namespace
}  // namespace rx
