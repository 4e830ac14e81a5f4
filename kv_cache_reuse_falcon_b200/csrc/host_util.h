// Host-side checks and device queries shared by the library's entry points.
#pragma once

#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "unipin.h"

namespace unipin {

constexpr int kNumSmsHint = 148;   // B200
constexpr int kMaxDevices = 64;

inline int g_num_sms[kMaxDevices] = {};

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// SM count of the current device (queried once per device; the B200 count if
// the query fails, e.g. on a machine without a device).
inline int current_sms()
{
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return kNumSmsHint;
    if (g_num_sms[dev] > 0) return g_num_sms[dev];
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) return kNumSmsHint;
    g_num_sms[dev] = n;
    return n;
}

// The pool's heads are key/value heads: H (query heads) must be a multiple of them.
inline int check_pool(const unipin_kvpool* pool, int H, int D, int layer)
{
    if (!pool || !pool->k || !pool->v) return UNIPIN_ERR_INVALID_ARG;
    if (pool->L < 1 || pool->S < 1 || pool->n_cap < 1 || pool->H < 1 || H % pool->H != 0 || pool->D != D)
        return UNIPIN_ERR_INVALID_ARG;
    if (pool->dtype != UNIPIN_POOL_BF16 && pool->dtype != UNIPIN_POOL_E4M3) return UNIPIN_ERR_INVALID_ARG;
    if (pool->dtype == UNIPIN_POOL_E4M3 &&
        (!(pool->k_scale > 0.f) || !std::isfinite(pool->k_scale) || !(pool->v_scale > 0.f) ||
         !std::isfinite(pool->v_scale) || !std::isfinite(1.f / pool->k_scale) || !std::isfinite(1.f / pool->v_scale)))
        return UNIPIN_ERR_INVALID_ARG;
    if (!aligned16(pool->k) || !aligned16(pool->v)) return UNIPIN_ERR_MISALIGNED;
    if (layer < 0 || layer >= pool->L) return UNIPIN_ERR_OUT_OF_RANGE;
    if ((uint64_t)pool->L * pool->S * pool->H >= (1ull << 31)) return UNIPIN_ERR_INVALID_ARG;
    return UNIPIN_OK;
}

inline bool supported_d(int D) { return D == 32 || D == 64 || D == 128; }

}  // namespace unipin
