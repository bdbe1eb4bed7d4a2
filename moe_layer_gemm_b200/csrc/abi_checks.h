// Argument checks shared by the files that implement the C ABI.
#pragma once
#include <cmath>
#include <cstddef>
#include <cstdint>

#include "../../include/moe_b200.h"

namespace moe {

constexpr int64_t kMaxT = int64_t(1) << 24;

inline size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline int check_dims(const moe_dims* d) {
    if (!d) return MOE_EINVAL;
    if (d->T < 1 || d->T > kMaxT) return MOE_EINVAL;
    if (d->E < 1 || d->E > 256) return MOE_EINVAL;
    if (d->K < 1 || d->K > d->E || d->K > 16) return MOE_EINVAL;
    if (d->d_model < 16 || d->d_ff < 16) return MOE_EINVAL;
    if (d->d_model > (1 << 16) || d->d_ff > (1 << 17)) return MOE_EINVAL;
    if (d->d_model % 16 != 0 || d->d_ff % 16 != 0) return MOE_EUNSUPPORTED;
    if (std::isnan(d->capacity_factor)) return MOE_EINVAL;
    return MOE_OK;
}

// Status of an internal launch function's result (0, -2: shape, else CUDA).
inline int map_launch(int r) {
    if (r == 0) return MOE_OK;
    if (r == -2) return MOE_EUNSUPPORTED;
    return MOE_ECUDA;
}

#define MOE_TRY(expr)               \
    do {                            \
        int _s = (expr);            \
        if (_s != MOE_OK) return _s; \
    } while (0)

}  // namespace moe
