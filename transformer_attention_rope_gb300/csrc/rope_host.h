// rope_host.h -- host-side pieces shared by the entry points that take rows of any strides
// and turn them by positions (cache_host.cu, norm_host.cu).
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "host_common.h"
#include "rope.h"

namespace apex {

inline bool aligned(const void *p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// Whether na bytes at a and nb at b share one (b may be NULL: no).
inline bool overlap(const void *a, size_t na, const void *b, size_t nb)
{
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return b && (x < y ? y - x < na : x - y < nb);
}

// theta_i / (2 pi linear) of d_rot / 2 pairs as 0.64 fixed-point fractions of a turn; false
// when the lock of the sets that are kept cannot be had
bool turns_of(const RopeFreq &f, float linear, int d_rot, uint64_t *out);

// Rows of a tensor: elements at + b * stride[0] + h * stride[1] + s * stride[2] + [0, d).
struct RowSet {
    __int128 at;
    long long stride[3];
    int count[3], d;
};

// Whether two sets of rows share an element (b == &a: whether two rows of a do); layouts that
// would take long to tell count as sharing.
bool share_elements(const RowSet &a, const RowSet &b);

}  // namespace apex
