// gdn_granules.h -- copying a piece of an unaligned row as the 16-byte granules that hold it
// (plain C++, so that the host can check which bytes it reads).
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define GDN_HD __host__ __device__ __forceinline__
#else
#define GDN_HD inline
#endif

namespace gdn {

// The elements E at addresses [row, end) of a tensor that lies in [lo, hi), by the granules
// first, first + STEP, ... of those that hold them (at most TRIPS of these): copy(offset, bytes)
// for `bytes` bytes of the granule `offset` bytes behind the first one, one(offset) for a single
// element.  Nothing outside [lo, hi) is read: the granule that reaches past hi is cut short, and
// the elements of one that begins ahead of lo go one by one.  (Both are rare: the tensor's first
// and last few elements.)
template <typename E, int STEP, int TRIPS, typename Copy, typename One>
GDN_HD void copy_granules(uintptr_t row, uintptr_t end, uintptr_t lo, uintptr_t hi, int first,
                          const Copy& copy, const One& one) {
    const uintptr_t from = row & ~(uintptr_t)15;
    const int n = (int)(end - from);
    const uintptr_t left = hi - from;
    const int rest = left < 4096 ? (int)left : 4096;  // (more than a row's granules)
#ifdef __CUDACC__
#pragma unroll
#endif
    for (int k = 0; k < TRIPS; ++k) {
        const int o = (first + k * STEP) * 16;
        if (o >= n) continue;
        if (k == 0 && first == 0 && from < lo) {
            for (int i = (int)(row - from); i < n && i < 16; i += (int)sizeof(E)) one(i);
        } else {
            copy(o, rest - o < 16 ? rest - o : 16);
        }
    }
}

}  // namespace gdn
