// Launches of attention with a bias, from positions (fpstok_attention_bias.hip)
// or from the plane of entries (fpstok_attention_plane.hip).
#pragma once

#include "fpstok_attention_kernels.h"

namespace fpstok {

// The sum of the row tiles' parts of the table's gradient.
void launch_bias_table(const BiasArgs& b, const AttnArgs& a, int tiles, hipStream_t s);
hipError_t launch_plane(const AttnArgs& a, const BiasArgs& b, const AttnPlan& plan, hipStream_t s);
hipError_t launch_plane_backward(const AttnArgs& a, const BiasArgs& b, hipStream_t s);

template <class T, BiasFrom FROM>
static hipError_t backward(const AttnArgs& a, BiasArgs b, hipStream_t s) {
    const bool rows = a.qs.rows > 0;
    if (!b.grad) {
        b.part = nullptr;
        if (rows) backward_q<T, FROM>(a, b, s);
    } else {
        // more than kTableEntries entries: a walk for each part of them
        const int tiles = rows ? (int)row_slots(a.qs, a.G, 7) : 0;
        for (b.from = 0; b.from < b.entries; b.from += b.count) {
            const int left = b.entries - b.from;
            b.count = left < kTableEntries ? left : kTableEntries;
            if (rows) backward_q<T, FROM>(a, b, s);
            launch_bias_table(b, a, tiles, s);
        }
    }
    backward_kv<T, FROM>(a, b, s);
    return hipGetLastError();
}

template <BiasFrom FROM>
static hipError_t launch(const AttnArgs& a, const BiasArgs& b, const AttnPlan& plan,
                         hipStream_t s) {
    return a.dtype == 0   ? forward<float, FROM>(a, b, plan, s)
           : a.dtype == 1 ? forward<_Float16, FROM>(a, b, plan, s)
                          : forward<__bf16, FROM>(a, b, plan, s);
}

template <BiasFrom FROM>
static hipError_t launch_backward(const AttnArgs& a, const BiasArgs& b, hipStream_t s) {
    return a.dtype == 0   ? backward<float, FROM>(a, b, s)
           : a.dtype == 1 ? backward<_Float16, FROM>(a, b, s)
                          : backward<__bf16, FROM>(a, b, s);
}

}  // namespace fpstok
