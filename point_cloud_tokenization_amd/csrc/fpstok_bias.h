// A learned bias of the scores by buckets of the rows' distance, for the
// attention kernels: per axis a of up to four,
//   D = x_key - x_query,  linear: clamp(floor(D + shift), 0, n - 1),
//   log: clamp(shift + sign(D) L, 0, n - 1), L = floor(g (E + F)) of
//        1 + |D| = 2^E (1 + F),
// each float32 operation rounded by itself, and the score gets table[head]
// [first[a] + bucket].  For g a power of two, L is 1 + |D|'s bits less those of
// 1.0, shifted: exponent and leading bits of the fraction.
#pragma once

#include <type_traits>

#include "fpstok_attention.h"
#include "fpstok_mma.h"

namespace fpstok {

// Where a kernel's scores get their bias from.
enum BiasFrom {
    kNoBias,
    kPositions,  // every head finds the pairs' entries itself
    kPlane       // they were found once for all heads (bias_plane_kernel)
};
struct NoBias {};
template <BiasFrom BIAS>
using BiasParam = std::conditional_t<BIAS != kNoBias, BiasArgs, NoBias>;

// Positions of a tile's rows in LDS, and of the rows across the lanes: float32
// times the axis's rate, or the int32 as they are.  [axis][row]; `span`: the least
// and the greatest of a wave's own 32 rows.
template <BiasFrom BIAS, int OWN, int ROWS>
struct BiasPos {
    uint32_t own[kMaxAxes][OWN];
    uint32_t tile[2][kMaxAxes][ROWS];
    uint32_t span[OWN / 32][kMaxAxes][2];
};
template <int OWN, int ROWS>
struct BiasPos<kNoBias, OWN, ROWS> {};

// The element of a small array in registers at a place that is the same in
// every lane.
template <class V>
__device__ __forceinline__ V pick(const V (&v)[kMaxAxes], int a) {
    return a == 0 ? v[0] : a == 1 ? v[1] : a == 2 ? v[2] : v[3];
}

// Positions of a tile's ROWS rows on their way to LDS, by THREADS threads.
template <int ROWS, int THREADS>
struct PosStage {
    static constexpr int kPer = ROWS * kMaxAxes > THREADS ? ROWS * kMaxAxes / THREADS : 1;
    uint32_t x[kPer];
    int row[kPer], axis[kPer];
    float rate[kPer];
    __device__ __forceinline__ PosStage(const BiasArgs& b, int tid) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int at = tid + i * THREADS;
            row[i] = (int)((uint32_t)at / (uint32_t)b.axes);
            axis[i] = at - row[i] * b.axes;
            rate[i] = pick(b.rate, axis[i]);
        }
    }
    // Rows at or past `rows` (at least 1) hold the last one's.
    __device__ __forceinline__ void load(const BiasArgs& b, const void* pos, int64_t row0,
                                         int rows) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int r = row[i] < rows ? row[i] : rows - 1;
            x[i] = ((const uint32_t*)pos)[(row0 + r) * b.axes + axis[i]];
        }
    }
    __device__ __forceinline__ void store(const BiasArgs& b, uint32_t (*tile)[ROWS]) const {
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (row[i] < ROWS)
                tile[axis[i]][row[i]] =
                    b.ints ? x[i] : __float_as_uint(__uint_as_float(x[i]) * rate[i]);
    }
};

// A position as a whole number of the same order, and back.
__device__ __forceinline__ int ordered(uint32_t x, bool ints) {
    return ints ? (int)x : (int)(x ^ ((uint32_t)((int)x >> 31) & 0x7fffffffu));
}
__device__ __forceinline__ uint32_t position(int x, bool ints) {
    return (uint32_t)ordered((uint32_t)x, ints);
}

// The least and the greatest over 32 lanes, the two halves of a wave alike.
__device__ __forceinline__ void span_of(int x, int& least, int& most) {
    least = most = x;
    auto step = [&](auto ctrl) {
        constexpr int kCtrl = decltype(ctrl)::value;
        const int a = __builtin_amdgcn_update_dpp(0, least, kCtrl, 0xf, 0xf, true);
        const int b = __builtin_amdgcn_update_dpp(0, most, kCtrl, 0xf, 0xf, true);
        least = a < least ? a : least;
        most = b > most ? b : most;
    };
    step(std::integral_constant<int, 0xb1>{});   // lanes l ^ 1
    step(std::integral_constant<int, 0x4e>{});   // l ^ 2
    step(std::integral_constant<int, 0x141>{});  // 7 - l % 8
    step(std::integral_constant<int, 0x140>{});  // 15 - l % 16
    const auto a = __builtin_amdgcn_permlane16_swap(least, least, false, false);
    const auto b = __builtin_amdgcn_permlane16_swap(most, most, false, false);
    least = (int)a[0] < (int)a[1] ? (int)a[0] : (int)a[1];
    most = (int)b[0] > (int)b[1] ? (int)b[0] : (int)b[1];
}

// Positions of the rows across a wave's lanes (lanes 0-31 write): row `row` of
// the buffer, or, not `live`, the first lane's (if that is not either, row 0).
template <int OWN>
__device__ __forceinline__ void own_positions(const BiasArgs& b, uint32_t (*own)[OWN],
                                              uint32_t (*span)[2], int at, const void* pos,
                                              int64_t row, bool live, int half) {
    const int first = __builtin_amdgcn_readfirstlane(live ? (int)row : 0);
#pragma unroll
    for (int a = 0; a < kMaxAxes; ++a) {
        if (a >= b.axes) break;
        uint32_t x = ((const uint32_t*)pos)[(live ? row : first) * b.axes + a];
        if (!b.ints) x = __float_as_uint(__uint_as_float(x) * b.rate[a]);
        if (half == 0) own[a][at] = x;
        int least, most;
        span_of(ordered(x, b.ints), least, most);
        if ((threadIdx.x & 63) == 0)
            span[a][0] = position(least, b.ints), span[a][1] = position(most, b.ints);
    }
}

// LDS that the launch adds to a kernel's own: the tables, then the sums of
// their gradients.
__device__ __forceinline__ float* bias_lds() {
    extern __shared__ __attribute__((aligned(256))) float fpstok_bias_lds[];
    return fpstok_bias_lds;
}
// Places of a row's sums: an entry each, and one that nobody reads for entries of
// another launch and for the half of a wave that has no axis.
__host__ __device__ inline int table_slots(const BiasArgs& b) {
    return b.count + (b.count != b.entries || (b.axes & 1) != 0);
}
// Values of one head's tables: an entry each, or (JOINT) two axes' sums.
__host__ __device__ inline int table_size(const BiasArgs& b, bool joint) {
    return joint ? b.joint[0] + b.joint[1] : b.entries;
}
inline size_t bias_lds_bytes(const BiasArgs& b, int G, bool joint, bool sums) {
    const size_t table = ((size_t)G * table_size(b, joint) + 63) & ~(size_t)63;
    return (table + (sums ? (size_t)4 * table_slots(b) * 64 : 0)) * sizeof(float);
}

using u32x16 = uint32_t __attribute__((ext_vector_type(16)));

// The bucket of a distance, from the own row's and another's position as they
// are in LDS.
template <bool INTS, bool LOG>
__device__ __forceinline__ int bucket_of(uint32_t k, uint32_t q, float rate, float zero, int top,
                                         int shift) {
    float d;
    if constexpr (INTS)
        d = (float)(int)(k - q) * rate;
    else
        d = __uint_as_float(k) - __uint_as_float(q);
    if constexpr (LOG) {
        const int steps = (int)((__float_as_uint(1.0f + fabsf(d)) - 0x3f800000u) >> shift);
        const int sign = (int)__float_as_uint(d) >> 31;
        const int bucket = (steps ^ sign) + ((int)zero - sign);
        return bucket < 0 ? 0 : bucket > top ? top : bucket;
    }
    // (0 where d is not a number)
    return (int)__builtin_amdgcn_fmed3f(d + zero, 0.0f, (float)top);
}

// Calls f(INTS, LOG) with what an axis is.
template <class F>
__device__ __forceinline__ void by_kind(bool ints, bool log, F f) {
    if (ints) {
        if (log)
            f(std::true_type{}, std::true_type{});
        else
            f(std::true_type{}, std::false_type{});
    } else {
        if (log)
            f(std::false_type{}, std::true_type{});
        else
            f(std::false_type{}, std::false_type{});
    }
}

// The same from the pairs' entries as they are in the plane (JOINT) or its bytes.
template <bool JOINT>
__device__ __forceinline__ void add_entries(f32x16& s, const u32x16& entries, int axes,
                                            const FPSTOK_LDS float* table) {
    const FPSTOK_LDS char* at = (const FPSTOK_LDS char*)table;
    if constexpr (JOINT) {
#pragma unroll
        for (int e = 0; e < 16; ++e)
            s[e] += *(const FPSTOK_LDS float*)(at + (entries[e] & 0xffffu));
        if (axes <= 2) return;
#pragma unroll
        for (int e = 0; e < 16; ++e)
            s[e] += *(const FPSTOK_LDS float*)(at + (entries[e] >> 16));
    } else {
#pragma unroll
        for (int a = 0; a < kMaxAxes; ++a) {
            if (a >= axes) break;
#pragma unroll
            for (int e = 0; e < 16; ++e)
                s[e] += *(const FPSTOK_LDS float*)(at + (entries[e] >> 8 * a & 255u));
        }
    }
}

// What bucket 1 of axis a adds to a pair's word, and what a word begins with.
template <bool JOINT>
__device__ __forceinline__ uint32_t entry_unit(const BiasArgs& b, int a) {
    if (!JOINT) return 4u << 8 * a;
    // (the first of two axes: as many as the second has)
    const uint32_t n = (a & 1) == 0 && a + 1 < b.axes ? (uint32_t)pick(b.top, a + 1) + 1 : 1u;
    return 4 * n << 16 * (a >> 1);
}
template <bool JOINT>
__device__ __forceinline__ uint32_t entry_base(const BiasArgs& b) {
    if (JOINT) return b.axes > 2 ? (uint32_t)b.joint[0] << 18 : 0;
    uint32_t x = 0;
#pragma unroll
    for (int a = 0; a < kMaxAxes; ++a) x += a < b.axes ? (uint32_t)b.first[a] << (8 * a + 2) : 0;
    return x;
}

// Entries of a block's pairs as the plane would hold them (places as for add_bias).
template <bool JOINT, bool KEY, int OWN, int ROWS>
__device__ __forceinline__ u32x16 find_entries(const BiasArgs& b, const FPSTOK_LDS uint32_t* own,
                                               const FPSTOK_LDS uint32_t* tile) {
    u32x16 entries = entry_base<JOINT>(b);
#pragma unroll 1
    for (int a = 0; a < b.axes; ++a) {
        const uint32_t mine = own[a * OWN], unit = entry_unit<JOINT>(b, a);
        const int top = pick(b.top, a), shift = pick(b.log_shift, a);
        const float rate = pick(b.rate, a), zero = pick(b.shift, a);
        by_kind(b.ints, shift >= 0, [&](auto ints, auto log) {
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const uint32_t other = tile[a * ROWS + (e >> 2) * 8 + (e & 3)];
                const int bucket = bucket_of<decltype(ints)::value, decltype(log)::value>(
                    KEY ? mine : other, KEY ? other : mine, rate, zero, top, shift);
                entries[e] += (uint32_t)bucket * unit;
            }
        });
    }
    return entries;
}

// Lane FROM of every four lanes' value, in all four (SHARE 4), or that of lane FROM
// of every two (SHARE 2).
template <int SHARE, int FROM>
__device__ __forceinline__ uint32_t from_lane(uint32_t x) {
    constexpr int kPerm = SHARE == 4 ? FROM * 0x55 : SHARE == 2 ? (FROM ? 0xf5 : 0xa0) : 0xe4;
    if (SHARE == 1) return x;
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, kPerm, 0xf, 0xf, true);
}

// Adds the bias of a block of 32 x 32 pairs to its scores (in units of log2): a
// lane's own row against the block's rows in its registers.  own: this lane's
// place in own[0], tile: that of the block's row 4 half in tile[0].
// KEY: the own row is the key.  PACK: entries, byte a of a pair's: the entry of
// axis a; bit a of `same`: it is one for all of the block's pairs.
// SHARE: that many lanes after one another hold one query (in heads of a group): each
// finds a part of the pairs' buckets for all of them.  (8192 + 5000 rows, causal, 16
// heads on 4 of 128: 788 us with one in four, 884 with all.)
//
// Rows in order (of time, of their place) and buckets that grow with the distance, or
// end, leave most blocks of a long walk in one bucket.  It grows or falls with the
// distance, so it is one for the block if the least key less the greatest query and the
// greatest less the least fall into the same: then a lane needs one value, not 16
// loads of LDS (the same rows: 703 us, 788 without).  Where a window hides the far
// keys, there are few, or several axes (of which one at most is in order), this would be
// looked for in vain (b.spans; 6000 + 2500 + 333 pulses, window of 256: a training step
// 369 us with it, 344 without; 64 events of up to 128 tokens, float32: 39 and 37; 6000 +
// 2111 + 64 rows, 4 axes: 11.4 and 9.7 ms).
template <bool KEY, bool PACK, bool SPANS, int SHARE, int OWN, int ROWS>
__device__ __forceinline__ uint32_t add_bias_shared(f32x16& s, u32x16* entries,
                                                    const BiasArgs& b,
                                                    const FPSTOK_LDS float* table,
                                                    const FPSTOK_LDS uint32_t* own,
                                                    const FPSTOK_LDS uint32_t* span,
                                                    const FPSTOK_LDS uint32_t* tile) {
    const int lane = threadIdx.x & 63;
    uint32_t same = 0;
    constexpr int kGroups = 4 / SHARE;  // of 4 adjacent rows that this lane looks at
    const int part = SHARE > 1 ? (int)(threadIdx.x & (SHARE - 1)) : 0;
#pragma unroll 1
    for (int a = 0; a < b.axes; ++a) {
        const uint32_t mine = own[a * OWN];
        const int first = pick(b.first, a), top = pick(b.top, a), shift = pick(b.log_shift, a);
        const float rate = pick(b.rate, a), zero = pick(b.shift, a);
        if (SPANS && b.spans) {
            int least, most, one = 0, other_end = 0;
            // (tile is at row 4 half)
            span_of(ordered(tile[a * ROWS + (lane & 31) - (lane >> 5) * 4], b.ints), least, most);
            by_kind(b.ints, shift >= 0, [&](auto ints, auto log) {
                const uint32_t lo = position(least, b.ints), hi = position(most, b.ints);
                const uint32_t k0 = KEY ? span[a * 2] : lo, k1 = KEY ? span[a * 2 + 1] : hi;
                const uint32_t q0 = KEY ? lo : span[a * 2], q1 = KEY ? hi : span[a * 2 + 1];
                one = bucket_of<decltype(ints)::value, decltype(log)::value>(k0, q1, rate, zero,
                                                                             top, shift);
                other_end = bucket_of<decltype(ints)::value, decltype(log)::value>(
                    k1, q0, rate, zero, top, shift);
                // (a distance that does not fit, or is not a number, says nothing of what
                // lies between)
                if constexpr (decltype(ints)::value) {
                    int d;
                    if (__builtin_sub_overflow((int)k0, (int)q1, &d) ||
                        __builtin_sub_overflow((int)k1, (int)q0, &d))
                        other_end = -1;
                } else {
                    if (!(__uint_as_float(k0) - __uint_as_float(q1) <=
                          __uint_as_float(k1) - __uint_as_float(q0)))
                        other_end = -1;
                }
            });
            if (__builtin_amdgcn_readfirstlane(one) == __builtin_amdgcn_readfirstlane(other_end)) {
                const float value = table[first + one];
#pragma unroll
                for (int e = 0; e < 16; ++e) s[e] += value;
                if constexpr (PACK) {
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        (*entries)[e] += (uint32_t)(first + one) << 8 * a;
                    same |= 1u << a;
                }
                continue;
            }
        }
        uint32_t found[kGroups * 4];
        by_kind(b.ints, shift >= 0, [&](auto ints, auto log) {
#pragma unroll
            for (int g = 0; g < kGroups; ++g) {
                const u32x4 other =
                    *(const FPSTOK_LDS u32x4*)(tile + a * ROWS + (part * kGroups + g) * 8);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    found[g * 4 + e] =
                        (uint32_t)(first +
                                   bucket_of<decltype(ints)::value, decltype(log)::value>(
                                       KEY ? mine : other[e], KEY ? other[e] : mine, rate, zero,
                                       top, shift))
                        << 2;
            }
        });
        auto add = [&](auto lane, int to) {
#pragma unroll
            for (int e = 0; e < kGroups * 4; ++e) {
                const uint32_t at = from_lane<SHARE, decltype(lane)::value>(found[e]);
                s[to + e] += *(const FPSTOK_LDS float*)((const FPSTOK_LDS char*)table + at);
                if constexpr (PACK) (*entries)[to + e] += at >> 2 << 8 * a;
            }
        };
        add(std::integral_constant<int, 0>{}, 0);
        if constexpr (SHARE > 1) add(std::integral_constant<int, 1>{}, kGroups * 4);
        if constexpr (SHARE > 2) {
            add(std::integral_constant<int, 2>{}, kGroups * 8);
            add(std::integral_constant<int, 3>{}, kGroups * 12);
        }
    }
    return same;
}

// share: 4, 2 or 1, the same in all lanes (query_share of the group).  Returns `same`.
template <bool KEY, bool PACK, bool SPANS, int OWN, int ROWS>
__device__ __forceinline__ uint32_t add_bias(f32x16& s, u32x16* entries, const BiasArgs& b,
                                             int share, const FPSTOK_LDS float* table,
                                             const FPSTOK_LDS uint32_t* own,
                                             const FPSTOK_LDS uint32_t* span,
                                             const FPSTOK_LDS uint32_t* tile) {
    if constexpr (PACK) *entries = 0;
    if constexpr (!KEY) {
        if (share == 4)
            return add_bias_shared<KEY, PACK, SPANS, 4, OWN, ROWS>(s, entries, b, table, own, span,
                                                                  tile);
        if (share == 2)
            return add_bias_shared<KEY, PACK, SPANS, 2, OWN, ROWS>(s, entries, b, table, own, span,
                                                                  tile);
    }
    return add_bias_shared<KEY, PACK, SPANS, 1, OWN, ROWS>(s, entries, b, table, own, span,
                                                                  tile);
}

// Lanes after one another that hold one query: tiles begin at a multiple of 32 rows,
// so rows of a group of 4 n heads come in fours.
__device__ __forceinline__ int query_share(int G) {
    return (G & 3) == 0 ? 4 : (G & 1) == 0 ? 2 : 1;
}

}  // namespace fpstok
