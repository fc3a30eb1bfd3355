// Matrix-product pieces of the attention kernels: 32 x 32 tiles by the matrix
// instructions of gfx950, their operands as fragments of 8 elements per lane,
// and the tiles of rows in LDS they are read from.
//
// One product step contracts 16 elements: lane l holds 8 of them (half
// l >> 5) for row (A) or column (B) l & 31; the 32 x 32 float32 result has
// column l & 31 and, in register r, row 8 (r / 4) + 4 (l >> 5) + r % 4.  Which
// 8 of the 16 a half holds is free as long as A and B agree:
//   natural  half h holds elements 8 h .. 8 h + 7 (16 adjacent bytes of a row
//            of a 16-bit type);
//   folded   half h holds 4 h .. 4 h + 3 and 8 + 4 h .. 8 + 4 h + 3: what
//            registers 0-7 (8-15) of a result hold, so the result of one
//            product is the operand of the next without moving between lanes.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fpstok {

using f32x16 = float __attribute__((ext_vector_type(16)));
using u32x4 = uint32_t __attribute__((ext_vector_type(4)));

#define FPSTOK_LDS __attribute__((address_space(3)))

template <class T>
struct Elem;

template <>
struct Elem<__bf16> {
    using Frag = __bf16 __attribute__((ext_vector_type(8)));
    static constexpr uint32_t kExp = 0x7f807f80u;  // exponent bits of two elements
    static constexpr uint32_t kOne = 0x00800080u;
    static constexpr uint32_t kUnit = 0x3f80u;  // 1.0
    static __device__ __forceinline__ f32x16 mma(Frag a, Frag b, f32x16 c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
    }
};

template <>
struct Elem<_Float16> {
    using Frag = _Float16 __attribute__((ext_vector_type(8)));
    static constexpr uint32_t kExp = 0x7c007c00u;
    static constexpr uint32_t kOne = 0x04000400u;
    static constexpr uint32_t kUnit = 0x3c00u;  // 1.0
    static __device__ __forceinline__ f32x16 mma(Frag a, Frag b, f32x16 c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
    }
};

template <>
struct Elem<float> {
    using Frag = float __attribute__((ext_vector_type(8)));
    static constexpr uint32_t kExp = 0x7f800000u;
    static constexpr uint32_t kOne = 0x00800000u;
    static constexpr uint32_t kUnit = 0x3f800000u;  // 1.0
    static __device__ __forceinline__ f32x16 mma(Frag a, Frag b, f32x16 c) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            c = __builtin_amdgcn_mfma_f32_32x32x2f32(a[j], b[j], c, 0, 0, 0);
        return c;
    }
};

// Registers 8 k .. 8 k + 7 of a result, rounded to the type, as the operand of
// the next product (folded order).
template <class T>
__device__ __forceinline__ typename Elem<T>::Frag to_frag(const f32x16& x, int k) {
    using f32x8 = float __attribute__((ext_vector_type(8)));
    const f32x8 v = k ? __builtin_shufflevector(x, x, 8, 9, 10, 11, 12, 13, 14, 15)
                      : __builtin_shufflevector(x, x, 0, 1, 2, 3, 4, 5, 6, 7);
    return __builtin_convertvector(v, typename Elem<T>::Frag);
}

// A tile of rows of DP elements in LDS, in 16-byte chunks; chunk c of a row is
// stored at place c ^ swz(row).  LDS has 64 banks of 4 bytes, 16 chunks wide;
// the swizzle spreads over them
//   the same chunk of the 16 rows that a 16-byte read takes at a time (lanes
//   0-3, 12-15 and 20-27, or 4-11, 16-19 and 28-31 of a half wave: measured);
//   the 64 bytes of 4 adjacent rows that a transposing read takes at a time,
//   or, of float32, the 128 bytes of the rows r and r + 4.
// It is linear: swz(x ^ y) = swz(x) ^ swz(y).  (A swizzle over 8 rows only
// measured a conflict on every read, half of all LDS cycles.)
template <class T, int DP>
struct Tile {
    static constexpr int kElems = 16 / (int)sizeof(T);  // per chunk
    static constexpr int kChunks = DP / kElems;         // per row
    static constexpr int kPitch = DP * (int)sizeof(T);  // bytes
    using Frag = typename Elem<T>::Frag;

    static __device__ __forceinline__ constexpr int swz(int row) {
        const int x = (row >> 3) & 1;
        if constexpr (sizeof(T) == 4) return ((row & 4) << 1) | ((row & 3) << 1) | x;
        // two rows of 128 bytes fill the banks: their parity is in the address
        if constexpr (kPitch == 128) return ((row & 2) << 1) | ((row & 4) >> 1) | x;
        return ((row & 3) << 2) | ((row & 4) >> 1) | x;
    }
    static __device__ __forceinline__ int place(int row, int chunk) {
        return row * kPitch + ((chunk ^ swz(row)) << 4);
    }

    // Row fragment of row `row` (lane-dependent), elements 16 step + 8 h ..
    // + 7 (natural order).
    static __device__ __forceinline__ Frag row_frag(const FPSTOK_LDS char* t, int row, int step,
                                                    int half) {
        if constexpr (sizeof(T) == 2) {
            return *(const FPSTOK_LDS Frag*)(t + place(row, 2 * step + half));
        } else {
            using f4 = float __attribute__((ext_vector_type(4)));
            const f4 a = *(const FPSTOK_LDS f4*)(t + place(row, 4 * step + 2 * half));
            const f4 b = *(const FPSTOK_LDS f4*)(t + place(row, 4 * step + 2 * half + 1));
            return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
        }
    }

    // Transposed fragment: elements `32 db + (lane & 31)` of the 16 rows from
    // row0 on, in folded order.  16-bit types read 4 rows x 16 elements per 16
    // lanes with one transposing read (lane i of the 16 addresses 4 elements
    // of row i / 4 and receives element i of the 4 rows).
    static __device__ __forceinline__ Frag col_frag(const FPSTOK_LDS char* t, int row0, int db,
                                                    int lane) {
        if constexpr (sizeof(T) == 2) {
            using s4 = short __attribute__((ext_vector_type(4)));
            const int i = lane & 15, r = ((lane >> 5) << 2) + (i >> 2);
            const int c = db * 4 + ((lane >> 4) & 1) * 2 + ((i & 3) >> 1);
            const int low = (i & 1) * 8;
            const s4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (FPSTOK_LDS s4*)(t + (row0 * kPitch + place(r, c ^ swz(row0)) + low)));
            const s4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (FPSTOK_LDS s4*)(t + ((row0 + 8) * kPitch + place(r, c ^ swz(row0 + 8)) + low)));
            return __builtin_bit_cast(Frag, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
        } else {
            const int d = db * 32 + (lane & 31), h4 = (lane >> 5) << 2;
            Frag f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int r = (j >> 2) * 8 + h4 + (j & 3);
                f[j] = *(const FPSTOK_LDS float*)(t + place(row0 + r, d >> 2) + (d & 3) * 4);
            }
            return f;
        }
    }
};

// True if a chunk holds an infinite or not-a-number element: the exponent
// bits of such an element carry into the bit above them when one is added.
template <class T>
__device__ __forceinline__ bool chunk_bad(u32x4 x) {
    uint32_t acc = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) acc |= (x[i] & Elem<T>::kExp) + Elem<T>::kOne;
    return (acc & (sizeof(T) == 2 ? 0x80008000u : 0x80000000u)) != 0;
}

// The chunk with its infinite and not-a-number elements replaced by zero, or,
// SIGN, by 1 of their sign.
template <class T, bool SIGN = false>
__device__ __forceinline__ u32x4 chunk_clean(u32x4 x) {
    constexpr uint32_t one = SIGN ? Elem<T>::kUnit : 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t c = (x[i] & Elem<T>::kExp) + Elem<T>::kOne;
        if constexpr (sizeof(T) == 2) {
            constexpr uint32_t sign = SIGN ? 0x8000u : 0;
            if (c & 0x80000000u) x[i] = (x[i] & (sign << 16 | 0xffffu)) | one << 16;
            if (c & 0x00008000u) x[i] = (x[i] & (sign | 0xffff0000u)) | one;
        } else {
            if (c & 0x80000000u) x[i] = (x[i] & (SIGN ? 0x80000000u : 0)) | one;
        }
    }
    return x;
}

// A lane's operand with its infinite and not-a-number elements replaced by zero.
template <class T>
__device__ __forceinline__ typename Elem<T>::Frag frag_clean(typename Elem<T>::Frag f) {
    u32x4* x = (u32x4*)&f;
#pragma unroll
    for (int e = 0; e < (int)sizeof(f) / 16; ++e) x[e] = chunk_clean<T>(x[e]);
    return f;
}

// Rows of a tile on their way from memory to LDS, by THREADS threads: load()
// issues the loads, store() writes them.  Rows at or past `rows` and elements
// at or past D become zero: their lanes load a place that exists instead (a
// load under a divergent branch would be waited for before the branch ends)
// and drop the value in store().  `rows` must be at least 1.
template <class T, int DP, int ROWS, int THREADS>
struct Stage {
    using Tl = Tile<T, DP>;
    static constexpr int kPer = ROWS * Tl::kChunks / THREADS;
    static constexpr int kStep = THREADS / Tl::kChunks;  // rows between a thread's chunks
    static_assert(ROWS * Tl::kChunks % THREADS == 0 && THREADS % Tl::kChunks == 0,
                  "whole chunks per thread");
    u32x4 x[kPer];
    int have;  // valid rows of the tile

    static __device__ __forceinline__ int row(int tid) { return tid / Tl::kChunks; }
    static __device__ __forceinline__ int chunk(int tid) { return tid % Tl::kChunks; }

    __device__ __forceinline__ void load(const T* base, int64_t stride, int rows, int D, int tid) {
        const int c = chunk(tid) * Tl::kElems < D ? chunk(tid) * Tl::kElems : 0;
        have = rows;
        if (rows >= ROWS) {
            const T* p = base + row(tid) * stride + c;
#pragma unroll
            for (int i = 0; i < kPer; ++i) x[i] = *(const u32x4*)(p + i * (kStep * stride));
        } else {
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const int r = i * kStep + row(tid);
                x[i] = *(const u32x4*)(base + (r < rows ? r : rows - 1) * stride + c);
            }
        }
    }
    __device__ __forceinline__ void store(FPSTOK_LDS char* t, int D, int tid) {
        if (have < ROWS || D < DP) {
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                if (i * kStep + row(tid) >= have || chunk(tid) * Tl::kElems >= D) x[i] = 0;
        }
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            *(FPSTOK_LDS u32x4*)(t + Tl::place(i * kStep + row(tid), chunk(tid))) = x[i];
    }
    // Rows whose bit is set become zero.
    __device__ __forceinline__ void drop(uint32_t rows, int tid) {
        static_assert(ROWS <= 32, "a bit per row");
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (rows >> (i * kStep + row(tid)) & 1) x[i] = 0;
    }
    // Infinite elements of rows whose bit is set become 1 of their sign.
    __device__ __forceinline__ void finite(uint32_t rows, int tid) {
        static_assert(ROWS <= 32, "a bit per row");
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (rows >> (i * kStep + row(tid)) & 1) x[i] = chunk_clean<T, true>(x[i]);
    }
    // Infinite and not-a-number elements of rows that exist become zero; a bit
    // for each chunk that had any (bit i of row i * kStep + row).
    __device__ __forceinline__ uint32_t clean(int tid) {
        static_assert(kPer <= 32, "a bit per chunk");
        uint32_t bad = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (i * kStep + row(tid) < have && chunk_bad<T>(x[i])) {
                x[i] = chunk_clean<T>(x[i]);
                bad |= 1u << i;
            }
        return bad;
    }
};

__device__ __forceinline__ const void* wave_uniform(const void* p) {
    const uint64_t x = (uint64_t)p;
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)x);
    const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(x >> 32));
    return (const void*)((uint64_t)hi << 32 | lo);
}

// 16 bytes per lane from base + off (bytes) straight to LDS at lds + 16 lane
// (base and lds the same in every lane), without a register in between; done
// once the wave's vmcnt is back at 0 (dma_wait).  The compiler would wait for such
// a load before the next LDS read of any kind; here the reads of one buffer go
// on while the other one fills.  The instruction takes its LDS address from M0,
// which the compiler itself does not use in these kernels (a check of the build
// looks for that; a clobber of a reserved register would not be kept).  It may
// follow the vector instruction that forms `base`, whose scalar registers a
// memory instruction can read 5 wait states later at the earliest: s_mov counts
// 1, s_nop 4 counts 5, and no pass of the compiler looks in here.
__device__ __forceinline__ void dma16(const void* base, uint32_t off, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tglobal_load_lds_dwordx4 %1, %2"
                 :
                 : "s"(__builtin_amdgcn_readfirstlane(lds)), "v"(off), "s"(wave_uniform(base))
                 : "memory");
}
__device__ __forceinline__ void dma4(const void* base, uint32_t off, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tglobal_load_lds_dword %1, %2"
                 :
                 : "s"(__builtin_amdgcn_readfirstlane(lds)), "v"(off), "s"(wave_uniform(base))
                 : "memory");
}
__device__ __forceinline__ void dma_wait() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

// Rows of a tile straight from memory to LDS by the 4 waves of a workgroup.
// Lane l of a load fills the l-th 16 bytes of its part of the tile, so the
// swizzle is in the address it reads from.  Rows at or past `rows` (at least
// 1) hold a copy of the last one: whoever reads the tile masks them.  Chunks
// at or past D are not loaded: they keep the zeros of zero().
template <class T, int DP, int ROWS>
struct Dma {
    using Tl = Tile<T, DP>;
    static constexpr int kPer = ROWS * Tl::kChunks / 256;
    static constexpr int kStep = 256 / Tl::kChunks;  // rows between a thread's chunks
    static constexpr int kBytes = ROWS * Tl::kPitch;
    static_assert(ROWS * Tl::kChunks % 256 == 0, "whole chunks per thread");
    int row, chunk;  // this thread's first row and the chunk it loads of it
    int D;
    __device__ __forceinline__ Dma(int D, int tid) : D(D) {
        row = tid / Tl::kChunks;
        chunk = (tid % Tl::kChunks) ^ Tl::swz(row);
    }
    // First element of the chunk this thread loads of row i * kStep + row.
    __device__ __forceinline__ int col(int i) const {
        return (chunk ^ Tl::swz(i * kStep)) * Tl::kElems;
    }
    static __device__ __forceinline__ void zero(FPSTOK_LDS char* buf, int bytes, int tid) {
        for (int i = tid * 16; i < bytes; i += 256 * 16) *(FPSTOK_LDS u32x4*)(buf + i) = 0;
    }
    // This thread's byte offset from a tile's first row, for load().
    __device__ __forceinline__ uint32_t offset(int64_t stride) const {
        return (uint32_t)(row * (int)stride + col(0)) * (uint32_t)sizeof(T);
    }
    __device__ __forceinline__ void load(const T* base, uint32_t offset, int64_t stride, int rows,
                                         FPSTOK_LDS char* buf, int wave) const {
        const uint32_t lds = (uint32_t)(uintptr_t)buf + wave * 1024;
        if (rows >= ROWS && Tl::swz(kStep) == 0) {
            if (col(0) < D) {
#pragma unroll
                for (int i = 0; i < kPer; ++i)
                    dma16(base, offset + (uint32_t)(i * kStep * (int)stride) * (uint32_t)sizeof(T),
                          lds + i * 4096);
            }
        } else {
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const int r = i * kStep + row < rows ? i * kStep + row : rows - 1;
                if (col(i) < D)
                    dma16(base, (uint32_t)(r * (int)stride + col(i)) * (uint32_t)sizeof(T),
                          lds + i * 4096);
            }
        }
    }
    // After dma_wait, of the chunks this thread loaded: rows whose bit is set
    // become zero; their infinite elements become 1 of their sign; all infinite
    // and not-a-number elements become zero (a bit for each chunk that had any:
    // bit i of row i * kStep + row).
    static __device__ __forceinline__ void drop(FPSTOK_LDS char* buf, uint64_t rows, int tid) {
        static_assert(ROWS <= 64, "a bit per row");
#pragma unroll 1
        for (int i = 0; i < kPer; ++i)
            if (rows >> (i * kStep + tid / Tl::kChunks) & 1)
                *(FPSTOK_LDS u32x4*)(buf + i * 4096 + tid * 16) = 0;
    }
    static __device__ __forceinline__ void finite(FPSTOK_LDS char* buf, uint64_t rows, int tid) {
        static_assert(ROWS <= 64, "a bit per row");
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            FPSTOK_LDS u32x4* p = (FPSTOK_LDS u32x4*)(buf + i * 4096 + tid * 16);
            const u32x4 x = *p;
            if (chunk_bad<T>(x) && (rows >> (i * kStep + tid / Tl::kChunks) & 1))
                *p = chunk_clean<T, true>(x);
        }
    }
    static __device__ __forceinline__ uint32_t clean(FPSTOK_LDS char* buf, int tid) {
        static_assert(kPer <= 32, "a bit per chunk");
        uint32_t bad = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            FPSTOK_LDS u32x4* p = (FPSTOK_LDS u32x4*)(buf + i * 4096 + tid * 16);
            const u32x4 x = *p;
            if (chunk_bad<T>(x)) {
                *p = chunk_clean<T>(x);
                bad |= 1u << i;
            }
        }
        return bad;
    }
};

// Orders a wave's own LDS writes and reads across its lanes (other waves are
// not waited for).
__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// max / sum of a value over the two lanes l and l ^ 32.
__device__ __forceinline__ float pair_max(float x) {
    const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false,
                                                    false);
    return fmaxf(__uint_as_float(s[0]), __uint_as_float(s[1]));
}

__device__ __forceinline__ float pair_sum(float x) {
    const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false,
                                                    false);
    return __uint_as_float(s[0]) + __uint_as_float(s[1]);
}

// Writes a transposed result (lane l: row l & 31 of the output, registers:
// elements of it) times `f` to `row`, D elements of it: 16 bytes per lane
// and store.
template <class T, int DB>
__device__ __forceinline__ void store_row(const f32x16* acc, float f, T* row, int D, int lane) {
    const int half = lane >> 5;
    if constexpr (sizeof(T) == 2) {
        using T4 = T __attribute__((ext_vector_type(4)));
        using f4 = float __attribute__((ext_vector_type(4)));
        using u2 = uint32_t __attribute__((ext_vector_type(2)));
#pragma unroll
        for (int db = 0; db < DB; ++db)
#pragma unroll
            for (int g = 0; g < 4; g += 2) {
                u2 p[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    f4 v;
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[e] = acc[db][(g + k) * 4 + e] * f;
                    p[k] = __builtin_bit_cast(u2, __builtin_convertvector(v, T4));
                }
                // half 0 collects elements 8g .. 8g+7, half 1 the next 8
                const auto a = __builtin_amdgcn_permlane32_swap(p[0][0], p[1][0], false, false);
                const auto b = __builtin_amdgcn_permlane32_swap(p[0][1], p[1][1], false, false);
                const u32x4 o = {a[0], b[0], a[1], b[1]};
                const int d = db * 32 + g * 8 + half * 8;
                if (row && d < D) *(u32x4*)(row + d) = o;
            }
    } else {
        using f4 = float __attribute__((ext_vector_type(4)));
#pragma unroll
        for (int db = 0; db < DB; ++db)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                f4 v;
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = acc[db][g * 4 + e] * f;
                const int d = db * 32 + g * 8 + half * 4;
                if (row && d < D) *(f4*)(row + d) = v;
            }
    }
}

}  // namespace fpstok
