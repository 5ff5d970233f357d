// Rows of bf16 or fp32 as the norms read and write them: eight elements (one
// chunk) per lane at a time, at any alignment of the rows' elements.
#pragma once
#include "moe_internal.h"

namespace moe {
namespace ops {

typedef u32x4 u32x4_e __attribute__((aligned(2)));   // 16 bytes at element alignment

// Eight consecutive elements as loaded: one 16-byte word per 8 bf16, two per 8 fp32.
template <typename XT>
struct Chunk {
    u32x4 w[sizeof(XT) / 2];
};

// Elements 0 .. n-1 of a chunk (n <= 8; the rest reads as zero).  TAIL: n may
// lie between 0 and 8 (rows whose length is no multiple of 8).
template <bool TAIL, typename XT>
__device__ __forceinline__ Chunk<XT> load_chunk(const XT* p, int n) {
    Chunk<XT> c;
    if (!TAIL || n >= 8) {
#pragma unroll
        for (int i = 0; i < (int)(sizeof(XT) / 2); ++i)
            c.w[i] = TAIL || n >= 8 ? ((const u32x4_e*)p)[i] : u32x4{0u, 0u, 0u, 0u};
        return c;
    }
    if constexpr (sizeof(XT) == 2) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t lo = 2 * i < n ? p[2 * i] : 0u, hi = 2 * i + 1 < n ? p[2 * i + 1] : 0u;
            c.w[0][i] = lo | (hi << 16);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) c.w[i / 4][i % 4] = i < n ? __float_as_uint(p[i]) : 0u;
    }
    return c;
}

template <typename XT>
__device__ __forceinline__ void unpack(const Chunk<XT>& c, float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if constexpr (sizeof(XT) == 2) v[i] = i & 1 ? bf16_hi(c.w[0][i / 2]) : bf16_lo(c.w[0][i / 2]);
        else v[i] = __uint_as_float(c.w[i / 4][i % 4]);
    }
}

// A row's chunk as the kernels fetch it ahead: the last one of a row that ends
// inside a chunk (n < 8) is read eight elements from the row's end back, so
// that it is one wide load as well and nothing of it is needed before its row
// is (assembled from single elements when fetched, it held up every row of the
// workgroup: 3001 x 7164 bf16, backward, 52.2 us against 38.9, forward 26.3
// against 22.8).  unpack_row moves the elements to their places.
template <bool TAIL, typename XT>
__device__ __forceinline__ Chunk<XT> fetch_chunk(const XT* p, int n, int H) {
    if (TAIL && H < 8) return load_chunk<true>(p, n);
    return load_chunk<false>(TAIL && n > 0 ? p - (8 - n) : p, n > 0 ? 8 : 0);
}
template <bool TAIL, typename XT>
__device__ __forceinline__ void unpack_row(const Chunk<XT>& c, int n, int H, float (&v)[8]) {
    unpack(c, v);
    if (!TAIL || H < 8 || n == 0 || n == 8) return;
    const int back = 8 - H % 8;   // the same for every row
    if (back & 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = v[i + 4];
    }
    if (back & 2) {
#pragma unroll
        for (int i = 0; i < 6; ++i) v[i] = v[i + 2];
    }
    if (back & 1) {
#pragma unroll
        for (int i = 0; i < 7; ++i) v[i] = v[i + 1];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? v[i] : 0.f;
}

// STREAM: nontemporal stores.
template <bool TAIL, bool STREAM = false, typename XT>
__device__ __forceinline__ void store_chunk(XT* p, int n, const float (&v)[8]) {
    if (n >= 8) {
        u32x4 w[sizeof(XT) / 2];
        if constexpr (sizeof(XT) == 2) {
            w[0] = u32x4{bf16x2_rne(v[0], v[1]), bf16x2_rne(v[2], v[3]), bf16x2_rne(v[4], v[5]),
                         bf16x2_rne(v[6], v[7])};
        } else {
#pragma unroll
            for (int i = 0; i < 2; ++i)
                w[i] = u32x4{__float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]), __float_as_uint(v[4 * i + 2]),
                             __float_as_uint(v[4 * i + 3])};
        }
#pragma unroll
        for (int i = 0; i < (int)(sizeof(XT) / 2); ++i) {
            if constexpr (STREAM) __builtin_nontemporal_store(w[i], (u32x4_e*)p + i);
            else ((u32x4_e*)p)[i] = w[i];
        }
        return;
    }
    if constexpr (!TAIL) return;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < n) {
            if constexpr (sizeof(XT) == 2) p[i] = (uint16_t)f32_to_bf16(v[i]);
            else p[i] = v[i];
        }
}

// Chunk of a weight or bias vector; `fill` where there is none.
template <bool TAIL>
__device__ __forceinline__ void load_param(const void* p, int dtype, int c, int n, float fill, float (&v)[8]) {
    if (!p) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = fill;
    } else if (dtype == MOE_BF16) {
        unpack(load_chunk<TAIL>((const uint16_t*)p + 8 * c, n), v);
    } else {
        unpack(load_chunk<TAIL>((const float*)p + 8 * c, n), v);
    }
}

}  // namespace ops
}  // namespace moe
