// Pieces of the products grouped by expert that their two kernels share: the
// operands, transfers to LDS, operand fragments and the outputs' epilogues.
#pragma once
#include "moe_internal.h"

namespace moe {
namespace grouped {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

// What happens to the sums.
enum Epilogue {
    kRows,         // out[row][a] in bf16
    kSwigluKeep,   // a = gate and up of a feature: h and silu(gate) * up, both in bf16
    kSwigluGrad,   // the sums are the activation's gradient: h's gradient and the activation again
    kWeight16,     // out[e][b][a] in bf16
    kWeight16Add,  // the same, added to what is there
    kWeight32      // the same in fp32, added to what is there or not
};

struct Args {
    const uint16_t* a;     // [E] x [.., ..] weights, or rows (weight's gradient)
    const uint16_t* b;     // rows
    const uint16_t* h;     // kSwigluGrad: the forward's pre-activations [R, 2 na]
    void* out;
    uint16_t* out2;        // kSwigluKeep, kSwigluGrad: activations [R, na]
    const int64_t* seg_off;
    const int32_t* kept;
    long long R;
    int E, na, nb, nk;     // features, columns of the gradient (weight's gradient), sum's length
    int accumulate;        // weight's gradient: add to out
};

typedef __attribute__((address_space(1))) const char gchar;
typedef __attribute__((address_space(3))) char lchar;
typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) i16x4 li16x4;
typedef __attribute__((address_space(3))) u32x4 lu32x4;
typedef __attribute__((address_space(3))) u32x2 lu32x2;

__device__ __forceinline__ gchar* uniform_ptr(const void* p) {
    const uint64_t v = (uint64_t)(uintptr_t)p;
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v);
    const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
    return (gchar*)(((uint64_t)hi << 32) | lo);
}
__device__ __forceinline__ int uniform(int v) { return (int)__builtin_amdgcn_readfirstlane((uint32_t)v); }

// 16 bytes per lane from sbase (wave-uniform) + voff (per lane) to LDS byte
// address lds + 16 * lane.  Inline asm, so that the compiler does not wait for
// it before other LDS reads; completion is awaited explicitly.  m0 is written
// only here; a load to LDS needs one wait state after that (s_nop 0).
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void to_lds16(gchar* sbase, uint32_t voff, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" : : "v"(voff), "s"(sbase), "s"(lds)
                 : "memory", "m0");
}
#pragma clang diagnostic pop
// Scalar bases that a vector instruction may have written (readfirstlane, a
// spilled register's return) need five wait states before a transfer reads them.
__device__ __forceinline__ void base_ready(gchar*& a, gchar*& b) {
    asm volatile("s_nop 4" : "+s"(a), "+s"(b) : : "memory");
}
template <int N>
__device__ __forceinline__ void wait_vm() {
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
// Workgroup barrier; this wavefront's LDS reads are complete before it
// arrives, its transfers may be in flight.
__device__ __forceinline__ void lds_barrier() {
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// Between a wavefront's LDS writes and its other lanes' reads of them: the
// hardware keeps their order, the compiler has to be told.
__device__ __forceinline__ void lanes_exchange() { asm volatile("" ::: "memory"); }

__device__ __forceinline__ int expert_rows(const Args& p, int e, long long* seg) {
    const long long so = p.seg_off[e];
    long long m = so < p.R ? (long long)p.kept[e] : 0;   // a segment may begin past the end
    if (m > 0 && so + m > p.R) m = p.R - so;
    *seg = so;
    return (int)m;
}

__device__ __forceinline__ float sigmoid(float v) { return 1.f / (1.f + __expf(-v)); }

constexpr int kNxcd = 8;

// One tile: a0, b0 are its first feature and row (column of the gradient), nb
// bounds the rows (columns), nk is the sum's length.
struct Tile {
    gchar* A;
    gchar* B;
    int a0, b0, nb, nk;
};

// Fragments of a stage of BK elements: lane l holds row l % 32 of a block,
// elements 8 * (l / 32) .. + 7 of a step of 16.  X: an operand read across
// comes through the transposing read: of 16 lanes, lane i takes column i of the
// 4 rows x 16 columns whose 8 bytes each lane addresses.  In LDS
//   not across  rows of BK elements in chunks of 16 bytes, chunk c of row r at
//               place c ^ (r / (64 / BK * 2)) % (BK / 8)
//   across      rows of PITCH bytes, one per element of the sum, in units of 64
//               bytes, unit u of row k at place u ^ k % 4
// so that each read touches every bank once.  Blocks first, first + step, ...
template <bool X, int BK, int PITCH, int NB>
struct Fragments {
    uint32_t at[X ? NB : 1];
    int stride;

    __device__ __forceinline__ void init(int first, int step, int lane) {
        stride = step * 32 * BK * 2;
        if (X) {
#pragma unroll
            for (int i = 0; i < NB; ++i)
                at[X ? i : 0] = (uint32_t)((8 * (lane >> 5) + ((lane & 15) >> 2)) * PITCH +
                                           ((first + i * step) ^ ((lane >> 2) & 3)) * 64 + ((lane >> 4) & 1) * 32 +
                                           (lane & 3) * 8);
        } else {
            const int r = lane & 31;
            at[0] = (uint32_t)((32 * first + r) * BK * 2 + ((lane >> 5) ^ ((r / (128 / BK)) & (BK / 8 - 1))) * 16);
        }
    }
    // Block i of step s.  Not across, chunk 2 s + l / 32 lies where chunk l / 32 does, with the bits of 2 s flipped.
    __device__ __forceinline__ u32x4 load(lchar* base, int s, int i) const {
        if constexpr (X) {
            const i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((li16x4*)(base + at[i] + 16 * s * PITCH));
            const i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((li16x4*)(base + at[i] + (16 * s + 4) * PITCH));
            const u32x2 l = __builtin_bit_cast(u32x2, lo), h = __builtin_bit_cast(u32x2, hi);
            return u32x4{l[0], l[1], h[0], h[1]};
        } else {
            return *(lu32x4*)(base + (at[0] ^ (uint32_t)(32 * s)) + i * stride);
        }
    }
};

__device__ __forceinline__ f32x16 multiply(const u32x4& a, const u32x4& b, const f32x16& c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// Elements `left` and on of a fragment's eight become zero.
__device__ __forceinline__ u32x4 keep_first(u32x4 f, int left) {
#pragma unroll
    for (int q = 0; q < 4; ++q) f[q] &= left >= 2 * q + 2 ? 0xffffffffu : left == 2 * q + 1 ? 0xffffu : 0u;
    return f;
}

// fp32 rows of 64 features in LDS: 16 chunks of 16 bytes and one to spare.
__device__ __forceinline__ lu32x4* fp32_chunk(lchar* st, int r, int c) { return (lu32x4*)(st + r * 272 + c * 16); }

// This lane's sums of its row in the two feature blocks.
__device__ __forceinline__ void write_fp32(const f32x16& lo, const f32x16& hi, lchar* st, int row, int lane) {
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const f32x16& v = j ? hi : lo;
            *fp32_chunk(st + (lane >> 5) * 16, row, 8 * j + 2 * g) =
                u32x4{__float_as_uint(v[4 * g]), __float_as_uint(v[4 * g + 1]), __float_as_uint(v[4 * g + 2]),
                      __float_as_uint(v[4 * g + 3])};
        }
}

// Outputs of a tile: 64 features (kSwigluKeep: 32, gate and up) from f0 on, row
// blocks first, first + step, ... of rows b0 .. b0 + nrows - 1.  A lane holds
// row b = lane % 32 of each row block and features 8 * (r / 4) + 4 * (lane / 32)
// + r % 4 of each feature block; R16 (R32) rows at a time they pass through
// this wavefront's part of LDS as bf16 (as fp32) and leave as whole row segments
// of 128 bytes, 16 per lane.  Only this wavefront touches its part and its LDS
// operations run in order, so no barrier is needed.
//
// The activations and h's gradient, operands of the next products, leave as
// bf16: the matrix unit multiplies bf16 by bf16, and what a rounding drops could
// only come back as a second bf16 operand, which makes the forward's products 8 R
// H F operations instead of 6 and the backward's 22 instead of 12.  The forward
// MLP rounds its activations in the same place.  One rounding of an operand and
// one of the output leave the MLP's bf16 results 2.4e-3 off (2-norm), where the
// output's own alone gives 1.7e-3.
template <Epilogue EPI, int R16, int R32, int NTB>
__device__ __forceinline__ void store_tile(const Args& p, int f0, int b0, int nrows, int first, int step,
                                           long long seg, int e, const f32x16 (&acc)[2][NTB], lchar* st, int lane) {
    constexpr bool WEIGHT = EPI == kWeight16 || EPI == kWeight16Add || EPI == kWeight32;
    const int r8 = lane >> 3, c8 = lane & 7;
    // addresses: a wave-uniform row and the lane's 32-bit offset from it
    const long long out_row = (WEIGHT ? (long long)e * p.nb : seg) + b0;
    const uint32_t width = (EPI == kSwigluKeep || EPI == kSwigluGrad ? 2u : 1u) * p.na;
    if constexpr (EPI == kRows || EPI == kSwigluKeep || EPI == kWeight16) {
        // In the order write, read, write the next, store: a part's stores wait for its reads while the next is on its
        // way.  kSwigluKeep takes two parts for each: h, then the activations.
        constexpr int PARTS = 32 / R16, KINDS = EPI == kSwigluKeep ? 2 : 1, N = NTB * PARTS * KINDS;
        const int f = EPI == kSwigluKeep ? f0 + 8 * (c8 & 3) : f0 + 8 * c8;
        const uint32_t lane_at = (uint32_t)r8 * width + (uint32_t)(EPI == kSwigluKeep ? (c8 >> 2) * p.na : 0) + f;
        const int r4 = lane >> 2, fa = f0 + 8 * (lane & 3);
        auto write = [&](int at) {
            const int i = at / (PARTS * KINDS), part = at / KINDS % PARTS;
            lchar* wr = st + (lane & (R16 - 1)) * 144 + (lane >> 5) * 8;
            if (R16 < 32 && (lane & 31) / R16 != part) return;
            if (at % KINDS == 0) {
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int g = 0; g < 4; ++g)
                        *(lu32x2*)(wr + j * 64 + g * 16) = u32x2{bf16x2_rne(acc[j][i][4 * g], acc[j][i][4 * g + 1]),
                                                                 bf16x2_rne(acc[j][i][4 * g + 2], acc[j][i][4 * g + 3])};
            } else {
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    float a[4];
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const float v = acc[0][i][4 * g + r];
                        a[r] = v * sigmoid(v) * acc[1][i][4 * g + r];
                    }
                    *(lu32x2*)(wr + g * 16) = u32x2{bf16x2_rne(a[0], a[1]), bf16x2_rne(a[2], a[3])};
                }
            }
        };
        if constexpr (N > 0) write(0);
#pragma unroll
        for (int at = 0; at < N; ++at) {
            const int row0 = 32 * (first + at / (PARTS * KINDS) * step) + at / KINDS % PARTS * R16;
            lanes_exchange();
            u32x4 v[R16 / 8];
            if (at % KINDS == 0) {
#pragma unroll
                for (int k = 0; k < R16 / 8; ++k) v[k] = *(lu32x4*)(st + (8 * k + r8) * 144 + c8 * 16);
            } else {
#pragma unroll
                for (int k = 0; k < R16 / 16; ++k) v[k] = *(lu32x4*)(st + (16 * k + r4) * 144 + (lane & 3) * 16);
            }
            lanes_exchange();
            if (at + 1 < N) write(at + 1);
            if (at % KINDS == 0) {
#pragma unroll
                for (int k = 0; k < R16 / 8; ++k) {
                    if (row0 + 8 * k + r8 >= nrows || f >= p.na) continue;
                    uint16_t* o = (uint16_t*)p.out + (size_t)(out_row + row0 + 8 * k) * width;
                    if constexpr (EPI == kWeight16) __builtin_nontemporal_store(v[k], (u32x4*)(o + lane_at));
                    else *(u32x4*)(o + lane_at) = v[k];
                }
            } else {
#pragma unroll
                for (int k = 0; k < R16 / 16; ++k)
                    if (row0 + 16 * k + r4 < nrows && fa < p.na)
                        *(u32x4*)(p.out2 + (size_t)(out_row + row0 + 16 * k) * p.na + ((uint32_t)r4 * p.na + fa)) = v[k];
            }
        }
    } else if constexpr (EPI == kWeight16Add || EPI == kWeight32) {
        const int r16 = lane >> 4, f = f0 + 4 * (lane & 15);
        typedef std::conditional_t<EPI == kWeight32, u32x4, u32x2> Four;   // four elements
        typedef std::conditional_t<EPI == kWeight32, float, uint16_t> Out;
#pragma unroll
        for (int i = 0; i < NTB; ++i) {
            const int row0 = 32 * (first + i * step);
            Out* o = (Out*)p.out + (size_t)(out_row + row0) * p.na;
            const uint32_t lane_at = (uint32_t)r16 * p.na + f;
            Four old[4];       // 16 rows' values to add to, all on their way together
#pragma unroll
            for (int part = 0; part < 32 / R32; ++part) {
                if (p.accumulate && part * R32 % 16 == 0) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int row = part * R32 + 4 * k;
                        if (row0 + row + r16 < nrows && f < p.na) 
                            old[k] = __builtin_nontemporal_load((const Four*)(o + (size_t)row * p.na + lane_at));
                    }
                }
                if ((lane & 31) / R32 == part) write_fp32(acc[0][i], acc[1][i], st, lane & (R32 - 1), lane);
                lanes_exchange();
#pragma unroll
                for (int z = 0; z < R32 / 4; ++z) {
                    const int k = part * (R32 / 4) + z;
                    const u32x4 w = *fp32_chunk(st, 4 * z + r16, lane & 15);
                    if (row0 + 4 * k + r16 >= nrows || f >= p.na) continue;
                    float v[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) v[q] = __uint_as_float(w[q]);
                    if constexpr (EPI == kWeight32) {
                        if (p.accumulate) {
#pragma unroll
                            for (int q = 0; q < 4; ++q) v[q] += __uint_as_float(old[k & 3][q]);
                        }
                        __builtin_nontemporal_store(u32x4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                                         __float_as_uint(v[3])}, (u32x4*)(o + (size_t)(4 * k) * p.na + lane_at));
                    } else {
                        __builtin_nontemporal_store(u32x2{bf16x2_rne(v[0] + bf16_lo(old[k & 3][0]), v[1] + bf16_hi(old[k & 3][0])),
                                         bf16x2_rne(v[2] + bf16_lo(old[k & 3][1]), v[3] + bf16_hi(old[k & 3][1]))},
                                   (u32x2*)(o + (size_t)(4 * k) * p.na + lane_at));
                    }
                }
                lanes_exchange();
            }
        }
    } else {
        constexpr int PARTS = 32 / R32, K8 = R32 / 8;
        const int f = f0 + 8 * c8;
        // the next part's pre-activations are on their way while one is stored
        u32x4 gw[2][K8], uw[2][K8];
        auto row_of = [&](int at, int k) { return 32 * (first + at / PARTS * step) + at % PARTS * R32 + 8 * k; };
        const uint32_t lane_at = (uint32_t)r8 * width + f;
        auto fetch = [&](int at) {
#pragma unroll
            for (int k = 0; k < K8; ++k)
                if (row_of(at, k) + r8 < nrows && f < p.na) {
                    const uint16_t* h = p.h + (size_t)(out_row + row_of(at, k)) * width;
                    gw[at & 1][k] = *(const u32x4*)(h + lane_at);
                    uw[at & 1][k] = *(const u32x4*)(h + p.na + lane_at);
                }
        };
        fetch(0);
#pragma unroll
        for (int at = 0; at < NTB * PARTS; ++at) {
            if (at + 1 < NTB * PARTS) fetch(at + 1);
            if ((lane & 31) / R32 == at % PARTS)
                write_fp32(acc[0][at / PARTS], acc[1][at / PARTS], st, lane & (R32 - 1), lane);
            lanes_exchange();
#pragma unroll
            for (int k = 0; k < K8; ++k) {
                const int row = row_of(at, k);
                const u32x4 lo = *fp32_chunk(st, 8 * k + r8, 2 * c8);
                const u32x4 hi = *fp32_chunk(st, 8 * k + r8, 2 * c8 + 1);
                if (row + r8 >= nrows || f >= p.na) continue;
                u32x4 og, ou, oa;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    float dg[2], du[2], a[2];
#pragma unroll
                    for (int z = 0; z < 2; ++z) {
                        const uint32_t wg = gw[at & 1][k][q], wu = uw[at & 1][k][q];
                        const float g = z ? bf16_hi(wg) : bf16_lo(wg), u = z ? bf16_hi(wu) : bf16_lo(wu);
                        const float s = sigmoid(g), d = __uint_as_float(q < 2 ? lo[2 * q + z] : hi[2 * q + z - 4]);
                        dg[z] = d * u * s * (1.f + g * (1.f - s));
                        du[z] = d * g * s;
                        a[z] = g * s * u;
                    }
                    og[q] = bf16x2_rne(dg[0], dg[1]);
                    ou[q] = bf16x2_rne(du[0], du[1]);
                    oa[q] = bf16x2_rne(a[0], a[1]);
                }
                uint16_t* gh = (uint16_t*)p.out + (size_t)(out_row + row) * width;
                *(u32x4*)(gh + lane_at) = og;
                *(u32x4*)(gh + p.na + lane_at) = ou;
                *(u32x4*)(p.out2 + (size_t)(out_row + row) * p.na + ((uint32_t)r8 * p.na + f)) = oa;
            }
            lanes_exchange();
        }
    }
}

// The wide kernel's launch (grouped_wide.hip).
hipError_t launch_wide(Epilogue epi, bool across, const Args& p, int num_cu, hipStream_t s);

}  // namespace grouped
}  // namespace moe
