// Matrix products grouped by expert over the dispatched rows, for sizes that
// are any multiple of 8: the rows' product with the expert's weight and with
// its transpose, the weight's gradient, and the two products of the SwiGLU
// MLP's training passes with the activation in their epilogue.
//
// Every one is C[b][a] = sum over k of A[a][k] * B[b][k] for one expert, fp32
// sums of bf16 products (MFMA), one rounding at the end:
//   product            a = feature of w, b = row, k = column of the rows
//   its transpose      the same with w read across its rows (k = row of w)
//   weight's gradient  a = column of the rows, b = column of the gradient, k = row (both read across)
// An operand is "across" when its k runs over rows of the array.
#include "moe_internal.h"

namespace moe {
namespace {

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
    int accumulate;
};

constexpr int kTA = 256;                    // features of a tile: 64 per wavefront
constexpr int kTB = 128;                    // rows (weight's gradient: columns of the gradient) of a tile
constexpr int kBK = 32;                     // sum's elements per stage
constexpr int kSlots = 3;                   // stages in LDS
constexpr int kABytes = kTA * kBK * 2, kBBytes = kTB * kBK * 2, kSlot = kABytes + kBBytes;
constexpr int kNxcd = 8;
constexpr int kPerThread = kMaxE / 256;     // experts whose tiles one thread counts

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
template <int N>
__device__ __forceinline__ void wait_vm() {
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
// At most n of this wavefront's transfers in flight.
__device__ __forceinline__ void wait_transfers(int n) {
    if (n == 6) wait_vm<6>();
    else if (n == 5) wait_vm<5>();
    else if (n == 4) wait_vm<4>();
    else wait_vm<0>();
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
    long long m = so < p.R ? (long long)p.kept[e] : 0;
    if (so + m > p.R) m = p.R - so;
    *seg = so;
    return (int)m;
}

__device__ __forceinline__ float sigmoid(float v) { return 1.f / (1.f + __expf(-v)); }

// One tile: na, nb, nk bound the operands' columns, rows and sums; a0, b0 are
// the tile's first feature and row (column of the gradient).
struct Tile {
    gchar* A;
    gchar* B;
    int a0, b0, nb, nk;
};

// A stage's transfers.  Not across: rows of 64 bytes, four chunks of 16, chunk
// c of row r at place c ^ (r / 4) % 4.  Across: rows of 512 (B: 256) bytes, one
// per element of the sum, in units of 64 bytes, unit u of row k at place
// u ^ k % 4.  Either way the reads below touch every bank once.
template <bool AX, bool BX, bool KEEP>
struct Transfers {
    uint32_t a[4], b[2];      // per-lane offsets
    int nb_mine;              // B transfers of this wavefront
    uint32_t pitch_a, pitch_b;

    __device__ __forceinline__ void init(const Args& p, const Tile& t, int ntb, int wave, int lane) {
        pitch_a = (uint32_t)(AX ? p.na : t.nk) * 2u;
        pitch_b = (uint32_t)(BX ? p.nb : t.nk) * 2u;
        const uint32_t c4 = (uint32_t)((lane & 3) ^ ((lane >> 4) & 3)) * 16u;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            if (AX) {
                const int k = 8 * q + 2 * wave + (lane >> 5), c = (lane & 31) ^ ((k & 3) << 2);
                a[q] = (uint32_t)k * pitch_a + (uint32_t)min(t.a0 + 8 * c, p.na - 8) * 2u;
            } else if (KEEP) {      // rows 64 q .. of the tile: 32 gate features, the same 32 up
                const int f = min(t.a0 + 32 * q + 16 * (wave & 1) + (lane >> 2), p.na - 1);
                a[q] = (uint32_t)(f + (wave >> 1) * p.na) * pitch_a + c4;
            } else {
                a[q] = (uint32_t)min(t.a0 + 64 * q + 16 * wave + (lane >> 2), p.na - 1) * pitch_a + c4;
            }
        }
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            if (BX) {
                const int k = 16 * q + 4 * wave + (lane >> 4), c = (lane & 15) ^ ((k & 3) << 2);
                b[q] = (uint32_t)k * pitch_b + (uint32_t)min(t.b0 + 8 * c, t.nb - 8) * 2u;
            } else {
                b[q] = (uint32_t)min(64 * q + 16 * wave + (lane >> 2), t.nb - t.b0 - 1) * pitch_b + c4;
            }
        }
        nb_mine = BX ? 2 : (2 * ntb - wave + 3) / 4;
    }
    __device__ __forceinline__ int count() const { return 4 + nb_mine; }

    // Stage kt into LDS from byte address `lds` on; elements past the sum's end read valid memory again.
    __device__ __forceinline__ void issue(const Tile& t, int kt, uint32_t lds, int wave, int lane) const {
        gchar* A = t.A + (AX ? (size_t)kt * kBK * pitch_a : (size_t)kt * kBK * 2);
        gchar* B = t.B + (BX ? (size_t)kt * kBK * pitch_b : (size_t)kt * kBK * 2);
        const int rem = t.nk - kt * kBK;
        uint32_t va[4], vb[2];
#pragma unroll
        for (int q = 0; q < 4; ++q) va[q] = a[q];
#pragma unroll
        for (int q = 0; q < 2; ++q) vb[q] = b[q];
        if (rem < kBK) {
            const uint32_t c = (uint32_t)((lane & 3) ^ ((lane >> 4) & 3));
            const uint32_t back = (int)(8 * c) >= rem ? 16u * c : 0u;
#pragma unroll
            for (int q = 0; q < 4; ++q)
                va[q] -= AX ? (uint32_t)max(8 * q + 2 * wave + (lane >> 5) - (rem - 1), 0) * pitch_a : back;
#pragma unroll
            for (int q = 0; q < 2; ++q)
                vb[q] -= BX ? (uint32_t)max(16 * q + 4 * wave + (lane >> 4) - (rem - 1), 0) * pitch_b : back;
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) to_lds16(A, va[q], lds + (uint32_t)(4 * q + wave) * 1024u);
#pragma unroll
        for (int q = 0; q < 2; ++q)
            if (BX || q < nb_mine) to_lds16(B, vb[q], lds + kABytes + (uint32_t)(4 * q + wave) * 1024u);
    }
};

// Fragments of a stage: lane l holds row l % 32 of a block, elements 8 * (l /
// 32) .. + 7 of a step of 16.  Across operands come through the transposing
// read: of 16 lanes, lane i takes column i of the 4 rows x 16 columns whose 8
// bytes each lane addresses.
template <bool X, int PITCH, int NB>
struct Fragments {
    uint32_t at[X ? NB : 2];

    __device__ __forceinline__ void init(int first_block, int lane) {
        if (X) {
#pragma unroll
            for (int i = 0; i < NB; ++i)
                at[i] = (uint32_t)((8 * (lane >> 5) + ((lane & 15) >> 2)) * PITCH +
                                   ((first_block + i) ^ ((lane >> 2) & 3)) * 64 + ((lane >> 4) & 1) * 32 +
                                   (lane & 3) * 8);
        } else {
            const int r = lane & 31;
#pragma unroll
            for (int s = 0; s < 2; ++s)
                at[s] = (uint32_t)((32 * first_block + r) * 64 + ((2 * s + (lane >> 5)) ^ ((r >> 2) & 3)) * 16);
        }
    }
    __device__ __forceinline__ u32x4 load(lchar* base, int s, int i) const {
        if constexpr (X) {
            const i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((li16x4*)(base + at[i] + 16 * s * PITCH));
            const i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((li16x4*)(base + at[i] + (16 * s + 4) * PITCH));
            const u32x2 l = __builtin_bit_cast(u32x2, lo), h = __builtin_bit_cast(u32x2, hi);
            return u32x4{l[0], l[1], h[0], h[1]};
        } else {
            return *(lu32x4*)(base + at[s] + i * 2048);
        }
    }
};

// Outputs of a tile.  A lane holds row b = lane % 32 of each row block and
// features 8 * (r / 4) + 4 * (lane / 32) + r % 4 of each feature block; they
// pass through this wavefront's 6 KB of a free slot and leave as whole row
// segments of 128 bytes, 16 per lane.  Only this wavefront touches its part and
// its LDS operations run in order, so no barrier is needed.
template <Epilogue EPI, int NTB>
__device__ __forceinline__ void store_tile(const Args& p, const Tile& t, long long seg, int e, f32x16 (&acc)[2][NTB],
                                           lchar* st, int wave, int lane) {
    const int nrows = t.nb - t.b0;              // rows of the tile that exist
    const int f0 = t.a0 + (EPI == kSwigluKeep ? 32 : 64) * wave;
    const int r8 = lane >> 3, c8 = lane & 7;
    auto pack = [&](const f32x16& v, int g) {
        return u32x2{bf16x2_rne(v[4 * g], v[4 * g + 1]), bf16x2_rne(v[4 * g + 2], v[4 * g + 3])};
    };
#pragma unroll
    for (int i = 0; i < NTB; ++i) {
        const int row0 = 32 * i;
        if constexpr (EPI == kRows || EPI == kSwigluKeep || EPI == kWeight16) {
            lchar* wr = st + (lane & 31) * 144 + (lane >> 5) * 8;
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int g = 0; g < 4; ++g) *(lu32x2*)(wr + j * 64 + g * 16) = pack(acc[j][i], g);
            lanes_exchange();
            const int f = EPI == kSwigluKeep ? f0 + 8 * (c8 & 3) : f0 + 8 * c8;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int row = row0 + 8 * k + r8;
                u32x4 v = *(lu32x4*)(st + (8 * k + r8) * 144 + c8 * 16);
                if (row >= nrows || f >= p.na) continue;
                if constexpr (EPI == kSwigluKeep) {
                    *(u32x4*)((uint16_t*)p.out + (size_t)(seg + t.b0 + row) * 2 * p.na + (c8 >> 2) * p.na + f) = v;
                } else if constexpr (EPI == kRows) {
                    *(u32x4*)((uint16_t*)p.out + (size_t)(seg + t.b0 + row) * p.na + f) = v;
                } else {
                    u32x4* o = (u32x4*)((uint16_t*)p.out + ((size_t)e * p.nb + t.b0 + row) * p.na + f);
                    *o = v;
                }
            }
            lanes_exchange();
            if constexpr (EPI == kSwigluKeep) {
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
                lanes_exchange();
                const int r4 = lane >> 2, c4 = lane & 3, fa = f0 + 8 * c4;
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int row = row0 + 16 * k + r4;
                    const u32x4 v = *(lu32x4*)(st + (16 * k + r4) * 144 + c4 * 16);
                    if (row < nrows && fa < p.na)
                        *(u32x4*)(p.out2 + (size_t)(seg + t.b0 + row) * p.na + fa) = v;
                }
                lanes_exchange();
            }
        } else {
            // fp32 sums: 16 rows of 64 features at a time
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                if ((lane & 31) / 16 == half) {
                    lchar* wr = st + (lane & 15) * 272 + (lane >> 5) * 16;
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int g = 0; g < 4; ++g)
                            *(lu32x4*)(wr + j * 128 + g * 32) =
                                u32x4{__float_as_uint(acc[j][i][4 * g]), __float_as_uint(acc[j][i][4 * g + 1]),
                                      __float_as_uint(acc[j][i][4 * g + 2]), __float_as_uint(acc[j][i][4 * g + 3])};
                }
                lanes_exchange();
                if constexpr (EPI == kWeight32) {
                    const int r16 = lane >> 4, c16 = lane & 15, f = f0 + 4 * c16;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int row = row0 + 16 * half + 4 * k + r16;
                        const u32x4 w = *(lu32x4*)(st + (4 * k + r16) * 272 + c16 * 16);
                        float4 v = make_float4(__uint_as_float(w[0]), __uint_as_float(w[1]), __uint_as_float(w[2]),
                                               __uint_as_float(w[3]));
                        if (row >= nrows || f >= p.na) continue;
                        float4* o = (float4*)((float*)p.out + ((size_t)e * p.nb + t.b0 + row) * p.na + f);
                        if (p.accumulate) {
                            const float4 old = *o;
                            v.x += old.x; v.y += old.y; v.z += old.z; v.w += old.w;
                        }
                        *o = v;
                    }
                } else if constexpr (EPI == kWeight16Add || EPI == kSwigluGrad) {
                    const int f = f0 + 8 * c8;
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const int row = row0 + 16 * half + 8 * k + r8;
                        const u32x4 lo = *(lu32x4*)(st + (8 * k + r8) * 272 + c8 * 32);
                        const u32x4 hi = *(lu32x4*)(st + (8 * k + r8) * 272 + c8 * 32 + 16);
                        if (row >= nrows || f >= p.na) continue;
                        float v[8];
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            v[q] = __uint_as_float(lo[q]);
                            v[4 + q] = __uint_as_float(hi[q]);
                        }
                        if constexpr (EPI == kWeight16Add) {
                            u32x4* o = (u32x4*)((uint16_t*)p.out + ((size_t)e * p.nb + t.b0 + row) * p.na + f);
                            u32x4 w = *o;
#pragma unroll
                            for (int q = 0; q < 4; ++q)
                                w[q] = bf16x2_rne(v[2 * q] + bf16_lo(w[q]), v[2 * q + 1] + bf16_hi(w[q]));
                            *o = w;
                        } else {
                            const size_t at = (size_t)(seg + t.b0 + row) * 2 * p.na + f;
                            const u32x4 gw = *(const u32x4*)(p.h + at), uw = *(const u32x4*)(p.h + at + p.na);
                            u32x4 og, ou, oa;
#pragma unroll
                            for (int q = 0; q < 4; ++q) {
                                float dg[2], du[2], a[2];
#pragma unroll
                                for (int z = 0; z < 2; ++z) {
                                    const float g = z ? bf16_hi(gw[q]) : bf16_lo(gw[q]);
                                    const float u = z ? bf16_hi(uw[q]) : bf16_lo(uw[q]);
                                    const float s = sigmoid(g), d = v[2 * q + z];
                                    dg[z] = d * u * s * (1.f + g * (1.f - s));
                                    du[z] = d * g * s;
                                    a[z] = g * s * u;
                                }
                                og[q] = bf16x2_rne(dg[0], dg[1]);
                                ou[q] = bf16x2_rne(du[0], du[1]);
                                oa[q] = bf16x2_rne(a[0], a[1]);
                            }
                            *(u32x4*)((uint16_t*)p.out + at) = og;
                            *(u32x4*)((uint16_t*)p.out + at + p.na) = ou;
                            *(u32x4*)(p.out2 + (size_t)(seg + t.b0 + row) * p.na + f) = oa;
                        }
                    }
                }
                lanes_exchange();
            }
        }
    }
}

template <bool AX, bool BX, Epilogue EPI, int NTB>
__device__ __forceinline__ void run_tile(const Args& p, const Tile& t, long long seg, int e, lchar* lds, int wave,
                                         int lane) {
    Transfers<AX, BX, EPI == kSwigluKeep> tr;
    tr.init(p, t, NTB, wave, lane);
    Fragments<AX, kTA * 2, 2> fa;
    Fragments<BX, kTB * 2, NTB> fb;
    fa.init(2 * wave, lane);
    fb.init(0, lane);
    f32x16 acc[2][NTB];
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < NTB; ++i)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[j][i][r] = 0.f;
    const uint32_t base = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)lds);
    const int n = (t.nk + kBK - 1) / kBK;
    int slot = 0;             // of the stage that is multiplied
    if (n > 0) tr.issue(t, 0, base, wave, lane);
    if (n > 1) tr.issue(t, 1, base + kSlot, wave, lane);
    // Stage kt has landed when at most the transfers of stage kt + 1 are in
    // flight; past the barrier every wavefront's have, and the slot of stage
    // kt - 1, which all have read, takes stage kt + 2.
    auto stage = [&](int kt, auto lastc) {
        constexpr bool LAST = decltype(lastc)::value;
        if (LAST) wait_vm<0>();
        else wait_transfers(tr.count());
        lds_barrier();
        if (!LAST && kt + 2 < n) tr.issue(t, kt + 2, base + (slot == 0 ? 2 : slot - 1) * kSlot, wave, lane);
        lchar* s0 = lds + slot * kSlot;
        u32x4 a[2][2], b[2][NTB];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
#pragma unroll
            for (int j = 0; j < 2; ++j) a[s][j] = fa.load(s0, s, j);
#pragma unroll
            for (int i = 0; i < NTB; ++i) b[s][i] = fb.load(s0 + kABytes, s, i);
        }
        if (LAST) {           // elements past the sum's end become zero in both operands
            const int rem = t.nk - kt * kBK;
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const int left = rem - 16 * s - 8 * (lane >> 5);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const uint32_t m = left >= 2 * q + 2 ? 0xffffffffu : left == 2 * q + 1 ? 0xffffu : 0u;
#pragma unroll
                    for (int j = 0; j < 2; ++j) a[s][j][q] &= m;
#pragma unroll
                    for (int i = 0; i < NTB; ++i) b[s][i][q] &= m;
                }
            }
        }
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int i = 0; i < NTB; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    acc[j][i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a[s][j]),
                                                                        __builtin_bit_cast(bf16x8, b[s][i]), acc[j][i],
                                                                        0, 0, 0);
        slot = slot == 2 ? 0 : slot + 1;
    };
    for (int kt = 0; kt + 1 < n; ++kt) stage(kt, std::false_type{});
    if (n > 0) stage(n - 1, std::true_type{});
    // the slot behind the last stage's was read two stages ago, before a barrier that all have passed
    store_tile<EPI, NTB>(p, t, seg, e, acc, lds + slot * kSlot + wave * (kSlot / 4), wave, lane);
}

template <bool AX, bool BX, Epilogue EPI>
__global__ __launch_bounds__(256, 2) void k_grouped(Args p) {
    constexpr bool WEIGHT = EPI == kWeight16 || EPI == kWeight16Add || EPI == kWeight32;
    constexpr int AW = EPI == kSwigluKeep ? kTA / 2 : kTA;     // features of a tile
    __shared__ u32x4 s_ring[kSlots * kSlot / 16];
    __shared__ int s_wave[4];
    __shared__ int s_expert, s_first, s_tiles, s_rows;
    __shared__ long long s_seg;
    lchar* lds = (lchar*)(__attribute__((address_space(3))) u32x4*)s_ring;
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    const int ta = (p.na + AW - 1) / AW;
    // rows: the tiles of rows of every expert, counted by each workgroup
    int mine[kPerThread], rows[kPerThread], before = 0;
    const int per = (p.E + 255) / 256;
    long long total;
    const int tb = WEIGHT ? (p.nb + kTB - 1) / kTB : 0;
    if (WEIGHT) {
        total = (long long)p.E * ta * tb;
    } else {
        int sum = 0;
#pragma unroll
        for (int i = 0; i < kPerThread; ++i) {
            const int e = tid * per + i;
            long long seg;
            rows[i] = i < per && e < p.E ? expert_rows(p, e, &seg) : 0;
            mine[i] = (rows[i] + kTB - 1) / kTB;
            sum += mine[i];
        }
        int run = sum;        // inclusive over the wavefront's lanes
        for (int d = 1; d < 64; d <<= 1) {
            const int o = __shfl_up(run, d);
            if (lane >= d) run += o;
        }
        if (lane == 63) s_wave[wave] = run;
        __syncthreads();
        before = run - sum;
        int all = 0;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            if (w < wave) before += s_wave[w];
            all += s_wave[w];
        }
        total = (long long)all * ta;
    }
    // each XCD takes one contiguous run of the tiles, so that tiles that share rows or weights share an L2
    const int xcd = blockIdx.x % kNxcd;
    const long long hi = total * (xcd + 1) / kNxcd;
    for (long long t = total * xcd / kNxcd + blockIdx.x / kNxcd; t < hi; t += gridDim.x / kNxcd) {
        int e, nrows;
        long long seg;
        Tile tile;
        if (WEIGHT) {
            e = (int)(t / ((long long)ta * tb));
            const int at = (int)(t - (long long)e * ta * tb);
            nrows = uniform(expert_rows(p, e, &seg));
            tile.a0 = (at % ta) * AW;
            tile.b0 = (at / ta) * kTB;
            tile.nb = p.nb;
            tile.nk = nrows;
            if (nrows == 0 && p.accumulate) continue;
            tile.A = uniform_ptr(p.a + (size_t)seg * p.na);
            tile.B = uniform_ptr(p.b + (size_t)seg * p.nb);
        } else {
            const int u = (int)(t / ta);
#pragma unroll
            for (int i = 0, at = before; i < kPerThread; at += mine[i], ++i)
                if (u >= at && u < at + mine[i]) {
                    s_expert = tid * per + i;
                    s_first = at;
                    s_tiles = mine[i];
                    s_rows = rows[i];
                    s_seg = p.seg_off[tid * per + i];
                }
            __syncthreads();
            e = uniform(s_expert);
            const int tiles = uniform(s_tiles), at = (int)(t - (long long)uniform(s_first) * ta);
            nrows = uniform(s_rows);
            seg = s_seg;
            seg = (long long)(((uint64_t)__builtin_amdgcn_readfirstlane((uint32_t)(seg >> 32)) << 32) |
                              __builtin_amdgcn_readfirstlane((uint32_t)seg));
            // an expert's rows in tiles of nearly one size, whole blocks of 32; its tiles of rows are neighbours
            const int blocks = ((nrows + 31) / 32 + tiles - 1) / tiles;
            tile.a0 = (at / tiles) * AW;
            tile.b0 = (at % tiles) * blocks * 32;
            tile.nb = min(nrows, tile.b0 + blocks * 32);
            tile.nk = p.nk;
            tile.A = uniform_ptr(p.a + (size_t)e * (EPI == kSwigluKeep ? 2 : 1) * p.na * p.nk);
            tile.B = uniform_ptr(p.b + (size_t)(seg + tile.b0) * p.nk);
        }
        asm volatile("s_nop 4" ::: "memory");   // wait states between readfirstlane and the transfers' base
        switch ((min(tile.nb - tile.b0, kTB) + 31) / 32) {
            case 1: run_tile<AX, BX, EPI, 1>(p, tile, seg, e, lds, wave, lane); break;
            case 2: run_tile<AX, BX, EPI, 2>(p, tile, seg, e, lds, wave, lane); break;
            case 3: run_tile<AX, BX, EPI, 3>(p, tile, seg, e, lds, wave, lane); break;
            default: run_tile<AX, BX, EPI, 4>(p, tile, seg, e, lds, wave, lane); break;
        }
        lds_barrier();        // the slots are free for the next tile
    }
}

constexpr long long kMaxGrid = 1 << 20;   // workgroups; more tiles than that are walked

unsigned grid_for(long long tiles) {
    const long long g = (tiles + kNxcd - 1) / kNxcd * kNxcd;
    return (unsigned)(g < kMaxGrid ? g : kMaxGrid);
}

Args make_args(const moe_handle* h) {
    Args p = {};
    p.seg_off = h->seg_off;
    p.kept = h->kept;
    p.R = h->desc.out_rows;
    p.E = h->desc.E;
    return p;
}

// Most tiles that the rows can make: each expert's last one may be partial.
long long row_tiles(const moe_handle* h) {
    const long long copies = (long long)h->desc.T * h->desc.K;
    return copies / kTB + (copies < h->desc.E ? copies : h->desc.E);
}

template <bool AX, Epilogue EPI>
hipError_t launch_rows(const moe_handle* h, const Args& p, hipStream_t s) {
    constexpr int AW = EPI == kSwigluKeep ? kTA / 2 : kTA;
    const long long tiles = row_tiles(h) * ((p.na + AW - 1) / AW);
    if (p.R == 0 || tiles == 0) return hipSuccess;
    hipLaunchKernelGGL((k_grouped<AX, false, EPI>), dim3(grid_for(tiles)), dim3(256), 0, s, p);
    return hipGetLastError();
}

template <Epilogue EPI>
void launch_weight(const Args& p, hipStream_t s) {
    const long long tiles = (long long)p.E * ((p.na + kTA - 1) / kTA) * ((p.nb + kTB - 1) / kTB);
    hipLaunchKernelGGL((k_grouped<true, true, EPI>), dim3(grid_for(tiles)), dim3(256), 0, s, p);
}

}  // namespace

hipError_t launch_grouped_product(const moe_handle* h, int N, int M, int transpose, const void* rows, const void* w,
                                  void* out, hipStream_t s) {
    Args p = make_args(h);
    p.a = (const uint16_t*)w;
    p.b = (const uint16_t*)rows;
    p.out = out;
    p.na = transpose ? M : N;
    p.nk = transpose ? N : M;
    return transpose ? launch_rows<true, kRows>(h, p, s) : launch_rows<false, kRows>(h, p, s);
}

hipError_t launch_grouped_swiglu_keep(const moe_handle* h, int F, const void* rows, const void* w1, void* hout,
                                      void* act, hipStream_t s) {
    Args p = make_args(h);
    p.a = (const uint16_t*)w1;
    p.b = (const uint16_t*)rows;
    p.out = hout;
    p.out2 = (uint16_t*)act;
    p.na = F;
    p.nk = h->desc.H;
    return launch_rows<false, kSwigluKeep>(h, p, s);
}

hipError_t launch_grouped_swiglu_grad(const moe_handle* h, int F, const void* grad_out, const void* w2, const void* hin,
                                      void* grad_h, void* act, hipStream_t s) {
    Args p = make_args(h);
    p.a = (const uint16_t*)w2;
    p.b = (const uint16_t*)grad_out;
    p.h = (const uint16_t*)hin;
    p.out = grad_h;
    p.out2 = (uint16_t*)act;
    p.na = F;
    p.nk = h->desc.H;
    return launch_rows<true, kSwigluGrad>(h, p, s);
}

hipError_t launch_grouped_weight_grad(const moe_handle* h, int N, int M, int out_dtype, int accumulate,
                                      const void* grad, const void* rows, void* out, hipStream_t s) {
    Args p = make_args(h);
    p.a = (const uint16_t*)rows;
    p.b = (const uint16_t*)grad;
    p.out = out;
    p.na = M;
    p.nb = N;
    p.accumulate = accumulate;
    if (out_dtype != MOE_BF16) launch_weight<kWeight32>(p, s);
    else if (accumulate) launch_weight<kWeight16Add>(p, s);
    else launch_weight<kWeight16>(p, s);
    return hipGetLastError();
}

}  // namespace moe
