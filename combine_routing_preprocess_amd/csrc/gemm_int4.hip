// Grouped expert MLP with 4-bit weights and one fp32 scale per weight row and
// 128 columns (W4A16), for decode-sized batches.
//
//   w[n][k] = (c[n][k] - 8) * s[n][k / 128],  c in 0..15, two codes per byte (even column in the low half)
//   FC1: g = W1[0:F] x, u = W1[F:2F] x, a = bf16(silu(g) * u);  FC2: y = bf16(W2 a)
//
// A few rows per expert share each weight, so streaming the codes bounds it:
// (1/2 + 4/128) bytes per weight from HBM, against a few multiply-adds each.
//
//  * Work unit = (expert, 16 features per wavefront) for FC1, (expert, 32
//    output rows per wavefront) for FC2, one workgroup of four or eight
//    wavefronts per unit; a wavefront owns two 16-row weight tiles (FC1: the
//    gate and up rows of its features).  Per step a unit takes one 128-byte
//    line (256 codes) of every weight row, the line's scales (two steps' at a
//    time) and the same 256 columns of its token rows, all straight from
//    memory into an LDS ring: no registers, no LDS writes by the wavefronts.
//    Weights and scales are the wavefront's own, tokens are shared (passes of
//    up to four rows have a copy per wavefront and no barriers).  Without the
//    arithmetic the transfers alone run at 6.8 TB/s.
//  * The loop is balanced between those transfers and some 190 vector (FC2:
//    157) and 24 matrix instructions per step and wavefront, so that many steps
//    have to overlap on a CU: three workgroups of two ring slots each (64 tokens, 256
//    experts top-8, 7168 x 2048: 876 us, against 914 with two workgroups of
//    three slots).  Where a CU gets one or two units the ring is deeper, and
//    two sets of wavefronts take every other step of a lone unit (one token:
//    43.5 us against 49).
//  * Rows per pass: 16 while the shape makes up to 8 rows per expert likely,
//    32 or, in units of eight wavefronts that share the tokens among more
//    weight rows, 64 above that (32 experts of 256 rows, 2048 x 1024: 278 us
//    with 64 against 326 with 32, 370 TFLOP/s), as far as the CUs all get a
//    workgroup.  More rows take more passes.
#include "device_ops.h"

namespace moe {
namespace {

using namespace ops;

constexpr int kCols = 256;            // columns of a step: a 128-byte line of codes, two scale groups
constexpr int kWaveBytes = 32 * 128;  // codes of a wavefront's step
constexpr int kWide = 32;             // rows per expert above which a unit may have eight wavefronts
constexpr int kBlock = 2;             // steps that share a transfer of scales: 4 groups of 32 rows
constexpr int kScaleBytes = 32 * 4 * 4;

// LDS of a kernel for passes of up to `rows` token rows and units of `waves`
// wavefronts: for each of the `split` sets that share a unit's columns the
// ring of `depth` steps and the blocks of scales per wavefront that may still
// be read while the ring's are loaded.
constexpr int scale_blocks(int depth, int split) { return split > 1 ? depth : (depth + kBlock - 1) / kBlock + 1; }
constexpr int set_bytes(int rows, int depth, int split, int waves) {
    return scale_blocks(depth, split) * waves * kScaleBytes + depth * (waves * kWaveBytes + rows * kCols * 2);
}
// Workgroups per CU that fit its 160 KB.
constexpr int per_cu(int rows, int depth, int split, int waves) {
    return 160 * 1024 / (split * set_bytes(rows, depth, split, waves));
}
static_assert(per_cu(16, 2, 1, 4) == 3 && per_cu(16, 3, 1, 4) == 2 && per_cu(16, 3, 2, 4) == 1 &&
                  per_cu(32, 2, 1, 4) == 2 && per_cu(64, 2, 1, 8) == 1,
              "LDS budget");

// Memory -> LDS transfers of 16 or 4 bytes per lane: from sbase
// (wave-uniform) + voff (per lane) to LDS byte address lds + 16 * lane (4 *
// lane).  Inline asm, so that the compiler does not wait for them before other
// LDS reads; their completion is awaited explicitly.  m0 is written only here;
// a load to LDS needs one wait state after that (s_nop 0), which the compiler
// does not add to inline asm.
typedef const char __attribute__((address_space(1))) gchar;
__device__ __forceinline__ gchar* uniform_ptr(const void* p) {
    const uint64_t v = (uint64_t)(uintptr_t)p;
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v);
    const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
    return (gchar*)(((uint64_t)hi << 32) | lo);
}
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void to_lds16(gchar* sbase, uint32_t voff, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" : : "v"(voff), "s"(sbase), "s"(lds)
                 : "memory", "m0");
}
__device__ __forceinline__ void to_lds16_once(gchar* sbase, uint32_t voff, uint32_t lds) {   // data read once
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1 nt" : : "v"(voff), "s"(sbase), "s"(lds)
                 : "memory", "m0");
}
__device__ __forceinline__ void to_lds4(gchar* sbase, uint32_t voff, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dword %0, %1" : : "v"(voff), "s"(sbase), "s"(lds)
                 : "memory", "m0");
}
#pragma clang diagnostic pop
template <int N>
__device__ __forceinline__ void wait_vm() {
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
// Workgroup barrier; this wavefront's LDS reads are complete before it
// arrives, its transfers may be in flight.
__device__ __forceinline__ void lds_barrier() {
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

__device__ __forceinline__ f32x4 mfma_bf16(const u32x4& a, const u32x4& b, const f32x4& c) {
    typedef __bf16 v8 __attribute__((ext_vector_type(8)));
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8, a), __builtin_bit_cast(v8, b), c, 0, 0, 0);
}

// Eight codes -> eight bf16 16 + c, in column order 0 4 1 5 2 6 3 7.  Mask and
// base are held in registers the compiler knows nothing of: as constants they
// would need two literals, and each and-or would become two instructions.
struct CodeBits {
    uint32_t mask = 0x00780078u, base = 0x41804180u;
    __device__ __forceinline__ CodeBits() { asm("" : "+v"(mask), "+v"(base)); }
    __device__ __forceinline__ u32x4 bf16(uint32_t w) const {
        return u32x4{((w << 3) & mask) | base, ((w >> 1) & mask) | base, ((w >> 5) & mask) | base,
                     ((w >> 9) & mask) | base};
    }
};

// Eight consecutive bf16 into the same column order.
__device__ __forceinline__ u32x4 pair_order(const u32x4& x) {
    return u32x4{__builtin_amdgcn_perm(x[2], x[0], 0x05040100u), __builtin_amdgcn_perm(x[2], x[0], 0x07060302u),
                 __builtin_amdgcn_perm(x[3], x[1], 0x05040100u), __builtin_amdgcn_perm(x[3], x[1], 0x07060302u)};
}

constexpr uint32_t kMinus24 = 0xc1c0c1c0u;   // two bf16 of -24

// One pass over rows m0 .. m0+mv-1 of the segment (mv <= ROWS) for the two
// weight tiles at t0 / t1 (byte 0 of each tile's first row) with scales at ws0
// and, scale_step bytes further, for the second tile.  On return lane l holds,
// for token 16 t + 4 * (l / 16) + j of the pass, the sums of the tiles' rows l
// % 16 in acc[.][t][j] (of the first set; `lds` is the set's own part of the
// workgroup's `shared`).
template <int MODE, int ROWS, int D, int SPLIT, int WAVES>
__device__ __forceinline__ void int4_accumulate(const uint16_t* __restrict__ X, const uint8_t* t0, const uint8_t* t1,
                                                const float* ws0, uint32_t scale_step, long long row0, int mv,
                                                int Kdim, int lane, int wave, int set, unsigned char* lds,
                                                unsigned char* shared, f32x4 (&acc)[2][(ROWS + 15) / 16]) {
    // Passes of up to 4 rows keep a copy of them per wavefront (in the room of 16 shared ones), so that no wavefront
    // waits for another.
    constexpr bool kOwnRows = ROWS <= 4;
    constexpr int NTB = (ROWS + 15) / 16, TL = kOwnRows ? 2 : ROWS / (2 * WAVES), SB = scale_blocks(D, SPLIT);
    constexpr int kScaleRing = SB * WAVES * kScaleBytes, kUnitBytes = WAVES * kWaveBytes;
    static_assert(TL > 0 && (kOwnRows || TL * 2 * WAVES == ROWS), "token transfers");
    // transfers of a wavefront per step, at least (scales where every step has its own; one of two token rows or more)
    constexpr int kLoads = 4 + (kOwnRows ? 1 : TL) + (SPLIT > 1);
    constexpr int kStage = kUnitBytes + (kOwnRows ? 16 : ROWS) * kCols * 2;
    const int own_rows_at = kOwnRows ? wave * 4 * kCols * 2 : 0;
    const int r16 = lane & 15, c1 = lane >> 4, row_bytes = Kdim / 2, groups = Kdim / 128;
    const int steps = (Kdim + kCols - 1) / kCols;
    const bool half_last = Kdim % kCols != 0;   // the last step holds one group only
    // this set's steps: its i-th is step i * SPLIT + set
    const int own = (steps - set + SPLIT - 1) / SPLIT, most = (steps + SPLIT - 1) / SPLIT;
    auto block_slot = [&](int i) { return SPLIT > 1 ? i % SB : i / kBlock % SB; };
#pragma unroll
    for (int t = 0; t < NTB; ++t) acc[0][t] = acc[1][t] = f32x4{0.f, 0.f, 0.f, 0.f};

    // Sources.  16-byte pieces are swizzled on the way (the LDS side of a
    // transfer is linear): piece p of weight row r lands in slot p ^ (r % 8) of
    // its 8, piece p of token row r in slot p ^ (r % 16) of its 32.
    const int wrow = lane >> 3, wpiece = (lane & 7) ^ wrow;
    const uint32_t woff = (uint32_t)(wrow * row_bytes + 16 * wpiece);
    // Half a last step: the pieces past the row's end read those of its first half again (nothing multiplies them).
    // The step back is one value for all rows of a lane (the swizzle by r % 16 leaves bit 4 of a token piece as
    // it is), so no second set of offsets is kept: 500 tokens, 24 experts of 1152 x 640 take 23.1 + 13.9 us
    // against 23.6 + 14.5 with such a set, and fewer registers spill.
    const uint32_t wback = half_last ? 16u * (uint32_t)(wpiece & 4) : 0u, xback = half_last ? 16u * (lane & 16) : 0u;
    // Scales of a block lie as [32 rows][4 groups].  Rows of whole 16-byte pieces on a base at a multiple of 16 take
    // one transfer (row lane of the lower 32 lanes), others, for which 4-byte alignment is enough, two (row 16 i +
    // lane / 4, one group); groups past the row's end repeat its last.
    const bool wide = groups % 4 == 0 && ((uintptr_t)ws0 & 15) == 0;
    auto scale_off = [&](int row, int g) {
        return (uint32_t)(((row & 15) * groups + g) * 4) + (row & 16 ? scale_step : 0u);
    };
    uint32_t xoff[TL];
#pragma unroll
    for (int j = 0; j < TL; ++j) {
        const int r = 2 * (kOwnRows ? j : wave + WAVES * j) + (lane >> 5), p = (lane & 31) ^ (r & 15);
        const uint32_t at = (uint32_t)min(r, mv - 1) * (uint32_t)Kdim * 2u;
        xoff[j] = at + 16u * (uint32_t)p;
    }
    gchar *b0 = uniform_ptr(t0), *b1 = uniform_ptr(t1), *bs = uniform_ptr(ws0);
    gchar* bx = uniform_ptr(X + (size_t)row0 * Kdim);
    const uint32_t ring = __builtin_amdgcn_readfirstlane(
        (uint32_t)(uintptr_t)(__attribute__((address_space(3))) unsigned char*)lds);
    auto load_scales = [&](int i) {
        const int blk = (i * SPLIT + set) / kBlock;
        const uint32_t at = ring + (uint32_t)(block_slot(i) * WAVES + wave) * kScaleBytes;
        if (wide) {
            if (lane < 32) to_lds16(bs, scale_off(lane, 4 * blk), at);
        } else {
#pragma unroll
            for (int j = 0; j < 2; ++j)
                to_lds4(bs, scale_off(16 * j + (lane >> 2), min(4 * blk + (lane & 3), groups - 1)), at + 256 * j);
        }
    };
    auto load = [&](int i) {
        if (SPLIT > 1 || i % kBlock == 0) load_scales(i);
        const int k = i * SPLIT + set;
        const bool last = k == steps - 1;
        const uint32_t at = ring + kScaleRing + (uint32_t)(i % D) * kStage;
        const uint32_t aw = at + (uint32_t)wave * kWaveBytes;
        const size_t line = (size_t)k * 128;
        const uint32_t wo = woff - (last ? wback : 0u), xb = last ? xback : 0u;
#pragma unroll
        for (int i = 0; i < 4; ++i)   // eight weight rows each
            to_lds16_once((i < 2 ? b0 : b1) + line + 8 * (i & 1) * (size_t)row_bytes, wo, aw + 1024u * i);
#pragma unroll
        for (int j = 0; j < TL; ++j)
            if (!kOwnRows || j == 0 || mv > 2)
                to_lds16(bx + (size_t)k * (kCols * 2), xoff[j] - xb,
                         at + kUnitBytes + (uint32_t)(own_rows_at + (kOwnRows ? j : wave + WAVES * j) * 1024));
    };
    const u32x4 off = {kMinus24, kMinus24, kMinus24, kMinus24};
    const CodeBits bits;
    auto tokens = [&](const u32x4& x) { return MODE == 0 ? pair_order(x) : x; };   // FC1 stores its output in pair order
    auto group = [&](int i0, int slot, int half) {
        const unsigned char* st = lds + kScaleRing + slot * kStage;
        const unsigned char* sw = st + wave * kWaveBytes;
        const float* ss = (const float*)(lds + (block_slot(i0) * WAVES + wave) * kScaleBytes) +
                          2 * ((i0 * SPLIT + set) % kBlock) + half;
        u32x4 b[2][4];
        float sc[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const u32x4 wq = *(const u32x4*)(sw + (16 * i + r16) * 128 + 16 * ((c1 + 4 * half) ^ (r16 & 7)));
            sc[i] = ss[4 * (16 * i + r16)];
#pragma unroll
            for (int q = 0; q < 4; ++q) b[i][q] = bits.bf16(wq[q]);
        }
#pragma unroll
        for (int t = 0; t < NTB; ++t) {
            const int r = 16 * t + (ROWS < 16 ? r16 % ROWS : r16);
            u32x4 a[4];
            f32x4 z = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int q = 0; q < 4; ++q)
                a[q] = tokens(*(const u32x4*)(st + kUnitBytes + own_rows_at + r * (kCols * 2) +
                                              16 * ((16 * half + 4 * c1 + q) ^ (r & 15))));
#pragma unroll
            for (int q = 0; q < 4; ++q) z = mfma_bf16(a[q], off, z);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                f32x4 p = z;
#pragma unroll
                for (int q = 0; q < 4; ++q) p = mfma_bf16(a[q], b[i][q], p);
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][t][j] = fmaf(sc[i], p[j], acc[i][t][j]);
            }
        }
    };
    wait_vm<0>();      // the counts below are of the transfers alone
    lds_barrier();     // nobody reads the previous pass's ring any more
#pragma unroll
    for (int i = 0; i < D - 1; ++i)
        if (i < own) load(i);
    auto arrive = [&](int i) {
        // The set's step i has landed; the transfers of up to D - 2 steps after it may be in flight.  They complete in
        // order, and counting the scales' among the steps' only waits for a little more.
        const int later = min(D - 2, own - 1 - i);
        if (D > 2 && later >= 1) wait_vm<kLoads>();
        else wait_vm<0>();
        if (kOwnRows) asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        else lds_barrier();
        if (i + D - 1 < own) load(i + D - 1);   // into the slot that step i - 1 was read from
    };
    static_assert(D <= 3, "arrive() lets one step be in flight");
    const int common = (steps - (half_last ? 1 : 0)) / SPLIT;   // whole steps that every set has
    for (int i0 = 0; i0 < common; i0 += D)
#pragma unroll
        for (int u = 0; u < D; ++u)   // step i0 + u is in slot u: a constant in every LDS address
            if (i0 + u < common) {
                arrive(i0 + u);
                group(i0 + u, u, 0);
                group(i0 + u, u, 1);
            }
    if (common < most) {   // a step that not every set has, or half a step
        arrive(common);
        if (common < own) {
            group(common, common % D, 0);
            if (!half_last || common * SPLIT + set < steps - 1) group(common, common % D, 1);
        }
    }
    if constexpr (SPLIT > 1) {   // the sets' sums join in the first one
        static_assert(SPLIT == 2, "one partner");
        f32x4* part = (f32x4*)shared + (wave * 64 + lane) * 2 * NTB;
        lds_barrier();
#pragma unroll
        for (int j = 0; j < 2 * NTB; ++j)
            if (set == 1) part[j] = acc[j / NTB][j % NTB];
        lds_barrier();
#pragma unroll
        for (int j = 0; j < 2 * NTB; ++j)
            if (set == 0) acc[j / NTB][j % NTB] += part[j];
    }
}

// MODE 0: SwiGLU of (gate, up) at feature f0 + l % 16; MODE 1: output rows
// f0 + l % 16 and f0 + 16 + l % 16.  Both stored as bf16 [R, Nout], the
// activations of MODE 0 with each 8 features in pair order, as FC2 reads them.
template <int MODE, int ROWS, int D, int SPLIT, int WAVES>
__device__ __forceinline__ void int4_pass(const uint16_t* __restrict__ X, const uint8_t* t0, const uint8_t* t1,
                                          const float* ws0, uint32_t scale_step, uint16_t* __restrict__ Out,
                                          long long row0, int mv, int Kdim, int Nout, int f0, bool mine, int lane,
                                          int wave, int set, unsigned char* lds, unsigned char* shared) {
    f32x4 acc[2][(ROWS + 15) / 16];
    int4_accumulate<MODE, ROWS, D, SPLIT, WAVES>(X, t0, t1, ws0, scale_step, row0, mv, Kdim, lane, wave, set, lds, shared,
                                       acc);
    if (!mine) return;
#pragma unroll
    for (int t = 0; t < (ROWS + 15) / 16; ++t)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int tok = 16 * t + 4 * (lane >> 4) + j;
            if (tok >= mv) continue;
            const int at = MODE == 0 ? (lane & 8) | ((lane & 3) << 1) | ((lane >> 2) & 1) : lane & 15;
            uint16_t* o = Out + (size_t)(row0 + tok) * Nout + f0 + at;
            if (MODE == 0) {
                o[0] = (uint16_t)f32_to_bf16(swiglu(acc[0][t][j], acc[1][t][j]));
            } else {
                o[0] = (uint16_t)f32_to_bf16(acc[0][t][j]);
                o[16] = (uint16_t)f32_to_bf16(acc[1][t][j]);
            }
        }
}

// The n-th expert that has rows, -1 if there are not as many; the same in every
// wavefront.
__device__ __forceinline__ int nth_with_rows(const int32_t* __restrict__ kept, int E, int n, int lane) {
    for (int e0 = 0; e0 < E; e0 += 256) {
        bool has[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int e = e0 + 64 * i + lane;
            has[i] = e < E && kept[min(e, E - 1)] > 0;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint64_t mask = __ballot(has[i]);
            const int c = __popcll(mask);
            if (n < c) {
                const int rank = __builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32),
                                                           __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0));
                return e0 + 64 * i + __ffsll((unsigned long long)__ballot(has[i] && rank == n)) - 1;
            }
            n -= c;
        }
    }
    return -1;
}

// Passes of up to ROWS token rows each: pass blockIdx.y and every gridDim.y-th
// after it.  `sparse`: blockIdx.x counts the units of the experts that have
// rows, otherwise of all.
// SPLIT sets of WAVES wavefronts share a unit's steps.
template <int MODE, int ROWS, int D, int SPLIT, int WAVES>
__global__ __launch_bounds__(64 * WAVES * SPLIT, WAVES / 4 * SPLIT * per_cu(ROWS, D, SPLIT, WAVES)) void k_gemm_int4(
    const uint16_t* __restrict__ X, const uint8_t* __restrict__ W, const float* __restrict__ Ws,
    uint16_t* __restrict__ Out, const int64_t* __restrict__ seg_off, const int32_t* __restrict__ kept, long long R,
    int E, int Kdim, int Wrows, int Nout, int units_per_expert, int sparse) {
    __shared__ __attribute__((aligned(16))) unsigned char s_ring[SPLIT * set_bytes(ROWS, D, SPLIT, WAVES)];
    const int lane = threadIdx.x & 63, any_wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wave = any_wave % WAVES, set = any_wave / WAVES;
    int e = blockIdx.x / units_per_expert;
    const int unit = blockIdx.x - e * units_per_expert;
    if (sparse) e = nth_with_rows(kept, E, e, lane);
    if (e < 0) return;
    const long long seg = seg_off[e];
    long long me_l = seg < R ? (long long)kept[e] : 0;
    if (seg + me_l > R) me_l = R - seg;
    const int me = (int)me_l;
    // the unit's features (FC1) or output rows (FC2); of a last unit that is not whole, wavefronts past the end repeat
    // the first half without storing it
    int f0 = (unit * WAVES + wave) * (MODE == 0 ? 16 : 32);
    const bool mine = set == 0 && f0 < Nout;
    if (f0 >= Nout) f0 -= WAVES / 2 * (MODE == 0 ? 16 : 32);
    const size_t r0 = (size_t)e * Wrows + f0, step = MODE == 0 ? Nout : 16;
    const uint8_t *t0 = W + r0 * (Kdim / 2), *t1 = t0 + step * (Kdim / 2);
    const float* ws0 = Ws + r0 * (Kdim / 128);
    const uint32_t scale_step = (uint32_t)(step * (Kdim / 128) * 4);
    for (int m0 = blockIdx.y * ROWS; m0 < me; m0 += gridDim.y * ROWS) {
        const int mv = min(ROWS, me - m0);
        const long long row0 = seg + m0;
        auto pass = [&](auto n) {
            int4_pass<MODE, decltype(n)::value, D, SPLIT, WAVES>(X, t0, t1, ws0, scale_step, Out, row0, mv, Kdim, Nout,
                                                                 f0, mine, lane, wave, set,
                                                                 s_ring + set * set_bytes(ROWS, D, SPLIT, WAVES),
                                                                 s_ring);
        };
        using std::integral_constant;
        if constexpr (ROWS == 16) {
            if (mv <= 4) pass(integral_constant<int, 4>{});
            else pass(integral_constant<int, 16>{});
        } else if constexpr (ROWS == 32) {
            if (mv <= 8) pass(integral_constant<int, 8>{});
            else if (mv <= 16) pass(integral_constant<int, 16>{});
            else pass(integral_constant<int, 32>{});
        } else {
            if (mv <= 16) pass(integral_constant<int, 16>{});
            else if (mv <= 32) pass(integral_constant<int, 32>{});
            else pass(integral_constant<int, 64>{});
        }
    }
}

}  // namespace

hipError_t launch_gemm_int4(const moe_handle* h, int stage, int F, const void* in, const void* w, const float* ws,
                            void* out, int num_cu, hipStream_t s) {
    const moe_desc& d = h->desc;
    const long long R = d.out_rows, copies = (long long)d.T * d.K;
    if (R == 0 || copies == 0) return hipSuccess;
    // experts that can have rows, and units to run; fewer copies than experts: skip the experts without rows by
    // counting (their empty workgroups would hold the CUs' LDS in turns: one token took 50 us in FC1 with them)
    const bool sparse = copies < d.E;
    const int experts = sparse ? (int)copies : d.E, nout = stage == 0 ? F : d.H, per_wave = stage == 0 ? 16 : 32;
    const long long avg = (copies + experts - 1) / experts;   // rows per expert, if they are spread evenly
    auto upe = [&](int waves) { return (nout + waves * per_wave - 1) / (waves * per_wave); };
    auto go = [&](auto rows, auto depth, auto split, auto waves) {
        constexpr int ROWS = decltype(rows)::value, D = decltype(depth)::value, SPLIT = decltype(split)::value,
                      WAVES = decltype(waves)::value;
        const long long units = (long long)experts * upe(WAVES);
        // passes of their own workgroups while the units alone leave room on the CUs
        const long long room = (long long)per_cu(ROWS, D, SPLIT, WAVES) * num_cu;
        const long long fill = (room + units - 1) / units, passes = (avg + ROWS - 1) / ROWS;
        const dim3 grid((unsigned)units, (unsigned)(fill < passes ? fill : passes)), block(64 * WAVES * SPLIT);
        if (stage == 0)
            hipLaunchKernelGGL((k_gemm_int4<0, ROWS, D, SPLIT, WAVES>), grid, block, 0, s, (const uint16_t*)in,
                               (const uint8_t*)w, ws, (uint16_t*)out, h->seg_off, h->kept, R, d.E, d.H, 2 * F, F,
                               upe(WAVES), sparse);
        else
            hipLaunchKernelGGL((k_gemm_int4<1, ROWS, D, SPLIT, WAVES>), grid, block, 0, s, (const uint16_t*)in,
                               (const uint8_t*)w, ws, (uint16_t*)out, h->seg_off, h->kept, R, d.E, F, d.H, d.H,
                               upe(WAVES), sparse);
    };
    using std::integral_constant;
    integral_constant<int, 1> one;
    integral_constant<int, 2> two;
    integral_constant<int, 3> three;
    integral_constant<int, 4> four;
    integral_constant<int, 8> eight;
    integral_constant<int, 16> r16;
    integral_constant<int, 32> r32;
    integral_constant<int, 64> r64;
    // The largest pass that still gives nearly every CU a workgroup: rows that share a dequantised weight against
    // CUs at work.  500 tokens, 24 experts of 1152 x 640 (240 units of 64 rows): 38.0 us with 64, 42.1 with 32; 100
    // tokens, 16 experts of 3584 x 512 (64 units of 64 rows, 256 of 32): 61.9 and 39.1, with 16 rows 44.1; 128 tokens,
    // 4 experts of 512 x 256 (16, 64 and 128 units): 19.4, 10.8 and 8.8.  In between, 2048 x 1024 with 128 units of 64
    // rows: 63.0 us against 41.6 with fewer rows a pass, 160: 50.0 and 55.1, 192: 51.5 and 58.2 (4096 x 2048 with 67
    // rows an expert, which 32 cut better: 84.0 and 68.7), 208: 70.4 and 70.5, 256: 77.2 and 83.2.  Seven eighths of the
    // CUs keep clear of the side that loses a third.
    auto workgroups = [&](int rows, int waves) { return (long long)experts * upe(waves) * ((avg + rows - 1) / rows); };
    const long long most = workgroups(16, 4);
    if (avg > kWide && 8 * workgroups(64, 8) >= 7ll * num_cu) go(r64, two, one, eight);
    else if (avg > 8 && workgroups(32, 4) >= num_cu) go(r32, two, one, four);
    else if (most <= num_cu) go(r16, three, two, four);
    else if (most <= 2 * num_cu) go(r16, three, one, four);
    else go(r16, two, one, four);
    return hipGetLastError();
}

}  // namespace moe
