// Grouped expert MLP with 4-bit weights and one fp32 scale per weight row and
// 128 columns (W4A16), for decode-sized batches.
//
//   w[n][k] = (c[n][k] - 8) * s[n][k / 128],  c in 0..15, two codes per byte (even column in the low half)
//   FC1: g = W1[0:F] x, u = W1[F:2F] x, a = bf16(silu(g) * u);  FC2: y = bf16(W2 a)
//
// A few rows per expert share each weight, so streaming the codes bounds it:
// (1/2 + 4/128) bytes per weight from HBM, against a few multiply-adds each.
//
//  * Work unit = (expert, 64 features) for FC1, (expert, 128 output rows) for
//    FC2, one workgroup of four wavefronts per unit; a wavefront owns two
//    16-row weight tiles (FC1: the gate and up rows of 16 features).  Whole
//    128-byte lines (256 codes of a row) go through the wavefront's own LDS
//    buffer into operand layout, as in the fp8 kernels.
//  * Products on v_mfma_f32_16x16x32_bf16: token rows are the A operand
//    (16 rows), weight rows the B operand (16 columns), so a lane dequantises
//    and scales one weight row only.  A lane's 16-byte piece holds 32
//    consecutive codes of its row; MFMA q of a 128-column group takes the 8
//    codes of the piece's word q, and the token operand the same 8 columns.
//  * A code becomes a bf16 by placing its four bits at the top of the
//    mantissa of 16.0: 16 + c, exact, one shift and one and-or per two codes.
//    The pairs come out as columns (0,4) (1,5) (2,6) (3,7); the token operand
//    is permuted the same way.  What is too much, 24 * sum(x) per token and
//    group, is an MFMA with a constant -24 operand whose result every tile's
//    accumulation starts from; it costs no vector instruction.
//  * After a group's MFMAs the fp32 block sum times the lane's scale is added
//    to the accumulator: scales are never rounded.  Activations between FC1
//    and FC2 are rounded once to bf16, as on the bf16 path.
//  * Up to 4 token blocks (64 rows) per pass; more rows take more passes.
#include "device_ops.h"

namespace moe {
namespace {

using namespace ops;

typedef short bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x2a __attribute__((ext_vector_type(2), aligned(4)));
typedef float f32x4a __attribute__((ext_vector_type(4), aligned(4)));

constexpr int kLine = 256;     // codes of a 128-byte line of a weight row: two scale groups

__device__ __forceinline__ f32x4 mfma_bf16(const u32x4& a, const u32x4& b, const f32x4& c) {
    typedef __bf16 v8 __attribute__((ext_vector_type(8)));
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8, a), __builtin_bit_cast(v8, b), c, 0, 0, 0);
}

// Eight codes -> eight bf16 16 + c, in column order 0 4 1 5 2 6 3 7.
__device__ __forceinline__ u32x4 codes_bf16(uint32_t w) {
    constexpr uint32_t kMask = 0x00780078u, kBase = 0x41804180u;
    return u32x4{((w << 3) & kMask) | kBase, ((w >> 1) & kMask) | kBase, ((w >> 5) & kMask) | kBase,
                 ((w >> 9) & kMask) | kBase};
}

// Eight consecutive bf16 into the same column order.
__device__ __forceinline__ u32x4 pair_order(const u32x4& x) {
    return u32x4{__builtin_amdgcn_perm(x[2], x[0], 0x05040100u), __builtin_amdgcn_perm(x[2], x[0], 0x07060302u),
                 __builtin_amdgcn_perm(x[3], x[1], 0x05040100u), __builtin_amdgcn_perm(x[3], x[1], 0x07060302u)};
}

constexpr uint32_t kMinus24 = 0xc1c0c1c0u;   // two bf16 of -24

// One 128-column group: wq[i] = the lane's 16-byte piece of tile i's row
// (columns 32 * (lane / 16) .. + 31 of the group), xg = the lane's token
// columns at the same place, sc[i] = the scales of the lane's rows.
template <int NTB>
__device__ __forceinline__ void group_mac(const u32x4 (&wq)[2], const uint16_t* const (&xg)[NTB], const float (&sc)[2],
                                          f32x4 (&acc)[2][NTB]) {
    u32x4 b[2][4];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) b[i][q] = codes_bf16(wq[i][q]);
    const u32x4 off = {kMinus24, kMinus24, kMinus24, kMinus24};
#pragma unroll
    for (int t = 0; t < NTB; ++t) {
        u32x4 a[4];
        f32x4 z = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int q = 0; q < 4; ++q) a[q] = pair_order(*(const u32x4*)(xg[t] + 8 * q));
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
}

// K loop of one pass over rows m0 .. m0+mv-1 of the segment for the two
// weight tiles at t0 / t1 (byte 0 of each tile's first row) with scales s0 /
// s1 (the lane's own row).  On return lane l holds, for token m0 + 16 t + 4 *
// (l / 16) + j, the sums of the tiles' rows l % 16 in acc[.][t][j].
template <int NTB>
__device__ __forceinline__ void int4_accumulate(const uint16_t* __restrict__ X, const uint8_t* t0, const uint8_t* t1,
                                                const float* s0, const float* s1, long long seg, int m0, int mv,
                                                int Kdim, int lane, unsigned char* lds, f32x4 (&acc)[2][NTB]) {
    const int r16 = lane & 15, c1 = lane >> 4, row_bytes = Kdim / 2;
#pragma unroll
    for (int t = 0; t < NTB; ++t) acc[0][t] = acc[1][t] = f32x4{0.f, 0.f, 0.f, 0.f};
    // the lane's token row in block t (clamped), at its 32 columns of a group
    const uint16_t* xr[NTB];
#pragma unroll
    for (int t = 0; t < NTB; ++t) xr[t] = X + (size_t)(seg + m0 + min(16 * t + r16, mv - 1)) * Kdim + 32 * c1;

    auto lines = [&](int kb0, auto uc) {   // UU whole lines of every row, all loads first
        constexpr int UU = decltype(uc)::value;
        u32x4 raw[UU][4];
        wl_load<UU>(t0, t1, row_bytes, kb0, lane, raw);
        wl_stash<UU>(lds, lane, raw);
#pragma unroll
        for (int u = 0; u < UU; ++u) {
            const unsigned char* buf = lds + u * 4096;
            const f32x2a sa = *(const f32x2a*)(s0 + 2 * (kb0 + u)), sb = *(const f32x2a*)(s1 + 2 * (kb0 + u));
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int ch = c1 + 4 * half;
                const u32x4 wq[2] = {*(const u32x4*)(buf + r16 * 128 + 16 * (ch ^ (r16 & 7))),
                                     *(const u32x4*)(buf + (16 + r16) * 128 + 16 * (ch ^ (r16 & 7)))};
                const float sc[2] = {sa[half], sb[half]};
                const uint16_t* xg[NTB];
#pragma unroll
                for (int t = 0; t < NTB; ++t) xg[t] = xr[t] + (size_t)(kb0 + u) * kLine + 128 * half;
                group_mac<NTB>(wq, xg, sc, acc);
            }
        }
    };
    const int nl = Kdim / kLine;
    int kb = 0;
    for (; kb + kU <= nl; kb += kU) lines(kb, std::integral_constant<int, kU>{});
    for (; kb < nl; ++kb) lines(kb, std::integral_constant<int, 1>{});
    if (Kdim % kLine) {   // an odd number of groups: the last one straight in operand layout
        const size_t o = (size_t)r16 * row_bytes + (size_t)nl * 128 + 16 * c1;
        const u32x4 wq[2] = {__builtin_nontemporal_load((const u32x4*)(t0 + o)),
                             __builtin_nontemporal_load((const u32x4*)(t1 + o))};
        const float sc[2] = {s0[2 * nl], s1[2 * nl]};
        const uint16_t* xg[NTB];
#pragma unroll
        for (int t = 0; t < NTB; ++t) xg[t] = xr[t] + (size_t)nl * kLine;
        group_mac<NTB>(wq, xg, sc, acc);
    }
}

// MODE 0: SwiGLU of (gate, up) at feature f0 + l % 16; MODE 1: output rows
// f0 + l % 16 and f0 + 16 + l % 16.  Both stored as bf16 [R, Nout].
template <int MODE, int NTB>
__device__ __forceinline__ void int4_pass(const uint16_t* __restrict__ X, const uint8_t* t0, const uint8_t* t1,
                                          const float* s0, const float* s1, uint16_t* __restrict__ Out, long long seg,
                                          int m0, int mv, int Kdim, int Nout, int f0, int lane, unsigned char* lds) {
    f32x4 acc[2][NTB];
    int4_accumulate<NTB>(X, t0, t1, s0, s1, seg, m0, mv, Kdim, lane, lds, acc);
#pragma unroll
    for (int t = 0; t < NTB; ++t)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int tok = 16 * t + 4 * (lane >> 4) + j;
            if (tok >= mv) continue;
            uint16_t* o = Out + (size_t)(seg + m0 + tok) * Nout + f0 + (lane & 15);
            if (MODE == 0) {
                o[0] = (uint16_t)f32_to_bf16(swiglu(acc[0][t][j], acc[1][t][j]));
            } else {
                o[0] = (uint16_t)f32_to_bf16(acc[0][t][j]);
                o[16] = (uint16_t)f32_to_bf16(acc[1][t][j]);
            }
        }
}

template <int MODE>
__global__ __launch_bounds__(256) void k_gemm_int4(const uint16_t* __restrict__ X, const uint8_t* __restrict__ W,
                                                   const float* __restrict__ Ws, uint16_t* __restrict__ Out,
                                                   const int64_t* __restrict__ seg_off,
                                                   const int32_t* __restrict__ kept, long long R, int Kdim, int Wrows,
                                                   int Nout, int units_per_expert) {
    __shared__ __attribute__((aligned(16))) unsigned char s_w[4 * kWaveLds];
    const int e = blockIdx.x / units_per_expert;
    const int unit = blockIdx.x - e * units_per_expert;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const long long seg = seg_off[e];
    long long me_l = seg < R ? (long long)kept[e] : 0;
    if (seg + me_l > R) me_l = R - seg;
    const int me = (int)me_l;
    if (me <= 0) return;
    const int f0 = MODE == 0 ? unit * kFeat + wave * 16 : unit * kFeat2 + wave * 32;
    const size_t r0 = (size_t)e * Wrows + f0, r1 = r0 + (MODE == 0 ? Nout : 16);
    const uint8_t *t0 = W + r0 * (Kdim / 2), *t1 = W + r1 * (Kdim / 2);
    const float *s0 = Ws + (r0 + (lane & 15)) * (Kdim / 128), *s1 = Ws + (r1 + (lane & 15)) * (Kdim / 128);
    unsigned char* lds = s_w + wave * kWaveLds;
    for (int m0 = 0; m0 < me; m0 += 16 * kMaxTB) {
        const int mv = min(16 * kMaxTB, me - m0);
        switch ((mv + 15) / 16) {
            case 1: int4_pass<MODE, 1>(X, t0, t1, s0, s1, Out, seg, m0, mv, Kdim, Nout, f0, lane, lds); break;
            case 2: int4_pass<MODE, 2>(X, t0, t1, s0, s1, Out, seg, m0, mv, Kdim, Nout, f0, lane, lds); break;
            case 3: int4_pass<MODE, 3>(X, t0, t1, s0, s1, Out, seg, m0, mv, Kdim, Nout, f0, lane, lds); break;
            default: int4_pass<MODE, 4>(X, t0, t1, s0, s1, Out, seg, m0, mv, Kdim, Nout, f0, lane, lds); break;
        }
    }
}

}  // namespace

hipError_t launch_gemm_int4(const moe_handle* h, int stage, int F, const void* in, const void* w, const float* ws,
                            void* out, hipStream_t s) {
    const moe_desc& d = h->desc;
    const long long R = d.out_rows;
    if (R == 0) return hipSuccess;
    if (stage == 0) {
        const int upe = F / kFeat;
        hipLaunchKernelGGL(k_gemm_int4<0>, dim3(d.E * upe), dim3(256), 0, s, (const uint16_t*)in, (const uint8_t*)w,
                           ws, (uint16_t*)out, h->seg_off, h->kept, R, d.H, 2 * F, F, upe);
    } else {
        const int upe = d.H / kFeat2;
        hipLaunchKernelGGL(k_gemm_int4<1>, dim3(d.E * upe), dim3(256), 0, s, (const uint16_t*)in, (const uint8_t*)w,
                           ws, (uint16_t*)out, h->seg_off, h->kept, R, F, d.H, d.H, upe);
    }
    return hipGetLastError();
}

}  // namespace moe
