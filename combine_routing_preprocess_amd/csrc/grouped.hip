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

constexpr int kTile = 64, kStep = 32, kPad = 8;

__device__ __forceinline__ int expert_rows(const Args& p, int e, long long* seg) {
    const long long so = p.seg_off[e];
    long long m = so < p.R ? (long long)p.kept[e] : 0;
    if (so + m > p.R) m = p.R - so;
    *seg = so;
    return (int)m;
}

__device__ __forceinline__ float sigmoid(float v) { return 1.f / (1.f + __expf(-v)); }

template <bool A_ACROSS, bool B_ACROSS, Epilogue EPI>
__global__ __launch_bounds__(256) void k_grouped(Args p) {
    constexpr bool WEIGHT = EPI == kWeight16 || EPI == kWeight32;
    __shared__ uint16_t sa[kTile][kStep + kPad], sb[kTile][kStep + kPad];
    __shared__ float sc[kTile][kTile + 4];
    __shared__ int s_e, s_first;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int a0 = blockIdx.x * (EPI == kSwigluKeep ? kTile / 2 : kTile);
    int e, b0;
    if (WEIGHT) {
        e = blockIdx.z;
        b0 = blockIdx.y * kTile;
    } else {
        if (tid == 0) {   // the expert that this tile of rows belongs to
            int at = blockIdx.y, i = 0;
            for (; i < p.E; ++i) {
                long long seg;
                const int n = (expert_rows(p, i, &seg) + kTile - 1) / kTile;
                if (at < n) break;
                at -= n;
            }
            s_e = i;
            s_first = at * kTile;
        }
        __syncthreads();
        e = s_e;
        b0 = s_first;
        if (e >= p.E) return;
    }
    long long seg;
    const int rows = expert_rows(p, e, &seg);
    const int nb = WEIGHT ? p.nb : rows;
    const int nk = WEIGHT ? rows : p.nk;
    const int arows = EPI == kSwigluKeep ? 2 * p.na : p.na;   // rows of a weight that is not read across
    const uint16_t* A = WEIGHT ? p.a + seg * p.na : p.a + (size_t)e * arows * p.nk;
    const uint16_t* B = WEIGHT ? p.b + seg * p.nb : p.b + seg * p.nk;
    f32x16 acc;
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[i] = 0.f;
    for (int k0 = 0; k0 < nk; k0 += kStep) {
        for (int i = tid; i < kTile * kStep; i += 256) {
            if (A_ACROSS) {
                const int k = i / kTile, a = i % kTile;
                sa[a][k] = a0 + a < p.na && k0 + k < nk ? A[(size_t)(k0 + k) * p.na + a0 + a] : 0;
            } else {
                const int a = i / kStep, k = i % kStep;
                int f = a0 + a;
                bool ok = f < p.na;
                if (EPI == kSwigluKeep) {   // gate rows, then up rows
                    f = a0 + a % (kTile / 2);
                    ok = f < p.na;
                    if (a >= kTile / 2) f += p.na;
                }
                sa[a][k] = ok && k0 + k < nk ? A[(size_t)f * p.nk + k0 + k] : 0;
            }
            if (B_ACROSS) {
                const int k = i / kTile, b = i % kTile;
                sb[b][k] = b0 + b < nb && k0 + k < nk ? B[(size_t)(k0 + k) * p.nb + b0 + b] : 0;
            } else {
                const int b = i / kStep, k = i % kStep;
                sb[b][k] = b0 + b < nb && k0 + k < nk ? B[(size_t)(b0 + b) * p.nk + k0 + k] : 0;
            }
        }
        __syncthreads();
#pragma unroll
        for (int s = 0; s < kStep / 16; ++s) {
            const int r = lane & 31, k = 16 * s + 8 * (lane >> 5);
            const bf16x8 fa = *(const bf16x8*)&sa[(wave >> 1) * 32 + r][k];
            const bf16x8 fb = *(const bf16x8*)&sb[(wave & 1) * 32 + r][k];
            acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa, fb, acc, 0, 0, 0);
        }
        __syncthreads();
    }
    // a lane holds column b = lane % 32 and rows a = 8 * (r / 4) + 4 * (lane / 32) + r % 4 of its block
#pragma unroll
    for (int r = 0; r < 16; ++r)
        sc[(wave & 1) * 32 + (lane & 31)][(wave >> 1) * 32 + 8 * (r / 4) + 4 * (lane >> 5) + r % 4] = acc[r];
    __syncthreads();
    for (int i = tid; i < kTile * kTile; i += 256) {
        const int b = b0 + i / kTile, a = a0 + i % kTile;
        const float v = sc[i / kTile][i % kTile];
        if (b >= nb) continue;
        if (EPI == kSwigluKeep) {
            const int f = i % kTile;
            if (f >= kTile / 2 || a >= p.na) continue;
            const float u = sc[i / kTile][f + kTile / 2];
            uint16_t* h = (uint16_t*)p.out + (seg + b) * 2 * p.na;
            h[a] = (uint16_t)f32_to_bf16(v);
            h[p.na + a] = (uint16_t)f32_to_bf16(u);
            p.out2[(seg + b) * p.na + a] = (uint16_t)f32_to_bf16(v * sigmoid(v) * u);
        } else if (a >= p.na) {
            continue;
        } else if (EPI == kRows) {
            ((uint16_t*)p.out)[(seg + b) * p.na + a] = (uint16_t)f32_to_bf16(v);
        } else if (EPI == kSwigluGrad) {
            const uint16_t* h = p.h + (seg + b) * 2 * p.na;
            const float g = bf16_lo(h[a]), u = bf16_lo(h[p.na + a]), s = sigmoid(g);
            uint16_t* gh = (uint16_t*)p.out + (seg + b) * 2 * p.na;
            gh[a] = (uint16_t)f32_to_bf16(v * u * s * (1.f + g * (1.f - s)));
            gh[p.na + a] = (uint16_t)f32_to_bf16(v * g * s);
            p.out2[(seg + b) * p.na + a] = (uint16_t)f32_to_bf16(g * s * u);
        } else if (EPI == kWeight16) {
            uint16_t* o = (uint16_t*)p.out + ((size_t)e * p.nb + b) * p.na + a;
            if (p.accumulate) *o = (uint16_t)f32_to_bf16(bf16_lo(*o) + v);
            else *o = (uint16_t)f32_to_bf16(v);
        } else {
            float* o = (float*)p.out + ((size_t)e * p.nb + b) * p.na + a;
            *o = p.accumulate ? *o + v : v;
        }
    }
}

Args make_args(const moe_handle* h) {
    Args p = {};
    p.seg_off = h->seg_off;
    p.kept = h->kept;
    p.R = h->desc.out_rows;
    p.E = h->desc.E;
    return p;
}

// Tiles that the rows can make: each expert's last one may be partial.
unsigned row_tiles(const moe_handle* h, int tile) {
    const long long copies = (long long)h->desc.T * h->desc.K;
    return (unsigned)(copies / tile + (copies < h->desc.E ? copies : h->desc.E));
}

template <bool AA, bool BA, Epilogue EPI>
hipError_t launch_rows(const moe_handle* h, const Args& p, hipStream_t s) {
    const unsigned tiles = row_tiles(h, kTile);
    if (p.R == 0 || tiles == 0) return hipSuccess;
    const int wide = EPI == kSwigluKeep ? kTile / 2 : kTile;
    hipLaunchKernelGGL((k_grouped<AA, BA, EPI>), dim3((p.na + wide - 1) / wide, tiles), dim3(256), 0, s, p);
    return hipGetLastError();
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
    return transpose ? launch_rows<true, false, kRows>(h, p, s) : launch_rows<false, false, kRows>(h, p, s);
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
    return launch_rows<false, false, kSwigluKeep>(h, p, s);
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
    return launch_rows<true, false, kSwigluGrad>(h, p, s);
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
    const dim3 grid((M + kTile - 1) / kTile, (N + kTile - 1) / kTile, p.E);
    if (out_dtype == MOE_BF16) hipLaunchKernelGGL((k_grouped<true, true, kWeight16>), grid, dim3(256), 0, s, p);
    else hipLaunchKernelGGL((k_grouped<true, true, kWeight32>), grid, dim3(256), 0, s, p);
    return hipGetLastError();
}

}  // namespace moe
