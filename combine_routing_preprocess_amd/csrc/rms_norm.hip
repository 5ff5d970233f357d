// RMS norm of token rows with the residual's addition and an output in 8 bits,
// and its backward pass: the norm in front of the MoE layer.
//
//   forward   t = x + residual,  r = 1 / sqrt(mean(t^2) + eps),  y = t * r * w
//             codes = e4m3(y / scale), scale = max |y| of 128 columns / 448
//   backward  xh = t * r,  q = gy * w,
//             gt = grad_total + r * (q - xh * mean(q * xh)),
//             gw = sum over the rows of gy * xh
//
// Both directions are bound by HBM: every row is read and written once.  As in
// the layer norm a row is held in registers by W wavefronts, 8 elements (one
// chunk) per lane and step, at most NC steps; G short rows share a workgroup;
// workgroups walk the rows with a stride, so the weight is loaded once per
// workgroup, and the loads of the next two rows are in flight during the
// current row's sum.  The 16 lanes that hold 128 columns are neighbours, so a
// block's maximum is four lane permutes.  The sum of squares is fp32, eight
// terms per lane and step, then lanes, then wavefronts: no cancellation, so one
// pass and one barrier per row.  Measured on MI355X, 8192 x 7168 bf16: forward
// with residual into 8-bit rows 81 us, backward with the residual stream's
// gradient and the weight's 91 us (5.1 and 5.2 TB/s, where a large device copy
// runs at 4.7); one row 4.1 us on the GPU, 8.7 us per call from the host; 3001 x
// 1537 fp32 backward 19 us, of which the second launch is 4.
#include "row_chunks.h"
#include "wave_ops.h"

namespace moe {
namespace {

using ops::Chunk;
using ops::fetch_chunk;
using ops::load_param;
using ops::row_sum;
using ops::store_chunk;
using ops::u32x4_e;
using ops::unpack_row;
using ops::wave_sum_dpp;

constexpr int kMaxWaves = 16;   // wavefronts of a workgroup

// Where the forward's outputs go; null where they are not wanted.
struct Outputs {
    void* y;
    uint8_t* codes;
    float* scales;
    void* total;
    float* rstd;
    int y_bf16;
};

// Largest of 16 neighbouring lanes' values, in every one of them.
__device__ __forceinline__ uint32_t row_max(uint32_t v) {
    v = max(v, ops::dpp<ops::kDppXor1>(v));
    v = max(v, ops::dpp<ops::kDppXor2>(v));
    v = max(v, ops::dpp<ops::kDppHalfMirror>(v));
    return max(v, ops::dpp<ops::kDppMirror>(v));
}

// x, the residual and the total may be the same rows, so none is __restrict__:
// an element is read, two rows ahead, by the lane that writes it (the chunk at
// a row's end is read with elements of its neighbour's, which it drops), and
// before a barrier that its row's stores come after.
template <typename XT, typename RT, int NC, bool TAIL, bool STREAM>
__global__ __launch_bounds__(1024) void k_rms_norm(const XT* x, const RT* res, int T, int H, int W, int G,
                                                   const void* __restrict__ weight, int wdtype, float eps, Outputs o) {
    __shared__ float s_part[2][kMaxWaves];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int grp = wave / W, part = wave - grp * W;
    constexpr bool KEEP = NC <= 2;   // the weight and the next rows in registers
    int col[NC], n[NC];
    float w[KEEP ? NC : 1][8];
#pragma unroll
    for (int k = 0; k < NC; ++k) {
        const int c = (part + k * W) * 64 + lane;
        col[k] = 8 * c;
        n[k] = min(max(H - col[k], 0), 8);
        if (KEEP) load_param<TAIL>(weight, wdtype, c, n[k], 1.f, w[KEEP ? k : 0]);
    }
    const float inv_h = 1.f / (float)H;
    const int peer = lane & 15;
    const long long stride = (long long)gridDim.x * G;
    long long row = (long long)blockIdx.x * G + grp;
    Chunk<XT> nx[2][NC];
    Chunk<RT> nr[2][NC];
    auto fetch = [&](int d, long long r) {
#pragma unroll
        for (int k = 0; k < NC; ++k) nx[d][k] = fetch_chunk<TAIL>(x + r * H + col[k], r < T ? n[k] : 0, H);
        if (res) {
#pragma unroll
            for (int k = 0; k < NC; ++k) nr[d][k] = fetch_chunk<TAIL>(res + r * H + col[k], r < T ? n[k] : 0, H);
        }
    };
    if (KEEP) {
        fetch(0, row);
        fetch(1, row + stride);
    }
    auto step = [&](int par) {
        const bool ok = row < T;
        float v[NC][8];
        if (!KEEP) fetch(par, row);
#pragma unroll
        for (int k = 0; k < NC; ++k) unpack_row<TAIL>(nx[par][k], ok ? n[k] : 0, H, v[k]);
        if (res) {
#pragma unroll
            for (int k = 0; k < NC; ++k) {
                float a[8];
                unpack_row<TAIL>(nr[par][k], ok ? n[k] : 0, H, a);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[k][i] += a[i];
            }
        }
        if (KEEP) fetch(par, row + 2 * stride);
        float q = 0.f;
#pragma unroll
        for (int k = 0; k < NC; ++k)
#pragma unroll
            for (int i = 0; i < 8; ++i) q = fmaf(v[k][i], v[k][i], q);
        q = wave_sum_dpp(q);
        if (W > 1) {
            if (lane == 0) s_part[par][wave] = q;
            // one barrier: who still reads the other parity passed its barrier before this row's writes
            __syncthreads();
            q = row_sum(peer < W ? s_part[par][grp * W + (peer < W ? peer : 0)] : 0.f);
        }
        const float r = 1.f / sqrtf(fmaf(q, inv_h, eps));
        if (ok) {
#pragma unroll
            for (int k = 0; k < NC; ++k) {
                const long long at = row * H + col[k];
                if (o.total) store_chunk<TAIL, STREAM>((RT*)o.total + at, n[k], v[k]);
                if (!KEEP) load_param<TAIL>(weight, wdtype, col[k] / 8, n[k], 1.f, w[0]);
                float y[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] = v[k][i] * r * w[KEEP ? k : 0][i];
                if (o.y) {
                    if (o.y_bf16) store_chunk<TAIL, STREAM>((uint16_t*)o.y + at, n[k], y);
                    else store_chunk<TAIL, STREAM>((float*)o.y + at, n[k], y);
                }
                if constexpr (!TAIL) {
                    if (o.codes) {
                        uint32_t top = 0;   // as integers NaN is above infinity, infinity above all numbers
#pragma unroll
                        for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(y[i]) & 0x7fffffffu);
                        top = row_max(top);
                        const float sc = top < 0x7f800000u ? e4m3_scale(__uint_as_float(top))
                                                           : __uint_as_float(0x7fc00000u);
                        if (n[k] > 0) {
                            *(u32x2*)(o.codes + at) = u32x2{e4m3_pack4(y[0], y[1], y[2], y[3], sc),
                                                            e4m3_pack4(y[4], y[5], y[6], y[7], sc)};
                            if (peer == 0) o.scales[at / 128] = sc;
                        }
                    }
                }
            }
            if (o.rstd && part == 0 && lane == 0) o.rstd[row] = r;
        }
        row += stride;
    };
    // the workgroup's rows advance together, so every wavefront meets the barriers
    for (long long row0 = (long long)blockIdx.x * G; row0 < T; row0 += 2 * stride) {
        step(0);
        if (row0 + stride < T) step(1);
    }
}

// Row gradients of the workgroup's rows, and its sums of gy * xh per column
// into pw + blockIdx * pstride.  The gradient may be grad_total: as above.
template <typename TT, typename YT, int NC, bool TAIL>
__global__ __launch_bounds__(1024) void k_rms_norm_backward(const YT* __restrict__ gy, const TT* __restrict__ t,
                                                            const float* __restrict__ rstd, const TT* gtot, int T,
                                                            int H, int W, int G, const void* __restrict__ weight,
                                                            int wdtype, TT* gx, float* __restrict__ pw,
                                                            long long pstride) {
    extern __shared__ float s_cols[];   // [groups that hand over][columns], G > 1 only
    __shared__ float s_part[2][kMaxWaves];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int grp = wave / W, part = wave - grp * W;
    int col[NC], n[NC];
    float w[NC][8], aw[NC][8];
#pragma unroll
    for (int k = 0; k < NC; ++k) {
        const int c = (part + k * W) * 64 + lane;
        col[k] = 8 * c;
        n[k] = min(max(H - col[k], 0), 8);
        load_param<TAIL>(weight, wdtype, c, n[k], 1.f, w[k]);
#pragma unroll
        for (int i = 0; i < 8; ++i) aw[k][i] = 0.f;
    }
    const float inv_h = 1.f / (float)H;
    const long long stride = (long long)gridDim.x * G;
    long long row = (long long)blockIdx.x * G + grp;
    constexpr int DEPTH = NC == 1 ? 2 : 1;   // rows in flight, as far as the registers go
    Chunk<TT> nt[DEPTH][NC], na[DEPTH][NC];
    Chunk<YT> ng[DEPTH][NC];
    float nr[DEPTH];
    auto fetch = [&](int d, long long r) {
        const bool ok = r < T;
#pragma unroll
        for (int k = 0; k < NC; ++k) {
            nt[d][k] = fetch_chunk<TAIL>(t + r * H + col[k], ok ? n[k] : 0, H);
            ng[d][k] = fetch_chunk<TAIL>(gy + r * H + col[k], ok ? n[k] : 0, H);
        }
        if (gtot) {
#pragma unroll
            for (int k = 0; k < NC; ++k) na[d][k] = fetch_chunk<TAIL>(gtot + r * H + col[k], ok ? n[k] : 0, H);
        }
        nr[d] = ok ? rstd[r] : 0.f;
    };
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) fetch(d, row + d * stride);
    auto step = [&](int par) {
        const int d = par % DEPTH;
        const bool ok = row < T;
        const float r = nr[d];
        float xh[NC][8], g[NC][8], add[NC][8];
        float b = 0.f;
#pragma unroll
        for (int k = 0; k < NC; ++k) {
            unpack_row<TAIL>(nt[d][k], ok ? n[k] : 0, H, xh[k]);
            unpack_row<TAIL>(ng[d][k], ok ? n[k] : 0, H, g[k]);
            if (gtot) unpack_row<TAIL>(na[d][k], ok ? n[k] : 0, H, add[k]);
        }
        fetch(d, row + DEPTH * stride);
#pragma unroll
        for (int k = 0; k < NC; ++k)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                // past the row's end t and gy read as 0; xh must be 0 there too (0 * inf)
                xh[k][i] = (TAIL ? i < n[k] : n[k] > 0) ? xh[k][i] * r : 0.f;
                aw[k][i] = fmaf(g[k][i], xh[k][i], aw[k][i]);
                g[k][i] *= w[k][i];
                b = fmaf(g[k][i], xh[k][i], b);
            }
        b = wave_sum_dpp(b);
        if (W > 1) {
            if (lane == 0) s_part[par][wave] = b;
            __syncthreads();
            const int peer = lane & 15;
            b = row_sum(peer < W ? s_part[par][grp * W + (peer < W ? peer : 0)] : 0.f);
        }
        b *= inv_h;
        if (ok) {
#pragma unroll
            for (int k = 0; k < NC; ++k) {
                float o[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    o[i] = r * (g[k][i] - xh[k][i] * b);
                    if (gtot) o[i] += add[k][i];
                }
                store_chunk<TAIL>(gx + row * H + col[k], n[k], o);
            }
        }
        row += stride;
    };
    for (long long row0 = (long long)blockIdx.x * G; row0 < T; row0 += 2 * stride) {
        step(0);
        if (row0 + stride < T) step(1);
    }
    if (!pw) return;
    // the row groups' columns join by halves: groups s .. 2s-1 hand theirs to groups 0 .. s-1
    const int span = W * NC * 512;   // columns that a group holds, those past H among them
    for (int half = 8; half >= 1; half >>= 1) {
        if (half >= G) continue;
        if (half < 8 && 2 * half < G) __syncthreads();   // the step before has been read
        float4* at = (float4*)(s_cols + (size_t)span * (grp % half)) + (part * 64 + lane) * 2;
        if (grp >= half && grp < 2 * half && grp < G) {
#pragma unroll
            for (int k = 0; k < NC; ++k)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    at[k * W * 128 + i] = make_float4(aw[k][4 * i], aw[k][4 * i + 1], aw[k][4 * i + 2], aw[k][4 * i + 3]);
        }
        __syncthreads();
        if (grp < half && grp + half < G) {
#pragma unroll
            for (int k = 0; k < NC; ++k)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float4 u = at[k * W * 128 + i];
                    aw[k][4 * i] += u.x; aw[k][4 * i + 1] += u.y; aw[k][4 * i + 2] += u.z; aw[k][4 * i + 3] += u.w;
                }
        }
    }
    if (grp > 0) return;
#pragma unroll
    for (int k = 0; k < NC; ++k) store_chunk<TAIL>(pw + (long long)blockIdx.x * pstride + col[k], n[k], aw[k]);
}

// gw = sum over the nb workgroups' partials [nb][H], in a fixed order (no
// atomics, so a call repeats bit for bit): 64 columns x 16 slices of the
// partials per workgroup, four columns per lane, four partials in flight.
// nb = 0 (no rows) writes zeros.
__global__ __launch_bounds__(256) void k_rms_weight_grad(const float* __restrict__ part, int nb, int H,
                                                         float* __restrict__ gw) {
    __shared__ float s[16][64];
    const int cl = (threadIdx.x & 15) * 4, sl = threadIdx.x >> 4;
    const int c = blockIdx.x * 64 + cl;
    const int n = min(max(H - c, 0), 4);
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    for (int i0 = sl; i0 < nb; i0 += 64) {
        float f[4][4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int i = i0 + 16 * u;
            const float* p = part + (long long)i * H + c;
            if (i < nb && n == 4) {
                const u32x4 q = *(const u32x4_e*)p;
#pragma unroll
                for (int k = 0; k < 4; ++k) f[u][k] = __uint_as_float(q[k]);
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k) f[u][k] = i < nb && k < n ? p[k] : 0.f;
            }
        }
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] += f[u][k];
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) s[sl][cl + k] = v[k];
    __syncthreads();
    const int h = blockIdx.x * 64 + threadIdx.x;
    if (threadIdx.x >= 64 || h >= H) return;
    float o = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) o += s[i][threadIdx.x];
    gw[h] = o;
}

static_assert(64 * 8 * kMaxWaves * 4 == MOE_NORM_MAX_H, "norm row limit: 4 steps of 16 wavefronts");
constexpr int kBackwardBlocks = 256;   // the scratch's size is a function of the shape alone
constexpr int kForwardWide = 8, kBackwardWide = kMaxWaves;

// Steps per lane and wavefronts per row: at most `wide` wavefronts share a row
// while 2 steps do.
void row_shape(int H, int wide, int* NC, int* W) {
    const int groups = (H + 511) / 512;   // 64-lane groups of chunks
    *NC = groups <= wide ? 1 : groups <= 2 * kMaxWaves ? 2 : 4;
    *W = (groups + *NC - 1) / *NC;
}

// Workgroups of the backward pass: one row per row group up to 64 of them, two from there on.
int backward_blocks(int T, int G) {
    const long long one = ((long long)T + G - 1) / G, two = (one + 1) / 2;
    return (int)(one <= 64 ? one : two <= 64 ? 64 : two < kBackwardBlocks ? two : kBackwardBlocks);
}

// Calls go with the two row types, the steps per lane and whether rows end
// inside a chunk.
template <typename F>
void by_variant(int a_dtype, int b_dtype, int NC, int H, F go) {
    auto by_nc = [&](auto at, auto bt) {
        auto by_tail = [&](auto nc) {
            if (H % 8) go(at, bt, nc, std::true_type{});
            else go(at, bt, nc, std::false_type{});
        };
        if (NC == 1) by_tail(std::integral_constant<int, 1>{});
        else if (NC == 2) by_tail(std::integral_constant<int, 2>{});
        else by_tail(std::integral_constant<int, 4>{});
    };
    const bool ab = a_dtype == MOE_BF16, bb = b_dtype == MOE_BF16;
    if (ab && bb) by_nc(uint16_t{}, uint16_t{});
    else if (ab) by_nc(uint16_t{}, float{});
    else if (bb) by_nc(float{}, uint16_t{});
    else by_nc(float{}, float{});
}

size_t width(int dtype) { return dtype == MOE_BF16 ? 2 : 4; }

}  // namespace

size_t rms_norm_backward_scratch_bytes(int T, int H) {
    int NC, W;
    row_shape(H, kBackwardWide, &NC, &W);
    return (size_t)backward_blocks(T, kMaxWaves / W) * H * sizeof(float);
}

hipError_t launch_rms_norm(int T, int H, int x_dtype, int r_dtype, int y_dtype, int w_dtype, const void* x,
                           const void* residual, const void* weight, float eps, void* y, void* codes, float* scales,
                           void* total, float* rstd, int num_cu, hipStream_t s) {
    if (T == 0) return hipSuccess;
    int NC, W;
    row_shape(H, kForwardWide, &NC, &W);
    const int G = W >= 4 ? 1 : 4 / W;
    const int per_cu = max(1, 32 / (W * G));
    // outputs past the 32 MB of L2 leave it anyway: nontemporal stores, as the layer norm's
    const size_t bytes = (size_t)T * H * ((y ? width(y_dtype) : 0) + (codes ? 1 : 0) + (total ? width(r_dtype) : 0));
    const bool stream = bytes > (32u << 20);
    const long long want = ((long long)T + G - 1) / G, most = (long long)num_cu * per_cu;
    const unsigned grid = (unsigned)(want < most ? want : most);
    const Outputs o = {y, (uint8_t*)codes, scales, total, rstd, y_dtype == MOE_BF16};
    auto go = [&](auto xt, auto rt, auto nc, auto tail) {
        using XT = decltype(xt);
        using RT = decltype(rt);
        auto launch = [&](auto st) {
            hipLaunchKernelGGL((k_rms_norm<XT, RT, decltype(nc)::value, decltype(tail)::value, decltype(st)::value>),
                               dim3(grid), dim3(64 * W * G), 0, s, (const XT*)x, (const RT*)residual, T, H, W, G,
                               weight, w_dtype, eps, o);
        };
        if (stream) launch(std::true_type{});
        else launch(std::false_type{});
    };
    by_variant(x_dtype, r_dtype, NC, H, go);
    return hipGetLastError();
}

hipError_t launch_rms_norm_backward(int T, int H, int t_dtype, int y_dtype, int w_dtype, const void* gy,
                                    const void* total, const float* rstd, const void* weight, const void* grad_total,
                                    void* gx, float* gw, void* scratch, hipStream_t s) {
    int NC, W;
    row_shape(H, kBackwardWide, &NC, &W);
    const int G = kMaxWaves / W;
    const int nb = T > 0 ? backward_blocks(T, G) : 0;
    if (nb > 0) {
        float* pw = !gw ? nullptr : nb == 1 ? gw : (float*)scratch;
        int half = 0;   // groups of the first joining step
        for (int i = 8; i >= 1 && !half; i >>= 1)
            if (i < G) half = i;
        const size_t lds = gw ? (size_t)half * W * NC * 512 * sizeof(float) : 0;
        auto go = [&](auto tt, auto yt, auto nc, auto tail) {
            using TT = decltype(tt);
            using YT = decltype(yt);
            hipLaunchKernelGGL((k_rms_norm_backward<TT, YT, decltype(nc)::value, decltype(tail)::value>), dim3(nb),
                               dim3(64 * W * G), lds, s, (const YT*)gy, (const TT*)total, rstd, (const TT*)grad_total,
                               T, H, W, G, weight, w_dtype, (TT*)gx, pw, (long long)H);
        };
        by_variant(t_dtype, y_dtype, NC, H, go);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess || nb == 1) return e;
    }
    if (!gw) return hipSuccess;
    hipLaunchKernelGGL(k_rms_weight_grad, dim3((unsigned)((H + 63) / 64)), dim3(256), 0, s, (const float*)scratch, nb,
                       H, gw);
    return hipGetLastError();
}

}  // namespace moe
