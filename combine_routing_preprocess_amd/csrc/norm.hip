// Layer norm of token rows, forward and backward, with the reduction of the
// weight's and bias's gradients: the norm in front of the MoE layer.
//
//   forward   y = (x - mu) * r * w + b,  mu = mean(x),  r = 1 / sqrt(mean((x - mu)^2) + eps)
//   backward  xh = (x - mu) * r,  g = gy * w,
//             gx = r * (g - mean(g) - xh * mean(g * xh)),
//             gw = sum over the rows of gy * xh,  gb = sum over the rows of gy
//
// Both directions are bound by HBM: the forward reads x and writes y once, the
// backward reads x and gy and writes gx once.  A row is held in registers by W
// wavefronts, 8 elements (one chunk) per lane and step, at most NC steps; G
// rows share a workgroup when they are short.  Workgroups walk the rows with a
// stride, so weight and bias are loaded once per workgroup, and the loads of
// the next two rows are in flight during the current row's reductions.
// Measured on MI355X, 8192 x 7168 bf16, in long runs of calls: forward 47.0 us
// (5.0 TB/s), backward with the sum of its parameter gradients 73.8 us (4.8
// TB/s), where a 1 GiB device copy runs at 5.08 TB/s.  The forward takes 2
// chunks per lane there (7 wavefronts per row), the backward one, for the
// column sums that each lane keeps (two chunks spill: 126 us; so do the two
// and four of wider rows, 57 M elements as 16384 columns in 158 us).
//
// Statistics are fp32 and need one barrier per row.  Each wavefront takes the
// mean m of its own part, then the sum e and the square sum q of what is left,
// x - m: e is the rounding that m carries, so the part's mean is m + e / n and
// its centred square sum q - e^2 / n, without the cancellation of E[x^2] -
// mu^2.  The parts join by the exact rule for means and square sums of
// disjoint sets, relative to the first part's m, so that a row whose offset is
// far larger than its spread keeps its precision.
//
// Rows need no alignment beyond their element's: chunks are loaded and stored
// as 16-byte accesses at element alignment, which the memory pipeline takes
// (the whole-line rows of a width that is a multiple of 8 are just the fast
// case), and a last partial chunk is loaded from the row's end back and stored
// element by element.
#include "row_chunks.h"
#include "wave_ops.h"

namespace moe {
namespace {

using ops::Chunk;
using ops::fetch_chunk;
using ops::load_chunk;
using ops::load_param;
using ops::readlane;
using ops::row_sum;
using ops::store_chunk;
using ops::u32x4_e;
using ops::unpack_row;
using ops::wave_sum_dpp;

constexpr int kMaxWaves = 16;   // wavefronts of a workgroup

// Elements that wavefront i of a row's W holds in all its NC steps.
template <int NC>
__device__ __forceinline__ int part_elems(int H, int W, int i) {
    int n = 0;
#pragma unroll
    for (int k = 0; k < NC; ++k) n += min(max(H - 512 * (i + k * W), 0), 512);
    return n;
}

template <typename XT, typename YT, int NC, bool TAIL, bool STREAM>
__global__ __launch_bounds__(1024) void k_layer_norm(const XT* __restrict__ x, int T, int H, int W, int G,
                                                     const void* __restrict__ weight, const void* __restrict__ bias,
                                                     int wdtype, float eps, YT* __restrict__ y,
                                                     float* __restrict__ mean, float* __restrict__ rstd) {
    __shared__ float4 s_part[2][kMaxWaves];   // each part's m, e, q
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int grp = wave / W, part = wave - grp * W;
    constexpr bool KEEP = NC <= 2;   // parameters and the next row in registers
    int col[NC], n[NC];
    float w[KEEP ? NC : 1][8], b[KEEP ? NC : 1][8];
#pragma unroll
    for (int k = 0; k < NC; ++k) {
        const int c = (part + k * W) * 64 + lane;
        col[k] = 8 * c;
        n[k] = min(max(H - col[k], 0), 8);
        if (KEEP) {
            load_param<TAIL>(weight, wdtype, c, n[k], 1.f, w[KEEP ? k : 0]);
            load_param<TAIL>(bias, wdtype, c, n[k], 0.f, b[KEEP ? k : 0]);
        }
    }
    const float inv_h = 1.f / (float)H;
    const float inv_mine = 1.f / (float)part_elems<NC>(H, W, part);
    const int peer = lane & 15;                       // the part of the row that this lane joins
    const float peer_n = peer < W ? (float)part_elems<NC>(H, W, peer) : 0.f;
    const long long stride = (long long)gridDim.x * G;
    long long row = (long long)blockIdx.x * G + grp;
    // rows in flight: each step takes the row in its slot and loads the one two steps on into it
    Chunk<XT> slot[2][NC];
    auto fetch = [&](Chunk<XT> (&c)[NC], long long r) {
#pragma unroll
        for (int k = 0; k < NC; ++k) c[k] = fetch_chunk<TAIL>(x + r * H + col[k], r < T ? n[k] : 0, H);
    };
    if (KEEP) {
        fetch(slot[0], row);
        fetch(slot[1], row + stride);
    }
    auto step = [&](int par) {
        Chunk<XT> (&next)[NC] = slot[par];
        const bool ok = row < T;
        float v[NC][8];
        if (!KEEP) fetch(next, row);
#pragma unroll
        for (int k = 0; k < NC; ++k) unpack_row<TAIL>(next[k], ok ? n[k] : 0, H, v[k]);
        if (KEEP) fetch(next, row + 2 * stride);
        float s = 0.f;
#pragma unroll
        for (int k = 0; k < NC; ++k)
#pragma unroll
            for (int i = 0; i < 8; ++i) s += v[k][i];
        // through a scalar register: m is one rounded value everywhere below (contracted into v - m, the
        // product would enter unrounded there and rounded elsewhere, and e would not be its rounding)
        float m = readlane(wave_sum_dpp(s) * inv_mine, 0);
        float e = 0.f, q = 0.f;
#pragma unroll
        for (int k = 0; k < NC; ++k)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float d = (TAIL ? i < n[k] : n[k] > 0) ? v[k][i] - m : 0.f;
                e += d;
                q = fmaf(d, d, q);
            }
        e = wave_sum_dpp(e);
        q = wave_sum_dpp(q);
        float delta, sq;   // mean relative to m, centred square sum of the row
        if (W == 1) {
            delta = e * inv_h;
            sq = q - e * delta;
        } else {
            if (lane == 0) s_part[par][wave] = make_float4(m, e, q, 0.f);
            // one barrier: who still reads the other parity passed its barrier before this row's writes
            __syncthreads();
            const float4 p = s_part[par][grp * W + (peer < W ? peer : 0)];
            m = readlane(p.x, 0);
            const float shift = p.x - m;
            delta = row_sum(peer < W ? fmaf(peer_n, shift, p.y) : 0.f) * inv_h;
            const float off = shift - delta;          // the part's m relative to the row's mean
            sq = row_sum(peer < W ? fmaf(off, fmaf(peer_n, off, 2.f * p.y), p.z) : 0.f);
        }
        if (sq < 0.f) sq = 0.f;   // NaN stays
        const float r = 1.f / sqrtf(fmaf(sq, inv_h, eps));
        if (ok) {
#pragma unroll
            for (int k = 0; k < NC; ++k) {
                float o[8];
                const int kk = KEEP ? k : 0;
                if (!KEEP) {
                    load_param<TAIL>(weight, wdtype, col[k] / 8, n[k], 1.f, w[0]);
                    load_param<TAIL>(bias, wdtype, col[k] / 8, n[k], 0.f, b[0]);
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) o[i] = fmaf(((v[k][i] - m) - delta) * r, w[kk][i], b[kk][i]);
                store_chunk<TAIL, STREAM>(y + row * H + col[k], n[k], o);
            }
            if (part == 0 && lane == 0) {
                if (mean) mean[row] = m + delta;
                if (rstd) rstd[row] = r;
            }
        }
        row += stride;
    };
    // the workgroup's rows advance together, so every wavefront meets the barriers
    for (long long row0 = (long long)blockIdx.x * G; row0 < T; row0 += 2 * stride) {
        step(0);
        if (row0 + stride < T) step(1);
    }
}

// Row gradients of the workgroup's rows, and its sums of gy * xh and gy per
// column into part[2 * blockIdx][H] and part[2 * blockIdx + 1][H] (straight
// into gw and gb when one workgroup has every row).
template <typename XT, typename YT, int NC, bool TAIL>
__global__ __launch_bounds__(1024) void k_layer_norm_backward(const YT* __restrict__ gy, const XT* __restrict__ x,
                                                              const float* __restrict__ mean,
                                                              const float* __restrict__ rstd, int T, int H, int W,
                                                              int G, const void* __restrict__ weight, int wdtype,
                                                              XT* __restrict__ gx, float* __restrict__ pw,
                                                              float* __restrict__ pb, long long pstride) {
    extern __shared__ float s_cols[];   // [groups that hand over][2][columns], G > 1 only
    __shared__ float2 s_part[2][kMaxWaves];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int grp = wave / W, part = wave - grp * W;
    int col[NC], n[NC];
    float w[NC][8], aw[NC][8], ab[NC][8];
#pragma unroll
    for (int k = 0; k < NC; ++k) {
        const int c = (part + k * W) * 64 + lane;
        col[k] = 8 * c;
        n[k] = min(max(H - col[k], 0), 8);
        load_param<TAIL>(weight, wdtype, c, n[k], 1.f, w[k]);
#pragma unroll
        for (int i = 0; i < 8; ++i) aw[k][i] = ab[k][i] = 0.f;
    }
    const float inv_h = 1.f / (float)H;
    const long long stride = (long long)gridDim.x * G;
    long long row = (long long)blockIdx.x * G + grp;
    constexpr int DEPTH = NC == 1 ? 2 : 1;   // rows in flight, as far as the registers go
    Chunk<XT> nx[DEPTH][NC];
    Chunk<YT> ng[DEPTH][NC];
    float nm[DEPTH], nr[DEPTH];
    auto fetch = [&](int d, long long r) {
        const bool ok = r < T;
#pragma unroll
        for (int k = 0; k < NC; ++k) {
            nx[d][k] = fetch_chunk<TAIL>(x + r * H + col[k], ok ? n[k] : 0, H);
            ng[d][k] = fetch_chunk<TAIL>(gy + r * H + col[k], ok ? n[k] : 0, H);
        }
        nm[d] = ok ? mean[r] : 0.f;
        nr[d] = ok ? rstd[r] : 0.f;
    };
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) fetch(d, row + d * stride);
    auto step = [&](int par) {
        const int d = par % DEPTH;
        const bool ok = row < T;
        const float m = nm[d], r = nr[d];
        float xh[NC][8], g[NC][8];
        float a = 0.f, b = 0.f;
#pragma unroll
        for (int k = 0; k < NC; ++k) {
            unpack_row<TAIL>(nx[d][k], ok ? n[k] : 0, H, xh[k]);
            unpack_row<TAIL>(ng[d][k], ok ? n[k] : 0, H, g[k]);
        }
        fetch(d, row + DEPTH * stride);
#pragma unroll
        for (int k = 0; k < NC; ++k)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                // past the row's end gy reads as 0; xh must be 0 there too (0 * inf)
                xh[k][i] = (TAIL ? i < n[k] : n[k] > 0) ? (xh[k][i] - m) * r : 0.f;
                aw[k][i] = fmaf(g[k][i], xh[k][i], aw[k][i]);
                ab[k][i] += g[k][i];
                g[k][i] *= w[k][i];
                a += g[k][i];
                b = fmaf(g[k][i], xh[k][i], b);
            }
        a = wave_sum_dpp(a);
        b = wave_sum_dpp(b);
        if (W > 1) {
            if (lane == 0) s_part[par][wave] = make_float2(a, b);
            __syncthreads();
            const int peer = lane & 15;
            const float2 p = s_part[par][grp * W + (peer < W ? peer : 0)];
            a = row_sum(peer < W ? p.x : 0.f);
            b = row_sum(peer < W ? p.y : 0.f);
        }
        a *= inv_h;
        b *= inv_h;
        if (ok) {
#pragma unroll
            for (int k = 0; k < NC; ++k) {
                float o[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) o[i] = r * (g[k][i] - a - xh[k][i] * b);
                store_chunk<TAIL>(gx + row * H + col[k], n[k], o);
            }
        }
        row += stride;
    };
    for (long long row0 = (long long)blockIdx.x * G; row0 < T; row0 += 2 * stride) {
        step(0);
        if (row0 + stride < T) step(1);
    }
    if (!pw && !pb) return;
    // the row groups' columns join by halves: groups s .. 2s-1 hand theirs to groups 0 .. s-1
    const int span = W * NC * 512;   // columns that a group holds, those past H among them
    for (int half = 8; half >= 1; half >>= 1) {
        if (half >= G) continue;
        if (half < 8 && 2 * half < G) __syncthreads();   // the step before has been read
        float4* at = (float4*)(s_cols + (size_t)2 * span * (grp % half)) + (part * 64 + lane) * 2;
        if (grp >= half && grp < 2 * half && grp < G) {
#pragma unroll
            for (int k = 0; k < NC; ++k)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    at[k * W * 128 + i] = make_float4(aw[k][4 * i], aw[k][4 * i + 1], aw[k][4 * i + 2], aw[k][4 * i + 3]);
                    at[span / 4 + k * W * 128 + i] = make_float4(ab[k][4 * i], ab[k][4 * i + 1], ab[k][4 * i + 2],
                                                                 ab[k][4 * i + 3]);
                }
        }
        __syncthreads();
        if (grp < half && grp + half < G) {
#pragma unroll
            for (int k = 0; k < NC; ++k)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float4 u = at[k * W * 128 + i], v = at[span / 4 + k * W * 128 + i];
                    aw[k][4 * i] += u.x; aw[k][4 * i + 1] += u.y; aw[k][4 * i + 2] += u.z; aw[k][4 * i + 3] += u.w;
                    ab[k][4 * i] += v.x; ab[k][4 * i + 1] += v.y; ab[k][4 * i + 2] += v.z; ab[k][4 * i + 3] += v.w;
                }
        }
    }
    if (grp > 0) return;
#pragma unroll
    for (int k = 0; k < NC; ++k) {
        if (pw) store_chunk<TAIL>(pw + (long long)blockIdx.x * pstride + col[k], n[k], aw[k]);
        if (pb) store_chunk<TAIL>(pb + (long long)blockIdx.x * pstride + col[k], n[k], ab[k]);
    }
}

// gw / gb = sum over the nb workgroups' partials [nb][2][H], in a fixed order
// (no atomics, so a call repeats bit for bit): 64 columns x 16 slices of the
// partials per workgroup, four columns per lane, four partials in flight.
// nb = 0 (no rows) writes zeros.
__global__ __launch_bounds__(256) void k_norm_param_grads(const float* __restrict__ part, int nb, int H,
                                                          float* __restrict__ gw, float* __restrict__ gb) {
    __shared__ float s[16][64];
    const int cl = (threadIdx.x & 15) * 4, sl = threadIdx.x >> 4;
    const int c = blockIdx.x * 64 + cl;   // column of [2][H]
    const int n = min(max(2 * H - c, 0), 4);
    const long long stride = 2ll * H;
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    for (int i0 = sl; i0 < nb; i0 += 64) {
        float f[4][4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int i = i0 + 16 * u;
            const float* p = part + i * stride + c;
            if (i < nb && n == 4) {
                const u32x4 w = *(const u32x4_e*)p;
#pragma unroll
                for (int k = 0; k < 4; ++k) f[u][k] = __uint_as_float(w[k]);
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
    if (threadIdx.x >= 64 || h >= 2 * H) return;
    float o = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) o += s[i][threadIdx.x];
    if (h < H) {
        if (gw) gw[h] = o;
    } else if (gb) {
        gb[h - H] = o;
    }
}

constexpr int kMaxRowElems = 64 * 8 * kMaxWaves * 4;   // 4 steps of 16 wavefronts
static_assert(kMaxRowElems == MOE_NORM_MAX_H, "norm row limit");
// One workgroup per CU of the whole chip walks the rows, whatever part of it the call runs on: the scratch's size is a
// function of the shape alone.  8192 x 7168 bf16: 72.8 us, 80.6 with 512 and 115.7 with 128; 114688 x 512: 68.9,
// 75.7 and 88.0.
constexpr int kBackwardBlocks = 256;

// Steps per lane and wavefronts per row: at most `wide` wavefronts share a row
// while 2 steps do.  The forward's 8 against 16 and 4, 57 M bf16 elements again
// and again: 2560 columns 49.2 us (16: 48.0, 4: 42.1), 4096 45.8 (45.1, 41.5),
// 4608 47.7 (47.4, 48.1), 5120 45.7 (58.4, 45.4), 6144 46.8 (45.5, 47.1), 7168
// 41.2 (46.7, 40.4), 8192 40.2 (44.3, 40.4); 256 rows of 2560 3.3 us (4: 3.6),
// of 4096 3.5 (3.8).  16 loses from 5120 columns on; 4 wins 10 to 14 % in large
// batches of 2560 to 4096 columns and loses 8 % in small ones, where 8 stays.
void row_shape(int H, int wide, int* NC, int* W) {
    const int groups = (H + 511) / 512;   // 64-lane groups of chunks
    *NC = groups <= wide ? 1 : groups <= 2 * kMaxWaves ? 2 : 4;
    *W = (groups + *NC - 1) / *NC;
}
constexpr int kForwardWide = 8, kBackwardWide = kMaxWaves;

// Workgroups of the backward pass.  Each writes 2 H partial sums, the traffic of two bf16 rows and more; rows in
// series cost a workgroup about a microsecond each while the GPU is not full.  So one row per row group up to 64
// workgroups, two from there on (256 rows of 7168: 11.5 us with two, 13.1 with one, 12.2 with four).
int backward_blocks(int T, int G) {
    const long long one = ((long long)T + G - 1) / G, two = (one + 1) / 2;
    return (int)(one <= 64 ? one : two <= 64 ? 64 : two < kBackwardBlocks ? two : kBackwardBlocks);
}

// Calls go with the row types, the steps per lane and whether rows end inside
// a chunk.
template <typename F>
void by_variant(int x_dtype, int y_dtype, int NC, int H, F go) {
    auto by_nc = [&](auto xt, auto yt) {
        auto by_tail = [&](auto nc) {
            if (H % 8) go(xt, yt, nc, std::true_type{});
            else go(xt, yt, nc, std::false_type{});
        };
        if (NC == 1) by_tail(std::integral_constant<int, 1>{});
        else if (NC == 2) by_tail(std::integral_constant<int, 2>{});
        else by_tail(std::integral_constant<int, 4>{});
    };
    const bool xb = x_dtype == MOE_BF16, yb = y_dtype == MOE_BF16;
    if (xb && yb) by_nc(uint16_t{}, uint16_t{});
    else if (xb) by_nc(uint16_t{}, float{});
    else if (yb) by_nc(float{}, uint16_t{});
    else by_nc(float{}, float{});
}

}  // namespace

size_t norm_backward_scratch_bytes(int T, int H) {
    int NC, W;
    row_shape(H, kBackwardWide, &NC, &W);
    return (size_t)backward_blocks(T, kMaxWaves / W) * 2 * H * sizeof(float);
}

hipError_t launch_layer_norm(int T, int H, int x_dtype, int y_dtype, int w_dtype, const void* x, const void* weight,
                             const void* bias, float eps, void* y, float* mean, float* rstd, int num_cu,
                             hipStream_t s) {
    if (T == 0) return hipSuccess;
    int NC, W;
    row_shape(H, kForwardWide, &NC, &W);
    const int G = W >= 4 ? 1 : 4 / W;
    const int per_cu = max(1, 32 / (W * G));
    // Outputs past the 32 MB of L2 leave it anyway: nontemporal stores; smaller ones stay for the router's product and
    // the dispatch that read them next.  8192 x 7168 bf16 with and without, and with who reads the rows: alone 51.3 and
    // 55.0 us, with the router's product 136.4 and 135.5, with the dispatch 248 and 240 (the rows stay in the last-level
    // cache), with product, gate, routing and dispatch as the layer runs them 337 and 340
    const bool stream = (long long)T * H * (y_dtype == MOE_BF16 ? 2 : 4) > (32ll << 20);
    const long long want = ((long long)T + G - 1) / G, most = (long long)num_cu * per_cu;
    const unsigned grid = (unsigned)(want < most ? want : most);
    auto go = [&](auto xt, auto yt, auto nc, auto tail) {
        using XT = decltype(xt);
        using YT = decltype(yt);
        auto launch = [&](auto st) {
            hipLaunchKernelGGL((k_layer_norm<XT, YT, decltype(nc)::value, decltype(tail)::value, decltype(st)::value>),
                               dim3(grid), dim3(64 * W * G), 0, s, (const XT*)x, T, H, W, G, weight, bias, w_dtype,
                               eps, (YT*)y, mean, rstd);
        };
        if (stream) launch(std::true_type{});
        else launch(std::false_type{});
    };
    by_variant(x_dtype, y_dtype, NC, H, go);
    return hipGetLastError();
}

hipError_t launch_layer_norm_backward(int T, int H, int x_dtype, int y_dtype, int w_dtype, const void* gy,
                                      const void* x, const float* mean, const float* rstd, const void* weight,
                                      void* gx, float* gw, float* gb, void* scratch, hipStream_t s) {
    int NC, W;
    row_shape(H, kBackwardWide, &NC, &W);
    const int G = kMaxWaves / W;
    const int nb = T > 0 ? backward_blocks(T, G) : 0;
    const bool params = gw || gb;
    if (nb > 0) {
        float* part = (float*)scratch;
        float* pw = nb == 1 ? gw : params ? part : nullptr;
        float* pb = nb == 1 ? gb : params ? part + H : nullptr;
        int half = 0;   // groups of the first joining step
        for (int i = 8; i >= 1 && !half; i >>= 1)
            if (i < G) half = i;
        const size_t lds = params ? (size_t)half * 2 * W * NC * 512 * sizeof(float) : 0;
        auto go = [&](auto xt, auto yt, auto nc, auto tail) {
            using XT = decltype(xt);
            using YT = decltype(yt);
            hipLaunchKernelGGL((k_layer_norm_backward<XT, YT, decltype(nc)::value, decltype(tail)::value>), dim3(nb), dim3(64 * W * G), lds,
                               s, (const YT*)gy, (const XT*)x, mean, rstd, T, H, W, G, weight, w_dtype, (XT*)gx, pw,
                               pb, 2ll * H);
        };
        by_variant(x_dtype, y_dtype, NC, H, go);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess || nb == 1) return e;
    }
    if (!params) return hipSuccess;
    hipLaunchKernelGGL(k_norm_param_grads, dim3((unsigned)((2 * H + 63) / 64)), dim3(256), 0, s,
                       (const float*)scratch, nb, H, gw, gb);
    return hipGetLastError();
}

}  // namespace moe
