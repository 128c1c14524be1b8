// Layer norm over rows, forward and backward, sm_103a.
//
// Forward, per row x of d channels (biased variance):
//     mean = sum x / d,  var = sum (x - mean)^2 / d,  rstd = 1 / sqrt(var + eps)
//     y = (x - mean) * rstd * w + b
// Backward, from dy and the saved mean and rstd, with z = (x - mean) * rstd and
// g = dy * w:
//     dx = rstd * (g - sum(g) / d - z * sum(g z) / d)
//     dw = sum over rows of dy * z,   db = sum over rows of dy
// w and b have one row for every group_rows rows of x (a modulation per sample)
// or one row for all.  Rows are stored in 16 or 32 bits; every sum, mean, rstd,
// dw and db is fp32, and y and dx are rounded once, to nearest even.
//
// Both are bound by HBM: x is read once and y written once (forward), x and dy
// are read once and dx written once (backward).  A row is held by a team of
// threads in registers, as 16-byte chunks in the storage type, so the second
// look at it (the centred squares; dx after the two sums) costs no traffic.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "kq_device.cuh"
#include "kq_internal.h"

namespace kq {
namespace {

// ---- 16-byte chunks of the storage types ---------------------------------------

template <int FMT>
struct Chunk {
    static constexpr int kN = FMT == KQ_F32 ? 4 : 8;   // elements per chunk
    static constexpr int kSize = FMT == KQ_F32 ? 4 : 2;
};

template <int FMT>
__device__ __forceinline__ void unpack(const uint4 &r, float (&v)[Chunk<FMT>::kN])
{
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (FMT == KQ_F32) {
            v[i] = __uint_as_float(w[i]);
        } else if constexpr (FMT == KQ_BF16) {
            v[2 * i] = bf16_lo(w[i]);
            v[2 * i + 1] = bf16_hi(w[i]);
        } else {
            v[2 * i] = f16_lo(w[i]);
            v[2 * i + 1] = f16_hi(w[i]);
        }
    }
}

template <int FMT>
__device__ __forceinline__ uint4 pack(const float (&v)[Chunk<FMT>::kN])
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (FMT == KQ_F32) {
            w[i] = __float_as_uint(v[i]);
        } else if constexpr (FMT == KQ_BF16) {
            const __nv_bfloat162 p = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&p);
        } else {
            const __half2 p = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&p);
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Streaming load: x and dy are read once.
__device__ __forceinline__ uint4 ldg_stream(const void *p)
{
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// Chunk `c` of a row of d elements: whole 16-byte chunks are loaded as such,
// the ragged end element by element (zeros past d).
template <int FMT>
__device__ __forceinline__ uint4 load_chunk(const uint8_t *row, int c, int d)
{
    constexpr int N = Chunk<FMT>::kN;
    if ((c + 1) * N <= d) return ldg_stream(row + 16 * c);
    uint32_t w[4] = {0, 0, 0, 0};
    for (int i = 0; c * N + i < d; ++i) {
        if constexpr (FMT == KQ_F32)
            w[i] = reinterpret_cast<const uint32_t *>(row)[c * N + i];
        else
            w[i >> 1] |= static_cast<uint32_t>(reinterpret_cast<const uint16_t *>(row)[c * N + i])
                         << (16 * (i & 1));
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

template <int FMT>
__device__ __forceinline__ void store_chunk(uint8_t *row, int c, int d, const uint4 &r)
{
    constexpr int N = Chunk<FMT>::kN;
    if ((c + 1) * N <= d) {
        stg128_cs(row + 16 * c, r);
        return;
    }
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < N; ++i) {
        if (c * N + i >= d) break;
        if constexpr (FMT == KQ_F32)
            reinterpret_cast<uint32_t *>(row)[c * N + i] = w[i];
        else
            reinterpret_cast<uint16_t *>(row)[c * N + i] =
                static_cast<uint16_t>(w[i >> 1] >> (16 * (i & 1)));
    }
}

// The fp32 parameters of chunk c; `vec`: their row is 16-byte aligned.
template <int N>
__device__ __forceinline__ void load_param(const float *p, int c, int d, bool vec, float fill,
                                           float (&v)[N])
{
    if (p == nullptr) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = fill;
    } else if (vec && (c + 1) * N <= d) {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const float4 f = __ldg(reinterpret_cast<const float4 *>(p + c * N + i));
            v[i] = f.x;
            v[i + 1] = f.y;
            v[i + 2] = f.z;
            v[i + 3] = f.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = c * N + i < d ? __ldg(p + c * N + i) : 0.f;
    }
}

// Sums `v` over a team of TPR threads (whole warps of the block); `red` holds
// the warps' partial sums of one row, and `buf` alternates from row to row so
// that one barrier per sum is enough.
template <int TPR>
__device__ __forceinline__ float2 team_sum(float2 v, float2 *red, int team, int buf)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
        v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
    }
    if constexpr (TPR > 32) {
        constexpr int W = TPR / 32;
        const int warp = (threadIdx.x % TPR) >> 5, lane = threadIdx.x & 31;
        float2 *r = red + (team * 2 + buf) * W;
        if (lane == 0) r[warp] = v;
        named_barrier(1 + static_cast<uint32_t>(team), TPR);
        v = lane < W ? r[lane] : make_float2(0.f, 0.f);
#pragma unroll
        for (int o = W / 2; o > 0; o >>= 1) {
            v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
            v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
        }
        v.x = __shfl_sync(0xffffffffu, v.x, 0);
        v.y = __shfl_sync(0xffffffffu, v.y, 0);
    }
    return v;
}

struct NormArgs {
    const uint8_t *x, *dy;       // rows of x (and dy); pitches in bytes
    int64_t xpitch, dypitch;
    uint8_t *y;                  // y (forward) or dx (backward, may be null)
    int64_t ypitch;
    int64_t m;
    int d;
    const float *weight, *bias;  // [groups][d] or null
    int64_t group_rows;          // > 0
    int vec;                     // every parameter row is 16-byte aligned
    float eps, inv_d;
    float *mean, *rstd;          // written (forward, may be null) or read (backward)
    int parts;                   // backward: row slices per group
    float *dweight, *dbias;      // backward, [groups][d], may be null
    float *work;                 // backward: [groups][parts][2][d] when parts > 1
};

template <int TPR>
struct Team {
    static constexpr int kPerBlock = TPR >= 128 ? 1 : 128 / TPR;
    static constexpr int kThreads = TPR * kPerBlock;
    static constexpr int kRed = TPR > 32 ? kPerBlock * 2 * (TPR / 32) : 1;
};

// ---- forward --------------------------------------------------------------------

template <int FMT, int TPR, int VPT>
__global__ void __launch_bounds__(Team<TPR>::kThreads) norm_forward_kernel(const NormArgs g)
{
    constexpr int N = Chunk<FMT>::kN;
    __shared__ float2 red[Team<TPR>::kRed];
    const int team = threadIdx.x / TPR, t = threadIdx.x % TPR;
    const int64_t row = blockIdx.x * static_cast<int64_t>(Team<TPR>::kPerBlock) + team;
    grid_dependency_wait();
    if (row >= g.m) return;
    const int nc = (g.d + N - 1) / N;
    const uint8_t *xr = g.x + row * g.xpitch;
    uint4 raw[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = t + i * TPR;
        raw[i] = c < nc ? load_chunk<FMT>(xr, c, g.d) : make_uint4(0, 0, 0, 0);
    }
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        float v[N];
        unpack<FMT>(raw[i], v);
#pragma unroll
        for (int j = 0; j < N; ++j) s += v[j];
    }
    const float mean = team_sum<TPR>(make_float2(s, 0.f), red, team, 0).x * g.inv_d;
    float q = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = t + i * TPR;
        float v[N];
        unpack<FMT>(raw[i], v);
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const float e = v[j] - mean;
            if (c * N + j < g.d) q = fmaf(e, e, q);
        }
    }
    const float var = team_sum<TPR>(make_float2(q, 0.f), red, team, 1).x * g.inv_d;
    const float rstd = 1.0f / sqrtf(var + g.eps);
    const int64_t grp = row / g.group_rows;
    const float *w = g.weight ? g.weight + grp * g.d : nullptr;
    const float *b = g.bias ? g.bias + grp * g.d : nullptr;
    uint8_t *yr = g.y + row * g.ypitch;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = t + i * TPR;
        if (c < nc) {
            float v[N], wv[N], bv[N];
            unpack<FMT>(raw[i], v);
            load_param<N>(w, c, g.d, g.vec, 1.f, wv);
            load_param<N>(b, c, g.d, g.vec, 0.f, bv);
#pragma unroll
            for (int j = 0; j < N; ++j) v[j] = fmaf((v[j] - mean) * rstd, wv[j], bv[j]);
            store_chunk<FMT>(yr, c, g.d, pack<FMT>(v));
        }
    }
    if (t == 0) {
        if (g.mean) g.mean[row] = mean;
        if (g.rstd) g.rstd[row] = rstd;
    }
}

// ---- backward -------------------------------------------------------------------

// A block takes slice p of group gi: teams walk its rows, keep the columns'
// sums of dy * z and dy in registers, and add them up at the end (in team
// order: the result does not depend on timing).
template <int FMT, int TPR, int VPT>
__global__ void __launch_bounds__(Team<TPR>::kThreads) norm_backward_kernel(const NormArgs g)
{
    constexpr int N = Chunk<FMT>::kN, PB = Team<TPR>::kPerBlock;
    __shared__ float2 red[Team<TPR>::kRed];
    extern __shared__ float sums[];              // [2][d], PB > 1 only
    const int team = threadIdx.x / TPR, t = threadIdx.x % TPR;
    const int64_t gi = blockIdx.x / static_cast<unsigned>(g.parts);
    const int p = static_cast<int>(blockIdx.x % static_cast<unsigned>(g.parts));
    const int64_t first = gi * g.group_rows, last = min(g.m, first + g.group_rows);
    const int nc = (g.d + N - 1) / N;
    const float *w = g.weight ? g.weight + gi * g.d : nullptr;
    float aw[VPT][N], ab[VPT][N];
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int j = 0; j < N; ++j) aw[i][j] = ab[i][j] = 0.f;
    grid_dependency_wait();
    int buf = 0;
    for (int64_t row = first + static_cast<int64_t>(p) * PB + team; row < last;
         row += static_cast<int64_t>(g.parts) * PB, buf ^= 1) {
        uint4 rx[VPT], rd[VPT];
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = t + i * TPR;
            rx[i] = c < nc ? load_chunk<FMT>(g.x + row * g.xpitch, c, g.d) : make_uint4(0, 0, 0, 0);
            rd[i] = c < nc ? load_chunk<FMT>(g.dy + row * g.dypitch, c, g.d) : make_uint4(0, 0, 0, 0);
        }
        const float mean = __ldg(g.mean + row), rstd = __ldg(g.rstd + row);
        float2 s = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = t + i * TPR;
            if (c < nc) {
                float x[N], dy[N], wv[N];
                unpack<FMT>(rx[i], x);
                unpack<FMT>(rd[i], dy);
                load_param<N>(w, c, g.d, g.vec, 1.f, wv);
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    // past d: dy = 0, and z must not turn it into a NaN
                    const float z = c * N + j < g.d ? (x[j] - mean) * rstd : 0.f;
                    const float gr = dy[j] * wv[j];
                    s.x += gr;
                    s.y = fmaf(gr, z, s.y);
                    aw[i][j] = fmaf(dy[j], z, aw[i][j]);
                    ab[i][j] += dy[j];
                }
            }
        }
        s = team_sum<TPR>(s, red, team, buf);
        if (g.y) {
            const float c1 = s.x * g.inv_d, c2 = s.y * g.inv_d;
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int c = t + i * TPR;
                if (c < nc) {
                    float x[N], dy[N], wv[N];
                    unpack<FMT>(rx[i], x);
                    unpack<FMT>(rd[i], dy);
                    load_param<N>(w, c, g.d, g.vec, 1.f, wv);
#pragma unroll
                    for (int j = 0; j < N; ++j) {
                        const float z = (x[j] - mean) * rstd;
                        x[j] = rstd * (fmaf(dy[j], wv[j], -c1) - z * c2);
                    }
                    store_chunk<FMT>(g.y + row * g.ypitch, c, g.d, pack<FMT>(x));
                }
            }
        }
    }
    if (g.dweight == nullptr && g.dbias == nullptr) return;
    float *ow, *ob;
    if (g.parts > 1) {
        ow = g.work + (gi * g.parts + p) * 2 * static_cast<int64_t>(g.d);
        ob = ow + g.d;
    } else {
        ow = g.dweight ? g.dweight + gi * g.d : nullptr;
        ob = g.dbias ? g.dbias + gi * g.d : nullptr;
    }
    for (int k = 0; k < PB; ++k) {
        if (team == k) {
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    const int col = (t + i * TPR) * N + j;
                    if (col < g.d) {
                        float a = aw[i][j], b = ab[i][j];
                        if (k > 0) {
                            a += sums[col];
                            b += sums[g.d + col];
                        }
                        if (k < PB - 1) {
                            sums[col] = a;
                            sums[g.d + col] = b;
                        } else {
                            if (ow) ow[col] = a;
                            if (ob) ob[col] = b;
                        }
                    }
                }
            }
        }
        if (k < PB - 1) __syncthreads();
    }
}

// dw and db from the slices' sums, in slice order.
__global__ void __launch_bounds__(256) norm_reduce_kernel(const NormArgs g, int64_t groups)
{
    grid_dependency_wait();
    const int64_t total = groups * 2 * g.d;
    for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < total; i += gridDim.x * 256ll) {
        const int64_t gi = i / (2 * g.d);
        const int64_t col = i % (2 * g.d);
        float *out = col < g.d ? g.dweight : g.dbias;
        if (out == nullptr) continue;
        const float *w = g.work + gi * g.parts * 2 * g.d + col;
        float s = 0.f;
        for (int p = 0; p < g.parts; ++p) s += w[p * 2ll * g.d];
        out[gi * g.d + (col < g.d ? col : col - g.d)] = s;
    }
}

template <int FMT, int TPR, int VPT>
kq_status forward_t(const NormArgs &g, cudaStream_t stream)
{
    constexpr int PB = Team<TPR>::kPerBlock;
    const int64_t blocks = (g.m + PB - 1) / PB;
    return launch_pdl(norm_forward_kernel<FMT, TPR, VPT>, static_cast<int>(blocks),
                      Team<TPR>::kThreads, 0, stream, g);
}

// A team is the smallest that holds a row in four chunks a thread.
template <int FMT>
kq_status forward_f(const NormArgs &g, cudaStream_t stream)
{
    const int nc = (g.d + Chunk<FMT>::kN - 1) / Chunk<FMT>::kN;
    if (nc <= 64) return forward_t<FMT, 32, 2>(g, stream);
    if (nc <= 160) return forward_t<FMT, 32, 5>(g, stream);
    if (nc <= 256) return forward_t<FMT, 64, 4>(g, stream);
    if (nc <= 512) return forward_t<FMT, 128, 4>(g, stream);
    if (nc <= 1024) return forward_t<FMT, 256, 4>(g, stream);
    if (nc <= 2048) return forward_t<FMT, 512, 4>(g, stream);
    if constexpr (FMT == KQ_F32) return forward_t<FMT, 1024, 4>(g, stream);
    return KQ_ERR_SHAPE;
}

template <int FMT, int TPR, int VPT>
kq_status backward_t(const NormArgs &g, int64_t groups, cudaStream_t stream)
{
    const size_t smem = Team<TPR>::kPerBlock > 1 ? 2 * sizeof(float) * static_cast<size_t>(g.d) : 0;
    return launch_pdl(norm_backward_kernel<FMT, TPR, VPT>, static_cast<int>(groups * g.parts),
                      Team<TPR>::kThreads, smem, stream, g);
}

template <int FMT>
kq_status backward_f(const NormArgs &g, int64_t groups, cudaStream_t stream)
{
    const int nc = (g.d + Chunk<FMT>::kN - 1) / Chunk<FMT>::kN;
    if (nc <= 64) return backward_t<FMT, 32, 2>(g, groups, stream);
    if (nc <= 128) return backward_t<FMT, 32, 4>(g, groups, stream);
    if (nc <= 192) return backward_t<FMT, 64, 3>(g, groups, stream);
    if (nc <= 384) return backward_t<FMT, 128, 3>(g, groups, stream);
    if (nc <= 768) return backward_t<FMT, 256, 3>(g, groups, stream);
    if (nc <= 1536) return backward_t<FMT, 512, 3>(g, groups, stream);
    if (nc <= 2048) return backward_t<FMT, 512, 4>(g, groups, stream);
    if constexpr (FMT == KQ_F32) return backward_t<FMT, 1024, 4>(g, groups, stream);
    return KQ_ERR_SHAPE;
}

// Row slices per group of the backward pass: about two blocks for each of the
// 152 SMs in all, no slice without a row.
constexpr int64_t kNormParts = 304;

}  // namespace

int64_t norm_parts(int64_t m, int64_t group_rows)
{
    const int64_t groups = (m + group_rows - 1) / group_rows;
    const int64_t rows = std::min(m, group_rows);
    return std::max<int64_t>(1, std::min((kNormParts + groups - 1) / groups, (rows + 3) / 4));
}

kq_status launch_norm_forward(const void *x, int64_t ldx, kq_format fmt, int64_t m, int64_t d,
                              const float *weight, const float *bias, int64_t group_rows, float eps,
                              void *y, int64_t ldy, float *mean, float *rstd, cudaStream_t stream)
{
    DeviceInfo info;
    const kq_status st = device_info(info);
    if (st != KQ_OK) return st;
    const int64_t size = fmt == KQ_F32 ? 4 : 2;
    NormArgs g{};
    g.x = static_cast<const uint8_t *>(x);
    g.xpitch = ldx * size;
    g.y = static_cast<uint8_t *>(y);
    g.ypitch = ldy * size;
    g.m = m;
    g.d = static_cast<int>(d);
    g.weight = weight;
    g.bias = bias;
    g.group_rows = group_rows;
    g.vec = group_rows >= m || d % 4 == 0;
    g.eps = eps;
    g.inv_d = 1.0f / static_cast<float>(d);
    g.mean = mean;
    g.rstd = rstd;
    if (fmt == KQ_BF16) return forward_f<KQ_BF16>(g, stream);
    if (fmt == KQ_F16) return forward_f<KQ_F16>(g, stream);
    return forward_f<KQ_F32>(g, stream);
}

kq_status launch_norm_backward(const void *dy, int64_t lddy, const void *x, int64_t ldx,
                               kq_format fmt, int64_t m, int64_t d, const float *weight,
                               int64_t group_rows, const float *mean, const float *rstd, void *dx,
                               int64_t lddx, float *dweight, float *dbias, void *workspace,
                               cudaStream_t stream)
{
    DeviceInfo info;
    kq_status st = device_info(info);
    if (st != KQ_OK) return st;
    const int64_t size = fmt == KQ_F32 ? 4 : 2, groups = (m + group_rows - 1) / group_rows;
    NormArgs g{};
    g.x = static_cast<const uint8_t *>(x);
    g.xpitch = ldx * size;
    g.dy = static_cast<const uint8_t *>(dy);
    g.dypitch = lddy * size;
    g.y = static_cast<uint8_t *>(dx);
    g.ypitch = lddx * size;
    g.m = m;
    g.d = static_cast<int>(d);
    g.weight = weight;
    g.group_rows = group_rows;
    g.vec = groups == 1 || d % 4 == 0;
    g.inv_d = 1.0f / static_cast<float>(d);
    g.mean = const_cast<float *>(mean);
    g.rstd = const_cast<float *>(rstd);
    g.parts = static_cast<int>(norm_parts(m, group_rows));
    g.dweight = dweight;
    g.dbias = dbias;
    g.work = static_cast<float *>(workspace);
    st = fmt == KQ_BF16  ? backward_f<KQ_BF16>(g, groups, stream)
         : fmt == KQ_F16 ? backward_f<KQ_F16>(g, groups, stream)
                         : backward_f<KQ_F32>(g, groups, stream);
    if (st != KQ_OK || g.parts == 1 || (dweight == nullptr && dbias == nullptr)) return st;
    const int64_t total = groups * 2 * d;
    const int blocks = static_cast<int>(
        std::min<int64_t>((total + 255) / 256, static_cast<int64_t>(info.sm_count) * 8));
    return launch_pdl(norm_reduce_kernel, blocks, 256, 0, stream, g, groups);
}

}  // namespace kq
