// Attention over packed sequences, sm_103a:
//     out[i] = sum_j softmax_j(scale q_i . k_j) v_j,   lse[i] = log sum_j exp(scale q_i . k_j)
// for every query row i over the keys j of its sequence (causal: the last query
// row sees the last key), with groups of query heads sharing a key/value head.
//
// One pass over the keys with a running maximum m and sum l per row (scores in
// units of log 2):
//     p_j = 2^(s_j - m),   l = sum p_j,   O = sum p_j v_j,   out = O / l
// where a larger maximum rescales l and O by 2^(m_old - m_new).  m is raised
// only when the scores exceed it by more than 8: p stays below 2^8, exact in
// range for both 16-bit types, and O is almost never read back.  Scores, p, l, m
// and O are fp32; p is rounded to the storage type for the product with V, whose
// operands have one type; l sums the unrounded p.
//
// Bound by the tensor cores: 4 D flops per (row, key), against one exponential
// (at D = 128 two M = 128 products of a tile take 1024 SM cycles, its 16384
// exponentials 512).  So two tiles of 128 query rows take turns: while the tensor
// cores work on one, a warpgroup turns the other's scores into P.  A tile holds
// the query heads of one key/value head for 128 / group tokens, so that a single
// token's heads share one read of the cache and causal tiles waste little.
//
// Roles: warps 0-3 and 4-7 softmax of tile 0 and 1 (thread = row), warp 8
// schedule and TMA loads, warp 9 the MMAs (10 and 11 only give their registers
// away).  Issuing an MMA costs its warp about as long as the tensor cores take for
// it, hence straight-line code on warp-uniform operands.  (A warp of its own for each
// tile's MMAs was slower: 1223 against 1106 us on the 16384-token prompt.)
// TMEM: scores of the tiles at columns 0 and 128 (P, 16-bit, over the first half
// of its scores), O at 256 and 384.
// Shared memory: Q of both tiles, and a ring of K and V tiles of 128 keys
// (K_0 V_0 K_1 V_1 ...), rows of 128 bytes in the 128-byte swizzle.
//
// Schedule: persistent CTAs.  With many items (tile pair x key/value head), a CTA
// takes whole items, long ones first, in an order that alternates direction from
// round to round.  With fewer items than SMs, all items' key tiles are laid end to
// end and cut into equal shares; an item cut by a share's border leaves
// normalised parts and their lse in the workspace, and a second kernel joins them.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "kq_device.cuh"
#include "kq_epilogue.cuh"
#include "kq_internal.h"
#include "kq_tcgen05.cuh"

namespace kq {
namespace {

constexpr int kAThreads = 384;                    // three warpgroups
// Registers a thread: a softmax thread holds a row of 128 scores.  The launch gives
// 168 to each of the 384; 256 * 216 + 128 * 72 = 384 * 168.
constexpr int kARegsSoftmax = 216, kARegsOther = 72;
constexpr int kABoxBytes = 128 * 128;            // 128 rows x 64 elements
constexpr int kASlotRows = 256;                  // rows of one part in the workspace
constexpr float kRescale = 8.0f;                 // log2 of the headroom of p

template <int DA>                                // boxes of 64 channels: D <= 64 DA
struct ACfg {
    static constexpr int kTile = DA * kABoxBytes;
    static constexpr int kStages = DA == 2 ? 5 : 10;
    static constexpr int kRingOff = 2 * kTile;
    static constexpr int kBarOff = kRingOff + kStages * kTile;
    static constexpr int kSmem = kBarOff + 512 + 1024;
};

struct AttnArgs {
    const int32_t *cu_q, *cu_k;
    int nseq;
    int tq, tk;                   // rows of q, of k and v
    int heads, group, gp;         // query heads, per kv head, per tile
    int tpt;                      // tokens per tile
    int units;                    // heads / gp: items per tile pair
    int d;
    int causal, split;
    float scale_log2;
    void *out;
    int64_t out_token, out_head;  // strides in elements
    float *lse;                   // [tq][heads] or null
    float *part, *part_lse;       // workspace of the split schedule
};

// One piece of work: query tokens q0 + t0 .. of a sequence against its key tiles
// j0 .. j1 - 1.
struct Segment {
    int q0, qlen, k0, klen;       // the sequence
    int t0;                       // first token of the tile pair, in the sequence
    int unit;                     // query heads unit * gp ...
    int j0, j1;
    int slot;                     // -1: writes the output; else the part's slot
    int valid;                    // 0: no more work
};

// Key tiles that some row of tile t (tokens t0 + t * tpt ...) sees.
__device__ __forceinline__ int tile_limit(const AttnArgs &g, int qlen, int klen, int t0, int t)
{
    const int first = t0 + t * g.tpt;
    if (first >= qlen) return 0;
    int seen = klen;
    if (g.causal) seen = min(klen, min(qlen, first + g.tpt) + klen - qlen);
    return seen > 0 ? (seen + 127) >> 7 : 0;
}

// A warp's cursor over the sequences, 32 at a time: finds the one that holds
// position w of the running count of work (items, or key tiles of items).
struct Cursor {
    int b0 = -32;
    int64_t base = 0, total = 0;  // count before and within the 32 sequences
    int64_t incl = 0;             // count up to and with this lane's sequence
    int q0 = 0, qlen = 0, k0 = 0, klen = 0;

    __device__ __forceinline__ int pairs(const AttnArgs &g) const { return (qlen + 2 * g.tpt - 1) / (2 * g.tpt); }
    __device__ __forceinline__ int tiles(const AttnArgs &g) const { return g.split ? max(1, (klen + 127) >> 7) : 1; }

    __device__ __forceinline__ bool next(const AttnArgs &g)
    {
        base += total;
        b0 += 32;
        if (b0 >= g.nseq) {
            total = 0;
            return false;
        }
        const int b = b0 + static_cast<int>(threadIdx.x & 31);
        q0 = qlen = k0 = klen = 0;
        if (b < g.nseq) {
            // offsets are the caller's: whatever they hold, rows stay in range
            q0 = min(max(__ldg(g.cu_q + b), 0), g.tq);
            qlen = max(min(__ldg(g.cu_q + b + 1), g.tq) - q0, 0);
            k0 = min(max(__ldg(g.cu_k + b), 0), g.tk);
            klen = max(min(__ldg(g.cu_k + b + 1), g.tk) - k0, 0);
        }
        incl = static_cast<int64_t>(pairs(g)) * g.units * tiles(g);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
            if (static_cast<int>(threadIdx.x & 31) >= o) incl += v;
        }
        total = __shfl_sync(0xffffffffu, incl, 31);
        return true;
    }

    // Position w, at or after the last one asked for: the segment it starts (one
    // item, or its key tiles up to `end`).  False past the end.
    __device__ __forceinline__ bool find(const AttnArgs &g, int64_t w, int64_t end, Segment &s)
    {
        while (w >= base + total)
            if (!next(g)) return false;
        const uint32_t hit = __ballot_sync(0xffffffffu, w < base + incl);
        const int src = __ffs(hit) - 1;
        s.q0 = __shfl_sync(0xffffffffu, q0, src);
        s.qlen = __shfl_sync(0xffffffffu, qlen, src);
        s.k0 = __shfl_sync(0xffffffffu, k0, src);
        s.klen = __shfl_sync(0xffffffffu, klen, src);
        const int np = __shfl_sync(0xffffffffu, pairs(g), src), nt = __shfl_sync(0xffffffffu, tiles(g), src);
        const int64_t before = base + __shfl_sync(0xffffffffu, incl, src) -
                               static_cast<int64_t>(np) * g.units * nt;
        const int64_t off = w - before;
        const int item = static_cast<int>(off / nt);
        s.t0 = (np - 1 - item / g.units) * 2 * g.tpt;      // the longest tiles first
        s.unit = item % g.units;
        s.slot = -1;
        s.valid = 1;
        if (!g.split) {
            s.j0 = 0;
            s.j1 = (s.klen + 127) >> 7;
        } else {
            s.j0 = static_cast<int>(off % nt);
            s.j1 = static_cast<int>(min(static_cast<int64_t>(nt), s.j0 + (end - w)));
        }
        return true;
    }
};

// ---- tensor core and TMEM pieces ----------------------------------------------------

// D += P V with P (A operand) in TMEM.
__device__ __forceinline__ void a_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}

// V, [128 keys][64 channels] boxes: the channels (N) are the contiguous
// dimension, 64 of them in the swizzle atom; the next 64 are a box further
// (leading offset), the next 8 keys 1 KB (stride offset).
__device__ __forceinline__ uint64_t a_desc_v(uint32_t saddr)
{
    return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) |
           (static_cast<uint64_t>(kABoxBytes >> 4) << 16) | (static_cast<uint64_t>(1024 >> 4) << 32) |
           (1ull << 46) | (2ull << 61);
}

#define KQ_R8(r, o) "=r"(r[o]), "=r"(r[o + 1]), "=r"(r[o + 2]), "=r"(r[o + 3]), "=r"(r[o + 4]), \
                    "=r"(r[o + 5]), "=r"(r[o + 6]), "=r"(r[o + 7])
#define KQ_I8(r, o) "r"(r[o]), "r"(r[o + 1]), "r"(r[o + 2]), "r"(r[o + 3]), "r"(r[o + 4]), \
                    "r"(r[o + 5]), "r"(r[o + 6]), "r"(r[o + 7])
#define KQ_IO8(r, o) "+r"(r[o]), "+r"(r[o + 1]), "+r"(r[o + 2]), "+r"(r[o + 3]), "+r"(r[o + 4]), \
                     "+r"(r[o + 5]), "+r"(r[o + 6]), "+r"(r[o + 7])

// 32 columns of the warp's lanes, complete after a_wait_ld on the registers.
__device__ __forceinline__ void a_ld32(uint32_t taddr, uint32_t *r)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : KQ_R8(r, 0), KQ_R8(r, 8), KQ_R8(r, 16), KQ_R8(r, 24)
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void a_st32(uint32_t taddr, const uint32_t *r)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
        "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
        KQ_I8(r, 0), KQ_I8(r, 8), KQ_I8(r, 16), KQ_I8(r, 24)
        : "memory");
}
// Waits for the loads; the registers pass through, so that no use of them can be
// moved ahead of the wait.
__device__ __forceinline__ void a_wait_ld(uint32_t *r)
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : KQ_IO8(r, 0), KQ_IO8(r, 8), KQ_IO8(r, 16), KQ_IO8(r, 24)
                 :
                 : "memory");
}
__device__ __forceinline__ void a_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *map, int32_t x, int32_t y,
                                            int32_t z, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}

// N words of a row, `left` bytes of them real (a multiple of 16): 32 bytes a store
// where the row allows it.  Every lane writes its own row, so what counts is the
// number of store instructions and whole 32-byte sectors.
template <int N>
__device__ __forceinline__ void store_row(uint8_t *dst, const uint32_t *o, int left, bool wide)
{
#pragma unroll
    for (int k = 0; k < N; k += 8) {
        if (wide && 4 * k + 32 <= left) {
            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst + 4 * k),
                         KQ_I8(o, k)
                         : "memory");
        } else {
            if (4 * k < left)
                *reinterpret_cast<uint4 *>(dst + 4 * k) = make_uint4(o[k], o[k + 1], o[k + 2], o[k + 3]);
            if (4 * k + 16 < left)
                *reinterpret_cast<uint4 *>(dst + 4 * k + 16) = make_uint4(o[k + 4], o[k + 5], o[k + 6], o[k + 7]);
        }
    }
}

__device__ __forceinline__ void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kARegsOther)); }
__device__ __forceinline__ void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kARegsSoftmax)); }

// ---- the kernel ------------------------------------------------------------------------

template <int DA, bool F16>
__global__ void __launch_bounds__(kAThreads, 1)
    attention_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV, const AttnArgs g)
{
    using C = ACfg<DA>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ Segment segs[2];
    const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
    const uint32_t ring = base + C::kRingOff;
    const uint32_t bar = base + C::kBarOff;
    const uint32_t kv_full = bar, kv_empty = bar + 8 * C::kStages;
    const uint32_t b1 = bar + 16 * C::kStages;
    // per tile: Q, scores, P (in halves), O; then the two segment buffers
    const uint32_t q_full = b1, q_empty = b1 + 16, s_full = b1 + 32, p_ready = b1 + 48, o_full = b1 + 80;
    const uint32_t drain = b1 + 96, seg_full = b1 + 112, seg_empty = b1 + 128;
    const uint32_t tmem_slot = b1 + 144;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        tma_prefetch_desc(&tmQ);
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(kv_full + 8 * s, 1);
            mbar_init(kv_empty + 8 * s, 1);
        }
        for (int q = 0; q < 2; ++q) {
            mbar_init(q_full + 8 * q, 1);
            mbar_init(q_empty + 8 * q, 1);
            mbar_init(s_full + 8 * q, 1);
            mbar_init(p_ready + 16 * q, 4);              // the softmax warps
            mbar_init(p_ready + 16 * q + 8, 4);
            mbar_init(o_full + 8 * q, 1);
            mbar_init(drain + 8 * q, 1);
            mbar_init(seg_full + 8 * q, 1);
            mbar_init(seg_empty + 8 * q, 9);             // MMA and softmax warps
        }
        mbar_fence_init();
    }
    if (warp == 9) g_tmem_alloc(tmem_slot, 512);
    g_fence_before();
    __syncthreads();
    g_fence_after();
    // All 512 columns are this CTA's, so they start at column 0: as a constant the
    // address costs the MMA warps no register traffic.
    constexpr uint32_t tmem = 0;
    grid_dependency_wait();

    // A role's segments: slot i of the pair of segment buffers.  False: no more
    // work, or the wait for it gave up.
    auto take = [&](int i, Segment &s) {
        if (!__all_sync(0xffffffffu, mbar_wait(seg_full + 8 * (i & 1), static_cast<uint32_t>((i >> 1) & 1))))
            return false;
        s = segs[i & 1];
        __syncwarp();
        if (lane == 0) mbar_arrive(seg_empty + 8 * (i & 1));
        return __shfl_sync(0xffffffffu, s.valid, 0) != 0;
    };
    // Key tiles of the segment that tile t works on.
    auto tiles_of = [&](const Segment &s, int t) {
        return max(0, min(s.j1, tile_limit(g, s.qlen, s.klen, s.t0, t)) - s.j0);
    };

    if (warp == 8) {
        // schedule and loads
        regs_dec();
        Cursor cur;
        int64_t w = blockIdx.x, end = 0, quota = 0;
        if (g.split) {
            Cursor all;
            while (all.next(g)) {
            }
            quota = (all.base + gridDim.x - 1) / gridDim.x;
            w = static_cast<int64_t>(blockIdx.x) * quota;
            end = min(all.base, w + quota);
        }
        const int64_t begin = w;
        int kv = 0, qn[2] = {0, 0};                      // stages and Q tiles loaded
        bool ok = true;
        for (int i = 0; ok; ++i) {
            Segment s;
            if (!g.split) {
                // round i, direction alternating: lengths even out over the rounds
                w = static_cast<int64_t>(i) * gridDim.x +
                    ((i & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
                if (!cur.find(g, w, 0, s)) s.valid = 0;
            } else {
                if (w >= end || !cur.find(g, w, end, s)) {
                    s.valid = 0;
                } else {
                    const int nt = max(1, (s.klen + 127) >> 7);
                    if (s.j1 - s.j0 < nt) s.slot = static_cast<int>(blockIdx.x) * 2 + (w == begin ? 0 : 1);
                    w += s.j1 - s.j0;
                }
            }
            if (i >= 2)
                ok = __all_sync(0xffffffffu, mbar_wait(seg_empty + 8 * (i & 1),
                                                       static_cast<uint32_t>(((i >> 1) - 1) & 1)));
            if (!ok) break;
            if (lane == 0) {
                segs[i & 1] = s;
                mbar_arrive(seg_full + 8 * (i & 1));
            }
            __syncwarp();
            if (!s.valid) break;
            const int n0 = tiles_of(s, 0), n1 = tiles_of(s, 1), n = max(n0, n1);
            if (n == 0) continue;
            if (lane == 0) {
                const int kvh = s.unit * g.gp / g.group, h0 = s.unit * g.gp;
                const uint32_t box = static_cast<uint32_t>(g.gp * g.tpt) * 128u;
                auto load_q = [&](int t) {
                    if ((t ? n1 : n0) == 0 || !ok) return;
                    if (qn[t] > 0) ok = mbar_wait(q_empty + 8 * t, static_cast<uint32_t>((qn[t] - 1) & 1));
                    if (!ok) return;
                    mbar_arrive_expect_tx(q_full + 8 * t, box * DA);
                    for (int a = 0; a < DA; ++a)
                        tma_load_3d(base + t * C::kTile + a * kABoxBytes, &tmQ, 64 * a, h0,
                                    s.q0 + s.t0 + t * g.tpt, q_full + 8 * t);
                    ++qn[t];
                };
                load_q(0);
                for (int j = 0; j < 2 * n && ok; ++j, ++kv) {
                    if (j == 1) load_q(1);               // after the first K: tile 0 can start
                    const int st = kv % C::kStages;
                    if (ok && kv >= C::kStages)
                        ok = mbar_wait(kv_empty + 8 * st, static_cast<uint32_t>((kv / C::kStages - 1) & 1));
                    if (!ok) break;
                    const uint32_t dst = ring + static_cast<uint32_t>(st) * C::kTile;
                    mbar_arrive_expect_tx(kv_full + 8 * st, C::kTile);
                    for (int a = 0; a < DA; ++a)
                        tma_load_3d(dst + a * kABoxBytes, (j & 1) ? &tmV : &tmK, 64 * a, kvh,
                                    s.k0 + (s.j0 + (j >> 1)) * 128, kv_full + 8 * st);
                }
            }
            ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
        }
        if (lane == 0) {
            // no copy is in flight when the CTA leaves
            for (int t = 0; t < 2; ++t)
                if (qn[t] > 0) (void)mbar_wait(q_full + 8 * t, static_cast<uint32_t>((qn[t] - 1) & 1));
            for (int j = max(0, kv - C::kStages); j < kv; ++j)
                (void)mbar_wait(kv_full + 8 * (j % C::kStages), static_cast<uint32_t>((j / C::kStages) & 1));
        }
        __syncwarp();
    } else if (warp == 9) {
        // MMAs: one elected lane issues, the warp waits converged.  Its operands are
        // warp-uniform and its full tiles straight-line code.
        regs_dec();
        const bool leader = elect_one();
        constexpr uint32_t kFmt = F16 ? 0u : ((1u << 7) | (1u << 10));
        constexpr uint32_t id_qk = (1u << 4) | kFmt | ((128u >> 3) << 17) | ((128u >> 4) << 24);
        const uint32_t nv = static_cast<uint32_t>((g.d + 15) & ~15);
        const uint32_t id_pv = (1u << 4) | kFmt | (1u << 16) | ((nv >> 3) << 17) | ((128u >> 4) << 24);
        const int ksteps = (g.d + 15) >> 4;
        const bool full_d = ksteps == 4 * DA;
        int st = 0;                                      // ring stage, its parity
        uint32_t par = 0;
        uint32_t qpar[2] = {0, 0}, ppar[2] = {0, 0};
        bool ok = true;
        auto wait = [&](uint32_t b, uint32_t p) {
            ok = ok && __all_sync(0xffffffffu, mbar_wait(b, p));
            g_fence_after();
        };
        auto advance = [&] {
            if (++st == C::kStages) {
                st = 0;
                par ^= 1;
            }
        };
        // S = Q K^T of tile t from the K tile of stage `k`
        auto qk = [&](int t, int k) {
            const uint32_t ts = tmem + 128 * t;
            const uint64_t dq = g_desc(base + t * C::kTile), dk = g_desc(ring + static_cast<uint32_t>(k) * C::kTile);
            if (leader) {
                if (full_d) {
#pragma unroll
                    for (int i = 0; i < 4 * DA; ++i) {
                        const int off = (i >> 2) * (kABoxBytes >> 4) + (i & 3) * 2;
                        g_mma_id(ts, dq + off, dk + off, id_qk, i > 0);
                    }
                } else {
                    for (int i = 0; i < ksteps; ++i) {
                        const int off = (i >> 2) * (kABoxBytes >> 4) + (i & 3) * 2;
                        g_mma_id(ts, dq + off, dk + off, id_qk, i > 0);
                    }
                }
                g_commit(s_full + 8 * t);
            }
            __syncwarp();
        };
        auto release = [&](uint32_t b) {
            if (leader) g_commit(b);
            __syncwarp();
        };
        Segment s;
        for (int i = 0; ok && take(i, s); ++i) {
            const int n0 = __shfl_sync(0xffffffffu, tiles_of(s, 0), 0);
            const int n1 = __shfl_sync(0xffffffffu, tiles_of(s, 1), 0), n = max(n0, n1);
            const int tail = __shfl_sync(0xffffffffu, s.klen - s.j0 * 128, 0);   // keys from tile j0 on
            if (n == 0) continue;
            wait(kv_full + 8 * st, par);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                if ((t ? n1 : n0) == 0) continue;
                wait(q_full + 8 * t, qpar[t]);
                qpar[t] ^= 1;
                if (!ok) break;
                qk(t, st);
                if ((t ? n1 : n0) == 1) release(q_empty + 8 * t);
            }
            if (!ok) break;
            release(kv_empty + 8 * st);
            advance();
            for (int j = 0; j < n && ok; ++j) {
                const int sv = st;
                wait(kv_full + 8 * sv, par);
                advance();
                const uint32_t va = ring + static_cast<uint32_t>(sv) * C::kTile;
                // keys of this tile; rows of V past the last one (another sequence's)
                // could hold NaN, which a weight of zero does not undo: the MMAs stop
                // at the next 16 keys, and the rows up to there are cleared
                const int keys = min(128, tail - j * 128);
                const int vsteps = (keys + 15) >> 4;
                if (ok && (keys & 15)) {
                    const int pad = vsteps * 16 - keys;
                    for (int c = lane; c < pad * 8 * DA; c += 32) {
                        const int row = keys + (c >> 3) % pad, box = (c >> 3) / pad;
                        sts128(va + box * kABoxBytes + row * 128 + (c & 7) * 16, make_uint4(0, 0, 0, 0));
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                }
                const uint64_t dv = a_desc_v(va);
                bool next = false;                       // the next K tile has been waited for
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const int mine = t ? n1 : n0;
                    if (j < mine) {
                        const uint32_t ts = tmem + 128 * t, to = tmem + 256 + 128 * t;
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            wait(p_ready + 16 * t + 8 * h, ppar[t]);
                            if (!ok) break;
                            const uint32_t acc = j > 0 || h > 0;
                            if (leader) {
                                if (vsteps == 8) {
#pragma unroll
                                    for (int k = 0; k < 4; ++k)
                                        a_mma_ts(to, ts + 32 * h + 8 * k, dv + 512 * h + 128 * k, id_pv,
                                                 k > 0 ? 1u : acc);
                                } else {
                                    for (int k = 0; k < 4 && 4 * h + k < vsteps; ++k)
                                        a_mma_ts(to, ts + 32 * h + 8 * k, dv + 512 * h + 128 * k, id_pv,
                                                 k > 0 ? 1u : acc);
                                }
                                if (h == 1 && j == mine - 1) g_commit(o_full + 8 * t);
                            }
                            __syncwarp();
                        }
                        ppar[t] ^= 1;
                    }
                    if (t == 1) release(kv_empty + 8 * sv);
                    if (j + 1 < mine) {
                        if (!next) wait(kv_full + 8 * st, par);
                        next = true;
                        if (!ok) break;
                        qk(t, st);
                        if (j + 2 == mine) release(q_empty + 8 * t);
                    }
                }
                if (j + 1 < n) {
                    if (!next) wait(kv_full + 8 * st, par);
                    release(kv_empty + 8 * st);
                    advance();
                }
            }
        }
        // nothing of the tensor cores' is in flight when the CTA leaves
        if (leader) g_commit(drain);
        __syncwarp();
        (void)mbar_wait(drain, 0);
    } else if (warp >= 10) {
        regs_dec();
    } else {
        regs_inc();
        const int t = warp >> 2, qtr = warp & 3;
        const int r = qtr * 32 + lane;                   // row of the tile
        const int rt = r / g.gp, rh = r - rt * g.gp;     // its token and head in the tile
        const uint32_t lanes = static_cast<uint32_t>(qtr * 32) << 16;
        const uint32_t ts = tmem + lanes + 128 * t, to = tmem + lanes + 256 + 128 * t;
        const uint32_t sbar = s_full + 8 * t, pbar = p_ready + 16 * t, obar = o_full + 8 * t;
        int sn = 0, on = 0;                              // scores and outputs consumed
        bool ok = true;
        Segment s;
        for (int i = 0; ok && take(i, s); ++i) {
            if (s.t0 + t * g.tpt >= s.qlen) continue;    // no tokens in this tile
            const int n = tiles_of(s, t);
            const int tok = s.t0 + t * g.tpt + rt;
            const bool real = rt < g.tpt && tok < s.qlen;
            // keys this row sees
            int lim = real ? (g.causal ? min(s.klen, tok + 1 + s.klen - s.qlen) : s.klen) : 0;
            lim -= s.j0 * 128;
            float m = -INFINITY, l = 0.f;
            for (int j = 0; j < n; ++j, lim -= 128, ++sn) {
                ok = __all_sync(0xffffffffu, mbar_wait(sbar, static_cast<uint32_t>(sn & 1)));
                if (!ok) break;
                g_fence_after();
                uint32_t v[128];
#pragma unroll
                for (int c = 0; c < 4; ++c) a_ld32(ts + 32 * c, v + 32 * c);
#pragma unroll
                for (int c = 0; c < 4; ++c) a_wait_ld(v + 32 * c);
                if (__any_sync(0xffffffffu, lim < 128)) {
#pragma unroll
                    for (int c = 0; c < 128; ++c)
                        if (c >= lim) v[c] = 0xFF800000u;
                }
                float top = -INFINITY;
                // weights of 64 keys against the maximum m, and their sums
                const float2 sc = make_float2(g.scale_log2, g.scale_log2);
                float2 sum[2];
                uint32_t p[32];
                auto weights = [&](int h) {
                    const float ref = m == -INFINITY ? 0.f : m;
                    const float2 rf = make_float2(-ref, -ref);
                    sum[0] = sum[1] = make_float2(0.f, 0.f);
#pragma unroll
                    for (int c = 0; c < 32; ++c) {
                        const int e = 64 * h + 2 * c;
                        float2 x = make_float2(__uint_as_float(v[e]), __uint_as_float(v[e + 1]));
                        x = __ffma2_rn(x, sc, rf);
                        x.x = ex2_approx(x.x);
                        x.y = ex2_approx(x.y);
                        sum[c & 1] = __fadd2_rn(sum[c & 1], x);
                        p[c] = pack16(x.x, x.y, F16);
                    }
                };
                auto maximum = [&] {
                    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int c = 0; c < 128; c += 8) {
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            mx[k] = fmax3(mx[k], __uint_as_float(v[c + 2 * k]), __uint_as_float(v[c + 2 * k + 1]));
                    }
                    top = fmaxf(fmax3(mx[0], mx[1], mx[2]), mx[3]) * g.scale_log2;
                };
                auto hand_over = [&](int h) {
                    a_st32(ts + 32 * h, p);
                    a_wait_st();
                    g_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(pbar + 8 * h);
                };
                // The first half's weights are computed against the old maximum
                // while the new one is found (the exponentials and the comparisons
                // use different pipes); they are computed again in the rare tile
                // that raises it.
                weights(0);
                maximum();
                if (__any_sync(0xffffffffu, top > m + kRescale)) {   // also from m = -inf
                    const float mn = top > m + kRescale ? top : m;
                    const float f = m == -INFINITY ? 0.f : ex2_approx(m - mn);
                    m = mn;
                    l *= f;
                    if (j > 0) {
                        for (int c = 0; c < g.d; c += 32) {
                            uint32_t o[32];
                            a_ld32(to + c, o);
                            a_wait_ld(o);
#pragma unroll
                            for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                            a_st32(to + c, o);
                        }
                    }
                    weights(0);
                }
                l += (sum[0].x + sum[1].x) + (sum[0].y + sum[1].y);
                hand_over(0);
                weights(1);
                l += (sum[0].x + sum[1].x) + (sum[0].y + sum[1].y);
                hand_over(1);
            }
            if (!ok) break;
            if (n > 0) {
                ok = __all_sync(0xffffffffu, mbar_wait(obar, static_cast<uint32_t>(on & 1)));
                ++on;
                if (!ok) break;
                g_fence_after();
            }
            // a row without keys is zero, and its lse -inf
            const float inv = l > 0.f || l != l ? 1.0f / l : 0.f;
            const float lse = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
            const int64_t row = s.q0 + tok;
            const int head = s.unit * g.gp + rh;
            // rows of the output start on 32 bytes (the workspace's always do)
            const bool wide = ((reinterpret_cast<uintptr_t>(g.out) & 31) | ((g.out_token | g.out_head) & 15)) == 0;
            uint8_t *dst;
            if (s.slot < 0) {
                dst = static_cast<uint8_t *>(g.out) + (row * g.out_token + head * g.out_head) * 2;
                if (real && g.lse != nullptr) g.lse[row * g.heads + head] = lse;
            } else {
                const int64_t pr = static_cast<int64_t>(s.slot) * kASlotRows + t * 128 + r;
                dst = reinterpret_cast<uint8_t *>(g.part + pr * g.d);
                if (real) g.part_lse[pr] = lse;
            }
            for (int c = 0; c < g.d; c += 32) {
                uint32_t o[32];
                if (n > 0) {
                    a_ld32(to + c, o);
                    a_wait_ld(o);
                } else {
#pragma unroll
                    for (int k = 0; k < 32; ++k) o[k] = 0;
                }
                if (!real) continue;
#pragma unroll
                for (int k = 0; k < 32; ++k)
                    o[k] = __float_as_uint(inv == 0.f ? 0.f : __uint_as_float(o[k]) * inv);
                if (s.slot < 0) {
#pragma unroll
                    for (int k = 0; k < 16; ++k)
                        o[k] = pack16(__uint_as_float(o[2 * k]), __uint_as_float(o[2 * k + 1]), F16);
                    store_row<16>(dst + c * 2, o, (g.d - c) * 2, wide);
                } else {
                    store_row<32>(dst + c * 4, o, (g.d - c) * 4, true);
                }
            }
            g_fence_before();
        }
    }
    g_fence_before();
    __syncthreads();
    if (warp == 9) {
        g_fence_after();
        uint32_t addr;
        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(addr) : "r"(tmem_slot) : "memory");
        g_tmem_dealloc(addr, 512);
    }
}

// Joins the parts of the items that the split schedule cut: one warp per query
// row and head.  out = sum_i w_i O_i / sum_i w_i with w_i = exp(lse_i - max lse),
// over the parts in the order of their keys.
template <bool F16>
__global__ void __launch_bounds__(256) attention_join_kernel(const AttnArgs g, int grid)
{
    const int lane = threadIdx.x & 31;
    const int64_t id = blockIdx.x * 8ll + (threadIdx.x >> 5);
    const int row = static_cast<int>(id / g.heads), head = static_cast<int>(id % g.heads);
    grid_dependency_wait();
    if (row >= g.tq) return;
    // the row's item, as the schedule counts: total work, and the item's first unit
    Cursor cur;
    int64_t u0 = -1;
    int nt = 0, r = 0;
    while (cur.next(g)) {
        const uint32_t hit = __ballot_sync(0xffffffffu, row >= cur.q0 && row < cur.q0 + cur.qlen);
        if (hit != 0 && u0 < 0) {
            const int src = __ffs(hit) - 1;
            const int tok = row - __shfl_sync(0xffffffffu, cur.q0, src);
            const int np = __shfl_sync(0xffffffffu, cur.pairs(g), src);
            nt = __shfl_sync(0xffffffffu, cur.tiles(g), src);
            const int64_t first = cur.base + __shfl_sync(0xffffffffu, cur.incl, src) -
                                  static_cast<int64_t>(np) * g.units * nt;
            const int pair = tok / (2 * g.tpt), in = tok - pair * 2 * g.tpt;
            u0 = first + (static_cast<int64_t>(np - 1 - pair) * g.units + head / g.gp) * nt;
            r = in / g.tpt * 128 + in % g.tpt * g.gp + head % g.gp;
        }
    }
    if (u0 < 0) return;                                  // a row of no sequence
    const int64_t quota = (cur.base + grid - 1) / grid;
    const int64_t c0 = u0 / quota, c1 = (u0 + nt - 1) / quota;
    if (c0 == c1) return;                                // written whole
    auto slot_row = [&](int64_t c) {
        const int64_t slot = 2 * c + (c == c0 && u0 != c0 * quota ? 1 : 0);
        return slot * kASlotRows + r;
    };
    float top = -INFINITY;
    for (int64_t c = c0 + lane; c <= c1; c += 32) top = fmaxf(top, g.part_lse[slot_row(c)]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float ref = top == -INFINITY ? 0.f : top;
    float acc[4] = {0.f, 0.f, 0.f, 0.f}, sum = 0.f;
    const int col = 4 * lane;                            // d <= 128: four channels a lane
    for (int64_t c = c0; c <= c1; ++c) {
        const int64_t pr = slot_row(c);
        const float w = ex2_approx((g.part_lse[pr] - ref) * kLog2e);
        sum += w;
        if (col < g.d && w != 0.f) {
            const float4 o = *reinterpret_cast<const float4 *>(g.part + pr * g.d + col);
            acc[0] = fmaf(w, o.x, acc[0]);
            acc[1] = fmaf(w, o.y, acc[1]);
            acc[2] = fmaf(w, o.z, acc[2]);
            acc[3] = fmaf(w, o.w, acc[3]);
        }
    }
    const float inv = sum > 0.f || sum != sum ? 1.0f / sum : 0.f;
    if (col < g.d)
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(g.out) + row * g.out_token +
                                   head * g.out_head + col) =
            make_uint2(pack16(acc[0] * inv, acc[1] * inv, F16), pack16(acc[2] * inv, acc[3] * inv, F16));
    if (lane == 0 && g.lse != nullptr)
        g.lse[static_cast<int64_t>(row) * g.heads + head] =
            sum == 0.f ? -INFINITY : ref + log2f(sum) * 0.69314718055994531f;
}

template <int DA, bool F16>
kq_status launch_t(const CUtensorMap &mq, const CUtensorMap &mk, const CUtensorMap &mv,
                   const AttnArgs &g, int grid, cudaStream_t stream)
{
    auto kern = attention_kernel<DA, F16>;
    static DeviceOnce once;
    kq_status st = once.run([&] {
        return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, ACfg<DA>::kSmem);
    });
    if (st != KQ_OK) return st;
    st = launch_pdl(kern, grid, kAThreads, static_cast<size_t>(ACfg<DA>::kSmem), stream, mq, mk, mv, g);
    if (st != KQ_OK || !g.split) return st;
    const int64_t rows = static_cast<int64_t>(g.tq) * g.heads;
    return launch_pdl(attention_join_kernel<F16>, static_cast<int>((rows + 7) / 8), 256, 0, stream, g, grid);
}

// Query heads per tile: the whole group, or for groups of more than 128 heads
// its largest divisor that fits.
int heads_per_tile(int group)
{
    int gp = std::min(group, 128);
    while (group % gp != 0) --gp;
    return gp;
}

constexpr int kAMaxGrid = 152;

// Upper bound of the items: every sequence has at most one partly filled pair.
int64_t items_most(int64_t tq, int64_t nseq, int64_t max_q, int64_t pair, int64_t units)
{
    const int64_t by_rows = std::min(tq, tq / pair + nseq);
    return units * std::max<int64_t>(1, std::min(by_rows, nseq * ((max_q + pair - 1) / pair)));
}

bool split_schedule(int64_t tq, int64_t nseq, int64_t heads, int64_t kv_heads, int64_t max_q)
{
    const int gp = heads_per_tile(static_cast<int>(heads / kv_heads));
    return items_most(tq, nseq, max_q, 2 * (128 / gp), heads / gp) < kAMaxGrid;
}

}  // namespace

size_t attention_bytes(int64_t tq, int64_t nseq, int64_t heads, int64_t kv_heads, int64_t d, int64_t max_q)
{
    if (!split_schedule(tq, nseq, heads, kv_heads, max_q)) return 0;
    return static_cast<size_t>(kAMaxGrid) * 2 * kASlotRows * (static_cast<size_t>(d) + 1) * sizeof(float);
}

kq_status launch_attention(const AttentionCall &c, cudaStream_t stream)
{
    DeviceInfo info;
    kq_status st = device_info(info);
    if (st != KQ_OK) return st;
    AttnArgs g{};
    g.cu_q = c.cu_q;
    g.cu_k = c.cu_k;
    g.nseq = static_cast<int>(c.nseq);
    g.tq = static_cast<int>(c.tq);
    g.tk = static_cast<int>(c.tk);
    g.heads = static_cast<int>(c.heads);
    g.group = static_cast<int>(c.heads / c.kv_heads);
    g.gp = heads_per_tile(g.group);
    g.tpt = 128 / g.gp;
    g.units = g.heads / g.gp;
    g.d = static_cast<int>(c.d);
    g.causal = c.causal ? 1 : 0;
    g.split = split_schedule(c.tq, c.nseq, c.heads, c.kv_heads, c.max_q) ? 1 : 0;
    g.scale_log2 = c.scale * 1.4426950408889634f;
    g.out = c.out;
    g.out_token = c.out_token;
    g.out_head = c.out_head;
    g.lse = c.lse;
    g.part = static_cast<float *>(c.workspace);
    g.part_lse = g.part + static_cast<int64_t>(kAMaxGrid) * 2 * kASlotRows * g.d;
    CUtensorMap mq, mk, mv;
    st = make_tensor_map_3d_16(&mq, c.q, c.d, c.heads, c.tq, c.q_head, c.q_token, 64,
                               static_cast<uint32_t>(g.gp), static_cast<uint32_t>(g.tpt));
    // no keys at all: no tile is loaded, and the maps only have to be well formed
    const int64_t tk = std::max<int64_t>(c.tk, 1);
    const void *kp = c.tk > 0 ? c.k : c.q, *vp = c.tk > 0 ? c.v : c.q;
    if (st == KQ_OK)
        st = make_tensor_map_3d_16(&mk, kp, c.d, c.kv_heads, tk, c.k_head, c.k_token, 64, 1, 128);
    if (st == KQ_OK)
        st = make_tensor_map_3d_16(&mv, vp, c.d, c.kv_heads, tk, c.v_head, c.v_token, 64, 1, 128);
    if (st != KQ_OK) return st;
    const int sms = std::min(info.sm_count, kAMaxGrid);
    const int64_t items = items_most(c.tq, c.nseq, c.max_q, 2 * g.tpt, g.units);
    const int grid = g.split ? sms : static_cast<int>(std::min<int64_t>(items, sms));
    if (c.d <= 64)
        return c.f16 ? launch_t<1, true>(mq, mk, mv, g, grid, stream)
                     : launch_t<1, false>(mq, mk, mv, g, grid, stream);
    return c.f16 ? launch_t<2, true>(mq, mk, mv, g, grid, stream)
                 : launch_t<2, false>(mq, mk, mv, g, grid, stream);
}

}  // namespace kq
