// The QKV projection with low-rank adapters of many requests, and its
// backward pass.
//
// Rows offsets[r] .. offsets[r+1] - 1 are request r's, with adapter
// a = adapter[r] (none where the id is not in 0 .. n_ad - 1):
//   t = scaling_a x A_a^T                     (rank R, fp32 sums, rounded to bf16)
//   qkv = s_n (x W^T + bias + t B_a^T)        (s_n = HD^-0.5 in the q block, else 1)
// Backward, with g = s_n dqkv:
//   u = scaling_a g B_a,  dx = g W + u A_a,
//   dA_a = sum over the adapter's rows of u^T x,  dB_a = sum of g^T t.
// The base weight and the scalings are frozen: they get no gradient.
//
// lora_down computes t and u. It writes them once for each pair of a 128-row
// tile and a request that meets it, zeros in the rows of others, so that the
// large product takes an adapter as R more columns of its contraction: the
// accumulator tile of lora_gemm gets t B_a^T from the tensor cores and leaves
// the SM once. Pair (tile i, request r) is block i + r of the workspace: along
// the rows one of the two grows from pair to pair, so no two share a block.
#include <atomic>
#include <cuda_bf16.h>

#include "na3d_host.cuh"
#include "na3d_lora.cuh"
#include "sm103_ptx.cuh"

namespace na3d {

__device__ unsigned int g_lora_timeout_flag = 0;

namespace {

__device__ __forceinline__ float f32(uint16_t h) { return __uint_as_float(uint32_t(h) << 16); }
__device__ __forceinline__ uint16_t b16(float f) { return __bfloat16_as_ushort(__float2bfloat16_rn(f)); }

// ------------------------------------------------------------------ requests

struct Requests {
    const int32_t *offsets, *adapter;
    int n_req, n_ad;
};

__device__ __forceinline__ Requests requests_of(const LoraParams& p) { return {p.offsets, p.adapter, p.n_req, p.n_ad}; }

// The first request that ends behind row m (n_req where none does).
__device__ __forceinline__ int first_request(const Requests& q, int m) {
    int lo = 0, hi = q.n_req;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (q.offsets[mid + 1] > m) hi = mid;
        else lo = mid + 1;
    }
    return lo;
}

// The same by a whole warp: few requests' offsets in one trip to memory, and
// the same search over them.
__device__ __forceinline__ int first_request_warp(const Requests& q, int m) {
    if (q.n_req > 32) return first_request(q, m);
    const int lane = threadIdx.x & 31, end = lane < q.n_req ? q.offsets[lane + 1] : 0;
    int lo = 0, hi = q.n_req;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (__shfl_sync(0xffffffffu, end, mid) > m) hi = mid;
        else lo = mid + 1;
    }
    return lo;
}

// The requests with an adapter that meet rows [m0, m0 + SPAN), in order. Every
// role of every kernel walks them alike.
template <int SPAN>
struct WalkOf {
    int r, a, lo, hi;   // request, its adapter, its rows
    __device__ __forceinline__ void start(const Requests& q, int m0) {
        r = first_request(q, m0) - 1;
        next(q, m0);
    }
    __device__ __forceinline__ void start_warp(const Requests& q, int m0) {
        r = first_request_warp(q, m0) - 1;
        next(q, m0);
    }
    __device__ __forceinline__ void next(const Requests& q, int m0) {
        for (++r; r < q.n_req; ++r) {
            lo = q.offsets[r];
            hi = q.offsets[r + 1];
            a = q.adapter[r];
            if (lo >= m0 + SPAN) break;
            if (hi > lo && hi > m0 && a >= 0 && a < q.n_ad) return;
        }
        r = q.n_req;
    }
    __device__ __forceinline__ bool more(const Requests& q) const { return r < q.n_req; }
};
using Walk = WalkOf<128>;

__host__ __device__ __forceinline__ int padded_rank(int R) { return R <= 16 ? 16 : R <= 32 ? 32 : R <= 64 ? 64 : 128; }

// ------------------------------------------------------------------ mma.sync pieces

__device__ __forceinline__ void ldsm4(uint32_t a, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t a, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void mma16816(float* d, const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// 16 bytes, zeros where not `in`.
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool in) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// Chunk c (16 bytes) of row r of a tile with rows of `row` bytes, permuted so
// that eight consecutive rows lie in different banks.
template <int ROW>
__device__ __forceinline__ uint32_t at(int r, int c) {
    if (ROW == 32) return r * 32 + ((c ^ ((r >> 2) & 1)) << 4);
    if (ROW == 64) return r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
    return r * ROW + ((c ^ (r & 7)) << 4);
}

// A kernel lets the next one of its stream start, and waits for the one before
// it to be through (nothing to wait for where it was launched plainly).
__device__ __forceinline__ void dependents_may_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_primary() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// ------------------------------------------------------------------ t and u

constexpr int kDownStages = 4;

// t (from x and A) or u (from g = s dqkv and B) of the pairs of one 128-row
// tile, RT rows a block: rows by 16 over the warps (RT 64), or, where there
// are few tiles, 16 rows whose contraction the four warps share (RT 16).
// Bound by the read of x (dqkv), which the large product then finds in L2
// where it fits: x of 49152 x 2048 at rank 64 in 38 us, 5.3 TB/s; x and dqkv of
// 65536 x (512 + 1536) at rank 16 in 46 us, 5.8 TB/s. RP: the rank, padded.
template <int RP, bool BWD, int RT>
__device__ __forceinline__ void down_rows(const LoraParams& p, uint16_t* out) {
    constexpr int X_TILE = RT * 128, B_TILE = RP * 128, STAGE = X_TILE + B_TILE, NT = RP / 8;
    extern __shared__ __align__(128) uint8_t smem[];
    const uint32_t base = smem_u32(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int m_first = blockIdx.x * RT, m0 = m_first & ~127;
    const int K = BWD ? p.N : p.C, blocks = (K + 63) / 64;
    const uint16_t* const src = BWD ? p.dqkv : p.x;
    const int g = lane >> 2, c2 = lane & 3;

    const Requests rq = requests_of(p);
    Walk w;
    int turn = 0;   // the requests of a tile in turns over the blocks along z
    for (w.start_warp(rq, m0); w.more(rq); w.next(rq, m0)) {
        if (turn++ % int(gridDim.z) != int(blockIdx.z)) continue;
        uint16_t* const to = out + ((int64_t(m0 >> 7) + w.r) * 128 + (m_first & 127)) * RP;
        const int lo = max(w.lo, m_first), hi = min(min(w.hi, p.M), m_first + RT);   // rows of this block
        if (lo >= hi) {
            for (int i = threadIdx.x; i < RT * RP / 8; i += 128) reinterpret_cast<uint4*>(to)[i] = make_uint4(0, 0, 0, 0);
            continue;
        }
        // this thread's 16-byte pieces of a stage, the same rows of x (of A, or columns of B) in
        // each: pointers that move on by a block, so that a load is an addition and a copy
        constexpr int XJ = RT * 8 / 128, BJ = RP / 16;
        const int xc = (threadIdx.x & 7) * 8;   // column in a 64-column block
        const uint16_t *xp[XJ], *bp[BJ];
        uint32_t x_in = 0, b_in = 0;
#pragma unroll
        for (int j = 0; j < XJ; ++j) {
            const int m = m_first + (threadIdx.x >> 3) + 16 * j;
            const bool in = m >= lo && m < hi;
            x_in |= uint32_t(in) << j;
            xp[j] = src + (in ? int64_t(m) * K + xc : 0);
        }
        constexpr int PR = RP / 8;   // pieces of a row of B
#pragma unroll
        for (int j = 0; j < BJ; ++j) {
            const int i = threadIdx.x + 128 * j, r = BWD ? i / PR : i >> 3, c = BWD ? i % PR : i & 7;
            const bool in = BWD ? c * 8 < p.R : r < p.R;
            b_in |= uint32_t(in) << j;
            bp[j] = BWD ? p.b + (in ? (int64_t(w.a) * K + r) * p.R + c * 8 : 0) : p.a + (in ? (int64_t(w.a) * p.R + r) * K + c * 8 : 0);
        }
        auto load = [&](int kb) {   // blocks in order, each once
            const uint32_t st = base + (kb % kDownStages) * STAGE;
            const int left = K - kb * 64;
#pragma unroll
            for (int j = 0; j < XJ; ++j) {
                const bool in = (x_in >> j & 1u) && xc < left;
                cp16(st + at<128>((threadIdx.x >> 3) + 16 * j, threadIdx.x & 7), in ? xp[j] : src, in);
                xp[j] += 64;
            }
#pragma unroll
            for (int j = 0; j < BJ; ++j) {
                const int i = threadIdx.x + 128 * j, r = BWD ? i / PR : i >> 3, c = BWD ? i % PR : i & 7;
                const bool in = (b_in >> j & 1u) && (BWD ? r : c * 8) < left;
                cp16(st + X_TILE + (BWD ? at<RP * 2>(r, c) : at<128>(r, c)), in ? bp[j] : src, in);
                bp[j] += BWD ? int64_t(64) * p.R : 64;
            }
        };
        float acc[NT][4] = {};
        auto step = [&](int kb, int kk, int row16) {   // 16 of the contraction
            const uint32_t st = base + (kb % kDownStages) * STAGE, bt = st + X_TILE;
            uint32_t a[4], f[NT / 2][4];   // all loads before the products that wait for them
            ldsm4(st + at<128>(row16 + (lane & 15), 2 * kk + (lane >> 4)), a);
#pragma unroll
            for (int j = 0; j < NT / 2; ++j) {
                if (!BWD) ldsm4(bt + at<128>(16 * j + (lane & 15), 2 * kk + (lane >> 4)), f[j]);
                else ldsm4t(bt + at<RP * 2>(16 * kk + (lane & 15), 2 * j + (lane >> 4)), f[j]);
            }
#pragma unroll
            for (int j = 0; j < NT / 2; ++j) {
                mma16816(acc[2 * j], a, f[j][0], f[j][BWD ? 1 : 2]);
                mma16816(acc[2 * j + 1], a, f[j][BWD ? 2 : 1], f[j][3]);
            }
        };
        __syncthreads();   // the stages of the request before are read
        for (int s = 0; s < kDownStages - 1; ++s) {
            if (s < blocks) load(s);
            cp_commit();
        }
        bool scaled = !BWD;   // the q block's sums have got their scale
        for (int kb = 0; kb < blocks; ++kb) {
            cp_wait<kDownStages - 2>();
            __syncthreads();
            if (kb + kDownStages - 1 < blocks) load(kb + kDownStages - 1);
            cp_commit();
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
                if (RT == 16 && kk != warp) continue;
                // the q block comes first: its sums are scaled once it is through (Nq is a
                // multiple of 16)
                if (!scaled && kb * 64 + kk * 16 >= p.Nq) {
                    scaled = true;
#pragma unroll
                    for (int j = 0; j < NT; ++j)
#pragma unroll
                        for (int i = 0; i < 4; ++i) acc[j][i] *= p.q_scale;
                }
                step(kb, kk, RT == 16 ? 0 : 16 * warp);
            }
        }
        cp_wait<0>();
        if (!scaled)   // a warp of RT 16 that met no column behind the q block
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[j][i] *= p.q_scale;
        const float by = p.scaling[w.a];
        if (RT == 16) {   // the warps' parts of the sum, in their order
            float* part = reinterpret_cast<float*>(smem);
            __syncthreads();
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    part[warp * 16 * RP + (g + 8 * (i >> 1)) * RP + 8 * j + 2 * c2 + (i & 1)] = acc[j][i];
            __syncthreads();
            for (int i = threadIdx.x; i < 16 * RP; i += 128) {
                const int m = m_first + i / RP;
                const float s = (part[i] + part[16 * RP + i]) + (part[32 * RP + i] + part[48 * RP + i]);
                to[i] = m >= lo && m < hi ? b16(s * by) : uint16_t(0);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = 16 * warp + g + 8 * i, m = m_first + r;
                const bool in = m >= lo && m < hi;
#pragma unroll
                for (int j = 0; j < NT; ++j)
                    *reinterpret_cast<uint32_t*>(to + r * RP + 8 * j + 2 * c2) =
                        in ? pack_bf16x2(acc[j][2 * i] * by, acc[j][2 * i + 1] * by) : 0u;
            }
        }
    }
}

template <int RP, int RT>
__global__ void __launch_bounds__(128) lora_down(const LoraParams p, uint16_t* t) {
    dependents_may_start();
    down_rows<RP, false, RT>(p, t);
}

// Both of the backward pass: u, then (blockIdx.y 1) t.
template <int RP, int RT>
__global__ void __launch_bounds__(128) lora_down_both(const LoraParams p, uint16_t* t, uint16_t* u) {
    wait_for_primary();   // the plan's offsets
    dependents_may_start();
    if (blockIdx.y == 0) down_rows<RP, true, RT>(p, u);
    else down_rows<RP, false, RT>(p, t);
}

// ------------------------------------------------------------------ the large product

constexpr int kBM = 128, kBN = 256, kBK = 64;
constexpr int kThreads = 320;   // eight epilogue warps, a loading and an issuing one

// As many requests are kept in shared memory: each role of a block walks them
// for each tile, and trips to memory for the offsets would hold up its loads
// (103 -> 95 us at 65536 x 512 x 1536).
constexpr int kFewRequests = 1024;

// Shared memory of a block, alone (CG 1) or one of a pair (CG 2): each block of
// a pair holds its own 128 rows of A and half of the columns of B.
template <int CG>
struct Shape {
    static constexpr int kStages = CG == 2 ? 6 : 4;
    static constexpr int BN = kBN / CG;
    static constexpr int A_TILE = kBM * kBK * 2, B_TILE = BN * kBK * 2, STAGE = A_TILE + B_TILE;
    static constexpr int OFF_BAR = kStages * STAGE;
    static constexpr int B_FULL = 0, B_EMPTY = kStages, B_AFULL = 2 * kStages, B_AEMPTY = B_AFULL + 2,
                         B_DRAIN = B_AEMPTY + 2, NBAR = B_DRAIN + 1;
    static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;   // tensor memory's address, abort flag, beat
    static constexpr int OFF_BEAT = OFF_MISC + 8;
    static constexpr int OFF_BIAS = (OFF_MISC + 16 + 15) & ~15;   // a tile's bias, fp32, for each epilogue warp its columns
    static constexpr int OFF_REQ = OFF_BIAS + 8 * 128 * 4;        // the requests, where they are few
    static constexpr int SMEM = OFF_REQ + (2 * kFewRequests + 1) * 4 + 1024;
};
constexpr uint64_t kWaitLimitNs = 2000000000ull;
constexpr uint64_t kDrainLimitNs = 500000000ull;

// About a millisecond a tick.
__device__ __forceinline__ uint32_t beat_clock() { return uint32_t(globaltimer_ns() >> 20); }

// Has the block given up? It does kWaitLimitNs after this wait began (t0) and after the last beat.
__device__ __noinline__ bool gave_up(volatile uint32_t* abort_flag, uint64_t t0) {
    if (abort_flag[0]) return true;
    if (globaltimer_ns() - t0 <= kWaitLimitNs || beat_clock() - abort_flag[1] <= uint32_t(kWaitLimitNs >> 20)) return false;
    abort_flag[0] = 1u;
    atomicOr(&g_lora_timeout_flag, 1u);
    return true;
}

struct Sync {
    uint32_t bar0;
    // behind it the beat: when a thread of the block or its pair was last on a value by itself (beat_clock())
    volatile uint32_t* abort_flag;
    __device__ __forceinline__ uint32_t bar(int i) const { return bar0 + 8u * i; }
    // (the other block of a pair arrives on some of the barriers)
    static __device__ __forceinline__ bool try_wait(uint32_t b, uint32_t parity) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok) : "r"(b), "r"(parity) : "memory");
        return ok != 0;
    }
    // Wait for a barrier phase; false once this block has given up.
    __device__ __forceinline__ bool wait(uint32_t b, uint32_t parity) const {
        if (try_wait(b, parity)) return true;
        const uint64_t t0 = globaltimer_ns();
        for (uint32_t it = 1;; ++it) {
            if (try_wait(b, parity)) return true;
            if ((it & 1023u) == 0u && gave_up(abort_flag, t0)) return false;
        }
    }
};

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int32_t c0, int32_t c1,
                                            int32_t c2) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2),
        "r"(bar) : "memory");
}

// Pairs of blocks (cta_group::2): a cluster of two whose tensor cores work on one
// tile of 256 rows. The leader (rank 0) issues; barriers that both sides of a
// pair signal are the leader's.
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ uint32_t leaders(uint32_t addr) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(addr));
    return r;
}
__device__ __forceinline__ void arrive_cluster(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
template <int CG>
__device__ __forceinline__ void load_2d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int32_t c0, int32_t c1) {
    if (CG == 1) {
        tma_load_2d(dst, map, bar, c0, c1);
    } else {
        asm volatile(
            "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar)
            : "memory");
    }
}
template <int CG>
__device__ __forceinline__ void load_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int32_t c0, int32_t c1, int32_t c2) {
    if (CG == 1) {
        tma_load_3d(dst, map, bar, c0, c1, c2);
    } else {
        asm volatile(
            "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2),
            "r"(bar) : "memory");
    }
}
template <int CG, uint32_t ACC>
__device__ __forceinline__ void umma(uint32_t d, uint32_t a_lo, uint32_t a_hi, uint32_t b_lo, uint32_t b_hi, uint32_t idesc) {
    if (CG == 1) {
        umma_ss_halves<ACC>(d, a_lo, a_hi, b_lo, b_hi, idesc);
    } else {
        asm volatile(
            "{\n\t.reg .b64 da, db;\n\t.reg .pred p;\n\t"
            "mov.b64 da, {%1, %2};\n\t"
            "mov.b64 db, {%3, %4};\n\t"
            "setp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], da, db, %5, p;\n\t}" ::"r"(d), "r"(a_lo), "r"(a_hi), "r"(b_lo),
            "r"(b_hi), "r"(idesc), "n"(ACC) : "memory");
    }
}
// Arrive on `bar` (of both blocks of a pair) once the products issued so far are done.
template <int CG>
__device__ __forceinline__ void commit(uint32_t bar) {
    if (CG == 1) {
        umma_commit(bar);
    } else {
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
                     "h"(uint16_t(3)) : "memory");
    }
}

struct GemmParams {
    int32_t K, cols;            // contraction and output columns
    int32_t n_tiles, n_tiles_n, k_blocks;
    int32_t out_v8;             // 1: output rows allow 32-byte stores
    int32_t t_rows;             // rows of t
    const uint16_t* t;          // pairs of t (u), [block][128][padded rank]
    uint16_t* out;
};

// The time into the beat of the block, or of both of a pair.
template <int CG>
__device__ __forceinline__ void give_beat(uint32_t addr) {
    const uint32_t now = beat_clock();
#pragma unroll
    for (uint32_t r = 0; r < CG; ++r) {
        uint32_t at = addr;
        if (CG == 2) asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(addr), "r"(r));
        if (CG == 2) asm volatile("st.relaxed.cluster.shared::cluster.u32 [%0], %1;" ::"r"(at), "r"(now) : "memory");
        else asm volatile("st.relaxed.cta.shared::cta.u32 [%0], %1;" ::"r"(at), "r"(now) : "memory");
    }
}

// One output value from the inputs, for a row whose tile holds another
// request's values that are not finite. The accumulator is held meanwhile,
// for a long contraction longer than the other roles' waits allow: every
// kBeat terms a thread leaves the time in shared memory, and they wait on.
constexpr int kBeat = 4096;
template <bool BWD, int CG>
__device__ __noinline__ float lone_value(const LoraParams& p, const GemmParams& q, int m, int col) {
    extern __shared__ uint8_t smem_raw[];
    const uint32_t beat = ((smem_u32(smem_raw) + 1023u) & ~1023u) + Shape<CG>::OFF_BEAT;
    float s = 0.f, sq = 0.f;
    const int rp = padded_rank(p.R), terms = BWD ? p.N : p.C;
    for (int k0 = 0, k1; k0 < terms; k0 = k1) {
        give_beat<CG>(beat);
        k1 = k0 + min(terms - k0, kBeat);
        if (!BWD) {
            for (int c = k0; c < k1; ++c) s = fmaf(f32(p.x[int64_t(m) * p.C + c]), f32(p.w[int64_t(col) * p.C + c]), s);
        } else {
            for (int n = k0; n < k1; ++n) {
                if (n == p.Nq) { sq = s * p.q_scale; s = 0.f; }
                s = fmaf(f32(p.dqkv[int64_t(m) * p.N + n]), f32(p.w[int64_t(n) * p.C + col]), s);
            }
        }
    }
    s += sq;
    const Requests rq = requests_of(p);
    Walk w;
    for (w.start(rq, m & ~127); w.more(rq); w.next(rq, m & ~127)) {
        if (m < w.lo || m >= w.hi) continue;
        const uint16_t* t = q.t + ((int64_t(m >> 7) + w.r) * 128 + (m & 127)) * rp;
        for (int r = 0; r < p.R; ++r)
            s = fmaf(f32(t[r]), f32(BWD ? p.a[(int64_t(w.a) * p.R + r) * p.C + col] : p.b[(int64_t(w.a) * p.N + col) * p.R + r]), s);
    }
    return s;
}

// FWD: qkv = s_n (x W^T + bias + t B^T); BWD: dx = g W + u A with W and A read
// along their columns. A persistent, warp-specialised tcgen05 product, one
// block per SM, tiles of 128 x 256:
//   warps 0..7  epilogue, two for each quarter of the rows (TMEM lanes), 128
//               columns each;
//   warp 8      TMA producer: 64-column blocks of the contraction into a ring
//               of four stages, then each adapter's block;
//   warp 9      MMA issuer, owns the tensor memory.
// FWD alternates two 256-column accumulators between tiles. BWD gives the q
// block's contraction one accumulator and the rest the other, since only the
// first is scaled (HD^-0.5 is no power of two for every HD): the epilogue
// takes the scaled q sums into registers while the rest accumulates, which
// frees that accumulator for the next tile.
// CG 2: pairs of blocks on tiles of 256 x 256, each bringing in half of B. At
// C = 512 what bounds the product is the 49 bytes a cycle that an SM takes in
// from L2: 96 bytes of operands for each of its 128 x 256 x 1 products alone,
// 64 in a pair. In pairs the epilogue follows: at 65536 x 512 x 1536, rank 32,
// t and product took 109 us with 64 columns at a time, 106 of those without any
// operand load, 90 without the stores of the results, 86 without the whole
// epilogue; 32 columns at a time take 103. Storing through shared memory, by
// TMA (103 -> 111 us then) or in whole lines (102), does not help. At
// 49152 x 2048 x 6144, rank 64, the tensor cores bound it (90 % of their cycles):
// 702 us, 1.82 PFLOP/s. The backward product of 65536 x 1536 x 512 takes 93 us;
// 97 while it stored before it freed the second accumulator.
template <bool BWD, int CG>
__global__ void __launch_bounds__(kThreads, 1)
lora_gemm(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
          const __grid_constant__ CUtensorMap tm_t, const __grid_constant__ CUtensorMap tm_l,
          const __grid_constant__ LoraParams p, const __grid_constant__ GemmParams q) {
    using S = Shape<CG>;
    constexpr int kStages = S::kStages, A_TILE = S::A_TILE, STAGE = S::STAGE, BN = S::BN;
    constexpr int B_FULL = S::B_FULL, B_EMPTY = S::B_EMPTY, B_AFULL = S::B_AFULL, B_AEMPTY = S::B_AEMPTY, B_DRAIN = S::B_DRAIN;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* base_ptr = smem_raw + (base - raw);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rp = padded_rank(p.R), rb = rp < 64 ? rp : 64;   // an adapter's columns, and a block's

    volatile uint32_t* misc = reinterpret_cast<volatile uint32_t*>(base_ptr + S::OFF_MISC);
    Sync sy{base + S::OFF_BAR, misc + 1};
    const int rank = CG == 2 ? int(cluster_rank()) : 0, unit = blockIdx.x / CG, units = gridDim.x / CG;
    if (threadIdx.x == 0) {
        for (int i = 0; i < S::NBAR; ++i) mbar_init(sy.bar(i), (i >= B_AEMPTY && i < B_AEMPTY + 2) ? 256u * CG : 1u);
        misc[1] = 0u;
        misc[2] = beat_clock() - uint32_t(kWaitLimitNs >> 20) - 1u;   // long ago
        fence_mbar_init();
    }
    Requests rq = requests_of(p);
    if (p.n_req <= kFewRequests) {
        int32_t* const kept = reinterpret_cast<int32_t*>(base_ptr + S::OFF_REQ);
        for (int r = threadIdx.x; r <= p.n_req; r += kThreads) kept[r] = p.offsets[r];
        for (int r = threadIdx.x; r < p.n_req; r += kThreads) kept[kFewRequests + 1 + r] = p.adapter[r];
        rq.offsets = kept;
        rq.adapter = kept + kFewRequests + 1;
    }
    if (warp == 8 && lane == 0) {
        tma_prefetch_desc(&tm_a);
        tma_prefetch_desc(&tm_b);
        tma_prefetch_desc(&tm_t);
        tma_prefetch_desc(&tm_l);
    }
    if (warp == 9) {
        if (CG == 1) {
            tmem_alloc(base + S::OFF_MISC, 512);
            tmem_relinquish();
        } else {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(base + S::OFF_MISC), "r"(512)
                         : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
        }
    }
    tc_fence_before();
    __syncthreads();
    if (CG == 2) cluster_sync();   // both blocks' barriers are there
    tc_fence_after();
    const uint32_t tmem = misc[0];

    if (warp == 8 && lane == 0) {
        // ---------------------------------------------------------- producer
        uint32_t it = 0;
        bool ok = true;
        for (int t = unit; ok && t < q.n_tiles; t += units) {
            const int i = t / q.n_tiles_n * CG + rank, m0 = i * kBM, span0 = m0 - rank * kBM;
            const int n0 = (t % q.n_tiles_n) * kBN + rank * BN;   // of this block's part of B
            for (int kb = 0; kb < q.k_blocks; ++kb, ++it) {
                const uint32_t st = it % kStages, to = base + st * STAGE;
                if (!sy.wait(sy.bar(B_EMPTY + st), ((it / kStages) & 1u) ^ 1u)) { ok = false; break; }
                const uint32_t full = CG == 2 ? leaders(sy.bar(B_FULL + st)) : sy.bar(B_FULL + st);
                if (rank == 0) mbar_arrive_expect_tx(sy.bar(B_FULL + st), STAGE * CG);
                load_2d<CG>(to, &tm_a, full, kb * kBK, m0);
                if (!BWD) {
                    load_2d<CG>(to + A_TILE, &tm_b, full, kb * kBK, n0);
                } else {
                    for (int c = 0; c < BN / 64; ++c)
                        load_2d<CG>(to + A_TILE + c * (kBK * 128), &tm_b, full, n0 + c * 64, kb * kBK);
                }
            }
            WalkOf<kBM * CG> w;
            w.start(rq, span0);
            if (w.more(rq)) wait_for_primary();   // t
            for (; ok && w.more(rq); w.next(rq, span0))
                for (int r0 = 0; r0 < rp; r0 += rb, ++it) {
                    const uint32_t st = it % kStages, to = base + st * STAGE;
                    if (!sy.wait(sy.bar(B_EMPTY + st), ((it / kStages) & 1u) ^ 1u)) { ok = false; break; }
                    const uint32_t full = CG == 2 ? leaders(sy.bar(B_FULL + st)) : sy.bar(B_FULL + st);
                    if (rank == 0) mbar_arrive_expect_tx(sy.bar(B_FULL + st), (kBM + BN) * rb * 2 * CG);
                    // the other block's request: zeros (rows past the tensor) for this one
                    const bool mine = w.lo < m0 + kBM && w.hi > m0;
                    load_2d<CG>(to, &tm_t, full, r0, mine ? (i + w.r) * kBM : q.t_rows);
                    if (!BWD) {
                        load_2d<CG>(to + A_TILE, &tm_l, full, r0, w.a * p.N + n0);
                    } else {
                        for (int c = 0; c < BN / 64; ++c)
                            load_3d<CG>(to + A_TILE + c * (rb * 128), &tm_l, full, n0 + c * 64, r0, w.a);
                    }
                }
        }
        wait_for_primary();
        // every issued load lands before the CTA may exit (the pair's end waits for the leader)
        for (uint32_t s = 0; rank == 0 && s < kStages; ++s) {
            const uint32_t f = it / kStages + (s < it % kStages ? 1u : 0u);
            if (f && !mbar_wait_bounded(sy.bar(B_FULL + s), (f - 1u) & 1u, kDrainLimitNs))
                atomicOr(&g_lora_timeout_flag, 1u);
        }
    } else if (warp == 9 && lane == 0 && rank == 0) {
        // ---------------------------------------------------------- MMA issuer
        const uint32_t idesc = make_idesc_bf16(kBM * CG, kBN, 0, BWD ? 1 : 0);
        const uint64_t ad0 = make_smem_desc(base, 16, 1024, kSwizzle128B);
        // BWD: columns outermost in memory (MN-major), 64 to a region of kBK rows
        const uint64_t bd0 = make_smem_desc(base + A_TILE, BWD ? kBK * 128 : 16, 1024, kSwizzle128B);
        const uint32_t swz = rb == 64 ? kSwizzle128B : rb == 32 ? kSwizzle64B : kSwizzle32B;
        const uint64_t td0 = make_smem_desc(base, 16, rb * 16, swz);
        const uint64_t ld0 = BWD ? make_smem_desc(base + A_TILE, rb * 128, 1024, kSwizzle128B)
                                 : make_smem_desc(base + A_TILE, 16, rb * 16, swz);
        const uint32_t a_hi = uint32_t(ad0 >> 32), b_hi = uint32_t(bd0 >> 32);
        const uint32_t t_hi = uint32_t(td0 >> 32), l_hi = uint32_t(ld0 >> 32);
        constexpr uint32_t b_step = BWD ? (16 * 128) >> 4 : 2;   // 16 of the contraction further
        uint32_t it = 0, lt = 0;
        bool ok = true;
        for (int t = unit; ok && t < q.n_tiles; t += units, ++lt) {
            const int m0 = (t / q.n_tiles_n) * kBM * CG;
            // FWD: this tile's accumulator; BWD: 0, then 1 behind the q block
            uint32_t buf = BWD ? 0u : lt & 1u;
            if (!sy.wait(sy.bar(B_AEMPTY + buf), ((BWD ? lt : lt >> 1) & 1u) ^ 1u)) break;
            tc_fence_after();
            uint32_t d = tmem + buf * kBN;
            bool fresh = true;
            for (int kb = 0; kb < q.k_blocks; ++kb, ++it) {
                const uint32_t st = it % kStages;
                if (!sy.wait(sy.bar(B_FULL + st), (it / kStages) & 1u)) { ok = false; break; }
                tc_fence_after();
                const uint32_t a_lo = uint32_t(ad0) + ((st * STAGE) >> 4), b_lo = uint32_t(bd0) + ((st * STAGE) >> 4);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                    if (BWD && buf == 0 && kb * kBK + kk * 16 >= p.Nq) {
                        commit<CG>(sy.bar(B_AFULL));
                        buf = 1;
                        if (!sy.wait(sy.bar(B_AEMPTY + 1), (lt & 1u) ^ 1u)) { ok = false; break; }
                        tc_fence_after();
                        d = tmem + kBN;
                        fresh = true;
                    }
                    if (fresh) umma<CG, 0>(d, a_lo + kk * 2, a_hi, b_lo + kk * b_step, b_hi, idesc);
                    else umma<CG, 1>(d, a_lo + kk * 2, a_hi, b_lo + kk * b_step, b_hi, idesc);
                    fresh = false;
                }
                if (!ok) break;
                commit<CG>(sy.bar(B_EMPTY + st));
            }
            WalkOf<kBM * CG> w;
            for (w.start(rq, m0); ok && w.more(rq); w.next(rq, m0))
                for (int r0 = 0; r0 < rp; r0 += rb, ++it) {
                    const uint32_t st = it % kStages;
                    if (!sy.wait(sy.bar(B_FULL + st), (it / kStages) & 1u)) { ok = false; break; }
                    tc_fence_after();
                    const uint32_t a_lo = uint32_t(td0) + ((st * STAGE) >> 4), b_lo = uint32_t(ld0) + ((st * STAGE) >> 4);
                    for (int kk = 0; kk < rb / 16; ++kk)
                        umma<CG, 1>(d, a_lo + kk * 2, t_hi, b_lo + kk * b_step, l_hi, idesc);
                    commit<CG>(sy.bar(B_EMPTY + st));
                }
            if (!ok) break;
            commit<CG>(sy.bar(B_AFULL + buf));
        }
        commit<CG>(sy.bar(B_DRAIN));
        if (!mbar_wait_bounded(sy.bar(B_DRAIN), 0, kDrainLimitNs)) atomicOr(&g_lora_timeout_flag, 1u);
    } else if (warp < 8) {
        // ---------------------------------------------------------- epilogue
        wait_for_primary();
        dependents_may_start();   // who reads t and u too
        const int quad = warp & 3, half = warp >> 2;
        const uint32_t t_row = tmem + (uint32_t(quad * 32) << 16) + half * 128;
        float* bias_s = reinterpret_cast<float*>(base_ptr + S::OFF_BIAS) + warp * 128;   // this warp's copy
        // the bias of a tile's columns (0 past N or without bias), read a tile ahead
        float bias_r[4];
        auto read_bias = [&](int t) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int c = (t % q.n_tiles_n) * kBN + half * 128 + 32 * i + lane;
                bias_r[i] = (p.bias && t < q.n_tiles && c < p.N) ? f32(p.bias[c]) : 0.f;
            }
        };
        if (!BWD) read_bias(unit);
        uint32_t lt = 0;
        for (int t = unit; t < q.n_tiles; t += units, ++lt) {
            const int m0 = ((t / q.n_tiles_n) * CG + rank) * kBM, n0 = (t % q.n_tiles_n) * kBN + half * 128;
            const int row = m0 + quad * 32 + lane;
            uint16_t* orow = q.out + int64_t(row) * q.cols;
            if (!BWD) {
#pragma unroll
                for (int i = 0; i < 4; ++i) bias_s[32 * i + lane] = bias_r[i];
                __syncwarp();
                read_bias(t + units);
            }
            float held[BWD ? 128 : 1];   // BWD: the scaled sums of the q block
            if (BWD) {
                if (!sy.wait(sy.bar(B_AFULL), lt & 1u)) break;
                tc_fence_after();
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_ld32(t_row + 32 * c, held + (BWD ? 32 * c : 0));
                tmem_wait_ld();
                tc_fence_before();
                if (CG == 2) arrive_cluster(leaders(sy.bar(B_AEMPTY)));
                else mbar_arrive(sy.bar(B_AEMPTY));
            }
            const uint32_t buf = BWD ? 1u : lt & 1u;
            if (!sy.wait(sy.bar(B_AFULL + buf), (BWD ? lt : lt >> 1) & 1u)) break;
            tc_fence_after();
            if (BWD) {   // all sums first: the next tile's are waiting for the accumulator
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    float acc[32];
                    tmem_ld32(t_row + kBN + 32 * c, acc);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 32; ++j) held[BWD ? 32 * c + j : 0] = fmaf(held[BWD ? 32 * c + j : 0], p.q_scale, acc[j]);
                }
                tc_fence_before();
                if (CG == 2) arrive_cluster(leaders(sy.bar(B_AEMPTY + 1)));
                else mbar_arrive(sy.bar(B_AEMPTY + 1));
            }
            constexpr int W = 32;   // columns at a time (64: longer bursts of stores, 109 us for 103 at 65536 x 512 x 1536)
#pragma unroll
            for (int c = 0; c < 128 / W; ++c) {
                const int c0 = n0 + W * c;
                float acc[W];
                if (BWD) {
#pragma unroll
                    for (int j = 0; j < W; ++j) acc[j] = held[BWD ? W * c + j : 0];
                } else {
                    __syncwarp();   // lanes with values by themselves come later; the load is the whole warp's
                    tmem_ld32(t_row + buf * kBN + W * c, acc);
                    tmem_wait_ld();
                    if (c == 128 / W - 1) {   // the accumulator is read
                        tc_fence_before();
                        if (CG == 2) arrive_cluster(leaders(sy.bar(B_AEMPTY + buf)));
                        else mbar_arrive(sy.bar(B_AEMPTY + buf));
                    }
                }
                if (c0 >= q.cols || row >= p.M) continue;
                float top = 0.f;
#pragma unroll
                for (int j = 0; j < W; j += 2)
                    asm("max.NaN.f32 %0, %0, %1, %2;" : "+f"(top) : "f"(fabsf(acc[j])), "f"(fabsf(acc[j + 1])));
                if (!(top < INFINITY)) {
                    // where the tile holds rows of more than one request, the value may be another's
                    const int span0 = m0 - rank * kBM;
                    WalkOf<kBM * CG> w;
                    w.start(rq, span0);
                    if (w.more(rq) && (w.lo > span0 || w.hi < min(span0 + kBM * CG, p.M)))
#pragma unroll 1
                        for (int j = 0; j < W && c0 + j < q.cols; ++j) {
                            const float x = lone_value<BWD, CG>(p, q, row, c0 + j);
#pragma unroll
                            for (int k = 0; k < W; ++k)
                                if (k == j) acc[k] = x;
                        }
                }
                uint32_t pk[W / 2];
#pragma unroll
                for (int j = 0; j < W / 2; j += 2) {
                    float v[4] = {acc[2 * j], acc[2 * j + 1], acc[2 * j + 2], acc[2 * j + 3]};
                    if (!BWD) {
                        const float4 b = *reinterpret_cast<const float4*>(bias_s + W * c + 2 * j);
                        // the q block (columns below NH * HD, a multiple of 16) carries the HD^-0.5 scale
                        const float by = c0 + (2 * j & ~15) < p.Nq ? p.q_scale : 1.f;
                        v[0] = (v[0] + b.x) * by;
                        v[1] = (v[1] + b.y) * by;
                        v[2] = (v[2] + b.z) * by;
                        v[3] = (v[3] + b.w) * by;
                    }
                    pk[j] = pack_bf16x2(v[0], v[1]);
                    pk[j + 1] = pack_bf16x2(v[2], v[3]);
                }
                const int nval = min(W, q.cols - c0);   // a multiple of 8
#pragma unroll
                for (int i = 0; i < W / 16; ++i) {
                    if (q.out_v8 && 16 * i + 16 <= nval) {
                        st_global_v8(orow + c0 + 16 * i, pk + 8 * i);
                    } else {
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            if (16 * i + 8 * h < nval)
                                *reinterpret_cast<uint4*>(orow + c0 + 16 * i + 8 * h) =
                                    make_uint4(pk[8 * i + 4 * h], pk[8 * i + 4 * h + 1], pk[8 * i + 4 * h + 2], pk[8 * i + 4 * h + 3]);
                    }
                }
            }
            __syncwarp();   // the bias copy is rewritten for the next tile
        }
    }

    tc_fence_before();
    __syncthreads();
    if (CG == 2) cluster_sync();   // no block ends while the other may still reach its memory
    if (warp == 9) {
        tc_fence_after();
        if (CG == 1) tmem_dealloc(tmem, 512);
        else asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
    }
}

// ------------------------------------------------------------------ few rows

// Up to here the product streams W past the rows: 32 rows of 2048 channels to
// 6144 take 10.8 us so, 19.9 in the large product (512 to 1536: 5.1 and 10.4).
constexpr int kSmallRows = 32;

// t of up to kSmallRows rows, [row][R]: a warp for each value. Latency: 7 us by
// itself, hidden behind the product's read of W.
__global__ void __launch_bounds__(256) lora_down_few(const LoraParams p, uint16_t* t) {
    dependents_may_start();
    const int m = blockIdx.x, r = blockIdx.y * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    const Requests rq = requests_of(p);
    Walk w;
    for (w.start_warp(rq, m); w.more(rq) && w.hi <= m; w.next(rq, m)) {}
    if (!w.more(rq) || w.lo > m) return;   // nothing reads this row's
    const uint4* x = reinterpret_cast<const uint4*>(p.x + int64_t(m) * p.C);
    const uint4* a = reinterpret_cast<const uint4*>(p.a + (int64_t(w.a) * p.R + r) * p.C);
    float s = 0.f;
#pragma unroll 4
    for (int i = lane; i < p.C / 8; i += 32) {
        const uint4 u = x[i], v = a[i];
        const uint32_t e[4] = {u.x, u.y, u.z, u.w}, f[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            s = fmaf(__uint_as_float(e[k] << 16), __uint_as_float(f[k] << 16), s);
            s = fmaf(__uint_as_float(e[k] & 0xffff0000u), __uint_as_float(f[k] & 0xffff0000u), s);
        }
    }
#pragma unroll
    for (int k = 16; k; k >>= 1) s += __shfl_xor_sync(0xffffffffu, s, k);
    if (lane == 0) t[m * p.R + r] = b16(s * p.scaling[w.a]);
}

// qkv of up to 8 * MT rows: a block takes 16 rows of W, read once from memory
// straight into fragments (a thread's 16 bytes are 8 consecutive channels, the
// same for W and x, so the contraction is permuted alike on both sides), its
// warps an eighth of the channels each. Bound by the read of W; t is waited for
// behind it only. Eight rows of 2048 channels to 6144 columns, W from memory:
// 12 us by itself, 2.2 TB/s; replayed with its t about 9 (the call's own work on
// the host is 24).
template <int MT>
__global__ void __launch_bounds__(256) lora_fwd_few(const LoraParams p, const uint16_t* t) {
    constexpr int U = MT <= 2 ? 4 : 2;   // blocks of 32 channels in flight
    __shared__ float part[8][16][8 * MT + 1];
    __shared__ int row_adapter[8 * MT];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c2 = lane & 3;
    const int n0 = blockIdx.x * 16;   // N is a multiple of 16
    const uint16_t* const w0 = p.w + int64_t(n0 + g) * p.C;
    const uint16_t* const w1 = w0 + int64_t(8) * p.C;
    if (int(threadIdx.x) < p.M) {   // one row's adapter, -1 for none
        const Requests rq = requests_of(p);
        const int m = threadIdx.x;
        Walk w;
        w.start(rq, m);
        row_adapter[m] = w.more(rq) && w.lo <= m ? w.a : -1;
    }
    const uint4 zero = make_uint4(0, 0, 0, 0);
    float acc[MT][4] = {};
    const int blocks = (p.C + 31) / 32;
    for (int b = warp; b < blocks; b += 8 * U) {
        uint4 a0[U], a1[U], x[U][MT];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = (b + 8 * u) * 32 + 8 * c2;
            const bool in = c < p.C;
            a0[u] = in ? *reinterpret_cast<const uint4*>(w0 + c) : zero;
            a1[u] = in ? *reinterpret_cast<const uint4*>(w1 + c) : zero;
#pragma unroll
            for (int i = 0; i < MT; ++i)
                x[u][i] = in && 8 * i + g < p.M ? *reinterpret_cast<const uint4*>(p.x + int64_t(8 * i + g) * p.C + c) : zero;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t lo[4] = {a0[u].x, a1[u].x, a0[u].y, a1[u].y}, hi[4] = {a0[u].z, a1[u].z, a0[u].w, a1[u].w};
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                mma16816(acc[i], lo, x[u][i].x, x[u][i].y);
                mma16816(acc[i], hi, x[u][i].z, x[u][i].w);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) part[warp][g + 8 * (k >> 1)][8 * i + 2 * c2 + (k & 1)] = acc[i][k];
    wait_for_primary();
    __syncthreads();
    for (int e = threadIdx.x; e < 16 * p.M; e += 256) {
        const int n = e & 15, m = e >> 4, col = n0 + n;
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) s += part[i][n][m];
        if (p.bias) s += f32(p.bias[col]);
        const int a = row_adapter[m];
        if (a >= 0) {
            const uint4* b = reinterpret_cast<const uint4*>(p.b + (int64_t(a) * p.N + col) * p.R);
            const uint4* tm = reinterpret_cast<const uint4*>(t + m * p.R);
            for (int i = 0; i < p.R / 8; ++i) {
                const uint4 u = b[i], v = tm[i];
                const uint32_t f[4] = {u.x, u.y, u.z, u.w}, h[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    s = fmaf(__uint_as_float(h[k] << 16), __uint_as_float(f[k] << 16), s);
                    s = fmaf(__uint_as_float(h[k] & 0xffff0000u), __uint_as_float(f[k] & 0xffff0000u), s);
                }
            }
        }
        p.qkv[int64_t(m) * p.N + col] = b16(s * (col < p.Nq ? p.q_scale : 1.f));
    }
}

// ------------------------------------------------------------------ adapters' gradients

constexpr int kChunk = 64;   // rows of a request that lora_grad takes at a time

// Where the rows of each adapter are: offsets made non-decreasing and kept in
// 0 .. M (which good ones are already), the requests with an adapter in the
// order of the adapters, and the chunks of each request and adapter.
struct Plan {
    int32_t *offsets;      // n_req + 1
    int32_t *request;      // n_req, by adapter
    int32_t *first;        // n_req + 1: first chunk of request[i]
    int32_t *ad_first;     // n_ad + 1: first chunk of an adapter
    int32_t *ad_req;       // n_ad + 1: first place of an adapter in request[]
};

__host__ __device__ __forceinline__ Plan plan_at(void* work, int n_req, int n_ad) {
    Plan q;
    q.offsets = static_cast<int32_t*>(work);
    q.request = q.offsets + n_req + 1;
    q.first = q.request + n_req;
    q.ad_first = q.first + n_req + 1;
    q.ad_req = q.ad_first + n_ad + 1;
    return q;
}

// One block; latency, 5 us for four requests. A thread looks at every request
// for each of its adapters, twice: 0.36 ms for 4096 requests of 64 adapters,
// 4.4 ms of 4096, and 67 ms for 16384 of as many, before anything else starts.
__global__ void __launch_bounds__(256) lora_plan(const LoraParams p, const Plan q) {
    dependents_may_start();
    __shared__ int top[256];
    const int per = (p.n_req + 256) / 256, lo = min(int(threadIdx.x) * per, p.n_req + 1), hi = min(lo + per, p.n_req + 1);
    int m = 0;
    for (int i = lo; i < hi; ++i) m = max(m, min(p.offsets[i], p.M));
    top[threadIdx.x] = m;
    __syncthreads();
    m = 0;
    for (int i = 0; i < int(threadIdx.x); ++i) m = max(m, top[i]);
    for (int i = lo; i < hi; ++i) {
        m = max(m, min(p.offsets[i], p.M));
        q.offsets[i] = m;
    }
    __syncthreads();
    for (int a = threadIdx.x; a < p.n_ad; a += 256) {
        int n = 0, c = 0;
        for (int r = 0; r < p.n_req; ++r)
            if (p.adapter[r] == a) {
                ++n;
                c += (q.offsets[r + 1] - q.offsets[r] + kChunk - 1) / kChunk;
            }
        q.ad_req[a + 1] = n;
        q.ad_first[a + 1] = c;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        q.ad_req[0] = q.ad_first[0] = 0;
        for (int a = 0; a < p.n_ad; ++a) {
            q.ad_req[a + 1] += q.ad_req[a];
            q.ad_first[a + 1] += q.ad_first[a];
        }
        q.first[q.ad_req[p.n_ad]] = q.ad_first[p.n_ad];
    }
    __syncthreads();
    for (int a = threadIdx.x; a < p.n_ad; a += 256) {
        int n = q.ad_req[a], c = q.ad_first[a];
        for (int r = 0; r < p.n_req; ++r)
            if (p.adapter[r] == a) {
                q.request[n] = r;
                q.first[n++] = c;
                c += (q.offsets[r + 1] - q.offsets[r] + kChunk - 1) / kChunk;
            }
    }
}

constexpr int kGradStages = 3;

// Part of dA_a = u^T x (blocks of columns below C) and dB_a^T = t^T dqkv (the
// others): one block takes 128 columns and an equal run of the chunks, which
// are in the order of the adapters, and writes a sum for each adapter that it
// meets. Part s + a: along the runs one of the two grows, so the parts are as
// few as splits and adapters together. Bound by the read of x and dqkv: 65536 x
// (512 + 1536) at rank 16 in 49 us, 5.5 TB/s.
template <int RP>
__global__ void __launch_bounds__(256) lora_grad(const LoraParams p, const Plan q, const uint16_t* tt, const uint16_t* uu,
                                                 float* part, int splits, bool beside) {
    // beside the large product, which started behind t and u; else behind those
    if (!beside) wait_for_primary();
    dependents_may_start();
    constexpr int X_TILE = kChunk * 256, U_TILE = kChunk * RP * 2, STAGE_G = X_TILE + U_TILE, MT = RP / 16;
    extern __shared__ __align__(128) uint8_t smem[];
    const uint32_t base = smem_u32(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c2 = lane & 3;
    const int c_blocks = (p.C + 127) / 128;
    const bool is_b = int(blockIdx.x) >= c_blocks;
    const int cols = is_b ? p.N : p.C, col0 = (is_b ? blockIdx.x - c_blocks : blockIdx.x) * 128;
    const uint16_t* const x = is_b ? p.dqkv : p.x;
    const uint16_t* const u = is_b ? tt : uu;
    const int total = q.ad_first[p.n_ad], per = (total + splits - 1) / splits;
    const int first = blockIdx.y * per, last = min(first + per, total);
    if (first >= last) {
        if (beside) wait_for_primary();
        return;
    }

    // the place of the first chunk: the last request that starts at or before it
    int j = 0;
    {
        int hi = q.ad_req[p.n_ad];
        while (j + 1 < hi) {
            const int mid = (j + hi) >> 1;
            if (q.first[mid] <= first) j = mid;
            else hi = mid;
        }
    }
    const int n_sorted = q.ad_req[p.n_ad];
    int jl = j;   // of the loads
    auto load = [&](int c) {
        const uint32_t st = base + (c - first) % kGradStages * STAGE_G;
        while (jl + 1 < n_sorted && q.first[jl + 1] <= c) ++jl;
        const int r = q.request[jl], m0 = q.offsets[r] + (c - q.first[jl]) * kChunk, end = q.offsets[r + 1];
        for (int i = threadIdx.x; i < kChunk * 16; i += 256) {
            const int k = i >> 4, cc = i & 15, m = m0 + k, col = col0 + cc * 8;
            const bool in = m < end && col < cols;
            cp16(st + (cc >> 3) * (kChunk * 128) + at<128>(k, cc & 7), x + (in ? int64_t(m) * cols + col : 0), in);
        }
        for (int i = threadIdx.x; i < kChunk * (RP / 8); i += 256) {
            const int k = i / (RP / 8), cc = i % (RP / 8), m = m0 + k;
            const bool in = m < end;
            cp16(st + X_TILE + at<RP * 2>(k, cc), u + (in ? ((int64_t(m >> 7) + r) * 128 + (m & 127)) * RP + cc * 8 : 0), in);
        }
    };
    float acc[MT][2][4] = {};
    int a = p.adapter[q.request[j]];
    auto flush = [&] {
        float* to = part + (int64_t(blockIdx.y) + a) * RP * (p.C + p.N) + (is_b ? p.C : 0);
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int row = 16 * t + g + 8 * (i >> 1), col = col0 + 16 * warp + 8 * n + 2 * c2 + (i & 1);
                    if (col < cols) to[int64_t(row) * (p.C + p.N) + col] = acc[t][n][i];
                    acc[t][n][i] = 0.f;
                }
    };
    for (int s = 0; s < kGradStages - 1; ++s) {
        if (first + s < last) load(first + s);
        cp_commit();
    }
    for (int c = first; c < last; ++c) {
        cp_wait<kGradStages - 2>();
        __syncthreads();
        if (c + kGradStages - 1 < last) load(c + kGradStages - 1);
        cp_commit();
        bool moved = false;
        while (j + 1 < n_sorted && q.first[j + 1] <= c) { ++j; moved = true; }
        if (moved && p.adapter[q.request[j]] != a) {
            flush();
            a = p.adapter[q.request[j]];
        }
        const uint32_t st = base + (c - first) % kGradStages * STAGE_G;
#pragma unroll
        for (int kk = 0; kk < kChunk / 16; ++kk) {
            uint32_t f[4], e[4];
            const int k = 16 * kk + (lane & 15), cc = 2 * warp + (lane >> 4);
            ldsm4t(st + (cc >> 3) * (kChunk * 128) + at<128>(k, cc & 7), f);
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                // rows of u are the contraction: transposed, 16 of its columns are the rows of A
                ldsm4t(st + X_TILE + at<RP * 2>(16 * kk + (lane & 7) + 8 * (lane >> 4), 2 * t + ((lane >> 3) & 1)), e);
                mma16816(acc[t][0], e, f[0], f[1]);
                mma16816(acc[t][1], e, f[2], f[3]);
            }
        }
    }
    cp_wait<0>();
    flush();
    if (beside) wait_for_primary();   // ends behind the product beside it
}

// The parts of each adapter, in their order, to dA (n_ad, R, C) and dB
// (n_ad, N, R), the q block's rows of dB scaled. A thread sums one value: the
// parts lie far apart, so what counts is how many reads are under way (eight:
// 45 -> 8 us for three adapters of rank 16 over 2048 columns).
__global__ void __launch_bounds__(256) lora_grad_sum(const LoraParams p, const Plan q, const float* part, int splits, int rp) {
    wait_for_primary();
    const int cols = p.C + p.N;
    const int64_t e = int64_t(blockIdx.x) * 256 + threadIdx.x;
    if (e >= int64_t(p.n_ad) * p.R * cols) return;
    const int col = int(e % cols), r = int(e / cols % p.R), a = int(e / cols / p.R);
    const int total = q.ad_first[p.n_ad], per = (total + splits - 1) / splits;
    const int c0 = q.ad_first[a], c1 = q.ad_first[a + 1];
    float s = 0.f;
    if (c0 < c1) {
        const int k1 = (c1 - 1) / per;
        const float* from = part + ((int64_t(c0 / per) + a) * rp + r) * cols + col;
        const int64_t next = int64_t(rp) * cols;
        int k = c0 / per;
        for (; k + 7 <= k1; k += 8, from += 8 * next) {
            float x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = from[i * next];
#pragma unroll
            for (int i = 0; i < 8; ++i) s += x[i];
        }
        for (; k <= k1; ++k, from += next) s += *from;
    }
    if (col < p.C) p.da[(int64_t(a) * p.R + r) * p.C + col] = b16(s);
    else p.db[(int64_t(a) * p.N + col - p.C) * p.R + r] = b16(s * (col - p.C < p.Nq ? p.q_scale : 1.f));
}

// ------------------------------------------------------------------ launch

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t align256(int64_t x) { return (x + 255) / 256 * 256; }

// Runs of chunks that lora_grad's blocks share a column block's rows by. Blocks
// that are all resident at once on 152 SMs (a fixed count, since the workspace
// and the order of the sums follow it): 65536 rows of 512 channels take, whole calls,
// at ranks 16, 32, 64 and 128 with 2 blocks an SM 216, 222, 242 and 332 us, with
// 3 194, 200, 259 and 363, with 4 186, 210, 246 and 337.
int grad_splits(int64_t M, int64_t C, int64_t N, int64_t R) {
    const int rp = padded_rank(int(R)), per_sm = rp == 16 ? 4 : rp == 32 ? 3 : 2;
    const int64_t s = per_sm * 152 / (ceil_div(C, 128) + ceil_div(N, 128)), most = ceil_div(M, kChunk);
    return int(s < 1 ? 1 : s > most ? most : s);
}

struct Work {
    int64_t t, u, plan, part, bytes;
};

Work lay_out(int64_t M, int64_t C, int64_t N, int64_t R, int64_t n_req, int64_t n_ad, bool backward) {
    Work w;
    const int64_t rp = padded_rank(int(R)), pairs = (ceil_div(M, 128) + n_req) * 128 * rp * 2;
    w.t = 0;
    w.u = w.t + align256(pairs);
    w.plan = w.u + (backward ? align256(pairs) : 0);
    w.part = w.plan + (backward ? align256((3 * n_req + 2 * n_ad + 4) * 4) : 0);
    w.bytes = w.part + (backward ? (grad_splits(M, C, N, R) + n_ad) * rp * (C + N) * 4 : 0);
    return w;
}

// A tensor map of up to three dimensions of bf16, strides in elements.
bool map_of(CUtensorMap* m, const void* ptr, int dims, const int64_t* size, const int64_t* stride, int box0, int box1) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    cuuint64_t d[3], s[2];
    const cuuint32_t box[3] = {cuuint32_t(box0), cuuint32_t(box1), 1}, one[3] = {1, 1, 1};
    for (int i = 0; i < dims; ++i) d[i] = cuuint64_t(size[i]);
    for (int i = 0; i + 1 < dims; ++i) s[i] = cuuint64_t(stride[i] * 2);
    const CUtensorMapSwizzle swz = box0 == 64   ? CU_TENSOR_MAP_SWIZZLE_128B
                                   : box0 == 32 ? CU_TENSOR_MAP_SWIZZLE_64B
                                                : CU_TENSOR_MAP_SWIZZLE_32B;
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, dims, const_cast<void*>(ptr), d, s, box, one,
              CU_TENSOR_MAP_INTERLEAVE_NONE, swz, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A launch that may start while the kernel before it, which lets it, still
// runs; it waits for that kernel itself where it reads its results.
template <class... P, class... A>
cudaError_t launch_dependent(void (*kernel)(P...), dim3 grid, unsigned threads, int smem, cudaStream_t stream, int cluster,
                             const A&... args) {
    cudaLaunchConfig_t c = {};
    cudaLaunchAttribute a[2] = {};
    a[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    a[0].val.programmaticStreamSerializationAllowed = 1;
    a[1].id = cudaLaunchAttributeClusterDimension;
    a[1].val.clusterDim.x = unsigned(cluster);
    a[1].val.clusterDim.y = a[1].val.clusterDim.z = 1;
    c.gridDim = grid;
    c.blockDim = dim3(threads);
    c.dynamicSmemBytes = smem;
    c.stream = stream;
    c.attrs = a;
    c.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&c, kernel, P(args)...);
}

// t, or with `u` both.
template <int RP, int RT>
cudaError_t down_t(const LoraParams& p, uint16_t* t, uint16_t* u, int sms, cudaStream_t stream) {
    constexpr int smem = kDownStages * (RT * 128 + RP * 128);
    static_assert(RT != 16 || 4 * 16 * RP * 4 <= smem, "the warps' parts fit the stages");
    if (smem > 48 * 1024) {
        const cudaError_t e =
            u ? cudaFuncSetAttribute(lora_down_both<RP, RT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)
              : cudaFuncSetAttribute(lora_down<RP, RT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
    }
    const unsigned grid = unsigned(ceil_div(p.M, 128) * 128 / RT);
    // Few rows of many requests: these in parallel too, up to four blocks an SM (16 requests in 40
    // rows, backward from 5760 columns to 896: 186 -> 61 us; 40 in 54, forward: 52 -> 28).
    const int64_t room = int64_t(4) * sms / (int64_t(grid) * (u ? 2 : 1));
    const unsigned turns = unsigned(room < 1 ? 1 : room > p.n_req ? p.n_req : room);
    if (u) return launch_dependent(lora_down_both<RP, RT>, dim3(grid, 2, turns), 128, smem, stream, 1, p, t, u);
    lora_down<RP, RT><<<dim3(grid, 1, turns), 128, smem, stream>>>(p, t);
    return cudaGetLastError();
}

cudaError_t down(const LoraParams& p, uint16_t* t, uint16_t* u, int sms, cudaStream_t stream) {
    // Whole calls of 128 rows of 2048 channels take 18 us with 16 rows a block and 29 with 64, 1024
    // rows 28.8 and 29.5; from 1536 rows on 64 are as good or better (512 channels: 11.6 and 9.4;
    // 4096 rows: 17.2 and 14.8), since 16 read the adapter four times as often.
    const bool small = p.M < 8 * sms;
    switch (padded_rank(p.R)) {
        case 16: return small ? down_t<16, 16>(p, t, u, sms, stream) : down_t<16, 64>(p, t, u, sms, stream);
        case 32: return small ? down_t<32, 16>(p, t, u, sms, stream) : down_t<32, 64>(p, t, u, sms, stream);
        case 64: return small ? down_t<64, 16>(p, t, u, sms, stream) : down_t<64, 64>(p, t, u, sms, stream);
        default: return small ? down_t<128, 16>(p, t, u, sms, stream) : down_t<128, 64>(p, t, u, sms, stream);
    }
}

template <bool BWD, int CG>
cudaError_t gemm_t(const LoraParams& p, const uint16_t* t, int sms, cudaStream_t stream) {
    GemmParams q{};
    q.K = BWD ? p.N : p.C;
    q.cols = BWD ? p.C : p.N;
    q.n_tiles_n = int32_t(ceil_div(q.cols, kBN));
    const int64_t tiles = ceil_div(p.M, kBM * CG) * q.n_tiles_n;
    if (tiles >= (int64_t(1) << 31)) return cudaErrorInvalidValue;
    q.n_tiles = int32_t(tiles);
    q.k_blocks = int32_t(ceil_div(q.K, kBK));
    q.t = t;
    q.out = BWD ? p.dx : p.qkv;
    q.out_v8 = reinterpret_cast<uintptr_t>(q.out) % 32 == 0 && q.cols % 16 == 0;
    const int rp = padded_rank(p.R), rb = rp < 64 ? rp : 64;
    CUtensorMap ta, tb, tt, tl;
    const int64_t blocks = (ceil_div(p.M, 128) + p.n_req) * 128;
    q.t_rows = int32_t(blocks);
    const int64_t sa[2] = {q.K, p.M}, ka[1] = {q.K}, st[2] = {rp, blocks}, kt[1] = {rp};
    const int64_t sw[2] = {p.C, p.N}, kw[1] = {p.C};
    const int64_t sb[2] = {p.R, int64_t(p.n_ad) * p.N}, kb[1] = {p.R};
    const int64_t sl[3] = {p.C, p.R, p.n_ad}, kl[2] = {p.C, int64_t(p.R) * p.C};
    bool ok = map_of(&ta, BWD ? p.dqkv : p.x, 2, sa, ka, 64, kBM) && map_of(&tt, t, 2, st, kt, rb, kBM);
    if (BWD) ok = ok && map_of(&tb, p.w, 2, sw, kw, 64, kBK) && map_of(&tl, p.a, 3, sl, kl, 64, rb);
    else ok = ok && map_of(&tb, p.w, 2, sw, kw, 64, Shape<CG>::BN) && map_of(&tl, p.b, 2, sb, kb, rb, Shape<CG>::BN);
    if (!ok) return cudaErrorInvalidValue;
    const cudaError_t e =
        cudaFuncSetAttribute(lora_gemm<BWD, CG>, cudaFuncAttributeMaxDynamicSharedMemorySize, Shape<CG>::SMEM);
    if (e != cudaSuccess) return e;
    const int64_t units = sms / CG;
    return launch_dependent(lora_gemm<BWD, CG>, dim3(unsigned((tiles < units ? tiles : units) * CG)), kThreads, Shape<CG>::SMEM,
                            stream, CG, ta, tb, tt, tl, p, q);
}

template <bool BWD>
cudaError_t gemm(const LoraParams& p, const uint16_t* t, int sms, cudaStream_t stream) {
    // Pairs where each has six tiles of 256 rows. Whole forward calls of 4096, 16384, 24576 and
    // 65536 rows of 512 channels to 1536 take 17.8, 33.5, 44.1 and 107 us by pairs and 16.4, 32.7,
    // 47.4 and 114 by blocks, 49152 of 2048 to 6144 753 and 794; backward 16384 and 65536 rows of 512
    // channels 63.4 and 187 by pairs, 61.5 and 190 by blocks, 49152 of 2048 1263 and 1294.
    return (p.M / (2 * kBM)) * ceil_div(BWD ? p.C : p.N, kBN) >= 3 * sms ? gemm_t<BWD, 2>(p, t, sms, stream)
                                                                        : gemm_t<BWD, 1>(p, t, sms, stream);
}

template <int RP>
cudaError_t grad(const LoraParams& p, const Plan& q, const uint16_t* t, const uint16_t* u, float* part, cudaStream_t stream) {
    constexpr int smem = kGradStages * (kChunk * 256 + kChunk * RP * 2);
    cudaError_t e = cudaFuncSetAttribute(lora_grad<RP>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    const int splits = grad_splits(p.M, p.C, p.N, p.R);
    const dim3 grid(unsigned(ceil_div(p.C, 128) + ceil_div(p.N, 128)), unsigned(splits));
    e = launch_dependent(lora_grad<RP>, grid, 256, smem, stream, 1, p, q, t, u, part, splits, p.dx != nullptr);
    if (e != cudaSuccess) return e;
    const int64_t n = int64_t(p.n_ad) * p.R * (int64_t(p.C) + p.N);
    return launch_dependent(lora_grad_sum, dim3(unsigned(ceil_div(n, 256))), 256, 0, stream, 1, p, q, part, splits, RP);
}

}  // namespace

static std::atomic<bool> g_launched{false};

int64_t lora_workspace(int64_t M, int64_t C, int64_t N, int64_t R, int64_t n_req, int64_t n_ad, bool backward) {
    return lay_out(M, C, N, R, n_req, n_ad, backward).bytes;
}

cudaError_t launch_lora_fwd(const LoraParams& p, int sms, cudaStream_t stream) {
    g_launched = true;
    uint16_t* t = static_cast<uint16_t*>(p.work);
    if (p.M <= kSmallRows) {
        lora_down_few<<<dim3(unsigned(p.M), unsigned(p.R / 8)), 256, 0, stream>>>(p, t);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
        const dim3 grid(unsigned(p.N / 16));
        if (p.M <= 8) return launch_dependent(lora_fwd_few<1>, grid, 256, 0, stream, 1, p, t);
        if (p.M <= 16) return launch_dependent(lora_fwd_few<2>, grid, 256, 0, stream, 1, p, t);
        return launch_dependent(lora_fwd_few<4>, grid, 256, 0, stream, 1, p, t);
    }
    const cudaError_t e = down(p, t, nullptr, sms, stream);
    return e != cudaSuccess ? e : gemm<false>(p, t, sms, stream);
}

cudaError_t launch_lora_bwd(const LoraParams& p0, int sms, cudaStream_t stream) {
    g_launched = true;
    const Work w = lay_out(p0.M, p0.C, p0.N, p0.R, p0.n_req, p0.n_ad, true);
    uint8_t* work = static_cast<uint8_t*>(p0.work);
    uint16_t *t = reinterpret_cast<uint16_t*>(work + w.t), *u = reinterpret_cast<uint16_t*>(work + w.u);
    const Plan q = plan_at(work + w.plan, p0.n_req, p0.n_ad);
    lora_plan<<<1, 256, 0, stream>>>(p0, q);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    LoraParams p = p0;   // every pass walks the plan's offsets
    p.offsets = q.offsets;
    if ((e = down(p, t, u, sms, stream)) != cudaSuccess) return e;
    if (p.dx && (e = gemm<true>(p, u, sms, stream)) != cudaSuccess) return e;
    float* part = reinterpret_cast<float*>(work + w.part);
    switch (padded_rank(p.R)) {
        case 16: return grad<16>(p, q, t, u, part, stream);
        case 32: return grad<32>(p, q, t, u, part, stream);
        case 64: return grad<64>(p, q, t, u, part, stream);
        default: return grad<128>(p, q, t, u, part, stream);
    }
}

// The flag is taken as for the attention kernel: one atomic exchange per
// status request, its old value left in a slot of that request's own. A process
// that has launched none of these kernels has nothing to ask for.
constexpr unsigned int kStatusSlots = 256;
__device__ unsigned int g_lora_status_slots[kStatusSlots];

__global__ void take_lora_flag(unsigned int slot) { g_lora_status_slots[slot] = atomicExch(&g_lora_timeout_flag, 0u); }

cudaError_t take_lora_error(cudaStream_t stream, unsigned int* flag) {
    *flag = 0;
    if (!g_launched) return cudaSuccess;
    static std::atomic<unsigned int> next{0};
    const unsigned int slot = next.fetch_add(1u) % kStatusSlots;
    take_lora_flag<<<1, 1, 0, stream>>>(slot);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    e = cudaMemcpyFromSymbolAsync(flag, g_lora_status_slots, sizeof(unsigned int), slot * sizeof(unsigned int),
                                  cudaMemcpyDeviceToHost, stream);
    if (e != cudaSuccess) return e;
    return cudaStreamSynchronize(stream);
}

}  // namespace na3d
