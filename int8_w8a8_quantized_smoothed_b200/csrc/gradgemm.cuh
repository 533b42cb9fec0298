// The gradients of a W8A8 linear on the 5th-generation tensor cores (tcgen05.mma kind::f16, bf16
// operands, binary32 accumulators):
//
//   C[i, j] = sum_r A(i, r) B(r, j),   B(r, j) = bf16(s[r] Q[r, j])
//
//   input gradient   i = token,   r = output channel, j = input channel:  A = dy, Q = wq, s = s_ch
//   weight gradient  i = output channel, r = token,   j = input channel:  A = dy^T, Q = xq, s = s_tok
//
// Both sum over the rows of the 8-bit matrix Q, which is the dimension its scales belong to, so
// the scale cannot wait for the epilogue: Q becomes a scaled bf16 operand, its codes exact in bf16
// and the product with the scale rounded once. That rounding, the same as a weight dequantized to
// bf16 has, is as large as the output's: with the two the 2-norm error is 2.3e-3 of the result's,
// with the output's alone 1.7e-3. Without it (dy s in two bf16 parts against the bare codes) there
// would be twice the MMAs, which set the time of all but the narrow form. Three forms:
//   narrow    at most 128 rows i of an input gradient: the codes are streamed once, converted into
//             tensor memory (below);
//   CONV      warps of the kernel turn Q's tiles into bf16 tiles in shared memory: a code is read
//             as one byte and never stored as two;
//   otherwise grad_dequant_kernel writes all of B first and the kernel loads both operands: each
//             of Q's tiles is converted once, not once for every tile of rows i.
// B's tiles keep Q's layout (rows r, j contiguous: the MMA's MN-major form), as does A in the
// weight gradient (dy's rows are r), so nothing is transposed in memory.
#pragma once

#include "gemm.cuh"

namespace w8a8 {

// warps: 0 A producer, 1 MMA, 2 Q producer (CONV); 4 .. 7 epilogue; from 8 on converters (CONV)
constexpr int kGradConvWarp0 = 8;
constexpr int kGradTile = 256; // columns j of a pair's tile, and rows i (of each half, if two)
constexpr int kGradBR = 64;    // r per k-block: one 128-byte row of bf16

// Tiles [0, whole) go to the pairs one after another; the remaining tiles' k-blocks are split
// evenly over rem_pairs pairs, whose partial tiles grad_fixup_kernel adds.
struct GradWork {
    int I, J, R;
    int tile_i, tile_j; // 256 or 512 x 256 for a CTA pair; narrow kernel: 16 .. 128 x 128 for a CTA
    int ni, nj, kblocks, group_i;
    int npairs, whole, rem, rem_pairs; // (narrow kernel: CTAs)
};

struct GradSegment {
    int tile, kb0, kb1;
    bool partial;
    int slot; // of a partial segment: 0 for the first tile of the pair's split range, 1 for the next
};

// A pair's segments in order; every role walks the same ones.
struct GradWalk {
    int next_whole;
    int64_t u, u1;
    __device__ __forceinline__ GradWalk(const GradWork &w, int pair)
    {
        next_whole = pair;
        const int64_t U = static_cast<int64_t>(w.rem) * w.kblocks;
        const bool in = pair < w.rem_pairs;
        u = in ? pair * U / w.rem_pairs : 0;
        u1 = in ? (pair + 1) * U / w.rem_pairs : 0;
        first = static_cast<int>(u / w.kblocks);
    }
    int first;
    __device__ __forceinline__ bool next(const GradWork &w, GradSegment &s)
    {
        if (next_whole < w.whole) {
            s = GradSegment{next_whole, 0, w.kblocks, false, 0};
            next_whole += w.npairs;
            return true;
        }
        if (u >= u1)
            return false;
        const SkSegment sg = sk_segment(u, u1, w.kblocks);
        const int t = static_cast<int>(sg.t);
        s = GradSegment{w.whole + t, sg.kb0, sg.kb1, sg.kb1 - sg.kb0 < w.kblocks, t != first};
        u += sg.kb1 - sg.kb0;
        return true;
    }
};

// A pair's k-blocks one after another across its segments, some at a time.
struct GradBlocks {
    GradWalk walk;
    GradSegment sg;
    int kb;
    bool ok;
    __device__ __forceinline__ GradBlocks(const GradWork &w, int pair, int skip) : walk(w, pair)
    {
        ok = walk.next(w, sg);
        kb = sg.kb0;
        if (ok)
            advance(w, skip);
    }
    __device__ __forceinline__ void advance(const GradWork &w, int n)
    {
        kb += n;
        while (ok && kb >= sg.kb1) {
            const int over = kb - sg.kb1;
            ok = walk.next(w, sg);
            kb = sg.kb0 + over;
        }
    }
};

// CONV: the kernel converts Q itself; otherwise B is a bf16 matrix loaded like A.
// H: the tile's halves of 256 rows i, both multiplied by the same converted tile of B.
template <bool CONV, int H> struct GradCfg {
    static_assert(H == 1 || (H == 2 && CONV), "halves");
    static constexpr int GROUPS = H == 2 ? 3 : 4; // of converter warps, each on its own k-block
    static constexpr int GROUP_WARPS = 4;
    static constexpr int STAGES = H == 2 ? 3 : CONV ? 4 : 6;
    static constexpr int QSTAGES = CONV ? 2 * GROUPS : 0; // two a group: one is loaded meanwhile
    // A converter group meets a stage of either ring again only after it has used it before (see
    // the narrow kernel's).
    static_assert(QSTAGES % GROUPS == 0 && (!CONV || STAGES % GROUPS == 0), "rings and groups");
    static constexpr int kThreads = (kGradConvWarp0 + (CONV ? GROUPS * GROUP_WARPS : 0)) * 32;
    static constexpr int kHalfBytes = 128 * kGradBR * 2;
    static constexpr int kABytes = H * kHalfBytes;
    static constexpr int kBBytes = 128 * kGradBR * 2;
    static constexpr int kQBytes = 128 * kGradBR;
    static constexpr int kBOff = STAGES * kABytes;
    static constexpr int kQOff = kBOff + STAGES * kBBytes;
    static constexpr int kOutOff = kQOff + QSTAGES * kQBytes; // 2 x 4 KB per epilogue warp
    static constexpr int kBarOff = kOutOff + 4 * 8192;
    // full[S], empty[S], qfull[QS], qempty[QS], tfull[2], tempty[2], tensor-memory slot
    static constexpr int kSmemBytes = kBarOff + (2 * STAGES + 2 * QSTAGES + 6) * 8 + 16 + 1024;
    static_assert(kSmemBytes <= 232448, "shared memory per CTA");
    // two 128 x 256 accumulators per CTA: of two tiles by turns, or of a tile's halves
    static constexpr int kTmemCols = 512;
};

// 256-row bf16 MMA over the pair (see umma_i8_pair).
__device__ __forceinline__ void umma_bf16_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                               uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Instruction descriptor of kind::f16 with bf16 A and B and a binary32 D, each operand K-major or
// MN-major.
__host__ __device__ constexpr uint32_t idesc_bf16(int m, int n, bool a_mn, bool b_mn)
{
    return (1u << 4)                                // D format: F32
           | (1u << 7)                              // A format: BF16
           | (1u << 10)                             // B format: BF16
           | ((a_mn ? 1u : 0u) << 15)               // A MN-major
           | ((b_mn ? 1u : 0u) << 16)               // B MN-major
           | (static_cast<uint32_t>(n >> 3) << 17)  // N / 8
           | (static_cast<uint32_t>(m >> 4) << 24); // M / 16
}

// MN-major operand in 128-byte-swizzled shared memory: chunks of 64 values of the M or N side,
// each [64 k][64 values] with rows of 128 bytes. Eight k rows form a 1024-byte swizzle atom (the
// stride byte offset); the next chunk starts 8192 bytes on (the leading byte offset). Advancing
// `saddr` by 2048 selects the next 16 k.
__device__ __forceinline__ uint64_t sw128_mnmajor_desc(uint32_t saddr)
{
    uint64_t d = 0;
    d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
    d |= static_cast<uint64_t>(8192u >> 4) << 16;
    d |= static_cast<uint64_t>(1024u >> 4) << 32;
    d |= static_cast<uint64_t>(1u) << 46;
    d |= static_cast<uint64_t>(2u) << 61;
    return d;
}

// Arrive on an mbarrier of either CTA of the pair (a cluster address), for the pair's MMA, which is
// issued in the even CTA and reads both CTAs' converted tiles. The release is at cluster scope, as
// the odd CTA's stores are published to a thread outside it, but of stores to this CTA's shared
// memory alone (each behind its own thread's proxy fence): a release of all of memory took about
// 2000 cycles, which four groups of converters could not hide (2048 x 28672 x 4096 in tiles of 256
// rows 440 us, 401 with this one), nor could a warp that passes the groups' arrivals on (in tiles of
// 512 rows 396 us, 343 to 351 with this one).
__device__ __forceinline__ void mbar_arrive_pair(uint32_t bar_cluster)
{
    asm volatile("fence.release.sync_restrict::shared::cta.cluster;\n\t"
                 "mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar_cluster)
                 : "memory");
}

// A ring's stage and the parity of its current round, kept running: the single-thread roles are
// chains of dependent instructions, and a remainder by the number of stages in each of them
// (with addresses computed anew) made a k-block's issue take 650 cycles.
template <int N> struct Ring {
    uint32_t s = 0, ph = 0;
    __device__ __forceinline__ void next()
    {
        if (++s == N) {
            s = 0;
            ph ^= 1u;
        }
    }
};

// mbar_wait for a barrier that the other CTA of the pair arrives on (the MMAs' commits reach both
// CTAs): acquire at cluster scope, which costs nothing that could be measured.
__device__ __forceinline__ bool mbar_wait_cluster(uint32_t bar, uint32_t parity, uint64_t limit_ns)
{
    uint64_t t0 = 0;
    while (true) {
#pragma unroll 1
        for (int i = 0; i < 32; ++i) {
            uint32_t ok;
            asm volatile("{\n\t.reg .pred p;\n\t"
                         "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
                         "selp.u32 %0, 1, 0, p;\n\t}"
                         : "=r"(ok)
                         : "r"(bar), "r"(parity)
                         : "memory");
            if (ok)
                return true;
        }
        const uint64_t now = globaltimer_ns();
        if (t0 == 0)
            t0 = now;
        if (now - t0 > limit_ns) {
            flag_timeout();
            return false;
        }
    }
}

__device__ __forceinline__ uint32_t sub_bf16x2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

__device__ __forceinline__ uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c)
{
    uint32_t r;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
    return r;
}

// Scales as the sum of two bf16 values, the nearest one and the nearest to what it leaves (2^-17
// relative together); hi and lo hold two scales' each, the first in the lower half. A scale that
// is not finite leaves a NaN.
__device__ __forceinline__ void split_scales(float s0, float s1, uint32_t &hi, uint32_t &lo)
{
    hi = pack_bf16x2(s0, s1);
    lo = pack_bf16x2(s0 - __uint_as_float(hi << 16), s1 - __uint_as_float(hi & 0xFFFF0000u));
}

// One scale's parts in both halves of a word.
struct RowScale {
    uint32_t hi, lo;
};

__device__ __forceinline__ RowScale row_scale(float s)
{
    RowScale r;
    split_scales(s, s, r.hi, r.lo);
    return r;
}

// Four codes (a 32-bit word) as exact bf16 values, v[0] the first two.
// INT8: the low 7 bits as the fraction of 128 make 128 + (q & 127), the sign bit as the lowest
// exponent bit of 128 makes 128 or 256; their difference is q.
// E4M3: exponent and fraction moved to a bf16's places make q 2^-120 (subnormals too).
template <bool F8> __device__ __forceinline__ void code_values(uint32_t w, uint32_t (&v)[2])
{
    if constexpr (F8) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const uint32_t t = __byte_perm(w, 0u, k ? 0x3424 : 0x1404);
            v[k] = mul_bf16x2(((t >> 4) & 0x07F007F0u) | (t & 0x80008000u), 0x7B807B80u);
        }
    } else {
        const uint32_t m = w & 0x7F7F7F7Fu, n = w & 0x80808080u;
#pragma unroll
        for (int k = 0; k < 2; ++k)
            v[k] = sub_bf16x2(__byte_perm(m, 0x43434343u, k ? 0x4342 : 0x4140),
                              __byte_perm(n, 0x43434343u, k ? 0x4342 : 0x4140));
    }
}

// Four codes of one row to bf16(s q), in packed bf16 arithmetic: q hi + bf16(q lo) is rounded once,
// so the result is bf16 of s q within 2^-16 relative.
template <bool F8>
__device__ __forceinline__ uint2 convert4(uint32_t w, const RowScale sc)
{
    uint32_t v[2];
    code_values<F8>(w, v);
    return make_uint2(fma_bf16x2(v[0], sc.hi, mul_bf16x2(v[0], sc.lo)),
                      fma_bf16x2(v[1], sc.hi, mul_bf16x2(v[1], sc.lo)));
}

// d(silu(g) u): with sig = 1 / (1 + exp(-g)), dg = da u sig (1 + g (1 - sig)), du = da g sig.
// exp of -|g| only, so nothing overflows; all in binary32.
__device__ __forceinline__ void silu_grad(float da, float g, float u, float &dg, float &du)
{
    const float e = __expf(-fabsf(g));
    const float inv = __fdividef(1.0f, 1.0f + e);
    const float small = e * inv;
    const float sig = g >= 0.0f ? inv : small;
    const float rest = g >= 0.0f ? small : inv;
    dg = da * u * (sig * fmaf(g, rest, 1.0f));
    du = da * (g * sig);
}

// Eight values of dg and du from eight of da and the stored bf16 gate and up values.
__device__ __forceinline__ void silu_grad8(const float (&da)[8], const uint4 rg, const uint4 ru,
                                           uint4 &og, uint4 &ou)
{
    float g[8], u[8], a[8], b[8];
    unpack8(rg, g);
    unpack8(ru, u);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        silu_grad(da[i], g[i], u[i], a[i], b[i]);
    og = make_uint4(pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3]), pack_bf16x2(a[4], a[5]),
                    pack_bf16x2(a[6], a[7]));
    ou = make_uint4(pack_bf16x2(b[0], b[1]), pack_bf16x2(b[2], b[3]), pack_bf16x2(b[4], b[5]),
                    pack_bf16x2(b[6], b[7]));
}

// A warp's 32 rows of ROW 16-byte words between global memory and its staging buffer, coalesced;
// word j of row r is kept at r * ROW + (j ^ (r * ROW / 8 & (ROW - 1))), so a lane's walk along its
// own row meets no bank conflict. Nothing is read or written outside the valid part.
template <int ROW> __device__ __forceinline__ int stage_at(int r, int j)
{
    return r * ROW + (j ^ ((r * ROW >> 3) & (ROW - 1)));
}

// Asynchronous (cp.async): stage_load_wait<N> waits for all but the last N of the lane's loads
// committed as groups; words outside the valid part keep what they held.
template <int ROW>
__device__ __forceinline__ void stage_load(uint4 *stage, int lane, const char *src, int64_t stride,
                                           int rows_valid, int bytes_valid)
{
#pragma unroll
    for (int i = 0; i < ROW; ++i) {
        const int r = (i * 32 + lane) / ROW, j = lane % ROW;
        if (r < rows_valid && j * 16 < bytes_valid)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                             smem_u32(stage + stage_at<ROW>(r, j))),
                         "l"(src + r * stride + j * 16)
                         : "memory");
    }
}

__device__ __forceinline__ void stage_load_commit()
{
    asm volatile("cp.async.commit_group;" ::: "memory");
}

template <int N> __device__ __forceinline__ void stage_load_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <int ROW>
__device__ __forceinline__ void stage_store(const uint4 *stage, int lane, char *dst, int64_t stride,
                                            int rows_valid, int bytes_valid)
{
#pragma unroll
    for (int i = 0; i < ROW; ++i) {
        const int r = (i * 32 + lane) / ROW, j = lane % ROW;
        if (r < rows_valid && j * 16 < bytes_valid)
            *reinterpret_cast<uint4 *>(dst + r * stride + j * 16) = stage[stage_at<ROW>(r, j)];
    }
}

// A CTA pair per 256 H x 256 tile (cta_group::2): each CTA holds 128 rows of A a half and 128
// columns of B and accumulates 128 x 256 a half. WGRAD: A is MN-major. SILU: the epilogue turns
// C = da into dg and du (out is [I, 2J]) with the forward call's gate|up values.
// Bound by the power limit in long runs: 2048 x 28672 x 4096 takes 347 us = 1.39 PFLOP/s, sustained
// 398 us at 1.57 GHz (the bare bf16 product by a library 316 and 351 us); a k-block of 512 rows
// takes about 1250 cycles, of them 1024 of MMA.
template <bool CONV, int H, bool WGRAD, bool F8, bool SILU>
__global__ void __launch_bounds__(GradCfg<CONV, H>::kThreads, 1)
    grad_gemm_kernel(const __grid_constant__ CUtensorMap tmA,
                     const __grid_constant__ CUtensorMap tmQ, const float *__restrict__ scale,
                     const GradWork w, const uint16_t *__restrict__ gate_up,
                     uint16_t *__restrict__ out, float *__restrict__ part,
                     unsigned long long limit_ns)
{
    using Cfg = GradCfg<CONV, H>;
    constexpr int kTileI = H * kGradTile;
    constexpr int STAGES = Cfg::STAGES, QSTAGES = CONV ? Cfg::QSTAGES : 1;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const uint32_t sbase = smem_u32(smem);
    const uint32_t sA = sbase, sB = sbase + Cfg::kBOff, sQ = sbase + Cfg::kQOff;
    const uint32_t bar_full = sbase + Cfg::kBarOff;       // used in the even CTA
    const uint32_t bar_empty = bar_full + 8 * STAGES;     // both
    const uint32_t bar_qfull = bar_empty + 8 * STAGES;    // each CTA its own
    const uint32_t bar_qempty = bar_qfull + 8 * QSTAGES;
    const uint32_t bar_tfull = bar_qempty + 8 * QSTAGES;  // both
    const uint32_t bar_tempty = bar_tfull + 16;           // used in the even CTA
    const uint32_t tslot = bar_tempty + 16;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const int pair = blockIdx.x >> 1;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            // the loads' bytes, and the group of converters of each CTA
            mbar_init(bar_full + 8 * s, CONV ? 1 + 2 * Cfg::GROUP_WARPS : 1);
            mbar_init(bar_empty + 8 * s, 1);
        }
        for (int s = 0; CONV && s < QSTAGES; ++s) {
            mbar_init(bar_qfull + 8 * s, 1);
            mbar_init(bar_qempty + 8 * s, Cfg::GROUP_WARPS);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(bar_tfull + 8 * b, 1);
            mbar_init(bar_tempty + 8 * b, 8); // 4 epilogue warps in each CTA
        }
        fence_mbar_init();
        tma_prefetch_desc(&tmA);
        tma_prefetch_desc(&tmQ);
    }
    __syncwarp();
    // both CTAs run, their barriers set, before the pair allocates tensor memory together
    cluster_sync();
    if (warp == 1)
        tmem_alloc_pair(tslot, Cfg::kTmemCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base =
        *reinterpret_cast<volatile uint32_t *>(smem + (tslot - sbase));

    // The roles' loops run on all lanes of their warp, so that the compiler keeps their state in
    // uniform registers; one lane issues.
    if (warp == 0) {
        pdl_wait();
        const uint32_t full0 = map_peer_smem(bar_full, 0);
        uint32_t it = 0;
        bool ok = true;
        Ring<STAGES> ring;
        GradWalk walk(w, pair);
        GradSegment sg;
        while (ok && walk.next(w, sg)) {
            int ib, jb;
            tile_coords(sg.tile, w.ni, w.nj, w.group_i, ib, jb);
            const int i0 = ib * kTileI + static_cast<int>(rank) * 128;
            const int j0 = jb * kGradTile + static_cast<int>(rank) * 128;
            int r0 = sg.kb0 * kGradBR;
            for (int n = sg.kb1 - sg.kb0; n > 0; --n, ++it, r0 += kGradBR) {
                if (!mbar_wait_cluster(bar_empty + 8 * ring.s, ring.ph ^ 1u, limit_ns)) {
                    ok = false;
                    break;
                }
                if (lane == 0) {
                    const uint32_t full = full0 + 8 * ring.s;
                    if (rank == 0)
                        mbar_expect_tx(bar_full + 8 * ring.s,
                                       2 * (Cfg::kABytes + (CONV ? 0 : Cfg::kBBytes)));
#pragma unroll
                    for (int h = 0; h < H; ++h) {
                        const uint32_t dst = sA + ring.s * Cfg::kABytes + h * Cfg::kHalfBytes;
                        const int i = i0 + h * kGradTile;
                        if constexpr (WGRAD) {
                            tma_load_2d_pair(dst, &tmA, full, i, r0);
                            tma_load_2d_pair(dst + 8192, &tmA, full, i + 64, r0);
                        } else {
                            tma_load_2d_pair(dst, &tmA, full, r0, i);
                        }
                    }
                    if constexpr (!CONV) {
                        const uint32_t b = sB + ring.s * Cfg::kBBytes;
                        tma_load_2d_pair(b, &tmQ, full, j0, r0);
                        tma_load_2d_pair(b + 8192, &tmQ, full, j0 + 64, r0);
                    }
                }
                __syncwarp();
                ring.next();
            }
        }
        if (ok) // every stage released by the MMAs before this CTA may leave
            drain_ring(bar_empty, it, STAGES, limit_ns);
        if (lane == 0)
            pdl_launch_dependents();
    } else if (warp == 1) {
        if (rank == 0) {
            constexpr uint32_t idesc = idesc_bf16(kGradTile, kGradTile, WGRAD, true);
            // stage 0's descriptors; a stage further on adds its bytes / 16 to the address field
            const uint64_t da = WGRAD ? sw128_mnmajor_desc(sA) : sw128_kmajor_desc(sA);
            const uint64_t db = sw128_mnmajor_desc(sB);
            constexpr uint32_t kStepA = (WGRAD ? 2048 : 32) / 16, kStepB = 2048 / 16;
            bool ok = true;
            Ring<STAGES> ring;
            // with one half the two accumulators take turns; with two each has its own
            Ring<2> acc;
            uint32_t tile_ph = 0;
            GradWalk walk(w, pair);
            GradSegment sg;
            auto free_acc = [&](int h) { // its last tile has been read out
                const uint32_t b = H == 2 ? h : acc.s, ph = H == 2 ? tile_ph : acc.ph;
                const bool got = mbar_wait_cluster(bar_tempty + 8 * b, ph ^ 1u, limit_ns);
                tc_fence_after();
                return got;
            };
            while (ok && walk.next(w, sg)) {
                if (!free_acc(0))
                    break;
                const uint32_t d = tmem_base + (H == 2 ? 0 : acc.s) * kGradTile;
                uint32_t accumulate = 0;
                for (int n = sg.kb1 - sg.kb0; n > 0; --n) {
                    if (!mbar_wait_cluster(bar_full + 8 * ring.s, ring.ph, limit_ns)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
#pragma unroll
                    for (int h = 0; h < H; ++h) {
                        if (h == 1 && !accumulate && !free_acc(1)) {
                            ok = false;
                            break;
                        }
                        if (lane == 0) {
                            const uint64_t a0 = da + ring.s * (Cfg::kABytes / 16) +
                                                h * (Cfg::kHalfBytes / 16);
                            const uint64_t b0 = db + ring.s * (Cfg::kBBytes / 16);
#pragma unroll
                            for (int k = 0; k < kGradBR / 16; ++k)
                                umma_bf16_pair(d + h * kGradTile, a0 + k * kStepA,
                                               b0 + k * kStepB, idesc, k > 0 ? 1u : accumulate);
                            if (h == H - 1)
                                umma_commit_pair(bar_empty + 8 * ring.s, 0x3);
                            if (H == 2 && n == 1)
                                umma_commit_pair(bar_tfull + 8 * h, 0x3);
                        }
                        __syncwarp();
                    }
                    if (!ok)
                        break;
                    accumulate = 1;
                    ring.next();
                }
                if (H == 1 && ok && lane == 0)
                    umma_commit_pair(bar_tfull + 8 * acc.s, 0x3);
                __syncwarp();
                acc.next();
                tile_ph ^= 1u;
            }
        }
    } else if (warp >= 4 && warp < 8) {
        // epilogue: this CTA's 128 rows of the tile, 32 per warp
        pdl_wait();
        const int quarter = warp & 3;
        uint4 *stage_w = reinterpret_cast<uint4 *>(smem + Cfg::kOutOff) + quarter * 512;
        const uint32_t tempty0 = map_peer_smem(bar_tempty, 0);
        uint32_t seg = 0;
        GradWalk walk(w, pair);
        GradSegment sg;
        while (walk.next(w, sg)) {
            int ib, jb;
            tile_coords(sg.tile, w.ni, w.nj, w.group_i, ib, jb);
            bool ok = true;
#pragma unroll 1
            for (int h = 0; h < H && ok; ++h) {
                const uint32_t buf = H == 2 ? h : seg & 1u, aph = (H == 2 ? seg : seg >> 1) & 1u;
                const int row0 = ib * kTileI + h * kGradTile + static_cast<int>(rank) * 128 + quarter * 32;
                const int rows = min(32, w.I - row0); // may be negative: nothing stored
                const int64_t ld = static_cast<int64_t>(w.J) * (SILU ? 4 : 2); // bytes
                float *slot = part + ((static_cast<int64_t>(pair) * 2 + sg.slot) * kTileI +
                                      h * kGradTile + rank * 128 + quarter * 32) * kGradTile;
                // SILU: the gate and up values of a chunk of 32 columns are on their way while the
                // chunk before it is worked on, the first ones while the tile is still multiplied
                auto fetch = [&](int c) {
                    const int j0 = jb * kGradTile + c * 32;
                    const char *gu = reinterpret_cast<const char *>(gate_up) + row0 * ld + j0 * 2;
                    const int bytes = 2 * min(32, w.J - j0);
                    uint4 *to = stage_w + (c & 1) * 256;
                    stage_load<4>(to, lane, gu, ld, rows, bytes);
                    stage_load<4>(to + 128, lane, gu + static_cast<int64_t>(w.J) * 2, ld, rows, bytes);
                    stage_load_commit();
                };
                if constexpr (SILU)
                    if (!sg.partial)
                        fetch(0);
                ok = mbar_wait_cluster(bar_tfull + 8 * buf, aph, limit_ns);
                if (!ok)
                    break;
                __syncwarp();
                tc_fence_after();
                const uint32_t tbase =
                    tmem_base + buf * kGradTile + (static_cast<uint32_t>(quarter * 32) << 16);
#pragma unroll 1
                for (int c = 0; c < kGradTile / 32; ++c) {
                    const int j0 = jb * kGradTile + c * 32;
                    uint32_t r[32];
                    if constexpr (SILU)
                        if (!sg.partial && c + 1 < kGradTile / 32)
                            fetch(c + 1);
                    tmem_ld_32x32b_x32(tbase + c * 32, r);
                    tmem_ld_wait();
                    if (sg.partial) {
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            stage_w[stage_at<8>(lane, j)] =
                                make_uint4(r[4 * j], r[4 * j + 1], r[4 * j + 2], r[4 * j + 3]);
                        __syncwarp();
                        stage_store<8>(stage_w, lane, reinterpret_cast<char *>(slot + c * 32),
                                       kGradTile * 4, rows, 128);
                    } else if constexpr (SILU) {
                        if (c + 1 < kGradTile / 32)
                            stage_load_wait<1>();
                        else
                            stage_load_wait<0>();
                        __syncwarp();
                        uint4 *st = stage_w + (c & 1) * 256;
#pragma unroll
                        for (int e = 0; e < 4; ++e) { // the lane's own row, in place
                            float da[8];
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                da[i] = __uint_as_float(r[e * 8 + i]);
                            uint4 *g = st + stage_at<4>(lane, e);
                            silu_grad8(da, g[0], g[128], g[0], g[128]);
                        }
                        __syncwarp();
                        char *dst = reinterpret_cast<char *>(out) + row0 * ld + j0 * 2;
                        const int bytes = 2 * min(32, w.J - j0);
                        stage_store<4>(st, lane, dst, ld, rows, bytes);
                        stage_store<4>(st + 128, lane, dst + static_cast<int64_t>(w.J) * 2, ld, rows,
                                       bytes);
                    } else { // two chunks of columns go out together, 128 bytes a row
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const uint32_t *f = &r[e * 8];
                            stage_w[stage_at<8>(lane, (c & 1) * 4 + e)] = make_uint4(
                                pack_bf16x2(__uint_as_float(f[0]), __uint_as_float(f[1])),
                                pack_bf16x2(__uint_as_float(f[2]), __uint_as_float(f[3])),
                                pack_bf16x2(__uint_as_float(f[4]), __uint_as_float(f[5])),
                                pack_bf16x2(__uint_as_float(f[6]), __uint_as_float(f[7])));
                        }
                        if (c & 1) {
                            __syncwarp();
                            stage_store<8>(stage_w, lane,
                                           reinterpret_cast<char *>(out) + row0 * ld + (j0 - 32) * 2, ld,
                                           rows, 2 * min(64, w.J - j0 + 32)); // J up to 2^30
                        }
                    }
                    __syncwarp();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive_cluster(tempty0 + 8 * buf); // the leader's accumulator is free
            }
            if (!ok)
                break;
            ++seg;
        }
    } else if (CONV && warp == 2) {
        pdl_wait();
        uint32_t it = 0;
        bool ok = true;
        Ring<QSTAGES> ring;
        GradWalk walk(w, pair);
        GradSegment sg;
        while (ok && walk.next(w, sg)) {
            int ib, jb;
            tile_coords(sg.tile, w.ni, w.nj, w.group_i, ib, jb);
            const int j0 = jb * kGradTile + static_cast<int>(rank) * 128;
            int r0 = sg.kb0 * kGradBR;
            for (int n = sg.kb1 - sg.kb0; n > 0; --n, ++it, r0 += kGradBR) {
                if (!mbar_wait(bar_qempty + 8 * ring.s, ring.ph ^ 1u, limit_ns)) {
                    ok = false;
                    break;
                }
                if (lane == 0) {
                    mbar_expect_tx(bar_qfull + 8 * ring.s, Cfg::kQBytes);
                    tma_load_2d(sQ + ring.s * Cfg::kQBytes, &tmQ, bar_qfull + 8 * ring.s, j0, r0);
                }
                __syncwarp();
                ring.next();
            }
        }
        if (ok)
            drain_ring(bar_qempty, it, QSTAGES, limit_ns);
    } else if (CONV && warp >= kGradConvWarp0) {
        // converters: group g (four warps) takes every GROUPS-th k-block, so the waits,
        // loads and fences of several k-blocks overlap. Two threads share a row r of the
        // k-block's [64 r][128 j] codes, every other 16-byte piece each, starting at the lane's
        // own, so that eight lanes of a load, or of a store into the swizzled bf16 tile, fill all
        // banks.
        pdl_wait();
        constexpr int kGroupThreads = 2 * kGradBR;
        static_assert(Cfg::GROUP_WARPS * 32 == kGroupThreads, "two threads a row");
        const int ct = threadIdx.x - kGradConvWarp0 * 32;
        const int group = ct / kGroupThreads;
        const int row = ct % kGradBR, half = ct / kGradBR & 1;
        const uint32_t full0 = map_peer_smem(bar_full, 0);
        float next = 0.0f;
        auto fetch = [&](int kb) {
            const int r = kb * kGradBR + row;
            next = r < w.R ? __ldg(scale + r) : 0.0f;
        };
        GradBlocks blk(w, pair, group);
        if (blk.ok)
            fetch(blk.kb);
        for (uint32_t it = group; blk.ok; it += Cfg::GROUPS) {
            const RowScale sc = row_scale(next);
            const uint32_t qs = it % QSTAGES, s = it % STAGES;
            if (!mbar_wait(bar_qfull + 8 * qs, (it / QSTAGES) & 1u, limit_ns))
                break;
            const uint8_t *src = smem + Cfg::kQOff + qs * Cfg::kQBytes + row * 128;
            uint4 raw[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                raw[k] = *reinterpret_cast<const uint4 *>(src + (((2 * k + half + lane) & 7) << 4));
            if (!mbar_wait_cluster(bar_empty + 8 * s, ((it / STAGES) & 1u) ^ 1u, limit_ns))
                break;
            uint8_t *bt = smem + Cfg::kBOff + s * Cfg::kBBytes + row * 128;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t piece = (2 * k + half + lane) & 7; // columns 16 piece .. + 15
                uint8_t *chunk = bt + (piece >> 2) * 8192;
                const uint32_t word = (piece & 3) * 2;
                const uint2 a = convert4<F8>(raw[k].x, sc), b = convert4<F8>(raw[k].y, sc);
                const uint2 c = convert4<F8>(raw[k].z, sc), d = convert4<F8>(raw[k].w, sc);
                *reinterpret_cast<uint4 *>(chunk + ((word ^ (row & 7)) << 4)) =
                    make_uint4(a.x, a.y, b.x, b.y);
                *reinterpret_cast<uint4 *>(chunk + (((word + 1) ^ (row & 7)) << 4)) =
                    make_uint4(c.x, c.y, d.x, d.y);
            }
            fence_proxy_async_smem(); // the tensor cores read what was stored
            __syncwarp();
            if (lane == 0) {
                mbar_arrive_pair(full0 + 8 * s);
                // Q's stage goes back only here: an arrival does not wait for loads in flight, and
                // right after the loads (stores of other warps before them in the queue) the next
                // bulk copy overwrote bytes not yet read, in one call of two hundred
                mbar_arrive(bar_qempty + 8 * qs);
            }
            // the scale of the group's next k-block, after the fence, which would wait for it
            blk.advance(w, Cfg::GROUPS);
            if (blk.ok)
                fetch(blk.kb);
        }
    }
    __syncwarp();
    if (warp == 1)
        tmem_relinquish_pair();
    // every MMA, commit and remote arrive is done before either CTA frees its tensor memory
    tc_fence_before();
    cluster_sync();
    tc_fence_after();
    if (warp == 1)
        tmem_dealloc_pair(tmem_base, Cfg::kTmemCols);
}

// ---------------------------------------------------------------- few rows (input gradients)
//
// For at most 128 rows i the MMAs of a 256 x 256 tile would be mostly empty, and each SM should do
// nothing but stream its share of the codes. Here a CTA takes 128 columns j and all rows i, and the
// converted operand is the MMA's first one, in tensor memory: D^T = B^T A^T with j on the 128
// lanes, i along 16 .. 128 columns. Q's tile is transposed on its way (rows r of bytes j, to lanes
// j of values r) by the byte form of ldmatrix, whose register layout is the one that the 16x256b
// store to tensor memory takes, so it is neither stored to shared memory again nor waited for by a
// proxy fence. (With 256 rows this form is the slower one: an MMA whose first operand is in tensor
// memory took 690 cycles a k-block where the pair's took 610.) The scales, which here vary along
// a register's bytes, are prepared by each converter warp, two rows a lane, and handed round by
// shuffles; a warp of its own that put them into shared memory was a chain of dependent steps
// of 670 cycles a k-block, the pace of the whole kernel.

// warps: 0 A producer, 1 MMA, 2 Q producer; 4 .. 7 epilogue; 8 .. 23 converters
constexpr int kNarrowThreads = 768;
constexpr int kNarrowConvWarp0 = 8;
constexpr int kNarrowGroups = 4; // groups of four converter warps, each on its own k-block
// r per k-block: twice the pair kernel's, as the MMA's issue (wait, instructions, commit: about
// 550 cycles with 64) was the pace
constexpr int kNarrowBR = 128;

template <int NT> struct NarrowCfg {
    static constexpr int STAGES = 4, QSTAGES = NT == 128 ? 4 : 8;
    // A converter group meets a stage of either ring again only after it has used it before: with
    // other numbers it could come to a stage of Q a whole round early, while another group still
    // waits for the load before it, and take that wait's parity for its own.
    static_assert(STAGES % kNarrowGroups == 0 && QSTAGES % kNarrowGroups == 0, "rings and groups");
    static constexpr int kABytes = NT * kNarrowBR * 2; // two swizzled tiles of 64 r
    static constexpr int kQBytes = 128 * kNarrowBR;
    static constexpr int kQOff = STAGES * kABytes;
    static constexpr int kOutOff = kQOff + QSTAGES * kQBytes; // 4 KB per epilogue warp
    static constexpr int kBarOff = kOutOff + 4 * 4096;
    // full[S], empty[S], qfull[QS], qempty[QS], tfull[2], tempty[2], tensor-memory slot
    static constexpr int kSmemBytes = kBarOff + (2 * STAGES + 2 * QSTAGES + 4) * 8 + 16 + 1024;
    static_assert(kSmemBytes <= 232448, "shared memory per CTA");
    // two accumulators of 128 lanes j x NT columns i, then the converted operand's stages
    static constexpr int kTmemCols = 512;
    static constexpr int kTmemB = 256;
    static_assert(2 * NT <= kTmemB && kTmemB + STAGES * kNarrowBR / 2 <= kTmemCols, "tensor memory");
};

// D (+)= A B^T with A in tensor memory and B in shared memory, bf16.
__device__ __forceinline__ void umma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                             uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Two 16 x 16 byte matrices (16 rows of 16 bytes each; lanes 0 .. 15 give the first one's row
// addresses, 16 .. 31 the second's), transposed: lane t gets bytes 4 (t % 4) .. + 3 of row t / 4
// in r[0] and of row t / 4 + 8 in r[1], and of the second matrix in r[2], r[3].
__device__ __forceinline__ void ldmatrix_b8_trans_x2(uint32_t addr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

// 16 lanes x 32 columns of tensor memory: of column group g (8 columns), lane t stores r[4g],
// r[4g + 1] to columns 2 (t % 4), + 1 of lane t / 4 and r[4g + 2], r[4g + 3] to those of lane
// t / 4 + 8.
__device__ __forceinline__ void tmem_st_16x256b_x4(uint32_t taddr, const uint32_t (&r)[16])
{
    asm volatile("tcgen05.st.sync.aligned.16x256b.x4.b32 [%0],"
                 " {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(
                     taddr),
                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]),
                 "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]),
                 "r"(r[14]), "r"(r[15])
                 : "memory");
}

__device__ __forceinline__ void tmem_st_wait()
{
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// Four codes (rows r .. r + 3 of one column, a byte each) to bf16(s q): convert4 with two scales'
// parts in a word. sc: the hi parts of r, r + 1 and of r + 2, r + 3, then the lo parts.
template <bool F8>
__device__ __forceinline__ void convert4_rows(uint32_t w, const uint4 sc, uint32_t &o0, uint32_t &o1)
{
    uint32_t v[2];
    code_values<F8>(w, v);
    o0 = fma_bf16x2(v[0], sc.x, mul_bf16x2(v[0], sc.z));
    o1 = fma_bf16x2(v[1], sc.y, mul_bf16x2(v[1], sc.w));
}

// Two 16-byte words, `second` and `first` by turns, from a staging buffer whose readers' rows are
// 128 bytes apart: lanes of odd rows read the second word first, so eight lanes fill all banks.
__device__ __forceinline__ void read_pair(const uint4 *p, int odd, uint4 &first, uint4 &second)
{
    const uint4 a = p[odd], b = p[odd ^ 1];
    first = odd ? b : a;
    second = odd ? a : b;
}

template <int NT, bool F8, bool SILU>
__global__ void __launch_bounds__(kNarrowThreads, 1)
    grad_narrow_kernel(const __grid_constant__ CUtensorMap tmA,
                     const __grid_constant__ CUtensorMap tmQ, const float *__restrict__ scale,
                     const GradWork w, const uint16_t *__restrict__ gate_up,
                     uint16_t *__restrict__ out, float *__restrict__ part,
                     unsigned long long limit_ns)
{
    using Cfg = NarrowCfg<NT>;
    constexpr int STAGES = Cfg::STAGES, QSTAGES = Cfg::QSTAGES;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const uint32_t sbase = smem_u32(smem);
    const uint32_t sA = sbase, sQ = sbase + Cfg::kQOff;
    const uint32_t bar_full = sbase + Cfg::kBarOff;
    const uint32_t bar_empty = bar_full + 8 * STAGES;
    const uint32_t bar_qfull = bar_empty + 8 * STAGES;
    const uint32_t bar_qempty = bar_qfull + 8 * QSTAGES;
    const uint32_t bar_tfull = bar_qempty + 8 * QSTAGES;
    const uint32_t bar_tempty = bar_tfull + 16;
    const uint32_t tslot = bar_tempty + 16;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int cta = blockIdx.x;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(bar_full + 8 * s, 1 + 4); // A's bytes, four converter warps
            mbar_init(bar_empty + 8 * s, 1);
        }
        for (int s = 0; s < QSTAGES; ++s) {
            mbar_init(bar_qfull + 8 * s, 1);
            mbar_init(bar_qempty + 8 * s, 4);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(bar_tfull + 8 * b, 1);
            mbar_init(bar_tempty + 8 * b, 4);
        }
        fence_mbar_init();
        tma_prefetch_desc(&tmA);
        tma_prefetch_desc(&tmQ);
    }
    __syncwarp();
    if (warp == 1)
        tmem_alloc(tslot, Cfg::kTmemCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base =
        *reinterpret_cast<volatile uint32_t *>(smem + (tslot - sbase));

    if (warp == 0) {
        pdl_wait();
        uint32_t it = 0;
        bool ok = true;
        Ring<STAGES> ring;
        GradWalk walk(w, cta);
        GradSegment sg;
        while (ok && walk.next(w, sg)) {
            int r0 = sg.kb0 * kNarrowBR;
            for (int n = sg.kb1 - sg.kb0; n > 0; --n, ++it, r0 += kNarrowBR) {
                if (!mbar_wait(bar_empty + 8 * ring.s, ring.ph ^ 1u, limit_ns)) {
                    ok = false;
                    break;
                }
                if (lane == 0) {
                    mbar_expect_tx(bar_full + 8 * ring.s, Cfg::kABytes);
                    const uint32_t dst = sA + ring.s * Cfg::kABytes;
                    tma_load_2d(dst, &tmA, bar_full + 8 * ring.s, r0, 0);
                    tma_load_2d(dst + Cfg::kABytes / 2, &tmA, bar_full + 8 * ring.s, r0 + 64, 0);
                }
                __syncwarp();
                ring.next();
            }
        }
        if (ok) // every stage released by the MMAs before this CTA may leave
            drain_ring(bar_empty, it, STAGES, limit_ns);
        if (lane == 0)
            pdl_launch_dependents();
    } else if (warp == 1) {
        constexpr uint32_t idesc = idesc_bf16(128, NT, false, false);
        const uint64_t da = sw128_kmajor_desc(sA);
        bool ok = true;
        Ring<STAGES> ring;
        Ring<2> acc;
        GradWalk walk(w, cta);
        GradSegment sg;
        while (ok && walk.next(w, sg)) {
            if (!mbar_wait(bar_tempty + 8 * acc.s, acc.ph ^ 1u, limit_ns))
                break;
            tc_fence_after();
            const uint32_t d = tmem_base + acc.s * NT;
            uint32_t accumulate = 0;
            for (int n = sg.kb1 - sg.kb0; n > 0; --n) {
                if (!mbar_wait(bar_full + 8 * ring.s, ring.ph, limit_ns)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                if (lane == 0) {
                    const uint64_t a0 = da + ring.s * (Cfg::kABytes / 16);
                    const uint32_t b0 = tmem_base + Cfg::kTmemB + ring.s * (kNarrowBR / 2);
#pragma unroll
                    for (int k = 0; k < kNarrowBR / 16; ++k)
                        umma_bf16_ts(d, b0 + k * 8,
                                     a0 + (k >> 2) * (Cfg::kABytes / 32) + (k & 3) * 2, idesc,
                                     k > 0 ? 1u : accumulate);
                    umma_commit(bar_empty + 8 * ring.s);
                }
                __syncwarp();
                accumulate = 1;
                ring.next();
            }
            if (ok && lane == 0)
                umma_commit(bar_tfull + 8 * acc.s);
            __syncwarp();
            acc.next();
        }
    } else if (warp == 2) {
        pdl_wait();
        uint32_t it = 0;
        bool ok = true;
        Ring<QSTAGES> ring;
        GradWalk walk(w, cta);
        GradSegment sg;
        while (ok && walk.next(w, sg)) {
            const int j0 = sg.tile * 128;
            int r0 = sg.kb0 * kNarrowBR;
            for (int n = sg.kb1 - sg.kb0; n > 0; --n, ++it, r0 += kNarrowBR) {
                if (!mbar_wait(bar_qempty + 8 * ring.s, ring.ph ^ 1u, limit_ns)) {
                    ok = false;
                    break;
                }
                if (lane == 0) {
                    mbar_expect_tx(bar_qfull + 8 * ring.s, Cfg::kQBytes);
                    tma_load_2d(sQ + ring.s * Cfg::kQBytes, &tmQ, bar_qfull + 8 * ring.s, j0, r0);
                }
                __syncwarp();
                ring.next();
            }
        }
        if (ok)
            drain_ring(bar_qempty, it, QSTAGES, limit_ns);
    } else if (warp >= 4 && warp < kNarrowConvWarp0) {
        // epilogue: the warp's lanes are 32 columns j; the rows i in chunks of 32
        pdl_wait();
        const int quarter = warp & 3;
        uint4 *stage = reinterpret_cast<uint4 *>(smem + Cfg::kOutOff) + quarter * 256;
        uint32_t *words = reinterpret_cast<uint32_t *>(stage);
        uint32_t seg = 0;
        GradWalk walk(w, cta);
        GradSegment sg;
        while (walk.next(w, sg)) {
            const uint32_t buf = seg & 1u, aph = (seg >> 1) & 1u;
            ++seg;
            if (!mbar_wait(bar_tfull + 8 * buf, aph, limit_ns))
                break;
            __syncwarp();
            tc_fence_after();
            const uint32_t tbase = tmem_base + buf * NT + (static_cast<uint32_t>(quarter * 32) << 16);
            const int jl = quarter * 32;
            const int j0 = sg.tile * 128 + jl;
            float *slot = part + (static_cast<int64_t>(cta) * 2 + sg.slot) * NT * 128 + jl + lane;
#pragma unroll 1
            for (int c = 0; c < (NT + 31) / 32; ++c) {
                const int i0 = c * 32;
                uint32_t r[32]; // of 16 rows' accumulator: columns past it, never stored
                tmem_ld_32x32b_x32(tbase + c * 32, r);
                tmem_ld_wait();
                if (c == (NT + 31) / 32 - 1) { // the accumulator is in registers
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(bar_tempty + 8 * buf);
                }
                if (sg.partial) {
#pragma unroll
                    for (int k = 0; k < 32; ++k)
                        if (i0 + k < w.I)
                            __stcg(slot + (i0 + k) * 128, __uint_as_float(r[k]));
                    continue;
                }
                if (i0 >= w.I)
                    continue;
                if constexpr (SILU) {
                    // da transposed through the staging buffer, then row by row
#pragma unroll
                    for (int k = 0; k < 32; ++k)
                        words[k * 32 + lane] = r[k];
                    __syncwarp();
#pragma unroll
                    for (int t = 0; t < 4; ++t) {
                        const int k = t * 8 + (lane >> 2), jg = lane & 3;
                        const int i = i0 + k, j = j0 + jg * 8;
                        if (i < w.I && j < w.J) {
                            const int64_t o = static_cast<int64_t>(i) * 2 * w.J + j;
                            uint4 g = ldg_nc_v4(gate_up + o), u = ldg_nc_v4(gate_up + o + w.J);
                            uint4 a, b;
                            read_pair(stage + k * 8 + jg * 2, k & 1, a, b);
                            const float da[8] = {
                                __uint_as_float(a.x), __uint_as_float(a.y), __uint_as_float(a.z),
                                __uint_as_float(a.w), __uint_as_float(b.x), __uint_as_float(b.y),
                                __uint_as_float(b.z), __uint_as_float(b.w)};
                            silu_grad8(da, g, u, g, u);
                            *reinterpret_cast<uint4 *>(out + o) = g;
                            *reinterpret_cast<uint4 *>(out + o + w.J) = u;
                        }
                    }
                } else {
                    // rows 2p and 2p + 1 of a column in one word; the readers take them apart
#pragma unroll
                    for (int p = 0; p < 16; ++p)
                        words[p * 32 + lane] =
                            pack_bf16x2(__uint_as_float(r[2 * p]), __uint_as_float(r[2 * p + 1]));
                    __syncwarp();
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        const int p = t * 8 + (lane >> 2), jg = lane & 3;
                        const int i = i0 + 2 * p, j = j0 + jg * 8;
                        uint4 a, b;
                        read_pair(stage + p * 8 + jg * 2, p & 1, a, b);
                        uint16_t *dst = out + static_cast<int64_t>(i) * w.J + j;
                        if (i < w.I && j < w.J)
                            *reinterpret_cast<uint4 *>(dst) = make_uint4(
                                __byte_perm(a.x, a.y, 0x5410), __byte_perm(a.z, a.w, 0x5410),
                                __byte_perm(b.x, b.y, 0x5410), __byte_perm(b.z, b.w, 0x5410));
                        if (i + 1 < w.I && j < w.J)
                            *reinterpret_cast<uint4 *>(dst + w.J) = make_uint4(
                                __byte_perm(a.x, a.y, 0x7632), __byte_perm(a.z, a.w, 0x7632),
                                __byte_perm(b.x, b.y, 0x7632), __byte_perm(b.z, b.w, 0x7632));
                    }
                }
                __syncwarp();
            }
        }
    } else if (warp >= kNarrowConvWarp0) {
        // converters: group g takes every kNarrowGroups-th k-block, its warp of lane quarter q
        // the columns j = 32 q .. 32 q + 31. Q's tile has rows r of 128 bytes, 16-byte pieces
        // swizzled by the row (TMA's 128-byte swizzle), so ldmatrix's eight rows fill all banks.
        pdl_wait();
        const int group = (warp - kNarrowConvWarp0) >> 2, quarter = warp & 3;
        const uint32_t src = (lane & 15) * 128 + (((2 * quarter + (lane >> 4)) ^ (lane & 7)) << 4);
        const uint32_t dst = tmem_base + Cfg::kTmemB + (static_cast<uint32_t>(quarter * 32) << 16);
        float next[4] = {0.0f, 0.0f, 0.0f, 0.0f}; // rows 4 lane .. + 3 of the next k-block
        GradBlocks blk(w, cta, group);
        auto fetch = [&]() {
            if (blk.ok) {
                const int r = blk.kb * kNarrowBR + 4 * lane;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    next[e] = r + e < w.R ? __ldg(scale + r + e) : 0.0f;
            }
        };
        fetch();
        for (uint32_t it = group; blk.ok; it += kNarrowGroups) {
            const uint32_t qs = it % QSTAGES, s = it % STAGES;
            uint4 own;
            split_scales(next[0], next[1], own.x, own.z);
            split_scales(next[2], next[3], own.y, own.w);
            blk.advance(w, kNarrowGroups);
            fetch(); // the group's next k-block's, in flight while this one is converted
            if (!mbar_wait(bar_qfull + 8 * qs, (it / QSTAGES) & 1u, limit_ns))
                break;
            __syncwarp();
            const uint32_t tile = sQ + qs * Cfg::kQBytes + src;
            bool ok = true;
#pragma unroll
            for (int half = 0; half < 2; ++half) { // 64 rows r each
                uint32_t m[4][4];
#pragma unroll
                for (int g = 0; g < 4; ++g)
                    ldmatrix_b8_trans_x2(tile + half * 8192 + g * 2048, m[g]);
                if (half == 0)
                    ok = mbar_wait(bar_empty + 8 * s, ((it / STAGES) & 1u) ^ 1u, limit_ns);
                __syncwarp();
                tc_fence_after();
                uint4 sc[4]; // rows 64 half + 16 g + 4 (lane % 4) .. + 3
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const int from = 16 * half + 4 * g + (lane & 3);
                    sc[g] = make_uint4(__shfl_sync(0xffffffffu, own.x, from),
                                       __shfl_sync(0xffffffffu, own.y, from),
                                       __shfl_sync(0xffffffffu, own.z, from),
                                       __shfl_sync(0xffffffffu, own.w, from));
                }
#pragma unroll
                for (int c = 0; c < 2; ++c) { // 16 columns j each
                    uint32_t o[16];
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        convert4_rows<F8>(m[g][2 * c], sc[g], o[4 * g], o[4 * g + 1]);
                        convert4_rows<F8>(m[g][2 * c + 1], sc[g], o[4 * g + 2], o[4 * g + 3]);
                    }
                    if (ok)
                        tmem_st_16x256b_x4(dst + s * (kNarrowBR / 2) + half * 32 +
                                               (static_cast<uint32_t>(16 * c) << 16),
                                           o);
                }
            }
            if (!ok)
                break;
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(bar_full + 8 * s);
                mbar_arrive(bar_qempty + 8 * qs); // not before the loads are done (see the pair's)
            }
        }
    }
    __syncwarp();
    if (warp == 1)
        tmem_relinquish();
    tc_fence_before(); // every MMA and load of the accumulators is done before they are freed
    __syncthreads();
    tc_fence_after();
    if (warp == 1)
        tmem_dealloc(tmem_base, Cfg::kTmemCols);
}

// The whole of Q to scaled bf16 ahead of the product, [R, J]: 16 codes a thread and step.
template <bool F8>
__global__ void __launch_bounds__(256) grad_dequant_kernel(const uint8_t *__restrict__ q,
                                                           const float *__restrict__ scale,
                                                           int64_t nvec, uint32_t row_vecs,
                                                           uint16_t *__restrict__ out)
{
    if (threadIdx.x == 0)
        pdl_launch_dependents();
    pdl_wait();
    // kFlight vectors of a thread in flight: the loads' latency, not HBM, set the pace with one
    constexpr int kFlight = 4;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * blockDim.x;
    for (int64_t v0 = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; v0 < nvec;
         v0 += kFlight * stride) {
        uint4 raw[kFlight];
        float s[kFlight];
#pragma unroll
        for (int f = 0; f < kFlight; ++f) {
            const int64_t v = v0 + f * stride;
            if (v < nvec) {
                raw[f] = ldg_nc_v4(reinterpret_cast<const uint4 *>(q) + v);
                const uint32_t row = nvec <= 0xFFFFFFFFll
                                         ? static_cast<uint32_t>(v) / row_vecs
                                         : static_cast<uint32_t>(v / row_vecs);
                s[f] = __ldg(scale + row);
            }
        }
#pragma unroll
        for (int f = 0; f < kFlight; ++f) {
            const int64_t v = v0 + f * stride;
            if (v < nvec) {
                const RowScale sc = row_scale(s[f]);
                const uint2 a = convert4<F8>(raw[f].x, sc), b = convert4<F8>(raw[f].y, sc);
                const uint2 c = convert4<F8>(raw[f].z, sc), d = convert4<F8>(raw[f].w, sc);
                uint4 *o = reinterpret_cast<uint4 *>(out) + 2 * v;
                o[0] = make_uint4(a.x, a.y, b.x, b.y);
                o[1] = make_uint4(c.x, c.y, d.x, d.y);
            }
        }
    }
}

// The pair whose range of the split holds unit v, in 32 bits where they do.
__device__ __forceinline__ int split_owner(int64_t v, int64_t U, int pairs)
{
    if (U * pairs < 0x7FFFFFFF) {
        const uint32_t u = static_cast<uint32_t>(U), n = static_cast<uint32_t>(pairs);
        const uint32_t x = static_cast<uint32_t>(v);
        uint32_t c = x * n / u;
        while (c + 1 < n && (c + 1) * u / n <= x)
            ++c;
        while (c > 0 && c * u / n > x)
            --c;
        return static_cast<int>(c);
    }
    return static_cast<int>(sk_owner_of(v, U, pairs));
}

// Adds the partial tiles of the split tiles, in the order of the pairs, and finishes them: block
// (x, y) takes 2048 values of remaining tile y.
template <bool SILU>
__global__ void __launch_bounds__(256) grad_fixup_kernel(const GradWork w,
                                                         const float *__restrict__ part,
                                                         const uint16_t *__restrict__ gate_up,
                                                         uint16_t *__restrict__ out)
{
    if (threadIdx.x == 0)
        pdl_launch_dependents();
    pdl_wait();
    const int t = blockIdx.y;
    int ib, jb;
    tile_coords(w.whole + t, w.ni, w.nj, w.group_i, ib, jb);
    const int at = (blockIdx.x * 256 + threadIdx.x) * 8;
    const int rl = at / w.tile_j, cl = at - rl * w.tile_j;
    const int row = ib * w.tile_i + rl, col = jb * w.tile_j + cl;
    if (rl >= w.tile_i || row >= w.I || col >= w.J)
        return;
    const int64_t U = static_cast<int64_t>(w.rem) * w.kblocks;
    const int64_t u0 = static_cast<int64_t>(t) * w.kblocks;
    const int p0 = split_owner(u0, U, w.rem_pairs);
    const int p1 = split_owner(u0 + w.kblocks - 1, U, w.rem_pairs);
    if (p0 == p1)
        return; // one pair had the whole tile and finished it
    float f[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        f[i] = 0.0f;
    // Only the first pair can have begun in an earlier tile (its slot 1); the others' ranges begin
    // here. Four parts are in flight, added in order.
    const float4 *src = reinterpret_cast<const float4 *>(
        part + static_cast<int64_t>(p0) * 2 * w.tile_i * w.tile_j + at);
    const int slot_words = w.tile_i * w.tile_j / 4;
    const bool second = static_cast<int64_t>(p0) * U / w.rem_pairs < u0;
    for (int p = p0; p <= p1; p += 4) {
        float4 v[4][2];
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (p + e <= p1) {
                const float4 *at = src + static_cast<int64_t>(p + e - p0) * 2 * slot_words +
                                   (second && p + e == p0 ? slot_words : 0);
                v[e][0] = __ldcs(at);
                v[e][1] = __ldcs(at + 1);
            }
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (p + e <= p1) {
                const float4 a = v[e][0], b = v[e][1];
                f[0] += a.x; f[1] += a.y; f[2] += a.z; f[3] += a.w;
                f[4] += b.x; f[5] += b.y; f[6] += b.z; f[7] += b.w;
            }
    }
    if constexpr (SILU) {
        const int64_t o = static_cast<int64_t>(row) * 2 * w.J + col;
        uint4 g = *reinterpret_cast<const uint4 *>(gate_up + o);
        uint4 u = *reinterpret_cast<const uint4 *>(gate_up + o + w.J);
        silu_grad8(f, g, u, g, u);
        *reinterpret_cast<uint4 *>(out + o) = g;
        *reinterpret_cast<uint4 *>(out + o + w.J) = u;
    } else {
        *reinterpret_cast<uint4 *>(out + static_cast<int64_t>(row) * w.J + col) =
            make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                       pack_bf16x2(f[6], f[7]));
    }
}

} // namespace w8a8
