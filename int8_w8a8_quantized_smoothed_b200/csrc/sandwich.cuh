// The row operators at a block boundary: the norm after a block (optional), its gate, the scaled
// residual add, the norm before the next block and its per-token quantization, in one pass over
// the row; and the backward pass of that chain.
//
//   n = (y r1) gamma_post           r1 = 1 / sqrt(mean(y^2) + eps_post)    (n = y without it)
//   h = bf16(res_scale residual + gate n)
//   z = (h r2) gamma_pre            r2 = 1 / sqrt(mean(h^2) + eps_pre)
//   s, q = per-token codes of z
#pragma once

#include "rowquant.cuh"

namespace w8a8 {

enum GateKind { kGateNone = 0, kGateToken = 1, kGateChannel = 2, kGateFull = 3 };

// Eight binary32 values of vector vi.
__device__ __forceinline__ void load8_f32(const float *__restrict__ p, int vi, float (&f)[8])
{
    const float4 a = __ldg(reinterpret_cast<const float4 *>(p) + 2 * vi);
    const float4 b = __ldg(reinterpret_cast<const float4 *>(p) + 2 * vi + 1);
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}

// 1 / sqrt(sum / K + eps), the mean in binary64 and rounded once, as every RMSNorm here.
__device__ __forceinline__ float rstd_of(double sum, int K, float eps)
{
    const double mean = (K & (K - 1)) == 0 ? __dmul_rn(sum, 1.0 / static_cast<double>(K))
                                           : __ddiv_rn(sum, static_cast<double>(K));
    return __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(__double2float_rn(mean), eps)));
}

template <int NCH> __device__ __forceinline__ double square_sum(const float (&v)[NCH][8])
{
    double ss = 0.0;
#pragma unroll
    for (int c = 0; c < NCH; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) // each square of a bf16 value is exact in binary32
            ss = __dadd_rn(ss, static_cast<double>(__fmul_rn(v[c][i], v[c][i])));
    return ss;
}

// One CTA per row, the row in registers (NCH vectors of 8 values per thread). GATE: kGateToken
// also serves no gate (factor 1, exact).
template <int NCH, bool POST, int GATE, bool F8>
__global__ void __launch_bounds__(NCH <= 2 ? 256 : 1024, NCH <= 2 ? 3 : 1)
    sandwich_quant_kernel(const uint16_t *__restrict__ y, const uint16_t *res,
                          const float *__restrict__ gamma_post, const void *__restrict__ gate,
                          float res_scale, const float *__restrict__ gamma_pre, float eps_post,
                          float eps_pre, int K, int M, uint16_t *h_out, int8_t *__restrict__ q,
                          float *__restrict__ s_tok)
{
    // the buffers take turns, so each is rewritten only after another one's barrier
    __shared__ double sh_y[32], sh_h[32];
    __shared__ float sh_max[32];
    if (threadIdx.x == 0)
        pdl_launch_dependents();
    pdl_wait(); // every input may come from the previous kernel
    const int nvec = K >> 3;
    for (int64_t row = blockIdx.x; row < M; row += gridDim.x) {
        uint4 ry[NCH], rr[NCH], rg[GATE == kGateFull ? NCH : 1];
        load_row<NCH>(reinterpret_cast<const uint4 *>(y + row * K), nvec, ry);
        const uint4 *resv = reinterpret_cast<const uint4 *>(res + row * K);
#pragma unroll
        for (int c = 0; c < NCH; ++c) { // plain loads: h_out may be the residual
            const int vi = c * blockDim.x + threadIdx.x;
            rr[c] = vi < nvec ? resv[vi] : make_uint4(0u, 0u, 0u, 0u);
        }
        if constexpr (GATE == kGateFull)
            load_row<NCH>(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(gate) + row * K),
                          nvec, rg);
        float gt = 1.0f;
        if constexpr (GATE == kGateToken)
            gt = gate ? __ldg(static_cast<const float *>(gate) + row) : 1.0f;
        float v[NCH][8];
#pragma unroll
        for (int c = 0; c < NCH; ++c)
            unpack8(ry[c], v[c]);
        float r1 = 1.0f;
        if constexpr (POST)
            r1 = rstd_of(block_sum(square_sum<NCH>(v), sh_y), K, eps_post);
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
            const int vi = c * blockDim.x + threadIdx.x;
            if (vi < nvec) {
                float r[8], w[8];
                unpack8(rr[c], r);
                if constexpr (POST) {
                    load8_f32(gamma_post, vi, w);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        v[c][i] = __fmul_rn(__fmul_rn(v[c][i], r1), w[i]);
                }
                if constexpr (GATE == kGateFull)
                    unpack8(rg[c], w);
                else if constexpr (GATE == kGateChannel)
                    load8_f32(static_cast<const float *>(gate), vi, w);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float b = __fmul_rn(GATE == kGateToken ? gt : w[i], v[c][i]);
                    v[c][i] = __fadd_rn(__fmul_rn(res_scale, r[i]), b);
                }
                uint4 hb;
                hb.x = pack_bf16x2(v[c][0], v[c][1]);
                hb.y = pack_bf16x2(v[c][2], v[c][3]);
                hb.z = pack_bf16x2(v[c][4], v[c][5]);
                hb.w = pack_bf16x2(v[c][6], v[c][7]);
                reinterpret_cast<uint4 *>(h_out + row * K)[vi] = hb;
                unpack8(hb, v[c]);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    v[c][i] = 0.0f;
            }
        }
        const float r2 = rstd_of(block_sum(square_sum<NCH>(v), sh_h), K, eps_pre);
        float amax = 0.0f;
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
            const int vi = c * blockDim.x + threadIdx.x;
            if (vi < nvec) {
                float w[8];
                load8_f32(gamma_pre, vi, w);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    v[c][i] = __fmul_rn(__fmul_rn(v[c][i], r2), w[i]);
                    amax = fmaxf(amax, fabsf(v[c][i]));
                }
            }
        }
        amax = block_max(amax, sh_max);
        quantize_and_store<NCH, F8>(v, amax, 0, nvec, q + row * K, s_tok + row);
    }
}

// Many rows of up to 8192 values. What bounded the kernel above was the chain of steps of one row
// (three reductions over a whole CTA, each with a barrier, and between them square roots and
// quotients): three CTAs an SM, each at one row, took 90 us for 8192 x 4096 with an elementwise
// gate, whether their loads were ahead or not. Here a row belongs to a team of one, two or four
// warps, 64 values a lane, so that up to sixteen rows of an SM are at different steps and a row's
// reductions cost few instructions. A team's row comes by bulk copies into its place in shared
// memory, given back as soon as h is formed; the gains are kept in shared memory for all teams.
struct SandwichRows {
    const uint16_t *y, *res;
    const float *gamma_post, *gamma_pre;
    const void *gate;
    uint16_t *h;
    int8_t *q;
    float *s_tok;
    float res_scale, eps_post, eps_pre;
    int K, M, teams;
    unsigned long long limit_ns;
};

constexpr int kTeamVecs = 8; // vectors of 8 values a lane
constexpr int kRowsMaxK = 4 * 32 * kTeamVecs * 8;

// Shared memory: the gains as two planes of half vectors each (so that lanes' reads of 16 bytes
// are consecutive), each team's row, its barrier and its sums.
__host__ __device__ constexpr int rows_smem_bytes(int K, int arrays, int gains, int teams)
{
    return K * 4 * gains + teams * (2 * K * arrays + 8 + 2 * 4 * 8 + 4 * 4);
}

template <int W> __device__ __forceinline__ void team_sync(int team)
{
    if constexpr (W == 1)
        __syncwarp();
    else
        named_bar_sync(1 + team, 32 * W);
}

// Running sum of squares of values that are exact in bf16 (so are their squares in binary32): a
// binary32 sum and the sum of its additions' exact errors, two lanes at a time, with a fraction of
// the time of binary64 conversions and additions. With u = 2^-24 and at most 32 values in a sum S,
// an addition's error is at most u S and the sum of i of them at most i u S, so rounding those sums
// costs at most (1 + .. + 32) u^2 S < 2^-38 S (2^-46 in practice). Where the binary32 sum
// overflows, value() is infinite or NaN, and the row is summed again in binary64.
struct SquareSum {
    float2 hi = make_float2(0.0f, 0.0f), lo = make_float2(0.0f, 0.0f);
    __device__ __forceinline__ void add(float2 a)
    {
        const float2 m1 = make_float2(-1.0f, -1.0f);
        const float2 p = mul2(a, a);
        const float2 t = add2(hi, p);
        const float2 z = fma2(hi, m1, t); // t - hi
        lo = add2(lo, add2(fma2(fma2(z, m1, t), m1, hi), fma2(z, m1, p))); // (hi - (t - z)) + (p - z)
        hi = t;
    }
    __device__ __forceinline__ double value() const
    {
        return (static_cast<double>(hi.x) + static_cast<double>(hi.y)) +
               (static_cast<double>(lo.x) + static_cast<double>(lo.y));
    }
};

template <int W>
__device__ __forceinline__ double team_sum(double v, double *sh, int team, int warp_in_team, int lane)
{
    v = warp_sum(v);
    if constexpr (W > 1) {
        if (lane == 0)
            sh[warp_in_team] = v;
        team_sync<W>(team);
        v = sh[0];
#pragma unroll
        for (int w = 1; w < W; ++w)
            v = __dadd_rn(v, sh[w]);
    }
    return v;
}

// The sum of squares of a team's row again, in binary64 as the kernel above has it; value(c, v)
// gives the thread's vector c.
template <int W, typename Value>
__device__ __forceinline__ double team_resum(Value value, int nvec, int tl, double *sh, int team,
                                             int warp_in_team, int lane)
{
    double t = 0.0;
#pragma unroll 1
    for (int c = 0; c < kTeamVecs; ++c)
        if (c * 32 * W + tl < nvec) {
            float v[1][8];
            value(c, v[0]);
            t = __dadd_rn(t, square_sum<1>(v));
        }
    team_sync<W>(team); // all have read the first sums
    return team_sum<W>(t, sh, team, warp_in_team, lane);
}

template <int W, bool POST, int GATE, bool F8>
__global__ void __launch_bounds__(512, 1) sandwich_rows_kernel(const SandwichRows a)
{
    extern __shared__ __align__(16) uint8_t rows_smem[];
    constexpr int kArrays = GATE == kGateFull ? 3 : 2;
    constexpr int kGains = 1 + (POST ? 1 : 0) + (GATE == kGateChannel ? 1 : 0);
    const int nvec = a.K >> 3;
    const int lane = threadIdx.x & 31;
    const int team = threadIdx.x / (32 * W), tl = threadIdx.x % (32 * W), wt = tl >> 5;
    float4 *gains = reinterpret_cast<float4 *>(rows_smem); // [gain][half][nvec]
    uint4 *rows = reinterpret_cast<uint4 *>(gains + kGains * 2 * nvec);
    uint64_t *bars = reinterpret_cast<uint64_t *>(rows + a.teams * kArrays * nvec);
    double *sums = reinterpret_cast<double *>(bars + a.teams) + team * 8; // two of four
    float *maxes = reinterpret_cast<float *>(reinterpret_cast<double *>(bars + a.teams) + a.teams * 8) +
                   team * 4;
    const uint32_t bar = smem_u32(bars + team);
    if (tl == 0) {
        mbar_init(bar, 1);
        fence_mbar_init();
    }
    if (threadIdx.x == 0)
        pdl_launch_dependents();
    __syncthreads();
    pdl_wait(); // every input may come from the previous kernel
    const int64_t stride = static_cast<int64_t>(gridDim.x) * a.teams;
    const int64_t first = blockIdx.x + static_cast<int64_t>(team) * gridDim.x;
    const uint4 *mine = rows + team * kArrays * nvec;
    auto fetch = [&](int64_t row) { // one thread of the team
        const uint32_t bytes = static_cast<uint32_t>(nvec) * 16, dst = smem_u32(mine);
        const int64_t at = row * nvec;
        mbar_expect_tx(bar, bytes * kArrays);
        bulk_load_g2s(dst, reinterpret_cast<const uint4 *>(a.y) + at, bytes, bar);
        bulk_load_g2s(dst + bytes, reinterpret_cast<const uint4 *>(a.res) + at, bytes, bar);
        if constexpr (GATE == kGateFull)
            bulk_load_g2s(dst + 2 * bytes, static_cast<const uint4 *>(a.gate) + at, bytes, bar);
    };
    if (tl == 0 && first < a.M)
        fetch(first);
    auto keep = [&](const float *src, int gain) {
        for (int i = threadIdx.x; i < 2 * nvec; i += blockDim.x)
            gains[(gain * 2 + (i & 1)) * nvec + (i >> 1)] =
                __ldg(reinterpret_cast<const float4 *>(src) + i);
    };
    keep(a.gamma_pre, 0);
    if constexpr (POST)
        keep(a.gamma_post, 1);
    if constexpr (GATE == kGateChannel)
        keep(static_cast<const float *>(a.gate), kGains - 1);
    __syncthreads();
    auto gain8 = [&](int gain, int vi, float (&g)[8]) {
        const float4 x = gains[gain * 2 * nvec + vi], y = gains[(gain * 2 + 1) * nvec + vi];
        g[0] = x.x; g[1] = x.y; g[2] = x.z; g[3] = x.w;
        g[4] = y.x; g[5] = y.y; g[6] = y.z; g[7] = y.w;
    };
    uint32_t ph = 0;
    for (int64_t row = first; row < a.M; row += stride, ph ^= 1u) {
        // a wait that ran out has raised the status word; the row is then worked on as it is
        (void)mbar_wait(bar, ph, a.limit_ns);
        __syncwarp();
        float v[kTeamVecs][8];
        float r1 = 1.0f;
        if constexpr (POST) {
            SquareSum ss;
#pragma unroll
            for (int c = 0; c < kTeamVecs; ++c) {
                const int vi = c * 32 * W + tl;
                if (vi < nvec) {
                    unpack8(mine[vi], v[c]);
#pragma unroll
                    for (int i = 0; i < 8; i += 2)
                        ss.add(make_float2(v[c][i], v[c][i + 1]));
                }
            }
            auto y = [&](int c, float (&x)[8]) { unpack8(mine[c * 32 * W + tl], x); };
            r1 = rstd_of(team_sum<W>(ss.value(), sums, team, wt, lane), a.K, a.eps_post);
            if (!(r1 > 0.0f)) // the sum has overflowed, for the whole team alike
                r1 = rstd_of(team_resum<W>(y, nvec, tl, sums, team, wt, lane), a.K, a.eps_post);
        }
        float gt = 1.0f;
        if constexpr (GATE == kGateToken)
            gt = a.gate ? __ldg(static_cast<const float *>(a.gate) + row) : 1.0f;
        SquareSum ss;
#pragma unroll
        for (int c = 0; c < kTeamVecs; ++c) {
            const int vi = c * 32 * W + tl;
            if (vi < nvec) {
                float r[8], g[8];
                unpack8(mine[vi], v[c]);
                uint32_t w[4];
                if constexpr (POST) {
                    gain8(1, vi, g);
#pragma unroll
                    for (int i = 0; i < 8; i += 2) {
                        const float2 x = mul2(mul2(make_float2(v[c][i], v[c][i + 1]), splat2(r1)),
                                              make_float2(g[i], g[i + 1]));
                        v[c][i] = x.x;
                        v[c][i + 1] = x.y;
                    }
                }
                if constexpr (GATE == kGateFull)
                    unpack8(mine[2 * nvec + vi], g);
                else if constexpr (GATE == kGateChannel)
                    gain8(kGains - 1, vi, g);
                unpack8(mine[nvec + vi], r);
#pragma unroll
                for (int i = 0; i < 8; i += 2) {
                    float2 x = mul2(GATE == kGateToken ? splat2(gt) : make_float2(g[i], g[i + 1]),
                                    make_float2(v[c][i], v[c][i + 1]));
                    x = add2(mul2(splat2(a.res_scale), make_float2(r[i], r[i + 1])), x);
                    w[i >> 1] = pack_bf16x2(x.x, x.y);
                }
                const uint4 hb = make_uint4(w[0], w[1], w[2], w[3]);
                reinterpret_cast<uint4 *>(a.h)[row * nvec + vi] = hb;
                unpack8(hb, v[c]);
#pragma unroll
                for (int i = 0; i < 8; i += 2)
                    ss.add(make_float2(v[c][i], v[c][i + 1]));
            }
        }
        const double hh = team_sum<W>(ss.value(), sums + 4, team, wt, lane);
        // the whole team has used what it read of this row: its place is free
        if (tl == 0 && row + stride < a.M)
            fetch(row + stride);
        float r2 = rstd_of(hh, a.K, a.eps_pre);
        if (!(r2 > 0.0f)) { // as r1; h comes from where this thread has just stored it
            auto h = [&](int c, float (&x)[8]) {
                unpack8(reinterpret_cast<const uint4 *>(a.h)[row * nvec + c * 32 * W + tl], x);
            };
            r2 = rstd_of(team_resum<W>(h, nvec, tl, sums + 4, team, wt, lane), a.K, a.eps_pre);
        }
        float amax = 0.0f;
#pragma unroll
        for (int c = 0; c < kTeamVecs; ++c) {
            const int vi = c * 32 * W + tl;
            if (vi < nvec) {
                float g[8];
                gain8(0, vi, g);
#pragma unroll
                for (int i = 0; i < 8; i += 2) {
                    const float2 x = mul2(mul2(make_float2(v[c][i], v[c][i + 1]), splat2(r2)),
                                          make_float2(g[i], g[i + 1]));
                    v[c][i] = x.x;
                    v[c][i + 1] = x.y;
                    amax = fmaxf(amax, fmaxf(fabsf(x.x), fabsf(x.y)));
                }
            }
        }
        amax = warp_max(amax);
        if constexpr (W > 1) {
            if (lane == 0)
                maxes[wt] = amax;
            team_sync<W>(team);
#pragma unroll
            for (int w = 0; w < W; ++w)
                amax = fmaxf(amax, maxes[w]);
        }
        const float s = __fdiv_rn(amax, F8 ? 448.0f : 127.0f);
        if (tl == 0)
            a.s_tok[row] = s;
        const bool by_product = s >= kProductScale;
        const float rs = by_product ? __frcp_rn(s) : 0.0f;
#pragma unroll
        for (int c = 0; c < kTeamVecs; ++c) {
            const int vi = c * 32 * W + tl;
            if (vi < nvec)
                reinterpret_cast<uint2 *>(a.q)[row * nvec + vi] =
                    quantize_vector<F8>(v[c], amax, s, rs, by_product);
        }
    }
}

// ------------------------------------------------------------------------------ backward
//
// With w = dz gamma_pre and p = gamma_post y (p = y without the first norm), per row:
//   D = dh + r2 w - h r2^3 A / K,                A = sum w h              (gradient of h)
//   dresidual = res_scale D,  dgate = D n
//   dy = r1 gate gamma_post D - y r1^3 S / K,    S = sum gate p D         (dy = gate D without it)
// S needs D, whose own sums are linear in it: sum p D = sum p dh + r2 sum p w - r2^3 A / K sum p h
// (p with the gate where it varies along the row), so one round of row sums gives all of them.
// dgamma_pre = sum_m dz h r2 and T = sum_m [gate] D y r1 are summed over the rows a CTA takes in
// registers (each thread keeps its eight columns for every row); sandwich_part_kernel adds the
// CTAs' sums in a fixed order.
//
// A CTA covers up to 8192 columns (1024 threads, one vector of 8 each); wider rows take a cluster
// of CTAs whose row sums meet through distributed shared memory, one barrier a row either way. The
// rows come by bulk copies into a ring of two or three in shared memory, so that the next rows'
// bytes are on their way without a register held for them, and are read twice from there, before
// and after the row's sums are known. (With the next row in registers, 512 threads and two CTAs a
// row of 8192, 8192 x 8192 took 470 us, 7900 cycles a row.)

constexpr int kBackMaxThreads = 1024;
constexpr int kBackSums = 6; // h h, w h, y y, p dh, p w, p h
struct SandwichBack {
    const uint16_t *dz, *dh, *y, *h;
    const float *gamma_post, *gamma_pre;
    const void *gate;
    uint16_t *dy, *dres, *dgate_full;
    float *dgate_tok;
    float *part; // [clusters][2][K]: dgamma_pre, T
    float res_scale, eps_post, eps_pre;
    int K, M, stages;
    unsigned long long limit_ns;
};

// Shared memory of a CTA with `cols` columns: the ring, the warps' sums by row parity, the ring's
// barriers.
__host__ __device__ constexpr int back_smem_bytes(int cols, int arrays, int stages)
{
    return 2 * cols * arrays * stages + 2 * kBackSums * 32 * 4 + stages * 8;
}

// Sums of eight values over the warp: of value j, all lanes with (lane >> 2) == j hold it (by
// exchanging halves of the values first, 9 shuffles instead of 5 for each).
__device__ __forceinline__ float warp_sum8(const float (&v)[8], int lane)
{
    float a[4], b[2];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float keep = (lane & 16) ? v[4 + i] : v[i], send = (lane & 16) ? v[i] : v[4 + i];
        a[i] = keep + __shfl_xor_sync(0xffffffffu, send, 16);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float keep = (lane & 8) ? a[2 + i] : a[i], send = (lane & 8) ? a[i] : a[2 + i];
        b[i] = keep + __shfl_xor_sync(0xffffffffu, send, 8);
    }
    const float keep = (lane & 4) ? b[1] : b[0], send = (lane & 4) ? b[0] : b[1];
    float c = keep + __shfl_xor_sync(0xffffffffu, send, 4);
    c += __shfl_xor_sync(0xffffffffu, c, 2);
    return c + __shfl_xor_sync(0xffffffffu, c, 1);
}

__device__ __forceinline__ float ld_dsmem_f32(uint32_t addr)
{
    float r;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(r) : "r"(addr) : "memory");
    return r;
}

// Columns 2e and 2e + 1 of a half vector's words.
__device__ __forceinline__ float2 bf16_pair(const uint2 v, int e)
{
    const uint32_t w = e ? v.y : v.x;
    return make_float2(bf16_lo(w), bf16_hi(w));
}

template <bool POST, int GATE, bool CLUSTER>
__global__ void __launch_bounds__(kBackMaxThreads, 1) sandwich_back_kernel(const SandwichBack a)
{
    extern __shared__ __align__(16) uint8_t back_smem[];
    const int K = a.K;
    const int nvec = K >> 3;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int nw = blockDim.x >> 5;
    uint32_t rank = 0, csize = 1;
    if constexpr (CLUSTER) {
        rank = cluster_ctarank();
        asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(csize));
    }
    const int cl = blockIdx.x / csize, ncl = gridDim.x / csize;
    const int per = (nvec + csize - 1) / csize; // vectors of a CTA; the last one may have fewer
    const int v0 = rank * per;
    const int have = min(per, nvec - v0);
    const int vi = v0 + threadIdx.x;
    const bool on = static_cast<int>(threadIdx.x) < have;
    const bool has_dh = a.dh != nullptr;
    const int arrays = 3 + (has_dh ? 1 : 0) + (GATE == kGateFull ? 1 : 0);
    const int stage_vecs = arrays * per;
    uint4 *ring = reinterpret_cast<uint4 *>(back_smem);
    float(*sh)[kBackSums][32] =
        reinterpret_cast<float(*)[kBackSums][32]>(ring + a.stages * stage_vecs);
    const uint32_t bars = smem_u32(sh + 2);

    if (threadIdx.x == 0) {
        pdl_launch_dependents();
        for (int s = 0; s < a.stages; ++s)
            mbar_init(bars + 8 * s, 1);
        fence_mbar_init();
    }
    __syncthreads();
    pdl_wait();
    auto fetch = [&](int64_t row, int s) { // one thread
        const uint32_t bytes = static_cast<uint32_t>(have) * 16;
        const uint32_t bar = bars + 8 * s;
        const int64_t at = row * nvec + v0;
        uint32_t dst = smem_u32(ring + s * stage_vecs);
        mbar_expect_tx(bar, bytes * arrays);
        auto copy = [&](const void *p) {
            bulk_load_g2s(dst, static_cast<const uint4 *>(p) + at, bytes, bar);
            dst += per * 16;
        };
        copy(a.dz);
        copy(a.y);
        copy(a.h);
        if (has_dh)
            copy(a.dh);
        if constexpr (GATE == kGateFull)
            copy(a.gate);
    };
    if (threadIdx.x == 0)
        for (int s = 0; s < a.stages; ++s)
            if (cl + static_cast<int64_t>(s) * ncl < a.M)
                fetch(cl + static_cast<int64_t>(s) * ncl, s);
    // gamma_smoothed, and gamma_post with the channel gate where there is one
    float gp[8], gq[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        gp[i] = gq[i] = 1.0f;
    if (on) {
        load8_f32(a.gamma_pre, vi, gp);
        if constexpr (POST)
            load8_f32(a.gamma_post, vi, gq);
        if constexpr (GATE == kGateChannel) {
            float g[8];
            load8_f32(static_cast<const float *>(a.gate), vi, g);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                gq[i] *= g[i];
        }
    }
    constexpr bool kSums = POST || GATE == kGateToken; // sums of p wanted
    constexpr bool kT = POST || GATE == kGateChannel;
    float acc_pre[8], acc_t[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        acc_pre[i] = acc_t[i] = 0.0f;
    const float invK = 1.0f / static_cast<float>(K);
    int s = 0;
    uint32_t ph = 0, parity = 0;
    for (int64_t row = cl; row < a.M; row += ncl, parity ^= 1u) {
        // a wait that ran out has raised the status word; the row is then worked on as it is
        (void)mbar_wait(bars + 8 * s, ph, a.limit_ns);
        const uint2 *st = reinterpret_cast<const uint2 *>(ring + s * stage_vecs + threadIdx.x);
        const int next = 2 * per; // from one array to the next
        float sum[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            sum[j] = 0.0f;
        if (on) {
#pragma unroll
            for (int hv = 0; hv < 2; ++hv) { // four columns at a time
                const uint2 dz = st[hv], y = st[next + hv], h = st[2 * next + hv];
                const uint2 dh = has_dh ? st[3 * next + hv] : make_uint2(0u, 0u);
                uint2 g = make_uint2(0u, 0u);
                if constexpr (GATE == kGateFull)
                    g = st[(arrays - 1) * next + hv];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float2 dz2 = bf16_pair(dz, e), y2 = bf16_pair(y, e), h2 = bf16_pair(h, e);
                    const float2 dh2 = bf16_pair(dh, e), g2 = bf16_pair(g, e);
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const int i = 4 * hv + 2 * e + c;
                        const float hh = c ? h2.y : h2.x, yy = c ? y2.y : y2.x;
                        const float w = (c ? dz2.y : dz2.x) * gp[i];
                        sum[0] = fmaf(hh, hh, sum[0]);
                        sum[1] = fmaf(w, hh, sum[1]);
                        if constexpr (POST)
                            sum[2] = fmaf(yy, yy, sum[2]);
                        if constexpr (kSums) {
                            float p = gq[i] * yy;
                            if constexpr (GATE == kGateFull)
                                p *= c ? g2.y : g2.x;
                            sum[3] = fmaf(p, c ? dh2.y : dh2.x, sum[3]);
                            sum[4] = fmaf(p, w, sum[4]);
                            sum[5] = fmaf(p, hh, sum[5]);
                        }
                    }
                }
            }
        }
        float(&buf)[kBackSums][32] = sh[parity];
        const float mine = warp_sum8(sum, lane);
        if ((lane & 3) == 0 && (lane >> 2) < kBackSums)
            buf[lane >> 2][warp] = mine;
        if constexpr (CLUSTER)
            cluster_sync();
        else
            __syncthreads();
        // every thread has used what it read of the row before this one: its stage is free
        if (threadIdx.x == 0 && row != cl) {
            const int64_t ahead = row + static_cast<int64_t>(a.stages - 1) * ncl;
            if (ahead < a.M)
                fetch(ahead, s == 0 ? a.stages - 1 : s - 1);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
            sum[j] = 0.0f;
        if (lane < nw) {
#pragma unroll
            for (int j = 0; j < kBackSums; ++j) {
                if constexpr (CLUSTER) {
                    for (uint32_t r = 0; r < csize; ++r)
                        sum[j] += ld_dsmem_f32(map_peer_smem(smem_u32(&buf[j][lane]), r));
                } else {
                    sum[j] = buf[j][lane];
                }
            }
        }
        const float all = warp_sum8(sum, lane);
        float t[kBackSums];
#pragma unroll
        for (int j = 0; j < kBackSums; ++j)
            t[j] = __shfl_sync(0xffffffffu, all, 4 * j);
        float gt = 1.0f;
        if constexpr (GATE == kGateToken)
            gt = a.gate ? __ldg(static_cast<const float *>(a.gate) + row) : 1.0f;
        const float r2 = 1.0f / sqrtf(fmaf(t[0], invK, a.eps_pre));
        // r2^3 A / K and r1^3 S / K without one factor, which goes to h and to y: 1 / rms may be large
        // enough (from 2^43 on) for its cube to overflow
        const float c2 = t[1] * invK * r2 * r2;
        const float r1 = POST ? 1.0f / sqrtf(fmaf(t[2], invK, a.eps_post)) : 1.0f;
        const float sp = fmaf(-c2, r2 * t[5], fmaf(r2, t[4], t[3])); // sum p D
        const float c1 = gt * sp * invK * r1 * r1;
        if constexpr (GATE == kGateToken)
            if (a.dgate_tok && threadIdx.x == 0 && rank == 0)
                a.dgate_tok[row] = r1 * sp;
        if (on) {
            uint32_t ores[4], ody[4], ogate[4];
#pragma unroll
            for (int hv = 0; hv < 2; ++hv) {
                const uint2 dz = st[hv], y = st[next + hv], h = st[2 * next + hv];
                const uint2 dh = has_dh ? st[3 * next + hv] : make_uint2(0u, 0u);
                uint2 g = make_uint2(0u, 0u);
                if constexpr (GATE == kGateFull)
                    g = st[(arrays - 1) * next + hv];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float2 dz2 = bf16_pair(dz, e), y2 = bf16_pair(y, e), h2 = bf16_pair(h, e);
                    const float2 dh2 = bf16_pair(dh, e), g2 = bf16_pair(g, e);
                    float od[2], oy[2], og[2];
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const int i = 4 * hv + 2 * e + c;
                        const float x2 = (c ? h2.y : h2.x) * r2, x1 = (c ? y2.y : y2.x) * r1;
                        const float zz = c ? dz2.y : dz2.x;
                        const float D = fmaf(r2, zz * gp[i], fmaf(-c2, x2, c ? dh2.y : dh2.x));
                        acc_pre[i] = fmaf(zz, x2, acc_pre[i]);
                        od[c] = D * a.res_scale;
                        // a gate that varies along the row is in gq (per channel) or in g
                        const float gd = GATE == kGateToken ? gt * D
                                         : GATE == kGateFull ? (c ? g2.y : g2.x) * D : D;
                        if constexpr (kT)
                            acc_t[i] = fmaf(gd, x1, acc_t[i]);
                        if constexpr (GATE == kGateFull)
                            og[c] = D * (x1 * gq[i]);
                        oy[c] = POST ? fmaf(r1 * gq[i], gd, -c1 * x1) : gq[i] * gd;
                    }
                    ores[2 * hv + e] = pack_bf16x2(od[0], od[1]);
                    ody[2 * hv + e] = pack_bf16x2(oy[0], oy[1]);
                    if constexpr (GATE == kGateFull)
                        ogate[2 * hv + e] = pack_bf16x2(og[0], og[1]);
                }
            }
            const int64_t off = row * nvec + vi;
            reinterpret_cast<uint4 *>(a.dres)[off] = make_uint4(ores[0], ores[1], ores[2], ores[3]);
            reinterpret_cast<uint4 *>(a.dy)[off] = make_uint4(ody[0], ody[1], ody[2], ody[3]);
            if constexpr (GATE == kGateFull)
                reinterpret_cast<uint4 *>(a.dgate_full)[off] =
                    make_uint4(ogate[0], ogate[1], ogate[2], ogate[3]);
        }
        if (++s == a.stages) {
            s = 0;
            ph ^= 1u;
        }
    }
    if (on) {
        float4 *p0 = reinterpret_cast<float4 *>(a.part + (static_cast<int64_t>(cl) * 2) * K) + 2 * vi;
        p0[0] = make_float4(acc_pre[0], acc_pre[1], acc_pre[2], acc_pre[3]);
        p0[1] = make_float4(acc_pre[4], acc_pre[5], acc_pre[6], acc_pre[7]);
        if constexpr (kT) {
            float4 *p1 = p0 + K / 4;
            p1[0] = make_float4(acc_t[0], acc_t[1], acc_t[2], acc_t[3]);
            p1[1] = make_float4(acc_t[4], acc_t[5], acc_t[6], acc_t[7]);
        }
    }
    if constexpr (CLUSTER)
        cluster_sync(); // a peer may still read this CTA's sums
}

// Column sums of the CTAs' parts, in a fixed order: dgamma_pre from array 0; T from array 1 gives
// dgamma_post = [gate_ch] T and dgate_ch = [gamma_post] T. A block takes 32 columns, its warps the
// parts in turn, four loads of each in flight: 8 warps (which find room beside the kernel before),
// or 32 for many parts.
__global__ void __launch_bounds__(1024) sandwich_part_kernel(const float *__restrict__ part,
                                                             int nparts, int K,
                                                             const float *__restrict__ gamma_post,
                                                             const float *__restrict__ gate_ch,
                                                             float *__restrict__ dgamma_pre,
                                                             float *__restrict__ dgamma_post,
                                                             float *__restrict__ dgate_ch)
{
    __shared__ float sh[32][32];
    if (threadIdx.x == 0)
        pdl_launch_dependents();
    pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
    const int col = blockIdx.x * 32 + lane;
    const int which = blockIdx.y;
    const float *src = part + static_cast<int64_t>(which) * K + col;
    float t = 0.0f;
    if (col < K)
        for (int p = warp; p < nparts; p += 4 * nw) {
            float v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                v[e] = p + nw * e < nparts ? __ldcs(src + static_cast<int64_t>(p + nw * e) * 2 * K)
                                           : 0.0f;
            t += (v[0] + v[1]) + (v[2] + v[3]);
        }
    sh[warp][lane] = t;
    __syncthreads();
    if (warp == 0 && col < K) {
        t = 0.0f;
        for (int w = 0; w < nw; ++w)
            t += sh[w][lane];
        if (which == 0) {
            dgamma_pre[col] = t;
        } else {
            if (dgamma_post)
                dgamma_post[col] = gate_ch ? gate_ch[col] * t : t;
            if (dgate_ch)
                dgate_ch[col] = gamma_post ? gamma_post[col] * t : t;
        }
    }
}

} // namespace w8a8
