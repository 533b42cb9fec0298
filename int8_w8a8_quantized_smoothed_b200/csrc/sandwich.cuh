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

// ------------------------------------------------------------------------------ backward
//
// With w = dz gamma_pre and p = gamma_post y (p = y without the first norm), per row:
//   D = dh + r2 w - h r2^3 A / K,                A = sum w h              (gradient of h)
//   dresidual = res_scale D,  dgate = D n
//   dy = r1 gate gamma_post D - y r1^3 S / K,    S = sum gate p D         (dy = gate D without it)
// S needs D, whose own sums are linear in it: sum p D = sum p dh + r2 sum p w - r2^3 A / K sum p h
// (p with the gate where it varies along the row), so one round of row sums gives all of them.
// dgamma_pre = sum_m dz h r2 and T = sum_m [gate] D y r1 are summed over the rows a CTA takes in
// registers (each thread keeps its eight columns for every row); part_kernel adds the CTAs'
// sums in a fixed order.
//
// A CTA covers up to 4096 columns (512 threads, one vector of 8 each); wider rows take a cluster
// of CTAs whose row sums meet through distributed shared memory, one barrier a row either way.

constexpr int kBackMaxThreads = 512;
constexpr int kBackSums = 6; // h h, w h, y y, p dh, p w, p h

struct SandwichBack {
    const uint16_t *dz, *dh, *y, *h;
    const float *gamma_post, *gamma_pre;
    const void *gate;
    uint16_t *dy, *dres, *dgate_full;
    float *dgate_tok;
    float *part; // [clusters][2][K]: dgamma_pre, T
    float res_scale, eps_post, eps_pre;
    int K, M;
};

__device__ __forceinline__ float warp_sum_f(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

__device__ __forceinline__ float ld_dsmem_f32(uint32_t addr)
{
    float r;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(r) : "r"(addr) : "memory");
    return r;
}

template <bool POST, int GATE, bool CLUSTER>
__global__ void __launch_bounds__(kBackMaxThreads, 1) sandwich_back_kernel(const SandwichBack a)
{
    __shared__ float sh[2][kBackSums][16]; // by row parity: one barrier a row
    if (threadIdx.x == 0)
        pdl_launch_dependents();
    pdl_wait();
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
    const int per = (nvec + csize - 1) / csize;
    const int vi = rank * per + threadIdx.x;
    const bool on = static_cast<int>(threadIdx.x) < per && vi < nvec;
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    constexpr bool kSums = POST || GATE == kGateToken; // sums of p wanted
    float gpost[8], gpre[8], gch[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        gpost[i] = gpre[i] = gch[i] = 1.0f;
    if (on) {
        load8_f32(a.gamma_pre, vi, gpre);
        if constexpr (POST)
            load8_f32(a.gamma_post, vi, gpost);
        if constexpr (GATE == kGateChannel)
            load8_f32(static_cast<const float *>(a.gate), vi, gch);
    }
    float acc_pre[8], acc_t[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        acc_pre[i] = acc_t[i] = 0.0f;
    uint4 ndz = zero, ndh = zero, ny = zero, nh = zero, ng = zero;
    auto fetch = [&](int64_t row) {
        if (on && row < a.M) {
            const int64_t o = row * nvec + vi;
            ndz = ldg_nc_v4(reinterpret_cast<const uint4 *>(a.dz) + o);
            if (a.dh)
                ndh = reinterpret_cast<const uint4 *>(a.dh)[o]; // dres may be dh: a plain load
            ny = ldg_nc_v4(reinterpret_cast<const uint4 *>(a.y) + o);
            nh = ldg_nc_v4(reinterpret_cast<const uint4 *>(a.h) + o);
            if constexpr (GATE == kGateFull)
                ng = ldg_nc_v4(reinterpret_cast<const uint4 *>(a.gate) + o);
        }
    };
    fetch(cl);
    const float invK = 1.0f / static_cast<float>(K);
    uint32_t it = 0;
    for (int64_t row = cl; row < a.M; row += ncl, ++it) {
        float dz[8], D[8], y[8], h[8], g[8];
        unpack8(ndz, dz);
        unpack8(ndh, D);
        unpack8(ny, y);
        unpack8(nh, h);
        if constexpr (GATE == kGateFull)
            unpack8(ng, g);
        else
#pragma unroll
            for (int i = 0; i < 8; ++i)
                g[i] = gch[i];
        float gt = 1.0f;
        if constexpr (GATE == kGateToken)
            gt = a.gate ? __ldg(static_cast<const float *>(a.gate) + row) : 1.0f;
        fetch(row + ncl);
        float s[kBackSums];
#pragma unroll
        for (int j = 0; j < kBackSums; ++j)
            s[j] = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float w = dz[i] * gpre[i];
            s[0] = fmaf(h[i], h[i], s[0]);
            s[1] = fmaf(w, h[i], s[1]);
            if constexpr (POST)
                s[2] = fmaf(y[i], y[i], s[2]);
            if constexpr (kSums) {
                const float p = GATE == kGateToken ? gpost[i] * y[i] : g[i] * gpost[i] * y[i];
                s[3] = fmaf(p, D[i], s[3]);
                s[4] = fmaf(p, w, s[4]);
                s[5] = fmaf(p, h[i], s[5]);
            }
        }
        float(&buf)[kBackSums][16] = sh[it & 1];
#pragma unroll
        for (int j = 0; j < kBackSums; ++j) {
            if ((j == 2 && !POST) || (j > 2 && !kSums))
                continue;
            s[j] = warp_sum_f(s[j]);
            if (lane == 0)
                buf[j][warp] = s[j];
        }
        if constexpr (CLUSTER)
            cluster_sync();
        else
            __syncthreads();
#pragma unroll
        for (int j = 0; j < kBackSums; ++j) {
            if ((j == 2 && !POST) || (j > 2 && !kSums))
                continue;
            float t = 0.0f;
            if constexpr (CLUSTER) {
                for (uint32_t r = 0; r < csize; ++r)
                    if (lane < nw)
                        t += ld_dsmem_f32(map_peer_smem(smem_u32(&buf[j][lane]), r));
            } else {
                t = lane < nw ? buf[j][lane] : 0.0f;
            }
            s[j] = warp_sum_f(t);
        }
        const float r2 = 1.0f / sqrtf(fmaf(s[0], invK, a.eps_pre));
        const float c2 = r2 * r2 * r2 * (s[1] * invK);
        const float r1 = POST ? 1.0f / sqrtf(fmaf(s[2], invK, a.eps_post)) : 1.0f;
        const float sp = fmaf(-c2, s[5], fmaf(r2, s[4], s[3])); // sum p D
        const float c1 = r1 * r1 * r1 * (gt * sp * invK);
        if constexpr (GATE == kGateToken)
            if (a.dgate_tok && threadIdx.x == 0 && rank == 0)
                a.dgate_tok[row] = r1 * sp;
        if (on) {
            float o[8], t8[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float w = dz[i] * gpre[i];
                D[i] = fmaf(r2, w, D[i]) - c2 * h[i];
                acc_pre[i] = fmaf(dz[i] * r2, h[i], acc_pre[i]);
                t8[i] = D[i] * a.res_scale;
            }
            const int64_t off = row * nvec + vi;
            reinterpret_cast<uint4 *>(a.dres)[off] =
                make_uint4(pack_bf16x2(t8[0], t8[1]), pack_bf16x2(t8[2], t8[3]),
                           pack_bf16x2(t8[4], t8[5]), pack_bf16x2(t8[6], t8[7]));
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float x1 = y[i] * r1;
                const float gate = GATE == kGateToken ? gt : g[i];
                if constexpr (GATE == kGateChannel)
                    acc_t[i] = fmaf(D[i], x1, acc_t[i]);
                else
                    acc_t[i] = fmaf(gate * D[i], x1, acc_t[i]);
                if constexpr (GATE == kGateFull)
                    t8[i] = D[i] * (x1 * gpost[i]);
                if constexpr (POST)
                    o[i] = fmaf(r1 * gpost[i], gate * D[i], -c1 * y[i]);
                else
                    o[i] = gate * D[i];
            }
            reinterpret_cast<uint4 *>(a.dy)[off] =
                make_uint4(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]),
                           pack_bf16x2(o[4], o[5]), pack_bf16x2(o[6], o[7]));
            if constexpr (GATE == kGateFull)
                reinterpret_cast<uint4 *>(a.dgate_full)[off] =
                    make_uint4(pack_bf16x2(t8[0], t8[1]), pack_bf16x2(t8[2], t8[3]),
                               pack_bf16x2(t8[4], t8[5]), pack_bf16x2(t8[6], t8[7]));
        }
    }
    if (on) {
        float4 *p0 = reinterpret_cast<float4 *>(a.part + (static_cast<int64_t>(cl) * 2) * K) + 2 * vi;
        p0[0] = make_float4(acc_pre[0], acc_pre[1], acc_pre[2], acc_pre[3]);
        p0[1] = make_float4(acc_pre[4], acc_pre[5], acc_pre[6], acc_pre[7]);
        if constexpr (POST || GATE == kGateChannel) {
            float4 *p1 = p0 + K / 4;
            p1[0] = make_float4(acc_t[0], acc_t[1], acc_t[2], acc_t[3]);
            p1[1] = make_float4(acc_t[4], acc_t[5], acc_t[6], acc_t[7]);
        }
    }
    if constexpr (CLUSTER)
        cluster_sync(); // a peer may still read this CTA's sums
}

// Column sums of the CTAs' parts, in order: dgamma_pre from array 0; T from array 1 gives
// dgamma_post = [gate_ch] T and dgate_ch = [gamma_post] T. A block takes 32 columns, a warp every
// eighth part.
__global__ void __launch_bounds__(256) sandwich_part_kernel(const float *__restrict__ part,
                                                            int nparts, int K,
                                                            const float *__restrict__ gamma_post,
                                                            const float *__restrict__ gate_ch,
                                                            float *__restrict__ dgamma_pre,
                                                            float *__restrict__ dgamma_post,
                                                            float *__restrict__ dgate_ch)
{
    __shared__ float sh[8][32];
    if (threadIdx.x == 0)
        pdl_launch_dependents();
    pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int col = blockIdx.x * 32 + lane;
    const int which = blockIdx.y;
    float t = 0.0f;
    if (col < K)
        for (int p = warp; p < nparts; p += 8)
            t += part[(static_cast<int64_t>(p) * 2 + which) * K + col];
    sh[warp][lane] = t;
    __syncthreads();
    if (warp == 0 && col < K) {
        t = 0.0f;
#pragma unroll
        for (int w = 0; w < 8; ++w)
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
