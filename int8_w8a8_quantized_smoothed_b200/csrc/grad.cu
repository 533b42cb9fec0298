// C ABI of the block-boundary norms and of the W8A8 linear's gradients (declared in
// include/w8a8.h): argument validation, launch shapes and launches. The kernels are in
// sandwich.cuh and gradgemm.cuh.
#include "gradgemm.cuh"
#include "host.cuh"
#include "sandwich.cuh"

#include <algorithm>

namespace w8a8 {

cudaError_t grad_status_read(unsigned int *word, cudaStream_t st)
{
    return cudaMemcpyFromSymbolAsync(word, g_status_word, sizeof(*word), 0, cudaMemcpyDeviceToHost,
                                     st);
}

cudaError_t grad_status_clear()
{
    const unsigned int zero = 0;
    return cudaMemcpyToSymbol(g_status_word, &zero, sizeof(zero));
}

} // namespace w8a8

namespace {

using namespace w8a8;

bool same(const void *a, const void *b)
{
    return a != nullptr && a == b;
}

// ------------------------------------------------------------------ norms at a block boundary

struct SandwichArgs {
    const uint16_t *y, *res;
    const float *gamma_post;
    const void *gate;
    float res_scale;
    const float *gamma_pre;
    float eps_post, eps_pre;
    int64_t M;
    int K;
    uint16_t *h;
    int8_t *q;
    float *s;
};

template <int NCH, bool POST, int GATE, bool F8>
int launch_sandwich(const SandwichArgs &a, int threads, int dev, int sms, cudaStream_t st)
{
    const void *fn = reinterpret_cast<const void *>(&sandwich_quant_kernel<NCH, POST, GATE, F8>);
    if (int rc = ensure_smem(fn, dev, 0))
        return rc;
    return launch_kernel(sandwich_quant_kernel<NCH, POST, GATE, F8>,
                         dim3(row_grid(fn, threads, a.M, dev, sms)), dim3(threads), 0, st, a.y,
                         a.res, a.gamma_post, a.gate, a.res_scale, a.gamma_pre, a.eps_post,
                         a.eps_pre, a.K, static_cast<int>(a.M), a.h, a.q, a.s);
}

// From this many values on, a call with rows of up to kRowsMaxK of them runs sandwich_rows_kernel
// (us, this kernel / one row a CTA: 300 x 4096 7.2 / 5.0, 600 x 4096 8.1 / 8.7, 333 x 5136 8.2 / 9.4,
// 8192 x 4096 with an elementwise gate 59 / 90; it begins by copying the gains).
constexpr int64_t kRowsFrom = 3 << 19;

template <int W, bool POST, int GATE, bool F8>
int launch_sandwich_rows_w(const SandwichArgs &a, int dev, int sms, cudaStream_t st)
{
    constexpr int kArrays = GATE == kGateFull ? 3 : 2;
    constexpr int kGains = 1 + (POST ? 1 : 0) + (GATE == kGateChannel ? 1 : 0);
    constexpr int kMax = 226 * 1024;
    const int64_t grid = std::min<int64_t>(a.M, sms);
    int teams = static_cast<int>(std::min<int64_t>(512 / (32 * W), (a.M + grid - 1) / grid));
    while (teams > 1 && rows_smem_bytes(a.K, kArrays, kGains, teams) > kMax)
        --teams;
    auto kernel = sandwich_rows_kernel<W, POST, GATE, F8>;
    static_assert(rows_smem_bytes(kRowsMaxK, 3, 3, 1) <= kMax, "shared memory per CTA");
    if (int rc = ensure_smem(reinterpret_cast<const void *>(kernel), dev, kMax))
        return rc;
    const SandwichRows r{a.y, a.res, a.gamma_post, a.gamma_pre, a.gate, a.h, a.q, a.s,
                         a.res_scale, a.eps_post, a.eps_pre, a.K, static_cast<int>(a.M), teams,
                         kWaitLimitNs};
    return launch_kernel(kernel, dim3(static_cast<unsigned>(grid)), dim3(teams * 32 * W),
                         rows_smem_bytes(a.K, kArrays, kGains, teams), st, r);
}

template <bool POST, int GATE, bool F8>
int launch_sandwich_rows_t(const SandwichArgs &a, int dev, int sms, cudaStream_t st)
{
    constexpr int kPerWarp = kRowsMaxK / 4;
    return a.K <= kPerWarp       ? launch_sandwich_rows_w<1, POST, GATE, F8>(a, dev, sms, st)
           : a.K <= 2 * kPerWarp ? launch_sandwich_rows_w<2, POST, GATE, F8>(a, dev, sms, st)
                                 : launch_sandwich_rows_w<4, POST, GATE, F8>(a, dev, sms, st);
}

template <bool F8>
int launch_sandwich_rows(const SandwichArgs &a, int gate_kind, int dev, int sms, cudaStream_t st)
{
    switch (gate_kind) {
    case kGateFull:
        return a.gamma_post ? launch_sandwich_rows_t<true, kGateFull, F8>(a, dev, sms, st)
                            : launch_sandwich_rows_t<false, kGateFull, F8>(a, dev, sms, st);
    case kGateChannel:
        return a.gamma_post ? launch_sandwich_rows_t<true, kGateChannel, F8>(a, dev, sms, st)
                            : launch_sandwich_rows_t<false, kGateChannel, F8>(a, dev, sms, st);
    default:
        return a.gamma_post ? launch_sandwich_rows_t<true, kGateToken, F8>(a, dev, sms, st)
                            : launch_sandwich_rows_t<false, kGateToken, F8>(a, dev, sms, st);
    }
}

template <int NCH, bool POST, bool F8>
int launch_sandwich_gate(const SandwichArgs &a, int gate_kind, int threads, int dev, int sms,
                         cudaStream_t st)
{
    switch (gate_kind) {
    case kGateFull: return launch_sandwich<NCH, POST, kGateFull, F8>(a, threads, dev, sms, st);
    case kGateChannel: return launch_sandwich<NCH, POST, kGateChannel, F8>(a, threads, dev, sms, st);
    default: return launch_sandwich<NCH, POST, kGateToken, F8>(a, threads, dev, sms, st);
    }
}

template <int NCH, bool F8>
int launch_sandwich_post(const SandwichArgs &a, int gate_kind, int threads, int dev, int sms,
                         cudaStream_t st)
{
    if (a.gamma_post)
        return launch_sandwich_gate<NCH, true, F8>(a, gate_kind, threads, dev, sms, st);
    return launch_sandwich_gate<NCH, false, F8>(a, gate_kind, threads, dev, sms, st);
}

bool gate_args_ok(const void *gate, int gate_kind)
{
    return gate_kind >= W8A8_GATE_NONE && gate_kind <= W8A8_GATE_FULL &&
           (gate != nullptr) == (gate_kind != W8A8_GATE_NONE);
}

bool finite(float v)
{
    return v - v == 0.0f;
}

template <bool F8>
int sandwich_quant_impl(const uint16_t *y, const uint16_t *residual, const float *gamma_post,
                        float eps_post, const void *gate, int gate_kind, float res_scale,
                        const float *gamma_smoothed, float eps, int64_t M, int64_t K,
                        uint16_t *h_out, int8_t *q, float *s_tok, w8a8_stream_t stream)
{
    if (!y || !residual || !gamma_smoothed || !h_out || !q || !s_tok ||
        !gate_args_ok(gate, gate_kind) || !finite(res_scale) || !(eps >= 0.0f) ||
        (gamma_post && !(eps_post >= 0.0f)))
        return W8A8_ERR_INVALID_ARG;
    int rc = check_row_shape(M, K);
    if (rc)
        return rc;
    if (!aligned16(y) || !aligned16(residual) || !aligned16(gamma_smoothed) || !aligned16(h_out) ||
        !aligned16(q) || (gamma_post && !aligned16(gamma_post)) ||
        (gate_kind >= W8A8_GATE_CHANNEL && !aligned16(gate)))
        return W8A8_ERR_ALIGNMENT;
    if (same(h_out, y) || same(h_out, gate) || same(q, y) || same(q, residual) || same(q, h_out) ||
        same(q, gate))
        return W8A8_ERR_INVALID_ARG;
    int dev, sms;
    if ((rc = current_device(&dev, &sms)))
        return rc;
    const SandwichArgs a{y, residual, gamma_post, gate, res_scale, gamma_smoothed, eps_post, eps,
                         M, static_cast<int>(K), h_out, q, s_tok};
    const RowLaunch L = row_launch(K);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (K <= kRowsMaxK && M * K >= kRowsFrom)
        return launch_sandwich_rows<F8>(a, gate_kind, dev, sms, st);
    switch (L.nch) {
    case 1: return launch_sandwich_post<1, F8>(a, gate_kind, L.threads, dev, sms, st);
    case 2: return launch_sandwich_post<2, F8>(a, gate_kind, L.threads, dev, sms, st);
    default: return launch_sandwich_post<4, F8>(a, gate_kind, L.threads, dev, sms, st);
    }
}

// Backward launch shape: clusters of `csize` CTAs of `threads`, one vector of 8 columns per
// thread, rings of three rows where two CTAs of 4096 columns (or one of 8192) leave the room, else
// of two. As many clusters as the device holds at 64 registers a thread, but beyond one CTA an SM
// only for at least four rows each, since each of them stores and adds sums as long as two rows.
struct SandwichBackPlan {
    int csize, threads, stages, smem;
    int64_t clusters;
};

SandwichBackPlan sandwich_back_plan(int64_t M, int64_t K, int arrays, int sms)
{
    constexpr int kSmemPerSm = 227 * 1024, kReserved = 1024;
    SandwichBackPlan p;
    const int64_t nvec = K / 8;
    p.csize = static_cast<int>((nvec + kBackMaxThreads - 1) / kBackMaxThreads);
    const int64_t per = (nvec + p.csize - 1) / p.csize;
    p.threads = static_cast<int>((per + 31) / 32 * 32);
    const int cols = static_cast<int>(per * 8);
    const int by_threads = kBackMaxThreads / p.threads;
    auto resident = [&](int stages) {
        return std::min(by_threads, kSmemPerSm / (back_smem_bytes(cols, arrays, stages) + kReserved));
    };
    p.stages = resident(3) >= std::min(by_threads, 2) ? 3 : 2;
    p.smem = back_smem_bytes(cols, arrays, p.stages);
    const int per_sm = std::max(1, std::min(resident(p.stages), 8));
    const int64_t one = std::max<int64_t>(1, sms / p.csize), all = sms * per_sm / p.csize;
    p.clusters = std::min<int64_t>(M, std::max(one, std::min<int64_t>(all, M / 4)));
    return p;
}

// The workspace does not depend on which inputs a call has: the most clusters of any.
size_t sandwich_back_ws(int64_t M, int64_t K, int sms)
{
    int64_t clusters = 0;
    for (int arrays = 3; arrays <= 5; ++arrays)
        clusters = std::max(clusters, sandwich_back_plan(M, K, arrays, sms).clusters);
    return static_cast<size_t>(clusters) * 2 * static_cast<size_t>(K) * sizeof(float);
}

// The most that a plan takes (resident() >= 1), and that the widest rows fit with two stages.
constexpr int kBackMaxSmem = 226 * 1024;
static_assert(back_smem_bytes(8 * kBackMaxThreads, 5, 2) <= kBackMaxSmem, "shared memory per CTA");

template <bool POST, int GATE>
int launch_sandwich_back(const SandwichBack &a, const SandwichBackPlan &p, int dev, cudaStream_t st)
{
    if (p.csize > 1) {
        const void *fn = reinterpret_cast<const void *>(&sandwich_back_kernel<POST, GATE, true>);
        if (int rc = ensure_smem(fn, dev, kBackMaxSmem))
            return rc;
        return launch_kernel_cluster(sandwich_back_kernel<POST, GATE, true>,
                                     dim3(static_cast<unsigned>(p.clusters * p.csize)),
                                     dim3(p.threads), p.smem, st, static_cast<unsigned>(p.csize), a);
    }
    const void *fn = reinterpret_cast<const void *>(&sandwich_back_kernel<POST, GATE, false>);
    if (int rc = ensure_smem(fn, dev, kBackMaxSmem))
        return rc;
    return launch_kernel(sandwich_back_kernel<POST, GATE, false>,
                         dim3(static_cast<unsigned>(p.clusters)), dim3(p.threads), p.smem, st, a);
}

template <bool POST>
int launch_sandwich_back_gate(const SandwichBack &a, int gate_kind, const SandwichBackPlan &p,
                              int dev, cudaStream_t st)
{
    switch (gate_kind) {
    case W8A8_GATE_FULL: return launch_sandwich_back<POST, kGateFull>(a, p, dev, st);
    case W8A8_GATE_CHANNEL: return launch_sandwich_back<POST, kGateChannel>(a, p, dev, st);
    default: return launch_sandwich_back<POST, kGateToken>(a, p, dev, st);
    }
}

// ------------------------------------------------------------------ gradients of a W8A8 linear

int check_grad_shape(int64_t M, int64_t N, int64_t K)
{
    if (M < 1 || N < 8 || K < 16)
        return W8A8_ERR_INVALID_ARG;
    if (N % 8 != 0 || K % 16 != 0 || M > (1 << 30) || N > (1 << 30) || K > (1 << 30))
        return W8A8_ERR_UNSUPPORTED_SHAPE;
    return W8A8_OK;
}

enum GradForm { kGradNarrow, kGradConv, kGradDequant };

struct GradPlan {
    GradWork w;
    GradForm form;
    int nt;          // rows of a narrow tile
    size_t part_off; // partial tiles of a split, after the bf16 operand
    size_t ws_bytes;
};

// Up to this many rows i an input gradient runs the narrow kernel.
constexpr int64_t kGradNarrowRows = 128;
// From this many rows i on and for sums of fewer than kGradDequantSum terms, Q is converted once
// ahead of the product: a pass over Q of 3 bytes a code, after which the GEMM is free of the
// conversions that the other form makes again for every 512 rows, and of that form's tile ends with
// nothing to hide behind. With longer sums the two take the same time and the pass would only cost
// its workspace (us, converting in the kernel / ahead: 4096 x 2048 x 4096 60 / 54, 8192 x 4096 x
// 4096 212 / 188, 4096 x 8192 x 4096 208 / 204, 4096 x 28672 x 4096 703 / 707;
// 2048 x 28672 x 4096 351 / 396).
constexpr int64_t kGradDequantRows = 4096, kGradDequantSum = 8192;
// The kernel that converts Q itself has tiles of 256 x 256, or of 512 x 256 with half the
// conversions but nothing to hide a tile's end behind: a k-block of either, and that end, us. (By
// 512 x 256 / 256 x 256: 2048 x 28672 x 4096 351 / 401 us, 2048 x 4096 x 4096 59 / 63, 512 x 4096 x
// 14336 with the SiLU epilogue 77 / 75, wgrad 1024 x 4000 x 4096 39 / 36. Of 45 random shapes the
// plan came within 5% of the better height in 43, within 6% in all.)
constexpr double kConvOneUs = 0.46, kConvTwoUs = 0.79, kTailUs = 5.0, kTailSiluUs = 8.0;
// Operands of up to this many bytes stay in L2 (126 MB) from one use to the next.
constexpr int64_t kGradL2Bytes = 64 << 20;

// The tiles of one form and how many pairs (CTAs) share the last ones; returns an estimate, us, for
// comparing plans. It is not the time: it leaves out a launch's start, and counts no end of the
// 256-row tiles (512 x 4096 x 14336 with the SiLU epilogue: 57, measured 75).
// The last tiles' k-blocks are split over more pairs where that saves more than the partial tiles
// cost: a k-block takes `each` us and a tile's end `tail` us more, the second launch about 3 us, and
// the partial tiles are stored and read at about 6 MB a us.
// Equal parts of every tile, so that the pairs walk r together and find each other's rows of Q and
// columns of dy in L2; uneven ones (all pairs busy, each at an r of its own) only where `uneven`
// says that both operands stay in L2 anyway: 1024 x 28672 x 4096 took 256 us uneven over 74 pairs,
// 219 us with 64 pairs of equal parts; 512 x 4096 x 14336 74 us uneven, 77 us without.
double plan_tiles(GradWork *w, int64_t I, int64_t J, int64_t R, int tile_i, int tile_j, int br,
                  int64_t pairs, double each, double tail, int min_share, bool uneven)
{
    const int64_t ni = (I + tile_i - 1) / tile_i, nj = (J + tile_j - 1) / tile_j;
    const int64_t kb = (R + br - 1) / br, tiles = ni * nj;
    w->I = static_cast<int>(I);
    w->J = static_cast<int>(J);
    w->R = static_cast<int>(R);
    w->tile_i = tile_i;
    w->tile_j = tile_j;
    w->ni = static_cast<int>(ni);
    w->nj = static_cast<int>(nj);
    w->kblocks = static_cast<int>(kb);
    w->group_i = tile_i > kGradTile ? 4 : 8;
    w->npairs = static_cast<int>(pairs);
    w->whole = static_cast<int>(tiles / pairs * pairs);
    w->rem = static_cast<int>(tiles % pairs);
    w->rem_pairs = w->rem;
    const double tile_bytes = 4.0 * std::min<int64_t>(I, tile_i) * tile_j;
    const double whole = static_cast<double>(tiles / pairs) * (each * static_cast<double>(kb) + tail);
    if (w->rem == 0)
        return whole;
    double best = each * static_cast<double>(kb) + tail;
    for (int k = 2; k <= 65; ++k) {
        int64_t split = static_cast<int64_t>(w->rem) * (k <= 64 ? k : pairs);
        if (split > pairs && !uneven)
            break;
        split = std::min(pairs, split);
        const double share = static_cast<double>((w->rem * kb + split - 1) / split);
        const double time = each * share + tail + 3.0 + (split + w->rem) * tile_bytes * 2 / 6e6;
        if (share >= min_share && time < best) {
            best = time;
            w->rem_pairs = static_cast<int>(split);
        }
        if (split == pairs)
            break;
    }
    return whole + best;
}

// False when there are more tiles than an int counts.
bool grad_plan(int64_t I, int64_t J, int64_t R, bool wgrad, bool silu, int sms, GradPlan *p)
{
    if ((I / kGradTile + 1) * (J / kGradTile + 1) > (1 << 30))
        return false;
    p->nt = I <= 16 ? 16 : I <= 32 ? 32 : I <= 64 ? 64 : 128;
    p->part_off = 0;
    const int pairs = sms / 2;
    const bool dequant = I >= kGradDequantRows && R < kGradDequantSum;
    const bool in_l2 = 2 * I * R + (dequant ? 2 : 1) * R * J <= kGradL2Bytes;
    if (dequant) {
        p->form = kGradDequant;
        plan_tiles(&p->w, I, J, R, kGradTile, kGradTile, kGradBR, pairs, 0.35, 0.0, 4, in_l2);
        p->part_off = (static_cast<size_t>(R) * static_cast<size_t>(J) * 2 + 255) / 256 * 256;
    } else if (!wgrad && I <= kGradNarrowRows) {
        p->form = kGradNarrow; // every CTA streams codes of its own
        plan_tiles(&p->w, I, J, R, p->nt, 128, kNarrowBR, sms, 0.4, 0.0, 2, true);
    } else {
        p->form = kGradConv;
        GradWork two;
        const double t1 = plan_tiles(&p->w, I, J, R, kGradTile, kGradTile, kGradBR, pairs,
                                     kConvOneUs, 0.0, 4, in_l2);
        const double t2 = plan_tiles(&two, I, J, R, 2 * kGradTile, kGradTile, kGradBR, pairs,
                                     kConvTwoUs, silu ? kTailSiluUs : kTailUs, 4, in_l2);
        if (t2 < t1)
            p->w = two;
    }
    p->ws_bytes = p->part_off;
    if (p->w.rem_pairs > p->w.rem)
        p->ws_bytes +=
            static_cast<size_t>(p->w.rem_pairs) * 2 * p->w.tile_i * p->w.tile_j * sizeof(float);
    return true;
}

// 2-D row-major tensor, `inner` elements of `esize` bytes per row, 128-byte boxes.
int encode_grad(CUtensorMap *map, const void *base, int64_t rows, int64_t inner, int esize,
                int box_rows, bool swizzle)
{
    cuuint64_t dims[2] = {static_cast<cuuint64_t>(inner), static_cast<cuuint64_t>(rows)};
    cuuint64_t strides[1] = {static_cast<cuuint64_t>(inner * esize)};
    cuuint32_t box[2] = {static_cast<cuuint32_t>(128 / esize), static_cast<cuuint32_t>(box_rows)};
    cuuint32_t estr[2] = {1, 1};
    CUresult r = encode_tiled(
        map, esize == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 2,
        const_cast<void *>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
        swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? W8A8_OK : W8A8_ERR_CUDA;
}

// The second launch, where tiles were split.
template <bool SILU>
int launch_fixup(const GradWork &w, const float *part, const uint16_t *gate_up, uint16_t *out,
                 int dev, cudaStream_t st)
{
    if (w.rem_pairs <= w.rem)
        return W8A8_OK;
    const void *fn = reinterpret_cast<const void *>(&grad_fixup_kernel<SILU>);
    if (int rc = ensure_smem(fn, dev, 0))
        return rc;
    const unsigned values = static_cast<unsigned>(std::min(w.I, w.tile_i) * w.tile_j);
    return launch_kernel(grad_fixup_kernel<SILU>,
                         dim3((values + 2047) / 2048, static_cast<unsigned>(w.rem)), dim3(256), 0,
                         st, w, part, gate_up, out);
}

template <bool CONV, int H, bool WGRAD, bool F8, bool SILU>
int launch_grad(const CUtensorMap &ta, const CUtensorMap &tq, const float *scale,
                const GradWork &w, const uint16_t *gate_up, uint16_t *out, float *part, int dev,
                cudaStream_t st)
{
    using Cfg = GradCfg<CONV, H>;
    auto kernel = grad_gemm_kernel<CONV, H, WGRAD, F8, SILU>;
    if (int rc = ensure_smem(reinterpret_cast<const void *>(kernel), dev, Cfg::kSmemBytes))
        return rc;
    const unsigned pairs = static_cast<unsigned>(w.whole > 0 ? w.npairs : w.rem_pairs);
    if (int rc = launch_kernel_cluster(kernel, dim3(2 * pairs), dim3(Cfg::kThreads),
                                       Cfg::kSmemBytes, st, 2u, ta, tq, scale, w, gate_up, out,
                                       part, kWaitLimitNs))
        return rc;
    return launch_fixup<SILU>(w, part, gate_up, out, dev, st);
}

template <bool WGRAD, bool F8, bool SILU>
int launch_conv(const CUtensorMap &ta, const CUtensorMap &tq, const float *scale,
                const GradWork &w, const uint16_t *gate_up, uint16_t *out, float *part, int dev,
                cudaStream_t st)
{
    return w.tile_i > kGradTile
               ? launch_grad<true, 2, WGRAD, F8, SILU>(ta, tq, scale, w, gate_up, out, part, dev, st)
               : launch_grad<true, 1, WGRAD, F8, SILU>(ta, tq, scale, w, gate_up, out, part, dev, st);
}

template <int NT, bool F8, bool SILU>
int launch_narrow(const CUtensorMap &ta, const CUtensorMap &tq, const float *scale,
                  const GradWork &w, const uint16_t *gate_up, uint16_t *out, float *part, int dev,
                  cudaStream_t st)
{
    using Cfg = NarrowCfg<NT>;
    auto kernel = grad_narrow_kernel<NT, F8, SILU>;
    if (int rc = ensure_smem(reinterpret_cast<const void *>(kernel), dev, Cfg::kSmemBytes))
        return rc;
    const unsigned ctas = static_cast<unsigned>(w.whole > 0 ? w.npairs : w.rem_pairs);
    if (int rc = launch_kernel(kernel, dim3(ctas), dim3(kNarrowThreads), Cfg::kSmemBytes, st, ta,
                               tq, scale, w, gate_up, out, part, kWaitLimitNs))
        return rc;
    return launch_fixup<SILU>(w, part, gate_up, out, dev, st);
}

template <bool F8, bool SILU>
int launch_narrow_nt(int nt, const CUtensorMap &ta, const CUtensorMap &tq, const float *scale,
                     const GradWork &w, const uint16_t *gate_up, uint16_t *out, float *part,
                     int dev, cudaStream_t st)
{
    switch (nt) {
    case 16: return launch_narrow<16, F8, SILU>(ta, tq, scale, w, gate_up, out, part, dev, st);
    case 32: return launch_narrow<32, F8, SILU>(ta, tq, scale, w, gate_up, out, part, dev, st);
    case 64: return launch_narrow<64, F8, SILU>(ta, tq, scale, w, gate_up, out, part, dev, st);
    default: return launch_narrow<128, F8, SILU>(ta, tq, scale, w, gate_up, out, part, dev, st);
    }
}

template <bool F8>
int launch_dequant(const void *q, const float *scale, int64_t R, int64_t J, uint16_t *out, int dev,
                   int sms, cudaStream_t st)
{
    const void *fn = reinterpret_cast<const void *>(&grad_dequant_kernel<F8>);
    if (int rc = ensure_smem(fn, dev, 0))
        return rc;
    const int64_t nvec = R * (J / 16);
    const int64_t grid = std::min<int64_t>((nvec + 255) / 256, static_cast<int64_t>(sms) * 8);
    return launch_kernel(grad_dequant_kernel<F8>, dim3(static_cast<unsigned>(grid)), dim3(256), 0,
                         st, static_cast<const uint8_t *>(q), scale, nvec,
                         static_cast<uint32_t>(J / 16), out);
}

// dy [M, N]; Q: wq [N, K] (input gradient) or xq [M, K] (weight gradient).
template <bool WGRAD, bool SILU>
int grad_impl(bool f8, const uint16_t *dy, const void *q, const float *scale, int64_t M, int64_t N,
              int64_t K, const uint16_t *gate_up, uint16_t *out, void *workspace,
              size_t workspace_bytes, w8a8_stream_t stream)
{
    if (!dy || !q || !scale || !out || (SILU && !gate_up))
        return W8A8_ERR_INVALID_ARG;
    int rc = check_grad_shape(M, N, K);
    if (rc)
        return rc;
    if (!aligned16(dy) || !aligned16(q) || !aligned16(out) || (SILU && !aligned16(gate_up)) ||
        (workspace && !aligned16(workspace)))
        return W8A8_ERR_ALIGNMENT;
    if (same(out, dy) || same(out, q) || same(out, gate_up))
        return W8A8_ERR_INVALID_ARG;
    int dev, sms;
    if ((rc = current_device(&dev, &sms)))
        return rc;
    const int64_t R = WGRAD ? M : N;
    GradPlan p;
    if (!grad_plan(WGRAD ? N : M, K, R, WGRAD, SILU, sms, &p))
        return W8A8_ERR_UNSUPPORTED_SHAPE;
    if (p.ws_bytes > 0 && (workspace == nullptr || workspace_bytes < p.ws_bytes))
        return W8A8_ERR_WORKSPACE;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    float *part = reinterpret_cast<float *>(static_cast<char *>(workspace) + p.part_off);
    CUtensorMap ta, tq;
    const int box_i = p.form == kGradNarrow ? p.nt : 128;
    if (encode_grad(&ta, dy, M, N, 2, WGRAD ? kGradBR : box_i, true))
        return W8A8_ERR_CUDA;
    if (p.form != kGradDequant) {
        if (encode_grad(&tq, q, R, K, 1, p.form == kGradNarrow ? kNarrowBR : kGradBR,
                        p.form == kGradNarrow))
            return W8A8_ERR_CUDA;
        if constexpr (!WGRAD)
            if (p.form == kGradNarrow)
                return f8 ? launch_narrow_nt<true, SILU>(p.nt, ta, tq, scale, p.w, gate_up, out,
                                                         part, dev, st)
                          : launch_narrow_nt<false, SILU>(p.nt, ta, tq, scale, p.w, gate_up, out,
                                                          part, dev, st);
        return f8 ? launch_conv<WGRAD, true, SILU>(ta, tq, scale, p.w, gate_up, out, part, dev, st)
                  : launch_conv<WGRAD, false, SILU>(ta, tq, scale, p.w, gate_up, out, part, dev, st);
    }
    uint16_t *b = static_cast<uint16_t *>(workspace);
    if (encode_grad(&tq, b, R, K, 2, kGradBR, true))
        return W8A8_ERR_CUDA;
    if ((rc = f8 ? launch_dequant<true>(q, scale, R, K, b, dev, sms, st)
                 : launch_dequant<false>(q, scale, R, K, b, dev, sms, st)))
        return rc;
    return launch_grad<false, 1, WGRAD, false, SILU>(ta, tq, scale, p.w, gate_up, out, part, dev, st);
}

size_t grad_workspace(int64_t M, int64_t N, int64_t K, bool wgrad)
{
    if (check_grad_shape(M, N, K))
        return 0;
    int dev, sms = 148;
    if (current_device(&dev, &sms))
        sms = 148;
    GradPlan p, q;
    if (!grad_plan(wgrad ? N : M, K, wgrad ? M : N, wgrad, false, sms, &p))
        return 0;
    if (wgrad)
        return p.ws_bytes;
    grad_plan(M, K, N, false, true, sms, &q); // one size serves the input gradient's two forms
    return std::max(p.ws_bytes, q.ws_bytes);
}

} // namespace

extern "C" {

size_t w8a8_gemm_dgrad_workspace_size(int64_t M, int64_t N, int64_t K)
{
    return grad_workspace(M, N, K, false);
}

size_t w8a8_gemm_wgrad_workspace_size(int64_t M, int64_t N, int64_t K)
{
    return grad_workspace(M, N, K, true);
}

int w8a8_gemm_dgrad(const w8a8_bf16 *dy, const int8_t *wq, const float *s_ch, int64_t M, int64_t N,
                    int64_t K, w8a8_bf16 *dx, void *workspace, size_t workspace_bytes,
                    w8a8_stream_t stream)
{
    return grad_impl<false, false>(false, dy, wq, s_ch, M, N, K, nullptr, dx, workspace,
                                   workspace_bytes, stream);
}

int w8a8_gemm_dgrad_fp8(const w8a8_bf16 *dy, const uint8_t *wq, const float *s_ch, int64_t M,
                        int64_t N, int64_t K, w8a8_bf16 *dx, void *workspace,
                        size_t workspace_bytes, w8a8_stream_t stream)
{
    return grad_impl<false, false>(true, dy, wq, s_ch, M, N, K, nullptr, dx, workspace,
                                   workspace_bytes, stream);
}

int w8a8_gemm_dgrad_silu(const w8a8_bf16 *dy, const int8_t *wq, const float *s_ch, int64_t M,
                         int64_t N, int64_t I, const w8a8_bf16 *gate_up, w8a8_bf16 *dgate_up,
                         void *workspace, size_t workspace_bytes, w8a8_stream_t stream)
{
    return grad_impl<false, true>(false, dy, wq, s_ch, M, N, I, gate_up, dgate_up, workspace,
                                  workspace_bytes, stream);
}

int w8a8_gemm_dgrad_silu_fp8(const w8a8_bf16 *dy, const uint8_t *wq, const float *s_ch, int64_t M,
                             int64_t N, int64_t I, const w8a8_bf16 *gate_up, w8a8_bf16 *dgate_up,
                             void *workspace, size_t workspace_bytes, w8a8_stream_t stream)
{
    return grad_impl<false, true>(true, dy, wq, s_ch, M, N, I, gate_up, dgate_up, workspace,
                                  workspace_bytes, stream);
}

int w8a8_gemm_wgrad(const w8a8_bf16 *dy, const int8_t *xq, const float *s_tok, int64_t M, int64_t N,
                    int64_t K, w8a8_bf16 *dw, void *workspace, size_t workspace_bytes,
                    w8a8_stream_t stream)
{
    return grad_impl<true, false>(false, dy, xq, s_tok, M, N, K, nullptr, dw, workspace,
                                  workspace_bytes, stream);
}

int w8a8_gemm_wgrad_fp8(const w8a8_bf16 *dy, const uint8_t *xq, const float *s_tok, int64_t M,
                        int64_t N, int64_t K, w8a8_bf16 *dw, void *workspace,
                        size_t workspace_bytes, w8a8_stream_t stream)
{
    return grad_impl<true, false>(true, dy, xq, s_tok, M, N, K, nullptr, dw, workspace,
                                  workspace_bytes, stream);
}

int w8a8_sandwich_rmsnorm_quant(const w8a8_bf16 *y, const w8a8_bf16 *residual,
                                const float *gamma_post, float eps_post, const void *gate,
                                int gate_kind, float res_scale, const float *gamma_smoothed,
                                float eps, int64_t M, int64_t K, w8a8_bf16 *h_out, int8_t *q,
                                float *s_tok, w8a8_stream_t stream)
{
    return sandwich_quant_impl<false>(y, residual, gamma_post, eps_post, gate, gate_kind,
                                      res_scale, gamma_smoothed, eps, M, K, h_out, q, s_tok,
                                      stream);
}

int w8a8_sandwich_rmsnorm_quant_fp8(const w8a8_bf16 *y, const w8a8_bf16 *residual,
                                    const float *gamma_post, float eps_post, const void *gate,
                                    int gate_kind, float res_scale, const float *gamma_smoothed,
                                    float eps, int64_t M, int64_t K, w8a8_bf16 *h_out, uint8_t *q,
                                    float *s_tok, w8a8_stream_t stream)
{
    return sandwich_quant_impl<true>(y, residual, gamma_post, eps_post, gate, gate_kind, res_scale,
                                     gamma_smoothed, eps, M, K, h_out,
                                     reinterpret_cast<int8_t *>(q), s_tok, stream);
}

size_t w8a8_sandwich_rmsnorm_backward_workspace_size(int64_t M, int64_t K)
{
    if (check_row_shape(M, K))
        return 0;
    int dev, sms = 148;
    if (current_device(&dev, &sms))
        sms = 148;
    return sandwich_back_ws(M, K, sms);
}

int w8a8_sandwich_rmsnorm_backward(const w8a8_bf16 *dz, const w8a8_bf16 *dh, const w8a8_bf16 *y,
                                   const w8a8_bf16 *h, const float *gamma_post, float eps_post,
                                   const void *gate, int gate_kind, float res_scale,
                                   const float *gamma_smoothed, float eps, int64_t M, int64_t K,
                                   w8a8_bf16 *dy, w8a8_bf16 *dresidual, float *dgamma_post,
                                   void *dgate, float *dgamma_smoothed, void *workspace,
                                   size_t workspace_bytes, w8a8_stream_t stream)
{
    if (!dz || !y || !h || !gamma_smoothed || !dy || !dresidual || !dgamma_smoothed ||
        !gate_args_ok(gate, gate_kind) || (dgate != nullptr) != (gate != nullptr) ||
        (dgamma_post != nullptr) != (gamma_post != nullptr) || !finite(res_scale) ||
        !(eps >= 0.0f) || (gamma_post && !(eps_post >= 0.0f)))
        return W8A8_ERR_INVALID_ARG;
    int rc = check_row_shape(M, K);
    if (rc)
        return rc;
    if (!aligned16(dz) || (dh && !aligned16(dh)) || !aligned16(y) || !aligned16(h) ||
        !aligned16(gamma_smoothed) || (gamma_post && !aligned16(gamma_post)) || !aligned16(dy) ||
        !aligned16(dresidual) || (workspace && !aligned16(workspace)) ||
        (gate_kind >= W8A8_GATE_CHANNEL && !aligned16(gate)) ||
        (gate_kind == W8A8_GATE_FULL && !aligned16(dgate)))
        return W8A8_ERR_ALIGNMENT;
    // dresidual may be dh (in place); every other output is written while inputs are still read
    const void *in[] = {dz, y, h, gate};
    for (const void *p : in)
        if (same(dy, p) || same(dresidual, p) || same(dgate, p))
            return W8A8_ERR_INVALID_ARG;
    if (same(dy, dh) || same(dgate, dh) || same(dy, dresidual) || same(dgate, dy) ||
        same(dgate, dresidual))
        return W8A8_ERR_INVALID_ARG;
    int dev, sms;
    if ((rc = current_device(&dev, &sms)))
        return rc;
    if (workspace == nullptr || workspace_bytes < sandwich_back_ws(M, K, sms))
        return W8A8_ERR_WORKSPACE;
    const SandwichBackPlan p =
        sandwich_back_plan(M, K, 3 + (dh ? 1 : 0) + (gate_kind == W8A8_GATE_FULL ? 1 : 0), sms);
    SandwichBack a;
    a.dz = dz;
    a.dh = dh;
    a.y = y;
    a.h = h;
    a.gamma_post = gamma_post;
    a.gamma_pre = gamma_smoothed;
    a.gate = gate;
    a.dy = dy;
    a.dres = dresidual;
    a.dgate_full = gate_kind == W8A8_GATE_FULL ? static_cast<uint16_t *>(dgate) : nullptr;
    a.dgate_tok = gate_kind == W8A8_GATE_TOKEN ? static_cast<float *>(dgate) : nullptr;
    a.part = static_cast<float *>(workspace);
    a.res_scale = res_scale;
    a.eps_post = eps_post;
    a.eps_pre = eps;
    a.K = static_cast<int>(K);
    a.M = static_cast<int>(M);
    a.stages = p.stages;
    a.limit_ns = kWaitLimitNs;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    rc = gamma_post ? launch_sandwich_back_gate<true>(a, gate_kind, p, dev, st)
                    : launch_sandwich_back_gate<false>(a, gate_kind, p, dev, st);
    if (rc)
        return rc;
    const bool channel = gate_kind == W8A8_GATE_CHANNEL;
    const void *fn = reinterpret_cast<const void *>(&sandwich_part_kernel);
    if ((rc = ensure_smem(fn, dev, 0)))
        return rc;
    return launch_kernel(sandwich_part_kernel,
                         dim3(static_cast<unsigned>((K + 31) / 32), gamma_post || channel ? 2 : 1),
                         dim3(p.clusters > 320 ? 1024 : 256), 0, st, static_cast<const float *>(workspace),
                         static_cast<int>(p.clusters), static_cast<int>(K), gamma_post,
                         channel ? static_cast<const float *>(gate) : nullptr, dgamma_smoothed,
                         dgamma_post, channel ? static_cast<float *>(dgate) : nullptr);
}

} // extern "C"
