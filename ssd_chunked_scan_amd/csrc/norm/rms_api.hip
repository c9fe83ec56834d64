// rms_api.hip -- host side of the root-mean-square norm (ssd_rms_norm_* in include/ssd.h).
// Validation is host-only and runs before any HIP call; nothing here allocates,
// frees or synchronises.
#include "ssd.h"

#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

#include "api_checks.hpp"
#include "rms_kernels.hpp"

using namespace ssd;
using namespace ssd::rms;

namespace {

ssd_status launched() { return hipGetLastError() == hipSuccess ? SSD_OK : SSD_ERR_HIP; }

constexpr int64_t kMaxDim = 65536;
// Rows of one launch: at up to 1024 threads each, fewer than 2^32 threads.
constexpr int64_t kLaunchRows = (int64_t)1 << 21;

ssd_status check_dims(int64_t rows, int64_t dim, int dtype, int res_dtype)
{
    if (!known_dtype(dtype) || !known_dtype(res_dtype)) return SSD_ERR_BAD_DTYPE;
    if (rows < 0 || dim < 1 || dim > kMaxDim || rows > INT32_MAX || rows > ((int64_t)1 << 40) / dim) return SSD_ERR_BAD_SHAPE;
    return SSD_OK;
}

// Rows of whole runs start at 16 bytes, others at any element.
bool rows_aligned(const void *p, int64_t dim, size_t esz) { return aligned_to(p, dim % kRun == 0 ? 16 : esz); }

// How a row of `dim` is held: lanes of a row and runs of 8 values a lane.  Rows that are not whole
// runs have fewer forms.  The backward's rows take up to four times the registers, so
// they have more lanes.
struct Plan {
    int L, IT;
};
constexpr Plan kFwdPlans[] = {{16, 1}, {64, 1}, {64, 2}, {64, 3}, {64, 5}, {256, 2}, {256, 3}, {256, 4}, {1024, 2}},
               kBwdPlans[] = {{16, 1}, {64, 1}, {64, 2}, {64, 3}, {256, 1}, {256, 2}, {256, 3}, {1024, 1}},
               kFwdOdd[] = {{16, 1}, {64, 2}, {256, 2}, {256, 4}, {1024, 2}}, kBwdOdd[] = {{16, 1}, {64, 2}, {256, 2}, {1024, 1}};
constexpr int64_t kFwdHeld = 16384, kBwdHeld = 8192;   // the longest rows of these
enum class Form { Fwd, Bwd, FwdOdd, BwdOdd };
template <Form F> constexpr int plans() { return F == Form::Fwd ? 9 : F == Form::Bwd ? 8 : F == Form::FwdOdd ? 5 : 4; }
template <Form F> constexpr Plan plan_at(int i)
{
    return F == Form::Fwd ? kFwdPlans[i] : F == Form::Bwd ? kBwdPlans[i] : F == Form::FwdOdd ? kFwdOdd[i] : kBwdOdd[i];
}
template <int N> using Int = std::integral_constant<int, N>;
// f(lanes, runs) of the first form that holds the row.
template <Form F, int I = 0, typename Fn> void with_plan(int64_t dim, Fn &&f)
{
    if constexpr (I < plans<F>()) {
        constexpr Plan p = plan_at<F>(I);
        if ((int64_t)p.L * p.IT * kRun >= dim) f(Int<p.L>{}, Int<p.IT>{});
        else with_plan<F, I + 1>(dim, f);
    }
}

// Rows per workgroup of the backward: about 512 strips, whole rounds of its row groups.
int64_t strip_of(int64_t rows, int64_t dim)
{
    int64_t groups = 1;
    auto of = [&](auto l, auto) { groups = decltype(l)::value < kThreads ? kThreads / decltype(l)::value : 1; };
    if (dim % kRun == 0) with_plan<Form::Bwd>(dim, of);
    else with_plan<Form::BwdOdd>(dim, of);
    return ceil_div(ceil_div(rows, 512), groups) * groups;
}

template <typename E, typename R, bool RES> void fwd_typed(const ssd_rms_norm_args *a, hipStream_t st)
{
    const int64_t nb = ceil_div(a->dim, 128);
    for (int64_t r0 = 0; r0 < a->rows; r0 += kLaunchRows) {
        FwdArgs k{};
        const int64_t o = r0 * a->dim;
        k.x = (const E *)a->x + o;
        k.res = RES ? (const R *)a->residual + o : nullptr;
        k.w = a->weight;
        k.res_out = RES ? (R *)a->residual_out + o : nullptr;
        k.y = a->y ? (E *)a->y + o : nullptr;
        k.q = a->q ? (uint8_t *)a->q + o : nullptr;
        k.scales = a->q ? a->scales + r0 * nb : nullptr;
        k.rstd = a->rstd ? a->rstd + r0 : nullptr;
        k.rows = a->rows - r0 < kLaunchRows ? a->rows - r0 : kLaunchRows;
        k.dim = (int)a->dim;
        k.eps = a->eps;
        auto launch = [&](auto al, auto l, auto it) {
            constexpr int L = decltype(l)::value;
            // few rows: a wave per workgroup, so they spread over the CUs
            const int threads = L >= kThreads ? L : k.rows * L <= 64 * 1024 ? 64 : kThreads;
            hipLaunchKernelGGL((k_rms_fwd<E, R, RES, decltype(al)::value, L, decltype(it)::value>),
                               dim3((unsigned)ceil_div(k.rows, threads / L)), dim3(threads), 0, st, k);
        };
        if (a->dim > kFwdHeld) hipLaunchKernelGGL((k_rms_fwd_long<E, R, RES>), dim3((unsigned)k.rows), dim3(kLong), 0, st, k);
        else if (a->dim % kRun == 0) with_plan<Form::Fwd>(a->dim, [&](auto l, auto it) { launch(std::true_type{}, l, it); });
        else with_plan<Form::FwdOdd>(a->dim, [&](auto l, auto it) { launch(std::false_type{}, l, it); });
    }
}

template <typename E, typename R> void bwd_typed(const ssd_rms_norm_bwd_args *a, hipStream_t st)
{
    BwdArgs k{};
    k.r = a->r;
    k.dy = a->dy;
    k.dres = a->dresidual_out;
    k.rstd = a->rstd;
    k.w = a->weight;
    k.dx = a->dx;
    k.dr = a->dresidual;
    k.parts = a->dweight ? static_cast<float *>(a->workspace) : nullptr;
    k.rows = a->rows;
    k.dim = (int)a->dim;
    k.strip = (int)strip_of(a->rows, a->dim);
    const unsigned strips = (unsigned)ceil_div(a->rows, k.strip);
    if (a->dim > kBwdHeld) {
        if (a->dweight)   // before dx, which may be dy
            hipLaunchKernelGGL((k_rms_cols_long<E, R>), dim3(strips, (unsigned)ceil_div(a->dim, kThreads)), dim3(kThreads), 0, st, k);
        for (int64_t r0 = 0; r0 < a->rows; r0 += kLaunchRows) {
            const int64_t n = a->rows - r0 < kLaunchRows ? a->rows - r0 : kLaunchRows, o = r0 * a->dim;
            BwdArgs b = k;
            b.r = (const R *)a->r + o;
            b.dy = (const E *)a->dy + o;
            b.dres = a->dresidual_out ? (const R *)a->dresidual_out + o : nullptr;
            b.rstd = a->rstd + r0;
            b.dx = (E *)a->dx + o;
            b.dr = a->dresidual ? (R *)a->dresidual + o : nullptr;
            hipLaunchKernelGGL((k_rms_dx_long<E, R>), dim3((unsigned)n), dim3(kLong), 0, st, b);
        }
    } else {
        auto launch = [&](auto al, auto l, auto it) {
            constexpr bool AL = decltype(al)::value;
            constexpr int L = decltype(l)::value, IT = decltype(it)::value;
            const dim3 block(L > kThreads ? L : kThreads);
            if (k.dres) hipLaunchKernelGGL((k_rms_bwd<E, R, true, AL, L, IT>), dim3(strips), block, 0, st, k);
            else hipLaunchKernelGGL((k_rms_bwd<E, R, false, AL, L, IT>), dim3(strips), block, 0, st, k);
        };
        if (a->dim % kRun == 0) with_plan<Form::Bwd>(a->dim, [&](auto l, auto it) { launch(std::true_type{}, l, it); });
        else with_plan<Form::BwdOdd>(a->dim, [&](auto l, auto it) { launch(std::false_type{}, l, it); });
    }
    if (a->dweight)
        hipLaunchKernelGGL(k_rms_sum, dim3((unsigned)ceil_div(a->dim, 32)), dim3(1024), 0, st, (const float *)k.parts, a->dweight,
                           (int)strips, (int)a->dim);
}

__global__ __launch_bounds__(kThreads) void k_rms_zero(float *p, int n)
{
    const int i = blockIdx.x * kThreads + threadIdx.x;
    if (i < n) p[i] = 0.f;
}

}  // namespace

extern "C" {

ssd_status ssd_rms_norm_fwd(const ssd_rms_norm_args *a, void *stream)
{
    if (!a) return SSD_ERR_NULL_POINTER;
    const ssd_status r = check_dims(a->rows, a->dim, a->dtype, a->residual_dtype);
    if (r != SSD_OK) return r;
    if (a->rows == 0) return SSD_OK;
    if (!a->x || (!a->y && !a->q) || (a->residual && !a->residual_out) || (!a->residual && a->residual_out) || (a->q && !a->scales))
        return SSD_ERR_NULL_POINTER;
    const size_t e = elem_size(a->dtype), re = elem_size(a->residual_dtype);
    if (!rows_aligned(a->x, a->dim, e) || !rows_aligned(a->y, a->dim, e) || !rows_aligned(a->residual, a->dim, re) ||
        !rows_aligned(a->residual_out, a->dim, re) || !rows_aligned(a->q, a->dim, 1) || !aligned_to(a->weight, 16))
        return SSD_ERR_MISALIGNED;
    if (!aligned_to(a->scales, 4) || !aligned_to(a->rstd, 4)) return SSD_ERR_MISALIGNED;
    const size_t n = (size_t)(a->rows * a->dim);
    const Range ins[] = {{a->x, n * e}, {a->residual, n * re}, {a->weight, (size_t)a->dim * 4}};
    const Range outs[] = {{a->residual_out, n * re}, {a->y, n * e}, {a->q, n},
                          {a->q ? a->scales : nullptr, (size_t)(a->rows * ceil_div(a->dim, 128)) * 4}, {a->rstd, (size_t)a->rows * 4}};
    for (int i = 0; i < 5; ++i) {
        for (int j = 0; j < 3; ++j) {
            // a value is written where it was read
            const bool same = outs[i].p == ins[j].p && outs[i].n == ins[j].n && ((i == 0 && j < 2) || (i == 1 && j == 0));
            if (!same && overlaps(outs[i], ins[j])) return SSD_ERR_ALIASING;
        }
        for (int j = i + 1; j < 5; ++j)
            if (overlaps(outs[i], outs[j])) return SSD_ERR_ALIASING;
    }
    hipStream_t st = static_cast<hipStream_t>(stream);
    const bool bf = a->dtype == SSD_DTYPE_BF16, rbf = a->residual_dtype == SSD_DTYPE_BF16;
    if (!a->residual) {
        if (bf) fwd_typed<bf16, bf16, false>(a, st);
        else fwd_typed<float, float, false>(a, st);
    } else if (bf) {
        if (rbf) fwd_typed<bf16, bf16, true>(a, st);
        else fwd_typed<bf16, float, true>(a, st);
    } else {
        if (rbf) fwd_typed<float, bf16, true>(a, st);
        else fwd_typed<float, float, true>(a, st);
    }
    return launched();
}

ssd_status ssd_rms_norm_bwd_workspace_size(const ssd_rms_norm_bwd_args *a, size_t *bytes)
{
    if (!a) return SSD_ERR_NULL_POINTER;
    const ssd_status r = check_dims(a->rows, a->dim, a->dtype, a->residual_dtype);
    if (r != SSD_OK) return r;
    if (!bytes) return SSD_ERR_NULL_POINTER;
    *bytes = a->rows ? (size_t)(ceil_div(a->rows, strip_of(a->rows, a->dim)) * a->dim) * 4 : 0;
    return SSD_OK;
}

ssd_status ssd_rms_norm_bwd(const ssd_rms_norm_bwd_args *a, void *stream)
{
    size_t need = 0;
    const ssd_status r = ssd_rms_norm_bwd_workspace_size(a, &need);
    if (r != SSD_OK) return r;
    hipStream_t st = static_cast<hipStream_t>(stream);
    const size_t e = elem_size(a->dtype), re = elem_size(a->residual_dtype);
    if (!rows_aligned(a->dy, a->dim, e) || !rows_aligned(a->dx, a->dim, e) || !rows_aligned(a->r, a->dim, re) ||
        !rows_aligned(a->dresidual_out, a->dim, re) || !rows_aligned(a->dresidual, a->dim, re))
        return SSD_ERR_MISALIGNED;
    const void *ptrs[] = {a->weight, a->dweight, a->workspace};
    for (const void *p : ptrs)
        if (!aligned_to(p, 16)) return SSD_ERR_MISALIGNED;
    if (!aligned_to(a->rstd, 4)) return SSD_ERR_MISALIGNED;
    if (a->rows > 0) {
        if (!a->r || !a->dy || !a->rstd || !a->dx) return SSD_ERR_NULL_POINTER;
        if (a->dweight && !a->workspace) return SSD_ERR_NULL_POINTER;
        if (a->dweight && a->workspace_bytes < need) return SSD_ERR_WORKSPACE_TOO_SMALL;
    }
    const size_t n = (size_t)(a->rows * a->dim), d = (size_t)a->dim * 4;
    const Range ins[] = {{a->dy, n * e}, {a->dresidual_out, n * re}, {a->r, n * re}, {a->rstd, (size_t)a->rows * 4}, {a->weight, d}};
    const Range outs[] = {{a->dx, n * e}, {a->dresidual, n * re}, {a->dweight, d}, {a->dweight ? a->workspace : nullptr, need}};
    for (int i = 0; i < 4; ++i) {
        for (int j = 0; j < 5; ++j) {
            const bool same = i == j && i < 2 && outs[i].p == ins[j].p;   // dx over dy, dresidual over dresidual_out
            if (!same && overlaps(outs[i], ins[j])) return SSD_ERR_ALIASING;
        }
        for (int j = i + 1; j < 4; ++j)
            if (overlaps(outs[i], outs[j])) return SSD_ERR_ALIASING;
    }
    if (a->rows == 0) {
        if (a->dweight)
            hipLaunchKernelGGL(k_rms_zero, dim3((unsigned)ceil_div(a->dim, kThreads)), dim3(kThreads), 0, st, a->dweight, (int)a->dim);
        return launched();
    }
    const bool bf = a->dtype == SSD_DTYPE_BF16, rbf = a->residual_dtype == SSD_DTYPE_BF16;
    if (bf && rbf) bwd_typed<bf16, bf16>(a, st);
    else if (bf) bwd_typed<bf16, float>(a, st);
    else if (rbf) bwd_typed<float, bf16>(a, st);
    else bwd_typed<float, float>(a, st);
    return launched();
}

}  // extern "C"
