// norm_api.hip -- host side of layer norm (ssd_layer_norm_* in include/ssd.h).
// Validation is host-only and runs before any HIP call; nothing here allocates,
// frees or synchronises.
#include "ssd.h"

#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

#include "norm_kernels.hpp"

using namespace ssd;
using namespace ssd::norm;

namespace {

struct Range {
    const void *p;
    size_t n;
};
bool overlaps(Range a, Range b)
{
    if (!a.p || !b.p || a.n == 0 || b.n == 0) return false;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
    return a0 < b0 + b.n && b0 < a0 + a.n;
}
bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
ssd_status launched() { return hipGetLastError() == hipSuccess ? SSD_OK : SSD_ERR_HIP; }

constexpr int64_t kMaxNormDim = 65536;

ssd_status check_dims(int64_t rows, int64_t dim, int dtype)
{
    if (dtype != SSD_DTYPE_F32 && dtype != SSD_DTYPE_BF16) return SSD_ERR_BAD_DTYPE;
    // rows are counted in 31 bits
    if (rows < 0 || dim < 1 || dim > kMaxNormDim || rows > INT32_MAX || rows > ((int64_t)1 << 40) / dim)
        return SSD_ERR_BAD_SHAPE;
    return SSD_OK;
}

// Rows of one launch: at up to 1024 threads each, fewer than 2^32 threads.
constexpr int64_t kLaunchRows = (int64_t)1 << 21;

// How a row of `dim` is held: vector width, lanes per row and vectors per lane (0:
// longer than the registers).
struct Plan {
    int V, L, IT;
};
Plan plan_of(int64_t dim, int dtype)
{
    const int full = dtype == SSD_DTYPE_BF16 ? 8 : 4;
    Plan p;
    p.V = dim % full == 0 ? full : 1;
    const int64_t nv = dim / p.V;
    auto pick = [&](int L, const int *its, int n) {
        for (int i = 0; i < n; ++i)
            if (nv <= (int64_t)L * its[i]) {
                p.L = L;
                p.IT = its[i];
                return true;
            }
        return false;
    };
    const int a[] = {1, 2}, b[] = {1, 2, 3, 5}, c[] = {2, 3, 5, 8};
    if (pick(16, a, 2) || pick(64, b, 4) || pick(256, c, 4)) return p;
    p.L = 0;
    p.IT = 0;
    return p;
}

// Rows per workgroup of the backward: as many workgroups (strips) as keep every CU loading,
// few enough that the rows of partial sums stay a small part of the traffic.  512 for rows of
// 2 KB and more and for fp32; bf16 rows that are shorter, or read by single elements, keep
// few bytes in flight per workgroup and take 1024.  2^26 elements in us, 512 against 1024:
// bf16 dim 64 131, 106; 320 114, 95; 1531 142, 109; 1024 77, 82; 5120 78, 86; fp32 320 149, 151.
int64_t strip_of(const Plan &p, int64_t rows, int64_t dim, int dtype)
{
    const bool few = dtype == SSD_DTYPE_BF16 && p.L != 0 && (p.V == 1 || dim < 1024);
    const int64_t strips = few ? 1024 : 512, groups = p.L ? kThreads / p.L : 1;
    const int64_t s = (rows + strips - 1) / strips;
    return (s + groups - 1) / groups * groups;
}

template <int N> using Int = std::integral_constant<int, N>;

template <typename E, typename F> void with_plan(const Plan &p, F &&f)
{
    constexpr int FULL = kVec16<E>;
    auto it = [&](auto v, auto l) {
        if constexpr (decltype(l)::value == 16) {
            if (p.IT == 1) f(v, l, Int<1>{});
            else f(v, l, Int<2>{});
        } else if constexpr (decltype(l)::value == 64) {
            if (p.IT == 1) f(v, l, Int<1>{});
            else if (p.IT == 2) f(v, l, Int<2>{});
            else if (p.IT == 3) f(v, l, Int<3>{});
            else f(v, l, Int<5>{});
        } else {
            if (p.IT == 2) f(v, l, Int<2>{});
            else if (p.IT == 3) f(v, l, Int<3>{});
            else if (p.IT == 5) f(v, l, Int<5>{});
            else f(v, l, Int<8>{});
        }
    };
    auto lanes = [&](auto v) {
        if (p.L == 16) it(v, Int<16>{});
        else if (p.L == 64) it(v, Int<64>{});
        else it(v, Int<256>{});
    };
    if (p.V == 1) lanes(Int<1>{});
    else lanes(Int<FULL>{});
}

template <typename E> ssd_status run_fwd(const ssd_norm_args *a, hipStream_t st)
{
    const int dim = (int)a->dim;
    const Plan p = plan_of(a->dim, a->dtype);
    for (int64_t r0 = 0; r0 < a->rows; r0 += kLaunchRows) {
        const int64_t rows = a->rows - r0 < kLaunchRows ? a->rows - r0 : kLaunchRows;
        const E *x = (const E *)a->x + r0 * dim;
        E *y = (E *)a->y + r0 * dim;
        float *mean = a->mean ? a->mean + r0 : nullptr, *rstd = a->rstd ? a->rstd + r0 : nullptr;
        if (p.L == 0) {
            hipLaunchKernelGGL(k_norm_fwd_long<E>, dim3((unsigned)rows), dim3(kLongThreads), 0, st, x, a->weight, a->bias, y,
                               mean, rstd, dim, a->eps);
            continue;
        }
        with_plan<E>(p, [&](auto v, auto l, auto it) {
            constexpr int L = decltype(l)::value;
            // few rows: a wave per workgroup, so they spread over the CUs
            const int threads = L == 256 ? 256 : rows * L <= 64 * 1024 ? 64 : kThreads;
            const int64_t per = threads / L;
            hipLaunchKernelGGL((k_norm_fwd<E, decltype(v)::value, L, decltype(it)::value>),
                               dim3((unsigned)((rows + per - 1) / per)), dim3(threads), 0, st, x, a->weight, a->bias, y, mean,
                               rstd, rows, dim, a->eps);
        });
    }
    return launched();
}

template <typename E> ssd_status run_bwd(const ssd_norm_bwd_args *a, hipStream_t st)
{
    const int dim = (int)a->dim;
    const bool sums = a->dweight || a->dbias;
    float *parts = static_cast<float *>(a->workspace);
    const Plan p = plan_of(a->dim, a->dtype);
    const int64_t strip = strip_of(p, a->rows, a->dim, a->dtype);
    const int64_t blocks = (a->rows + strip - 1) / strip;
    if (p.L == 0) {
        if (sums)   // before dx, which may be dy
            hipLaunchKernelGGL(k_norm_cols_long<E>, dim3((unsigned)blocks, (unsigned)((dim + kThreads - 1) / kThreads)),
                               dim3(kThreads), 0, st, (const E *)a->x, (const E *)a->dy, a->mean, a->rstd, parts, a->rows,
                               dim, (int)strip);
        for (int64_t r0 = 0; r0 < a->rows; r0 += kLaunchRows) {
            const int64_t rows = a->rows - r0 < kLaunchRows ? a->rows - r0 : kLaunchRows;
            hipLaunchKernelGGL(k_norm_dx_long<E>, dim3((unsigned)rows), dim3(kLongThreads), 0, st, (const E *)a->x + r0 * dim,
                               (const E *)a->dy + r0 * dim, a->mean + r0, a->rstd + r0, a->weight, (E *)a->dx + r0 * dim, dim);
        }
    } else {
        with_plan<E>(p, [&](auto v, auto l, auto it) {
            auto launch = [&](auto kern) {
                hipLaunchKernelGGL(kern, dim3((unsigned)blocks), dim3(kThreads), 0, st, (const E *)a->x,
                                   (const E *)a->dy, a->mean, a->rstd, a->weight, (E *)a->dx, parts, a->rows, dim,
                                   (int)strip);
            };
            constexpr int V = decltype(v)::value, L = decltype(l)::value, IT = decltype(it)::value;
            if (sums) launch(k_norm_bwd<E, V, L, IT, true>);
            else launch(k_norm_bwd<E, V, L, IT, false>);
        });
    }
    if (sums)
        hipLaunchKernelGGL(k_norm_sum, dim3((unsigned)((2 * dim + 31) / 32)), dim3(1024), 0, st, (const float *)parts,
                           a->dweight, a->dbias, (int)blocks, dim);
    return launched();
}

}  // namespace

extern "C" {

ssd_status ssd_layer_norm_fwd(const ssd_norm_args *a, void *stream)
{
    if (!a) return SSD_ERR_NULL_POINTER;
    const ssd_status r = check_dims(a->rows, a->dim, a->dtype);
    if (r != SSD_OK) return r;
    if (a->rows == 0) return SSD_OK;
    if (!a->x || !a->y) return SSD_ERR_NULL_POINTER;
    const void *ptrs[] = {a->x, a->weight, a->bias, a->y};
    for (const void *p : ptrs)
        if (!aligned16(p)) return SSD_ERR_MISALIGNED;
    if (!aligned4(a->mean) || !aligned4(a->rstd)) return SSD_ERR_MISALIGNED;
    const size_t n = (size_t)(a->rows * a->dim) * (a->dtype == SSD_DTYPE_BF16 ? 2 : 4), d = (size_t)a->dim * 4,
                 s = (size_t)a->rows * 4;
    const Range ins[] = {{a->x, n}, {a->weight, d}, {a->bias, d}};
    const Range outs[] = {{a->y, n}, {a->mean, s}, {a->rstd, s}};
    for (int i = 0; i < 3; ++i) {
        for (const Range &in : ins)
            if (overlaps(outs[i], in) && !(i == 0 && in.p == a->x && a->y == a->x)) return SSD_ERR_ALIASING;
        for (int j = i + 1; j < 3; ++j)
            if (overlaps(outs[i], outs[j])) return SSD_ERR_ALIASING;
    }
    hipStream_t st = static_cast<hipStream_t>(stream);
    return a->dtype == SSD_DTYPE_BF16 ? run_fwd<bf16>(a, st) : run_fwd<float>(a, st);
}

ssd_status ssd_layer_norm_bwd_workspace_size(const ssd_norm_bwd_args *a, size_t *bytes)
{
    if (!a) return SSD_ERR_NULL_POINTER;
    const ssd_status r = check_dims(a->rows, a->dim, a->dtype);
    if (r != SSD_OK) return r;
    if (!bytes) return SSD_ERR_NULL_POINTER;
    const Plan p = plan_of(a->dim, a->dtype);
    const int64_t strip = strip_of(p, a->rows, a->dim, a->dtype);
    *bytes = a->rows ? (size_t)((a->rows + strip - 1) / strip) * 2 * (size_t)a->dim * 4 : 0;
    return SSD_OK;
}

ssd_status ssd_layer_norm_bwd(const ssd_norm_bwd_args *a, void *stream)
{
    size_t need = 0;
    const ssd_status r = ssd_layer_norm_bwd_workspace_size(a, &need);
    if (r != SSD_OK) return r;
    hipStream_t st = static_cast<hipStream_t>(stream);
    const void *ptrs[] = {a->x, a->dy, a->weight, a->dx, a->dweight, a->dbias, a->workspace};
    for (const void *p : ptrs)
        if (!aligned16(p)) return SSD_ERR_MISALIGNED;
    if (!aligned4(a->mean) || !aligned4(a->rstd)) return SSD_ERR_MISALIGNED;
    const bool sums = a->dweight || a->dbias;
    if (a->rows > 0) {
        if (!a->x || !a->dy || !a->mean || !a->rstd || !a->dx) return SSD_ERR_NULL_POINTER;
        if (sums && !a->workspace) return SSD_ERR_NULL_POINTER;
        if (sums && a->workspace_bytes < need) return SSD_ERR_WORKSPACE_TOO_SMALL;
    }
    const size_t n = (size_t)(a->rows * a->dim) * (a->dtype == SSD_DTYPE_BF16 ? 2 : 4), d = (size_t)a->dim * 4,
                 s = (size_t)a->rows * 4;
    const Range ins[] = {{a->x, n}, {a->dy, n}, {a->mean, s}, {a->rstd, s}, {a->weight, d}};
    const Range outs[] = {{a->dx, n}, {a->dweight, d}, {a->dbias, d}, {sums ? a->workspace : nullptr, need}};
    for (int i = 0; i < 4; ++i) {
        for (const Range &in : ins)
            if (overlaps(outs[i], in) && !(i == 0 && in.p == a->dy && a->dx == a->dy)) return SSD_ERR_ALIASING;
        for (int j = i + 1; j < 4; ++j)
            if (overlaps(outs[i], outs[j])) return SSD_ERR_ALIASING;
    }
    if (a->rows == 0) {
        if (sums)
            hipLaunchKernelGGL(k_norm_zero, dim3((unsigned)((a->dim + kThreads - 1) / kThreads)), dim3(kThreads), 0, st,
                               a->dweight, a->dbias, (int)a->dim);
        return launched();
    }
    return a->dtype == SSD_DTYPE_BF16 ? run_bwd<bf16>(a, st) : run_bwd<float>(a, st);
}

}  // extern "C"
