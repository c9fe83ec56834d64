// mm_api.hip -- host side of the 8-bit block-scaled matrix product (ssd_matmul_fp8 in
// include/ssd.h).  Validation is host-only and runs before any HIP call; nothing here
// allocates, frees or synchronises.
#include "ssd.h"

#include <hip/hip_runtime.h>

#include <cstdint>

#include "api_checks.hpp"
#include "mm_kernels.hpp"

using namespace ssd;
using namespace ssd::mm;

namespace {

ssd_status launched() { return hipGetLastError() == hipSuccess ? SSD_OK : SSD_ERR_HIP; }

constexpr int64_t kMaxInner = (int64_t)1 << 22;   // a tile's rows are addressed in 31 bits
constexpr int64_t kMaxSide = ((int64_t)1 << 31) - 512;

struct Plan {
    int bm;              // rows of a tile
    bool few;
    int64_t tm, tn, kb, per, shares;
};
Plan plan_of(int64_t m, int64_t n, int64_t k)
{
    Plan p{};
    p.kb = ceil_div(k, kBlock);
    p.per = p.kb;
    p.shares = 1;
    if (m == 0 || n == 0) return p;   // no tiles
    auto tiles = [&](int bm, int bn) {
        p.bm = bm;
        p.tm = ceil_div(m, bm);
        p.tn = ceil_div(n, bn);
        return p.tm * p.tn;
    };
    // tiles of 128 where they keep a quarter of the CUs busy, or where the other form could not share k out further.  400 x 2560
    // of k = 2560, 80 tiles: 25 us so, 36 in the other form; 640 x 1280, 50 tiles: 24 against 19, and of k = 512 8 against 11
    if (m > 64 && (tiles(128, 128) >= 64 || p.kb <= 4)) return p;
    p.few = true;
    const int64_t groups = tiles(m <= 16 ? 16 : m <= 32 ? 32 : 64, 64);
    // where the tiles are too few to keep half of the CUs loading, k is shared out over workgroups, at least four blocks
    // each
    const int64_t want = groups >= 128 ? 1 : ceil_div(256, groups), most = ceil_div(p.kb, 4);
    const int64_t shares = want < most ? want : most;
    p.per = ceil_div(p.kb, shares);
    p.shares = ceil_div(p.kb, p.per);
    return p;
}
size_t bytes_of(const Plan &p, int64_t m, int64_t n) { return p.shares > 1 ? (size_t)(p.shares * m * n) * 4 : 0; }

ssd_status check_dims(const ssd_matmul_fp8_args *a, Plan *p)
{
    if (!a) return SSD_ERR_NULL_POINTER;
    if (!known_dtype(a->dtype)) return SSD_ERR_BAD_DTYPE;
    constexpr int64_t most = (int64_t)1 << 40;
    if (a->m < 0 || a->n < 0 || a->k < 1 || a->k % 16 != 0 || a->m > kMaxSide || a->n > kMaxSide || a->k > kMaxInner) return SSD_ERR_BAD_SHAPE;
    if (a->m * a->k > most || a->n * a->k > most || (a->m > 0 && a->n > most / a->m)) return SSD_ERR_BAD_SHAPE;
    *p = plan_of(a->m, a->n, a->k);
    if (p->tm > 0 && p->tn > 0 && p->tm > (p->few ? kMaxGroups / 2 / p->shares : INT32_MAX / 2) / p->tn) return SSD_ERR_BAD_SHAPE;
    return SSD_OK;
}

template <typename O> void run(const ssd_matmul_fp8_args *a, const Plan &p, hipStream_t st)
{
    MmArgs k{};
    k.a = static_cast<const uint8_t *>(a->a);
    k.w = static_cast<const uint8_t *>(a->w);
    k.as = a->a_scales;
    k.ws = a->w_scales;
    k.bias = a->bias;
    k.out = a->out;
    k.part = static_cast<float *>(a->workspace);
    k.m = (int)a->m;
    k.n = (int)a->n;
    k.k = (int)a->k;
    k.kb = (int)p.kb;
    k.per = (int)p.per;
    k.tm = (int)p.tm;
    k.tn = (int)p.tn;
    const dim3 grid((unsigned)(p.tm * p.tn * p.shares));
    if (!p.few) {
        auto tile = [&](auto whole) {
            constexpr bool WHOLE = decltype(whole)::value;
            // workgroups: what the card holds at a time (LDS: two a CU)
            hipLaunchKernelGGL((k_mm_tile<O, WHOLE>), dim3((unsigned)(p.tm * p.tn < 512 ? p.tm * p.tn : 512)), dim3(256), 0, st, k);
        };
        // such a tile is addressed in 31 bits
        if (std::is_same<O, bf16>::value && a->n % 8 == 0 && a->n <= (int64_t)1 << 21) {
            if constexpr (std::is_same<O, bf16>::value) tile(std::true_type{});
        } else tile(std::false_type{});
        return;
    }
    auto few = [&](auto mi) {
        constexpr int MI = decltype(mi)::value;
        if (p.shares > 1) hipLaunchKernelGGL((k_mm_few<O, MI, true>), grid, dim3(512), 0, st, k);
        else hipLaunchKernelGGL((k_mm_few<O, MI, false>), grid, dim3(512), 0, st, k);
    };
    if (p.bm == 16) few(std::integral_constant<int, 1>{});
    else if (p.bm == 32) few(std::integral_constant<int, 2>{});
    else few(std::integral_constant<int, 4>{});
    if (p.shares == 1) return;
    const int64_t mn = a->m * a->n;
    auto join = [&](auto v) {
        constexpr int V = decltype(v)::value;
        hipLaunchKernelGGL((k_mm_join<O, V>), dim3((unsigned)ceil_div(mn, kThreads * V)), dim3(kThreads), 0, st, (const float *)k.part,
                           a->bias, (O *)a->out, mn, (int)a->n, (int)p.shares);
    };
    if (a->n % 4 == 0) join(std::integral_constant<int, 4>{});
    else join(std::integral_constant<int, 1>{});
}

}  // namespace

extern "C" {

ssd_status ssd_matmul_fp8_workspace_size(const ssd_matmul_fp8_args *a, size_t *bytes)
{
    Plan p;
    const ssd_status r = check_dims(a, &p);
    if (r != SSD_OK) return r;
    if (!bytes) return SSD_ERR_NULL_POINTER;
    *bytes = a->m > 0 && a->n > 0 ? bytes_of(p, a->m, a->n) : 0;
    return SSD_OK;
}

ssd_status ssd_matmul_fp8(const ssd_matmul_fp8_args *a, void *stream)
{
    Plan p;
    const ssd_status r = check_dims(a, &p);
    if (r != SSD_OK) return r;
    if (a->m == 0 || a->n == 0) return SSD_OK;
    if (!a->a || !a->a_scales || !a->w || !a->w_scales || !a->out) return SSD_ERR_NULL_POINTER;
    const void *ptrs[] = {a->a, a->w, a->out, a->workspace};
    for (const void *q : ptrs)
        if (!aligned_to(q, 16)) return SSD_ERR_MISALIGNED;
    if (!aligned_to(a->a_scales, 4) || !aligned_to(a->w_scales, 4) || !aligned_to(a->bias, 4)) return SSD_ERR_MISALIGNED;
    const size_t need = bytes_of(p, a->m, a->n);
    if (need > 0 && !a->workspace) return SSD_ERR_NULL_POINTER;
    if (a->workspace_bytes < need) return SSD_ERR_WORKSPACE_TOO_SMALL;
    const Range ins[] = {{a->a, (size_t)(a->m * a->k)}, {a->w, (size_t)(a->n * a->k)}, {a->a_scales, (size_t)(a->m * p.kb) * 4},
                         {a->w_scales, (size_t)(ceil_div(a->n, kBlock) * p.kb) * 4}, {a->bias, (size_t)a->n * 4}};
    const Range outs[] = {{a->out, (size_t)(a->m * a->n) * elem_size(a->dtype)}, {need ? a->workspace : nullptr, need}};
    if (!apart(ins, outs)) return SSD_ERR_ALIASING;
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (a->dtype == SSD_DTYPE_BF16) run<bf16>(a, p, st);
    else run<float>(a, p, st);
    return launched();
}

}  // extern "C"
