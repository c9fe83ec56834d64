// conv_api.hip -- host side of the causal convolution with a carried window
// (ssd_causal_conv_* in include/ssd.h).  Validation is host-only and runs before any
// HIP call; nothing here allocates, frees or synchronises.
#include "ssd.h"

#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

#include "api_checks.hpp"
#include "conv_kernels.hpp"

using namespace ssd;
using namespace ssd::conv;

namespace {

ssd_status launched() { return hipGetLastError() == hipSuccess ? SSD_OK : SSD_ERR_HIP; }

constexpr int64_t kMaxWidth = (int64_t)1 << 22, kMaxStride = (int64_t)1 << 31;

struct Shape {
    int64_t b, T, C, K, rows, tokens;
    int dtype;
    size_t esz;
    bool packed;
};
ssd_status check_dims(int64_t b, int64_t C, int64_t K, int dtype, int64_t stride)
{
    if (!known_dtype(dtype)) return SSD_ERR_BAD_DTYPE;
    if (b < 1 || C < 1 || C > kMaxWidth || K < 1 || K > 4 || (stride != 0 && (stride < C || stride >= kMaxStride)))
        return SSD_ERR_BAD_SHAPE;
    return SSD_OK;
}
ssd_status parse_shape(const ssd_causal_conv_args *a, Shape *s)
{
    if (!a) return SSD_ERR_NULL_POINTER;
    const ssd_status r = check_dims(a->batch, a->dim, a->width, a->dtype, a->x_stride);
    if (r != SSD_OK) return r;
    constexpr int64_t most = ((int64_t)1 << 31) - 64;
    if (a->seqlen < 0 || a->seqlen >= most || a->batch >= most || a->batch * a->seqlen >= most) return SSD_ERR_BAD_SHAPE;
    if (a->seq_idx && (a->batch != 1 || a->nseq < 1 || a->nseq > ((int64_t)1 << 30))) return SSD_ERR_SEQ_IDX;
    s->b = a->batch;
    s->T = a->seqlen;
    s->C = a->dim;
    s->K = a->width;
    s->packed = a->seq_idx != nullptr;
    s->rows = s->packed ? a->nseq : s->b;
    s->tokens = s->b * s->T;
    s->dtype = a->dtype;
    s->esz = elem_size(a->dtype);
    // a thread an element of a strip of 16 tokens at least, and one a window's element, in one launch
    if (s->b * ceil_div(s->T, kFwdStrip) + s->rows * (s->K - 1) > (kMaxGroups - 2) * kThreads / s->C) return SSD_ERR_BAD_SHAPE;
    return SSD_OK;
}
size_t span(int64_t tokens, int64_t stride, int64_t width, size_t esz)
{
    return tokens > 0 ? (size_t)((tokens - 1) * (stride ? stride : width) + width) * esz : 0;
}
// Tokens of a strip of the backward: its sums over tokens are one row of width + 1 fp32 numbers,
// written and read again, so long strips where there are threads enough (16384 tokens of 5120
// channels: 64 tokens 141 us, 128 tokens 151 us, with half the sums but half the threads).
int64_t bwd_strip(const Shape &s)
{
    for (int64_t strip = 64; strip > 16; strip /= 2)
        if (s.b * ceil_div(s.T, strip) * s.C >= (int64_t)4 * 131072) return strip;
    return 16;
}
size_t bwd_bytes(const Shape &s) { return (size_t)(s.b * ceil_div(s.T, bwd_strip(s)) * (s.K + 1) * s.C) * 4; }

ConvArgs conv_args(const Shape &s, const ssd_causal_conv_args *a, int64_t strip)
{
    ConvArgs k{};
    k.x = a->x;
    k.xs = a->x_stride ? a->x_stride : s.C;
    k.w = a->weight;
    k.bias = a->bias;
    k.win0 = a->initial_window;
    k.ids = a->seq_idx;
    k.T = (int)s.T;
    k.C = (int)s.C;
    k.rows = (int)s.rows;
    k.strip = (int)strip;
    k.nb = (int)ceil_div(s.T, strip);
    k.silu = a->silu != 0;
    return k;
}
template <int N> using Int = std::integral_constant<int, N>;
template <typename F> void with_width(int64_t K, F &&f)
{
    if (K == 1) f(Int<1>{});
    else if (K == 2) f(Int<2>{});
    else if (K == 3) f(Int<3>{});
    else f(Int<4>{});
}
// E, vector width, taps and packing of a call.  Four elements to a thread in both types: 16
// bytes of bf16 take twice the registers (packed prompts of 18 K tokens, 5120 channels: 110
// against 97 us; gradients of 16384 tokens: 283 against 141 us, at one wave a SIMD).
template <typename F> void dispatch(const Shape &s, F &&f)
{
    with_width(s.K, [&](auto kw) {
        auto typed = [&](auto e) {
            auto packed = [&](auto v) {
                if (s.packed) f(e, v, kw, std::true_type{});
                else f(e, v, kw, std::false_type{});
            };
            if (s.C >= 4) packed(Int<4>{});
            else packed(Int<1>{});
        };
        if (s.dtype == SSD_DTYPE_BF16) typed(bf16{});
        else typed(float{});
    });
}

// Workgroups of a launch for V channels a thread: the strips', and in front of them, if windows go out, those of the windows of a packed
// stream's segments without tokens.
unsigned groups_of(const Shape &s, ConvArgs &k, int V, bool windows)
{
    const int64_t gv = ceil_div(s.C, V);
    k.items = s.b * k.nb * gv;
    k.ahead = s.packed && windows ? (int)ceil_div(s.rows * gv, kThreads) : 0;
    return (unsigned)(k.ahead + ceil_div(k.items, kThreads));
}

void keep(const Shape &s, const void *from, void *to, hipStream_t st)
{
    const int64_t n = s.rows * (s.K - 1) * s.C;
    if (!to || n == 0) return;
    const dim3 grid((unsigned)ceil_div(n, kThreads)), block(kThreads);
    if (s.dtype == SSD_DTYPE_BF16) hipLaunchKernelGGL(k_conv_keep<bf16>, grid, block, 0, st, (const bf16 *)from, (bf16 *)to, n);
    else hipLaunchKernelGGL(k_conv_keep<float>, grid, block, 0, st, (const float *)from, (float *)to, n);
}

ssd_status check_inputs(const Shape &s, const ssd_causal_conv_args *a)
{
    if (!a->weight || (s.tokens > 0 && !a->x)) return SSD_ERR_NULL_POINTER;
    if (!aligned_to(a->x, s.esz) || !aligned_to(a->initial_window, s.esz) || !aligned_to(a->weight, 4) || !aligned_to(a->bias, 4) ||
        !aligned_to(a->seq_idx, 4))
        return SSD_ERR_MISALIGNED;
    return SSD_OK;
}

}  // namespace

extern "C" {

ssd_status ssd_causal_conv_fwd(const ssd_causal_conv_args *a, void *stream)
{
    Shape s;
    ssd_status r = parse_shape(a, &s);
    if (r != SSD_OK) return r;
    if ((r = check_inputs(s, a)) != SSD_OK) return r;
    if (s.tokens > 0 && !a->y) return SSD_ERR_NULL_POINTER;
    if (!aligned_to(a->y, s.esz) || !aligned_to(a->final_window, s.esz)) return SSD_ERR_MISALIGNED;
    const size_t win = (size_t)(s.rows * (s.K - 1) * s.C) * s.esz;
    const Range ins[] = {{a->x, span(s.tokens, a->x_stride, s.C, s.esz)}, {a->weight, (size_t)(s.C * s.K) * 4}, {a->bias, (size_t)s.C * 4},
                         {a->initial_window, win}, {a->seq_idx, s.packed ? (size_t)s.T * 4 : 0}};
    const Range outs[] = {{a->y, span(s.tokens, 0, s.C, s.esz)}, {a->final_window, win}};
    if (!apart(ins, outs)) return SSD_ERR_ALIASING;
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (s.T == 0) {
        keep(s, a->initial_window, a->final_window, st);
        return launched();
    }
    ConvArgs k = conv_args(s, a, kFwdStrip);
    k.y = a->y;
    k.win1 = s.K > 1 ? a->final_window : nullptr;
    dispatch(s, [&](auto e, auto v, auto kw, auto packed) {
        constexpr int V = decltype(v)::value;
        const unsigned groups = groups_of(s, k, V, k.win1 != nullptr);
        hipLaunchKernelGGL((k_conv_fwd<decltype(e), V, decltype(kw)::value, decltype(packed)::value>), dim3(groups), dim3(kThreads), 0, st, k);
    });
    return launched();
}

ssd_status ssd_causal_conv_bwd_workspace_size(const ssd_causal_conv_args *a, size_t *bytes)
{
    Shape s;
    const ssd_status r = parse_shape(a, &s);
    if (r != SSD_OK) return r;
    if (!bytes) return SSD_ERR_NULL_POINTER;
    *bytes = bwd_bytes(s);
    return SSD_OK;
}

ssd_status ssd_causal_conv_bwd(const ssd_causal_conv_args *a, const ssd_causal_conv_bwd_args *g, void *stream)
{
    Shape s;
    ssd_status r = parse_shape(a, &s);
    if (r != SSD_OK) return r;
    if (!g) return SSD_ERR_NULL_POINTER;
    if ((r = check_inputs(s, a)) != SSD_OK) return r;
    if (!g->dweight || (s.tokens > 0 && (!g->dy || !g->dx))) return SSD_ERR_NULL_POINTER;
    const void *els[] = {g->dy, g->dfinal_window, g->dx, g->dinitial_window};
    for (const void *p : els)
        if (!aligned_to(p, s.esz)) return SSD_ERR_MISALIGNED;
    if (!aligned_to(g->dweight, 4) || !aligned_to(g->dbias, 4) || !aligned_to(g->workspace, 16)) return SSD_ERR_MISALIGNED;
    const size_t need = bwd_bytes(s);
    if (need > 0 && !g->workspace) return SSD_ERR_NULL_POINTER;
    if (g->workspace_bytes < need) return SSD_ERR_WORKSPACE_TOO_SMALL;
    const size_t win = (size_t)(s.rows * (s.K - 1) * s.C) * s.esz, par = (size_t)(s.C * s.K) * 4, tok = span(s.tokens, 0, s.C, s.esz);
    const Range ins[] = {{a->x, span(s.tokens, a->x_stride, s.C, s.esz)}, {a->weight, par}, {a->bias, (size_t)s.C * 4},
                         {a->initial_window, win}, {a->seq_idx, s.packed ? (size_t)s.T * 4 : 0}, {g->dy, tok}, {g->dfinal_window, win}};
    const Range outs[] = {{g->dx, tok}, {g->dweight, par}, {g->dbias, (size_t)s.C * 4}, {g->dinitial_window, win},
                          {need ? g->workspace : nullptr, need}};
    if (!apart(ins, outs)) return SSD_ERR_ALIASING;
    hipStream_t st = static_cast<hipStream_t>(stream);
    ConvArgs k = conv_args(s, a, bwd_strip(s));
    k.dy = g->dy;
    k.dx = g->dx;
    k.dwin1 = s.K > 1 ? g->dfinal_window : nullptr;
    k.dwin0 = s.K > 1 ? g->dinitial_window : nullptr;
    k.parts = static_cast<float *>(g->workspace);
    if (s.T == 0) keep(s, g->dfinal_window, g->dinitial_window, st);
    else {
        dispatch(s, [&](auto e, auto v, auto kw, auto packed) {
            constexpr int V = decltype(v)::value;
            const unsigned groups = groups_of(s, k, V, k.dwin0 != nullptr);
            hipLaunchKernelGGL((k_conv_bwd<decltype(e), V, decltype(kw)::value, decltype(packed)::value>), dim3(groups), dim3(kThreads), 0, st, k);
        });
    }
    hipLaunchKernelGGL(k_conv_sum, dim3((unsigned)ceil_div((s.K + 1) * s.C, 32)), dim3(1024), 0, st, (const float *)k.parts, g->dweight,
                       g->dbias, (int)(s.b * k.nb), (int)s.C, (int)s.K);
    return launched();
}

ssd_status ssd_causal_conv_step(const ssd_causal_conv_step_args *a, void *stream)
{
    if (!a) return SSD_ERR_NULL_POINTER;
    const ssd_status r = check_dims(a->batch, a->dim, a->width, a->dtype, a->x_stride);
    if (r != SSD_OK) return r;
    if (a->batch > kMaxGroups * kThreads / a->dim) return SSD_ERR_BAD_SHAPE;
    if (!a->x || !a->weight || !a->y || (a->width > 1 && !a->window)) return SSD_ERR_NULL_POINTER;
    Shape s{};
    s.b = a->batch;
    s.C = a->dim;
    s.K = a->width;
    s.dtype = a->dtype;
    s.esz = elem_size(a->dtype);
    if (!aligned_to(a->x, s.esz) || !aligned_to(a->window, s.esz) || !aligned_to(a->y, s.esz) || !aligned_to(a->weight, 4) ||
        !aligned_to(a->bias, 4))
        return SSD_ERR_MISALIGNED;
    const Range ins[] = {{a->x, span(s.b, a->x_stride, s.C, s.esz)}, {a->weight, (size_t)(s.C * s.K) * 4}, {a->bias, (size_t)s.C * 4}};
    const Range outs[] = {{a->window, (size_t)(s.b * (s.K - 1) * s.C) * s.esz}, {a->y, span(s.b, 0, s.C, s.esz)}};
    if (!apart(ins, outs)) return SSD_ERR_ALIASING;
    hipStream_t st = static_cast<hipStream_t>(stream);
    const int64_t xs = a->x_stride ? a->x_stride : s.C;
    const bool vec = s.C % 4 == 0;   // the window is moved in place: no element may be two threads'
    with_width(s.K, [&](auto kw) {
        constexpr int K = decltype(kw)::value;
        auto launch = [&](auto e, auto v) {
            using E = decltype(e);
            constexpr int V = decltype(v)::value;
            const int64_t items = s.b * (s.C / V);
            hipLaunchKernelGGL((k_conv_step<E, V, K>), dim3((unsigned)ceil_div(items, kThreads)), dim3(kThreads), 0, st,
                               (const E *)a->x, xs, a->weight, a->bias, (E *)a->window, (E *)a->y, items, (int)s.C, a->silu != 0);
        };
        auto typed = [&](auto e) {
            if (vec) launch(e, Int<4>{});
            else launch(e, Int<1>{});
        };
        if (s.dtype == SSD_DTYPE_BF16) typed(bf16{});
        else typed(float{});
    });
    return launched();
}

}  // extern "C"
