// scan_api.hip -- host side of the selective scan (ssd_selective_scan_* in include/ssd.h):
// argument validation, workspace layout and launches.  Validation is host-only and
// runs before any HIP call; nothing here allocates, frees or synchronises.
#include "ssd.h"

#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

#include "api_checks.hpp"
#include "scan_kernels.hpp"

using namespace ssd;
using namespace ssd::sscan;

namespace {

ssd_status launched() { return hipGetLastError() == hipSuccess ? SSD_OK : SSD_ERR_HIP; }

constexpr int64_t kMaxWidth = (int64_t)1 << 20;
constexpr int64_t kMaxStride = (int64_t)1 << 22;       // tiles of tokens are addressed in 31 bits
constexpr int64_t kMaxStepStride = (int64_t)1 << 36;   // single tokens in 64

struct Shape {
    int64_t b, T, D, N, G, nseq;
    int64_t rows;       // batch rows or segments
    int64_t tokens;     // b T
    int64_t per, bpg, nblk;   // channels of a group, tiles of channels of a group and in all
    int LN, dtype;
    size_t esz;
    bool packed;
};
struct Chunking {
    int lq;             // log2 of the chunk
    int64_t nch, slots;
    int64_t limit;      // packed: rows up to this long are not cut
    bool cut;           // whether rows may be cut at all
};

int lanes_of(int64_t N) { return N <= 4 ? 1 : N <= 8 ? 2 : N <= 16 ? 4 : N <= 32 ? 8 : 16; }

ssd_status check_dims(int64_t b, int64_t D, int64_t N, int64_t G, int dtype, Shape *s)
{
    if (!known_dtype(dtype)) return SSD_ERR_BAD_DTYPE;
    if (b < 1 || D < 1 || N < 1 || G < 1 || D > kMaxWidth || N > 64 || G > kMaxWidth || G * N > kMaxWidth) return SSD_ERR_BAD_SHAPE;
    if (D % G != 0) return SSD_ERR_GROUPS;
    s->b = b;
    s->D = D;
    s->N = N;
    s->G = G;
    s->LN = lanes_of(N);
    s->per = D / G;
    s->bpg = ceil_div(s->per, kThreads / s->LN);
    s->nblk = G * s->bpg;
    s->dtype = dtype;
    s->esz = elem_size(dtype);
    return SSD_OK;
}

// Chunks of the forward.  Rows are cut where their waves would not fill the card; a cut row
// costs its tokens' exponentials twice.
Chunking fwd_chunks(const Shape &s)
{
    Chunking c{};
    const int64_t waves = s.nblk * 4, want = 4096;
    int lq = 6;
    while (lq < 28 && waves * (s.packed ? ceil_div(s.T, (int64_t)1 << lq) : s.b * ceil_div(s.T, (int64_t)1 << lq)) > want) ++lq;
    c.lq = lq;
    if (s.packed) {
        c.cut = s.T > ((int64_t)1 << lq);
        const int64_t share = waves * s.T / 1024;   // tokens a SIMD has if all share alike
        c.limit = share > 128 ? share : 128;
        if (c.limit > s.T) c.cut = false;
    } else {
        c.cut = s.b * waves < 1024 && s.T > 128 && s.T > ((int64_t)1 << lq);
    }
    if (!c.cut) c.lq = kUncut;
    c.nch = s.T > 0 ? ceil_div(s.T, (int64_t)1 << c.lq) : 1;
    c.slots = s.packed ? (c.cut ? (s.T >> c.lq) : 0) + s.nseq : s.b * c.nch;
    return c;
}
Chunking bwd_chunks(const Shape &s)
{
    Chunking c{};
    c.lq = grad_log2(s.LN);
    const int64_t q = (int64_t)1 << c.lq;
    c.limit = -1;
    c.cut = true;
    c.nch = s.T > 0 ? ceil_div(s.T, q) : 1;
    c.slots = s.packed ? s.T / q + s.nseq : s.b * c.nch;
    return c;
}

ssd_status parse_shape(const ssd_selective_scan_args *a, bool bwd, Shape *s)
{
    if (!a) return SSD_ERR_NULL_POINTER;
    const ssd_status r = check_dims(a->batch, a->dim, a->dstate, a->ngroups, a->dtype, s);
    if (r != SSD_OK) return r;
    constexpr int64_t most = ((int64_t)1 << 31) - 64;
    if (a->seqlen < 0 || a->seqlen >= most || a->batch >= most || a->batch * a->seqlen >= most) return SSD_ERR_BAD_SHAPE;
    if (a->seq_idx && (a->batch != 1 || a->nseq < 1 || a->nseq > ((int64_t)1 << 30))) return SSD_ERR_SEQ_IDX;
    s->T = a->seqlen;
    s->packed = a->seq_idx != nullptr;
    s->nseq = s->packed ? a->nseq : 0;
    s->rows = s->packed ? s->nseq : s->b;
    s->tokens = s->b * s->T;
    if (s->packed && s->T > ((int64_t)1 << 28)) return SSD_ERR_BAD_SHAPE;   // ids are read with 31-bit byte offsets
    if (s->tokens > ((int64_t)1 << 40) / s->D) return SSD_ERR_BAD_SHAPE;
    // grids: a direction's own chunks, a thread a state from chunk to chunk, and in the backward one a key's gradient
    const int64_t slots = (bwd ? bwd_chunks(*s) : fwd_chunks(*s)).slots;
    if (slots > kMaxGroups / s->nblk || s->rows > kMaxGroups / ceil_div(s->D * s->N, kThreads)) return SSD_ERR_BAD_SHAPE;
    if (bwd && s->tokens * s->G > kMaxGroups * kThreads / (8 * s->LN)) return SSD_ERR_BAD_SHAPE;
    // byte counts stay far below 2^63
    if (slots * s->D > ((int64_t)1 << 52) / s->N || s->rows * s->D > ((int64_t)1 << 52) / s->N) return SSD_ERR_BAD_SHAPE;
    return SSD_OK;
}

struct Workspace {
    size_t plan, order, S, sum, R, pD, pbias, part, total;
};
Workspace layout(const Shape &s, const Chunking &c, bool bwd)
{
    Workspace w{};
    size_t o = 0;
    auto take = [&](size_t n) { const size_t at = o; o = align256(o + n); return at; };
    const size_t states = (size_t)(c.slots * s.D * s.N) * 4, chans = (size_t)(c.slots * s.D) * 4;
    if (s.packed) w.plan = take((size_t)(s.nseq + 1) * 4);
    if (s.packed && !bwd) w.order = take((size_t)(s.nseq + 1) * 4);
    if (c.cut) {
        w.S = take(states);
        w.sum = take(chans);
    }
    if (bwd) {
        w.R = take(states);
        w.pD = take(chans);
        w.pbias = take(chans);
        w.part = take((size_t)(s.tokens * s.nblk) * 8 * s.LN * 4);
    }
    w.total = o;
    return w;
}

bool strides_ok(const Shape &s, int64_t xs, int64_t dts, int64_t Bs, int64_t Cs, int64_t zs, int64_t most)
{
    const int64_t d[] = {xs, dts, zs}, k[] = {Bs, Cs};
    for (int64_t v : d)
        if (v != 0 && (v < s.D || v > most)) return false;
    for (int64_t v : k)
        if (v != 0 && (v < s.G * s.N || v > most)) return false;
    return true;
}
size_t span(int64_t tokens, int64_t stride, int64_t width, size_t esz)
{
    return tokens > 0 ? (size_t)((tokens - 1) * (stride ? stride : width) + width) * esz : 0;
}

ssd_status check_inputs(const Shape &s, const ssd_selective_scan_args *a)
{
    if (!strides_ok(s, a->x_stride, a->dt_stride, a->B_stride, a->C_stride, a->z_stride, kMaxStride)) return SSD_ERR_BAD_SHAPE;
    if (!a->A) return SSD_ERR_NULL_POINTER;
    if (s.tokens > 0 && (!a->x || !a->dt || !a->B || !a->C)) return SSD_ERR_NULL_POINTER;
    const void *els[] = {a->x, a->dt, a->B, a->C, a->z}, *f[] = {a->A, a->D, a->dt_bias, a->initial_states, a->seq_idx};
    for (const void *p : els)
        if (!aligned_to(p, s.esz)) return SSD_ERR_MISALIGNED;
    for (const void *p : f)
        if (!aligned_to(p, 4)) return SSD_ERR_MISALIGNED;
    return SSD_OK;
}
struct Inputs {
    Range r[10];
};
Inputs inputs_of(const Shape &s, const ssd_selective_scan_args *a)
{
    const size_t d = (size_t)s.D * 4, states = (size_t)(s.rows * s.D * s.N) * 4;
    return Inputs{{{a->x, span(s.tokens, a->x_stride, s.D, s.esz)},
                   {a->dt, span(s.tokens, a->dt_stride, s.D, s.esz)},
                   {a->B, span(s.tokens, a->B_stride, s.G * s.N, s.esz)},
                   {a->C, span(s.tokens, a->C_stride, s.G * s.N, s.esz)},
                   {a->z, span(s.tokens, a->z_stride, s.D, s.esz)},
                   {a->A, d * s.N},
                   {a->D, d},
                   {a->dt_bias, d},
                   {a->initial_states, states},
                   {a->seq_idx, s.packed ? (size_t)s.T * 4 : 0}}};
}

ScanArgs scan_args(const Shape &s, const Chunking &c, const ssd_selective_scan_args *a, char *ws, const Workspace &w)
{
    ScanArgs k{};
    k.x = a->x;
    k.dt = a->dt;
    k.B = a->B;
    k.C = a->C;
    k.z = a->z;
    k.A = a->A;
    k.D_ = a->D;
    k.bias = a->dt_bias;
    k.xs = a->x_stride ? a->x_stride : s.D;
    k.dts = a->dt_stride ? a->dt_stride : s.D;
    k.zs = a->z_stride ? a->z_stride : s.D;
    k.Bs = a->B_stride ? a->B_stride : s.G * s.N;
    k.Cs = a->C_stride ? a->C_stride : s.G * s.N;
    k.s0 = a->initial_states;
    k.plan = s.packed ? reinterpret_cast<const int32_t *>(ws + w.plan) : nullptr;
    k.S = c.cut ? reinterpret_cast<float *>(ws + w.S) : nullptr;
    k.sum = c.cut ? reinterpret_cast<float *>(ws + w.sum) : nullptr;
    k.T = (int)s.T;
    k.D = (int)s.D;
    k.N = (int)s.N;
    k.per = (int)s.per;
    k.bpg = (int)s.bpg;
    k.nblk = (int)s.nblk;
    k.rows = (int)s.rows;
    k.lq = c.lq;
    k.nch = (int)c.nch;
    k.softplus = a->dt_softplus != 0;
    return k;
}

template <int N> using Int = std::integral_constant<int, N>;
template <typename F> void with_lanes(int LN, F &&f)
{
    if (LN == 1) f(Int<1>{});
    else if (LN == 2) f(Int<2>{});
    else if (LN == 4) f(Int<4>{});
    else if (LN == 8) f(Int<8>{});
    else f(Int<16>{});
}

// The segments' first tokens; for the forward also their order and whether they are cut.
void plan(const Shape &s, const Chunking &c, const ssd_selective_scan_args *a, ScanArgs &k, char *ws, const Workspace &w, bool order, hipStream_t st)
{
    hipLaunchKernelGGL(k_scan_starts, dim3((unsigned)(s.T > 0 ? ceil_div(s.T, 4 * kThreads) : ceil_div(s.nseq + 1, kThreads))), dim3(kThreads), 0, st,
                       a->seq_idx, reinterpret_cast<int32_t *>(ws + w.plan), (int)s.T, (int)s.nseq);
    if (!order) return;
    int32_t *o = reinterpret_cast<int32_t *>(ws + w.order);
    hipLaunchKernelGGL(k_scan_plan, dim3(1), dim3(kPlanThreads), 0, st, k, o, c.lq, (int)(c.limit < INT32_MAX ? c.limit : INT32_MAX));
    k.order = o;
}

template <typename E> ssd_status fwd_typed(const Shape &s, const ssd_selective_scan_args *a, hipStream_t st)
{
    const Chunking c = fwd_chunks(s);
    const Workspace w = layout(s, c, false);
    char *ws = static_cast<char *>(a->workspace);
    ScanArgs k = scan_args(s, c, a, ws, w);
    k.y = a->y;
    k.s1 = a->final_states;
    if (s.packed) plan(s, c, a, k, ws, w, true, st);
    const dim3 grid((unsigned)(c.slots * s.nblk)), block(kThreads);
    with_lanes(s.LN, [&](auto ln) {
        constexpr int LN = decltype(ln)::value;
        if (c.cut) {
            const int blocks = (int)ceil_div(s.D * s.N, kThreads);
            hipLaunchKernelGGL((k_scan<E, LN, false, 1>), grid, block, 0, st, k);
            hipLaunchKernelGGL(k_scan_pass<false>, dim3((unsigned)(s.rows * blocks)), block, 0, st, k, blocks);
        }
        if (k.z) hipLaunchKernelGGL((k_scan<E, LN, true, 0>), grid, block, 0, st, k);
        else hipLaunchKernelGGL((k_scan<E, LN, false, 0>), grid, block, 0, st, k);
    });
    return launched();
}

template <typename E>
ssd_status bwd_typed(const Shape &s, const ssd_selective_scan_args *a, const ssd_selective_scan_bwd_args *g, hipStream_t st)
{
    const Chunking c = bwd_chunks(s);
    const Workspace w = layout(s, c, true);
    char *ws = static_cast<char *>(g->workspace);
    ScanArgs k = scan_args(s, c, a, ws, w);
    k.dy = g->dy;
    k.d1 = g->dfinal_states;
    k.d0 = g->dinitial_states;
    k.dx = g->dx;
    k.ddt = g->ddt;
    k.dz = g->dz;
    k.R = reinterpret_cast<float *>(ws + w.R);
    k.pD = reinterpret_cast<float *>(ws + w.pD);
    k.pbias = reinterpret_cast<float *>(ws + w.pbias);
    k.part = reinterpret_cast<float *>(ws + w.part);
    if (s.packed) plan(s, c, a, k, ws, w, false, st);
    const dim3 grid((unsigned)(c.slots * s.nblk)), block(kThreads);
    const int blocks = (int)ceil_div(s.D * s.N, kThreads);
    with_lanes(s.LN, [&](auto ln) {
        constexpr int LN = decltype(ln)::value;
        auto gated = [&](auto gate) {
            constexpr bool GATE = decltype(gate)::value;
            hipLaunchKernelGGL((k_scan<E, LN, GATE, 2>), grid, block, 0, st, k);
            hipLaunchKernelGGL(k_scan_pass<true>, dim3((unsigned)(s.rows * blocks)), block, 0, st, k, blocks);
            hipLaunchKernelGGL((k_scan_grad<E, LN, GATE>), grid, block, 0, st, k);
        };
        if (k.z) gated(std::true_type{});
        else gated(std::false_type{});
        const int64_t items = s.tokens * s.G * 8 * LN;
        if (items > 0)
            hipLaunchKernelGGL((k_scan_keys<E>), dim3((unsigned)ceil_div(items, kThreads)), block, 0, st, (const float *)k.part,
                               (E *)g->dB, (E *)g->dC, items, (int)s.bpg, (int)s.N, 4 * LN);
    });
    auto sum = [&](const float *part, float *out, int64_t n) {
        hipLaunchKernelGGL(k_scan_sum, dim3((unsigned)ceil_div(n, 32)), dim3(1024), 0, st, part, out, (int)c.slots, n);
    };
    sum(k.S, g->dA, s.D * s.N);
    if (g->dD) sum(k.pD, g->dD, s.D);
    if (g->ddt_bias) sum(k.pbias, g->ddt_bias, s.D);
    return launched();
}

}  // namespace

extern "C" {

ssd_status ssd_selective_scan_fwd_workspace_size(const ssd_selective_scan_args *a, size_t *bytes)
{
    Shape s;
    const ssd_status r = parse_shape(a, false, &s);
    if (r != SSD_OK) return r;
    if (!bytes) return SSD_ERR_NULL_POINTER;
    *bytes = layout(s, fwd_chunks(s), false).total;
    return SSD_OK;
}

ssd_status ssd_selective_scan_bwd_workspace_size(const ssd_selective_scan_args *a, size_t *bytes)
{
    Shape s;
    const ssd_status r = parse_shape(a, true, &s);
    if (r != SSD_OK) return r;
    if (!bytes) return SSD_ERR_NULL_POINTER;
    *bytes = layout(s, bwd_chunks(s), true).total;
    return SSD_OK;
}

ssd_status ssd_selective_scan_fwd(const ssd_selective_scan_args *a, void *stream)
{
    Shape s;
    ssd_status r = parse_shape(a, false, &s);
    if (r != SSD_OK) return r;
    if ((r = check_inputs(s, a)) != SSD_OK) return r;
    if (s.tokens > 0 && !a->y) return SSD_ERR_NULL_POINTER;
    if (!aligned_to(a->y, s.esz) || !aligned_to(a->final_states, 4) || !aligned_to(a->workspace, 16)) return SSD_ERR_MISALIGNED;
    const size_t need = layout(s, fwd_chunks(s), false).total;
    if (need > 0 && !a->workspace) return SSD_ERR_NULL_POINTER;
    if (a->workspace_bytes < need) return SSD_ERR_WORKSPACE_TOO_SMALL;
    const Inputs in = inputs_of(s, a);
    const Range outs[] = {{a->y, span(s.tokens, 0, s.D, s.esz)},
                          {a->final_states, (size_t)(s.rows * s.D * s.N) * 4},
                          {need ? a->workspace : nullptr, need}};
    if (!apart(in.r, outs)) return SSD_ERR_ALIASING;
    hipStream_t st = static_cast<hipStream_t>(stream);
    return s.dtype == SSD_DTYPE_BF16 ? fwd_typed<bf16>(s, a, st) : fwd_typed<float>(s, a, st);
}

ssd_status ssd_selective_scan_bwd(const ssd_selective_scan_args *a, const ssd_selective_scan_bwd_args *g, void *stream)
{
    Shape s;
    ssd_status r = parse_shape(a, true, &s);
    if (r != SSD_OK) return r;
    if (!g) return SSD_ERR_NULL_POINTER;
    if ((r = check_inputs(s, a)) != SSD_OK) return r;
    if (s.tokens > 0 && (!g->dy || !g->dx || !g->ddt || !g->dB || !g->dC || (a->z && !g->dz))) return SSD_ERR_NULL_POINTER;
    if (!g->dA) return SSD_ERR_NULL_POINTER;
    const void *els[] = {g->dy, g->dx, g->ddt, g->dB, g->dC, a->z ? g->dz : nullptr};
    const void *f[] = {g->dfinal_states, g->dA, g->dD, g->ddt_bias, g->dinitial_states};
    for (const void *p : els)
        if (!aligned_to(p, s.esz)) return SSD_ERR_MISALIGNED;
    for (const void *p : f)
        if (!aligned_to(p, 4)) return SSD_ERR_MISALIGNED;
    if (!aligned_to(g->workspace, 16)) return SSD_ERR_MISALIGNED;
    const size_t need = layout(s, bwd_chunks(s), true).total;
    if (!g->workspace) return SSD_ERR_NULL_POINTER;
    if (g->workspace_bytes < need) return SSD_ERR_WORKSPACE_TOO_SMALL;
    const Inputs in = inputs_of(s, a);
    const size_t tok = span(s.tokens, 0, s.D, s.esz), key = span(s.tokens, 0, s.G * s.N, s.esz), states = (size_t)(s.rows * s.D * s.N) * 4;
    Range ins[12];
    for (int i = 0; i < 10; ++i) ins[i] = in.r[i];
    ins[10] = {g->dy, tok};
    ins[11] = {g->dfinal_states, states};
    const Range outs[] = {{g->dx, tok}, {g->ddt, tok}, {g->dB, key}, {g->dC, key}, {a->z ? g->dz : nullptr, tok},
                          {g->dA, (size_t)(s.D * s.N) * 4}, {g->dD, (size_t)s.D * 4}, {g->ddt_bias, (size_t)s.D * 4},
                          {g->dinitial_states, states}, {g->workspace, need}};
    if (!apart(ins, outs)) return SSD_ERR_ALIASING;
    hipStream_t st = static_cast<hipStream_t>(stream);
    return s.dtype == SSD_DTYPE_BF16 ? bwd_typed<bf16>(s, a, g, st) : bwd_typed<float>(s, a, g, st);
}

ssd_status ssd_selective_scan_step(const ssd_selective_scan_step_args *a, void *stream)
{
    if (!a) return SSD_ERR_NULL_POINTER;
    Shape s{};
    const ssd_status r = check_dims(a->batch, a->dim, a->dstate, a->ngroups, a->dtype, &s);
    if (r != SSD_OK) return r;
    if (s.b > kMaxGroups / s.nblk) return SSD_ERR_BAD_SHAPE;
    if (!strides_ok(s, a->x_stride, a->dt_stride, a->B_stride, a->C_stride, a->z_stride, kMaxStepStride)) return SSD_ERR_BAD_SHAPE;
    if (!a->x || !a->dt || !a->A || !a->B || !a->C || !a->state || !a->y) return SSD_ERR_NULL_POINTER;
    const void *els[] = {a->x, a->dt, a->B, a->C, a->z, a->y}, *f[] = {a->A, a->D, a->dt_bias, a->state};
    for (const void *p : els)
        if (!aligned_to(p, s.esz)) return SSD_ERR_MISALIGNED;
    for (const void *p : f)
        if (!aligned_to(p, 4)) return SSD_ERR_MISALIGNED;
    const Range ins[] = {{a->x, span(s.b, a->x_stride, s.D, s.esz)},       {a->dt, span(s.b, a->dt_stride, s.D, s.esz)},
                         {a->B, span(s.b, a->B_stride, s.G * s.N, s.esz)}, {a->C, span(s.b, a->C_stride, s.G * s.N, s.esz)},
                         {a->z, span(s.b, a->z_stride, s.D, s.esz)},       {a->A, (size_t)(s.D * s.N) * 4},
                         {a->D, (size_t)s.D * 4},                          {a->dt_bias, (size_t)s.D * 4}};
    const Range outs[] = {{a->state, (size_t)(s.b * s.D * s.N) * 4}, {a->y, span(s.b, 0, s.D, s.esz)}};
    if (!apart(ins, outs)) return SSD_ERR_ALIASING;
    StepArgs k{};
    k.x = a->x;
    k.dt = a->dt;
    k.B = a->B;
    k.C = a->C;
    k.z = a->z;
    k.A = a->A;
    k.D = a->D;
    k.bias = a->dt_bias;
    k.xs = a->x_stride ? a->x_stride : s.D;
    k.dts = a->dt_stride ? a->dt_stride : s.D;
    k.zs = a->z_stride ? a->z_stride : s.D;
    k.Bs = a->B_stride ? a->B_stride : s.G * s.N;
    k.Cs = a->C_stride ? a->C_stride : s.G * s.N;
    k.state = a->state;
    k.y = a->y;
    k.dim = (int)s.D;
    k.N = (int)s.N;
    k.per = (int)s.per;
    k.bpg = (int)s.bpg;
    k.nblk = (int)s.nblk;
    k.softplus = a->dt_softplus != 0;
    hipStream_t st = static_cast<hipStream_t>(stream);
    with_lanes(s.LN, [&](auto ln) {
        const dim3 grid((unsigned)(s.b * s.nblk)), block(kThreads);
        if (s.dtype == SSD_DTYPE_BF16) hipLaunchKernelGGL((k_scan_step<bf16, decltype(ln)::value>), grid, block, 0, st, k);
        else hipLaunchKernelGGL((k_scan_step<float, decltype(ln)::value>), grid, block, 0, st, k);
    });
    return launched();
}

}  // extern "C"
