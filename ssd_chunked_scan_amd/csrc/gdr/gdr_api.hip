// gdr_api.hip -- host side of the gated delta rule (ssd_gdr_* in include/ssd.h):
// argument validation, workspace layout and launches.  Validation is host-only and
// runs before any HIP call; nothing here allocates, frees or synchronises.
#include "ssd.h"

#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

#include "gdr_kernels.hpp"

using namespace ssd;
using namespace ssd::gdr;

namespace {

constexpr int64_t kMaxDim = (int64_t)1 << 30;
constexpr int64_t kMaxGroups = ((int64_t)1 << 24) - 1;   // workgroups of 256 threads in a launch

struct Shape {
    int64_t b, T, H, P, N, G, nseq;
    int64_t nc;       // chunks per batch row
    int64_t nct;      // chunks in all (an upper bound for packed streams)
    int64_t chains;   // batch rows or segments
    int64_t NT, Pp, np;
    int dtype;
    size_t esz;
    bool packed;
};

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
// g, beta and their gradients are read and written one element at a time
bool aligned_to(const void *p, int dtype) { return (reinterpret_cast<uintptr_t>(p) & (dtype == SSD_DTYPE_BF16 ? 1u : 3u)) == 0; }
size_t align256(size_t v) { return (v + 255) & ~(size_t)255; }
ssd_status launched() { return hipGetLastError() == hipSuccess ? SSD_OK : SSD_ERR_HIP; }

// P, N, heads and groups, common to the chunked calls and the step.
ssd_status check_dims(int64_t b, int64_t H, int64_t P, int64_t N, int64_t G, int dtype)
{
    if (dtype != SSD_DTYPE_F32 && dtype != SSD_DTYPE_BF16) return SSD_ERR_BAD_DTYPE;
    if (b < 1 || H < 1 || P < 16 || N < 16 || G < 1) return SSD_ERR_BAD_SHAPE;
    if (P % 16 != 0 || N % 16 != 0 || N > kMaxStateDim || P > 4096) return SSD_ERR_BAD_SHAPE;
    if (b > kMaxDim || H > kMaxDim || b * H > INT32_MAX) return SSD_ERR_BAD_SHAPE;
    if (H % G != 0) return SSD_ERR_GROUPS;
    return SSD_OK;
}

ssd_status parse_shape(const ssd_gdr_args *a, Shape *s)
{
    if (!a) return SSD_ERR_NULL_POINTER;
    const ssd_status r = check_dims(a->batch, a->nheads, a->headdim, a->dstate, a->ngroups, a->dtype);
    if (r != SSD_OK) return r;
    if (a->seqlen < 0 || a->seqlen > kMaxDim) return SSD_ERR_BAD_SHAPE;
    if (a->seq_idx && (a->batch != 1 || a->nseq < 1 || a->nseq > kMaxDim)) return SSD_ERR_SEQ_IDX;
    s->b = a->batch;
    s->T = a->seqlen;
    s->H = a->nheads;
    s->P = a->headdim;
    s->N = a->dstate;
    s->G = a->ngroups;
    s->dtype = a->dtype;
    s->esz = a->dtype == SSD_DTYPE_BF16 ? 2 : 4;
    s->packed = a->seq_idx != nullptr;
    s->nseq = s->packed ? a->nseq : 0;
    s->nc = (s->T + kC - 1) / kC;
    // every segment starts a chunk of its own: a bound that the host knows
    s->nct = s->packed ? s->T / kC + (s->nseq < s->T ? s->nseq : s->T) : s->b * s->nc;
    s->chains = s->packed ? s->nseq : s->b;
    s->NT = s->N <= 64 ? 64 : s->N <= 128 ? 128 : 256;
    s->Pp = (s->P + 31) / 32 * 32;
    s->np = (s->Pp + kC - 1) / kC;
    if (s->packed && s->T > ((int64_t)1 << 28)) return SSD_ERR_BAD_SHAPE;   // ids are read with 31-bit byte offsets
    // a chunk's rows of all heads or groups are addressed with 31-bit byte offsets
    if (s->H * s->P > (1 << 22) || s->G * s->N > (1 << 22)) return SSD_ERR_BAD_SHAPE;
    // int32 indices, and grids: a launch has fewer than 2^32 threads (the chains of both
    // directions, 4 preparing waves to a workgroup, 512 threads of the gradient kernel)
    if (s->chains > kMaxGroups / 2 / s->H / s->np || s->nct > kMaxGroups * 4 / (s->H + 2 * s->G) || s->nct * kC > INT32_MAX)
        return SSD_ERR_BAD_SHAPE;
    // byte counts stay far below 2^63
    if (s->nct * s->H > ((int64_t)1 << 40) / (s->P * s->NT) * 64 || s->chains * s->H > ((int64_t)1 << 44) / (s->P * s->N))
        return SSD_ERR_BAD_SHAPE;
    return SSD_OK;
}

struct Sizes {
    size_t kq, v, gate, states, seq;
};
Sizes sizes_of(const Shape &s)
{
    Sizes z;
    z.kq = (size_t)(s.b * s.T * s.G * s.N) * s.esz;
    z.v = (size_t)(s.b * s.T * s.H * s.P) * s.esz;
    z.gate = (size_t)(s.b * s.T * s.H) * s.esz;
    z.states = (size_t)(s.chains * s.H * s.P * s.N) * 4;
    z.seq = s.packed ? (size_t)s.T * 4 : 0;
    return z;
}

// The heads of a group go to `hsplit` workgroups of the gradient kernel.  One workgroup is
// what a CU holds, so a run takes rounds of 256.  In half heads' time: a workgroup takes its
// heads and 2 to start and to end, and every split adds fp32 sums of dq and dk to write and
// read back, about 1 (with 4 and 2, or 6 and 3, nine backwards of 55 to 1530 us took the same
// or up to 2 us more).
int64_t head_split(const Shape &s)
{
    const int64_t tiles = s.nct * s.G, hpg = s.H / s.G;
    const int64_t ends = 2, sums = 1;
    int64_t best = 1, cost = INT64_MAX;
    for (int64_t k = 1; k <= hpg && k <= 32; ++k) {
        const int64_t c = (tiles * k + 255) / 256 * (2 * ((hpg + k - 1) / k) + ends) + (k > 1 ? sums : 0);
        if (c < cost) {
            cost = c;
            best = k;
        }
    }
    return best;
}

ssd_status parse_bwd(const ssd_gdr_args *a, Shape *s)
{
    const ssd_status r = parse_shape(a, s);
    if (r != SSD_OK) return r;
    return s->nct * s->G * head_split(*s) > kMaxGroups / 2 ? SSD_ERR_BAD_SHAPE : SSD_OK;
}

// Narrow chains share a step among a workgroup's waves, wide ones have fewer bytes to load
// per column.  Narrow where wide workgroups (of both directions together) would not come
// near one per CU: up to 144 in bf16, 192 for its forward with N = 256 and for fp32.  2048
// tokens, heads of 64, whole passes in us, wide against narrow:
//   bf16, forward   N = 64   128 heads 119, 113   160 heads 127, 138   192 heads 136, 152   256 heads 157, 217
//                   N = 128            140, 118             146, 154             155, 167             167, 241
//                   N = 256            241, 155             243, 213             260, 228             272, 310
//   bf16, backward  N = 64   64 heads  198, 182   80 heads  219, 232   96 heads  229, 273   128 heads 271, 356
//                   N = 128            256, 210             275, 282             292, 330             347, 445
//                   N = 256            412, 354             445, 451             480, 533             574, 707
//   fp32, forward   N = 64   128 heads 268, 180   192 heads 287, 331   256 heads 291, 371
//                   N = 128            383, 232             403, 343             413, 438
//                   N = 256           1457, 430            1526, 629            1804, 838
//   fp32, backward  N = 64   64 heads  402, 302   96 heads  459, 460   128 heads 522, 554
//                   N = 128            611, 419             697, 647             797, 818
//                   N = 256           1820, 797            1992, 1171           2264, 1518
int64_t narrow_up_to(const Shape &s, int directions)
{
    return s.dtype == SSD_DTYPE_F32 || (s.N > 128 && directions == 1) ? 192 : 144;
}
constexpr size_t kCacheBytes = (size_t)256 << 20;

struct Workspace {
    size_t cmap, chain, range, order, kq, vec, tri, sst, ust, dst, hst, part, total;
};
Workspace layout(const Shape &s, bool bwd)
{
    Workspace w{};
    size_t o = 0;
    auto take = [&](size_t n) { const size_t at = o; o = align256(o + n); return at; };
    if (s.packed) {
        w.cmap = take((size_t)s.nct * 8);
        w.chain = take((size_t)s.nseq * 16);
        w.range = take((size_t)s.nseq * 8);
        w.order = take((size_t)s.nseq * 4);
    }
    const size_t u = (size_t)(s.nct * s.H);
    const int tri = s.dtype == SSD_DTYPE_BF16 ? tri_elems<bf16>(bwd) : tri_elems<float>(bwd);
    w.kq = take((size_t)(s.nct * s.G) * (bwd ? 4 : 3) * kC * (size_t)s.NT * s.esz);
    w.vec = take(u * kVec * 4);
    w.tri = take(u * (size_t)tri * s.esz);
    if (bwd) {
        const size_t col = (size_t)s.Pp * (s.dtype == SSD_DTYPE_BF16 ? kPlanes<bf16> : kPlanes<float>) * s.esz;
        w.sst = take(u * (size_t)s.NT * col);
        w.ust = take(u * kC * col);
        w.dst = take(u * (size_t)s.NT * col);
        w.hst = take(u * kC * col);
        const int64_t hs = head_split(s);
        w.part = take(hs > 1 ? (size_t)(s.nct * s.G * hs) * 2 * kC * (size_t)s.NT * 4 : 0);
    }
    w.total = o;
    return w;
}

template <typename F> ssd_status with_nt(int64_t NT, F &&f)
{
    if (NT == 64) return f(std::integral_constant<int, 64>{});
    if (NT == 128) return f(std::integral_constant<int, 128>{});
    return f(std::integral_constant<int, 256>{});
}

// What both directions form first: the chunk map, the operand copies, the triangles.
template <typename E, bool BWD>
ssd_status prepare(const Shape &s, const ssd_gdr_args *a, char *ws, const Workspace &w, Chunks *m, hipStream_t st)
{
    *m = Chunks{nullptr, nullptr, nullptr, (int)s.T, (int)s.nc};
    if (s.packed) {
        int2 *cmap = reinterpret_cast<int2 *>(ws + w.cmap);
        int4 *chain = reinterpret_cast<int4 *>(ws + w.chain);
        hipLaunchKernelGGL(k_gdr_map, dim3(1), dim3(kMapThreads), 0, st, a->seq_idx,
                           reinterpret_cast<int2 *>(ws + w.range), chain, cmap,
                           reinterpret_cast<int *>(ws + w.order), (int)s.T, (int)s.nseq, (int)s.nct);
        m->cmap = cmap;
        m->chain = chain;
        m->order = reinterpret_cast<const int *>(ws + w.order);
        if (launched() != SSD_OK) return SSD_ERR_HIP;
    }
    return with_nt(s.NT, [&](auto nt) {
        constexpr int NT = decltype(nt)::value;
        // heads per wave: 2048 waves (two per SIMD) run at a time, and a wave pays for its start,
        // K K^T and Q K^T once, about 1 + NT / 256 heads' time.  Whole forwards with 1, 2, 4 and 8
        // heads a wave: 16640 tokens of 64 heads, 8 a group, N = 128: 700, 672, 664, 686 us; 16384
        // of 32 heads in one group, N = 256: 745, 710, 694, 690 us
        const int64_t hpg = s.H / s.G;
        int64_t hpw = 1;
        double cost = 1e300;
        for (int64_t k = 1; k <= hpg && k <= 32; ++k) {
            const int64_t waves = s.nct * s.G * ((hpg + k - 1) / k);
            const double t = (double)((waves + 2047) / 2048) * ((double)k + 1 + (double)NT / 256);
            if (t < cost) {
                cost = t;
                hpw = k;
            }
        }
        const int64_t units = s.nct * s.G * ((hpg + hpw - 1) / hpw);
        // triangles that the last level of cache cannot hold are written past it: 410 MB of a
        // forward over 16640 tokens of 64 heads, all kernels 683 -> 664 us; 750 MB of a backward
        // over 8 x 2048 tokens of 80 heads 1595 -> 1570 us; but 57 MB of 2 x 2048 tokens of 24 heads
        // 151 -> 170 us
        const bool once = (size_t)(s.nct * s.H) * tri_elems<E>(BWD) * sizeof(E) > kCacheBytes;
        auto launch = [&](auto past) {
            hipLaunchKernelGGL((k_gdr_prep<E, NT, BWD, decltype(past)::value>),
                               dim3((unsigned)((units + 2 * s.nct * s.G + 3) / 4)), dim3(kThreads), 0, st, (const E *)a->k,
                               (const E *)a->q, (const E *)a->g, (const E *)a->beta, reinterpret_cast<E *>(ws + w.kq),
                               reinterpret_cast<float *>(ws + w.vec), reinterpret_cast<E *>(ws + w.tri), *m, (int)s.H,
                               (int)s.G, (int)s.N, a->scale, (int)hpw, (int)units);
        };
        if (once) launch(std::true_type{});
        else launch(std::false_type{});
        return launched();
    });
}

template <typename E> ChainArgs chain_args(const Shape &s, const ssd_gdr_args *a, char *ws, const Workspace &w, const Chunks &m)
{
    ChainArgs c{};
    c.kq = ws + w.kq;
    c.tri = ws + w.tri;
    c.vec = reinterpret_cast<const float *>(ws + w.vec);
    c.v = a->v;
    c.s0 = a->initial_states;
    c.m = m;
    c.H = (int)s.H;
    c.G = (int)s.G;
    c.P = (int)s.P;
    c.N = (int)s.N;
    c.Pp = (int)s.Pp;
    c.np = (int)s.np;
    c.units = (int)(s.chains * s.H * s.np);
    c.scale = a->scale;
    return c;
}

// Whether `directions` chains of these units run narrow; if so c is set for 16 columns per
// workgroup.
bool narrowed(ChainArgs &c, const Shape &s, int directions)
{
    if ((int64_t)c.units * directions > narrow_up_to(s, directions)) return false;
    c.np = (int)(s.Pp / 16);
    c.units = (int)(s.chains * s.H * c.np);
    return true;
}

template <typename E> ssd_status fwd_typed(const Shape &s, const ssd_gdr_args *a, hipStream_t st)
{
    const Workspace w = layout(s, false);
    char *ws = static_cast<char *>(a->workspace);
    Chunks m;
    ssd_status r = prepare<E, false>(s, a, ws, w, &m, st);
    if (r != SSD_OK) return r;
    ChainArgs c = chain_args<E>(s, a, ws, w, m);
    c.y = a->y;
    c.s1 = a->final_states;
    return with_nt(s.NT, [&](auto nt) {
        constexpr int NT = decltype(nt)::value;
        if (narrowed(c, s, 1))
            hipLaunchKernelGGL((k_gdr_chain_narrow<E, NT / 16>), dim3((unsigned)c.units), dim3(64 * kNW<NT / 16>), 0, st, c);
        else
            hipLaunchKernelGGL((k_gdr_chain<E, NT / 16, kStaged<E, NT>>), dim3((unsigned)c.units), dim3(kThreads), 0, st, c);
        return launched();
    });
}

template <typename E> ssd_status bwd_typed(const Shape &s, const ssd_gdr_args *a, const ssd_gdr_bwd_args *g, hipStream_t st)
{
    const Workspace w = layout(s, true);
    char *ws = static_cast<char *>(g->workspace);
    Chunks m;
    ssd_status r = prepare<E, true>(s, a, ws, w, &m, st);
    if (r != SSD_OK) return r;
    ChainArgs c = chain_args<E>(s, a, ws, w, m);
    c.dy = g->dy;
    c.dv = g->dv;
    c.d1 = g->dfinal_states;
    c.d0 = g->dinitial_states;
    c.sst = ws + w.sst;
    c.ust = ws + w.ust;
    c.dst = ws + w.dst;
    c.hst = ws + w.hst;
    const int64_t hs = head_split(s);
    GradArgs ga{};
    ga.kq = c.kq;
    ga.k = a->k;
    ga.q = a->q;
    ga.dy = g->dy;
    ga.sst = c.sst;
    ga.ust = c.ust;
    ga.dst = c.dst;
    ga.hst = c.hst;
    ga.vec = reinterpret_cast<float *>(ws + w.vec);
    ga.dq = g->dq;
    ga.dk = g->dk;
    ga.dg = g->dg;
    ga.dbeta = g->dbeta;
    ga.part = reinterpret_cast<float *>(ws + w.part);
    ga.m = m;
    ga.H = c.H;
    ga.G = c.G;
    ga.P = c.P;
    ga.N = c.N;
    ga.Pp = c.Pp;
    ga.hsplit = (int)hs;
    ga.scale = a->scale;
    return with_nt(s.NT, [&](auto nt) {
        constexpr int NT = decltype(nt)::value;
        if (narrowed(c, s, 2))
            hipLaunchKernelGGL((k_gdr_chains_narrow<E, NT / 16>), dim3(2u * (unsigned)c.units), dim3(64 * kNW<NT / 16>), 0,
                               st, c);
        else
            hipLaunchKernelGGL((k_gdr_chains<E, NT / 16, kStaged<E, NT>>), dim3(2u * (unsigned)c.units), dim3(kThreads), 0,
                               st, c);
        hipLaunchKernelGGL((k_gdr_grad<E, NT / 16>), dim3((unsigned)(s.nct * s.G * hs)), dim3(kGradThreads), 0, st, ga);
        if (hs > 1)
            hipLaunchKernelGGL((k_gdr_grad_sum<E, NT>), dim3((unsigned)(s.nct * s.G), NT / 16), dim3(kThreads), 0, st,
                               (const float *)ga.part, (E *)g->dq, (E *)g->dk, m, (int)s.G, (int)s.N, (int)hs);
        return launched();
    });
}

void copy_states(float *dst, const float *src, const Shape &s, hipStream_t st)
{
    if (!dst) return;
    const int64_t n = s.chains * s.H * s.P * s.N, blocks = (n / 4 + kThreads - 1) / kThreads;
    hipLaunchKernelGGL(k_gdr_copy, dim3((unsigned)(blocks < (1 << 20) ? blocks : 1 << 20)), dim3(kThreads), 0, st, dst, src, n);
}

// Inputs of the chunked calls: present, aligned.
ssd_status check_inputs(const ssd_gdr_args *a, const Shape &s)
{
    if (s.T > 0 && (!a->q || !a->k || !a->v || !a->g || !a->beta)) return SSD_ERR_NULL_POINTER;
    const void *ptrs[] = {a->q, a->k, a->v, a->initial_states, a->seq_idx};
    for (const void *p : ptrs)
        if (!aligned16(p)) return SSD_ERR_MISALIGNED;
    if (!aligned_to(a->g, s.dtype) || !aligned_to(a->beta, s.dtype)) return SSD_ERR_MISALIGNED;
    return SSD_OK;
}

template <size_t NO, size_t NI> bool clash(const Range (&outs)[NO], const Range (&ins)[NI])
{
    for (size_t i = 0; i < NO; ++i) {
        for (const Range &in : ins)
            if (overlaps(outs[i], in)) return true;
        for (size_t j = i + 1; j < NO; ++j)
            if (overlaps(outs[i], outs[j])) return true;
    }
    return false;
}

template <typename E> ssd_status run_step(const ssd_gdr_step_args *a, hipStream_t st)
{
    const int N = (int)a->dstate, P = (int)a->headdim;
    auto launch = [&](auto nl) {
        constexpr int NL = decltype(nl)::value;
        constexpr int rows = kThreads / NL * kStepRows;
        const dim3 grid((unsigned)(a->batch * a->nheads), (unsigned)((P + rows - 1) / rows));
        hipLaunchKernelGGL((k_gdr_step<E, NL>), grid, dim3(kThreads), 0, st, (const E *)a->q, (const E *)a->k,
                           (const E *)a->v, (const E *)a->g, (const E *)a->beta, a->state, (E *)a->y, (int)a->nheads,
                           (int)a->ngroups, P, N, a->scale);
        return launched();
    };
    const int need = N / 4;   // lanes per state row
    if (need <= 4) return launch(std::integral_constant<int, 4>{});
    if (need <= 8) return launch(std::integral_constant<int, 8>{});
    if (need <= 16) return launch(std::integral_constant<int, 16>{});
    if (need <= 32) return launch(std::integral_constant<int, 32>{});
    return launch(std::integral_constant<int, 64>{});
}

}  // namespace

extern "C" {

ssd_status ssd_gdr_fwd_workspace_size(const ssd_gdr_args *args, size_t *bytes)
{
    Shape s;
    const ssd_status r = parse_shape(args, &s);
    if (r != SSD_OK) return r;
    if (!bytes) return SSD_ERR_NULL_POINTER;
    *bytes = layout(s, false).total;
    return SSD_OK;
}

ssd_status ssd_gdr_bwd_workspace_size(const ssd_gdr_args *args, size_t *bytes)
{
    Shape s;
    const ssd_status r = parse_bwd(args, &s);
    if (r != SSD_OK) return r;
    if (!bytes) return SSD_ERR_NULL_POINTER;
    *bytes = layout(s, true).total;
    return SSD_OK;
}

ssd_status ssd_gdr_fwd(const ssd_gdr_args *a, void *stream)
{
    Shape s;
    ssd_status r = parse_shape(a, &s);
    if (r != SSD_OK) return r;
    if ((r = check_inputs(a, s)) != SSD_OK) return r;
    const bool empty = s.T == 0;
    if (!empty && (!a->y || !a->workspace)) return SSD_ERR_NULL_POINTER;
    if (!aligned16(a->y) || !aligned16(a->final_states) || !aligned16(a->workspace)) return SSD_ERR_MISALIGNED;
    const size_t wtotal = layout(s, false).total;
    if (!empty && a->workspace_bytes < wtotal) return SSD_ERR_WORKSPACE_TOO_SMALL;
    const Sizes z = sizes_of(s);
    const Range ins[] = {{a->q, z.kq}, {a->k, z.kq}, {a->v, z.v}, {a->g, z.gate}, {a->beta, z.gate},
                         {a->initial_states, z.states}, {a->seq_idx, z.seq}};
    const Range outs[] = {{a->y, z.v}, {a->final_states, z.states}, {empty ? nullptr : a->workspace, wtotal}};
    if (clash(outs, ins)) return SSD_ERR_ALIASING;
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (empty) {
        copy_states(a->final_states, a->initial_states, s, st);
        return launched();
    }
    return s.dtype == SSD_DTYPE_BF16 ? fwd_typed<bf16>(s, a, st) : fwd_typed<float>(s, a, st);
}

ssd_status ssd_gdr_bwd(const ssd_gdr_args *a, const ssd_gdr_bwd_args *g, void *stream)
{
    Shape s;
    ssd_status r = parse_bwd(a, &s);
    if (r != SSD_OK) return r;
    if (!g) return SSD_ERR_NULL_POINTER;
    if ((r = check_inputs(a, s)) != SSD_OK) return r;
    const bool empty = s.T == 0;
    if (!empty && (!g->dy || !g->dq || !g->dk || !g->dv || !g->dg || !g->dbeta || !g->workspace))
        return SSD_ERR_NULL_POINTER;
    const void *ptrs[] = {g->dy, g->dfinal_states, g->dq, g->dk, g->dv, g->dinitial_states, g->workspace};
    for (const void *p : ptrs)
        if (!aligned16(p)) return SSD_ERR_MISALIGNED;
    if (!aligned_to(g->dg, s.dtype) || !aligned_to(g->dbeta, s.dtype)) return SSD_ERR_MISALIGNED;
    const size_t wtotal = layout(s, true).total;
    if (!empty && g->workspace_bytes < wtotal) return SSD_ERR_WORKSPACE_TOO_SMALL;
    const Sizes z = sizes_of(s);
    const Range ins[] = {{a->q, z.kq}, {a->k, z.kq}, {a->v, z.v}, {a->g, z.gate}, {a->beta, z.gate},
                         {a->initial_states, z.states}, {a->seq_idx, z.seq}, {g->dy, z.v}, {g->dfinal_states, z.states}};
    const Range outs[] = {{g->dq, z.kq}, {g->dk, z.kq}, {g->dv, z.v}, {g->dg, z.gate}, {g->dbeta, z.gate},
                          {g->dinitial_states, z.states}, {empty ? nullptr : g->workspace, wtotal}};
    if (clash(outs, ins)) return SSD_ERR_ALIASING;
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (empty) {
        copy_states(g->dinitial_states, g->dfinal_states, s, st);
        return launched();
    }
    return s.dtype == SSD_DTYPE_BF16 ? bwd_typed<bf16>(s, a, g, st) : bwd_typed<float>(s, a, g, st);
}

ssd_status ssd_gdr_step(const ssd_gdr_step_args *a, void *stream)
{
    if (!a) return SSD_ERR_NULL_POINTER;
    const ssd_status r = check_dims(a->batch, a->nheads, a->headdim, a->dstate, a->ngroups, a->dtype);
    if (r != SSD_OK) return r;
    if (a->batch * a->nheads > kMaxGroups) return SSD_ERR_BAD_SHAPE;
    if (!a->q || !a->k || !a->v || !a->g || !a->beta || !a->state || !a->y) return SSD_ERR_NULL_POINTER;
    const void *ptrs[] = {a->q, a->k, a->v, a->state, a->y};
    for (const void *p : ptrs)
        if (!aligned16(p)) return SSD_ERR_MISALIGNED;
    if (!aligned_to(a->g, a->dtype) || !aligned_to(a->beta, a->dtype)) return SSD_ERR_MISALIGNED;
    const size_t esz = a->dtype == SSD_DTYPE_BF16 ? 2 : 4;
    const size_t bh = (size_t)(a->batch * a->nheads), kq = (size_t)(a->batch * a->ngroups * a->dstate) * esz;
    const Range ins[] = {{a->q, kq}, {a->k, kq}, {a->v, bh * a->headdim * esz}, {a->g, bh * esz}, {a->beta, bh * esz}};
    const Range outs[] = {{a->state, bh * a->headdim * a->dstate * 4}, {a->y, bh * a->headdim * esz}};
    if (clash(outs, ins)) return SSD_ERR_ALIASING;
    hipStream_t st = static_cast<hipStream_t>(stream);
    return a->dtype == SSD_DTYPE_BF16 ? run_step<bf16>(a, st) : run_step<float>(a, st);
}

}  // extern "C"
