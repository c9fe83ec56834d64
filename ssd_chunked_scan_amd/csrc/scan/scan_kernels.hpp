// scan_kernels.hpp -- the selective scan (a decay rate for every channel and state),
// forward, backward and one token, for gfx950.
//
//   Delta = softplus(dt + bias),  h_t = e^{Delta A} h_{t-1} + Delta x_t B_t,
//   y_t = (C_t . h_t + D x_t) SiLU(z_t)
//
// The decays differ in every channel d and state n, so no product of matrices forms the
// scan: it is an exponential and a few multiply-adds for each (t, d, n), and these bound
// it, not the bytes (N = 16: 16 exponentials for 8 bytes of x, dt, z and y).  A wave issues an
// fp32 instruction in 4 cycles and an exponential in 9.
//
// Layout.  LN neighbouring lanes share a channel, each holding 4 of its states (LN = N / 4
// rounded up to a power of two), so a wave has 64 / LN channels.  The LN lanes also share
// the work that a channel has once per token: lane j loads x, dt and z of token j of LN
// tokens, forms Delta and Delta x there, and the others read them by DPP.  B and C of a tile of
// tokens are in LDS as fp32.
//
// Chunks.  A row (a batch row, or a segment of a packed stream) is one after another in
// time; where the rows and channels are too few to fill the card, rows are cut into chunks:
// first every chunk's end state from a zero start, then the states from chunk to chunk,
// then every chunk from its own entering state.
#pragma once

#include <type_traits>

#include "segment_ids.hpp"
#include "ssd_device.hpp"

namespace ssd {
namespace sscan {

constexpr float kLn2 = 0.6931471805599453f;
// Tokens of a chunk of the backward (their Delta and x are in LDS, for 256 / LN channels).
constexpr int grad_log2(int LN) { return LN == 1 ? 4 : LN == 2 || LN == 16 ? 5 : 6; }
template <int LN> constexpr int kGradQ = 1 << grad_log2(LN);

constexpr int kUncut = 31;      // log2 of the chunk of rows that are not cut
constexpr int kRanked = 1024;   // rows that are put in order

struct ScanArgs {
    const void *x, *dt, *B, *C, *z;
    const float *A, *D_, *bias;    // D_: the skip term
    int64_t xs, dts, Bs, Cs, zs;   // elements from token to token
    const float *s0;               // initial states
    float *s1;                     // final states
    void *y;
    const int32_t *plan;           // packed streams: first token of every segment, T
    const int32_t *order;          // rows by length, then log2 of the chunk (NULL: lq), where the device decides
    float *S, *sum;                // chunk states [slots][D][N], sums of Delta [slots][D]
    const void *dy;
    const float *d1;               // gradient of the final states
    float *d0;                     // gradient of the initial states
    void *dx, *ddt, *dz;
    float *R;                      // gradients of the chunk states [slots][D][N]
    float *part;                   // dB, dC of every tile of channels [tokens][nblk][2][4 LN]
    float *pD, *pbias;             // dD, ddt_bias of every chunk [slots][D]
    int T, D, N, per, bpg, nblk, rows, lq, nch, softplus;
};

// The LN lanes of a channel, lane I's value in all of them.
template <int LN, int I> __device__ __forceinline__ float from_lane(float v)
{
    if constexpr (LN == 1) return v;
    else if constexpr (LN == 2) return dpp_mov<I | I << 2 | (2 + I) << 4 | (2 + I) << 6>(v);
    else if constexpr (LN == 4) return dpp_mov<I * 0x55>(v);
    else {   // 0x150 + i: lane i of each row of 16
        const int s = __float_as_int(v), lo = __builtin_amdgcn_update_dpp(0, s, 0x150 + I, 0xf, 0xf, true);
        if constexpr (LN == 16) return __int_as_float(lo);
        else return __int_as_float(__builtin_amdgcn_update_dpp(lo, s, 0x150 + 8 + I, 0xf, 0xc, false));
    }
}
// The sum over the LN lanes of a channel, in all of them.
constexpr int kDppRowMirror = 0x140, kDppRowRor4 = 0x124;
template <int LN> __device__ __forceinline__ float lane_sum(float v)
{
    if constexpr (LN >= 2) v += dpp_mov<kDppQuadXor1>(v);
    if constexpr (LN >= 4) v += dpp_mov<kDppQuadXor2>(v);
    if constexpr (LN >= 8) v += dpp_mov<kDppRowHalfMirror>(v);
    if constexpr (LN >= 16) v += dpp_mov<kDppRowMirror>(v);
    return v;
}
template <int N, typename F> __device__ __forceinline__ void unrolled(F &&f)
{
    if constexpr (N > 0) {
        unrolled<N - 1>(f);
        f(std::integral_constant<int, N - 1>{});
    }
}

// A barrier for what is in LDS: accesses of global memory stay in flight across it.
__device__ __forceinline__ void lds_barrier()
{
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}
// One element of a row's buffer, zero past its end, as it is in memory: what is loaded ahead is turned into a
// float where it is used, since that waits for the load.
template <typename E> __device__ __forceinline__ uint32_t bload_raw(__amdgpu_buffer_rsrc_t r, uint32_t off)
{
    if constexpr (sizeof(E) == 2) return (uint32_t)__builtin_amdgcn_raw_buffer_load_b16(r, off, 0, 0);
    else return __builtin_amdgcn_raw_buffer_load_b32(r, off, 0, 0);
}
template <typename E> __device__ __forceinline__ float float_of(uint32_t raw) { return __uint_as_float(sizeof(E) == 2 ? raw << 16 : raw); }
// The same to memory, rounded; lost past the buffer's end.  Stores without branches around them leave
// the number of outstanding accesses known, so a wait for loads issued before them is not one for the stores.
template <typename E> __device__ __forceinline__ void bstore_el(__amdgpu_buffer_rsrc_t r, uint32_t off, float v)
{
    if constexpr (sizeof(E) == 2)
        __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(unsigned short, from_float<E>(v)), r, off, 0, 0);
    else __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v), r, off, 0, 0);
}
// `tokens` tokens of a tensor from token t0 on, `width` elements each.
template <typename E>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t token_rsrc(const void *p, int64_t t0, int64_t stride, int tokens, int width)
{
    return make_rsrc(static_cast<const E *>(p) + t0 * stride, tokens > 0 ? ((tokens - 1) * stride + width) * (int64_t)sizeof(E) : 0);
}

// ---------------------------------------------------------------------------
// rows and chunks
// ---------------------------------------------------------------------------
// Chunk slot c.  Segment i of a packed stream that starts at token s_i has the slots from
// s_i / Q + i on: as many as its chunks, whatever the lengths (floor(a) + ceil(b) <=
// floor(a + b) + 1), so no list of chunks is needed, and T / Q + segments slots hold them
// all.  Slots without tokens have count <= 0.
struct Slot {
    int row, j, count;   // the chunk's row, its number there, its tokens
    int64_t t0;          // its first token
    int len;             // tokens of the row
    bool last;
};
// The first token of segment i; in [0, T] whatever an invalid stream has left there.
__device__ __forceinline__ int start_of(const ScanArgs &a, int i)
{
    const int v = a.plan[i];
    return v < 0 ? 0 : v > a.T ? a.T : v;
}
__device__ __forceinline__ Slot slot_at(const ScanArgs &a, int c)
{
    Slot s;
    int lq = a.lq, start = 0;
    if (a.plan) {
        if (a.order) lq = a.order[a.rows];
        int lo = 0, hi = a.rows - 1;
        if (lq == kUncut) lo = c < a.rows && a.rows <= kRanked ? a.order[c] : c < a.rows ? c : hi;
        else
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if ((int64_t)(start_of(a, mid) >> lq) + mid <= c) lo = mid;
                else hi = mid - 1;
            }
        s.row = lo;
        start = start_of(a, lo);
        s.len = start_of(a, lo + 1) - start;
        s.j = lq == kUncut ? (c < a.rows ? 0 : -1) : c - ((start >> lq) + lo);
        s.t0 = start;
    } else {
        s.row = c / a.nch;
        s.j = c - s.row * a.nch;
        s.len = a.T;
        s.t0 = (int64_t)s.row * a.T;
    }
    const int64_t at = (int64_t)s.j << lq, left = s.len - at, q = (int64_t)1 << lq;
    s.t0 += at;
    s.count = s.j < 0 || left <= 0 ? 0 : (int)(left < q ? left : q);
    s.last = left <= q;
    return s;
}

// start[from] .. start[to - 1] = t of every lane: a few by the lane itself, a long list (segments without tokens) by its wave (64 tokens and
// 65536 segments, 16 channels, one state: the forward 141 us, with every list by its lane 1785).
__device__ __forceinline__ void put_starts(int32_t *start, int from, int to, int t)
{
    constexpr int FEW = 8;
    const int n = to - from;
    if (n <= FEW)
        for (int i = from; i < to; ++i) start[i] = t;
    for (uint64_t many = __ballot(n > FEW); many; many &= many - 1) {
        const int l = __ffsll((unsigned long long)many) - 1;
        const int first = __builtin_amdgcn_readlane(from, l), last = __builtin_amdgcn_readlane(to, l), v = __builtin_amdgcn_readlane(t, l);
        for (int i = first + (threadIdx.x & 63); i < last; i += 64) start[i] = v;
    }
}
// start[i]: the first token of segment i (or of the next one that has any), start[nseq] = T, for non-decreasing
// ids; four tokens a thread, a start a thread where there are no tokens.  Whatever the ids, i is in [0, nseq].
__global__ __launch_bounds__(kThreads) void k_scan_starts(const int32_t *__restrict__ seq_idx, int32_t *__restrict__ start, int T, int nseq)
{
    const int at = blockIdx.x * kThreads + threadIdx.x;
    if (T == 0) {
        if (at <= nseq) start[at] = 0;
        return;
    }
    const int t0 = at * 4;
    const __amdgpu_buffer_rsrc_t rs = make_rsrc_n(seq_idx, T * 4);
    int id[5];
    id[0] = t0 > 0 && t0 < T ? (int)__builtin_amdgcn_raw_buffer_load_b32(rs, 4u * t0 - 4, 0, 0) : -1;
#pragma unroll
    for (int e = 0; e < 4; ++e) id[e + 1] = (int)__builtin_amdgcn_raw_buffer_load_b32(rs, 4u * (t0 + e), 0, 0);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int t = t0 + e;
        const Segments here = segments_through(id[e], id[e + 1], nseq);   // this id's, and those of ids left out
        put_starts(start, here.from, t < T ? here.to : here.from, t);
        put_starts(start, here.to, t == T - 1 ? nseq + 1 : here.to, T);
    }
}
// Where the device decides: rows in the order of their lengths, the longest first (a long one that starts last
// would run alone at the end), and whether any is long enough beside the whole to be cut.
constexpr int kPlanThreads = 1024;
__global__ __launch_bounds__(kPlanThreads) void k_scan_plan(ScanArgs a, int32_t *__restrict__ order, int lq_long, int limit)
{
    __shared__ int most, len[kRanked];
    const int tid = threadIdx.x;
    if (tid == 0) most = 0;
    __syncthreads();
    int m = 0;
    for (int i = tid; i < a.rows; i += kPlanThreads) {
        const int n = start_of(a, i + 1) - start_of(a, i);
        m = max(m, n);
        if (a.rows <= kRanked) len[i] = n;
    }
    atomicMax(&most, m);
    __syncthreads();
    if (a.rows <= kRanked && tid < a.rows) {
        const int n = len[tid];
        int rank = 0;
        for (int o = 0; o < a.rows; ++o) rank += len[o] > n || (len[o] == n && o < tid) ? 1 : 0;
        order[rank] = tid;
    }
    if (tid == 0) order[a.rows] = most <= limit ? kUncut : lq_long;
}

// ---------------------------------------------------------------------------
// one tile of channels
// ---------------------------------------------------------------------------
template <int LN> struct Lanes {
    static constexpr int CB = kThreads / LN;          // channels of a workgroup
    static constexpr int NP = 4 * LN;                 // states, padded
    static constexpr int TT = LN <= 2 ? 16 : LN == 4 ? 32 : 64;   // tokens of a tile
    static constexpr int NG = TT / LN;                // groups of LN tokens
    static constexpr int NL = (TT * NP + kThreads - 1) / kThreads;   // B (and C) values of a tile a thread loads
};
struct Place {
    int g, d, j;     // group, channel, lane of the channel
    bool live;       // whether the lane has a channel of its own
};
template <int LN> __device__ __forceinline__ Place place_of(const ScanArgs &a, int blk)
{
    Place p;
    p.g = blk / a.bpg;
    const int c = (blk - p.g * a.bpg) * Lanes<LN>::CB + threadIdx.x / LN;
    p.live = c < a.per;
    p.d = p.g * a.per + (p.live ? c : a.per - 1);
    p.j = threadIdx.x % LN;
    return p;
}
// Four neighbours of a row of N, in one access where rows hold whole fours; it need not be
// aligned to more than an element.
template <typename E> using four_t = E __attribute__((ext_vector_type(4), aligned(sizeof(E))));
template <typename E> __device__ __forceinline__ void load_four(const E *p, int n0, int N, float (&h)[4])
{
    if ((N & 3) == 0) {
        four_t<E> v = {};
        if (n0 < N) v = *reinterpret_cast<const four_t<E> *>(p + n0);
#pragma unroll
        for (int k = 0; k < 4; ++k) h[k] = (float)v[k];
        return;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) h[k] = n0 + k < N ? to_float(p[n0 + k]) : 0.f;
}
__device__ __forceinline__ void load_state(const float *p, int n0, int N, float (&h)[4]) { load_four<float>(p, n0, N, h); }
__device__ __forceinline__ void store_state(float *p, int n0, int N, const float (&h)[4])
{
    if ((N & 3) == 0) {
        if (n0 < N) *reinterpret_cast<four_t<float> *>(p + n0) = four_t<float>{h[0], h[1], h[2], h[3]};
        return;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
        if (n0 + k < N) p[n0 + k] = h[k];
}

// B or C of `tokens` tokens from t0 on for LDS: element e of a tile is token e / NP, state e % NP.
template <typename E, int LN, int NL>
__device__ __forceinline__ void fetch_keys(const void *p, int64_t t0, int64_t stride, int g, int N, int tokens, uint32_t (&v)[NL])
{
    constexpr int NP = Lanes<LN>::NP;
    const __amdgpu_buffer_rsrc_t r = token_rsrc<E>(static_cast<const E *>(p) + (int64_t)g * N, t0, stride, tokens, N);
#pragma unroll
    for (int i = 0; i < NL; ++i) {
        const int e = i * kThreads + threadIdx.x, t = e / NP, n = e % NP;
        v[i] = bload_raw<E>(r, n < N && t < tokens ? (uint32_t)((t * stride + n) * sizeof(E)) : kOffNone);
    }
}
template <typename E, int LN, int NL> __device__ __forceinline__ void put_keys(float *dst, const uint32_t (&v)[NL], int elems)
{
#pragma unroll
    for (int i = 0; i < NL; ++i) {
        const int e = i * kThreads + threadIdx.x;
        if (e < elems) dst[e] = float_of<E>(v[i]);
    }
}

// softplus as softplus_f, with the hardware's reciprocal (1 ulp) for its quotient: once for every channel and token.
__device__ __forceinline__ float step_size(float raw, int softplus)
{
    if (!softplus) return raw;
    const float u = exp2_(-fabsf(raw) * kLog2e), w = 1.f + u;
    const float l1p = w == 1.f ? u : __builtin_amdgcn_logf(w) * kLn2 * (u * __builtin_amdgcn_rcpf(w - 1.f));
    return fmaxf(raw, 0.f) + l1p;
}

// Forward over a chunk.  MODE 0: y and the final states, from the state that enters the chunk.
// MODE 1: the chunk's end state from a zero start into S, and the sum of its Delta.  MODE 2:
// that, and what the chunk's dy add to the gradient of the state that enters it, R = sum over
// t of (product of the decays up to t's) C_t dy_t SiLU(z_t).
//
// 16 prompts of 18 K tokens in all, 5120 channels, 16 states, bf16: 495 us (MODE 0), of which the recurrence
// and its output (per 4 states and token 4 exponentials and 17 other instructions) are 360 and the loads, softplus, SiLU and
// the sum over lanes the rest; the bytes would take 140.  Workgroups of longer rows start first: 690 without that and with four waves.
// Three waves a SIMD keep it busy; with four, which the registers would let in, the longest rows share a SIMD with
// more of the others and end later (532 against 505 us; 555 with two; the same tokens of N = 8 456 either way, of N = 32, where four do
// not fit, 828 told so and 850 without).  For N <= 4 a limit of three would put 19 registers into scratch (636 against 430 us), for N > 32 two
// fit (1735 either way).  Forms that need more registers have their own limit.
template <int LN, int MODE> constexpr bool kThree = MODE == 0 && LN > 1 && LN < 16;
template <typename E, int LN, bool GATE, int MODE>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(kThree<LN, MODE> ? 3 : 1, kThree<LN, MODE> ? 3 : 8)))
void k_scan(ScanArgs a)
{
    using L = Lanes<LN>;
    constexpr int TT = L::TT, NP = L::NP, NG = L::NG, NL = L::NL;
    constexpr bool HASC = MODE != 1, HASZ = GATE && MODE != 1, HASG = MODE == 2;
    __shared__ float keys[2][HASC ? 2 : 1][TT * NP];
    const int c = blockIdx.x / a.nblk, blk = blockIdx.x - c * a.nblk;
    const Slot s = slot_at(a, c);
    const Place p = place_of<LN>(a, blk);
    const int n0 = 4 * p.j;
    const int64_t dn = (int64_t)p.d * a.N, DN = (int64_t)a.D * a.N;
    if (MODE == 0 ? s.count <= 0 && !(s.len <= 0 && s.j == 0) : s.count <= 0 || (s.last && (MODE == 1 || s.j == 0))) return;
    float h[4] = {0.f, 0.f, 0.f, 0.f}, R[4] = {0.f, 0.f, 0.f, 0.f}, cum[4] = {1.f, 1.f, 1.f, 1.f};
    if (MODE == 0) {
        if (s.j > 0) load_state(a.S + c * DN + dn, n0, a.N, h);
        else if (a.s0) load_state(a.s0 + s.row * DN + dn, n0, a.N, h);
    }
    float A2[4];
    load_state(a.A + dn, n0, a.N, A2);
#pragma unroll
    for (int k = 0; k < 4; ++k) A2[k] *= kLog2e;
    const float bias = a.bias ? a.bias[p.d] : 0.f, skip = a.D_ ? a.D_[p.d] : 0.f;
    float total = 0.f;

    // the next tile's values are on their way while this one is computed
    uint32_t xr[NG], dr[NG], zr[HASZ ? NG : 1], gr[HASG ? NG : 1], kb[NL], kc[HASC ? NL : 1];
    auto fetch = [&](int t1) {
        const int64_t t = s.t0 + t1;
        const int left = s.count - t1 < TT ? s.count - t1 : TT;
        const __amdgpu_buffer_rsrc_t rx = token_rsrc<E>(a.x, t, a.xs, left, a.D), rd = token_rsrc<E>(a.dt, t, a.dts, left, a.D);
#pragma unroll
        for (int q = 0; q < NG; ++q) {
            const int at = q * LN + p.j;
            xr[q] = bload_raw<E>(rx, (uint32_t)((at * (int)a.xs + p.d) * (int)sizeof(E)));
            dr[q] = bload_raw<E>(rd, (uint32_t)((at * (int)a.dts + p.d) * (int)sizeof(E)));
        }
        if constexpr (HASZ) {
            const __amdgpu_buffer_rsrc_t rz = token_rsrc<E>(a.z, t, a.zs, left, a.D);
#pragma unroll
            for (int q = 0; q < NG; ++q) zr[q] = bload_raw<E>(rz, (uint32_t)(((q * LN + p.j) * (int)a.zs + p.d) * (int)sizeof(E)));
        }
        if constexpr (HASG) {
            const __amdgpu_buffer_rsrc_t rg = token_rsrc<E>(a.dy, t, a.D, left, a.D);
#pragma unroll
            for (int q = 0; q < NG; ++q) gr[q] = bload_raw<E>(rg, (uint32_t)(((q * LN + p.j) * a.D + p.d) * (int)sizeof(E)));
        }
        fetch_keys<E, LN, NL>(a.B, t, a.Bs, p.g, a.N, left, kb);
        if constexpr (HASC) fetch_keys<E, LN, NL>(a.C, t, a.Cs, p.g, a.N, left, kc);
    };
    if (s.count > 0) fetch(0);
    for (int t1 = 0, b = 0; t1 < s.count; t1 += TT, b ^= 1) {
        put_keys<E, LN, NL>(keys[b][0], kb, TT * NP);
        if constexpr (HASC) put_keys<E, LN, NL>(keys[b][HASC ? 1 : 0], kc, TT * NP);
        float xv[NG], dl[NG], zv[HASZ ? NG : 1], gv[HASG ? NG : 1];
#pragma unroll
        for (int q = 0; q < NG; ++q) {
            // tokens past the chunk: no step, so that the state stays
            const bool in = t1 + q * LN + p.j < s.count;
            xv[q] = float_of<E>(xr[q]);
            dl[q] = in ? step_size(float_of<E>(dr[q]) + bias, a.softplus) : 0.f;
            if constexpr (HASZ) zv[q] = float_of<E>(zr[q]);
            if constexpr (HASG) gv[q] = HASZ ? float_of<E>(gr[q]) * silu(zv[q]) : float_of<E>(gr[q]);
        }
        if (t1 + TT < s.count) fetch(t1 + TT);
        const __amdgpu_buffer_rsrc_t ry =
            token_rsrc<E>(MODE == 0 ? a.y : a.x, s.t0 + t1, a.D, MODE != 0 ? 0 : s.count - t1 < TT ? s.count - t1 : TT, a.D);
        lds_barrier();   // the tile's keys are there, and the tile before last is done with
        const float *kB = keys[b][0] + n0, *kC = keys[b][HASC ? 1 : 0] + n0;
#pragma unroll
        for (int q = 0; q < NG; ++q) {
            const float dx = dl[q] * xv[q];
            float y = 0.f;
            unrolled<LN>([&](auto ic) {
                constexpr int i = decltype(ic)::value;
                const float di = from_lane<LN, i>(dl[q]), dxi = from_lane<LN, i>(dx);
                const floatx4 B = *reinterpret_cast<const floatx4 *>(kB + (q * LN + i) * NP);
                floatx4 C;
                if constexpr (HASC) C = *reinterpret_cast<const floatx4 *>(kC + (q * LN + i) * NP);
                float dyi = 0.f, acc = 0.f;
                if constexpr (HASG) dyi = from_lane<LN, i>(gv[q]);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float e = exp2_(di * A2[k]);
                    h[k] = e * h[k] + dxi * B[k];
                    if constexpr (MODE == 0) acc += h[k] * C[k];
                    if constexpr (MODE == 2) {
                        cum[k] *= e;
                        R[k] += cum[k] * (C[k] * dyi);
                    }
                }
                if constexpr (MODE == 0) {
                    acc = lane_sum<LN>(acc);
                    y = p.j == i ? acc : y;
                }
            });
            if constexpr (MODE == 0) {
                y += skip * xv[q];
                if constexpr (HASZ) y *= silu(zv[q]);
                bstore_el<E>(ry, p.live ? (uint32_t)(((q * LN + p.j) * a.D + p.d) * (int)sizeof(E)) : kOffNone, y);
            } else total += dl[q];
        }
    }
    if (!p.live) return;
    if constexpr (MODE == 0) {
        if (a.s1 && s.last) store_state(a.s1 + s.row * DN + dn, n0, a.N, h);
    } else {
        store_state(a.S + c * DN + dn, n0, a.N, h);
        total = lane_sum<LN>(total);
        if (p.j == 0) a.sum[(int64_t)c * a.D + p.d] = total;
        if constexpr (MODE == 2) store_state(a.R + c * DN + dn, n0, a.N, R);
    }
}

// From chunk to chunk, a state a thread: S becomes the state that enters the chunk, R (BWD) the
// gradient of the state that leaves it.  The first chunk's S and the last one's R stay: those
// come from the initial states and the final states' gradient.
template <bool BWD> __global__ __launch_bounds__(kThreads) void k_scan_pass(ScanArgs a, int blocks)
{
    constexpr int U = 8;   // chunks in flight
    const int row = blockIdx.x / blocks;
    const int64_t DN = (int64_t)a.D * a.N, e = (int64_t)(blockIdx.x - row * blocks) * kThreads + threadIdx.x;
    int lq = a.lq, len = a.T, c0 = row * a.nch;
    if (a.plan) {
        if (a.order) lq = a.order[a.rows];
        const int start = start_of(a, row);
        len = start_of(a, row + 1) - start;
        c0 = (start >> lq) + row;
    }
    const int n = len <= 0 ? 0 : (int)(((int64_t)len + ((int64_t)1 << lq) - 1) >> lq);
    if (n < 2 || e >= DN) return;
    const int d = (int)(e / a.N);
    const float A2 = a.A[e] * kLog2e;
    float h = a.s0 ? a.s0[row * DN + e] : 0.f;
    for (int j = 0; j < n - 1; j += U) {
        float s[U], t[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t c = c0 + (j + u < n - 1 ? j + u : n - 2);
            s[u] = a.S[c * DN + e];
            t[u] = a.sum[c * a.D + d];
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (j + u < n - 1) {
                if (j + u > 0) a.S[(c0 + j + u) * DN + e] = h;
                h = exp2_(A2 * t[u]) * h + s[u];
            }
    }
    a.S[(c0 + n - 1) * DN + e] = h;
    if constexpr (BWD) {
        float g = a.d1 ? a.d1[row * DN + e] : 0.f;
        for (int j = n - 1; j > 0; j -= U) {
            float s[U], t[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t c = c0 + (j - u > 0 ? j - u : 1);
                s[u] = a.R[c * DN + e];
                t[u] = a.sum[c * a.D + d];
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (j - u > 0) {
                    if (j - u < n - 1) a.R[(c0 + j - u) * DN + e] = g;
                    g = exp2_(A2 * t[u]) * g + s[u];
                }
        }
        a.R[(int64_t)c0 * DN + e] = g;
    }
}

// Every gradient of a chunk.  Delta and x of the whole chunk go to LDS first, then the states at the start
// of each 8 tokens; then, from the last 8 tokens to the first, the states in between again and the way back
// through them,
//
//   g_t = e^{Delta_t+1 A} g_t+1 + C_t dy_t,   dB_t = sum over d of Delta x g_t,  dC_t = sum over d of dy h_t,
//   dx = Delta (B . g) + D dy,  dDelta = x (B . g) + sum_n A e^{Delta A} g h_t-1,  dA = sum_t Delta e^{Delta A} g h_t-1
//
// with dy the gradient before the gate.  Over the four rows of 16 lanes the sum over channels of dB and dC is a
// product with a one-hot row on the matrix cores, which are idle here: v_mfma_f32_16x16x4 adds the four
// lanes of a column into row t (dB) or 8 + t (dC) of an accumulator that 8 tokens share; over the lanes of a
// row and over the waves it is taken once for the 8 tokens.  Over tiles of channels k_scan_keys adds it up.
//
// 0 x inf is NaN, so such a product spreads what is not finite over all 8 tokens; where a sum is not finite, the wave takes
// the 8 tokens' sums one by one from the states at their start and the gradient at their end (that check and its registers
// take 0.4 % of the time for N = 16, 4 % for N = 64).
//
// 16384 tokens of 5120 channels, 16 states, bf16: 1660 us, of k_scan's MODE 2 before it 433; the bytes would take 230.
// 256 registers a thread, 8 more in scratch: two waves a SIMD (three spill more: 2890 us).  In scratch are also, of the gated forms, some 160
// for N <= 4 and 13 for N = 5 to 8, and 50 of the ungated one for N <= 4 (all gradients of these tokens: 1990 us for N = 4 gated, 790
// ungated, 1485 and 1150 for N = 8).  Sums over channels by DPP and LDS alone, and Delta and x formed where
// they are used instead of staged, took 3045.  Chunks of 64 tokens: a shorter one rebuilds its states more often.
template <typename E, int LN, bool GATE>
__global__ __launch_bounds__(kThreads, 2) void k_scan_grad(ScanArgs a)
{
    constexpr int Q = kGradQ<LN>, NP = 4 * LN, SC = 8, TL = LN < SC ? LN : SC, GS = SC / TL, NSUB = Q / SC, SL = kThreads / LN;
    constexpr int NL = (Q * NP + kThreads - 1) / kThreads, NT = Q * SL / kThreads;
    __shared__ float keys[2][Q * NP];
    __shared__ floatx4 hs[NSUB][kThreads];
    __shared__ float red[2][4][SC][2][NP];
    __shared__ float sdl[Q * SL], sx[Q * SL];
    const int c = blockIdx.x / a.nblk, blk = blockIdx.x - c * a.nblk;
    const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
    const Slot s = slot_at(a, c);
    const Place p = place_of<LN>(a, blk);
    const int n0 = 4 * p.j, jt = p.j % TL, slot = tid / LN;
    const int64_t dn = (int64_t)p.d * a.N, DN = (int64_t)a.D * a.N;
    if (s.count <= 0) {
        const float none[4] = {0.f, 0.f, 0.f, 0.f};
        if (!p.live) return;
        // a segment without tokens hands its gradient on; a slot without tokens adds nothing
        if (s.len <= 0 && s.j == 0 && a.d0) {
            float g[4] = {0.f, 0.f, 0.f, 0.f};
            if (a.d1) load_state(a.d1 + s.row * DN + dn, n0, a.N, g);
            store_state(a.d0 + s.row * DN + dn, n0, a.N, g);
        }
        store_state(a.S + c * DN + dn, n0, a.N, none);
        if (p.j == 0) a.pD[(int64_t)c * a.D + p.d] = a.pbias[(int64_t)c * a.D + p.d] = 0.f;
        return;
    }
    const __amdgpu_buffer_rsrc_t rd = token_rsrc<E>(a.dt, s.t0, a.dts, s.count, a.D),
                                 rz = token_rsrc<E>(GATE ? a.z : a.x, s.t0, GATE ? a.zs : a.xs, s.count, a.D),
                                 rg = token_rsrc<E>(a.dy, s.t0, a.D, s.count, a.D), wx = token_rsrc<E>(a.dx, s.t0, a.D, s.count, a.D),
                                 wd = token_rsrc<E>(a.ddt, s.t0, a.D, s.count, a.D),
                                 wz = token_rsrc<E>(GATE ? a.dz : a.dx, s.t0, a.D, s.count, a.D),
                                 wp = token_rsrc<float>(a.part + blk * (2 * NP), s.t0, (int64_t)a.nblk * (2 * NP), s.count, 2 * NP);
    float h[4] = {0.f, 0.f, 0.f, 0.f}, g[4] = {0.f, 0.f, 0.f, 0.f}, A2[4] = {0.f, 0.f, 0.f, 0.f};
    // the gradient of the state that leaves the chunk
    auto load_end = [&](float(&v)[4]) {
        if (!p.live) return;
        if (!s.last) load_state(a.R + c * DN + dn, n0, a.N, v);
        else if (a.d1) load_state(a.d1 + s.row * DN + dn, n0, a.N, v);
    };
    if (p.live) {
        if (s.j > 0) load_state(a.S + c * DN + dn, n0, a.N, h);
        else if (a.s0) load_state(a.s0 + s.row * DN + dn, n0, a.N, h);
        load_state(a.A + dn, n0, a.N, A2);
    }
    load_end(g);
#pragma unroll
    for (int k = 0; k < 4; ++k) A2[k] *= kLog2e;
    const float bias = a.bias ? a.bias[p.d] : 0.f, skip = a.D_ ? a.D_[p.d] : 0.f;
    const int nsub = (s.count + SC - 1) / SC;
    const float *kB = keys[0] + n0, *kC = keys[1] + n0;
    // the first tokens of the way back are on their way meanwhile
    uint32_t nraw[GS], nz[GS], ng[GS];
    auto fetch = [&](int u) {
#pragma unroll
        for (int q = 0; q < GS; ++q) {
            const int t = u * SC + q * TL + jt;
            nraw[q] = bload_raw<E>(rd, (uint32_t)((t * (int)a.dts + p.d) * (int)sizeof(E)));
            ng[q] = bload_raw<E>(rg, p.live ? (uint32_t)((t * a.D + p.d) * (int)sizeof(E)) : kOffNone);
            nz[q] = GATE ? bload_raw<E>(rz, p.live ? (uint32_t)((t * (int)a.zs + p.d) * (int)sizeof(E)) : kOffNone) : 0u;
        }
    };
    fetch(nsub - 1);
    // LDS position of a token and channel: the TL tokens that a wave's lanes read together lie in different banks
    auto place = [&](int t, int ch) { return t * SL + (ch ^ ((t % TL) * (64 / LN) & (SL - 1))); };
    {
        const __amdgpu_buffer_rsrc_t rx = token_rsrc<E>(a.x, s.t0, a.xs, s.count, a.D);
        const int ch = tid % SL, cc = (blk - p.g * a.bpg) * SL + ch, dd = p.g * a.per + (cc < a.per ? cc : a.per - 1);
        const float b = a.bias ? a.bias[dd] : 0.f;
        uint32_t xr[NT], dr[NT], kb[NL], kc[NL];
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            const int t = i * LN + tid / SL;
            xr[i] = bload_raw<E>(rx, cc < a.per ? (uint32_t)((t * (int)a.xs + dd) * (int)sizeof(E)) : kOffNone);
            dr[i] = bload_raw<E>(rd, (uint32_t)((t * (int)a.dts + dd) * (int)sizeof(E)));
        }
        fetch_keys<E, LN, NL>(a.B, s.t0, a.Bs, p.g, a.N, s.count, kb);
        fetch_keys<E, LN, NL>(a.C, s.t0, a.Cs, p.g, a.N, s.count, kc);
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            const int t = i * LN + tid / SL;
            // none for a lane without a channel, none past the chunk
            sdl[place(t, ch)] = t < s.count && cc < a.per ? step_size(float_of<E>(dr[i]) + b, a.softplus) : 0.f;
            sx[place(t, ch)] = float_of<E>(xr[i]);
        }
        put_keys<E, LN, NL>(keys[0], kb, Q * NP);
        put_keys<E, LN, NL>(keys[1], kc, Q * NP);
    }
    lds_barrier();
    for (int u = 0; u < nsub; ++u) {
        hs[u][tid] = floatx4{h[0], h[1], h[2], h[3]};
        if (u == nsub - 1) break;
        float dxs[GS], dl[GS];
#pragma unroll
        for (int q = 0; q < GS; ++q) {
            const int at = place(u * SC + q * TL + jt, slot);
            dl[q] = sdl[at];
            dxs[q] = dl[q] * sx[at];
        }
        unrolled<SC>([&](auto tc) {
            constexpr int t = decltype(tc)::value, q = t / TL, i = t % TL;
            const float di = from_lane<LN, i>(dl[q]), dxi = from_lane<LN, i>(dxs[q]);
            const floatx4 B = *reinterpret_cast<const floatx4 *>(kB + (u * SC + t) * NP);
#pragma unroll
            for (int k = 0; k < 4; ++k) h[k] = exp2_(di * A2[k]) * h[k] + dxi * B[k];
        });
    }
    float dA[4] = {0.f, 0.f, 0.f, 0.f}, sD = 0.f, sb = 0.f;
    for (int u = nsub - 1; u >= 0; --u) {
        float raw[GS], x[GS], dl[GS], zv[GS], go[GS], dy[GS], dxs[GS], ys[GS];
#pragma unroll
        for (int q = 0; q < GS; ++q) {
            const int at = place(u * SC + q * TL + jt, slot);
            dl[q] = sdl[at];
            x[q] = sx[at];
            raw[q] = float_of<E>(nraw[q]) + bias;
            go[q] = float_of<E>(ng[q]);
            zv[q] = float_of<E>(nz[q]);
            dy[q] = GATE ? go[q] * silu(zv[q]) : go[q];
            dxs[q] = dl[q] * x[q];
            ys[q] = 0.f;
        }
        fetch(u > 0 ? u - 1 : 0);
        float hh[SC + 1][4], ee[SC][4];
        {
            const floatx4 v = hs[u][tid];
            if (u < nsub - 1) hs[u + 1][tid] = floatx4{g[0], g[1], g[2], g[3]};   // for the sums token by token below
#pragma unroll
            for (int k = 0; k < 4; ++k) hh[0][k] = v[k];
        }
        unrolled<SC>([&](auto tc) {
            constexpr int t = decltype(tc)::value, q = t / TL, i = t % TL;
            const floatx4 B = *reinterpret_cast<const floatx4 *>(kB + (u * SC + t) * NP);
            floatx4 C;
            if constexpr (GATE) C = *reinterpret_cast<const floatx4 *>(kC + (u * SC + t) * NP);
            const float di = from_lane<LN, i>(dl[q]), dxi = from_lane<LN, i>(dxs[q]);
            float acc = 0.f;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                ee[t][k] = exp2_(di * A2[k]);
                hh[t + 1][k] = ee[t][k] * hh[t][k] + dxi * B[k];
                if constexpr (GATE) acc += hh[t + 1][k] * C[k];
            }
            if constexpr (GATE) {
                acc = lane_sum<LN>(acc);
                ys[q] = jt == i ? acc : ys[q];
            }
        });
        float along[GS], dd[GS];
        floatx4 keysum[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) keysum[k] = floatx4{0.f, 0.f, 0.f, 0.f};
        unrolled<SC>([&](auto tc) {
            constexpr int t = SC - 1 - decltype(tc)::value, q = t / TL, i = t % TL;
            const floatx4 B = *reinterpret_cast<const floatx4 *>(kB + (u * SC + t) * NP);
            const floatx4 C = *reinterpret_cast<const floatx4 *>(kC + (u * SC + t) * NP);
            const float di = from_lane<LN, i>(dl[q]), dxi = from_lane<LN, i>(dxs[q]), dyi = from_lane<LN, i>(dy[q]);
            const float to = (lane & 15) == t + (lane < 32 ? 0 : 8) ? 1.f : 0.f;
            float al = 0.f, de = 0.f;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                g[k] += dyi * C[k];
                const auto v = __builtin_amdgcn_permlane32_swap(__float_as_uint(dxi * g[k]), __float_as_uint(dyi * hh[t + 1][k]), false, false);
                keysum[k] = __builtin_amdgcn_mfma_f32_16x16x4f32(to, __uint_as_float(v[0]) + __uint_as_float(v[1]), keysum[k], 0, 0, 0);
                al += g[k] * B[k];
                g[k] *= ee[t][k];
                const float gh = g[k] * hh[t][k];
                de += gh * A2[k];
                dA[k] += gh * di;
            }
            al = lane_sum<LN>(al);
            de = lane_sum<LN>(de);
            along[q] = i == TL - 1 || jt == i ? al : along[q];
            dd[q] = i == TL - 1 || jt == i ? de : dd[q];
        });
        // a product with a row of zeros and a one spreads what is not finite over all 8 tokens, so that one of a column's rows shows
        // it: such sums are taken token by token
        const float odd = (keysum[0][0] + keysum[1][0]) + (keysum[2][0] + keysum[3][0]);
        if (__builtin_expect(__any(!__builtin_isfinite(odd)), 0)) {
            float As[4], xs[GS], ds[GS], gy[GS], v[4];
            // formed again, not kept in registers from above
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                As[k] = A2[k];
                asm volatile("" : "+v"(As[k]));
            }
#pragma unroll
            for (int q = 0; q < GS; ++q) {
                ds[q] = dl[q];
                xs[q] = x[q];
                gy[q] = dy[q];
                asm volatile("" : "+v"(ds[q]), "+v"(xs[q]), "+v"(gy[q]));
                xs[q] *= ds[q];
            }
            // v, summed over the wave's channels, as token t's dB (0) or dC (1)
            auto put = [&](int t, int which) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
#pragma unroll
                    for (int d = LN; d < 64; d <<= 1) v[k] += __shfl_xor(v[k], d);
                if (lane < LN) *reinterpret_cast<floatx4 *>(&red[u & 1][wv][t][which][n0]) = floatx4{v[0], v[1], v[2], v[3]};
                __builtin_amdgcn_sched_barrier(0);
            };
            floatx4 st = hs[u][tid];
            unrolled<SC>([&](auto tc) {
                constexpr int t = decltype(tc)::value, q = t / TL, i = t % TL;
                const floatx4 B = *reinterpret_cast<const floatx4 *>(kB + (u * SC + t) * NP);
                const float di = from_lane<LN, i>(ds[q]), dxi = from_lane<LN, i>(xs[q]), dyi = from_lane<LN, i>(gy[q]);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    st[k] = exp2_(di * As[k]) * st[k] + dxi * B[k];
                    v[k] = dyi * st[k];
                }
                put(t, 1);
            });
            float gs[4] = {0.f, 0.f, 0.f, 0.f};
            if (u == nsub - 1) load_end(gs);
            else {
                const floatx4 w = hs[u + 1][tid];
#pragma unroll
                for (int k = 0; k < 4; ++k) gs[k] = w[k];
            }
            unrolled<SC>([&](auto tc) {
                constexpr int t = SC - 1 - decltype(tc)::value, q = t / TL, i = t % TL;
                const floatx4 C = *reinterpret_cast<const floatx4 *>(kC + (u * SC + t) * NP);
                const float di = from_lane<LN, i>(ds[q]), dxi = from_lane<LN, i>(xs[q]), dyi = from_lane<LN, i>(gy[q]);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    gs[k] += dyi * C[k];
                    v[k] = dxi * gs[k];
                    gs[k] *= exp2_(di * As[k]);
                }
                put(t, 0);
            });
        } else
        // keysum[k][r]: row 4 (lane / 16) + r of column lane % 16; over the columns of one state
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            float v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                v[k] = keysum[k][r];
                if constexpr (LN <= 8) v[k] += dpp_mov<kDppRowRor8>(v[k]);
                if constexpr (LN <= 4) v[k] += dpp_mov<kDppRowRor4>(v[k]);
                if constexpr (LN <= 2) v[k] += dpp_mov<kDppQuadXor2>(v[k]);
                if constexpr (LN == 1) v[k] += dpp_mov<kDppQuadXor1>(v[k]);
            }
            const int row = 4 * (lane >> 4) + r;
            if ((lane & 15) < LN) *reinterpret_cast<floatx4 *>(&red[u & 1][wv][row & 7][row >> 3][n0]) = floatx4{v[0], v[1], v[2], v[3]};
        }
#pragma unroll
        for (int q = 0; q < GS; ++q) {
            const int t = u * SC + q * TL + jt;
            const uint32_t at = p.live && p.j < TL ? (uint32_t)((t * a.D + p.d) * (int)sizeof(E)) : kOffNone;
            float dd_ = x[q] * along[q] + kLn2 * dd[q];
            if (a.softplus) dd_ *= __builtin_amdgcn_rcpf(1.f + exp2_(-raw[q] * kLog2e));
            bstore_el<E>(wx, at, dl[q] * along[q] + dy[q] * skip);
            bstore_el<E>(wd, at, dd_);
            // tokens past the chunk have neither
            const bool in = t < s.count && p.j < TL;
            sD += in ? dy[q] * x[q] : 0.f;
            sb += in ? dd_ : 0.f;
            if constexpr (GATE) {
                const float sg = __builtin_amdgcn_rcpf(1.f + exp2_(-zv[q] * kLog2e));
                bstore_el<E>(wz, at, go[q] * (ys[q] + skip * x[q]) * (sg * (1.f + zv[q] * (1.f - sg))));
            }
        }
        lds_barrier();   // once for 8 tokens: the next ones' sums go to the other half
        for (int e = tid; e < SC * 2 * NP; e += kThreads) {
            const int t = u * SC + e / (2 * NP);
            const float *r = &red[u & 1][0][0][0][0] + e;
            constexpr int W = SC * 2 * NP;
            bstore_el<float>(wp, (uint32_t)(t * a.nblk * (2 * NP) + e % (2 * NP)) * 4u, (r[0] + r[W]) + (r[2 * W] + r[3 * W]));
        }
    }
    sD = lane_sum<LN>(sD);
    sb = lane_sum<LN>(sb);
    if (!p.live) return;
    if (s.j == 0 && a.d0) store_state(a.d0 + s.row * DN + dn, n0, a.N, g);
    store_state(a.S + c * DN + dn, n0, a.N, dA);   // this workgroup alone has read it
    if (p.j == 0) {
        a.pD[(int64_t)c * a.D + p.d] = sD;
        a.pbias[(int64_t)c * a.D + p.d] = sb;
    }
}

// dB and dC: the sums of a token's and group's tiles of channels.
template <typename E>
__global__ __launch_bounds__(kThreads) void k_scan_keys(const float *__restrict__ part, E *__restrict__ dB, E *__restrict__ dC,
                                                        int64_t items, int bpg, int N, int NP)
{
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (i >= items) return;
    const int n = (int)(i % (2 * NP));
    const int64_t tg = i / (2 * NP);
    const float *p = part + tg * bpg * (2 * NP) + n;
    float s = 0.f;
    for (int b = 0; b < bpg; ++b) s += p[(int64_t)b * 2 * NP];
    const int k = n % NP;
    if (k < N) (n < NP ? dB : dC)[tg * N + k] = from_float<E>(s);
}

// out[e] = the sum over the slots of part[slot][e]: 32 values and 32 slices of the slots a workgroup.
__global__ __launch_bounds__(1024) void k_scan_sum(const float *__restrict__ part, float *__restrict__ out, int slots, int64_t n)
{
    __shared__ float s[32][33];
    const int cl = threadIdx.x & 31, sl = threadIdx.x >> 5;
    const int64_t e = (int64_t)blockIdx.x * 32 + cl;
    float v = 0.f;
    if (e < n)
        for (int c = sl; c < slots; c += 32) v += part[c * n + e];
    s[sl][cl] = v;
    __syncthreads();
    if (sl == 0 && e < n) {
        float t = 0.f;
#pragma unroll
        for (int r = 0; r < 32; ++r) t += s[r][cl];
        out[e] = t;
    }
}

// One token of every batch row: the state is read and written once, 16 bytes a lane, and that
// is what should bound it.  64 rows of 5120 channels and 16 states: 42 MB in 13 us (single elements 23; a copy of as
// many bytes, in the last cache, takes 5.5).
struct StepArgs {
    const void *x, *dt, *B, *C, *z;
    const float *A, *D, *bias;
    int64_t xs, dts, Bs, Cs, zs;
    float *state;
    void *y;
    int dim, N, per, bpg, nblk, softplus;
};
template <typename E, int LN>
__global__ __launch_bounds__(kThreads) void k_scan_step(StepArgs a)
{
    constexpr int CB = kThreads / LN;
    const int b = blockIdx.x / a.nblk, blk = blockIdx.x - b * a.nblk;
    const int g = blk / a.bpg, c = (blk - g * a.bpg) * CB + threadIdx.x / LN, j = threadIdx.x % LN, n0 = 4 * j;
    if (c >= a.per) return;   // all lanes of the channel
    const int d = g * a.per + c;
    const E *Bp = static_cast<const E *>(a.B) + b * a.Bs + (int64_t)g * a.N, *Cp = static_cast<const E *>(a.C) + b * a.Cs + (int64_t)g * a.N;
    float *sp = a.state + ((int64_t)b * a.dim + d) * a.N;
    float h[4], A[4], B[4], C[4];
    load_state(sp, n0, a.N, h);
    load_state(a.A + (int64_t)d * a.N, n0, a.N, A);
    load_four<E>(Bp, n0, a.N, B);
    load_four<E>(Cp, n0, a.N, C);
    const float x = to_float(static_cast<const E *>(a.x)[b * a.xs + d]);
    const float dl = step_size(to_float(static_cast<const E *>(a.dt)[b * a.dts + d]) + (a.bias ? a.bias[d] : 0.f), a.softplus);
    float y = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        h[k] = exp2_(dl * (A[k] * kLog2e)) * h[k] + dl * x * B[k];
        y += h[k] * C[k];
    }
    store_state(sp, n0, a.N, h);
    y = lane_sum<LN>(y);
    if (j) return;
    if (a.D) y += a.D[d] * x;
    if (a.z) y *= silu(to_float(static_cast<const E *>(a.z)[b * a.zs + d]));
    static_cast<E *>(a.y)[(int64_t)b * a.dim + d] = from_float<E>(y);
}


}  // namespace sscan
}  // namespace ssd
