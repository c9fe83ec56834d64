// conv_kernels.hpp -- the causal convolution with a carried window, forward, backward and one
// token, for gfx950.
//
//   v_t = bias + sum_k w[k] x_{t-K+1+k},  y_t = SiLU(v_t) or v_t        for every channel
//   dv_t = dy_t SiLU'(v_t),  dx_t = sum_d w[K-1-d] dv_{t+d},  dw[k] = sum_t dv_t x_{t-K+1+k}
//
// Bound by its bytes: a thread has V neighbouring channels (four, at any element; one where there
// are fewer) and walks a strip of tokens with the last K-1 inputs in
// registers, so that every row is read once, but for the K-1 rows around a strip.  The inputs
// before a sequence's first token are its window's.
#pragma once

#include <type_traits>

#include "segment_ids.hpp"
#include "ssd_device.hpp"

namespace ssd {
namespace conv {

struct ConvArgs {
    const void *x;
    int64_t xs;              // elements from token to token
    const float *w, *bias;
    const void *win0;        // windows [rows][K-1][C]
    const int32_t *ids;      // packed streams: segment ids
    void *y, *win1;
    const void *dy, *dwin1;
    void *dx, *dwin0;
    float *parts;            // dweight, dbias of every strip [strips][K+1][C]
    int T, C, rows, nb, strip, silu;
    int ahead;               // workgroups in front of the strips': windows of segments without tokens
    int64_t items;           // threads: rows of strips times vectors of a row
};

// V elements of E as they are in memory, and as floats.
template <typename E, int V> using vec_t = typename std::conditional<V * sizeof(E) == 16, uint4, typename std::conditional<V * sizeof(E) == 8, uint2, E>::type>::type;
template <typename E, int V> __device__ __forceinline__ void to_floats(const vec_t<E, V> &r, float (&o)[V])
{
    if constexpr (V == 1) o[0] = to_float(r);
    else {
        typedef E ev __attribute__((ext_vector_type(V)));
        typedef float fv __attribute__((ext_vector_type(V)));
        const fv f = __builtin_convertvector(__builtin_bit_cast(ev, r), fv);
#pragma unroll
        for (int i = 0; i < V; ++i) o[i] = f[i];
    }
}
template <typename E, int V> __device__ __forceinline__ vec_t<E, V> from_floats(const float (&v)[V])
{
    if constexpr (V == 1) return from_float<E>(v[0]);
    else {
        typedef E ev __attribute__((ext_vector_type(V)));
        typedef float fv __attribute__((ext_vector_type(V)));
        fv f;
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = v[i];
        return __builtin_bit_cast(vec_t<E, V>, __builtin_convertvector(f, ev));   // to nearest even
    }
}
// In memory they are aligned to an element only.
template <typename E, int V> using any_t = E __attribute__((ext_vector_type(V), aligned(sizeof(E))));
template <typename E, int V> __device__ __forceinline__ vec_t<E, V> load_vec(const void *p, int64_t at)
{
    if constexpr (V == 1) return static_cast<const E *>(p)[at];
    else {
        typedef E ev __attribute__((ext_vector_type(V)));
        const ev v = *reinterpret_cast<const any_t<E, V> *>(static_cast<const E *>(p) + at);
        return __builtin_bit_cast(vec_t<E, V>, v);
    }
}
template <typename E, int V> __device__ __forceinline__ void store_raw(void *p, int64_t at, const vec_t<E, V> &v)
{
    if constexpr (V == 1) static_cast<E *>(p)[at] = v;
    else {
        typedef E ev __attribute__((ext_vector_type(V)));
        *reinterpret_cast<any_t<E, V> *>(static_cast<E *>(p) + at) = __builtin_bit_cast(ev, v);
    }
}
template <typename E, int V> __device__ __forceinline__ void store_vec(void *p, int64_t at, const float (&v)[V])
{
    store_raw<E, V>(p, at, from_floats<E, V>(v));
}

// A thread's place: its channels c .., its sequence row b and first token.
struct Strip {
    int c, t0, t1;       // tokens [t0, t1) of the row
    int64_t row0;        // the row's first token
    int64_t index;       // number of the strip
    int b;
};
template <int V> __device__ __forceinline__ bool strip_of(const ConvArgs &a, Strip &s)
{
    // XCD-aware order: strips that share rows run on one XCD
    const int64_t it = (int64_t)xcd_remap(blockIdx.x - a.ahead, gridDim.x - a.ahead) * kThreads + threadIdx.x;
    if (it >= a.items) return false;
    // the last channels of a number that V does not divide are two threads', which write the same values
    const int gv = (a.C + V - 1) / V;
    s.index = it / gv;
    s.c = (int)(it - s.index * gv) * V;
    if (s.c > a.C - V) s.c = a.C - V;
    s.b = (int)(s.index / a.nb);
    s.t0 = (int)(s.index - (int64_t)s.b * a.nb) * a.strip;
    s.t1 = a.T - s.t0 < a.strip ? a.T : s.t0 + a.strip;
    s.row0 = (int64_t)s.b * a.T;
    return true;
}
// Row `i` of sequence `seq`'s window (zeros without one, or for an id out of range).
template <typename E, int V, int K>
__device__ __forceinline__ void window_row(const ConvArgs &a, const void *win, int seq, int i, int c, float (&o)[V])
{
#pragma unroll
    for (int e = 0; e < V; ++e) o[e] = 0.f;
    if (win && (unsigned)seq < (unsigned)a.rows) to_floats<E, V>(load_vec<E, V>(win, ((int64_t)seq * (K - 1) + i) * a.C + c), o);
}
template <typename E, int V, int K>
__device__ __forceinline__ void put_window_row(const ConvArgs &a, void *win, int seq, int i, int c, const float (&v)[V])
{
    if ((unsigned)seq < (unsigned)a.rows) store_vec<E, V>(win, ((int64_t)seq * (K - 1) + i) * a.C + c, v);
}
// Windows of the segments without tokens: from -> to (zeros without a `from`), V channels of one segment a thread, in workgroups
// of their own, the launch's first (64 tokens and 65536 segments, 16 channels, bf16: 11 us; with a segment after
// another in the thread of the strip in front of them 43 ms).
template <typename E, int V, int K> __device__ __forceinline__ void pass_windows(const ConvArgs &a, const void *from, void *to)
{
    const int gv = (a.C + V - 1) / V;
    const int64_t it = (int64_t)blockIdx.x * kThreads + threadIdx.x, q = it / gv;
    if (q >= a.rows) return;
    const int at = first_from(a.ids, a.T, (int)q);
    if (at < a.T && a.ids[at] == (int)q) return;
    int c = (int)(it - q * gv) * V;
    if (c > a.C - V) c = a.C - V;
#pragma unroll
    for (int i = 0; i < K - 1; ++i) {
        float v[V];
        window_row<E, V, K>(a, from, (int)q, i, c, v);
        put_window_row<E, V, K>(a, to, (int)q, i, c, v);
    }
}
// The last K-1 inputs before the strip's first token, and how many of them (up to K-1) are of
// its sequence.
template <typename E, int V, int K, bool PACKED>
__device__ __forceinline__ int history(const ConvArgs &a, const Strip &s, int seq, float (&hist)[K][V])
{
    int p = 0;
    if constexpr (PACKED) {
#pragma unroll
        for (int d = 1; d < K; ++d)
            if (p == d - 1 && s.t0 - d >= 0 && a.ids[s.t0 - d] == seq) p = d;
    } else p = s.t0 < K - 1 ? s.t0 : K - 1;
#pragma unroll
    for (int i = 0; i < K - 1; ++i) {
        if (K - 1 - i <= p) to_floats<E, V>(load_vec<E, V>(a.x, (s.row0 + s.t0 - (K - 1) + i) * a.xs + s.c), hist[i]);
        else window_row<E, V, K>(a, a.win0, seq, p + i, s.c, hist[i]);
    }
    return p;
}
template <int V, int K> __device__ __forceinline__ void load_taps(const ConvArgs &a, int c, float (&w)[K][V], float (&bias)[V])
{
#pragma unroll
    for (int e = 0; e < V; ++e) {
        bias[e] = a.bias ? a.bias[c + e] : 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k) w[k][e] = a.w[(int64_t)(c + e) * K + k];
    }
}

// All of a strip's rows are loaded before the first is used: 16 of them.  Packed prompts of
// 18 K tokens, 5120 channels, bf16: 97 us with 16 (105 with 8, 195 with 32, which leave too few
// waves), 3.8 of the 5.05 TB/s
// that a large copy reaches; the rest is the 3 rows that a strip reads twice, and SiLU.
constexpr int kFwdStrip = 16;

template <typename E, int V, int K, bool PACKED>
__global__ __launch_bounds__(kThreads) void k_conv_fwd(ConvArgs a)
{
    if (PACKED && (int)blockIdx.x < a.ahead) {
        pass_windows<E, V, K>(a, a.win0, a.win1);
        return;
    }
    Strip s;
    if (!strip_of<V>(a, s)) return;
    vec_t<E, V> raw[kFwdStrip];
    int id[PACKED ? kFwdStrip + 1 : 1];
#pragma unroll
    for (int j = 0; j < kFwdStrip; ++j) {
        const int t = s.t0 + j < s.t1 ? s.t0 + j : s.t1 - 1;
        raw[j] = load_vec<E, V>(a.x, (s.row0 + t) * a.xs + s.c);
        if constexpr (PACKED) id[j] = a.ids[t];
    }
    if constexpr (PACKED) id[kFwdStrip] = s.t1 < a.T ? a.ids[s.t1] : a.rows;
    float w[K][V], bias[V], hist[K][V];
    load_taps<V, K>(a, s.c, w, bias);
    history<E, V, K, PACKED>(a, s, PACKED ? id[0] : s.b, hist);
#pragma unroll
    for (int j = 0; j < kFwdStrip; ++j) {
        const int t = s.t0 + j;
        if (t >= s.t1) break;
        const int seq = PACKED ? id[PACKED ? j : 0] : s.b;
        if constexpr (PACKED)
            if (j > 0 && seq != id[j > 0 ? j - 1 : 0])
#pragma unroll
                for (int i = 0; i < K - 1; ++i) window_row<E, V, K>(a, a.win0, seq, i, s.c, hist[i]);
        to_floats<E, V>(raw[j], hist[K - 1]);
        float o[V];
#pragma unroll
        for (int e = 0; e < V; ++e) o[e] = bias[e];
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int e = 0; e < V; ++e) o[e] += w[k][e] * hist[k][e];
        if (a.silu)
#pragma unroll
            for (int e = 0; e < V; ++e) o[e] = silu(o[e]);
        store_vec<E, V>(a.y, (s.row0 + t) * a.C + s.c, o);
#pragma unroll
        for (int k = 0; k < K - 1; ++k)
#pragma unroll
            for (int e = 0; e < V; ++e) hist[k][e] = hist[k + 1][e];
        // the id behind the last token of the strip is the next strip's
        const int next = PACKED ? (t == s.t1 - 1 ? id[PACKED ? kFwdStrip : 0] : id[PACKED ? j + 1 : 0]) : 0;
        const bool end = PACKED ? t == a.T - 1 || next != seq : t == a.T - 1;
        if (a.win1 && end)
#pragma unroll
            for (int i = 0; i < K - 1; ++i) put_window_row<E, V, K>(a, a.win1, seq, i, s.c, hist[i]);
    }
}

// The gradients.  Walking up a strip, token t adds w[K-1-d] dv_t to the K gradients that it
// reaches, those of tokens t - d, which wait in `pend` until token t + K - 1 has added its
// share; what reaches before the sequence's first token belongs to its window.  K - 1 tokens
// past the strip are formed again for the strip's last gradients.  Four tokens are in flight.
// 16384 tokens of 5120 channels in bf16: 123 us and 10 us for the sums of the strips, 4.1 and
// 3.8 TB/s; a branch for tokens away from a sequence's start takes 9 multiplications out.
template <typename E, int V, int K, bool PACKED>
__global__ __launch_bounds__(kThreads) void k_conv_bwd(ConvArgs a)
{
    if (PACKED && (int)blockIdx.x < a.ahead) {
        pass_windows<E, V, K>(a, a.dwin1, a.dwin0);
        return;
    }
    Strip s;
    if (!strip_of<V>(a, s)) return;
    constexpr int U = 4;   // tokens in flight
    float w[K][V], bias[V], hist[K][V], pend[K][V], dw[K][V], db[V], dwin[K][V];
    load_taps<V, K>(a, s.c, w, bias);
#pragma unroll
    for (int e = 0; e < V; ++e) {
        db[e] = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k) pend[k][e] = dw[k][e] = dwin[k][e] = 0.f;
    }
    const int stop = s.t1 + K - 1;   // one past the last token looked at
    vec_t<E, V> xr[U], gr[U];
    int idr[U];
    auto fetch = [&](int t) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int tt = t + u < a.T ? t + u : a.T - 1;
            xr[u] = load_vec<E, V>(a.x, (s.row0 + tt) * a.xs + s.c);
            gr[u] = load_vec<E, V>(a.dy, (s.row0 + tt) * a.C + s.c);
            idr[u] = PACKED ? a.ids[tt] : s.b;
        }
    };
    fetch(s.t0);
    int seq = idr[0];
    int q = history<E, V, K, PACKED>(a, s, seq, hist);   // tokens of the sequence before this one, up to K - 1
    bool own = q == 0;   // the sequence's first token is in this strip
    for (int tb = s.t0; tb < stop; tb += U) {
        vec_t<E, V> xc[U], gc[U];
        int ic[U + 1];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            xc[u] = xr[u];
            gc[u] = gr[u];
            ic[u] = idr[u];
        }
        if (tb + U < stop || PACKED) fetch(tb + U);
        ic[U] = idr[0];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int t = tb + u;
            if (t >= stop) break;
            const bool in = t < a.T;
            if (PACKED && in && ic[u] != seq) {
                seq = ic[u];
                q = 0;
                own = t < s.t1;
#pragma unroll
                for (int i = 0; i < K - 1; ++i) window_row<E, V, K>(a, a.win0, seq, i, s.c, hist[i]);
#pragma unroll
                for (int k = 0; k < K; ++k)
#pragma unroll
                    for (int e = 0; e < V; ++e) dwin[k][e] = 0.f;
            }
            float dv[V];
            to_floats<E, V>(xc[u], hist[K - 1]);
            to_floats<E, V>(gc[u], dv);
            if (a.silu) {
                float v[V];
#pragma unroll
                for (int e = 0; e < V; ++e) v[e] = bias[e];
#pragma unroll
                for (int k = 0; k < K; ++k)
#pragma unroll
                    for (int e = 0; e < V; ++e) v[e] += w[k][e] * hist[k][e];
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float sg = __builtin_amdgcn_rcpf(1.f + exp2_(-v[e] * kLog2e));
                    dv[e] *= sg * (1.f + v[e] * (1.f - sg));
                }
            }
            if (!in)
#pragma unroll
                for (int e = 0; e < V; ++e) dv[e] = 0.f;
            if (t < s.t1)
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    db[e] += dv[e];
#pragma unroll
                    for (int k = 0; k < K; ++k) dw[k][e] += dv[e] * hist[k][e];
                }
#pragma unroll
            for (int e = 0; e < V; ++e) pend[K - 1][e] = 0.f;
            if (q == K - 1) {
#pragma unroll
                for (int d = 0; d < K; ++d)
#pragma unroll
                    for (int e = 0; e < V; ++e) pend[K - 1 - d][e] += w[K - 1 - d][e] * dv[e];
            } else {   // near the sequence's start
#pragma unroll
                for (int d = 0; d < K; ++d)
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        const float g = w[K - 1 - d][e] * dv[e];
                        pend[K - 1 - d][e] += d <= q ? g : 0.f;
                        // row K - 1 + q - d of the window
#pragma unroll
                        for (int r = 0; r < K - 1; ++r) dwin[r][e] += r == K - 1 + q - d && d > q ? g : 0.f;
                    }
            }
            const bool end = in && (t == a.T - 1 || (PACKED && ic[u + 1] != seq));
            if (end && a.dwin1) {
#pragma unroll
                for (int d = 0; d < K - 1; ++d) {   // the window's row K - 2 - d is token t - d
                    float g[V];
                    window_row<E, V, K>(a, a.dwin1, seq, K - 2 - d, s.c, g);
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        pend[K - 1 - d][e] += d <= q ? g[e] : 0.f;
#pragma unroll
                        for (int r = 0; r < K - 1; ++r) dwin[r][e] += r == K - 1 + q - d && d > q ? g[e] : 0.f;
                    }
                }
            }
            if (K > 1 && a.dwin0 && own && in && (end || q == K - 2)) {
                own = false;
#pragma unroll
                for (int i = 0; i < K - 1; ++i) put_window_row<E, V, K>(a, a.dwin0, seq, i, s.c, dwin[i]);
            }
            const int done = t - (K - 1);
            if (done >= s.t0 && done < s.t1) store_vec<E, V>(a.dx, (s.row0 + done) * a.C + s.c, pend[0]);
#pragma unroll
            for (int k = 0; k < K - 1; ++k)
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    hist[k][e] = hist[k + 1][e];
                    pend[k][e] = pend[k + 1][e];
                }
            q = q < K - 1 ? q + 1 : K - 1;
        }
    }
    float *out = a.parts + s.index * (K + 1) * a.C + s.c;
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int e = 0; e < V; ++e) out[(int64_t)k * a.C + e] = dw[k][e];
#pragma unroll
    for (int e = 0; e < V; ++e) out[(int64_t)K * a.C + e] = db[e];
}

// dweight [C][K] and dbias from the strips' sums [strips][K+1][C]: 32 columns and 32 slices.
__global__ __launch_bounds__(1024) void k_conv_sum(const float *__restrict__ parts, float *__restrict__ dweight,
                                                   float *__restrict__ dbias, int strips, int C, int K)
{
    __shared__ float s[32][33];
    const int cl = threadIdx.x & 31, sl = threadIdx.x >> 5;
    const int64_t e = (int64_t)blockIdx.x * 32 + cl, n = (int64_t)(K + 1) * C;
    float v = 0.f;
    if (e < n)
        for (int r = sl; r < strips; r += 32) v += parts[r * n + e];
    s[sl][cl] = v;
    __syncthreads();
    if (sl == 0 && e < n) {
        float t = 0.f;
#pragma unroll
        for (int r = 0; r < 32; ++r) t += s[r][cl];
        const int k = (int)(e / C), c = (int)(e - (int64_t)k * C);
        if (k < K) dweight[(int64_t)c * K + k] = t;
        else if (dbias) dbias[c] = t;
    }
}

// No tokens: the windows stay as they are.
template <typename E> __global__ __launch_bounds__(kThreads) void k_conv_keep(const E *from, E *to, int64_t n)
{
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (i < n) to[i] = from ? from[i] : from_float<E>(0.f);
}

template <typename E, int V, int K>
__global__ __launch_bounds__(kThreads) void k_conv_step(const E *__restrict__ x, int64_t xs, const float *__restrict__ w,
                                                        const float *__restrict__ bias, E *__restrict__ window,
                                                        E *__restrict__ y, int64_t items, int C, int act)
{
    const int64_t it = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (it >= items) return;
    const int gv = C / V;
    const int64_t b = it / gv;
    const int c = (int)(it - b * gv) * V;
    vec_t<E, V> raw[K];
#pragma unroll
    for (int i = 0; i < K - 1; ++i) raw[i] = load_vec<E, V>(window, (b * (K - 1) + i) * C + c);
    raw[K - 1] = load_vec<E, V>(x, b * xs + c);
    float o[V];
#pragma unroll
    for (int e = 0; e < V; ++e) o[e] = bias ? bias[c + e] : 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        float v[V];
        to_floats<E, V>(raw[k], v);
#pragma unroll
        for (int e = 0; e < V; ++e) o[e] += w[(int64_t)(c + e) * K + k] * v[e];
    }
    if (act)
#pragma unroll
        for (int e = 0; e < V; ++e) o[e] = silu(o[e]);
    store_vec<E, V>(y, b * C + c, o);
#pragma unroll
    for (int i = 0; i < K - 1; ++i) store_raw<E, V>(window, (b * (K - 1) + i) * C + c, raw[i + 1]);
}

}  // namespace conv
}  // namespace ssd
