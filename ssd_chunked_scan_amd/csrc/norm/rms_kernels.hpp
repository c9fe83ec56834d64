// rms_kernels.hpp -- root-mean-square norm with the residual's addition, forward (to the dtype
// or to 8 bits with a scale for every 128 values) and backward, for gfx950.
//
//   r = x + residual (rounded to the residual's type),  y = r rstd w,  rstd = 1 / sqrt(avg(r^2) + eps)
//   dr = rstd (g - hat avg(g hat)) + dresidual,  g = dy w,  hat = r rstd,  dw = sum over rows of dy hat
//
// Bound by bytes: a row is read once into registers, summed there and written once.  L lanes share a
// row, each with IT runs of 8 neighbouring values (16 bytes of bf16, 32 of fp32), so that a block
// of 128 values, which shares a scale, lies in 16 lanes: one DPP row.  Rows whose length is not a
// multiple of 8 start at any element: the same vectors, not aligned (8000 rows of 2561, fp32: 66 us; by single
// elements 186 us), and single elements where the row's end cuts a run.
//
// The backward's sum over rows: every workgroup keeps its lanes' columns in registers over a strip of
// rows, joins its row groups through LDS and writes one fp32 row of partial sums; a second kernel
// adds those.  No atomics: the order is fixed.
#pragma once

#include <type_traits>

#include "ssd_device.hpp"

namespace ssd {
namespace rms {

constexpr int kRun = 8;            // values of a lane's run
constexpr float kMax8 = 448.f;     // largest e4m3 value
constexpr float kLeastScale = 0x1p-126f;
constexpr int kDppRowMirror = 0x140;

// A run of 8 values as it is in memory.
template <typename T> struct Run {
    uint4 v[(int)sizeof(T) / 2];
};
// Vectors in memory that are aligned to an element only.
template <typename T, typename V, int N> using any_t = V __attribute__((ext_vector_type(N), aligned(sizeof(T))));
// Loads the run at column c of a row; past the row's end its first values are loaded instead
// (`unpack_run` drops them).  AL: rows are whole runs, which start at 16 bytes; otherwise vectors start
// at any element, and a run that the row's end cuts is loaded by single elements.
template <bool AL, typename T> __device__ __forceinline__ void load_run(Run<T> &r, const T *row, int c, int dim)
{
    if constexpr (AL) {
        typedef unsigned int uint4v __attribute__((ext_vector_type(4)));
        const uint4v *p = reinterpret_cast<const uint4v *>(row + (c < dim ? c : 0));
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.v[i] = __builtin_bit_cast(uint4, __builtin_nontemporal_load(p + i));   // read once
    } else if (c + kRun <= dim) {
        typedef any_t<T, unsigned int, 4> uint4v;
        const uint4v *p = reinterpret_cast<const uint4v *>(row + c);
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.v[i] = uint4{p[i].x, p[i].y, p[i].z, p[i].w};
    } else {
        typedef T tv __attribute__((ext_vector_type(16 / sizeof(T))));
        constexpr int W = 16 / (int)sizeof(T);
#pragma unroll
        for (int i = 0; i < kRun / W; ++i) {
            tv t;
#pragma unroll
            for (int e = 0; e < W; ++e) t[e] = row[c + i * W + e < dim ? c + i * W + e : 0];
            r.v[i] = __builtin_bit_cast(uint4, t);
        }
    }
}
template <bool AL, typename T> __device__ __forceinline__ void unpack_run(const Run<T> &r, float (&o)[kRun], int c, int dim)
{
    if constexpr (sizeof(T) == 2) {
        const floatx8 f = __builtin_convertvector(__builtin_bit_cast(bf16x8, r.v[0]), floatx8);
#pragma unroll
        for (int e = 0; e < kRun; ++e) o[e] = f[e];
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            o[4 * i] = __uint_as_float(r.v[i].x);
            o[4 * i + 1] = __uint_as_float(r.v[i].y);
            o[4 * i + 2] = __uint_as_float(r.v[i].z);
            o[4 * i + 3] = __uint_as_float(r.v[i].w);
        }
    }
#pragma unroll
    for (int e = 0; e < kRun; ++e)
        if ((AL ? c : c + e) >= dim) o[e] = 0.f;
}
template <bool AL, typename T> __device__ __forceinline__ void store_run(T *row, const float (&v)[kRun], int c, int dim)
{
    if (AL ? c < dim : c + kRun <= dim) {
        if constexpr (sizeof(T) == 2) {
            floatx8 f;
#pragma unroll
            for (int e = 0; e < kRun; ++e) f[e] = v[e];
            const bf16x8 o = __builtin_convertvector(f, bf16x8);
            if constexpr (AL) *reinterpret_cast<bf16x8 *>(row + c) = o;
            else *reinterpret_cast<any_t<T, T, 8> *>(row + c) = o;
        } else if constexpr (AL) {
            store4_f32(row + c, v);
            store4_f32(row + c + 4, v + 4);
        } else {
#pragma unroll
            for (int i = 0; i < kRun; i += 4)
                *reinterpret_cast<any_t<T, T, 4> *>(row + c + i) = any_t<T, T, 4>{v[i], v[i + 1], v[i + 2], v[i + 3]};
        }
    } else if constexpr (!AL) {
#pragma unroll
        for (int e = 0; e < kRun; ++e)
            if (c + e < dim) row[c + e] = from_float<T>(v[e]);
    }
}
template <bool AL> __device__ __forceinline__ void load_weight(const float *w, float (&o)[kRun], int c, int dim)
{
#pragma unroll
    for (int e = 0; e < kRun; ++e) o[e] = 1.f;
    if (!w) return;
    // weights start at 16 bytes, and so do a row's runs of them
    if (AL || c + kRun <= dim) {
        const int cc = c < dim ? c : 0;
        load4_f32(w + cc, o);
        load4_f32(w + cc + 4, o + 4);
    } else {
#pragma unroll
        for (int e = 0; e < kRun; ++e) o[e] = w[c + e < dim ? c + e : 0];
    }
}

// The sum over the L lanes of a row (L > 64: the whole workgroup, through `red`, L / 64 floats that
// no earlier sum may still be reading).
template <int L> __device__ __forceinline__ float row_sum(float a, float *red)
{
#pragma unroll
    for (int d = 1; d < (L < 64 ? L : 64); d <<= 1) a += __shfl_xor(a, d);
    if constexpr (L > 64) {
        if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = a;
        __syncthreads();
        a = 0.f;
#pragma unroll
        for (int i = 0; i < L / 64; ++i) a += red[i];
    }
    return a;
}
// The largest over the 16 lanes of a DPP row.
__device__ __forceinline__ float max16(float v)
{
    v = fmaxf(v, dpp_mov<kDppQuadXor1>(v));
    v = fmaxf(v, dpp_mov<kDppQuadXor2>(v));
    v = fmaxf(v, dpp_mov<kDppRowHalfMirror>(v));
    return fmaxf(v, dpp_mov<kDppRowMirror>(v));
}

// A run's values times `inv` as e4m3, to nearest even; `left`: values up to the row's end.
template <bool AL> __device__ __forceinline__ void put_8bit(uint8_t *q, const float (&w)[kRun], float inv, int left)
{
    uint32_t b[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int p = __builtin_amdgcn_cvt_pk_fp8_f32(w[4 * h] * inv, w[4 * h + 1] * inv, 0, false);
        b[h] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(w[4 * h + 2] * inv, w[4 * h + 3] * inv, p, true);
    }
    if constexpr (AL) *reinterpret_cast<uint2 *>(q) = uint2{b[0], b[1]};
    else if (left >= kRun) *reinterpret_cast<any_t<uint8_t, unsigned int, 2> *>(q) = any_t<uint8_t, unsigned int, 2>{b[0], b[1]};
    else
#pragma unroll
        for (int e = 0; e < kRun; ++e)
            if (e < left) q[e] = (uint8_t)(b[e / 4] >> (8 * (e % 4)));
}

struct FwdArgs {
    const void *x, *res;
    const float *w;
    void *res_out, *y;
    uint8_t *q;
    float *scales, *rstd;
    int64_t rows;
    int dim;
    float eps;
};

// Threads of a workgroup: L = 1024 a row, else 256 or (few rows) 64, whole rows each.
template <typename E, typename R, bool RES, bool AL, int L, int IT>
__global__ __launch_bounds__(L > kThreads ? L : kThreads) void k_rms_fwd(FwdArgs a)
{
    __shared__ float red[L > 64 ? L / 64 : 1];
    const int ln = threadIdx.x % L;
    const int64_t row = (int64_t)blockIdx.x * (blockDim.x / L) + threadIdx.x / L;
    if (L <= 64 && row >= a.rows) return;   // longer rows: one a workgroup, always there
    const E *x = static_cast<const E *>(a.x) + row * a.dim;
    const R *res = static_cast<const R *>(a.res) + row * a.dim;
    Run<E> rx[IT];
    Run<R> rr[RES ? IT : 1];
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        const int c = (i * L + ln) * kRun;
        load_run<AL>(rx[i], x, c, a.dim);
        if constexpr (RES) load_run<AL>(rr[i], res, c, a.dim);
    }
    float v[IT][kRun], s = 0.f;
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        const int c = (i * L + ln) * kRun;
        unpack_run<AL>(rx[i], v[i], c, a.dim);
        if constexpr (RES) {
            float o[kRun];
            unpack_run<AL>(rr[i], o, c, a.dim);
#pragma unroll
            for (int e = 0; e < kRun; ++e) v[i][e] = to_float(from_float<R>(v[i][e] + o[e]));   // what the stream holds
            store_run<AL>(static_cast<R *>(a.res_out) + row * a.dim, v[i], c, a.dim);
        }
#pragma unroll
        for (int e = 0; e < kRun; ++e) s += v[i][e] * v[i][e];
    }
    s = row_sum<L>(s, red);
    const float rs = 1.f / sqrtf(s / (float)a.dim + a.eps);
    if (ln == 0 && a.rstd) a.rstd[row] = rs;
    const int nb = (a.dim + 127) / 128;
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        const int c = (i * L + ln) * kRun;
        float w[kRun], m = 0.f;
        load_weight<AL>(a.w, w, c, a.dim);
#pragma unroll
        for (int e = 0; e < kRun; ++e) {
            w[e] = v[i][e] * rs * w[e];
            m = fmaxf(m, fabsf(w[e]));
        }
        if (a.y) store_run<AL>(static_cast<E *>(a.y) + row * a.dim, w, c, a.dim);
        if (!a.q) continue;
        const float scale = fmaxf(max16(m) / kMax8, kLeastScale), inv = 1.f / scale;
        if (c >= a.dim) continue;
        if ((ln & 15) == 0) a.scales[row * nb + c / 128] = scale;
        put_8bit<AL>(a.q + row * a.dim + c, w, inv, a.dim - c);
    }
}

// Rows too long for the registers of the above, a workgroup each: read twice (with a residual the
// second time from residual_out).
constexpr int kLong = 1024;
template <typename E, typename R, bool RES> __global__ __launch_bounds__(kLong) void k_rms_fwd_long(FwdArgs a)
{
    __shared__ float red[kLong / 64];
    const int64_t at = (int64_t)blockIdx.x * a.dim;
    const E *x = static_cast<const E *>(a.x) + at;
    const R *res = static_cast<const R *>(a.res) + at;
    R *out = static_cast<R *>(a.res_out) + at;
    const int nb = (a.dim + 127) / 128;
    float s = 0.f;
    for (int c = threadIdx.x * kRun; c < a.dim; c += kLong * kRun)
#pragma unroll
        for (int e = 0; e < kRun; ++e) {
            if (c + e >= a.dim) break;
            float v = to_float(x[c + e]);
            if constexpr (RES) {
                const R r = from_float<R>(v + to_float(res[c + e]));
                out[c + e] = r;
                v = to_float(r);
            }
            s += v * v;
        }
    s = row_sum<kLong>(s, red);
    const float rs = 1.f / sqrtf(s / (float)a.dim + a.eps);
    if (threadIdx.x == 0 && a.rstd) a.rstd[blockIdx.x] = rs;
    // whole rounds, so that the 16 lanes of a block of 128 take part together
    for (int c0 = 0; c0 < a.dim; c0 += kLong * kRun) {
        const int c = c0 + threadIdx.x * kRun;
        float w[kRun], m = 0.f;
#pragma unroll
        for (int e = 0; e < kRun; ++e) {
            w[e] = 0.f;
            if (c + e >= a.dim) continue;
            w[e] = (RES ? to_float(out[c + e]) : to_float(x[c + e])) * rs * (a.w ? a.w[c + e] : 1.f);
            m = fmaxf(m, fabsf(w[e]));
        }
        const float scale = fmaxf(max16(m) / kMax8, kLeastScale), inv = 1.f / scale;
        if (c >= a.dim) continue;
        if (a.y) store_run<false>(static_cast<E *>(a.y) + at, w, c, a.dim);
        if (!a.q) continue;
        if ((threadIdx.x & 15) == 0) a.scales[(int64_t)blockIdx.x * nb + c / 128] = scale;
        put_8bit<false>(a.q + at + c, w, inv, a.dim - c);
    }
}

struct BwdArgs {
    const void *r, *dy, *dres;
    const float *rstd, *w;
    void *dx, *dr;
    float *parts;
    int64_t rows;
    int dim, strip;
};

// Rows [strip * blockIdx.x, ...) of the workgroup, and their part of dweight, parts[blockIdx.x][dim].
template <typename E, typename R, bool DRES, bool AL, int L, int IT>
__global__ __launch_bounds__(L > kThreads ? L : kThreads) void k_rms_bwd(BwdArgs a)
{
    constexpr int NT = L > kThreads ? L : kThreads, G = NT / L;   // rows at a time
    __shared__ float red[2][L > 64 ? L / 64 : 1];
    __shared__ float join[G > 1 ? G * L * IT * kRun : 1];
    const int ln = threadIdx.x % L, rg = threadIdx.x / L;
    float w[IT][kRun], dw[IT][kRun];
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        load_weight<AL>(a.w, w[i], (i * L + ln) * kRun, a.dim);
#pragma unroll
        for (int e = 0; e < kRun; ++e) dw[i][e] = 0.f;
    }
    const int64_t r0 = (int64_t)blockIdx.x * a.strip, r1 = r0 + a.strip < a.rows ? r0 + a.strip : a.rows;
    // the next row is on its way while this one is summed; rows past the strip load its first
    Run<R> nr[IT], nd[DRES ? IT : 1];
    Run<E> ng[IT];
    float nrs;
    auto fetch = [&](int64_t row) {
        const int64_t rr = row < r1 ? row : r0, at = rr * a.dim;
        nrs = a.rstd[rr];
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int c = (i * L + ln) * kRun;
            load_run<AL>(nr[i], static_cast<const R *>(a.r) + at, c, a.dim);
            load_run<AL>(ng[i], static_cast<const E *>(a.dy) + at, c, a.dim);
            if constexpr (DRES) load_run<AL>(nd[i], static_cast<const R *>(a.dres) + at, c, a.dim);
        }
    };
    const float inv = 1.f / (float)a.dim;
    fetch(r0 + rg);
    int flip = 0;
    for (int64_t rb = r0; rb < r1; rb += G, flip ^= 1) {
        const int64_t row = rb + rg, at = row * a.dim;
        const bool live = row < r1;   // the whole row group agrees
        float h[IT][kRun], g[IT][kRun];
        Run<R> cd[DRES ? IT : 1];
        const float rs = nrs;
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int c = live ? (i * L + ln) * kRun : a.dim;
            unpack_run<AL>(nr[i], h[i], c, a.dim);
            unpack_run<AL>(ng[i], g[i], c, a.dim);
            if constexpr (DRES) cd[i] = nd[i];
        }
        if (rb + G < r1) fetch(row + G);
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < IT; ++i)
#pragma unroll
            for (int e = 0; e < kRun; ++e) {
                h[i][e] *= rs;
                dw[i][e] += g[i][e] * h[i][e];
                g[i][e] *= w[i][e];
                s += g[i][e] * h[i][e];
            }
        s = row_sum<L>(s, red[flip]) * inv;
        if (!live) continue;
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int c = (i * L + ln) * kRun;
            float o[kRun];
            if constexpr (DRES) unpack_run<AL>(cd[i], o, c, a.dim);
#pragma unroll
            for (int e = 0; e < kRun; ++e) o[e] = rs * (g[i][e] - h[i][e] * s) + (DRES ? o[e] : 0.f);
            store_run<AL>(static_cast<E *>(a.dx) + at, o, c, a.dim);
            if (a.dr) store_run<AL>(static_cast<R *>(a.dr) + at, o, c, a.dim);
        }
    }
    if (!a.parts) return;
    float *out = a.parts + (int64_t)blockIdx.x * a.dim;
    if constexpr (G > 1) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < IT; ++i)
#pragma unroll
            for (int e = 0; e < kRun; ++e) join[(rg * L * IT + i * L + ln) * kRun + e] = dw[i][e];
        __syncthreads();
        for (int c = threadIdx.x; c < a.dim; c += NT) {
            float s = 0.f;
#pragma unroll
            for (int r = 0; r < G; ++r) s += join[r * L * IT * kRun + c];
            out[c] = s;
        }
    } else {
#pragma unroll
        for (int i = 0; i < IT; ++i)
#pragma unroll
            for (int e = 0; e < kRun; ++e) {
                const int c = (i * L + ln) * kRun + e;
                if (c < a.dim) out[c] = dw[i][e];
            }
    }
}

// Rows too long for the registers of the above: read twice, the sums over rows by columns.
template <typename E, typename R> __global__ __launch_bounds__(kLong) void k_rms_dx_long(BwdArgs a)
{
    __shared__ float red[kLong / 64];
    const int64_t at = (int64_t)blockIdx.x * a.dim;
    const R *r = static_cast<const R *>(a.r) + at, *dres = a.dres ? static_cast<const R *>(a.dres) + at : nullptr;
    const E *dy = static_cast<const E *>(a.dy) + at;
    E *dx = static_cast<E *>(a.dx) + at;
    R *dr = a.dr ? static_cast<R *>(a.dr) + at : nullptr;
    const float rs = a.rstd[blockIdx.x];
    float s = 0.f;
    for (int c = threadIdx.x; c < a.dim; c += kLong) s += to_float(dy[c]) * (a.w ? a.w[c] : 1.f) * (to_float(r[c]) * rs);
    s = row_sum<kLong>(s, red) / (float)a.dim;
    for (int c = threadIdx.x; c < a.dim; c += kLong) {
        const float o = rs * (to_float(dy[c]) * (a.w ? a.w[c] : 1.f) - to_float(r[c]) * rs * s) + (dres ? to_float(dres[c]) : 0.f);
        dx[c] = from_float<E>(o);
        if (dr) dr[c] = from_float<R>(o);
    }
}
template <typename E, typename R> __global__ __launch_bounds__(kThreads) void k_rms_cols_long(BwdArgs a)
{
    const int c = blockIdx.y * kThreads + threadIdx.x;
    if (c >= a.dim) return;
    const int64_t r0 = (int64_t)blockIdx.x * a.strip, r1 = r0 + a.strip < a.rows ? r0 + a.strip : a.rows;
    float s = 0.f;
    for (int64_t r = r0; r < r1; ++r)
        s += to_float(static_cast<const E *>(a.dy)[r * a.dim + c]) * (to_float(static_cast<const R *>(a.r)[r * a.dim + c]) * a.rstd[r]);
    a.parts[(int64_t)blockIdx.x * a.dim + c] = s;
}

// dweight from `n` rows of partial sums: 32 columns and 32 slices of the rows.
__global__ __launch_bounds__(1024) void k_rms_sum(const float *__restrict__ parts, float *__restrict__ dweight, int n, int dim)
{
    __shared__ float s[32][33];
    const int cl = threadIdx.x & 31, sl = threadIdx.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * 32 + cl;
    float v = 0.f;
    if (c < dim)
        for (int r = sl; r < n; r += 32) v += parts[(int64_t)r * dim + c];
    s[sl][cl] = v;
    __syncthreads();
    if (sl == 0 && c < dim) {
        float t = 0.f;
#pragma unroll
        for (int r = 0; r < 32; ++r) t += s[r][cl];
        dweight[c] = t;
    }
}

}  // namespace rms
}  // namespace ssd
