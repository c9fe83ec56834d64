// norm_kernels.hpp -- layer norm over the last axis, forward and backward, for gfx950.
//
//   y = (x - mean) rstd weight + bias
//   dx = rstd (w - avg(w) - xhat avg(w xhat)),  w = dy weight,  xhat = (x - mean) rstd
//   dweight = sum over rows of dy xhat,  dbias = sum over rows of dy
//
// Both directions are bound by the bytes of their rows: every row is read once into
// registers, both of its sums are taken there (the mean first, then the squares
// around it, so no cancellation), and it is written once.  L lanes share a row (16,
// 64 or the whole workgroup, by its length), each holding IT vectors of V elements:
// 16 bytes where dim is a multiple of such a vector, else single elements, since
// the rows of an odd dim start at any address.  Rows longer than the registers
// take the "long" kernels, which read their row again from L2.
//
// The sums over rows: every workgroup keeps its lanes' columns in registers over a
// strip of rows, joins its row groups through LDS and writes one fp32 row of
// partial sums; a second kernel adds those rows.  No atomics: the order is fixed.
//
// 16384 rows of bf16, against 5.1 TB/s of a copy: forward, dim 2560, 168 MB in 37 us (41 with
// ordinary loads); backward, dim 5120, 503 MB in 111 us with other data in the caches and 95
// with its own (147 and 112 with ordinary loads), 7 of them for the sums.  2^26 elements,
// backward, dims 1024 to 5120: 4.8 to 5.2 TB/s in bf16, 5.4 to 6.0 in fp32; rows of odd length
// 3.7 and 4.9, the long kernels, which read twice, 2.3.
#pragma once

#include <type_traits>

#include "ssd_device.hpp"

namespace ssd {
namespace norm {

constexpr int kLongThreads = 1024;

// 16 bytes that are read once: past the caches, whose other contents they would push out and,
// where dirty, have written back first.
__device__ __forceinline__ uint4 load16_once(const void *p)
{
    typedef unsigned int uint4v __attribute__((ext_vector_type(4)));
    return __builtin_bit_cast(uint4, __builtin_nontemporal_load(reinterpret_cast<const uint4v *>(p)));
}
template <int V, typename E> __device__ __forceinline__ void store_v(E *p, const float (&v)[V])
{
    if constexpr (V == 1) *p = from_float<E>(v[0]);
    else if constexpr (V == 4) store4_f32(p, v);
    else {
        floatx8 f;
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = v[i];
        *reinterpret_cast<bf16x8 *>(p) = __builtin_convertvector(f, bf16x8);
    }
}
// A vector as it is in memory (one or four words), and its floats.
template <int V, typename E> struct Raw {
    typedef typename std::conditional<V == 1, E, uint4>::type type;
};
template <int V, typename E> __device__ __forceinline__ void unpack(const typename Raw<V, E>::type &r, float (&o)[V])
{
    if constexpr (V == 1) o[0] = to_float(r);
    else if constexpr (V == 4) {
        o[0] = __uint_as_float(r.x); o[1] = __uint_as_float(r.y);
        o[2] = __uint_as_float(r.z); o[3] = __uint_as_float(r.w);
    } else {
        const floatx8 f = __builtin_convertvector(__builtin_bit_cast(bf16x8, r), floatx8);
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = f[i];
    }
}
// V floats of an fp32 vector at any 4-byte-aligned place of a 16-byte-aligned run.
template <int V> __device__ __forceinline__ void load_p(const float *p, float (&o)[V])
{
    if constexpr (V == 1) o[0] = *p;
    else
#pragma unroll
        for (int i = 0; i < V; i += 4) load4_f32(p + i, o + i);
}

// Two sums over the L lanes of a row.  L <= 64: inside the wave; L = 256: through LDS
// (`red`: 8 floats, free again after the next barrier of the caller).
template <int L> __device__ __forceinline__ void row_sums(float &a, float &b, float *red)
{
#pragma unroll
    for (int d = 1; d < (L < 64 ? L : 64); d <<= 1) {
        a += __shfl_xor(a, d);
        b += __shfl_xor(b, d);
    }
    if constexpr (L > 64) {
        const int w = threadIdx.x >> 6;
        if ((threadIdx.x & 63) == 0) {
            red[w] = a;
            red[4 + w] = b;
        }
        __syncthreads();
        a = red[0] + red[1] + red[2] + red[3];
        b = red[4] + red[5] + red[6] + red[7];
    }
}

// Rows per workgroup at a time: blockDim / L.
template <typename E, int V, int L, int IT>
__global__ __launch_bounds__(kThreads) void k_norm_fwd(const E *x, const float *__restrict__ weight,
                                                       const float *__restrict__ bias, E *y, float *__restrict__ mean,
                                                       float *__restrict__ rstd, int64_t rows, int dim, float eps)
{
    __shared__ float red[16];
    const int ln = threadIdx.x % L;
    const int64_t row = (int64_t)blockIdx.x * (blockDim.x / L) + threadIdx.x / L;
    if (L <= 64 && row >= rows) return;   // L = 256: one row per workgroup, always in range
    const int nv = dim / V;
    const E *xr = x + row * dim;
    float v[IT][V];
    float s = 0.f, z = 0.f;
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        const int c = i * L + ln;
#pragma unroll
        for (int e = 0; e < V; ++e) v[i][e] = 0.f;
        if (c >= nv) continue;
        if constexpr (V == 1) v[i][0] = to_float(xr[c]);
        else unpack<V, E>(load16_once(xr + c * V), v[i]);
    }
#pragma unroll
    for (int i = 0; i < IT; ++i)
#pragma unroll
        for (int e = 0; e < V; ++e) s += v[i][e];
    row_sums<L>(s, z, red);
    const float inv = 1.f / (float)dim, mu = s * inv;
    float q = 0.f;
#pragma unroll
    for (int i = 0; i < IT; ++i)
        if (i * L + ln < nv)
#pragma unroll
            for (int e = 0; e < V; ++e) {
                v[i][e] -= mu;
                q += v[i][e] * v[i][e];
            }
    row_sums<L>(q, z, red + 8);
    const float rs = 1.f / sqrtf(q * inv + eps);
    if (ln == 0) {
        if (mean) mean[row] = mu;
        if (rstd) rstd[row] = rs;
    }
    E *yr = y + row * dim;
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        const int c = i * L + ln;
        if (c >= nv) continue;
        float w[V], b[V];
#pragma unroll
        for (int e = 0; e < V; ++e) {
            w[e] = 1.f;
            b[e] = 0.f;
        }
        if (weight) load_p<V>(weight + c * V, w);
        if (bias) load_p<V>(bias + c * V, b);
#pragma unroll
        for (int e = 0; e < V; ++e) w[e] = v[i][e] * rs * w[e] + b[e];
        store_v<V>(yr + c * V, w);
    }
}

// Rows [strip * blockIdx.x, ...) of the workgroup; PARTS: also the partial sums
// over them, parts[blockIdx.x][2][dim] (dy xhat, then dy).
template <typename E, int V, int L, int IT, bool PARTS>
__global__ __launch_bounds__(kThreads) void k_norm_bwd(const E *__restrict__ x, const E *dy, const float *__restrict__ mean,
                                                       const float *__restrict__ rstd, const float *__restrict__ weight,
                                                       E *dx, float *__restrict__ parts, int64_t rows, int dim, int strip)
{
    constexpr int R = kThreads / L;   // rows at a time
    __shared__ float red[2][8];
    __shared__ float join[PARTS && R > 1 ? R * L * IT * V : 1];
    const int ln = threadIdx.x % L, rg = threadIdx.x / L;
    const int nv = dim / V;
    const float inv = 1.f / (float)dim;
    float dw[PARTS ? IT : 1][V], db[PARTS ? IT : 1][V];
#pragma unroll
    for (int i = 0; i < (PARTS ? IT : 1); ++i)
#pragma unroll
        for (int e = 0; e < V; ++e) dw[i][e] = db[i][e] = 0.f;
    const int64_t r0 = (int64_t)blockIdx.x * strip, r1 = r0 + strip < rows ? r0 + strip : rows;
    // the next row's vectors are on their way while this one is summed; vectors past the row
    // and rows past the strip load its first ones instead of branching
    typename Raw<V, E>::type xr[IT], gr[IT];
    float mu_n, rs_n;
    auto fetch = [&](int64_t row) {
        const int64_t rr = row < r1 ? row : r0, at = rr * dim;
        mu_n = mean[rr];
        rs_n = rstd[rr];
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int c = i * L + ln < nv ? i * L + ln : 0;
            if constexpr (V == 1) {
                xr[i] = x[at + c];
                gr[i] = dy[at + c];
            } else {
                xr[i] = load16_once(x + at + c * V);
                gr[i] = load16_once(dy + at + c * V);
            }
        }
    };
    // this lane's part of the weight, once for all rows (read again for every row it came
    // from L1 beside them: 16384 rows of 5120 bf16 121 -> 102 us, 2^20 of 64 210 -> 136 us,
    // both before the loads went past the caches)
    float wt[IT][V];
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        const int c = i * L + ln < nv ? i * L + ln : 0;
#pragma unroll
        for (int e = 0; e < V; ++e) wt[i][e] = 1.f;
        if (weight) load_p<V>(weight + c * V, wt[i]);
    }
    fetch(r0 + rg);
    int flip = 0;
    for (int64_t rb = r0; rb < r1; rb += R, flip ^= 1) {
        const int64_t row = rb + rg;
        const bool live = row < r1;   // the whole row group agrees
        const int64_t at = row * dim;
        float xv[IT][V], gv[IT][V];
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            unpack<V, E>(xr[i], xv[i]);
            unpack<V, E>(gr[i], gv[i]);
            if (!live)
#pragma unroll
                for (int e = 0; e < V; ++e) xv[i][e] = gv[i][e] = 0.f;
        }
        const float mu = mu_n, rs = rs_n;
        if (rb + R < r1) fetch(row + R);
        float s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int c = i * L + ln;
            if (c >= nv) continue;
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float xh = (xv[i][e] - mu) * rs, gy = gv[i][e];
                if (PARTS) {
                    dw[i][e] += gy * xh;
                    db[i][e] += gy;
                }
                const float gw = gy * wt[i][e];
                xv[i][e] = xh;
                gv[i][e] = gw;
                s1 += gw;
                s2 += gw * xh;
            }
        }
        row_sums<L>(s1, s2, red[flip]);
        s1 *= inv;
        s2 *= inv;
        if (!live) continue;
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int c = i * L + ln;
            if (c >= nv) continue;
            float o[V];
#pragma unroll
            for (int e = 0; e < V; ++e) o[e] = rs * (gv[i][e] - s1 - xv[i][e] * s2);
            store_v<V>(dx + at + c * V, o);
        }
    }
    if constexpr (PARTS) {
        float *out = parts + (int64_t)blockIdx.x * 2 * dim;
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            if constexpr (R == 1) {
#pragma unroll
                for (int i = 0; i < IT; ++i) {
                    const int c = i * L + ln;
                    if (c < nv)
#pragma unroll
                        for (int e = 0; e < V; ++e) out[(int64_t)which * dim + c * V + e] = which ? db[i][e] : dw[i][e];
                }
            } else {
                __syncthreads();
#pragma unroll
                for (int i = 0; i < IT; ++i)
#pragma unroll
                    for (int e = 0; e < V; ++e)
                        join[(rg * L * IT + i * L + ln) * V + e] = which ? db[i][e] : dw[i][e];
                __syncthreads();
                for (int c = threadIdx.x; c < dim; c += kThreads) {
                    float s = 0.f;
#pragma unroll
                    for (int r = 0; r < R; ++r) s += join[r * L * IT * V + c];
                    out[(int64_t)which * dim + c] = s;
                }
            }
        }
    }
}

// dweight and dbias from `n` rows of partial sums: 32 columns x 32 slices of the rows.
__global__ __launch_bounds__(1024) void k_norm_sum(const float *__restrict__ parts, float *__restrict__ dweight,
                                                   float *__restrict__ dbias, int n, int dim)
{
    __shared__ float s[32][33];
    const int cl = threadIdx.x & 31, sl = threadIdx.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * 32 + cl;
    float a = 0.f;
    if (c < 2 * (int64_t)dim)
        for (int r = sl; r < n; r += 32) a += parts[(int64_t)r * 2 * dim + c];
    s[sl][cl] = a;
    __syncthreads();
    if (sl == 0 && c < 2 * (int64_t)dim) {
        float t = 0.f;
#pragma unroll
        for (int r = 0; r < 32; ++r) t += s[r][cl];
        if (c < dim) {
            if (dweight) dweight[c] = t;
        } else if (dbias) dbias[c - dim] = t;
    }
}

// ---- rows longer than the registers: a workgroup of 1024 per row ----
__device__ __forceinline__ void block_sums(float &a, float &b, float *red)
{
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        a += __shfl_xor(a, d);
        b += __shfl_xor(b, d);
    }
    __syncthreads();
    if ((threadIdx.x & 63) == 0) {
        red[threadIdx.x >> 6] = a;
        red[16 + (threadIdx.x >> 6)] = b;
    }
    __syncthreads();
    a = b = 0.f;
#pragma unroll
    for (int i = 0; i < kLongThreads / 64; ++i) {
        a += red[i];
        b += red[16 + i];
    }
}

template <typename E>
__global__ __launch_bounds__(kLongThreads) void k_norm_fwd_long(const E *x, const float *__restrict__ weight,
                                                                const float *__restrict__ bias, E *y,
                                                                float *__restrict__ mean, float *__restrict__ rstd,
                                                                int dim, float eps)
{
    __shared__ float red[32];
    const int64_t row = blockIdx.x;
    const E *xr = x + row * dim;
    float s = 0.f, z = 0.f, q = 0.f;
    for (int c = threadIdx.x; c < dim; c += kLongThreads) s += to_float(xr[c]);
    block_sums(s, z, red);
    const float inv = 1.f / (float)dim, mu = s * inv;
    for (int c = threadIdx.x; c < dim; c += kLongThreads) {
        const float d = to_float(xr[c]) - mu;
        q += d * d;
    }
    block_sums(q, z, red);
    const float rs = 1.f / sqrtf(q * inv + eps);
    if (threadIdx.x == 0) {
        if (mean) mean[row] = mu;
        if (rstd) rstd[row] = rs;
    }
    for (int c = threadIdx.x; c < dim; c += kLongThreads)
        y[row * dim + c] =
            from_float<E>((to_float(xr[c]) - mu) * rs * (weight ? weight[c] : 1.f) + (bias ? bias[c] : 0.f));
}

template <typename E>
__global__ __launch_bounds__(kLongThreads) void k_norm_dx_long(const E *__restrict__ x, const E *dy,
                                                               const float *__restrict__ mean,
                                                               const float *__restrict__ rstd,
                                                               const float *__restrict__ weight, E *dx, int dim)
{
    __shared__ float red[32];
    const int64_t row = blockIdx.x, at = row * dim;
    const float mu = mean[row], rs = rstd[row], inv = 1.f / (float)dim;
    float s1 = 0.f, s2 = 0.f;
    for (int c = threadIdx.x; c < dim; c += kLongThreads) {
        const float gw = to_float(dy[at + c]) * (weight ? weight[c] : 1.f);
        s1 += gw;
        s2 += gw * ((to_float(x[at + c]) - mu) * rs);
    }
    block_sums(s1, s2, red);
    s1 *= inv;
    s2 *= inv;
    for (int c = threadIdx.x; c < dim; c += kLongThreads) {
        const float gw = to_float(dy[at + c]) * (weight ? weight[c] : 1.f);
        dx[at + c] = from_float<E>(rs * (gw - s1 - (to_float(x[at + c]) - mu) * rs * s2));
    }
}

// Partial sums of a strip of rows, a column per thread.
template <typename E>
__global__ __launch_bounds__(kThreads) void k_norm_cols_long(const E *__restrict__ x, const E *__restrict__ dy,
                                                             const float *__restrict__ mean,
                                                             const float *__restrict__ rstd, float *__restrict__ parts,
                                                             int64_t rows, int dim, int strip)
{
    const int c = blockIdx.y * kThreads + threadIdx.x;
    if (c >= dim) return;
    const int64_t r0 = (int64_t)blockIdx.x * strip, r1 = r0 + strip < rows ? r0 + strip : rows;
    float dw = 0.f, db = 0.f;
    for (int64_t r = r0; r < r1; ++r) {
        const float gy = to_float(dy[r * dim + c]);
        dw += gy * ((to_float(x[r * dim + c]) - mean[r]) * rstd[r]);
        db += gy;
    }
    float *out = parts + (int64_t)blockIdx.x * 2 * dim;
    out[c] = dw;
    out[dim + c] = db;
}

__global__ __launch_bounds__(kThreads) void k_norm_zero(float *__restrict__ a, float *__restrict__ b, int dim)
{
    const int c = blockIdx.x * kThreads + threadIdx.x;
    if (c >= dim) return;
    if (a) a[c] = 0.f;
    if (b) b[c] = 0.f;
}

}  // namespace norm
}  // namespace ssd
