// mm_kernels.hpp -- the matrix product of e4m3 numbers with a scale for each block of 128 along
// the inner axis, for gfx950.
//
//   out[m][n] = bias[n] + sum_i a_scales[m][i] w_scales[n/128][i] sum_{k in block i} a[m][k] w[n][k]
//
// For bf16 outputs one v_mfma_f32_16x16x128 takes a whole block of 128, so its result (from a zero
// accumulator) is the block's sum, which one multiply-add per value scales into the fp32 total.  The matrix
// cores add e4m3 products to about 13 bits below the largest of them: 1.5e-5 of the result in norm with
// normal values, 5e-5 with a few large ones among them, whatever the instruction's length; far inside bf16's
// rounding (1.7e-3), but not fp32's.  fp32 outputs therefore turn both operands to bf16, exactly, and take
// four v_mfma_f32_16x16x32_bf16 a block (1e-8), at half the rate or less.
//
// The weights are the first operand and the rows of a the second: a lane then holds 4 neighbouring n of one
// m, so a lane has one scale for a 16 x 16 tile and stores its 4 values together.  What a lane group
// g = lane / 16 feeds is bytes 16 g .. and 64 + 16 g .. of a block, in both operands alike (the order inside a
// block does not change its sum).
#pragma once

#include <type_traits>

#include "ssd_device.hpp"

namespace ssd {
namespace mm {

typedef int intx8 __attribute__((ext_vector_type(8)));

constexpr int kBlock = 128;   // bytes of a row that share a scale

struct MmArgs {
    const uint8_t *a, *w;
    const float *as, *ws, *bias;
    void *out;
    float *part;        // sums of the shares of k [share][m][n]
    int m, n, k, kb;    // kb: blocks of 128 along k
    int per;            // blocks of a share
    int tm, tn;         // tiles along m and n
};

// What a lane feeds of 16 rows of a block: 32 numbers as they are, or as bf16.
template <bool BF> struct Operand {
    typename std::conditional<BF, bf16x8, intx8>::type v[BF ? 4 : 1];
};
__device__ __forceinline__ bf16x8 bf16_of(uint32_t a, uint32_t b)
{
    const bf16x2 p = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.f, false), q = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.f, true),
                 r = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.f, false), t = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.f, true);
    return bf16x8{p[0], p[1], q[0], q[1], r[0], r[1], t[0], t[1]};
}
template <bool BF> __device__ __forceinline__ Operand<BF> operand(const uint4 &lo, const uint4 &hi)
{
    Operand<BF> o;
    if constexpr (BF) {
        o.v[0] = bf16_of(lo.x, lo.y);
        o.v[1] = bf16_of(lo.z, lo.w);
        o.v[2] = bf16_of(hi.x, hi.y);
        o.v[3] = bf16_of(hi.z, hi.w);
    } else o.v[0] = intx8{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
    return o;
}
template <bool BF> __device__ __forceinline__ floatx4 block_product(const Operand<BF> &a, const Operand<BF> &b)
{
    floatx4 t = {0.f, 0.f, 0.f, 0.f};
    if constexpr (BF) {
#pragma unroll
        for (int i = 0; i < 4; ++i) mma(t, a.v[i], b.v[i]);
    } else t = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a.v[0], b.v[0], t, 0, 0, 0, 0, 0, 0);   // scales of zero: the form without
    return t;
}

// Rows of 128 bytes in LDS: 16-byte chunk c of row r at position c ^ (r & 7), so that 8 lanes that read
// one chunk of 8 rows touch every bank once.
template <bool BF> __device__ __forceinline__ Operand<BF> lds_operand(const uint8_t *tile, int row, int g)
{
    const uint8_t *p = tile + row * kBlock;
    const uint4 lo = *reinterpret_cast<const uint4 *>(p + 16 * (g ^ (row & 7)));
    const uint4 hi = *reinterpret_cast<const uint4 *>(p + 16 * ((g + 4) ^ (row & 7)));
    return operand<BF>(lo, hi);
}
typedef __attribute__((address_space(3))) void *lds_t;
// 8 rows of block `kb` from row `row` (of the buffer's tile) on into LDS: 16 bytes a lane; rows past the
// buffer and bytes past k are zero.
__device__ __forceinline__ void rows_to_lds(__amdgpu_buffer_rsrc_t r, uint8_t *dst, int row, int kb, int k)
{
    const int lane = threadIdx.x & 63, rr = lane >> 3, at = kb * kBlock + 16 * ((lane & 7) ^ rr);
    const uint32_t off = at < k ? (uint32_t)(row + rr) * (uint32_t)k + (uint32_t)at : kOffNone;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_t)dst, 16, off, 0, 0, 0);
}

// 4 neighbouring n of row m, to the output's type (or as fp32 sums).
template <typename O> __device__ __forceinline__ void store4(O *row, int n, int N, const floatx4 &v, bool vec)
{
    if (vec && n + 3 < N) {
        const float f[4] = {v[0], v[1], v[2], v[3]};
        store4_f32(row + n, f);
    } else
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (n + i < N) row[n + i] = from_float<O>(v[i]);
}

// Tile of BM rows of a and BN rows of w, WM x WN waves.  Two stages of LDS: the next block of both
// operands is on its way while this one is multiplied.
template <typename O, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN) void k_mm_tile(MmArgs p)
{
    constexpr bool BF = std::is_same<O, float>::value;
    constexpr int NW = WM * WN, TM = BM / WM, TN = BN / WN, MI = TM / 16, NI = TN / 16;
    static_assert(128 % TN == 0 && BN % 128 == 0, "a wave's columns share a scale");
    __shared__ __attribute__((aligned(128))) uint8_t sa[2][BM * kBlock], sw[2][BN * kBlock];
    __shared__ float sc[2][BM];
    const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int lr = lane & 15, g = lane >> 4;
    // groups of 8 tiles along m share their weights' tiles while they are in an XCD's L2
    constexpr int GM = 8;
    const int id = xcd_remap(blockIdx.x, gridDim.x);
    const int first = id / (GM * p.tn) * GM, gm = p.tm - first < GM ? p.tm - first : GM, in = id - first * p.tn;
    const int m0 = (first + in % gm) * BM, n0 = in / gm * BN;
    const int rows = p.m - m0 < BM ? p.m - m0 : BM, cols = p.n - n0 < BN ? p.n - n0 : BN;
    const __amdgpu_buffer_rsrc_t ra = make_rsrc(p.a + (int64_t)m0 * p.k, (int64_t)rows * p.k);
    const __amdgpu_buffer_rsrc_t rw = make_rsrc(p.w + (int64_t)n0 * p.k, (int64_t)cols * p.k);
    const __amdgpu_buffer_rsrc_t rs = make_rsrc(p.as + (int64_t)m0 * p.kb, (int64_t)rows * p.kb * 4);
    auto stage = [&](int s, int kb) {
        for (int i = wv; i < BM / 8; i += NW) rows_to_lds(ra, sa[s] + i * 8 * kBlock, i * 8, kb, p.k);
        for (int i = wv; i < BN / 8; i += NW) rows_to_lds(rw, sw[s] + i * 8 * kBlock, i * 8, kb, p.k);
        if (tid < BM)
            sc[s][tid] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rs, (uint32_t)(tid * p.kb + kb) * 4u, 0, 0));
    };
    floatx4 acc[MI][NI];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NI; ++j) acc[i][j] = floatx4{0.f, 0.f, 0.f, 0.f};
    const int wm = wv % WM * TM, wn = wv / WM * TN;
    const float *wsp = p.ws + (int64_t)((n0 + wn < p.n ? n0 + wn : 0) / kBlock) * p.kb;
    stage(0, 0);
    for (int kb = 0; kb < p.kb; ++kb) {
        __syncthreads();   // this block is there, and the other stage is read out
        const int s = kb & 1;
        if (kb + 1 < p.kb) stage(s ^ 1, kb + 1);
        const float ws = wsp[kb];
        Operand<BF> fw[NI];
#pragma unroll
        for (int j = 0; j < NI; ++j) fw[j] = lds_operand<BF>(sw[s], wn + 16 * j + lr, g);
#pragma unroll
        for (int i = 0; i < MI; ++i) {
            const Operand<BF> fa = lds_operand<BF>(sa[s], wm + 16 * i + lr, g);
            const float f = sc[s][wm + 16 * i + lr] * ws;
#pragma unroll
            for (int j = 0; j < NI; ++j) {
                const floatx4 t = block_product<BF>(fw[j], fa);
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[i][j][e] += f * t[e];
            }
        }
    }
    const bool vec = (p.n & 3) == 0;
#pragma unroll
    for (int i = 0; i < MI; ++i) {
        const int m = m0 + wm + 16 * i + lr;
        if (m >= p.m) continue;
        O *row = static_cast<O *>(p.out) + (int64_t)m * p.n;
#pragma unroll
        for (int j = 0; j < NI; ++j) {
            const int n = n0 + wn + 16 * j + 4 * g;
            floatx4 v = acc[i][j];
            if (p.bias)
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] += p.bias[n + e < p.n ? n + e : 0];
            store4(row, n, p.n, v, vec);
        }
    }
}

// Few rows: bound by the weights' bytes.  A workgroup has 16 MI rows of a and 128 rows of w, 16 a wave,
// and a share of k.  A wave reads its weights straight into registers, U blocks ahead; the rows of a come
// through LDS, U blocks at a time.
template <typename O, int MI, bool SHARED>
__global__ __launch_bounds__(512) void k_mm_few(MmArgs p)
{
    constexpr bool BF = std::is_same<O, float>::value;
    constexpr int BM = 16 * MI, U = 4;
    __shared__ __attribute__((aligned(128))) uint8_t sa[2][U][BM * kBlock];
    const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int lr = lane & 15, g = lane >> 4;
    const int id = xcd_remap(blockIdx.x, gridDim.x);
    // tiles along m next to each other: they share weights
    const int tmi = id % p.tm, rest = id / p.tm, tni = rest % p.tn, share = rest / p.tn;
    const int m0 = tmi * BM, n0 = tni * 128 + wv * 16;
    const int b0 = share * p.per, b1 = b0 + p.per < p.kb ? b0 + p.per : p.kb;
    const int rows = p.m - m0 < BM ? p.m - m0 : BM, cols = n0 < p.n ? (p.n - n0 < 16 ? p.n - n0 : 16) : 0;
    const __amdgpu_buffer_rsrc_t ra = make_rsrc(p.a + (int64_t)m0 * p.k, (int64_t)rows * p.k);
    const __amdgpu_buffer_rsrc_t rw = make_rsrc(p.w + (int64_t)(cols ? n0 : 0) * p.k, (int64_t)cols * p.k);
    const __amdgpu_buffer_rsrc_t rs = make_rsrc(p.as + (int64_t)m0 * p.kb, (int64_t)rows * p.kb * 4);
    const float *wsp = p.ws + (int64_t)tni * p.kb;
    uint4 lo[U], hi[U];
    float fs[U][MI];
    auto stage = [&](int s, int kb) {
        for (int i = wv; i < U * (BM / 8); i += 8) {
            const int u = i / (BM / 8), r = i % (BM / 8);
            if (kb + u < b1) rows_to_lds(ra, sa[s][u] + r * 8 * kBlock, r * 8, kb + u, p.k);
        }
    };
    auto fetch = [&](int kb) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int at = (kb + u) * kBlock + 16 * g;
            const uint32_t off = (uint32_t)lr * (uint32_t)p.k + (uint32_t)at;
            const bool in = kb + u < b1;
            lo[u] = bload16(rw, in && at < p.k ? off : kOffNone);
            hi[u] = bload16(rw, in && at + 64 < p.k ? off + 64 : kOffNone);
#pragma unroll
            for (int i = 0; i < MI; ++i)
                fs[u][i] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(
                    rs, in ? (uint32_t)((16 * i + lr) * p.kb + kb + u) * 4u : kOffNone, 0, 0));
        }
    };
    floatx4 acc[MI];
#pragma unroll
    for (int i = 0; i < MI; ++i) acc[i] = floatx4{0.f, 0.f, 0.f, 0.f};
    stage(0, b0);
    fetch(b0);
    int s = 0;
    for (int kb = b0; kb < b1; kb += U, s ^= 1) {
        Operand<BF> fw[U];
        float f[U][MI];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            fw[u] = operand<BF>(lo[u], hi[u]);
            const float ws = kb + u < b1 ? wsp[kb + u] : 0.f;
#pragma unroll
            for (int i = 0; i < MI; ++i) f[u][i] = fs[u][i] * ws;
        }
        __syncthreads();
        if (kb + U < b1) {
            stage(s ^ 1, kb + U);
            fetch(kb + U);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (kb + u >= b1) break;
#pragma unroll
            for (int i = 0; i < MI; ++i) {
                const floatx4 t = block_product<BF>(fw[u], lds_operand<BF>(sa[s][u], 16 * i + lr, g));
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[i][e] += f[u][i] * t[e];
            }
        }
    }
    const bool vec = (p.n & 3) == 0;
    const int n = n0 + 4 * g;
#pragma unroll
    for (int i = 0; i < MI; ++i) {
        const int m = m0 + 16 * i + lr;
        if (m >= p.m || n >= p.n) continue;
        floatx4 v = acc[i];
        if constexpr (SHARED) store4(p.part + ((int64_t)share * p.m + m) * p.n, n, p.n, v, vec);
        else {
            if (p.bias)
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] += p.bias[n + e < p.n ? n + e : 0];
            store4(static_cast<O *>(p.out) + (int64_t)m * p.n, n, p.n, v, vec);
        }
    }
}

// The shares of k, added in their order, V values a thread.
template <typename O, int V>
__global__ __launch_bounds__(kThreads) void k_mm_join(const float *__restrict__ part, const float *__restrict__ bias, O *__restrict__ out,
                                                      int64_t mn, int n, int shares)
{
    const int64_t i = ((int64_t)blockIdx.x * kThreads + threadIdx.x) * V;
    if (i >= mn) return;
    float s[V];
    const int c = (int)(i % n);
#pragma unroll
    for (int e = 0; e < V; ++e) s[e] = bias ? bias[c + e] : 0.f;
    for (int r = 0; r < shares; ++r) {
        float v[V];
        if constexpr (V == 4) load4_f32(part + r * mn + i, v);
        else v[0] = part[r * mn + i];
#pragma unroll
        for (int e = 0; e < V; ++e) s[e] += v[e];
    }
    if constexpr (V == 4) store4_f32(out + i, s);
    else out[i] = from_float<O>(s[0]);
}

}  // namespace mm
}  // namespace ssd
