// mm_kernels.hpp -- the matrix product of e4m3 numbers with a scale for each block of 128 along
// the inner axis, for gfx950.
//
//   out[m][n] = bias[n] + sum_i a_scales[m][i] w_scales[n/128][i] sum_{k in block i} a[m][k] w[n][k]
//
// Both operands become bf16 in registers, which is exact, and four v_mfma_f32_16x16x32_bf16 form a block's sum in
// fp32; one multiply-add per value scales it into the total.  The matrix cores' own e4m3 products run at twice the rate
// (410 against 780 us for 16384 x 10240 of k = 2560), but add to about 13 bits below the largest product: where a channel
// stands out of a block, what is beside it is lost, 1.4e-4 of the terms' sizes where two such channels cancel.
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

// What a lane feeds of 16 rows of a block: 32 numbers.
struct Operand {
    bf16x8 v[4];
};
__device__ __forceinline__ bf16x8 bf16_of(uint32_t a, uint32_t b)
{
    const bf16x2 p = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.f, false), q = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.f, true),
                 r = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.f, false), t = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.f, true);
    return bf16x8{p[0], p[1], q[0], q[1], r[0], r[1], t[0], t[1]};
}
__device__ __forceinline__ Operand operand(const uint4 &lo, const uint4 &hi)
{
    return Operand{{bf16_of(lo.x, lo.y), bf16_of(lo.z, lo.w), bf16_of(hi.x, hi.y), bf16_of(hi.z, hi.w)}};
}
__device__ __forceinline__ floatx4 block_product(const Operand &a, const Operand &b)
{
    floatx4 t = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 4; ++i) mma(t, a.v[i], b.v[i]);
    return t;
}

// Rows of 128 bytes in LDS: 16-byte chunk c of row r at position c ^ (r & 7), so that 8 lanes that read
// one chunk of 8 rows touch every bank once.  A lane reads row lane % 16 of 16-row groups: its two places there.
struct Places {
    int lo, hi;
};
__device__ __forceinline__ Places places_of(int lane)
{
    const int r = lane & 15, g = lane >> 4;
    return Places{r * kBlock + 16 * (g ^ (r & 7)), r * kBlock + 16 * ((g + 4) ^ (r & 7))};
}
__device__ __forceinline__ Operand lds_operand(const uint8_t *rows16, const Places &p)
{
    return operand(*reinterpret_cast<const uint4 *>(rows16 + p.lo), *reinterpret_cast<const uint4 *>(rows16 + p.hi));
}
typedef __attribute__((address_space(3))) void *lds_t;
// The byte of a row's block that this lane brings to LDS (8 lanes a row, 8 rows an access).
__device__ __forceinline__ int byte_of(int lane) { return 16 * ((lane & 7) ^ (lane >> 3)); }
// 8 rows of a block into LDS: 16 bytes a lane from `off` (row, byte_of) plus the block's first byte; rows past the
// buffer and bytes past k are zero.
__device__ __forceinline__ void rows_to_lds(__amdgpu_buffer_rsrc_t r, uint8_t *dst, uint32_t off, int kb, int byte, int k)
{
    const int at = kb * kBlock;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_t)dst, 16, at + byte < k ? off + (uint32_t)at : kOffNone, 0, 0, 0);
}

// Every wave's loads have landed and every wave's reads are over.
__device__ __forceinline__ void stage_done()
{
    __builtin_amdgcn_s_waitcnt(0x0070);   // vmcnt(0) lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");   // nothing is read ahead of the barrier
}
// Vectors in memory that are aligned to an element only: rows of n values start anywhere.
template <typename T, int N> using any_t = T __attribute__((ext_vector_type(N), aligned(sizeof(T))));
// 4 neighbouring n of row m, to the output's type (or as fp32 sums).
template <typename O> __device__ __forceinline__ void store4(O *row, int n, int N, const floatx4 &v)
{
    if (n + 3 < N) *reinterpret_cast<any_t<O, 4> *>(row + n) = __builtin_convertvector(v, any_t<O, 4>);   // to nearest even
    else
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (n + i < N) row[n + i] = from_float<O>(v[i]);
}

// A wave's values as bf16, 8 neighbouring n a lane: of two 16 x 16 tiles next to each other along n the lanes of
// group g hold n 4 g .. of each; the halves that are in the wrong lanes swap.  A store then writes 64 bytes of each of 16
// rows (32 with 4 values a lane: 16384 x 10240 of k = 2560 in 813 us, 780 so), past the caches, which would write
// them all back at once when every workgroup's tile ends (791 us).
// Rows that are not whole vectors take ordinary stores, aligned to an element, and single elements at their ends.
constexpr int kCpolPast = 18;   // streaming, written through
template <bool WHOLE, int MI, int NI>
__device__ __forceinline__ void store_wide(const float (&acc)[MI][NI][4], bf16 *tile, int row, int col, int g, int rows, int cols, int stride)
{
    const __amdgpu_buffer_rsrc_t r = make_rsrc(tile, WHOLE ? ((int64_t)(rows - 1) * stride + cols) * 2 : 0);
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NI; j += 2) {
            const auto &a = acc[i][j], &b = acc[i][j + 1];
            const auto x = __builtin_amdgcn_permlane32_swap(pack_bf16x2(a[0], a[1]), pack_bf16x2(b[0], b[1]), false, false);
            const auto y = __builtin_amdgcn_permlane32_swap(pack_bf16x2(a[2], a[3]), pack_bf16x2(b[2], b[3]), false, false);
            const auto u = __builtin_amdgcn_permlane16_swap(x[0], x[1], false, false);
            const auto v = __builtin_amdgcn_permlane16_swap(y[0], y[1], false, false);
            typedef unsigned int u32x4 __attribute__((__vector_size__(16)));
            const u32x4 o = {u[0], v[0], u[1], v[1]};
            const int c = col + 16 * j + 8 * g;   // groups 0 and 1 have the first tile's, 2 and 3 the second's
            if constexpr (WHOLE)
                __builtin_amdgcn_raw_buffer_store_b128(o, r, c < cols ? ((uint32_t)(row + 16 * i) * (uint32_t)stride + (uint32_t)c) * 2u : kOffNone, 0,
                                                       kCpolPast);
            else if (row + 16 * i < rows) {
                bf16 *to = tile + (int64_t)(row + 16 * i) * stride + c;
                const any_t<bf16, 8> e = __builtin_bit_cast(bf16x8, o);
                if (c + 8 <= cols) *reinterpret_cast<any_t<bf16, 8> *>(to) = e;
                else
#pragma unroll
                    for (int q = 0; q < 8; ++q)
                        if (c + q < cols) to[q] = e[q];
            }
        }
}

// Tile of BM rows of a and BN rows of w, WM x WN waves.  16384 x 10240 of k = 2560 to bf16: 780 us, 1.10 PFLOP/s, where a large library
// product of bf16 numbers reaches 1.13 to 1.27: the matrix cores bound it.  (Tiles of 256 x 128 and 8 waves took 754
// there, 388 for 2560 columns of k = 5120 either way, and for 4096 rows of those 142 instead of 100.)
// Two stages of LDS, filled straight from memory:
// the next block of both operands is on its way while this one is multiplied.  The stages are arrays of their
// own, so that a read of one does not wait for the loads into the other.  A workgroup stays for tile after
// tile: the next one's first block comes while this one's last is multiplied and its values are stored.  WHOLE: rows of
// whole 16-byte vectors of bf16 (11844 x 5154 of k = 112, not so: 138 us with single elements, 43 with vectors).
template <typename O, bool WHOLE>
__global__ __launch_bounds__(kThreads) void k_mm_tile(MmArgs p)
{
    constexpr int BM = 128, BN = 128, WM = 2, WN = 2, NW = WM * WN, TM = BM / WM, TN = BN / WN, MI = TM / 16, NI = TN / 16;
    static_assert(128 % TN == 0 && BN % 128 == 0, "a wave's columns share a scale");
    static_assert(BM < 64 * NW && BM % 64 == 0, "a wave loads the scales of 64 rows, the last one those of w");
    __shared__ __attribute__((aligned(128))) uint8_t sa0[BM * kBlock], sw0[BN * kBlock], sa1[BM * kBlock], sw1[BN * kBlock];
    __shared__ float sc0[BM + 64], sc1[BM + 64];   // scales of the rows of a, then of the blocks of w
    const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int lr = lane & 15, g = lane >> 4, byte = byte_of(lane);
    const Places at = places_of(lane);
    const int wm = wv % WM * TM, wn = wv / WM * TN;
    const uint32_t off = (uint32_t)(wv * 8 + (lane >> 3)) * (uint32_t)p.k + (uint32_t)byte, step = (uint32_t)(NW * 8) * (uint32_t)p.k;
    const int tiles = p.tm * p.tn;
    struct Tile {
        int m0, n0;
        __amdgpu_buffer_rsrc_t a, w, as, ws;
    };
    auto tile_at = [&](int v) {
        // groups of 8 tiles along m share their weights' tiles while they are in an XCD's L2
        constexpr int GM = 8;
        const int id = xcd_remap(v, tiles);
        const int first = id / (GM * p.tn) * GM, gm = p.tm - first < GM ? p.tm - first : GM, in = id - first * p.tn;
        Tile t;
        t.m0 = (first + in % gm) * BM;
        t.n0 = in / gm * BN;
        const int rows = p.m - t.m0 < BM ? p.m - t.m0 : BM, cols = p.n - t.n0 < BN ? p.n - t.n0 : BN;
        t.a = make_rsrc(p.a + (int64_t)t.m0 * p.k, (int64_t)rows * p.k);
        t.w = make_rsrc(p.w + (int64_t)t.n0 * p.k, (int64_t)cols * p.k);
        t.as = make_rsrc(p.as + (int64_t)t.m0 * p.kb, (int64_t)rows * p.kb * 4);
        t.ws = make_rsrc(p.ws + (int64_t)(t.n0 / kBlock) * p.kb, (int64_t)((cols + kBlock - 1) / kBlock) * p.kb * 4);
        return t;
    };
    auto stage = [&](uint8_t *sa, uint8_t *sw, float *sc, const Tile &t, int kb) {
#pragma unroll
        for (int i = 0; i < BM / 8 / NW; ++i) rows_to_lds(t.a, sa + (i * NW + wv) * 8 * kBlock, off + i * step, kb, byte, p.k);
#pragma unroll
        for (int i = 0; i < BN / 8 / NW; ++i) rows_to_lds(t.w, sw + (i * NW + wv) * 8 * kBlock, off + i * step, kb, byte, p.k);
        if (wv < BM / 64)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(t.as, (lds_t)(sc + 64 * wv), 4, kb < p.kb ? (uint32_t)(tid * p.kb + kb) * 4u : kOffNone, 0,
                                                     0, 0);
        else if (wv == NW - 1)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(t.ws, (lds_t)(sc + BM), 4,
                                                     kb < p.kb && lane < BN / kBlock ? (uint32_t)(lane * p.kb + kb) * 4u : kOffNone, 0, 0, 0);
    };
    float acc[MI][NI][4];   // vectors of four would be copied from block to block
    // a product is scaled and added three products later, when it is there
    constexpr int AHEAD = 3;
    auto multiply = [&](const uint8_t *sa, const uint8_t *sw, const float *sc) {
        sa += wm * kBlock;
        sw += wn * kBlock;
        Operand fw[NI];
#pragma unroll
        for (int j = 0; j < NI; ++j) fw[j] = lds_operand(sw + 16 * j * kBlock, at);
        Operand fa[2];
        fa[0] = lds_operand(sa, at);
        floatx4 t[AHEAD + 1];
        float f[MI];
        const float ws = sc[BM + wn / kBlock];
#pragma unroll
        for (int i = 0; i < MI; ++i) f[i] = sc[wm + lr + 16 * i] * ws;
#pragma unroll
        for (int n = 0; n < MI * NI + AHEAD; ++n) {
            const int i = n / NI, j = n % NI;
            if (n < MI * NI) {
                if (j == 0 && i + 1 < MI) fa[(i + 1) & 1] = lds_operand(sa + 16 * (i + 1) * kBlock, at);
                t[n % (AHEAD + 1)] = block_product(fw[j], fa[i & 1]);
            }
            if (n >= AHEAD) {
                const int pi = (n - AHEAD) / NI, pj = (n - AHEAD) % NI;
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[pi][pj][e] += f[pi] * t[(n - AHEAD) % (AHEAD + 1)][e];
                // here, not after the loop's next barrier, where the compiler would rather have all of them
                asm volatile("" : "+v"(acc[pi][pj][0]), "+v"(acc[pi][pj][1]), "+v"(acc[pi][pj][2]), "+v"(acc[pi][pj][3]));
            }
            __builtin_amdgcn_sched_barrier(0);   // further ahead the scheduler runs out of registers
        }
    };
    Tile t = tile_at(blockIdx.x);
    stage(sa0, sw0, sc0, t, 0);
    for (int v = blockIdx.x; v < tiles; v += gridDim.x) {
        const Tile next = tile_at(v + (int)gridDim.x < tiles ? v + (int)gridDim.x : v);
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int j = 0; j < NI; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[i][j][e] = 0.f;
        // in pairs; past an odd number of blocks there is a block of zeros (a way out between the two would keep
        // the sums in registers twice)
        for (int kb = 0; kb < p.kb; kb += 2) {
            stage_done();   // this block is there, and the other stage is read out
            stage(sa1, sw1, sc1, t, kb + 1);
            multiply(sa0, sw0, sc0);
            stage_done();
            if (kb + 2 < p.kb) stage(sa0, sw0, sc0, t, kb + 2);
            else if (v + (int)gridDim.x < tiles) stage(sa0, sw0, sc0, next, 0);
            multiply(sa1, sw1, sc1);
        }
        if (p.bias)
#pragma unroll
            for (int j = 0; j < NI; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int n = t.n0 + wn + 16 * j + 4 * g + e;
                    const float b = p.bias[n < p.n ? n : 0];
#pragma unroll
                    for (int i = 0; i < MI; ++i) acc[i][j][e] += b;
                }
        if constexpr (std::is_same<O, bf16>::value) {
            O *tile = static_cast<O *>(p.out) + (int64_t)t.m0 * p.n + t.n0;
            const int rows = p.m - t.m0 < BM ? p.m - t.m0 : BM, cols = p.n - t.n0 < BN ? p.n - t.n0 : BN;
            store_wide<WHOLE>(acc, tile, wm + lr, wn, g, rows, cols, p.n);
        } else {
#pragma unroll
            for (int i = 0; i < MI; ++i) {
                const int m = t.m0 + wm + 16 * i + lr;
                if (m >= p.m) continue;
                O *row = static_cast<O *>(p.out) + (int64_t)m * p.n;
#pragma unroll
                for (int j = 0; j < NI; ++j)
                    store4(row, t.n0 + wn + 16 * j + 4 * g, p.n, floatx4{acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]});
            }
        }
        t = next;
    }
}

// This wave's loads but the last N have landed and its reads are over; the same for every wave behind the barrier.
template <int N> __device__ __forceinline__ void loads_done()
{
    static_assert(N < 64, "");
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt((N & 15) | (N >> 4) << 14 | 0x70);   // vmcnt(N) lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}
template <int N, typename F> __device__ __forceinline__ void unrolled(F &&f)
{
    if constexpr (N > 0) {
        unrolled<N - 1>(f);
        f(std::integral_constant<int, N - 1>{});
    }
}

// Few rows: bound by the weights' bytes.  A workgroup has 16 MI rows of a and 64 rows of w, in 4 waves of 16 twice: each
// half takes half of the workgroup's blocks, and the halves are added in LDS.  A wave reads its weights straight
// into registers, up to 8 blocks ahead, since they come from memory (two halves of every line, so not past the caches).  Where
// its loop of 8 blocks ends the compiler moves what is on its way to other registers, which waits for it: a wave with
// more than 8 blocks sees the memory's latency once more every 8.  The rows of a, which the 4 waves share, come through
// LDS a phase of U blocks ahead.  SHARED: the blocks are shared out over workgroups too, and k_mm_join adds their sums.
// 64 rows of 10240 x 2560: 18.7 us, 16 rows 11.0; the weights' bytes would take 5.2.
template <typename O, int MI, bool SHARED>
__global__ __launch_bounds__(512) void k_mm_few(MmArgs p)
{
    constexpr int BM = 16 * MI, U = MI == 4 ? 2 : 4, R = 8 / U;
    __shared__ __attribute__((aligned(128))) uint8_t sa0[2 * U * BM * kBlock], sa1[2 * U * BM * kBlock];
    __shared__ float ss0[2 * U * 64], ss1[2 * U * 64];   // scales of the rows of a
    const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int lr = lane & 15, g = lane >> 4, byte = byte_of(lane), half = wv >> 2;
    const Places at = places_of(lane);
    const int id = xcd_remap(blockIdx.x, gridDim.x);
    // tiles along m next to each other: they share weights
    const int tmi = id % p.tm, rest = id / p.tm, tni = rest % p.tn, share = rest / p.tn;
    const int m0 = tmi * BM, n0 = tni * 64 + (wv & 3) * 16;
    const int first = share * p.per, last = first + p.per < p.kb ? first + p.per : p.kb, each = (last - first + 1) / 2;
    const int b0 = first + half * each, b1 = half ? last : first + each;   // the half's blocks
    const int rows = p.m - m0 < BM ? p.m - m0 : BM, cols = n0 < p.n ? (p.n - n0 < 16 ? p.n - n0 : 16) : 0;
    const __amdgpu_buffer_rsrc_t ra = make_rsrc(p.a + (int64_t)m0 * p.k, (int64_t)rows * p.k);
    const __amdgpu_buffer_rsrc_t rw = make_rsrc(p.w + (int64_t)(cols ? n0 : 0) * p.k, (int64_t)cols * p.k);
    const __amdgpu_buffer_rsrc_t rs = make_rsrc(p.as + (int64_t)m0 * p.kb, (int64_t)rows * p.kb * 4);
    const __amdgpu_buffer_rsrc_t rws = make_rsrc(p.ws + (int64_t)(tni * 64 / kBlock) * p.kb, (int64_t)p.kb * 4);
    // both halves' rows of a, 8 rows of a block an access; nothing is read past the last block, but the accesses
    // are there, so that a wait can count them
    constexpr int ND = 2 * U * BM / 8 / 8, NF = U * 3;
    static_assert(ND * 8 == 2 * U * BM / 8, "");
    auto stage = [&](uint8_t *sa, float *ss, int ph) {
#pragma unroll
        for (int i = 0; i < ND; ++i) {
            const int x = i * 8 + wv, r = x % (BM / 8), u = x / (BM / 8) % U, h = x / (BM / 8) / U;
            const int kb = first + h * each + ph * U + u;
            rows_to_lds(ra, sa + x * 8 * kBlock, (uint32_t)(r * 8 + (lane >> 3)) * (uint32_t)p.k + (uint32_t)byte,
                        kb < (h ? last : first + each) ? kb : p.kb, byte, p.k);
        }
        // a wave the scales of one block (some the same ones as another wave)
        const int u = wv % U, h = wv / U & 1, kb = first + h * each + ph * U + u;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_t)(ss + (h * U + u) * 64), 4,
                                                 kb < (h ? last : first + each) && lane < BM ? (uint32_t)(lane * p.kb + kb) * 4u : kOffNone, 0, 0, 0);
    };
    uint4 lo[R][U], hi[R][U];
    float fw[R][U];
    auto fetch = [&](auto set, int ph) {
        constexpr int S = decltype(set)::value;
        // in this place: loads_done counts these NF loads behind the rows of a
        asm volatile("" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int kb = b0 + ph * U + u, b = kb * kBlock + 16 * g;
            const uint32_t off = (uint32_t)lr * (uint32_t)p.k + (uint32_t)b;
            const bool in = kb < b1;
            lo[S][u] = bload16(rw, in && b < p.k ? off : kOffNone);
            hi[S][u] = bload16(rw, in && b + 64 < p.k ? off + 64 : kOffNone);
            fw[S][u] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rws, in ? (uint32_t)kb * 4u : kOffNone, 0, 0));
        }
        asm volatile("" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
    };
    float acc[MI][4];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][e] = 0.f;
    const int phases = (each + U - 1) / U;
    // a phase's rows of a were asked for before the last weights: those may still be on their way
    auto phase = [&](auto set, int ph) {
        constexpr int S = decltype(set)::value;
        const uint8_t *sa = S & 1 ? sa1 : sa0;
        const float *ss = (S & 1 ? ss1 : ss0) + half * U * 64 + lr;
        loads_done<NF>();
        stage(S & 1 ? sa0 : sa1, S & 1 ? ss0 : ss1, ph + 1);
        Operand w[U];
        float ws[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            w[u] = operand(lo[S][u], hi[S][u]);
            ws[u] = fw[S][u];
        }
        fetch(set, ph + R);
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < MI; ++i) {
                const floatx4 t = block_product(w[u], lds_operand(sa + ((half * U + u) * BM + 16 * i) * kBlock, at));
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[i][e] += ss[u * 64 + 16 * i] * ws[u] * t[e];
            }
    };
    unrolled<R - 1>([&](auto s) { fetch(s, decltype(s)::value); });
    stage(sa0, ss0, 0);
    fetch(std::integral_constant<int, R - 1>{}, R - 1);
    for (int ph = 0; ph < phases; ph += R) unrolled<R>([&](auto s) { phase(s, ph + decltype(s)::value); });   // past the last: nothing
    // the second half's sums through LDS
    stage_done();
    float *sums = reinterpret_cast<float *>(sa0) + (wv & 3) * MI * 256 + lane * 4;
    if (half)
#pragma unroll
        for (int i = 0; i < MI; ++i) store4_f32(sums + i * 256, acc[i]);
    stage_done();
    if (half) return;
    const int n = n0 + 4 * g;
#pragma unroll
    for (int i = 0; i < MI; ++i) {
        const int m = m0 + 16 * i + lr;
        if (m >= p.m || n >= p.n) continue;
        float o[4];
        load4_f32(sums + i * 256, o);
        floatx4 v = {acc[i][0] + o[0], acc[i][1] + o[1], acc[i][2] + o[2], acc[i][3] + o[3]};
        if constexpr (SHARED) store4(p.part + ((int64_t)share * p.m + m) * p.n, n, p.n, v);
        else {
            if (p.bias)
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] += p.bias[n + e < p.n ? n + e : 0];
            store4(static_cast<O *>(p.out) + (int64_t)m * p.n, n, p.n, v);
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
