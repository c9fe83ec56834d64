// gdr_kernels.hpp -- the gated delta rule for gfx950: chunked forward, backward
// and the one-token step.
//
// Per head (keys and queries are shared by the heads of a group), state S [N][P]:
//
//   u_t = v_t - e^{g_t} S_{t-1}^T k_t,   S_t = e^{g_t} S_{t-1} + beta_t k_t u_t^T,
//   y_t = scale S_t^T q_t
//
// Over a chunk of 64 tokens with entering state S, cs = the inclusive prefix sum
// of g, Gam[t][s] = e^{cs_t - cs_s} (s <= t) and A = the strictly lower part of
// Gam o K K^T, the 64 u's solve the unit lower triangular system
//
//   (I + A Db) U = R,   R = V - e^{cs} o (K S),   Db = diag(beta)
//
// and with N = (I + A Db)^-1 A (strictly lower, defined for beta = 0 too)
//
//   U = R - N (beta o R)
//   Y = scale (e^{cs} o (Q S) + (Gam o Q K^T) (beta o U))
//   S' = e^{cs_last} S + K^T (e^{cs_last - cs} o beta o U).
//
// The gradient runs the same chain backwards: with D = dL/dS' and
// W = scale (Gam o Q K^T)^T dY + e^{cs_last - cs} o (K D),
//
//   H = W - N^T (beta o W)       (= dL/d(beta u)),   dV = beta o H
//   dL/dS = e^{cs_last} D + scale Q^T (e^{cs} o dY) - K^T (e^{cs} o beta o H),
//
// which needs no state, so both chains run at the same time.  Everything that no
// state enters (N, Gam o Q K^T, the operand copies) is formed first, for all
// chunks in parallel; the gradients of q, k, g and beta are formed last, again
// for all chunks in parallel, from the stored S, U, D and H of every chunk.
//
// Register layout of a chain.  A wave owns 16 value columns of one head and all
// of their state: N / 16 accumulators S[nb], lane l holding rows n = 16 nb +
// 4 (l/16) + r of column p = l % 16.  A matrix-core product contracts over 32
// slots, 8 per lane group l/16, and does not care which row a slot stands for as
// long as both operands agree: with slot j of lane group g standing for row
// 4g + j (j < 4) or 16 + 4g + j - 4 (j >= 4) of a 32-row block, two accumulators
// ARE the second operand of the next product.  So the chain K S -> U -> S' runs
// from registers to registers, without a shuffle or a barrier between products;
// only the first operands (K, K^T, Q, N, Gam o Q K^T) come from memory, laid out
// once per chunk in that slot order ("slot order" below).
//
// Numerics.  Inputs are exact in their type.  For bf16 problems S, U, D and every
// sum are fp32, and whatever is not an input goes to the matrix cores as a sum of
// two bf16 numbers (16 bits of significand; a product drops that of the two small
// parts, about 2^-18 of its size).  So y and the gradients are off by the one
// rounding of their type (1.7e-3 in norm), states by 3e-6 to 4e-5.  With single bf16
// numbers for the operands of the outputs that do not feed the chain (S, beta U and
// Gam o Q K^T of y; S, U, D, H and the pair matrices of the gradients) random keys
// gave 2.9e-3; but with similar keys, beta near 1 and weak decay the terms are
// several times the sum, and keys at cosines of 0.9 gave 1.6e-2 for y and up to
// 6e-2 for dg.  The second numbers cost 592 -> 694 us for 16K tokens forward,
// 326 -> 367 for packed prompts and 1112 -> 1494 for the 2.7B-scale backward.
// fp32 problems use the fp32 matrix instructions throughout.
#pragma once

#include <type_traits>

#include "ssd_device.hpp"

namespace ssd {
namespace gdr {

constexpr int kC = 64;            // tokens per chunk
constexpr int kTri = 6;           // 16 x 32 operand blocks in a triangle of 64 x 64
// Per-token scalars of a (chunk, head), 64 floats each: e^{cs}, beta, scale e^{cs},
// beta e^{cs_last - cs}, e^{cs_last - cs}, -beta e^{cs}, and cs as a sum of two floats.
// Then, for the gradients, Gam between different blocks of 16 tokens as a product: with
// the reference r_b = cs before block b, for t in block b and s before it
//   Gam_ts = e^{cs_t - r_b} e^{r_b - cs_s}   (both at most 1)
// scale e^{cs_t - r_b}, beta_t e^{cs_t - r_b} (zero past the count), and beta_s e^{r_b -
// cs_s} for b = 1, 2, 3; and room for one vector (dg of the first pass).
constexpr int kVec = 16 * kC, kVecChain = 8 * kC;
constexpr int kSince = 0, kBeta = kC, kScaled = 2 * kC, kTillBeta = 3 * kC, kTill = 4 * kC, kErase = 5 * kC,
              kCsHi = 6 * kC, kCsLo = 7 * kC, kRowScale = 8 * kC, kRowBeta = 9 * kC, kColBeta = 10 * kC, kDgPass = 13 * kC;
constexpr double kLog2eD = 1.4426950408889634;
constexpr float kMinLogDecay = -64.f;   // e^-64 = 1.6e-28: smaller decays act as this one

// Planes of a split operand: a bf16 chain value is the sum of two bf16 numbers.
template <typename E> constexpr int kPlanes = sizeof(E) == 2 ? 2 : 1;

// ---------------------------------------------------------------------------
// chunks and chains
// ---------------------------------------------------------------------------
// A chain is one batch row, or one segment of a packed stream; its chunks are
// consecutive.  Packed streams: cmap[c] = {first token, token count} and
// chain[i] = {first chunk, chunks, first token, tokens} are built on the device from
// seq_idx (every segment starts a chunk of its own); otherwise both are null and
// arithmetic.
struct Chunks {
    const int2 *cmap;
    const int4 *chain;
    const int *order;   // packed: the chains by falling length, or null
    int T, nc;   // tokens and chunks per batch row (not packed)
};

__device__ __forceinline__ void chunk_at(const Chunks &m, int c, int64_t &t0, int &count)
{
    if (m.cmap) {
        const int2 v = m.cmap[c];
        t0 = __builtin_amdgcn_readfirstlane(v.x);
        count = __builtin_amdgcn_readfirstlane(v.y);
    } else {
        const int row = c / m.nc, i = c - row * m.nc;
        t0 = (int64_t)row * m.T + (int64_t)i * kC;
        count = m.T - i * kC < kC ? m.T - i * kC : kC;
    }
}

__device__ __forceinline__ void chain_at(const Chunks &m, int &i, int &c0, int &n, int64_t &t0, int &len)
{
    if (m.chain) {
        i = __builtin_amdgcn_readfirstlane(m.order[i]);   // the i-th longest
        const int4 v = m.chain[i];
        c0 = __builtin_amdgcn_readfirstlane(v.x);
        n = __builtin_amdgcn_readfirstlane(v.y);
        t0 = __builtin_amdgcn_readfirstlane(v.z);
        len = __builtin_amdgcn_readfirstlane(v.w);
    } else {
        c0 = i * m.nc;
        n = m.nc;
        t0 = (int64_t)i * m.T;
        len = m.T;
    }
}

// The chunk map of a packed stream, by one workgroup.  `range` [nseq] is scratch.
// Ids outside [0, nseq) are skipped and nothing is written past ncmax chunks, so
// an invalid stream gives wrong chunks but no access out of bounds.
constexpr int kMapThreads = 1024;
__global__ __launch_bounds__(kMapThreads) void k_gdr_map(const int32_t *__restrict__ seq_idx, int2 *__restrict__ range,
                                                         int4 *__restrict__ chain, int2 *__restrict__ cmap,
                                                         int *__restrict__ order, int T, int nseq, int ncmax)
{
    // chunks before a segment: 64 bits, since the overlapping ranges of an invalid stream may
    // add up to more than 2^31
    __shared__ int64_t wsum[kMapThreads / 64], base;
    __shared__ int chunks[kMapThreads];
    const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
    for (int i = tid; i < nseq; i += kMapThreads) range[i] = int2{0, 0};
    if (tid == 0) base = 0;
    __syncthreads();
    // range[id] = {start, end}: the words of one id are written by the threads of its
    // first and its last token.  Four tokens per thread, four such groups in flight.
    int *words = reinterpret_cast<int *>(range);
    const __amdgpu_buffer_rsrc_t rs = make_rsrc_n(seq_idx, T * 4);   // past the end: 0, not used
    constexpr int U = 4;
    for (int tb = 0; tb < T; tb += U * 4 * kMapThreads) {
        int id[U][6];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int t = tb + (u * kMapThreads + tid) * 4;
            const uint4 v = bload16(rs, 4u * t);
            id[u][0] = t > 0 ? __builtin_amdgcn_raw_buffer_load_b32(rs, 4u * t - 4, 0, 0) : -1;
            id[u][1] = v.x;
            id[u][2] = v.y;
            id[u][3] = v.z;
            id[u][4] = v.w;
            id[u][5] = __builtin_amdgcn_raw_buffer_load_b32(rs, 4u * t + 16, 0, 0);
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int t = tb + (u * kMapThreads + tid) * 4 + e, me = id[u][e + 1];
                if (t >= T || me < 0 || me >= nseq) continue;
                if (t == 0 || id[u][e] != me) words[2 * me] = t;
                if (t == T - 1 || id[u][e + 2] != me) words[2 * me + 1] = t + 1;
            }
    }
    __syncthreads();
    for (int i0 = 0; i0 < nseq; i0 += kMapThreads) {
        const int i = i0 + tid;
        const int2 r = i < nseq ? range[i] : int2{0, 0};
        const int len = r.y > r.x ? r.y - r.x : 0, n = (len + kC - 1) / kC;
        int64_t s = n;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int64_t o = __shfl_up((long long)s, d);
            if (lane >= d) s += o;
        }
        if (lane == 63) wsum[wv] = s;
        chunks[tid] = n;
        __syncthreads();
        int64_t before = base;
        for (int w = 0; w < wv; ++w) before += wsum[w];
        const int64_t c0 = before + s - n;
        if (i < nseq) {
            const int lo = c0 < ncmax ? (int)c0 : ncmax;
            chain[i] = int4{lo, c0 + n <= ncmax ? n : ncmax - lo, r.x, len};
            // long chains first (up to kMapThreads of them, each with its rank): a long one
            // started last would run alone at the end
            int rank = i;
            if (nseq <= kMapThreads) {
                rank = 0;
                for (int o = 0; o < nseq; ++o) rank += chunks[o] > n || (chunks[o] == n && o < i) ? 1 : 0;
            }
            order[rank] = i;
        }
        __syncthreads();
        if (tid == kMapThreads - 1) base = before + s;
        __syncthreads();
    }
    // one wave per segment writes its chunks
    for (int i = wv; i < nseq; i += kMapThreads / 64) {
        const int2 r = range[i];
        const int4 ch = chain[i];
        for (int j = lane; j < ch.y; j += 64) {
            const int left = r.y - r.x - j * kC;
            cmap[ch.x + j] = int2{r.x + j * kC, left < kC ? left : kC};
        }
    }
    for (int64_t c = base + tid; c < ncmax; c += kMapThreads) cmap[c] = int2{0, 0};
}

// ---------------------------------------------------------------------------
// operand blocks
// ---------------------------------------------------------------------------
// An operand block is 16 rows x 32 slots, 512 elements, lane l's 8 slots at
// element 8 l: one coalesced 16-byte (fp32: 32-byte) load per lane feeds one
// product.  The position in a 32-row block of slot j of lane group g:
__device__ __forceinline__ int slot_row(int g, int j) { return j < 4 ? 4 * g + j : 16 + 4 * g + j - 4; }
// Blocks of a lower triangle (rows t, slots s <= t) and of an upper one (rows s,
// slots t >= s) of a 64 x 64 matrix, 32-slot block kb of row block b.
__device__ __forceinline__ int lower_block(int b, int kb) { return b < 2 ? b : 2 + 2 * (b - 2) + kb; }
__device__ __forceinline__ int upper_block(int b, int kb) { return b < 2 ? 2 * b + kb : 4 + (b - 2); }

// Two accumulators (32 rows of 16 columns) as a second operand, hi + lo: both
// rounded to nearest even, the remainder x - hi exact in fp32.  Pairwise, so that one
// conversion serves the operand and the remainder.
__device__ __forceinline__ void split_pair(const floatx4 &a, const floatx4 &b, bf16x8 &hi, bf16x8 &lo)
{
    uint32_t h[4], o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float x = i < 2 ? a[2 * i] : b[2 * i - 4], y = i < 2 ? a[2 * i + 1] : b[2 * i - 3];
        h[i] = pack_bf16x2(x, y);
        o[i] = pack_bf16x2(x - __uint_as_float(h[i] << 16), y - __uint_as_float(h[i] & 0xffff0000u));
    }
    hi = __builtin_bit_cast(bf16x8, uint4{h[0], h[1], h[2], h[3]});
    lo = __builtin_bit_cast(bf16x8, uint4{o[0], o[1], o[2], o[3]});
}
__device__ __forceinline__ void split_pair(const floatx4 &a, const floatx4 &b, floatx8 &hi, floatx8 &)
{
    hi = __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}
template <typename E> __device__ __forceinline__ frag_t<E> round_pair(const floatx4 &a, const floatx4 &b)
{
    return from_f32<frag_t<E>>(__builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
}

// Four consecutive slots of a split matrix into its planes (`plane` elements apart).
__device__ __forceinline__ void store_split4(bf16 *p, int64_t plane, const floatx4 &v)
{
    const bf16x4 hi = __builtin_convertvector(v, bf16x4);
    *reinterpret_cast<bf16x4 *>(p) = hi;
    *reinterpret_cast<bf16x4 *>(p + plane) = __builtin_convertvector(v - __builtin_convertvector(hi, floatx4), bf16x4);
}
__device__ __forceinline__ void store_split4(float *p, int64_t, const floatx4 &v) { *reinterpret_cast<floatx4 *>(p) = v; }
__device__ __forceinline__ void store_round4(bf16 *p, const floatx4 &v)
{
    *reinterpret_cast<bf16x4 *>(p) = __builtin_convertvector(v, bf16x4);
}
__device__ __forceinline__ void store_round4(float *p, const floatx4 &v) { *reinterpret_cast<floatx4 *>(p) = v; }
// The same, past the caches where ONCE (non-temporal).
typedef unsigned int uint2v __attribute__((ext_vector_type(2)));
typedef unsigned int uint4v __attribute__((ext_vector_type(4)));
template <bool ONCE> __device__ __forceinline__ void store_round4(bf16 *p, const floatx4 &v)
{
    if (ONCE) __builtin_nontemporal_store(uint2v{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])}, reinterpret_cast<uint2v *>(p));
    else store_round4(p, v);
}
template <bool ONCE> __device__ __forceinline__ void store_round4(float *p, const floatx4 &v)
{
    if (ONCE) __builtin_nontemporal_store(v, reinterpret_cast<floatx4 *>(p));
    else store_round4(p, v);
}
template <bool ONCE, typename E> __device__ __forceinline__ void store_block(E *p, const frag_t<E> &f)
{
    if constexpr (!ONCE) store_frag(p, f);
    else if constexpr (sizeof(E) == 2) __builtin_nontemporal_store(__builtin_bit_cast(uint4v, f), reinterpret_cast<uint4v *>(p));
    else {
        store_round4<true>(p, __builtin_shufflevector(f, f, 0, 1, 2, 3));
        store_round4<true>(p + 4, __builtin_shufflevector(f, f, 4, 5, 6, 7));
    }
}

__device__ __forceinline__ floatx4 vec4(const float *p) { return *reinterpret_cast<const floatx4 *>(p); }
// Rows of the identity as a second operand: slot row (g, j) of a 32-row block against
// column 16 HALF + l.  An operand read as a first operand is its transpose; a product
// with these moves it to accumulators, exactly, with rows and columns exchanged.  That
// is how tiles enter and leave a chain with four consecutive elements per lane instead
// of one (4 accesses of 8 bytes instead of 16 of 2).
template <typename E> struct Select {
    frag_t<E> half[2];
    __device__ __forceinline__ void init(int lane)
    {
        const int g = lane >> 4, l = lane & 15;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int j = 0; j < 8; ++j) half[h][j] = from_float<E>(slot_row(g, j) == 16 * h + l ? 1.f : 0.f);
    }
};
// One element through a buffer resource: out of range reads are zero and writes are
// dropped, so ragged tiles need no branches (a branch around each of 16 loads makes
// each wait for its own).
template <typename E> __device__ __forceinline__ E bload_elem(__amdgpu_buffer_rsrc_t r, uint32_t off)
{
    if constexpr (sizeof(E) == 2)
        return __builtin_bit_cast(E, (unsigned short)__builtin_amdgcn_raw_buffer_load_b16(r, off, 0, 0));
    else return __builtin_bit_cast(E, (unsigned int)__builtin_amdgcn_raw_buffer_load_b32(r, off, 0, 0));
}
// The buffer of one head's rows of a chunk: `count` rows of P elements, `ld` apart
// (the host keeps 64 ld elements below 2^31 bytes).
template <typename E> __device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_rsrc(const E *base, int count, int64_t ld, int P)
{
    return make_rsrc(base, ((count - 1) * ld + P) * (int64_t)sizeof(E));
}
// K and Q of one chunk and group are kept as operand blocks in slot order: rows (64
// tokens, slots over N: 4 x NT/32 blocks) and transposed (NT rows n, slots over tokens:
// NT/16 x 2 blocks), in the order K, K^T, Q, Q^T (the last for the backward only).  Tokens
// past the chunk's count and columns past N are zero.

// Elements of one (chunk, head) of the prepared triangles, all in their planes: N and Gam
// o Q K^T; for the backward N, N^T and (Gam o Q K^T)^T.
template <typename E> __host__ __device__ constexpr int tri_elems(bool bwd)
{
    return 512 * kTri * kPlanes<E> * (bwd ? 3 : 2);
}

// Everything of one chunk and head that no state enters, by one wave: no barrier, and the
// four waves of a workgroup keep a CU's SIMDs busy with four of them.  A wave takes `hpw`
// heads of a group one after another, so that K K^T and Q K^T, which they share, are
// formed once.  Further waves write the operand blocks of K and Q.  cs is summed in 64 bits,
// since Gam takes differences of it.
//
// 8 x 2048 tokens of 80 heads, backward: 168 us, 0.9 GB (36 KB of triangles and 4 KB of
// scalars to write per chunk and head) at 5.4 TB/s.  (235 us while Gam o Q K^T was formed
// before the inverse, with more spilled registers, which came back from memory behind the
// stores; the bf16 backward that stores past the caches still spills 9.)  The forward writes
// two thirds and is bound by latency at two waves a SIMD (247 registers): packed prompts of 64
// heads 131 us, matrix and vector pipes about a quarter busy.  Workgroups of four waves that
// shared one head, with barriers between the blocks, took 177 us there while they wrote less.
//
// Blocks of 16 x 16 (i, j <= i), as accumulators with rows s of block j and columns t of
// block i: four consecutive slots of an operand block with rows t.  Between different
// blocks Gam is a product of two prepared factors (kVec), on the diagonal an exponential.
// The inverse goes by blocks too: the diagonal blocks' inverses Tm = (I + Db A)^-1 by
// substitution, the four of them side by side (lane group g: block g, a column per lane),
// then block row i of N from right to left,
//   N_ij = (A_ij - sum_{j < k <= i} N_ik (Db A)_kj) Tm_jj,
// transposed, so that an accumulator is the next product's second operand.  fp32 matrix
// instructions; A's blocks lie in LDS for the first operands.
constexpr int kPrepRow = 20, kPrepBlock = 16 * kPrepRow + 4;   // floats: 16-byte rows, blocks on other banks
constexpr int kPrepTables = 7 * kC;                            // row factor, 3 column factors, cs hi, lo, beta
constexpr int kPrepWave = 10 * kPrepBlock + 4 * 16 * 17 + kPrepTables;
__device__ __forceinline__ constexpr int tri_block(int i, int j) { return i * (i + 1) / 2 + j; }

// What this wave's lanes wrote to LDS is there for all of them (LDS serves a wave in order;
// the compiler has to keep that order too).
__device__ __forceinline__ void wave_sync()
{
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

template <typename E, int NT, bool BWD, bool ONCE>
__global__ __launch_bounds__(kThreads, 2) void k_gdr_prep(const E *__restrict__ kin, const E *__restrict__ qin,
                                                          const E *__restrict__ gate, const E *__restrict__ beta,
                                                          E *__restrict__ kq, float *__restrict__ vec,
                                                          E *__restrict__ tri, Chunks m, int H, int G, int N, float scale,
                                                          int hpw, int units)
{
    constexpr int NK = NT / 32, kMat = kC * NT, PL = 512 * kTri;
    __shared__ __attribute__((aligned(16))) float lds[4 * kPrepWave];
    const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), g = lane >> 4, l = lane & 15;
    float *A = lds + wv * kPrepWave, *Tm = A + 10 * kPrepBlock, *row = Tm + 4 * 16 * 17, *col = row + kC, *chi = row + 4 * kC,
          *clo = chi + kC, *bt = clo + kC;
    // units: (chunk, group, part of its heads), and after them (chunk, group, K or Q) to copy
    const int job = blockIdx.x * 4 + wv, hpg = H / G, parts = (hpg + hpw - 1) / hpw;
    const bool copies = job >= units;
    const int unit = copies ? job - units : job, per = copies ? 2 : parts;
    const int part = unit % per, grp = unit / per % G, c = unit / (per * G);
    if (copies && unit >= 2 * (units / parts)) return;
    int64_t t0;
    int count;
    chunk_at(m, c, t0, count);
    if (count <= 0) return;
    E *copy = kq + ((int64_t)c * G + grp) * (BWD ? 4 : 3) * kMat + 8 * lane;
    const __amdgpu_buffer_rsrc_t krs = rows_rsrc(kin + (t0 * G + grp) * N, count, (int64_t)G * N, N);
    const __amdgpu_buffer_rsrc_t qrs = rows_rsrc(qin + (t0 * G + grp) * N, count, (int64_t)G * N, N);
    Select<E> sel;
    sel.init(lane);
    floatx4 kk[10], qk[10];
#pragma unroll
    for (int b = 0; b < 10; ++b) kk[b] = qk[b] = floatx4{0, 0, 0, 0};
    // 32 columns at a time, straight from the rows: slots 0..3 are columns 4 g .., 4..7 are 16 + 4 g ..
    auto fetch = [&](__amdgpu_buffer_rsrc_t rs, int i, int kb) {
        const int n = 32 * kb + 4 * g;
        const uint32_t o = (uint32_t)((16 * i + l) * (G * N) + n) * (uint32_t)sizeof(E);
        const uint32_t o0 = n < N ? o : kOffNone, o1 = n + 16 < N ? o + 16 * (uint32_t)sizeof(E) : kOffNone;
        frag_t<E> f;
        if constexpr (sizeof(E) == 2) {
            const uint2 x = bload8s(rs, o0, 0), y = bload8s(rs, o1, 0);
            f = __builtin_bit_cast(bf16x8, uint4{x.x, x.y, y.x, y.y});
        } else {
            const floatx4 x = __builtin_bit_cast(floatx4, bload16(rs, o0)), y = __builtin_bit_cast(floatx4, bload16(rs, o1));
            f = __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7);
        }
        return f;
    };
    if (copies) {
        const __amdgpu_buffer_rsrc_t rs = part ? qrs : krs;
        E *o = copy + 2 * part * kMat;
        const bool both = BWD || part == 0;
#pragma unroll 2
        for (int kb = 0; kb < NK; ++kb) {
            frag_t<E> f[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) f[i] = fetch(rs, i, kb);
#pragma unroll
            for (int i = 0; i < 4; ++i) store_frag(o + (i * NK + kb) * 512, f[i]);
            if (!both) continue;
            // the columns' blocks of the transpose, through products with the identity
#pragma unroll
            for (int half = 0; half < 2; ++half)
#pragma unroll
                for (int tb = 0; tb < 2; ++tb) {
                    floatx4 a = floatx4{0, 0, 0, 0}, b = a;
                    mma(a, f[2 * tb], sel.half[half]);
                    mma(b, f[2 * tb + 1], sel.half[half]);
                    store_frag(o + kMat + (2 * (2 * kb + half) + tb) * 512, round_pair<E>(a, b));
                }
        }
        return;
    }
    // (for the pairs any order of the slots will do: eight consecutive columns, one load)
    auto fetch8 = [&](__amdgpu_buffer_rsrc_t rs, int i, int kb) {
        const int n = 32 * kb + 8 * g;
        frag_t<E> f;
        bload_frag(rs, n < N ? (uint32_t)((16 * i + l) * (G * N) + n) * (uint32_t)sizeof(E) : kOffNone, f);
        return f;
    };
    frag_t<E> kn[4], qn[4];   // the next 32 columns, on their way
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        kn[i] = fetch8(krs, i, 0);
        qn[i] = fetch8(qrs, i, 0);
    }
    for (int kb = 0; kb < NK; ++kb) {
        frag_t<E> k[4], q[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            k[i] = kn[i];
            q[i] = qn[i];
            kn[i] = fetch8(krs, i, kb + 1);   // (past the end: zero)
            qn[i] = fetch8(qrs, i, kb + 1);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j <= i; ++j) {
                mma(kk[tri_block(i, j)], k[j], k[i]);
                mma(qk[tri_block(i, j)], k[j], q[i]);
            }
    }
    const int h0 = grp * hpg + part * hpw, h1 = h0 + hpw < (grp + 1) * hpg ? h0 + hpw : (grp + 1) * hpg;
    // a head's gates are requested while the head before it is worked on, ahead of that
    // one's stores (a load waits for the stores issued before it)
    const int64_t gat = (t0 + (lane < count ? lane : count - 1)) * H;
    E g_next = gate[gat + h0], b_next = beta[gat + h0];
    {   // (the first ones have arrived: the loop's wait for the next ones then leaves the stores
        // behind them in flight)
        float gw = to_float(g_next), bw = to_float(b_next);
        asm volatile("" : "+v"(gw), "+v"(bw));
    }
    for (int h = h0; h < h1; ++h) {
        const int64_t u = (int64_t)c * H + h;
        {
            const float gv = lane < count ? to_float(g_next) : 0.f, bv = lane < count ? to_float(b_next) : 0.f;
            const int hn = h + 1 < h1 ? h + 1 : h;
            g_next = gate[gat + hn];
            b_next = beta[gat + hn];
            double s = gv < kMinLogDecay ? kMinLogDecay : gv;
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) {
                const double o = __shfl_up(s, d);
                if (lane >= d) s += o;
            }
            const double last = __shfl(s, 63);
            float *vo = vec + u * kVec;
            const float hi = (float)s, lo = (float)(s - (double)hi);
            const float since = exp2_((float)(s * kLog2eD)), till = exp2_((float)((last - s) * kLog2eD));
            const double ref[4] = {0.0, __shfl(s, 15), __shfl(s, 31), __shfl(s, 47)};
            const double r = g == 0 ? ref[0] : g == 1 ? ref[1] : g == 2 ? ref[2] : ref[3];
            const float rf = exp2_((float)((s - r) * kLog2eD));
            vo[kSince + lane] = since;
            vo[kBeta + lane] = bv;
            vo[kScaled + lane] = scale * since;
            vo[kTillBeta + lane] = till * bv;
            vo[kTill + lane] = till;
            vo[kErase + lane] = -bv * since;
            vo[kCsHi + lane] = hi;
            vo[kCsLo + lane] = lo;
            row[lane] = rf;
            chi[lane] = hi;
            clo[lane] = lo;
            bt[lane] = bv;
            if (BWD) {
                vo[kRowScale + lane] = lane < count ? scale * rf : 0.f;
                vo[kRowBeta + lane] = lane < count ? bv * rf : 0.f;
            }
#pragma unroll
            for (int k = 1; k < 4; ++k) {
                const float cf = lane < 16 * k ? exp2_((float)((ref[k] - s) * kLog2eD)) : 0.f;
                col[(k - 1) * kC + lane] = cf;
                if (BWD) vo[kColBeta + (k - 1) * kC + lane] = bv * cf;
            }
        }
        wave_sync();
        E *n_o = tri + u * tri_elems<E>(BWD), *p_o = n_o + kPlanes<E> * PL, *nt_o = p_o, *pt_o = nt_o + kPlanes<E> * PL;
        floatx4 a[10], gd[4];   // gd: Gam of the diagonal blocks
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j <= i; ++j) {
                const int b = tri_block(i, j), t = 16 * i + l;
                floatx4 gam;
                if (j < i) {
                    gam = row[t] * vec4(col + (i - 1) * kC + 16 * j + 4 * g);
                    a[b] = gam * kk[b];
                } else {
                    const floatx4 oh = vec4(chi + 16 * j + 4 * g), ol = vec4(clo + 16 * j + 4 * g);
                    const float th = chi[t], tl = clo[t];
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int s = 4 * g + r;
                        gam[r] = exp2_(s <= l ? ((th - oh[r]) + (tl - ol[r])) * kLog2e : 0.f);
                        a[b][r] = s < l ? gam[r] * kk[b][r] : 0.f;
                    }
                    gd[i] = gam;
                }
                *reinterpret_cast<floatx4 *>(A + b * kPrepBlock + l * kPrepRow + 4 * g) = a[b];
            }
        wave_sync();
        {
            // column l of Tm of diagonal block g
            const float *D = A + tri_block(0, 0) * kPrepBlock;
            D = A + (g == 0 ? tri_block(0, 0) : g == 1 ? tri_block(1, 1) : g == 2 ? tri_block(2, 2) : tri_block(3, 3)) * kPrepBlock;
            float x[16];
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                float s = 0.f;
#pragma unroll
                for (int e = 0; e < r; ++e) s += D[r * kPrepRow + e] * x[e];
                x[r] = (r == l ? 1.f : 0.f) - bt[16 * g + r] * s;
                Tm[(16 * g + r) * 17 + l] = x[r];
            }
        }
        wave_sync();
        // first operands: -(Db A)_kj (rows: tokens of block j) and Tm_jj^T
        float op[6][4], tm[4][4];
#pragma unroll
        for (int k = 1; k < 4; ++k)
#pragma unroll
            for (int j = 0; j < k; ++j)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    op[k * (k - 1) / 2 + j][r] = -bt[16 * k + 4 * g + r] * A[tri_block(k, j) * kPrepBlock + (4 * g + r) * kPrepRow + l];
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r) tm[j][r] = Tm[(16 * j + 4 * g + r) * 17 + l];
        // N^T, all block rows i at once (they are independent), j falling
#pragma unroll
        for (int dj = 0; dj < 4; ++dj)
#pragma unroll
            for (int i = dj; i < 4; ++i) {
                const int j = i - dj;
                floatx4 x = a[tri_block(i, j)], n = floatx4{0, 0, 0, 0};
#pragma unroll
                for (int k = j + 1; k <= i; ++k)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        x = __builtin_amdgcn_mfma_f32_16x16x4f32(op[k * (k - 1) / 2 + j][r], a[tri_block(i, k)][r], x, 0, 0, 0);
#pragma unroll
                for (int r = 0; r < 4; ++r) n = __builtin_amdgcn_mfma_f32_16x16x4f32(tm[j][r], x[r], n, 0, 0, 0);
                a[tri_block(i, j)] = n;   // A_ij is not needed again
            }
        // N with rows t; Gam Q K^T with rows t (forward); both with rows s (backward), through
        // products with the identity, plane by plane
        const floatx4 none = floatx4{0, 0, 0, 0};
        auto pair = [&](int i, int j) {   // block (i, j) of scale Gam o Q K^T
            const int b = tri_block(i, j), t = 16 * i + l;
            if (j < i) return (scale * (row[t] * vec4(col + (i - 1) * kC + 16 * j + 4 * g))) * qk[b];
            floatx4 d;
#pragma unroll
            for (int r = 0; r < 4; ++r) d[r] = 4 * g + r <= l ? scale * gd[i][r] * qk[b][r] : 0.f;
            return d;
        };
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int kb = 0; kb <= i / 2; ++kb) {
                const int j = 2 * kb;
                const bool two = j + 1 <= i;
                frag_t<E> f[2 * 2];   // hi, lo of N; hi, lo of the pair matrix
                split_pair(a[tri_block(i, j)], two ? a[tri_block(i, two ? j + 1 : j)] : none, f[0], f[1]);
                store_block<ONCE>(n_o + lower_block(i, kb) * 512 + 8 * lane, f[0]);
                if (kPlanes<E> == 2) store_block<ONCE>(n_o + PL + lower_block(i, kb) * 512 + 8 * lane, f[1]);
                split_pair(pair(i, j), two ? pair(i, two ? j + 1 : j) : none, f[2], f[3]);
                if (!BWD) {
                    store_block<ONCE>(p_o + lower_block(i, kb) * 512 + 8 * lane, f[2]);
                    if (kPlanes<E> == 2) store_block<ONCE>(p_o + PL + lower_block(i, kb) * 512 + 8 * lane, f[3]);
                    continue;
                }
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    E *o = (x ? pt_o : nt_o) + 8 * lane + 4 * (i & 1);
#pragma unroll
                    for (int half = 0; half < 2; ++half)
#pragma unroll
                        for (int pl = 0; pl < kPlanes<E>; ++pl) {
                            floatx4 d = none;
                            mma(d, f[2 * x + pl], sel.half[half]);
                            store_round4<ONCE>(o + pl * PL + upper_block(j + half, i >> 1) * 512, d);
                        }
                }
            }
        wave_sync();
    }
}

// ---------------------------------------------------------------------------
// the chains
// ---------------------------------------------------------------------------
struct ChainArgs {
    const void *kq, *tri;        // operand blocks per (chunk, group) and (chunk, head)
    const float *vec;
    const void *v, *dy;          // values; output gradients (backward)
    void *y, *dv;                // outputs of the forward / backward chain
    const float *s0, *d1;        // [chains,H,P,N] initial state, gradient of the final state, or null
    float *s1, *d0;              // final state, gradient of the initial state, or null
    void *sst, *ust, *dst, *hst; // backward only: S, U, D, H of every (chunk, head)
    Chunks m;
    int H, G, P, N, Pp, np;      // Pp: P rounded up to 32; np: workgroups per head
    int units;                   // chains * H * np
    float scale;
};

// The state of 16 columns as second operands.
template <typename E, int NB> struct StateOps {
    frag_t<E> hi[NB / 2], lo[NB / 2];
    __device__ __forceinline__ void of(const floatx4 (&s)[NB])
    {
#pragma unroll
        for (int kb = 0; kb < NB / 2; ++kb) split_pair(s[2 * kb], s[2 * kb + 1], hi[kb], lo[kb]);
    }
};

template <typename E, int NB>
__device__ __forceinline__ void load_state(const float *src, floatx4 (&s)[NB], int p, int g, int P, int N, int n0 = 0)
{
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
        const int n = n0 + 16 * nb + 4 * g;
        s[nb] = floatx4{0, 0, 0, 0};
        if (src && p < P && n < N) s[nb] = *reinterpret_cast<const floatx4 *>(src + (int64_t)p * N + n);
    }
}
template <int NB>
__device__ __forceinline__ void save_state(float *dst, const floatx4 (&s)[NB], int p, int g, int P, int N, int n0 = 0)
{
    if (!dst || p >= P) return;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
        const int n = n0 + 16 * nb + 4 * g;
        if (n < N) *reinterpret_cast<floatx4 *>(dst + (int64_t)p * N + n) = s[nb];
    }
}

// S, U, D and H of a chunk and head are kept as operand blocks with their columns p as
// slots (in order, 8 per lane): for every 32 columns the row blocks of each plane, so that
// what the gradient kernel takes at a time is contiguous.  Where lane (g, l) puts columns
// p0 + 4 g .. + 3 of row l of row block b (a wave's 16 x 16 piece is 512 contiguous bytes of
// bf16):
template <typename E> __device__ __forceinline__ int64_t piece(int b, int rows, int p0, int g, int l, int plane)
{
    const int block = ((p0 >> 5) * kPlanes<E> + plane) * rows + b;
    return ((int64_t)block * 64 + l + 16 * (((p0 & 31) >> 3) + (g >> 1))) * 8 + 4 * (g & 1);
}
template <typename E, int NF> __device__ __forceinline__ void store_pieces(E *dst, const frag_t<E> (&hi)[NF],
                                                                           const frag_t<E> (&lo)[NF], const Select<E> &sel,
                                                                           int p0, int lane, int rows = 2 * NF, int row0 = 0)
{
#pragma unroll
    for (int b = 0; b < 2 * NF; ++b)
#pragma unroll
        for (int pl = 0; pl < kPlanes<E>; ++pl) {
            floatx4 d = floatx4{0, 0, 0, 0};
            mma(d, pl ? lo[b >> 1] : hi[b >> 1], sel.half[b & 1]);
            store_round4<true>(dst + piece<E>(row0 + b, rows, p0, lane >> 4, lane & 15, pl), d);
        }
}
// One 16 x 16 accumulator of such a matrix of 64 rows.
template <typename E> __device__ __forceinline__ void store_piece(E *dst, const floatx4 &v, const Select<E> &sel, int b,
                                                                  int p0, int lane)
{
    frag_t<E> hi, lo;
    split_pair(v, floatx4{0, 0, 0, 0}, hi, lo);
#pragma unroll
    for (int pl = 0; pl < kPlanes<E>; ++pl) {
        floatx4 d = floatx4{0, 0, 0, 0};
        mma(d, pl ? lo : hi, sel.half[0]);
        store_round4(dst + piece<E>(b, 4, p0, lane >> 4, lane & 15, pl), d);
    }
}

// A [64 tokens][16 columns] tile of a caller's tensor: lane (g, l) moves columns
// 4 g .. 4 g + 3 of token 16 tb + l (`off`: byte offset of column p0 + 4 g, kOffNone past P).
template <typename E> struct Tile {
    typedef E vec __attribute__((ext_vector_type(4)));
    vec x[4];
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t rs, uint32_t ld, uint32_t off, int l)
    {
#pragma unroll
        for (int tb = 0; tb < 4; ++tb) {
            const uint32_t o = off + (16 * tb + l) * ld;
            if constexpr (sizeof(E) == 2)
                x[tb] = __builtin_bit_cast(vec, __builtin_amdgcn_raw_buffer_load_b64(rs, o, 0, 0));
            else x[tb] = __builtin_bit_cast(vec, __builtin_amdgcn_raw_buffer_load_b128(rs, o, 0, 0));
        }
    }
    // to accumulators: rows t = 16 tb + 4 g + r, column p0 + l
    __device__ __forceinline__ void rows(floatx4 (&o)[4], const Select<E> &sel) const
    {
#pragma unroll
        for (int tb = 0; tb < 4; ++tb) {
            frag_t<E> f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                f[j] = x[tb][j];
                f[4 + j] = from_float<E>(0.f);
            }
            o[tb] = floatx4{0, 0, 0, 0};
            mma(o[tb], f, sel.half[0]);
        }
    }
};
template <typename E>
__device__ __forceinline__ void store_tile(__amdgpu_buffer_rsrc_t rs, uint32_t ld, uint32_t off, const floatx4 (&x)[4],
                                           const Select<E> &sel, int l)
{
    const frag_t<E> f[2] = {round_pair<E>(x[0], x[1]), round_pair<E>(x[2], x[3])};
#pragma unroll
    for (int tb = 0; tb < 4; ++tb) {
        floatx4 d = floatx4{0, 0, 0, 0};
        mma(d, f[tb >> 1], sel.half[tb & 1]);
        const uint32_t o = off + (16 * tb + l) * ld;
        if constexpr (sizeof(E) == 2) {
            const uint2 v = uint2{pack_bf16x2(d[0], d[1]), pack_bf16x2(d[2], d[3])};
            __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(__attribute__((__vector_size__(8))) unsigned int, v),
                                                  rs, o, 0, 0);
        } else {
            __builtin_amdgcn_raw_buffer_store_b128(
                __builtin_bit_cast(__attribute__((__vector_size__(16))) unsigned int, d), rs, o, 0, 0);
        }
    }
}


// ---- operands of a chain's step, staged through LDS ----
// The waves of a workgroup own different columns and read the same first operands, 44
// to 72 KB a step at N = 128.  They come straight from memory into LDS (16 bytes per
// lane, no registers), in two regions: phase 1 of a step reads what meets the entering
// state (K, and Q or the pair matrix), phase 2 the rest.  While a phase computes from one
// region, the other one's next contents are in flight; one barrier before each phase says
// both that its operands are there and that the other region is free.  Sets too large for
// LDS (fp32 at N = 256) are read from global memory by every wave (STAGED false).
//
// 8 x 2048 tokens of 80 heads of 64, N = 128, both directions: 720 us for 3.6 GB, 5.0 TB/s of
// the 5.1 that a copy reaches.  (While S, U, D and H were kept as single bf16 numbers, 2.5 GB
// took 620 us; without the operand loads or without the stores 480 and 440 us, without both
// 305 us, the arithmetic's own time at two workgroups a CU.)  Packed prompts of 64 heads,
// forward: 229 us.
template <typename E, int NT> constexpr bool kStaged = sizeof(E) * NT <= 512;

// KIND 0: the forward (y), 1: the forward for the backward (S and U), 2: the backward
template <typename E, int NB, int KIND, bool STAGED> struct Regions {
    static constexpr int kMat = 4 * NB / 2;   // blocks of K, K^T, Q or Q^T (64 x NT)
    static constexpr int kN = kTri * kPlanes<E>;
    // phase 1: K | Q (KIND 0) or the transposed pair matrix (KIND 2)
    static constexpr int kOne = kMat + (KIND == 0 ? kMat : KIND == 2 ? kN : 0);
    // phase 2: N or N^T | the pair matrix (KIND 0) | K^T | Q^T (KIND 2)
    static constexpr int kTwo = kN + (KIND == 0 ? kN : 0) + kMat + (KIND == 2 ? kMat : 0);
    static constexpr int kBytes = STAGED ? (kOne + kTwo) * 512 * (int)sizeof(E) + 2 * kVecChain * 4 : 16;
};

typedef __attribute__((address_space(1))) const void *gptr_t;
typedef __attribute__((address_space(3))) void *lptr_t;

// What is read by one workgroup only is loaded, and what another kernel reads much later
// is stored, past the caches (non-temporal), which keeps them for K and Q, whose blocks a
// group's heads share: 8 x 2048 tokens of 80 heads, chains 666 -> 639 us, gradients 592 ->
// 558 us; packed prompts' chains 245 -> 238 us (all while the outputs took single bf16 numbers).
constexpr int kOnce = 2;

// `n` operand blocks from memory to LDS, a wave every fourth block.
template <typename E, int n, int HOW = 0> __device__ __forceinline__ void stage(const E *src, E *dst, int wv, int lane)
{
    constexpr int V = kVec16<E>;
#pragma unroll
    for (int b0 = 0; b0 < n; b0 += 4) {
        const int b = b0 + wv;
        if (n % 4 == 0 || b < n)
#pragma unroll
            for (int j = 0; j < 512; j += 64 * V)
                __builtin_amdgcn_global_load_lds((gptr_t)(src + b * 512 + j + V * lane), (lptr_t)(dst + b * 512 + j), 16,
                                                 0, HOW);
    }
}
// This wave's loads have arrived.  Called before a step's stores are issued, so that
// the next barrier does not wait for them.
__device__ __forceinline__ void loads_done() { __builtin_amdgcn_s_waitcnt(0x0f70); }   // vmcnt(0)

// A step's operand pointers: in LDS, or in memory.
template <typename E, int NB, int KIND, bool STAGED> struct Operands {
    using R = Regions<E, NB, KIND, STAGED>;
    static constexpr int kMatE = kC * 16 * NB;
    E *one, *two;
    float *vecs;
    const E *kq, *tri;
    const float *vec;
    int wv, lane, turn;   // turn: which of the two copies of the scalars is being staged

    __device__ __forceinline__ void init(char *smem, int wv_, int lane_)
    {
        one = reinterpret_cast<E *>(smem);
        two = one + R::kOne * 512;
        vecs = reinterpret_cast<float *>(two + R::kTwo * 512);
        wv = wv_;
        lane = lane_;
        turn = 0;
    }
    // where chunk c's operands are in memory
    __device__ __forceinline__ void at(const ChainArgs &a, int c, int h, int grp)
    {
        const int64_t u = (int64_t)c * a.H + h;
        kq = (const E *)a.kq + ((int64_t)c * a.G + grp) * (KIND == 0 ? 3 : 4) * kMatE;
        tri = (const E *)a.tri + u * tri_elems<E>(KIND != 0);
        vec = a.vec + u * kVec;
    }
    // in `tri`: N | Gam QK^T, or N | N^T | (Gam QK^T)^T; in `kq`: K | K^T | Q | Q^T
    static constexpr int kPL = 512 * kTri, kNt = kPlanes<E> * kPL, kPt = 2 * kPlanes<E> * kPL;
    __device__ __forceinline__ void stage_one()
    {
        if constexpr (STAGED) {
            stage<E, R::kMat>(kq, one, wv, lane);
            if (KIND == 0) stage<E, R::kMat>(kq + 2 * kMatE, one + kMatE, wv, lane);
            if (KIND == 2) stage<E, R::kN, kOnce>(tri + kPt, one + kMatE, wv, lane);
            if (wv >= 2)   // kVecChain floats: two loads
                __builtin_amdgcn_global_load_lds((gptr_t)(vec + 256 * (wv - 2) + 4 * lane),
                                                 (lptr_t)(vecs + kVecChain * turn + 256 * (wv - 2)), 16, 0, 0);
        }
    }
    __device__ __forceinline__ void stage_two()
    {
        if constexpr (STAGED) {
            E *o = two;
            stage<E, R::kN, kOnce>(tri + (KIND == 2 ? kNt : 0), o, wv, lane);
            o += R::kN * 512;
            if (KIND == 0) {
                stage<E, R::kN, kOnce>(tri + kPlanes<E> * kPL, o, wv, lane);
                o += R::kN * 512;
            }
            stage<E, R::kMat>(kq + kMatE, o, wv, lane);
            if (KIND == 2) stage<E, R::kMat>(kq + 3 * kMatE, o + kMatE, wv, lane);
        }
    }
    __device__ __forceinline__ const E *k() const { return (STAGED ? one : kq) + 8 * lane; }
    __device__ __forceinline__ const E *q() const { return (STAGED ? one + kMatE : kq + 2 * kMatE) + 8 * lane; }
    __device__ __forceinline__ const E *pt() const { return (STAGED ? one + kMatE : tri + kPt) + 8 * lane; }
    __device__ __forceinline__ const E *n() const { return (STAGED ? two : tri + (KIND == 2 ? kNt : 0)) + 8 * lane; }
    __device__ __forceinline__ const E *p() const { return (STAGED ? two + R::kN * 512 : tri + kPlanes<E> * kPL) + 8 * lane; }
    __device__ __forceinline__ const E *kt() const
    {
        return (STAGED ? two + (R::kN + (KIND == 0 ? R::kN : 0)) * 512 : kq + kMatE) + 8 * lane;
    }
    __device__ __forceinline__ const E *qt() const { return (STAGED ? two + R::kN * 512 + kMatE : kq + 3 * kMatE) + 8 * lane; }
    // the scalars of the step whose turn is t
    __device__ __forceinline__ const float *scalars(int t) const { return STAGED ? vecs + kVecChain * t : vec; }
};

// Workgroup -> unit (chain, head, column tile).  Workgroups go round the 8 XCDs; where a
// chain's units divide by 8, an XCD takes consecutive ones, so that the heads of a group find
// its K and Q in one L2 (packed prompts, 8 groups of 8 heads: chains 235 -> 209 us, before y
// took two bf16 numbers for its operands; ragged fp32, 3 groups of 2: 38 -> 34 us).  Not with all heads in one group, whose K and Q every L2
// holds anyway.
__device__ __forceinline__ int by_group(const ChainArgs &a, int unit)
{
    const int per = a.np * a.H, i = unit % per;
    return a.G > 1 && per % 8 == 0 ? unit - i + (i & 7) * (per >> 3) + (i >> 3) : unit;
}

// One forward chain.  KEEP: for the backward, which wants S and U of every chunk
// and not y.
template <typename E, int NB, bool KEEP, bool STAGED>
__device__ __forceinline__ void chain_fwd(const ChainArgs &a, int unit, char *smem)
{
    constexpr int NT = 16 * NB, NK = NT / 32, PL = 512 * kTri;
    const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), g = lane >> 4, l = lane & 15;
    const int ptile = unit % a.np, h = (unit / a.np) % a.H;
    int ch = unit / (a.np * a.H);
    const int p0 = ptile * kC + 16 * wv;
    const bool keep = p0 < a.Pp;
    int c0, n, len;
    int64_t t0;
    chain_at(a.m, ch, c0, n, t0, len);
    const int64_t so = ((int64_t)ch * a.H + h) * a.P * a.N, ld = (int64_t)a.H * a.P;
    floatx4 S[NB];
    load_state<E, NB>(a.s0 ? a.s0 + so : nullptr, S, p0 + l, g, a.P, a.N);
    const uint32_t ldb = (uint32_t)ld * sizeof(E), poff = p0 < a.P ? (p0 + 4 * g) * sizeof(E) : kOffNone;
    const int grp = h / (a.H / a.G);
    auto rows_of = [&](const void *base, int i) {   // the head's rows of the chain's chunk i
        const int left = len - i * kC;
        return rows_rsrc((const E *)base + ((t0 + i * kC) * a.H + h) * a.P, left < kC ? left : kC, ld, a.P);
    };
    Select<E> sel;
    sel.init(lane);
    Operands<E, NB, KEEP ? 1 : 0, STAGED> op;
    op.init(smem, wv, lane);
    Tile<E> v;
    if (n > 0) {
        op.at(a, c0, h, grp);
        op.stage_one();
        v.load(rows_of(a.v, 0), ldb, poff, l);
    }
    for (int i = 0; i < n; ++i) {
        const int64_t u = (int64_t)(c0 + i) * a.H + h;
        if (STAGED) {
            if (i == 0) loads_done();
            __syncthreads();
        }
        op.stage_two();
        floatx4 R[4], X[4];
        v.rows(R, sel);
        const float *vec = op.scalars(op.turn);
        StateOps<E, NB> so_;
        so_.of(S);
        floatx4 ks[4], qs[4];
        const E *kf = op.k(), *qf = op.q();
#pragma unroll
        for (int tb = 0; tb < 4; ++tb) ks[tb] = qs[tb] = floatx4{0, 0, 0, 0};
#pragma unroll
        for (int kb = 0; kb < NK; ++kb)
#pragma unroll
            for (int tb = 0; tb < 4; ++tb) {
                const frag_t<E> f = load_frag(kf + (tb * NK + kb) * 512);
                mma(ks[tb], f, so_.hi[kb]);
                if (kPlanes<E> == 2) mma(ks[tb], f, so_.lo[kb]);
                if (!KEEP) {
                    const frag_t<E> fq = load_frag(qf + (tb * NK + kb) * 512);
                    mma(qs[tb], fq, so_.hi[kb]);
                    if (kPlanes<E> == 2) mma(qs[tb], fq, so_.lo[kb]);
                }
            }
        floatx4 bt[4];
#pragma unroll
        for (int tb = 0; tb < 4; ++tb) {
            bt[tb] = vec4(vec + kBeta + 16 * tb + 4 * g);
            R[tb] -= vec4(vec + kSince + 16 * tb + 4 * g) * ks[tb];
            X[tb] = bt[tb] * R[tb];
        }
        frag_t<E> xh[2], xl[2];
        split_pair(X[0], X[1], xh[0], xl[0]);
        split_pair(X[2], X[3], xh[1], xl[1]);
        if (STAGED) {
            loads_done();
            __syncthreads();
        }
        const E *nf = op.n(), *pf = op.p(), *ktf = op.kt();
        if (i + 1 < n) {
            op.at(a, c0 + i + 1, h, grp);
            op.turn ^= 1;
            op.stage_one();
            v.load(rows_of(a.v, i + 1), ldb, poff, l);
        }
#pragma unroll
        for (int tb = 0; tb < 4; ++tb) {
            floatx4 d = floatx4{0, 0, 0, 0};
#pragma unroll
            for (int kb = 0; kb <= tb / 2; ++kb) {
                const frag_t<E> f = load_frag(nf + lower_block(tb, kb) * 512);
                mma(d, f, xh[kb]);
                if (kPlanes<E> == 2) {
                    mma(d, f, xl[kb]);
                    mma(d, load_frag(nf + PL + lower_block(tb, kb) * 512), xh[kb]);
                }
            }
            R[tb] -= d;   // U
            X[tb] = vec4(vec + kTillBeta + 16 * tb + 4 * g) * R[tb];
        }
        // beta U for y, or U itself for the backward
        frag_t<E> w[2], wl[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            if (KEEP) split_pair(R[2 * j], R[2 * j + 1], w[j], wl[j]);
            else split_pair(bt[2 * j] * R[2 * j], bt[2 * j + 1] * R[2 * j + 1], w[j], wl[j]);
        }
        split_pair(X[0], X[1], xh[0], xl[0]);
        split_pair(X[2], X[3], xh[1], xl[1]);
        const float whole = vec[kSince + kC - 1];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) S[nb] *= whole;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int kb = 0; kb < 2; ++kb) {
                const frag_t<E> f = load_frag(ktf + (2 * nb + kb) * 512);
                mma(S[nb], f, xh[kb]);
                if (kPlanes<E> == 2) mma(S[nb], f, xl[kb]);
            }
        if (KEEP) {
            if (STAGED) loads_done();
            if (keep) {
                store_pieces<E>((E *)a.sst + u * kPlanes<E> * NT * a.Pp, so_.hi, so_.lo, sel, p0, lane);
                store_pieces<E>((E *)a.ust + u * kPlanes<E> * kC * a.Pp, w, wl, sel, p0, lane);
            }
        } else {
            floatx4 y[4];
#pragma unroll
            for (int tb = 0; tb < 4; ++tb) {
                y[tb] = vec4(vec + kScaled + 16 * tb + 4 * g) * qs[tb];
#pragma unroll
                for (int kb = 0; kb <= tb / 2; ++kb) {
                    const frag_t<E> f = load_frag(pf + lower_block(tb, kb) * 512);
                    mma(y[tb], f, w[kb]);
                    if (kPlanes<E> == 2) {
                        mma(y[tb], f, wl[kb]);
                        mma(y[tb], load_frag(pf + PL + lower_block(tb, kb) * 512), w[kb]);
                    }
                }
            }
            if (STAGED) loads_done();
            store_tile<E>(rows_of(a.y, i), ldb, poff, y, sel, l);
        }
    }
    save_state<NB>(a.s1 ? a.s1 + so : nullptr, S, p0 + l, g, a.P, a.N);
}

// One backward chain: D of every chunk (the gradient of the state that leaves it),
// H, and dv.
template <typename E, int NB, bool STAGED>
__device__ __forceinline__ void chain_bwd(const ChainArgs &a, int unit, char *smem)
{
    constexpr int NT = 16 * NB, NK = NT / 32, PL = 512 * kTri;
    const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), g = lane >> 4, l = lane & 15;
    const int ptile = unit % a.np, h = (unit / a.np) % a.H;
    int ch = unit / (a.np * a.H);
    const int p0 = ptile * kC + 16 * wv;
    const bool keep = p0 < a.Pp;
    int c0, n, len;
    int64_t t0;
    chain_at(a.m, ch, c0, n, t0, len);
    const int64_t so = ((int64_t)ch * a.H + h) * a.P * a.N, ld = (int64_t)a.H * a.P;
    floatx4 D[NB];
    load_state<E, NB>(a.d1 ? a.d1 + so : nullptr, D, p0 + l, g, a.P, a.N);
    const uint32_t ldb = (uint32_t)ld * sizeof(E), poff = p0 < a.P ? (p0 + 4 * g) * sizeof(E) : kOffNone;
    const int grp = h / (a.H / a.G);
    auto rows_of = [&](const void *base, int i) {
        const int left = len - i * kC;
        return rows_rsrc((const E *)base + ((t0 + i * kC) * a.H + h) * a.P, left < kC ? left : kC, ld, a.P);
    };
    Select<E> sel;
    sel.init(lane);
    Operands<E, NB, 2, STAGED> op;
    op.init(smem, wv, lane);
    Tile<E> dy;
    if (n > 0) {
        op.at(a, c0 + n - 1, h, grp);
        op.stage_one();
        dy.load(rows_of(a.dy, n - 1), ldb, poff, l);
    }
    for (int i = n - 1; i >= 0; --i) {
        const int64_t u = (int64_t)(c0 + i) * a.H + h;
        if (STAGED) {
            if (i == n - 1) loads_done();
            __syncthreads();
        }
        op.stage_two();
        floatx4 yt[4];
        dy.rows(yt, sel);
        const float *vec = op.scalars(op.turn);
        StateOps<E, NB> dop;
        dop.of(D);
        const frag_t<E> y0 = round_pair<E>(yt[0], yt[1]), y1 = round_pair<E>(yt[2], yt[3]);   // exact
        const E *kf = op.k(), *ptf = op.pt();
        floatx4 W[4], X[4], bt[4];
#pragma unroll
        for (int tb = 0; tb < 4; ++tb) W[tb] = floatx4{0, 0, 0, 0};
#pragma unroll
        for (int kb = 0; kb < NK; ++kb)
#pragma unroll
            for (int tb = 0; tb < 4; ++tb) {
                const frag_t<E> f = load_frag(kf + (tb * NK + kb) * 512);
                mma(W[tb], f, dop.hi[kb]);
                if (kPlanes<E> == 2) mma(W[tb], f, dop.lo[kb]);
            }
#pragma unroll
        for (int tb = 0; tb < 4; ++tb) {
            W[tb] *= vec4(vec + kTill + 16 * tb + 4 * g);
            bt[tb] = vec4(vec + kBeta + 16 * tb + 4 * g);
#pragma unroll
            for (int kb = tb / 2; kb < 2; ++kb)
#pragma unroll
                for (int pl = 0; pl < kPlanes<E>; ++pl)
                    mma(W[tb], load_frag(ptf + pl * PL + upper_block(tb, kb) * 512), kb ? y1 : y0);
            X[tb] = bt[tb] * W[tb];
        }
        frag_t<E> xh[2], xl[2];
        split_pair(X[0], X[1], xh[0], xl[0]);
        split_pair(X[2], X[3], xh[1], xl[1]);
        if (STAGED) {
            loads_done();
            __syncthreads();
        }
        const E *nt = op.n(), *ktf = op.kt(), *qtf = op.qt();
        if (i > 0) {
            op.at(a, c0 + i - 1, h, grp);
            op.turn ^= 1;
            op.stage_one();
            dy.load(rows_of(a.dy, i - 1), ldb, poff, l);
        }
        const float whole = vec[kSince + kC - 1];
        frag_t<E> yh[2], yl[2];
#pragma unroll
        for (int tb = 0; tb < 4; ++tb) yt[tb] *= vec4(vec + kScaled + 16 * tb + 4 * g);
        split_pair(yt[0], yt[1], yh[0], yl[0]);
        split_pair(yt[2], yt[3], yh[1], yl[1]);
#pragma unroll
        for (int tb = 0; tb < 4; ++tb) {
            floatx4 d = floatx4{0, 0, 0, 0};
#pragma unroll
            for (int kb = tb / 2; kb < 2; ++kb) {
                const frag_t<E> f = load_frag(nt + upper_block(tb, kb) * 512);
                mma(d, f, xh[kb]);
                if (kPlanes<E> == 2) {
                    mma(d, f, xl[kb]);
                    mma(d, load_frag(nt + PL + upper_block(tb, kb) * 512), xh[kb]);
                }
            }
            W[tb] -= d;             // H
            X[tb] = bt[tb] * W[tb]; // dv
        }
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) D[nb] *= whole;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int kb = 0; kb < 2; ++kb) {
                const frag_t<E> fq = load_frag(qtf + (2 * nb + kb) * 512);
                mma(D[nb], fq, yh[kb]);
                if (kPlanes<E> == 2) mma(D[nb], fq, yl[kb]);
            }
        frag_t<E> hf[2], hl[2];
        split_pair(W[0], W[1], hf[0], hl[0]);
        split_pair(W[2], W[3], hf[1], hl[1]);
#pragma unroll
        for (int tb = 0; tb < 4; ++tb) W[tb] *= vec4(vec + kErase + 16 * tb + 4 * g);
        split_pair(W[0], W[1], xh[0], xl[0]);
        split_pair(W[2], W[3], xh[1], xl[1]);
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int kb = 0; kb < 2; ++kb) {
                const frag_t<E> f = load_frag(ktf + (2 * nb + kb) * 512);
                mma(D[nb], f, xh[kb]);
                if (kPlanes<E> == 2) mma(D[nb], f, xl[kb]);
            }
        if (STAGED) loads_done();
        store_tile<E>(rows_of(a.dv, i), ldb, poff, X, sel, l);
        if (keep) {
            store_pieces<E>((E *)a.dst + u * kPlanes<E> * NT * a.Pp, dop.hi, dop.lo, sel, p0, lane);
            store_pieces<E>((E *)a.hst + u * kPlanes<E> * kC * a.Pp, hf, hl, sel, p0, lane);
        }
    }
    save_state<NB>(a.d0 ? a.d0 + so : nullptr, D, p0 + l, g, a.P, a.N);
}

// ---- narrow chains ----
// With fewer chains than CUs a step's length is all that counts.  Here a workgroup owns 16
// columns and its kNW waves share a step: the state's rows n are split over them (each
// holds its part, and multiplies its part of K, Q and K^T), and so are the chunk's tokens
// (16 or 32 each) for what is not a product with the state.  Three exchanges through LDS a
// step: the partial products K S (and Q S), the right-hand sides X, and U.  Every first
// operand is now used by one wave once, so it comes from memory into registers, requested
// for the next step as soon as this step has used it.
//
// 16K tokens of 32 heads, N = 256: 645 us, 2.5 us a step; 545 us (wide: 1.36 ms), 2.1 us a
// step, before y took two bf16 numbers for its operands: 1.4 us for the chain of products and
// exchanges and the rest for 112 KB of operands at a CU's 64 bytes a cycle.  2 x 2048 tokens
// of 24 heads, N = 64, both directions: 82 us.  Requests issued earlier, between the products,
// made no difference then (570 us), nor did touching the operands of two steps ahead for L2
// (570 us).
template <int NB> constexpr int kNW = NB / 2 < 4 ? NB / 2 : 4;
template <typename E, int NB, int KIND> struct Narrow {
    static constexpr int NW = kNW<NB>, NBW = NB / NW, TBW = 4 / NW, KBW = NBW / 2, NK = NB / 2;
    static constexpr int kPart = NW * 4 * 64 * 4;                         // floats: [wave][tb][lane][4]
    static constexpr int kFrag = 512 * kPlanes<E>;                        // elements of a split operand
    static constexpr int kBytes = (KIND == 0 ? 2 : 1) * kPart * 4 + (KIND == 0 ? 3 : 2) * 2 * kFrag * (int)sizeof(E);
};
// The half of a split second operand that the 16 tokens of row block tb are, and the operand.
template <typename E> __device__ __forceinline__ void put_half(E *f, int tb, int lane, const floatx4 &v)
{
    store_split4(f + (tb >> 1) * 512 * kPlanes<E> + 8 * lane + 4 * (tb & 1), 512, v);
}
template <typename E> __device__ __forceinline__ void get_split(const E *f, int kb, int lane, frag_t<E> &hi, frag_t<E> &lo)
{
    hi = load_frag(f + kb * 512 * kPlanes<E> + 8 * lane);
    if (kPlanes<E> == 2) lo = load_frag(f + kb * 512 * kPlanes<E> + 512 + 8 * lane);
}
// Operand blocks of one chunk behind a buffer resource: lane offset fixed, block number in
// the scalar offset (a 64-bit address per load costs two vector instructions each).
template <typename E> struct Blocks {
    __amdgpu_buffer_rsrc_t rs;
    uint32_t off;   // the lane's
    __device__ __forceinline__ void at(const E *base, int elems, int lane)
    {
        rs = make_rsrc_n(base, elems * (int)sizeof(E));
        off = lane * 8 * sizeof(E);
    }
    __device__ __forceinline__ frag_t<E> get(int elem0) const   // block starting at element elem0
    {
        const uint32_t so = __builtin_amdgcn_readfirstlane(elem0 * (int)sizeof(E));
        if constexpr (sizeof(E) == 2) return __builtin_bit_cast(bf16x8, bload16s(rs, off, so));
        else {
            const floatx4 lo = __builtin_bit_cast(floatx4, bload16s(rs, off, so));
            const floatx4 hi = __builtin_bit_cast(floatx4, bload16s(rs, off + 16, so));
            return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
        }
    }
};
// acc += T X for row block tb of a triangle T (blocks given by block(tb, kb), planes PL
// apart) and split X; `from`, `to`: the range of kb.
template <typename E> struct TriRow {
    frag_t<E> hi[2], lo[2];
    template <typename B> __device__ __forceinline__ void load(const Blocks<E> &t, int e0, int k0, int k1, B block)
    {
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {   // a block outside the triangle: another one in its place
            const int b = block(kb < k0 ? k0 : kb > k1 ? k1 : kb);
            hi[kb] = t.get(e0 + b * 512);
            if (kPlanes<E> == 2) lo[kb] = t.get(e0 + 512 * kTri + b * 512);
        }
    }
    __device__ __forceinline__ void product(floatx4 &d, int k0, int k1, const frag_t<E> (&xh)[2], const frag_t<E> (&xl)[2]) const
    {
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
            if (kb >= k0 && kb <= k1) {
                mma(d, hi[kb], xh[kb]);
                if (kPlanes<E> == 2) {
                    mma(d, hi[kb], xl[kb]);
                    mma(d, lo[kb], xh[kb]);
                }
            }
    }
};
// One 16 x 16 tile of a caller's rows, as Tile.
template <typename E> __device__ __forceinline__ floatx4 tile_rows(const typename Tile<E>::vec &x, const Select<E> &sel)
{
    frag_t<E> f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        f[j] = x[j];
        f[4 + j] = from_float<E>(0.f);
    }
    floatx4 o = floatx4{0, 0, 0, 0};
    mma(o, f, sel.half[0]);
    return o;
}
template <typename E> __device__ __forceinline__ typename Tile<E>::vec tile_load(__amdgpu_buffer_rsrc_t rs, uint32_t off)
{
    if constexpr (sizeof(E) == 2) return __builtin_bit_cast(typename Tile<E>::vec, __builtin_amdgcn_raw_buffer_load_b64(rs, off, 0, 0));
    else return __builtin_bit_cast(typename Tile<E>::vec, __builtin_amdgcn_raw_buffer_load_b128(rs, off, 0, 0));
}
template <typename E> __device__ __forceinline__ floatx4 transposed(const floatx4 &v, const Select<E> &sel)
{
    floatx4 d = floatx4{0, 0, 0, 0};
    mma(d, round_pair<E>(v, floatx4{0, 0, 0, 0}), sel.half[0]);
    return d;
}
template <typename E> __device__ __forceinline__ void tile_store(__amdgpu_buffer_rsrc_t rs, uint32_t off, const floatx4 &v,
                                                                 const Select<E> &sel)
{
    const floatx4 d = transposed<E>(v, sel);
    if constexpr (sizeof(E) == 2)
        __builtin_amdgcn_raw_buffer_store_b64(
            __builtin_bit_cast(__attribute__((__vector_size__(8))) unsigned int, uint2{pack_bf16x2(d[0], d[1]), pack_bf16x2(d[2], d[3])}),
            rs, off, 0, 0);
    else
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(__attribute__((__vector_size__(16))) unsigned int, d), rs, off, 0, 0);
}

template <typename E, int NB, bool KEEP>
__device__ __forceinline__ void narrow_fwd(const ChainArgs &a, int unit, char *smem)
{
    constexpr int KIND = KEEP ? 1 : 0;
    using C = Narrow<E, NB, KIND>;
    constexpr int NT = 16 * NB, kMat = kC * NT, NW = C::NW, NBW = C::NBW, TBW = C::TBW, KBW = C::KBW, NK = C::NK;
    constexpr int kTriE = 512 * kTri;
    float *part = reinterpret_cast<float *>(smem), *partq = part + C::kPart;
    E *xf = reinterpret_cast<E *>(part + (KEEP ? 1 : 2) * C::kPart), *uf = xf + 2 * C::kFrag, *wf = uf + 2 * C::kFrag;
    const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), g = lane >> 4, l = lane & 15;
    const int ptile = unit % a.np, h = (unit / a.np) % a.H;
    int ch = unit / (a.np * a.H);
    const int p0 = 16 * ptile;
    int c0, n, len;
    int64_t t0;
    chain_at(a.m, ch, c0, n, t0, len);
    const int64_t so = ((int64_t)ch * a.H + h) * a.P * a.N, ld = (int64_t)a.H * a.P;
    floatx4 S[NBW];
    load_state<E, NBW>(a.s0 ? a.s0 + so : nullptr, S, p0 + l, g, a.P, a.N, 16 * NBW * wv);
    const uint32_t ldb = (uint32_t)ld * sizeof(E), poff = p0 < a.P ? (p0 + 4 * g) * sizeof(E) : kOffNone;
    const int grp = h / (a.H / a.G);
    auto rows_of = [&](const void *base, int i) {
        const int left = len - i * kC;
        return rows_rsrc((const E *)base + ((t0 + i * kC) * a.H + h) * a.P, left < kC ? left : kC, ld, a.P);
    };
    Select<E> sel;
    sel.init(lane);
    frag_t<E> kf[4][KBW], qf[KEEP ? 1 : 4][KBW], ktf[NBW][2];
    TriRow<E> nf[TBW], pf[KEEP ? 1 : TBW];
    floatx4 since[TBW], bt[TBW], tillb[TBW], scaled[TBW];
    typename Tile<E>::vec v[TBW];
    float whole;
    Blocks<E> kq, tri;
    __amdgpu_buffer_rsrc_t vec;
    auto at = [&](int i) {
        const int64_t u = (int64_t)(c0 + i) * a.H + h;
        constexpr int kq_e = (KEEP ? 4 : 3) * kMat, tri_e = tri_elems<E>(KEEP);
        kq.at((const E *)a.kq + ((int64_t)(c0 + i) * a.G + grp) * kq_e, kq_e, lane);
        tri.at((const E *)a.tri + u * tri_e, tri_e, lane);
        vec = make_rsrc_n(a.vec + u * kVec, kVec * 4);
    };
    auto scalars = [&](int which, int tb) {
        return __builtin_bit_cast(floatx4, bload16s(vec, 16 * g, __builtin_amdgcn_readfirstlane(4 * (which + 16 * tb))));
    };
    auto load_k = [&]() {
#pragma unroll
        for (int tb = 0; tb < 4; ++tb)
#pragma unroll
            for (int kb = 0; kb < KBW; ++kb) kf[tb][kb] = kq.get((tb * NK + wv * KBW + kb) * 512);
    };
    auto load_q = [&]() {
        if (!KEEP)
#pragma unroll
            for (int tb = 0; tb < 4; ++tb)
#pragma unroll
                for (int kb = 0; kb < KBW; ++kb) qf[tb][kb] = kq.get(2 * kMat + (tb * NK + wv * KBW + kb) * 512);
    };
    auto load_v = [&](int i) {
        const __amdgpu_buffer_rsrc_t rs = rows_of(a.v, i);
#pragma unroll
        for (int j = 0; j < TBW; ++j) {
            const int tb = wv * TBW + j;
            v[j] = tile_load<E>(rs, poff + (16 * tb + l) * ldb);
            since[j] = scalars(kSince, tb);
            bt[j] = scalars(kBeta, tb);
        }
    };
    auto load_tri = [&]() {
#pragma unroll
        for (int j = 0; j < TBW; ++j) {
            const int tb = wv * TBW + j;
            nf[j].load(tri, 0, 0, tb >> 1, [&](int kb) { return lower_block(tb, kb); });
            if (!KEEP) pf[j].load(tri, kPlanes<E> * kTriE, 0, tb >> 1, [&](int kb) { return lower_block(tb, kb); });
        }
    };
    auto load_rest = [&]() {
#pragma unroll
        for (int j = 0; j < TBW; ++j) {
            const int tb = wv * TBW + j;
            tillb[j] = scalars(kTillBeta, tb);
            if (!KEEP) scaled[j] = scalars(kScaled, tb);
        }
        whole = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(vec, 4 * (kSince + kC - 1), 0, 0));
#pragma unroll
        for (int nb = 0; nb < NBW; ++nb)
#pragma unroll
            for (int kb = 0; kb < 2; ++kb) ktf[nb][kb] = kq.get(kMat + (2 * (wv * NBW + nb) + kb) * 512);
    };
    if (n > 0) {
        at(0);
        load_k();
        load_q();
        load_v(0);
        load_tri();
        load_rest();
    }
    for (int i = 0; i < n; ++i) {
        const int64_t u = (int64_t)(c0 + i) * a.H + h;
        // the last step requests its own operands again: no load is conditional, so that the
        // waits for them count exactly; and they stay in order (the scheduling barriers), since a
        // wait for one is a wait for all before it
        const int next = i + 1 < n ? i + 1 : i;
        StateOps<E, NBW> so_;
        so_.of(S);
        floatx4 ks[4], qs[4];
#pragma unroll
        for (int tb = 0; tb < 4; ++tb) ks[tb] = qs[tb] = floatx4{0, 0, 0, 0};
#pragma unroll
        for (int kb = 0; kb < KBW; ++kb)
#pragma unroll
            for (int tb = 0; tb < 4; ++tb) {
                mma(ks[tb], kf[tb][kb], so_.hi[kb]);
                if (kPlanes<E> == 2) mma(ks[tb], kf[tb][kb], so_.lo[kb]);
            }
#pragma unroll
        for (int tb = 0; tb < 4; ++tb) *reinterpret_cast<floatx4 *>(part + ((wv * 4 + tb) * 64 + lane) * 4) = ks[tb];
        at(next);
        load_k();
        __builtin_amdgcn_sched_barrier(0);
        __syncthreads();
        floatx4 R[TBW], sum[TBW][NW];
#pragma unroll
        for (int j = 0; j < TBW; ++j)
#pragma unroll
            for (int o = 0; o < NW; ++o) sum[j][o] = vec4(part + ((o * 4 + wv * TBW + j) * 64 + lane) * 4);
        if (!KEEP) {   // while these arrive: y's part of the state product, off the step's critical path
#pragma unroll
            for (int kb = 0; kb < KBW; ++kb)
#pragma unroll
                for (int tb = 0; tb < 4; ++tb) {
                    mma(qs[tb], qf[tb][kb], so_.hi[kb]);
                    if (kPlanes<E> == 2) mma(qs[tb], qf[tb][kb], so_.lo[kb]);
                }
        }
#pragma unroll
        for (int j = 0; j < TBW; ++j) {
            const int tb = wv * TBW + j;
            floatx4 s = sum[j][0];
#pragma unroll
            for (int o = 1; o < NW; ++o) s += sum[j][o];
            R[j] = tile_rows<E>(v[j], sel) - since[j] * s;
            put_half<E>(xf, tb, lane, bt[j] * R[j]);
        }
        floatx4 b_now[TBW];
#pragma unroll
        for (int j = 0; j < TBW; ++j) b_now[j] = bt[j];
        if (!KEEP)
#pragma unroll
            for (int tb = 0; tb < 4; ++tb) *reinterpret_cast<floatx4 *>(partq + ((wv * 4 + tb) * 64 + lane) * 4) = qs[tb];
        load_q();
        load_v(next);
        __builtin_amdgcn_sched_barrier(0);
        __syncthreads();
        frag_t<E> xh[2], xl[2];
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) get_split<E>(xf, kb, lane, xh[kb], xl[kb]);
#pragma unroll
        for (int j = 0; j < TBW; ++j) {
            const int tb = wv * TBW + j;
            floatx4 d = floatx4{0, 0, 0, 0};
            nf[j].product(d, 0, tb >> 1, xh, xl);
            R[j] -= d;   // U
            put_half<E>(uf, tb, lane, tillb[j] * R[j]);
            if (!KEEP) put_half<E>(wf, tb, lane, b_now[j] * R[j]);
        }
        __syncthreads();
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) get_split<E>(uf, kb, lane, xh[kb], xl[kb]);
#pragma unroll
        for (int nb = 0; nb < NBW; ++nb) S[nb] *= whole;
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
#pragma unroll
            for (int nb = 0; nb < NBW; ++nb) {
                mma(S[nb], ktf[nb][kb], xh[kb]);
                if (kPlanes<E> == 2) mma(S[nb], ktf[nb][kb], xl[kb]);
            }
        if (KEEP) {
#pragma unroll
            for (int j = 0; j < TBW; ++j)
                store_piece<E>((E *)a.ust + u * kPlanes<E> * kC * a.Pp, R[j], sel, wv * TBW + j, p0, lane);
            store_pieces<E>((E *)a.sst + u * kPlanes<E> * NT * a.Pp, so_.hi, so_.lo, sel, p0, lane, NB, NBW * wv);
        } else {
            const __amdgpu_buffer_rsrc_t rs = rows_of(a.y, i);
            frag_t<E> w[2], wl[2];
#pragma unroll
            for (int kb = 0; kb < 2; ++kb) get_split<E>(wf, kb, lane, w[kb], wl[kb]);
#pragma unroll
            for (int j = 0; j < TBW; ++j) {
                const int tb = wv * TBW + j;
                floatx4 s = vec4(partq + (tb * 64 + lane) * 4);   // (written again only after two meetings)
#pragma unroll
                for (int o = 1; o < NW; ++o) s += vec4(partq + ((o * 4 + tb) * 64 + lane) * 4);
                s *= scaled[j];
                pf[j].product(s, 0, tb >> 1, w, wl);
                tile_store<E>(rs, poff + (16 * tb + l) * ldb, s, sel);
            }
        }
        load_tri();
        load_rest();
        __builtin_amdgcn_sched_barrier(0);
    }
    save_state<NBW>(a.s1 ? a.s1 + so : nullptr, S, p0 + l, g, a.P, a.N, 16 * NBW * wv);
}

template <typename E, int NB>
__device__ __forceinline__ void narrow_bwd(const ChainArgs &a, int unit, char *smem)
{
    using C = Narrow<E, NB, 2>;
    constexpr int NT = 16 * NB, kMat = kC * NT, NW = C::NW, NBW = C::NBW, TBW = C::TBW, KBW = C::KBW, NK = C::NK;
    constexpr int kTriE = 512 * kTri;
    float *part = reinterpret_cast<float *>(smem);
    E *xf = reinterpret_cast<E *>(part + C::kPart), *uf = xf + 2 * C::kFrag;
    const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), g = lane >> 4, l = lane & 15;
    const int ptile = unit % a.np, h = (unit / a.np) % a.H;
    int ch = unit / (a.np * a.H);
    const int p0 = 16 * ptile;
    int c0, n, len;
    int64_t t0;
    chain_at(a.m, ch, c0, n, t0, len);
    const int64_t so = ((int64_t)ch * a.H + h) * a.P * a.N, ld = (int64_t)a.H * a.P;
    floatx4 D[NBW];
    load_state<E, NBW>(a.d1 ? a.d1 + so : nullptr, D, p0 + l, g, a.P, a.N, 16 * NBW * wv);
    const uint32_t ldb = (uint32_t)ld * sizeof(E), poff = p0 < a.P ? (p0 + 4 * g) * sizeof(E) : kOffNone;
    const int grp = h / (a.H / a.G);
    auto rows_of = [&](const void *base, int i) {
        const int left = len - i * kC;
        return rows_rsrc((const E *)base + ((t0 + i * kC) * a.H + h) * a.P, left < kC ? left : kC, ld, a.P);
    };
    Select<E> sel;
    sel.init(lane);
    frag_t<E> kf[4][KBW], ktf[NBW][2], qtf[NBW][2];
    TriRow<E> nf[TBW], pf[TBW];
    floatx4 till[TBW], bt[TBW], erase[TBW], scaled[4];
    Tile<E> dy;
    float whole;
    Blocks<E> kq, tri;
    __amdgpu_buffer_rsrc_t vec;
    auto at = [&](int i) {
        const int64_t u = (int64_t)(c0 + i) * a.H + h;
        kq.at((const E *)a.kq + ((int64_t)(c0 + i) * a.G + grp) * 4 * kMat, 4 * kMat, lane);
        tri.at((const E *)a.tri + u * tri_elems<E>(true), tri_elems<E>(true), lane);
        vec = make_rsrc_n(a.vec + u * kVec, kVec * 4);
    };
    auto scalars = [&](int which, int tb) {
        return __builtin_bit_cast(floatx4, bload16s(vec, 16 * g, __builtin_amdgcn_readfirstlane(4 * (which + 16 * tb))));
    };
    auto load_k = [&]() {
#pragma unroll
        for (int tb = 0; tb < 4; ++tb)
#pragma unroll
            for (int kb = 0; kb < KBW; ++kb) kf[tb][kb] = kq.get((tb * NK + wv * KBW + kb) * 512);
    };
    auto load_dy = [&](int i) {
        dy.load(rows_of(a.dy, i), ldb, poff, l);
#pragma unroll
        for (int j = 0; j < TBW; ++j) {
            const int tb = wv * TBW + j;
            till[j] = scalars(kTill, tb);
            pf[j].load(tri, 2 * kPlanes<E> * kTriE, tb >> 1, 1, [&](int kb) { return upper_block(tb, kb); });
        }
    };
    auto load_tri = [&]() {
#pragma unroll
        for (int j = 0; j < TBW; ++j) {
            const int tb = wv * TBW + j;
            nf[j].load(tri, kPlanes<E> * kTriE, tb >> 1, 1, [&](int kb) { return upper_block(tb, kb); });
            bt[j] = scalars(kBeta, tb);
            erase[j] = scalars(kErase, tb);
        }
    };
    auto load_rest = [&]() {
#pragma unroll
        for (int tb = 0; tb < 4; ++tb) scaled[tb] = scalars(kScaled, tb);
        whole = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(vec, 4 * (kSince + kC - 1), 0, 0));
#pragma unroll
        for (int nb = 0; nb < NBW; ++nb)
#pragma unroll
            for (int kb = 0; kb < 2; ++kb) {
                ktf[nb][kb] = kq.get(kMat + (2 * (wv * NBW + nb) + kb) * 512);
                qtf[nb][kb] = kq.get(3 * kMat + (2 * (wv * NBW + nb) + kb) * 512);
            }
    };
    if (n > 0) {
        at(n - 1);
        load_k();
        load_dy(n - 1);
        load_tri();
        load_rest();
    }
    for (int i = n - 1; i >= 0; --i) {
        const int64_t u = (int64_t)(c0 + i) * a.H + h;
        const int next = i > 0 ? i - 1 : 0;   // (as in the forward: no conditional loads)
        StateOps<E, NBW> dop;
        dop.of(D);
        floatx4 ks[4];
#pragma unroll
        for (int tb = 0; tb < 4; ++tb) ks[tb] = floatx4{0, 0, 0, 0};
#pragma unroll
        for (int kb = 0; kb < KBW; ++kb)
#pragma unroll
            for (int tb = 0; tb < 4; ++tb) {
                mma(ks[tb], kf[tb][kb], dop.hi[kb]);
                if (kPlanes<E> == 2) mma(ks[tb], kf[tb][kb], dop.lo[kb]);
            }
#pragma unroll
        for (int tb = 0; tb < 4; ++tb) *reinterpret_cast<floatx4 *>(part + ((wv * 4 + tb) * 64 + lane) * 4) = ks[tb];
        floatx4 yt[4];
        dy.rows(yt, sel);
        const frag_t<E> y01[2] = {round_pair<E>(yt[0], yt[1]), round_pair<E>(yt[2], yt[3])};   // exact
        floatx4 W[TBW];
#pragma unroll
        for (int j = 0; j < TBW; ++j) {
            const int tb = wv * TBW + j;
            W[j] = floatx4{0, 0, 0, 0};
#pragma unroll
            for (int kb = 0; kb < 2; ++kb)
                if (kb >= tb >> 1) {
                    mma(W[j], pf[j].hi[kb], y01[kb]);
                    if (kPlanes<E> == 2) mma(W[j], pf[j].lo[kb], y01[kb]);
                }
        }
#pragma unroll
        for (int tb = 0; tb < 4; ++tb) yt[tb] *= scaled[tb];
        frag_t<E> yh[2], yl[2];
        split_pair(yt[0], yt[1], yh[0], yl[0]);
        split_pair(yt[2], yt[3], yh[1], yl[1]);
        at(next);
        load_k();
        __builtin_amdgcn_sched_barrier(0);
        __syncthreads();
#pragma unroll
        for (int j = 0; j < TBW; ++j) {
            const int tb = wv * TBW + j;
            floatx4 s = vec4(part + (tb * 64 + lane) * 4);
#pragma unroll
            for (int o = 1; o < NW; ++o) s += vec4(part + ((o * 4 + tb) * 64 + lane) * 4);
            W[j] += till[j] * s;
            put_half<E>(xf, tb, lane, bt[j] * W[j]);
        }
        load_dy(next);
        __builtin_amdgcn_sched_barrier(0);
        __syncthreads();
        frag_t<E> xh[2], xl[2];
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) get_split<E>(xf, kb, lane, xh[kb], xl[kb]);
        floatx4 X[TBW];
#pragma unroll
        for (int j = 0; j < TBW; ++j) {
            const int tb = wv * TBW + j;
            floatx4 d = floatx4{0, 0, 0, 0};
            nf[j].product(d, tb >> 1, 1, xh, xl);
            W[j] -= d;              // H
            X[j] = bt[j] * W[j];    // dv
            put_half<E>(uf, tb, lane, erase[j] * W[j]);
        }
        load_tri();
        __builtin_amdgcn_sched_barrier(0);
        __syncthreads();
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) get_split<E>(uf, kb, lane, xh[kb], xl[kb]);
#pragma unroll
        for (int nb = 0; nb < NBW; ++nb) D[nb] *= whole;
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
#pragma unroll
            for (int nb = 0; nb < NBW; ++nb) {
                mma(D[nb], qtf[nb][kb], yh[kb]);
                if (kPlanes<E> == 2) mma(D[nb], qtf[nb][kb], yl[kb]);
                mma(D[nb], ktf[nb][kb], xh[kb]);
                if (kPlanes<E> == 2) mma(D[nb], ktf[nb][kb], xl[kb]);
            }
        load_rest();
        __builtin_amdgcn_sched_barrier(0);
        const __amdgpu_buffer_rsrc_t rs = rows_of(a.dv, i);
#pragma unroll
        for (int j = 0; j < TBW; ++j) {
            const int tb = wv * TBW + j;
            tile_store<E>(rs, poff + (16 * tb + l) * ldb, X[j], sel);
            store_piece<E>((E *)a.hst + u * kPlanes<E> * kC * a.Pp, W[j], sel, tb, p0, lane);
        }
        store_pieces<E>((E *)a.dst + u * kPlanes<E> * NT * a.Pp, dop.hi, dop.lo, sel, p0, lane, NB, NBW * wv);
    }
    save_state<NBW>(a.d0 ? a.d0 + so : nullptr, D, p0 + l, g, a.P, a.N, 16 * NBW * wv);
}

template <typename E, int NB, bool STAGED>
__global__ __launch_bounds__(kThreads, 2) void k_gdr_chain(ChainArgs a)
{
    __shared__ __attribute__((aligned(16))) char smem[Regions<E, NB, 0, STAGED>::kBytes];
    chain_fwd<E, NB, false, STAGED>(a, by_group(a, blockIdx.x), smem);
}
template <typename E, int NB>
__global__ __launch_bounds__(64 * kNW<NB>, 1) void k_gdr_chain_narrow(ChainArgs a)
{
    __shared__ __attribute__((aligned(16))) char smem[Narrow<E, NB, 0>::kBytes];
    // the workgroups of a head next to each other on one XCD share its triangles' lines
    // (16K tokens, N = 256: 547 against 578 us; the backward's two chains gain nothing)
    narrow_fwd<E, NB, false>(a, xcd_remap(blockIdx.x, a.units), smem);
}

// The backward's two chains in one launch: neither needs the other.
template <typename E, int NB, bool STAGED>
__global__ __launch_bounds__(kThreads, 2) void k_gdr_chains(ChainArgs a)
{
    __shared__ __attribute__((aligned(16))) char smem[Regions<E, NB, 2, STAGED>::kBytes];   // the larger of both
    if (blockIdx.x < (unsigned)a.units) chain_bwd<E, NB, STAGED>(a, by_group(a, blockIdx.x), smem);
    else chain_fwd<E, NB, true, STAGED>(a, by_group(a, blockIdx.x - a.units), smem);
}
template <typename E, int NB>
__global__ __launch_bounds__(64 * kNW<NB>, 1) void k_gdr_chains_narrow(ChainArgs a)
{
    __shared__ __attribute__((aligned(16))) char smem[Narrow<E, NB, 2>::kBytes];   // as large as KIND 1's
    if (blockIdx.x < (unsigned)a.units) narrow_bwd<E, NB>(a, by_group(a, blockIdx.x), smem);
    else narrow_fwd<E, NB, true>(a, by_group(a, blockIdx.x - a.units), smem);
}

// ---------------------------------------------------------------------------
// gradients of q, k, g and beta
// ---------------------------------------------------------------------------
// With W_ts = scale Gam_ts beta_s (dy_t . u_s) (s <= t) and Z_ts = Gam_ts beta_t
// beta_s (H_t . u_s) (s < t), per head
//   dq = scale e^{cs} o (dY S^T) + W K
//   dk = -e^{cs} beta o (H S^T) + e^{cs_last - cs} beta o (U D^T) + W^T Q - (Z + Z^T) K
//   dbeta_t = H_t . u_t
// and dq, dk are summed over the heads of the group, in order.  For dg_t every
// path from before t to at or after t counts once: with
//   X_ts = W_ts q_t.k_s - Z_ts k_t.k_s,
//   a_t = q_t . scale e^{cs_t} S dy_t - k_t . e^{cs_t} beta_t S H_t,
//   b_s = k_s . e^{cs_last - cs_s} beta_s D u_s,
//   dg_t = sum_{u >= t} (sum_s X_us - sum_s X_su + a_u - b_u) + sum_s b_s + e^{cs_last} <D, S>.
// The pairs on one side of t cancel, and do so to fp32 whatever U, H, S and D were
// rounded to, because both sums take the same X.  (q.dq - v.dv, the shorter form of
// the same sum, would need dq and dv far beyond bf16: 9e-3 against 2e-3 of dg.)
struct GradArgs {
    const void *kq, *k, *q, *dy, *sst, *ust, *dst, *hst;
    float *vec;                  // (written: kDgPass)
    void *dq, *dk, *dg, *dbeta;
    float *part;                 // hsplit > 1: fp32 sums of dq and dk per split
    Chunks m;
    int H, G, P, N, Pp, hsplit;
    float scale;
};

// One workgroup per (chunk, group, part of the group's heads), 8 waves: wave (tb, half)
// owns 16 tokens and half of the columns n of dq and dk, in registers over all heads.
// What a head brings (S, D, U, H and dy, 32 columns p at a time) comes into LDS as
// operand blocks without passing through registers, for the next stage while this one
// computes where LDS holds it twice (TWICE).  At N = 256 registers and LDS hold half of the
// columns n: a workgroup goes over its heads twice, forms the pair matrices again and adds
// up dg, whose terms are sums over n (in one pass it spilled 141 registers in bf16 and 196 in
// fp32: 16K tokens of 32 heads 2380 against 1535 us for the whole backward, fp32 of 2048
// tokens of 128 heads 2680 against 2240; 32 and 44 are left).
//
// 8 x 2048 tokens of 80 heads, N = 128: 690 us, 2.3 GB read at 3.4 TB/s.  What holds it is
// the chain inside a stage at two waves a SIMD (247 registers): waves wait a third of the
// time, the matrix pipe is busy 27 %.  (410 us, half the bytes, with single bf16 numbers; 900
// before half the waves formed W and the others Z; 70 more with a head's dg finished by one
// wave at its end and the next stage requested first.)
constexpr int kGradThreads = 512;
constexpr int kDgHeads = 4;   // heads whose dg is finished at a time
template <typename E, int NB> struct GradPlan {
    static constexpr int PL = kPlanes<E>;
    static constexpr int kPasses = NB == 16 ? 2 : 1, kRows = NB / kPasses;   // row blocks n of a pass
    static constexpr int kBlocks = (2 * kRows + 8) * PL + 4;              // of 32 columns: S | D | U | H | dy
    static constexpr int kRoom = kBlocks < 24 * PL ? 24 * PL : kBlocks;   // (at least what is exchanged below)
    static constexpr int kStage = kRoom * 512 * (int)sizeof(E);
    static constexpr int kMats = 2 * 2 * kRows * 512 * (int)sizeof(E);    // K^T and Q^T
    static constexpr int kDg = kDgHeads * (4 * kC + 17) * 4;              // dcs and red
    static constexpr int kLds = 160 * 1024;
    static constexpr bool TWICE = 2 * kStage + kMats + 2 * kVec * 4 + kDg <= kLds;
    static constexpr int kVecs = (TWICE ? 2 : 1) * kVec;
    static_assert((TWICE ? 2 : 1) * kStage + kMats + kVecs * 4 + kDg <= kLds, "a workgroup's LDS");
};

// acc + the sum of eight products (bf16: two per instruction, in fp32).
__device__ __forceinline__ float dot8(const bf16x8 &x, const bf16x8 &y, float acc)
{
#pragma unroll
    for (int i = 0; i < 8; i += 2)
        acc = __builtin_amdgcn_fdot2_f32_bf16(bf16x2{x[i], x[i + 1]}, bf16x2{y[i], y[i + 1]}, acc, false);
    return acc;
}
__device__ __forceinline__ float dot8(const floatx8 &x, const floatx8 &y, float acc)
{
#pragma unroll
    for (int i = 0; i < 8; ++i) acc += x[i] * y[i];
    return acc;
}
// The sum over a row of 16 lanes, in all of them.
__device__ __forceinline__ float row_sum16(float v)
{
    v += dpp_mov<kDppQuadXor1>(v);
    v += dpp_mov<kDppQuadXor2>(v);
    v += dpp_mov<kDppRowHalfMirror>(v);
    return v + dpp_mov<kDppRowRor8>(v);
}

// The sum over lanes l, l + 16, l + 32, l + 48, in all of them (row swaps: no LDS).
__device__ __forceinline__ float cross_sum4(float v)
{
    const int x = __float_as_int(v);
    const auto a = __builtin_amdgcn_permlane16_swap(x, x, false, false);
    const float s = __int_as_float(a[0]) + __int_as_float(a[1]);
    const int y = __float_as_int(s);
    const auto b = __builtin_amdgcn_permlane32_swap(y, y, false, false);
    return __int_as_float(b[0]) + __int_as_float(b[1]);
}
// Inclusive prefix sum over the wave: shifts by 1, 2, 4, 8 inside each row of 16, then the
// last lane of row 0 (2) to row 1 (3), and of row 1 to rows 2 and 3.
__device__ __forceinline__ float prefix_sum64(float v)
{
    auto add = [&](auto ctrl, auto rows) {
        v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), decltype(ctrl)::value, decltype(rows)::value, 0xf, false));
    };
    using std::integral_constant;
    add(integral_constant<int, 0x111>{}, integral_constant<int, 0xf>{});
    add(integral_constant<int, 0x112>{}, integral_constant<int, 0xf>{});
    add(integral_constant<int, 0x114>{}, integral_constant<int, 0xf>{});
    add(integral_constant<int, 0x118>{}, integral_constant<int, 0xf>{});
    add(integral_constant<int, 0x142>{}, integral_constant<int, 0xa>{});
    add(integral_constant<int, 0x143>{}, integral_constant<int, 0xc>{});
    return v;
}

template <typename E, int NB>
__global__ __launch_bounds__(kGradThreads, 2) void k_gdr_grad(GradArgs a)
{
    using Plan = GradPlan<E, NB>;
    constexpr int NT = 16 * NB, NK = NT / 32, kMat = kC * NT, PL = Plan::PL, NBP = Plan::kRows, HB = NBP / 2, V = kVec16<E>;
    constexpr int kHalf = kMat / Plan::kPasses;   // of K^T and Q^T, what a pass takes
    __shared__ __attribute__((aligned(16))) E stage_m[(Plan::TWICE ? 2 : 1) * Plan::kRoom * 512];
    __shared__ __attribute__((aligned(16))) E mats[2 * kHalf];
    __shared__ __attribute__((aligned(16))) float vs2[Plan::kVecs];
    __shared__ float dcs[kDgHeads][4][kC], red[kDgHeads][17];
    const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), g = lane >> 4, l = lane & 15;
    const int w = wv & 3, half = wv >> 2;
    int x = blockIdx.x;
    const int sp = x % a.hsplit;
    x /= a.hsplit;
    const int grp = x % a.G, c = x / a.G;
    int64_t t0;
    int count;
    chunk_at(a.m, c, t0, count);
    if (count <= 0) return;
    const int hpg = a.H / a.G;
    const int h0 = grp * hpg + (int)((int64_t)hpg * sp / a.hsplit), h1 = grp * hpg + (int)((int64_t)hpg * (sp + 1) / a.hsplit);
    const int NPC = a.Pp / 32, J = (h1 - h0) * NPC;
    const E *kf = (const E *)a.kq + ((int64_t)c * a.G + grp) * 4 * kMat;
    const E *ktg = kf + kMat, *qf = kf + 2 * kMat, *qtg = kf + 3 * kMat;
    const int64_t yld = (int64_t)a.H * a.P;

    // stage j: head h0 + j / NPC, columns 32 (j % NPC) ...
    int pass = 0;
    const int mine = wv * 64 * V + V * lane;
    auto run = [&](const E *src, E *dst, auto n) {   // n blocks, 1 KiB at a time from wave to wave
        constexpr int kParts = decltype(n)::value * 512 / (64 * V);
#pragma unroll
        for (int i = 0; i < kParts; i += 8)
            if (kParts % 8 == 0 || i + wv < kParts)
                __builtin_amdgcn_global_load_lds((gptr_t)(src + mine + i * 64 * V), (lptr_t)(dst + (i + wv) * 64 * V), 16, 0, kOnce);
    };
    auto issue = [&](int j) {
        const int hi = j / NPC, pc = j - hi * NPC, h = h0 + hi;
        const int64_t u = (int64_t)c * a.H + h;
        E *dst = stage_m + (Plan::TWICE ? (j & 1) : 0) * Plan::kRoom * 512;
        const int64_t so = (u * a.Pp + 32 * pc) * (PL * NT), uo = (u * a.Pp + 32 * pc) * (PL * kC);
        using BS = std::integral_constant<int, NBP * (Plan::kPasses == 1 ? PL : 1)>;
        using BU = std::integral_constant<int, 4 * PL>;
        for (int pl = 0; pl < (Plan::kPasses == 1 ? 1 : PL); ++pl) {   // (one pass: the planes lie one behind the other)
            const int from = (pl * NB + pass * NBP) * 512, to = pl * NBP * 512;
            run((const E *)a.sst + so + from, dst + to, BS{});
            run((const E *)a.dst + so + from, dst + NBP * PL * 512 + to, BS{});
        }
        dst += 2 * NBP * PL * 512;
        run((const E *)a.ust + uo, dst, BU{});
        run((const E *)a.hst + uo, dst + 4 * PL * 512, BU{});
        dst += 8 * PL * 512;
        // dy, a KiB per wave.  Rows past the count and columns past P: any element of the row's
        // own data (masked below; columns past P meet zeros of S, U and H)
        if (mine < 4 * 512) {
            const int e = mine % 512, t = 16 * (mine / 512) + (e >> 3) % 16, pp = 32 * pc + 8 * (e >> 7) + (e & 7);
            const E *dy = (const E *)a.dy + (t0 * a.H + h) * a.P;
            __builtin_amdgcn_global_load_lds((gptr_t)(dy + (int64_t)(t < count ? t : count - 1) * yld + (pp < a.P ? pp : 0)),
                                             (lptr_t)(dst + wv * 64 * V), 16, 0, 0);
        }
        if (pc == 0 && wv >= 4)
            __builtin_amdgcn_global_load_lds((gptr_t)(a.vec + u * kVec + 256 * (wv - 4) + 4 * lane),
                                             (lptr_t)(vs2 + (Plan::TWICE ? hi & 1 : 0) * kVec + 256 * (wv - 4)), 16, 0, 0);
    };
    auto issue_mats = [&]() {
        constexpr int n = 2 * kHalf * (int)sizeof(E) / 1024;   // K^T and Q^T, 1 KiB each
        static_assert(n % 16 == 0, "whole rounds");
#pragma unroll
        for (int i = 0; i < n / 8; ++i) {
            const int b = 8 * i + wv, e = b * 64 * V;
            const E *src = (e < kHalf ? ktg + e : qtg + (e - kHalf)) + pass * kHalf;
            __builtin_amdgcn_global_load_lds((gptr_t)(src + V * lane), (lptr_t)(mats + e), 16, 0, 0);
        }
    };
    if (Plan::TWICE) issue(0);
    issue_mats();
    const E *ktf = mats + 8 * lane, *qtf = mats + kHalf + 8 * lane;

    // The pair matrices of the wave's 16 tokens (half 0: W, half 1: Z): block i holds rows of
    // block i against columns of block w, as (s, t) pairs where i <= w and as (t, s) pairs
    // where i > w; the diagonal block is needed both ways (mD: as (t, s)).  kq: q.k or k.k
    // of the same pairs.
    floatx4 kq[4], kqD = floatx4{0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i) kq[i] = floatx4{0, 0, 0, 0};
    {
        const E *xf = half ? kf : qf;   // what stands for t
        // (where from is selected, not branched on, so that the loads go out together)
#pragma unroll 2
        for (int kb = 0; kb < NK; ++kb) {
            const frag_t<E> kw = load_frag(kf + (w * NK + kb) * 512 + 8 * lane), xw = load_frag(xf + (w * NK + kb) * 512 + 8 * lane);
            frag_t<E> f[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) f[i] = load_frag((i <= w ? kf : xf) + (i * NK + kb) * 512 + 8 * lane);
            mma(kqD, xw, kw);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i <= w) mma(kq[i], f[i], xw);
                else mma(kq[i], f[i], kw);
        }
    }
    // the wave's q and k in accumulator layout: token 16 w + 4 g + r, column 16 nb + l
    // (packed in pairs, for the registers)
    constexpr int QW = sizeof(E) == 2 ? 2 : 4;
    uint32_t qe[HB][QW], ke[HB][QW];
    const int64_t kq0 = (t0 * a.G + grp) * a.N;
    const uint32_t kqld = (uint32_t)(a.G * a.N) * sizeof(E);
    const __amdgpu_buffer_rsrc_t qrs = rows_rsrc((const E *)a.q + kq0, count, (int64_t)a.G * a.N, a.N);
    const __amdgpu_buffer_rsrc_t krs = rows_rsrc((const E *)a.k + kq0, count, (int64_t)a.G * a.N, a.N);
    floatx4 dq[HB], dk[HB];
    floatx4 m[4], mD, aq, ak, bk;
    float db = 0.f, sd = 0.f;
    const int tl0 = 16 * w + l;
    // N = 256: one pass over the heads for each half of the columns n (their registers and LDS
    // are those of N = 128; the pair matrices are formed twice)
    for (; pass < Plan::kPasses; ++pass) {
        if (pass) {
            __syncthreads();   // the last pass has read its operands
            if (Plan::TWICE) issue(0);
            issue_mats();
        }
#pragma unroll
        for (int nb = 0; nb < HB; ++nb)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int t = 16 * w + 4 * g + r, n = 16 * (pass * NBP + half * HB + nb) + l;
                const uint32_t off = n < a.N ? t * kqld + n * sizeof(E) : kOffNone;
                if constexpr (sizeof(E) == 2) {
                    const uint32_t qv = __builtin_bit_cast(unsigned short, bload_elem<E>(qrs, off));
                    const uint32_t kv = __builtin_bit_cast(unsigned short, bload_elem<E>(krs, off));
                    qe[nb][r / 2] = r % 2 ? qe[nb][r / 2] | qv << 16 : qv;
                    ke[nb][r / 2] = r % 2 ? ke[nb][r / 2] | kv << 16 : kv;
                } else {
                    qe[nb][r] = __builtin_bit_cast(uint32_t, bload_elem<E>(qrs, off));
                    ke[nb][r] = __builtin_bit_cast(uint32_t, bload_elem<E>(krs, off));
                }
            }
#pragma unroll
        for (int nb = 0; nb < HB; ++nb) dq[nb] = dk[nb] = floatx4{0, 0, 0, 0};

        for (int j = 0; j < J; ++j) {
            const int h = h0 + j / NPC, pc = j % NPC;
            if (!Plan::TWICE) {
                __syncthreads();
                issue(j);
            }
            loads_done();
            __syncthreads();
            E *room = stage_m + (Plan::TWICE ? (j & 1) : 0) * Plan::kRoom * 512;
            const E *buf = room + 8 * lane;
            const E *Sb = buf, *Db = buf + NBP * PL * 512, *Ub = buf + 2 * NBP * PL * 512, *Hb = Ub + 4 * PL * 512,
                    *Yb = Hb + 4 * PL * 512, *Xb = half ? Hb : Yb;
            const float *vs = vs2 + (Plan::TWICE ? (h - h0) & 1 : 0) * kVec;
            if (pc == 0) {
#pragma unroll
                for (int i = 0; i < 4; ++i) m[i] = floatx4{0, 0, 0, 0};
                mD = aq = ak = bk = floatx4{0, 0, 0, 0};
                db = sd = 0.f;
            }
            // (a second plane's products are those that hi and lo of both factors give, without lo
            // lo; dy is exact in one)
            frag_t<E> uw[PL], hw[PL];
            const frag_t<E> yw = load_frag(Yb + w * 512), xw = load_frag(Xb + w * 512);
#pragma unroll
            for (int pl = 0; pl < PL; ++pl) {
                uw[pl] = load_frag(Ub + (4 * pl + w) * 512);
                hw[pl] = load_frag(Hb + (4 * pl + w) * 512);
            }
            {
                frag_t<E> f[4], fl[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) f[i] = load_frag((i <= w ? Ub : Xb) + i * 512);
                if (PL == 2)
#pragma unroll
                    for (int i = 0; i < 4; ++i) fl[i] = load_frag((i <= w ? Ub : Hb) + (4 + i) * 512);
                if (half) db = dot8(uw[0], hw[0], db);
                mma(mD, xw, uw[0]);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (i <= w) mma(m[i], f[i], xw);
                    else mma(m[i], f[i], uw[0]);
                if (PL == 2) {
                    mma(mD, xw, uw[PL - 1]);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (i <= w) mma(m[i], fl[i], xw);
                        else mma(m[i], f[i], uw[PL - 1]);
                    if (half) {
                        db = dot8(uw[0], hw[PL - 1], dot8(uw[PL - 1], hw[0], db));
                        mma(mD, hw[PL - 1], uw[0]);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (i <= w) mma(m[i], f[i], hw[PL - 1]);
                            else mma(m[i], fl[i], uw[0]);
                    }
                }
            }
            // (requested here and not at the head of the stage, where the compiler has the first LDS
            // read wait for it; the exchange below waits for it in any case)
            if (Plan::TWICE && j + 1 < J) issue(j + 1);
            // the state products
            {
                const floatx4 cq = vec4(vs + kScaled + 16 * w + 4 * g), cd = vec4(vs + kTillBeta + 16 * w + 4 * g),
                              ch = vec4(vs + kErase + 16 * w + 4 * g);
#pragma unroll
                for (int nb = 0; nb < HB; ++nb) {
                    floatx4 ys = floatx4{0, 0, 0, 0}, hs = ys, ud = ys;
                    frag_t<E> sf[PL], df[PL];
#pragma unroll
                    for (int pl = 0; pl < PL; ++pl) {
                        sf[pl] = load_frag(Sb + (pl * NBP + half * HB + nb) * 512);
                        df[pl] = load_frag(Db + (pl * NBP + half * HB + nb) * 512);
                    }
                    mma(ys, yw, sf[0]);
                    mma(hs, hw[0], sf[0]);
                    mma(ud, uw[0], df[0]);
                    if (PL == 2) {
                        mma(ys, yw, sf[PL - 1]);
                        mma(hs, hw[0], sf[PL - 1]);
                        mma(ud, uw[0], df[PL - 1]);
                        mma(hs, hw[PL - 1], sf[0]);
                        mma(ud, uw[PL - 1], df[0]);
                    }
                    if ((nb & 3) == w) {
                        sd = dot8(sf[0], df[0], sd);
                        if (PL == 2) sd = dot8(sf[0], df[PL - 1], dot8(sf[PL - 1], df[0], sd));
                    }
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        uint32_t qw = qe[nb][r * QW / 4], kw = ke[nb][r * QW / 4];
                        asm volatile("" : "+v"(qw), "+v"(kw));   // (unpacked here, not kept unpacked)
                        if (QW == 2) {
                            qw = r % 2 ? qw & 0xffff0000u : qw << 16;
                            kw = r % 2 ? kw & 0xffff0000u : kw << 16;
                        }
                        aq[r] += __uint_as_float(qw) * ys[r];
                        ak[r] += __uint_as_float(kw) * hs[r];
                        bk[r] += __uint_as_float(kw) * ud[r];
                        dq[nb][r] += cq[r] * ys[r];
                        dk[nb][r] += cd[r] * ud[r];
                        dk[nb][r] += ch[r] * hs[r];
                    }
                }
            }
            if (pc != NPC - 1) continue;
            // the head's pair matrix and its part of dg.  Rows past the count hold data of the last
            // row; their factors are zero.
            // (sums over s and over t apart, so that what cancels does so exactly)
            float dx = 0.f, dx_s = 0.f;
            // (opaque, so that the comparisons below are made here and not kept in registers)
            int tl = tl0, o0 = 4 * g;
            asm volatile("" : "+v"(tl), "+v"(o0));
            const float *row = vs + (half ? kRowBeta : kRowScale);
            // the factors of every block first, then the branches, so that the reads go out together
            floatx4 fo[4];   // of o: before t (i < w), or t itself
            float fl[4];     // of tl: t itself, or before t
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                fo[i] = vec4((i < w ? vs + kColBeta + (w - 1) * kC : row) + 16 * i + o0);
                fl[i] = (i < w ? row : vs + kColBeta + (i - 1) * kC)[tl];
            }
            const float chi = vs[kCsHi + tl], clo = vs[kCsLo + tl], bl = vs[kBeta + tl];
            const floatx4 oh = vec4(vs + kCsHi + 16 * w + o0), ol = vec4(vs + kCsLo + 16 * w + o0),
                          bo = vec4(vs + kBeta + 16 * w + o0);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i != w) {   // t = tl, s = o (i < w); t = o, s = tl
                    m[i] *= fl[i] * fo[i];
                    float d = 0.f;
#pragma unroll
                    for (int r = 0; r < 4; ++r) d += m[i][r] * kq[i][r];
                    dx += i < w ? d : 0.f;
                    dx_s += i < w ? 0.f : d;
                } else {
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int o = 16 * i + o0 + r;
                        const float d = ((chi - oh[r]) + (clo - ol[r])) * kLog2e;
                        const bool down = half ? o < tl : o <= tl, up = half ? tl < o : tl <= o;
                        const float f = exp2_(down ? d : 0.f) * bo[r] * (half ? bl : a.scale);
                        m[i][r] = down && tl < count ? f * m[i][r] : 0.f;
                        const float fD = exp2_(up ? -d : 0.f) * bl * (half ? bo[r] : a.scale);
                        mD[r] = up && o < count ? fD * mD[r] : 0.f;
                        dx += m[i][r] * kq[i][r];
                        dx_s += mD[r] * kqD[r];
                    }
                }
            dx = pass ? 0.f : dx - dx_s;   // (no columns n in it: counted once)
            // its operands change hands through what this stage no longer needs
            __syncthreads();
            {
                const floatx4 none = floatx4{0, 0, 0, 0};
                E *mine = room + w * 6 * PL * 512 + 8 * lane;   // W up | W down | Z, two blocks each, in their planes
                auto give = [&](int k, const floatx4 &x, const floatx4 &y) {
                    frag_t<E> hi, lo;
                    split_pair(x, y, hi, lo);
                    store_frag(mine + k * PL * 512, hi);
                    if (PL == 2) store_frag(mine + (k * PL + 1) * 512, lo);
                };
                if (half == 0) {
                    floatx4 up[4], dn[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        up[i] = i <= w ? m[i] : none;
                        dn[i] = i < w ? none : i == w ? mD : m[i];
                    }
                    give(0, up[0], up[1]);
                    give(1, up[2], up[3]);
                    give(2, dn[0], dn[1]);
                    give(3, dn[2], dn[3]);
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) m[i] = i == w ? -m[i] - mD : -m[i];
                    give(4, m[0], m[1]);
                    give(5, m[2], m[3]);
                    dx = -dx;
                }
            }
            // dg and dbeta
            floatx4 ab;
            float sb = 0.f;
            {
                const floatx4 cq = vec4(vs + kScaled + 16 * w + 4 * g), cd = vec4(vs + kTillBeta + 16 * w + 4 * g),
                              ch = vec4(vs + kErase + 16 * w + 4 * g);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const bool in = 16 * w + 4 * g + r < count;
                    const float b = cd[r] * bk[r];
                    sb += b;
                    ab[r] = in ? row_sum16(cq[r] * aq[r] + ch[r] * ak[r] - b) : 0.f;
                }
            }
            sb = cross_sum4(row_sum16(sb));
            sd = cross_sum4(row_sum16(sd));
            dx = cross_sum4(dx);
            if (half) {
                db = cross_sum4(db);
                if (g == 0 && tl < count && pass == 0) ((E *)a.dbeta)[(t0 + tl) * a.H + h] = from_float<E>(db);
            }
            const int slot = (h - h0) % kDgHeads;
            if (g == 0) dcs[slot][2 + half][tl] = dx;
            if (l == 0)
#pragma unroll
                for (int r = 0; r < 4; ++r) dcs[slot][half][16 * w + 4 * g + r] = ab[r];
            if (lane == 0) {
                red[slot][wv] = sb;
                red[slot][8 + wv] = sd;
                if (wv == 0) red[slot][16] = vs[kSince + kC - 1];
            }
            __syncthreads();
            // W K, W^T Q and (Z + Z^T) K
            {
                const E *theirs = room + w * 6 * PL * 512 + 8 * lane;
                frag_t<E> x[6][PL];
#pragma unroll
                for (int k = 0; k < 6; ++k)
#pragma unroll
                    for (int pl = 0; pl < PL; ++pl) x[k][pl] = load_frag(theirs + (k * PL + pl) * 512);
#pragma unroll
                for (int nb = 0; nb < HB; ++nb) {
                    const E *kt = ktf + 2 * (half * HB + nb) * 512, *qt = qtf + 2 * (half * HB + nb) * 512;
                    const frag_t<E> k0 = load_frag(kt), k1 = load_frag(kt + 512), q0 = load_frag(qt), q1 = load_frag(qt + 512);
#pragma unroll
                    for (int pl = 0; pl < PL; ++pl) {
                        mma(dq[nb], x[0][pl], k0);
                        mma(dk[nb], x[2][pl], q0);
                        mma(dq[nb], x[1][pl], k1);
                        mma(dk[nb], x[4][pl], k0);
                        mma(dk[nb], x[3][pl], q1);
                        mma(dk[nb], x[5][pl], k1);
                    }
                }
            }
            // dg of several heads at a time, a wave each: once per head it would hold the other
            // waves up
            if ((slot == kDgHeads - 1 || h == h1 - 1) && wv <= slot) {
                const int t = 63 - lane;
                const float(&d)[4][kC] = dcs[wv];
                const float *rd = red[wv];
                float s = prefix_sum64(d[0][t] + d[1][t] + d[2][t] + d[3][t]), sum_b = 0.f, sum_sd = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    sum_b += rd[i];
                    sum_sd += rd[8 + i];
                }
                s += sum_b + rd[16] * sum_sd;
                const int hw = h - slot + wv;
                if (t < count) {   // (the same lane in every pass)
                    float *before = a.vec + ((int64_t)c * a.H + hw) * kVec + kDgPass + t;
                    if (pass) s += *before;
                    if (pass + 1 < Plan::kPasses) *before = s;
                    else ((E *)a.dg)[(t0 + t) * a.H + hw] = from_float<E>(s);
                }
            }
        }
#pragma unroll
        for (int nb = 0; nb < HB; ++nb)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int t = 16 * w + 4 * g + r, n = 16 * (pass * NBP + half * HB + nb) + l;
                if (a.hsplit > 1) {
                    float *o = a.part + (((int64_t)c * a.G + grp) * a.hsplit + sp) * 2 * kMat + (int64_t)t * NT + n;
                    o[0] = dq[nb][r];
                    o[kMat] = dk[nb][r];
                } else if (t < count && n < a.N) {
                    const int64_t at = ((t0 + t) * a.G + grp) * a.N + n;
                    ((E *)a.dq)[at] = from_float<E>(dq[nb][r]);
                    ((E *)a.dk)[at] = from_float<E>(dk[nb][r]);
                }
            }
    }
}

// dq and dk of one chunk and group from their parts, added in order of the split.  Many
// small workgroups, each a strip of the block: 13 us where one per block took 34.
template <typename E, int NT>
__global__ __launch_bounds__(kThreads) void k_gdr_grad_sum(const float *__restrict__ part, E *__restrict__ dq,
                                                           E *__restrict__ dk, Chunks m, int G, int N, int hsplit)
{
    constexpr int kMat = kC * NT;
    const int c = blockIdx.x / G, grp = blockIdx.x % G;
    int64_t t0;
    int count;
    chunk_at(m, c, t0, count);
    const float *p = part + ((int64_t)c * G + grp) * hsplit * 2 * kMat;
    for (int i = blockIdx.y * kThreads + threadIdx.x; i < 2 * kMat / 4; i += gridDim.y * kThreads) {
        const int which = i / (kMat / 4), e = 4 * (i % (kMat / 4)), t = e / NT, n = e % NT;
        if (t >= count || n >= N) continue;
        floatx4 s = floatx4{0, 0, 0, 0};
        for (int k = 0; k < hsplit; ++k) s += vec4(p + (int64_t)(2 * k + which) * kMat + e);
        store_round4((which ? dk : dq) + ((t0 + t) * G + grp) * N + n, s);
    }
}

// ---------------------------------------------------------------------------
// one token
// ---------------------------------------------------------------------------
// One step of the recurrence for every (batch row, head), the state [P][N] in
// fp32, read and written once.  NL lanes share a row of the state (four
// consecutive n each, 16-byte accesses); the two sums over n (with k before the
// update, with q after it) are reduced inside those lanes.  Bound by the state's
// bytes, like any step of a recurrence.  The state goes past the caches (non-temporal): it
// comes back only after all the other layers' states.  64 sequences of 80 heads of 64 x 128,
// 337 MB, of which a copy's rate makes 66 us: 65 us between events with other data in the
// caches (with ordinary accesses 81, with 4 rows a thread 67), 58 us with its own in the last
// level (55).
constexpr int kStepRows = 2;   // rows in flight per thread
template <typename E, int NL>
__global__ __launch_bounds__(kThreads) void k_gdr_step(const E *__restrict__ q, const E *__restrict__ k,
                                                       const E *__restrict__ v, const E *__restrict__ gate,
                                                       const E *__restrict__ beta, float *__restrict__ state,
                                                       E *__restrict__ y, int H, int G, int P, int N, float scale)
{
    const int bh = blockIdx.x, b = bh / H, h = bh - b * H, grp = h / (H / G);
    const int ln = threadIdx.x % NL, row = threadIdx.x / NL, n = 4 * ln;
    constexpr int RPB = kThreads / NL;
    const bool in = n < N;
    const int64_t kq = ((int64_t)b * G + grp) * N + n;
    float kv[4] = {0, 0, 0, 0}, qv[4] = {0, 0, 0, 0};
    const int p0 = blockIdx.y * RPB * kStepRows + row;
    float *st = state + (int64_t)bh * P * N;
    floatx4 s[kStepRows];
#pragma unroll
    for (int i = 0; i < kStepRows; ++i) {
        const int p = p0 + i * RPB;
        s[i] = floatx4{0, 0, 0, 0};
        if (in && p < P) s[i] = __builtin_nontemporal_load(reinterpret_cast<const floatx4 *>(st + (int64_t)p * N + n));
    }
    if (in) {
        load4_f32(k + kq, kv);
        load4_f32(q + kq, qv);
    }
    float gv = to_float(gate[bh]);
    gv = gv < kMinLogDecay ? kMinLogDecay : gv;
    const float al = exp2_(gv * kLog2e), bt = to_float(beta[bh]);
#pragma unroll
    for (int i = 0; i < kStepRows; ++i) {
        const int p = p0 + i * RPB;
        s[i] *= al;
        float d = s[i][0] * kv[0] + s[i][1] * kv[1] + s[i][2] * kv[2] + s[i][3] * kv[3];
#pragma unroll
        for (int o = 1; o < NL; o <<= 1) d += __shfl_xor(d, o);
        const float u = p < P ? bt * (to_float(v[(int64_t)bh * P + p]) - d) : 0.f;
        float o = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            s[i][e] += u * kv[e];
            o += s[i][e] * qv[e];
        }
#pragma unroll
        for (int x = 1; x < NL; x <<= 1) o += __shfl_xor(o, x);
        if (p < P) {
            if (in) __builtin_nontemporal_store(s[i], reinterpret_cast<floatx4 *>(st + (int64_t)p * N + n));
            if (ln == 0) y[(int64_t)bh * P + p] = from_float<E>(scale * o);
        }
    }
}

// final_states = initial_states (or zero): no tokens.
__global__ __launch_bounds__(kThreads) void k_gdr_copy(float *__restrict__ dst, const float *__restrict__ src, int64_t n)
{
    for (int64_t i = ((int64_t)blockIdx.x * kThreads + threadIdx.x) * 4; i < n; i += (int64_t)gridDim.x * kThreads * 4)
        *reinterpret_cast<floatx4 *>(dst + i) = src ? vec4(src + i) : floatx4{0, 0, 0, 0};
}

}  // namespace gdr
}  // namespace ssd
