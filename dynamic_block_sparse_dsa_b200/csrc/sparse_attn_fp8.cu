// sparse_attn_fp8.cu -- exact attention over the selected blocks of the 8-bit
// (E4M3) cache.
//
// "Day-0 Adaptation for Massive LLMs: Overcoming Sparse Attention and MXFP4
// Expert Weights", section 4(3): gather the selected blocks by their ids and
// attend under a valid mask.  The 8-bit storage has no counterpart there.
//
// Per 64-token tile of a selected block, with E4M3 codes K, V, the tile's fp32
// scales s_k, s_v and the query heads Q of the KV head:
//     S^T = (s_k * scale) * (K Q^T),  P = 2^(S - m),  O^T += s_v * (V^T P^T)
// The products run as mma.m16n8k16 f16 with fp32 accumulation (keys or dims are
// the M dimension, the <= 8 or 16 heads N):
//   * an E4M3 code is exact in f16, so K and V lose nothing in the conversion
//     (one cvt per two codes);
//   * a query row is multiplied by the power of two that brings its largest
//     entry into [2^14, 2^15): its bf16 significands then fit f16 exactly down
//     to 2^-31 of that entry, and below that are off by at most 2^-39 of it --
//     far under the fp32 accumulation's own rounding;
//   * P is in [0, 1] and rounds to f16 (half a step: 2^-11 relative, 2^-25
//     absolute below 2^-14); the softmax sum is taken in fp32 before that.
// The e4m3 form of mma.sync would take the codes as they are, with the other
// operand as a sum of two codes; measured, it is slower (4.52 against 3.16 ms
// for the 4096-query chunk, at that state of the rest): 16.5 tensor cycles per
// m16n8k32 and 1,200 instructions a tile, as if every operand were converted for
// every product.
//
// The 8-bit operands reach the fragments without byte shuffles of K: an
// ldmatrix lane holds four neighbouring dims of one token, which serve as the
// k indexes (2c, 2c+1) and (2c+8, 2c+9) of one mma when the query fragments are
// laid out the same way.  For V the transposing 8-bit ldmatrix gives a lane four
// rows of one column; the rows' addresses are permuted so that these are the
// tokens 2c, 2c+1, 2c+8 and 2c+9 of the column's dim, again the k indexes of one
// mma (of the weights as the 16-bit transpose leaves them).
//
// Feeding.  Every warp is its own producer: it holds kSlots 8-KiB slots, one
// for K tiles and one for V tiles, and issues the TMA box of its next tile as
// soon as it has read a slot.  Nothing is handed from warp to warp, so a tile
// costs no queue words, fences or polls.  (A producer warp for the whole CTA,
// as over the bf16 cache, needed about 600 cycles a tile here, with no
// arithmetic at all: 4.4 of 5.5 ms of the 4096-query chunk.)
//
// Work.  With P (query, KV head) pairs and W warps on the GPU, floor(P / W)
// rounds give each warp a pair of its own, which it writes out by itself; the
// pairs go KV-head-major, so that all warps read one KV head's slice of the
// pool at a time and the queries that select the same block find it in L2.
// The pairs left over (all of a decode batch) go to teams of several warps of
// one CTA, the largest that still leave a team for every pair: a team's warps
// take the pair's tiles in turn and merge their softmax states through shared
// memory.  With less than half as many pairs as CTAs, the tiles of a pair are
// split over several CTAs; their states meet in the workspace, and the CTA that
// completes the pair's count merges them (nobody waits).
// All waits are bounded (DSA_DEV_ERR_WAIT on timeout, no hang).
//
// Bounds (one B200).  The 4096-query chunk (2.1 M tiles, 34 GB gathered from L2)
// takes 2.40 ms: 680 instructions a tile, of them 256 conversions at two cycles
// each, keep the ALU pipe 55 % and the tensor pipe 41 % busy; the gather alone
// takes 1.67 ms (20 TB/s).  Decode reads its tiles once: 64 contexts of 8K, 135
// MB, take 26.6 us (5.1 TB/s, 0.78 of the copy bandwidth) and 25.1 us without the
// arithmetic.
#include "dsa_kernels.h"
#include "dsa_tma.cuh"

#include <cuda_fp16.h>

#include <atomic>

namespace dsa {

namespace {

constexpr int kTileBytes = kBlockSize * kHeadDim;   // 8 KiB: 64 rows x 128 codes
constexpr int kSlots = 2;                           // per warp: a K tile and a V tile
constexpr int kRingBytes = kSlots * kTileBytes;
constexpr int kMergeStride = 132;                   // floats per merge row (padded against bank conflicts)
constexpr int kMaxSmemSeqs = 256;                   // cu_q entries cached in shared memory
constexpr float kLn2 = 0.6931471805599453f;

// shared memory: the rings (a warp's ring takes its state in the merge, when its
// last tile is read), then the rest
struct Plan {
    int ml, cuq, bars, words, bytes;
    __host__ __device__ constexpr explicit Plan(int warps)
        : ml(warps * kRingBytes),                              // [warp][16] (m, l)
          cuq(ml + warps * 16 * 8),
          bars((cuq + (kMaxSmemSeqs + 1) * 4 + 7) / 8 * 8),
          words(bars + warps * kSlots * 8),                    // never, last, end of the queries
          bytes(words + 12 + 1024) {}                          // + base alignment slack
};
static_assert(Plan(kFp8ManyWarps).bytes <= 227 * 1024, "shared memory");
static_assert(16 * kMergeStride * 4 <= kRingBytes, "a warp's state fits its ring");

using unit_t = uint32_t;

// D(16x8 f32) += A(16x16 f16, row) * B(16x8 f16, col)
__device__ __forceinline__ void mma_f16_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// two 16x16 byte matrices, transposed: lane (g, c) gets bytes of rows 4c .. 4c+3
// of column g (r0; r2 of the second matrix) and of column g + 8 (r1; r3).  Lane
// i gives the address of row i (16 + i: the second matrix).
__device__ __forceinline__ void ldmatrix_b8_x2_trans(uint32_t addr, uint32_t &r0, uint32_t &r1, uint32_t &r2,
                                                     uint32_t &r3) {
    asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0,%1,%2,%3}, [%4];\n"
                 : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
                 : "r"(addr));
}

// four E4M3 codes -> two pairs of f16 (exact)
__device__ __forceinline__ void codes_to_f16(uint32_t w, uint32_t &lo, uint32_t &hi) {
    asm("{\n\t.reg .b16 l, h;\n\t"
        "mov.b32 {l, h}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, l;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// 2^x; results below 2^-126 become 0 (-inf gives 0)
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// the larger of two, NaN if either is
__device__ __forceinline__ float max_nan(float x, float y) {
    float z;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(z) : "f"(x), "f"(y));
    return z;
}

__device__ __forceinline__ float max3_nan(float x, float y, float z) {
    float w;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(w) : "f"(x), "f"(y), "f"(z));
    return w;
}

// natural log-sum-exp from a base-2 maximum and sum; -inf for an empty row, NaN kept
__device__ __forceinline__ float lse_of(float m, float l) {
    return !(l <= 0.f) ? (m + log2f(l)) * kLn2 : -INFINITY;
}
// 1 / l; 0 for an empty row (its O is 0), NaN kept
__device__ __forceinline__ float inv_of(float l) { return !(l <= 0.f) ? 1.f / l : 0.f; }

// B fragments of the query heads (8 nt + g), scaled to f16: step kk covers dims
// 16 kk .. 16 kk + 15, this lane's 16 kk + 4 cq .. + 3.  mul[nt][h]: from an
// accumulator of head 8 nt + 2 cq + h to base-2 logits.
template <int NT>
__device__ __forceinline__ void load_queries(const __nv_bfloat16 *q, int group, float scale_log2,
                                             uint32_t (&qb)[8][NT][2], float (&mul)[NT][2]) {
    const int lane = threadIdx.x & 31, g = lane >> 2, cq = lane & 3;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        int w[8][2];
        const bool in = 8 * nt + g < group;
        const int *row = reinterpret_cast<const int *>(q + (size_t)(in ? 8 * nt + g : 0) * kHeadDim) + 2 * cq;
#pragma unroll
        for (int k = 0; k < 8; ++k) {   // 16 dims each
            w[k][0] = w[k][1] = 0;
            if (in)   // the rows may come from the append just before: kept behind the wait
                asm volatile("ld.global.v2.b32 {%0, %1}, [%2];" : "=r"(w[k][0]), "=r"(w[k][1]) : "l"(row + 8 * k));
        }
        float top = 0.f;
        bool odd = false;   // a NaN or an infinity in the row
#pragma unroll
        for (int k = 0; k < 8; ++k)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float x = fabsf(__uint_as_float((uint32_t)w[k][i] << 16));
                const float y = fabsf(__uint_as_float((uint32_t)w[k][i] & 0xffff0000u));
                top = fmaxf(top, fmaxf(x, y));
                odd |= !(x <= 3.4e38f) || !(y <= 3.4e38f);
            }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // top = 2^(e - 127) * [1, 2): times 2^(14 - (e - 127)); a row below 2^-99
        // takes the largest factor (both factors stay normal numbers)
        const int e = max((int)(__float_as_uint(top) >> 23), 28);
        const float up = __uint_as_float((uint32_t)(268 - e) << 23);
        const float down = __uint_as_float((uint32_t)(e - 14) << 23);
#pragma unroll
        for (int k = 0; k < 8; ++k)
#pragma unroll
            for (int i = 0; i < 2; ++i)
                qb[k][nt][i] = pack_f16x2(__uint_as_float((uint32_t)w[k][i] << 16) * up,
                                          __uint_as_float((uint32_t)w[k][i] & 0xffff0000u) * up);
        // a NaN or an infinity in the query makes the row's result NaN
        odd |= __shfl_xor_sync(0xffffffffu, (int)odd, 1) != 0;
        odd |= __shfl_xor_sync(0xffffffffu, (int)odd, 2) != 0;
        const float m = odd ? __uint_as_float(0x7fc00000u) : scale_log2 * down;
        mul[nt][0] = __shfl_sync(0xffffffffu, m, 8 * cq);       // the lane with g = 2 cq
        mul[nt][1] = __shfl_sync(0xffffffffu, m, 8 * cq + 4);   // g = 2 cq + 1
    }
}

// A warp's running state for one pair: O^T accumulators of dims 16 dm + g (+8) x
// heads 8 nt + 2 cq (+1), and per head the maximum and this lane's part of the sum
template <int NT>
struct State {
    float o[8][NT][4], m[NT][2], l[NT][2];
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            m[nt][0] = m[nt][1] = -INFINITY;
            l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
            for (int dm = 0; dm < 8; ++dm) o[dm][nt][0] = o[dm][nt][1] = o[dm][nt][2] = o[dm][nt][3] = 0.f;
        }
    }
    __device__ __forceinline__ void sum_lanes() {   // l over the token rows g
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                l[nt][h] += __shfl_xor_sync(0xffffffffu, l[nt][h], 4);
                l[nt][h] += __shfl_xor_sync(0xffffffffu, l[nt][h], 8);
                l[nt][h] += __shfl_xor_sync(0xffffffffu, l[nt][h], 16);
            }
    }
};

// S^T of one K tile (swizzled 64 x 128 bytes): raw accumulators
template <int NT>
__device__ __forceinline__ void scores(uint32_t tk, const uint32_t (&qb)[8][NT][2], float (&sc)[4][NT][4]) {
    const int lane = threadIdx.x & 31;
    const int lr = lane & 15, lc = lane >> 4;   // ldmatrix row and chunk of this lane
#pragma unroll
    for (int mt = 0; mt < 4; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) sc[mt][nt][0] = sc[mt][nt][1] = sc[mt][nt][2] = sc[mt][nt][3] = 0.f;
#pragma unroll
    for (int kp = 0; kp < 4; ++kp)   // 32 dims: two k-steps per ldmatrix
#pragma unroll
        for (int mt = 0; mt < 4; ++mt) {
            uint32_t w[4], a0[4], a1[4];
            ldmatrix_x4(tk + swz128(16 * mt + lr, 2 * kp + lc), w[0], w[1], w[2], w[3]);
            codes_to_f16(w[0], a0[0], a0[2]);
            codes_to_f16(w[1], a0[1], a0[3]);
            codes_to_f16(w[2], a1[0], a1[2]);
            codes_to_f16(w[3], a1[1], a1[3]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                mma_f16_16816(sc[mt][nt], a0, qb[2 * kp][nt][0], qb[2 * kp][nt][1]);
                mma_f16_16816(sc[mt][nt], a1, qb[2 * kp + 1][nt][0], qb[2 * kp + 1][nt][1]);
            }
        }
}

// Online softmax of a tile whose last visible token is lim; P^T as f16 B
// fragments pb[k-step of 16 tokens].
template <int NT>
__device__ __forceinline__ void softmax(float (&sc)[4][NT][4], const float (&mul)[NT][2], float s_k, int lim,
                                        State<NT> &st, uint32_t (&pb)[4][NT][2]) {
    const int g = (threadIdx.x & 31) >> 2;
    float alpha[NT][2];
    bool moved = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const float f[2] = {mul[nt][0] * s_k, mul[nt][1] * s_k};
        float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int mt = 0; mt < 4; ++mt)
#pragma unroll
            for (int k = 0; k < 4; ++k) sc[mt][nt][k] *= f[k & 1];
        if (lim < kBlockSize - 1) {   // the query's own tile
#pragma unroll
            for (int mt = 0; mt < 4; ++mt)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (16 * mt + g + 8 * (k >> 1) > lim) sc[mt][nt][k] = -INFINITY;
        }
#pragma unroll
        for (int mt = 0; mt < 4; ++mt)
#pragma unroll
            for (int k = 0; k < 2; ++k) mx[k] = max3_nan(mx[k], sc[mt][nt][k], sc[mt][nt][k + 2]);
        float ref[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            mx[h] = max_nan(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 4));
            mx[h] = max_nan(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 8));
            mx[h] = max_nan(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 16));
            // a NaN logit counts as +inf: its weight 2^(NaN - inf) makes the row
            // NaN, and the +inf carries that through every later merge
            if (mx[h] != mx[h]) mx[h] = INFINITY;
            const float m_new = fmaxf(st.m[nt][h], mx[h]);
            ref[h] = m_new == -INFINITY ? 0.f : m_new;   // nothing visible yet: every weight is 2^-inf = 0
            alpha[nt][h] = exp2_fast(st.m[nt][h] - ref[h]);
            moved |= m_new != st.m[nt][h];
            st.m[nt][h] = m_new;
        }
        float rs[2] = {0.f, 0.f};
#pragma unroll
        for (int mt = 0; mt < 4; ++mt) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                sc[mt][nt][k] = exp2_fast(sc[mt][nt][k] - ref[k & 1]);
                rs[k & 1] += sc[mt][nt][k];
            }
            pb[mt][nt][0] = movmatrix_trans(pack_f16x2(sc[mt][nt][0], sc[mt][nt][1]));
            pb[mt][nt][1] = movmatrix_trans(pack_f16x2(sc[mt][nt][2], sc[mt][nt][3]));
        }
        st.l[nt][0] = st.l[nt][0] * alpha[nt][0] + rs[0];
        st.l[nt][1] = st.l[nt][1] * alpha[nt][1] + rs[1];
    }
    // past the first tiles the maxima rarely move, and O keeps its scale
    if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
        for (int dm = 0; dm < 8; ++dm)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int k = 0; k < 4; ++k) st.o[dm][nt][k] *= alpha[nt][k & 1];
    }
}

// O^T += s_v (V^T P^T) for one V tile; the tile's product is formed on its own,
// since every tile has its own scale
template <int NT>
__device__ __forceinline__ void weigh(uint32_t tv, float s_v, const uint32_t (&pb)[4][NT][2],
                                      State<NT> &st) {
    const int lane = threadIdx.x & 31;
    // the token whose row this lane addresses: row 4 c + i of a matrix is token
    // 2 c + (i & 1) + 8 (i >> 1) of its 16
    const int r = lane & 15, tok = (lane & 16) + 2 * (r >> 2) + (r & 1) + 8 * ((r >> 1) & 1);
#pragma unroll
    for (int dm = 0; dm < 8; ++dm) {
        float pv[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) pv[nt][0] = pv[nt][1] = pv[nt][2] = pv[nt][3] = 0.f;
#pragma unroll
        for (int mp = 0; mp < 2; ++mp) {   // 32 tokens: two k-steps per ldmatrix
            uint32_t w[4], a0[4], a1[4];
            ldmatrix_b8_x2_trans(tv + swz128(32 * mp + tok, dm), w[0], w[1], w[2], w[3]);
            codes_to_f16(w[0], a0[0], a0[2]);
            codes_to_f16(w[1], a0[1], a0[3]);
            codes_to_f16(w[2], a1[0], a1[2]);
            codes_to_f16(w[3], a1[1], a1[3]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                mma_f16_16816(pv[nt], a0, pb[2 * mp][nt][0], pb[2 * mp][nt][1]);
                mma_f16_16816(pv[nt], a1, pb[2 * mp + 1][nt][0], pb[2 * mp + 1][nt][1]);
            }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int k = 0; k < 4; ++k) st.o[dm][nt][k] = fmaf(pv[nt][k], s_v, st.o[dm][nt][k]);
    }
}

// a tile of the warp's stream: its place in the stream, sequence tile and pool row
struct Tile {
    int x;   // < 0: the stream has ended
    int blk, row, kvh;
};

}  // namespace

// NT: query-head n-tiles of 8 (the GQA group is <= 8 * NT); kWarps: warps per CTA
template <int NT, int kWarps>
__global__ void __launch_bounds__(kWarps * 32, 1)
sparse_attn_fp8_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, AttnArgs a) {
    constexpr int warps = kWarps, threads = kWarps * 32;
    constexpr Plan plan(kWarps);
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
    uint8_t *gbase = smem_raw + (base - raw);
    float *s_ml = reinterpret_cast<float *>(gbase + plan.ml);   // [warp][16][2]
    int *s_cuq = reinterpret_cast<int *>(gbase + plan.cuq);
    volatile int *s_never = reinterpret_cast<volatile int *>(gbase + plan.words);   // stays 0: no abort flag
    volatile int *s_last = s_never + 1, *s_end = s_never + 2;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, c = blockIdx.x;
    const uint32_t ring = base + warp * kRingBytes, bars = base + plan.bars + warp * kSlots * 8;
    const int G = a.group, T = a.total_q;
    const unit_t K = (unit_t)a.k_max << a.tile_shift;   // tiles per pair

    pdl_trigger();
    if (lane == 0)
        for (int s = 0; s < kSlots; ++s) mbar_init(bars + 8 * s, 1);
    if (tid == 0) *s_never = 0;
    if (lane == 0) {
        fence_barrier_init();
        if (warp == 0) {
            prefetch_tensormap(&tm_k);
            prefetch_tensormap(&tm_v);
        }
    }
    const bool cached = a.num_seqs + 1 <= kMaxSmemSeqs;
    if (cached)
        for (int i = tid; i <= a.num_seqs; i += threads) s_cuq[i] = __ldg(a.cu_q + i);
    // queries behind the last sequence's (a padded batch) are not attended to, their rows not written
    if (tid == 0) *s_end = __ldg(a.cu_q + a.num_seqs);
    __syncthreads();

    const int W = gridDim.x * warps, pairs = T * a.num_kv_heads;
    const int own0 = c * warps + warp;                 // this warp's own pairs: own0 + i * W
    const unit_t n_own = (unit_t)a.warp_rounds * K;     // the warp's stream: their tiles, then its share
    // of a team's pair: tiles j_first, j_first + team, ... of the CTA's part [j_lo, j_hi)
    const int team = a.team, splits = a.splits, member = team > 0 ? warp % team : 0;
    int tail_pair = -1;
    unit_t j_lo = 0, j_hi = 0;
    if (team > 0) {
        const int i = splits > 1 ? c / splits : own0 / team;
        if (a.warp_rounds * W + i < pairs) {
            tail_pair = a.warp_rounds * W + i;
            const unsigned long long part = splits > 1 ? c - i * splits : 0;   // times K: past 32 bits
            j_lo = (unit_t)(part * K / (unsigned)splits);
            j_hi = (unit_t)((part + 1) * K / (unsigned)splits);
        }
    }
    const unit_t j_first = j_lo + (unit_t)member;
    const unit_t n_all = n_own + (j_hi > j_first ? (j_hi - j_first + team - 1) / team : 0);

    // ---- the stream: 32 places at a time are resolved to pool rows, a lane each
    uint32_t err_bits = 0;
    unsigned ready = 0;           // resolved places not yet taken
    int x_base = -32;
    int l_blk = 0, l_row = 0, l_kvh = 0;
    auto resolve = [&]() {
        const unit_t x = (unit_t)x_base + lane;
        bool good = false;
        if (x < n_all) {
            unit_t pair, ju;
            if (x < n_own) {
                const unit_t i = x / K;
                pair = (unit_t)own0 + i * W;
                ju = x - i * K;
            } else {
                pair = (unit_t)tail_pair;
                ju = j_first + (x - n_own) * (unit_t)team;
            }
            if (pair < (unit_t)pairs) {
                l_kvh = (int)(pair / (unit_t)T);
                const int t = (int)(pair - (unit_t)l_kvh * (unit_t)T);
                int s;
                if (cached) {
                    int lo = 0, hi = a.num_seqs - 1;
                    while (lo < hi) {
                        const int mid = (lo + hi + 1) >> 1;
                        if (s_cuq[mid] <= t) lo = mid; else hi = mid - 1;
                    }
                    s = lo;
                } else {
                    s = find_seq(a.cu_q, a.num_seqs, t);
                }
                const int p = __ldg(a.q_pos + t), len = __ldg(a.seq_lens + s);
                const int j = (int)(ju >> a.tile_shift), sub = (int)ju & ((1 << a.tile_shift) - 1);
                pdl_wait();   // returns at once after the first time
                int n_sel = ld_ordered_cg(a.cnt + t);
                const int b = ld_ordered_cg(a.sel + (size_t)t * a.k_max + j);
                const int n_vis = (p >> a.block_shift) + 1;
                if (p < 0 || p >= len || n_vis > a.max_blocks || n_sel < 0 || n_sel > a.k_max || t >= *s_end)
                    n_sel = 0;
                if (j < n_sel) {
                    if (b < 0 || b >= n_vis) {
                        err_bits |= DSA_DEV_ERR_SEL;
                    } else {
                        const int pg = __ldg(a.block_table + (size_t)s * a.max_blocks + b);
                        l_blk = (b << a.tile_shift) + sub;
                        if (pg < 0 || pg >= a.num_pages) {
                            err_bits |= DSA_DEV_ERR_PAGE;
                        } else if (l_blk <= p >> 6) {   // tiles past the position (own block only) hold nothing visible
                            l_row = (pg << a.block_shift) + (sub << 6);
                            good = true;
                        }
                    }
                }
            }
        }
        ready = __ballot_sync(0xffffffffu, good);
    };
    auto next = [&]() {
        Tile d;
        d.x = -1;
        while (ready == 0) {
            if (x_base >= 0 && (unit_t)x_base + 32 >= n_all) return d;
            x_base += 32;
            if ((unit_t)x_base >= n_all) return d;
            resolve();
        }
        const int src = __ffs(ready) - 1;
        ready &= ready - 1;
        d.x = x_base + src;
        d.blk = __shfl_sync(0xffffffffu, l_blk, src);
        d.row = __shfl_sync(0xffffffffu, l_row, src);
        d.kvh = __shfl_sync(0xffffffffu, l_kvh, src);
        return d;
    };
    // ---- the ring: every K tile in slot 0, every V tile in slot 1, each refilled
    // as soon as it is read
    auto issue = [&](int slot, const Tile &d) {
        if (d.x >= 0 && lane == 0) {
            mbar_arrive_expect_tx(bars + 8 * slot, kTileBytes);
            tma_load_3d(ring + slot * kTileBytes, slot ? &tm_v : &tm_k, 0, d.kvh, d.row, bars + 8 * slot);
        }
    };
    uint32_t phase = 0;   // of the current tile, in both slots
    auto arrived = [&](int slot) {
        return __all_sync(0xffffffffu, mbar_wait(bars + 8 * slot, phase, s_never)) != 0;
    };

    uint32_t qb[8][NT][2];
    float mul[NT][2];
    State<NT> st;
    Tile cur = next();
    pdl_wait();
    issue(0, cur);
    issue(1, cur);
    // a tile's scales (one address for the whole warp) are loaded a tile ahead: they
    // come from memory as slowly as the codes do
    auto scales_of = [&](const Tile &d, float &k, float &v) {
        if (d.x >= 0) {
            const size_t i = (size_t)(d.row >> 6) * a.num_kv_heads + d.kvh;
            k = ld_ordered_cg(a.k_scale + i);
            v = ld_ordered_cg(a.v_scale + i);
        }
    };
    float s_k = 0.f, s_v = 0.f;
    scales_of(cur, s_k, s_v);
    Tile nxt = next();
    bool dead = false, dead_behind_k = false;   // a wait gave up; behind the next K tile's copy
    // the warp's tiles before place x_end, all of one pair at position p
    auto run = [&](unit_t x_end, int p) {
        while (!dead && cur.x >= 0 && (unit_t)cur.x < x_end) {
            float sc[4][NT][4];
            uint32_t pb[4][NT][2];
            float nxt_k = 0.f, nxt_v = 0.f;
            scales_of(nxt, nxt_k, nxt_v);
            if (!arrived(0)) { dead = true; break; }
            scores<NT>(ring, qb, sc);
            __syncwarp();
            issue(0, nxt);
            const int lim = p - cur.blk * kBlockSize;   // >= 63 but in the query's own tile
            softmax<NT>(sc, mul, s_k, lim, st, pb);
            const Tile after = next();
            if (!arrived(1)) { dead = dead_behind_k = true; break; }
            const uint32_t tile = ring + kTileBytes;
            if (lim < kBlockSize - 1) {
                // slots past the query's position hold whatever the cache had there;
                // a zero weight times a NaN is NaN, so their value rows are cleared
                for (int e = lane; e < (kBlockSize - 1 - lim) * 8; e += 32)
                    st_shared_zero16(tile + swz128(lim + 1 + (e >> 3), e & 7));
                __syncwarp();
            }
            weigh<NT>(tile, s_v, pb, st);
            // generic-proxy stores (the cleared rows) before the TMA refills the slot
            if (lim < kBlockSize - 1) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            issue(1, nxt);
            phase ^= 1;
            cur = nxt;
            nxt = after;
            s_k = nxt_k;
            s_v = nxt_v;
        }
    };

    // ---- this warp's own pairs
    for (int i = 0; i < a.warp_rounds; ++i) {
        const int pair = own0 + i * W;
        if (pair >= pairs) break;
        const int kvh = pair / T, t = pair - kvh * T;
        if (t >= *s_end) continue;
        const size_t row0 = (size_t)t * a.num_q_heads + (size_t)kvh * G;
        st.clear();
        load_queries<NT>(a.q + row0 * kHeadDim, G, a.scale_log2, qb, mul);
        run((unit_t)(i + 1) * K, __ldg(a.q_pos + t));
        st.sum_lanes();
        const int g = lane >> 2, cq = lane & 3;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const float inv[2] = {inv_of(st.l[nt][0]), inv_of(st.l[nt][1])};
            // neighbouring lanes g, g ^ 1 trade a head each: 4-byte stores of two dims
            const int h = 8 * nt + 2 * cq + (g & 1);
            __nv_bfloat16 *dst = a.out + (row0 + h) * kHeadDim + (g & ~1);
#pragma unroll
            for (int dm = 0; dm < 8; ++dm)
#pragma unroll
                for (int k = 0; k < 4; k += 2) {
                    const float x = st.o[dm][nt][k] * inv[0], y = st.o[dm][nt][k + 1] * inv[1];
                    const float other = __shfl_xor_sync(0xffffffffu, (g & 1) ? x : y, 4);
                    const uint32_t v = (g & 1) ? pack_bf16x2(other, y) : pack_bf16x2(x, other);
                    if (h < G) *reinterpret_cast<uint32_t *>(dst + 16 * dm + 4 * k) = v;
                }
            if (a.lse && g < 2 && 8 * nt + 2 * cq + g < G)
                a.lse[row0 + 8 * nt + 2 * cq + g] = lse_of(g ? st.m[nt][1] : st.m[nt][0], g ? st.l[nt][1] : st.l[nt][0]);
        }
    }

    // ---- the team's pair (its warps agree on tail_pair)
    if (tail_pair >= 0) {
        const int kvh = tail_pair / T, t = tail_pair - kvh * T;
        const size_t row0 = (size_t)t * a.num_q_heads + (size_t)kvh * G;
        st.clear();
        if (cur.x >= 0) {
            load_queries<NT>(a.q + row0 * kHeadDim, G, a.scale_log2, qb, mul);
            run(n_all, __ldg(a.q_pos + t));
        }
        st.sum_lanes();
        const int g = lane >> 2, cq = lane & 3;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int h0 = 8 * nt + 2 * cq;
            float *r0 = reinterpret_cast<float *>(gbase + warp * kRingBytes) + h0 * kMergeStride, *r1 = r0 + kMergeStride;
#pragma unroll
            for (int dm = 0; dm < 8; ++dm) {
                const int d = 16 * dm + g;
                r0[d] = st.o[dm][nt][0];
                r1[d] = st.o[dm][nt][1];
                r0[d + 8] = st.o[dm][nt][2];
                r1[d + 8] = st.o[dm][nt][3];
            }
            if (g == 0) {
                float *ml = s_ml + (warp * 16 + h0) * 2;
                ml[0] = st.m[nt][0]; ml[1] = st.l[nt][0];
                ml[2] = st.m[nt][1]; ml[3] = st.l[nt][1];
            }
        }
        const int w0 = warp - member, bar = 1 + warp / team;   // a named barrier per team
        named_barrier(bar, team * 32);
        for (int e = member * 32 + lane; e < G * 32; e += team * 32) {
            const int r = e >> 5, d0 = (e & 31) * 4;
            const float *ml = s_ml + (w0 * 16 + r) * 2;
            const float *mo = reinterpret_cast<const float *>(gbase + w0 * kRingBytes) + r * kMergeStride + d0;
            float M = -INFINITY, L = 0.f;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int w = 0; w < team; ++w) M = fmaxf(M, ml[w * 32]);
            if (M != -INFINITY)
                for (int w = 0; w < team; ++w) {
                    const float m = ml[w * 32];
                    if (m == -INFINITY) continue;
                    const float f = exp2f(m - M);
                    L += ml[w * 32 + 1] * f;
                    const float4 v = *reinterpret_cast<const float4 *>(mo + w * (kRingBytes / 4));
                    acc.x += v.x * f; acc.y += v.y * f; acc.z += v.z * f; acc.w += v.w * f;
                }
            if (t >= *s_end) continue;
            if (splits == 1) {
                const float inv = inv_of(L);
                *reinterpret_cast<uint2 *>(a.out + (row0 + r) * kHeadDim + d0) =
                    make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
                if (a.lse && d0 == 0) a.lse[row0 + r] = lse_of(M, L);
            } else {
                float *dst = a.part + ((size_t)c * G + r) * kAttnPartStride;
                *reinterpret_cast<float4 *>(dst + d0) = acc;
                if (d0 == 0) *reinterpret_cast<float2 *>(dst + 128) = make_float2(M, L);
            }
        }
        if (splits > 1) {   // the team is the CTA
            __syncthreads();   // the partial's stores are ordered before the count
            if (tid == 0) *s_last = atomic_add_acq_rel_gpu(a.counters + tail_pair, 1) + 1 == splits;
            __syncthreads();
            if (*s_last) {
                const int c0 = c / splits * splits;
                for (int e = tid; e < (t < *s_end ? G * 32 : 0); e += threads) {
                    const int r = e >> 5, d0 = (e & 31) * 4;
                    float M = -INFINITY, L = 0.f;
                    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
                    constexpr int kBatch = 4;   // partials in flight per round trip
                    for (int k0 = 0; k0 < splits; k0 += kBatch) {
                        float2 ml[kBatch];
                        float4 ov[kBatch];
#pragma unroll
                        for (int k = 0; k < kBatch; ++k) {
                            ml[k] = make_float2(-INFINITY, 0.f);
                            ov[k] = make_float4(0.f, 0.f, 0.f, 0.f);
                            if (k0 + k < splits) {
                                const float *src = a.part + ((size_t)(c0 + k0 + k) * G + r) * kAttnPartStride;
                                ml[k] = __ldcg(reinterpret_cast<const float2 *>(src + 128));
                                ov[k] = __ldcg(reinterpret_cast<const float4 *>(src + d0));
                            }
                        }
                        float Mn = M;
#pragma unroll
                        for (int k = 0; k < kBatch; ++k) Mn = fmaxf(Mn, ml[k].x);
                        if (Mn == -INFINITY) continue;
                        const float fo = M == -INFINITY ? 0.f : exp2f(M - Mn);
                        L *= fo;
                        acc.x *= fo; acc.y *= fo; acc.z *= fo; acc.w *= fo;
#pragma unroll
                        for (int k = 0; k < kBatch; ++k) {
                            if (ml[k].x == -INFINITY) continue;
                            const float f = exp2f(ml[k].x - Mn);
                            L += ml[k].y * f;
                            acc.x += ov[k].x * f; acc.y += ov[k].y * f;
                            acc.z += ov[k].z * f; acc.w += ov[k].w * f;
                        }
                        M = Mn;
                    }
                    const float inv = inv_of(L);
                    *reinterpret_cast<uint2 *>(a.out + (row0 + r) * kHeadDim + d0) =
                        make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
                    if (a.lse && d0 == 0) a.lse[row0 + r] = lse_of(M, L);
                }
                if (tid == 0) a.counters[tail_pair] = 0;
            }
        }
    }
    err_bits = __reduce_or_sync(0xffffffffu, err_bits);
    if (lane == 0 && err_bits) set_err(a.dev_err, err_bits);
    if (dead) {
        // a wait gave up: say so, and let the copies in flight land (again with a
        // limit) before the CTA's shared memory goes to the next one
        if (lane == 0) {
            set_err(a.dev_err, DSA_DEV_ERR_WAIT);
            // the current tile's phase of each slot, and the next tile's where it was issued
            for (int slot = 0; slot < kSlots; ++slot) {
                mbar_wait(bars + 8 * slot, phase, s_never);
                if (slot == 0 && dead_behind_k && nxt.x >= 0) mbar_wait(bars, phase ^ 1, s_never);
            }
        }
        __syncwarp();
    }
}

namespace {

using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                   const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
    static const EncodeTiledFn fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<EncodeTiledFn>(p);
    }();
    return fn;
}

// pool of codes: dims (head_dim, kv_head, page * B + token), boxes of one tile of one head
cudaError_t pool_map(CUtensorMap &m, const void *pool, const AttnArgs &a) {
    const EncodeTiledFn enc = encode_fn();
    if (!enc) return cudaErrorNotSupported;
    const cuuint64_t dims[3] = {(cuuint64_t)kHeadDim, (cuuint64_t)a.num_kv_heads,
                                (cuuint64_t)a.num_pages << a.block_shift};
    const cuuint64_t strides[2] = {(cuuint64_t)kHeadDim, (cuuint64_t)a.num_kv_heads * kHeadDim};
    const cuuint32_t box[3] = {(cuuint32_t)kHeadDim, 1, kBlockSize};
    const cuuint32_t estr[3] = {1, 1, 1};
    return enc(&m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void *>(pool), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? cudaSuccess
               : cudaErrorInvalidValue;
}

template <int NT, int kWarps>
cudaError_t launch(const AttnArgs &a, const CUtensorMap &k, const CUtensorMap &v, cudaStream_t stream) {
    // the shared-memory opt-in, once per device
    static std::atomic<unsigned long long> done{0};
    constexpr int bytes = Plan(kWarps).bytes;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || !(done.load() >> dev & 1)) {
        e = cudaFuncSetAttribute(sparse_attn_fp8_kernel<NT, kWarps>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != cudaSuccess) return e;
        if (dev < 64) done.fetch_or(1ull << dev);
    }
    return launch_pdl(sparse_attn_fp8_kernel<NT, kWarps>, dim3(a.num_ctas), dim3(kWarps * 32), (size_t)bytes, stream, k,
                      v, a);
}

}  // namespace

cudaError_t launch_sparse_attn_fp8(const AttnArgs &a, cudaStream_t stream) {
    CUtensorMap k, v;
    cudaError_t e = pool_map(k, a.k_pool, a);
    if (e == cudaSuccess) e = pool_map(v, a.v_pool, a);
    if (e != cudaSuccess) return e;
    if (a.group > 8) return launch<2, kFp8Warps>(a, k, v, stream);
    return a.warps == kFp8Warps ? launch<1, kFp8Warps>(a, k, v, stream) : launch<1, kFp8ManyWarps>(a, k, v, stream);
}

}  // namespace dsa
