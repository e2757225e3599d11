// attn_fp8.cuh -- one 64-token tile of an 8-bit (E4M3) cache against the query
// heads of its KV head, for one consumer warp of the sparse attention kernel.
//
//     S^T = (s_k * scale) * (K Q^T),  P = 2^(S - m),  O^T += s_v * (V^T P^T)
//
// with E4M3 codes K, V and the tile's fp32 scales s_k, s_v.  The products run
// as mma.m16n8k16 f16 with fp32 accumulation, in the same swap-AB form as the
// bf16 tile (tokens or dims are the M dimension, the <= 8 or 16 heads N):
//   * an E4M3 code is exact in f16, so K and V lose nothing in the conversion
//     (one cvt per two codes);
//   * a query row is multiplied by the power of two that brings its largest
//     entry into [2^14, 2^15): its bf16 significands then fit f16 exactly down
//     to 2^-29 of that entry, and below that are off by at most 2^-40 of it --
//     far under the fp32 accumulation's own rounding;
//   * P is in [0, 1] and rounds to f16 (half a step: 2^-12 relative, 2^-26
//     absolute below 2^-14); the softmax sum is taken in fp32 before that.
// E4M3 mma instructions (K as it is, P as 8 bits) would drop the conversions
// but hold P to 2^-4 and accumulate in fewer bits.
//
// The 8-bit operands reach the fragments without byte shuffles of K: an
// ldmatrix lane holds four neighbouring dims of one token, which serve as the
// k indexes (2c, 2c+1) and (2c+8, 2c+9) of one mma when the query fragments are
// laid out the same way.  For V the transposing ldmatrix moves byte pairs, so
// a lane holds dims (2g, 2g+1) of tokens 2c and 2c+1; one byte permutation per
// register makes them the rows g and g+8 of V^T, i.e. accumulator rows g and
// g+8 of a 16-dim group are its dims 2g and 2g+1.
#pragma once

#include "dsa_tma.cuh"

#include <cuda_fp16.h>

namespace dsa {
namespace fp8 {

constexpr int kTileBytes = kBlockSize * kHeadDim;   // 8 KiB: 64 rows x 128 codes

// D(16x8 f32) += A(16x16 f16, row) * B(16x8 f16, col)
__device__ __forceinline__ void mma_f16_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
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

// 2^x for x <= 0 (-inf gives 0); results below 2^-126 become 0
__device__ __forceinline__ float exp2_neg(float x) {
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

// Query fragments of head row 8 * nt + g from the swizzled bf16 tile (two
// halves of 64 dims, `half_bytes` apart), as scaled f16: step kk covers dims
// 16 kk .. 16 kk + 15, this lane's 16 kk + 4 cq .. + 3.  mul[nt][h] is the
// factor from a raw accumulator of head 8 * nt + 2 * cq + h to base-2 logits.
template <int NT>
__device__ __forceinline__ void load_queries(uint32_t tile, uint32_t half_bytes, bool ok, float scale_log2,
                                             uint32_t (&qb)[8][NT][2], float (&mul)[NT][2]) {
    const int lane = threadIdx.x & 31, g = lane >> 2, cq = lane & 3;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        uint2 w[8];
        float top = 0.f;
        bool odd = false;   // a NaN or an infinity in the row
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
            const int r = 8 * nt + g, ch = 2 * kk + (cq >> 1);
            w[kk] = make_uint2(0u, 0u);
            if (ok)
                asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];"
                             : "=r"(w[kk].x), "=r"(w[kk].y)
                             : "r"(tile + (ch >> 3) * half_bytes + swz128(r, ch & 7) + (cq & 1) * 8));
            const float x[4] = {__uint_as_float(w[kk].x << 16), __uint_as_float(w[kk].x & 0xffff0000u),
                                __uint_as_float(w[kk].y << 16), __uint_as_float(w[kk].y & 0xffff0000u)};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                top = fmaxf(top, fabsf(x[k]));
                odd |= !(fabsf(x[k]) <= 3.4e38f);
            }
        }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // top = 2^(e - 127) * [1, 2): multiply by 2^(14 - (e - 127)); a row below
        // 2^-99 takes the largest factor (both factors stay normal numbers)
        const int e = max((int)(__float_as_uint(top) >> 23), 28);
        const float up = __uint_as_float((uint32_t)(268 - e) << 23);
        const float down = __uint_as_float((uint32_t)(e - 14) << 23);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
            qb[kk][nt][0] = pack_f16x2(__uint_as_float(w[kk].x << 16) * up, __uint_as_float(w[kk].x & 0xffff0000u) * up);
            qb[kk][nt][1] = pack_f16x2(__uint_as_float(w[kk].y << 16) * up, __uint_as_float(w[kk].y & 0xffff0000u) * up);
        }
        // a NaN or an infinity in the query makes the row's result NaN
        odd |= __shfl_xor_sync(0xffffffffu, odd, 1) != 0;
        odd |= __shfl_xor_sync(0xffffffffu, odd, 2) != 0;
        const float m = odd ? __uint_as_float(0x7fc00000u) : scale_log2 * down;
        mul[nt][0] = __shfl_sync(0xffffffffu, m, 8 * cq);        // the lane with g = 2 cq
        mul[nt][1] = __shfl_sync(0xffffffffu, m, 8 * cq + 4);    // g = 2 cq + 1
    }
}

// One tile: tk / tv are the swizzled 64 x 128-byte code tiles, lim the last
// visible token (value rows behind it are already cleared), s_k / s_v the
// scales; o, m_run and l_run the warp's running state.
template <int NT>
__device__ __forceinline__ void attend_tile(uint32_t tk, uint32_t tv, int lim, float s_k, float s_v,
                                            const uint32_t (&qb)[8][NT][2], const float (&mul)[NT][2],
                                            float (&o)[8][NT][4], float (&m_run)[NT][2], float (&l_run)[NT][2]) {
    const int lane = threadIdx.x & 31, g = lane >> 2;
    const int lr = (lane & 7) + 8 * ((lane >> 3) & 1), lc = lane >> 4;   // ldmatrix row and chunk of this lane
    float sc[4][NT][4];
#pragma unroll
    for (int mt = 0; mt < 4; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) sc[mt][nt][0] = sc[mt][nt][1] = sc[mt][nt][2] = sc[mt][nt][3] = 0.f;
#pragma unroll
    for (int kp = 0; kp < 4; ++kp) {   // 32 dims: two k-steps per ldmatrix
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
    // online softmax per head column
    float alpha[NT][2];
    uint32_t pb[4][NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const float f[2] = {mul[nt][0] * s_k, mul[nt][1] * s_k};
        float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int mt = 0; mt < 4; ++mt)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float x = 16 * mt + g + 8 * (k >> 1) <= lim ? sc[mt][nt][k] * f[k & 1] : -INFINITY;
                sc[mt][nt][k] = x;
                mx[k & 1] = max_nan(mx[k & 1], x);
            }
        float ref[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            mx[h] = max_nan(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 4));
            mx[h] = max_nan(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 8));
            mx[h] = max_nan(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 16));
            // a NaN logit counts as +inf: its weight 2^(NaN - inf) makes the row
            // NaN, and the +inf carries that through every later merge
            if (mx[h] != mx[h]) mx[h] = INFINITY;
            const float m_new = fmaxf(m_run[nt][h], mx[h]);
            ref[h] = m_new == -INFINITY ? 0.f : m_new;   // nothing visible yet: every weight is 2^-inf = 0
            alpha[nt][h] = exp2_neg(m_run[nt][h] - ref[h]);
            m_run[nt][h] = m_new;
        }
        float rs[2] = {0.f, 0.f};
#pragma unroll
        for (int mt = 0; mt < 4; ++mt) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                sc[mt][nt][k] = exp2_neg(sc[mt][nt][k] - ref[k & 1]);
                rs[k & 1] += sc[mt][nt][k];
            }
            pb[mt][nt][0] = movmatrix_trans(pack_f16x2(sc[mt][nt][0], sc[mt][nt][1]));
            pb[mt][nt][1] = movmatrix_trans(pack_f16x2(sc[mt][nt][2], sc[mt][nt][3]));
        }
        l_run[nt][0] = l_run[nt][0] * alpha[nt][0] + rs[0];
        l_run[nt][1] = l_run[nt][1] * alpha[nt][1] + rs[1];
    }
    // O^T = alpha O^T + s_v (V^T P^T): the tile's product is formed on its own,
    // since every tile has its own scale
#pragma unroll
    for (int dg = 0; dg < 4; ++dg) {   // 32 dims: two groups of 16 per ldmatrix
        float pv[2][NT][4];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) pv[i][nt][0] = pv[i][nt][1] = pv[i][nt][2] = pv[i][nt][3] = 0.f;
#pragma unroll
        for (int mt = 0; mt < 4; ++mt) {
            uint32_t w[4], a0[4], a1[4];
            ldmatrix_x4_trans(tv + swz128(16 * mt + lr, 2 * dg + lc), w[0], w[1], w[2], w[3]);
            codes_to_f16(__byte_perm(w[0], 0u, 0x3120), a0[0], a0[1]);
            codes_to_f16(__byte_perm(w[1], 0u, 0x3120), a0[2], a0[3]);
            codes_to_f16(__byte_perm(w[2], 0u, 0x3120), a1[0], a1[1]);
            codes_to_f16(__byte_perm(w[3], 0u, 0x3120), a1[2], a1[3]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                mma_f16_16816(pv[0][nt], a0, pb[mt][nt][0], pb[mt][nt][1]);
                mma_f16_16816(pv[1][nt], a1, pb[mt][nt][0], pb[mt][nt][1]);
            }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    o[2 * dg + i][nt][k] = fmaf(pv[i][nt][k], s_v, o[2 * dg + i][nt][k] * alpha[nt][k & 1]);
    }
}

}  // namespace fp8
}  // namespace dsa
