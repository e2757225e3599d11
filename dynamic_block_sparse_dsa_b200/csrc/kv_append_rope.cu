// kv_append_rope.cu -- appending new tokens with the position rotation applied
// on the way, into the bf16 cache and into the 8-bit (E4M3) cache.
//
// "Day-0 Readiness for Trillion-Parameter Models: Engineering Sparse Attention
// and Expert Weight Compression", section "KV Cache Layout": prefill writes
// blocks in batch, decode appends one token, both through one block table.
// The rotation and the 8-bit storage have no counterpart on the pages.
//
// Rotation.  Pair i of a row at position p turns by the angle p * inv_freq[i]:
//     (x, y) -> (x cos - y sin, y cos + x sin) * scale.
// At a million tokens p * inv_freq in fp32 is off by up to 0.06 rad, so the
// angle is kept in turns as a 64-bit fraction: f = inv_freq / (2 pi) mod 1
// times 2^64, and p * f mod 2^64 is the fraction of a turn.  f is off by at most
// 2^-63 (turns_q64), the fraction at any int32 position by 2^-32.  Its upper 32
// bits give the nearest quarter turn and a remainder in [-pi/4, pi/4], rounded
// to fp32 (2^-26 of a turn), whose sine and cosine are Taylor sums (to x^9 and
// x^8: the next terms are below 2^-25 there).  The rotation itself is fp32,
// rounded once to the stored type.
//
// E4M3 cache.  A tile is 64 tokens of a block; each (tile, KV head) has one
// scale for K and one for V, a power of two when written here:
//     need = the least 2^e, e >= -100, with max |x| <= 448 * 2^e over the new rows
//     s'   = need for a tile whose first token is new, else max(s, need)
//     new rows: e4m3(x / s');  rows held from before: e4m3(code * s / s') if s' != s.
// A power of two keeps the 4-bit significand of every code that stays normal,
// so growing the scale again and again does not add up roundings; a scale of
// max/448 would spread the codes by up to 2x more evenly but re-round each.
//
// Work and bounds (one B200).  The bf16 kernel runs a CTA of 256 threads per
// token: its K, V and query rows, 32 bytes a thread and row, with the rows'
// loads issued before the (cos, sin) table is ready.  4096 tokens of 64 query
// and 8 KV heads take 31.3 us in calls back to back, 5.4 TB/s of rows read and
// written (0.82 of the copy bandwidth): memory-bound, with a gap between the
// calls (28.6 us when the next call's loads filled it, before its wait).  The
// E4M3 kernel runs a CTA of 512 threads per
// (tile, K or V, up to eight heads) and per two queries: the first wait on
// tables, maxima and barriers, the second on memory, and they share the SMs.
// 4160 tokens (64 of them decode tokens) take 30.9 us, 5.2 TB/s (0.80); 32 decode
// tokens take 2.3 us back to back.
#include "dsa_kernels.h"

#include <cuda_fp8.h>
#include <float.h>

namespace dsa {

namespace {

constexpr int kThreads = 256, kSlots = kThreads / 8;   // eight threads (32 bytes of a row each) per row
constexpr int kTileThreads = 2 * kThreads;             // E4M3 append: a row of a full tile per eight threads
constexpr int kPairs = kHeadDim / 2;
// CTAs per SM of the two kernels: with the SMs, the first wave, which may start
// before the kernel ahead ends
constexpr int kRopeCtas = 5, kTileCtas = 2, kSms = 148;
constexpr int kMinScaleExp = -100;
constexpr int kMaxAxes = 4;

// The fraction of a turn per position as a 64-bit fixed-point number.  1 / (2 pi)
// is the sum of two doubles, and the product with the first is kept with its
// rounding error: the product of one double alone is off by 2^-53 of its size,
// which at inv_freq 100 and position 2^31 is 2.6e-6 of a turn.  The whole turns
// drop out exactly (hi - rint(hi)); the two conversions cut off below 2^-64 each.
__device__ __forceinline__ unsigned long long turns_q64(float inv_freq) {
    constexpr double kHi = 0.15915494309189535, kLo = -9.839338337591243e-18;
    constexpr double kOne = 18446744073709551616.0;   // 2^64
    const double x = inv_freq, hi = x * kHi, lo = fma(x, kHi, -hi) + x * kLo;
    return (unsigned long long)((long long)((hi - rint(hi)) * kOne) + (long long)(lo * kOne));
}

// (cos, sin) of the angle at position p, times the rotation's scale
__device__ __forceinline__ float2 rope_cs(int p, unsigned long long f, float scale) {
    const uint32_t turn = (uint32_t)(((unsigned long long)(long long)p * f) >> 32);   // of 2^32
    const uint32_t quarter = (turn + 0x20000000u) >> 30;                               // nearest quarter turn
    const float x = (float)(int)(turn - (quarter << 30)) * (float)(3.14159265358979323846 / 2147483648.0);
    const float y = x * x;
    float s = fmaf(y, fmaf(y, fmaf(y, 1.f / 362880.f, -1.f / 5040.f), 1.f / 120.f), -1.f / 6.f);
    s = fmaf(x * y, s, x);
    const float c = fmaf(y, fmaf(y, fmaf(y, fmaf(y, 1.f / 40320.f, -1.f / 720.f), 1.f / 24.f), -0.5f), 1.f);
    // a quarter turn on: (c, s) -> (-s, c)
    const float u = (quarter & 1u) ? s : c, v = (quarter & 1u) ? c : s;
    const float cs = ((quarter + 1u) & 2u) ? -u : u, sn = (quarter & 2u) ? -v : v;
    return make_float2(cs * scale, sn * scale);
}

// the (cos, sin) table of one row: thread j of the row owns pairs 8j..8j+7,
// kept as [pair of pairs m][j] so that the eight threads' 16-byte reads are
// free of bank conflicts
struct RopeTab {
    float4 cs[4][8];
};
__device__ __forceinline__ void put_cs(RopeTab &t, int pair, float2 cs) {
    reinterpret_cast<float2 *>(&t.cs[(pair >> 1) & 3][pair >> 3])[pair & 1] = cs;
}

// 16-byte chunks (8 dims each) of a row that thread j owns.  Rotated threads
// (j < rotary_dim / 16) own both halves of eight pairs: chunks j and
// j + rotary_dim / 16 when a pair is (i, i + rotary_dim / 2), adjacent chunks
// when it is (2i, 2i + 1); the others own two chunks that are only copied.
__device__ __forceinline__ void own_chunks(const RopeArgs &r, int j, int &c0, int &c1) {
    const bool halves = !r.interleaved && j < (r.rotary_dim >> 4);
    c0 = halves ? j : 2 * j;
    c1 = halves ? j + (r.rotary_dim >> 4) : 2 * j + 1;
}

__device__ __forceinline__ void unpack8(const uint4 &u, float *x) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        x[2 * k] = __uint_as_float(w[k] << 16);
        x[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
    }
}
__device__ __forceinline__ uint4 pack8(const float *x) {
    return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                      pack_bf16x2(x[6], x[7]));
}

// rotate the sixteen values of thread j (chunk c0, then chunk c1)
__device__ __forceinline__ void rotate16(float *x, const RopeTab &t, int j, int interleaved) {
#pragma unroll
    for (int m = 0; m < 4; ++m) {
        const float4 cs = t.cs[m][j];
        const float cc[2] = {cs.x, cs.z}, ss[2] = {cs.y, cs.w};
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int e = 2 * m + k;   // both layouts by constant indexes, so that x stays in registers
            if (interleaved) {
                const float u = x[2 * e], v = x[2 * e + 1];
                x[2 * e] = u * cc[k] - v * ss[k];
                x[2 * e + 1] = v * cc[k] + u * ss[k];
            } else {
                const float u = x[e], v = x[8 + e];
                x[e] = u * cc[k] - v * ss[k];
                x[8 + e] = v * cc[k] + u * ss[k];
            }
        }
    }
}

// Last index s in [0, n) whose value is <= i (values ascend), by one warp: 32
// independent loads per step while n is small, a binary search beyond that.
template <typename F>
__device__ __forceinline__ int last_le_warp(int n, int i, F value) {
    if (n <= 256) {
        int count = 0;
        for (int b = 0; b < n; b += 32) {
            const int s = b + (int)(threadIdx.x & 31);
            count += __popc(__ballot_sync(0xffffffffu, s < n && value(s) <= i));
        }
        return max(count - 1, 0);
    }
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (value(mid) <= i) lo = mid; else hi = mid - 1;
    }
    return lo;
}

// the axis that `pair` turns by
__device__ __forceinline__ int axis_of(const RopeArgs &r, int pair, uint32_t &err) {
    const int axis = r.pair_axis ? __ldg(r.pair_axis + pair) : 0;
    if (axis >= 0 && axis < r.num_axes) return axis;
    err |= DSA_DEV_ERR_POS;
    return 0;
}

// where a new token lands; page < 0 when it is skipped
struct Place {
    int pos, page, slot;
    bool ends_block;   // the last new token of its block
};
__device__ __forceinline__ Place place_of(const KvAppendArgs &a, int i, uint32_t &err) {
    Place p{0, -1, 0, false};
    const int s = last_le_warp(a.num_seqs, i, [&](int k) { return __ldg(a.cu_new + k); });
    const int first = __ldg(a.cu_new + s), last = __ldg(a.cu_new + s + 1);
    const int len = __ldg(a.seq_lens + s), n = last - first;
    if (i < first || i >= last || n > len) {
        err |= DSA_DEV_ERR_POS;
        return p;
    }
    p.pos = len - n + (i - first);
    const int blk = p.pos >> a.block_shift;
    p.slot = p.pos & ((1 << a.block_shift) - 1);
    if (blk >= a.max_blocks) {
        err |= DSA_DEV_ERR_POS;
        return p;
    }
    p.page = __ldg(a.block_table + (size_t)s * a.max_blocks + blk);
    if (p.page < 0 || p.page >= a.num_pages) {
        err |= DSA_DEV_ERR_PAGE;
        p.page = -1;
    }
    p.ends_block = i == last - 1 || p.slot == (1 << a.block_shift) - 1;
    return p;
}

// the rotated query rows of one query and, in the bf16 cache, the K and V rows
// of one new token: row r of the CTA's list is K head r, then V head, then
// query head.  The rows may come from a kernel ahead and are read behind the wait
// for it.  A CTA of the first wave (early) looks up the token's place and forms
// the tables (s_tab: K, q) before that wait; the others, for which it is over,
// have the rows' first loads (kBatch per thread) under way meanwhile.  (8 decode
// tokens: 2.4 us early, 3.4 us not; 4096 tokens: 34.6 and 31.2 us.)  kThreads
// threads numbered tid share it; all threads of the CTA call it.
template <bool kKv>
__device__ __forceinline__ void token_rows(const AppendRopeArgs &a, int i, int tid, bool early, RopeTab *s_tab) {
    constexpr int kBatch = 2;
    const int j = tid & 7, slot = tid >> 3;
    const bool has_new = kKv && i < a.kv.total_new, has_q = i < a.total_q;
    const int hkv = has_new ? a.kv.num_kv_heads : 0, nq = has_q ? a.num_q_heads : 0;
    const int rows = 2 * hkv + nq;
    const RopeArgs &r = a.rope;
    int c0, c1;
    own_chunks(r, j, c0, c1);
    const bool turned = j < (r.rotary_dim >> 4);
    uint4 lo[kBatch], hi[kBatch];
    auto load = [&](int base) {
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int row = base + b * kSlots + slot;
            if (row < rows) {
                const __nv_bfloat16 *src;
                if (row < hkv) src = static_cast<const __nv_bfloat16 *>(a.kv.k_new) + i * a.k_stride + row * kHeadDim;
                else if (row < 2 * hkv) src = static_cast<const __nv_bfloat16 *>(a.kv.v_new) + i * a.v_stride + (row - hkv) * kHeadDim;
                else src = a.q + i * a.q_stride + (row - 2 * hkv) * kHeadDim;
                lo[b] = reinterpret_cast<const uint4 *>(src)[c0];
                hi[b] = reinterpret_cast<const uint4 *>(src)[c1];
            }
        }
    };
    uint32_t err = 0;
    Place p{0, -1, 0, false};
    auto prepare = [&]() {
        if (has_new) p = place_of(a.kv, i, err);
        if (tid >= 2 * kPairs) return;
        const int pair = tid & (kPairs - 1);
        const bool is_q = tid >= kPairs;
        if (pair < (r.rotary_dim >> 1) && (is_q ? has_q : has_new)) {
            const int axis = axis_of(r, pair, err);
            int pos = p.pos;
            if (is_q) pos = a.pos_q ? __ldg(a.pos_q + (size_t)axis * a.total_q + i) : __ldg(a.q_pos + i);
            else if (a.pos_new) pos = __ldg(a.pos_new + (size_t)axis * a.kv.total_new + i);
            put_cs(s_tab[is_q], pair, rope_cs(pos, turns_q64(__ldg(r.inv_freq + pair)), r.scale));
        }
    };
    if (early) prepare();
    pdl_wait();
    load(0);
    if (!early) prepare();
    if (err) set_err(a.kv.dev_err, err);
    __syncthreads();
    for (int base = 0; base < rows; base += kBatch * kSlots) {
        if (base) load(base);
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int row = base + b * kSlots + slot;
            if (row >= rows) break;
            const bool is_q = row >= 2 * hkv, is_v = !is_q && row >= hkv;
            if (turned && !is_v) {
                float x[16];
                unpack8(lo[b], x);
                unpack8(hi[b], x + 8);
                rotate16(x, s_tab[is_q], j, r.interleaved);
                lo[b] = pack8(x);
                hi[b] = pack8(x + 8);
            }
            uint4 *dst;
            if (is_q) {
                dst = reinterpret_cast<uint4 *>(a.q_out + ((size_t)i * a.num_q_heads + (row - 2 * hkv)) * kHeadDim);
            } else {
                if (p.page < 0) continue;
                __nv_bfloat16 *pool = static_cast<__nv_bfloat16 *>(is_v ? a.kv.v_pool : a.kv.k_pool);
                const size_t tok = ((size_t)p.page << a.kv.block_shift) + p.slot;
                dst = reinterpret_cast<uint4 *>(pool + (tok * hkv + (is_v ? row - hkv : row)) * kHeadDim);
            }
            dst[c0] = lo[b];
            dst[c1] = hi[b];
        }
    }
    if (has_new && a.kv.kc_new && p.page >= 0 && p.ends_block && tid < kIdxDim / 16)
        reinterpret_cast<int4 *>(a.kv.kc_pool)[(size_t)p.page * (kIdxDim / 16) + tid] =
            ld_ordered(reinterpret_cast<const int4 *>(a.kv.kc_new) + (size_t)i * (kIdxDim / 16) + tid);
}

// ------------------------------------------------------------------ E4M3 cache

// least 2^e >= 2^kMinScaleExp with amax <= 448 * 2^e, for a finite amax >= 0:
// 448 = 1.75 * 2^8, so e is amax's exponent - 8, one more if its significand
// exceeds 1.75.  (A subnormal amax lands on the floor.)
__device__ __forceinline__ float scale_for(float amax) {
    const uint32_t u = __float_as_uint(amax);
    const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
    return __uint_as_float((uint32_t)(max(e, kMinScaleExp) + 127) << 23);
}

__device__ __forceinline__ uint2 to_e4m3x8(const float *x, float inv) {
    uint32_t h[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
        h[k] = __nv_cvt_float2_to_fp8x2(make_float2(x[2 * k] * inv, x[2 * k + 1] * inv), __NV_SATFINITE, __NV_E4M3);
    return make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
}

__device__ __forceinline__ uint32_t rescale_e4m3x4(uint32_t w, float ratio) {
    float x[4];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> (16 * k)), __NV_E4M3);
        const float2 f = __half22float2(__half2(h));
        x[2 * k] = f.x * ratio;
        x[2 * k + 1] = f.y * ratio;
    }
    const uint32_t a = __nv_cvt_float2_to_fp8x2(make_float2(x[0], x[1]), __NV_SATFINITE, __NV_E4M3);
    const uint32_t b = __nv_cvt_float2_to_fp8x2(make_float2(x[2], x[3]), __NV_SATFINITE, __NV_E4M3);
    return a | (b << 16);
}

constexpr int kPassRows = kTileThreads / 8;
static_assert(kPassRows == kBlockSize, "a pass holds a full tile of one head");

// an append item: the new rows of one tile, K or V, for the heads [h_begin, h_end)
struct Item {
    int page, t0, len;      // t0: the tile's first position
    int held, cnt, i0;      // slots filled before, new tokens (0: nothing to do), the first of them
    int h_begin, h_end;
    bool is_v;
};

// Item number `item` = ((unit * 2) + is_v) * groups + head group, by one warp.
// Sequence s owns the units from cu_new[s] / 64 + 2 s on: n tokens lie in at
// most n / 64 + 2 tiles, and the next sequence starts no earlier.  Units behind a
// sequence's tiles have nothing to do.  (Counting the tiles exactly, 32
// sequences at a time, left fewer idle CTAs but took 2 us longer to find one's
// work: 32 decode tokens 5.0 against 2.8 us.)
__device__ __forceinline__ Item find_item(const AppendRopeArgs &a, int item) {
    const KvAppendArgs &kv = a.kv;
    const int H = kv.num_kv_heads, groups = (H + a.heads_per_item - 1) / a.heads_per_item;
    Item it{};
    const int g = item % groups;
    it.h_begin = g * a.heads_per_item;
    it.is_v = (item / groups) & 1;
    const int unit = item / (2 * groups);
    const bool reports = (threadIdx.x & 31) == 0 && g == 0 && !it.is_v;
    const int s = last_le_warp(kv.num_seqs, unit, [&](int k) { return (__ldg(kv.cu_new + k) >> 6) + 2 * k; });
    const int first = __ldg(kv.cu_new + s), last = __ldg(kv.cu_new + s + 1);
    it.len = __ldg(kv.seq_lens + s);
    if (unit == 0 && reports && __ldg(kv.cu_new + kv.num_seqs) < kv.total_new) set_err(kv.dev_err, DSA_DEV_ERR_POS);
    const int n = last - first;
    if (first < 0 || n < 0 || last > kv.total_new || n > it.len) {
        if (reports) set_err(kv.dev_err, DSA_DEV_ERR_POS);
        return it;
    }
    const int pos0 = it.len - n;                                 // first new position
    const long long t0 = ((long long)(pos0 >> 6) + unit - ((first >> 6) + 2 * s)) << 6;
    if (n == 0 || t0 >= it.len) return it;
    it.t0 = (int)t0;
    it.held = max(pos0 - it.t0, 0);
    const int cnt = min(it.len - it.t0, kBlockSize) - it.held;   // 1..64
    // where one pass holds every head, the first group takes them all
    const bool one_pass = cnt * H <= kPassRows;
    if (one_pass && g > 0) return it;
    const int blk = it.t0 >> kv.block_shift;
    if (blk >= kv.max_blocks) {
        if (reports) set_err(kv.dev_err, DSA_DEV_ERR_POS);
        return it;
    }
    it.page = __ldg(kv.block_table + (size_t)s * kv.max_blocks + blk);
    if (it.page < 0 || it.page >= kv.num_pages) {
        if (reports) set_err(kv.dev_err, DSA_DEV_ERR_PAGE);
        return it;
    }
    it.i0 = first + (it.t0 + it.held - pos0);
    it.h_end = one_pass ? H : min(it.h_begin + a.heads_per_item, H);
    it.cnt = cnt;
    return it;
}

// One item by the CTA.  A pass takes as many heads as fit 64 rows -- one head of
// a full tile, all heads of a decode token -- and holds their values in
// registers between the maximum and the stores, so the new rows are read once.
__device__ __forceinline__ void tile_rows(const AppendRopeArgs &a, int item, bool early, RopeTab *s_tab) {
    __shared__ int s_pos[kMaxAxes][kBlockSize];
    __shared__ uint32_t s_amax[kPassRows];
    __shared__ float s_old[kPassRows], s_new[kPassRows];
    __shared__ Item s_item;
    const KvAppendArgs &kv = a.kv;
    const RopeArgs &r = a.rope;
    const int tid = threadIdx.x, j = tid & 7, slot = tid >> 3;
    if (tid < 32) {   // one warp: copies of this chain in every warp would cost more than the rows
        const Item it = find_item(a, item);
        if (tid == 0) s_item = it;
    }
    __syncthreads();
    const Item it = s_item;
    const int cnt = it.cnt, held = it.held, H = kv.num_kv_heads;
    if (cnt == 0) return;
    const int per_pass = min(kPassRows / cnt, it.h_end - it.h_begin);   // heads per pass
    const size_t row0 = ((size_t)it.page << kv.block_shift) + (it.t0 & ((1 << kv.block_shift) - 1));   // pool row of slot 0
    uint8_t *pool = static_cast<uint8_t *>(it.is_v ? kv.v_pool : kv.k_pool) + row0 * H * kHeadDim;
    float *scales = (it.is_v ? a.v_scale : a.k_scale) + (row0 >> 6) * H;
    const __nv_bfloat16 *src = static_cast<const __nv_bfloat16 *>(it.is_v ? kv.v_new : kv.k_new);
    const long long stride = it.is_v ? a.v_stride : a.k_stride;
    const bool rotated = !it.is_v && r.rotary_dim > 0;
    const bool turned = rotated && j < (r.rotary_dim >> 4);
    int c0 = 2 * j, c1 = 2 * j + 1;
    if (rotated) own_chunks(r, j, c0, c1);

    // row `slot` of a pass is (head, token); a pass of one head needs no division
    const int rh = per_pass == 1 ? (slot < cnt ? 0 : kPassRows) : slot / cnt;
    const int rt = per_pass == 1 ? slot : slot - rh * cnt;
    const __nv_bfloat16 *mine = src + (it.i0 + rt) * stride + rh * kHeadDim;
    uint4 raw0, raw1;
    auto fetch = [&](int hb, int nh) {
        if (rh < nh) {
            raw0 = reinterpret_cast<const uint4 *>(mine + hb * kHeadDim)[c0];
            raw1 = reinterpret_cast<const uint4 *>(mine + hb * kHeadDim)[c1];
        }
    };
    uint32_t err = 0;
    auto tables = [&]() {
        if (!rotated) return;
        for (int e = tid; e < r.num_axes * cnt; e += kTileThreads) {
            const int axis = e / cnt, tok = e - axis * cnt;
            s_pos[axis][tok] = a.pos_new ? __ldg(a.pos_new + (size_t)axis * kv.total_new + it.i0 + tok)
                                         : it.t0 + held + tok;
        }
        __syncthreads();
        const int pair = tid % kPairs;   // the same pair for all of the thread's entries
        if (pair < (r.rotary_dim >> 1)) {
            const int axis = axis_of(r, pair, err);
            const unsigned long long f = turns_q64(__ldg(r.inv_freq + pair));
            for (int tok = tid / kPairs; tok < cnt; tok += kTileThreads / kPairs)
                put_cs(s_tab[tok], pair, rope_cs(s_pos[axis][tok], f, r.scale));
        }
    };
    if (early) tables();
    // rows, held scales and codes, and every store, come after the kernels ahead
    pdl_wait();
    fetch(it.h_begin, per_pass);
    if (!early) tables();   // the rows are on their way
    for (int hb = it.h_begin; hb < it.h_end; hb += per_pass) {
        const int nh = min(per_pass, it.h_end - hb);
        if (tid < nh) {
            s_amax[tid] = 0u;
            if (held > 0) s_old[tid] = ld_ordered_cg(scales + hb + tid);
        }
        float x[16];
        unpack8(raw0, x);
        unpack8(raw1, x + 8);
        if (hb + per_pass < it.h_end) fetch(hb + per_pass, min(per_pass, it.h_end - hb - per_pass));   // the next pass's rows
        __syncthreads();     // tables, cleared maxima, held scales
        uint32_t top = 0u;   // magnitudes order as their bits, infinities and NaN above them
        if (rh < nh) {
            if (turned) rotate16(x, s_tab[rt], j, r.interleaved);
#pragma unroll
            for (int e = 0; e < 16; ++e) top = max(top, __float_as_uint(x[e]) & 0x7fffffffu);
            if (top >= 0x7f800000u) {   // some are not finite: the largest of the others
                err |= DSA_DEV_ERR_VALUE;
                top = 0u;
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const uint32_t v = __float_as_uint(x[e]) & 0x7fffffffu;
                    if (v < 0x7f800000u) top = max(top, v);
                }
            }
        }
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 4));
        // the maximum does not depend on the order
        if (j == 0 && rh < nh) atomicMax(&s_amax[rh], top);
        __syncthreads();
        bool grows = false;
        if (tid < nh) {
            const float need = scale_for(__uint_as_float(s_amax[tid]));
            const float was = held > 0 ? s_old[tid] : 0.f;
            // a held scale that is not a positive finite number says nothing about its codes
            const bool good = was > 0.f && was <= FLT_MAX;
            const float now = good ? fmaxf(was, need) : need;
            if (now != was) scales[hb + tid] = now;
            grows = good && now != was;
            if (!grows) s_old[tid] = now;   // no rescaling
            s_new[tid] = now;
        }
        const bool grown = __syncthreads_or(grows);
        if (rh < nh) {
            const float inv = 1.f / s_new[rh];
            uint2 *dst = reinterpret_cast<uint2 *>(pool + ((size_t)(held + rt) * H + hb + rh) * kHeadDim);
            dst[c0] = to_e4m3x8(x, inv);
            dst[c1] = to_e4m3x8(x + 8, inv);
        }
        if (grown)   // held rows (head, token) over the slots
            for (int row = slot; row < nh * held; row += kPassRows) {
                const int h = row / held, tok = row - h * held;
                if (s_old[h] == s_new[h]) continue;
                const float ratio = s_old[h] / s_new[h];
                uint4 *w = reinterpret_cast<uint4 *>(pool + ((size_t)tok * H + hb + h) * kHeadDim) + j;
                uint4 c = *w;
                c.x = rescale_e4m3x4(c.x, ratio);
                c.y = rescale_e4m3x4(c.y, ratio);
                c.z = rescale_e4m3x4(c.z, ratio);
                c.w = rescale_e4m3x4(c.w, ratio);
                *w = c;
            }
        __syncthreads();   // the shared words of this pass are free
    }
    if (err) set_err(kv.dev_err, err);
    // the coarse key of the block that the tile's last new token ends
    const int end = it.t0 + held + cnt;                          // position behind it
    const bool ends_block = end == it.len || (end & ((1 << kv.block_shift) - 1)) == 0;
    if (!it.is_v && it.h_begin == 0 && kv.kc_new && ends_block && tid < kIdxDim / 16)
        reinterpret_cast<int4 *>(kv.kc_pool)[(size_t)it.page * (kIdxDim / 16) + tid] =
            ld_ordered(reinterpret_cast<const int4 *>(kv.kc_new) + (size_t)(it.i0 + cnt - 1) * (kIdxDim / 16) + tid);
}

}  // namespace

// kEarly: the whole grid is its first wave
template <bool kEarly>
__global__ void __launch_bounds__(kThreads, kRopeCtas) kv_append_rope_kernel(AppendRopeArgs a) {
    __shared__ RopeTab s_tab[2];
    pdl_trigger();
    token_rows<true>(a, blockIdx.x, threadIdx.x, kEarly, s_tab);
}

__global__ void __launch_bounds__(kTileThreads, kTileCtas) kv_append_fp8_kernel(AppendRopeArgs a) {
    __shared__ RopeTab s_tab[kBlockSize];
    pdl_trigger();
    // append and query CTAs in turn as long as there are both: the former wait on
    // latencies (tables, maxima), the latter on memory
    const int b = blockIdx.x, both = min(a.tile_ctas, (int)gridDim.x - a.tile_ctas);
    const bool appends = b < 2 * both ? !(b & 1) : a.tile_ctas > both;
    const int i = b < 2 * both ? b >> 1 : b - both;
    const bool early = b < kSms * kTileCtas;
    if (appends) {
        tile_rows(a, i, early, s_tab);
    } else {   // a query per half of the CTA
        const int half = threadIdx.x / kThreads;
        token_rows<false>(a, 2 * i + half, threadIdx.x % kThreads, early, s_tab + 2 * half);
    }
    // also where a CTA had nothing to do: whatever waits for this kernel waits
    // for the kernels ahead of it too
    pdl_wait();
}

cudaError_t launch_kv_append_rope(const AppendRopeArgs &a, cudaStream_t stream) {
    const int ctas = a.kv.total_new > a.total_q ? a.kv.total_new : a.total_q;
    if (ctas == 0) return cudaSuccess;
    return launch_pdl(ctas <= kSms * kRopeCtas ? kv_append_rope_kernel<true> : kv_append_rope_kernel<false>, dim3(ctas),
                      dim3(kThreads), 0, stream, a);
}

cudaError_t launch_kv_append_fp8(const AppendRopeArgs &a, cudaStream_t stream) {
    const long long ctas = (long long)a.tile_ctas + (a.total_q + 1ll) / 2;
    if (ctas == 0) return cudaSuccess;
    return launch_pdl(kv_append_fp8_kernel, dim3((unsigned)ctas), dim3(kTileThreads), 0, stream, a);
}

}  // namespace dsa
