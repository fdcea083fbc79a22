// kvq_tree.cuh -- attention of drafted tokens over a cache: the kernel.
//
// The rows of one (sequence, KV head) are its nodes * gqa queries, cut into row tiles of N
// columns; its tokens -- the packed ones, then the unpacked ones (the bf16 window, the drafts)
// -- into tiles of up to 128.  Per tile, on the tensor cores,
//   S^T [128 tokens x N]   = K [128 x D] Q^T [D x N]
//   O^T [D x N]           += V^T [D x 128] P [128 x N]
// with the tokens (and the channels) on the instruction's M side, so that its cost follows the
// number of queries, 16 to 128, and a cache byte is dequantised once for all of them.  A
// thread owns a token (a TMEM lane of S^T) and half of the columns.
//
// Softmax, in base 2.  A token's value row is stored in binary16 as v 2^-e (or as its code),
// v = stored * s; the weight that multiplies it is P = 2^(x + log2 s - m) with a running
// reference m per column: 8 under the largest x + log2 s seen, so that P <= 2^8 and weights
// down to 2^-22 of the largest keep binary16's 11 bits.  m moves only when some entry of a
// tile reaches 2^15 above it (every first tile; hardly ever later): then O^T is rescaled in
// TMEM.  The sum l takes P / s in binary32, per thread, and is joined at the end; O / l is the
// output.  A masked entry has x = -infinity and takes no part in anything.
#pragma once

#include <cuda_fp8.h>

#include "kvq_elements.cuh"
#include "kvq_internal.cuh"
#include "kvq_rope_angle.cuh"
#include "kvq_tcgen05.cuh"

namespace kvq {

constexpr int kTreeThreads = 256;
constexpr int kMaxTreeBlocks = 608;     // of a launch: bounds the workspace's partial results
constexpr float kNoMax = -1.0e30f;      // reference of a column that has seen nothing
constexpr float kHead = 8.0f;           // P of the largest entry, log2
constexpr float kReach = 15.0f;         // P may grow to 2^15 before the reference moves

struct TreeArgs {
    Layout lo;
    const uint8_t* cache;
    int layer, nodes, rows, RT;         // rows = nodes * gqa, RT row tiles of N columns
    int gshift;                         // log2 gqa
    int NB;                             // blocks of the launch
    int TT;                             // tokens of a full packed tile
    int staged;                         // the packed bytes of a tile pass through shared memory
    const __nv_bfloat16 *q, *k, *v;
    const uint8_t* mask;
    const int32_t* n_nodes;
    float qscale;                       // softmax scale * log2 e
    __nv_bfloat16* out;
    uint8_t* ws;
    int64_t ml_off, o_off;              // partials in the workspace: (m, l), then O
    float rope_w[128];
};

// Where a block's share lies: sequence, KV head, row tile, and the tile in it.
struct TreeSeq {
    int n, qn, nodes, packed, tiles, live;   // live: row tiles with queries in them
};
__device__ __forceinline__ TreeSeq tree_seq(const TreeArgs& a, int b, int N) {
    const int32_t* st = state_ptr(a.lo, a.cache, a.layer, b);
    TreeSeq s;
    s.n = st[0];
    s.qn = st[1];
    s.nodes = a.n_nodes ? a.n_nodes[b] : a.nodes;
    s.nodes = s.nodes < 0 ? 0 : (s.nodes > a.nodes ? a.nodes : s.nodes);
    s.packed = (s.qn + a.TT - 1) / a.TT;
    s.tiles = s.packed + (s.n - s.qn + s.nodes + 127) / 128;
    s.live = ((s.nodes << a.gshift) + N - 1) / N;
    return s;
}
// Tiles of all the row tiles of one KV head of a sequence (a row tile without queries is one
// empty tile: its outputs are set to 0).
__device__ __forceinline__ int64_t tree_head_tiles(const TreeArgs& a, const TreeSeq& s) {
    return (int64_t)s.live * s.tiles + (a.RT - s.live);
}

// Exclusive place of this thread's value in the block's sum, and the sum.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* tmp, int64_t* sum) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) tmp[warp] = x;
    __syncthreads();
    int64_t before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kTreeThreads / 32; ++w) {
        if (w < warp) before += tmp[w];
        all += tmp[w];
    }
    *sum = all;
    return before + x - v;
}

// All tiles of the launch.
__device__ __forceinline__ int64_t tree_total(const TreeArgs& a, int N, int64_t* tmp) {
    int64_t total = 0;
    for (int b0 = 0; b0 < a.lo.B; b0 += kTreeThreads) {
        const int b = b0 + threadIdx.x;
        int64_t sum;
        block_scan(b < a.lo.B ? a.lo.H * tree_head_tiles(a, tree_seq(a, b, N)) : 0, tmp, &sum);
        total += sum;
    }
    return total;
}

// Index of (token row, 16-byte chunk) in an operand tile.
__device__ __forceinline__ uint32_t core_at(int row, int chunk, uint32_t sbo) {
    return (row >> 3) * sbo + chunk * kCoreBytes + (row & 7) * 16;
}
// Order of the tokens of packed KIVI and FP8 tiles: row r of a tile's 16 is token
// (r & 1) * 8 + r / 2 (the order of the value codes and parameters of the records).
__device__ __forceinline__ int packed_token(int row) { return (row & ~15) + ((row & 1) << 3) + ((row & 15) >> 1); }
__device__ __forceinline__ int packed_row(int token) { return (token & ~15) + 2 * (token & 7) + ((token & 15) >> 3); }

// The channels of a key row are kept in the order in which two codes come out of one word of
// the packed row: KIVI, INT8 and INT4 blocks of W = 16, 8 or 4 channels (2, 4 or 8 bits),
// (i, i + W / 2) adjacent; FP8 quarters as the record has them.
__device__ __forceinline__ int key_block(const Layout& lo) {
    if (is_fp8(lo.scheme)) return 0;
    const int bits = lo.scheme == KVQ_SCHEME_KIVI ? lo.bits : (lo.scheme == KVQ_SCHEME_INT8 ? 8 : 4);
    return 32 / bits;
}
__device__ __forceinline__ int channel_place(int c, int W, int D) {
    if (W == 0) {
        const int r = c & 15;
        return ((r & 7) >> 1) * (D / 4) + 4 * (c >> 4) + 2 * (r >> 3) + (r & 1);
    }
    const int i = c & (W - 1), half = W >> 1;
    return (c & ~(W - 1)) + (i < half ? 2 * i : 2 * (i - half) + 1);
}
__device__ __forceinline__ int place_channel(int p, int W, int D) {
    if (W == 0) {
        const int quarter = p / (D / 4), x = p % (D / 4);
        return 16 * (x >> 2) + 2 * quarter + (x & 1) + 8 * ((x >> 1) & 1);
    }
    const int i = p & (W - 1);
    return (p & ~(W - 1)) + (i >> 1) + (i & 1) * (W >> 1);
}
// Eight words of 16 channels in natural order into the pairs' order.
__device__ __forceinline__ void pair_words(const uint32_t (&w)[8], int W, uint32_t (&o)[8]) {
    if (W == 16) {
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = prmt(w[i / 2], w[4 + i / 2], i & 1 ? 0x7632 : 0x5410);
    } else if (W == 8) {
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = prmt(w[(i & 4) + (i & 3) / 2], w[(i & 4) + 2 + (i & 3) / 2], i & 1 ? 0x7632 : 0x5410);
    } else if (W == 4) {
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = prmt(w[i & 6], w[(i & 6) + 1], i & 1 ? 0x7632 : 0x5410);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = w[i];
    }
}
// Stores 16 channels of a key (or query) row: 8 words in natural order.
template <int D>
__device__ __forceinline__ void store_unit(uint8_t* tile, int row, int unit, const uint32_t (&w)[8], int W) {
    constexpr uint32_t sbo = D / 8 * kCoreBytes;
    if (W != 0) {
        uint32_t o[8];
        pair_words(w, W, o);
        *reinterpret_cast<uint4*>(tile + core_at(row, 2 * unit, sbo)) = make_uint4(o[0], o[1], o[2], o[3]);
        *reinterpret_cast<uint4*>(tile + core_at(row, 2 * unit + 1, sbo)) = make_uint4(o[4], o[5], o[6], o[7]);
    } else {
        // channels 2i, 2i + 1, 2i + 8, 2i + 9 to quarter i, places 4 unit ..
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int p = i * (D / 4) + 4 * unit;
            *reinterpret_cast<uint2*>(tile + core_at(row, p >> 3, sbo) + (p & 7) * 2) = make_uint2(w[i], w[i + 4]);
        }
    }
}

__device__ __forceinline__ uint32_t hfma2u(uint32_t a, uint32_t b, uint32_t c) {
    return h2_as_u32(__hfma2(u32_as_h2(a), u32_as_h2(b), u32_as_h2(c)));
}
__device__ __forceinline__ constexpr uint32_t dup16(uint32_t h) { return h | (h << 16); }
// Codes of two halves of a word at bit POS (+ 16) as exact binary16 numbers: 1024 + code *
// 2^POS is one AND and one OR, and one fused multiply-add takes the code out of it.
template <int BITS, int POS>
__device__ __forceinline__ uint32_t code_pair(uint32_t x) {
    constexpr uint32_t mask = ((1u << BITS) - 1) << POS;
    constexpr uint32_t mul = (15 - POS) << 10;                 // 2^-POS
    constexpr uint32_t add = 0x8000u | ((25 - POS) << 10);     // -1024 * 2^-POS
    return hfma2u((x & dup16(mask)) | 0x64006400u, dup16(mul), dup16(add));
}
// The 16 codes of a unit (BITS / 2 words) as 8 pairs, in the pairs' order.
template <int BITS>
__device__ __forceinline__ void unit_codes(const uint32_t (&x)[4], uint32_t (&c)[8]) {
    if (BITS == 2) {
        const uint32_t y = x[0] >> 8;
        c[0] = code_pair<2, 0>(x[0]); c[1] = code_pair<2, 2>(x[0]); c[2] = code_pair<2, 4>(x[0]); c[3] = code_pair<2, 6>(x[0]);
        c[4] = code_pair<2, 0>(y); c[5] = code_pair<2, 2>(y); c[6] = code_pair<2, 4>(y); c[7] = code_pair<2, 6>(y);
    } else if (BITS == 4) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t y = x[i] >> 8;
            c[4 * i] = code_pair<4, 0>(x[i]); c[4 * i + 1] = code_pair<4, 4>(x[i]);
            c[4 * i + 2] = code_pair<4, 0>(y); c[4 * i + 3] = code_pair<4, 4>(y);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            c[2 * i] = code_pair<8, 0>(x[i]);
            c[2 * i + 1] = code_pair<8, 0>(x[i] >> 8);
        }
    }
}

// One packed tile: its groups' records (KIVI), or its rows (the other schemes).
struct PackedTile {
    const uint8_t* base;          // staged: the records one after another, or the rows
    int stride;
    const uint8_t* const* recs;   // not staged: the records' places (base is NULL)
    const uint8_t* codes[2];      // others: key rows and value rows (FP8: value tiles) of the tile
    const float* scales[2];       // INT8, INT4
    int cnt;                      // tokens
    __device__ __forceinline__ const uint8_t* rec(int g) const { return base ? base + g * stride : recs[g]; }
};

// KIVI keys.  A warp takes 64 channels of 2 D / 64 octets of rows; a lane 16 channels of one row
// of each octet, with the group's scales and zeros of its channels in registers.  x = code * s +
// z is one binary16 fused multiply-add of exact operands: rounded once.
template <int D, int BITS>
__device__ __forceinline__ void kivi_keys(const Layout& lo, const PackedTile& t, uint8_t* kt) {
    constexpr int QUADS = D / 64;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int unit = (warp % QUADS) * 4 + (lane >> 3), o0 = (warp / QUADS) * 2 * QUADS;
    uint32_t s[8], z[8];
    int have = -1;
#pragma unroll 2
    for (int o = o0; o < o0 + 2 * QUADS; ++o) {
        const int row = 8 * o + (lane & 7), tok = packed_token(row);
        if (8 * (o & ~1) >= t.cnt) break;
        const int g = (8 * (o & ~1)) / lo.G, tin = tok - g * lo.G;
        const uint8_t* rec = t.rec(g);
        if (g != have) {
            have = g;
            const uint4* ps = reinterpret_cast<const uint4*>(rec + lo.kc + lo.vc + 32 * unit);
            const uint4* pz = reinterpret_cast<const uint4*>(rec + lo.kc + lo.vc + 2 * D + 32 * unit);
            const uint4 s0 = ps[0], s1 = ps[1], z0 = pz[0], z1 = pz[1];
            const uint32_t sw[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
            const uint32_t zw[8] = {z0.x, z0.y, z0.z, z0.w, z1.x, z1.y, z1.z, z1.w};
            pair_words(sw, 32 / BITS, s);
            pair_words(zw, 32 / BITS, z);
        }
        uint32_t x[4] = {}, c[8];
        const uint8_t* src = rec + tin * (D * BITS / 8) + unit * (2 * BITS);
        if (BITS == 2) {
            x[0] = *reinterpret_cast<const uint32_t*>(src);
        } else if (BITS == 4) {
            const uint2 v = *reinterpret_cast<const uint2*>(src);
            x[0] = v.x; x[1] = v.y;
        } else {
            const uint4 v = *reinterpret_cast<const uint4*>(src);
            x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
        }
        unit_codes<BITS>(x, c);
#pragma unroll
        for (int i = 0; i < 8; ++i) c[i] = hfma2u(c[i], s[i], z[i]);
        constexpr uint32_t sbo = D / 8 * kCoreBytes;
        *reinterpret_cast<uint4*>(kt + core_at(row, 2 * unit, sbo)) = make_uint4(c[0], c[1], c[2], c[3]);
        *reinterpret_cast<uint4*>(kt + core_at(row, 2 * unit + 1, sbo)) = make_uint4(c[4], c[5], c[6], c[7]);
    }
}

// KIVI values, [channel][token] (K-major): a thread takes one word pair index of two adjacent
// lanes' codes, four tokens 4 ip .. and their partners 8 later, over 16 / BITS channels.
template <int D, int BITS>
__device__ __forceinline__ void kivi_values(const Layout& lo, const PackedTile& t, uint8_t* vt) {
    constexpr int HW = 16 / BITS, WPL = D * BITS / 64, SW = WPL < 4 ? WPL : 4;
    const int g8 = threadIdx.x & 7, ip = (threadIdx.x >> 3) & 1;
    for (int it = threadIdx.x >> 4; it < 8 * (WPL / 2); it += kTreeThreads / 16) {
        const int a = it / (WPL / 2), mm = it % (WPL / 2);     // 16-token tile, word pair
        if (16 * a >= t.cnt) break;
        const int g = 16 * a / lo.G, ti = 16 * a - g * lo.G;   // group, first token in it
        const uint8_t* rec = t.rec(g);
        const int w = 2 * mm;
        const uint8_t* src = rec + lo.kc + 4 * ((ti / 16) * 32 * WPL + (w / SW) * 32 * SW + (4 * g8 + 2 * ip) * SW + w % SW);
        const uint2 lo2 = *reinterpret_cast<const uint2*>(src), hi2 = *reinterpret_cast<const uint2*>(src + 4 * SW);
        const uint32_t x[4] = {lo2.x, lo2.y, hi2.x, hi2.y};    // tokens 4 ip + 0 .. 3 (and + 8)
        const uint8_t* par = rec + lo.kc + lo.vc + lo.kp + 2 * (ti + 8 * ip);
        uint4 s, z;
        int have = -1;
#pragma unroll
        for (int m = 0; m < HW; ++m) {
            const int j = mm * HW + m, c = 16 * (j >> 1) + g8 + 8 * (j & 1);
            const int gv = c / lo.Gv;
            if (gv != have) {
                have = gv;
                s = *reinterpret_cast<const uint4*>(par + 2 * gv * lo.G);
                z = *reinterpret_cast<const uint4*>(par + 2 * (lo.NGv + gv) * lo.G);
            }
            uint32_t y[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (BITS == 2)
                    y[i] = m == 0 ? code_pair<2, 0>(x[i]) : m == 1 ? code_pair<2, 2>(x[i]) : m == 2 ? code_pair<2, 4>(x[i])
                         : m == 3 ? code_pair<2, 6>(x[i]) : m == 4 ? code_pair<2, 0>(x[i] >> 8)
                         : m == 5 ? code_pair<2, 2>(x[i] >> 8) : m == 6 ? code_pair<2, 4>(x[i] >> 8)
                                  : code_pair<2, 6>(x[i] >> 8);
                else if (BITS == 4)
                    y[i] = m == 0 ? code_pair<4, 0>(x[i]) : m == 1 ? code_pair<4, 4>(x[i])
                         : m == 2 ? code_pair<4, 0>(x[i] >> 8) : code_pair<4, 4>(x[i] >> 8);
                else
                    y[i] = m == 0 ? code_pair<8, 0>(x[i]) : code_pair<8, 0>(x[i] >> 8);
            }
            *reinterpret_cast<uint4*>(vt + core_at(c, 2 * a + ip, 16 * kCoreBytes)) =
                make_uint4(hfma2u(y[0], s.x, z.x), hfma2u(y[1], s.y, z.y), hfma2u(y[2], s.z, z.z), hfma2u(y[3], s.w, z.w));
        }
    }
}

// Largest |value| that the keys (kv = 0) or values of the tile's groups can have, over this
// thread's share of their parameters; what is not finite is left out.
__device__ __forceinline__ float kivi_bound(const Layout& lo, const PackedTile& t, int kv) {
    const float levels = static_cast<float>((1 << lo.bits) - 1);
    const int pairs = kv ? lo.NGv * lo.G : lo.D;
    float top = 0.0f;
    for (int g = 0; g * lo.G < t.cnt; ++g) {
        const __half* par = reinterpret_cast<const __half*>(t.rec(g) + lo.kc + lo.vc + (kv ? lo.kp : 0));
        const uint32_t* side = reinterpret_cast<const uint32_t*>(t.rec(g) + lo.kc + lo.vc + lo.kp + lo.vp + (kv ? lo.ko : 0));
        for (int i = 2 * threadIdx.x; i < pairs; i += 2 * kTreeThreads) {
            const float2 s = __half22float2(*reinterpret_cast<const __half2*>(par + i));
            const float2 z = __half22float2(*reinterpret_cast<const __half2*>(par + pairs + i));
            const float x = fmaf(levels, s.x, fabsf(z.x)), y = fmaf(levels, s.y, fabsf(z.y));
            top = fmaxf(top, fmaxf(x < INFINITY ? x : 0.0f, y < INFINITY ? y : 0.0f));
        }
        for (int i = threadIdx.x; i < lo.K * pairs; i += kTreeThreads) {
            const float x = fabsf(__uint_as_float(side[i] & 0xffff0000u));
            top = fmaxf(top, x < INFINITY ? x : 0.0f);
        }
    }
    return top;
}

// The same tile where binary16 does not hold its values: element by element, times `scale`.
template <int D>
__device__ void kivi_keys_scaled(const Layout& lo, const PackedTile& t, uint8_t* kt, float scale, int W) {
    for (int i = threadIdx.x; i < 128 * D; i += kTreeThreads) {
        const int row = i / D, c = i % D, tok = packed_token(row);
        if (tok >= t.cnt) continue;
        const uint8_t* rec = t.rec(tok / lo.G);
        const __half* par = reinterpret_cast<const __half*>(rec + lo.kc + lo.vc);
        const int bit = ((tok % lo.G) * D + c) * lo.bits;
        const float x = scaled_code((rec[bit >> 3] >> (bit & 7)) & ((1 << lo.bits) - 1), __half2float(par[c]),
                                    __half2float(par[D + c]));
        const int p = channel_place(c, W, D);
        *reinterpret_cast<__half*>(kt + core_at(row, p >> 3, D / 8 * kCoreBytes) + (p & 7) * 2) = __float2half_rn(x * scale);
    }
}
template <int D>
__device__ void kivi_values_scaled(const Layout& lo, const PackedTile& t, uint8_t* vt, float scale) {
    for (int i = threadIdx.x; i < 128 * D; i += kTreeThreads) {
        const int tok = i / D, c = i % D;
        if (tok >= t.cnt) continue;
        const uint8_t* rec = t.rec(tok / lo.G);
        const int tin = tok % lo.G, pi = record_value_param(lo, tin, c), bit = record_value_bit(lo, tin, c);
        const __half* par = reinterpret_cast<const __half*>(rec + lo.kc + lo.vc + lo.kp);
        const float x = scaled_code((rec[lo.kc + (bit >> 3)] >> (bit & 7)) & ((1 << lo.bits) - 1), __half2float(par[pi]),
                                    __half2float(par[lo.G * lo.NGv + pi]));
        const int row = packed_row(tok);
        *reinterpret_cast<__half*>(vt + core_at(c, row >> 3, 16 * kCoreBytes) + (row & 7) * 2) = __float2half_rn(x * scale);
    }
}
// The side lists' elements over the dense ones.
template <int D>
__device__ void kivi_outliers(const Layout& lo, const PackedTile& t, uint8_t* tile, int kv, float scale, int W) {
    const int per = kv ? lo.NGv * lo.G : D;
    for (int g = 0; g * lo.G < t.cnt; ++g) {
        const uint32_t* side = reinterpret_cast<const uint32_t*>(t.rec(g) + lo.kc + lo.vc + lo.kp + lo.vp + (kv ? lo.ko : 0));
        for (int i = threadIdx.x; i < lo.K * per; i += kTreeThreads) {
            const uint32_t e = side[i];
            const int idx = static_cast<int>(e & 0xffffu), at = i % per;
            const __half x = __float2half_rn(__uint_as_float(e & 0xffff0000u) * scale);
            if (kv) {
                const int row = g * lo.G + at % lo.G, c = at / lo.G * lo.Gv + idx;
                *reinterpret_cast<__half*>(tile + core_at(c, row >> 3, 16 * kCoreBytes) + (row & 7) * 2) = x;
            } else {
                const int row = packed_row(g * lo.G + idx), p = channel_place(at, W, D);
                *reinterpret_cast<__half*>(tile + core_at(row, p >> 3, D / 8 * kCoreBytes) + (p & 7) * 2) = x;
            }
        }
    }
}

// FP8 keys and values: every code is a binary16 number.
__device__ __forceinline__ uint32_t fp8_pair(uint32_t two, bool e4m3) {
    uint32_t r;
    if (e4m3)
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(two)));
    else
        asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(two)));
    return r;
}
__device__ __forceinline__ void fp8_16(const uint4& v, bool e4m3, uint32_t (&o)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        o[2 * i] = fp8_pair(w[i] & 0xffffu, e4m3);
        o[2 * i + 1] = fp8_pair(w[i] >> 16, e4m3);
    }
}
template <int D>
__device__ __forceinline__ void fp8_keys(const PackedTile& t, bool e4m3, uint8_t* kt) {
    constexpr uint32_t sbo = D / 8 * kCoreBytes;
    for (int i = threadIdx.x; i < 128 * D / 16; i += kTreeThreads) {
        const int row = (i & 7) + 8 * (i / (D / 2)), unit = (i >> 3) % (D / 16), tok = packed_token(row);
        if ((row & ~15) >= t.cnt) break;
        uint32_t o[8];
        fp8_16(*reinterpret_cast<const uint4*>(t.codes[0] + tok * D + 16 * unit), e4m3, o);
        *reinterpret_cast<uint4*>(kt + core_at(row, 2 * unit, sbo)) = make_uint4(o[0], o[1], o[2], o[3]);
        *reinterpret_cast<uint4*>(kt + core_at(row, 2 * unit + 1, sbo)) = make_uint4(o[4], o[5], o[6], o[7]);
    }
}
template <int D>
__device__ __forceinline__ void fp8_values(const PackedTile& t, bool e4m3, bool negative, uint8_t* vt) {
    for (int i = threadIdx.x; i < 8 * D; i += kTreeThreads) {
        const int c = i % D, a = i / D;
        if (16 * a >= t.cnt) break;
        uint32_t o[8];
        fp8_16(*reinterpret_cast<const uint4*>(t.codes[1] + (16 * a * D + 16 * c)), e4m3, o);
        if (negative) {                     // the value scale's sign (its size goes to the weights)
#pragma unroll
            for (int r = 0; r < 8; ++r) o[r] ^= 0x80008000u;
        }
        if (16 * a + 16 > t.cnt) {          // tokens that the cache does not hold: any bytes
#pragma unroll
            for (int r = 0; r < 16; ++r)
                if (packed_token(16 * a + r) >= t.cnt) o[r / 2] &= r & 1 ? 0x0000ffffu : 0xffff0000u;
        }
        *reinterpret_cast<uint4*>(vt + core_at(c, 2 * a, 16 * kCoreBytes)) = make_uint4(o[0], o[1], o[2], o[3]);
        *reinterpret_cast<uint4*>(vt + core_at(c, 2 * a + 1, 16 * kCoreBytes)) = make_uint4(o[4], o[5], o[6], o[7]);
    }
}

// INT8 and INT4 rows: the codes as exact binary16 numbers (the scales go to the scores and the
// weights); keys K-major, values with their channels inside a row (MN-major).
template <int D>
__device__ __forceinline__ void rows_codes(const PackedTile& t, int kv, bool int8, uint8_t* tile) {
    for (int i = threadIdx.x; i < 128 * D / 16; i += kTreeThreads) {
        const int row = (i & 7) + 8 * (i / (D / 2)), unit = (i >> 3) % (D / 16);
        if ((row & ~15) >= t.cnt) break;
        uint32_t o[8] = {};
        if (row < t.cnt) {
            if (int8) {
                const uint4 v = *reinterpret_cast<const uint4*>(t.codes[kv] + row * D + 16 * unit);
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {       // code + 128 as an unsigned byte, less 1152
                    const uint32_t x = w[j] ^ 0x80808080u;
                    o[2 * j] = hfma2u((x & 0x00ff00ffu) | 0x64006400u, 0x3c003c00u, 0xe480e480u);
                    o[2 * j + 1] = hfma2u(((x >> 8) & 0x00ff00ffu) | 0x64006400u, 0x3c003c00u, 0xe480e480u);
                }
            } else {
                const uint2 v = *reinterpret_cast<const uint2*>(t.codes[kv] + row * (D / 2) + 8 * unit);
                const uint32_t w[2] = {v.x, v.y};
#pragma unroll
                for (int j = 0; j < 8; ++j) {       // code + 8 as an unsigned nibble, less 1032
                    const uint32_t x = (w[j / 4] ^ 0x88888888u) >> (4 * (j & 3));
                    o[j] = hfma2u((x & 0x000f000fu) | 0x64006400u, 0x3c003c00u, 0xe408e408u);
                }
            }
        }
        const uint4 a = make_uint4(o[0], o[1], o[2], o[3]), b = make_uint4(o[4], o[5], o[6], o[7]);
        if (kv == 0) {
            constexpr uint32_t sbo = D / 8 * kCoreBytes;
            *reinterpret_cast<uint4*>(tile + core_at(row, 2 * unit, sbo)) = a;
            *reinterpret_cast<uint4*>(tile + core_at(row, 2 * unit + 1, sbo)) = b;
        } else {
            uint8_t* at = tile + (row >> 3) * kCoreBytes + (row & 7) * 16 + 2 * unit * 16 * kCoreBytes;
            *reinterpret_cast<uint4*>(at) = a;
            *reinterpret_cast<uint4*>(at + 16 * kCoreBytes) = b;
        }
    }
}

// The exponent e of a power of two with |x| 2^-e < 2^14 for |x| <= top (top finite; under 2^-80
// it stays as there, which keeps the sums of P / s finite), and 2^e.
__device__ __forceinline__ int range_exponent(float top) {
    const int e = static_cast<int>((__float_as_uint(top) >> 23) & 255) - 127;
    return (e < -80 ? -80 : e) - 13;
}
__device__ __forceinline__ float pow2i(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

// (key scale, value scale) of an FP8 cache's KV head.
__device__ __forceinline__ const float* fp8_scale(const TreeArgs& a, int h) {
    return reinterpret_cast<const float*>(a.cache + a.lo.scales_off) + ((int64_t)a.layer * a.lo.H + h) * 2;
}

// 16 bf16 channels as binary16 pairs times 2^-e.  zero: what is not finite becomes 0.
__device__ __forceinline__ void half_words(const uint32_t (&w)[8], float f, bool zero, uint32_t (&o)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float x = __uint_as_float(w[i] << 16), y = __uint_as_float(w[i] & 0xffff0000u);
        if (zero) {
            x = fabsf(x) < INFINITY ? x : 0.0f;
            y = fabsf(y) < INFINITY ? y : 0.0f;
        }
        o[i] = h2_as_u32(__floats2half2_rn(x * f, y * f));
    }
}
// Largest finite |x| of 16 bf16 channels; *bad: one is not finite.
__device__ __forceinline__ float unit_top(const uint32_t (&w)[8], bool* bad) {
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float x = fabsf(__uint_as_float(w[i] << 16)), y = fabsf(__uint_as_float(w[i] & 0xffff0000u));
        *bad |= !(x < INFINITY) || !(y < INFINITY);
        top = fmaxf(top, fmaxf(x < INFINITY ? x : 0.0f, y < INFINITY ? y : 0.0f));
    }
    return top;
}
__device__ __forceinline__ void load_words(const uint16_t* p, uint32_t (&w)[8]) {
    const uint4 a = reinterpret_cast<const uint4*>(p)[0], b = reinterpret_cast<const uint4*>(p)[1];
    w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w; w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
}

// bf16 rows (the window's tokens, then the drafts) [r0, r0 + cnt) of unit (b, h): keys, values
// and their powers of two.  A warp takes an octet of rows, a lane 16 channels of one row at a
// time; each row is scaled by its own largest element.  *bad: a draft's value is not finite
// (it is 0 in the tile).
template <int D>
__device__ __forceinline__ void raw_rows(const TreeArgs& a, int b, int h, const TreeSeq& s, int r0, int cnt, int W,
                                         bool paired_values, uint8_t* kt, uint8_t* vt, float* kf, float* vlog,
                                         bool* bad) {
    constexpr int UNITS = D / 16, STEPS = (UNITS + 3) / 4;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int window = s.n - s.qn;
    for (int o = warp; o < 16; o += kTreeThreads / 32) {
        const int row = 8 * o + (lane & 7), r = r0 + row;
        if ((8 * o & ~15) >= cnt) break;
        const uint16_t *kp = nullptr, *vp = nullptr;
        if (row < cnt) {
            if (r < window) {
                kp = reinterpret_cast<const uint16_t*>(a.cache + a.lo.ring_off + (unit_index(a.lo, a.layer, b, h) * a.lo.C +
                                                                                 (s.qn + (int64_t)r) % a.lo.C) * (4 * D));
                vp = kp + D;
            } else {
                const int64_t at = (((int64_t)b * a.nodes + (r - window)) * a.lo.H + h) * D;
                kp = reinterpret_cast<const uint16_t*>(a.k) + at;
                vp = reinterpret_cast<const uint16_t*>(a.v) + at;
            }
        }
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
            const uint16_t* p = kv ? vp : kp;
            uint32_t w[STEPS][8];
            float top = 0.0f;
            bool odd = false;
#pragma unroll
            for (int i = 0; i < STEPS; ++i) {
                const int unit = (lane >> 3) + 4 * i;
#pragma unroll
                for (int j = 0; j < 8; ++j) w[i][j] = 0u;
                if (p && unit < UNITS) load_words(p + 16 * unit, w[i]);
                top = fmaxf(top, unit_top(w[i], &odd));
            }
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
            const int e = range_exponent(top);
            const float f = pow2i(-e);
            const bool draft = r >= window;
            if (kv && odd && draft) *bad = true;
#pragma unroll
            for (int i = 0; i < STEPS; ++i) {
                const int unit = (lane >> 3) + 4 * i;
                if (unit >= UNITS) continue;
                uint32_t hw[8];
                half_words(w[i], f, kv && draft, hw);
                if (kv == 0) {
                    store_unit<D>(kt, row, unit, hw, W);
                } else {
                    uint32_t pw[8];
                    pair_words(hw, paired_values ? W : 0, pw);
                    uint8_t* at = vt + (row >> 3) * kCoreBytes + (row & 7) * 16 + 2 * unit * 16 * kCoreBytes;
                    *reinterpret_cast<uint4*>(at) = make_uint4(pw[0], pw[1], pw[2], pw[3]);
                    *reinterpret_cast<uint4*>(at + 16 * kCoreBytes) = make_uint4(pw[4], pw[5], pw[6], pw[7]);
                }
            }
            if (lane < 8) {
                if (kv)
                    vlog[row] = static_cast<float>(e);
                else
                    kf[row] = pow2i(e);
            }
        }
    }
}

// Turns the tile's cached keys by their positions: row r of the tile is token t0 + (its place),
// rows from `rows` on stay.
template <int D>
__device__ void turn_keys(uint8_t* kt, const float* w, int64_t t0, int rows, bool packed_order) {
    constexpr uint32_t sbo = D / 8 * kCoreBytes;
    constexpr int CH = D / 16;                  // 8-channel chunks of half a row
    for (int i = threadIdx.x; i < 128 * CH; i += kTreeThreads) {
        const int row = (i & 7) + 8 * (i / (8 * CH)), ch = (i >> 3) % CH;
        const int tok = packed_order ? packed_token(row) : row;
        if (tok >= rows) continue;
        uint4* pa = reinterpret_cast<uint4*>(kt + core_at(row, ch, sbo));
        uint4* pb = reinterpret_cast<uint4*>(kt + core_at(row, ch + CH, sbo));
        const uint4 va = *pa, vb = *pb;
        const uint32_t x[4] = {va.x, va.y, va.z, va.w}, y[4] = {vb.x, vb.y, vb.z, vb.w};
        uint32_t ox[4], oy[4];
        const float pos = static_cast<float>(t0 + tok);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 fx = __half22float2(u32_as_h2(x[j])), fy = __half22float2(u32_as_h2(y[j]));
            float s0, c0, s1, c1;
            rope_sincos(__fmul_rn(pos, w[8 * ch + 2 * j]), &s0, &c0);
            rope_sincos(__fmul_rn(pos, w[8 * ch + 2 * j + 1]), &s1, &c1);
            ox[j] = h2_as_u32(__floats2half2_rn(fx.x * c0 - fy.x * s0, fx.y * c1 - fy.y * s1));
            oy[j] = h2_as_u32(__floats2half2_rn(fy.x * c0 + fx.x * s0, fy.y * c1 + fx.y * s1));
        }
        *pa = make_uint4(ox[0], ox[1], ox[2], ox[3]);
        *pb = make_uint4(oy[0], oy[1], oy[2], oy[3]);
    }
}

template <int N, int D>
struct TreeSmem {
    static constexpr int kVBytes = D > 128 ? 65536 : 32768;     // the product reads 128 channel rows
    static constexpr int kK = 0, kV = 256 * D, kQ = kV + kVBytes, kP = kQ + 2 * N * D, kStage = kP + 256 * N;
    static constexpr int kDN = D > 128 ? 2 : 1;                 // accumulators of 128 channels
    static constexpr uint32_t kCols = N * (1 + kDN) <= 32 ? 32 : N * (1 + kDN) <= 64 ? 64 : N * (1 + kDN) <= 128 ? 128
                                      : N * (1 + kDN) <= 256 ? 256 : 512;
    static constexpr int kBlocks = N >= 128 || D > 128 ? 1 : 2;
};

__device__ __forceinline__ float fast_log2(float x) {
    float r;
    asm("lg2.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float tree_exp2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float warp_max(float x) {
    float r;
    asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
    return r;
}

template <int N, int D>
__global__ void __launch_bounds__(kTreeThreads, TreeSmem<N, D>::kBlocks) k_tree(const __grid_constant__ TreeArgs a) {
    using S = TreeSmem<N, D>;
    constexpr int NH = N / 2;                       // columns of a thread
    constexpr int STEP = NH < 32 ? NH : 32;         // columns of one TMEM access
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ __align__(16) float2 col[N];         // (query scale, -reference) of a column
    __shared__ float fac[N], cmax[4][N], lsum[4][N], kf[128], vlog[128], wt[D / 2];
    __shared__ int64_t scan[8], start[4];
    __shared__ uint64_t bar_stage, bar_s, bar_pv;
    __shared__ uint32_t tmem_slot, top[2];
    __shared__ const uint8_t* recs[8];
    __shared__ int dead;

    const Layout& lo = a.lo;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, quad = warp & 3, half = warp >> 2;
    const int H = lo.H, gqa = lo.gqa, W = key_block(lo);
    uint8_t *kt = smem + S::kK, *vt = smem + S::kV, *qt = smem + S::kQ, *pt = smem + S::kP, *stage = smem + S::kStage;
    const bool kivi = lo.scheme == KVQ_SCHEME_KIVI, fp8 = is_fp8(lo.scheme), rows_scheme = is_rows(lo.scheme);
    const bool rope = lo.rope_base > 0.0f;
    const int64_t row_bytes = lo.scheme == KVQ_SCHEME_INT4 ? D / 2 : D;     // of a code row

    grid_dependency_wait();
    grid_launch_dependents();
    // this block's tiles: positions [x0, x1) of all tiles, in the order sequence, KV head, row
    // tile, tile
    const int64_t total = tree_total(a, N, scan);
    const int64_t nb = total < a.NB ? total : a.NB;     // blocks with a share
    if (blockIdx.x >= nb) return;
    const int64_t x0 = total * blockIdx.x / nb, x1 = total * (blockIdx.x + 1) / nb;
    {
        int64_t base = 0;
        for (int b0 = 0; b0 < lo.B; b0 += kTreeThreads) {
            const int b = b0 + tid;
            const int64_t w = b < lo.B ? H * tree_head_tiles(a, tree_seq(a, b, N)) : 0;
            int64_t sum;
            const int64_t at = base + block_scan(w, scan, &sum);
            if (at <= x0 && x0 < at + w) {
                start[0] = b;
                start[1] = x0 - at;
            }
            base += sum;
        }
    }
    if (warp == 0) tmem_alloc(&tmem_slot, S::kCols);
    if (tid == 32) {
        mbar_init(&bar_stage, 1);
        mbar_init(&bar_s, 1);
        mbar_init(&bar_pv, 1);
        dead = 0;
    }
    if (rope)
        for (int i = tid; i < D / 2; i += kTreeThreads) wt[i] = a.rope_w[place_channel(i, W, D)];
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    const uint32_t tm_s = tmem_slot, tm_o = tm_s + N;
    const uint32_t my_s = tm_s + (static_cast<uint32_t>(32 * quad) << 16) + half * NH;

    auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (*static_cast<volatile int*>(&dead)) return;
        if (!mbar_wait_bounded(bar, parity, kWaitLimitNs)) {
            dead = 1;
            atomicOr(reinterpret_cast<uint32_t*>(a.ws), KVQ_STATUS_TIMEOUT);
        }
    };
    // tile `tile` of (b, h) brought to the stage: thread 0
    auto issue = [&](int b, int h, int tile, int qn) {
        const int64_t t0 = (int64_t)tile * a.TT;
        const int cnt = static_cast<int>(qn - t0 < a.TT ? qn - t0 : a.TT);
        if (kivi) {
            const int ng = cnt / lo.G;
            mbar_arrive_expect_tx(&bar_stage, static_cast<uint32_t>(ng * lo.rec));
            if (lo.PG == 0) {
                bulk_copy_g2s(stage, a.cache + group_offset(lo, a.layer, b, h, t0 / lo.G), ng * lo.rec, &bar_stage);
            } else {
                for (int g = 0; g < ng; ++g) {
                    int64_t off = group_offset(lo, a.layer, b, h, t0 / lo.G + g);
                    if (off < 0) {      // a table entry outside the pool: page 0 in its place, reported
                        atomicOr(reinterpret_cast<uint32_t*>(a.ws), KVQ_STATUS_BAD_PAGE);
                        off = lo.data_off + (((int64_t)a.layer * H + h) * lo.PG + (t0 / lo.G + g) % lo.PG) * lo.rec;
                    }
                    bulk_copy_g2s(stage + g * lo.rec, a.cache + off, lo.rec, &bar_stage);
                }
            }
        } else {
            const int c16 = (cnt + 15) & ~15;
            const uint8_t* base = a.cache + lo.data_off + unit_index(lo, a.layer, b, h) * lo.unit;
            const uint32_t bytes = static_cast<uint32_t>(c16 * row_bytes);
            mbar_arrive_expect_tx(&bar_stage, 2 * bytes + (rows_scheme ? 8 * c16 : 0));
            bulk_copy_g2s(stage, base + t0 * row_bytes, bytes, &bar_stage);
            bulk_copy_g2s(stage + 128 * row_bytes, base + (lo.T16 + t0) * row_bytes, bytes, &bar_stage);
            if (rows_scheme) {
                const uint8_t* sc = base + 2 * (int64_t)lo.T16 * row_bytes;
                bulk_copy_g2s(stage + 256 * row_bytes, sc + 4 * t0, 4 * c16, &bar_stage);
                bulk_copy_g2s(stage + 256 * row_bytes + 512, sc + 4 * (lo.T16 + t0), 4 * c16, &bar_stage);
            }
        }
    };

    int b = static_cast<int>(start[0]), h, rt, tile;
    TreeSeq s = tree_seq(a, b, N);
    {
        const int64_t per = tree_head_tiles(a, s), in = start[1] % per;
        h = static_cast<int>(start[1] / per);
        if (in < (int64_t)s.live * s.tiles) {
            rt = static_cast<int>(in / s.tiles);
            tile = static_cast<int>(in % s.tiles);
        } else {
            rt = static_cast<int>(s.live + (in - (int64_t)s.live * s.tiles));
            tile = 0;
        }
    }
    uint32_t ph_stage = 0, ph_s = 0, ph_pv = 0;
    bool fetched = false;                       // the current tile is on its way to the stage
    bool pv_open = false;                       // a value product has not been waited for
    int64_t left = x1 - x0;

    while (left > 0) {
        // ------------------------------------------------------------ a segment: tiles [tile, end)
        const bool live = rt < s.live;
        const int unit_tiles = live ? s.tiles : 1;
        const int first = tile;
        const int end = static_cast<int>(left < unit_tiles - tile ? tile + left : unit_tiles);
        if (live && !fetched && first < s.packed && a.staged) {
            if (tid == 0) issue(b, h, first, s.qn);
            fetched = true;
        }
        const int row0 = rt * N, row_end = s.nodes << a.gshift;
        bool nonfinite = false;
        float l[NH];
#pragma unroll
        for (int i = 0; i < NH; ++i) l[i] = 0.0f;
        if (live) {
            // queries: a warp takes an octet of columns, a lane 16 channels at a time
            constexpr int UNITS = D / 16, STEPS = (UNITS + 3) / 4;
            for (int o = warp; o < N / 8; o += kTreeThreads / 32) {
                const int c = 8 * o + (lane & 7), r = row0 + c;
                const uint16_t* p = nullptr;
                if (r < row_end)
                    p = reinterpret_cast<const uint16_t*>(a.q) +
                        (((int64_t)b * a.nodes + (r >> a.gshift)) * lo.Hq + h * gqa + (r & (gqa - 1))) * D;
                uint32_t w[STEPS][8];
                float mx = 0.0f;
                bool odd = false;
#pragma unroll
                for (int i = 0; i < STEPS; ++i) {
                    const int unit = (lane >> 3) + 4 * i;
#pragma unroll
                    for (int j = 0; j < 8; ++j) w[i][j] = 0u;
                    if (p && unit < UNITS) load_words(p + 16 * unit, w[i]);
                    mx = fmaxf(mx, unit_top(w[i], &odd));
                }
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                const int e = range_exponent(mx);
                const float f = pow2i(-e);
#pragma unroll
                for (int i = 0; i < STEPS; ++i) {
                    const int unit = (lane >> 3) + 4 * i;
                    if (unit >= UNITS) continue;
                    uint32_t hw[8];
                    half_words(w[i], f, false, hw);
                    store_unit<D>(qt, c, unit, hw, W);
                }
                if (lane < 8) col[c] = make_float2(a.qscale * pow2i(e), -kNoMax);
            }
        }

        // ------------------------------------------------------------ tiles
        bool have_o = false;                    // O^T holds this segment's sum
        for (; tile < end; ++tile) {
            if (!live) continue;
            const bool packed = tile < s.packed;
            const int r0 = (tile - s.packed) * 128;                     // of the raw rows
            int cnt;
            PackedTile t;
            t.stride = lo.rec;
            t.recs = recs;
            if (packed) {
                const int64_t t0 = (int64_t)tile * a.TT;
                cnt = static_cast<int>(s.qn - t0 < a.TT ? s.qn - t0 : a.TT);
                if (a.staged) {
                    wait(&bar_stage, ph_stage);
                    ph_stage ^= 1;
                    fetched = false;
                    t.base = stage;
                    t.codes[0] = stage;
                    t.codes[1] = stage + 128 * row_bytes;
                    t.scales[0] = reinterpret_cast<const float*>(stage + 256 * row_bytes);
                    t.scales[1] = t.scales[0] + 128;
                } else {
                    // records too large to pass through shared memory next to the tiles
                    if (tid < 8 && tid * lo.G < cnt) {
                        int64_t off = group_offset(lo, a.layer, b, h, t0 / lo.G + tid);
                        if (off < 0) {
                            atomicOr(reinterpret_cast<uint32_t*>(a.ws), KVQ_STATUS_BAD_PAGE);
                            off = lo.data_off + (((int64_t)a.layer * H + h) * lo.PG + (t0 / lo.G + tid) % lo.PG) * lo.rec;
                        }
                        recs[tid] = a.cache + off;
                    }
                    __syncthreads();
                    t.base = nullptr;
                }
                t.cnt = cnt;
            } else {
                const int all = s.n - s.qn + s.nodes - r0;
                cnt = all < 128 ? all : 128;
            }
            const int steps = (cnt + 15) >> 4;                         // of 16 tokens
            float kscale = 1.0f, vscale = 1.0f;                        // KIVI: stored = value * scale
            int ke = 0, ve = 0;
            if (packed && kivi) {
                if (tid < 2) top[tid] = 0u;
                __syncthreads();
#pragma unroll
                for (int kv = 0; kv < 2; ++kv) {
                    const float m = warp_max(kivi_bound(lo, t, kv));
                    if (lane == 0) atomicMax(&top[kv], __float_as_uint(m));
                }
                __syncthreads();
                const float kb = __uint_as_float(top[0]), vb = __uint_as_float(top[1]);
                if (kb >= 32768.0f) {
                    ke = range_exponent(kb);
                    kscale = pow2i(-ke);
                }
                if (vb >= 32768.0f) {
                    ve = range_exponent(vb);
                    vscale = pow2i(-ve);
                }
            }
            // ---- keys (the previous tile's score product is done: its scores were read)
            if (!packed) {
                if (pv_open) {                                          // the rows write both tiles
                    wait(&bar_pv, ph_pv);
                    ph_pv ^= 1;
                    pv_open = false;
                }
                raw_rows<D>(a, b, h, s, r0, cnt, W, rows_scheme, kt, vt, kf, vlog, &nonfinite);
            } else if (kivi) {
                if (kscale != 1.0f)
                    kivi_keys_scaled<D>(lo, t, kt, kscale, W);
                else if constexpr (D >= 64) {
                    if (lo.bits == 2) kivi_keys<D, 2>(lo, t, kt);
                    else if (lo.bits == 4) kivi_keys<D, 4>(lo, t, kt);
                    else kivi_keys<D, 8>(lo, t, kt);
                }
                if (lo.K > 0) {
                    __syncthreads();
                    kivi_outliers<D>(lo, t, kt, 0, kscale, W);
                }
            } else if (fp8) {
                fp8_keys<D>(t, lo.scheme == KVQ_SCHEME_FP8_E4M3, kt);
            } else {
                rows_codes<D>(t, 0, lo.scheme == KVQ_SCHEME_INT8, kt);
            }
            if (rope) {
                __syncthreads();
                if (packed)
                    turn_keys<D>(kt, wt, (int64_t)tile * a.TT, cnt, true);
                else
                    turn_keys<D>(kt, wt, (int64_t)s.qn + r0, s.n - s.qn - r0 < cnt ? s.n - s.qn - r0 : cnt, false);
            }
            smem_to_async();
            tmem_fence_before();
            __syncthreads();
            if (tid == 0) {
                tmem_fence_after();
                const uint64_t da = mma_desc(smem_addr(kt), D / 8 * kCoreBytes), db = mma_desc(smem_addr(qt), D / 8 * kCoreBytes);
#pragma unroll
                for (int k = 0; k < D / 16; ++k)
                    mma_f16(tm_s, da + k * (2 * kCoreBytes >> 4), db + k * (2 * kCoreBytes >> 4),
                            mma_idesc(128, N, false, false), k > 0);
                mma_commit(&bar_s);
            }
            // ---- values, while the scores are computed
            if (pv_open) {
                wait(&bar_pv, ph_pv);
                ph_pv ^= 1;
                pv_open = false;
            }
            if (packed) {
                if (kivi) {
                    if (vscale != 1.0f)
                        kivi_values_scaled<D>(lo, t, vt, vscale);
                    else if constexpr (D >= 64) {
                        if (lo.bits == 2) kivi_values<D, 2>(lo, t, vt);
                        else if (lo.bits == 4) kivi_values<D, 4>(lo, t, vt);
                        else kivi_values<D, 8>(lo, t, vt);
                    }
                    if (lo.K > 0) {
                        __syncthreads();
                        kivi_outliers<D>(lo, t, vt, 1, vscale, W);
                    }
                } else if (fp8) {
                    fp8_values<D>(t, lo.scheme == KVQ_SCHEME_FP8_E4M3, fp8_scale(a, h)[1] < 0.0f, vt);
                } else {
                    rows_codes<D>(t, 1, lo.scheme == KVQ_SCHEME_INT8, vt);
                }
            }
            // ---- this thread's token: factor of its scores, log2 of its values' scale
            const int row = 32 * quad + lane;
            const int tok = packed && (kivi || fp8) ? packed_token(row) : row;
            const bool valid = tok < cnt;
            float f = 0.0f, lv = 0.0f;
            int draft = -1;
            if (valid) {
                if (!packed) {
                    f = kf[row];
                    lv = vlog[row];
                    draft = r0 + row - (s.n - s.qn);
                } else if (kivi) {
                    f = pow2i(ke);
                    lv = static_cast<float>(ve);
                } else if (fp8) {
                    const float* sc = fp8_scale(a, h);
                    f = sc[0];
                    lv = fast_log2(fabsf(sc[1]));
                } else {
                    f = t.scales[0][tok];
                    lv = fast_log2(t.scales[1][tok]);
                }
                lv = fmaxf(lv, -110.0f);        // (a scale of 0 belongs to codes of 0)
            }
            const float inv = tree_exp2(-lv);
            __syncthreads();                    // the stage is read: the next tile may come
            {
                // the next packed tile of this block, in this segment (the next segment's first
                // tile is fetched when it begins)
                if (a.staged && tile + 1 < end && tile + 1 < s.packed) {
                    if (tid == 0) issue(b, h, tile + 1, s.qn);
                    fetched = true;
                }
            }
            wait(&bar_s, ph_s);
            ph_s ^= 1;
            tmem_fence_after();
            // ---- softmax
            float x[NH];
#pragma unroll
            for (int c = 0; c < NH; c += STEP) {
                float y[STEP];
                tmem_load(my_s + c, y);
#pragma unroll
                for (int i = 0; i < STEP; ++i) x[c + i] = y[i];
            }
            float hi = kNoMax;
            const bool masked = cnt < 128 || !packed;
            if (masked) {
#pragma unroll
                for (int i = 0; i < NH; ++i) {
                    const int c = half * NH + i;
                    bool see = valid;
                    if (draft >= 0) {
                        const int r = row0 + c, node = r >> a.gshift;
                        see = r < row_end;
                        if (see) see = a.mask ? a.mask[((int64_t)b * a.nodes + node) * a.nodes + draft] != 0 : draft <= node;
                    }
                    const float2 g = col[c];
                    x[i] = see ? fmaf(x[i], f * g.x, lv) : -INFINITY;
                    hi = fmaxf(hi, x[i] + g.y);
                }
            } else {
#pragma unroll
                for (int i = 0; i < NH; ++i) {
                    const float2 g = col[half * NH + i];
                    x[i] = fmaf(x[i], f * g.x, lv);
                    hi = fmaxf(hi, x[i] + g.y);
                }
            }
            if (__syncthreads_or(hi > kReach)) {
                // the columns' maxima over the tile, and the new references
#pragma unroll
                for (int i = 0; i < NH; ++i) {
                    const float m = warp_max(x[i]);
                    if (lane == 0) cmax[quad][half * NH + i] = m;
                }
                __syncthreads();
                if (tid < N) {
                    const float m = fmaxf(fmaxf(cmax[0][tid], cmax[1][tid]), fmaxf(cmax[2][tid], cmax[3][tid])) - kHead;
                    const float old = -col[tid].y, now = fmaxf(old, m);
                    col[tid].y = -now;
                    fac[tid] = tree_exp2(old - now);
                }
                __syncthreads();
#pragma unroll
                for (int i = 0; i < NH; ++i) l[i] *= fac[half * NH + i];
                if (have_o) {
#pragma unroll
                    for (int d = 0; d < S::kDN; ++d)
#pragma unroll
                        for (int c = 0; c < NH; c += STEP) {
                            float o[STEP];
                            const uint32_t at = tm_o + d * N + (static_cast<uint32_t>(32 * quad) << 16) + half * NH + c;
                            tmem_load(at, o);
#pragma unroll
                            for (int i = 0; i < STEP; ++i) o[i] *= fac[half * NH + c + i];
                            tmem_store(at, o);
                        }
                }
            }
#pragma unroll
            for (int c = 0; c < NH; c += 8) {
                uint32_t p[4];
#pragma unroll
                for (int i = 0; i < 8; i += 2) {
                    const float p0 = tree_exp2(x[c + i] + col[half * NH + c + i].y);
                    const float p1 = tree_exp2(x[c + i + 1] + col[half * NH + c + i + 1].y);
                    l[c + i] = fmaf(p0, inv, l[c + i]);
                    l[c + i + 1] = fmaf(p1, inv, l[c + i + 1]);
                    p[i / 2] = h2_as_u32(__floats2half2_rn(p0, p1));
                }
                *reinterpret_cast<uint4*>(pt + ((half * NH + c) >> 3) * (16 * kCoreBytes) + (row >> 3) * kCoreBytes + (row & 7) * 16) =
                    make_uint4(p[0], p[1], p[2], p[3]);
            }
            smem_to_async();
            tmem_fence_before();
            __syncthreads();
            if (tid == 0) {
                tmem_fence_after();
                const bool mn = !packed || rows_scheme;                 // values with channels inside a row
                const uint64_t db = mma_desc(smem_addr(pt), 16 * kCoreBytes);
#pragma unroll
                for (int d = 0; d < S::kDN; ++d) {
                    const uint64_t da = mma_desc(smem_addr(vt) + d * 32768, 16 * kCoreBytes);
                    for (int k = 0; k < steps; ++k)
                        mma_f16(tm_o + d * N, da + k * (2 * kCoreBytes >> 4), db + k * (2 * kCoreBytes >> 4),
                                mma_idesc(128, N, mn, true), have_o || k > 0);
                }
                mma_commit(&bar_pv);
            }
            pv_open = true;
            have_o = true;
        }
        // ------------------------------------------------------------ the segment's result
        const bool whole = first == 0 && end == unit_tiles;
        const int64_t unit = ((int64_t)b * H + h) * a.RT + rt;
        const int64_t slot = blockIdx.x + unit;
        if (pv_open) {
            wait(&bar_pv, ph_pv);
            ph_pv ^= 1;
            pv_open = false;
        }
        tmem_fence_after();
        const bool odd = __syncthreads_or(nonfinite);
        // the sums over a column's tokens
#pragma unroll
        for (int i = 0; i < NH; ++i) {
            float v = l[i];
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
            if (lane == 0) lsum[quad][half * NH + i] = v;
        }
        __syncthreads();
        if (tid < N) {
            // rows of padding nodes saw the cached tokens with a query of 0: their output is 0
            const float v = live && row0 + tid < row_end ? (lsum[0][tid] + lsum[1][tid]) + (lsum[2][tid] + lsum[3][tid]) : 0.0f;
            if (whole) {
                fac[tid] = v != 0.0f ? 1.0f / v : 0.0f;
            } else {
                fac[tid] = v != 0.0f ? 1.0f : 0.0f;
                reinterpret_cast<float2*>(a.ws + a.ml_off)[slot * N + tid] = make_float2(-col[tid].y, v);
            }
        }
        __syncthreads();
#pragma unroll
        for (int d = 0; d < S::kDN; ++d) {
            const int ch0 = 128 * d + 32 * quad;
            if (ch0 >= D) continue;
            // lane -> channel: the order of the tile's value rows
            const int c0 = rows_scheme ? place_channel(ch0 + lane, W, D) : ch0 + lane;
#pragma unroll
            for (int c = 0; c < NH; c += STEP) {
                float o[STEP];
                if (live)
                    tmem_load(tm_o + d * N + (static_cast<uint32_t>(32 * quad) << 16) + half * NH + c, o);
#pragma unroll
                for (int i = 0; i < STEP; ++i) {
                    const int cc = half * NH + c + i, r = row0 + cc;
                    if (r >= a.rows) continue;
                    const float fc = fac[cc];
                    float v = fc != 0.0f ? o[i] * fc : 0.0f;
                    if (odd && r < row_end) {   // drafts whose value is not finite, in the rows that see them
                        const int node = r >> a.gshift;
                        for (int j = 0; j < s.nodes; ++j) {
                            const float y = __bfloat162float(a.v[(((int64_t)b * a.nodes + j) * H + h) * D + c0]);
                            if (fabsf(y) < INFINITY) continue;
                            if (a.mask ? a.mask[((int64_t)b * a.nodes + node) * a.nodes + j] != 0 : j <= node) v += y;
                        }
                    }
                    if (whole)
                        a.out[(((int64_t)b * a.nodes + (r >> a.gshift)) * lo.Hq + h * gqa + (r & (gqa - 1))) * D + c0] =
                            __float2bfloat16_rn(v);
                    else
                        reinterpret_cast<float*>(a.ws + a.o_off)[(slot * N + cc) * D + c0] = v;
                }
            }
        }
        tmem_fence_before();
        __syncthreads();
        tmem_fence_after();
        // ------------------------------------------------------------ the next unit
        left -= end - first;
        if (tile >= unit_tiles) {
            tile = 0;
            if (++rt == a.RT) {
                rt = 0;
                if (++h == H) {
                    h = 0;
                    ++b;
                    if (left > 0) s = tree_seq(a, b, N);
                }
            }
        }
    }
    __syncthreads();
    if (warp == 0) tmem_free(tm_s, S::kCols);
}

// Joins the partial results of row tiles that several blocks worked on.  A block takes CW
// columns of one row tile: it finds the blocks whose shares meet the row tile's tiles, and for
// each column sums their O 2^(m - M) and l 2^(m - M).
template <int N, int D>
__global__ void __launch_bounds__(kTreeThreads) k_tree_merge(const __grid_constant__ TreeArgs a) {
    constexpr int CW = N < 32 ? N / 2 : 16;
    __shared__ int64_t scan[8], start;
    const Layout& lo = a.lo;
    const int64_t unit = blockIdx.x / (N / CW);
    const int c0 = static_cast<int>(blockIdx.x % (N / CW)) * CW;
    const int rt = static_cast<int>(unit % a.RT);
    const int64_t bh = unit / a.RT;
    const int b = static_cast<int>(bh / lo.H), h = static_cast<int>(bh % lo.H);
    const int row0 = rt * N;
    // the token counts are not written by the attention: the plan needs no wait for it
    const int64_t total = tree_total(a, N, scan);
    int64_t base = 0;
    for (int b0 = 0; b0 <= b; b0 += kTreeThreads) {
        const int bb = b0 + threadIdx.x;
        int64_t sum;
        const int64_t at = base + block_scan(bb < lo.B ? lo.H * tree_head_tiles(a, tree_seq(a, bb, N)) : 0, scan, &sum);
        if (bb == b) start = at;
        base += sum;
    }
    __syncthreads();
    const TreeSeq s = tree_seq(a, b, N);
    const int64_t nb = total < a.NB ? total : a.NB;
    const int64_t y0 = start + h * tree_head_tiles(a, s) + (int64_t)rt * s.tiles, y1 = y0 + s.tiles;
    // block j has the positions [total j / nb, total (j + 1) / nb)
    int64_t j0 = y0 * nb / total, j1;
    while (total * (j0 + 1) / nb <= y0) ++j0;
    while (total * j0 / nb > y0) --j0;
    for (j1 = j0; total * (j1 + 1) / nb < y1;) ++j1;
    // every block waits, also one with nothing to join: the launch after this one may rely on it
    grid_dependency_wait();
    if (rt >= s.live || j0 == j1) return;
    const float2* ml = reinterpret_cast<const float2*>(a.ws + a.ml_off);
    const float* po = reinterpret_cast<const float*>(a.ws + a.o_off);
    for (int i = threadIdx.x; i < CW * D; i += kTreeThreads) {
        const int c = c0 + i / D, ch = i % D, r = row0 + c;
        if (r >= a.rows) continue;
        float M = -INFINITY;
        for (int64_t j = j0; j <= j1; ++j) {
            const float2 x = ml[(j + unit) * N + c];
            if (x.y != 0.0f) M = fmaxf(M, x.x);
        }
        float L = 0.0f, O = 0.0f;
        for (int64_t j = j0; j <= j1; ++j) {
            const float2 x = ml[(j + unit) * N + c];
            const float o = po[((j + unit) * N + c) * D + ch];
            if (x.y == 0.0f) {
                if (!(fabsf(o) < INFINITY)) O += o;     // a visible draft's value that is not finite
                continue;
            }
            const float f = tree_exp2(x.x - M);
            L = fmaf(x.y, f, L);
            O += fabsf(o) < INFINITY ? o * f : o;
        }
        a.out[(((int64_t)b * a.nodes + (r >> a.gshift)) * lo.Hq + h * lo.gqa + (r & (lo.gqa - 1))) * D + ch] =
            __float2bfloat16_rn(L != 0.0f ? O / L : 0.0f);
    }
}

// `stage`: bytes of shared memory that a tile's packed bytes pass through.
int launch_tree_d32(TreeArgs& a, int N, int64_t stage, cudaStream_t stream);
int launch_tree_d64(TreeArgs& a, int N, int64_t stage, cudaStream_t stream);
int launch_tree_d128(TreeArgs& a, int N, int64_t stage, cudaStream_t stream);
int launch_tree_d256(TreeArgs& a, int N, int64_t stage, cudaStream_t stream);

}  // namespace kvq
