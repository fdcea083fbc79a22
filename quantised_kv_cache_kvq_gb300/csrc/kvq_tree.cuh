// kvq_tree.cuh -- attention of drafted tokens over a cache: the kernel.
//
// The rows of one (sequence, KV head) are its nodes * gqa queries, cut into row tiles of N
// columns; its tokens -- the packed ones, then the unpacked ones (the bf16 window, the drafts)
// -- into tiles of up to 128.  Per tile, on the tensor cores,
//   S^T [128 tokens x N]   = K [128 x D] Q^T [D x N]
//   O^T [D x N]           += V^T [D x 128] P [128 x N]
// with the tokens (and the channels) on the instruction's M side, so that its cost follows the
// number of queries, 16 to 128, and a cache byte is dequantised once for all of them.
//
// Per tile a block unpacks the keys, issues the scores' product, unpacks the values while it
// runs, takes the scores out of TMEM, writes the weights to shared memory and issues their
// product, which runs under the next tile's keys.  Two blocks share an SM where their tiles fit
// (heads of up to 128 channels, up to 64 columns), so that one computes while the other waits.
//
// Measured (a call: this kernel and the join of its parts; 32 query and 8 KV heads of 128):
//   16 drafts, 2-bit, 8 x 4096 tokens       53 us   (its bytes take 4.6 us at the copy bandwidth)
//   32 drafts, 4-bit, 131072 tokens        178 us   (its products take 35 us at the dense bf16 rate)
//   8 drafts, FP8, 64 x 8192 tokens        306 us   (its bytes take 160 us)
// The kernel issues instructions in 33 to 52% of its cycles, and the tensor pipe is busy in 8 to
// 17%: a tile is a chain of short phases (unpack, product, unpack, softmax, product), each of a
// few hundred instructions a warp behind a barrier, and 128 registers a thread allow two blocks
// of 8 warps to fill each other's gaps.  Measured slower: warps in roles (copy, keys, values,
// product, softmax) that hand tiles on through mbarriers (133 us where the phases took 113: the
// roles' code, side by side, missed the instruction cache, their waits took issue slots, and 20
// to 24 warps left too few registers); 16 warps of 64 registers a block (78 us for 53: spills);
// row tiles of 64 columns in place of 128, so that two blocks fit (237 us for 192); the weights
// written before the vote on the references, to save its barrier (FP8 349 us for 333).
//
// Softmax, in base 2.  A token's value row is stored in binary16 as v 2^-e (or as its code),
// v = stored * s; the weight that multiplies it is P = 2^(x + log2 s - m) with a running
// reference m per column: 8 under the largest x + log2 s seen, so that P <= 2^8 and weights
// down to 2^-22 of the largest keep binary16's 11 bits.  m is set on a segment's first tile
// and moves later only when some entry of a tile reaches 2^15 above it: then O^T is rescaled
// in TMEM.  The sum l takes P / s in binary32, per thread, and is joined at the end; O / l is
// the output.  A masked entry has x = -infinity and takes no part in anything.
//
// Roundings to 16 bits: a product's operands only.  Queries and raw rows (bf16, 8 bits) go into
// binary16's 11 exactly, under a power of two, but for what lies 2^-30 below their largest;
// a KIVI key or value is rounded once, behind its fused multiply-add, a turned key behind the
// turn; FP8, INT8 and INT4 codes are exact; a weight is rounded once, by 2^-11 of itself.
#pragma once

#include <cuda_fp8.h>

#include "kvq_elements.cuh"
#include "kvq_internal.cuh"
#include "kvq_rope_angle.cuh"
#include "kvq_tcgen05.cuh"

namespace kvq {

constexpr int kMergeThreads = 256;
constexpr int kMaxTreeBlocks = 608;     // of a launch: bounds the workspace's partial results
constexpr float kHead = 8.0f;           // P of the largest entry, log2
constexpr float kReach = 15.0f;         // P may grow to 2^15 before the reference moves

// What a kernel unpacks: KIVI records of 2, 4 or 8 bits, KIVI records read where they lie (any
// bits; those that do not fit next to the operand tiles), INT8 and INT4 rows, FP8 tiles.  The
// kinds are kernels of their own: together in one, their code costs every path registers.
enum TreeKind { kKivi2 = 2, kKivi4 = 4, kKivi8 = 8, kInPlace = 16, kRows = 32, kFp8 = 64 };

struct TreeArgs {
    Layout lo;
    const uint8_t* cache;
    int layer, nodes, rows, RT;         // rows = nodes * gqa, RT row tiles of N columns
    int gshift;                         // log2 gqa
    int NB, blocks;                     // blocks of the launch, and of an SM
    int TT, TG;                         // tokens, and groups, of a full packed tile
    int gvshift;                        // log2 of the value group (it divides a power of two)
    int pieces;                         // KIVI: pieces of 8 key and value parameters of a group
    uint32_t pieces_inverse;            // 2^32 / pieces, rounded up
    int group_of[8];                    // KIVI: the group of a tile's 16-token piece
    int stages, stage_bytes;            // buffers that a tile's packed bytes pass through (0: none)
    int share;                          // the weights lie in the key tile (written when its scores are done)
    int stage_at;                       // where the buffers begin
    const __nv_bfloat16 *q, *k, *v;
    const uint8_t* mask;
    const int32_t* n_nodes;
    float qscale;                       // softmax scale * log2 e
    __nv_bfloat16* out;
    uint8_t* ws;
    int64_t span_off, ml_off, o_off;    // in the workspace: each row tile's blocks, partials (m, l), O
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
// Cost of the tiles of one row tile, in packed tiles: an unpacked one takes about as long as
// kRawCost of them (measured).
constexpr int kRawCost = 3;
__device__ __forceinline__ int tree_cost(const TreeSeq& s) { return s.packed + (s.tiles - s.packed) * kRawCost; }
// The first tile that begins at or behind cost position x of a row tile.
__device__ __forceinline__ int tree_tile_at(const TreeSeq& s, int64_t x) {
    if (x <= s.packed) return static_cast<int>(x);
    const int64_t t = s.packed + (x - s.packed + kRawCost - 1) / kRawCost;
    return t < s.tiles ? static_cast<int>(t) : s.tiles;
}
// Cost of all the row tiles of one KV head of a sequence (a row tile without queries is one
// empty tile: its outputs are set to 0).
__device__ __forceinline__ int64_t tree_head_tiles(const TreeArgs& a, const TreeSeq& s) {
    return (int64_t)s.live * tree_cost(s) + (a.RT - s.live);
}

// Exclusive place of this thread's value in the block's sum, and the sum.
template <int NT>
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
    for (int w = 0; w < NT / 32; ++w) {
        if (w < warp) before += tmp[w];
        all += tmp[w];
    }
    *sum = all;
    return before + x - v;
}

// All tiles of the launch.
template <int NT>
__device__ __forceinline__ int64_t tree_total(const TreeArgs& a, int N, int64_t* tmp) {
    int64_t total = 0;
    for (int b0 = 0; b0 < a.lo.B; b0 += NT) {
        const int b = b0 + threadIdx.x;
        int64_t sum;
        block_scan<NT>(b < a.lo.B ? a.lo.H * tree_head_tiles(a, tree_seq(a, b, N)) : 0, tmp, &sum);
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

// One packed tile: its groups' records (KIVI), or its rows (the other schemes).  STAGED: in
// shared memory, one record after another; else the records are read where they lie.
template <bool STAGED>
struct PackedTile {
    const uint8_t* base;          // STAGED
    int stride;
    const uint8_t* const* recs;   // not STAGED: the records' places
    int cnt;                      // tokens
    __device__ __forceinline__ const uint8_t* rec(int g) const {
        if constexpr (STAGED) return base + g * stride;
        else return recs[g];
    }
};

// KIVI keys.  A warp takes 64 channels of some octets of rows; a lane 16 channels of one row
// of each octet, with the group's scales and zeros of its channels in registers.  x = code * s +
// z is one binary16 fused multiply-add of exact operands: rounded once.
template <int D, int BITS, int DT, typename Tile>
__device__ __forceinline__ void kivi_keys(const TreeArgs& a, const Tile t, uint8_t* kt, int tid) {
    constexpr int QUADS = D / 64, PER = 16 * QUADS / (DT / 32);       // octets of a warp
    const Layout& lo = a.lo;
    const int warp = tid >> 5, lane = tid & 31;
    const int unit = (warp % QUADS) * 4 + (((lane >> 3) + lane) & 3), o0 = (warp / QUADS) * PER;
    uint32_t s[8], z[8];
    int have = -1;
#pragma unroll 4
    for (int o = o0; o < o0 + PER; ++o) {
        const int row = 8 * o + (lane & 7), tok = packed_token(row);
        if (8 * (o & ~1) >= t.cnt) break;
        const int g = a.group_of[o >> 1], tin = tok - g * lo.G;
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
template <int D, int BITS, int DT, typename Tile>
__device__ __forceinline__ void kivi_values(const TreeArgs& args, const Tile t, uint8_t* vt, int tid) {
    constexpr int HW = 16 / BITS, WPL = D * BITS / 64, SW = WPL < 4 ? WPL : 4;
    const Layout& lo = args.lo;
    const int g8 = tid & 7, ip = (tid >> 3) & 1;
    for (int it = tid >> 4; it < 8 * (WPL / 2); it += DT / 16) {
        const int a = it / (WPL / 2), mm = it % (WPL / 2);     // 16-token tile, word pair
        if (16 * a >= t.cnt) break;
        const int g = args.group_of[a], ti = 16 * a - g * lo.G;   // group, first token in it
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
            const int gv = c >> args.gvshift;
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

// Largest magnitude in the tile's side lists (as bf16 << 16), over a thread's share.
template <int DT, typename Tile>
__device__ __noinline__ uint32_t side_wide(const Layout& lo, const Tile t, int tid) {
    uint32_t top = 0;
    for (int g = 0; g * lo.G < t.cnt; ++g) {
        const uint32_t* side = reinterpret_cast<const uint32_t*>(t.rec(g) + lo.kc + lo.vc + lo.kp + lo.vp);
        for (int i = tid; i < (lo.ko + lo.vo) / 4; i += DT) top = max(top, side[i] & 0x7fff0000u);
    }
    return top;
}
// Whether some |value| that the tile's keys or values can have reaches 2^15, over a thread's
// share of their parameters (in binary16: levels * s + |z|, an infinity counts).  Piece i of 8
// parameters of a tile lies `piece` bytes into its group's record.
template <int DT, typename Tile>
__device__ __forceinline__ bool kivi_wide(const TreeArgs& a, const Tile& t, int tid) {
    const Layout& lo = a.lo;
    const __half2 levels = __float2half2_rn(static_cast<float>((1 << lo.bits) - 1));
    __half2 top = __float2half2_rn(0.0f);
    uint32_t side_top = 0;
    for (int i = tid; i < a.TG * a.pieces; i += DT) {
        const int g = static_cast<int>(__umulhi(i, a.pieces_inverse));      // i / pieces
        if (g * lo.G >= t.cnt) break;
        const int at = i - g * a.pieces, kpieces = lo.D / 8;
        const bool v = at >= kpieces;
        const uint8_t* p = t.rec(g) + lo.kc + lo.vc + 16 * at + (v ? 2 * lo.D : 0);
        const uint4 s = *reinterpret_cast<const uint4*>(p), z = *reinterpret_cast<const uint4*>(p + (v ? 16 * (a.pieces - kpieces) : 2 * lo.D));
        const uint32_t sw[4] = {s.x, s.y, s.z, s.w}, zw[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) top = __hmax2(top, __hfma2(levels, u32_as_h2(sw[j]), __habs2(u32_as_h2(zw[j]))));
    }
    if (lo.K > 0) side_top = side_wide<DT>(lo, t, tid);
    const uint32_t h = h2_as_u32(top);
    return (h & 0xffffu) >= 0x7800u || (h >> 16) >= 0x7800u || side_top >= 0x47000000u;
}
// Their largest finite |value|, of the keys (kv = 0) or values, over a thread's share.
template <int DT, typename Tile>
__device__ __noinline__ float kivi_bound(const Layout& lo, const Tile t, int kv, int lane) {
    const float levels = static_cast<float>((1 << lo.bits) - 1);
    const int pairs = kv ? lo.NGv * lo.G : lo.D;
    float top = 0.0f;
    for (int g = 0; g * lo.G < t.cnt; ++g) {
        const __half* par = reinterpret_cast<const __half*>(t.rec(g) + lo.kc + lo.vc + (kv ? lo.kp : 0));
        const uint32_t* side = reinterpret_cast<const uint32_t*>(t.rec(g) + lo.kc + lo.vc + lo.kp + lo.vp + (kv ? lo.ko : 0));
        for (int i = lane; i < pairs; i += DT) {
            const float x = fmaf(levels, __half2float(par[i]), fabsf(__half2float(par[pairs + i])));
            top = fmaxf(top, x < INFINITY ? x : 0.0f);
        }
        for (int i = lane; i < lo.K * pairs; i += DT) {
            const float x = fabsf(__uint_as_float(side[i] & 0xffff0000u));
            top = fmaxf(top, x < INFINITY ? x : 0.0f);
        }
    }
    return top;
}

// The same tile where binary16 does not hold its values: element by element, times `scale`.
template <int D, int DT, typename Tile>
__device__ __noinline__ void kivi_keys_scaled(const Layout& lo, const Tile t, uint8_t* kt, float scale, int W, int tid) {
    for (int i = tid; i < 128 * D; i += DT) {
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
template <int D, int DT, typename Tile>
__device__ __noinline__ void kivi_values_scaled(const Layout& lo, const Tile t, uint8_t* vt, float scale, int tid) {
    for (int i = tid; i < 128 * D; i += DT) {
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
template <int D, int DT, typename Tile>
__device__ __noinline__ void kivi_outliers(const Layout& lo, const Tile t, uint8_t* tile, int kv, float scale, int W, int tid) {
    const int per = kv ? lo.NGv * lo.G : D;
    for (int g = 0; g * lo.G < t.cnt; ++g) {
        const uint32_t* side = reinterpret_cast<const uint32_t*>(t.rec(g) + lo.kc + lo.vc + lo.kp + lo.vp + (kv ? lo.ko : 0));
        for (int i = tid; i < lo.K * per; i += DT) {
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
template <int D, int DT>
__device__ __forceinline__ void fp8_keys(const uint8_t* codes, int cnt, bool e4m3, uint8_t* kt, int tid) {
    constexpr uint32_t sbo = D / 8 * kCoreBytes;
#pragma unroll 4
    for (int i = tid; i < 128 * D / 16; i += DT) {
        const int row = (i & 7) + 8 * (i / (D / 2)), unit = ((i >> 3) + row) % (D / 16), tok = packed_token(row);
        if ((row & ~15) >= cnt) break;
        uint32_t o[8];
        fp8_16(*reinterpret_cast<const uint4*>(codes + tok * D + 16 * unit), e4m3, o);
        *reinterpret_cast<uint4*>(kt + core_at(row, 2 * unit, sbo)) = make_uint4(o[0], o[1], o[2], o[3]);
        *reinterpret_cast<uint4*>(kt + core_at(row, 2 * unit + 1, sbo)) = make_uint4(o[4], o[5], o[6], o[7]);
    }
}
template <int D, int DT>
__device__ __forceinline__ void fp8_values(const uint8_t* codes, int cnt, bool e4m3, bool negative, uint8_t* vt, int tid) {
#pragma unroll 4
    for (int i = tid; i < 8 * D; i += DT) {
        const int c = i % D, a = i / D;
        if (16 * a >= cnt) break;
        uint32_t o[8];
        fp8_16(*reinterpret_cast<const uint4*>(codes + (16 * a * D + 16 * c)), e4m3, o);
        if (negative) {                     // the value scale's sign (its size goes to the weights)
#pragma unroll
            for (int r = 0; r < 8; ++r) o[r] ^= 0x80008000u;
        }
        if (16 * a + 16 > cnt) {          // tokens that the cache does not hold: any bytes
#pragma unroll
            for (int r = 0; r < 16; ++r)
                if (packed_token(16 * a + r) >= cnt) o[r / 2] &= r & 1 ? 0x0000ffffu : 0xffff0000u;
        }
        *reinterpret_cast<uint4*>(vt + core_at(c, 2 * a, 16 * kCoreBytes)) = make_uint4(o[0], o[1], o[2], o[3]);
        *reinterpret_cast<uint4*>(vt + core_at(c, 2 * a + 1, 16 * kCoreBytes)) = make_uint4(o[4], o[5], o[6], o[7]);
    }
}

// INT8 and INT4 rows: the codes as exact binary16 numbers (the scales go to the scores and the
// weights); keys K-major, values with their channels inside a row (MN-major).
template <int D, int DT>
__device__ __forceinline__ void rows_codes(const uint8_t* codes, int cnt, int kv, bool int8, uint8_t* tile, int tid) {
#pragma unroll 4
    for (int i = tid; i < 128 * D / 16; i += DT) {
        const int row = (i & 7) + 8 * (i / (D / 2)), unit = ((i >> 3) + row) % (D / 16);
        if ((row & ~15) >= cnt) break;
        uint32_t o[8] = {};
        if (row < cnt) {
            if (int8) {
                const uint4 v = *reinterpret_cast<const uint4*>(codes + row * D + 16 * unit);
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {       // code + 128 as an unsigned byte, less 1152
                    const uint32_t x = w[j] ^ 0x80808080u;
                    o[2 * j] = hfma2u((x & 0x00ff00ffu) | 0x64006400u, 0x3c003c00u, 0xe480e480u);
                    o[2 * j + 1] = hfma2u(((x >> 8) & 0x00ff00ffu) | 0x64006400u, 0x3c003c00u, 0xe480e480u);
                }
            } else {
                const uint2 v = *reinterpret_cast<const uint2*>(codes + row * (D / 2) + 8 * unit);
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

// 16 bf16 channels as binary16 pairs times f.
__device__ __forceinline__ void half_words(const uint32_t (&w)[8], float f, uint32_t (&o)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
        o[i] = h2_as_u32(__floats2half2_rn(__uint_as_float(w[i] << 16) * f, __uint_as_float(w[i] & 0xffff0000u) * f));
}
// Largest magnitude of 16 bf16 channels, as a pattern (0x7f80 and above: not finite).
__device__ __forceinline__ uint32_t unit_top(const uint32_t (&w)[8]) {
    uint32_t m = w[0] & 0x7fff7fffu;
#pragma unroll
    for (int i = 1; i < 8; ++i) m = __vmaxu2(m, w[i] & 0x7fff7fffu);
    return max(m & 0xffffu, m >> 16);
}
// The same over the finite ones, which are left alone where `keep`; the others become 0 if not.
__device__ __forceinline__ uint32_t finite_top(uint32_t (&w)[8], bool keep) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t lo = w[i] & 0x7fffu, hi = (w[i] >> 16) & 0x7fffu;
        if (lo < 0x7f80u) m = max(m, lo);
        else if (!keep) w[i] &= 0xffff0000u;
        if (hi < 0x7f80u) m = max(m, hi);
        else if (!keep) w[i] &= 0x0000ffffu;
    }
    return m;
}
// Largest finite magnitude of the row that lanes l, l + 8, l + 16 and l + 24 hold.
template <int STEPS>
__device__ __forceinline__ float row_top(uint32_t (&w)[STEPS][8], bool keep, bool* odd) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < STEPS; ++i) m = max(m, unit_top(w[i]));
    if (m >= 0x7f80u) {
        *odd = true;
        m = 0;
#pragma unroll
        for (int i = 0; i < STEPS; ++i) m = max(m, finite_top(w[i], keep));
    }
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 8));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 16));
    return __uint_as_float(m << 16);
}
__device__ __forceinline__ void load_words(const uint16_t* p, uint32_t (&w)[8]) {
    const uint4 a = reinterpret_cast<const uint4*>(p)[0], b = reinterpret_cast<const uint4*>(p)[1];
    w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w; w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
}

// The channels' order as a compile-time number where the kind fixes it (else -1).
template <int KIND>
__device__ __forceinline__ constexpr int fixed_block() {
    return KIND <= kKivi8 ? 32 / KIND : KIND == kFp8 ? 0 : -1;
}

// bf16 rows (the window's tokens, then the drafts) [r0, r0 + cnt) of unit (b, h): keys and
// values into their tiles, with their powers of two.  A warp takes an octet of rows, a lane 16
// channels of one row at a time; each row is scaled by its own largest element (the second
// loads hit the cache).  *bad: a draft's value is not finite (it is 0 in the tile).  The loops
// are not unrolled: what runs once or twice in a block costs its instructions' fetch first.
template <int D, int DT, int KIND>
__device__ __noinline__ void raw_rows(const TreeArgs& a, int b, int h, int n, int qn, int r0, int cnt, uint8_t* kt, uint8_t* vt,
                                      float* kf, float* vlog, int* bad, int tid) {
    constexpr int UNITS = D / 16, STEPS = (UNITS + 3) / 4, WK = fixed_block<KIND>();
    const int W = WK >= 0 ? WK : key_block(a.lo);
    const int warp = tid >> 5, lane = tid & 31, window = n - qn, C = a.lo.C;
    const uint32_t slot0 = C > 0 ? static_cast<uint32_t>(qn) % static_cast<uint32_t>(C) : 0u;
    const uint16_t* ring = reinterpret_cast<const uint16_t*>(a.cache + a.lo.ring_off) + unit_index(a.lo, a.layer, b, h) * C * (2 * D);
    const int64_t draft0 = (((int64_t)b * a.nodes - window) * a.lo.H + h) * D;      // row r: + r H D
#pragma unroll 1
    for (int o = warp; o < 16; o += DT / 32) {
        const int row = 8 * o + (lane & 7), r = r0 + row;
        if ((8 * o & ~15) >= cnt) break;
        const uint16_t *kp = nullptr, *vp = nullptr;
        if (row < cnt) {
            if (r < window) {
                uint32_t slot = slot0 + r;                  // window token r is in slot (qn + r) mod C
                if (slot >= static_cast<uint32_t>(C)) slot -= C;
                kp = ring + (int64_t)slot * (2 * D);
                vp = kp + D;
            } else {
                const int64_t at = draft0 + (int64_t)r * a.lo.H * D;
                kp = reinterpret_cast<const uint16_t*>(a.k) + at;
                vp = reinterpret_cast<const uint16_t*>(a.v) + at;
            }
        }
        const bool draft = r >= window;
        uint32_t ktop = 0, vtop = 0;
#pragma unroll
        for (int i = 0; i < STEPS; ++i) {
            const int unit = (lane >> 3) + 4 * i;
            if (!kp || unit >= UNITS) continue;
            uint32_t x[8], y[8];
            load_words(kp + 16 * unit, x);
            load_words(vp + 16 * unit, y);
            ktop = max(ktop, unit_top(x));
            vtop = max(vtop, unit_top(y));
        }
#pragma unroll 1
        for (int kv = 0; kv < 2; ++kv) {
            const uint16_t* p = kv ? vp : kp;
            uint32_t top = kv ? vtop : ktop;
            const bool odd = top >= 0x7f80u, clear = kv && draft;
            uint32_t w[8];
            if (odd) {
                top = 0;
                for (int unit = lane >> 3; unit < UNITS; unit += 4) {
                    load_words(p + 16 * unit, w);
                    top = max(top, finite_top(w, true));
                }
                if (clear) *bad = 1;
            }
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 8));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 16));
            const int e = range_exponent(__uint_as_float(top << 16));
            const float f = pow2i(-e);
#pragma unroll 1
            for (int unit = lane >> 3; unit < UNITS; unit += 4) {
#pragma unroll
                for (int j = 0; j < 8; ++j) w[j] = 0u;
                if (p) load_words(p + 16 * unit, w);
                if (odd && clear) finite_top(w, false);
                uint32_t hw[8];
                half_words(w, f, hw);
                if (kv == 0) {
                    store_unit<D>(kt, row, unit, hw, W);
                } else {
                    if (KIND == kRows) {
                        pair_words(hw, W, w);
                    } else {
#pragma unroll
                        for (int j = 0; j < 8; ++j) w[j] = hw[j];
                    }
                    uint8_t* at = vt + (row >> 3) * kCoreBytes + (row & 7) * 16 + 2 * unit * 16 * kCoreBytes;
                    *reinterpret_cast<uint4*>(at) = make_uint4(w[0], w[1], w[2], w[3]);
                    *reinterpret_cast<uint4*>(at + 16 * kCoreBytes) = make_uint4(w[4], w[5], w[6], w[7]);
                }
            }
            if (lane < 8) {
                if (kv) vlog[row] = static_cast<float>(e);
                else kf[row] = pow2i(e);
            }
        }
    }
}

// Rows [r0, r1) of the unpacked ones (the window's part) into L2.
template <int D, int DT>
__device__ __noinline__ void prefetch_rows(const TreeArgs& a, int b, int h, int n, int qn, int nodes, int r0, int r1, int tid) {
    const int window = n - qn, C = a.lo.C, lines = D * 4 / 128;         // of a token's key and value
    r1 = r1 < window ? r1 : window;
    if (r0 >= r1) return;
    const uint8_t* ring = a.cache + a.lo.ring_off + unit_index(a.lo, a.layer, b, h) * C * (int64_t)(4 * D);
    const uint32_t slot0 = static_cast<uint32_t>(qn) % static_cast<uint32_t>(C);
    for (int i = r0 * lines + tid; i < r1 * lines; i += DT) {
        uint32_t slot = slot0 + i / lines;
        if (slot >= static_cast<uint32_t>(C)) slot -= C;
        prefetch_l2(ring + (int64_t)slot * (4 * D) + (i % lines) * 128);
    }
}

// Turns the tile's cached keys by their positions: row r of the tile is token t0 + (its place),
// rows from `rows` on stay.
template <int D, int DT>
__device__ __noinline__ void turn_keys(uint8_t* kt, const float* w, int64_t t0, int rows, int tid) {
    constexpr uint32_t sbo = D / 8 * kCoreBytes;
    constexpr int CH = D / 16;                  // 8-channel chunks of half a row
    for (int i = tid; i < 128 * CH; i += DT) {
        const int row = (i & 7) + 8 * (i / (8 * CH)), ch = (i >> 3) % CH;
        if (row >= rows) continue;
        uint4* pa = reinterpret_cast<uint4*>(kt + core_at(row, ch, sbo));
        uint4* pb = reinterpret_cast<uint4*>(kt + core_at(row, ch + CH, sbo));
        const float pos = static_cast<float>(t0 + row);
#pragma unroll 1
        for (int j = 0; j < 8; ++j) {           // (one sine's code, not eight)
            __half* px = reinterpret_cast<__half*>(pa) + j;
            __half* py = reinterpret_cast<__half*>(pb) + j;
            const float x = __half2float(*px), y = __half2float(*py);
            float sn, cs;
            rope_sincos(__fmul_rn(pos, w[8 * ch + j]), &sn, &cs);
            *px = __float2half_rn(x * cs - y * sn);
            *py = __float2half_rn(y * cs + x * sn);
        }
    }
}
// A dequantised key (times `scale`) in binary32 where h is its binary16 rounding, else h: an
// outlier lies over it.
__device__ __forceinline__ float unrounded_key(const Layout& lo, const uint8_t* rec, int tin, int c, float scale, __half h) {
    const __half* par = reinterpret_cast<const __half*>(rec + lo.kc + lo.vc);
    const int bit = (tin * lo.D + c) * lo.bits;
    const float x = scale * scaled_code((rec[bit >> 3] >> (bit & 7)) & ((1 << lo.bits) - 1), __half2float(par[c]),
                                        __half2float(par[lo.D + c]));
    return __half_as_ushort(__float2half_rn(x)) == __half_as_ushort(h) ? x : __half2float(h);
}
// The same for a KIVI tile (tokens in the packed order), from the values before their rounding
// to binary16: a turned key is rounded once.
template <int D, int DT, typename Tile>
__device__ __noinline__ void turn_kivi_keys(const Layout& lo, const Tile t, uint8_t* kt, const float* w, int64_t t0, float scale, int W,
                                            int tid) {
    constexpr uint32_t sbo = D / 8 * kCoreBytes;
    constexpr int CH = D / 16;
    for (int i = tid; i < 128 * CH; i += DT) {
        const int row = (i & 7) + 8 * (i / (8 * CH)), ch = (i >> 3) % CH, tok = packed_token(row);
        if (tok >= t.cnt) continue;
        uint4* pa = reinterpret_cast<uint4*>(kt + core_at(row, ch, sbo));
        uint4* pb = reinterpret_cast<uint4*>(kt + core_at(row, ch + CH, sbo));
        const float pos = static_cast<float>(t0 + tok);
        const int g = tok / lo.G, tin = tok - g * lo.G;
        const uint8_t* rec = t.rec(g);
#pragma unroll 1
        for (int j = 0; j < 8; ++j) {
            __half* px = reinterpret_cast<__half*>(pa) + j;
            __half* py = reinterpret_cast<__half*>(pb) + j;
            const int c = place_channel(8 * ch + j, W, D);
            const float x = unrounded_key(lo, rec, tin, c, scale, *px), y = unrounded_key(lo, rec, tin, c + D / 2, scale, *py);
            float sn, cs;
            rope_sincos(__fmul_rn(pos, w[8 * ch + j]), &sn, &cs);
            *px = __float2half_rn(x * cs - y * sn);
            *py = __float2half_rn(y * cs + x * sn);
        }
    }
}

// Shapes of an instantiation: N columns, D channels.
template <int N, int D>
struct TreeShape {
    static constexpr int kThreads = N > 64 || (D > 128 && N > 16) ? 512 : 256;
    static constexpr int kBlocks = N > 64 || D > 128 ? 1 : 2;   // of an SM
    static constexpr int NH = N / (kThreads / 128);             // columns of a thread
    static constexpr int B = NH;                                // of one TMEM access
    static constexpr int kDN = D > 128 ? 2 : 1;                 // accumulators of 128 channels
    static constexpr int kTmem = N * (1 + kDN);                 // the scores and O^T
    static constexpr uint32_t kCols = kTmem <= 32 ? 32 : kTmem <= 64 ? 64 : kTmem <= 128 ? 128 : kTmem <= 256 ? 256 : 512;
    // shared memory: K, V (the product reads 128 channel rows of it), Q, P, then the stages
    static constexpr int kVBytes = D > 128 ? 65536 : 32768;
    static constexpr int kK = 0, kV = 256 * D, kQ = kV + kVBytes, kP = kQ + 2 * N * D;
};

__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(r));
    return r != 0;
}
// Bounded wait of about a second.  The thread sleeps in the instruction (up to a millisecond at
// a time): warps that poll take the issue slots and the shared-memory pipe of those that work.
__device__ __forceinline__ bool mbar_wait_asleep(uint64_t* bar, uint32_t parity) {
    const uint32_t at = smem_addr(bar);
    for (int i = 0; i < 2000; ++i) {
        uint32_t ok;
        asm volatile(
            "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n selp.u32 %0, 1, 0, p;\n}"
            : "=r"(ok)
            : "r"(at), "r"(parity), "r"(1000000u)
            : "memory");
        if (ok) return true;
    }
    return false;
}
// Two binary32 lanes at a time.
__device__ __forceinline__ uint64_t pack2(float x, float y) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float* x, float* y) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(*x), "=f"(*y) : "l"(v));
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// Where block j of nb's share of `total` tiles begins: total j / nb (in 32 bits where they do).
__device__ __forceinline__ int64_t share_start(int64_t total, int64_t j, int64_t nb) {
    if (total < (1 << 21)) return static_cast<uint32_t>(total) * static_cast<uint32_t>(j) / static_cast<uint32_t>(nb);
    return total * j / nb;
}
// A block's walk over its share of the tiles: segments, each the tiles [first, end) of one row
// tile of one KV head: those that begin in [pos, pos + left) of its cost.
struct TreeWalk {
    int b, h, rt, first, end, unit_tiles;
    bool live;
    TreeSeq s;
    int64_t pos, left;
    __device__ __forceinline__ int64_t unit_cost() const { return live ? tree_cost(s) : 1; }
    __device__ __forceinline__ void segment() {
        live = rt < s.live;
        unit_tiles = live ? s.tiles : 1;
        const int64_t to = left < unit_cost() - pos ? pos + left : unit_cost();
        first = live ? tree_tile_at(s, pos) : 0;
        end = live ? tree_tile_at(s, to) : 1;
    }
    // the share of `n` from position `at` of sequence b_ on
    __device__ __forceinline__ void begin(const TreeArgs& a, const TreeSeq& seq, int b_, int64_t at, int64_t n) {
        b = b_;
        left = n;
        s = seq;
        const int64_t per = tree_head_tiles(a, s);
        h = static_cast<int>(at >> 31 ? at / per : static_cast<uint32_t>(at) / static_cast<uint32_t>(per));
        const int in = static_cast<int>(at - h * per), cost = tree_cost(s), run = s.live * cost;
        rt = in < run ? in / cost : s.live + (in - run);
        pos = in < run ? in - rt * cost : 0;
        segment();
    }
    // to the next segment; false at the end of the share
    __device__ __forceinline__ bool next(const TreeArgs& a, int N) {
        const int64_t took = unit_cost() - pos;
        left -= took;
        if (left <= 0) return false;
        pos = 0;
        if (++rt == a.RT) {
            rt = 0;
            if (++h == a.lo.H) {
                h = 0;
                ++b;
                s = tree_seq(a, b, N);
            }
        }
        segment();
        return true;
    }
    __device__ __forceinline__ int packed_count(const TreeArgs& a, int tile) const {
        const int64_t t0 = (int64_t)tile * a.TT;
        return static_cast<int>(s.qn - t0 < a.TT ? s.qn - t0 : a.TT);
    }
    __device__ __forceinline__ int raw_count(int tile) const {
        const int all = s.n - s.qn + s.nodes - (tile - s.packed) * 128;
        return all < 128 ? all : 128;
    }
};

// What a block shares next to the operand tiles.
template <int N, int D>
struct TreeShared {
    float colg[N], colr[N];         // a column's query scale and minus its reference
    int seen[N];                    // it has a reference
    float fac[N], part[4][N];       // per column: factors; per quadrant: maxima, sums
    float kf[128], vl[128];         // a raw row's score factor and log2 of its value scale
    float kscale, vscale, vscale_log;       // FP8: the KV head's scales, log2 of the values'
    float wt[D / 2];                // rotary frequencies in the order of the key tile
    int64_t scan[32], start;
    uint64_t stage_full[2], keys_full[2], s_full, pv_done;   // (keys_full: rows and FP8, whose keys come apart)
    const uint8_t* recs[8];         // records read in place
    int qtop, qlow;                 // exponents of the largest and the smallest query
    uint32_t tmem, top[2];
    TreeWalk walk;                  // the segment
    int more;
    // the next packed tile to bring in: its segment, where it lies, what is left of the segment's
    // packed part (KIVI: groups; others: tokens); paged: the table's entry, the group in its page, the
    // page (negative: not looked up yet)
    TreeWalk ahead;
    const uint8_t* ahead_src;
    int ahead_left, ahead_entry, ahead_in, ahead_page;
    uint32_t ahead_slot;
    bool keys_sent;                 // rows and FP8: the next tile's keys are on their way
    int dead, odd;                  // a wait gave up; a draft's value is not finite
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

// The queries of a segment's columns into their tile: a warp takes an octet of columns, a lane
// 16 channels at a time.  All are stored under the largest one's power of two; a query 2^20
// below it keeps binary16's subnormal steps, 2^-39 of the largest.  Where one is smaller
// still, each gets a power of its own, and the scores their columns' factors.  Returns (such
// factors are needed, the factor of all scores); ends behind a block barrier.
template <int N, int D, int KIND>
__device__ __noinline__ float2 load_queries(const TreeArgs& a, int row0, int row_end, uint8_t* qt,
                                            TreeShared<N, D>& sh) {
    const TreeWalk& w = sh.walk;
    constexpr int WK = fixed_block<KIND>();
    const int W = WK >= 0 ? WK : key_block(a.lo);
    constexpr int UNITS = D / 16, STEPS = (UNITS + 3) / 4, WARPS = TreeShape<N, D>::kThreads / 32;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gqa = a.lo.gqa;
    if (tid == 0) {
        sh.qtop = -200;
        sh.qlow = 200;
        if constexpr (KIND == kFp8) {
            const float* sc = fp8_scale(a, w.h);
            sh.kscale = sc[0];
            sh.vscale = sc[1];
            sh.vscale_log = fmaxf(fast_log2(fabsf(sc[1])), -110.0f);    // (a scale of 0 belongs to codes of 0)
        }
    }
    __syncthreads();
    // (at most one octet per warp: 16 columns have 2, 64 have 8 of 8 warps, 128 have 16 of 16)
    static_assert(N / 8 <= WARPS, "");
    uint32_t q[STEPS][8];
    const int c = 8 * warp + (lane & 7), r = row0 + c;
    float mx = 0.0f;
    if (warp < N / 8) {
        const uint16_t* p = reinterpret_cast<const uint16_t*>(a.q) +
                            (((int64_t)w.b * a.nodes + (r >> a.gshift)) * a.lo.Hq + w.h * gqa + (r & (gqa - 1))) * D;
#pragma unroll
        for (int i = 0; i < STEPS; ++i) {
            const int unit = (lane >> 3) + 4 * i;
#pragma unroll
            for (int j = 0; j < 8; ++j) q[i][j] = 0u;
            if (r < row_end && unit < UNITS) load_words(p + 16 * unit, q[i]);
        }
        bool odd = false;
        mx = row_top(q, true, &odd);
        if (lane < 8 && mx > 0.0f) {
            atomicMax(&sh.qtop, range_exponent(mx));
            atomicMin(&sh.qlow, range_exponent(mx));
        }
    }
    __syncthreads();
    const bool mixed = sh.qtop - sh.qlow > 20;
    const int common = sh.qtop > -200 ? sh.qtop : 0;
    if (warp < N / 8) {
        const int e = mixed ? range_exponent(mx) : common;
        const float f = pow2i(-e);
#pragma unroll
        for (int i = 0; i < STEPS; ++i) {
            const int unit = (lane >> 3) + 4 * i;
            if (unit >= UNITS) continue;
            uint32_t hw[8];
            half_words(q[i], f, hw);
            store_unit<D>(qt, c, unit, hw, W);
        }
        if (lane < 8) {
            sh.colg[c] = a.qscale * pow2i(e);
            sh.colr[c] = 0.0f;
            sh.seen[c] = 0;
        }
    }
    __syncthreads();
    return make_float2(mixed ? 1.0f : 0.0f, mixed ? 1.0f : a.qscale * pow2i(common));
}

// The result of a segment: O^T (TMEM, from `tm` on for this warp's lanes and columns) over the
// columns' sums (sh.part), as bf16 outputs where the segment is a whole row tile, else as a
// partial result (m, l, O).
template <int N, int D, bool ROWS>
__device__ __noinline__ void finish_segment(const TreeArgs& a, int first, uint32_t tm, int row0, int row_end,
                                            int W, TreeShared<N, D>& sh) {
    using S = TreeShape<N, D>;
    const Layout& lo = a.lo;
    const TreeWalk& w = sh.walk;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, quad = warp & 3, col0 = (warp >> 2) * S::NH;
    const bool whole = first == 0 && w.end == w.unit_tiles;
    const int64_t unit = ((int64_t)w.b * lo.H + w.h) * a.RT + w.rt, slot = blockIdx.x + unit;
    if (tid == 0) {             // which blocks have a part of the row tile: none to join, or first and last
        int* span = reinterpret_cast<int*>(a.ws + a.span_off) + 2 * unit;
        if (first == 0) span[0] = whole ? -1 : static_cast<int>(blockIdx.x);
        if (w.end == w.unit_tiles) span[1] = static_cast<int>(blockIdx.x);
    }
    for (int c = tid; c < N; c += S::kThreads) {
        // rows of padding nodes saw the cached tokens with a query of 0: their output is 0
        const float v = w.live && row0 + c < row_end ? (sh.part[0][c] + sh.part[1][c]) + (sh.part[2][c] + sh.part[3][c]) : 0.0f;
        if (whole) {
            sh.fac[c] = v != 0.0f ? 1.0f / v : 0.0f;
        } else {
            sh.fac[c] = v != 0.0f ? 1.0f : 0.0f;
            reinterpret_cast<float2*>(a.ws + a.ml_off)[slot * N + c] = make_float2(-sh.colr[c], v);
        }
    }
    __syncthreads();
    const bool odd = sh.odd != 0;
    const int gmask = lo.gqa - 1, out_row = lo.Hq * D;
    __nv_bfloat16* out = a.out + ((int64_t)w.b * a.nodes * lo.Hq + w.h * lo.gqa) * D;
    float* part = reinterpret_cast<float*>(a.ws + a.o_off) + slot * N * D;
#pragma unroll 1
    for (int d = 0; d < S::kDN; ++d) {
        const int ch0 = 128 * d + 32 * quad;
        if (ch0 >= D) continue;
        // lane -> channel: the order of the tile's value rows
        const int ch = ROWS ? place_channel(ch0 + lane, W, D) : ch0 + lane;
#pragma unroll 1
        for (int c0 = 0; c0 < S::NH; c0 += S::NH < 16 ? 8 : 16) {
            constexpr int Q = S::NH < 16 ? 8 : 16;
            float o[Q];
            if (w.live) {
                tmem_load(tm + d * N + c0, o);
            } else {
#pragma unroll
                for (int i = 0; i < Q; ++i) o[i] = 0.0f;
            }
#pragma unroll
            for (int i = 0; i < Q; ++i) {
                const float fc = sh.fac[col0 + c0 + i];
                o[i] = fc != 0.0f ? o[i] * fc : 0.0f;
            }
            if (odd) {      // drafts whose value is not finite, in the rows that see them
                for (int j = 0; j < w.s.nodes; ++j) {
                    const float y = __bfloat162float(a.v[(((int64_t)w.b * a.nodes + j) * lo.H + w.h) * D + ch]);
                    if (fabsf(y) < INFINITY) continue;
#pragma unroll
                    for (int i = 0; i < Q; ++i) {
                        const int r = row0 + col0 + c0 + i, node = r >> a.gshift;
                        if (r < row_end && (a.mask ? a.mask[((int64_t)w.b * a.nodes + node) * a.nodes + j] != 0 : j <= node)) o[i] += y;
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < Q; ++i) {
                const int c = col0 + c0 + i, r = row0 + c;
                if (r >= a.rows) break;
                if (whole)
                    out[(r >> a.gshift) * out_row + (r & gmask) * D + ch] = __float2bfloat16_rn(o[i]);
                else
                    part[c * D + ch] = o[i];
            }
        }
    }
}

// A share that covers only the inside of one tile's cost: a part that the join passes over.
template <int N, int D>
__device__ __noinline__ void finish_empty(const TreeArgs& a, TreeShared<N, D>& sh) {
    const TreeWalk& w = sh.walk;
    const int64_t slot = blockIdx.x + ((int64_t)w.b * a.lo.H + w.h) * a.RT + w.rt;
    for (int c = threadIdx.x; c < N; c += TreeShape<N, D>::kThreads)
        reinterpret_cast<float2*>(a.ws + a.ml_off)[slot * N + c] = make_float2(-INFINITY, 0.0f);
    __syncthreads();
}

// A KIVI key tile's further steps: the scaled tile (scaled: always, else where ke != 0), the
// outliers, the rotation; behind and before block barriers.
template <int D, int DT, typename Tile>
__device__ __noinline__ void kivi_keys_rest(const TreeArgs& a, const Tile t, uint8_t* kt, const float* wt, int64_t t0, int ke,
                                            bool scaled, int W, int tid) {
    if (ke != 0 || scaled) {
        kivi_keys_scaled<D, DT>(a.lo, t, kt, pow2i(-ke), W, tid);
        __syncthreads();
    }
    if (a.lo.K > 0) {
        kivi_outliers<D, DT>(a.lo, t, kt, 0, pow2i(-ke), W, tid);
        __syncthreads();
    }
    if (a.lo.rope_base > 0.0f) turn_kivi_keys<D, DT>(a.lo, t, kt, wt, t0, pow2i(-ke), W, tid);
}
// The exponents of the keys and values of a tile that may reach outside binary16 (0: they do
// not); behind and before block barriers.
template <int DT, typename Tile>
__device__ __noinline__ void kivi_exponents(const Layout& lo, const Tile t, uint32_t* top, int* ke, int* ve, int tid) {
    if (tid < 2) top[tid] = 0u;
    __syncthreads();
    for (int kv = 0; kv < 2; ++kv) atomicMax(&top[kv], __float_as_uint(kivi_bound<DT>(lo, t, kv, tid)));
    __syncthreads();
    const float k = __uint_as_float(top[0]), v = __uint_as_float(top[1]);
    *ke = k >= 32768.0f ? range_exponent(k) : 0;
    *ve = v >= 32768.0f ? range_exponent(v) : 0;
    __syncthreads();
}

// The segment that sh.ahead is in, for copy_next; the next one with packed tiles where it has
// none left (`on`).  One thread.
template <int N, int D, int KIND>
__device__ __noinline__ void copy_segment(const TreeArgs& a, TreeShared<N, D>& sh, bool on) {
    TreeWalk& w = sh.ahead;
    for (;; on = true) {
        if (on && !w.next(a, N)) {
            sh.ahead_left = -1;         // nothing more
            return;
        }
        const int end = w.live ? (w.end < w.s.packed ? w.end : w.s.packed) : 0;
        if (w.first >= end) continue;
        const uint8_t* base = a.cache + a.lo.data_off + unit_index(a.lo, a.layer, w.b, w.h) * a.lo.unit;
        const int all = w.s.qn < end * a.TT ? w.s.qn : end * a.TT, rest = all - w.first * a.TT;
        if constexpr (KIND <= kInPlace) {
            const int group = w.first * a.TG;
            sh.ahead_left = rest / a.lo.G;
            sh.ahead_src = base + (int64_t)group * a.lo.rec;
            if (a.lo.PG > 0) {
                sh.ahead_entry = group / a.lo.PG;
                sh.ahead_in = group - sh.ahead_entry * a.lo.PG;
                sh.ahead_page = -1;
            }
        } else {
            sh.ahead_left = rest;
            sh.ahead_src = base + (int64_t)w.first * 128 * (a.lo.scheme == KVQ_SCHEME_INT4 ? D / 2 : D);
        }
        return;
    }
}
// `ng` group records from the pages that sh.ahead's block table names: a copy for each page (a
// head's records lie one after another in it), whose entry is looked up once.
template <int N, int D>
__device__ __noinline__ void copy_pages(const TreeArgs& a, TreeShared<N, D>& sh, uint8_t* to, uint64_t* bar, int ng) {
    const Layout& lo = a.lo;
    while (ng > 0) {
        int in = sh.ahead_in, page = sh.ahead_page;
        if (page < 0) {
            page = lo.table[(int64_t)sh.ahead.b * lo.MP + sh.ahead_entry];
            if (page < 0 || page >= lo.NP) {    // outside the pool: page 0 in its place, reported
                atomicOr(reinterpret_cast<uint32_t*>(a.ws), KVQ_STATUS_BAD_PAGE);
                page = 0;
            }
            sh.ahead_page = page;
        }
        const int run = ng < lo.PG - in ? ng : lo.PG - in;
        bulk_copy_g2s(to, a.cache + lo.data_off + (int64_t)page * lo.page + (((int64_t)a.layer * lo.H + sh.ahead.h) * lo.PG + in) * lo.rec,
                      run * lo.rec, bar);
        to += run * lo.rec;
        ng -= run;
        in += run;
        if (in == lo.PG) {
            in = 0;
            ++sh.ahead_entry;
            sh.ahead_page = -1;
        }
        sh.ahead_in = in;
    }
}
// Brings the block's next packed tile, if there is one, to the next stage; one thread.  KIVI: its
// records.  Rows and FP8: its keys (copy_keys), then its values and scales (copy_next), each as
// soon as the stage's last ones are read.
template <int N, int D, int KIND>
__device__ __forceinline__ bool copy_ready(const TreeArgs& a, TreeShared<N, D>& sh) {
    if (sh.ahead_left == 0) copy_segment<N, D, KIND>(a, sh, true);
    return sh.ahead_left > 0 && !*static_cast<volatile int*>(&sh.dead);
}
template <int N, int D, int KIND>
__device__ __forceinline__ void copy_keys(const TreeArgs& a, TreeShared<N, D>& sh, uint8_t* stage) {
    sh.keys_sent = copy_ready<N, D, KIND>(a, sh);
    if (!sh.keys_sent) return;
    const int row_bytes = a.lo.scheme == KVQ_SCHEME_INT4 ? D / 2 : D, left = sh.ahead_left;
    const uint32_t bytes = static_cast<uint32_t>((((left < 128 ? left : 128) + 15) & ~15) * row_bytes), slot = sh.ahead_slot;
    mbar_arrive_expect_tx(&sh.keys_full[slot], bytes);
    bulk_copy_g2s(stage + slot * a.stage_bytes, sh.ahead_src, bytes, &sh.keys_full[slot]);
}
template <int N, int D, int KIND>
__device__ __forceinline__ void copy_next(const TreeArgs& a, TreeShared<N, D>& sh, uint8_t* stage) {
    const Layout& lo = a.lo;
    if constexpr (KIND <= kInPlace) {
        if (!copy_ready<N, D, KIND>(a, sh)) return;
    } else {
        if (sh.ahead_left <= 0 || !sh.keys_sent) return;
    }
    const int left = sh.ahead_left;
    const uint32_t slot = sh.ahead_slot;
    if (a.stages == 2) sh.ahead_slot = slot ^ 1;
    uint8_t* to = stage + slot * a.stage_bytes;
    uint64_t* bar = &sh.stage_full[slot];
    const uint8_t* src = sh.ahead_src;
    if constexpr (KIND <= kInPlace) {
        const int ng = left < a.TG ? left : a.TG;
        sh.ahead_left = left - ng;
        sh.ahead_src = src + a.TG * lo.rec;
        mbar_arrive_expect_tx(bar, static_cast<uint32_t>(ng * lo.rec));
        if (lo.PG == 0)
            bulk_copy_g2s(to, src, ng * lo.rec, bar);
        else
            copy_pages(a, sh, to, bar, ng);
    } else {
        const int cnt = left < 128 ? left : 128, c16 = (cnt + 15) & ~15;
        const int row_bytes = lo.scheme == KVQ_SCHEME_INT4 ? D / 2 : D;
        sh.ahead_left = left - cnt;
        sh.ahead_src = src + 128 * row_bytes;
        const uint32_t bytes = static_cast<uint32_t>(c16 * row_bytes);
        mbar_arrive_expect_tx(bar, bytes + (KIND == kRows ? 8 * c16 : 0));
        bulk_copy_g2s(to + 128 * row_bytes, src + (int64_t)lo.T16 * row_bytes, bytes, bar);
        if constexpr (KIND == kRows) {          // the scales: 4 bytes a row from the unit's codes' end on
            const uint8_t* base = a.cache + lo.data_off + unit_index(lo, a.layer, sh.ahead.b, sh.ahead.h) * lo.unit;
            const uint8_t* sc = base + 2 * (int64_t)lo.T16 * row_bytes + (src - base) / row_bytes * 4;
            bulk_copy_g2s(to + 256 * row_bytes, sc, 4 * c16, bar);
            bulk_copy_g2s(to + 256 * row_bytes + 512, sc + 4 * (int64_t)lo.T16, 4 * c16, bar);
        }
    }
}

template <int N, int D, int KIND>
__global__ void __launch_bounds__(TreeShape<N, D>::kThreads, TreeShape<N, D>::kBlocks) k_tree(const __grid_constant__ TreeArgs a) {
    using S = TreeShape<N, D>;
    constexpr int NT = S::kThreads, CT = S::kThreads, NH = S::NH, B = S::B;
    constexpr bool kivi = KIND <= kInPlace, staged_tiles = KIND != kInPlace, fp8 = KIND == kFp8, rows_scheme = KIND == kRows;
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ __align__(16) TreeShared<N, D> sh;

    const Layout& lo = a.lo;
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31, quad = warp & 3, col0 = (warp >> 2) * NH;
    const int row = 32 * quad + lane;                                   // this thread's token of a tile
    const uint32_t lanes = static_cast<uint32_t>(32 * quad) << 16;
    constexpr int WK = fixed_block<KIND>();
    const int H = lo.H, W = WK >= 0 ? WK : key_block(lo);
    uint8_t *kt = smem + S::kK, *vt = smem + S::kV, *qt = smem + S::kQ, *pt = smem + (a.share ? S::kK : S::kP), *stage = smem + a.stage_at;
    const bool rope = kivi && lo.rope_base > 0.0f;
    const int row_bytes = lo.scheme == KVQ_SCHEME_INT4 ? D / 2 : D;     // of a code row

    if (warp == 0) tmem_alloc(&sh.tmem, S::kCols);
    if (tid == 32) {
        mbar_init(&sh.stage_full[0], 1);
        mbar_init(&sh.stage_full[1], 1);
        mbar_init(&sh.keys_full[0], 1);
        mbar_init(&sh.keys_full[1], 1);
        mbar_init(&sh.s_full, 1);
        mbar_init(&sh.pv_done, 1);
        sh.dead = 0;
        sh.odd = 0;
    }
    if (rope)
        for (int i = tid; i < D / 2; i += NT) sh.wt[i] = a.rope_w[place_channel(i, W, D)];
    grid_dependency_wait();
    grid_launch_dependents();
    // this block's tiles: positions [x0, x1) of all tiles, in the order sequence, KV head, row
    // tile, tile
    TreeSeq seq;
    if (tid < lo.B) seq = tree_seq(a, tid, N);
    int64_t total, mine = tid < lo.B ? H * tree_head_tiles(a, seq) : 0;
    int64_t at = block_scan<NT>(mine, sh.scan, &total);
    if (lo.B > NT) total = tree_total<NT>(a, N, sh.scan);
    const int64_t nb = total < a.NB ? total : a.NB;     // blocks with a share
    const int64_t x0 = share_start(total, blockIdx.x, nb), x1 = share_start(total, blockIdx.x + 1, nb);
    for (int b0 = 0;;) {
        if (at <= x0 && x0 < at + mine && static_cast<int64_t>(blockIdx.x) < nb)
            sh.walk.begin(a, seq, b0 + tid, x0 - at, x1 - x0);
        if ((b0 += NT) >= lo.B) break;
        const int64_t base = at + mine;                 // of the last thread: the next round's start
        if (tid == NT - 1) sh.start = base;
        __syncthreads();
        const int b = b0 + tid;
        const int64_t from = sh.start;                  // (read before the scan's barriers: it is written again behind them)
        int64_t sum;
        if (b < lo.B) seq = tree_seq(a, b, N);
        mine = b < lo.B ? H * tree_head_tiles(a, seq) : 0;
        at = from + block_scan<NT>(mine, sh.scan, &sum);
    }
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    const uint32_t tm_s = sh.tmem, tm_o = tm_s + N, my_s = tm_s + lanes + col0;

    auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (mbar_try_wait(bar, parity & 1)) return;
        if (*static_cast<volatile int*>(&sh.dead)) return;
        if (!mbar_wait_asleep(bar, parity & 1)) {
            sh.dead = 1;
            atomicOr(reinterpret_cast<uint32_t*>(a.ws), KVQ_STATUS_TIMEOUT);
        }
    };
    // the stage that the i-th packed tile of this block passes through, and how often it did
    auto slot_of = [&](uint32_t i) { return a.stages == 2 ? i & 1 : 0u; };
    auto turn_of = [&](uint32_t i) { return a.stages == 2 ? i >> 1 : i; };
    if (static_cast<int64_t>(blockIdx.x) < nb) {
        // the walk is kept in shared memory: its fields are needed now and then, and a register
        // that does not hold one of them saves a trip to local memory
        TreeWalk& w = sh.walk;
        if (staged_tiles && warp == CT / 32 - 1 && elect_one()) {
            sh.ahead = w;
            sh.ahead_slot = 0;
            copy_segment<N, D, KIND>(a, sh, false);
            for (int i = 0; i < a.stages; ++i) {
                if constexpr (!kivi) copy_keys<N, D, KIND>(a, sh, stage);
                copy_next<N, D, KIND>(a, sh, stage);
            }
        }
        uint32_t it = 0, used = 0;              // tiles, and packed tiles, so far
        do {
            const int row0 = w.rt * N, row_end = w.s.nodes << a.gshift, first = w.first, end = w.end, packed_end = w.s.packed;
            const bool live = w.live;
            bool mixed = false;
            float gscale = 1.0f;
            float l[NH];
#pragma unroll
            for (int i = 0; i < NH; ++i) l[i] = 0.0f;
            if (live && first < end) {
                // the segment's unpacked rows are needed behind its packed tiles: into L2 meanwhile
                if (end > packed_end)
                    prefetch_rows<D, CT>(a, w.b, w.h, w.s.n, w.s.qn, w.s.nodes, (first > packed_end ? first - packed_end : 0) * 128,
                                         (end - packed_end) * 128, tid);
                const float2 m = load_queries<N, D, KIND>(a, row0, row_end, qt, sh);
                mixed = m.x != 0.0f;
                gscale = m.y;
            }
            bool seen_cached = false;           // a tile with cached tokens is behind us
            for (int tile = first; live && tile < end; ++tile, ++it) {
                const bool packed = tile < packed_end;
                const int cnt = packed ? w.packed_count(a, tile) : w.raw_count(tile);
                int ke = 0, ve = 0;                                     // KIVI: exponents outside binary16
                const uint32_t slot = slot_of(used), turn = turn_of(used);
                const uint8_t* raw = stage + slot * a.stage_bytes;
                PackedTile<staged_tiles> t;
                t.base = raw;
                t.stride = lo.rec;
                t.recs = sh.recs;
                t.cnt = cnt;
                // ---- keys (the scores of the tile before are out of TMEM: its votes are behind a barrier)
                if (!packed) {
                    const int r0 = (tile - w.s.packed) * 128, held = w.s.n - w.s.qn - r0;
                    wait(&sh.pv_done, it + 1);                          // the rows write both tiles
                    raw_rows<D, CT, KIND>(a, w.b, w.h, w.s.n, w.s.qn, r0, cnt, kt, vt, sh.kf, sh.vl, &sh.odd, tid);
                    if (rope) {
                        __syncthreads();
                        turn_keys<D, CT>(kt, sh.wt, (int64_t)w.s.qn + r0, held < cnt ? held : cnt, tid);
                    }
                    smem_to_async();
                    tmem_fence_before();
                    __syncthreads();
                } else {
                    if constexpr (staged_tiles) {
                        wait(kivi ? &sh.stage_full[slot] : &sh.keys_full[slot], turn);
                    } else {
                        // records too large to pass through shared memory next to the tiles
                        if (tid < 8 && tid * lo.G < cnt) {
                            int64_t off = group_offset(lo, a.layer, w.b, w.h, (int64_t)tile * a.TG + tid);
                            if (off < 0) {
                                atomicOr(reinterpret_cast<uint32_t*>(a.ws), KVQ_STATUS_BAD_PAGE);
                                off = lo.data_off + (((int64_t)a.layer * H + w.h) * lo.PG + (tile * a.TG + tid) % lo.PG) * lo.rec;
                            }
                            sh.recs[tid] = a.cache + off;
                        }
                        __syncthreads();
                    }
                    ++used;
                    if (a.share) wait(&sh.pv_done, it + 1);             // the weights lie in the key tile
                    bool wide = false;
                    if constexpr (kivi) {
                        wide = kivi_wide<CT>(a, t, tid);
                        if constexpr (KIND <= kKivi8) kivi_keys<D, KIND, CT>(a, t, kt, tid);
                        if (lo.K > 0 || rope || KIND == kInPlace) {
                            if (__syncthreads_or(wide)) kivi_exponents<CT>(lo, t, sh.top, &ke, &ve, tid);
                            kivi_keys_rest<D, CT>(a, t, kt, sh.wt, (int64_t)tile * a.TT, ke, KIND == kInPlace, W, tid);
                            wide = false;
                        }
                    } else {
                        if constexpr (fp8) fp8_keys<D, CT>(raw, cnt, lo.scheme == KVQ_SCHEME_FP8_E4M3, kt, tid);
                        else rows_codes<D, CT>(raw, cnt, 0, lo.scheme == KVQ_SCHEME_INT8, kt, tid);
                    }
                    smem_to_async();
                    tmem_fence_before();
                    if (__syncthreads_or(wide)) {
                        if constexpr (kivi) {   // some value may be outside binary16: the tile again, scaled
                            kivi_exponents<CT>(lo, t, sh.top, &ke, &ve, tid);
                            if (ke != 0) kivi_keys_rest<D, CT>(a, t, kt, sh.wt, (int64_t)tile * a.TT, ke, false, W, tid);
                            smem_to_async();
                            __syncthreads();
                        }
                    }
                }
                // the tile's key bytes are read
                if constexpr (!kivi) {
                    if (packed && warp == CT / 32 - 1 && elect_one()) copy_keys<N, D, KIND>(a, sh, stage);
                }
                if (warp == 0 && elect_one()) {
                    tmem_fence_after();
                    const uint64_t dk = mma_desc(smem_addr(kt), D / 8 * kCoreBytes), dq = mma_desc(smem_addr(qt), D / 8 * kCoreBytes);
#pragma unroll
                    for (int k = 0; k < D / 16; ++k)
                        mma_f16(tm_s, dk + k * (2 * kCoreBytes >> 4), dq + k * (2 * kCoreBytes >> 4),
                                mma_idesc(128, N, false, false), k > 0);
                    mma_commit(&sh.s_full);
                }
                __syncwarp();
                if (!kivi && packed) wait(&sh.stage_full[slot], turn);      // its values and scales
                // ---- this thread's token: factor of its scores, log2 of its values' scale
                const int tok = packed && !rows_scheme ? packed_token(row) : row;
                const bool valid = tok < cnt, masked = cnt < 128 || !packed;
                int draft = -1;
                float f = 0.0f, lv = 0.0f;
                if (valid) {
                    if (!packed) {
                        f = sh.kf[row];
                        lv = sh.vl[row];
                        draft = (tile - w.s.packed) * 128 + row - (w.s.n - w.s.qn);
                    } else if constexpr (kivi) {
                        f = pow2i(ke);
                        lv = static_cast<float>(ve);
                    } else if constexpr (fp8) {
                        f = sh.kscale;
                        lv = sh.vscale_log;
                    } else {
                        const float* sc = reinterpret_cast<const float*>(raw + 256 * row_bytes);
                        f = sc[tok];
                        lv = fmaxf(fast_log2(sc[128 + tok]), -110.0f);  // (a scale of 0 belongs to codes of 0)
                    }
                    f *= gscale;
                }
                // ---- values, while the scores are computed
                if (packed) {
                    wait(&sh.pv_done, it + 1);                          // the tile before has been read
                    if constexpr (kivi) {
                        if (ve != 0 || KIND == kInPlace) {
                            kivi_values_scaled<D, CT>(lo, t, vt, pow2i(-ve), tid);
                        } else if constexpr (KIND <= kKivi8) {
                            kivi_values<D, KIND, CT>(a, t, vt, tid);
                        }
                        if (lo.K > 0) {
                            __syncthreads();
                            kivi_outliers<D, CT>(lo, t, vt, 1, pow2i(-ve), W, tid);
                        }
                    } else {
                        const uint8_t* vraw = raw + 128 * row_bytes;
                        if constexpr (fp8) fp8_values<D, CT>(vraw, cnt, lo.scheme == KVQ_SCHEME_FP8_E4M3, sh.vscale < 0.0f, vt, tid);
                        else rows_codes<D, CT>(vraw, cnt, 1, lo.scheme == KVQ_SCHEME_INT8, vt, tid);
                    }
                }
                // ---- softmax
                const float inv = tree_exp2(-lv);
                const uint64_t f2 = pack2(f, f), lv2 = pack2(lv, lv), inv2 = pack2(inv, inv);
                // which columns see this token
                uint32_t sees = valid ? 0xffffffffu : 0u;
                if (draft >= 0) {
                    const uint8_t* mask = a.mask ? a.mask + (int64_t)w.b * a.nodes * a.nodes + draft : nullptr;
                    sees = 0u;
#pragma unroll 1
                    for (int c = 0; c < B; c += 8) {        // 8 loads on their way at a time
                        uint32_t bits = 0u;
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const int r = row0 + col0 + c + i, node = r >> a.gshift;
                            const bool in = r < row_end;
                            const uint32_t byte = mask ? (in ? mask[node * a.nodes] : 0u) : (in && draft <= node ? 1u : 0u);
                            bits |= (byte != 0u ? 1u : 0u) << i;
                        }
                        sees |= bits << c;
                    }
                }
                wait(&sh.s_full, it);
                tmem_fence_after();
                // x = score + log2 s, less the column's reference.  Until a column has one, which it
                // surely has behind a tile with cached tokens, the references are set first
                bool fresh = tile == first || (!packed && !seen_cached);
                seen_cached |= packed || (tile - packed_end) * 128 < w.s.n - w.s.qn;
                float x[B];
                for (;;) {
                    tmem_load(my_s, x);
                    if (mixed) {
#pragma unroll
                        for (int i = 0; i < B; ++i) x[i] *= sh.colg[col0 + i];
                    }
#pragma unroll
                    for (int i = 0; i < B; i += 4) {
                        const ulonglong2 r = *reinterpret_cast<const ulonglong2*>(&sh.colr[col0 + i]);
                        const uint64_t u = add2(fma2(pack2(x[i], x[i + 1]), f2, lv2), r.x);
                        const uint64_t v = add2(fma2(pack2(x[i + 2], x[i + 3]), f2, lv2), r.y);
                        unpack2(u, &x[i], &x[i + 1]);
                        unpack2(v, &x[i + 2], &x[i + 3]);
                    }
                    if (masked) {
#pragma unroll
                        for (int i = 0; i < B; ++i) x[i] = sees >> i & 1u ? x[i] : -INFINITY;
                    }
                    float hi = -INFINITY;
#pragma unroll
                    for (int i = 0; i < B; i += 2) hi = max3(hi, x[i], x[i + 1]);
                    if (!__syncthreads_or(fresh || hi > kReach)) break;
                    // the columns' maxima over the tile, the new references, and everything so far
                    // under them
#pragma unroll
                    for (int i = 0; i < B; ++i) {
                        const float m = warp_max(x[i]);
                        if (lane == 0) sh.part[quad][col0 + i] = m;
                    }
                    __syncthreads();
                    for (int c = tid; c < N; c += CT) {
                        const float top = fmaxf(fmaxf(sh.part[0][c], sh.part[1][c]), fmaxf(sh.part[2][c], sh.part[3][c]));
                        const float old = -sh.colr[c], m = top + old - kHead;
                        const bool had = sh.seen[c] != 0, any = top > -INFINITY;
                        const float now = any ? (had ? fmaxf(old, m) : m) : old;
                        sh.seen[c] = had || any;
                        sh.colr[c] = -now;
                        sh.fac[c] = had ? tree_exp2(old - now) : 1.0f;
                    }
                    __syncthreads();
                    if (tile > first) {
#pragma unroll
                        for (int i = 0; i < NH; ++i) l[i] *= sh.fac[col0 + i];
#pragma unroll 1
                        for (int d = 0; d < S::kDN; ++d)
#pragma unroll 1
                            for (int c0 = 0; c0 < NH; c0 += 8) {
                                float o[8];
                                const uint32_t at = tm_o + d * N + lanes + col0 + c0;
                                tmem_load(at, o);
#pragma unroll
                                for (int i = 0; i < 8; ++i) o[i] *= sh.fac[col0 + c0 + i];
                                tmem_store(at, o);
                            }
                    }
                    fresh = false;
                }
                // behind the vote's barrier the tile's packed bytes are read: the next ones may come
                if (staged_tiles && packed && warp == CT / 32 - 1 && elect_one()) copy_next<N, D, KIND>(a, sh, stage);
                __syncwarp();
                uint8_t* prow = pt + (row >> 3) * kCoreBytes + (row & 7) * 16;
#pragma unroll
                for (int c = 0; c < B; c += 8) {
                    uint32_t p[4];
#pragma unroll
                    for (int i = 0; i < 8; i += 2) {
                        const float p0 = tree_exp2(x[c + i]), p1 = tree_exp2(x[c + i + 1]);
                        unpack2(fma2(pack2(p0, p1), inv2, pack2(l[c + i], l[c + i + 1])), &l[c + i], &l[c + i + 1]);
                        p[i / 2] = h2_as_u32(__floats2half2_rn(p0, p1));
                    }
                    *reinterpret_cast<uint4*>(prow + ((col0 + c) >> 3) * (16 * kCoreBytes)) = make_uint4(p[0], p[1], p[2], p[3]);
                }
                smem_to_async();
                tmem_fence_before();
                __syncthreads();
                if (warp == CT / 32 - 2 && elect_one()) {       // (not the warp that issued the scores)
                    tmem_fence_after();
                    const uint64_t dp = mma_desc(smem_addr(pt), 16 * kCoreBytes);
                    const int steps = (cnt + 15) >> 4;
                    const bool mn = !packed || rows_scheme;             // values with channels inside a row
                    const uint32_t idesc = mn ? mma_idesc(128, N, true, true) : mma_idesc(128, N, false, true);
#pragma unroll
                    for (int d = 0; d < S::kDN; ++d) {
                        const uint64_t dv = mma_desc(smem_addr(vt) + d * 32768, 16 * kCoreBytes);
#pragma unroll 4
                        for (int k = 0; k < steps; ++k)
                            mma_f16(tm_o + d * N, dv + k * (2 * kCoreBytes >> 4), dp + k * (2 * kCoreBytes >> 4), idesc,
                                    tile > first || k > 0);
                    }
                    mma_commit(&sh.pv_done);
                }
                __syncwarp();
            }
            // ---------------------------------------------------------- the segment's result
            if (live && first >= end) {         // none of the unit's tiles begins in this share
                finish_empty<N, D>(a, sh);
            } else {
            if (live) wait(&sh.pv_done, it + 1);
            tmem_fence_after();
            // the sums over a column's tokens, through the key tile's memory: [column][token]
            float* sums = reinterpret_cast<float*>(smem);
#pragma unroll
            for (int i = 0; i < NH; ++i) sums[(col0 + i) * 128 + row] = l[i];
            __syncthreads();
            for (int i = tid; i < 4 * N; i += CT) {         // a quarter of a column each, in a fixed order
                float v = 0.0f;
#pragma unroll 8
                for (int j = 0; j < 32; ++j) v += sums[32 * i + ((j + lane) & 31)];
                sh.part[i & 3][i >> 2] = v;
            }
            __syncthreads();
            finish_segment<N, D, rows_scheme>(a, first, tm_o + lanes + col0, row0, row_end, W, sh);
            tmem_fence_before();
            __syncthreads();
            tmem_fence_after();
            }
            if (tid == 0) sh.more = w.next(a, N);
            __syncthreads();
        } while (sh.more);
        // where a wait gave up, the copies in flight land before the block ends
        if (staged_tiles && tid == 0 && sh.dead)
            for (uint32_t i = used; i < used + a.stages; ++i) {
                if (!kivi) mbar_wait_asleep(&sh.keys_full[slot_of(i)], turn_of(i) & 1);
                mbar_wait_asleep(&sh.stage_full[slot_of(i)], turn_of(i) & 1);
            }
    }
    __syncthreads();
    if (warp == 0) tmem_free(tm_s, S::kCols);
}

// Joins the partial results of row tiles that several blocks worked on: a block takes 4 columns
// of one row tile, weighs the blocks' parts by 2^(m - M) and sums their O and l.
constexpr int kMergeColumns = 4;
template <int N, int D>
__global__ void __launch_bounds__(kMergeThreads) k_tree_merge(const __grid_constant__ TreeArgs a) {
    constexpr int CW = kMergeColumns, QUADS = CW * D / 4, GROUPS = kMergeThreads / QUADS;
    __shared__ float2 part[kMaxTreeBlocks * CW];        // (m, l), then (weight, -)
    __shared__ float sum[CW];
    __shared__ float4 red[GROUPS > 1 ? kMergeThreads : 1];
    const Layout& lo = a.lo;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int unit = blockIdx.x / (N / CW), c0 = (blockIdx.x % (N / CW)) * CW;
    const int rt = unit % a.RT, bh = unit / a.RT, b = bh / lo.H, h = bh - b * lo.H, row0 = rt * N + c0;
    // every block waits, also one with nothing to join: the launch after this one may rely on it
    grid_dependency_wait();
    const int2 span = reinterpret_cast<const int2*>(a.ws + a.span_off)[unit];
    if (span.x < 0 || row0 >= a.rows) return;
    const int J = span.y - span.x + 1;
    const int64_t slot0 = (int64_t)span.x + unit;
    const float2* ml = reinterpret_cast<const float2*>(a.ws + a.ml_off) + slot0 * N + c0;
    for (int i = tid; i < J * CW; i += kMergeThreads) part[i] = ml[(int64_t)(i / CW) * N + i % CW];
    __syncthreads();
    if (warp < CW) {
        float M = -INFINITY, L = 0.0f;
        for (int j = lane; j < J; j += 32)
            if (part[j * CW + warp].y != 0.0f) M = fmaxf(M, part[j * CW + warp].x);
        M = warp_max(M);
        for (int j = lane; j < J; j += 32) {
            const float2 x = part[j * CW + warp];
            const float f = x.y != 0.0f ? tree_exp2(x.x - M) : 0.0f;
            L = fmaf(x.y, f, L);
            // a negative weight: nothing was written for this part
            part[j * CW + warp].x = x.x == -INFINITY ? -1.0f : f;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
        if (lane == 0) sum[warp] = L != 0.0f ? 1.0f / L : 0.0f;
    }
    __syncthreads();
    const int quad = tid % QUADS, group = tid / QUADS, c = quad / (D / 4);
    const float4* po = reinterpret_cast<const float4*>(a.ws + a.o_off) + slot0 * (N * D / 4) + c0 * (D / 4) + quad;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    // (a value that is not finite -- a visible draft's -- goes through unweighted)
    auto add = [](float& s, float x, float f) { s += fabsf(x) < INFINITY ? x * f : x; };
#pragma unroll 4
    for (int j = group; j < J; j += GROUPS) {
        const float f = part[j * CW + c].x;
        if (f < 0.0f) continue;
        const float4 x = po[(int64_t)j * (N * D / 4)];
        add(o.x, x.x, f);
        add(o.y, x.y, f);
        add(o.z, x.z, f);
        add(o.w, x.w, f);
    }
    if constexpr (GROUPS > 1) {
        red[tid] = o;
        __syncthreads();
        if (group > 0) return;
        for (int g = 1; g < GROUPS; ++g) {
            const float4 x = red[g * QUADS + quad];
            o.x += x.x;
            o.y += x.y;
            o.z += x.z;
            o.w += x.w;
        }
    }
    const int r = row0 + c;
    if (r >= a.rows) return;
    const float f = sum[c];
    auto out = [&](float x) { return fabsf(x) < INFINITY ? x * f : x; };
    __nv_bfloat162 lo2 = __floats2bfloat162_rn(out(o.x), out(o.y)), hi2 = __floats2bfloat162_rn(out(o.z), out(o.w));
    *reinterpret_cast<uint2*>(a.out + (((int64_t)b * a.nodes + (r >> a.gshift)) * lo.Hq + h * lo.gqa + (r & (lo.gqa - 1))) * D +
                              4 * (quad % (D / 4))) =
        make_uint2(*reinterpret_cast<uint32_t*>(&lo2), *reinterpret_cast<uint32_t*>(&hi2));
}

}  // namespace kvq
