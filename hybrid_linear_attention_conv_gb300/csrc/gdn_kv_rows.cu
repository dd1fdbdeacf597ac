// gdn_kv_rows.cu -- attention over the paged 8-bit cache for few query rows:
// eight rows (queries x heads of one key/value head) at a time, over that
// head's tokens.
//
// For a row with query q, tokens j with key codes c_j, value codes w_j and the
// scales a_j, b_j of their blocks (logits to base 2):
//   s_j = scale log2(e) a_j (q . c_j),   t_j = s_j + log2 b_j,   m = max_j t_j,
//   o   = sum_j 2^(t_j - m) w_j / sum_j 2^(t_j - m) / b_j.
// Taking b_j into the exponent keeps every weight within (0, 1] whatever the
// blocks' scales are, and leaves w_j as the raw codes.
//
// Bound by the cache's bytes: 2 d bytes a token and key/value head, against
// 4 d flops for each of at most eight rows.  Both products run on
// mma.sync.m16n8k16 with the codes, converted exactly to f16, as the 16-row
// operand, and the eight rows as the n = 8 one, so no part of a tile is empty:
//   S^T [tokens x rows] = K Q^T,     O^T [columns x rows] += V^T P^T.
// q (bf16, times a power of two) is exact in f16, a weight, held times 2^15, is within
// 2^-11 of itself, or 2^-40 of the row's largest.
// (mma.sync on e4m3 operands is no shorter way: it took 870 instructions for a tile of
// 32 tokens x 128, with q and the weights as two e4m3 numbers each.  tcgen05's
// tiles of 128 rows would be fifteen sixteenths empty here.)
//
// Layout.  A contraction's index may be permuted as long as both operands
// agree, and so may an output's rows, so everything comes straight from 16-byte
// shared-memory reads and from the thread's own accumulators.  Lane = 4 g + q4:
//   keys    tokens 8 j + g of a 32-token tile, bytes 32 q4 .. 32 q4 + 31 of
//           each 128: chunks 2 q4 and 2 q4 + 1 (c ^ (token & 7) after the swizzle:
//           a quarter-warp's eight chunks fall into eight bank groups);
//   logits  tokens g and g + 8 of each 16, rows 2 q4 and 2 q4 + 1; the weights of eight
//           tokens become the second product's operand by one 8 x 8 transpose;
//   values  tokens 2 q4, 2 q4 + 1 of each eight, chunk g of each 128 columns; bytes of
//           two tokens are paired by a permute before they are converted;
//   output  rows 2 q4 and 2 q4 + 1, columns 16 g .. 16 g + 15 of each 128.
//
// A warp is a worker of its own: it has a ring of tiles that it fills with TMA
// loads and its own m, sum and output, and takes every fourth 32-token tile of
// the CTA's part; nothing synchronises the CTA inside a part.  The list of all
// (request, head, row block, tile) is cut evenly over the CTAs, two or three to an SM;
// a (request, head, row block) that spans several CTAs leaves its parts in the
// workspace, and a second kernel joins them, in CTA order, so results do not
// depend on timing.  (Joined by the last CTA to finish, the 76 parts of an item
// took 15 us and more: one SM's reads, a round after another, by code that the
// stream of the cache had driven out of the L2.)
//
// Measured, 24/4 heads of 256, one token a request: 64 requests of 4,096 to 12,288
// tokens 167 to 171 us (by box) = 6.3 to 6.2 TB/s of cache, 95 to 92 % of a plain copy's rate; one of 131,072 in
// 55 us = 4.9 TB/s and of 4,097 in 11.4 us, where the chain of a launch (scan of
// the requests, table entry, scales, first tile, join) shows.  32/8 heads of 128, 251
// requests of up to 3,000: 131 to 135 us = 5.8 to 5.6 TB/s, with an item's ends once in 47 tiles.
#include <algorithm>
#include <mutex>

#include "gdn_kv.cuh"
#include "gdn_kv_tc.cuh"
#include "gdn_tc.cuh"

namespace gdn {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kTile = 32;               // tokens
constexpr int kRows = 8;
// CTAs of an SM, and a warp's ring (3 units of 8 KB, or 4 of 4 KB): with 256
// columns a thread needs more than the 168 registers that twelve warps leave it.
__host__ __device__ constexpr int per_sm(int d) { return d == 256 ? 2 : 3; }
__host__ __device__ constexpr int ring_bytes(int d) { return d == 256 ? 24 * 1024 : 16 * 1024; }
constexpr float kPScale = 15.0f;        // weights, at most 1, are held times 2^15: f16's largest binade
constexpr uint64_t kDrainNs = 200000000ull;
// An item's beginning and end, in tiles.  251 requests of up to 3,000 tokens, 32/8
// heads of 128: 162 us without, 146 with 4, 132 with 8 and 16; 64 long ones of 256 172,
// 170, 169, 173; one of 4,097 tokens 15.3, 13.9, 11.6, 11.4.
constexpr int kItemCost = 8;
// What a CTA takes at least: fewer CTAs leave fewer parts to join, more share the
// latency.  One request of 4,097 tokens: 11.6 us at 8, 14.5 at 16; longer ones the same.
constexpr int kMinTiles = 8;

template <int D>
struct RowsSmem {
    alignas(1024) uint8_t ring[kWarps][ring_bytes(D)];
    alignas(16) float merge[kRows * D];     // one warp's output on its way to another
    float ml[kWarps][2][kRows];
    alignas(8) uint64_t full[kWarps][4];
    long long scan[kWarps];
    long long at_rest;                      // the CTA's first tile inside request at_b
    int at_b;
};

// A request's part of the list of tiles.  An item (head, row block) takes
// kItemCost places of the list before its tiles' own, so that CTAs with many
// short items get fewer tiles.
struct Request {
    int n, L, row0;        // queries, tokens, first row of q
    int row_blocks, tiles; // of eight rows; of 32 tokens (at least one)
    int items;             // row_blocks * Hkv
    long long work;        // items * (tiles + kItemCost)
};

__device__ __forceinline__ Request request(const KvAttnParams& p, int b) {
    Request r;
    r.row0 = p.start[b];
    r.n = max(0, min(p.start[b + 1], p.T) - r.row0);
    if (r.row0 < 0) r.n = 0;
    r.L = max(0, min(p.lens[b], p.width << p.log2_page));
    r.row_blocks = (r.n * p.G + kRows - 1) / kRows;
    r.tiles = max(1, (r.L + kTile - 1) / kTile);
    r.items = r.row_blocks * p.Hkv;
    r.work = (long long)r.items * (r.tiles + kItemCost);
    return r;
}

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Transpose of an 8 x 8 matrix of f16: lane 4 g + q holds elements 2 q, 2 q + 1 of row g.
__device__ __forceinline__ uint32_t transpose8(uint32_t w) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(w));
    return r;
}

__device__ __forceinline__ uint32_t word_of(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

__device__ __forceinline__ float factor(float m, float top) { return m == top ? 1.0f : ex2(m - top); }

__device__ __forceinline__ float lse_of(float m, float l) {
    return l == 0.0f ? -INFINITY : ((m == -INFINITY ? 0.0f : m) - kPScale + log2f(l)) * 0.69314718055994531f;
}

// A part: an item's rows [8][d] as summed up, their m, their l.
__host__ __device__ constexpr int part_floats(int d) { return kRows * d + 2 * kRows; }

template <int D>
__global__ void __launch_bounds__(kThreads, per_sm(D)) gdn_kv_attn_rows_kernel(const __grid_constant__ KvAttnParams p) {
    constexpr int kUnit = kTile * D;                 // a tile's keys or values
    constexpr int kUnits = ring_bytes(D) / kUnit;
    constexpr int kHalves = D / 128;
    extern __shared__ uint8_t smem_raw[];
    RowsSmem<D>& sm = *reinterpret_cast<RowsSmem<D>*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, q4 = lane & 3;
    const uint8_t* ring = sm.ring[warp];
    const uint32_t ring_at = tc::smem_u32(ring), bars = tc::smem_u32(sm.full[warp]);
    if (lane == 0)
        for (int i = 0; i < kUnits; ++i) tc::mbar_init(bars + 8 * i, 1);
    if (tid == 0) {
        tc::prefetch_map(&p.tm_k);
        tc::prefetch_map(&p.tm_v);
    }
    // A programmatic dependent launch: nothing above touches memory that an earlier kernel may write.
    tc::grid_wait();
    if (tid == 0) p.spans[blockIdx.x] = 0;

    // Where this CTA's part of the list of tiles begins: prefix sums of the
    // requests' work, a stretch of requests to a thread.
    const int per = (p.B + kThreads - 1) / kThreads;
    const int rb0 = min(tid * per, p.B), rb1 = min(rb0 + per, p.B);
    long long mine = 0;
    for (int b = rb0; b < rb1; ++b) mine += request(p, b).work;
    long long upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long u = __shfl_up_sync(~0u, upto, o);
        if (lane >= o) upto += u;
    }
    if (lane == 31) sm.scan[warp] = upto;
    __syncthreads();
    long long total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) upto += sm.scan[w];
        total += sm.scan[w];
    }
    const long long W = max((total + gridDim.x - 1) / gridDim.x, (long long)kMinTiles);  // places a CTA
    const long long x0 = blockIdx.x * W, x1 = min(x0 + W, total);
    if (x0 >= x1) return;  // uniform; nothing is in flight
    if (upto - mine <= x0 && x0 < upto) {
        long long rest = x0 - (upto - mine);
        int b = rb0;
        for (; b < rb1; ++b) {
            const long long w = request(p, b).work;
            if (rest < w) break;
            rest -= w;
        }
        sm.at_b = b;
        sm.at_rest = rest;
    }
    __syncthreads();
    CopyRing<kUnits> units;

    // The stretch at hand: request b's item `item`, tiles t0 .. t1 - 1; x is the
    // place of the list that its place v0 lies at.
    int b = sm.at_b;
    Request r = request(p, b);
    int item = (int)(sm.at_rest / (r.tiles + kItemCost)), v0 = (int)(sm.at_rest - (long long)item * (r.tiles + kItemCost));
    int t0 = 0, t1 = 0;
    long long x = x0;
    auto settle = [&]() {  // false: the CTA's part is done
        while (x < x1) {
            if (item >= r.items) {
                r = request(p, ++b);
                item = 0;
                continue;
            }
            const int v1 = (int)min((long long)r.tiles + kItemCost, v0 + (x1 - x));
            t0 = max(0, v0 - kItemCost);
            t1 = max(0, v1 - kItemCost);
            if (t0 < t1) return true;
            x += v1 - v0;
            v0 = 0;
            ++item;
        }
        return false;
    };
    // This warp's tiles of it: t0 + warp + 4 i, i < nt.  32 tiles' places and
    // scales at a time, a lane each; the ones looked up last, and the ones in use.
    int nt = 0, h = 0, yI = 0;
    float ksI = 0.0f, vsI = 1.0f, ksC = 0.0f, vsC = 1.0f;
    auto lookup = [&](int i0) {
        const int i = i0 + lane;
        if (i < nt) {
            const int pos = (t0 + warp + kWarps * i) * kTile;
            const int idx = pos >> p.log2_page;
            const int page = idx < p.width ? p.table[(int64_t)b * p.width + idx] : -1;
            const bool good = page >= 0 && page < p.pages;
            yI = cache_row(page, p.pages, p.Hkv, h, p.log2_page, pos);
            ksI = good ? p.k_scale[(int64_t)page * p.Hkv + h] : __int_as_float(0x7fffffff);
            vsI = good ? p.v_scale[(int64_t)page * p.Hkv + h] : __int_as_float(0x7fffffff);
        }
    };
    int issued = 0;  // units
    auto issue = [&]() {
        if (issued >= 2 * nt || units.gave_up) return;
        const int i = issued >> 1;
        if ((issued & 63) == 0) lookup(i);
        const int y = __shfl_sync(~0u, yI, i & 31);
        if (tc::elect_one()) {  // (a copy's operands are uniform registers: not under a test of the lane number)
            const void* map = (issued & 1) ? &p.tm_v : &p.tm_k;
            tc::mbar_arrive_expect_tx(bars + 8 * units.send, kUnit);
#pragma unroll
            for (int hf = 0; hf < kHalves; ++hf)
                tc::tma_load_2d(ring_at + units.send * kUnit + hf * (kTile * 128), map, hf * 128, y, bars + 8 * units.send);
        }
        units.sent();
        ++issued;
    };
    auto begin = [&]() {  // the stretch's first copies
        nt = t1 - t0 > warp ? (t1 - t0 - warp + kWarps - 1) / kWarps : 0;
        h = item % p.Hkv;
        issued = 0;
        for (int i = 0; i < kUnits; ++i) issue();
    };

    bool more = settle();
    if (more) begin();
    while (more) {
        // rows of this block: row -> query i, head of the group
        const int block = item / p.Hkv, base = r.L - r.n;  // base: tokens that every query sees
        auto find = [&](int local, int& qi, int64_t& at) {  // at: of the row's output; false: no such row
            const int row = block * kRows + local;
            const bool have = row < r.n * p.G;
            qi = have ? row / p.G : 0;
            at = have ? (int64_t)(r.row0 + qi) * p.Hq + h * p.G + row - qi * p.G : 0;
            return have;
        };
        int qi[2];
        int64_t at[2];
        const bool have[2] = {find(2 * q4, qi[0], at[0]), find(2 * q4 + 1, qi[1], at[1])};
        const int seen[2] = {have[0] ? base + qi[0] + 1 : 0, have[1] ? base + qi[1] + 1 : 0};  // causal: tokens below this
        const int all_see = max(0, min(r.L, p.tree != nullptr ? base : base + (block * kRows) / p.G + 1));
        ksC = ksI;
        vsC = vsI;

        // q (row g), times a power of two that brings its largest to (224, 448], in f16
        uint32_t qb[kHalves * 8][2];
        float rf[2];  // of rows 2 q4 and 2 q4 + 1
        {
            int qig;
            int64_t atg;
            const bool haveg = find(g, qig, atg);
            const uint16_t* src = p.q + (int64_t)(r.row0 + qig) * p.ldq + (atg - (int64_t)(r.row0 + qig) * p.Hq) * D + 32 * q4;
            uint4 w[kHalves][4];
            uint32_t m2 = 0;
#pragma unroll
            for (int hf = 0; hf < kHalves; ++hf)
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    w[hf][c] = haveg ? *reinterpret_cast<const uint4*>(src + hf * 128 + c * 8) : make_uint4(0, 0, 0, 0);
                    m2 = __vmaxu2(m2, w[hf][c].x & 0x7fff7fffu);
                    m2 = __vmaxu2(m2, w[hf][c].y & 0x7fff7fffu);
                    m2 = __vmaxu2(m2, w[hf][c].z & 0x7fff7fffu);
                    m2 = __vmaxu2(m2, w[hf][c].w & 0x7fff7fffu);
                }
            uint32_t top = max(m2 & 0xffffu, m2 >> 16);
            top = max(top, __shfl_xor_sync(~0u, top, 1));
            top = max(top, __shfl_xor_sync(~0u, top, 2));
            const bool finite = top < 0x7f80u;
            const int e = finite ? scale_exp_of_bf16(top) : 0;
            const float inv = exp2_int(-e);
            // a query that is not finite makes its row NaN, through the row's factor
            const float mine = finite ? exp2_int(e) * p.scale_log2 : __int_as_float(0x7fffffff);
            rf[0] = __shfl_sync(~0u, mine, 8 * q4);
            rf[1] = __shfl_sync(~0u, mine, 8 * q4 + 4);
#pragma unroll
            for (int hf = 0; hf < kHalves; ++hf)
#pragma unroll
                for (int c = 0; c < 4; ++c)
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint32_t u = finite ? word_of(w[hf][c], k) : 0u;
                        qb[hf * 8 + 2 * c + (k >> 1)][k & 1] = f16x2(__uint_as_float(u << 16) * inv, __uint_as_float(u & 0xffff0000u) * inv);
                    }
        }

        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
        float o[kHalves * 8][4];
#pragma unroll
        for (int e = 0; e < kHalves * 8; ++e) o[e][0] = o[e][1] = o[e][2] = o[e][3] = 0.0f;

        auto wait_unit = [&]() {
            if (units.gave_up) return;
            if (!__all_sync(~0u, tc::mbar_wait(bars + 8 * units.slot, units.parity, p.wait_ns))) {
                if (lane == 0) report_give_up(p, 1);
                units.gave_up = true;
                CopyRing<kUnits> left = units;  // what is in flight lands before the CTA ends
                for (int i = units.pending(); i > 0; --i, left.read()) tc::mbar_wait(bars + 8 * left.slot, left.parity, kDrainNs);
            }
        };
        auto next_unit = [&]() {
            __syncwarp();
            units.read();
            issue();
        };

        for (int i = 0; i < nt; ++i) {
            const int pos0 = (t0 + warp + kWarps * i) * kTile;
            if ((i & 31) == 0 && i > 0) {
                ksC = ksI;
                vsC = vsI;
            }
            const float ks = __shfl_sync(~0u, ksC, i & 31), vs = __shfl_sync(~0u, vsC, i & 31), lv = __log2f(vs);
            // ---- logits: s[mt] of tokens 16 mt + g (0, 1) and 16 mt + 8 + g (2, 3), rows 2 q4 and 2 q4 + 1
            wait_unit();
            float s[2][4];
#pragma unroll
            for (int mt = 0; mt < 2; ++mt) s[mt][0] = s[mt][1] = s[mt][2] = s[mt][3] = 0.0f;
#pragma unroll
            for (int hf = 0; hf < kHalves; ++hf)
#pragma unroll
                for (int cc = 0; cc < 2; ++cc) {
                    uint4 k[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        k[j] = *reinterpret_cast<const uint4*>(ring + units.slot * kUnit + hf * (kTile * 128) + (8 * j + g) * 128 + (((2 * q4 + cc) ^ g) << 4));
#pragma unroll
                    for (int c = 0; c < 4; ++c)
#pragma unroll
                        for (int mt = 0; mt < 2; ++mt) {
                            const uint32_t w0 = word_of(k[2 * mt], c), w1 = word_of(k[2 * mt + 1], c);
                            const uint32_t(&b)[2] = qb[hf * 8 + cc * 4 + c];
                            mma_f16(s[mt], f16x2_of_e4m3x2(w0), f16x2_of_e4m3x2(w1), f16x2_of_e4m3x2(w0 >> 16), f16x2_of_e4m3x2(w1 >> 16), b[0], b[1]);
                        }
                }
            next_unit();
            // ---- weights
            float t[4][2];  // tokens 8 j + g
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int z = 0; z < 2; ++z) t[j][z] = fmaf(s[j >> 1][2 * (j & 1) + z], rf[z] * ks, lv);
            if (pos0 + kTile > all_see) {  // some row does not see some token
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                    const unsigned long long tree = p.tree != nullptr && have[z] ? (unsigned long long)p.tree[r.row0 + qi[z]] : 0ull;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int pos = pos0 + 8 * j + g, node = pos - base;
                        const bool vis = p.tree != nullptr ? have[z] && pos < r.L && (node < 0 || (node < 64 && ((tree >> (node & 63)) & 1)))
                                                           : pos < seen[z];
                        t[j][z] = vis ? t[j][z] : -INFINITY;
                    }
                }
            }
            float top[2];
#pragma unroll
            for (int z = 0; z < 2; ++z) {
                top[z] = fmaxf(fmaxf(t[0][z], t[1][z]), fmaxf(t[2][z], t[3][z]));
                top[z] = fmaxf(top[z], __shfl_xor_sync(~0u, top[z], 4));
                top[z] = fmaxf(top[z], __shfl_xor_sync(~0u, top[z], 8));
                top[z] = fmaxf(top[z], __shfl_xor_sync(~0u, top[z], 16));
                top[z] = fmaxf(top[z], m[z]);
            }
            if (__any_sync(~0u, top[0] > m[0] || top[1] > m[1])) {
                const float c0 = factor(m[0], top[0]), c1 = factor(m[1], top[1]);
                l[0] *= c0;
                l[1] *= c1;
#pragma unroll
                for (int e = 0; e < kHalves * 8; ++e) {
                    o[e][0] *= c0;
                    o[e][1] *= c1;
                    o[e][2] *= c0;
                    o[e][3] *= c1;
                }
                m[0] = top[0];
                m[1] = top[1];
            }
            uint32_t pb[4];
            {
                const float a0 = kPScale - (m[0] == -INFINITY ? 0.0f : m[0]), a1 = kPScale - (m[1] == -INFINITY ? 0.0f : m[1]);
                float sum[2] = {0.0f, 0.0f};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float e0 = ex2(t[j][0] + a0), e1 = ex2(t[j][1] + a1);  // a token that is not seen: 2^-inf = 0
                    sum[0] += e0;
                    sum[1] += e1;
                    pb[j] = transpose8(f16x2(e0, e1));
                }
                // a row that sees nothing here takes nothing from the block's scale
                const float iv = __fdividef(1.0f, vs);
                if (sum[0] != 0.0f) l[0] = fmaf(sum[0], iv, l[0]);
                if (sum[1] != 0.0f) l[1] = fmaf(sum[1], iv, l[1]);
            }
            // ---- output: column tile e holds columns 16 g + 2 e (0, 1) and 16 g + 2 e + 1 (2, 3)
            wait_unit();
            const bool tail = pos0 + kTile > r.L;
#pragma unroll
            for (int hf = 0; hf < kHalves; ++hf) {
                uint4 v[8];
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    v[k] = *reinterpret_cast<const uint4*>(ring + units.slot * kUnit + hf * (kTile * 128) + (8 * (k >> 1) + 2 * q4 + (k & 1)) * 128 +
                                                           ((g ^ ((2 * q4 + (k & 1)) & 7)) << 4));
                if (tail) {  // whatever lies past the end: zeros
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        if (pos0 + 8 * (k >> 1) + 2 * q4 + (k & 1) >= r.L) v[k] = make_uint4(0, 0, 0, 0);
                }
#pragma unroll
                for (int c = 0; c < 4; ++c)
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const uint32_t sel = half ? 0x7362 : 0x5140;  // bytes 2 half, 2 half + 1 of two tokens, paired
                        uint32_t x[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) x[k] = __byte_perm(word_of(v[2 * k], c), word_of(v[2 * k + 1], c), sel);
#pragma unroll
                        for (int u = 0; u < 2; ++u)
                            mma_f16(o[hf * 8 + 2 * c + half], f16x2_of_e4m3x2(x[2 * u]), f16x2_of_e4m3x2(x[2 * u] >> 16), f16x2_of_e4m3x2(x[2 * u + 1]),
                                    f16x2_of_e4m3x2(x[2 * u + 1] >> 16), pb[2 * u], pb[2 * u + 1]);
                    }
            }
            next_unit();
        }
#pragma unroll
        for (int z = 0; z < 2; ++z) {
            l[z] += __shfl_xor_sync(~0u, l[z], 4);
            l[z] += __shfl_xor_sync(~0u, l[z], 8);
            l[z] += __shfl_xor_sync(~0u, l[z], 16);
        }

        // ---- the next stretch's copies go out before this one's output is put together
        const long long tile0 = x - v0 + kItemCost;  // the place of the item's first tile
        const int c0 = (int)(tile0 / W), c1 = (int)((tile0 + r.tiles - 1) / W);
        const bool from_start = t0 == 0;
        x += t1 + kItemCost - v0;
        v0 = 0;
        ++item;
        more = settle();
        if (more) begin();

        // ---- the four warps' states into warp 0's, one after another
        auto take = [&](float mo0, float mo1, float lo0, float lo1, const float* from) {  // from: this lane's values, 32 lanes apart by float4
            const float top0 = fmaxf(m[0], mo0), top1 = fmaxf(m[1], mo1);
            const float a0 = factor(m[0], top0), a1 = factor(m[1], top1), b0 = factor(mo0, top0), b1 = factor(mo1, top1);
            l[0] = l[0] * a0 + lo0 * b0;
            l[1] = l[1] * a1 + lo1 * b1;
            m[0] = top0;
            m[1] = top1;
#pragma unroll
            for (int e = 0; e < kHalves * 8; ++e) {
                const float4 u = *reinterpret_cast<const float4*>(from + e * 128 + lane * 4);
                o[e][0] = o[e][0] * a0 + u.x * b0;
                o[e][1] = o[e][1] * a1 + u.y * b1;
                o[e][2] = o[e][2] * a0 + u.z * b0;
                o[e][3] = o[e][3] * a1 + u.w * b1;
            }
        };
        auto give = [&](float* to) {
#pragma unroll
            for (int e = 0; e < kHalves * 8; ++e) *reinterpret_cast<float4*>(to + e * 128 + lane * 4) = make_float4(o[e][0], o[e][1], o[e][2], o[e][3]);
        };
        auto merge_warps = [&]() {
            if (g == 0) {
                sm.ml[warp][0][2 * q4] = m[0];
                sm.ml[warp][0][2 * q4 + 1] = m[1];
                sm.ml[warp][1][2 * q4] = l[0];
                sm.ml[warp][1][2 * q4 + 1] = l[1];
            }
            for (int w = 1; w < kWarps; ++w) {
                if (warp == w) give(sm.merge);
                __syncthreads();
                if (warp == 0) take(sm.ml[w][0][2 * q4], sm.ml[w][0][2 * q4 + 1], sm.ml[w][1][2 * q4], sm.ml[w][1][2 * q4 + 1], sm.merge);
                __syncthreads();
            }
        };
        merge_warps();

        // ---- the whole item here: write it; else leave a part
        if (warp == 0 && c0 != c1) {
            float* left = p.partials + ((size_t)blockIdx.x * 2 + (from_start ? 1 : 0)) * part_floats(D);
#pragma unroll
            for (int z = 0; z < 2; ++z) {
                const int local = 2 * q4 + z;
#pragma unroll
                for (int hf = 0; hf < kHalves; ++hf) {
                    float4* dst = reinterpret_cast<float4*>(left + local * D + hf * 128 + 16 * g);
#pragma unroll
                    for (int e = 0; e < 8; e += 2)
                        dst[e / 2] = make_float4(o[hf * 8 + e][z], o[hf * 8 + e][2 + z], o[hf * 8 + e + 1][z], o[hf * 8 + e + 1][2 + z]);
                }
                if (g == 0) {
                    left[kRows * D + local] = m[z];
                    left[kRows * D + kRows + local] = l[z];
                    if (from_start) p.span_rows[blockIdx.x * kRows + local] = have[z] ? at[z] : -1;
                }
            }
            if (tid == 0 && from_start) p.spans[blockIdx.x] = c1 - c0;
        }
        const bool write = warp == 0 && c0 == c1;
        if (write) {
#pragma unroll
            for (int z = 0; z < 2; ++z) {
                if (!have[z]) continue;
                const bool empty = l[z] == 0.0f;  // no token seen: zeros
                const float inv = empty ? 0.0f : 1.0f / l[z];
#pragma unroll
                for (int hf = 0; hf < kHalves; ++hf) {
                    uint4* dst = reinterpret_cast<uint4*>(p.out + at[z] * D + hf * 128 + 16 * g);
                    uint32_t u[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        u[e] = tc::pack_bf16(__float2bfloat16_rn(o[hf * 8 + e][z] * inv), __float2bfloat16_rn(o[hf * 8 + e][2 + z] * inv));
                    dst[0] = make_uint4(u[0], u[1], u[2], u[3]);
                    dst[1] = make_uint4(u[4], u[5], u[6], u[7]);
                }
                if (p.lse != nullptr && g == 0) p.lse[at[z]] = lse_of(m[z], l[z]);
            }
        }
    }
}

// Joins the parts of the item that begins in CTA blockIdx.y and goes on in later
// ones.  A block has 512 consecutive values of the item's eight rows, a lane four times four
// of them; its warps, eight or sixteen, take the parts in turn.
constexpr int kJoinWarps = 16;
template <int D>
__global__ void __launch_bounds__(kJoinWarps * 32) gdn_kv_join_rows_kernel(const int* spans, const int64_t* span_rows, const float* partials,
                                                                           uint16_t* out, float* lse) {
    __shared__ float4 acc[kJoinWarps][4][32];
    __shared__ float ml[kJoinWarps][4][2];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5, c0 = blockIdx.y;
    tc::grid_wait();
    const int more = spans[c0];
    if (more == 0) return;
    auto part_of = [&](int c) { return partials + ((size_t)(c0 + c) * 2 + (c == 0 ? 1 : 0)) * part_floats(D); };
    const int at0 = blockIdx.x * 128 + lane;  // by float4
    float m[4], l[4];
    float4 sum[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        m[k] = -INFINITY;
        l[k] = 0.0f;
        sum[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
#pragma unroll 1
    for (int c = warp; c <= more; c += warps) {
        const float* part = part_of(c);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int row = (blockIdx.x * 128 + k * 32) / (D / 4);
            const float mo = part[kRows * D + row], lo = part[kRows * D + kRows + row];
            const float4 u = reinterpret_cast<const float4*>(part)[at0 + k * 32];
            const float top = fmaxf(m[k], mo), a = factor(m[k], top), b = factor(mo, top);
            m[k] = top;
            l[k] = l[k] * a + lo * b;
            sum[k] = make_float4(sum[k].x * a + u.x * b, sum[k].y * a + u.y * b, sum[k].z * a + u.z * b, sum[k].w * a + u.w * b);
        }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        acc[warp][k][lane] = sum[k];
        if (lane == 0) {
            ml[warp][k][0] = m[k];
            ml[warp][k][1] = l[k];
        }
    }
    __syncthreads();
    if (warp >= 4) return;
    // warp k: the k-th of the block's four stretches of 128 values
    const int k = warp, i4 = at0 + k * 32, row = i4 / (D / 4);
    float top = -INFINITY, total = 0.0f;
    for (int w = 0; w < warps; ++w) top = fmaxf(top, ml[w][k][0]);
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int w = 0; w < warps; ++w) {
        const float f = factor(ml[w][k][0], top);
        const float4 u = acc[w][k][lane];
        total = fmaf(ml[w][k][1], f, total);
        v = make_float4(fmaf(u.x, f, v.x), fmaf(u.y, f, v.y), fmaf(u.z, f, v.z), fmaf(u.w, f, v.w));
    }
    const int64_t to = span_rows[c0 * kRows + row];
    if (to < 0) return;
    const float inv = total == 0.0f ? 0.0f : 1.0f / total;
    const int col = i4 % (D / 4) * 4;
    *reinterpret_cast<uint2*>(out + to * D + col) = make_uint2(tc::pack_bf16(__float2bfloat16_rn(v.x * inv), __float2bfloat16_rn(v.y * inv)),
                                                              tc::pack_bf16(__float2bfloat16_rn(v.z * inv), __float2bfloat16_rn(v.w * inv)));
    if (lse != nullptr && col == 0) lse[to] = lse_of(top, total);
}

template <int D>
cudaError_t launch(KvAttnParams& p, cudaStream_t s) {
    constexpr int smem = (int)sizeof(RowsSmem<D>) + 1024;
    static std::once_flag once[64];
    static cudaError_t err[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || dev < 0 || dev >= 64) return e != cudaSuccess ? e : cudaErrorInvalidDevice;
    std::call_once(once[dev], [dev] {
        err[dev] = cudaFuncSetAttribute(gdn_kv_attn_rows_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    });
    if (err[dev] != cudaSuccess) return err[dev];
    const int grid = std::min(per_sm(D) * device_sm_count(), kKvMaxCtas);
    e = launch_dependent(gdn_kv_attn_rows_kernel<D>, dim3((unsigned)grid), kThreads, smem, s, p);
    if (e != cudaSuccess) return e;
    // Sixteen warps shorten the rounds of an item of many parts (one request of 131,072 tokens,
    // 76 parts an item: 58.0 -> 55.0 us), where every block has a few parts or none they only take
    // longer to place (64 requests: 170.2 -> 173.0).
    const int64_t items = (int64_t)p.B * p.Hkv * std::max<int64_t>(1, ((int64_t)p.T * p.G / p.B + kRows - 1) / kRows);
    const int warps = grid > 8 * items ? kJoinWarps : kJoinWarps / 2;
    return launch_dependent(gdn_kv_join_rows_kernel<D>, dim3(kRows * D / 512, (unsigned)grid), warps * 32, 0, s, (const int*)p.spans,
                            (const int64_t*)p.span_rows, (const float*)p.partials, p.out, p.lse);
}

}  // namespace

size_t kv_attn_rows_workspace(int d) { return (size_t)2 * std::min(per_sm(d) * device_sm_count(), kKvMaxCtas) * part_floats(d) * 4; }

cudaError_t launch_kv_attn_rows(KvAttnParams& p, int d, cudaStream_t s) { return d == 256 ? launch<256>(p, s) : launch<128>(p, s); }

}  // namespace gdn
