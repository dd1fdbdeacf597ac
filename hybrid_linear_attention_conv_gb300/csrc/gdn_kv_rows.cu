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
// mma.sync.m16n8k32 with e4m3 operands, so no code is ever converted: the
// eight rows' q, and their weights, are split into two e4m3 numbers (hi + lo),
// hi in rows 0..7 of the tile and lo in rows 8..15, which this many rows would
// leave empty.  An accumulator's two halves then lie in one thread.
// tcgen05's tiles of 128 rows would be fifteen sixteenths empty here.
//
// Layout.  A contraction's index may be permuted as long as both operands
// agree, and so may an output's columns, so both operands of both products
// come straight from 16-byte shared-memory reads and from the thread's own
// accumulators.  Lane = 4 g + q4:
//   keys    token 8 j + g of a 32-token tile, its bytes 32 q4 .. 32 q4 + 31 of
//           each 128: chunks 2 q4 and 2 q4 + 1 (c ^ (token & 7) after the swizzle:
//           a quarter-warp's eight chunks fall into eight bank groups);
//   logits  row g, tokens 8 j + 2 q4 and + 1;
//   values  for the same eight tokens, chunk g of each 128 columns, transposed
//           4 x 4 bytes at a time; column tile e then holds columns 16 g + e;
//   output  row g, columns 32 q4 + e and 32 q4 + 16 + e: 32 in a row.
//
// A warp is a worker of its own: it has a ring of tiles that it fills with TMA
// loads and its own m, sum and output, and takes every fourth 32-token tile of
// the CTA's part; nothing synchronises the CTA inside a part.  The list of all
// (request, head, row block, tile) is cut evenly over the CTAs, two to an SM;
// a (request, head, row block) that spans several CTAs is joined by the last
// of them to finish, in CTA order, so results do not depend on timing.
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
constexpr int kRingBytes = 24 * 1024;   // a warp's ring: 3 units of 8 KB or 6 of 4 KB
constexpr float kPScale = 8.0f;         // weights are held times 2^8: e4m3 reaches 448
constexpr uint64_t kDrainNs = 200000000ull;
constexpr int kItemCost = 8;            // an item's beginning and end, in tiles
constexpr int kMinTiles = 16;           // what a CTA takes at least

template <int D>
struct RowsSmem {
    alignas(1024) uint8_t ring[kWarps][kRingBytes];
    alignas(16) float merge[kRows * D];     // one warp's output on its way to another
    float ml[kWarps][2][kRows];
    alignas(8) uint64_t full[kWarps][6];
    long long scan[kWarps];
    long long at_rest;                      // the CTA's first tile inside request at_b
    int at_b;
    unsigned last;
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

__device__ __forceinline__ void mma_e4m3(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Bytes of four tokens (words r0..r3, four columns each) to four columns of
// four tokens each.
__device__ __forceinline__ void transpose4(uint32_t r0, uint32_t r1, uint32_t r2, uint32_t r3, uint32_t (&w)[4]) {
    const uint32_t x0 = __byte_perm(r0, r1, 0x5140), x1 = __byte_perm(r0, r1, 0x7362);
    const uint32_t y0 = __byte_perm(r2, r3, 0x5140), y1 = __byte_perm(r2, r3, 0x7362);
    w[0] = __byte_perm(x0, y0, 0x5410);
    w[1] = __byte_perm(x0, y0, 0x7632);
    w[2] = __byte_perm(x1, y1, 0x5410);
    w[3] = __byte_perm(x1, y1, 0x7632);
}

__device__ __forceinline__ uint32_t word_of(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// Running softmax state of one row (row g, the same in its four lanes but for
// l and the output columns, which are the lane's own).
template <int D>
struct RowState {
    float m, l;
    float o[D / 8][2];  // [half * 16 + e]: columns half * 128 + 32 q4 + e and + 16 + e
};

__device__ __forceinline__ float factor(float m, float top) { return m == top ? 1.0f : ex2(m - top); }

template <int D>
__global__ void __launch_bounds__(kThreads, 2) gdn_kv_attn_rows_kernel(const __grid_constant__ KvAttnParams p) {
    constexpr int kUnit = kTile * D;                 // a tile's keys or values
    constexpr int kUnits = kRingBytes / kUnit;
    constexpr int kHalves = D / 128;
    extern __shared__ uint8_t smem_raw[];
    RowsSmem<D>& sm = *reinterpret_cast<RowsSmem<D>*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, q4 = lane & 3;
    const uint8_t* ring = sm.ring[warp];
    const uint32_t ring_at = tc::smem_u32(ring), bars = tc::smem_u32(sm.full[warp]);
    if (lane == 0)
        for (int i = 0; i < kUnits; ++i) tc::mbar_init(bars + 8 * i, 1);

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
    int slot = 0;                 // ring position and parity of the next unit to be read,
    uint32_t parity = 0;
    int islot = 0;                // and position of the next to be filled

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
        if (issued >= 2 * nt) return;
        const int i = issued >> 1;
        if ((issued & 63) == 0) lookup(i);
        const int y = __shfl_sync(~0u, yI, i & 31);
        if (tc::elect_one()) {  // (a copy's operands are uniform registers: not under a test of the lane number)
            const void* map = (issued & 1) ? &p.tm_v : &p.tm_k;
            tc::mbar_arrive_expect_tx(bars + 8 * islot, kUnit);
#pragma unroll
            for (int hf = 0; hf < kHalves; ++hf)
                tc::tma_load_2d(ring_at + islot * kUnit + hf * (kTile * 128), map, hf * 128, y, bars + 8 * islot);
        }
        islot = islot + 1 == kUnits ? 0 : islot + 1;
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
        const int block = item / p.Hkv, row = block * kRows + g;
        const bool have = row < r.n * p.G;
        const int qi = have ? row / p.G : 0, head = h * p.G + (have ? row - qi * p.G : 0);
        const int base = r.L - r.n;                     // tokens that every query sees
        const int seen = have ? base + qi + 1 : 0;      // causal: tokens below this
        const unsigned long long tree = p.tree != nullptr && have ? (unsigned long long)p.tree[r.row0 + qi] : 0ull;
        const int all_see = max(0, min(r.L, p.tree != nullptr ? base : base + (block * kRows) / p.G + 1));
        ksC = ksI;
        vsC = vsI;

        // q as hi + lo, times a power of two that brings its largest to (224, 448]
        uint32_t qa[kHalves * 4][4];
        float rf;
        {
            const uint16_t* src = p.q + (int64_t)(r.row0 + qi) * p.ldq + (int64_t)head * D + 32 * q4;
            uint4 w[kHalves][4];
            uint32_t m2 = 0;
#pragma unroll
            for (int hf = 0; hf < kHalves; ++hf)
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    w[hf][c] = have ? *reinterpret_cast<const uint4*>(src + hf * 128 + c * 8) : make_uint4(0, 0, 0, 0);
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
            rf = finite ? exp2_int(e) * p.scale_log2 : __int_as_float(0x7fffffff);
#pragma unroll
            for (int hf = 0; hf < kHalves; ++hf)
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const uint32_t u[4] = {w[hf][c].x, w[hf][c].y, w[hf][c].z, w[hf][c].w};
                    float f[8];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        f[2 * k] = finite ? __uint_as_float(u[k] << 16) * inv : 0.0f;
                        f[2 * k + 1] = finite ? __uint_as_float(u[k] & 0xffff0000u) * inv : 0.0f;
                    }
                    split4_f16(f[0], f[1], f[2], f[3], qa[hf * 4 + c][0], qa[hf * 4 + c][1]);
                    split4_f16(f[4], f[5], f[6], f[7], qa[hf * 4 + c][2], qa[hf * 4 + c][3]);
                }
        }

        float m = -INFINITY, l = 0.0f;
        float o[kHalves * 16][4];
#pragma unroll
        for (int e = 0; e < kHalves * 16; ++e) o[e][0] = o[e][1] = o[e][2] = o[e][3] = 0.0f;

        auto wait_unit = [&]() {
            if (!tc::mbar_wait(bars + 8 * slot, parity, p.wait_ns)) {
                if (lane == 0) atomicOr(p.status, 1);
                tc::mbar_wait(bars + 8 * slot, parity, kDrainNs);  // the copy lands before its place is used again
            }
        };
        auto next_unit = [&]() {
            __syncwarp();
            if (++slot == kUnits) {
                slot = 0;
                parity ^= 1;
            }
            issue();
        };

        for (int i = 0; i < nt; ++i) {
            const int pos0 = (t0 + warp + kWarps * i) * kTile;
            if ((i & 31) == 0 && i > 0) {
                ksC = ksI;
                vsC = vsI;
            }
            const float ks = __shfl_sync(~0u, ksC, i & 31), vs = __shfl_sync(~0u, vsC, i & 31), lv = __log2f(vs);
            // ---- logits
            wait_unit();
            float s[4][4];
#pragma unroll
            for (int j = 0; j < 4; ++j) s[j][0] = s[j][1] = s[j][2] = s[j][3] = 0.0f;
#pragma unroll
            for (int hf = 0; hf < kHalves; ++hf)
#pragma unroll
                for (int cc = 0; cc < 2; ++cc)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {  // four accumulators in turn: an MMA's result is 22 cycles away
                        const uint4 k = *reinterpret_cast<const uint4*>(ring + slot * kUnit + hf * (kTile * 128) + (8 * j + g) * 128 + (((2 * q4 + cc) ^ g) << 4));
                        mma_e4m3(s[j], qa[hf * 4 + 2 * cc], k.x, k.y);
                        mma_e4m3(s[j], qa[hf * 4 + 2 * cc + 1], k.z, k.w);
                    }
            next_unit();
            // ---- weights
            const float f = rf * ks;
            float t[8];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                t[2 * j] = fmaf(s[j][0] + s[j][2], f, lv);
                t[2 * j + 1] = fmaf(s[j][1] + s[j][3], f, lv);
            }
            if (pos0 + kTile > all_see) {  // some row does not see some token
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const int pos = pos0 + 8 * (k >> 1) + 2 * q4 + (k & 1);
                    const int node = pos - base;
                    const bool vis = p.tree != nullptr ? have && pos < r.L && (node < 0 || (node < 64 && ((tree >> (node & 63)) & 1)))
                                                       : pos < seen;
                    t[k] = vis ? t[k] : -INFINITY;
                }
            }
            float top = t[0];
#pragma unroll
            for (int k = 1; k < 8; ++k) top = fmaxf(top, t[k]);
            top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
            top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
            const float m_new = fmaxf(m, top);
            if (__any_sync(~0u, m_new > m)) {
                const float c = factor(m, m_new);
                l *= c;
#pragma unroll
                for (int e = 0; e < kHalves * 16; ++e) {
                    o[e][0] *= c;
                    o[e][1] *= c;
                    o[e][2] *= c;
                    o[e][3] *= c;
                }
                m = m_new;
            }
            const float shift = kPScale - (m == -INFINITY ? 0.0f : m);
            float w[8], sum = 0.0f;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                w[k] = ex2(t[k] + shift);  // a token that is not seen: 2^-inf = 0
                sum += w[k];
            }
            if (sum != 0.0f) l = fmaf(sum, __fdividef(1.0f, vs), l);  // a row that sees nothing here takes nothing from the block's scale
            uint32_t pa[4];
            {
                split4_f16(w[0], w[1], w[2], w[3], pa[0], pa[1]);
                split4_f16(w[4], w[5], w[6], w[7], pa[2], pa[3]);
            }
            // ---- output
            wait_unit();
            const bool tail = pos0 + kTile > r.L;
#pragma unroll
            for (int hf = 0; hf < kHalves; ++hf) {
                uint4 v[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const int tok = 8 * (k >> 1) + 2 * q4 + (k & 1);
                    v[k] = *reinterpret_cast<const uint4*>(ring + slot * kUnit + hf * (kTile * 128) + tok * 128 + ((g ^ (tok & 7)) << 4));
                    if (tail && pos0 + tok >= r.L) v[k] = make_uint4(0, 0, 0, 0);  // whatever lies past the end
                }
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t b0[4], b1[4];
                    transpose4(word_of(v[0], c), word_of(v[1], c), word_of(v[2], c), word_of(v[3], c), b0);
                    transpose4(word_of(v[4], c), word_of(v[5], c), word_of(v[6], c), word_of(v[7], c), b1);
#pragma unroll
                    for (int k = 0; k < 4; ++k) mma_e4m3(o[hf * 16 + 4 * c + k], pa, b0[k], b1[k]);
                }
            }
            next_unit();
        }
        l += __shfl_xor_sync(~0u, l, 1);
        l += __shfl_xor_sync(~0u, l, 2);

        // ---- the next stretch's copies go out before this one's output is put together
        const long long tile0 = x - v0 + kItemCost;  // the place of the item's first tile
        const int c0 = (int)(tile0 / W), c1 = (int)((tile0 + r.tiles - 1) / W);
        const bool from_start = t0 == 0;
        const int64_t at = (int64_t)(r.row0 + qi) * p.Hq + head;
        x += t1 + kItemCost - v0;
        v0 = 0;
        ++item;
        more = settle();
        if (more) begin();

        // ---- the four warps' states into warp 0's, one after another
        float acc[kHalves * 16][2];
#pragma unroll
        for (int e = 0; e < kHalves * 16; ++e) {
            acc[e][0] = o[e][0] + o[e][2];
            acc[e][1] = o[e][1] + o[e][3];
        }
        auto take = [&](float m_other, float l_other, const float* from) {  // from: this lane's values, 32 lanes apart by float4
            const float top = fmaxf(m, m_other), fa = factor(m, top), fb = factor(m_other, top);
            l = l * fa + l_other * fb;
            m = top;
#pragma unroll
            for (int e = 0; e < kHalves * 16; e += 2) {
                const float4 u = *reinterpret_cast<const float4*>(from + (e / 2) * 128 + lane * 4);
                acc[e][0] = acc[e][0] * fa + u.x * fb;
                acc[e][1] = acc[e][1] * fa + u.y * fb;
                acc[e + 1][0] = acc[e + 1][0] * fa + u.z * fb;
                acc[e + 1][1] = acc[e + 1][1] * fa + u.w * fb;
            }
        };
        auto give = [&](float* to) {
#pragma unroll
            for (int e = 0; e < kHalves * 16; e += 2)
                *reinterpret_cast<float4*>(to + (e / 2) * 128 + lane * 4) =
                    make_float4(acc[e][0], acc[e][1], acc[e + 1][0], acc[e + 1][1]);
        };
        auto merge_warps = [&]() {
            if (q4 == 0) {
                sm.ml[warp][0][g] = m;
                sm.ml[warp][1][g] = l;
            }
            for (int w = 1; w < kWarps; ++w) {
                if (warp == w) give(sm.merge);
                __syncthreads();
                if (warp == 0) take(sm.ml[w][0][g], sm.ml[w][1][g], sm.merge);
                __syncthreads();
            }
        };
        merge_warps();

        // ---- the whole item here: write it; else leave a part, and the last
        // CTA of the item joins them all
        bool write = warp == 0;
        constexpr int kPart = kRows * D + 2 * kRows;
        if (c0 != c1) {
            float* part = p.partials + ((size_t)blockIdx.x * 2 + (from_start ? 1 : 0)) * kPart;
            if (warp == 0) {
                give(part);
                if (q4 == 0) {
                    part[kRows * D + g] = m;
                    part[kRows * D + kRows + g] = l;
                }
                __threadfence();
                __syncwarp();
                if (lane == 0) {
                    const unsigned n = atomicAdd(p.counters + c0, 1u);
                    sm.last = n == (unsigned)(c1 - c0);
                    if (sm.last) p.counters[c0] = 0;  // as the next call finds it
                }
            }
            __syncthreads();
            const bool join = sm.last != 0;
            __syncthreads();
            write = false;
            if (join) {  // uniform in the CTA
                __threadfence();
                m = -INFINITY;
                l = 0.0f;
#pragma unroll
                for (int e = 0; e < kHalves * 16; ++e) acc[e][0] = acc[e][1] = 0.0f;
                for (int c = c0 + warp; c <= c1; c += kWarps) {
                    const float* other = p.partials + ((size_t)c * 2 + (c == c0 ? 1 : 0)) * kPart;
                    take(__ldcg(other + kRows * D + g), __ldcg(other + kRows * D + kRows + g), other);
                }
                merge_warps();
                write = warp == 0;
            }
        }
        if (write && have) {
            const bool empty = l == 0.0f;  // no token seen: zeros
            const float inv = empty ? 0.0f : 1.0f / l;
#pragma unroll
            for (int hf = 0; hf < kHalves; ++hf) {
                uint16_t* dst = p.out + at * D + hf * 128 + 32 * q4;
#pragma unroll
                for (int c = 0; c < 4; ++c) {  // columns 8 c .. 8 c + 7
                    uint32_t u[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int e = (8 * c + 2 * k) & 15, z = c >> 1;
                        u[k] = tc::pack_bf16(__float2bfloat16_rn(acc[hf * 16 + e][z] * inv), __float2bfloat16_rn(acc[hf * 16 + e + 1][z] * inv));
                    }
                    *reinterpret_cast<uint4*>(dst + 8 * c) = make_uint4(u[0], u[1], u[2], u[3]);
                }
            }
            if (p.lse != nullptr && q4 == 0)
                p.lse[at] = empty ? -INFINITY : ((m == -INFINITY ? 0.0f : m) - kPScale + log2f(l)) * 0.69314718055994531f;
        }
    }
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
    const int grid = std::min(2 * device_sm_count(), kKvMaxCtas);
    gdn_kv_attn_rows_kernel<D><<<grid, kThreads, smem, s>>>(p);
    return cudaGetLastError();
}

}  // namespace

size_t kv_attn_rows_workspace(int d) { return (size_t)2 * std::min(2 * device_sm_count(), kKvMaxCtas) * (kRows * d + 2 * kRows) * 4; }

cudaError_t launch_kv_attn_rows(KvAttnParams& p, int d, cudaStream_t s) { return d == 256 ? launch<256>(p, s) : launch<128>(p, s); }

}  // namespace gdn
