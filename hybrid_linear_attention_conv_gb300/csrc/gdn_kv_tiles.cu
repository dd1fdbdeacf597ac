// gdn_kv_tiles.cu -- attention over the paged 8-bit cache for many query rows:
// 128 rows (queries x heads of one key/value head) against 128 tokens at a
// time on the tcgen05 tensor cores.  The mathematics is gdn_kv_rows.cu's: with
// a_j, b_j the scales of token j's blocks,
//   t_j = scale log2(e) a_j (q . c_j) + log2 b_j,   o = sum 2^(t_j - m) w_j / sum 2^(t_j - m) / b_j.
//
// Both products take the cache's codes as they are: q and the weights are split
// into two 8-bit numbers, hi + lo (e4m3; q's lo is e5m2, which makes the pair exact), and
// every contraction runs over both, twice the products at twice bf16's rate,
// with half its bytes of operands and no conversion of a tile.
//
// The weights' product is the block-scaled kind (mxf8f6f4).  A row's weights of 32
// tokens, which share a value scale b, are a block with a power of two of its own, 2^e with the
// block's largest weight in (2^7, 2^8] 2^e, and lo's is 2^(e - 5): a weight is
// within 2^-8 of itself, or within 2^-22 of its block's largest where it is below 2^-14 of that,
// however far the block lies below the row's maximum.  (With one power
// for a whole row the smallest step was 2^-14 of the row's maximum: a flat tail behind
// one token with much of the softmax, or behind a page with a large value scale, was lost.)
//
// Roles of the CTA's 24 warps: one loads tiles (TMA) and their scales; one
// issues the MMAs; sixteen are the softmax, in two teams that take turns at the
// tiles, two threads a row; six split the next item's q, fetched into the L2 an
// item ahead, while the last tiles run.  (A tile's softmax is a chain of
// latencies -- logits out of tensor memory, maximum, exponentials at one every
// 5.5 cycles of a lone pair of warps, stores -- so it is more warps that make it
// short: eight of them took 3,400 cycles a tile and team.)
// Tensor memory: tiles of logits (128 columns each: two for d = 256, three for
// 128), over which their weights are written as the second product's A operand,
// and the output (d columns).  The tensor pipe runs the logits of one or two
// tiles ahead, then O += P V of the tile whose weights are ready.  The exponents of a
// tile's blocks go by way of shared memory, from where the product's issuer copies
// them into columns of the logits that are free by then.
//
// The reference m of a row is raised, and the output rescaled in tensor
// memory, only when a tile's maximum exceeds it by more than 2^8: what
// bounds that is fp32's range (sums of 2^8 times the scales' 2^-100 to 2^120), not the weights' format.
//
// The list of all (request, row tile, head, token tile) is cut evenly over
// the CTAs, one to an SM, causal tiles that nobody sees left out; an item that
// spans several CTAs leaves its parts in the workspace, and a second kernel joins
// them, in CTA order.
//
// Bound by the tensor cores, 8 d flops a row and token (both products, hi and
// lo) at twice bf16's rate, so 4 d at bf16's; for d = 128 by the softmax, whose
// exponentials and moves are the same for half the products.  Measured: a
// prompt of 8,192, 24/4 heads of 256, causal, 578 to 637 us (by box) = 1.43 to 1.29
// PFLOP/s of visible pairs, about 3,000 cycles a tile of 128 x 128 against
// 2,048 of products; 1,024 queries after 30,000 tokens 475 us = 1.62 PFLOP/s.
// d = 128: 2,300 cycles a tile against 1,024 (1,024 queries of 32/8 heads after 30,000
// tokens 458 us).  ptxas spills 100 B of stores a thread for d = 128 and 40 for 256
// around the tile loop's 88 registers.  Small steps pay 20 to 25 us beside
// their tiles: the list and the first q 7 to 10, an item's beginning and end, the
// join's launch and reads.
#include <algorithm>
#include <mutex>

#include "gdn_kv.cuh"
#include "gdn_kv_tc.cuh"
#include "gdn_tc.cuh"

namespace gdn {
namespace {

constexpr int kSoftWarps = 16, kQWarps = 6;
constexpr int kLoadWarp = kSoftWarps, kMmaWarp = kSoftWarps + 1, kQWarp0 = kSoftWarps + 2, kMmaWarp2 = kSoftWarps + 7;
constexpr int kThreads = (kSoftWarps + 2 + kQWarps) * 32;
constexpr int kTeamWarps = kSoftWarps / 2;
constexpr int kM = 128;                 // rows of an item
constexpr int kN = 128;                 // tokens of a tile
constexpr float kGrow = 8.0f;           // how far a weight may exceed the reference, in powers of two
constexpr float kBlockExp = 8.0f;       // a block's largest weight is held at most 2^8,
constexpr int kLoExp = 5;               // and what is left of a weight times 2^5
constexpr int kScaleRing = 8;
constexpr int kSoftRegs = 88, kOtherRegs = 64;  // 512 x 88 + 256 x 64 = 768 x 80
// An item's beginning and end, in tiles (the 8,192-token prompt took 606 us at 6, and 864,
// 637, 619, 628 at 2, 4, 8, 10).
constexpr int kItemCost = 6;
constexpr int kMinTiles = 8;            // what a CTA takes at least
constexpr uint64_t kDrainNs = 200000000ull;

template <int D>
struct TilesSmem {
    static constexpr int kSlot = kN * D;                      // a tile's keys or values
    static constexpr int kSlots = D == 256 ? 4 : 8;
    static constexpr int kBufs = D == 256 ? 2 : 3;            // tiles of logits in tensor memory
    static constexpr int kQBufs = D == 256 ? 1 : 2;           // items' q
    static constexpr bool kTwo = D == 128;                    // two warps issue MMAs
    static constexpr bool kEarly = D == 256;                  // the product starts on half the weights
    alignas(1024) uint8_t q[kQBufs][2][kM * D];               // hi, lo
    alignas(1024) uint8_t ring[kSlots][kSlot];
    float2 scales[kScaleRing][4];                             // of 32 tokens: key scale, log2 of the value scale
    float rf[kQBufs][kM];
    float ref[2][2][kM];                                      // the rows' references after a team's tiles, two of them in turn
    float top[2][2][2][kM];                                   // by team and half: the rows' maxima of two tiles in turn
    float ml[2][2][kM], mr[2][2][2][kM];                      // by item: the teams' references; each half's sum
    // exponents of a tile's blocks: for tokens 0 .. 31 of each half, and 32 .. 63, row 32 j + i's word
    // at 16 i + 4 j, byte 2 half + part; and a page of exponents 0 for the values
    alignas(128) uint8_t block_exp[kBufs][2][512], no_exp[512];
    union {
        alignas(16) uint8_t stage[kSoftWarps][32 * 32];       // a warp's 32 rows x 16 columns of output on their way out
        int qbase[kThreads];                                  // (before the first item)
    };
    alignas(8) uint64_t full[kSlots], empty[kSlots], s_full[kBufs], p_ready[2][kBufs], o_done[kBufs], scales_full[kScaleRing];
    uint64_t q_full[kQBufs], q_empty[kQBufs], item_done, o_free, drained;
    long long scan[kThreads / 32];
    int at_b, at_t, at_h, at_v;
    uint32_t tmem;
    int dead;
};

struct Request {
    int n, L, row0, tiles;  // queries, tokens, first row of q, row tiles
};

__device__ __forceinline__ Request request(const KvAttnParams& p, int b) {
    Request r;
    r.row0 = p.start[b];
    r.n = max(0, min(p.start[b + 1], p.T) - r.row0);
    if (r.row0 < 0) r.n = 0;
    r.L = max(0, min(p.lens[b], p.width << p.log2_page));
    r.tiles = (r.n * p.G + kM - 1) / kM;
    return r;
}

// Token tiles that some row of row tile t sees (at least one).
__device__ __forceinline__ int token_tiles(const KvAttnParams& p, const Request& r, int t) {
    const int last = min(r.n - 1, (t * kM + kM - 1) / p.G);
    const int seen = p.tree != nullptr ? r.L : min(r.L, r.L - r.n + last + 1);
    return max(1, (seen + kN - 1) / kN);
}

// One stretch of an item's token tiles, and the walk over a CTA's stretches.  An
// item takes kItemCost places of the list before its tiles' own, so that CTAs
// with many short items get fewer tiles.
struct Walk {
    int b, t, h, v0, j0, j1, kt;
    long long x, x1;
    Request r;
    __device__ __forceinline__ bool settle(const KvAttnParams& p) {  // false: the CTA's part is done
        while (x < x1) {
            r = request(p, b);
            while (t >= r.tiles) {
                t = 0;
                r = request(p, ++b);
            }
            kt = token_tiles(p, r, t);
            const int v1 = (int)min((long long)kt + kItemCost, v0 + (x1 - x));
            j0 = max(0, v0 - kItemCost);
            j1 = max(0, v1 - kItemCost);
            if (j0 < j1) return true;
            next(p, v1);
        }
        return false;
    }
    __device__ __forceinline__ void next(const KvAttnParams& p, int v1) {
        x += v1 - v0;
        v0 = 0;
        if (++h == p.Hkv) {
            h = 0;
            ++t;
        }
    }
    __device__ __forceinline__ void advance(const KvAttnParams& p) { next(p, j1 + kItemCost); }
};

// Rows of an item -> query and head of the group, without a division for each:
// local + rem < G + 128 <= 1152, and x * ceil(2^22 / G) >> 22 is x / G there.
struct RowMap {
    int G, q0, rem;
    unsigned magic;
    __device__ __forceinline__ RowMap(const KvAttnParams& p, int t) {
        G = p.G;
        q0 = t * kM / G;
        rem = t * kM - q0 * G;
        magic = p.group_magic;
    }
    __device__ __forceinline__ void find(int local, int& q, int& h) const {
        const int x = rem + local, d = (int)(((unsigned)x * magic) >> 22);
        q = q0 + d;
        h = x - d * G;
    }
};

__device__ __forceinline__ float factor(float m, float top) { return m == top ? 1.0f : ex2(m - top); }

__device__ __forceinline__ float lse_of(float m, float l) {
    return l == 0.0f ? -INFINITY : ((m == -INFINITY ? 0.0f : m) + log2f(l)) * 0.69314718055994531f;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) gdn_kv_attn_tiles_kernel(const __grid_constant__ KvAttnParams p) {
    using Smem = TilesSmem<D>;
    constexpr int kSlot = Smem::kSlot, kSlots = Smem::kSlots, kBufs = Smem::kBufs, kQBufs = Smem::kQBufs, kHalves = D / 128;
    constexpr bool kTwo = Smem::kTwo, kEarly = Smem::kEarly;
    constexpr int kQ = kTwo ? kQWarps - 1 : kQWarps;  // warps that split q
    constexpr uint32_t kHalfBytes = kN * 128;
    constexpr int kPart = kM * D + 2 * kM;
    extern __shared__ uint8_t smem_raw[];
    Smem& sm = *reinterpret_cast<Smem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

    if (tid == 0) {
        tc::prefetch_map(&p.tm_k);
        tc::prefetch_map(&p.tm_v);
    }
    tc::grid_wait();  // nothing above touches memory that an earlier kernel may write
    if (tid == 0) p.spans[blockIdx.x] = 0;

    // ---- this CTA's part of the list
    const int per = (p.B + kThreads - 1) / kThreads;
    const int rb0 = min(tid * per, p.B), rb1 = min(rb0 + per, p.B);
    auto scan = [&](long long v, long long& total) {  // exclusive prefix over the CTA's threads
        long long u = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long w = __shfl_up_sync(~0u, u, o);
            if (lane >= o) u += w;
        }
        if (lane == 31) sm.scan[warp] = u;
        __syncthreads();
        total = 0;
        for (int w = 0; w < kThreads / 32; ++w) {
            if (w < warp) u += sm.scan[w];
            total += sm.scan[w];
        }
        __syncthreads();
        return u - v;
    };
    long long mine = 0, total = 0;
    for (int b = rb0; b < rb1; ++b) mine += request(p, b).tiles;
    sm.qbase[tid] = (int)scan(mine, total);
    __syncthreads();
    const int nq = (int)total, perq = (nq + kThreads - 1) / kThreads;
    const int q0 = min(tid * perq, nq), q1 = min(q0 + perq, nq);
    int b0 = 0, t0 = 0;  // the first of this thread's row tiles
    mine = 0;
    if (q0 < q1) {
        int lo = 0, hi = kThreads;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (sm.qbase[mid] <= q0) lo = mid;
            else hi = mid;
        }
        b0 = lo * per;
        t0 = q0 - sm.qbase[lo];
        Request r = request(p, b0);
        for (; t0 >= r.tiles; r = request(p, ++b0)) t0 -= r.tiles;
        int b = b0, t = t0;
        for (int q = q0; q < q1; ++q, ++t) {
            while (t >= r.tiles) {
                t = 0;
                r = request(p, ++b);
            }
            mine += token_tiles(p, r, t) + kItemCost;
        }
    }
    const long long before = scan(mine, total) * p.Hkv;
    total *= p.Hkv;
    const long long W = max((total + gridDim.x - 1) / gridDim.x, (long long)kMinTiles);
    const long long x0 = blockIdx.x * W, x1 = min(x0 + W, total);
    if (x0 >= x1) return;  // uniform; nothing is in flight
    if (before <= x0 && x0 < before + mine * p.Hkv) {
        long long rest = x0 - before;
        int b = b0, t = t0;
        Request r = request(p, b);
        for (;; ++t) {
            while (t >= r.tiles) {
                t = 0;
                r = request(p, ++b);
            }
            const int len = token_tiles(p, r, t) + kItemCost;
            if (rest < (long long)len * p.Hkv) {
                sm.at_b = b;
                sm.at_t = t;
                sm.at_h = (int)(rest / len);
                sm.at_v = (int)(rest % len);
                break;
            }
            rest -= (long long)len * p.Hkv;
        }
    }

    // ---- barriers and tensor memory
    const uint32_t full = tc::smem_u32(sm.full), empty = tc::smem_u32(sm.empty), s_full = tc::smem_u32(sm.s_full),
                   p_ready = tc::smem_u32(sm.p_ready), scales_full = tc::smem_u32(sm.scales_full),
                   q_full = tc::smem_u32(sm.q_full), q_empty = tc::smem_u32(sm.q_empty),
                   o_done = tc::smem_u32(sm.o_done), o_free = tc::smem_u32(&sm.o_free), item_done = tc::smem_u32(&sm.item_done),
                   drained = tc::smem_u32(&sm.drained);
    if (tid == 0) {
        sm.dead = 0;
        for (int i = 0; i < kSlots; ++i) {
            tc::mbar_init(full + 8 * i, 1);
            tc::mbar_init(empty + 8 * i, 1);
        }
        for (int i = 0; i < kBufs; ++i) {
            tc::mbar_init(s_full + 8 * i, 1);
            tc::mbar_init(o_done + 8 * i, 1);
            tc::mbar_init(p_ready + 8 * i, kTeamWarps);
            tc::mbar_init(p_ready + 8 * (kBufs + i), kTeamWarps);
        }
        for (int i = 0; i < kScaleRing; ++i) tc::mbar_init(scales_full + 8 * i, 1);
        for (int i = 0; i < kQBufs; ++i) {
            tc::mbar_init(q_full + 8 * i, kQ);
            tc::mbar_init(q_empty + 8 * i, 1 + kSoftWarps);
        }
        tc::mbar_init(o_free, kSoftWarps);
        tc::mbar_init(item_done, 1);
        tc::mbar_init(drained, kTwo ? 2 : 1);
    }
    if (tid < 128) reinterpret_cast<uint32_t*>(sm.no_exp)[tid] = 0x7f7f7f7fu;
    tc::fence_async_smem();
    if (warp == kMmaWarp) tc::tmem_alloc(tc::smem_u32(&sm.tmem), 512);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = sm.tmem, tO = tmem + kBufs * kN;  // logits and weights before the output
    volatile int* dead = &sm.dead;

    // A bounded wait.  The first that gives up ends all waiting of the CTA, and its
    // copies: the roles run through on whatever is there, and the status word tells.
    // (Arrivals without bytes may then come in any number: a phase just completes.)
    auto wait = [&](uint32_t bar, uint32_t parity) {
        parity &= 1;
        if (tc::mbar_test(bar, parity)) return;
        if (*dead) return;
        if (!tc::mbar_wait(bar, parity, p.wait_ns)) {
            *dead = 1;
            report_give_up(p, 2);
        }
    };

    Walk w;
    w.b = sm.at_b;
    w.t = sm.at_t;
    w.h = sm.at_h;
    w.v0 = sm.at_v;
    w.x = x0;
    w.x1 = x1;

    // Warp me of n splits its share of the rows of v's item into q's buffer qb.
    auto split_q = [&](const Walk& v, int qb, int me, int n, auto&& may_write) {
        constexpr int kLanes = D / 16;              // of a row, 16 values each
        constexpr int kAtOnce = 32 / kLanes;        // rows of a warp's step
        constexpr int kBatch = 2;                   // steps whose loads go out together
        const int sub = lane / kLanes, c = lane % kLanes;
        const int rows = min(v.r.n * p.G - v.t * kM, kM);
        const RowMap map(p, v.t);
#pragma unroll 1
        for (int i0 = me; i0 < kM / kAtOnce; i0 += kBatch * n) {
            uint4 x[kBatch][2];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int local = (i0 + i * n) * kAtOnce + sub;
                x[i][0] = x[i][1] = make_uint4(0, 0, 0, 0);
                if (local < rows) {
                    int qi, hg;
                    map.find(local, qi, hg);
                    const uint4* src = reinterpret_cast<const uint4*>(p.q + (int64_t)(v.r.row0 + qi) * p.ldq + (int64_t)(v.h * p.G + hg) * D) + 2 * c;
                    x[i][0] = src[0];
                    x[i][1] = src[1];
                }
            }
            may_write();
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int local = (i0 + i * n) * kAtOnce + sub;
                if (i0 + i * n >= kM / kAtOnce) break;  // uniform in the warp
                const uint32_t word[8] = {x[i][0].x, x[i][0].y, x[i][0].z, x[i][0].w, x[i][1].x, x[i][1].y, x[i][1].z, x[i][1].w};
                uint32_t m2 = 0;
#pragma unroll
                for (int k = 0; k < 8; ++k) m2 = __vmaxu2(m2, word[k] & 0x7fff7fffu);
                uint32_t top = max(m2 & 0xffffu, m2 >> 16);
#pragma unroll
                for (int o = 1; o < kLanes; o <<= 1) top = max(top, __shfl_xor_sync(~0u, top, o));
                const bool finite = top < 0x7f80u;
                const int e = finite ? scale_exp_of_bf16(top) : 0;
                const float inv = exp2_int(-e);
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t a = finite ? word[2 * k] : 0u, b = finite ? word[2 * k + 1] : 0u;
                    split4_queries(__uint_as_float(a << 16) * inv, __uint_as_float(a & 0xffff0000u) * inv, __uint_as_float(b << 16) * inv,
                               __uint_as_float(b & 0xffff0000u) * inv, hi[k], lo[k]);
                }
                const uint32_t at = (c >> 3) * (kM * 128) + local * 128 + (((c & 7) ^ (local & 7)) << 4);
                *reinterpret_cast<uint4*>(sm.q[qb][0] + at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                *reinterpret_cast<uint4*>(sm.q[qb][1] + at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                // a query that is not finite makes its row NaN, through the row's factor
                if (c == 0) sm.rf[qb][local] = finite ? exp2_int(e) * p.scale_log2 : __int_as_float(0x7fffffff);
            }
        }
        tc::fence_async_smem();
    };

    // Inside the branches: code after a join of the two would have to fit the smaller number.
    if (warp >= kSoftWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == kLoadWarp) {
        // ------------------------------------------------------------ tiles
        const int page_rows = 1 << p.log2_page;  // of a box: 32, 64 or 128
        int u = 0, g = 0, issued = 0;  // ring units (keys, values), tiles
        for (; w.settle(p); w.advance(p)) {
            // eight tiles' places and scales at a time: lane = 4 tile + 32-token stretch
            int y = 0, y_next = 0;
            float ks = 0.0f, lv = 0.0f, ks_next = 0.0f, lv_next = 0.0f;
            auto lookup = [&](int j) {
                const int pos = (j + (lane >> 2)) * kN + (lane & 3) * 32, idx = pos >> p.log2_page;
                const int page = pos < w.r.L && idx < p.width ? p.table[(int64_t)w.b * p.width + idx] : -1;
                const bool good = page >= 0 && page < p.pages;
                y_next = cache_row(page, p.pages, p.Hkv, w.h, p.log2_page, pos);
                ks_next = good ? p.k_scale[(int64_t)page * p.Hkv + w.h] : __int_as_float(0x7fffffff);
                lv_next = good ? log2f(p.v_scale[(int64_t)page * p.Hkv + w.h]) : __int_as_float(0x7fffffff);
            };
            lookup(w.j0);
            for (int j = w.j0; j < w.j1; ++j, ++g) {
                const int k = (j - w.j0) & 7;
                if (k == 0) {
                    y = y_next;
                    ks = ks_next;
                    lv = lv_next;
                    lookup(j + 8);
                }
#pragma unroll
                for (int kv = 0; kv < 2; ++kv, ++u) {
                    const int slot = u % kSlots;
                    if (u >= kSlots) wait(empty + 8 * slot, u / kSlots - 1);
                    if (kv == 0) {
                        // the place in the ring is free: its last readers were done before the
                        // weights of the tile whose keys lay in this slot were
                        if ((lane >> 2) == k) sm.scales[g % kScaleRing][lane & 3] = make_float2(ks, lv);
                        __syncwarp();
                        if (lane == 0) tc::mbar_arrive(scales_full + 8 * (g % kScaleRing));
                    }
                    // Never into a slot whose wait gave up: a second arrival in a phase that still
                    // awaits its bytes is a fault.  (A wait that returned for `dead` sees it set here.)
                    if (*dead) continue;
                    issued = u + 1;
                    const uint32_t dst = tc::smem_u32(sm.ring[slot]);
                    int row[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) row[i] = __shfl_sync(~0u, y, 4 * k + i);
                    const void* map = kv ? &p.tm_v : &p.tm_k;
                    if (tc::elect_one()) {  // (a copy's operands are uniform registers: not under a test of the lane number)
                        tc::mbar_arrive_expect_tx(full + 8 * slot, kSlot);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if ((i * 32) % page_rows == 0)
#pragma unroll
                                for (int hf = 0; hf < kHalves; ++hf)
                                    tc::tma_load_2d(dst + hf * kHalfBytes + i * 32 * 128, map, hf * 128, row[i], full + 8 * slot);
                    }
                    __syncwarp();
                }
            }
        }
        // Copies that nobody waited for (after a wait that gave up) land before the CTA ends.
        for (int i = max(0, issued - kSlots); i < issued; ++i) tc::mbar_wait(full + 8 * (i % kSlots), (i / kSlots) & 1, kDrainNs);
    } else if (warp == kMmaWarp || (kTwo && warp == kMmaWarp2)) {
        // ------------------------------------------------------------- MMAs
        // A whole warp walks and waits; one elected lane issues.  (An MMA takes its
        // descriptors from uniform registers: under a test of the lane number
        // instead, each one costs about 185 cycles of issue, three times its own 64.)
        // Beside the softmax a tile's issue takes about 850 cycles a product.  For
        // d = 256, where the products take 1,024 each, one warp issues both, and the
        // tensor pipe's order keeps a tile's weights until their product has read
        // them; for d = 128 (512 each) a warp for each, the logits' one waiting for that product.
        constexpr uint32_t id_hi = tc::idesc_f8(kM, kN, false), id_lo = tc::idesc_f8(kM, kN, true);
        const uint32_t ring = tc::smem_u32(sm.ring[0]);
        auto logits = [&](int g, int qb, bool last) {
            const int u = 2 * g, slot = u % kSlots, buf = g % kBufs;
            wait(full + 8 * slot, u / kSlots);
            tc::fence_after_sync();
            const uint64_t q_hi = tc::smem_desc_sw128(tc::smem_u32(sm.q[0][0]) + qb * 2 * kM * D), q_lo = q_hi + (kM * D >> 4);
            const uint64_t k = tc::smem_desc_sw128(ring + slot * kSlot);
            const uint32_t d = tmem + buf * kN;
            if (tc::elect_one()) {
#pragma unroll
                for (int part = 0; part < 2; ++part)
#pragma unroll
                    for (int ks = 0; ks < D / 32; ++ks) {
                        const uint32_t at = ((ks >> 2) * kHalfBytes + (ks & 3) * 32) >> 4;
                        tc::mma_f8(d, (part ? q_lo : q_hi) + at, k + at, part ? id_lo : id_hi, part + ks > 0);
                    }
                tc::mma_commit(empty + 8 * slot);
                tc::mma_commit(s_full + 8 * buf);
                if (last) tc::mma_commit(q_empty + 8 * qb);
            }
            __syncwarp();
        };
        auto product = [&](int g, int item, bool first, bool last) {
            const int u = 2 * g + 1, slot = u % kSlots, buf = g % kBufs;
            if (first && item > 0) wait(o_free, item - 1);
            wait(full + 8 * slot, u / kSlots);
            const uint64_t v = tc::smem_desc_mn_sw128(ring + slot * kSlot, kHalfBytes);
            const uint32_t a = tmem + buf * kN;
            // the exponents: columns 16 .. 31 of the logits, whose readers were done before the weights were
            const uint32_t exps = a + 16, no_exps = exps + 8;
            const uint64_t from = tc::smem_desc_rows16(tc::smem_u32(sm.block_exp[buf][0])), none = tc::smem_desc_rows16(tc::smem_u32(sm.no_exp));
            // kEarly: the weights come in two halves, of tokens 0 .. 31 and 64 .. 95 first, and the
            // product of those runs while the others' exponentials do (d = 256: 529 -> 511 us for 1,024
            // queries after 30,000 tokens; d = 128, where the softmax is the longer, 369 -> 388 us)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                if (kEarly || c == 0) {
                    wait(p_ready + 8 * (c * kBufs + buf), g / kBufs);
                    tc::fence_after_sync();
                }
                if (tc::elect_one()) {
                    if (c == 0)
#pragma unroll
                        for (int n = 0; n < kHalves; ++n) tc::copy_scales(no_exps + 4 * n, none);
                    tc::copy_scales(exps + 4 * c, from + (c * 512 >> 4));
#pragma unroll
                    for (int half = 0; half < 2; ++half)
#pragma unroll
                        for (int part = 0; part < 2; ++part)
                            tc::mma_mx_e4m3_ts(tO, a + half * 64 + c * 32 + part * 8, v + ((2 * half + c) * 32 * 128 >> 4),
                                               tc::idesc_mx_e4m3(kM, D, 2 * half + part), exps + 4 * c, no_exps, c + half + part > 0 || !first);
                }
                __syncwarp();
            }
            if (tc::elect_one()) {
                tc::mma_commit(empty + 8 * slot);
                tc::mma_commit(o_done + 8 * buf);
                if (last) tc::mma_commit(item_done);
            }
            __syncwarp();
        };
        if constexpr (kTwo) {
            int g = 0, item = 0;
            for (; w.settle(p); w.advance(p), ++item) {
                if (warp == kMmaWarp) wait(q_full + 8 * (item % kQBufs), item / kQBufs);
                for (int j = w.j0; j < w.j1; ++j, ++g) {
                    if (warp == kMmaWarp) {
                        if (g >= kBufs) wait(o_done + 8 * (g % kBufs), g / kBufs - 1);
                        logits(g, item % kQBufs, j == w.j1 - 1);
                    } else {
                        product(g, item, j == w.j0, j == w.j1 - 1);
                    }
                }
            }
        } else {
            int gs = 0, gp = 0;                   // tiles whose logits, whose product have been issued
            uint32_t firsts = 0, lasts = 0;       // of the items, by tile modulo 32
            int item = 0, item_p = 0;
            auto product_next = [&]() {
                const bool last = (lasts >> (gp & 31)) & 1;
                product(gp, item_p, (firsts >> (gp & 31)) & 1, last);
                if (last) ++item_p;
                ++gp;
            };
            for (; w.settle(p); w.advance(p), ++item) {
                const int qb = item % kQBufs;
                // the products that are due first, unless this item's q is there already
                if (!__all_sync(~0u, tc::mbar_test(q_full + 8 * qb, (item / kQBufs) & 1)))
                    while (gp < gs) product_next();
                wait(q_full + 8 * qb, item / kQBufs);
                for (int j = w.j0; j < w.j1; ++j) {
                    while (gp <= gs - kBufs) product_next();  // the buffer's last reader
                    logits(gs, qb, j == w.j1 - 1);
                    const uint32_t bit = 1u << (gs & 31);
                    firsts = j == w.j0 ? firsts | bit : firsts & ~bit;
                    lasts = j == w.j1 - 1 ? lasts | bit : lasts & ~bit;
                    ++gs;
                }
            }
            while (gp < gs) product_next();
        }
        // every MMA has ended before tensor memory is given back
        if (tc::elect_one()) tc::mma_commit(drained);
        __syncwarp();
        tc::mbar_wait(drained, 0, kDrainNs);
    } else {
        // ----------------------------------------------------------- queries
        // The first item's rows are split by the softmax's warps too, which have nothing to do yet.
        int item = 0;
        auto fetch = [&]() {  // an item's rows towards the L2 (a row is 2 or 4 lines)
            const int rows_next = w.r.n * p.G - w.t * kM;
            const RowMap map_next(p, w.t);
#pragma unroll 1
            for (int i = (warp - kQWarp0) * 32 + lane; i < kM * (D / 64); i += kQ * 32) {
                const int local = i / (D / 64);
                if (local < rows_next) {
                    int qi, hg;
                    map_next.find(local, qi, hg);
                    asm volatile("prefetch.global.L2 [%0];" ::"l"(p.q + (int64_t)(w.r.row0 + qi) * p.ldq + (int64_t)(w.h * p.G + hg) * D + (i % (D / 64)) * 64));
                }
            }
        };
        bool more = w.settle(p);
        for (; more; ++item) {
            const int qb = item % kQBufs;
            bool waited = item < kQBufs;
            split_q(w, qb, warp - kQWarp0, item == 0 ? kQ + kSoftWarps : kQ, [&] {
                if (!waited) wait(q_empty + 8 * qb, item / kQBufs - 1);
                waited = true;
            });
            if (item == 0) tc::named_sync(14, (kQ + kSoftWarps) * 32);
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(q_full + 8 * qb);
            w.advance(p);
            more = w.settle(p);
            if (more) fetch();
        }
    }
    } else {
        // ----------------------------------------------------------- softmax
        // Team 0 has the even tiles of the CTA, team 1 the odd ones, a thread half a
        // row: 64 tokens, two blocks.  A block's weights replace the first 16 columns of its own
        // logits (hi, then lo).
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
        const int quad = warp & 3, half = (warp >> 2) & 1, team = warp >> 3, local = quad * 32 + lane;
        const uint32_t lanes = (uint32_t)(quad * 32) << 16, tH = tmem + lanes + half * 64;
        // One barrier a tile, team and quad of lanes: both halves' maxima are there, and the
        // other team's reference after the tile before (from its first half).
        const int my_bar = 1 + 4 * team + quad, other_bar = 1 + 4 * (team ^ 1) + quad;
        int g = 0, item = 0;
        Walk w_next = w;
        bool more = w_next.settle(p);
        if (more && team == 1 && half == 0) tc::named_arrive(other_bar, 96);  // there is no tile before the first
        if (more) {
            split_q(w_next, 0, kQ + warp, kQ + kSoftWarps, [] {});
            tc::named_arrive(14, (kQ + kSoftWarps) * 32);
        }
        for (; more; ++item) {
            w = w_next;
            w_next.advance(p);
            more = w_next.settle(p);
            const RowMap rows(p, w.t);
            const bool have = w.t * kM + local < w.r.n * p.G;
            int qi, hg;
            rows.find(local, qi, hg);
            if (!have) qi = hg = 0;
            const int64_t at = (int64_t)(w.r.row0 + qi) * p.Hq + w.h * p.G + hg;
            const int base = w.r.L - w.r.n;
            const int seen = have ? base + qi + 1 : 0;
            const int all_see = max(0, min(w.r.L, p.tree != nullptr ? base : base + rows.q0 + 1));
            const int qb = item % kQBufs;
            wait(q_full + 8 * qb, item / kQBufs);
            const float rf = sm.rf[qb][local];
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(q_empty + 8 * qb);
            float m = -INFINITY, l = 0.0f;  // l: this thread's, relative to m
            for (int j = w.j0; j < w.j1; ++j, ++g) {
                if ((g & 1) != team) continue;
                const int buf = g % kBufs;
                const uint32_t tS = tH + buf * kN;
                wait(scales_full + 8 * (g % kScaleRing), g / kScaleRing);
                const float2 sc0 = sm.scales[g % kScaleRing][2 * half], sc1 = sm.scales[g % kScaleRing][2 * half + 1];
                const float f0 = rf * sc0.x, f1 = rf * sc1.x;
                // the thread's 64 tokens as bits: those below its limit, or below the tree and the nodes it sees
                const bool masked = j * kN + kN > all_see;
                uint32_t vis[2] = {~0u, ~0u};
                if (masked) {
                    auto below = [](int n) { return n >= 64 ? ~0ull : n <= 0 ? 0ull : (1ull << n) - 1; };
                    const int pos0 = j * kN + half * 64, first = base - pos0;  // column of the tree's first node
                    unsigned long long bits = below(seen - pos0);
                    if (p.tree != nullptr) {
                        const unsigned long long tree = have ? (unsigned long long)p.tree[w.r.row0 + qi] : 0ull;
                        bits = below(first) | (first >= 64 || first <= -64 ? 0ull : first >= 0 ? tree << first : tree >> -first);
                        bits = have ? bits & below(w.r.L - pos0) : 0ull;
                    }
                    vis[0] = (uint32_t)bits;
                    vis[1] = (uint32_t)(bits >> 32);
                }
                wait(s_full + 8 * buf, g / kBufs);
                tc::fence_after_sync();

                // ---- the blocks' maxima and the tile's
                float top0 = -INFINITY, top1 = -INFINITY;
                // (unrolled where the softmax is the longer: d = 128, 494 -> 477 us for 1,024 queries of 32/8
                // heads after 30,000 tokens; d = 256, 482 -> 485)
#pragma unroll (D == 128 ? 2 : 1)
                for (int c = 0; c < 2; ++c) {
                    float s[32];
                    tc::tmem_ld32(tS + c * 32, s);
                    if (masked) {
                        const uint32_t bits = c ? vis[1] : vis[0];
#pragma unroll
                        for (int k = 0; k < 32; ++k) s[k] = (bits >> k) & 1 ? s[k] : -INFINITY;
                    }
                    float t4[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) t4[k] = fmaxf(fmaxf(s[8 * k], s[8 * k + 1]), s[8 * k + 2]);
#pragma unroll
                    for (int k = 0; k < 4; ++k) t4[k] = fmaxf(fmaxf(t4[k], s[8 * k + 3]), s[8 * k + 4]);
#pragma unroll
                    for (int k = 0; k < 4; ++k) t4[k] = fmaxf(fmaxf(t4[k], s[8 * k + 5]), fmaxf(s[8 * k + 6], s[8 * k + 7]));
                    const float t = fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3]));
                    const float u = fmaf(t, c ? f1 : f0, c ? sc1.y : sc0.y);
                    if (c) top1 = u;
                    else top0 = u;
                }
                float top = fmaxf(top0, top1);
                sm.top[(g >> 1) & 1][team][half][local] = top;
                tc::named_sync(my_bar, 96);

                // ---- the reference: the other team's after the tile before, raised where this tile asks for it
                top = fmaxf(top, sm.top[(g >> 1) & 1][team][half ^ 1][local]);
                float ref = j > w.j0 ? sm.ref[((g - 1) >> 1) & 1][team ^ 1][local] : -INFINITY;
                const bool grows = ref > -INFINITY && top > ref + kGrow;
                const float old = ref;
                if (ref == -INFINITY || grows) ref = fmaxf(ref, top);
                if (half == 0) {
                    sm.ref[(g >> 1) & 1][team][local] = ref;  // (the second half of the other team may still read the last one)
                    if (j + 1 < w.j1 || more) tc::named_arrive(other_bar, 96);
                }
                if (__any_sync(~0u, ref != m)) {
                    l *= factor(m, ref);
                    m = ref;
                    if (j > w.j0 && __any_sync(~0u, grows)) {
                        // This tile's logits came after product g - kBufs, and product g waits for this team: the
                        // barrier is in the phase of product g - 1 or just past it, which its parity tells apart.
                        wait(o_done + 8 * ((g - 1) % kBufs), (g - 1) / kBufs);
                        tc::fence_after_sync();
                        const float c = grows ? ex2(old - ref) : 1.0f;
#pragma unroll 1
                        for (int k = 0; k < D / 64; ++k) {
                            float o[32];
                            tc::tmem_ld32(tO + lanes + half * (D / 2) + 32 * k, o);
#pragma unroll
                            for (int i = 0; i < 32; ++i) o[i] *= c;
                            tc::tmem_st32(tO + lanes + half * (D / 2) + 32 * k, o);
                        }
                    }
                }

                if (j * kN + kN > w.r.L) {  // whatever lies past the end: zeros for the product
                    const int u = 2 * g + 1, slot = u % kSlots;
                    wait(full + 8 * slot, u / kSlots);
                    const int first = max(0, w.r.L - j * kN);
                    for (int i = half * kM + local; i < (kN - first) * (D / 16); i += 2 * kM) {
                        const int tok = first + i / (D / 16), cc = i % (D / 16);
                        *reinterpret_cast<uint4*>(sm.ring[slot] + (cc >> 3) * kHalfBytes + tok * 128 + (cc & 7) * 16) = make_uint4(0, 0, 0, 0);
                    }
                    tc::fence_async_smem();
                }
                // ---- weights
                // A block's exponent n: its largest weight, 2^(top - ref), is held within [2^7, 2^8].  Far
                // below the reference n stops where its byte does and the weights fade (a block that is not
                // seen is there too).  n comes as the low bits of a sum with 1.5 * 2^23.
                const float ref0 = m == -INFINITY ? 0.0f : m;
                auto exponent = [&](int c, float t, float lv) {
                    constexpr float kRound = 12582912.0f;
                    const float u = fmaxf(t - (ref0 - 0.5f), -110.0f) + (kRound - kBlockExp);
                    const uint32_t x = __float_as_uint(u) - __float_as_uint(kRound) + 127;  // below 256, so both bytes by one product
                    *reinterpret_cast<uint16_t*>(&sm.block_exp[buf][c][16 * lane + 4 * quad + 2 * half]) = (uint16_t)(x * 0x101 - (kLoExp << 8));
                    return lv - ref0 - (u - kRound);
                };
                const float a0 = exponent(0, top0, sc0.y), a1 = exponent(1, top1, sc1.y);
                tc::fence_async_smem();
#pragma unroll 1
                for (int c = 0; c < 2; ++c) {
                    float s[32];
                    tc::tmem_ld32(tS + c * 32, s);
                    const float f = c ? f1 : f0, a = c ? a1 : a0;
                    float2 part[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
                    const float2 f2 = make_float2(f, f), a2 = make_float2(a, a);
                    uint32_t hi[8], lo[8];
                    if (!masked) {
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const float2 x = __ffma2_rn(make_float2(s[4 * k], s[4 * k + 1]), f2, a2), y = __ffma2_rn(make_float2(s[4 * k + 2], s[4 * k + 3]), f2, a2);
                            const float2 p0 = make_float2(ex2(x.x), ex2(x.y)), p1 = make_float2(ex2(y.x), ex2(y.y));
                            part[0] = __fadd2_rn(part[0], p0);
                            part[1] = __fadd2_rn(part[1], p1);
                            split4_weights(p0.x, p0.y, p1.x, p1.y, hi[k], lo[k]);
                        }
                    } else {
                        const uint32_t bits = c ? vis[1] : vis[0];
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            float e[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i) e[i] = (bits >> (4 * k + i)) & 1 ? ex2(fmaf(s[4 * k + i], f, a)) : 0.0f;
                            part[0] = __fadd2_rn(part[0], make_float2(e[0], e[1]));
                            part[1] = __fadd2_rn(part[1], make_float2(e[2], e[3]));
                            split4_weights(e[0], e[1], e[2], e[3], hi[k], lo[k]);
                        }
                    }
                    tc::tmem_st8(tS + c * 32, hi);
                    tc::tmem_st8(tS + c * 32 + 8, lo);
                    // a row that sees nothing here takes nothing from the block's scale
                    const float sum = (part[0].x + part[0].y) + (part[1].x + part[1].y);
                    if (sum != 0.0f) l = fmaf(sum, ex2(-ref0 - a), l);  // 2^n over the value scale
                    if (kEarly || c == 1) {
                        tc::tmem_wait_st();
                        tc::fence_before_sync();
                        __syncwarp();
                        if (lane == 0) tc::mbar_arrive(p_ready + 8 * ((kEarly ? c : 0) * kBufs + buf));
                    }
                }
            }

            // ---- the item's output: whole, or this CTA's part of it.  A team and half has a quarter of the columns.
            const int part_id = team * 2 + half, col0 = part_id * (D / 4);
            if (half == 0) sm.ml[item & 1][team][local] = m;
            sm.mr[item & 1][team][half][local] = l;
            tc::named_sync(9 + quad, 128);
            {
                const float m0 = sm.ml[item & 1][0][local], m1 = sm.ml[item & 1][1][local];
                // the last tile's team has the final reference; O is relative to it
                m = ((g - 1) & 1) == 0 ? m0 : m1;
                l = (sm.mr[item & 1][0][0][local] + sm.mr[item & 1][0][1][local]) * factor(m0, m) +
                    (sm.mr[item & 1][1][0][local] + sm.mr[item & 1][1][1][local]) * factor(m1, m);
            }
            const long long tile0 = w.x - w.v0 + kItemCost;  // the place of the item's first tile
            const int c0 = (int)(tile0 / W), c1 = (int)((tile0 + w.kt - 1) / W);
            // Sixteen columns from `col` of the warp's 32 rows, through shared memory: a row's
            // 32 bytes then leave from two lanes (a thread storing its own row would touch 32
            // lines with every instruction).  Called from rolled loops: between two items this
            // code has left the instruction caches, and its fetch is most of its time.
            const int rows_here = min(kM, w.r.n * p.G - w.t * kM);
            auto put = [&](int col, const float (&o)[16], float inv) {
                uint4* stage = reinterpret_cast<uint4*>(sm.stage[warp]);
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    uint32_t u[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        u[e] = tc::pack_bf16(__float2bfloat16_rn(o[8 * i + 2 * e] * inv), __float2bfloat16_rn(o[8 * i + 2 * e + 1] * inv));
                    stage[lane * 2 + (i ^ ((lane >> 2) & 1))] = make_uint4(u[0], u[1], u[2], u[3]);
                }
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int r = i * 16 + (lane >> 1);
                    const int64_t to = __shfl_sync(~0u, at, r);
                    if (quad * 32 + r < rows_here)
                        reinterpret_cast<uint4*>(p.out + to * D + col)[lane & 1] = stage[r * 2 + ((lane & 1) ^ ((r >> 2) & 1))];
                }
            };
            auto put_lse = [&]() {
                if (p.lse != nullptr && have && part_id == 0) p.lse[at] = lse_of(m, l);
            };
            wait(item_done, item);
            tc::fence_after_sync();
            if (c0 == c1) {
                const float inv = l == 0.0f ? 0.0f : 1.0f / l;  // no token seen: zeros
#pragma unroll 1
                for (int k = 0; k < D / 64; ++k) {
                    float o[16];
                    tc::tmem_ld16(tO + lanes + col0 + 16 * k, o);
                    put(col0 + 16 * k, o, inv);
                }
                put_lse();
            } else {
                float* part = p.partials + ((size_t)blockIdx.x * 2 + (w.j0 == 0 ? 1 : 0)) * kPart;
#pragma unroll 1
                for (int k = 0; k < D / 64; ++k) {
                    float o[16];
                    tc::tmem_ld16(tO + lanes + col0 + 16 * k, o);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        reinterpret_cast<float4*>(part)[(col0 / 4 + 4 * k + i) * kM + local] =
                            make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                }
                if (part_id == 0) {
                    part[kM * D + local] = m;
                    part[kM * D + kM + local] = l;
                }
            }
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(o_free);
            if (c0 != c1 && w.j0 == 0 && tid == 0) {  // the item begins here: what the join needs
                p.spans[blockIdx.x] = c1 - c0;
                reinterpret_cast<int4*>(p.span_rows)[blockIdx.x * 4] = make_int4(w.r.row0, w.r.n, w.t, w.h);
            }
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == kMmaWarp) tc::tmem_dealloc(tmem, 512);
}

// Joins the parts of the item that begins in CTA blockIdx.y and goes on in later
// ones.  A block has 32 rows x 64 columns: four warps take the parts in turn for
// each half of the columns, a lane a row, then each of them has eight of the columns.
// (By the last CTA of an item, inside the kernel above: a 64-node tree after 8,000
// tokens, nine parts an item, 42 us instead of 34.5; eight 32-node trees 98.3 instead of 95.8; a
// first prompt of 2,000 tokens 77 instead of 79.6, for its launch.)
template <int D>
__global__ void __launch_bounds__(256) gdn_kv_join_tiles_kernel(const __grid_constant__ KvAttnParams p) {
    constexpr int kPart = kM * D + 2 * kM;
    __shared__ float acc[8][32][33];
    __shared__ float ml[8][2][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c0 = blockIdx.y;
    tc::grid_wait();
    const int more = p.spans[c0];
    if (more == 0) return;
    const int4 item = reinterpret_cast<const int4*>(p.span_rows)[c0 * 4];  // first row of q, queries, row tile, head
    const int quad = blockIdx.x & 3, rows = item.y * p.G - item.z * kM;
    if (quad * 32 >= rows) return;
    const int side = warp & 1, turn = warp >> 1, local = quad * 32 + lane, col = (blockIdx.x >> 2) * 64 + side * 32;
    float m = -INFINITY, l = 0.0f, o[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) o[i] = 0.0f;
#pragma unroll 1
    for (int c = c0 + turn; c <= c0 + more; c += 4) {
        const float* part = p.partials + ((size_t)c * 2 + (c == c0 ? 1 : 0)) * kPart;
        const float mo = part[kM * D + local], lo = part[kM * D + kM + local];
        float4 u[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) u[i] = reinterpret_cast<const float4*>(part)[(col / 4 + i) * kM + local];
        const float top = fmaxf(m, mo), a = factor(m, top), b = factor(mo, top);
        m = top;
        l = l * a + lo * b;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            o[4 * i] = o[4 * i] * a + u[i].x * b;
            o[4 * i + 1] = o[4 * i + 1] * a + u[i].y * b;
            o[4 * i + 2] = o[4 * i + 2] * a + u[i].z * b;
            o[4 * i + 3] = o[4 * i + 3] * a + u[i].w * b;
        }
    }
#pragma unroll
    for (int i = 0; i < 32; ++i) acc[warp][i][lane] = o[i];
    ml[warp][0][lane] = m;
    ml[warp][1][lane] = l;
    __syncthreads();
    float top = -INFINITY, total = 0.0f, v[8];
#pragma unroll
    for (int w = 0; w < 4; ++w) top = fmaxf(top, ml[2 * w + side][0][lane]);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.0f;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        const float f = factor(ml[2 * w + side][0][lane], top);
        total = fmaf(ml[2 * w + side][1][lane], f, total);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = fmaf(acc[2 * w + side][8 * turn + i][lane], f, v[i]);
    }
    if (local >= rows) return;
    int qi, hg;
    RowMap(p, item.z).find(local, qi, hg);
    const int64_t at = (int64_t)(item.x + qi) * p.Hq + item.w * p.G + hg;
    const float inv = total == 0.0f ? 0.0f : 1.0f / total;
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = tc::pack_bf16(__float2bfloat16_rn(v[2 * i] * inv), __float2bfloat16_rn(v[2 * i + 1] * inv));
    *reinterpret_cast<uint4*>(p.out + at * D + col + 8 * turn) = make_uint4(u[0], u[1], u[2], u[3]);
    if (p.lse != nullptr && col == 0 && turn == 0) p.lse[at] = lse_of(top, total);
}

template <int D>
cudaError_t launch(KvAttnParams& p, cudaStream_t s) {
    constexpr int smem = (int)sizeof(TilesSmem<D>) + 1024;
    static_assert(smem <= 227 * 1024, "shared memory of a CTA");
    static std::once_flag once[64];
    static cudaError_t err[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || dev < 0 || dev >= 64) return e != cudaSuccess ? e : cudaErrorInvalidDevice;
    std::call_once(once[dev], [dev] {
        err[dev] = cudaFuncSetAttribute(gdn_kv_attn_tiles_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    });
    if (err[dev] != cudaSuccess) return err[dev];
    const int grid = std::min(device_sm_count(), kKvMaxCtas);
    e = launch_dependent(gdn_kv_attn_tiles_kernel<D>, dim3((unsigned)grid), kThreads, smem, s, p);
    if (e != cudaSuccess) return e;
    return launch_dependent(gdn_kv_join_tiles_kernel<D>, dim3(4 * D / 64, (unsigned)grid), 256, 0, s, p);
}

}  // namespace

size_t kv_attn_tiles_workspace(int d) { return (size_t)2 * std::min(device_sm_count(), kKvMaxCtas) * (kM * d + 2 * kM) * 4; }

cudaError_t launch_kv_attn_tiles(KvAttnParams& p, int d, cudaStream_t s) { return d == 256 ? launch<256>(p, s) : launch<128>(p, s); }

}  // namespace gdn
