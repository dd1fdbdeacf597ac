// gdn_latent_tiles.cu -- latent attention, absorbed form: every head's query against the cached rows
// themselves, on the tcgen05 tensor cores.  For the rows r = (query, head) of a request,
//   t_jr = scale log2(e) x_j . q_r over 576 channels,   o_r = sum_j 2^(t_jr - m_r) c_j / sum_j 2^(t_jr - m_r) over 512.
//
// Both products are computed transposed, S^T = X Q^T and O^T += C^T P^T: the tokens, and then the
// latent channels, are the MMAs' rows, and the N = 16, 32 or 64 query rows of an item their columns.
// So a decode step of few heads leaves no part of an MMA empty (128 rows of queries would), the 512
// output channels of 64 rows are 256 columns of tensor memory, and one copy of a tile in shared memory
// serves both products: 64 tokens x 64 channels lie as 128-byte rows, K-major for the first, MN-major
// for the second.
//
// Roles of the CTA's 11 warps: four are the softmax; one loads tiles (TMA); one issues the first
// product, one the second; four copy the next item's queries (cp.async) and write the last one's output.  A tile of 64
// tokens is three copies, the key part and two units of 256 channels; a unit is free again once the second
// product has read it.
//
// The softmax's threads hold S^T as an MMA's fragments (16 tokens x 8 rows at a time), write the
// weights transposed (stmatrix) as the second product's K-major operand, and agree through one barrier with
// a vote whether a row's reference m has to be raised: only when a logit exceeds it by 2^8.  The
// weights are rounded to bf16, as the values are: within 2^-8 of themselves, however far below
// the reference; their sum is of the unrounded ones, in fp32.
//
// 64 requests of 4,096 to 12,288 tokens, 128 heads, one token each: 217 us, 659 TFLOP/s, 2.8 TB/s.  A tile of 64 tokens
// and 64 rows takes about 3,100 cycles, 1,950 of them products: bound by shared memory, which serves the MMAs' operands and
// takes the next tile in.  251 requests of up to 3,000 tokens, 20 heads: 95 us, 4.8 TB/s, HBM and the items' ends.  One
// request of 131,072 tokens, 64 heads: 53 us, of which 27 are the first copies, the last output and the join.
//
// The list of all (request, row tile, token tile) is cut evenly over the CTAs, one to an SM; an item that
// spans several leaves its parts in the workspace, and a second kernel joins them, in order.  With two row tiles a request or
// more, CTAs work in pairs (of few rows each, in up to eights) on the same tokens, so that the others read them out of the L2.
#include <algorithm>
#include <mutex>

#include "gdn_kv_tc.cuh"
#include "gdn_latent.cuh"
#include "gdn_latent_tc.cuh"
#include "gdn_tc.cuh"

namespace gdn {
namespace {

constexpr int kSoftWarps = 4, kQWarps = 4;
constexpr int kLoadWarp = kSoftWarps, kKeyWarp = kSoftWarps + 1, kValueWarp = kSoftWarps + 2, kQWarp0 = kSoftWarps + 3;
constexpr int kThreads = (kSoftWarps + 3 + kQWarps) * 32;
constexpr int kTok = 64;                 // tokens of a tile
constexpr int kBox = kTok * 128;         // 64 tokens x 64 channels
constexpr int kUnits = 2;                // of 256 channels
constexpr int kUnit = 4 * kBox;
constexpr int kBlocks = kLatent / 128;   // of 128 channels, the second product's rows
constexpr float kGrow = 8.0f;            // how far a weight may exceed the reference, in powers of two
constexpr int kItemCost = 2;             // an item's beginning and end, in tiles
constexpr int kMinShare = 2;             // what a CTA takes at least, in tiles
constexpr int kInfo = 8;
constexpr int kAhead = 2;                // tiles
constexpr int kMaxCtas = 512;
static_assert(kMaxCtas <= kKvMaxCtas, "the workspace's words");
constexpr uint64_t kDrainNs = 200000000ull;

template <int N>
struct LatentSmem {
    static constexpr int kRing = N == 64 ? 4 : N == 32 ? 5 : 6;  // units
    alignas(1024) uint8_t q[9][N * 128];
    alignas(1024) uint8_t ring[kRing][kUnit];
    alignas(1024) uint8_t keys[kBox];
    alignas(1024) uint8_t p[2][N * 128]; // two tiles of weights
    union {
        float top[kSoftWarps][N];        // a tile's maxima, or the sums, by warp
        long long scan[kThreads / 32];   // (before the first item)
    };
    float ref[N], fac[2][N];             // the rows' references; what the output's columns are multiplied by, items in turn
    short query[N];                      // the rows' queries, from the first one's on, -1 where there is none
    alignas(8) int limit[N];             // without a tree: a row sees the tokens before this
    alignas(8) uint64_t full[kRing], empty[kRing], info_full[kInfo], s_full[2], p_ready[2], o_done[2];
    uint64_t key_full, key_empty, q_full, q_empty, item_done, sums_there, o_free, drained[2];
    int bad[kInfo];                      // a tile's pages that are not in the cache, by 32 tokens
    int at_b, at_t, at_v;
    uint32_t tmem;
    int dead;
};

struct Request {
    int n, L, row0;   // queries, tokens, first row of q,
    unsigned groups;  // groups of row tiles
};

template <int N>
struct List {
    const LatentAttnParams& p;
    unsigned per_group;  // rows of a group (a request's are below 2^31)
    __device__ __forceinline__ List(const LatentAttnParams& p_) : p(p_), per_group(N * p_.pair) {}
    __device__ __forceinline__ Request request(int b) const {
        Request r;
        r.row0 = p.start[b];
        r.n = max(0, min(p.start[b + 1], p.T) - r.row0);
        if (r.row0 < 0) r.n = 0;
        r.L = max(0, min(p.lens[b], p.width << p.log2_page));
        r.groups = ((unsigned)r.n * p.H + per_group - 1) / per_group;
        return r;
    }
    // Token tiles that some row of group t sees (at least one).
    __device__ __forceinline__ int token_tiles(const Request& r, unsigned t) const {
        const int last = min(r.n - 1, (int)(((t + 1) * per_group - 1) / (unsigned)p.H));
        const int seen = p.tree != nullptr ? r.L : min(r.L, r.L - r.n + last + 1);
        return max(1, (seen + kTok - 1) / kTok);
    }
};

// One stretch of an item's token tiles, and the walk over a CTA's stretches.
template <int N>
struct Walk {
    List<N> list;
    int b, v0, j0, j1, kt;
    unsigned t;
    long long x, x1;
    Request r;
    __device__ __forceinline__ Walk(const LatentAttnParams& p) : list(p) {}
    __device__ __forceinline__ Walk& operator=(const Walk& w) {  // (one of the same list)
        b = w.b, t = w.t, v0 = w.v0, j0 = w.j0, j1 = w.j1, kt = w.kt, x = w.x, x1 = w.x1, r = w.r;
        return *this;
    }
    __device__ __forceinline__ bool settle(int side) {  // false: the CTA's part is done
        while (x < x1) {
            r = list.request(b);
            while (t >= r.groups) {
                t = 0;
                r = list.request(++b);
            }
            kt = list.token_tiles(r, t);
            const int v1 = (int)min((long long)kt + kItemCost, v0 + (x1 - x));
            j0 = max(0, v0 - kItemCost);
            j1 = max(0, v1 - kItemCost);
            // (a group's last row tiles may have no rows: their CTAs have nothing to do in it)
            if (j0 < j1 && t * list.per_group + side * N < (unsigned)r.n * list.p.H) return true;
            next(v1);
        }
        return false;
    }
    __device__ __forceinline__ void next(int v1) {
        x += v1 - v0;
        v0 = 0;
        ++t;
    }
    __device__ __forceinline__ void advance() { next(j1 + kItemCost); }
    __device__ __forceinline__ int row(int side) const { return (int)(t * list.per_group) + side * N; }  // first of the request's rows
};

__device__ __forceinline__ float factor(float m, float top) { return m == top ? 1.0f : ex2(m - top); }

__device__ __forceinline__ float lse_of(float m, float l) {
    return l == 0.0f ? -INFINITY : ((m == -INFINITY ? 0.0f : m) + log2f(l)) * 0.69314718055994531f;
}

// Whether any of `threads` threads at barrier `id` says so.
__device__ __forceinline__ bool vote_any(int id, int threads, bool mine) {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.b32 q, %1, 0;\n\tbar.red.or.pred p, %2, %3, q;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(r)
                 : "r"((uint32_t)mine), "r"(id), "r"(threads)
                 : "memory");
    return r != 0;
}

// A warp's 16 lanes x N columns as MMA fragments: s[4 g ..] = (row lane / 4, columns 8 g + 2 (lane % 4) and
// the next), (row + 8, the same).
__device__ __forceinline__ void tmem_ld_fragments(uint32_t taddr, float (&s)[8]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=f"(s[0]), "=f"(s[1]), "=f"(s[2]), "=f"(s[3]), "=f"(s[4]), "=f"(s[5]), "=f"(s[6]), "=f"(s[7])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_ld_fragments(uint32_t taddr, float (&s)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=f"(s[0]), "=f"(s[1]), "=f"(s[2]), "=f"(s[3]), "=f"(s[4]), "=f"(s[5]), "=f"(s[6]), "=f"(s[7]), "=f"(s[8]), "=f"(s[9]),
          "=f"(s[10]), "=f"(s[11]), "=f"(s[12]), "=f"(s[13]), "=f"(s[14]), "=f"(s[15])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_ld_fragments(uint32_t taddr, float (&s)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, "
        "%19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=f"(s[0]), "=f"(s[1]), "=f"(s[2]), "=f"(s[3]), "=f"(s[4]), "=f"(s[5]), "=f"(s[6]), "=f"(s[7]), "=f"(s[8]), "=f"(s[9]),
          "=f"(s[10]), "=f"(s[11]), "=f"(s[12]), "=f"(s[13]), "=f"(s[14]), "=f"(s[15]), "=f"(s[16]), "=f"(s[17]), "=f"(s[18]),
          "=f"(s[19]), "=f"(s[20]), "=f"(s[21]), "=f"(s[22]), "=f"(s[23]), "=f"(s[24]), "=f"(s[25]), "=f"(s[26]), "=f"(s[27]),
          "=f"(s[28]), "=f"(s[29]), "=f"(s[30]), "=f"(s[31])
        : "r"(taddr)
        : "memory");
}

// Four 8 x 8 matrices of 16-bit fragments, transposed: lane 8 i + k gives the address of matrix i's column k.
__device__ __forceinline__ void store_transposed(uint32_t saddr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(saddr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// Reduces values of 2, 4 or 8 pairs of columns over the eight lanes that have them (those of equal lane % 4), the lanes
// left with a pair (16 values), one (8) or one in common with another lane (4) each: v[0], of column my_col.
template <int C, class Op>
__device__ __forceinline__ void halve(float (&v)[C], int lane, Op op) {
    int n = C;
#pragma unroll
    for (int o = 16; o >= 4; o >>= 1) {
        if (n == 1) {
            v[0] = op(v[0], __shfl_xor_sync(~0u, v[0], o));
            continue;
        }
        n /= 2;
        const bool upper = (lane & o) != 0;
#pragma unroll
        for (int i = 0; i < C / 2; ++i)
            if (i < n) {
                const float keep = upper ? v[i + n] : v[i], give = upper ? v[i] : v[i + n];
                v[i] = op(keep, __shfl_xor_sync(~0u, give, o));
            }
    }
}

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

template <int N>
__global__ void __launch_bounds__(kThreads, 1) gdn_latent_tiles_kernel(const __grid_constant__ LatentAttnParams p) {
    using Smem = LatentSmem<N>;
    constexpr int kRing = Smem::kRing;
    constexpr int kPart = N * kLatent + 2 * N;
    constexpr int kCols = N / 4;  // of a softmax thread
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    Smem& sm = *reinterpret_cast<Smem*>(smem_raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int side = blockIdx.x % p.pair, share = blockIdx.x / p.pair, shares = gridDim.x / p.pair;
    const List<N> list(p);
    if ((tc::smem_u32(smem_raw) & 1023) != 0) {  // (the swizzle's atoms; the kernel has no other shared memory)
        if (tid == 0) {
            tc::grid_wait();
            p.spans[blockIdx.x] = 0;
            atomicOr(p.status, 8);
            atomicOr(p.gave_up, 8);
        }
        return;
    }

    // ---- barriers and tensor memory
    const uint32_t full = tc::smem_u32(sm.full), empty = tc::smem_u32(sm.empty), key_full = tc::smem_u32(&sm.key_full),
                   key_empty = tc::smem_u32(&sm.key_empty), info_full = tc::smem_u32(sm.info_full), s_full = tc::smem_u32(sm.s_full),
                   p_ready = tc::smem_u32(sm.p_ready), o_done = tc::smem_u32(sm.o_done), q_full = tc::smem_u32(&sm.q_full),
                   q_empty = tc::smem_u32(&sm.q_empty), item_done = tc::smem_u32(&sm.item_done), sums_there = tc::smem_u32(&sm.sums_there), o_free = tc::smem_u32(&sm.o_free),
                   drained = tc::smem_u32(sm.drained);
    if (tid == 0) {
        tc::prefetch_map(&p.tm);
        tc::prefetch_map(&p.tm_key);
        sm.dead = 0;
        for (int i = 0; i < kRing; ++i) {
            tc::mbar_init(full + 8 * i, 1);
            tc::mbar_init(empty + 8 * i, 1);
        }
        tc::mbar_init(key_full, 1);
        tc::mbar_init(key_empty, 1);
        for (int i = 0; i < kInfo; ++i) tc::mbar_init(info_full + 8 * i, 1);
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(s_full + 8 * i, 1);
            tc::mbar_init(p_ready + 8 * i, kSoftWarps);
            tc::mbar_init(o_done + 8 * i, 1);
            tc::mbar_init(drained + 8 * i, 1);
        }
        tc::mbar_init(q_full, kQWarps);
        tc::mbar_init(q_empty, 1);
        tc::mbar_init(item_done, 1);
        tc::mbar_init(sums_there, kSoftWarps);
        tc::mbar_init(o_free, kQWarps);
    }
    if (warp == kKeyWarp) tc::tmem_alloc(tc::smem_u32(&sm.tmem), 512);
    tc::fence_before_sync();
    tc::grid_wait();  // nothing above touches memory that an earlier kernel may write
    if (tid == 0) p.spans[blockIdx.x] = 0;

    // ---- this CTA's part of the list, from a prefix over the requests
    const int per = (p.B + kThreads - 1) / kThreads;
    const int b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
    long long mine = 0;
    for (int b = b0; b < b1; ++b) {
        const Request r = list.request(b);
#pragma unroll 1
        for (unsigned t = 0; t < r.groups; ++t) mine += list.token_tiles(r, t) + kItemCost;
    }
    long long before = mine, total = 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(~0u, before, o);
        if (lane >= o) before += x;
    }
    if (lane == 31) sm.scan[warp] = before;
    before -= mine;
    __syncthreads();
    tc::fence_after_sync();
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) {
        if (i < warp) before += sm.scan[i];
        total += sm.scan[i];
    }
    const long long W = max((total + shares - 1) / shares, (long long)kMinShare);
    const long long x0 = share * W, x1 = min(x0 + W, total);
    if (before <= x0 && x0 < before + mine) {
        long long rest = x0 - before;
        int b = b0;
        unsigned t = 0;
        Request r = list.request(b);
#pragma unroll 1
        for (;; ++t) {
            while (t >= r.groups) {
                t = 0;
                r = list.request(++b);
            }
            const int len = list.token_tiles(r, t) + kItemCost;
            if (rest < len) {
                sm.at_b = b;
                sm.at_t = t;
                sm.at_v = (int)rest;
                break;
            }
            rest -= len;
        }
    }
    __syncthreads();
    if (sm.tmem != 0 && tid == 0) {
        atomicOr(p.status, 8);
        atomicOr(p.gave_up, 8);
    }
    constexpr uint32_t tmem = 0, tO = tmem + 2 * N;  // (all of tensor memory is this CTA's); two tiles of logits before the output
    volatile int* dead = &sm.dead;

    // A bounded wait.  The first that gives up ends all waiting of the CTA, and its copies: the roles run
    // through on whatever is there, and the status words tell.
    auto wait = [&](uint32_t bar, uint32_t parity) {
        parity &= 1;
        if (tc::mbar_test(bar, parity)) return;
        if (*dead) return;
        if (!tc::mbar_wait(bar, parity, p.wait_ns)) {
            *dead = 1;
            atomicOr(p.status, 4);
            atomicOr(p.gave_up, 4);
        }
    };

    // Whether the CTA's copies have ended, the same answer for a warp's lanes: what they then do or leave out has votes in it.
    auto over = [&]() { return __any_sync(~0u, *dead != 0) != 0; };

    // The same for a barrier in each lane at once (each that has one to wait for).
    auto wait_lanes = [&](bool mine, uint32_t bar, uint32_t parity) {
        const bool there = !mine || tc::mbar_test(bar, parity & 1);
        if (!__all_sync(~0u, there)) {
            if (!there) wait(bar, parity);
            __syncwarp();
        }
        tc::fence_after_sync();
    };

    Walk<N> w(p);
    w.b = sm.at_b;
    w.t = sm.at_t;
    w.v0 = sm.at_v;
    w.x = x0;
    w.x1 = x1;

    if (warp == kLoadWarp) {
        // ------------------------------------------------------------ tiles
        const int box_rows = min(1 << p.log2_page, kTok), none = p.pages << p.log2_page;
        int g = 0;
        // copies that have been sent, by barrier: key parts, units
        int sent_keys = 0, sent_units = 0;
        for (; w.settle(side); w.advance()) {
            // 16 tiles' places at a time: lane = 2 tile + half of its tokens
            int y = 0, y_next = 0;
            auto lookup = [&](int j) {
                const int pos = (j + (lane >> 1)) * kTok + (lane & 1) * 32, idx = pos >> p.log2_page;
                const int page = pos < w.r.L && idx < p.width ? p.table[(int64_t)w.b * p.width + idx] : -1;
                y_next = cache_row(page, p.pages, 1, 0, p.log2_page, pos);
                if (pos >= w.r.L) y_next |= (int)0x80000000;  // nothing there, and nothing wrong
            };
            lookup(w.j0);
            for (int j = w.j0; j < w.j1; ++j, ++g) {
                const int k = (j - w.j0) & 15;
                if (k == 0) {
                    y = y_next;
                    lookup(j + 16);
                }
                const int ya = __shfl_sync(~0u, y, 2 * k), yb = __shfl_sync(~0u, y, 2 * k + 1);
                if (lane == 0) {
                    // the place in the ring is free: its reader was done before this tile's units were
                    sm.bad[g % kInfo] = (ya == none ? 1 : 0) | (yb == none ? 2 : 0);
                    tc::mbar_arrive(info_full + 8 * (g % kInfo));
                }
                const int row[2] = {ya & 0x7fffffff, yb & 0x7fffffff};
                // `groups` of 64 channels; pages of 32 tokens come one by one, others four groups in a box
                auto load = [&](uint32_t dst, const void* map, int group, int groups, uint32_t bar) {
                    if (box_rows == kTok) {
                        tc::tma_load_3d(dst, map, 0, row[0], group, bar);
                    } else {
#pragma unroll 1
                        for (int i = 0; i < 2 * groups; ++i) tc::tma_load_3d(dst + i * (kBox / 2), &p.tm_key, 0, i & 1 ? row[1] : row[0], group + (i >> 1), bar);
                    }
                };
                if (g > 0) wait(key_empty, g - 1);
                // Never into a slot whose wait gave up: a second arrival in a phase that still awaits its bytes is a fault.
                if (!over()) {
                    sent_keys = g + 1;
                    if (tc::elect_one()) {
                        tc::mbar_arrive_expect_tx(key_full, kBox);
                        load(tc::smem_u32(sm.keys), &p.tm_key, kLatent / 64, 1, key_full);
                    }
                    __syncwarp();
                }
                // A later tile's rows towards the L2 (of a pair, by the first): the ring's two tiles are too few bytes on their way
                // for the memory's latency.  (By the copy engine's own prefetch, or three tiles ahead, slower: 251 requests 107 us
                // without, 96 two tiles ahead, 105 three.)
                if (side == 0 && j + kAhead < w.j1) {
                    const int k2 = k + kAhead;
                    const int pa = __shfl_sync(~0u, k2 < 16 ? y : y_next, 2 * (k2 & 15)), pb = __shfl_sync(~0u, k2 < 16 ? y : y_next, 2 * (k2 & 15) + 1);
#pragma unroll
                    for (int i = 0; i < kLatentRow / 64; ++i) {  // 32 rows are nine times 32 lines
                        if ((unsigned)pa < (unsigned)none)
                            asm volatile("prefetch.global.L2 [%0];" ::"l"(p.cache + (int64_t)pa * kLatentRow + (i * 32 + lane) * 64));
                        if ((unsigned)pb < (unsigned)none)
                            asm volatile("prefetch.global.L2 [%0];" ::"l"(p.cache + (int64_t)pb * kLatentRow + (i * 32 + lane) * 64));
                    }
                }
                for (int i = 0; i < kUnits; ++i) {
                    const int u = g * kUnits + i, slot = u % kRing;
                    if (u >= kRing) wait(empty + 8 * slot, u / kRing - 1);
                    if (over()) continue;
                    sent_units = u + 1;
                    if (tc::elect_one()) {
                        tc::mbar_arrive_expect_tx(full + 8 * slot, kUnit);
                        load(tc::smem_u32(sm.ring[slot]), &p.tm, 4 * i, 4, full + 8 * slot);
                    }
                    __syncwarp();
                }
            }
        }
        // Copies that nobody waited for (after a wait that gave up) land before the CTA ends.
        if (sent_keys > 0) tc::mbar_wait(key_full, (sent_keys - 1) & 1, kDrainNs);
        for (int i = max(0, sent_units - kRing); i < sent_units; ++i) tc::mbar_wait(full + 8 * (i % kRing), (i / kRing) & 1, kDrainNs);
    } else if (warp == kKeyWarp) {
        // ------------------------------------------------------------ S^T = X Q^T
        constexpr uint32_t id = tc::idesc_bf16(kTok, N);
        constexpr uint32_t hi = tc::kDescHiSw128;
        const uint32_t q = tc::desc_lo_sw128(tc::smem_u32(sm.q[0])), part = tc::desc_lo_sw128(tc::smem_u32(sm.keys));
        // An MMA takes its descriptors from uniform registers.  With loops that the compiler knows to be uniform (their
        // conditions are votes) they are made there; moved there from others, an MMA takes twice as long to issue as to run.
        int g = 0, item = 0;
        for (; __any_sync(~0u, w.settle(side)); w.advance(), ++item) {
            wait(q_full, item);
            for (int j = w.j0; __any_sync(~0u, j < w.j1); ++j, ++g) {
                const bool last = __any_sync(~0u, j == w.j1 - 1);
                const uint32_t d = tmem + (g & 1) * N;
#pragma unroll
                for (int i = 0; i < kUnits; ++i) {
                    const int u = g * kUnits + i;
                    // first: the logits of the tile before last have been read (their buffer is free), and the key part
                    if (i == 0)
                        wait_lanes(lane < 2 || (lane == 2 && g >= 2), lane == 0 ? full + 8 * (u % kRing) : lane == 1 ? key_full : p_ready + 8 * (g & 1),
                                   lane == 0 ? u / kRing : lane == 1 ? g : g / 2 - 1);
                    else
                        wait_lanes(lane == 0, full + 8 * (u % kRing), u / kRing);
                    const uint32_t x = tc::desc_lo_sw128(tc::smem_u32(sm.ring[0]) + u % kRing * kUnit);
                    if (tc::elect_one()) {
                        if (i == 0) {
#pragma unroll
                            for (int ks = 0; ks < 4; ++ks) tc::mma_bf16_lo(d, part + 2 * ks, q + (8 * N * 128 >> 4) + 2 * ks, hi, id, ks > 0);
                            tc::mma_commit(key_empty);
                        }
#pragma unroll
                        for (int ks = 0; ks < 16; ++ks)
                            tc::mma_bf16_lo(d, x + (ks >> 2) * (kBox >> 4) + 2 * (ks & 3), q + ((4 * i + (ks >> 2)) * N * 128 >> 4) + 2 * (ks & 3), hi, id, 1);
                        if (i == kUnits - 1) {
                            tc::mma_commit(s_full + 8 * (g & 1));
                            if (last) tc::mma_commit(q_empty);
                        }
                    }
                    __syncwarp();
                }
            }
        }
        if (tc::elect_one()) tc::mma_commit(drained);
        __syncwarp();
        tc::mbar_wait(drained, 0, kDrainNs);
    } else if (warp == kValueWarp) {
        // ------------------------------------------------------------ O^T += C^T P^T
        constexpr uint32_t id = tc::idesc_bf16(128, N) | 1u << 15;  // the first operand MN-major
        constexpr uint32_t hi = tc::kDescHiSw128;
        int g = 0, item = 0;
        for (; __any_sync(~0u, w.settle(side)); w.advance(), ++item) {
            int done = 0;  // tiles of this item
            for (int j = w.j0; __any_sync(~0u, j < w.j1); ++j, ++g, ++done) {
                const bool last = __any_sync(~0u, j == w.j1 - 1);
                const int u = g * kUnits + (lane & 1);
                wait_lanes(lane < 3 || (lane == 3 && done == 0 && item > 0),
                           lane < 2 ? full + 8 * (u % kRing) : lane == 2 ? p_ready + 8 * (g & 1) : o_free, lane < 2 ? u / kRing : lane == 2 ? g / 2 : item - 1);
                const uint32_t pt = tc::desc_lo_sw128(tc::smem_u32(sm.p[0]) + (g & 1) * N * 128);
                if (tc::elect_one()) {
#pragma unroll
                    for (int i = 0; i < kUnits; ++i) {
                        const int slot = (g * kUnits + i) % kRing;
                        const uint32_t c = tc::desc_lo_mn_sw128(tc::smem_u32(sm.ring[0]) + slot * kUnit, kBox);
#pragma unroll
                        for (int m = 0; m < 2; ++m)
#pragma unroll
                            for (int ks = 0; ks < kTok / 16; ++ks)
                                tc::mma_bf16_lo(tO + (2 * i + m) * N, c + m * (2 * kBox >> 4) + ks * (16 * 128 >> 4), pt + 2 * ks, hi, id, ks > 0 || done > 0);
                        tc::mma_commit(empty + 8 * slot);
                    }
                    tc::mma_commit(o_done + 8 * (g & 1));
                    if (last) tc::mma_commit(item_done);
                }
                __syncwarp();
            }
        }
        // every MMA has ended before tensor memory is given back
        if (tc::elect_one()) tc::mma_commit(drained + 8);
        __syncwarp();
        tc::mbar_wait(drained + 8, 0, kDrainNs);
    } else if (warp >= kQWarp0) {
        // ------------------------------------------------------------ queries and output
        const int quad = warp & 3;
        const uint32_t lanes = (uint32_t)(quad * 32) << 16;
        Walk<N> w_next = w;
        bool more = w_next.settle(side);
        for (int item = -1; more || item >= 0; ++item) {
            // the next item's queries, while this one's last tile is in its softmax
            const bool load = more;
            if (load) {
                if (item >= 0) wait(q_empty, item);
                const int first = w_next.row(side), rows = min(w_next.r.n * p.H - first, N);
                for (int local = warp - kQWarp0; local < N; local += kQWarps) {
                    const int r = first + min(local, rows - 1), i = r / p.H, h = r - i * p.H;
                    const uint16_t* src = p.q + (int64_t)(w_next.r.row0 + i) * p.q_row + (int64_t)h * p.q_head;
                    const uint16_t* part = p.q_rope + (int64_t)(w_next.r.row0 + i) * p.r_row + (int64_t)h * p.r_head;
#pragma unroll
                    for (int k = 0; k < 3; ++k) {
                        const int c = lane + 32 * k;
                        if (k < 2 || lane < 8)
                            tc::cp_async16(tc::smem_u32(sm.q[c >> 3]) + local * 128 + (((c & 7) ^ (local & 7)) << 4),
                                           k < 2 ? src + 8 * c : part + 8 * lane, local < rows);
                    }
                }
                tc::cp_async_commit();
                tc::cp_async_wait_all();
                tc::fence_async_smem();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(q_full);
            }
            if (item >= 0) {
                // this item's output: whole, or the CTA's part of it
                const int first = w.row(side), rows = min(w.r.n * p.H - first, N);
                const long long tile0 = w.x - w.v0 + kItemCost;  // the place of the item's first tile
                const bool whole = tile0 / W == (tile0 + w.kt - 1) / W;
                uint16_t* out = p.out + ((int64_t)w.r.row0 * p.H + first) * kLatent + quad * 32;
                float* part = p.partials + ((size_t)blockIdx.x * 2 + (w.j0 == 0 ? 1 : 0)) * kPart + quad * 32 + lane;
                // (A barrier in shared memory, bounded as every wait between roles: at a hardware barrier the softmax's warps, which
                // do not wait there, would meet themselves once a wait that gave up has let them come twice, and these for ever.)
                wait(sums_there, item);
                wait(item_done, item);
                tc::fence_after_sync();
                float o[2][16];
                tc::tmem_ld16_start(tO + lanes, o[0]);
#pragma unroll 1
                for (int k2 = 0; k2 < kBlocks * N / 16; k2 += 2) {
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const int k = k2 + half, col = 16 * k % N, block = 16 * k / N;
                        tc::tmem_wait_ld(o[half]);
                        if (k + 1 < kBlocks * N / 16) tc::tmem_ld16_start(tO + lanes + 16 * (k + 1), o[half ^ 1]);
                        if (whole) {
                            tc::mul16(o[half], sm.fac[item & 1] + col);
                            // a pair of lanes has two channels of two rows: each stores both of one
                            uint16_t* to = out + (col + (lane & 1)) * kLatent + block * 128 + (lane & ~1);
#pragma unroll
                            for (int i = 0; i < 16; i += 2) {
                                const float a = o[half][i], b = o[half][i + 1], other = __shfl_xor_sync(~0u, lane & 1 ? a : b, 1);
                                if (col + i + (lane & 1) < rows) *reinterpret_cast<uint32_t*>(to + i * kLatent) = lane & 1 ? bf16x2(other, b) : bf16x2(a, other);
                            }
                        } else {
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                if (col + i < rows) part[(col + i) * kLatent + block * 128] = o[half][i];
                        }
                    }
                }
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(o_free);
            }
            if (!load) break;
            w = w_next;
            w_next.advance();
            more = w_next.settle(side);
        }
    } else {
        // ------------------------------------------------------------ softmax
        // Thread: tokens tok and tok + 8 of a tile, columns 8 g + col2 and the next, g < N / 8.
        const int tok = warp * 16 + (lane >> 2), col2 = 2 * (lane & 3);
        const uint32_t lanes = (uint32_t)(warp * 32) << 16;
        // where this lane's matrix column goes: rows (heads) of 128 bytes, the warp's tokens in chunks 2 warp, 2 warp + 1
        const uint32_t p_row = (uint32_t)((lane >> 4) * 8 + (lane & 7)), p_chunk = (uint32_t)(2 * warp + ((lane >> 3) & 1));
        const uint32_t p_at = p_row * 128 + ((p_chunk ^ (p_row & 7)) << 4);
        const int my_col = kCols == 16 ? (lane >> 2) * 8 + col2 : kCols == 8 ? (lane >> 3) * 8 + col2 + (lane >> 2 & 1) : (lane >> 4) * 8 + col2 + (lane >> 3 & 1);
        const float f = p.scale_log2;
        int g = 0, item = 0;
        for (; w.settle(side); w.advance(), ++item) {
            const int first = w.row(side), rows = min(w.r.n * p.H - first, N), base = w.r.L - w.r.n;
            const int all_see = max(0, min(w.r.L, p.tree != nullptr ? base : base + first / p.H + 1));
            if (tid < N) {  // (what an item's last tile read of these was read before its output's barriers)
                sm.ref[tid] = -INFINITY;
                const int q0 = first / p.H, q = (first + tid) / p.H;
                sm.query[tid] = tid < rows ? q - q0 : -1;
                sm.limit[tid] = tid < rows ? min(w.r.L, base + q + 1) : 0;
            }
            float l[kCols];  // this thread's sums, relative to the references
#pragma unroll
            for (int c = 0; c < kCols; ++c) l[c] = 0.0f;
            float sub[kCols];  // the references in powers of two, 0 where a row has seen nothing
#pragma unroll
            for (int c = 0; c < kCols; ++c) sub[c] = 0.0f;
            tc::named_sync(1, kSoftWarps * 32);
            for (int j = w.j0; j < w.j1; ++j, ++g) {
                // the tile's pages, its logits, and the weights' place (the second product of the tile before last)
                wait_lanes(lane < 2 || (lane == 2 && g >= 2), lane == 0 ? info_full + 8 * (g % kInfo) : lane == 1 ? s_full + 8 * (g & 1) : o_done + 8 * (g & 1),
                           lane == 0 ? g / kInfo : lane == 1 ? g / 2 : g / 2 - 1);
                const int bad = sm.bad[g % kInfo];
                const bool masked = j * kTok + kTok > all_see || bad != 0;
                float s[N / 2];
                // A pass through this loop has the tile's logits in powers of two less the references; a second one
                // follows where the references had to be raised.  (The code is one for both, and loops are rolled where they
                // are not a tile's every time: between items it leaves the instruction caches, and its fetch was most of a
                // short item's time.)
                uint32_t vis = ~0u, lost = 0;  // a bit for each of s: the row sees the token; the token's row is not finite
#pragma unroll 1
                for (int pass = 0;; ++pass) {
                    tmem_ld_fragments(tmem + lanes + (g & 1) * N, s);
                    if (masked) {
                        if (pass == 0) {
                            // A token whose values are not finite has no finite logit in any column (those without a row, of
                            // zeros, among them): zeros in its place for the second product, and NaN for the rows that see it.
                            // (So it goes for what lies past the request's end, too; finite values there meet weights of zero.)
                            // Logits alone say it of a row whose key part is not finite, or whose sums leave fp32's range, too: its
                            // values are looked at, below, and where they are finite its weights are what its logits make them.
                            bool gone[2] = {true, true};
#pragma unroll
                            for (int i = 0; i < N / 2; ++i) gone[(i >> 1) & 1] = gone[(i >> 1) & 1] && !(fabsf(s[i]) < INFINITY);
                            const int pos = j * kTok + tok;
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                gone[k] = __all_sync(0xfu << (lane & 28), gone[k]) || (bad >> (warp >> 1) & 1);
                                if (gone[k]) lost |= 0x33333333u << 2 * k;
                            }
                            vis = 0;
                            if (p.tree == nullptr) {
#pragma unroll
                                for (int c = 0; c < kCols / 2; ++c) {
                                    const int2 limit = *reinterpret_cast<const int2*>(sm.limit + 8 * c + col2);
                                    vis |= ((pos < limit.x ? 1u : 0u) | (pos < limit.y ? 2u : 0u) | (pos + 8 < limit.x ? 4u : 0u) | (pos + 8 < limit.y ? 8u : 0u)) << 4 * c;
                                }
                            } else {
                                const int qf = first / p.H;
#pragma unroll 1
                                for (int c = 0; c < kCols; ++c) {
                                    const int q = sm.query[(c >> 1) * 8 + col2 + (c & 1)];
                                    if (q < 0) continue;
                                    const unsigned long long word = (unsigned long long)p.tree[w.r.row0 + qf + q];
#pragma unroll
                                    for (int k = 0; k < 2; ++k) {
                                        const int at = pos + 8 * k, node = at - base;
                                        if (at < w.r.L && (node < 0 || (node < 64 && (word >> node & 1)))) vis |= 1u << ((c >> 1) * 4 + 2 * k + (c & 1));
                                    }
                                }
                            }
                            // (the second product has not begun: it waits for this warp)  A lane has 16 bytes of a row in each unit.
                            static_assert(kUnits == 2 && kUnit == 32 * kTok * 16, "two units of 32 lanes' 16 bytes a token");
                            uint8_t* const part = sm.ring[g * kUnits % kRing] + (lane >> 3) * kBox + (lane & 7) * 16;
                            uint8_t* const more = sm.ring[(g * kUnits + 1) % kRing] + (lane >> 3) * kBox + (lane & 7) * 16;
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                unsigned rows_gone = __ballot_sync(~0u, (lane & 3) == 0 && (lost >> 2 * k & 1));
#pragma unroll 1
                                while (rows_gone) {
                                    const int four = (__ffs(rows_gone) - 1) >> 2, t = warp * 16 + four + 8 * k;  // lanes 4 four .. have the logits
                                    rows_gone &= rows_gone - 1;
                                    uint4* const at[2] = {reinterpret_cast<uint4*>(part + t * 128), reinterpret_cast<uint4*>(more + t * 128)};
                                    const __nv_bfloat162 none = __floats2bfloat162_rn(0.0f, 0.0f);
                                    __nv_bfloat162 sum = none;  // 0 x is 0 of what is finite, else NaN
#pragma unroll
                                    for (int i = 0; i < 2; ++i) {
                                        const uint4 v = *at[i];
                                        sum = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&v.x), none, sum);
                                        sum = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&v.y), none, sum);
                                        sum = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&v.z), none, sum);
                                        sum = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&v.w), none, sum);
                                    }
                                    if (!__any_sync(~0u, !__hbeq2(sum, none))) {
                                        if (lane >> 2 == four && !(bad >> (warp >> 1) & 1)) lost &= ~(0x33333333u << 2 * k);
                                        continue;
                                    }
                                    *at[0] = make_uint4(0, 0, 0, 0);
                                    *at[1] = make_uint4(0, 0, 0, 0);
                                }
                            }
                        }
#pragma unroll
                        for (int i = 0; i < N / 2; ++i) {
                            if (lost >> i & 1) s[i] = __int_as_float(0x7fffffff);
                            if (!(vis >> i & 1)) s[i] = -INFINITY;
                        }
                    }
                    float high = -INFINITY;
#pragma unroll
                    for (int i = 0; i < N / 2; ++i) {
                        s[i] = fmaf(s[i], f, -sub[(i >> 2) * 2 + (i & 1)]);
                        high = fmaxf(high, s[i]);
                    }
                    // (masked tiles: a row may have seen nothing before them, and its reference of 0 is none)
                    if (pass == 1 || !vote_any(1, kSoftWarps * 32, high > kGrow || masked || j == w.j0)) break;
                    // ---- the tile's maxima, by warp, then over the warps; the references, raised where it asks for it
                    float top[kCols];
#pragma unroll
                    for (int c = 0; c < kCols; ++c)
                        top[c] = fmaxf(s[(c >> 1) * 4 + (c & 1)], s[(c >> 1) * 4 + 2 + (c & 1)]) + sub[c];
                    halve(top, lane, [](float a, float b) { return fmaxf(a, b); });
                    sm.top[warp][my_col] = top[0];
                    if (kCols == 16) sm.top[warp][my_col + 1] = top[1];
                    tc::named_sync(1, kSoftWarps * 32);
                    bool moved = false;
                    if (tid < N) {
                        const float t = fmaxf(fmaxf(sm.top[0][tid], sm.top[1][tid]), fmaxf(sm.top[2][tid], sm.top[3][tid])), old = sm.ref[tid];
                        moved = t > old + kGrow || (old == -INFINITY && t > -INFINITY);
                        sm.fac[item & 1][tid] = !moved ? 1.0f : old == -INFINITY ? 0.0f : ex2(old - t);
                        if (moved) sm.ref[tid] = t;
                    }
                    moved = vote_any(1, kSoftWarps * 32, moved);
                    if (!moved) break;
#pragma unroll
                    for (int c = 0; c < kCols; c += 2) {
                        const int col = c * 4 + col2;
                        const float2 by = *reinterpret_cast<const float2*>(sm.fac[item & 1] + col), ref = *reinterpret_cast<const float2*>(sm.ref + col);
                        l[c] *= by.x;
                        l[c + 1] *= by.y;
                        sub[c] = ref.x == -INFINITY ? 0.0f : ref.x;
                        sub[c + 1] = ref.y == -INFINITY ? 0.0f : ref.y;
                    }
                    if (j > w.j0) {
                        wait(o_done + 8 * ((g - 1) & 1), (g - 1) / 2);
                        tc::fence_after_sync();
#pragma unroll 1
                        for (int k = 0; k < kBlocks * N / 16; ++k) {
                            float o[16];
                            tc::tmem_ld16(tO + lanes + 16 * k, o);
                            tc::mul16(o, sm.fac[item & 1] + 16 * k % N);
                            tc::tmem_st16(tO + lanes + 16 * k, o);
                        }
                        tc::tmem_wait_st();
                    }
                }
                // ---- weights
                const uint32_t pb = tc::smem_u32(sm.p[g & 1]) + p_at;
#pragma unroll
                for (int i = 0; i < N / 2; ++i) s[i] = ex2(s[i]);
#pragma unroll
                for (int i = 0; i < N / 2; i += 8)
                    store_transposed(pb + (i / 8) * 16 * 128, bf16x2(s[i], s[i + 1]), bf16x2(s[i + 2], s[i + 3]), bf16x2(s[i + 4], s[i + 5]),
                                     bf16x2(s[i + 6], s[i + 7]));
                tc::fence_async_smem();
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(p_ready + 8 * (g & 1));
#pragma unroll
                for (int i = 0; i < N / 2; i += 4) {
                    l[i >> 1] += s[i] + s[i + 2];
                    l[(i >> 1) + 1] += s[i + 1] + s[i + 3];
                }
            }

            // ---- the item's sums, for its output; the output before it has been read and its factors used
            if (item > 0) wait(o_free, item - 1);
            halve(l, lane, [](float a, float b) { return a + b; });
            tc::named_sync(1, kSoftWarps * 32);  // the last tile's maxima have been read
            sm.top[warp][my_col] = l[0];
            if (kCols == 16) sm.top[warp][my_col + 1] = l[1];
            tc::named_sync(1, kSoftWarps * 32);
            const long long tile0 = w.x - w.v0 + kItemCost;  // the place of the item's first tile
            const int c0 = (int)(tile0 / W), c1 = (int)((tile0 + w.kt - 1) / W);
            const int64_t at = (int64_t)w.r.row0 * p.H + first;
            if (tid < N) {
                const float sum = (sm.top[0][tid] + sm.top[1][tid]) + (sm.top[2][tid] + sm.top[3][tid]), ref = sm.ref[tid];
                sm.fac[item & 1][tid] = sum == 0.0f ? 0.0f : 1.0f / sum;  // no token seen: zeros
                if (c0 != c1) {
                    float* part = p.partials + ((size_t)blockIdx.x * 2 + (w.j0 == 0 ? 1 : 0)) * kPart;
                    part[N * kLatent + tid] = ref;
                    part[N * kLatent + N + tid] = sum;
                } else if (p.lse != nullptr && tid < rows) {
                    p.lse[at + tid] = lse_of(ref, sum);
                }
            }
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(sums_there);
            if (c0 != c1 && w.j0 == 0 && tid == 0) {  // the item begins here: what the join needs
                p.spans[blockIdx.x] = c1 - c0;
                p.span_rows[blockIdx.x * 2] = at;
                p.span_rows[blockIdx.x * 2 + 1] = rows;
            }
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == kKeyWarp) tc::tmem_dealloc(tmem, 512);
}

// The joins of the items' parts, in order.  Of items that begin in CTA c0 and go on in `more` shares after it:
template <int N>
__device__ __forceinline__ const float* part_of(const LatentAttnParams& p, int c0, int i) {
    constexpr int kPart = N * kLatent + 2 * N;
    return p.partials + ((size_t)(c0 + i * p.pair) * 2 + (i == 0 ? 1 : 0)) * kPart;
}

// Items of a few parts: a block has four rows of the item that begins in CTA blockIdx.x, a warp a row (64 requests of 128 heads
// 216 us in all; with sixteen rows, which one block fills an SM with, 219).
constexpr int kJoinWarps = 4;
template <int N>
__global__ void __launch_bounds__(kJoinWarps * 32) gdn_latent_join_kernel(const __grid_constant__ LatentAttnParams p) {
    const int c0 = blockIdx.x, row = blockIdx.y * kJoinWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    tc::grid_wait();
    const int more = p.spans[c0];
    const int64_t at = p.span_rows[c0 * 2] + row, rows = p.span_rows[c0 * 2 + 1];
    if (more == 0 || row >= rows) return;
    // Everything is asked for before anything is waited for: the references and sums, and the first two parts.
    auto values = [&](int i, float4(&v)[4]) {
        const float4* part = reinterpret_cast<const float4*>(part_of<N>(p, c0, i) + row * kLatent);
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = part[lane + 32 * k];
    };
    float4 v[2][4];
    values(0, v[0]);
    values(1, v[1]);
    float m0 = -INFINITY, l0 = 0.0f;  // of part `lane`
    if (lane <= more) {
        const float* part = part_of<N>(p, c0, lane) + N * kLatent + row;
        m0 = part[0], l0 = part[N];
    }
    float top = m0;
    for (int i = lane + 32; i <= more; i += 32) top = fmaxf(top, part_of<N>(p, c0, i)[N * kLatent + row]);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
    const float by0 = factor(m0, top);
    float sum = l0 * by0;
    for (int i = lane + 32; i <= more; i += 32) {
        const float* part = part_of<N>(p, c0, i) + N * kLatent + row;
        sum = fmaf(part[N], factor(part[0], top), sum);
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) sum += __shfl_xor_sync(~0u, sum, o);
    float4 o[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) o[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 1
    for (int i = 0; i <= more; i += 2) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            if (i + j > more) break;
            const float shared = __shfl_sync(~0u, by0, (i + j) & 31);
            const float by = i + j < 32 ? shared : factor(part_of<N>(p, c0, i + j)[N * kLatent + row], top);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                o[k].x = fmaf(v[j][k].x, by, o[k].x);
                o[k].y = fmaf(v[j][k].y, by, o[k].y);
                o[k].z = fmaf(v[j][k].z, by, o[k].z);
                o[k].w = fmaf(v[j][k].w, by, o[k].w);
            }
            if (i + j + 2 <= more) values(i + j + 2, v[j]);
        }
    }
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
    for (int k = 0; k < 4; ++k)
        reinterpret_cast<uint2*>(p.out + at * kLatent)[lane + 32 * k] = make_uint2(bf16x2(o[k].x * inv, o[k].y * inv), bf16x2(o[k].z * inv, o[k].w * inv));
    if (p.lse != nullptr && lane == 0) p.lse[at] = lse_of(top, sum);
}

// A few items of many parts: a block has half of a row's channels, eight groups of 64 threads take the parts in turn;
// the blocks of a row and half take the items in turn.
constexpr int kJoinThreads = 512;
template <int N>
__global__ void __launch_bounds__(kJoinThreads) gdn_latent_join_long_kernel(const __grid_constant__ LatentAttnParams p) {
    constexpr int kTurns = kJoinThreads / 64;
    __shared__ float weight[kMaxCtas];
    __shared__ float4 acc[kTurns][64];
    __shared__ float red[2][kJoinThreads / 32];
    const int row = blockIdx.x >> 1, half = blockIdx.x & 1, tid = threadIdx.x, lane = tid & 31;
    constexpr int kEarly = 5;
    __shared__ int spans[kMaxCtas];
    tc::grid_wait();
    if (tid < kMaxCtas) spans[tid] = tid < p.ctas ? p.spans[tid] : 0;
    __syncthreads();
    int turn = 0;
#pragma unroll 1
    for (int word = 0; 32 * word < p.ctas; ++word) {
        const int span = spans[32 * word + lane];
        unsigned found = __ballot_sync(~0u, span > 0);  // (the same in all of the block's warps)
#pragma unroll 1
        for (; found != 0; found &= found - 1) {
            const int c0 = 32 * word + __ffs(found) - 1, more = __shfl_sync(~0u, span, __ffs(found) - 1);
            if (turn++ % (int)gridDim.y != (int)blockIdx.y) continue;
            const int64_t at = p.span_rows[c0 * 2] + row, rows = p.span_rows[c0 * 2 + 1];
            if (row >= rows) continue;
            // Asked for before anything is waited for: the references and sums (there are fewer parts than threads), and this
            // thread's first parts.
            auto value = [&](int i) {
                return reinterpret_cast<const float4*>(part_of<N>(p, c0, i) + row * kLatent + half * (kLatent / 2))[tid & 63];
            };
            static_assert(kMaxCtas <= kJoinThreads && kMaxCtas % 32 == 0, "a part to a thread");
            float m = -INFINITY, l = 0.0f;
            if (tid <= more) {
                const float* part = part_of<N>(p, c0, tid) + N * kLatent + row;
                m = part[0], l = part[N];
            }
            float4 early[kEarly];
#pragma unroll
            for (int i = 0; i < kEarly; ++i)
                early[i] = (tid >> 6) + i * kTurns <= more ? value((tid >> 6) + i * kTurns) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            float top = m;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
            if (lane == 0) red[0][tid >> 5] = top;
            __syncthreads();
#pragma unroll
            for (int i = 0; i < kJoinThreads / 32; ++i) top = fmaxf(top, red[0][i]);
            const float mine = factor(m, top);
            if (tid <= more) weight[tid] = mine;
            float sum = l * mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) sum += __shfl_xor_sync(~0u, sum, o);
            if (lane == 0) red[1][tid >> 5] = sum;
            __syncthreads();
            sum = 0.0f;
#pragma unroll
            for (int i = 0; i < kJoinThreads / 32; ++i) sum += red[1][i];
            float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            auto add = [&](const float4& v, float by) {
                o.x = fmaf(v.x, by, o.x);
                o.y = fmaf(v.y, by, o.y);
                o.z = fmaf(v.z, by, o.z);
                o.w = fmaf(v.w, by, o.w);
            };
#pragma unroll
            for (int i = 0; i < kEarly; ++i) {
                const int part = (tid >> 6) + i * kTurns;
                if (part <= more) add(early[i], weight[part]);
            }
#pragma unroll 10
            for (int i = (tid >> 6) + kEarly * kTurns; i <= more; i += kTurns) add(value(i), weight[i]);
            acc[tid >> 6][tid & 63] = o;
            __syncthreads();
            if (tid < 64) {
#pragma unroll
                for (int i = 1; i < kTurns; ++i) {
                    const float4 v = acc[i][tid];
                    o.x += v.x;
                    o.y += v.y;
                    o.z += v.z;
                    o.w += v.w;
                }
                const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
                reinterpret_cast<uint2*>(p.out + at * kLatent + half * (kLatent / 2))[tid] = make_uint2(bf16x2(o.x * inv, o.y * inv), bf16x2(o.z * inv, o.w * inv));
                if (p.lse != nullptr && tid == 0 && half == 0) p.lse[at] = lse_of(top, sum);
            }
            __syncthreads();
        }
    }
}

template <int N>
cudaError_t launch(LatentAttnParams& p, cudaStream_t s) {
    constexpr int smem = (int)sizeof(LatentSmem<N>);
    static_assert(smem <= 227 * 1024, "shared memory of a CTA");
    static std::once_flag once[64];
    static cudaError_t err[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || dev < 0 || dev >= 64) return e != cudaSuccess ? e : cudaErrorInvalidDevice;
    std::call_once(once[dev], [dev] {
        err[dev] = cudaFuncSetAttribute(gdn_latent_tiles_kernel<N>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    });
    if (err[dev] != cudaSuccess) return err[dev];
    const int grid = std::min(device_sm_count(), kMaxCtas) / p.pair * p.pair;
    p.ctas = grid;
    e = launch_dependent(gdn_latent_tiles_kernel<N>, dim3((unsigned)grid), kThreads, smem, s, p);
    if (e != cudaSuccess) return e;
    // Items by the requests' mean: where each goes to sixteen shares or more, by blocks that split the parts.  (One kernel
    // of a block to a row for all: 49 of 264 us for 64 requests of 128 heads.)
    const int64_t items = (((int64_t)p.T * p.H + p.B - 1) / p.B + N * p.pair - 1) / (N * p.pair) * p.B;
    if (items * 16 <= grid / p.pair)
        return launch_dependent(gdn_latent_join_long_kernel<N>, dim3(2 * N, (unsigned)std::min<int64_t>(items * p.pair, 8)), kJoinThreads, 0, s, p);
    return launch_dependent(gdn_latent_join_kernel<N>, dim3((unsigned)grid, N / kJoinWarps), kJoinWarps * 32, 0, s, p);
}

}  // namespace

// The largest: 64 rows.
size_t latent_tiles_workspace() { return (size_t)2 * std::min(device_sm_count(), kMaxCtas) * (64 * kLatent + 2 * 64) * 4; }

// Rows of an item: what the requests have on average, up to 64.  Fewer where the contexts that the table has room for are so
// short that a CTA gets a few tiles only: an item's queries, products and output are then most of the time, and the rows of
// one request go to up to eight CTAs that work on the same tokens.  Measured in us at 16, 32 and 64 rows for contexts that
// give a CTA t tiles of 16 rows: one request of 32 heads, 4,096 tokens (t = 0.8) 13.0, 15.3; 16 of 32 heads, 2,000 (6.7) 20.8,
// 20.8; 4 of 128 heads, 2,000 (6.7) 20.6, 21.2, 27.9; 4,096 (13.5) 26.4, 23.8, 31.4; 8 of 64 heads, 1,000 (3.4) 16.2, 17.4, 28.2;
// 16 of 64 heads, 2,000 (13.5) 27.5, 25.2, 23.9; one of 64 heads, 16,000 (6.6) 19.7, 20.1, 19.2; 40,000 (16) 30.4, 26.6, 24.3;
// 4 of 64 heads, 16,000 (26) 41.9, 37.2, 32.2.  The host knows the table's width and not the lengths: a table with room
// for much more than its contexts gets the rows of long ones (the last of three figures, or of two).
cudaError_t launch_latent_tiles(LatentAttnParams& p, cudaStream_t s) {
    const int64_t rows = ((int64_t)p.T * p.H + p.B - 1) / p.B, sms = device_sm_count();
    const int64_t tiles = (((int64_t)p.width << p.log2_page) + kTok - 1) / kTok;  // of the longest request that the table has room for
    auto of = [&](int n) { return (rows + n - 1) / n; };
    const double t = (double)of(16) * (double)p.B * (double)tiles / (double)sms;
    const int n = rows <= 16 || t <= 8.0 ? 16 : rows <= 32 || t <= 14.0 ? 32 : 64;
    p.pair = (int)std::min(std::min(of(n), (int64_t)(n == 64 ? 2 : 128 / n)), sms);
    return n == 16 ? launch<16>(p, s) : n == 32 ? launch<32>(p, s) : launch<64>(p, s);
}

}  // namespace gdn
