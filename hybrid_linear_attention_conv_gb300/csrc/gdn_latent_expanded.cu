// gdn_latent_expanded.cu -- latent attention, expanded form: heads of keys [128 | 64 shared] and values of 128,
// 256 queries of a head against 128 tokens at a time on the tcgen05 tensor cores.  For row i of a head,
//   t_ij = scale log2(e) q_i . k_j,   o_i = sum_j 2^(t_ij - m_i) v_j / sum_j 2^(t_ij - m_i).
//
// A CTA has two tiles of 128 queries (a tile's row is a lane of tensor memory, and has two threads of the
// softmax, 64 tokens each), which share the keys and values in its ring.  Tensor memory: two tiles of logits (128 columns each),
// over which their weights are written (bf16) as the second product's A operand, and two
// outputs (128 columns each).  Two warps issue the MMAs, one for each tile of queries, P V of a tile of tokens and then
// the next one's Q K^T: while one is in its softmax the tensor pipe works for the other.  (One warp for both, each
// unit waited for by itself: 6,200 cycles for 256 x 128, twice the products' own, in the waits between its issues.)
//
// The reference m of a row is raised, and the output rescaled, only when a tile's maximum exceeds it by more than
// 2^16: weights are rounded to bf16, whose exponents are fp32's, so that costs no precision, only range.
// Their sum is of the unrounded ones, in fp32.
//
// Blocks of 256 queries are CTAs of the grid, those with the most tokens first (23 ragged chunks: 193 us with requests in
// order, 167 so; 151 with what came after; requests past kSorted come in their order: 128 of 8 heads 322 us, 129 337).  A CTA that has done one takes over the next that has not begun (cluster launch control), so that
// a block's queries and first keys are on their way while the one before it ends.
//
// Bound by the tensor pipe, in a chain: 8,192 queries and tokens of 32 heads take 525 to 545 us (by box), 1.26 to 1.31 PFLOP/s, 3,900 cycles for
// 256 x 128 of which the products need 2,584.  Few queries after long contexts: by HBM, 4.0 to 4.8 TB/s.
#include <cuda_bf16.h>

#include <algorithm>
#include <mutex>

#include "gdn_kv_tc.cuh"
#include "gdn_latent.cuh"
#include "gdn_latent_tc.cuh"
#include "gdn_tc.cuh"

namespace gdn {
namespace {

constexpr int kSoftWarps = 16;
constexpr int kLoadWarp = kSoftWarps, kMmaWarp = kSoftWarps + 1, kGuardWarp = kSoftWarps + 3;  // two for the MMAs
constexpr int kThreads = (kSoftWarps + 4) * 32;
constexpr int kM = 128;                  // queries of a tile
constexpr int kN = 128;                  // tokens of a tile
constexpr int kBlock = 2 * kM;           // queries of a CTA
constexpr int kGroup = kM * 128;         // 128 rows x 64 channels
constexpr int kKeyUnits = (kNope + kKeyPart) / 64, kValueUnits = kValue / 64;
constexpr int kRing = 8;                 // units of a group
constexpr float kGrow = 16.0f;           // how far a weight may exceed the reference, in powers of two
constexpr int kSoftRegs = 104, kOtherRegs = 64;  // 512 x 104 + 128 x 64 = 640 x 96
constexpr int kTurnAt = kKeyUnits - 1;   // the unit of keys before whose products the turn passes
constexpr int kSorted = 128;             // requests whose blocks are sorted by their tokens
constexpr int kAhead = 1;                // tiles requested into the L2 before the loader waits for their places
constexpr uint64_t kDrainNs = 200000000ull;

struct Item {
    int n, L, row0, u0;  // queries and tokens of the request, its first rows of q and of k
    int block, h;        // block of queries, head; h < 0: the end
};

struct ExpandedSmem {
    alignas(1024) uint8_t q[2][kKeyUnits][kGroup];
    alignas(1024) uint8_t ring[kRing][kGroup];
    alignas(16) uint4 next;              // the launch control's answer
    Item item[2];
    alignas(8) uint64_t full[kRing], empty[kRing], s_full[2], p_ready[2][2], o_done[2], o_free[2], item_full[2], item_empty[2], turn[2];
    uint64_t q_full, q_empty, next_full, drained[2], guarded[2], joined;
    uint32_t tmem;
    int at[kSoftWarps][3];               // a softmax warp's place: its block's first unit of the ring, guarded tiles before it, meetings
    int bad[2];                          // of guarded tiles in turn: there is a value that is not finite
    int dead;
    float row[2][2][kM];                 // by tile and half: the rows' maxima, or sums
};

__device__ __forceinline__ Item read_item(const volatile Item& x) {
    Item it;
    it.n = x.n, it.L = x.L, it.row0 = x.row0, it.u0 = x.u0, it.block = x.block, it.h = x.h;
    return it;
}

// What a tile of queries of a block takes part in: its first query, and of the tiles of tokens, 0 to tiles - 1 in the
// ring, those from `from` in steps of `step` below `end` (none: it has no queries).  A block with one tile of queries
// only goes to both halves of the CTA, which take the tiles of tokens in turn and join their outputs at the end.
struct Part {
    int first, tiles, from, step, end;
    bool joined;
    __device__ __forceinline__ bool has(int j) const { return j >= from && j < end && (!joined || ((j - from) & 1) == 0); }
    __device__ __forceinline__ int last() const { return end - 1 - (joined ? (end - 1 - from) & 1 : 0); }
};
// Queries and tokens of request b (none: it is not there), as far as they lie within the tensors.
struct Lengths {
    int row0, n, k0, L;
};
__device__ __forceinline__ Lengths lengths(const ExpandedAttnParams& p, int b) {
    Lengths x{0, 0, 0, 0};
    if (b < p.B) {
        x.row0 = p.start[b];
        x.n = x.row0 < 0 ? 0 : max(0, min(p.start[b + 1], p.T) - x.row0);
        x.k0 = max(0, p.key_start[b]);
        x.L = max(0, min(p.key_start[b + 1], p.S) - x.k0);
    }
    return x;
}
__device__ __forceinline__ int token_tiles(const Item& it, int first) {
    const int seen = min(it.L, it.L - it.n + min(it.n, first + kM));
    return max(1, (seen + kN - 1) / kN);
}
__device__ __forceinline__ Part part_of(const Item& it, int side) {
    const int first = it.block * kBlock;
    const bool second = first + kM < it.n;  // the block has a second tile of queries
    Part t;
    t.tiles = token_tiles(it, second ? first + kM : first);
    t.joined = !second && t.tiles > 1;
    t.first = first + (second ? side * kM : 0);
    t.step = t.joined ? 2 : 1;
    t.from = t.joined ? side : 0;
    t.end = !second && !t.joined && side == 1 ? 0 : token_tiles(it, t.first);
    return t;
}

// The first of a block's tiles of tokens that some of its queries do not see all of: from there on they are guarded.
__device__ __forceinline__ int first_guarded(const Item& it, int tiles) {
    return min(tiles, max(0, min(it.L, it.L - it.n + it.block * kBlock + 1)) / kN);
}

__device__ __forceinline__ float lse_of(float m, float l) {
    return l == 0.0f ? -INFINITY : ((m == -INFINITY ? 0.0f : m) + log2f(l)) * 0.69314718055994531f;
}

__device__ __forceinline__ float factor(float m, float top) { return m == top ? 1.0f : ex2(m - top); }

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
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

// Of two lanes, `apart` lanes from one another, the one without `upper` gets both a's, the other both b's, its own lane's place first
// where it is the lower one.
__device__ __forceinline__ void swap_chunks(bool upper, int apart, const uint4& a, const uint4& b, uint4& low, uint4& high) {
    const uint4 give = upper ? a : b, keep = upper ? b : a;
    const uint4 got = make_uint4(__shfl_xor_sync(~0u, give.x, apart), __shfl_xor_sync(~0u, give.y, apart), __shfl_xor_sync(~0u, give.z, apart),
                                 __shfl_xor_sync(~0u, give.w, apart));
    low = upper ? got : keep;
    high = upper ? keep : got;
}

// Asks the launch control for a CTA of the grid that has not begun; its answer comes with 16 bytes on `bar`.
__device__ __forceinline__ void ask_next(uint32_t answer, uint32_t bar) {
    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(answer), "r"(bar) : "memory");
}
// The answer: the CTA's index, or -1 when there was none (then it is not to be asked again).
__device__ __forceinline__ int next_of(uint32_t answer) {
    uint32_t got, x;
    asm volatile(
        "{\n\t.reg .b128 a;\n\t.reg .pred p;\n\tld.shared.b128 a, [%2];\n\t"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, a;\n\tselp.u32 %0, 1, 0, p;\n\tmov.u32 %1, 0;\n\t"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, a;\n\t}"
        : "=r"(got), "=r"(x)
        : "r"(answer)
        : "memory");
    return got ? (int)x : -1;
}

__global__ void __launch_bounds__(kThreads, 1) gdn_latent_expanded_kernel(const __grid_constant__ ExpandedAttnParams p) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    ExpandedSmem& sm = *reinterpret_cast<ExpandedSmem*>(smem_raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if ((tc::smem_u32(smem_raw) & 1023) != 0) {  // (the swizzle's atoms; the kernel has no other shared memory)
        if (tid == 0) atomicOr(p.gave_up, 8);
        return;
    }
    const uint32_t full = tc::smem_u32(sm.full), empty = tc::smem_u32(sm.empty), s_full = tc::smem_u32(sm.s_full),
                   p_ready = tc::smem_u32(sm.p_ready), o_done = tc::smem_u32(sm.o_done), o_free = tc::smem_u32(sm.o_free),
                   item_full = tc::smem_u32(sm.item_full), item_empty = tc::smem_u32(sm.item_empty), q_full = tc::smem_u32(&sm.q_full),
                   q_empty = tc::smem_u32(&sm.q_empty), next_full = tc::smem_u32(&sm.next_full), drained = tc::smem_u32(sm.drained),
                   turn = tc::smem_u32(sm.turn), guarded = tc::smem_u32(sm.guarded), joined = tc::smem_u32(&sm.joined);
    if (tid == 0) {
        tc::prefetch_map(&p.tm_q);
        tc::prefetch_map(&p.tm_k);
        tc::prefetch_map(&p.tm_r);
        tc::prefetch_map(&p.tm_v);
        sm.dead = 0;
        for (int i = 0; i < kRing; ++i) {
            tc::mbar_init(full + 8 * i, 1);
            tc::mbar_init(empty + 8 * i, 3);  // two tiles of queries, the guard
        }
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(drained + 8 * i, 1);
            tc::mbar_init(guarded + 8 * i, 1);
            tc::mbar_init(turn + 8 * i, 1);
            tc::mbar_init(s_full + 8 * i, 1);
            tc::mbar_init(o_done + 8 * i, 1);
            tc::mbar_init(o_free + 8 * i, kSoftWarps / 2);
            tc::mbar_init(item_full + 8 * i, 1);
            tc::mbar_init(item_empty + 8 * i, kSoftWarps + 3);
        }
        for (int i = 0; i < 4; ++i) tc::mbar_init(p_ready + 8 * i, kSoftWarps / 4);
        tc::mbar_init(q_full, 1);
        tc::mbar_init(q_empty, 2);
        tc::mbar_init(next_full, 1);
        tc::mbar_init(joined, kSoftWarps);
    }
    if (warp == kMmaWarp) tc::tmem_alloc(tc::smem_u32(&sm.tmem), 512);
    tc::fence_before_sync();
    tc::grid_wait();  // nothing above touches memory that an earlier kernel may write
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = sm.tmem, tO = tmem + 2 * kN;
    volatile int* dead = &sm.dead;

    // A bounded wait.  The first that gives up ends all waiting of the CTA, and its copies: the roles run
    // through on whatever is there, and the device's status word tells.
    auto wait = [&](uint32_t bar, uint32_t parity) {
        parity &= 1;
        if (tc::mbar_test(bar, parity)) return;
        if (*dead) return;
        if (!tc::mbar_wait(bar, parity, p.wait_ns)) {
            *dead = 1;
            atomicOr(p.gave_up, 16);
        }
    };

    // Whether the CTA's copies have ended, the same answer for a warp's lanes: what they then do or leave out has votes in it.
    auto over = [&]() { return __any_sync(~0u, *dead != 0) != 0; };

    // A wait for a barrier in each lane at once (each that has one to wait for).
    auto wait_lanes = [&](bool mine, uint32_t bar, uint32_t parity) {
        const bool there = !mine || tc::mbar_test(bar, parity & 1);
        if (!__all_sync(~0u, there)) {
            if (!there) wait(bar, parity);
            __syncwarp();
        }
        tc::fence_after_sync();
    };

    // Inside the branches: code after a join of the two would have to fit the smaller number.
    if (warp >= kSoftWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == kLoadWarp) {
        // ------------------------------------------------------------ items and tiles
        int count = 0, u = 0, sent = 0, sent_q = 0, asked = 0;
        auto ask = [&]() {
            __syncwarp();
            if (lane == 0) {
                tc::mbar_arrive_expect_tx(next_full, 16);
                ask_next(tc::smem_u32(&sm.next), next_full);
            }
            __syncwarp();
        };
        // The block of CTA `index` of the grid (h < 0: the requests have none).  Of up to kSorted requests the blocks come in the
        // order of their tokens, the most first: a lane has some of the requests, and the number of a block's tiles is searched
        // for by counting, from the requests' lengths, the blocks that have as many or more.
        constexpr int kEach = kSorted / 32;
        const bool sorted = p.B > 1 && p.B <= kSorted;
        int n_of[kEach], L_of[kEach], most = 0;
        if (sorted) {
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
                const Lengths x = lengths(p, i * 32 + lane);
                n_of[i] = x.n, L_of[i] = x.L;
                most = max(most, x.L);
            }
            most = max(1, (__reduce_max_sync(~0u, most) + kN - 1) / kN);
        }
        // blocks of a request's that have `tiles` tiles of tokens or more (its last ones)
        auto long_blocks = [&](int n, int L, int tiles) {
            const int blocks = (n + kBlock - 1) / kBlock;
            if (tiles <= 1) return blocks;
            const int64_t more = (int64_t)(tiles - 1) * kN;  // tokens that such a block's last query sees more than
            return L <= more ? 0 : blocks - (int)(max((int64_t)0, more - L + n) / kBlock);
        };
        auto find_sorted = [&](int index) {
            Item it;
            it.h = -1;
            const int rank = index / p.H;
            auto all = [&](int tiles) {
                int c = 0;
#pragma unroll
                for (int i = 0; i < kEach; ++i) c += long_blocks(n_of[i], L_of[i], tiles);
                return (int)__reduce_add_sync(~0u, c);
            };
            if (rank >= all(1)) return it;
            int lo = 1, hi = most + 1, before = 0;  // all(lo) > rank >= all(hi)
            while (hi - lo > 1) {
                const int x = (lo + hi) >> 1, c = all(x);
                if (c > rank) lo = x;
                else hi = x, before = c;
            }
            int mine = 0;
#pragma unroll
            for (int i = 0; i < kEach; ++i) mine += long_blocks(n_of[i], L_of[i], lo) - long_blocks(n_of[i], L_of[i], hi);
            int upto = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int x = __shfl_up_sync(~0u, upto, o);
                if (lane >= o) upto += x;
            }
            const int at = __ffs(__ballot_sync(~0u, rank - before < upto)) - 1;
            int rest = rank - before - (upto - mine), b = 0, block = 0;
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
                const int longer = long_blocks(n_of[i], L_of[i], hi), c = long_blocks(n_of[i], L_of[i], lo) - longer;
                if (rest >= 0 && rest < c) {
                    b = i * 32 + lane;
                    block = (n_of[i] + kBlock - 1) / kBlock - longer - 1 - rest;
                }
                rest -= c;
            }
            const Lengths x = lengths(p, __shfl_sync(~0u, b, at));
            it.row0 = x.row0, it.n = x.n, it.u0 = x.k0, it.L = x.L;
            it.block = __shfl_sync(~0u, block, at);
            it.h = index % p.H;
            return it;
        };
        // Of one request, or of more of them, requests in order, 32 at a time.
        auto find = [&](int index) {
            if (sorted) return find_sorted(index);
            Item it;
            it.h = -1;
            int rest = index / p.H;
            for (int b0 = 0; b0 < p.B; b0 += 32) {
                const Lengths x = lengths(p, b0 + lane);
                const int blocks = (x.n + kBlock - 1) / kBlock;
                int upto = blocks;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int add = __shfl_up_sync(~0u, upto, o);
                    if (lane >= o) upto += add;
                }
                const unsigned past = __ballot_sync(~0u, rest < upto);
                if (past != 0) {
                    const int at = __ffs(past) - 1;
                    it.row0 = __shfl_sync(~0u, x.row0, at);
                    it.n = __shfl_sync(~0u, x.n, at);
                    it.block = __shfl_sync(~0u, upto, at) - 1 - rest;  // the last first
                    it.h = index % p.H;
                    it.u0 = __shfl_sync(~0u, x.k0, at);
                    it.L = __shfl_sync(~0u, x.L, at);
                    break;
                }
                rest -= __shfl_sync(~0u, upto, 31);
            }
            return it;
        };
        ask();
        Item it = find(blockIdx.x), it_next = it;
        bool more = true;
        // the block after this one, and the question for the one after that
        auto look_ahead = [&]() {
            wait(next_full, asked);
            if (over()) {  // (the answer may be on its way: waited for below)
                more = false;
                return;
            }
            const int index = next_of(tc::smem_u32(&sm.next));
            tc::fence_async_smem();  // read before it is written again
            more = index >= 0;       // (after the first without, it is not to be asked again)
            if (!more) return;
            ++asked;
            ask();
            it_next = find(index);
        };
        // Tile j of a block into the L2: the ring's tile and a half are what the tensor pipe takes in 2 us, no longer than a
        // copy from HBM under way with all SMs' (23 ragged chunks 167 -> 152 us with it).
        auto prefetch = [&](const Item& it, int j) {
            if (tc::elect_one()) {
                for (int i = 0; i < kNope / 64; ++i) tc::tma_prefetch_3d(&p.tm_k, 64 * i, it.h, it.u0 + j * kN);
                tc::tma_prefetch_3d(&p.tm_r, 0, 0, it.u0 + j * kN);
                for (int i = 0; i < kValueUnits; ++i) tc::tma_prefetch_3d(&p.tm_v, 64 * i, it.h, it.u0 + j * kN);
            }
            __syncwarp();
        };
        while (true) {
            if (it.h < 0) {
                look_ahead();
            } else {
                const int slot = count & 1;
                if (count >= 2) wait(item_empty + 8 * slot, count / 2 - 1);
                if (over()) break;  // (its place may still be read)
                if (lane == 0) {
                    sm.item[slot] = it;
                    tc::mbar_arrive(item_full + 8 * slot);
                }
                __syncwarp();
                const int tiles = part_of(it, 0).tiles, second = part_of(it, 1).first;
                // Never into a place whose wait gave up: a second arrival in a phase that still awaits its bytes is a fault.
                auto unit = [&](const CUtensorMap* map, int x, int h, int y) {
                    const int s = u % kRing;
                    if (u >= kRing) wait(empty + 8 * s, u / kRing - 1);
                    if (!over()) {
                        sent = u + 1;
                        if (tc::elect_one()) {
                            tc::mbar_arrive_expect_tx(full + 8 * s, kGroup);
                            tc::tma_load_3d(tc::smem_u32(sm.ring[s]), map, x, h, y, full + 8 * s);
                        }
                        __syncwarp();
                    }
                    ++u;
                };
                if (count > 0) wait(q_empty, count - 1);
                if (!over()) {
                    sent_q = count + 1;
                    if (tc::elect_one()) {
                        tc::mbar_arrive_expect_tx(q_full, 2 * kKeyUnits * kGroup);
                        for (int i = 0; i < 2 * kKeyUnits; ++i)
                            tc::tma_load_3d(tc::smem_u32(sm.q[i / kKeyUnits][i % kKeyUnits]), &p.tm_q, 64 * (i % kKeyUnits), it.h,
                                            it.row0 + (i < kKeyUnits ? it.block * kBlock : second), q_full);
                    }
                    __syncwarp();
                }
                ++count;
                for (int j = 0; j < tiles; ++j) {
                    if (j + kAhead < tiles) prefetch(it, j + kAhead);
                    if (j == max(0, tiles - 2) && more && it_next.h >= 0 && tiles > 2) {
                        prefetch(it_next, 0);
                        if (tc::elect_one()) {
                            const int second_next = part_of(it_next, 1).first;
                            for (int i = 0; i < 2 * kKeyUnits; ++i)
                                tc::tma_prefetch_3d(&p.tm_q, 64 * (i % kKeyUnits), it_next.h, it_next.row0 + (i < kKeyUnits ? it_next.block * kBlock : second_next));
                        }
                        __syncwarp();
                    }
                    for (int i = 0; i < kNope / 64; ++i) unit(&p.tm_k, 64 * i, it.h, it.u0 + j * kN);
                    unit(&p.tm_r, 0, 0, it.u0 + j * kN);
                    for (int i = 0; i < kValueUnits; ++i) unit(&p.tm_v, 64 * i, it.h, it.u0 + j * kN);
                    if (j == min(1, tiles - 1)) look_ahead();  // (the ring is full by now)
                }
            }
            if (!more) break;
            it = it_next;
        }
        // The end, in a place that is free.  After a wait that gave up it may still be the place of a block whose output
        // goes by it: it stays as it is, and the other warps, which look at `dead` behind every block, leave by that.
        const int slot = count & 1;
        if (count >= 2) wait(item_empty + 8 * slot, count / 2 - 1);
        if (lane == 0) {
            if (!*dead) sm.item[slot].h = -1;
            tc::mbar_arrive(item_full + 8 * slot);
        }
        __syncwarp();
        // Everything on its way lands before the CTA ends, also that of a block whose other warps' waits give up after this.
        tc::mbar_wait(next_full, asked & 1, kDrainNs);  // (done, if its answer has been read)
        if (sent_q > 0) tc::mbar_wait(q_full, (sent_q - 1) & 1, kDrainNs);
        for (int i = max(0, sent - kRing); i < sent; ++i) tc::mbar_wait(full + 8 * (i % kRing), (i / kRing) & 1, kDrainNs);
    } else if (warp == kMmaWarp || warp == kMmaWarp + 1) {
        // ------------------------------------------------------------ MMAs of one tile of queries
        constexpr uint32_t id_s = tc::idesc_bf16(kM, kN), id_o = tc::idesc_bf16(kM, 64) | 1u << 16;  // values MN-major
        const int side = warp - kMmaWarp;
        const uint32_t tS = tmem + side * kN, tOut = tO + side * kValue;
        // Turns: a tile's group of MMAs (the product of its weights, the next logits), then the other's.
        // (Without them the two fell into step, both in their products, then both in their softmax: 693 us for 8,192 queries.)
        constexpr uint32_t hi = tc::kDescHiSw128;
        const uint32_t ring = tc::smem_u32(sm.ring[0]), queries = tc::smem_u32(sm.q[side][0]);
        int u = 0, done = 0, items_done = 0, turns = 0, guards = 0;
        for (int count = 0;; ++count) {
            wait(item_full + 8 * (count & 1), count / 2);
            const Item it = sm.item[count & 1];
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(item_empty + 8 * (count & 1));
            if (over() || it.h < 0) break;
            const Part part = part_of(it, side);
            const int tiles = part.tiles, from_guard = first_guarded(it, tiles);
            const int all_see = max(0, min(it.L, it.L - it.n + part.first + 1));
            // Group j: the product of tile j's weights and values, the logits of tile j + 1.  What this tile's queries do not
            // see is given back (once it is there: the other tile may be a turn of the ring behind).
            for (int j = -1; j < tiles; ++j, ++turns) {
                const int u_value = u - kValueUnits, u_key = u;
                const int guard = guards + j - from_guard;
                const bool product = part.has(j), logits = part.has(j + 1), keys = j + 1 < tiles, start = j == part.from;
                {
                    // lanes: the keys' units, the queries, the values' units, the weights, the output's place, the turn, the guard
                    const bool key = lane < kKeyUnits, value = lane >= 4 && lane < 4 + kValueUnits;
                    const int unit = key ? u_key + lane : u_value + lane - 4;
                    const bool mine = key ? keys : lane == 3 ? j < 0 : value ? j >= 0 : lane == 6 || lane == 7 ? product : lane == 8 ? product && start && items_done > 0
                                                                                                                   : lane == 9  ? side == 1 || turns > 0
                                                                                                                   : lane == 10 && product && j >= from_guard;
                    wait_lanes(mine, key || value ? full + 8 * (unit % kRing) : lane == 3 ? q_full : lane < 8 ? p_ready + 8 * (2 * side + lane - 6) : lane == 8 ? o_free + 8 * side : lane == 9 ? turn + 8 * side : guarded + 8 * (guard & 1),
                               key || value ? unit / kRing : lane == 3 ? count : lane < 8 ? done : lane == 8 ? items_done - 1 : lane == 9 ? turns - (side == 0) : guard / 2);
                }
                // (as its softmax has it)
                const bool skip = product && j * kN + kN > all_see && *(volatile int*)&sm.bad[guard & 1] != 0;
                if (tc::elect_one()) {
                    if (product) {
                        if (!skip)
#pragma unroll
                            for (int ks = 0; ks < 8; ++ks)
#pragma unroll
                                for (int i = 0; i < kValueUnits; ++i)
                                    tc::mma_bf16_ts_lo(tOut + 64 * i, tS + (ks >> 2) * 64 + (ks & 3) * 8, tc::desc_lo_sw128(ring + (u_value + i) % kRing * kGroup) + ks * (16 * 128 >> 4),
                                                       hi, id_o, ks > 0 || !start);
#pragma unroll
                        for (int i = 0; i < kValueUnits; ++i) tc::mma_commit(empty + 8 * ((u_value + i) % kRing));
                        tc::mma_commit(o_done + 8 * side);
                    }
                    if (!logits) tc::mbar_arrive(turn + 8 * (side ^ 1));
                    if (logits) {
#pragma unroll
                        for (int i = 0; i < kKeyUnits; ++i) {
                            if (i == kTurnAt) tc::mbar_arrive(turn + 8 * (side ^ 1));  // by the time that the other warp has seen it these are done
                            const uint32_t q = tc::desc_lo_sw128(queries + i * kGroup), k = tc::desc_lo_sw128(ring + (u_key + i) % kRing * kGroup);
#pragma unroll
                            for (int ks = 0; ks < 4; ++ks) tc::mma_bf16_lo(tS, q + 2 * ks, k + 2 * ks, hi, id_s, i + ks > 0);
                            tc::mma_commit(empty + 8 * ((u_key + i) % kRing));
                        }
                        tc::mma_commit(s_full + 8 * side);
                        if (j + 1 == part.last()) tc::mma_commit(q_empty);
                    }
                }
                __syncwarp();
                if (j >= 0 && !product && lane < kValueUnits) tc::mbar_arrive(empty + 8 * ((u_value + lane) % kRing));
                if (keys && !logits && lane < kKeyUnits) tc::mbar_arrive(empty + 8 * ((u_key + lane) % kRing));
                if (j < 0 && part.end == 0 && lane == 0) tc::mbar_arrive(q_empty);  // it has no queries
                done += product;
                if (keys) u += kKeyUnits + kValueUnits;
            }
            items_done += part.end > 0;
            guards += tiles - from_guard;
        }
        // every MMA has ended before tensor memory is given back
        if (tc::elect_one()) tc::mma_commit(drained + 8 * side);
        __syncwarp();
        tc::mbar_wait(drained + 8 * side, 0, kDrainNs);
    } else if (warp == kGuardWarp) {
        // ------------------------------------------------------------ values of tiles that not every query sees
        // The product multiplies what a row does not see by weights of zero.  Values past the request's end, whatever they
        // are, become zeros here where they are not all finite; of a value that is not finite, which other rows may see, the
        // softmax's warps are told.
        int u0 = 0, guards = 0;
        for (int count = 0;; ++count) {
            wait(item_full + 8 * (count & 1), count / 2);
            const Item it = sm.item[count & 1];
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(item_empty + 8 * (count & 1));
            if (over() || it.h < 0) break;
            const int tiles = part_of(it, 0).tiles;
            const int from_guard = first_guarded(it, tiles);
            for (int j = 0; j < tiles; ++j) {
                const int unit = u0 + (kKeyUnits + kValueUnits) * j, u = unit + lane;
                const bool mine = lane < kKeyUnits + kValueUnits;
                wait_lanes(mine, full + 8 * (u % kRing), u / kRing);
                if (j >= from_guard) {
                    // Looked over without a branch (the softmax waits for it), and again, row by row, where there is such a value.
                    const __nv_bfloat162 none = __floats2bfloat162_rn(0.0f, 0.0f);
                    auto look = [&](const uint4& v, __nv_bfloat162(&bad)[4]) {  // 0 x is 0 of what is finite, else NaN
                        bad[0] = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&v.x), none, bad[0]);
                        bad[1] = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&v.y), none, bad[1]);
                        bad[2] = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&v.z), none, bad[2]);
                        bad[3] = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&v.w), none, bad[3]);
                    };
                    auto told = [&](const __nv_bfloat162(&bad)[4]) {
                        return __any_sync(~0u, !__hbeq2(__hadd2(__hadd2(bad[0], bad[1]), __hadd2(bad[2], bad[3])), none)) != 0;
                    };
                    __nv_bfloat162 bad[4] = {none, none, none, none};
#pragma unroll
                    for (int i = 0; i < kValueUnits; ++i) {
                        const uint4* chunk = reinterpret_cast<const uint4*>(sm.ring[(unit + kKeyUnits + i) % kRing]) + lane;
#pragma unroll 8
                        for (int c = 0; c < kM / 4; ++c) look(chunk[32 * c], bad);  // four rows at a time
                    }
                    bool any = told(bad);
                    if (any) {
                        for (int i = 0; i < 4; ++i) bad[i] = none;
#pragma unroll 1
                        for (int i = 0; i < kValueUnits; ++i) {
                            uint4* chunk = reinterpret_cast<uint4*>(sm.ring[(unit + kKeyUnits + i) % kRing]) + lane;
#pragma unroll 1
                            for (int c = 0; c < kM / 4; ++c) {
                                if (j * kN + 4 * c + (lane >> 3) >= it.L) chunk[32 * c] = make_uint4(0, 0, 0, 0);
                                else look(chunk[32 * c], bad);
                            }
                        }
                        tc::fence_async_smem();
                        any = told(bad);
                    }
                    if (lane == 0) {
                        sm.bad[guards & 1] = any;
                        tc::mbar_arrive(guarded + 8 * (guards & 1));
                    }
                    ++guards;
                    __syncwarp();
                }
                if (mine) tc::mbar_arrive(empty + 8 * (u % kRing));  // (so it is never a turn of the ring behind)
                __syncwarp();
            }
            u0 += (kKeyUnits + kValueUnits) * tiles;
        }
    }
    } else {
        // ---------------------------------------------------------------- softmax and output
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
        const int side = warp >> 3, half = warp >> 2 & 1, quad = warp & 3, local = quad * 32 + lane;
        const int pair_bar = 1 + 4 * side + quad;  // a row's two threads
        const uint32_t lanes = (uint32_t)(quad * 32) << 16, tS = tmem + lanes + side * kN, tOut = tO + lanes + side * kValue;
        const float f = p.scale_log2;
        int done = 0;
        if (lane < 3) sm.at[warp][lane] = 0;
        __syncwarp();
        volatile int* place = sm.at[warp];
        for (int count = 0;; ++count) {
            wait(item_full + 8 * (count & 1), count / 2);
            // What the loop needs of the item, and the output again (its registers are few).  The two warps that meet at a
            // barrier go on together or not at all, whatever a wait that gave up let them read.
            int limit, all_see, from, step, end;
            {
                const Item it = read_item(sm.item[count & 1]);
                if (vote_any(pair_bar, 64, it.h < 0 || *dead)) break;
                const Part part = part_of(it, side);
                const int i = part.first + local;
                limit = i < it.n ? min(it.L, it.L - it.n + i + 1) : 0;               // this row sees the tokens before it
                all_see = max(0, min(it.L, it.L - it.n + part.first + 1));         // every row those
                from = part.from;
                step = part.step;
                end = part.end;
                if (lane == 0) place[1] = place[1] - first_guarded(it, part.tiles);
                __syncwarp();
            }
            float ref = -INFINITY, l = 0.0f;  // l: of this thread's tokens
#pragma unroll 1
            for (int j = from; j < end; j += step, ++done) {
                const bool start = j == from;
                const bool masked = j * kN + kN > all_see;
                bool skip = false;
                wait(s_full + 8 * side, done);
                tc::fence_after_sync();
                if (masked) {  // with a value that is not finite the tile's product is done row by row, below
                    const int guard = place[1] + j;
                    wait(guarded + 8 * (guard & 1), guard / 2);
                    skip = vote_any(pair_bar, 64, *(volatile int*)&sm.bad[guard & 1] != 0);
                }
                const int seen = limit - j * kN - half * 64;  // this row sees the thread's tokens before it
                // ---- logits in powers of two less the reference, and their weights beside the maximum; where that asks
                // for another reference, once more from the logits.
                float2 sum[2];
                float w[32];
#pragma unroll 1
                for (int pass = 0;; ++pass) {
                    float s[64];
                    tc::tmem_ld32_start(tS + 64 * half, s);
                    tc::tmem_ld32_start(tS + 64 * half + 32, s + 32);
                    tc::tmem_wait_ld32(s);
                    tc::tmem_wait_ld32(s + 32);
                    if (masked) {
#pragma unroll
                        for (int c = 0; c < 64; ++c) s[c] = c < seen ? s[c] : -INFINITY;
                    }
                    const float sub = ref == -INFINITY ? 0.0f : ref;
                    const float2 f2 = make_float2(f, f), sub2 = make_float2(-sub, -sub);
                    float high[2] = {-INFINITY, -INFINITY};
                    sum[0] = sum[1] = make_float2(0.0f, 0.0f);
#pragma unroll
                    for (int c = 0; c < 32; ++c) {
                        const float2 x = __ffma2_rn(make_float2(s[2 * c], s[2 * c + 1]), f2, sub2);
                        high[c & 1] = fmaxf(fmaxf(high[c & 1], x.x), x.y);
                        const float2 e = make_float2(ex2(x.x), ex2(x.y));
                        sum[c & 1] = __fadd2_rn(sum[c & 1], e);
                        w[c] = __uint_as_float(bf16x2(e.x, e.y));
                    }
                    const float top = fmaxf(high[0], high[1]);
                    if (pass == 1 || !vote_any(pair_bar, 64, top > kGrow || (ref == -INFINITY && top > -INFINITY))) break;
                    sm.row[side][half][local] = top;
                    tc::named_sync(pair_bar, 64);
                    const float both = fmaxf(top, sm.row[side][half ^ 1][local]);
                    const bool grows = both > kGrow || (ref == -INFINITY && both > -INFINITY);
                    const float by = !grows ? 1.0f : ref == -INFINITY ? 0.0f : ex2(-both);
                    if (grows) ref = sub + both;
                    l *= by;
                    if (!start) {
                        wait(o_done + 8 * side, done - 1);
                        tc::fence_after_sync();
#pragma unroll 1
                        for (int k = 0; k < kValue / 32; ++k) {
                            float o[16];
                            tc::tmem_ld16(tOut + 64 * half + 16 * k, o);
#pragma unroll
                            for (int c = 0; c < 16; ++c) o[c] *= by;
                            tc::tmem_st16(tOut + 64 * half + 16 * k, o);
                        }
                        tc::tmem_wait_st();
                    }
                }
                tc::tmem_st32(tS + 64 * half, w);  // over this thread's own logits
                tc::tmem_wait_st();
                tc::fence_before_sync();
                l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
                if (skip) {
                    tc::named_sync(pair_bar, 64);  // both halves' weights; a thread 64 of its row's channels
                    tc::fence_after_sync();
                    if (!start) wait(o_done + 8 * side, done - 1);
                    tc::fence_after_sync();
                    const uint8_t* unit = sm.ring[(place[0] + (kKeyUnits + kValueUnits) * j + kKeyUnits + half) % kRing];
                    const int sees = limit - j * kN;
#pragma unroll 1
                    for (int k = 0; k < kValue / 32; ++k) {
                        float o[16];
                        tc::tmem_ld16(tOut + 64 * half + 16 * k, o);
#pragma unroll
                        for (int c = 0; c < 16; ++c) o[c] = start ? 0.0f : o[c];
#pragma unroll 1
                        for (int t = 0; t < kN; ++t) {
                            uint32_t two;
                            asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];\n\ttcgen05.wait::ld.sync.aligned;"
                                         : "=r"(two)
                                         : "r"(tS + (t >> 6) * 64 + (t & 63) / 2)
                                         : "memory");
                            const float e = __uint_as_float(t & 1 ? two & 0xffff0000u : two << 16);
                            if (t < sees) {
#pragma unroll
                                for (int c = 0; c < 16; ++c) {
                                    const uint16_t v = *reinterpret_cast<const uint16_t*>(unit + t * 128 + (((2 * k + (c >> 3)) ^ (t & 7)) << 4) + 2 * (c & 7));
                                    o[c] = fmaf(e, __uint_as_float((uint32_t)v << 16), o[c]);
                                }
                            }
                            __syncwarp();
                        }
                        tc::tmem_st16(tOut + 64 * half + 16 * k, o);
                    }
                    tc::tmem_wait_st();
                    tc::fence_before_sync();
                }
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(p_ready + 8 * (2 * side + half));
            }
            if (end > 0) {
                const Item it = read_item(sm.item[count & 1]);
                const Part part = part_of(it, side);
                const int i = part.first + local;
                // ---- output: 64 channels of a row, or, of a block that both halves of the CTA have, 32
                // all of the softmax's warps, of a joined block (a bounded wait: the two halves may leave at different blocks)
                auto meet = [&]() {
                    tc::fence_before_sync();
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive(joined);
                    wait(joined, place[2]);
                    __syncwarp();
                    if (lane == 0) place[2] = place[2] + 1;
                    __syncwarp();
                    tc::fence_after_sync();
                };
                tc::named_sync(pair_bar, 64);  // the last maxima have been read
                sm.row[side][half][local] = l;
                tc::named_sync(pair_bar, 64);
                l = sm.row[side][0][local] + sm.row[side][1][local];
                wait(o_done + 8 * side, done - 1);
                tc::fence_after_sync();
                float by = 1.0f, by_other = 0.0f;  // what the halves' outputs are multiplied by
                if (part.joined) {
                    tc::named_sync(pair_bar, 64);  // both have read the sums
                    sm.row[side][half][local] = half == 0 ? ref : l;
                    meet();
                    const float other = sm.row[side ^ 1][0][local], top = fmaxf(ref, other);
                    by = factor(ref, top);
                    by_other = factor(other, top);
                    // (in the same order on both sides)
                    const float mine = l * by, its = sm.row[side ^ 1][1][local] * by_other;
                    l = side == 0 ? mine + its : its + mine;
                    ref = top;
                }
                const float inv = l == 0.0f ? 0.0f : 1.0f / l;  // no token seen: zeros
                by *= inv;
                by_other *= inv;
                const int64_t at = ((int64_t)it.row0 + i) * p.H + it.h;
                const int channel0 = 64 * half + (part.joined ? 32 * side : 0);
#pragma unroll 1
                for (int k = 0; k < (part.joined ? 1 : 2); ++k) {
                    const int channel = channel0 + 32 * k;
                    float o[32];
                    tc::tmem_ld32(tOut + channel, o);
#pragma unroll
                    for (int c = 0; c < 32; ++c) o[c] *= by;
                    if (part.joined) {
#pragma unroll
                        for (int n = 0; n < 2; ++n) {
                            float o2[16];
                            tc::tmem_ld16(tO + lanes + (side ^ 1) * kValue + channel + 16 * n, o2);
#pragma unroll
                            for (int c = 0; c < 16; ++c) o[16 * n + c] = fmaf(o2[c], by_other, o[16 * n + c]);
                        }
                    }
                    // Four lanes change chunks of eight channels, so that they store 64 bytes of a row together: a lane
                    // storing its own row touches 32 lines an instruction, 4,000 cycles for a block.
                    uint4 x[4], y[2][2];
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        x[c] = make_uint4(bf16x2(o[8 * c], o[8 * c + 1]), bf16x2(o[8 * c + 2], o[8 * c + 3]), bf16x2(o[8 * c + 4], o[8 * c + 5]),
                                          bf16x2(o[8 * c + 6], o[8 * c + 7]));
                    const bool b0 = lane & 1, b1 = lane & 2;
#pragma unroll
                    for (int c = 0; c < 2; ++c) swap_chunks(b0, 1, x[2 * c], x[2 * c + 1], y[c][0], y[c][1]);
#pragma unroll
                    for (int c = 0; c < 2; ++c) swap_chunks(b1, 2, y[0][c], y[1][c], x[c], x[2 + c]);
                    const int row = i - (lane & 3);
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if (row + r < it.n)
                            *reinterpret_cast<uint4*>(p.out + (((int64_t)it.row0 + row + r) * p.H + it.h) * kValue + channel + 8 * (lane & 3)) = x[r];
                }
                if (p.lse != nullptr && i < it.n && half == 0 && (side == 0 || !part.joined)) p.lse[at] = lse_of(ref, l);
                if (part.joined) meet();  // both outputs have been read
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(o_free + 8 * side);
            }
            __syncwarp();
            if (lane == 0) {
                const int tiles = part_of(read_item(sm.item[count & 1]), 0).tiles;
                place[0] = place[0] + (kKeyUnits + kValueUnits) * tiles;
                place[1] = place[1] + tiles;
                tc::mbar_arrive(item_empty + 8 * (count & 1));
            }
            __syncwarp();
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == kMmaWarp) tc::tmem_dealloc(tmem, 512);
}

}  // namespace

// A CTA for every block that the requests may have: rows in blocks of their own, a last one each that is not full.
cudaError_t launch_latent_expanded(const ExpandedAttnParams& p, cudaStream_t s) {
    constexpr int smem = (int)sizeof(ExpandedSmem);
    static_assert(smem <= 227 * 1024, "shared memory of a CTA");
    static std::once_flag once[64];
    static cudaError_t err[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || dev < 0 || dev >= 64) return e != cudaSuccess ? e : cudaErrorInvalidDevice;
    std::call_once(once[dev], [dev] {
        err[dev] = cudaFuncSetAttribute(gdn_latent_expanded_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    });
    if (err[dev] != cudaSuccess) return err[dev];
    const int64_t blocks = std::min<int64_t>((int64_t)p.T / kBlock + p.B, p.T);
    return launch_dependent(gdn_latent_expanded_kernel, dim3((unsigned)(blocks * p.H)), kThreads, smem, s, p);
}

}  // namespace gdn
