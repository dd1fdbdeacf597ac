// gdn_kv.cu -- the paged 8-bit key/value cache of the decoder's attention
// layers: the host side of its entry points (validation and launches), the
// plan kernel (pages, slots and row offsets from the requests' lengths) and
// the append kernel (a step's k and v rows into e4m3 codes and scales).
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <mutex>

#include "gdn_kv.cuh"
#include "gdn_kv_tc.cuh"
#include "gdn_tc.cuh"

namespace gdn {
namespace {

// ---------------------------------------------------------------------------
// plan
//
// start = exclusive prefix of the new tokens, off = exclusive prefix of the
// pages wanted, over the requests; every table entry and slot then follows
// from two binary searches.  Each CTA computes both prefixes for itself (two
// reads of 12 bytes a request, out of the L2 but for the first) and writes its
// share of the outputs, so nothing waits on another CTA.  A slot takes its page from
// the table's old entries or straight from the free stack, never from the
// entries this launch writes.
// Bound by latency, a chain of five dependent reads: in a graph 2.9 us for 64
// requests of one token, 5.6 us for 1,500 requests and 45,000 tokens.
// ---------------------------------------------------------------------------
constexpr int kPlanThreads = 512;
constexpr int kPlanMaxB = 12288;  // 2 x 4 bytes a request of shared memory

__device__ __forceinline__ long long warp_scan_ll(long long v) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long u = __shfl_up_sync(~0u, v, o);
        if ((threadIdx.x & 31) >= o) v += u;
    }
    return v;
}

// Largest i in [0, n) with a[i] <= x, for ascending a with a[0] <= x.
__device__ __forceinline__ int find_last(const int32_t* a, int n, int x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a[mid] <= x) lo = mid;
        else hi = mid;
    }
    return lo;
}

__global__ void __launch_bounds__(kPlanThreads) gdn_kv_plan_kernel(KvPlanParams p) {
    extern __shared__ int32_t plan_smem[];
    int32_t* start = plan_smem;       // [B]
    int32_t* off = plan_smem + p.B;   // [B]
    __shared__ long long sums[2][kPlanThreads / 32];
    __shared__ int bad;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int P = 1 << p.log2_page;
    if (tid == 0) bad = 0;
    tc::grid_wait();
    __syncthreads();

    const int per = (p.B + kPlanThreads - 1) / kPlanThreads;
    const int b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
    long long rows = 0, need = 0;
    int wrong = 0;
    for (int b = b0; b < b1; ++b) {
        const int len = p.lens[b], add = p.add[b], held = p.held[b];
        if (len < 0 || add < 0 || held < 0 || held > p.width) {
            wrong |= 8;
            continue;
        }
        const long long want = ((long long)len + add + P - 1) >> p.log2_page;
        if (want > p.width) wrong |= 2;
        rows += add;
        need += want > held ? want - held : 0;
    }
    const long long in_rows = warp_scan_ll(rows), in_need = warp_scan_ll(need);
    if (lane == 31) {
        sums[0][warp] = in_rows;
        sums[1][warp] = in_need;
    }
    if (wrong) atomicOr(&bad, wrong);
    __syncthreads();
    long long before_rows = in_rows - rows, before_need = in_need - need, all_rows = 0, all_need = 0;
#pragma unroll
    for (int w = 0; w < kPlanThreads / 32; ++w) {
        if (w < warp) {
            before_rows += sums[0][w];
            before_need += sums[1][w];
        }
        all_rows += sums[0][w];
        all_need += sums[1][w];
    }
    const int count = p.free_count[0];
    int status = bad;
    if (count < 0 || count > p.free_cap) status |= 8;
    if (all_need > count) status |= 1;
    if (all_rows > p.rows) status |= 4;
    const bool ok = status == 0;

    for (int b = b0; b < b1; ++b) {  // ok: every prefix fits 32 bits
        const int len = p.lens[b], add = p.add[b], held = p.held[b];
        int want = held;
        if (ok) {
            start[b] = (int)before_rows;
            off[b] = (int)before_need;
            want = max(held, (int)(((long long)len + add + P - 1) >> p.log2_page));
        }
        if (blockIdx.x == 0) {
            p.start[b] = ok ? (int)before_rows : 0;
            p.lens_out[b] = ok ? len + add : len;
            p.held_out[b] = want;
        }
        before_rows += add;
        before_need += want - held;
    }
    if (blockIdx.x == 0 && tid == 0) {
        p.start[p.B] = ok ? (int)all_rows : 0;
        p.free_count_out[0] = ok ? count - (int)all_need : count;
        p.status[0] = status;
    }
    __syncthreads();

    const int n_rows = ok ? (int)all_rows : 0, n_need = ok ? (int)all_need : 0;
    const int first = blockIdx.x * kPlanThreads + tid, stride = gridDim.x * kPlanThreads;
    for (int i = first; i < n_need; i += stride) {
        const int b = find_last(off, p.B, i);
        p.table[(int64_t)b * p.width + p.held[b] + (i - off[b])] = p.free_pages[count - 1 - i];
    }
    for (int r = first; r < p.rows; r += stride) {
        int64_t slot = -1;
        if (r < n_rows) {
            const int b = find_last(start, p.B, r);
            const int pos = p.lens[b] + r - start[b], j = pos >> p.log2_page, held = p.held[b];
            const int page = j < held ? p.table[(int64_t)b * p.width + j] : p.free_pages[count - 1 - off[b] - (j - held)];
            slot = ((int64_t)page << p.log2_page) + (pos & (P - 1));
        }
        p.slots[r] = slot;
    }
}

// ---------------------------------------------------------------------------
// append
//
// A run is a stretch of rows with consecutive slots in one page.  Its block
// (page, head) gets the scale 2^e: e the smallest with amax <= 448 * 2^e over
// the run's finite values, or the block's old exponent where that is larger
// and the page holds earlier tokens.  Scaling by a power of two is exact, so a
// code is the e4m3 number nearest to the value, whatever else is in the block;
// where the scale grows, the earlier rows' codes move by the same power, which
// only rounds what falls below e4m3's smallest normal number.  (A scale of
// amax / 448 would round every code twice, and re-round every code at each
// growth; the power of two costs at most one bit of e4m3's 18 binades.)
//
// The work is one pass over bf16 rows (2 bytes in, 1 out), bound by memory
// for prompts and by latency for single tokens.  A CTA looks at `tile` rows of
// one head of k or v, finds the runs that begin there with a ballot, lets a
// warp take each short run, and takes the long ones as a whole, a thread
// holding its part of the run in registers between the maximum and the
// conversion.
// Measured in a graph, 4 heads of 256: 64 single tokens 4.5 us; 8,192 rows
// 10.0 us = 4.9 TB/s (a CTA's life is load, maximum, barrier, conversion, store, and
// there are 1.7 CTAs for each that is resident: two waves, the second not full; the
// conversion keeps the integer pipe 55 % busy).  37 chunks of up to 2,000 rows, 8 heads
// of 128: 23.5 us = 3.4 TB/s, with pages begun and ended inside the chunks.
// ---------------------------------------------------------------------------
constexpr int kAppendThreads = 256;
constexpr int kAppendWarps = kAppendThreads / 32;
constexpr int kAppendShort = 4;  // rows that one warp takes

// The larger magnitudes of two bf16 pairs (m's not negative); NaN stays.
__device__ __forceinline__ uint32_t max_abs2(uint32_t m, uint32_t w) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(m), "r"(w & 0x7fff7fffu));
    return r;
}

// 8 bf16 (packed) times f to 8 e4m3 codes; values that are not finite give 0.
__device__ __forceinline__ uint2 codes8(uint4 x, float f, bool finite) {
    uint32_t w[4] = {x.x, x.y, x.z, x.w};
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float a = __uint_as_float(w[i] << 16), b = __uint_as_float(w[i] & 0xffff0000u);
        if (!finite) {
            a = isfinite(a) ? a : 0.0f;
            b = isfinite(b) ? b : 0.0f;
        }
        c[i] = e4m3x2(a * f, b * f);
    }
    return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

// The largest magnitudes of two bf16 pairs among m and 8 bf16.
__device__ __forceinline__ uint32_t max_abs8(uint32_t m, uint4 x) { return max_abs2(max_abs2(max_abs2(max_abs2(m, x.x), x.y), x.z), x.w); }

// The largest finite |x| of 8 bf16, as bits, where some are not finite.
__device__ __forceinline__ uint32_t max_finite8(uint32_t m, uint4 x) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t a = w[i] & 0x7fffu, b = (w[i] >> 16) & 0x7fffu;
        if (a < 0x7f80u) m = max(m, a);
        if (b < 0x7f80u) m = max(m, b);
    }
    return m;
}

// 16 codes times 2^-k (k > 0), to nearest even.
__device__ __forceinline__ uint32_t shrink4(uint32_t w, float f) {
    const float2 a = float2_of_e4m3x2(w & 0xffffu), b = float2_of_e4m3x2(w >> 16);
    return e4m3x2(a.x * f, a.y * f) | (e4m3x2(b.x * f, b.y * f) << 16);
}

// The run of n rows from row t, by `threads` threads of which this is `who`,
// each holding up to CH chunks of 8 values; Max reduces a maximum over them.
template <int CH, class Max>
__device__ __forceinline__ void append_run(const KvAppendParams& p, int t, int n, int64_t slot, int head, bool is_v, int who,
                                           int threads, Max&& reduce_max) {
    const uint16_t* src = (is_v ? p.v : p.k) + (int64_t)head * p.d;
    const int64_t ld = is_v ? p.ldv : p.ldk;
    const int per_row = p.d >> 3, shift = p.d == 256 ? 5 : 4;
    const int64_t page = slot >> p.log2_page;
    const int at = (int)(slot & ((1 << p.log2_page) - 1));
    float* scale = (is_v ? p.v_scale : p.k_scale) + page * p.Hkv + head;
    uint8_t* block = (is_v ? p.v_cache : p.k_cache) + ((page * p.Hkv + head) << p.log2_page) * p.d;
    // read before the maximum's barrier, replaced after it
    const float old = at > 0 ? __uint_as_float(scale_before(__float_as_uint(*scale), at)) : 0.0f;
    // chunk who + i * threads: row r0 + i * step of the run, always the same columns
    const int r0 = who >> shift, step = threads >> shift;
    const uint16_t* col = src + (who & (per_row - 1)) * 8;
    uint4 x[CH];
    uint32_t m2 = 0;
    if (p.rows == nullptr) {
        const uint16_t* from = col + (int64_t)(t + r0) * ld;
        const int64_t stride = (int64_t)step * ld;
#pragma unroll
        for (int i = 0; i < CH; ++i) x[i] = r0 + i * step < n ? *reinterpret_cast<const uint4*>(from + i * stride) : make_uint4(0, 0, 0, 0);
    } else {
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            x[i] = make_uint4(0, 0, 0, 0);
            if (r0 + i * step < n) {
                const int row = p.rows[t + r0 + i * step];
                if (row < 0 || row >= p.n_src) x[i] = make_uint4(~0u, ~0u, ~0u, ~0u);  // a source row that is not there is not finite
                else x[i] = *reinterpret_cast<const uint4*>(col + (int64_t)row * ld);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < CH; ++i) m2 = max_abs8(m2, x[i]);
    uint32_t top = reduce_max(max(m2 & 0xffffu, m2 >> 16));
    const bool finite = top < 0x7f80u;
    if (!finite) {
        uint32_t f = 0;
#pragma unroll
        for (int i = 0; i < CH; ++i) f = max_finite8(f, x[i]);
        top = reduce_max(f);
    }
    const float fresh = exp2_int(scale_exp_of_bf16(top));
    const bool poisoned = at > 0 && !(old > 0.0f && old < INFINITY);  // earlier rows that are not numbers stay so
    const float now = poisoned ? fresh : fmaxf(old, fresh);
    // the scales that this kernel writes are powers of two; one that is not
    // (the caller's own) divides once, and its codes are re-rounded on growth
    const float inv = 1.0f / now;
    if (at > 0 && !poisoned && now > old) {
        const float f = old * inv;
        for (int c = who; c < (at * p.d) >> 4; c += threads) {
            uint4* q = reinterpret_cast<uint4*>(block) + c;
            const uint4 w = *q;
            *q = make_uint4(shrink4(w.x, f), shrink4(w.y, f), shrink4(w.z, f), shrink4(w.w, f));
        }
    }
    uint2* to = reinterpret_cast<uint2*>(block + (int64_t)at * p.d) + who;
#pragma unroll
    for (int i = 0; i < CH; ++i)
        if (r0 + i * step < n) to[i * threads] = codes8(x[i], inv, finite);
    uint32_t bits = poisoned ? kLostScale : __float_as_uint(now);
    if (!finite) {
        uint32_t left = 0;  // rows from the first that is not finite on, for the maximum
#pragma unroll 1
        for (int r = r0; r < n && left == 0; r += step) {  // read again: rare, and the registers were full
            const int row = p.rows == nullptr ? t + r : p.rows[t + r];
            const uint32_t m = row < 0 || row >= p.n_src ? ~0u : max_abs8(0, *reinterpret_cast<const uint4*>(col + (int64_t)row * ld));
            if (max(m & 0x7fffu, m >> 16 & 0x7fffu) >= 0x7f80u) left = n - r;
        }
        bits = marked_scale(bits, at + n - (int)reduce_max(left));
    }
    if (who == 0 && !(poisoned && old != old)) *scale = __uint_as_float(bits);  // (a NaN stays the one that it is)
}

template <int CH>
__global__ void __launch_bounds__(kAppendThreads, CH > 8 ? 2 : 4) gdn_kv_append_kernel(KvAppendParams p) {
    __shared__ uint32_t warp_max[2][kAppendWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int head = blockIdx.y, t0 = blockIdx.x * p.tile, P = 1 << p.log2_page;
    const bool is_v = blockIdx.z != 0;
    const int64_t last_slot = (int64_t)p.pages << p.log2_page;
    tc::grid_wait();

    // Rows t0 .. t0 + tile - 1: a row begins a run unless it follows the row
    // before it inside a page.  A run ends within P rows of its first, so the
    // slots of tile + P rows, read at once, a word of 32 to a warp, tell all.
    __shared__ uint32_t goes_on[kAppendWarps], begins[kAppendWarps];  // bit l of word k: row t0 + 32 k + l
    {
        const int t = t0 + tid;
        const int64_t slot = t < p.T && tid < p.tile + P ? p.slots[t] : -1;
        int64_t prev = __shfl_up_sync(~0u, slot, 1);
        if (lane == 0) prev = t > 0 && t < p.T ? p.slots[t - 1] : -2;
        const bool valid = slot >= 0 && slot < last_slot;
        const bool follows = valid && prev == slot - 1 && (slot & (P - 1)) != 0;
        const uint32_t goes = __ballot_sync(~0u, follows), first = __ballot_sync(~0u, valid && !follows && tid < p.tile);
        if (lane == 0) {
            goes_on[warp] = goes;
            begins[warp] = first;
        }
    }
    __syncthreads();
    int phase = 0, nth = 0;
    uint32_t left = begins[0];
    for (int word = 0;;) {  // uniform in the CTA
        if (left == 0) {
            if (32 * ++word >= p.tile) break;
            left = begins[word];
            continue;
        }
        const int l = __ffs(left) - 1;
        left &= left - 1;
        int n = 1, k = word, from = l + 1;  // rows that go on from the next one
        while (true) {
            if (from == 32) {
                from = 0;
                if (++k == kAppendWarps) break;
            }
            const uint32_t ends = ~goes_on[k] >> from;
            const int run = ends ? min(__ffs(ends) - 1, 32 - from) : 32 - from;
            n += run;
            if (run < 32 - from) break;
            from = 32;
        }
        const int t_run = t0 + 32 * word + l;
        const int64_t s0 = p.slots[t_run];
        if (n <= kAppendShort) {
            if (nth++ % kAppendWarps == warp)
                append_run<kAppendShort>(p, t_run, n, s0, head, is_v, lane, 32,
                                         [](uint32_t m) { return __reduce_max_sync(~0u, m); });
        } else {
            append_run<CH>(p, t_run, n, s0, head, is_v, tid, kAppendThreads, [&](uint32_t m) {
                m = __reduce_max_sync(~0u, m);
                if (lane == 0) warp_max[phase][warp] = m;
                __syncthreads();
                uint32_t r = 0;
#pragma unroll
                for (int w = 0; w < kAppendWarps; ++w) r = max(r, warp_max[phase][w]);
                phase ^= 1;  // the next use writes the other half; the one after it lies behind a barrier
                return r;
            });
        }
    }
}

// ---------------------------------------------------------------------------
// validation
// ---------------------------------------------------------------------------
int check_kv_shape(const gdn_kv_shape* s) {
    if (s == nullptr) return report_error(GDN_ERR_INVALID_ARG, "shape is NULL");
    if (s->B < 0 || s->Hq < 1 || s->Hkv < 1 || s->pages < 0 || s->width < 0)
        return report_error(GDN_ERR_UNSUPPORTED_SHAPE, "bad sizes: B=%d Hq=%d Hkv=%d pages=%d width=%d", s->B, s->Hq,
                            s->Hkv, s->pages, s->width);
    if (s->Hq % s->Hkv != 0)
        return report_error(GDN_ERR_UNSUPPORTED_SHAPE, "Hq=%d is not a multiple of Hkv=%d", s->Hq, s->Hkv);
    if (s->Hq > 1024) return report_error(GDN_ERR_UNSUPPORTED_SHAPE, "Hq=%d above 1024", s->Hq);
    if (s->d != 128 && s->d != 256)
        return report_error(GDN_ERR_UNSUPPORTED_SHAPE, "head size d=%d not in {128, 256}", s->d);
    if (s->page != 32 && s->page != 64 && s->page != 128)
        return report_error(GDN_ERR_UNSUPPORTED_SHAPE, "page=%d tokens not in {32, 64, 128}", s->page);
    if ((int64_t)s->pages * s->Hkv * s->page > 0x7fffff00LL)
        return report_error(GDN_ERR_UNSUPPORTED_SHAPE, "the cache has %lld rows, at most 2^31 - 256 are supported",
                            (long long)s->pages * s->Hkv * s->page);
    return GDN_OK;
}

int log2_of(int page) { return page == 32 ? 5 : page == 64 ? 6 : 7; }

int check_row_stride(int64_t ld, int64_t row, const char* name) {
    if (ld < row) return report_error(GDN_ERR_INVALID_ARG, "%s=%lld below a row's %lld elements", name, (long long)ld, (long long)row);
    if (ld % 8 != 0) return report_error(GDN_ERR_MISALIGNED, "%s=%lld is not a multiple of 8 elements (16 bytes)", name, (long long)ld);
    return GDN_OK;
}

// Rows a CTA looks at.  Few rows are mostly single tokens, a warp each; the CTA
// of a long run takes it as a whole, and one begins in about every P rows.  Which of
// the two many rows are the host does not know.  Measured (us, eight rows a CTA and P), 4
// heads of 256, pages of 128: 4,000 rows of long runs 17.9, 6.5, of single tokens 53.2,
// 50.3; 1,025 rows 7.9, 4.9 and 16.5, 45.2: a decode batch just above 1,024 pays for
// the prompts of its size.  Pages of 32: 1,025 rows 5.1, 3.4 and 11.4, 14.1.
int append_tile_rows(int T, int P) { return T <= 1024 ? kAppendWarps : P; }

// cuTensorMapEncodeTiled from the driver, looked up once.
PFN_cuTensorMapEncodeTiled_v12000 tmap_encoder() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
        (void)cudaGetLastError();
    });
    return fn;
}

// The device's give-up word, which every attention call on it reports to.
__device__ int g_kv_gave_up = 0;

cudaError_t gave_up_word(int** word) {  // its address on the current device, looked up once
    static std::once_flag once[64];
    static cudaError_t err[64];
    static void* at[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || dev < 0 || dev >= 64) return e != cudaSuccess ? e : cudaErrorInvalidDevice;
    std::call_once(once[dev], [dev] { err[dev] = cudaGetSymbolAddress(&at[dev], g_kv_gave_up); });
    *word = static_cast<int*>(at[dev]);
    return err[dev];
}

// A cache as rows of d codes, loaded in boxes of `rows` rows x 128 bytes with the
// 128-byte swizzle (16-byte chunk c of row r lies at c ^ (r & 7)).
bool encode_cache_map(CUtensorMap* map, const uint8_t* cache, const gdn_kv_shape* s, int rows) {
    const PFN_cuTensorMapEncodeTiled_v12000 enc = tmap_encoder();
    if (enc == nullptr) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)s->d, (cuuint64_t)s->pages * s->Hkv * s->page};
    const cuuint64_t strides[1] = {(cuuint64_t)s->d};
    const cuuint32_t box[2] = {128, (cuuint32_t)rows}, unit[2] = {1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(cache), dims, strides, box, unit,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Which attention kernel: eight rows (queries x heads of a group) at a time over
// tiles of 32 tokens, which reads a request's cache once for every eight of its
// rows, or 128 rows over tiles of 128.  Both sides' times, in tiles of the first
// (2.6 ns of the whole GPU for d = 256, 1.3 for 128): a tile of the second takes
// 5 of them (d = 256) or 6.5, an item's beginning and end 8 tiles of the first
// and 6 of the second, and a launch of the second 3 << 20 / d more where its
// items are fewer than the SMs (each is spread over several CTAs and joined),
// 1 << 20 / d where they are not.  All that the host knows of the lengths is the
// table's width: where that bound is loose, both sides grow, and more than
// eight rows a request go to the second.  Measured (rows, tiles, us): 64 requests of
// 8,000 tokens, 24/4 heads of 256, 6 rows 169, 217; 12 rows 321, 218; one of
// 8,000 tokens, 60 rows 25, 31; 252 rows 59, 33; a first prompt of 85 tokens 17, 27;
// 64/4 heads of 128, 64 requests of 8,000, 16 rows 173, 146; over 199 such pairs
// the rule loses 1.18x at most; eight rows a request as the border loses up to 2.7x.
// Those are steps of requests alike: the rule goes by their mean, and one kernel takes all.  63
// single tokens at 4,000 to 12,000 and 512 queries after 8,000, 24/4 heads of 256: 698, 287
// (each in its own 180 + 89); 250 single tokens at 16,000 and 250 queries after as many, 32/8
// heads of 128, which the mean leaves with the first: 1,497, 1,901 (1,254 + 79).
bool use_tiles(const gdn_kv_shape* s, int T) {
    const double L = (double)s->width * s->page, heads = (double)s->B * s->Hkv;
    const double rows = std::ceil((double)T * (s->Hq / s->Hkv) / s->B);
    const double items = heads * std::ceil(rows / 128);
    const double by_eight = heads * std::ceil(rows / 8) * (L / 32 + 8);
    const double by_tiles = items * (L / 128 + 6) * (s->d == 256 ? 5.0 : 6.5) + (double)((items < device_sm_count() ? 3 << 20 : 1 << 20) / s->d);
    return by_eight > by_tiles;
}

}  // namespace

cudaError_t launch_kv_plan(const KvPlanParams& p, cudaStream_t s) {
    static std::once_flag once[64];
    static cudaError_t err[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || dev < 0 || dev >= 64) return e != cudaSuccess ? e : cudaErrorInvalidDevice;
    std::call_once(once[dev], [dev] {
        err[dev] = cudaFuncSetAttribute(gdn_kv_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kPlanMaxB * 8);
    });
    if (err[dev] != cudaSuccess) return err[dev];
    // a CTA for every two rows of its threads, up to one per SM
    const int grid = std::max(1, std::min(device_sm_count(), (p.rows + 2 * kPlanThreads - 1) / (2 * kPlanThreads)));
    return launch_dependent(gdn_kv_plan_kernel, dim3((unsigned)grid), kPlanThreads, (size_t)p.B * 8, s, p);
}

cudaError_t launch_kv_append(const KvAppendParams& p0, cudaStream_t s) {
    KvAppendParams p = p0;
    p.tile = append_tile_rows(p.T, 1 << p.log2_page);
    const dim3 grid((unsigned)((p.T + p.tile - 1) / p.tile), (unsigned)p.Hkv, 2);
    const int chunks = ((1 << p.log2_page) * p.d) / (8 * kAppendThreads);  // a whole page's, for each thread
    switch (chunks) {
        case 2: return launch_dependent(gdn_kv_append_kernel<2>, grid, kAppendThreads, 0, s, p);
        case 4: return launch_dependent(gdn_kv_append_kernel<4>, grid, kAppendThreads, 0, s, p);
        case 8: return launch_dependent(gdn_kv_append_kernel<8>, grid, kAppendThreads, 0, s, p);
        default: return launch_dependent(gdn_kv_append_kernel<16>, grid, kAppendThreads, 0, s, p);
    }
}

}  // namespace gdn

using namespace gdn;

extern "C" {

int gdn_kv_plan(const gdn_kv_shape* shape, const int32_t* lens, const int32_t* add, const int32_t* held,
                const int32_t* free_pages, int32_t free_cap, const int32_t* free_count, int32_t* table, int32_t rows,
                int32_t* lens_out, int32_t* held_out, int32_t* free_count_out, int32_t* start, int64_t* slots,
                int32_t* status, void* stream) {
    int rc;
    if ((rc = check_kv_shape(shape)) != GDN_OK) return rc;
    if (shape->B > kPlanMaxB)
        return report_error(GDN_ERR_UNSUPPORTED_SHAPE, "B=%d requests, one plan takes at most %d", shape->B, kPlanMaxB);
    if ((int64_t)shape->width * shape->page > kKvMaxCount)
        return report_error(GDN_ERR_UNSUPPORTED_SHAPE, "width=%d pages of %d tokens exceed %lld tokens", shape->width, shape->page,
                            (long long)kKvMaxCount);
    if (rows > kKvMaxCount || free_cap > kKvMaxCount)
        return report_error(GDN_ERR_UNSUPPORTED_SHAPE, "rows=%d or free_cap=%d above %lld", rows, free_cap, (long long)kKvMaxCount);
    if (rows < 0 || free_cap < 0) return report_error(GDN_ERR_INVALID_ARG, "negative size rows=%d free_cap=%d", rows, free_cap);
    const bool some = shape->B > 0;
    if ((some && ((rc = check_pointer(lens, "lens")) || (rc = check_pointer(add, "add")) || (rc = check_pointer(held, "held")) ||
                  (rc = check_pointer(lens_out, "lens_out")) || (rc = check_pointer(held_out, "held_out")))) ||
        (some && shape->width > 0 && (rc = check_pointer(table, "table"))) ||
        (free_cap > 0 && (rc = check_pointer(free_pages, "free_pages"))) || (rc = check_pointer(free_count, "free_count")) ||
        (rc = check_pointer(free_count_out, "free_count_out")) || (rc = check_pointer(start, "start")) ||
        (rows > 0 && (rc = check_pointer(slots, "slots"))) || (rc = check_pointer(status, "status")))
        return rc;
    // every CTA reads all of these while others write the outputs
    const void* in[4] = {lens, add, held, free_count};
    const void* out[3] = {lens_out, held_out, free_count_out};
    for (const void* a : in)
        for (const void* b : out)
            if (a != nullptr && a == b) return report_error(GDN_ERR_INVALID_ARG, "an output is one of the inputs (they must be distinct buffers)");
    KvPlanParams p{};
    p.lens = lens;
    p.add = add;
    p.held = held;
    p.free_pages = free_pages;
    p.free_count = free_count;
    p.table = table;
    p.lens_out = lens_out;
    p.held_out = held_out;
    p.free_count_out = free_count_out;
    p.start = start;
    p.slots = slots;
    p.status = status;
    p.B = shape->B;
    p.width = shape->width;
    p.log2_page = log2_of(shape->page);
    p.free_cap = free_cap;
    p.rows = rows;
    cudaError_t e = launch_kv_plan(p, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? GDN_OK : cuda_error(e, "cache plan launch");
}

int gdn_kv_append(const gdn_kv_shape* shape, int32_t T, const gdn_bf16* k, int64_t ldk, const gdn_bf16* v, int64_t ldv,
                  int32_t n_src, const int64_t* slots, const int32_t* rows, uint8_t* k_cache, uint8_t* v_cache,
                  float* k_scale, float* v_scale, void* stream) {
    int rc;
    if ((rc = check_kv_shape(shape)) != GDN_OK) return rc;
    if (T < 0 || n_src < 0) return report_error(GDN_ERR_INVALID_ARG, "negative size T=%d n_src=%d", T, n_src);
    if (T > kKvMaxCount) return report_error(GDN_ERR_UNSUPPORTED_SHAPE, "T=%d above %lld", T, (long long)kKvMaxCount);
    if (shape->Hkv > 65535) return report_error(GDN_ERR_UNSUPPORTED_SHAPE, "Hkv=%d exceeds the grid limit 65535", shape->Hkv);
    const int64_t row = (int64_t)shape->Hkv * shape->d;
    if ((rc = check_row_stride(ldk, row, "ldk")) || (rc = check_row_stride(ldv, row, "ldv"))) return rc;
    if (rows == nullptr && n_src < T)
        return report_error(GDN_ERR_INVALID_ARG, "k and v have %d rows, T=%d are to be appended", n_src, T);
    if (T == 0 || shape->pages == 0) return GDN_OK;  // nothing to do; pointers may be NULL
    if ((rc = check_pointer(slots, "slots")) || (rc = check_pointer(k_cache, "k_cache")) ||
        (rc = check_pointer(v_cache, "v_cache")) || (rc = check_pointer(k_scale, "k_scale")) ||
        (rc = check_pointer(v_scale, "v_scale")))
        return rc;
    if (n_src > 0 && ((rc = check_pointer(k, "k")) || (rc = check_pointer(v, "v")))) return rc;
    if (rows != nullptr && (rc = check_pointer(rows, "rows")) != GDN_OK) return rc;
    KvAppendParams p{};
    p.k = k;
    p.v = v;
    p.slots = slots;
    p.rows = rows;
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.ldk = ldk;
    p.ldv = ldv;
    p.T = T;
    p.n_src = n_src;
    p.Hkv = shape->Hkv;
    p.d = shape->d;
    p.log2_page = log2_of(shape->page);
    p.pages = shape->pages;
    cudaError_t e = launch_kv_append(p, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? GDN_OK : cuda_error(e, "cache append launch");
}

size_t gdn_kv_attention_workspace_bytes(const gdn_kv_shape* shape) {
    if (check_kv_shape(shape) != GDN_OK) return 0;
    return kKvPartialsAt + std::max(kv_attn_rows_workspace(shape->d), kv_attn_tiles_workspace(shape->d));
}

int gdn_kv_attention(const gdn_kv_shape* shape, int32_t T, const gdn_bf16* q, int64_t ldq, const uint8_t* k_cache,
                     const uint8_t* v_cache, const float* k_scale, const float* v_scale, const int32_t* table,
                     const int32_t* start, const int32_t* lens, const int64_t* tree, float scale, gdn_bf16* out,
                     float* lse, void* workspace, size_t workspace_bytes, void* stream) {
    int rc;
    if ((rc = check_kv_shape(shape)) != GDN_OK) return rc;
    if (T < 0) return report_error(GDN_ERR_INVALID_ARG, "T=%d < 0", T);
    if ((int64_t)T * (shape->Hq / shape->Hkv) > kKvMaxCount || (int64_t)shape->width * shape->page > kKvMaxCount)
        return report_error(GDN_ERR_UNSUPPORTED_SHAPE, "T=%d rows or width=%d pages exceed %lld rows (of a group) or tokens", T, shape->width,
                            (long long)kKvMaxCount);
    if ((rc = check_row_stride(ldq, (int64_t)shape->Hq * shape->d, "ldq")) != GDN_OK) return rc;
    if (!(scale > 0.0f) || scale > 1e6f) return report_error(GDN_ERR_INVALID_ARG, "scale=%g outside (0, 1e6]", (double)scale);
    if (T == 0 || shape->B == 0) return GDN_OK;  // nothing to do; pointers may be NULL
    if (shape->pages < 1 || shape->width < 1)
        return report_error(GDN_ERR_UNSUPPORTED_SHAPE, "pages=%d width=%d: there is no cache to read", shape->pages, shape->width);
    if ((rc = check_pointer(q, "q")) || (rc = check_pointer(k_cache, "k_cache")) || (rc = check_pointer(v_cache, "v_cache")) ||
        (rc = check_pointer(k_scale, "k_scale")) || (rc = check_pointer(v_scale, "v_scale")) ||
        (rc = check_pointer(table, "table")) || (rc = check_pointer(start, "start")) || (rc = check_pointer(lens, "lens")) ||
        (rc = check_pointer(out, "out")))
        return rc;
    if (tree != nullptr && (rc = check_pointer(tree, "tree")) != GDN_OK) return rc;
    if (lse != nullptr && (rc = check_pointer(lse, "lse")) != GDN_OK) return rc;
    if (workspace == nullptr) return report_error(GDN_ERR_WORKSPACE, "workspace is NULL");
    if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
        return report_error(GDN_ERR_MISALIGNED, "workspace (%p) is not 256-byte aligned", workspace);
    const size_t need = gdn_kv_attention_workspace_bytes(shape);
    if (workspace_bytes < need)
        return report_error(GDN_ERR_WORKSPACE, "workspace of %zu bytes, %zu needed", workspace_bytes, need);
    KvAttnParams p{};
    const bool tiles = use_tiles(shape, T);
    const int box = tiles ? shape->page : 32;
    if (!encode_cache_map(&p.tm_k, k_cache, shape, box) || !encode_cache_map(&p.tm_v, v_cache, shape, box))
        return report_error(GDN_ERR_CUDA, "the driver refused the cache's tensor maps");
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    p.q = q;
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.table = table;
    p.start = start;
    p.lens = lens;
    p.tree = tree;
    p.out = out;
    p.lse = lse;
    cudaError_t e = gave_up_word(&p.gave_up);
    if (e != cudaSuccess) return cuda_error(e, "looking up the attention's give-up word");
    p.status = reinterpret_cast<int*>(ws);
    p.spans = reinterpret_cast<int*>(ws + kKvSpansAt);
    p.span_rows = reinterpret_cast<int64_t*>(ws + kKvSpanRowsAt);
    p.partials = reinterpret_cast<float*>(ws + kKvPartialsAt);
    p.wait_ns = wait_limit_ns();
    p.ldq = ldq;
    p.T = T;
    p.B = shape->B;
    p.Hq = shape->Hq;
    p.Hkv = shape->Hkv;
    p.G = shape->Hq / shape->Hkv;
    p.width = shape->width;
    p.pages = shape->pages;
    p.log2_page = log2_of(shape->page);
    p.scale_log2 = scale * 1.4426950408889634f;
    p.group_magic = ((1u << 22) + p.G - 1) / p.G;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    e = tiles ? launch_kv_attn_tiles(p, shape->d, st) : launch_kv_attn_rows(p, shape->d, st);
    return e == cudaSuccess ? GDN_OK : cuda_error(e, "cache attention launch");
}

int gdn_kv_attention_status(const void* workspace, void* stream, int32_t* status) {
    if (workspace == nullptr) return report_error(GDN_ERR_WORKSPACE, "workspace is NULL");
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    int32_t word = 0;
    cudaError_t e = cudaMemcpyAsync(&word, workspace, sizeof word, cudaMemcpyDeviceToHost, st);
    if (e == cudaSuccess) e = cudaStreamSynchronize(st);
    if (e != cudaSuccess) return cuda_error(e, "reading the attention's status word");
    if (status != nullptr) *status = word;
    if (word != 0) return report_error(GDN_ERR_TIMEOUT, "a bounded device wait of an attention call gave up (status %d)", word);
    return GDN_OK;
}

int gdn_kv_attention_device_status(void* stream, int32_t* status) {
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    int* word = nullptr;
    int32_t value = 0;
    cudaError_t e = gave_up_word(&word);
    if (e == cudaSuccess) e = cudaMemcpyAsync(&value, word, sizeof value, cudaMemcpyDeviceToHost, st);
    if (e == cudaSuccess) e = cudaStreamSynchronize(st);
    if (e == cudaSuccess && value != 0) e = cudaMemsetAsync(word, 0, sizeof value, st);
    if (e != cudaSuccess) return cuda_error(e, "reading the attention's give-up word");
    if (status != nullptr) *status = value;
    if (value != 0)
        return report_error(GDN_ERR_TIMEOUT, "a bounded device wait of an attention call gave up (status %d)", value);
    return GDN_OK;
}

}  // extern "C"
