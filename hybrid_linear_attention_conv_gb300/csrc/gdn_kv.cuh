// gdn_kv.cuh -- what the paged 8-bit cache's kernels share: the launch
// parameters that gdn_kv.cu fills after validation, the power-of-two scales,
// and the split of a value into two 8-bit numbers.  Nothing here is part of
// the ABI.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "gdn_internal.h"

namespace gdn {

// The most rows, free pages and tokens of a table row that a call takes.  The
// kernels count them in 32 bits and step past the last: by a grid's stride
// (a thread to a row), by the tiles that they look ahead.
constexpr int64_t kKvMaxCount = 0x7ff00000;

// A block's scale is 2^e.  e4m3's largest number is 448 = 1.75 * 2^8.
constexpr int kScaleMinExp = -100, kScaleMaxExp = 120;

// Smallest e with amax <= 448 * 2^e, clamped, for the finite bf16 with these
// bits (sign cleared).  amax = m * 2^E: e = E - 8 while m <= 1.75.
__host__ __device__ inline int scale_exp_of_bf16(uint32_t bits) {
    const int E = (int)(bits >> 7) - 127;
    const int e = E - 8 + ((bits & 0x7f) > 0x60 ? 1 : 0);
    return e < kScaleMinExp ? kScaleMinExp : e > kScaleMaxExp ? kScaleMaxExp : e;
}

// A block with a row that is not finite has a NaN for its scale, whose payload
// keeps what its other rows need should that row be taken back (a rejected draft):
// the scale's biased exponent in bits 0 to 7 and the first such row in bits 8 to 14.
// A scale that is no power of two (the caller's own) leaves a NaN without.
constexpr uint32_t kLostScale = 0x7fffffffu, kMarkedScale = 0x7fc08000u;
__host__ __device__ inline uint32_t marked_scale(uint32_t scale_bits, int row) {
    const uint32_t e = scale_bits >> 23;
    return (scale_bits & 0x807fffffu) != 0 || e == 0 || e == 255 ? kLostScale : kMarkedScale | (uint32_t)row << 8 | e;
}
// The scale of the rows before row `at`, as bits: a marked block's where its first row
// that is not finite is none of them.
__host__ __device__ inline uint32_t scale_before(uint32_t scale_bits, int at) {
    const bool marked = (scale_bits & 0xffff8000u) == kMarkedScale;
    const uint32_t e = scale_bits & 0xff;
    return marked && e != 0 && e != 255 && (int)(scale_bits >> 8 & 0x7f) >= at ? e << 23 : scale_bits;
}

// Row coordinate of tokens [pos, pos + 32) of a sequence in the cache seen as
// rows of d codes: rows of a page's head are adjacent.  A page that the table
// does not have (outside the table's width or the cache) gives `rows`, one
// past the last row, which the copy engine fills with zeros.
__host__ __device__ inline int32_t cache_row(int32_t page, int32_t pages, int32_t Hkv, int32_t h, int32_t log2_page,
                                             int32_t pos) {
    if (page < 0 || page >= pages) return (int32_t)((int64_t)pages * Hkv << log2_page);
    return (int32_t)((((int64_t)page * Hkv + h) << log2_page) + (pos & ((1 << log2_page) - 1)));
}

// A worker's ring of copies: a copy's place and its barrier's phase, in turn.
// A barrier must not be armed while its phase still awaits bytes (that is a
// fault), so a slot is filled again only after its copy was waited for with
// success: the first wait that gives up ends the sending for good.  The copies
// then in flight, pending() from the slot at hand on, are waited for once more (with a
// limit of their own), and everything after runs through on what is there.
template <int kUnits>
struct CopyRing {
    int slot = 0;          // of the copy to be read next,
    uint32_t parity = 0;   // its phase,
    int send = 0;          // and the slot to be filled next
    bool gave_up = false;
    __host__ __device__ void sent() { send = send + 1 == kUnits ? 0 : send + 1; }
    __host__ __device__ void read() {
        if (++slot == kUnits) {
            slot = 0;
            parity ^= 1;
        }
    }
    // Copies sent and not read, when the one at hand is among them: 1 to kUnits.
    __host__ __device__ int pending() const { return send > slot ? send - slot : send - slot + kUnits; }
};

struct KvPlanParams {
    const int32_t* lens;        // [B] tokens cached
    const int32_t* add;         // [B] tokens to come
    const int32_t* held;        // [B] pages held
    const int32_t* free_pages;  // [free_cap] a stack: the next page is the last
    const int32_t* free_count;  // [1]
    int32_t* table;             // [B, width]
    int32_t* lens_out;
    int32_t* held_out;
    int32_t* free_count_out;
    int32_t* start;             // [B + 1]
    int64_t* slots;             // [rows]
    int32_t* status;            // [1]
    int B, width, log2_page, free_cap, rows;
};

struct KvAppendParams {
    const uint16_t* k;          // bf16 rows [n_src, Hkv, d], row stride ldk
    const uint16_t* v;
    const int64_t* slots;       // [T]
    const int32_t* rows;        // [T] source rows, or nullptr (row t)
    uint8_t* k_cache;           // [pages, Hkv, P, d]
    uint8_t* v_cache;
    float* k_scale;             // [pages, Hkv]
    float* v_scale;
    int64_t ldk, ldv;
    int T, n_src, Hkv, d, log2_page, pages;
    int tile;                   // rows that a CTA looks at for the beginnings of runs
};

struct KvAttnParams {
    CUtensorMap tm_k, tm_v;     // the caches as [pages * Hkv * P, d] bytes, in boxes of 128 bytes x 32 rows, or x a page
    const uint16_t* q;          // bf16 rows [T, Hq, d], row stride ldq
    const float* k_scale;       // [pages, Hkv]
    const float* v_scale;
    const int32_t* table;       // [B, width]
    const int32_t* start;       // [B + 1]
    const int32_t* lens;        // [B]
    const int64_t* tree;        // [T] or nullptr
    uint16_t* out;              // bf16 [T, Hq, d]
    float* lse;                 // [T, Hq] or nullptr
    int* gave_up;               // the device's word: calls without a workspace of the caller's
    int* status;                // workspace: the status word,
    int* spans;                 // how many CTAs further the item goes that begins in a CTA,
    int64_t* span_rows;         // its eight rows' places in out (-1: none), or {first row of q, queries, row tile, head},
    float* partials;            // and the partial results
    uint64_t wait_ns;
    int64_t ldq;
    int T, B, Hq, Hkv, G, width, pages, log2_page;
    float scale_log2;           // scale * log2(e)
    unsigned group_magic;       // ceil(2^22 / G)
};

// Workspace: 256 bytes of status, the spans and their rows, then the partial results.
constexpr int kKvMaxCtas = 1024;
constexpr size_t kKvSpansAt = 256;
constexpr size_t kKvSpanRowsAt = kKvSpansAt + (size_t)kKvMaxCtas * 4;
constexpr size_t kKvPartialsAt = kKvSpanRowsAt + (size_t)kKvMaxCtas * 8 * 8;

cudaError_t launch_kv_append(const KvAppendParams& p, cudaStream_t s);
cudaError_t launch_kv_plan(const KvPlanParams& p, cudaStream_t s);
// One to eight query rows of a key/value head at a time (mma.sync).
cudaError_t launch_kv_attn_rows(KvAttnParams& p, int d, cudaStream_t s);
size_t kv_attn_rows_workspace(int d);
// 128 query rows at a time (tcgen05).
cudaError_t launch_kv_attn_tiles(KvAttnParams& p, int d, cudaStream_t s);
size_t kv_attn_tiles_workspace(int d);

#ifdef __CUDACC__
// A bounded wait gave up.
__device__ __forceinline__ void report_give_up(const KvAttnParams& p, int bit) {
    atomicOr(p.status, bit);
    atomicOr(p.gave_up, bit);
}

// Every kernel of a step is launched as a programmatic dependent of the one
// before it on the stream: its blocks may be placed while that one drains, and
// touch no memory that it may write before tc::grid_wait().
template <class... Args>
cudaError_t launch_dependent(void (*kernel)(Args...), dim3 grid, int threads, size_t smem, cudaStream_t s, Args... args) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// 2^e for e in the normal range.
__device__ __forceinline__ float exp2_int(int e) { return __int_as_float((e + 127) << 23); }

// Two e4m3 codes (a in the low byte), to nearest even, saturating; NaN stays NaN.
__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
    return r;
}
// The two e4m3 codes in the low half of w, as f16 (exact).
__device__ __forceinline__ uint32_t f16x2_of_e4m3x2(uint32_t w) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)w));
    return r;
}
__device__ __forceinline__ float2 float2_of_e4m3x2(uint32_t w) {
    const uint32_t h = f16x2_of_e4m3x2(w);
    float2 r;
    asm("{\n\t.reg .f16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.f32.f16 %0, lo;\n\tcvt.f32.f16 %1, hi;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "r"(h));
    return r;
}

// Four bf16 values, |x| <= 448, as hi (e4m3) + lo (e5m2): hi = RNE(x), and
// x - hi is at most eight steps of x, which e5m2's three significant bits hold
// exactly while x is above 2^-6; below, hi + lo is within 2^-14 of x (half a step of lo
// next to half a step of hi, 2^-10).  So a bf16 value is held exactly while it is
// within 2^-14 of its row's largest.  The values go by way of f16 pairs, whose
// conversions are half the instructions: exact, but for 2^-25 of what is that small.
__device__ __forceinline__ uint32_t f16x2(float a, float b) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}
__device__ __forceinline__ uint32_t e4m3x2_of_f16x2(uint32_t w) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(w));
    return r;
}
__device__ __forceinline__ uint32_t sub_f16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t e5m2x2_of_f16x2(uint32_t w) {
    uint16_t r;
    asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(r) : "r"(w));
    return r;
}
__device__ __forceinline__ void split4_queries(float e0, float e1, float e2, float e3, uint32_t& hi, uint32_t& lo) {
    const uint32_t a = f16x2(e0, e1), b = f16x2(e2, e3);
    const uint32_t ha = e4m3x2_of_f16x2(a), hb = e4m3x2_of_f16x2(b);
    const uint32_t la = e5m2x2_of_f16x2(sub_f16x2(a, f16x2_of_e4m3x2(ha)));
    const uint32_t lb = e5m2x2_of_f16x2(sub_f16x2(b, f16x2_of_e4m3x2(hb)));
    hi = ha | (hb << 16);
    lo = la | (lb << 16);
}

// Four softmax weights of a block, 0 <= w <= 256 and the block's largest above 2^7, as
// e4m3 hi + 2^-5 lo: hi = RNE(w), within 2^3 of w, and lo = RNE(2^5 (w - hi)), 2^8 at
// most.  Within 2^-8 of w (and f16's 2^-12) while w is above 2^-6, and within
// 2^-15, which is 2^-22 of the block's largest, below.
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ void split4_weights(float e0, float e1, float e2, float e3, uint32_t& hi, uint32_t& lo) {
    constexpr uint32_t k32 = 0x50005000u;  // 2^5, twice
    const uint32_t a = f16x2(e0, e1), b = f16x2(e2, e3);
    const uint32_t ha = e4m3x2_of_f16x2(a), hb = e4m3x2_of_f16x2(b);
    const uint32_t la = e4m3x2_of_f16x2(mul_f16x2(sub_f16x2(a, f16x2_of_e4m3x2(ha)), k32));
    const uint32_t lb = e4m3x2_of_f16x2(mul_f16x2(sub_f16x2(b, f16x2_of_e4m3x2(hb)), k32));
    hi = ha | (hb << 16);
    lo = la | (lb << 16);
}

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
#endif

}  // namespace gdn
