// gdn_rotary.cu -- RMS norm of the heads of q and k (optional) and rotation of
// their first channels by the tokens' positions:
//   y = x / sqrt(mean x^2 + eps) * w,   (y_a, y_b) <- (y_a c - y_b s, y_b c + y_a s),
// c, s the cosine and sine of pos * frequency, for the pairs (i, i + rot / 2) or (2 i, 2 i + 1).
//
// A group of 2^n lanes has a head and walks over tokens, a lane eight channels, one load and one store
// of 16 bytes each (two in fp32): addresses step by constants, the norm's weights stay in registers.  A CTA's groups have
// heads of their own over the same tokens, whose cosines and sines it makes once, after its first loads have gone out.
// Pairs that lie rot / 2 apart meet through shuffles, after the norm.
//
// Each value is read once and written once.  8,192 tokens of 28 heads of 256, normed, the first 64 channels turned: 47.8 us,
// 4.9 TB/s, bound by the chain from a token's loads to its stores, of which 24 warps to an SM fill two issue slots of three
// (with a group's heads and tokens found anew for each, about 300 instructions instead of 90: 74 us).  In fp32 76.6 us,
// 6.1 TB/s, HBM.  3,001 tokens of 64 heads of 64, no norm: 7.4 us, 6.6 TB/s, HBM.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "gdn_internal.h"
#include "gdn_kv.cuh"
#include "gdn_kv_tc.cuh"
#include "gdn_rotary.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 256;
constexpr int kUnits = 2;       // tokens that a group of lanes has in flight
constexpr int kRounds = 8;      // of them in a CTA
constexpr int kTable = 2048;    // cosines and sines of a CTA's tokens
constexpr int kMaxHead = 256;
constexpr double kPairCost = 0.4;

struct RotaryParams {
    const void* x[2];           // q, k
    void* y[2];
    const float* norm[2];       // [d], or nullptr
    int64_t row[2], head[2], out_row[2], out_head[2];
    const int32_t* positions;   // [T]
    const uint64_t* turns;      // [rot / 2]
    float factor, eps, inv_d;
    int T, Hq, H;               // H: heads of q and k
    int touched[2];             // channels of a head of q and of k that are read and written
    int rot_chunks;             // of eight channels, the rotated ones
    int log2_lanes;             // lanes of a head
    int tokens, heads;          // of a CTA
    int step;                   // from a group's token to its next
    int interleaved;
};

template <class E>
struct Eight;  // eight channels as they lie in memory
template <>
struct Eight<__nv_bfloat16> {
    uint4 w;
    __device__ __forceinline__ void load(const void* x, int64_t at) { w = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(x) + at); }
    __device__ __forceinline__ void clear() { w = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(u[i] << 16);
            v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ void store(void* y, int64_t at, const float (&v)[8]) {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            u[i] = *reinterpret_cast<const uint32_t*>(&b);
        }
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(y) + at) = make_uint4(u[0], u[1], u[2], u[3]);
    }
};
template <>
struct Eight<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const void* x, int64_t at) {
        const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(x) + at);
        a = p[0];
        b = p[1];
    }
    __device__ __forceinline__ void clear() { a = b = make_float4(0.0f, 0.0f, 0.0f, 0.0f); }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    }
    static __device__ __forceinline__ void store(void* y, int64_t at, const float (&v)[8]) {
        float4* p = reinterpret_cast<float4*>(static_cast<float*>(y) + at);
        p[0] = make_float4(v[0], v[1], v[2], v[3]);
        p[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
};

template <class E>
__global__ void __launch_bounds__(kThreads, 3) gdn_rotary_kernel(const __grid_constant__ RotaryParams p) {
    __shared__ float4 table[kTable / 2];  // two pairs' cosines and sines
    const int lanes = 1 << p.log2_lanes, lane = threadIdx.x & (lanes - 1), group = threadIdx.x >> p.log2_lanes;
    const int t0 = blockIdx.x * p.tokens, nt = min(p.tokens, p.T - t0), half = p.rot_chunks * 4;
    const bool first = 2 * lane < p.rot_chunks, turned = lane < p.rot_chunks;
    int token = group / p.heads;
    const int h = blockIdx.y * p.heads + group % p.heads;
    const int which = h >= p.Hq;
    const bool have = h < p.H && token < p.step && 8 * lane < p.touched[which];
    const int hw = min(h, p.H - 1) - (which ? p.Hq : 0);
    const int64_t row = p.row[which], out_row = p.out_row[which];
    int64_t from = (t0 + token) * row + hw * p.head[which] + 8 * lane, to = (t0 + token) * out_row + hw * p.out_head[which] + 8 * lane;
    const void* x = p.x[which];
    void* y = p.y[which];
    const float* norm = p.norm[which];
    const bool any_norm = p.norm[0] != nullptr || p.norm[1] != nullptr;
    tc::grid_wait();
    float w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = 1.0f;
    if (norm != nullptr && have) {
        const float4 a = reinterpret_cast<const float4*>(norm)[2 * lane], b = reinterpret_cast<const float4*>(norm)[2 * lane + 1];
        w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
    }
    const int shift = p.rot_chunks >> 1, partner = first ? lane + shift : turned ? lane - shift : lane;
    // A token's table: the first two pairs of each lane that turns some, their next two, and so on, so that lanes read neighbours.
    const int log2_each = p.interleaved ? 1 : 2, apart = half >> (1 + log2_each);
    const int at = p.interleaved || first ? lane : turned ? lane - shift : 0;
    const float sign = first ? -1.0f : 1.0f;

    // Tokens beyond nt come to groups of a warp at different times: its lanes leave together.
    Eight<E> next[kUnits];
    auto request = [&](int token) {
#pragma unroll
        for (int i = 0; i < kUnits; ++i) {
            next[i].clear();
            if (have && token + i * p.step < nt) next[i].load(x, from + i * p.step * row);
        }
        from += kUnits * p.step * row;
    };
    request(token);
    for (int i = threadIdx.x; i < nt * half; i += kThreads) {
        const int t = i / half, pair = i - t * half, two = pair >> 1;
        reinterpret_cast<float2*>(table)[t * half + 2 * ((two & ((1 << log2_each) - 1)) * apart + (two >> log2_each)) + (pair & 1)] =
            rotary_pair(p.turns[pair], p.positions[t0 + t], p.factor);
    }
    __syncthreads();
    while (__any_sync(~0u, token < nt)) {
        Eight<E> raw[kUnits];
#pragma unroll
        for (int i = 0; i < kUnits; ++i) raw[i] = next[i];
        request(token + kUnits * p.step);
        // (no branch between the tokens in flight: their chains of shuffles run beside one another)
        float inv[kUnits];
        if (any_norm) {
            float sum[kUnits];
#pragma unroll
            for (int i = 0; i < kUnits; ++i) {
                float v[8];
                raw[i].get(v);
                float2 two = make_float2(0.0f, 0.0f);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 x2 = make_float2(v[2 * e], v[2 * e + 1]);
                    two = __ffma2_rn(x2, x2, two);
                }
                sum[i] = two.x + two.y;
            }
            for (int o = 1; o < lanes; o <<= 1)
#pragma unroll
                for (int i = 0; i < kUnits; ++i) sum[i] += __shfl_xor_sync(~0u, sum[i], o);
#pragma unroll
            for (int i = 0; i < kUnits; ++i) inv[i] = norm != nullptr ? rsqrtf(fmaf(sum[i], p.inv_d, p.eps)) : 1.0f;
        }
#pragma unroll
        for (int i = 0; i < kUnits; ++i) {
            const int t = token + i * p.step;
            float v[8];
            raw[i].get(v);
            if (any_norm) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 by = __fmul2_rn(make_float2(w[2 * e], w[2 * e + 1]), make_float2(inv[i], inv[i]));
                    const float2 x2 = __fmul2_rn(make_float2(v[2 * e], v[2 * e + 1]), by);
                    v[2 * e] = x2.x, v[2 * e + 1] = x2.y;
                }
            }
            const float4* pairs = table + min(t, nt - 1) * (half >> 1) + at;
            if (p.interleaved) {
                if (turned) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float4 cs = pairs[e * apart];
                        const float a = v[4 * e], b = v[4 * e + 1], c = v[4 * e + 2], d = v[4 * e + 3];
                        v[4 * e] = a * cs.x - b * cs.y;
                        v[4 * e + 1] = b * cs.x + a * cs.y;
                        v[4 * e + 2] = c * cs.z - d * cs.w;
                        v[4 * e + 3] = d * cs.z + c * cs.w;
                    }
                }
            } else {
                float u[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) u[e] = __shfl_sync(~0u, v[e], partner, lanes);
                if (turned) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float4 cs = pairs[e * apart];
                        const float2 a = __fmul2_rn(make_float2(u[2 * e], u[2 * e + 1]), make_float2(sign * cs.y, sign * cs.w));
                        const float2 x2 = __ffma2_rn(make_float2(v[2 * e], v[2 * e + 1]), make_float2(cs.x, cs.z), a);
                        v[2 * e] = x2.x, v[2 * e + 1] = x2.y;
                    }
                }
            }
            if (have && t < nt) Eight<E>::store(y, to + i * p.step * out_row, v);
        }
        token += kUnits * p.step;
        to += kUnits * p.step * out_row;
    }
}

// A strided view [T, H, d] as byte offsets from its address.
struct View {
    uintptr_t at;
    int64_t row, head, span, extent;  // strides, bytes of a row (first to last head), of the whole view
    View(const void* x, int64_t row_, int64_t head_, int T, int H, int d, int size) {
        at = reinterpret_cast<uintptr_t>(x);
        row = T > 1 ? row_ * size : 0;
        head = H > 1 ? head_ * size : 0;
        span = (H > 1 ? (H - 1) * head : 0) + (int64_t)d * size;
        extent = (T > 1 ? (T - 1) * row : 0) + span;
    }
};

// Whether two views of [T, H, d] that are not the same view share an element, as far as that can be told from
// common strides; where it cannot, views whose extents meet count as sharing one.
bool meet(const View& a, const View& b, int64_t chunk) {
    if (a.at + (uint64_t)a.extent <= b.at || b.at + (uint64_t)b.extent <= a.at) return false;
    auto apart = [](uintptr_t x, int64_t nx, uintptr_t y, int64_t ny, int64_t period) {
        if (period <= 0) return false;
        const int64_t d = (int64_t)((y - x) % (uint64_t)period);
        return y >= x ? d >= nx && d + ny <= period : false;
    };
    auto both = [&](int64_t na, int64_t nb, int64_t period) {
        return a.at <= b.at ? apart(a.at, na, b.at, nb, period) : apart(b.at, nb, a.at, na, period);
    };
    if (a.row == b.row && both(a.span, b.span, a.row)) return false;  // different columns of the same rows
    auto parts = [&](int64_t inner, int64_t outer) { return inner > 0 && outer % inner == 0 && both(chunk, chunk, inner); };
    if (a.row == b.row && a.head == b.head && (parts(a.head, a.row) || parts(a.row, a.head))) return false;  // different parts of wider heads
    return true;
}

int check_view(const void* x, int64_t row, int64_t head, int T, int H, int d, int size, bool written, const char* name) {
    int rc;
    if ((rc = check_pointer(x, name)) != GDN_OK) return rc;
    if ((T > 1 && row < 0) || (H > 1 && head < 0)) return report_error(GDN_ERR_INVALID_ARG, "%s: negative stride", name);
    if ((T > 1 && row * size % 16 != 0) || (H > 1 && head * size % 16 != 0))
        return report_error(GDN_ERR_MISALIGNED, "%s: strides %lld, %lld are not multiples of 16 bytes", name, (long long)row, (long long)head);
    if ((T > 1 ? (double)T * row : 0.0) + (H > 1 ? (double)H * head : 0.0) > 0x1p60)
        return report_error(GDN_ERR_INVALID_ARG, "%s: strides %lld, %lld are too large", name, (long long)row, (long long)head);
    if (!written) return GDN_OK;
    const int64_t r = T > 1 ? row : INT64_MAX, h = H > 1 ? head : INT64_MAX;
    const bool rows_apart = h >= d && (T == 1 || r >= (H - 1) * (H > 1 ? head : 0) + d);
    const bool heads_apart = r >= d && (H == 1 || h >= (T - 1) * (T > 1 ? row : 0) + d);
    if (!rows_apart && !heads_apart) return report_error(GDN_ERR_INVALID_ARG, "%s: strides %lld, %lld make rows overlap", name, (long long)row, (long long)head);
    return GDN_OK;
}

}  // namespace
}  // namespace gdn

using namespace gdn;

extern "C" {

int gdn_rotary_frequencies(int32_t rot, double base, int32_t scaling, double factor, int32_t context, double fast, double slow,
                           uint64_t* turns, float* values) {
    if (rot < 2 || rot > kMaxHead || rot % 2 != 0) return report_error(GDN_ERR_UNSUPPORTED_SHAPE, "rot=%d is not even and in 2 .. %d", rot, kMaxHead);
    if (!(base > 1.0) || !std::isfinite(base)) return report_error(GDN_ERR_INVALID_ARG, "base=%g is not above 1", base);
    if (scaling != GDN_ROTARY_PLAIN && scaling != GDN_ROTARY_LINEAR && scaling != GDN_ROTARY_PARTS)
        return report_error(GDN_ERR_INVALID_ARG, "scaling=%d unknown", scaling);
    if (scaling != GDN_ROTARY_PLAIN && (!(factor >= 1.0) || !std::isfinite(factor)))
        return report_error(GDN_ERR_INVALID_ARG, "factor=%g below 1", factor);
    if (scaling == GDN_ROTARY_PARTS && (context < 1 || !(slow > 0.0) || !(fast > slow) || !std::isfinite(fast)))
        return report_error(GDN_ERR_INVALID_ARG, "context=%d fast=%g slow=%g: a context of 1 or more, fast > slow > 0", context, fast, slow);
    if (turns == nullptr) return report_error(GDN_ERR_INVALID_ARG, "turns is NULL");
    constexpr double kTurn = 6.283185307179586476925286766559;
    double lo = 0.0, hi = 0.0;
    if (scaling == GDN_ROTARY_PARTS) {
        auto at = [&](double n) { return rot * std::log(context / (n * kTurn)) / (2.0 * std::log(base)); };
        lo = std::max(std::floor(at(fast)), 0.0);
        hi = std::min(std::ceil(at(slow)), rot - 1.0);
    }
    for (int i = 0; i < rot / 2; ++i) {
        double f = std::pow(base, -2.0 * i / rot);
        if (scaling == GDN_ROTARY_LINEAR) f /= factor;
        if (scaling == GDN_ROTARY_PARTS) {
            const double keep = 1.0 - std::min(std::max((i - lo) / std::max(hi - lo, 0.001), 0.0), 1.0);
            f = f * keep + f / factor * (1.0 - keep);
        }
        turns[i] = (uint64_t)(f / kTurn * 18446744073709551616.0);  // f <= 1: below 2^62
    }
    if (values != nullptr) *values = scaling == GDN_ROTARY_PARTS ? (float)(0.1 * std::log(factor) + 1.0) : 1.0f;
    return GDN_OK;
}

int gdn_rotary(const gdn_rotary_shape* s, const void* q, int64_t q_row, int64_t q_head, const void* k, int64_t k_row, int64_t k_head,
               void* q_out, int64_t q_out_row, int64_t q_out_head, void* k_out, int64_t k_out_row, int64_t k_out_head,
               const int32_t* positions, const uint64_t* turns, float factor, const float* q_norm, const float* k_norm, float eps,
               uint32_t flags, void* stream) {
    int rc;
    if (s == nullptr) return report_error(GDN_ERR_INVALID_ARG, "shape is NULL");
    if (flags & ~(uint32_t)(GDN_IN_F32 | GDN_ROTARY_INTERLEAVED)) return report_error(GDN_ERR_INVALID_ARG, "unknown flags 0x%x", flags);
    if (s->T < 0) return report_error(GDN_ERR_INVALID_ARG, "T=%d < 0", s->T);
    if (s->Hq < 0 || s->Hk < 0 || s->Hq + (int64_t)s->Hk < 1 || s->Hq > 65536 || s->Hk > 65536)
        return report_error(GDN_ERR_UNSUPPORTED_SHAPE, "Hq=%d Hk=%d heads: together one or more, 65536 each at most", s->Hq, s->Hk);
    if (s->d < 16 || s->d > kMaxHead || s->d % 8 != 0) return report_error(GDN_ERR_UNSUPPORTED_SHAPE, "d=%d is not a multiple of 8 in 16 .. %d", s->d, kMaxHead);
    if (s->rot < 16 || s->rot > s->d || s->rot % 16 != 0)
        return report_error(GDN_ERR_UNSUPPORTED_SHAPE, "rot=%d is not a multiple of 16 in 16 .. d=%d", s->rot, s->d);
    if (s->T > kKvMaxCount) return report_error(GDN_ERR_UNSUPPORTED_SHAPE, "T=%d above %lld", s->T, (long long)kKvMaxCount);
    if (!std::isfinite(factor)) return report_error(GDN_ERR_INVALID_ARG, "factor=%g is not finite", (double)factor);
    if (!(eps >= 0.0f && eps <= 1.0f)) return report_error(GDN_ERR_INVALID_ARG, "eps=%g outside [0, 1]", (double)eps);
    if (s->T == 0) return GDN_OK;  // nothing to do; pointers may be NULL
    const int size = flags & GDN_IN_F32 ? 4 : 2;
    const int H[2] = {s->Hq, s->Hk};
    const void* x[2] = {q, k};
    void* y[2] = {q_out, k_out};
    const int64_t row[2] = {q_row, k_row}, head[2] = {q_head, k_head}, out_row[2] = {q_out_row, k_out_row}, out_head[2] = {q_out_head, k_out_head};
    const float* norm[2] = {q_norm, k_norm};
    const char *xn[2] = {"q", "k"}, *yn[2] = {"q_out", "k_out"}, *nn[2] = {"q_norm", "k_norm"};
    int touched[2] = {0, 0};
    for (int i = 0; i < 2; ++i) {
        if (H[i] == 0) continue;
        if ((rc = check_view(x[i], row[i], head[i], s->T, H[i], s->d, size, false, xn[i])) ||
            (rc = check_view(y[i], out_row[i], out_head[i], s->T, H[i], s->d, size, true, yn[i])) ||
            (norm[i] != nullptr && (rc = check_pointer(norm[i], nn[i]))))
            return rc;
        const bool same = x[i] == y[i] && (s->T == 1 || row[i] == out_row[i]) && (H[i] == 1 || head[i] == out_head[i]);
        touched[i] = same && norm[i] == nullptr ? s->rot : s->d;
        const View out(y[i], out_row[i], out_head[i], s->T, H[i], s->d, size);
        for (int j = 0; j < 2; ++j) {
            if (H[j] == 0) continue;
            if (!(j == i && same) && meet(out, View(x[j], row[j], head[j], s->T, H[j], s->d, size), (int64_t)s->d * size))
                return report_error(GDN_ERR_INVALID_ARG, "%s overlaps %s without being it", yn[i], xn[j]);
            if (j > i && meet(out, View(y[j], out_row[j], out_head[j], s->T, H[j], s->d, size), (int64_t)s->d * size))
                return report_error(GDN_ERR_INVALID_ARG, "q_out overlaps k_out");
        }
    }
    if ((rc = check_pointer(positions, "positions")) || (rc = check_pointer(turns, "turns"))) return rc;
    RotaryParams p{};
    for (int i = 0; i < 2; ++i) {
        p.x[i] = x[i];
        p.y[i] = y[i];
        p.norm[i] = H[i] == 0 ? nullptr : norm[i];
        p.row[i] = s->T > 1 ? row[i] : 0;
        p.head[i] = H[i] > 1 ? head[i] : 0;
        p.out_row[i] = s->T > 1 ? out_row[i] : 0;
        p.out_head[i] = H[i] > 1 ? out_head[i] : 0;
        p.touched[i] = touched[i];
    }
    p.positions = positions;
    p.turns = turns;
    p.factor = factor;
    p.eps = eps;
    p.inv_d = 1.0f / s->d;
    p.T = s->T;
    p.Hq = s->Hq;
    p.H = s->Hq + s->Hk;
    p.rot_chunks = s->rot / 8;
    p.interleaved = (flags & GDN_ROTARY_INTERLEAVED) != 0;
    while (8 << p.log2_lanes < std::max(touched[0], touched[1])) ++p.log2_lanes;
    // A CTA's groups have a head each, or, where the heads are fewer, several tokens at a time; its tokens are what a group
    // has in flight eight times over, more for few heads, fewer while there are not four CTAs for every SM.
    const int groups = kThreads >> p.log2_lanes;
    // Heads of a CTA: few enough to leave no group without one, many enough to share the cosines and sines (a pair's cost
    // kPairCost of a lane's eight channels').  28 heads of 256: 4 (8,192 tokens 47 us; 7, and one group of eight idle, 51).
    double best = 1e30;
    for (int heads = 1; heads <= std::min(groups, p.H); ++heads) {
        const int blocks = (p.H + heads - 1) / heads;
        const double cost = (double)blocks * (groups + kPairCost * (s->rot / 2) * (groups / heads) / (1 << p.log2_lanes)) / (groups / heads);
        if (cost < best) best = cost, p.heads = heads;
    }
    const int blocks_y = (p.H + p.heads - 1) / p.heads;
    p.step = groups / p.heads;
    p.tokens = std::min(p.step * kUnits * kRounds, kTable / (s->rot / 2));
    const int64_t spread = ((int64_t)s->T * blocks_y + 4 * device_sm_count() - 1) / (4 * device_sm_count());
    p.tokens = (int)std::min<int64_t>(p.tokens, std::max<int64_t>(spread, 1));
    const dim3 grid((unsigned)((s->T + p.tokens - 1) / p.tokens), (unsigned)blocks_y);
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = size == 4 ? launch_dependent(gdn_rotary_kernel<float>, grid, kThreads, 0, st, p)
                                    : launch_dependent(gdn_rotary_kernel<__nv_bfloat16>, grid, kThreads, 0, st, p);
    return e == cudaSuccess ? GDN_OK : cuda_error(e, "rotary launch");
}

}  // extern "C"
