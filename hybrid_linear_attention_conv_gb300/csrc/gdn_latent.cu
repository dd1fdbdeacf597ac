// gdn_latent.cu -- latent attention: one latent vector of 512 and one rotated
// key part of 64 a token, for all heads.  The host side of its entry points
// (validation and launches), the append of a step's rows to the paged cache,
// and the attention's two forms.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "gdn_kv_tc.cuh"
#include "gdn_latent.cuh"
#include "gdn_rotary.cuh"
#include "gdn_tc.cuh"

namespace gdn {
namespace {

__device__ __forceinline__ void unpack8(uint4 w, float (&v)[8]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(u[i] << 16);
        v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = tc::pack_bf16(__float2bfloat16_rn(v[2 * i]), __float2bfloat16_rn(v[2 * i + 1]));
    return make_uint4(u[0], u[1], u[2], u[3]);
}

// ---------------------------------------------------------------------------
// append
//
// A warp has a row: two chunks of eight latent channels a lane, whose sum of
// squares it reduces, and the key part's eight chunks in its first lanes; lane i
// makes the cosine and sine of pair i.  Bound by the chain slot -> row -> reduction ->
// store, of which 9,421 tokens of 37 prompts have enough under way for 3.9 TB/s (5.5 us); 64 single tokens take 2.1 us.
// ---------------------------------------------------------------------------
constexpr int kAppendThreads = 128;

__global__ void __launch_bounds__(kAppendThreads) gdn_latent_append_kernel(const __grid_constant__ LatentAppendParams p) {
    const int lane = threadIdx.x & 31, t = blockIdx.x * (kAppendThreads / 32) + (threadIdx.x >> 5);
    tc::grid_wait();
    if (t >= p.T) return;  // uniform in the warp
    const int64_t slot = p.slots[t];
    const int src = p.rows != nullptr ? p.rows[t] : t;
    if (slot < 0 || slot >= p.capacity) return;
    uint4* dst = reinterpret_cast<uint4*>(p.cache + slot * kLatentRow);
    if (src < 0 || src >= p.n_src) {  // no such row
        const uint4 nan = make_uint4(0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu);
        dst[lane] = dst[lane + 32] = nan;
        if (lane < 8) dst[lane + 64] = nan;
        return;
    }
    const uint4* x = reinterpret_cast<const uint4*>(p.x + src * p.ldx);
    const uint4 a = x[lane], b = x[lane + 32], r = lane < 8 ? x[lane + 64] : make_uint4(0, 0, 0, 0);
    const float2 mine = rotary_pair(p.turns[lane], p.positions[src], p.factor);
    float v[2][8];
    unpack8(a, v[0]);
    unpack8(b, v[1]);
    if (p.norm != nullptr) {
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) sum = fmaf(v[i >> 3][i & 7], v[i >> 3][i & 7], sum);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) sum += __shfl_xor_sync(~0u, sum, o);
        const float inv = 1.0f / sqrtf(fmaf(sum, 1.0f / kLatent, p.eps));
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const float4* w = reinterpret_cast<const float4*>(p.norm) + 2 * (lane + 32 * c);
            const float4 w0 = w[0], w1 = w[1];
            v[c][0] *= inv * w0.x, v[c][1] *= inv * w0.y, v[c][2] *= inv * w0.z, v[c][3] *= inv * w0.w;
            v[c][4] *= inv * w1.x, v[c][5] *= inv * w1.y, v[c][6] *= inv * w1.z, v[c][7] *= inv * w1.w;
        }
    }
    dst[lane] = p.norm != nullptr ? pack8(v[0]) : a;
    dst[lane + 32] = p.norm != nullptr ? pack8(v[1]) : b;
    float k[8], o[8];
    unpack8(r, k);
    if (p.interleaved) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float c = __shfl_sync(~0u, mine.x, (4 * lane + e) & 31), s = __shfl_sync(~0u, mine.y, (4 * lane + e) & 31);
            o[2 * e] = k[2 * e] * c - k[2 * e + 1] * s;
            o[2 * e + 1] = k[2 * e + 1] * c + k[2 * e] * s;
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float u = __shfl_xor_sync(~0u, k[e], 4);
            const float c = __shfl_sync(~0u, mine.x, (8 * lane + e) & 31), s = __shfl_sync(~0u, mine.y, (8 * lane + e) & 31);
            o[e] = k[e] * c + (lane & 4 ? u : -u) * s;
        }
    }
    if (lane < 8) dst[lane + 64] = pack8(o);
}

int check_latent_shape(const gdn_latent_shape* s) {
    if (s == nullptr) return report_error(GDN_ERR_INVALID_ARG, "shape is NULL");
    if (s->B < 0 || s->pages < 0 || s->width < 0 || s->H < 1)
        return report_error(GDN_ERR_UNSUPPORTED_SHAPE, "B=%d pages=%d width=%d H=%d: no negative counts, one head or more", s->B, s->pages, s->width, s->H);
    if (s->H > 1024) return report_error(GDN_ERR_UNSUPPORTED_SHAPE, "H=%d above 1024", s->H);
    if (s->page != 32 && s->page != 64 && s->page != 128)
        return report_error(GDN_ERR_UNSUPPORTED_SHAPE, "page=%d tokens not in {32, 64, 128}", s->page);
    if ((int64_t)s->pages * s->page > 0x7fffff00LL)
        return report_error(GDN_ERR_UNSUPPORTED_SHAPE, "the cache has %lld rows, at most 2^31 - 256 are supported", (long long)s->pages * s->page);
    return GDN_OK;
}

// A bf16 view [n, H, d]: strides in elements, multiples of 8, of any order (0 repeats a row or a head).
int check_strides(int64_t row, int64_t head, int64_t n, int H, const char* name) {
    if ((n > 1 && row < 0) || (H > 1 && head < 0)) return report_error(GDN_ERR_INVALID_ARG, "%s: negative stride", name);
    if ((n > 1 && row % 8 != 0) || (H > 1 && head % 8 != 0))
        return report_error(GDN_ERR_MISALIGNED, "%s: strides %lld, %lld are not multiples of 8 elements (16 bytes)", name, (long long)row, (long long)head);
    if ((n > 1 ? (double)n * row : 0.0) + (H > 1 ? (double)H * head : 0.0) > 0x1p60)
        return report_error(GDN_ERR_INVALID_ARG, "%s: strides %lld, %lld are too large", name, (long long)row, (long long)head);
    return GDN_OK;
}

// The cache's rows as nine groups of 64 channels, loaded in boxes of `groups` groups with the 128-byte swizzle.
bool encode_rows_map(CUtensorMap* map, const gdn_bf16* cache, const gdn_latent_shape* s, int groups) {
    const PFN_cuTensorMapEncodeTiled_v12000 enc = tmap_encoder();
    if (enc == nullptr) return false;
    const cuuint64_t dims[3] = {64, (cuuint64_t)s->pages * s->page, kLatentRow / 64};
    const cuuint64_t strides[2] = {(cuuint64_t)kLatentRow * 2, 128};
    const cuuint32_t box[3] = {64, (cuuint32_t)std::min(s->page, 64), (cuuint32_t)groups}, unit[3] = {1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<gdn_bf16*>(cache), dims, strides, box, unit,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A view [rows, H, d] in boxes of one head's 64 channels x 128 rows.
bool encode_heads_map(CUtensorMap* map, const gdn_bf16* x, int rows, int H, int d, int64_t row, int64_t head) {
    const PFN_cuTensorMapEncodeTiled_v12000 enc = tmap_encoder();
    if (enc == nullptr) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)H, (cuuint64_t)rows};
    const cuuint64_t strides[2] = {H > 1 ? (cuuint64_t)head * 2 : 256, rows > 1 ? (cuuint64_t)row * 2 : 256};
    const cuuint32_t box[3] = {64, 1, 128}, unit[3] = {1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<gdn_bf16*>(x), dims, strides, box, unit, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Its strides as a tensor map takes them: positive, below 2^40 bytes.
int check_map_strides(int64_t row, int64_t head, int64_t n, int H, const char* name) {
    if ((n > 1 && (row < 8 || row >= 1ll << 39)) || (H > 1 && (head < 8 || head >= 1ll << 39)))
        return report_error(GDN_ERR_UNSUPPORTED_SHAPE, "%s: strides %lld, %lld are not in 8 .. 2^39 - 1", name, (long long)row, (long long)head);
    return GDN_OK;
}

int check_scale(float scale) {
    if (!(scale > 0.0f) || scale > 1e6f) return report_error(GDN_ERR_INVALID_ARG, "scale=%g outside (0, 1e6]", (double)scale);
    return GDN_OK;
}

}  // namespace
}  // namespace gdn

using namespace gdn;

extern "C" {

int gdn_latent_append(const gdn_latent_shape* shape, int32_t T, const gdn_bf16* x, int64_t ldx, int32_t n_src, const int32_t* positions,
                      const int64_t* slots, const int32_t* rows, const uint64_t* turns, float factor, const float* norm, float eps,
                      gdn_bf16* cache, uint32_t flags, void* stream) {
    int rc;
    if ((rc = check_latent_shape(shape)) != GDN_OK) return rc;
    if (flags & ~(uint32_t)GDN_ROTARY_INTERLEAVED) return report_error(GDN_ERR_INVALID_ARG, "unknown flags 0x%x", flags);
    if (T < 0 || n_src < 0) return report_error(GDN_ERR_INVALID_ARG, "negative size T=%d n_src=%d", T, n_src);
    if (T > kKvMaxCount) return report_error(GDN_ERR_UNSUPPORTED_SHAPE, "T=%d above %lld", T, (long long)kKvMaxCount);
    if (n_src > 1 && ldx < kLatentRow) return report_error(GDN_ERR_INVALID_ARG, "ldx=%lld below a row's %d elements", (long long)ldx, kLatentRow);
    if ((rc = check_strides(ldx, 0, n_src, 1, "x")) != GDN_OK) return rc;
    if (rows == nullptr && n_src < T) return report_error(GDN_ERR_INVALID_ARG, "x has %d rows, T=%d are to be appended", n_src, T);
    if (!std::isfinite(factor)) return report_error(GDN_ERR_INVALID_ARG, "factor=%g is not finite", (double)factor);
    if (!(eps >= 0.0f && eps <= 1.0f)) return report_error(GDN_ERR_INVALID_ARG, "eps=%g outside [0, 1]", (double)eps);
    if (T == 0 || shape->pages == 0) return GDN_OK;  // nothing to do; pointers may be NULL
    if ((n_src > 0 && ((rc = check_pointer(x, "x")) || (rc = check_pointer(positions, "positions")))) || (rc = check_pointer(slots, "slots")) ||
        (rc = check_pointer(turns, "turns")) || (rc = check_pointer(cache, "cache")) || (rows != nullptr && (rc = check_pointer(rows, "rows"))) ||
        (norm != nullptr && (rc = check_pointer(norm, "norm"))))
        return rc;
    LatentAppendParams p{};
    p.x = x;
    p.positions = positions;
    p.slots = slots;
    p.rows = rows;
    p.turns = turns;
    p.norm = norm;
    p.cache = cache;
    p.ldx = n_src > 1 ? ldx : 0;
    p.capacity = (int64_t)shape->pages * shape->page;
    p.factor = factor;
    p.eps = eps;
    p.T = T;
    p.n_src = n_src;
    p.interleaved = (flags & GDN_ROTARY_INTERLEAVED) != 0;
    constexpr int per = kAppendThreads / 32;
    const cudaError_t e = launch_dependent(gdn_latent_append_kernel, dim3((unsigned)((T + per - 1) / per)), kAppendThreads, 0,
                                           static_cast<cudaStream_t>(stream), p);
    return e == cudaSuccess ? GDN_OK : cuda_error(e, "latent append launch");
}

size_t gdn_latent_attention_workspace_bytes(void) { return kKvPartialsAt + latent_tiles_workspace(); }

int gdn_latent_attention(const gdn_latent_shape* shape, int32_t T, const gdn_bf16* q, int64_t q_row, int64_t q_head, const gdn_bf16* q_rope,
                         int64_t r_row, int64_t r_head, const gdn_bf16* cache, const int32_t* table, const int32_t* start,
                         const int32_t* lens, const int64_t* tree, float scale, gdn_bf16* out, float* lse, void* workspace,
                         size_t workspace_bytes, void* stream) {
    int rc;
    if ((rc = check_latent_shape(shape)) != GDN_OK) return rc;
    if (T < 0) return report_error(GDN_ERR_INVALID_ARG, "T=%d < 0", T);
    if ((int64_t)T * shape->H > kKvMaxCount || (int64_t)shape->width * shape->page > kKvMaxCount)
        return report_error(GDN_ERR_UNSUPPORTED_SHAPE, "T=%d times H=%d rows or width=%d pages exceed %lld rows or tokens", T, shape->H, shape->width,
                            (long long)kKvMaxCount);
    if ((rc = check_strides(q_row, q_head, T, shape->H, "q")) || (rc = check_strides(r_row, r_head, T, shape->H, "q_rope")) ||
        (rc = check_scale(scale)))
        return rc;
    if (T == 0 || shape->B == 0) return GDN_OK;  // nothing to do; pointers may be NULL
    if (shape->pages < 1 || shape->width < 1)
        return report_error(GDN_ERR_UNSUPPORTED_SHAPE, "pages=%d width=%d: there is no cache to read", shape->pages, shape->width);
    if ((rc = check_pointer(q, "q")) || (rc = check_pointer(q_rope, "q_rope")) || (rc = check_pointer(cache, "cache")) ||
        (rc = check_pointer(table, "table")) || (rc = check_pointer(start, "start")) || (rc = check_pointer(lens, "lens")) ||
        (rc = check_pointer(out, "out")) || (tree != nullptr && (rc = check_pointer(tree, "tree"))) || (lse != nullptr && (rc = check_pointer(lse, "lse"))))
        return rc;
    if (workspace == nullptr) return report_error(GDN_ERR_WORKSPACE, "workspace is NULL");
    if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
        return report_error(GDN_ERR_MISALIGNED, "workspace (%p) is not 256-byte aligned", workspace);
    const size_t need = gdn_latent_attention_workspace_bytes();
    if (workspace_bytes < need) return report_error(GDN_ERR_WORKSPACE, "workspace of %zu bytes, %zu needed", workspace_bytes, need);
    LatentAttnParams p{};
    p.q = q;
    p.q_rope = q_rope;
    p.cache = cache;
    p.table = table;
    p.start = start;
    p.lens = lens;
    p.tree = tree;
    p.out = out;
    p.lse = lse;
    p.q_row = T > 1 ? q_row : 0;
    p.q_head = shape->H > 1 ? q_head : 0;
    p.r_row = T > 1 ? r_row : 0;
    p.r_head = shape->H > 1 ? r_head : 0;
    p.T = T;
    p.B = shape->B;
    p.H = shape->H;
    p.width = shape->width;
    p.pages = shape->pages;
    p.log2_page = shape->page == 32 ? 5 : shape->page == 64 ? 6 : 7;
    p.scale_log2 = scale * 1.4426950408889634f;
    if (!encode_rows_map(&p.tm, cache, shape, 4) || !encode_rows_map(&p.tm_key, cache, shape, 1))
        return report_error(GDN_ERR_CUDA, "the driver refused the cache's tensor maps");
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    cudaError_t e = gave_up_word(&p.gave_up);
    if (e != cudaSuccess) return cuda_error(e, "looking up the attention's give-up word");
    p.status = reinterpret_cast<int*>(ws);
    p.spans = reinterpret_cast<int*>(ws + kKvSpansAt);
    p.span_rows = reinterpret_cast<int64_t*>(ws + kKvSpanRowsAt);
    p.partials = reinterpret_cast<float*>(ws + kKvPartialsAt);
    p.wait_ns = wait_limit_ns();
    e = launch_latent_tiles(p, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? GDN_OK : cuda_error(e, "latent attention launch");
}

int gdn_latent_attention_expanded(int32_t B, int32_t H, int32_t T, int32_t S, const gdn_bf16* q, int64_t q_row, int64_t q_head,
                                  const gdn_bf16* k, int64_t k_row, int64_t k_head, const gdn_bf16* k_rope, int64_t r_row, const gdn_bf16* v,
                                  int64_t v_row, int64_t v_head, const int32_t* start, const int32_t* key_start, float scale, gdn_bf16* out,
                                  float* lse, void* stream) {
    int rc;
    if (B < 0 || T < 0 || S < 0) return report_error(GDN_ERR_INVALID_ARG, "negative size B=%d T=%d S=%d", B, T, S);
    if (H < 1 || H > 1024) return report_error(GDN_ERR_UNSUPPORTED_SHAPE, "H=%d not in 1 .. 1024", H);
    if ((int64_t)T * H > kKvMaxCount || S > kKvMaxCount)
        return report_error(GDN_ERR_UNSUPPORTED_SHAPE, "T=%d times H=%d rows or S=%d keys exceed %lld", T, H, S, (long long)kKvMaxCount);
    if ((rc = check_strides(q_row, q_head, T, H, "q")) || (rc = check_strides(k_row, k_head, S, H, "k")) ||
        (rc = check_strides(r_row, 0, S, 1, "k_rope")) || (rc = check_strides(v_row, v_head, S, H, "v")) || (rc = check_scale(scale)))
        return rc;
    if (((int64_t)T / 256 + B) * H > 0x7fffffff) return report_error(GDN_ERR_UNSUPPORTED_SHAPE, "T=%d B=%d H=%d: more blocks than a grid has", T, B, H);
    if (T == 0 || B == 0) return GDN_OK;  // nothing to do; pointers may be NULL
    if ((rc = check_map_strides(q_row, q_head, T, H, "q")) || (rc = check_map_strides(k_row, k_head, S, H, "k")) ||
        (rc = check_map_strides(r_row, 0, S, 1, "k_rope")) || (rc = check_map_strides(v_row, v_head, S, H, "v")))
        return rc;
    if ((rc = check_pointer(q, "q")) || (rc = check_pointer(start, "start")) || (rc = check_pointer(key_start, "key_start")) ||
        (rc = check_pointer(out, "out")) || (lse != nullptr && (rc = check_pointer(lse, "lse"))))
        return rc;
    if (S > 0 && ((rc = check_pointer(k, "k")) || (rc = check_pointer(k_rope, "k_rope")) || (rc = check_pointer(v, "v")))) return rc;
    ExpandedAttnParams p{};
    // without keys nothing is read of them: any memory serves their maps
    const bool none = S == 0;
    if (!encode_heads_map(&p.tm_q, q, T, H, kNope + kKeyPart, q_row, q_head) ||
        !encode_heads_map(&p.tm_k, none ? q : k, none ? 1 : S, none ? 1 : H, kNope, k_row, k_head) ||
        !encode_heads_map(&p.tm_r, none ? q : k_rope, none ? 1 : S, 1, kKeyPart, r_row, 0) ||
        !encode_heads_map(&p.tm_v, none ? q : v, none ? 1 : S, none ? 1 : H, kValue, v_row, v_head))
        return report_error(GDN_ERR_CUDA, "the driver refused the tensor maps of q, k and v");
    cudaError_t e = gave_up_word(&p.gave_up);
    if (e != cudaSuccess) return cuda_error(e, "looking up the attention's give-up word");
    p.start = start;
    p.key_start = key_start;
    p.out = out;
    p.lse = lse;
    p.wait_ns = wait_limit_ns();
    p.T = T;
    p.S = S;
    p.B = B;
    p.H = H;
    p.scale_log2 = scale * 1.4426950408889634f;
    e = launch_latent_expanded(p, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? GDN_OK : cuda_error(e, "expanded attention launch");
}

}  // extern "C"
