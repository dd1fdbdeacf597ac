// gdn_latent.cuh -- what the latent attention's kernels share: their launch
// parameters, which gdn_latent.cu fills after validation.  Nothing here is
// part of the ABI.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "gdn_internal.h"
#include "gdn_kv.cuh"

namespace gdn {

constexpr int kLatent = 512;                // channels of a token's latent vector: key and value of every head
constexpr int kKeyPart = 64;                // of its rotated key part, which the heads share
constexpr int kLatentRow = kLatent + kKeyPart;
constexpr int kNope = 128, kValue = 128;    // expanded form: a head's own key channels, its value

struct LatentAppendParams {
    const uint16_t* x;          // bf16 rows [n_src, 576], row stride ldx
    const int32_t* positions;   // [n_src]
    const int64_t* slots;       // [T]
    const int32_t* rows;        // [T] source rows, or nullptr (row t)
    const uint64_t* turns;      // [32]
    const float* norm;          // [512] or nullptr
    uint16_t* cache;            // [capacity, 576]
    int64_t ldx, capacity;
    float factor, eps;
    int T, n_src, interleaved;
};

struct LatentAttnParams {
    CUtensorMap tm, tm_key;     // the cache as [9 groups, rows, 64 channels], in boxes of four groups (one) of min(page, 64) rows
    const uint16_t* q;          // bf16 [T, H, 512]
    const uint16_t* q_rope;     // bf16 [T, H, 64]
    const uint16_t* cache;      // bf16 [pages, page, 576]
    const int32_t* table;       // [B, width]
    const int32_t* start;       // [B + 1]
    const int32_t* lens;        // [B]
    const int64_t* tree;        // [T] or nullptr
    uint16_t* out;              // bf16 [T, H, 512]
    float* lse;                 // [T, H] or nullptr
    int* gave_up;               // the device's word: calls without a workspace of the caller's
    int* status;                // workspace: the status word,
    int* spans;                 // how many shares further the item goes that begins in a CTA,
    int64_t* span_rows;         // the first of its rows in out, and how many,
    float* partials;            // and the partial results
    uint64_t wait_ns;
    int64_t q_row, q_head, r_row, r_head;
    int T, B, H, width, pages, log2_page;
    int ctas;                   // of the grid
    int pair;                   // CTAs that take row tiles of the same tokens: 1 to 2 of 64 rows, 4 of 32, 8 of 16
    float scale_log2;           // scale * log2(e)
};

struct ExpandedAttnParams {
    CUtensorMap tm_q;           // bf16 [T, H, 192], boxes of 128 rows x 64 channels
    CUtensorMap tm_k, tm_v;     // [S, H, 128]
    CUtensorMap tm_r;           // [S, 1, 64]
    const int32_t* start;       // [B + 1] rows of q
    const int32_t* key_start;   // [B + 1] rows of k
    uint16_t* out;              // bf16 [T, H, 128]
    float* lse;                 // [T, H] or nullptr
    int* gave_up;               // the device's word
    uint64_t wait_ns;
    int T, S, B, H;
    float scale_log2;
};

cudaError_t launch_latent_expanded(const ExpandedAttnParams& p, cudaStream_t s);
cudaError_t launch_latent_tiles(LatentAttnParams& p, cudaStream_t s);
size_t latent_tiles_workspace();

}  // namespace gdn
