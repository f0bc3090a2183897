// kamera_paged.h -- what the kernels of decode attention over the paged pool
// share: the launch parameters, the layout of partial softmax states in the
// workspace, and the launchers.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "kamera.h"

namespace kamera {

// Partial states: row r = sequence * Hq + query head holds `slots` of them, the
// prefix's first, then the own tokens'.  Slot i of row r is an unnormalised
// output (d floats at o[(r * slots + i) * d]) and, at ml[r * slots + i], the
// running maximum in log2 units and the sum of weights.  A slot is written iff
// its share of the tokens is not empty, which the merge works out again from
// the lengths.
struct PagedParams {
    const __nv_bfloat16* q;         // [n_seqs][H * G][d]
    __nv_bfloat16* out;
    float* lse;                     // or null
    int32_t n_seqs, H, G, d, P;
    int64_t num_pages;
    float scale;
    // own tokens
    const int32_t* pages;           // [n_seqs][max_pages]
    const int32_t* lens;
    int32_t max_pages, max_len;
    const int32_t* selected;        // [n_seqs][H][n_select], or null: every page
    int32_t n_select;
    int32_t own_split, own_slots;   // 16-token pieces of a split; splits at most
    // shared prefixes
    const int32_t* group_start;
    const int32_t* prefix_pages;    // [n_groups][max_prefix_pages]
    const int32_t* prefix_lens;
    int32_t n_groups, max_prefix_pages, max_prefix, max_group;
    int32_t two_tile;               // prefix CTAs: up to two 128-row tiles (1) or one, its tokens in two halves (0)
    int32_t row_blocks;             // prefix CTAs of a (group, KV head, split)
    int32_t block_rows;             // rows of each
    int32_t prefix_split;           // 128-token tiles of a split
    int32_t prefix_splits;          // splits at most
    int32_t prefix_slots;           // prefix_splits * (two_tile ? 1 : 2)
    int32_t slots;                  // prefix_slots + own_slots
    float* o;
    float2* ml;
    int32_t* err;
    uint64_t wait_ns;
    int32_t withhold;               // test hook: no tile is loaded
};

struct PagedLaunch {
    PagedParams p;
    CUtensorMap map_k, map_v;       // prefix: groups of eight rows, boxes of box_rows rows of a head; own pages:
                                    // rows, boxes of 64 columns x 16 rows
    const __nv_bfloat16* v;         // the value rows themselves, slot_stride elements apart
    int64_t slot_stride;
    int32_t box_rows;
};

// Tokens of sequence s read by the call (0 when its length is out of range).
__device__ __forceinline__ int own_len(const PagedParams& p, int s)
{
    if (p.max_len == 0)
        return 0;
    const int len = p.lens[s];
    return len >= 0 && len <= p.max_len ? len : 0;
}

// Group g's sequences [s0, s1) and prefix length; false if malformed.
__device__ __forceinline__ bool group_range(const PagedParams& p, int g, int& s0, int& s1, int& len)
{
    s0 = p.group_start[g];
    s1 = p.group_start[g + 1];
    len = p.prefix_lens[g];
    if (len < 0 || len > p.max_prefix)
        len = 0;
    return s0 >= 0 && s1 >= s0 && s1 <= p.n_seqs && s1 - s0 <= p.max_group;
}

// Softmax weights as the tensor cores take them: hi + lo, two bf16 parts, about 16
// significant bits (lo is rounded by at most 2^-16 of the weight).  hi is the weight
// rounded towards zero, its upper half word; lo what is left and 2^-24 of hi.  Both are
// positive, so that an infinite value reaches the sum as it is; with hi rounded to
// nearest, lo has half the error but either sign or is zero, and an infinite value
// became NaN.
constexpr float kLessHi = -0.99999994f;   // -(1 - 2^-24): lo = weight + kLessHi hi

__device__ __forceinline__ uint32_t weight_hi(float a, float b)
{
    return __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
}

cudaError_t launch_prefix(const PagedLaunch& L, cudaStream_t stream);

// The own tokens' part alone, for a caller that joins their partial states with others:
// the argument checks and the plan (a KAMERA_* status; 0 splits: nothing to read), and
// the launch, with p's pointers filled in and its states in p.o, p.ml (row r's split i
// at r * own_slots + i, written where it has tokens).
int plan_own_pages(const KameraPagedKV* kv, const KameraPagedQuery* q, const KameraPageTable* own, PagedParams* p);
cudaError_t launch_own_pages(const PagedParams& p, const KameraPagedKV* kv, cudaStream_t stream);

}  // namespace kamera
