// The paged KV cache as the kernels see it: where a token's sequence, a
// position's page and a query's visible keys are.  Shared by the paged append
// (paged_append.cu) and the attention kernels.
#pragma once

#include <limits.h>

#include "common.cuh"

namespace arops {

constexpr unsigned kDeviceErrBadIndexBit = AROPS_DEVICE_ERR_BAD_INDEX;

// Positions are mapped to pages by a shift where the page size is a power of
// two (page_shift >= 0), else by a 32-bit division.
struct PageMap {
    int64_t num_pages;
    int32_t page_size;
    int32_t page_shift;  // log2(page_size), or -1
};

inline PageMap make_page_map(const arops_paged_cache& c)
{
    PageMap m;
    m.num_pages = c.num_pages;
    m.page_size = c.page_size;
    m.page_shift = -1;
    for (int s = 0; s < 31; ++s)
        if (c.page_size == (1 << s))
            m.page_shift = s;
    return m;
}

__device__ __forceinline__ void split_position(const PageMap& m, int32_t p, int32_t& page,
                                               int32_t& slot)
{
    if (m.page_shift >= 0) {
        page = p >> m.page_shift;
        slot = p & (m.page_size - 1);
    } else {
        page = (int32_t)((uint32_t)p / (uint32_t)m.page_size);
        slot = p - page * m.page_size;
    }
}

// The sequence that token t belongs to: the last s with start[s] <= t, checked
// against start[s + 1]; -1 for a token of no sequence.  A search in 32 parts a
// round, one load a lane; the whole warp takes part with one t.  Whatever the
// array holds, only start[0 .. n] is read.
__device__ __forceinline__ int find_sequence(const int32_t* start, int n, int64_t t, int lane)
{
    int lo = 0, hi = n;  // the answer, if any, is in [lo, hi)
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32;
        const int at = lo + lane * step;
        const bool le = at < hi && (int64_t)__ldg(start + at) <= t;
        const unsigned mask = __ballot_sync(0xFFFFFFFFu, le);
        if (mask == 0)
            return -1;
        lo += (31 - __clz(mask)) * step;
        hi = min(hi, lo + step);
    }
    if (hi <= lo)
        return -1;
    const int64_t a = __ldg(start + lo), b = __ldg(start + lo + 1);
    return (a <= t && t < b) ? lo : -1;
}

// A length read from the device, brought into [0, capacity].
__device__ __forceinline__ int32_t clamp_length(int32_t len, int32_t capacity, bool& bad)
{
    if (len > capacity) {
        bad = true;
        return capacity;
    }
    return len > 0 ? len : 0;
}

// The keys that the query at position i sees are an interval [lo, hi): causal
// or among the first `bidir` positions, inside the window, below len.  Empty
// intervals come back with lo == hi.  i may be negative (more queries than
// positions).
__device__ __forceinline__ void visible_keys(int32_t i, int32_t len, int32_t bidir, int32_t window,
                                             int32_t& lo, int32_t& hi)
{
    lo = (window > 0 && i >= window) ? i - window + 1 : 0;
    hi = min(len, max(i < INT_MAX ? i + 1 : INT_MAX, bidir));
    hi = max(hi, lo);
}

// Arguments of the attention kernels (validated on the host).  With groups
// (group_start != nullptr) every sequence has one query token and its group's
// prefix before its own keys; otherwise q_start gives the tokens.
struct AttentionParams {
    const void* q;
    void* out;
    const void* k_pages;
    const void* v_pages;
    const int32_t* q_start;
    const int32_t* kv_lens;
    const int32_t* block_table;
    const int32_t* group_start;
    const int32_t* prefix_lens;
    const int32_t* prefix_table;
    const float* slopes;
    const int32_t* bidir_lens;
    unsigned* err;
    int64_t q_stride;
    int64_t tokens;
    PageMap map;
    int32_t n_seqs, max_pages;
    int32_t n_groups, max_prefix_pages;
    int32_t hq, hk, head_dim;
    int32_t window;
    float scale, softcap;
};

struct PagedAppendArgs {
    const void* q;
    const void* k;
    const void* v;
    void* q_out;
    void* k_pages;
    void* v_pages;
    int64_t q_stride, k_stride, v_stride, q_out_stride;
    const int32_t* q_start;
    const int32_t* kv_lens;
    const int32_t* block_table;
    const int32_t* pos;
    const void* gamma_q;
    const void* gamma_k;
    int64_t tokens;
    PageMap map;
    int32_t n_seqs, max_pages;
    int32_t hq, hk, head_dim;
    int32_t sections[3];
    float theta, eps;
};

cudaError_t launch_paged_append(const PagedAppendArgs& a, arops_dtype dtype, cudaStream_t stream);

// Attention (paged_attention.cu).  The workspace starts with
// attention_counter_bytes() of arrival counters, zero between calls; only shared
// prefixes have results of their own in it.
size_t attention_counter_bytes();
size_t attention_workspace_bytes(int64_t tokens, int hq, int head_dim, bool shared_prefix);
cudaError_t launch_attention(const AttentionParams& p, arops_dtype dtype, void* workspace,
                             cudaStream_t stream);

}  // namespace arops
