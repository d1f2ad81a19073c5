// Attention over a paged KV cache (sm_100a): the row kernel.
//
//   out_i = sum_j p_ij v_j / sum_j p_ij,  p_ij = exp(s_ij - m_i),  m_i = max_j s_ij
// over the keys j that query i sees, in one pass over the keys with a running
// maximum: when m grows, the sums so far are scaled by exp(m_old - m_new).
#include "paged.cuh"

namespace arops {
namespace {

constexpr int kCounterBytes = 16384;
constexpr float kLog2e = 1.4426950408889634f;

// One warp a (token, head); lanes over head_dim, keys one after another.
template <typename T>
__global__ void __launch_bounds__(128)
attention_simple_kernel(const __grid_constant__ AttentionParams p)
{
    pdl_wait();
    pdl_allow_dependents();
    constexpr int R = 16;  // head_dim <= 512
    const int lane = threadIdx.x & 31;
    const int d = p.head_dim, g = p.hq / p.hk, ps = p.map.page_size;
    const T* q = static_cast<const T*>(p.q);
    T* out = static_cast<T*>(p.out);
    const int64_t units = p.tokens * p.hq;
    for (int64_t u = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5); u < units;
         u += (int64_t)gridDim.x * 4) {
        const int64_t t = u / p.hq;
        const int h = (int)(u % p.hq);
        const int kvh = h / g;
        bool bad = false;
        int s, grp = 0;
        int32_t prefix = 0, bidir = 0, i, len;
        if (p.group_start) {
            s = (int)t;
            grp = find_sequence(p.group_start, p.n_groups, t, lane);
            if (grp < 0)
                continue;
            prefix = clamp_length(__ldg(p.prefix_lens + grp), p.max_prefix_pages * ps, bad);
            len = prefix + clamp_length(__ldg(p.kv_lens + s), p.max_pages * ps, bad);
            i = len - 1;
        } else {
            s = find_sequence(p.q_start, p.n_seqs, t, lane);
            if (s < 0)
                continue;
            len = clamp_length(__ldg(p.kv_lens + s), p.max_pages * ps, bad);
            i = (int32_t)(len - (__ldg(p.q_start + s + 1) - t));
            bidir = p.bidir_lens ? __ldg(p.bidir_lens + s) : 0;
        }
        int32_t lo, hi;
        visible_keys(i, len, bidir, p.window, lo, hi);
        float qr[R], o[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int e = lane + 32 * r;
            qr[r] = e < d ? load_elem(q + t * p.q_stride + (int64_t)h * d + e) : 0.f;
            o[r] = 0.f;
        }
        const float slope = p.slopes ? __ldg(p.slopes + h) : 0.f;
        float m = -INFINITY, l = 0.f;
        for (int32_t j = lo; j < hi; ++j) {
            const bool in_prefix = j < prefix;
            int32_t pi, slot;
            split_position(p.map, in_prefix ? j : j - prefix, pi, slot);
            const int64_t page = in_prefix
                ? __ldg(p.prefix_table + (int64_t)grp * p.max_prefix_pages + pi)
                : __ldg(p.block_table + (int64_t)s * p.max_pages + pi);
            const bool ok = page >= 0 && page < p.map.num_pages;
            bad |= !ok;
            const int64_t off = ok ? ((page * p.hk + kvh) * ps + slot) * (int64_t)d : 0;
            const T* kp = static_cast<const T*>(p.k_pages) + off;
            const T* vp = static_cast<const T*>(p.v_pages) + off;
            float x = 0.f;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const int e = lane + 32 * r;
                if (e < d && ok)
                    x += qr[r] * load_elem(kp + e);
            }
#pragma unroll
            for (int w = 16; w > 0; w >>= 1)
                x += __shfl_xor_sync(0xFFFFFFFFu, x, w);
            x *= p.scale;
            if (p.softcap > 0.f)
                x = p.softcap * tanhf(x / p.softcap);
            x -= slope * fabsf((float)(i - j));
            const float mn = fmaxf(m, x);
            const float f = m == -INFINITY ? 0.f : expf(m - mn);
            const float w = mn == -INFINITY ? 0.f : expf(x - mn);
            l = l * f + w;
            m = mn;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const int e = lane + 32 * r;
                if (e < d)
                    o[r] = o[r] * f + (ok ? w * load_elem(vp + e) : 0.f);
            }
        }
        if (bad && lane == 0)
            record_device_error(p.err, kDeviceErrBadIndexBit);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int e = lane + 32 * r;
            if (e < d)
                store_elem(out + (t * p.hq + h) * (int64_t)d + e, l > 0.f ? o[r] / l : 0.f);
        }
    }
}

}  // namespace

size_t attention_counter_bytes()
{
    return kCounterBytes;
}

size_t attention_workspace_bytes(int64_t, int, int)
{
    return kCounterBytes;
}

cudaError_t launch_attention(const AttentionParams& p, arops_dtype dtype, void*,
                             cudaStream_t stream)
{
    const int64_t grid = std::min<int64_t>(ceil_div(p.tokens * p.hq, 4), 148 * 16);
    if (dtype == AROPS_BF16)
        return launch(attention_simple_kernel<__nv_bfloat16>, dim3((unsigned)grid), dim3(128), 0,
                      stream, p);
    return launch(attention_simple_kernel<float>, dim3((unsigned)grid), dim3(128), 0, stream, p);
}

}  // namespace arops
