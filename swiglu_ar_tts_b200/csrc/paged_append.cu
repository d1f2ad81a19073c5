// M-RoPE with the append to a paged KV cache (sm_100a): every token's q and k
// heads are normalised (optional), rotated and stored, k and v into the slot
// that the block table names for the token's position.
//
// For a head x of D values, pairs (x[j], x[j + D/2]), j < D/2:
//   x' = gamma * x / sqrt(sum(x^2)/D + eps)            (where a weight is given)
//   out[j] = x'[j] cos - x'[j + D/2] sin,  out[j + D/2] = x'[j + D/2] cos + x'[j] sin
// with the angle pos[row(j)] * theta^(-2j/D).  Everything is fp32 in registers,
// rounded once at the store.  The operator reads and writes (2 Hq + 4 Hk) D
// values a token and computes ~8 operations on each, so memory bounds it; a
// decode step is bound by latency: positions, lengths and the block table form
// a chain of three dependent loads, the activations' loads run beside it (5
// tokens: 3.3-3.5 us a launch back to back).  A ragged batch of 7,443 tokens, 122 MB,
// takes 27.1 us, 69% of the measured copy rate: 950 instructions a warp and half
// token (angles, norms, rotation) keep half of the issue slots busy, and an SM's
// sixteen warps do not cover the rest of each other's latencies; more warps of
// fewer registers, weights kept in registers, or the next token's data brought
// into L2 ahead measured the same or slower.
#include "paged.cuh"
#include "rope.cuh"

namespace arops {
namespace {

constexpr int kAppendWarps = 4;

// Cache slot of token t, found by the whole warp: the element offset of
// (page, head 0, slot) or -1, and whether the token belongs to a sequence.
struct TokenSlot {
    int64_t offset;
    bool owned;
};

__device__ __forceinline__ TokenSlot token_slot(const PagedAppendArgs& a, int64_t t, int lane,
                                                unsigned* err)
{
    // a decode step has one token a sequence: then s == t, and the search ends
    // before it starts
    int s = -1;
    if (t < a.n_seqs && __ldg(a.q_start + t) == t && __ldg(a.q_start + t + 1) == t + 1)
        s = (int)t;
    else
        s = find_sequence(a.q_start, a.n_seqs, t, lane);
    TokenSlot r;
    r.offset = -1;
    r.owned = s >= 0;
    if (s < 0)
        return r;
    const int64_t end = __ldg(a.q_start + s + 1);
    const int64_t p = (int64_t)__ldg(a.kv_lens + s) - (end - t);
    if (p >= 0 && p < (int64_t)a.max_pages * a.map.page_size) {
        int32_t pi, slot;
        split_position(a.map, (int32_t)p, pi, slot);
        const int64_t page = __ldg(a.block_table + (int64_t)s * a.max_pages + pi);
        if (page >= 0 && page < a.map.num_pages)
            r.offset = (page * a.hk * a.map.page_size + slot) * a.head_dim;
    }
    if (r.offset < 0 && a.hk > 0 && lane == 0)
        record_device_error(err, kDeviceErrBadIndexBit);
    return r;
}

// A 16-byte vector as pairs of floats, and back.
template <typename T>
__device__ __forceinline__ void unpack2(const uint4& v, float2* f)
{
    float x[Vec<T>::N];
    Vec<T>::unpack(v, x);
#pragma unroll
    for (int i = 0; i < Vec<T>::N / 2; ++i)
        f[i] = make_float2(x[2 * i], x[2 * i + 1]);
}

template <typename T>
__device__ __forceinline__ uint4 pack2(const float2* f)
{
    float x[Vec<T>::N];
#pragma unroll
    for (int i = 0; i < Vec<T>::N / 2; ++i) {
        x[2 * i] = f[i].x;
        x[2 * i + 1] = f[i].y;
    }
    return Vec<T>::pack(x);
}

// 16-byte vectors: lane pv of a head's P lanes owns one vector of the first
// half and its partner of the second; a warp takes G = 32/P heads a pass and U
// passes at once (mrope.cu's layout, whose angles it shares).  A head's sum of
// squares is a shuffle over its P lanes.
template <typename T, int P, int U>
__global__ void __launch_bounds__(32 * kAppendWarps)
paged_append_kernel(const __grid_constant__ PagedAppendArgs a,
                    const __grid_constant__ MropeParams prm, int splits, unsigned* err)
{
    constexpr int E = Vec<T>::N;
    constexpr int G = 32 / P;
    constexpr int HALF = P * E;
    constexpr int D = 2 * HALF;
    constexpr bool kStream = U > 1;
    const int lane = threadIdx.x & 31;
    const int pv = lane % P;
    const int hg = lane / P;
    const int j0 = pv * E;
    const int hq = a.hq, hk = a.hk, nh = hq + 2 * hk;
    const T* q = static_cast<const T*>(a.q);
    const T* k = static_cast<const T*>(a.k);
    const T* v = static_cast<const T*>(a.v);
    T* q_out = static_cast<T*>(a.q_out);
    T* kc = static_cast<T*>(a.k_pages);
    T* vc = static_cast<T*>(a.v_pages);
    __shared__ double inv_freq[HALF];

    fill_inv_freq(inv_freq, HALF, prm);
    pdl_wait();
    pdl_allow_dependents();

    const int64_t head_step = (int64_t)a.map.page_size * D;
    const int64_t units = a.tokens * splits;
    const int64_t stride = (int64_t)gridDim.x * kAppendWarps;
    const bool norm = a.gamma_q || a.gamma_k;
    for (int64_t unit = (int64_t)blockIdx.x * kAppendWarps + (threadIdx.x >> 5); unit < units;
         unit += stride) {
        const int64_t t = splits == 1 ? unit : (int64_t)((uint32_t)unit / (uint32_t)splits);
        const int part = splits == 1 ? 0 : (int)((uint32_t)unit % (uint32_t)splits);
        const int h_first = hg + part * G * U;

        uint4 lo[U], hi[U];
        auto load_batch = [&](int h0) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int h = h0 + u * G;
                if (h < nh) {
                    const T* src = h < hq        ? q + t * a.q_stride + (int64_t)h * D
                                   : h < hq + hk ? k + t * a.k_stride + (int64_t)(h - hq) * D
                                                 : v + t * a.v_stride + (int64_t)(h - hq - hk) * D;
                    lo[u] = ld_stream(src + j0);
                    hi[u] = ld_stream(src + HALF + j0);
                }
            }
        };
        load_batch(h_first);
        const int32_t pt = __ldg(a.pos + t), ph = __ldg(a.pos + a.tokens + t),
                      pw = __ldg(a.pos + 2 * a.tokens + t);
        const TokenSlot slot = token_slot(a, t, lane, err);
        if (!slot.owned)
            continue;
        float c[E], s[E];
        token_angles<E, P>(pt, ph, pw, inv_freq, prm, lane, c, s);

        for (int h0 = h_first; h0 - hg < nh; h0 += G * U * splits) {
            if (h0 != h_first)
                load_batch(h0);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int h = h0 + u * G;
                // the lanes of absent heads stay for the shuffles
                if (h - hg >= nh)
                    break;
                const bool rotated = h < hq + hk;
                float2 x[E / 2], y[E / 2];  // two values an operation
                if (h < nh) {
                    unpack2<T>(lo[u], x);
                    unpack2<T>(hi[u], y);
                }
                if (norm) {
                    float2 ss = make_float2(0.f, 0.f);
                    if (h < nh) {
#pragma unroll
                        for (int m = 0; m < E / 2; ++m)
                            ss = fma2(x[m], x[m], fma2(y[m], y[m], ss));
                    }
                    float sum = ss.x + ss.y;
#pragma unroll
                    for (int o = P / 2; o > 0; o >>= 1)
                        sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
                    const T* gamma = static_cast<const T*>(h < hq ? a.gamma_q : a.gamma_k);
                    if (rotated && gamma) {
                        const float r = rsqrtf(sum * (1.0f / D) + a.eps);
                        float2 g0[E / 2], g1[E / 2];
                        unpack2<T>(__ldg(reinterpret_cast<const uint4*>(gamma + j0)), g0);
                        unpack2<T>(__ldg(reinterpret_cast<const uint4*>(gamma + HALF + j0)), g1);
#pragma unroll
                        for (int m = 0; m < E / 2; ++m) {
                            x[m] = mul2(mul2(x[m], make_float2(r, r)), g0[m]);
                            y[m] = mul2(mul2(y[m], make_float2(r, r)), g1[m]);
                        }
                    }
                }
                if (h >= nh)
                    continue;
                T* dst;
                if (h < hq)
                    dst = q_out + t * a.q_out_stride + (int64_t)h * D;
                else if (slot.offset < 0)
                    continue;
                else if (rotated)
                    dst = kc + slot.offset + (h - hq) * head_step;
                else
                    dst = vc + slot.offset + (h - hq - hk) * head_step;
                if (rotated) {
                    float2 ox[E / 2], oy[E / 2];
#pragma unroll
                    for (int m = 0; m < E / 2; ++m) {
                        const float2 cm = make_float2(c[2 * m], c[2 * m + 1]);
                        const float2 sm = make_float2(s[2 * m], s[2 * m + 1]);
                        ox[m] = fma2(x[m], cm, mul2(y[m], make_float2(-sm.x, -sm.y)));
                        oy[m] = fma2(y[m], cm, mul2(x[m], sm));
                    }
                    st_out<kStream>(dst + j0, pack2<T>(ox));
                    st_out<kStream>(dst + HALF + j0, pack2<T>(oy));
                } else {  // v keeps its bits
                    st_out<kStream>(dst + j0, lo[u]);
                    st_out<kStream>(dst + HALF + j0, hi[u]);
                }
            }
        }
    }
}

// Any even head_dim, any alignment: one warp per (token, head), lanes over the
// pairs.  A head's values are read twice when it is normalised (the second
// time from L1).
template <typename T>
__global__ void __launch_bounds__(32 * kAppendWarps)
paged_append_any_kernel(const __grid_constant__ PagedAppendArgs a,
                        const __grid_constant__ MropeParams prm, unsigned* err)
{
    __shared__ double inv_freq[256];
    const int half = a.head_dim / 2;
    fill_inv_freq(inv_freq, half, prm);
    pdl_wait();
    pdl_allow_dependents();
    const int lane = threadIdx.x & 31;
    const int hq = a.hq, hk = a.hk, nh = hq + 2 * hk, d = a.head_dim;
    const int64_t head_step = (int64_t)a.map.page_size * d;
    const int64_t units = a.tokens * nh;
    const int64_t stride = (int64_t)gridDim.x * kAppendWarps;
    for (int64_t unit = (int64_t)blockIdx.x * kAppendWarps + (threadIdx.x >> 5); unit < units;
         unit += stride) {
        const int64_t t = unit / nh;
        const int h = (int)(unit % nh);
        const TokenSlot slot = token_slot(a, t, lane, err);
        if (!slot.owned || (h >= hq && slot.offset < 0))
            continue;
        const T* src = h < hq ? static_cast<const T*>(a.q) + t * a.q_stride + (int64_t)h * d
                       : h < hq + hk
                           ? static_cast<const T*>(a.k) + t * a.k_stride + (int64_t)(h - hq) * d
                           : static_cast<const T*>(a.v) + t * a.v_stride +
                                 (int64_t)(h - hq - hk) * d;
        if (h >= hq + hk) {
            T* dst = static_cast<T*>(a.v_pages) + slot.offset + (h - hq - hk) * head_step;
            for (int e = lane; e < d; e += 32)
                dst[e] = src[e];
            continue;
        }
        const T* gamma = static_cast<const T*>(h < hq ? a.gamma_q : a.gamma_k);
        T* dst = h < hq ? static_cast<T*>(a.q_out) + t * a.q_out_stride + (int64_t)h * d
                        : static_cast<T*>(a.k_pages) + slot.offset + (h - hq) * head_step;
        float r = 1.f;
        if (gamma) {
            float ss = 0.f;
            for (int e = lane; e < d; e += 32) {
                const float x = load_elem(src + e);
                ss += x * x;
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
            r = rsqrtf(ss / (float)d + a.eps);
        }
        const int32_t pt = __ldg(a.pos + t), ph = __ldg(a.pos + a.tokens + t),
                      pw = __ldg(a.pos + 2 * a.tokens + t);
        for (int j = lane; j < half; j += 32) {
            float c, s;
            rope_cos_sin(inv_freq[j], position_of(j, prm, pt, ph, pw), &c, &s);
            float x = load_elem(src + j), y = load_elem(src + half + j);
            if (gamma) {
                x = x * r * load_elem(gamma + j);
                y = y * r * load_elem(gamma + half + j);
            }
            store_elem(dst + j, x * c - y * s);
            store_elem(dst + half + j, y * c + x * s);
        }
    }
}

template <typename T, int P, int U>
cudaError_t launch_append(const PagedAppendArgs& a, const MropeParams& prm, unsigned* err,
                          int sm_count, int splits, cudaStream_t st)
{
    int64_t cap = (int64_t)sm_count * 64;
    if (U > 1)
        cap = std::min<int64_t>(cap, wave_ctas<paged_append_kernel<T, P, U>>(32 * kAppendWarps,
                                                                            sm_count, 1));
    const int64_t grid = std::min<int64_t>(ceil_div(a.tokens * splits, kAppendWarps), cap);
    return launch(paged_append_kernel<T, P, U>, dim3((unsigned)grid), dim3(32 * kAppendWarps), 0,
                  st, a, prm, splits, err);
}

// As arops_mrope_kv_append's launcher: one pass a warp while every pass fits
// the warps resident at once, else one or two warps a token on one wave (7,443
// tokens of 16 + 8 + 8 heads of 128 with norms: 29.3 us with two warps and four
// passes in flight each, 32.2 with one warp, 33.2 with four warps of two
// passes, 50.8 with eight of one).
template <typename T, int P>
cudaError_t launch_append_p(const PagedAppendArgs& a, const MropeParams& prm, unsigned* err,
                            int sm_count, cudaStream_t st)
{
    constexpr int G = 32 / P;
    const int64_t passes = ceil_div((int64_t)a.hq + 2 * (int64_t)a.hk, G);
    if (a.tokens * passes <= (int64_t)sm_count * 64)
        return launch_append<T, P, 1>(a, prm, err, sm_count, (int)passes, st);
    if (passes <= 2)
        return launch_append<T, P, 2>(a, prm, err, sm_count, 1, st);
    if (passes <= 4 || a.tokens > INT32_MAX / 2)
        return launch_append<T, P, 4>(a, prm, err, sm_count, 1, st);
    return launch_append<T, P, 4>(a, prm, err, sm_count, 2, st);
}

template <typename T>
cudaError_t launch_append_t(const PagedAppendArgs& a, const MropeParams& prm, cudaStream_t st)
{
    DeviceInfo di;
    cudaError_t e = current_device_info(&di);
    if (e != cudaSuccess)
        return e;
    unsigned* err = nullptr;
    e = device_error_word(&err);
    if (e != cudaSuccess)
        return e;
    constexpr int E = Vec<T>::N;
    auto vec = [](const void* p, int64_t stride) { return aligned16(p) && stride % E == 0; };
    const int half = a.head_dim / 2;
    const bool aligned =
        (a.hq == 0 || (vec(a.q, a.q_stride) && vec(a.q_out, a.q_out_stride))) &&
        (a.hk == 0 || (vec(a.k, a.k_stride) && vec(a.v, a.v_stride) && aligned16(a.k_pages) &&
                       aligned16(a.v_pages))) &&
        aligned16(a.gamma_q) && aligned16(a.gamma_k);
    if (aligned && half % E == 0) {
        switch (half / E) {
        case 1: return launch_append_p<T, 1>(a, prm, err, di.sm_count, st);
        case 2: return launch_append_p<T, 2>(a, prm, err, di.sm_count, st);
        case 4: return launch_append_p<T, 4>(a, prm, err, di.sm_count, st);
        case 8: return launch_append_p<T, 8>(a, prm, err, di.sm_count, st);
        case 16: return launch_append_p<T, 16>(a, prm, err, di.sm_count, st);
        case 32: return launch_append_p<T, 32>(a, prm, err, di.sm_count, st);
        default: break;
        }
    }
    const int64_t units = a.tokens * ((int64_t)a.hq + 2 * (int64_t)a.hk);
    const int64_t grid =
        std::min<int64_t>(ceil_div(units, kAppendWarps), (int64_t)di.sm_count * 16);
    return launch(paged_append_any_kernel<T>, dim3((unsigned)grid), dim3(32 * kAppendWarps), 0, st,
                  a, prm, err);
}

}  // namespace

cudaError_t launch_paged_append(const PagedAppendArgs& a, arops_dtype dtype, cudaStream_t stream)
{
    MropeParams prm;
    prm.sec0 = a.sections[0];
    prm.sec01 = a.sections[0] + a.sections[1];
    prm.freq_scale = 2.0 * log2((double)a.theta) / (double)a.head_dim;
    if (dtype == AROPS_BF16)
        return launch_append_t<__nv_bfloat16>(a, prm, stream);
    return launch_append_t<float>(a, prm, stream);
}

}  // namespace arops
