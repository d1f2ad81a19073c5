// Pieces that the attention kernels share: base-2 softmax arithmetic, the
// score options, the workspace's layout.
#pragma once

#include "paged.cuh"

namespace arops {

constexpr float kLog2e = 1.4426950408889634f;

// The workspace: 16 KiB of the row kernel's arrival counters (one a CTA, zero
// between calls), then partial results.
constexpr int kCounterBytes = 16384;

__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float reciprocal_fast(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// What a partial result with maximum m_x is multiplied by when the joined
// maximum is m: 2^(m_x - m), and 0 if m_x is -inf.  Such a part's O and l are
// multiplied by the 0, not left out: where all scores are NaN the maximum stays
// -inf, and the row keeps its NaN.
__device__ __forceinline__ float part_factor(float mx, float m)
{
    return mx == -INFINITY ? 0.0f : exp2_fast(mx - m);
}

// cap * tanh(s / cap).  A cap may be far above the scores (a large one means
// none), so the error goes by the score, not by the cap:
//   |s| <= cap / 2: s (1 + y Q(y)), y = (s / cap)^2, Q of degree 3 with the least
//   largest relative error of the whole (1.5e-8; Lawson's iteration on Chebyshev
//   nodes): with its roundings 7.5e-8 of the result at most (2.7e-8 rms), and s
//   itself where the cap is far away.
//   Above: 1 - 2 / (1 + e^2|x|), a few 2^-24 of the cap, of which the result is 0.46
//   at least.  (Taken for every score, as it was, it left decode scores of size 2
//   an error of 2.5e-6 at cap 50, 0.46 at cap 1e7.)
// A NaN stays one; where e^2|x| overflows the quotient is 0.
constexpr float kCap1 = -0.33333144f, kCap2 = 0.13325879f, kCap3 = -0.053045493f,
                kCap4 = 0.017241491f;

__device__ __forceinline__ float soft_cap_large(float s, float cap, float inv_cap)
{
    const float e = exp2_fast(fabsf(s) * inv_cap * (2.0f * kLog2e));
    return copysignf(cap * fmaf(-2.0f, reciprocal_fast(1.0f + e), 1.0f), s);
}

// Whether the form above is the score's.
__device__ __forceinline__ bool cap_is_near(float s, float inv_cap)
{
    return !(fabsf(s * inv_cap) <= 0.5f);
}

__device__ __forceinline__ float soft_cap_small(float s, float inv_cap)
{
    const float x = s * inv_cap, y = x * x;
    return fmaf(s, fmaf(fmaf(fmaf(kCap4, y, kCap3), y, kCap2), y, kCap1) * y, s);
}

__device__ __forceinline__ float soft_cap(float s, float cap, float inv_cap)
{
    const float small = soft_cap_small(s, inv_cap), large = soft_cap_large(s, cap, inv_cap);
    return cap_is_near(s, inv_cap) ? large : small;
}

// The tile kernel's form of it, for bf16: tanh(x) = x P(x^2) for |x| <= 1/2, P of
// degree 3 with the least largest relative error (5.4e-7; as above), its
// coefficients multiplied by what scores are multiplied by anyway.  That is
// 2^-20 of a score with its roundings.
constexpr float kTanh0 = 0.99999946f, kTanh1 = -0.33326319f, kTanh2 = 0.13190296f,
                kTanh3 = -0.044402227f;

// What a kernel does to a raw product q.k, in base 2: with neither cap nor
// slopes only scale * log2(e).
struct ScoreMap {
    float scale;      // plain: scale * log2e; with options: scale
    float cap, inv_cap;
};

inline ScoreMap make_score_map(const AttentionParams& p)
{
    ScoreMap m;
    const bool full = p.softcap > 0.0f || p.slopes != nullptr;
    m.scale = full ? p.scale : p.scale * kLog2e;
    m.cap = p.softcap;
    m.inv_cap = p.softcap > 0.0f ? 1.0f / p.softcap : 0.0f;
    return m;
}

// The scores of a lane from its products, in base 2: slope[e >> 1], i[e >> 1] and
// j0 + 8 t + (e & 1) are the bias's factor, the query's and the key's position.
// All lanes of the warp take part: it computes the cap's second form only where
// one of its scores needs it (256 sequences of 60-4,100 keys under a cap: 341 us,
// 357 where all need it; 366 and 393 with a branch a score).
template <bool FULL>
__device__ __forceinline__ void map_scores(float (&s)[2][4], const ScoreMap& m, const float* slope,
                                           const int32_t* i, int32_t j0)
{
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            s[t][e] *= m.scale;
    if constexpr (FULL) {
        if (m.cap > 0.0f) {
            bool near = false;
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    near = near || cap_is_near(s[t][e], m.inv_cap);
            if (__any_sync(0xFFFFFFFFu, near)) {
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        s[t][e] = soft_cap(s[t][e], m.cap, m.inv_cap);
            } else {
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        s[t][e] = soft_cap_small(s[t][e], m.inv_cap);
            }
        }
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int32_t j = j0 + t * 8 + (e & 1);
                s[t][e] = (s[t][e] - slope[e >> 1] * fabsf((float)(i[e >> 1] - j))) * kLog2e;
            }
    }
}

// Rows run over an entity's tokens, n heads each: row / n is its token.
struct RowDivide {
    uint32_t n;
    int32_t shift;  // log2(n), or -1
    __device__ __forceinline__ uint32_t operator()(uint32_t row) const
    {
        return shift >= 0 ? row >> shift : row / n;
    }
};

inline RowDivide make_row_divide(int32_t n)
{
    RowDivide d;
    d.n = (uint32_t)n;
    d.shift = -1;
    for (int s = 0; s < 31; ++s)
        if (n == (1 << s))
            d.shift = s;
    return d;
}

// Units of UNIT keys that [lo, hi) takes.
template <int UNIT>
__device__ __forceinline__ int32_t units_between(int32_t lo, int32_t hi)
{
    return hi > lo ? (int32_t)(((uint32_t)(hi - lo) + UNIT - 1) / UNIT) : 0;
}

// A sequence of a ragged batch: its first token, tokens, length.
struct Ragged {
    int32_t t0, ntok, len, bidir;
};

__device__ __forceinline__ Ragged load_ragged(const AttentionParams& p, int32_t s, bool& bad)
{
    Ragged r;
    const int64_t a = __ldg(p.q_start + s), b = __ldg(p.q_start + s + 1);
    const bool ok = a >= 0 && b >= a && b <= p.tokens;
    bad = bad || !ok;
    r.t0 = ok ? (int32_t)a : 0;
    r.ntok = ok ? (int32_t)(b - a) : 0;
    r.len = clamp_length(__ldg(p.kv_lens + s), p.max_pages * p.map.page_size, bad);
    r.bidir = p.bidir_lens ? __ldg(p.bidir_lens + s) : 0;
    return r;
}

// Keys that some of rows [row0, row0 + n) sees; rows run over the tokens, g a
// token.  The first row's keys begin first (at `seen`) and the last row's end
// last.  lo is `seen` rounded down to a unit.
template <int UNIT>
__device__ __forceinline__ void ragged_range(const AttentionParams& p, const Ragged& r,
                                             const RowDivide& g, uint32_t row0,
                                             uint32_t n, int32_t& lo, int32_t& hi,
                                             int32_t& seen)
{
    const int32_t first = (int32_t)g(row0);
    const int32_t last = min(r.ntok - 1, (int32_t)g(row0 + n - 1));
    int32_t x;
    visible_keys(r.len - r.ntok + first, r.len, r.bidir, p.window, seen, x);
    visible_keys(r.len - r.ntok + last, r.len, r.bidir, p.window, x, hi);
    lo = seen & ~(UNIT - 1);
}

// The tile kernel (attention_tiles.cu).  With prefix_o it takes the prefixes of
// a shared batch and leaves O (unnormalised, [tokens, hq, padded head_dim]) and
// (m, l) of every (sequence, head) there; otherwise it writes p.out.
bool tiles_can_run(const AttentionParams& p, arops_dtype dtype);
size_t tile_part_bytes(int dp);
cudaError_t launch_attention_tiles(const AttentionParams& p, float* parts, float* prefix_o,
                                   float* prefix_ml, int sm_count, cudaStream_t stream);

}  // namespace arops
