// Pieces that the attention kernels share: base-2 softmax arithmetic, the
// score options, the workspace's layout.
#pragma once

#include "paged.cuh"

namespace arops {

constexpr float kLog2e = 1.4426950408889634f;

// The workspace: 16 KiB of arrival counters (zero between calls), 2048 for the
// row kernel and 2048 for the tile kernel, then their partial results.
constexpr int kCounterBytes = 16384;
constexpr int kMaxAttentionCtas = 2048;

__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// s / cap through tanh, times cap: tanh(x) = 1 - 2 / (1 + e^2x).  Its absolute
// error is a few 2^-24 of cap whatever x is, which is what a score needs (the
// quotient is 0 where e^2x overflows).
__device__ __forceinline__ float soft_cap(float s, float cap, float inv_cap)
{
    const float e = exp2_fast(s * inv_cap * (2.0f * kLog2e));
    return cap - cap * __fdividef(2.0f, 1.0f + e);
}

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

template <bool FULL>
__device__ __forceinline__ float map_score(float s, const ScoreMap& m, float slope, int32_t i,
                                           int32_t j)
{
    if constexpr (!FULL) {
        return s * m.scale;
    } else {
        s *= m.scale;
        if (m.cap > 0.0f)
            s = soft_cap(s, m.cap, m.inv_cap);
        return (s - slope * fabsf((float)(i - j))) * kLog2e;
    }
}

}  // namespace arops
