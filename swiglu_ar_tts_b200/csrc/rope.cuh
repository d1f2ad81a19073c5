// Angles of the multi-section rotary embedding, shared by the M-RoPE kernels
// (mrope.cu) and the paged append (paged_append.cu).
#pragma once

#include <math.h>

#include "common.cuh"

namespace arops {
namespace {

struct MropeParams {
    int32_t sec0;       // pairs j < sec0 take row 0 (t)
    int32_t sec01;      // pairs sec0 <= j < sec01 take row 1 (h); the rest row 2 (w)
    double freq_scale;  // 2 log2(theta) / head_dim: inverse frequency j is 2^(-j * freq_scale)
};

// theta^(-2j/head_dim) = 2^(-j * 2 log2(theta) / head_dim), the textbook RoPE
// inverse frequency, in fp64.
__device__ __forceinline__ double inv_freq_of(int j, const MropeParams& prm)
{
    return exp2(-(double)j * prm.freq_scale);
}

// Each CTA tabulates the head's inverse frequencies in shared memory once; this
// touches no global memory, so it runs before the dependency wait.
__device__ __forceinline__ void fill_inv_freq(double* table, int half, const MropeParams& prm)
{
    for (int j = threadIdx.x; j < half; j += blockDim.x)
        table[j] = inv_freq_of(j, prm);
    __syncthreads();
}

constexpr double kTwoPi = 6.283185307179586;
constexpr double kInvTwoPi = 0.15915494309189535;

__device__ __forceinline__ void rope_cos_sin(double inv_freq, int32_t p, float* c, float* s)
{
    const double phi = (double)p * inv_freq;
    const double k = rint(phi * kInvTwoPi);
    const double r = fma(-k, kTwoPi, phi);
    sincosf((float)r, s, c);
}

__device__ __forceinline__ int32_t position_of(int j, const MropeParams& prm, int32_t pt,
                                               int32_t ph, int32_t pw)
{
    return (j < prm.sec0) ? pt : ((j < prm.sec01) ? ph : pw);
}

// cos/sin of the angles a lane applies, for token t: the lanes of pair block
// pv split the block's E angles between them (F each) and share them with
// shuffles, so every lane of the warp must take part.
template <int E, int P>
__device__ __forceinline__ void token_angles(int32_t pt, int32_t ph, int32_t pw,
                                             const double* inv_freq, const MropeParams& prm,
                                             int lane, float* c, float* s)
{
    constexpr int G = 32 / P;                // heads per warp pass
    constexpr int F = (E >= G) ? E / G : 1;  // angles evaluated per lane
    const int pv = lane % P;
    const int hg = lane / P;
    const int j0 = pv * E;
    float cs[F], sn[F];
#pragma unroll
    for (int f = 0; f < F; ++f) {
        const int j = j0 + ((hg * F + f) % E);
        rope_cos_sin(inv_freq[j], position_of(j, prm, pt, ph, pw), &cs[f], &sn[f]);
    }
#pragma unroll
    for (int m = 0; m < E; ++m) {
        const int src = pv + P * ((m / F) % G);
        c[m] = __shfl_sync(0xFFFFFFFFu, cs[m % F], src);
        s[m] = __shfl_sync(0xFFFFFFFFu, sn[m % F], src);
    }
}

}  // namespace
}  // namespace arops
