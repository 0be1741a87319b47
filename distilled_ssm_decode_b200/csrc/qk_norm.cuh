// qk_norm.cuh -- norm and rotation of one head's query or key vector (device code shared by the
// prompt kernel of qk_norm.cu and the single-token step of linattn_decode.cu).
//
//   x <- x rsqrt(mean(x^2) + eps) w,   (a, b) <- (a cos t - b sin t, b cos t + a sin t)
//
// The vector is handled as hd/2 pairs: pair p of the first rot/2 is rotated by t = position *
// inv_freq[p]; the entries behind rot form pairs of neighbours that are only normed.  Both pairings
// ((i, i + rot/2) and (2i, 2i+1)) then differ only in where a pair's two entries lie.
#pragma once

#include "common.cuh"

namespace hyena {

struct QKPrepArgs {
    int norm;
    float eps;
    const float *qw, *kw;     // [hd] or null
    int rot;                  // rotated entries
    const float *inv_freq;    // [rot / 2]
    int interleaved;
};

// entries (e0, e1) of pair p
__device__ __forceinline__ void pair_entries(int p, int half, int interleaved, int &e0, int &e1) {
    if (interleaved || p >= half) {
        e0 = 2 * p;           // behind the rotated part: rot + 2 (p - rot/2) = 2 p
        e1 = 2 * p + 1;
    } else {
        e0 = p;
        e1 = p + half;
    }
}

// (cos t, sin t) of t = pos * freq.  The angle is formed in turns and reduced in fp64: pos * freq
// reaches 1e6 rad and more, where fp32 keeps no digits behind the point; after the reduction the
// rounding to fp32 is at most 2^-25 of half a turn.
__device__ __forceinline__ float2 rotation_of(int pos, float freq) {
    double a = (double)pos * (double)freq * 0.15915494309189533577;    // 1 / (2 pi)
    a -= rint(a);
    float c, s;
    sincospif((float)(2.0 * a), &s, &c);
    return make_float2(c, s);
}

__device__ __forceinline__ float2 rotate(float a, float b, float2 cs) {
    return make_float2(fmaf(a, cs.x, -b * cs.y), fmaf(b, cs.x, a * cs.y));
}

// One head's vector by one warp: x[at .. at + hd) of a tensor of n elements (hd even, <= 256) -> out [hd] fp32.
template <class Act>
__device__ __forceinline__ void norm_rotate_warp(const typename Act::T *__restrict__ x, long long at, long long n,
                                                 const float *__restrict__ w, const QKPrepArgs &a, int pos, int hd,
                                                 float *out, int lane) {
    (void)n;
    const int half = a.rot >> 1;
    float xa[4], xb[4], ss = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int p = lane + 32 * i;
        xa[i] = xb[i] = 0.f;
        if (p < hd / 2) {
            int e0, e1;
            pair_entries(p, half, a.interleaved, e0, e1);
            xa[i] = Act::ld(x + HB_IDX(at + e0, n));
            xb[i] = Act::ld(x + HB_IDX(at + e1, n));
        }
        ss = fmaf(xa[i], xa[i], fmaf(xb[i], xb[i], ss));
    }
    float r = 1.f;
    if (a.norm) {
#pragma unroll
        for (int m = 16; m >= 1; m >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
        r = rsqrtf(ss / (float)hd + a.eps);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int p = lane + 32 * i;
        if (p < hd / 2) {
            int e0, e1;
            pair_entries(p, half, a.interleaved, e0, e1);
            float ya = xa[i], yb = xb[i];
            if (a.norm) {
                ya *= r * (w ? __ldg(w + HB_IDX(e0, hd)) : 1.f);
                yb *= r * (w ? __ldg(w + HB_IDX(e1, hd)) : 1.f);
            }
            if (p < half) {
                const float2 y = rotate(ya, yb, rotation_of(pos, __ldg(a.inv_freq + HB_IDX(p, half))));
                ya = y.x;
                yb = y.y;
            }
            out[e0] = ya;
            out[e1] = yb;
        }
    }
}

}  // namespace hyena
