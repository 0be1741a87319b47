// qk_norm.cu -- norm of queries and keys for each head with the position rotation, for prompts.
//
// Bound by memory: every entry is read once and written once (2 a bytes).  A block takes a few
// tokens, tabulates their (cos, sin) once in shared memory -- they are the same for all heads, so the
// fp64 angles cost one evaluation per (token, pair), not per entry -- and runs over the tokens' query
// and key heads.
#include "kernels.h"
#include "qk_norm.cuh"

namespace hyena {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxTile = 8;                               // tokens of one block at most
constexpr int kMaxHalf = HYENA_MAX_HEAD_DIM / 2;

struct QKArgs {
    const void *q, *k;
    void *qo, *ko;
    long long ntok, ldq, ldk, ldqo, ldko;
    int L, H, Hk, hd, tile;
    const int *pos;
    int pos0;
    QKPrepArgs p;
};

// Scalar form: a warp per head, a pair per lane and step; any even hd, alignment of one element.
template <class Act>
__global__ void __launch_bounds__(kThreads) qk_norm_kernel(const QKArgs a) {
    using T = typename Act::T;
    __shared__ float2 cs[kMaxTile * kMaxHalf];
    const int tid = threadIdx.x, lane = tid & 31, half = a.p.rot >> 1, heads = a.H + a.Hk;
    const long long t0 = (long long)blockIdx.x * a.tile;
    const int nt = (int)min((long long)a.tile, a.ntok - t0);
    for (int i = tid; i < nt * half; i += kThreads) {
        const long long t = t0 + i / half;
        const int pos = a.pos ? a.pos[HB_IDX(t, a.ntok)] : a.pos0 + (int)(t % a.L);
        cs[i] = rotation_of(pos, a.p.inv_freq[HB_IDX(i % half, half)]);
    }
    __syncthreads();
    for (int it = tid >> 5; it < nt * heads; it += kThreads / 32) {
        const int tt = it / heads, h = it % heads;
        const bool isq = h < a.H;
        const long long t = t0 + tt;
        const long long si = isq ? t * a.ldq + (long long)h * a.hd : t * a.ldk + (long long)(h - a.H) * a.hd;
        const long long di = isq ? t * a.ldqo + (long long)h * a.hd : t * a.ldko + (long long)(h - a.H) * a.hd;
        const T *src = static_cast<const T *>(isq ? a.q : a.k);
        T *dst = static_cast<T *>(isq ? a.qo : a.ko);
        const long long ns = (a.ntok - 1) * (isq ? a.ldq : a.ldk) + (long long)(isq ? a.H : a.Hk) * a.hd;
        const long long nd = (a.ntok - 1) * (isq ? a.ldqo : a.ldko) + (long long)(isq ? a.H : a.Hk) * a.hd;
        (void)ns; (void)nd;
        const float *w = isq ? a.p.qw : a.p.kw;
        float xa[4], xb[4], ss = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int p = lane + 32 * i;
            xa[i] = xb[i] = 0.f;
            if (p < a.hd / 2) {
                int e0, e1;
                pair_entries(p, half, a.p.interleaved, e0, e1);
                xa[i] = Act::ld(src + HB_IDX(si + e0, ns));
                xb[i] = Act::ld(src + HB_IDX(si + e1, ns));
            }
            ss = fmaf(xa[i], xa[i], fmaf(xb[i], xb[i], ss));
        }
        float r = 1.f;
        if (a.p.norm) {
#pragma unroll
            for (int m = 16; m >= 1; m >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
            r = rsqrtf(ss / (float)a.hd + a.p.eps);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int p = lane + 32 * i;
            if (p < a.hd / 2) {
                int e0, e1;
                pair_entries(p, half, a.p.interleaved, e0, e1);
                float ya = xa[i], yb = xb[i];
                if (a.p.norm) {
                    ya *= r * (w ? __ldg(w + HB_IDX(e0, a.hd)) : 1.f);
                    yb *= r * (w ? __ldg(w + HB_IDX(e1, a.hd)) : 1.f);
                }
                if (p < half) {
                    const float2 y = rotate(ya, yb, cs[tt * half + p]);
                    ya = y.x;
                    yb = y.y;
                }
                if (HB_OK(di + e0, nd)) Act::st(dst + di + e0, ya);
                if (HB_OK(di + e1, nd)) Act::st(dst + di + e1, yb);
            }
        }
    }
}

}  // namespace

HYENA_BOUNDS_READER(qk_norm)

cudaError_t launch_qk_norm(const void *q, const void *k, int dtype, int B, int L, int H, int Hk, int hd, long long ldq,
                           long long ldk, const hyena_qk_prep &p, const int *pos, int pos0, void *qo, void *ko,
                           long long ldqo, long long ldko, cudaStream_t s) {
    QKArgs a;
    a.q = q; a.k = k; a.qo = qo; a.ko = ko;
    a.ntok = (long long)B * L;
    a.ldq = ldq; a.ldk = ldk; a.ldqo = ldqo; a.ldko = ldko;
    a.L = L; a.H = H; a.Hk = Hk; a.hd = hd;
    a.pos = pos; a.pos0 = pos0;
    a.p = QKPrepArgs{p.norm, p.eps, p.q_weight, p.k_weight, p.rot_dim, p.inv_freq, p.interleaved};
    // a few tokens per block, but enough blocks to fill the GPU
    a.tile = a.ntok >= 148 * 8 * 4 ? 4 : 1;
    const long long blocks = (a.ntok + a.tile - 1) / a.tile;
    if (blocks > 0x7fffffffll) return cudaErrorInvalidValue;
    if (dtype == HYENA_BF16) qk_norm_kernel<ActBF16><<<(unsigned)blocks, kThreads, 0, s>>>(a);
    else qk_norm_kernel<ActF32><<<(unsigned)blocks, kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace hyena
