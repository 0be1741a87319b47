// qk_norm.cu -- norm of queries and keys for each head with the position rotation, for prompts.
//
// Bound by memory: every entry is read once and written once (2 a bytes).  A block takes a few tokens.
// It first issues the loads of its heads (VEC entries per lane, PP lanes per head), then tabulates the
// tokens' cos and sin in shared memory -- they are the same for all heads, so the fp64 angles cost one evaluation
// per (token, pair), not per entry, and run while the loads are in flight -- and then norms, rotates and stores.
// With whole heads rotated a lane has both entries of its pairs (56 us where shuffles took 68, 8 x 4096 tokens of 2 x 8
// heads of 128); otherwise the other entry comes from the lane that has it, by a shuffle.  Sizes, strides or pointers that do not
// fit a vector take the scalar kernel (a warp per head).
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
    float inv_hd;
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

// VEC entries as they lie in memory
template <class Act, int VEC> struct Raw {
    static constexpr int kWords = VEC * Act::bytes / 4;
    uint32_t r[kWords];
    __device__ __forceinline__ void load(const void *p) {
        if constexpr (kWords >= 4) {
#pragma unroll
            for (int i = 0; i < kWords / 4; ++i) {
                const uint4 t = static_cast<const uint4 *>(p)[i];
                r[4 * i] = t.x; r[4 * i + 1] = t.y; r[4 * i + 2] = t.z; r[4 * i + 3] = t.w;
            }
        } else if constexpr (kWords == 2) {
            const uint2 t = *static_cast<const uint2 *>(p);
            r[0] = t.x; r[1] = t.y;
        } else {
            r[0] = *static_cast<const uint32_t *>(p);
        }
    }
    __device__ __forceinline__ void store(void *p) const {
        if constexpr (kWords >= 4) {
#pragma unroll
            for (int i = 0; i < kWords / 4; ++i)
                static_cast<uint4 *>(p)[i] = make_uint4(r[4 * i], r[4 * i + 1], r[4 * i + 2], r[4 * i + 3]);
        } else if constexpr (kWords == 2) {
            *static_cast<uint2 *>(p) = make_uint2(r[0], r[1]);
        } else {
            *static_cast<uint32_t *>(p) = r[0];
        }
    }
    // the two halves from two places
    __device__ __forceinline__ void load(const void *p, const void *q) {
        Raw<Act, VEC / 2> a, b;
        a.load(p);
        b.load(q);
#pragma unroll
        for (int i = 0; i < kWords / 2; ++i) { r[i] = a.r[i]; r[kWords / 2 + i] = b.r[i]; }
    }
    __device__ __forceinline__ void store(void *p, void *q) const {
        Raw<Act, VEC / 2> a, b;
#pragma unroll
        for (int i = 0; i < kWords / 2; ++i) { a.r[i] = r[i]; b.r[i] = r[kWords / 2 + i]; }
        a.store(p);
        b.store(q);
    }
    __device__ __forceinline__ float get(int i) const {
        if constexpr (Act::bytes == 4) return __uint_as_float(r[i]);
        else return __uint_as_float(i & 1 ? r[i / 2] & 0xffff0000u : r[i / 2] << 16);
    }
    __device__ __forceinline__ void set2(int i, float a, float b) {     // entries i, i + 1 (i even)
        if constexpr (Act::bytes == 4) {
            r[i] = __float_as_uint(a);
            r[i + 1] = __float_as_uint(b);
        } else {
            const __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
            r[i / 2] = *reinterpret_cast<const uint32_t *>(&p);
        }
    }
};

// Vector form.  PP lanes (a power of two) per head, the first hd / VEC of them with entries; kThreads / PP / tile groups
// of lanes share a token and take its heads in turn, U of q and U of k in flight.  An entry's output is
// r (x A + y B) with y the pair's other entry and A = w cos, B = -+ w_y sin fixed for the group's token (A = w, B = 0
// without rotation), so a head costs three operations per entry beside its norm.
// Pairs (i, i + rot/2) need rot/2 to be a multiple of VEC, so that a lane's entries lie on one side.
// kWhole: pairs (i, i + hd/2) of whole heads, both entries of a pair in one lane; kHalves: (i, i + rot/2) of a part
enum { kNoRotation, kHalves, kNeighbours, kWhole };
template <class Act, int VEC, int PP, int MODE>
__global__ void __launch_bounds__(kThreads, 3) qk_norm_vec_kernel(const QKArgs a) {
    using T = typename Act::T;
    using R = Raw<Act, VEC>;
    constexpr int kGroups = kThreads / PP, U = R::kWords > 4 ? 2 : 4, HV = VEC / 2;
    __shared__ __align__(16) float cs[2][kMaxTile * kMaxHalf];      // cos, sin
    __shared__ __align__(16) float ws[2][HYENA_MAX_HEAD_DIM];       // norm weights of q and k
    const int tid = threadIdx.x, l = tid % PP, grp = tid / PP, half = a.p.rot >> 1;
    const int gpt = kGroups / a.tile, tt = grp / gpt, slot = grp % gpt;
    const int e = MODE == kWhole ? l * HV : l * VEC, far = MODE == kWhole ? a.hd / 2 - HV : 0;      // far: from its first half's end to its second half
    const int side = MODE != kHalves || e >= 2 * half ? 0 : e < half ? 1 : -1;
    const bool on = l * VEC < a.hd;
    const int mate = (tid & 31) + side * (half / VEC);              // the lane with the pairs' other entries
    const long long t = (long long)blockIdx.x * a.tile + tt;
    const int nt = (int)min((long long)a.tile, a.ntok - (long long)blockIdx.x * a.tile);
    R x[2][U];
    auto load = [&](int s, int base) {
        const int heads = s ? a.Hk : a.H;
        const long long ld = s ? a.ldk : a.ldq, ext = (a.ntok - 1) * ld + (long long)heads * a.hd;
        (void)ext;
        const long long at = t * ld + (long long)(base + slot) * a.hd + e;
        const T *src = static_cast<const T *>(s ? a.k : a.q);
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int i = 0; i < R::kWords; ++i) x[s][u].r[i] = 0u;
            const long long xat = at + (long long)u * gpt * a.hd;
            if (on && tt < nt && base + u * gpt + slot < heads && HB_OK(xat + far + VEC - 1, ext)) {
                if constexpr (MODE == kWhole) x[s][u].load(src + xat, src + xat + a.hd / 2);
                else x[s][u].load(src + xat);
            }
        }
    };
    constexpr int kRead = MODE == kWhole ? HV : VEC;
    auto read = [&](const float *p, float *v) {
        if constexpr (kRead == 2) {
            const float2 f = *reinterpret_cast<const float2 *>(p);
            v[0] = f.x; v[1] = f.y;
        } else {
#pragma unroll
            for (int i = 0; i < kRead; i += 4) {
                const float4 f = *reinterpret_cast<const float4 *>(p + i);
                v[i] = f.x; v[i + 1] = f.y; v[i + 2] = f.z; v[i + 3] = f.w;
            }
        }
    };
    float c[VEC], sn[VEC];                       // this lane's entries: cos, and the sine with its sign (0: no rotation)
    auto angles = [&]() {
#pragma unroll
        for (int i = 0; i < VEC; ++i) { c[i] = 1.f; sn[i] = 0.f; }
        if (MODE == kWhole) {
            if (on) {
                read(cs[0] + tt * half + e, c);
                read(cs[1] + tt * half + e, sn);
            }
        } else if (MODE == kHalves && side) {
            const int at = tt * half + (side > 0 ? e : e - half);
            read(cs[0] + at, c);
            read(cs[1] + at, sn);
#pragma unroll
            for (int i = 0; i < VEC; ++i) sn[i] = side > 0 ? -sn[i] : sn[i];
        } else if (MODE == kNeighbours) {
#pragma unroll
            for (int i = 0; i < VEC; i += 2)
                if (e + i < 2 * half) {
                    const int at = tt * half + (e + i) / 2;
                    c[i] = c[i + 1] = cs[0][at];
                    sn[i + 1] = cs[1][at];
                    sn[i] = -sn[i + 1];
                }
        }
    };
    auto finish = [&](int s, int base) {
        const int heads = s ? a.Hk : a.H;
        if (base >= heads) return;
        const long long ld = s ? a.ldko : a.ldqo, ext = (a.ntok - 1) * ld + (long long)heads * a.hd;
        (void)ext;
        T *dst = static_cast<T *>(s ? a.ko : a.qo);
        const long long at = t * ld + (long long)(base + slot) * a.hd + e;
        float A[VEC], B[VEC];
        {
            float w0[VEC], w1[VEC];
            read(ws[s] + (on ? e : 0), w0);
            if constexpr (MODE == kWhole) {
                read(ws[s] + (on ? e + a.hd / 2 : 0), w1);
#pragma unroll
                for (int i = 0; i < HV; ++i) {
                    A[i] = w0[i] * c[i];
                    B[i] = -w1[i] * sn[i];
                    A[HV + i] = w1[i] * c[i];
                    B[HV + i] = w0[i] * sn[i];
                }
            } else if (MODE != kHalves) {
#pragma unroll
                for (int i = 0; i < VEC; ++i) w1[i] = w0[i ^ 1];
            } else {
                read(ws[s] + (on ? e + side * half : 0), w1);
            }
            if constexpr (MODE != kWhole) {
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    A[i] = w0[i] * c[i];
                    B[i] = w1[i] * sn[i];
                }
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (base + u * gpt >= heads) break;          // the same for the whole block
            const R &z = x[s][u];
            float r = 1.f;
            if (a.p.norm) {
                float ss = 0.f;
#pragma unroll
                for (int i = 0; i < VEC; ++i) ss = fmaf(z.get(i), z.get(i), ss);
#pragma unroll
                for (int m = PP / 2; m >= 1; m >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
                r = rsqrtf(fmaf(ss, a.inv_hd, a.p.eps));
            }
            R y, o;
            if (MODE == kHalves) {
#pragma unroll
                for (int i = 0; i < R::kWords; ++i) {
                    y.r[i] = __shfl_sync(0xffffffffu, z.r[i], mate);
                    if (!side) y.r[i] = 0u;
                }
            }
#pragma unroll
            for (int i = 0; i < VEC; i += 2) {
                float y0 = 0.f, y1 = 0.f;
                if (MODE == kWhole) {
                    y0 = z.get((i + HV) % VEC);
                    y1 = z.get((i + 1 + HV) % VEC);
                } else if (MODE == kHalves) {
                    y0 = y.get(i);
                    y1 = y.get(i + 1);
                } else if (MODE == kNeighbours && e + i < 2 * half) {
                    y0 = z.get(i + 1);
                    y1 = z.get(i);
                }
                o.set2(i, r * fmaf(z.get(i), A[i], y0 * B[i]), r * fmaf(z.get(i + 1), A[i + 1], y1 * B[i + 1]));
            }
            const long long xat = at + (long long)u * gpt * a.hd;
            if (on && tt < nt && base + u * gpt + slot < heads && HB_OK(xat + far + VEC - 1, ext)) {
                if constexpr (MODE == kWhole) o.store(dst + xat, dst + xat + a.hd / 2);
                else o.store(dst + xat);
            }
        }
    };
    load(0, 0);
    load(1, 0);
    const long long tb = (long long)blockIdx.x * a.tile;
    // a warp per token, or all warps for a single one
    const bool one = nt == 1;
    for (int i = one ? 0 : tid >> 5; i < nt; i += kThreads / 32) {
        const long long ta = tb + i;
        const int pos = a.pos ? a.pos[HB_IDX(ta, a.ntok)] : a.pos0 + (int)(ta % a.L);
        for (int p = one ? tid : tid & 31; p < half; p += one ? kThreads : 32) {
            const float2 v = rotation_of(pos, a.p.inv_freq[HB_IDX(p, half)]);
            cs[0][i * half + p] = v.x;
            cs[1][i * half + p] = v.y;
        }
    }
    for (int i = tid; i < 2 * a.hd; i += kThreads) {
        const int s = i >= a.hd, j = i - s * a.hd;
        const float *w = s ? a.p.kw : a.p.qw;
        ws[s][j] = a.p.norm && w ? w[HB_IDX(j, a.hd)] : 1.f;
    }
    __syncthreads();
    angles();
    for (int base = 0;;) {
        finish(0, base);
        finish(1, base);
        base += U * gpt;
        if (base >= max(a.H, a.Hk)) break;
        load(0, base);
        load(1, base);
    }
}

template <class Act, int VEC, int PP>
void launch_mode(const QKArgs &a, unsigned blocks, cudaStream_t s) {
    if (a.p.rot == 0) qk_norm_vec_kernel<Act, VEC, PP, kNoRotation><<<blocks, kThreads, 0, s>>>(a);
    else if (!a.p.interleaved && a.p.rot == a.hd) qk_norm_vec_kernel<Act, VEC, PP, kWhole><<<blocks, kThreads, 0, s>>>(a);
    else if (!a.p.interleaved) qk_norm_vec_kernel<Act, VEC, PP, kHalves><<<blocks, kThreads, 0, s>>>(a);
    else qk_norm_vec_kernel<Act, VEC, PP, kNeighbours><<<blocks, kThreads, 0, s>>>(a);
}

template <class Act, int VEC>
void launch_vec(const QKArgs &a, unsigned blocks, int pp, cudaStream_t s) {
    switch (pp) {
    case 4: launch_mode<Act, VEC, 4>(a, blocks, s); break;
    case 8: launch_mode<Act, VEC, 8>(a, blocks, s); break;
    case 16: launch_mode<Act, VEC, 16>(a, blocks, s); break;
    default: launch_mode<Act, VEC, 32>(a, blocks, s); break;
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
    a.inv_hd = 1.f / (float)hd;
    a.pos = pos; a.pos0 = pos0;
    a.p = QKPrepArgs{p.norm, p.eps, p.q_weight, p.k_weight, p.rot_dim, p.inv_freq, p.interleaved};
    // Vectors of 8 or 4 entries: the widest that divides the head, the strides and (pairs (i, i + rot/2)) rot / 2,
    // with the pointers aligned to it and the head within a warp.  Measured, bf16, 8 x 4096 tokens
    // of 2 x 8 heads of 128: 56 us (4.8 TB/s of 6.5 measured; 155 us with the scalar kernel alone), fp32, 3 x 1999
    // tokens of 8 heads of 80: 13 us (20 us).
    const int bytes = dtype == HYENA_BF16 ? 2 : 4;
    int vec = 8;
    auto fits = [&](int n) {
        auto at = [&](const void *x) { return reinterpret_cast<uintptr_t>(x) % ((size_t)min(16, n * bytes)) == 0; };
        return hd % n == 0 && hd / n <= 32 && (p.interleaved || p.rot_dim == hd || (p.rot_dim / 2) % n == 0) && ldq % n == 0 && ldk % n == 0 &&
               ldqo % n == 0 && ldko % n == 0 && at(q) && at(k) && at(qo) && at(ko);
    };
    while (vec > 2 && !fits(vec)) vec /= 2;
    if (vec == 2) vec = 1;
    int pp = 4;
    while (pp * vec < hd) pp *= 2;
    // Tokens of a block (a power of two): as many as let every group of lanes have its U heads in flight, fewer where
    // that would leave SMs without a block.
    const int most = H > Hk ? H : Hk, groups = kThreads / pp, inflight = vec * bytes > 16 ? 2 : 4;
    a.tile = vec > 1 ? 1 : a.ntok >= 148 * 8 * 4 ? 4 : 1;
    while (vec > 1 && 2 * a.tile <= kMaxTile && 2 * a.tile <= groups && (long long)most * 2 * a.tile <= (long long)inflight * groups &&
           a.ntok >= 148ll * 2 * 2 * a.tile)
        a.tile *= 2;
    const long long blocks = (a.ntok + a.tile - 1) / a.tile;
    if (blocks > 0x7fffffffll) return cudaErrorInvalidValue;
    if (vec > 1) {
        const unsigned n = (unsigned)blocks;
        if (dtype == HYENA_BF16) vec == 8 ? launch_vec<ActBF16, 8>(a, n, pp, s) : launch_vec<ActBF16, 4>(a, n, pp, s);
        else vec == 8 ? launch_vec<ActF32, 8>(a, n, pp, s) : launch_vec<ActF32, 4>(a, n, pp, s);
        return cudaGetLastError();
    }
    if (dtype == HYENA_BF16) qk_norm_kernel<ActBF16><<<(unsigned)blocks, kThreads, 0, s>>>(a);
    else qk_norm_kernel<ActF32><<<(unsigned)blocks, kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace hyena
