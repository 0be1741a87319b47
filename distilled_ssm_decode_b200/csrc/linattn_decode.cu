// linattn_decode.cu -- one token of linear attention with a decay for each head.
//
//   S <- g S + k v^T,   o = scale S^T q      (S [dk][dv] fp32 per sequence and key/value head)
//
// Bound by memory: S is read and written once (8 dk dv bytes against 4 dk dv operations).  A block
// owns one state, or a slice of its columns when there are too few states to fill the GPU (columns
// are independent, so a slice needs no exchange).  Threads lie as rows x columns: CT threads across a
// slice, V columns each, 256 / CT row groups; a thread's rows are loaded in batches of kRows before the
// first is used, the first batch even before the queries and keys are ready.  All query heads of the
// group use the loaded rows, so a shared state is read once for all of them.
#include "kernels.h"
#include "qk_norm.cuh"

namespace hyena {

namespace {

constexpr int kThreads = 256;
constexpr int kRows = 8;

struct DecArgs {
    const void *q, *k, *v;
    void *o;
    float *state;
    const float *decay;
    float scale;
    int B, H, Hk, dk, dv, slices;
    long long ldq, ldk, ldv;
    int prep;
    QKPrepArgs p;
    const int *pos;
    int pos0;
};

template <int V> struct Vec;
template <> struct Vec<4> {
    float x[4];
    __device__ __forceinline__ void load(const float *p) {
        const float4 t = __ldcs(reinterpret_cast<const float4 *>(p));
        x[0] = t.x; x[1] = t.y; x[2] = t.z; x[3] = t.w;
    }
    __device__ __forceinline__ void store(float *p) const {
        __stcs(reinterpret_cast<float4 *>(p), make_float4(x[0], x[1], x[2], x[3]));
    }
};
template <> struct Vec<1> {
    float x[1];
    __device__ __forceinline__ void load(const float *p) { x[0] = *p; }
    __device__ __forceinline__ void store(float *p) const { *p = x[0]; }
};

// G query heads per state are taken GT at a time (the first round updates the state, later rounds
// read it back).
template <class Act, int V, int CT, int GT>
__global__ void __launch_bounds__(kThreads) linattn_decode_kernel(const DecArgs a) {
    using T = typename Act::T;
    constexpr int RG = kThreads / CT, CS = CT * V, kWarps = kThreads / 32;
    __shared__ float ks[HYENA_MAX_HEAD_DIM], qs[GT][HYENA_MAX_HEAD_DIM];
    __shared__ float red[kWarps][GT][CS];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int sl = blockIdx.x % a.slices, unit = blockIdx.x / a.slices;
    const int hk = unit % a.Hk, b = unit / a.Hk, G = a.H / a.Hk;
    const int c = tid % CT, rg = tid / CT, col = sl * CS + c * V;
    const bool on = col < a.dv;
    const T *q = static_cast<const T *>(a.q), *k = static_cast<const T *>(a.k), *v = static_cast<const T *>(a.v);
    const long long qat = (long long)b * a.ldq + (long long)hk * G * a.dk, kat = (long long)b * a.ldk + (long long)hk * a.dk,
                    vat = (long long)b * a.ldv + (long long)hk * a.dv;
    const long long nq = (a.B - 1) * a.ldq + (long long)a.H * a.dk, nk = (a.B - 1) * a.ldk + (long long)a.Hk * a.dk,
                    nv = (a.B - 1) * a.ldv + (long long)a.Hk * a.dv;
    const long long sbase = (long long)unit * a.dk * a.dv, ns = (long long)a.B * a.Hk * a.dk * a.dv;
    (void)nq; (void)nk; (void)nv; (void)ns;
    float *S = a.state;
    auto at = [&](int r) { return sbase + (long long)r * a.dv + col; };

    Vec<V> s[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int r = rg + i * RG;
        if (on && r < a.dk) s[i].load(S + HB_IDX(at(r), ns - V + 1));
    }
    float vv[V];
#pragma unroll
    for (int j = 0; j < V; ++j) vv[j] = on && col + j < a.dv ? Act::ld(v + HB_IDX(vat + col + j, nv)) : 0.f;
    const float g = a.decay[HB_IDX(hk, a.Hk)];
    const int pos = a.prep ? (a.pos ? a.pos[HB_IDX(b, a.B)] : a.pos0) : 0;

    for (int g0 = 0; g0 < G; g0 += GT) {
        const int ng = min(GT, G - g0);
        // this round's queries, and the key
        if (a.prep) {
            for (int i = warp; i < ng + (g0 == 0); i += kWarps) {
                if (i < ng) norm_rotate_warp<Act>(q, qat + (long long)(g0 + i) * a.dk, nq, a.p.qw, a.p, pos, a.dk, qs[i], lane);
                else norm_rotate_warp<Act>(k, kat, nk, a.p.kw, a.p, pos, a.dk, ks, lane);
            }
        } else {
            for (int i = tid; i < ng * a.dk; i += kThreads)
                qs[i / a.dk][i % a.dk] = Act::ld(q + HB_IDX(qat + (long long)g0 * a.dk + i, nq));
            if (g0 == 0)
                for (int i = tid; i < a.dk; i += kThreads) ks[i] = Act::ld(k + HB_IDX(kat + i, nk));
        }
        __syncthreads();
        float acc[GT][V];
#pragma unroll
        for (int i = 0; i < GT; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) acc[i][j] = 0.f;
        for (int r0 = rg; r0 < a.dk; r0 += RG * kRows) {
            if (r0 != rg || g0 != 0) {
#pragma unroll
                for (int i = 0; i < kRows; ++i) {
                    const int r = r0 + i * RG;
                    if (on && r < a.dk) s[i].load(S + HB_IDX(at(r), ns - V + 1));
                }
            }
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
                const int r = r0 + i * RG;
                if (on && r < a.dk) {
                    if (g0 == 0) {
                        const float kr = ks[r];
#pragma unroll
                        for (int j = 0; j < V; ++j) s[i].x[j] = fmaf(g, s[i].x[j], kr * vv[j]);
                        if (HB_OK(at(r) + V - 1, ns)) s[i].store(S + at(r));
                    }
#pragma unroll
                    for (int h = 0; h < GT; ++h)
                        if (GT == 1 || h < ng) {
                            const float qr = qs[h][r];
#pragma unroll
                            for (int j = 0; j < V; ++j) acc[h][j] = fmaf(qr, s[i].x[j], acc[h][j]);
                        }
                }
            }
        }
        // sum the row groups: those of a warp by shuffles, the warps through shared memory (a fixed order)
#pragma unroll
        for (int h = 0; h < GT; ++h)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                float x = acc[h][j];
#pragma unroll
                for (int m = 16; m >= CT; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
                if (lane < CT) red[warp][h][lane * V + j] = x;
            }
        __syncthreads();
        T *o = static_cast<T *>(a.o);
        for (int i = tid; i < ng * CS; i += kThreads) {
            const int h = i / CS, cc = i % CS;
            if (sl * CS + cc < a.dv) {
                float x = 0.f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) x += red[w][h][cc];
                const long long oi = ((long long)b * a.H + (long long)hk * G + g0 + h) * a.dv + sl * CS + cc;
                if (HB_OK(oi, (long long)a.B * a.H * a.dv)) Act::st(o + oi, a.scale * x);
            }
        }
        if (g0 + GT < G) __syncthreads();      // qs and red are written again
    }
}

template <class Act, int V, int CT>
cudaError_t launch_g(const DecArgs &a, unsigned grid, cudaStream_t s) {
    const int G = a.H / a.Hk;
    if (G == 1) linattn_decode_kernel<Act, V, CT, 1><<<grid, kThreads, 0, s>>>(a);
    else if (G <= 4) linattn_decode_kernel<Act, V, CT, 4><<<grid, kThreads, 0, s>>>(a);
    else linattn_decode_kernel<Act, V, CT, 8><<<grid, kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

template <class Act>
cudaError_t launch_t(DecArgs &a, cudaStream_t s) {
    const long long units = (long long)a.B * a.Hk;
    auto grid = [&](int cs) -> long long { a.slices = (a.dv + cs - 1) / cs; return units * a.slices; };
    long long n;
    if (a.dv % 4) return (n = grid(32)) > 0x7fffffffll ? cudaErrorInvalidValue : launch_g<Act, 1, 32>(a, (unsigned)n, s);
    // 128-column slices stream best; narrower ones where those would leave SMs idle
    if ((n = grid(128)) >= 2 * 148) return n > 0x7fffffffll ? cudaErrorInvalidValue : launch_g<Act, 4, 32>(a, (unsigned)n, s);
    if ((n = grid(64)) >= 2 * 148) return launch_g<Act, 4, 16>(a, (unsigned)n, s);
    return launch_g<Act, 4, 8>(a, (unsigned)grid(32), s);
}

}  // namespace

HYENA_BOUNDS_READER(linattn_decode)

cudaError_t launch_linattn_decode(const void *q, const void *k, const void *v, int dtype, int B, int H, int Hk, int dk,
                                  int dv, long long ldq, long long ldk, long long ldv, const float *decay, float scale,
                                  const hyena_qk_prep *p, const int *pos, int pos0, float *state, void *o,
                                  cudaStream_t s) {
    DecArgs a{};
    a.q = q; a.k = k; a.v = v; a.o = o; a.state = state; a.decay = decay; a.scale = scale;
    a.B = B; a.H = H; a.Hk = Hk; a.dk = dk; a.dv = dv;
    a.ldq = ldq; a.ldk = ldk; a.ldv = ldv;
    a.prep = p != nullptr;
    if (p) a.p = QKPrepArgs{p->norm, p->eps, p->q_weight, p->k_weight, p->rot_dim, p->inv_freq, p->interleaved};
    a.pos = pos; a.pos0 = pos0;
    return dtype == HYENA_BF16 ? launch_t<ActBF16>(a, s) : launch_t<ActF32>(a, s);
}

}  // namespace hyena
