// linattn.cu -- linear attention with a decay for each head over a prompt: the CUDA-core route, the
// split of long prompts into segments (both routes), and the launcher.
//
// Mathematics, for a block of T tokens with entering state S (g the head's decay):
//   o_t = scale (g^(t+1) S^T q_t + sum_{j<=t} g^(t-j) (q_t . k_j) v_j),   t = 0..T-1
//   S  <- g^T S + sum_j g^(T-1-j) k_j v_j^T
// This is an exact regrouping of S <- g S + k v^T, o = scale S^T q; every weight is a power of g
// between 0 and 1, so nothing overflows for any decay in [0, 1].
//
// The block form takes 2 dk dv multiply-adds per token (output and update) plus 1/T of that for the
// decay, against 3 dk dv operations for the token-by-token form.  A thread block owns 64 columns of
// one state, held in registers: warp w keeps the rows [w RK, (w+1) RK), a lane two columns, so q and k
// are read from shared memory as broadcasts (one 16-byte read feeds 8 multiply-adds).
#include "linattn.cuh"

namespace hyena {

namespace {

constexpr int kThreads = 256, kWarps = 8;
constexpr int kT = 8;            // tokens of a block
constexpr int kTV = 64;          // state columns of a thread block

template <class Act, int RK>
__global__ void __launch_bounds__(kThreads, 2) linattn_kernel(const LinArgs a, int states_only) {
    using T = typename Act::T;
    constexpr int DKP = kWarps * RK;             // dk, padded with zeros
    constexpr int LD = DKP + 16;                 // row stride: rows of the score products fall into different banks
    constexpr int KI = kT * DKP / kThreads, VI = kT * kTV / kThreads;
    __shared__ __align__(16) float qs[kT][LD], ks[kT][LD];
    __shared__ float vs[kT][kTV], sc[kT][kT], pw[kT + 1];
    __shared__ float red[kWarps][kT][kTV];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    long long id = blockIdx.x;
    const int vt = (int)(id % a.vtiles);
    id /= a.vtiles;
    const int hk = (int)(id % a.Hk);
    id /= a.Hk;
    const int b = (int)(id % a.B), seg = (int)(id / a.B);
    const int G = a.H / a.Hk, c0 = vt * kTV;
    const int len = row_tokens(a, b);
    const int t_beg = min(len, seg * a.seg_tokens), t_end = min((long long)len, (long long)t_beg + a.seg_tokens);
    const double g = (double)a.decay[HB_IDX(hk, a.Hk)];
    const long long unit = (long long)b * a.Hk + hk, ns = (long long)a.B * a.Hk * a.dk * a.dv;
    (void)ns;
    const T *q = static_cast<const T *>(a.q), *k = static_cast<const T *>(a.k), *v = static_cast<const T *>(a.v);
    const long long row0 = (long long)b * a.L;
    const long long rows = (long long)a.B * a.L - 1;
    const long long nk = rows * a.ldk + (long long)a.Hk * a.dk, nv = rows * a.ldv + (long long)a.Hk * a.dv,
                    nq = rows * a.ldq + (long long)a.H * a.dk;
    (void)nk; (void)nv; (void)nq;
    if (tid <= kT) pw[tid] = (float)decay_pow(g, tid);

    // this thread's part of the state: rows warp * RK + i, columns c0 + lane, c0 + lane + 32
    float S0[RK], S1[RK];
    const float *init = states_only || !a.init ? nullptr : a.init + (long long)seg * a.init_stride;
#pragma unroll
    for (int i = 0; i < RK; ++i) {
        const int r = warp * RK + i;
        const long long x = (unit * a.dk + r) * a.dv + c0 + lane;
        S0[i] = init && r < a.dk && c0 + lane < a.dv ? init[HB_IDX(x, ns)] : 0.f;
        S1[i] = init && r < a.dk && c0 + lane + 32 < a.dv ? init[HB_IDX(x + 32, ns)] : 0.f;
    }

    // tokens t .. t + kT - 1 of k and v, one block ahead in registers
    float kr[KI], vr[VI], qr[KI];
    auto fetch_kv = [&](int t) {
#pragma unroll
        for (int i = 0; i < KI; ++i) {
            const int e = tid + i * kThreads, j = e / DKP, r = e % DKP;
            kr[i] = t + j < t_end && r < a.dk ? Act::ld(k + HB_IDX((row0 + t + j) * a.ldk + (long long)hk * a.dk + r, nk)) : 0.f;
        }
#pragma unroll
        for (int i = 0; i < VI; ++i) {
            const int e = tid + i * kThreads, j = e / kTV, c = e % kTV;
            vr[i] = t + j < t_end && c0 + c < a.dv ? Act::ld(v + HB_IDX((row0 + t + j) * a.ldv + (long long)hk * a.dv + c0 + c, nv)) : 0.f;
        }
    };
    auto fetch_q = [&](int t, int h) {
#pragma unroll
        for (int i = 0; i < KI; ++i) {
            const int e = tid + i * kThreads, j = e / DKP, r = e % DKP;
            qr[i] = t + j < t_end && r < a.dk ? Act::ld(q + HB_IDX((row0 + t + j) * a.ldq + (long long)h * a.dk + r, nq)) : 0.f;
        }
    };
    if (t_beg < t_end) {
        fetch_kv(t_beg);
        if (!states_only) fetch_q(t_beg, hk * G);
    }
    for (int t = t_beg; t < t_end; t += kT) {
        const int n = min(kT, t_end - t);
        __syncthreads();              // the last block's reads are done
#pragma unroll
        for (int i = 0; i < KI; ++i) {
            const int e = tid + i * kThreads;
            ks[e / DKP][e % DKP] = kr[i];
            if (!states_only) qs[e / DKP][e % DKP] = qr[i];
        }
#pragma unroll
        for (int i = 0; i < VI; ++i) {
            const int e = tid + i * kThreads;
            vs[e / kTV][e % kTV] = vr[i];
        }
        __syncthreads();
        if (t + kT < t_end) fetch_kv(t + kT);
        if (!states_only) {
            for (int x = 0; x < G; ++x) {
                if (x + 1 < G) fetch_q(t, hk * G + x + 1);
                else if (t + kT < t_end) fetch_q(t + kT, hk * G);
                {   // scores: four threads per (t, j) pair
                    const int i = tid >> 5, j = (tid >> 2) & 7, u = tid & 3;
                    float d = 0.f;
                    if (j <= i) {
#pragma unroll
                        for (int r = 4 * u; r < DKP; r += 16) {
                            const float4 x4 = *reinterpret_cast<const float4 *>(&qs[i][r]);
                            const float4 y4 = *reinterpret_cast<const float4 *>(&ks[j][r]);
                            d = fmaf(x4.x, y4.x, fmaf(x4.y, y4.y, fmaf(x4.z, y4.z, fmaf(x4.w, y4.w, d))));
                        }
                    }
                    d += __shfl_xor_sync(0xffffffffu, d, 1);
                    d += __shfl_xor_sync(0xffffffffu, d, 2);
                    if (u == 0) sc[i][j] = j <= i ? d * pw[i - j] : 0.f;
                }
                // this warp's rows of S^T q
#pragma unroll
                for (int i = 0; i < kT; ++i) {
                    float o0 = 0.f, o1 = 0.f;
#pragma unroll
                    for (int r = 0; r < RK; r += 4) {
                        const float4 x4 = *reinterpret_cast<const float4 *>(&qs[i][warp * RK + r]);
                        o0 = fmaf(x4.x, S0[r], fmaf(x4.y, S0[r + 1], fmaf(x4.z, S0[r + 2], fmaf(x4.w, S0[r + 3], o0))));
                        o1 = fmaf(x4.x, S1[r], fmaf(x4.y, S1[r + 1], fmaf(x4.z, S1[r + 2], fmaf(x4.w, S1[r + 3], o1))));
                    }
                    red[warp][i][lane] = o0;
                    red[warp][i][lane + 32] = o1;
                }
                __syncthreads();
#pragma unroll
                for (int y = 0; y < kT * kTV / kThreads; ++y) {
                    const int e = tid + y * kThreads, i = e / kTV, c = e % kTV;
                    if (i < n && c0 + c < a.dv) {
                        float acc = 0.f;
#pragma unroll
                        for (int w = 0; w < kWarps; ++w) acc += red[w][i][c];
                        acc *= pw[i + 1];
#pragma unroll
                        for (int j = 0; j < kT; ++j)
                            if (j <= i) acc = fmaf(sc[i][j], vs[j][c], acc);
                        const long long oi = ((row0 + t + i) * a.H + hk * G + x) * a.dv + c0 + c;
                        if (HB_OK(oi, (rows + 1) * a.H * a.dv)) Act::st(static_cast<T *>(a.o) + oi, a.scale * acc);
                    }
                }
                if (x + 1 < G) {
                    __syncthreads();
#pragma unroll
                    for (int i = 0; i < KI; ++i) {
                        const int e = tid + i * kThreads;
                        qs[e / DKP][e % DKP] = qr[i];
                    }
                    __syncthreads();
                }
            }
        }
        // the state after the block
        const float gn = pw[n];
#pragma unroll
        for (int i = 0; i < RK; ++i) {
            S0[i] *= gn;
            S1[i] *= gn;
        }
#pragma unroll
        for (int j = 0; j < kT; ++j) {
            if (j < n) {
                const float w = pw[n - 1 - j], v0 = w * vs[j][lane], v1 = w * vs[j][lane + 32];
#pragma unroll
                for (int r = 0; r < RK; r += 4) {
                    const float4 x4 = *reinterpret_cast<const float4 *>(&ks[j][warp * RK + r]);
                    S0[r] = fmaf(x4.x, v0, S0[r]);
                    S0[r + 1] = fmaf(x4.y, v0, S0[r + 1]);
                    S0[r + 2] = fmaf(x4.z, v0, S0[r + 2]);
                    S0[r + 3] = fmaf(x4.w, v0, S0[r + 3]);
                    S1[r] = fmaf(x4.x, v1, S1[r]);
                    S1[r + 1] = fmaf(x4.y, v1, S1[r + 1]);
                    S1[r + 2] = fmaf(x4.z, v1, S1[r + 2]);
                    S1[r + 3] = fmaf(x4.w, v1, S1[r + 3]);
                }
            }
        }
    }
    // this route has no waits: its error words are 0
    for (long long i = (long long)blockIdx.x * kThreads + tid; i < a.nerr; i += (long long)gridDim.x * kThreads) a.err[HB_IDX(i, a.nerr)] = 0;
    float *dst = states_only ? a.states + (long long)(seg + 1) * a.init_stride : seg == a.nseg - 1 ? a.state_out : nullptr;
    if (dst) {
#pragma unroll
        for (int i = 0; i < RK; ++i) {
            const int r = warp * RK + i;
            const long long x = (unit * a.dk + r) * a.dv + c0 + lane;
            if (r < a.dk && c0 + lane < a.dv && HB_OK(x, ns)) dst[x] = S0[i];
            if (r < a.dk && c0 + lane + 32 < a.dv && HB_OK(x + 32, ns)) dst[x + 32] = S1[i];
        }
    }
}

// The states entering the segments, in place over the segments' contributions: slot 0 becomes
// state_in (or zero), slot s + 1 becomes g^(tokens of segment s) * slot s + its contribution.
// A thread carries V neighbouring entries through the segments, kAhead contributions in flight.
constexpr int kStateThreads = 64, kAhead = 8;

template <int V>
__global__ void __launch_bounds__(kStateThreads) linattn_states_kernel(float *states, const float *state_in, long long n,
                                                                       long long per_head, int Hk, int L, int B, int nseg,
                                                                       int seg_tokens, const float *decay, const int *lens) {
    struct alignas(4 * V) Vec { float x[V]; };
    const long long i = ((long long)blockIdx.x * kStateThreads + threadIdx.x) * V;
    if (i >= n) return;
    const long long unit = i / per_head;
    const int hk = (int)(unit % Hk), b = (int)(unit / Hk);
    const double g = (double)decay[HB_IDX(hk, Hk)];
    const float whole = (float)decay_pow(g, seg_tokens);
    const int len = lens ? min(max(lens[HB_IDX(b, B)], 0), L) : L;
    auto at = [&](int s) { return reinterpret_cast<Vec *>(states + HB_IDX(s * n + i + V - 1, n * nseg) - (V - 1)); };
    Vec x;
#pragma unroll
    for (int v = 0; v < V; ++v) x.x[v] = 0.f;
    if (state_in) x = *reinterpret_cast<const Vec *>(state_in + HB_IDX(i, n - V + 1));
    for (int s0 = 0; s0 + 1 < nseg; s0 += kAhead) {
        Vec c[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            if (s0 + k + 1 < nseg) c[k] = *at(s0 + k + 1);
        if (s0 == 0) *at(0) = x;
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int s = s0 + k;
            if (s + 1 >= nseg) break;
            const int m = min(max(len - s * seg_tokens, 0), seg_tokens);
            const float w = m == seg_tokens ? whole : (float)decay_pow(g, m);
#pragma unroll
            for (int v = 0; v < V; ++v) x.x[v] = fmaf(w, x.x[v], c[k].x[v]);
            *at(s + 1) = x;
        }
    }
}

// CUDA-core route: 64-column tiles; two blocks fit on an SM.
LinPlan simt_plan(int B, int L, int Hk, int dv) {
    LinPlan p{};
    p.vtiles = (dv + kTV - 1) / kTV;
    const long long units = B > 0 ? (long long)B * Hk * p.vtiles : 1;
    long long want = units >= 148 ? 1 : (2 * 148 + units - 1) / units;
    const int tiles = (L + 63) / 64;             // segments are multiples of 64 tokens
    if (want > tiles) want = tiles;
    if (want < 1) want = 1;
    const int segt = tiles > 0 ? (int)((tiles + want - 1) / want) : 1;
    p.seg_tokens = segt * 64;
    p.nseg = tiles > 0 ? (tiles + segt - 1) / segt : 1;
    return p;
}

size_t al256(size_t x) { return (x + 255) & ~size_t(255); }

template <class Act>
cudaError_t launch_simt(const LinArgs &a, bool states_only, cudaStream_t s) {
    const long long blocks = (long long)(states_only ? a.nseg - 1 : a.nseg) * a.B * a.Hk * a.vtiles;
    if (blocks > 0x7fffffffll) return cudaErrorInvalidValue;
    if (a.dk <= 64) linattn_kernel<Act, 8><<<(unsigned)blocks, kThreads, 0, s>>>(a, states_only);
    else if (a.dk <= 128) linattn_kernel<Act, 16><<<(unsigned)blocks, kThreads, 0, s>>>(a, states_only);
    else linattn_kernel<Act, 32><<<(unsigned)blocks, kThreads, 0, s>>>(a, states_only);
    return cudaGetLastError();
}

}  // namespace

HYENA_BOUNDS_READER(linattn)

bool linattn_uses_tc(int dtype, int L, int H, int Hk, int dk, int dv, long long ldq, long long ldk, long long ldv, const void *q,
                     const void *k, const void *v, const void *o) {
    auto ok = [](const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; };
    // A prompt of one block of tokens (kT) costs the CUDA cores less than the tensor cores' pipeline takes to fill:
    // 64 x 16 states of 128 x 128, carried, 8 tokens 52 us against 100, 16 tokens 85 against 101; 31 x 12 of 64 x 128 with 3
    // query heads each, 8 tokens 23 against 31 (16: 40); 200 x 8 of 128 x 128 with 4, 8 tokens 184 against 117.
    // (The rule does not ask whether a state is carried: without one the tensor cores took 44 for the first of these.)
    if (L <= kT && (long long)L * (H / Hk) <= 3 * kT) return false;
    return linattn_tc_dims(dtype, dk, dv) && ldq % 8 == 0 && ldk % 8 == 0 && ldv % 8 == 0 && ok(q) && ok(k) && ok(v) && ok(o);
}

// Workspace: [segment states][error words of the state pass][error words of the main pass].  The queries know
// neither strides nor pointers, so there is room for whichever route is taken.
size_t linattn_err_offset(int dtype, int B, int L, int H, int Hk, int dk, int dv) {
    int nseg = simt_plan(B, L, Hk, dv).nseg;
    if (linattn_tc_dims(dtype, dk, dv))
        nseg = max(nseg, max(linattn_tc_plan(B, L, H, Hk, dk, dv, false).nseg, linattn_tc_plan(B, L, H, Hk, dk, dv, true).nseg));
    return al256(nseg > 1 ? (size_t)nseg * B * Hk * dk * dv * sizeof(float) : 0);
}

size_t linattn_ws_bytes(int dtype, int B, int L, int H, int Hk, int dk, int dv) {
    return linattn_err_offset(dtype, B, L, H, Hk, dk, dv) + 2 * kLinMaxBlocks * sizeof(int);
}

cudaError_t launch_linattn_prefill(const void *q, const void *k, const void *v, int dtype, int B, int L, int H, int Hk,
                                   int dk, int dv, long long ldq, long long ldk, long long ldv, const float *decay,
                                   float scale, const int *lens, const float *state_in, void *o, float *state_out,
                                   void *ws, cudaStream_t s) {
    const bool tc = linattn_uses_tc(dtype, L, H, Hk, dk, dv, ldq, ldk, ldv, q, k, v, o);
    const LinPlan p = tc ? linattn_tc_plan(B, L, H, Hk, dk, dv, lens != nullptr) : simt_plan(B, L, Hk, dv);
    LinArgs a{};
    a.q = q; a.k = k; a.v = v; a.o = o;
    a.B = B; a.L = L; a.H = H; a.Hk = Hk; a.dk = dk; a.dv = dv;
    a.ldq = ldq; a.ldk = ldk; a.ldv = ldv;
    a.decay = decay; a.scale = scale; a.lens = lens;
    a.state_out = state_out;
    a.seg_tokens = p.seg_tokens; a.nseg = p.nseg; a.vtiles = p.vtiles; a.nv = p.nv;
    a.init_stride = (long long)B * Hk * dk * dv;
    a.states = static_cast<float *>(ws);
    int *err = reinterpret_cast<int *>(static_cast<char *>(ws) + linattn_err_offset(dtype, B, L, H, Hk, dk, dv));
    auto run = [&](bool states_only) {
        // both sets of words are written when there is no state pass
        a.err = states_only || p.nseg == 1 ? err : err + kLinMaxBlocks;
        a.nerr = p.nseg == 1 ? 2 * kLinMaxBlocks : kLinMaxBlocks;
        return tc ? launch_linattn_tc(a, states_only, s)
                  : dtype == HYENA_BF16 ? launch_simt<ActBF16>(a, states_only, s) : launch_simt<ActF32>(a, states_only, s);
    };
    if (p.nseg > 1) {
        cudaError_t e = run(true);
        if (e != cudaSuccess) return e;
        const int per = dv % 4 == 0 ? 4 * kStateThreads : kStateThreads;
        const long long blocks = (a.init_stride + per - 1) / per;
        if (blocks > 0x7fffffffll) return cudaErrorInvalidValue;
        auto combine = dv % 4 == 0 ? linattn_states_kernel<4> : linattn_states_kernel<1>;
        combine<<<(unsigned)blocks, kStateThreads, 0, s>>>(a.states, state_in, a.init_stride, (long long)dk * dv, Hk, L, B,
                                                           p.nseg, p.seg_tokens, decay, lens);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
        a.init = a.states;
    } else {
        a.init = state_in;
        a.init_stride = 0;
    }
    return run(false);
}

}  // namespace hyena
