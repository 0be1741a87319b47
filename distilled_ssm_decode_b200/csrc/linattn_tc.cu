// linattn_tc.cu -- linear attention with a decay for each head over a prompt, on the tensor cores.
//
// Per chunk of n <= C = 128 tokens with entering state S [dk][dv] (g the head's decay, i, j in the chunk):
//   A_ij = q_i . k_j                                           (scores)
//   P_ij = scale g^(i-j) A_ij for j <= i, else 0
//   O    = diag(scale g^(i+1)) (Q S) + P V
//   S    <- g^n S + sum_j (g^(n-1-j) k_j) v_j^T
// an exact regrouping of S <- g S + k v^T, o = scale S^T q.  All weights are powers of g in [0, 1].
//
// Four products per chunk, accumulated in fp32 in tensor memory:
//   scores  128 x 128 x dk   Q (shared) x K (shared)            -> columns kColP
//   Q S     128 x dv x dk    Q (shared) x S as bf16 (shared)    -> columns kColO, then scaled in place
//   P V     128 x dv x n     P as bf16 (tensor memory, over the scores) x V (shared), onto kColO
//   state   dk x dv x n      weighted keys (tensor memory) x V (shared), from zero -> kColU
// Roundings to bf16: the scores' P and the state's copy that multiplies q (operands only; both reach o, itself bf16: its error
// in the 2-norm is 2.3e-3 where one rounding of the exact value leaves 1.7e-3; a second term for each would double two products).
// The state itself stays fp32, in registers; its weighted keys enter as the sum of four bf16 terms, which keeps them to
// 2^-25: one term would leave 2^-9, two 2^-17 of each token in a state that every later token reads.  A chunk's
// contribution is summed from zero and joined by one fp32 multiply-add: summing onto the state in tensor memory
// cut off (the units truncate) at every product at the state's size, 1e-6 and more over a long prompt.
//
// Bound: 2 (dk + dv) (1 + 1) bytes per token and head of q, k, v, o against 2 C (dk + dv) + (2 + 8) dk dv operations:
// memory-bound (at dk = dv = 128 the products need 64% of the time that the bytes need), if the chain
// scores -> P -> P V -> o of a chunk overlaps the loads of the next and the state's own chain.  Hence one
// persistent block per SM (a chunk's tiles fill shared memory) with a role for each warp or warp group:
//   warp 0 loads K, V, Q; warp 1 stores O; warp 2 issues the products of the outputs, warp 3 those of the state
//   warps 4-7   P group: a token row per thread: scores -> P, scaling of Q S, then O -> shared memory
//   warps 8-11  K group: keys -> weighted keys, by ldmatrix and packed bf16 fma -> tensor memory
//   warps 12-19 S groups: half a row of the state per thread, in registers: its decay and sum, its bf16 copy
// They meet at mbarriers only.  Every wait is bounded; on timeout the block records it in its error word,
// drains its copies and products, frees tensor memory and returns.
//
// Measured (us of the launches alone, bf16): 64 sequences x 512 tokens x 16 heads of 128 x 128 138 (67% of measured HBM),
// 8 x 4096 x 8 heads 95 (44%), 65536 x 12 heads of 64 x 64 199 (31%: a second pass over K and V for the states).  What holds
// it there is the length of a chunk's chains, not a unit: tensor cores 39% busy, issue slots 45%; a chunk takes 5.0 us where
// its bytes take 3.0.  What was tried and not kept: the outputs by the S groups (their row of the state spills: 141 ->
// 160), sleeping waits (no change), scores and state rows loaded two pieces ahead (185: spills), the next head's
// powers computed ahead (142).
//
// Tensor-memory rows: tokens for the first three products, entries of k for the state.  With dk <= 64 the state's
// rows 64..127 hold what the unused lanes give; nothing reads them.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>

#include <atomic>

#include "linattn.cuh"
#include "tc.cuh"

namespace hyena {

namespace {

constexpr int kC = 128;                 // tokens of a chunk
constexpr int kThreads = 640;
constexpr int kBlk = kC * 128;          // bytes of a [128 tokens][64 entries] bf16 tile, 128-byte swizzled
constexpr uint32_t kColP = 0, kColO = 128, kColU = 256, kColW = 384;   // tensor-memory columns
constexpr uint32_t kTmemCols = 512;
constexpr int kTerms = 4;               // bf16 terms of a weighted key
// Decays of kUp and more: the sums are kept as O g^(127-i) / scale, so that P's factor g^(127-j) depends on the column
// alone and the state's copy takes the rest of Q S, g^128; the row's factor scale g^(i-127) comes in with the output's
// rounding.  No factor inside the sums is above 1, so nothing passes fp32's range that the formula keeps inside it; at the
// other end they are as small as g^127 > 2^-25, so that scores below 2^-101 count as 0.  Smaller decays would lose more
// there (0.75: scores below 2^-73): they scale P by rows and columns and Q S in place, which costs another pass over
// Q S.  us of the launches alone that way and this: 64 x 512 x 16 heads of 128 x 128 160 and 137, 8 x 4096 x 8 heads 131 and
// 100, 65536 x 12 heads of 64 x 64 240 and 207.
constexpr double kUp = 0.875;
constexpr int kSub = 32;                // tokens of weighted keys in one of two buffers
constexpr int kWBufs = 2, kWCols = kTerms * kSub / 2;
static_assert(kColW + kWBufs * kWCols <= kTmemCols, "tensor memory");

// Registers: the S groups hold half a row of the state in fp32.  The shares of the five warp groups must not exceed the
// launch's 5 x 96 (checked before the first launch: a larger sum would wait for ever).
constexpr int kRegsLaunch = 96;

struct Maps {
    CUtensorMap q, k, v, o;
};

template <int NK, int NV>
struct Geo {
    static constexpr int kKB = NK / 64, kVB = NV / 64, kNH = NV / 2;   // 64-entry blocks; columns of an S group
    static constexpr int kStage = (kKB + kVB) * kBlk;                  // K, then V
    static constexpr int kQSlot = (kKB > kVB ? kKB : kVB) * kBlk;      // Q, then O
    static constexpr int kStages = NK + NV == 256 ? 2 : NK + NV == 192 ? 3 : 4, kQSlots = NK + NV == 128 ? 4 : 2;
    static constexpr int kRegsMisc = NV == 128 ? 72 : 56, kRegsS = NV == 128 ? 104 : 112;
    static_assert(kRegsMisc + 2 * kRegsLaunch + 2 * kRegsS <= 5 * kRegsLaunch, "register shares");
    static constexpr int kSBytes = NK * NV * 2;
    static constexpr int kSmQ = kStages * kStage;
    static constexpr int kSmS = kSmQ + kQSlots * kQSlot;
    static constexpr int kSmPw = kSmS + kSBytes;                       // float pw[kC], PairWeights rw[kC / 2]
    static constexpr int kSmBar = kSmPw + 4 * kC + 16 * (kC / 2);
    enum { KVFull = 0, KVEmpty = KVFull + kStages, QFull = KVEmpty + kStages, QEmpty = QFull + kQSlots,
           OStaged = QEmpty + kQSlots, T1Done = OStaged + kQSlots, QSDone, PReady, VReady, T2Done = VReady + kStages, OFree, WReady, WFree = WReady + kWBufs,
           SReady = WFree + kWBufs, SFree, UDone, UFree, Drain, DrainU, PSync, KSync, SSync, kNumBars };
    static constexpr int kSmMisc = kSmBar + 8 * kNumBars;
    static constexpr int kSmem = kSmMisc + 16 + 1024;
    static_assert(kSmem <= 227 * 1024, "shared memory");
    static_assert(kSmBar % 8 == 0 && kSmS % 1024 == 0, "alignment");
    __host__ __device__ static constexpr int count(int b) {
        return b == SReady || b == UFree || b == SSync ? 8       // warps
               : (b >= OStaged && b < T1Done) || b == OFree || b == PReady || (b >= VReady && b < T2Done) || (b >= WReady && b < WFree) || b == PSync || b == KSync ? 4
               : b >= KVEmpty && b < QFull ? 2 : 1;
    }
};

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t *>(&p);
}

// f lo, f hi in fp32 (one packed multiply), then as bf16
__device__ __forceinline__ uint32_t pack2_scaled(float f, float lo, float hi) {
    float a, b;
    asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %4};\n\tmul.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "=f"(a), "=f"(b) : "f"(lo), "f"(hi), "f"(f));
    return pack2(a, b);
}

struct Item {
    int seg, b, hk, c0, t0, ntok, nck;      // first column, first token, tokens, chunks
};

__device__ __forceinline__ Item item_of(const LinArgs &a, int id, int nv) {
    Item it;
    it.c0 = (id % a.vtiles) * nv;
    id /= a.vtiles;
    it.hk = id % a.Hk;
    id /= a.Hk;
    it.b = id % a.B;
    it.seg = id / a.B;
    const int len = row_tokens(a, it.b);
    it.t0 = (int)min((long long)len, (long long)it.seg * a.seg_tokens);
    it.ntok = min(len - it.t0, a.seg_tokens);
    it.nck = (it.ntok + kC - 1) / kC;
    return it;
}

// w = w1 + w2 + w3 in bf16, for two tokens: |w - w1 - w2 - w3| <= 2^-27 |w|.
struct __align__(16) PairWeights {
    __nv_bfloat162 w1, w2, w3;
    uint32_t pad;
};
__device__ __forceinline__ PairWeights split_weights(float a, float b) {
    PairWeights p;
    p.w1 = __floats2bfloat162_rn(a, b);
    a -= __low2float(p.w1);
    b -= __high2float(p.w1);
    p.w2 = __floats2bfloat162_rn(a, b);
    p.w3 = __floats2bfloat162_rn(a - __low2float(p.w2), b - __high2float(p.w2));
    p.pad = 0;
    return p;
}

template <int NK, int NV>
__global__ void __launch_bounds__(kThreads, 1)
linattn_tc_kernel(const __grid_constant__ Maps m, const LinArgs a, const int items, const int states_only) {
    using G = Geo<NK, NV>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = tc::smem_u32(sm);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    float *pw = reinterpret_cast<float *>(sm + G::kSmPw);            // pw[x] = g^x, or g^(127 - x) (the P group's)
    PairWeights *rw = reinterpret_cast<PairWeights *>(pw + kC);      // rw[x]: g^(n - 1 - 2 x), g^(n - 2 - 2 x) (the K group's)
    volatile int *misc = reinterpret_cast<volatile int *>(sm + G::kSmMisc);   // abort (= error code), tensor memory, never
    volatile int *abort = misc, *never = misc + 2;
    auto bar = [&](int b) { return sbase + G::kSmBar + 8u * b; };
    const int Gq = a.H / a.Hk;

    if (tid == 0) {
        misc[0] = 0;
        misc[2] = 0;
        // without queries the K and the P group both weigh keys
        for (int i = 0; i < G::kNumBars; ++i)
            tc::mbar_init(bar(i), states_only && (i == G::KSync || (i >= G::VReady && i < G::T2Done)) ? 8 : G::count(i));
        tc::fence_mbar_init();
    } else if (tid == 32) {
        tc::prefetch_tensormap(&m.q);
        tc::prefetch_tensormap(&m.k);
        tc::prefetch_tensormap(&m.v);
        tc::prefetch_tensormap(&m.o);
    }
    if (warp == 2) {
        tc::tmem_alloc(tc::smem_u32((const void *)(misc + 1)), kTmemCols);
        tc::tmem_relinquish();
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = (uint32_t)misc[1];
    auto uni = [&](bool x) -> bool { return __all_sync(0xffffffffu, x); };
    // one arrival for each warp of a group (32 arrivals of a warp would be serialised)
    auto arrive = [&](int b) {
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(bar(b));
    };

    // the warps of a group meet (bounded, as every wait here); `n` counts the meetings
    auto meet = [&](int b, int &n) -> bool {
        arrive(b);
        return uni(tc::mbar_wait(bar(b), n++ & 1, abort));
    };
    // one query tile's outputs: tensor memory -> bf16 -> shared memory (whole chunks, stored by warp 1) or o
    auto outputs = [&](const Item &it, int c, int x, int qc, float f, int row, uint32_t lane_base) -> bool {
        if (!uni(tc::mbar_wait(bar(G::T2Done), qc & 1, abort))) return false;
        tc::tc_fence_after();
        const int s = qc % G::kQSlots, n = min(kC, it.ntok - c * kC);
        uint8_t *ob = sm + G::kSmQ + s * G::kQSlot + row * 128;
        const long long at = (((long long)it.b * a.L + it.t0 + c * kC + row) * a.H + it.hk * Gq + x) * a.dv + it.c0;
#pragma unroll 1
        for (int p = 0; p < NV / 32; ++p) {
            float z[32];
            tc::tmem_ld32(lane_base + kColO + 32 * p, z);
            tc::tmem_wait_ld();
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const float *t = z + 8 * y;
                const uint4 v4 = make_uint4(pack2(f * t[0], f * t[1]), pack2(f * t[2], f * t[3]),
                                            pack2(f * t[4], f * t[5]), pack2(f * t[6], f * t[7]));
                const int ch = 4 * p + y;               // 16-byte piece of the row
                if (n == kC)
                    *reinterpret_cast<uint4 *>(ob + (ch / 8) * kBlk + (((ch & 7) ^ (row & 7)) << 4)) = v4;
                else if (row < n && it.c0 + 8 * ch < a.dv &&
                         HB_OK(at + 8 * ch + 7, (long long)a.B * a.L * a.H * a.dv))
                    *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.o) + at + 8 * ch) = v4;
            }
        }
        tc::tc_fence_before();
        arrive(G::OFree);
        tc::fence_proxy_async_smem();
        arrive(G::OStaged + s);
        return true;
    };

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(G::kRegsMisc));
        if (warp == 0) {
            // ------------------------------------------------------------ loads
            // K and V of the next chunk go out right behind the first queries of this one
            if (lane == 0) {
                int cc = 0, qc = 0, kv_id = blockIdx.x, kv_c = 0;
                Item kv{};
                if (kv_id < items) kv = item_of(a, kv_id, NV);
                bool ok = true;
                auto load_kv = [&]() {
                    while (kv_id < items && kv_c >= kv.nck) {
                        kv_id += gridDim.x;
                        kv_c = 0;
                        if (kv_id < items) kv = item_of(a, kv_id, NV);
                    }
                    if (kv_id >= items) return;
                    const int st = cc % G::kStages, t = kv.t0 + kv_c * kC;
                    if (!(ok = ok && tc::mbar_wait(bar(G::KVEmpty + st), ((cc / G::kStages) & 1) ^ 1, abort))) return;
                    const uint32_t dst = sbase + st * G::kStage;
                    tc::mbar_expect_tx(bar(G::KVFull + st), G::kStage);
                    for (int x = 0; x < G::kKB; ++x) tc::tma_load_4d(dst + x * kBlk, &m.k, bar(G::KVFull + st), 64 * x, kv.hk, t, kv.b);
                    for (int x = 0; x < G::kVB; ++x)
                        tc::tma_load_4d(dst + (G::kKB + x) * kBlk, &m.v, bar(G::KVFull + st), kv.c0 + 64 * x, kv.hk, t, kv.b);
                    ++cc;
                    ++kv_c;
                };
                load_kv();
                for (int id = blockIdx.x; id < items && ok; id += gridDim.x) {
                    const Item it = item_of(a, id, NV);
                    for (int c = 0; c < it.nck && ok; ++c) {
                        for (int x = 0; x < Gq && ok && !states_only; ++x, ++qc) {
                            const int s = qc % G::kQSlots;
                            if (!(ok = tc::mbar_wait(bar(G::QEmpty + s), ((qc / G::kQSlots) & 1) ^ 1, abort))) break;
                            tc::mbar_expect_tx(bar(G::QFull + s), G::kKB * kBlk);
                            for (int y = 0; y < G::kKB; ++y)
                                tc::tma_load_4d(sbase + G::kSmQ + s * G::kQSlot + y * kBlk, &m.q, bar(G::QFull + s), 64 * y,
                                                it.hk * Gq + x, it.t0 + c * kC, it.b);
                            if (x == 0) load_kv();
                        }
                        if (states_only) load_kv();
                    }
                }
                if (!ok) *abort = 1;
                // No copy may be in flight when the block leaves: another role's wait can run out after this one has issued
                // its last copies, so they are waited for here either way (without a timeout each has a consumer that
                // needs it before the block can end, so this costs nothing).
                for (int j = max(0, cc - G::kStages); j < cc; ++j)
                    tc::mbar_wait(bar(G::KVFull + j % G::kStages), (j / G::kStages) & 1, never);
                for (int j = max(0, qc - G::kQSlots); j < qc; ++j)
                    tc::mbar_wait(bar(G::QFull + j % G::kQSlots), (j / G::kQSlots) & 1, never);
            }
        } else if (warp == 1) {
            // ------------------------------------------------------------ O stores (whole chunks)
            if (lane == 0 && !states_only) {
                int qc = 0;
                bool ok = true;
                for (int id = blockIdx.x; id < items && ok; id += gridDim.x) {
                    const Item it = item_of(a, id, NV);
                    for (int c = 0; c < it.nck && ok; ++c)
                        for (int x = 0; x < Gq; ++x, ++qc) {
                            const int s = qc % G::kQSlots;
                            if (!(ok = tc::mbar_wait(bar(G::OStaged + s), (qc / G::kQSlots) & 1, abort))) break;
                            if (it.ntok - c * kC >= kC)
                                for (int y = 0; y < G::kVB; ++y)
                                    if (it.c0 + 64 * y < a.dv)
                                        tc::tma_store_4d(&m.o, sbase + G::kSmQ + s * G::kQSlot + y * kBlk, it.c0 + 64 * y,
                                                         it.hk * Gq + x, it.t0 + c * kC, it.b);
                            tc::bulk_commit();
                            tc::bulk_wait_read<0>();
                            tc::mbar_arrive(bar(G::QEmpty + s));
                        }
                }
                if (!ok) *abort = 1;
                tc::bulk_wait<0>();
            }
        } else if (warp == 2) {
            // ------------------------------------------------------------ products of the outputs
            // the scores of the next query tile go out as soon as P V of this one has read P, while the outputs are stored
            if (tc::elect_one()) {
                int cc = 0, qc = 0, sc = 0, id = blockIdx.x, c = 0, x = 0;
                bool ok = true;
                const uint32_t id_score = tc::idesc_bf16(128, 128, false), id_v = tc::idesc_bf16(128, NV, true);
                const uint32_t s_lo = tc::sw128_desc_lo(sbase + G::kSmS, NK * 128);
                auto wait = [&](int b, int phase) { return ok = ok && tc::mbar_wait(bar(b), phase & 1, abort); };
                Item it{};
                auto settle = [&]() {
                    for (; id < items; id += gridDim.x) {
                        it = item_of(a, id, NV);
                        if (it.nck > 0) return true;
                    }
                    return false;
                };
                auto q_at = [&]() { return tc::sw128_desc_lo(sbase + G::kSmQ + (qc % G::kQSlots) * G::kQSlot, 16); };
                bool live = settle();
                if (states_only) {
                    // the stage's second arrival (the first is the state's warp's), once both groups that weigh keys have
                    // passed it: one of them may have no piece of this chunk
                    for (; live && ok; ++cc) {
                        if (!wait(G::VReady + cc % G::kStages, cc / G::kStages)) break;
                        tc::mma_commit(bar(G::KVEmpty + cc % G::kStages));
                        if (++c == it.nck) {
                            c = 0;
                            id += gridDim.x;
                            live = settle();
                        }
                    }
                    live = false;
                }
                for (bool first = true; live && ok; first = false) {
                    const int st = cc % G::kStages;
                    if (!first && !wait(G::T2Done, qc - 1)) break;
                    if ((x == 0 && !wait(G::KVFull + st, cc / G::kStages)) || !wait(G::QFull + qc % G::kQSlots, qc / G::kQSlots)) break;
                    tc::tc_fence_after();
                    const uint32_t q_lo = q_at(), k_lo = tc::sw128_desc_lo(sbase + st * G::kStage, 16);
#pragma unroll
                    for (int kb = 0; kb < G::kKB; ++kb)
#pragma unroll
                        for (int ks = 0; ks < 4; ++ks) {
                            const uint32_t off = kb * (kBlk >> 4) + ks * 2;
                            tc::mma_bf16_sw128(tmem + kColP, q_lo + off, k_lo + off, id_score, kb + ks > 0);
                        }
                    tc::mma_commit(bar(G::T1Done));
                    const bool has_state = c > 0 || a.init;
                    if (has_state && x == 0 && !wait(G::SReady, sc++)) break;
                    if (!wait(G::OFree, qc + 1)) break;
                    tc::tc_fence_after();
                    if (has_state) {
#pragma unroll
                        for (int kb = 0; kb < G::kKB; ++kb)
#pragma unroll
                            for (int ks = 0; ks < 4; ++ks)
                                tc::mma_bf16_sw128(tmem + kColO, q_lo + kb * (kBlk >> 4) + ks * 2,
                                                   s_lo + (4 * kb + ks) * (2048 >> 4), id_v, kb + ks > 0);
                    }
                    tc::mma_commit(bar(G::QSDone));
                    if (has_state && x == Gq - 1) tc::mma_commit(bar(G::SFree));
                    if (!wait(G::PReady, qc) || (x == 0 && !wait(G::VReady + st, cc / G::kStages))) break;
                    tc::tc_fence_after();
                    const uint32_t v_lo = tc::sw128_desc_lo(sbase + st * G::kStage + G::kKB * kBlk, kBlk);
                    const int steps = (min(kC, it.ntok - c * kC) + 15) / 16;
#pragma unroll
                    for (int ks = 0; ks < kC / 16; ++ks)
                        if (ks < steps) tc::mma_bf16_ta_sw128(tmem + kColO, tmem + kColP + 8 * ks, v_lo + ks * (2048 >> 4), id_v,
                                              has_state || ks > 0);
                    tc::mma_commit(bar(G::T2Done));
                    ++qc;
                    if (++x == Gq) {
                        tc::mma_commit(bar(G::KVEmpty + st));
                        x = 0;
                        ++cc;
                        if (++c == it.nck) {
                            c = 0;
                            id += gridDim.x;
                            live = settle();
                        }
                    }
                }
                if (!ok) *abort = 1;
                tc::mma_commit(bar(G::Drain));
                tc::mbar_wait(bar(G::Drain), 0, never);
            }
        } else {
            // ------------------------------------------------------------ products of the state
            // the chunk's own contribution, from zero: kSub tokens of weighted keys at a time
            if (tc::elect_one()) {
                int cc = 0, wc = 0;
                bool ok = true;
                const uint32_t id_v = tc::idesc_bf16(128, NV, true);
                auto wait = [&](int b, int phase) { return ok = ok && tc::mbar_wait(bar(b), phase & 1, abort); };
                for (int id = blockIdx.x; id < items && ok; id += gridDim.x) {
                    const Item it = item_of(a, id, NV);
                    for (int c = 0; c < it.nck && ok; ++c, ++cc) {
                        const int st = cc % G::kStages, n = min(kC, it.ntok - c * kC), steps = (n + 15) / 16;
                        const uint32_t v_lo = tc::sw128_desc_lo(sbase + st * G::kStage + G::kKB * kBlk, kBlk);
                        if (!wait(G::KVFull + st, cc / G::kStages) || !wait(G::UFree, cc + 1)) break;
                        for (int h = 0; h * kSub < n; ++h, ++wc) {
                            const int wb = wc % kWBufs;
                            if (!wait(G::WReady + wb, wc / kWBufs)) break;
                            tc::tc_fence_after();
#pragma unroll
                            for (int ks = 0; ks < kSub / 16; ++ks)
                                if (h * (kSub / 16) + ks < steps)
#pragma unroll
                                    for (int t = 0; t < kTerms; ++t)
                                        tc::mma_bf16_ta_sw128(tmem + kColU, tmem + kColW + wb * kWCols + (kSub / 2) * t + 8 * ks,
                                                              v_lo + (h * (kSub / 16) + ks) * (2048 >> 4), id_v,
                                                              h > 0 || ks > 0 || t > 0);
                            tc::mma_commit(bar(G::WFree + wb));
                        }
                        if (!ok) break;
                        if (!a.hold || blockIdx.x != 0) tc::mma_commit(bar(G::UDone));
                        tc::mma_commit(bar(G::KVEmpty + st));
                    }
                }
                if (!ok) *abort = 1;
                tc::mma_commit(bar(G::DrainU));
                tc::mbar_wait(bar(G::DrainU), 0, never);
            }
        }
    } else if (warp < 8 && !states_only) {
        // ------------------------------------------------------------ P group
        const int w = warp & 3, row = 32 * w + lane;
        const uint32_t lane_base = tmem + ((uint32_t)(32 * w) << 16);
        int qc = 0, hk_cur = -1, met = 0;
        float f_row = 0.f;          // scale g^(i+1) of this row, or scale g^(i-127)
        bool up = false, ok = true;
        for (int id = blockIdx.x; id < items && ok; id += gridDim.x) {
            const Item it = item_of(a, id, NV);
            // the head's powers (this group writes its own table for itself)
            if (it.hk != hk_cur && it.nck > 0) {
                if (!(ok = meet(G::PSync, met))) break;
                const double g = (double)a.decay[HB_IDX(it.hk, a.Hk)];
                up = g >= kUp;
                pw[row] = (float)decay_pow(g, up ? kC - 1 - row : row);
                f_row = a.scale * (float)(up ? decay_pow(1.0 / g, kC - 1 - row) : decay_pow(g, row + 1));
                if (!(ok = meet(G::PSync, met))) break;
                hk_cur = it.hk;
            }
            for (int c = 0; c < it.nck && ok; ++c) {
                const int n = min(kC, it.ntok - c * kC);
                const bool has_state = c > 0 || a.init;
                for (int x = 0; x < Gq; ++x, ++qc) {
                    if (!(ok = uni(tc::mbar_wait(bar(G::T1Done), qc & 1, abort)))) break;
                    tc::tc_fence_after();
#pragma unroll 1
                    for (int p = 0; 32 * p < n; ++p) {
                        uint32_t out[16];
                        if (p > w) {
#pragma unroll
                            for (int j = 0; j < 16; ++j) out[j] = 0;      // later tokens
                        } else {
                            float z[32];
                            tc::tmem_ld32(lane_base + kColP + 32 * p, z);
                            tc::tmem_wait_ld();
                            if (up) {
#pragma unroll
                                for (int j = 0; j < 32; j += 4) {
                                    const float4 r4 = *reinterpret_cast<const float4 *>(pw + 32 * p + j);
                                    z[j] *= r4.x; z[j + 1] *= r4.y; z[j + 2] *= r4.z; z[j + 3] *= r4.w;
                                }
                            } else {
#pragma unroll
                                for (int j = 0; j < 32; ++j) z[j] *= a.scale * pw[max(row - 32 * p - j, 0)];
                            }
                            if (p == w) {
#pragma unroll
                                for (int j = 0; j < 32; ++j) z[j] = j <= lane ? z[j] : 0.f;
                            }
#pragma unroll
                            for (int j = 0; j < 16; ++j) out[j] = pack2(z[2 * j], z[2 * j + 1]);
                        }
                        tc::tmem_st16(lane_base + kColP + 16 * p, out);
                    }
                    if (has_state && !up) {
                        if (!(ok = uni(tc::mbar_wait(bar(G::QSDone), qc & 1, abort)))) break;
                        tc::tc_fence_after();
#pragma unroll 1
                        for (int p = 0; p < NV / 32; ++p) {
                            float z[32];
                            tc::tmem_ld32(lane_base + kColO + 32 * p, z);
                            tc::tmem_wait_ld();
                            uint32_t out[32];
#pragma unroll
                            for (int j = 0; j < 32; ++j) out[j] = __float_as_uint(f_row * z[j]);
                            tc::tmem_st32(lane_base + kColO + 32 * p, out);
                        }
                    }
                    tc::tmem_wait_st();
                    tc::tc_fence_before();
                    arrive(G::PReady);
                    if (!(ok = outputs(it, c, x, qc, up ? f_row : 1.f, row, lane_base))) break;
                }
            }
        }
        if (!ok) {
            *abort = 1;
            tc::tmem_wait_st();         // scores may be on their way to tensor memory, which is freed below
        }
    } else if (warp < 12) {
        // ------------------------------------------------------------ K group
        // without queries the P group weighs every other piece of keys
        const int w = warp & 3, d = 32 * w + lane, kg = warp < 8 ? 1 : 0;
        const uint32_t lane_base = tmem + ((uint32_t)(32 * w) << 16);
        int cc = 0, wc = 0, hk_cur = -1, n_cur = 0, met = 0;         // the table's head and chunk length
        bool ok = true;
        for (int id = blockIdx.x; id < items && ok; id += gridDim.x) {
            const Item it = item_of(a, id, NV);
            for (int c = 0; c < it.nck && ok; ++c, ++cc) {
                const int st = cc % G::kStages, n = min(kC, it.ntok - c * kC);
                if (it.hk != hk_cur || n != n_cur) {
                    if (!(ok = meet(G::KSync, met))) break;
                    if (d < kC / 2 && kg == 0) {
                        const double g = (double)a.decay[HB_IDX(it.hk, a.Hk)];
                        rw[d] = split_weights((float)decay_pow(g, max(n - 1 - 2 * d, 0)), (float)decay_pow(g, max(n - 2 - 2 * d, 0)));
                    }
                    if (!(ok = meet(G::KSync, met))) break;
                    hk_cur = it.hk;
                    n_cur = n;
                }
                if (!(ok = uni(tc::mbar_wait(bar(G::KVFull + st), (cc / G::kStages) & 1, abort)))) break;
                const uint32_t kt = sbase + st * G::kStage;
                if (n & 15) {
                    // rows of V behind the last token, up to the products' step of 16: whatever they hold must not
                    // reach a sum
                    uint8_t *vt = sm + st * G::kStage + G::kKB * kBlk;
                    const int rows = 16 - (n & 15);
                    for (int i = d; i < rows * 8 * G::kVB; i += 128)
                        *reinterpret_cast<uint4 *>(vt + (i / (rows * 8)) * kBlk + (n + (i / 8) % rows) * 128 + (i & 7) * 16) =
                            make_uint4(0, 0, 0, 0);
                    tc::fence_proxy_async_smem();
                }
                arrive(G::VReady + st);
                for (int h = 0; h * kSub < n; ++h, ++wc) {
                    const int wb = wc % kWBufs;
                    if (states_only && wb != kg) continue;
                    // x = w k as four bf16 terms.  The product of two bf16 numbers is the sum of its rounding and
                    // of what fma leaves, both exact: k w1 = t0 + e0, k w2 = t1 + e1; the last, k w3 + e1, is
                    // rounded at 2^-26 |x|.  Two tokens to a column, the terms kSub / 2 columns apart.
                    if (32 * w < NK) {
                        PairWeights pwt[4];
#pragma unroll
                        for (int m = 0; m < 4; ++m) pwt[m] = rw[h * (kSub / 2) + 4 * m + (lane & 3)];
                        const uint32_t k_row = kt + (w / 2) * kBlk + (h * kSub + (lane >> 4) * 8 + (lane & 7)) * 128;
                        uint32_t xs[2][8];
#pragma unroll
                        for (int hf = 0; hf < 2; ++hf) {              // 16 entries of k
                            const int ch = (w & 1) * 4 + hf * 2 + ((lane >> 3) & 1);      // this lane's 16-byte piece of its row
                            tc::ldmatrix_x4_trans(k_row + ((ch ^ (lane & 7)) << 4), xs[hf]);
                            tc::ldmatrix_x4_trans(k_row + 16 * 128 + ((ch ^ (lane & 7)) << 4), xs[hf] + 4);
                        }
                        if (!(ok = uni(tc::mbar_wait(bar(G::WFree + wb), ((wc / kWBufs) & 1) ^ 1, abort)))) break;
                        tc::tc_fence_after();
#pragma unroll
                        for (int hf = 0; hf < 2; ++hf) {
                            uint32_t *x = xs[hf];
                            if (n != kC) {
#pragma unroll
                                for (int i = 0; i < 8; ++i) {
                                    const int t = h * kSub + (i / 2) * 8 + (lane & 3) * 2;
                                    x[i] = t + 1 < n ? x[i] : t < n ? x[i] & 0xffffu : 0u;
                                }
                            }
                            uint32_t t[kTerms][8];
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                const PairWeights &p = pwt[i / 2];
                                const __nv_bfloat162 k = *reinterpret_cast<const __nv_bfloat162 *>(&x[i]);
                                const __nv_bfloat162 t0 = __hmul2_rn(k, p.w1), e0 = __hfma2(k, p.w1, __hneg2(t0));
                                const __nv_bfloat162 t1 = __hmul2_rn(k, p.w2), e1 = __hfma2(k, p.w2, __hneg2(t1));
                                const __nv_bfloat162 t2 = __hfma2(k, p.w3, e1);
                                t[0][i] = *reinterpret_cast<const uint32_t *>(&t0);
                                t[1][i] = *reinterpret_cast<const uint32_t *>(&e0);
                                t[2][i] = *reinterpret_cast<const uint32_t *>(&t1);
                                t[3][i] = *reinterpret_cast<const uint32_t *>(&t2);
                            }
                            const uint32_t cols = lane_base + ((uint32_t)(16 * hf) << 16) + kColW + wb * kWCols;
#pragma unroll
                            for (int y = 0; y < kTerms; ++y) tc::tmem_st_16x128b_x4(cols + y * (kSub / 2), t[y]);
                        }
                        tc::tmem_wait_st();
                    } else if (!(ok = uni(tc::mbar_wait(bar(G::WFree + wb), ((wc / kWBufs) & 1) ^ 1, abort)))) break;
                    tc::tc_fence_before();
                    arrive(G::WReady + wb);
                }
            }
        }
        if (!ok) *abort = 1;
    } else {
        // ------------------------------------------------------------ S groups
        // each has half of the columns of the state's rows, in registers
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(G::kRegsS));
        constexpr int NH = G::kNH;
        const int w = warp & 3, d = 32 * w + lane, sg = (warp - 12) >> 2;        // d: row of the state
        const uint32_t lane_base = tmem + ((uint32_t)(32 * w) << 16);
        int cc = 0, sc = 0, met = 0;                         // chunks, copies of the state so far
        bool ok = true;
        const long long ns = (long long)a.B * a.Hk * a.dk * a.dv;
        (void)ns; (void)met;
        for (int id = blockIdx.x; id < items && ok; id += gridDim.x) {
            const Item it = item_of(a, id, NV);
            const double g = (double)a.decay[HB_IDX(it.hk, a.Hk)];
            const float g_all = (float)decay_pow(g, kC), g_last = (float)decay_pow(g, it.ntok - (it.nck - 1) * kC);
            const float g_copy = g >= kUp ? g_all : 1.f;         // what the copy that multiplies the queries takes of Q S's factor
            const int col0 = it.c0 + sg * NH;
            const long long at = (((long long)it.b * a.Hk + it.hk) * a.dk + 32 * w) * a.dv + col0;       // this warp's rows
            const float *init = states_only || !a.init ? nullptr : a.init + (long long)it.seg * a.init_stride;
            float *dst = states_only ? a.states + (long long)(it.seg + 1) * a.init_stride
                                     : it.seg == a.nseg - 1 ? a.state_out : nullptr;
            float S[NH];
#pragma unroll
            for (int j = 0; j < NH; ++j) S[j] = 0.f;
            // Between global memory and the registers a warp's 32 rows pass through the copy's room, half of the group's
            // columns at a time (16-byte pieces swizzled by row), so that global accesses are whole lines: a row per
            // lane would cost one line per lane, and the other groups' shared-memory accesses would wait behind
            // them.  With NV = 128 a row is staged where this thread copies it; with NV = 64 the rooms and the rows of
            // the copy lie across one another, so all S warps meet in between.
            constexpr int kPc = NH / 8;                      // 16-byte pieces of a staged row
            const bool mine = 32 * w < NK;
            auto stage = [&](int r, int pc) {
                return reinterpret_cast<float4 *>(sm + G::kSmS + sg * (NK * NH * 2) + (32 * w + r) * (16 * kPc) + ((pc ^ (r & (kPc - 1))) << 4));
            };
            if (init) {
                if (!(ok = uni(tc::mbar_wait(bar(G::SFree), (sc & 1) ^ 1, abort)))) break;
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    if (mine) {
#pragma unroll
                        for (int i = 0; i < kPc; ++i) {
                            const int r = (i * 32 + lane) / kPc, pc = lane % kPc, col = hf * (NH / 2) + 4 * pc;
                            float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
                            if (32 * w + r < a.dk && col0 + col < a.dv)
                                t = *reinterpret_cast<const float4 *>(init + HB_IDX(at + (long long)r * a.dv + col, ns - 3));
                            *stage(r, pc) = t;
                        }
                        __syncwarp();
#pragma unroll
                        for (int pc = 0; pc < kPc; ++pc) {
                            const float4 t = *stage(lane, pc);
                            const int j = hf * (NH / 2) + 4 * pc;
                            S[j] = t.x; S[j + 1] = t.y; S[j + 2] = t.z; S[j + 3] = t.w;
                        }
                        __syncwarp();
                    }
                }
                if (NV == 64 && !(ok = meet(G::SSync, met))) break;
            }
            // the next item's entering state on its way to L2: read cold it would cost a dependent trip to memory
            if (init && id + (int)gridDim.x < items) {
                const Item nx = item_of(a, id + gridDim.x, NV);
                const long long base = (long long)nx.seg * a.init_stride + ((long long)nx.b * a.Hk + nx.hk) * a.dk * a.dv;
                for (int i = sg * 128 + d; i < (a.dk * a.dv + 31) / 32; i += 256)
                    asm volatile("prefetch.global.L2 [%0];" ::"l"(a.init + base + 32ll * i));
            }
            // c = -1: only the copy of the entering state
            for (int c = -1; c < it.nck; ++c) {
                if (c >= 0) {
                    if (!(ok = uni(tc::mbar_wait(bar(G::UDone), cc & 1, abort)))) break;
                    tc::tc_fence_after();
                    const float gn = c == it.nck - 1 ? g_last : g_all;
                    if (mine) {
#pragma unroll
                        for (int p = 0; p < NH / 16; ++p) {
                            float z[16];
                            tc::tmem_ld16(lane_base + kColU + sg * NH + 16 * p, z);
                            tc::tmem_wait_ld();
#pragma unroll
                            for (int j = 0; j < 16; ++j) S[16 * p + j] = fmaf(gn, S[16 * p + j], z[j]);
                        }
                    }
                    tc::tc_fence_before();
                    arrive(G::UFree);
                    ++cc;
                }
                if (states_only) continue;
                if (c + 1 < it.nck && (c >= 0 || init)) {
                    // the copy that multiplies the queries, once every product with the last one is done
                    if (!(ok = uni(tc::mbar_wait(bar(G::SFree), (sc & 1) ^ 1, abort)))) break;
                    if (mine) {
                        uint8_t *row = sm + G::kSmS + d * 128;
#pragma unroll
                        for (int i = 0; i < NH / 8; ++i) {
                            const int ch = sg * (NH / 8) + i;
                            *reinterpret_cast<uint4 *>(row + (ch / 8) * (NK * 128) + (((ch & 7) ^ (d & 7)) << 4)) =
                                make_uint4(pack2_scaled(g_copy, S[8 * i], S[8 * i + 1]), pack2_scaled(g_copy, S[8 * i + 2], S[8 * i + 3]),
                                           pack2_scaled(g_copy, S[8 * i + 4], S[8 * i + 5]), pack2_scaled(g_copy, S[8 * i + 6], S[8 * i + 7]));
                        }
                        tc::fence_proxy_async_smem();
                    }
                    arrive(G::SReady);
                    ++sc;
                }
            }
            if (!ok) break;
            if (dst) {
                if (!states_only && !(ok = uni(tc::mbar_wait(bar(G::SFree), (sc & 1) ^ 1, abort)))) break;
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    if (mine) {
#pragma unroll
                        for (int pc = 0; pc < kPc; ++pc) {
                            const int j = hf * (NH / 2) + 4 * pc;
                            *stage(lane, pc) = make_float4(S[j], S[j + 1], S[j + 2], S[j + 3]);
                        }
                        __syncwarp();
#pragma unroll 2
                        for (int i = 0; i < kPc; ++i) {
                            const int r = (i * 32 + lane) / kPc, pc = lane % kPc, col = hf * (NH / 2) + 4 * pc;
                            const long long x = at + (long long)r * a.dv + col;
                            if (32 * w + r < a.dk && col0 + col < a.dv && HB_OK(x + 3, ns)) *reinterpret_cast<float4 *>(dst + x) = *stage(r, pc);
                        }
                        __syncwarp();
                    }
                }
                if (NV == 64 && !states_only && !(ok = meet(G::SSync, met))) break;
            }
        }
        if (!ok) *abort = 1;
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    if (warp == 2) tc::tmem_dealloc(tmem, kTmemCols);
    if (tid == 0)
        for (int i = blockIdx.x; i < a.nerr; i += gridDim.x) a.err[HB_IDX(i, a.nerr)] = i == (int)blockIdx.x ? *abort : 0;
}

// tests: a wait of block 0 runs out in every later launch (hyena_test_linattn_hold)
std::atomic<int> g_hold{0};

// [B][L][heads][width] bf16 with rows `ld` elements apart; boxes of 64 entries x 1 head x 128 tokens
bool make_map(CUtensorMap *m, const void *base, int B, int L, int heads, int width, long long ld) {
    static PFN_cuTensorMapEncodeTiled_v12000 enc = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    }();
    if (!enc) return false;
    cuuint64_t dims[4] = {(cuuint64_t)width, (cuuint64_t)heads, (cuuint64_t)L, (cuuint64_t)B};
    cuuint64_t strides[3] = {(cuuint64_t)width * 2, (cuuint64_t)ld * 2, (cuuint64_t)ld * 2 * L};
    cuuint32_t box[4] = {64, 1, (cuuint32_t)kC, 1}, estr[4] = {1, 1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int NK, int NV>
cudaError_t launch(const Maps &m, const LinArgs &a, int items, bool states_only, cudaStream_t s) {
    constexpr int smem = Geo<NK, NV>::kSmem;
    // the kernel's attributes, once per device
    static std::atomic<unsigned long long> ready{0};
    int dev;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || !(ready.load(std::memory_order_acquire) >> dev & 1)) {
        e = cudaFuncSetAttribute(linattn_tc_kernel<NK, NV>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        cudaFuncAttributes fa;
        if ((e = cudaFuncGetAttributes(&fa, linattn_tc_kernel<NK, NV>)) != cudaSuccess) return e;
        // 640 threads leave at most 96 registers each, the shares need at least 94, and counts come in eights: only 96 will do
        if (fa.numRegs != kRegsLaunch) return cudaErrorInvalidConfiguration;
        if (dev < 64) ready.fetch_or(1ull << dev, std::memory_order_release);
    }
    const int grid = items < kLinMaxBlocks ? items : kLinMaxBlocks;
    linattn_tc_kernel<NK, NV><<<grid, kThreads, smem, s>>>(m, a, items, states_only);
    return cudaGetLastError();
}

}  // namespace

HYENA_BOUNDS_READER(linattn_tc)

void linattn_hold(int enable) { g_hold.store(enable); }

bool linattn_tc_dims(int dtype, int dk, int dv) { return dtype == HYENA_BF16 && dk <= 128 && dk % 8 == 0 && dv % 8 == 0; }

// How a prompt is cut, by a model of the time in us (blocks take their items one after the other, so the longest one
// counts).  A chunk of the main pass costs `base` + `query` for each query head of its key head, one of the state pass
// `state`, the entry of an item (its state, the filling of the pipeline) `entry`; cutting adds the state pass, the
// combination of the states and two launches.  Narrow tiles repeat the scores and the weighing of the keys, but give twice
// the items: where sequences x heads leave SMs idle they cost less than a second pass over the tokens.
// The figures were measured on whole grids when the rule was made.  Now a chunk takes 5.0 us (128 x 128), 3.0 (128 x 64, and
// 64 x 64) or 1.9 (64 x 64 without queries), and an item's entry hides behind the item before, so the model reads 1.1 to 1.7
// times too high (210, 134 and 285 us for the three shapes at the top of this file) and serves to compare cuts only.  The choices were compared
// with both widths and 1 to 64 segments on eleven shapes: the fastest, or within 2 us of it, on ten (few sequences, one
// long prompt, shared heads, a padded batch of 32 rows); 13 padded rows of 1537 tokens x 4 x 3 heads of 96 x 80 take 96 us
// in the rule's five segments and 78 in four.
// Padded rows (lens) are taken to be half full.
LinPlan linattn_tc_plan(int B, int L, int H, int Hk, int dk, int dv, bool lens) {
    struct Cost { double base, query, state, entry; };
    const double kCut = 15.0;
    LinPlan best{};
    double best_us = 0;
    const int chunks = L > 0 ? (L + kC - 1) / kC : 1, Gq = H / Hk;
    const double fill = lens ? 0.5 : 1.0;
    auto waves = [&](double items) { const double w = (double)(long long)((items * fill + kLinMaxBlocks - 1) / kLinMaxBlocks); return w < 1 ? 1.0 : w; };
    for (int nv = 64; nv <= (dv > 64 ? 128 : 64); nv += 64) {
        const Cost c = dk <= 64 ? (nv == 64 ? Cost{0.4, 3.0, 2.7, 5.0} : Cost{0.5, 3.7, 3.0, 6.0})
                                : (nv == 64 ? Cost{0.5, 3.5, 3.0, 6.0} : Cost{0.5, 4.5, 3.5, 10.0});
        const int vtiles = (dv + nv - 1) / nv;
        const double units = (double)(B > 0 ? B : 1) * Hk * vtiles;
        for (int want = 1; want <= chunks && want <= kLinMaxBlocks; ++want) {
            const int sc = (chunks + want - 1) / want, ns = (chunks + sc - 1) / sc;
            double us = waves(units * ns) * (sc * (c.base + c.query * Gq) + c.entry);
            if (ns > 1) us += waves(units * (ns - 1)) * (sc * c.state + c.entry / 2) + kCut;
            if (best.vtiles == 0 || us < best_us) {
                best_us = us;
                best.vtiles = vtiles;
                best.nv = nv;
                best.seg_tokens = sc * kC;
                best.nseg = ns;
            }
        }
    }
    return best;
}

cudaError_t launch_linattn_tc(LinArgs a, bool states_only, cudaStream_t s) {
    a.hold = g_hold.load(std::memory_order_relaxed);
    const long long items = (long long)(states_only ? a.nseg - 1 : a.nseg) * a.B * a.Hk * a.vtiles;
    if (items > 0x7fffffffll - kLinMaxBlocks) return cudaErrorInvalidValue;
    Maps m;
    if (!make_map(&m.q, a.q, a.B, a.L, a.H, a.dk, a.ldq) || !make_map(&m.k, a.k, a.B, a.L, a.Hk, a.dk, a.ldk) ||
        !make_map(&m.v, a.v, a.B, a.L, a.Hk, a.dv, a.ldv) || !make_map(&m.o, a.o, a.B, a.L, a.H, a.dv, (long long)a.H * a.dv))
        return cudaErrorInvalidValue;
    if (a.dk <= 64) return a.nv == 64 ? launch<64, 64>(m, a, (int)items, states_only, s) : launch<64, 128>(m, a, (int)items, states_only, s);
    return a.nv == 64 ? launch<128, 64>(m, a, (int)items, states_only, s) : launch<128, 128>(m, a, (int)items, states_only, s);
}

}  // namespace hyena
