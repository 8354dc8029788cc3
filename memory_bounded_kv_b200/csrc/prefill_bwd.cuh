// Gradients of the prompt attention (kvb_prefill_attn_bwd) on the 5th-generation tensor cores, as two
// kernels, so that every sum runs in one CTA in a fixed order (no atomics, no fp32 copy of dq):
//
//   prefill_dq_kernel   per block of query rows: S = Q K^T, dP = dO V^T, P = exp2(C S - lse),
//                       dS = P (dP - delta), dQ += dS K; leaves delta for the second kernel
//   prefill_dkv_kernel  per block of keys: S^T, dP^T, then dV += P^T dO, dK += dS^T Q, and
//                       d log beta_j = sum_i dS_ij max(i - j, 0) in fp32
//
// delta_i = sum_j p_ij dP_ij - dlse_i. dO . o would give it from the output, but o is held in bf16
// (2^-8 relative), which d log beta, an fp32 result whose terms cancel, would show. The first kernel
// starts from that estimate e_i = dO . o - dlse_i; its row sums of dS are then sum_j p_ij dP_ij - e_i,
// so e_i + their sum - dlse_i is delta to fp32, for one addition per score. In dq_i = sum_j dS_ij k_j the
// estimate's error eps_i = delta_i - e_i leaves eps_i sum_j p_ij k_j. Beside weights that are spread, that is less
// than the rounding of dS to bf16; where one key has almost all, dS_ij = p_ij (dP_ij - delta_i) is small and eps_i
// is not. So a key of weight above 1/2 (a row has one at most) is kept, and eps_i p_ij k_j is taken from dq_i.
// Log beta of -3 to -5, 1000 tokens, 8/2 heads: dq off by 4 % in the middle row and 1.3 % in all -> 0.25 % each,
// for 3 % of the time on documents of 250 tokens and next to none on one of 8192. Rows whose keys fit one tile
// take delta itself at once.
//
// What bounds both is shared memory and the hand-over between products and softmax. A product of two
// shared-memory operands reads 16 (128 + N) x 2 bytes per K step of 16: at N = 64 that is 48 clocks of
// the 128 bytes a clock for 32 clocks of mathematics, at N = 128 it is 64 for 64 (measured: 48.8 and
// 64.4 clocks a step; with the first operand in tensor memory 32.7 and 63.4).
//   By query rows, the block's Q and dO live in tensor memory (written there once per unit), so that S
// and dP leave shared memory to the copies. The next S is issued as soon as the warpgroups have read one;
// dS goes over dP, so dQ += dS K comes before the next dP, which the exponentials hide.
//   By keys there is no room for that (dK, dV, S and dP fill the tensor memory). S and dP alternate:
// P done -> dV += P^T dO and the next S, while the warpgroups turn dP into dS; dS done -> dK += dS^T Q
// and the next dP, while they turn the next S into P.
// Its key blocks are cut into pieces of equal length for the CTAs (StepLine), and prefill_dkv_sum_kernel
// adds up the few that a cut goes through.
//   The two warpgroups share a tile: each takes 64 of its 128 columns, a thread per row.
// The bias rides the S product as in prefill_fwd_kernel; by keys, - lse and - delta ride S and dP too.
// One document of 8192 tokens, 32/8 heads, d 128: by query rows 725 us (3 products, 1.14 PFLOP/s), by keys
// 925 us (4 products, 1.19 PFLOP/s), both near the power cap in long runs; d 64 627 and 617 us; d 128 with a cap
// of 50 1155 and 1250 us.
#pragma once

#include "prefill_units.cuh"

namespace kvb {

// The extra columns of prefill_dkv_kernel, where one block of keys meets queries at any distance: with
// i - last = a0 + 256 a1 + 65536 a2 (each term exact in bf16, tokens <= 2^24) and the three bf16 parts
// of b, of (last - j) b and of a per-query number y (- lse / scale for S, - delta for dP) the product is
// (i - last) b + (last - j) b + y; both terms of the bias have one sign.
__device__ __forceinline__ void far_query(int dist, float y, uint4& c0, uint4& c1) {
    const uint32_t a0 = pack_bf16((float)(dist & 255), (float)(dist & 255));
    const uint32_t a1 = pack_bf16((float)(dist & 0xff00), (float)(dist & 0xff00));
    const uint32_t a2 = pack_bf16((float)(dist & 0xff0000), (float)(dist & 0xff0000)), one = 0x3f803f80u;
    uint32_t yh, ym, yl;
    split3_bf16(y, yh, ym, yl);
    c0 = make_uint4(a0, (a0 & 0xffffu) | (a1 & 0xffff0000u), a1, a2);
    c1 = make_uint4((a2 & 0xffffu) | (one & 0xffff0000u), one, yh | (ym << 16), yl);
}
__device__ __forceinline__ void far_key(float b, int last_minus_j, uint4& c0, uint4& c1) {
    uint32_t h, m, l, ch, cm, cl;
    split3_bf16(b, h, m, l);
    split3_bf16((float)last_minus_j * b, ch, cm, cl);
    c0 = make_uint4(h | (m << 16), l | (h << 16), m | (l << 16), h | (m << 16));
    c1 = make_uint4(l | (ch << 16), cm | (cl << 16), 0x3f803f80u, 0x3f80u);
}

template <int D>
struct DqShape {
    static constexpr int R = 128, KT = 128;
    static constexpr int ST = D == 128 ? 3 : 6;          // K/V ring stages
    static constexpr int NT = 12 * 32;
    static constexpr int REG_SOFT = 208, REG_REST = 88;  // 2 x 208 + 88 = 3 x 168, the launch's registers
    static constexpr int KHALF = KT * 128, KTILE = KHALF * (D / 64);
    static constexpr int KV_OFF = 0;                     // [ST] K, V
    static constexpr int QX_OFF = KV_OFF + ST * 2 * KTILE;
    static constexpr int KX_OFF = QX_OFF + R * 32;
    static constexpr int LB_OFF = KX_OFF + ST * KT * 32;
    static constexpr int EST_OFF = LB_OFF + ST * KT * 4; // [128] estimates, [128] row sums of the second warpgroup
    static constexpr int PART_OFF = EST_OFF + 2 * R * 4; // [2][128] each warpgroup's part of delta (units of one tile); in
                                                         // other units EST and PART also hold what passes at the end
    static constexpr int INFO_OFF = PART_OFF + 2 * R * 4;
    static constexpr int BAR_OFF = INFO_OFF + 2 * 8 * 4;
    static constexpr int NBAR = 4 + 3 * ST + 6 + 4;
    static constexpr int MISC_OFF = BAR_OFF + NBAR * 8;
    static constexpr size_t SMEM = 1024 + MISC_OFF + 32;
    static constexpr int TM_Q = 0, TM_DO = 64, TM_S = 128, TM_DP = 256, TM_DQ = 384, TM_COLS = 512;
    static_assert(SMEM <= 227 * 1024, "shared memory");
};

template <int D, bool BETA, bool CAP>
__global__ void __launch_bounds__(DqShape<D>::NT, 1)
    prefill_dq_kernel(const __grid_constant__ PrefillParams p, const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV) {
    using SH = DqShape<D>;
    constexpr int ST = SH::ST, R = SH::R, KT = SH::KT;
    extern __shared__ unsigned char smem_dyn[];
    unsigned char* smem = reinterpret_cast<unsigned char*>(
        (reinterpret_cast<uintptr_t>(smem_dyn) + 1023) & ~static_cast<uintptr_t>(1023));
    const uint32_t sbase = smem_u32(smem);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + SH::BAR_OFF);
    uint64_t* a_full = bars;             // Q and dO are in tensor memory, the previous dQ is read
    uint64_t* est_full = bars + 1;
    uint64_t* sum_full = bars + 2;
    uint64_t* o_full = bars + 3;         // dQ
    uint64_t* kv_full = bars + 4;
    uint64_t* kv_empty = kv_full + ST;
    uint64_t* x_full = kv_empty + ST;    // the bias columns and slopes; K's and V's rows past the document cleared
    uint64_t* s_full = x_full + ST;
    uint64_t* s_read = s_full + 1;
    uint64_t* dp_full = s_full + 2;
    uint64_t* ds_full = s_full + 3;
    uint64_t* part_full = s_full + 4;
    uint64_t* fix_full = s_full + 5;     // the first warpgroup's answer to sum_full
    uint64_t* u_full = s_full + 6;
    uint64_t* u_empty = u_full + 2;
    int* info = reinterpret_cast<int*>(smem + SH::INFO_OFF);
    uint32_t* tslot = reinterpret_cast<uint32_t*>(smem + SH::MISC_OFF);
    volatile int* s_abort = reinterpret_cast<int*>(smem + SH::MISC_OFF) + 1;
    int* s_steps = reinterpret_cast<int*>(smem + SH::MISC_OFF) + 2;
    uint64_t* fin = reinterpret_cast<uint64_t*>(smem + SH::MISC_OFF + 16);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int lg = 31 - __clz(p.G), sh = 7 - lg;        // 2^sh tokens a unit
    if (tid == 0) {
        mbar_init(a_full, 8);
        mbar_init(est_full, 4);
        mbar_init(sum_full, 4);
        mbar_init(o_full, 1);
        for (int s = 0; s < ST; ++s) {
            mbar_init(&kv_full[s], 1);
            mbar_init(&kv_empty[s], 1);
            mbar_init(&x_full[s], 1);
        }
        mbar_init(s_full, 1);
        mbar_init(s_read, 8);
        mbar_init(dp_full, 1);
        mbar_init(ds_full, 8);
        mbar_init(part_full, 8);
        mbar_init(fix_full, 4);
        for (int t = 0; t < 2; ++t) {
            mbar_init(&u_full[t], 1);
            mbar_init(&u_empty[t], 10);   // products, bias, 8 softmax warps
        }
        mbar_init(fin, 1);
        *s_abort = 0;
        s_steps[0] = 0;
        fence_mbar_init();
    }
    if (warp == 9 && lane == 0) {
        prefetch_tensormap(&tmK);
        prefetch_tensormap(&tmV);
    }
    if (BETA && !CAP) {
        for (int x = tid; x < R; x += SH::NT) {
            *reinterpret_cast<uint4*>(smem + SH::QX_OFF + plain16_off(x, 0)) = bias_query(x >> lg);
            *reinterpret_cast<uint4*>(smem + SH::QX_OFF + plain16_off(x, 1)) = make_uint4(0u, 0u, 0u, 0u);
        }
        for (int x = tid; x < ST * KT; x += SH::NT)
            *reinterpret_cast<uint4*>(smem + SH::KX_OFF + (x >> 7) * KT * 32 + plain16_off(x & 127, 1)) =
                make_uint4(0u, 0u, 0u, 0u);
        fence_proxy_async_smem();
    }
    if (warp == 8) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tslot)),
                     "r"(SH::TM_COLS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    griddep_wait();
    griddep_launch_dependents();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tslot;
    auto fail = [&]() {
        raise_error(KVB_DERR_TIMEOUT);
        *s_abort = 1;
    };

    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(SH::REG_REST));
        if (warp == 9) {
            // ======================= units and loads =======================
            const PrefillWalk walk(p, sh);
            const long long units = walk.units;
            int step = 0, uc = 0;
            bool stop = false;
            for (long long r = 0; !stop; ++r, ++uc) {
                const long long u = PrefillWalk::nth(r, blockIdx.x, gridDim.x);
                const bool end = r * gridDim.x >= units;
                if (!end && u >= units) { --uc; continue; }
                PrefillUnit x{};
                int n = 0;
                if (!end) {
                    x = walk.unit(u);
                    n = (max(min((x.blk + 1) << sh, x.len), x.pre) + KT - 1) / KT;
                }
                const int ub = uc & 1;
                if (uc >= 2 && !warp_wait(&u_empty[ub], (unsigned)((uc >> 1) - 1) & 1u, p.wait_ns)) { stop = true; break; }
                if (__any_sync(kFull, *s_abort != 0)) break;
                if (lane == 0) {
                    int* m = info + ub * 8;
                    m[0] = end ? -1 : x.s;
                    m[1] = x.len;
                    m[2] = x.blk << sh;
                    m[3] = x.g;
                    m[4] = x.pre;
                    m[5] = n;
                    mbar_arrive(&u_full[ub]);
                }
                __syncwarp();
                if (end) break;
                const int loads = p.withhold == blockIdx.x + 1 ? min(n, max(1 - step, 0)) : n;   // test hook: one tile in all
                for (int tile = n - 1; tile >= n - loads; --tile, ++step) {
                    const int st = step % ST;
                    if (step >= ST && !warp_wait(&kv_empty[st], (unsigned)((step / ST) - 1) & 1u, p.wait_ns)) { stop = true; break; }
                    if (lane == 0) {
                        mbar_arrive_expect_tx(&kv_full[st], (unsigned)(2 * SH::KTILE));
                        for (int h = 0; h < D / 64; ++h) {
                            unsigned char* at = smem + SH::KV_OFF + st * 2 * SH::KTILE + h * SH::KHALF;
                            tma_load_3d(at, &tmK, 64 * h, x.g, x.s + tile * KT, &kv_full[st]);
                            tma_load_3d(at + SH::KTILE, &tmV, 64 * h, x.g, x.s + tile * KT, &kv_full[st]);
                        }
                        s_steps[0] = step + 1;
                    }
                    if (__any_sync(kFull, *s_abort != 0)) { stop = true; break; }
                }
                if (loads < n) break;
            }
            if (stop && lane == 0) fail();
        } else if (warp == 10) {
            // ======================= bias columns, K and V past a document's end =======================
            // the log betas of the next step load while it writes this one's
            const float unit_b = CAP ? kLog2e : 1.f / p.scale;
            int step = 0;
            bool stop = false;
            for (int uc = 0; !stop; ++uc) {
                const int ub = uc & 1;
                if (!warp_wait(&u_full[ub], (unsigned)(uc >> 1) & 1u, p.wait_ns)) { stop = true; break; }
                const int* m = info + ub * 8;
                const int s = m[0], len = m[1], i0 = m[2], g = m[3], n = m[5];
                __syncwarp();
                if (lane == 0) mbar_arrive(&u_empty[ub]);
                if (s < 0) break;
                float nb[4] = {0.f, 0.f, 0.f, 0.f};
                auto load = [&](int tile) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int j = tile * KT + lane + 32 * e;
                        nb[e] = tile >= 0 && j < len ? p.lb[(long long)(s + j) * p.lb_st + g * p.lb_sh] : 0.f;
                    }
                };
                if (BETA) load(n - 1);
                for (int q = 0; q < n; ++q) {
                    const int tile = n - 1 - q, k = step + q, st = k % ST;
                    const unsigned ph = (unsigned)(k / ST) & 1u;
                    float b[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) b[e] = clamp_log_beta(nb[e]) * unit_b;
                    if (BETA) load(tile - 1);
                    if (k >= ST && !warp_wait(&kv_empty[st], ph ^ 1u, p.wait_ns)) { stop = true; break; }
                    if (BETA) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int c = lane + 32 * e;
                            reinterpret_cast<float*>(smem + SH::LB_OFF)[st * KT + c] = b[e];
                            if (!CAP)
                                *reinterpret_cast<uint4*>(smem + SH::KX_OFF + st * KT * 32 + plain16_off(c, 0)) =
                                    bias_columns(b[e], i0 - tile * KT - c);
                        }
                    }
                    if ((tile + 1) * KT > len) {
                        if (!warp_wait(&kv_full[st], ph, p.wait_ns)) { stop = true; break; }
                        const int rows = len - tile * KT;
                        unsigned char* kt = smem + SH::KV_OFF + st * 2 * SH::KTILE;
                        for (int x = lane; x < (KT - rows) * 16 * (D / 64); x += 32) {
                            const int row = rows + x / (16 * (D / 64)), c = x % (16 * (D / 64));   // chunks of K, then of V
                            *reinterpret_cast<uint4*>(kt + (c >> 3) * SH::KHALF + row * 128 + ((c & 7) << 4)) =
                                make_uint4(0u, 0u, 0u, 0u);
                        }
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&x_full[st]);
                    if (__any_sync(kFull, *s_abort != 0)) { stop = true; break; }
                }
                step += n;
            }
            if (stop && lane == 0) fail();
        } else if (warp == 8) {
            // ======================= products =======================
            // the warp stays together (its values are uniform); one lane issues
            constexpr uint32_t idesc_s = umma_idesc_bf16(R, KT), idesc_o = umma_idesc_bf16_bmn(R, D);
            int step = 0;
            bool stop = false;
            const uint32_t k_lo = desc_sw128_lo(sbase + SH::KV_OFF), kr_lo = desc_mn_lo(sbase + SH::KV_OFF, SH::KHALF);
            const uint32_t qx_lo = desc_plain_lo(sbase + SH::QX_OFF), kx_lo = desc_plain_lo(sbase + SH::KX_OFF);
            auto scores = [&](int st, bool past) {
                umma_kmajor_ts<D / 16>(tmem + SH::TM_S, tmem + SH::TM_Q, k_lo + st * (2 * SH::KTILE >> 4), SH::KHALF, idesc_s);
                if (BETA && !CAP && past)
                    umma_bf16(tmem + SH::TM_S, desc(qx_lo, kDescPlainHi), desc(kx_lo + st * (KT * 32 >> 4), kDescPlainHi), idesc_s, 1u);
                umma_commit(s_full);
            };
            auto pulls = [&](int st) {
                umma_kmajor_ts<D / 16>(tmem + SH::TM_DP, tmem + SH::TM_DO, k_lo + (st * 2 + 1) * (SH::KTILE >> 4), SH::KHALF, idesc_s);
                umma_commit(dp_full);
            };
            auto loaded = [&](int k) {
                return warp_wait(&kv_full[k % ST], (unsigned)(k / ST) & 1u, p.wait_ns) &&
                       warp_wait(&x_full[k % ST], (unsigned)(k / ST) & 1u, p.wait_ns);
            };
            for (int uc = 0; !stop; ++uc) {
                const int ub = uc & 1;
                if (!warp_wait(&u_full[ub], (unsigned)(uc >> 1) & 1u, p.wait_ns)) { stop = true; break; }
                const int* m = info + ub * 8;
                const int s = __shfl_sync(kFull, m[0], 0), i0 = __shfl_sync(kFull, m[2], 0), n = __shfl_sync(kFull, m[5], 0);
                if (lane == 0) mbar_arrive(&u_empty[ub]);
                if (s < 0) break;
                if (!warp_wait(a_full, (unsigned)uc & 1u, p.wait_ns) || !loaded(step)) { stop = true; break; }
                tc_fence_after();
                if (elect_one()) {
                    scores(step % ST, n * KT <= i0 + 1);
                    pulls(step % ST);
                }
                __syncwarp();
                for (int tile = n - 1; tile >= 0; --tile, ++step) {
                    const int st = step % ST, nst = (step + 1) % ST;
                    const bool more = tile > 0;
                    // the next scores as soon as these are read
                    if (more && !loaded(step + 1)) { stop = true; break; }
                    if (!warp_wait(s_read, (unsigned)step & 1u, p.wait_ns)) { stop = true; break; }
                    tc_fence_after();
                    if (elect_one() && more) scores(nst, tile * KT <= i0 + 1);
                    __syncwarp();
                    if (!warp_wait(ds_full, (unsigned)step & 1u, p.wait_ns)) { stop = true; break; }
                    tc_fence_after();
                    if (elect_one()) {
                        // dS: a warpgroup's 64 columns as 32 words at the start of its half of dP
                        const uint32_t b = kr_lo + st * (2 * SH::KTILE >> 4);
                        umma_rows<4>(tmem + SH::TM_DQ, tmem + SH::TM_DP, b, idesc_o, tile == n - 1);
                        umma_rows<4>(tmem + SH::TM_DQ, tmem + SH::TM_DP + 64, b + 64 * 128 / 16, idesc_o, false);
                        umma_commit(&kv_empty[st]);
                        if (more) {
                            pulls(nst);
                        } else {
                            umma_commit(o_full);
                        }
                    }
                    __syncwarp();
                }
            }
            if (stop && lane == 0) fail();
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(SH::REG_SOFT));
        // ======================= Q and dO into tensor memory, dS, dQ and delta =======================
        const int t = warp >> 2, quarter = warp & 3;
        const int r = 32 * quarter + lane;
        const uint32_t tl = tmem + ((uint32_t)(32 * quarter) << 16);
        const float C = CAP ? 1.f : p.scale * kLog2e;
        const float cap2 = CAP ? p.softcap * kLog2e : 0.f, per_cap = CAP ? p.scale / p.softcap : 0.f;
        const float inv_cap2 = CAP ? -1.f / (cap2 * cap2) : 0.f;
        float* s_est = reinterpret_cast<float*>(smem + SH::EST_OFF);
        float* s_sum = s_est + R;
        float* s_part = reinterpret_cast<float*>(smem + SH::PART_OFF);
        unsigned singles = 0;   // parity of the units of one tile
        int step = 0;
        bool stop = false;
        int s = -1, len = 0, i0 = 0, g = 0, pre = 0, n = 0;
        uint32_t a[D / 2];
        // the unit's record, and this thread's row of Q (first warpgroup) or dO (second)
        auto next = [&](int uc) {
            const int ub = uc & 1;
            if (!warp_wait(&u_full[ub], (unsigned)(uc >> 1) & 1u, p.wait_ns)) return false;
            const int* m = info + ub * 8;
            s = m[0], len = m[1], i0 = m[2], g = m[3], pre = m[4], n = m[5];
            __syncwarp();
            if (lane == 0) mbar_arrive(&u_empty[ub]);
            const int i = i0 + (r >> lg), h = (g << lg) + (r & (p.G - 1));
            const bool row = s >= 0 && i < len;
            const uint16_t* src = t ? p.d_o + ((size_t)(s + i) * p.Hq + h) * D : p.q + (long long)(s + i) * p.q_st + h * p.q_sh;
#pragma unroll
            for (int c = 0; c < D / 8; ++c) {
                const uint4 v = row ? reinterpret_cast<const uint4*>(src)[c] : make_uint4(0u, 0u, 0u, 0u);
                a[4 * c] = v.x;
                a[4 * c + 1] = v.y;
                a[4 * c + 2] = v.z;
                a[4 * c + 3] = v.w;
            }
            return true;
        };
        if (!next(0)) stop = true;
        for (int uc = 0; !stop && s >= 0; ++uc) {
#pragma unroll
            for (int c = 0; c < D / 2; c += 32) tmem_st32(tl + (t ? SH::TM_DO : SH::TM_Q) + c, a + c);
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(a_full);
            const int first = i0, i = i0 + (r >> lg);
            const int lim = min(max(i + 1, pre), len);
            const bool valid = i < len;
            const size_t row = (size_t)(s + i) * p.Hq + (g << lg) + (r & (p.G - 1));
            // the estimate of delta from the output; lse in log2 units (a row past the document: P = 0)
            float est = 0.f, dlse = 0.f;
            const float lse2 = valid ? p.lse[row] * kLog2e : INFINITY;
            if (valid && p.d_lse != nullptr) dlse = p.d_lse[row];
            if (t == 1) {
                if (valid) {
                    const uint4* o = reinterpret_cast<const uint4*>(p.o + row * D);
                    float e0 = 0.f, e1 = 0.f;
#pragma unroll
                    for (int c = 0; c < D / 8; ++c) {
                        const uint4 v = o[c];
                        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            e0 = fmaf(bf16_lo(a[4 * c + e]), bf16_lo(w[e]), e0);
                            e1 = fmaf(bf16_hi(a[4 * c + e]), bf16_hi(w[e]), e1);
                        }
                    }
                    est = e0 + e1 - dlse;
                }
                s_est[r] = est;
                __syncwarp();
                if (lane == 0) mbar_arrive(est_full);
            } else {
                if (!warp_wait(est_full, (unsigned)uc & 1u, p.wait_ns)) { stop = true; break; }
                est = s_est[r];
            }
            const uint16_t* keys = p.k + (long long)s * p.kv_st + g * p.kv_sh;
            float top = 0.f;                           // a weight above 1/2 (times the cap's slope), and its key
            int top_j = 0;
            float rsum = 0.f;
            for (int tile = n - 1; tile >= 0; --tile, ++step) {
                const int st = step % ST, j0 = tile * KT + 64 * t;   // this warpgroup's keys
                if (!warp_wait(s_full, (unsigned)step & 1u, p.wait_ns)) { stop = true; break; }
                tc_fence_after();
                float x[64], th[CAP ? 64 : 1];
                tmem_ld32(tl + SH::TM_S + t * 64, x);
                tmem_ld32(tl + SH::TM_S + t * 64 + 32, x + 32);
                tmem_ld_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(s_read);
                const bool past = (tile + 1) * KT <= first + 1;
                if (CAP) {
                    cap_scores<64>(x, per_cap, cap2);
#pragma unroll
                    for (int c = 0; c < 64; ++c) th[c] = x[c];
                }
                if (BETA && (CAP || !past)) {
                    if (!warp_wait(&x_full[st], (unsigned)(step / ST) & 1u, p.wait_ns)) { stop = true; break; }
                    const float4* lb = reinterpret_cast<const float4*>(smem + SH::LB_OFF + (st * KT + 64 * t) * 4);
                    add_bias(x, lb, (float)(i - j0), past);
                    add_bias(x + 32, lb + 8, (float)(i - j0 - 32), past);
                }
                if (j0 + 64 > max(first + 1, pre)) {
#pragma unroll
                    for (int c = 0; c < 64; ++c) x[c] = c < lim - j0 ? x[c] : -INFINITY;
                }
                const uint64_t c2 = same2(C), n2 = same2(-lse2);
#pragma unroll
                for (int c = 0; c < 64; c += 2) {
                    float u, v;
                    upk2(fma2(pk2(x[c], x[c + 1]), c2, n2), u, v);
                    if (D == 64 && c % 8 == 6) {   // a quarter of the exponentials on the FMA pipe, as forward
                        exp2_poly2<5>(u, v);
                    } else {
                        u = ex2_approx(u);
                        v = ex2_approx(v);
                    }
                    x[c] = u;
                    x[c + 1] = v;
                }
                float most[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int c = 0; c < 64; c += 2) most[(c / 2) & 3] = max3(most[(c / 2) & 3], x[c], x[c + 1]);
                if (__any_sync(kFull, max3(most[0], most[1], fmaxf(most[2], most[3])) > 0.5f)) {
#pragma unroll
                    for (int c = 0; c < 64; ++c)
                        if (x[c] > 0.5f) {
                            top = x[c] * (CAP ? fmaf(th[c] * th[c], inv_cap2, 1.f) : 1.f);
                            top_j = j0 + c;
                        }
                }
                uint64_t sums[4] = {0ull, 0ull, 0ull, 0ull};
                if (!warp_wait(dp_full, (unsigned)step & 1u, p.wait_ns)) { stop = true; break; }
                tc_fence_after();
                if (n == 1) {
                    // all keys of these rows are here: delta itself before dS. Rows of few keys can have p near 1,
                    // where dP - delta cancels and the estimate's error shows in dq (a document of one token has
                    // dq = 0; two tokens: 0.0029 -> 0.0011 of dq besides its rounding)
                    uint64_t part = 0ull;
#pragma unroll 1
                    for (int c0 = 0; c0 < 64; c0 += 32) {
                        float dp[32];
                        tmem_ld32(tl + SH::TM_DP + t * 64 + c0, dp);
                        tmem_ld_wait();
#pragma unroll
                        for (int e = 0; e < 32; e += 2)
                            part = fma2(c0 ? pk2(x[32 + e], x[33 + e]) : pk2(x[e], x[e + 1]), pk2(dp[e], dp[e + 1]), part);
                    }
                    float p0, p1;
                    upk2(part, p0, p1);
                    s_part[t * R + r] = p0 + p1;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(part_full);
                    if (!warp_wait(part_full, singles, p.wait_ns)) { stop = true; break; }
                    singles ^= 1u;
                    est = s_part[r] + s_part[R + r] - dlse;
                }
                const uint64_t e2 = same2(-est);
#pragma unroll
                for (int c0 = 0; c0 < 64; c0 += 32) {
                    float dp[32];
                    tmem_ld32(tl + SH::TM_DP + t * 64 + c0, dp);
                    tmem_ld_wait();
                    uint32_t w[16];
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        const uint64_t ds = mul2(pk2(x[c0 + e], x[c0 + e + 1]), add2(pk2(dp[e], dp[e + 1]), e2));
                        sums[(e / 2) & 3] = add2(sums[(e / 2) & 3], ds);
                        float u, v;
                        upk2(CAP ? mul2(ds, cap_slope2(th[c0 + e], th[c0 + e + 1], inv_cap2)) : ds, u, v);
                        w[e / 2] = pack_bf16(u, v);   // dS enters dS K as bf16: 2^-8 each, as dq's own rounding
                    }
                    tmem_st16(tl + SH::TM_DP + t * 64 + c0 / 2, w);
                }
                float s0, s1;
                upk2(add2(add2(sums[0], sums[1]), add2(sums[2], sums[3])), s0, s1);
                rsum += s0 + s1;
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(ds_full);
            }
            if (stop) break;
            float fix = 0.f;   // eps p of the key that is kept
            if (t == 1) {
                // the first warpgroup has begun this unit, so it has read the last one's sums and parts, and with more
                // than one tile (both warpgroups take part in each) this one's estimates
                if (!warp_wait(a_full, (unsigned)uc & 1u, p.wait_ns)) { stop = true; break; }
                s_sum[r] = rsum;
                if (n > 1) {
                    s_est[r] = top;
                    reinterpret_cast<int*>(s_part)[r] = top_j;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(sum_full);
                if (!warp_wait(fix_full, (unsigned)uc & 1u, p.wait_ns)) { stop = true; break; }
                if (n > 1) {
                    fix = s_sum[r];
                    top_j = reinterpret_cast<int*>(s_part)[r];
                }
            } else {
                if (!warp_wait(sum_full, (unsigned)uc & 1u, p.wait_ns)) { stop = true; break; }
                const float eps = rsum + s_sum[r] - dlse;
                if (valid) p.delta[row] = est + eps;
                if (n > 1) {
                    if (s_est[r] > 0.f) {
                        top = s_est[r];
                        top_j = reinterpret_cast<int*>(s_part)[r];
                    }
                    if (valid) fix = eps * top;
                    s_sum[r] = fix;
                    reinterpret_cast<int*>(s_part)[r] = top_j;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(fix_full);
            }
            const bool fixes = __any_sync(kFull, fix != 0.f);
            // the next unit's rows are on their way while this one's last product runs
            if (!next(uc + 1) || !warp_wait(o_full, (unsigned)uc & 1u, p.wait_ns)) { stop = true; break; }
            tc_fence_after();
            uint4* dst = reinterpret_cast<uint4*>(p.dq + row * D);
#pragma unroll 1
            for (int c0 = t * (D / 2); c0 < (t + 1) * (D / 2); c0 += 32) {
                float o[32];
                tmem_ld32(tl + SH::TM_DQ + c0, o);
                tmem_ld_wait();
                if (fixes) {
                    const uint4* k4 = reinterpret_cast<const uint4*>(keys + (long long)top_j * p.kv_st + c0);
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        float kf[8];
                        unpack8(k4[c], kf);
#pragma unroll
                        for (int e = 0; e < 8; ++e) o[8 * c + e] = fmaf(-fix, kf[e], o[8 * c + e]);
                    }
                }
                if (valid) store_bf16x32(dst + c0 / 8, o, p.scale);
            }
        }
        if (stop && lane == 0) fail();
    }

    // ---- teardown: copies and products in flight finish (bounded) before the tensor memory goes
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 8) {
        if (elect_one()) umma_commit(fin);   // by the lane that issued the products
        __syncwarp();
        mbar_wait(fin, 0u);
    }
    if (tid == 0 && *s_abort) {
        for (int k = max(0, s_steps[0] - ST); k < s_steps[0]; ++k)
            mbar_wait(&kv_full[k % ST], (unsigned)(k / ST) & 1u, 100000000ull);
    }
    if (tid == 0) p.dq_done[blockIdx.x] = *s_abort ? 0 : 1;
    __syncthreads();
    if (warp == 8) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(SH::TM_COLS) : "memory");
    }
}

template <int D>
struct DkvShape {
    static constexpr int KT = 128, QT = 128;             // keys of a unit; query rows of a step (QT / G tokens)
    static constexpr int ST = D == 128 ? 2 : 4;
    static constexpr int NT = 12 * 32;
    static constexpr int REG_SOFT = 208, REG_REST = 88;
    // P is handed over in two halves where the products are short beside the exponentials (d 64: 681 -> 636 us
    // at 8192 tokens, 32/8 heads); at d 128 the products bound the kernel and the extra hand-over costs (858 -> 897)
    static constexpr bool SPLIT_P = D == 64;
    static constexpr int HALF = 128 * 128, TILE = HALF * (D / 64);
    static constexpr int K_OFF = 0;                      // K, V
    static constexpr int QO_OFF = K_OFF + 2 * TILE;      // [ST] Q, dO
    static constexpr int KX_OFF = QO_OFF + ST * 2 * TILE;
    static constexpr int ONE_OFF = KX_OFF + KT * 32;     // key columns without a bias
    static constexpr int QX_OFF = ONE_OFF + KT * 32;     // [ST] extra columns of Q, of dO
    static constexpr int ROW_OFF = QX_OFF + ST * 2 * QT * 32;   // [ST][128] lse in log2 units
    static constexpr int TOK_OFF = ROW_OFF + ST * QT * 4;   // [64] token of a row within its half step, as float
    static constexpr int DB_OFF = TOK_OFF + 64 * 4;      // [128] d log beta of the second warpgroup's columns
    static constexpr int INFO_OFF = DB_OFF + KT * 4;
    static constexpr int BAR_OFF = INFO_OFF + 2 * 8 * 4;
    static constexpr int NBAR = 2 + 3 * ST + 7 + 4;
    static constexpr int MISC_OFF = BAR_OFF + NBAR * 8;
    static constexpr size_t SMEM = 1024 + MISC_OFF + 32;
    static constexpr int TM_S = 0, TM_DP = 128, TM_DV = 256, TM_DK = 384, TM_COLS = 512;
    static_assert(SMEM <= 227 * 1024, "shared memory");
};

template <int D, bool BETA, bool CAP>
__global__ void __launch_bounds__(DkvShape<D>::NT, 1)
    prefill_dkv_kernel(const __grid_constant__ PrefillParams p, const __grid_constant__ CUtensorMap tmQ,
                       const __grid_constant__ CUtensorMap tmO, const __grid_constant__ CUtensorMap tmK,
                       const __grid_constant__ CUtensorMap tmV) {
    using SH = DkvShape<D>;
    constexpr int ST = SH::ST, KT = SH::KT, QT = SH::QT;
    extern __shared__ unsigned char smem_dyn[];
    unsigned char* smem = reinterpret_cast<unsigned char*>(
        (reinterpret_cast<uintptr_t>(smem_dyn) + 1023) & ~static_cast<uintptr_t>(1023));
    const uint32_t sbase = smem_u32(smem);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + SH::BAR_OFF);
    uint64_t* k_full = bars;
    uint64_t* k_empty = bars + 1;
    uint64_t* q_full = bars + 2;
    uint64_t* q_empty = q_full + ST;
    uint64_t* x_full = q_empty + ST;     // extra columns, row values; rows past the document cleared
    uint64_t* s_full = x_full + ST;
    uint64_t* dp_full = s_full + 1;
    uint64_t* p_half = s_full + 2;       // the weights of each half's first 32 columns, all of them
    uint64_t* p_full = s_full + 3;
    uint64_t* ds_full = s_full + 4;
    uint64_t* o_full = s_full + 5;       // dV, dK
    uint64_t* db_full = s_full + 6;      // the second warpgroup's part of d log beta
    uint64_t* u_full = db_full + 1;
    uint64_t* u_empty = u_full + 2;
    int* info = reinterpret_cast<int*>(smem + SH::INFO_OFF);
    uint32_t* tslot = reinterpret_cast<uint32_t*>(smem + SH::MISC_OFF);
    volatile int* s_abort = reinterpret_cast<int*>(smem + SH::MISC_OFF) + 1;
    int* s_steps = reinterpret_cast<int*>(smem + SH::MISC_OFF) + 2;
    uint64_t* fin = reinterpret_cast<uint64_t*>(smem + SH::MISC_OFF + 16);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int lg = 31 - __clz(p.G), bt = QT >> lg;      // tokens of a step
    if (tid == 0) {
        mbar_init(k_full, 1);
        mbar_init(k_empty, 1);
        for (int s = 0; s < ST; ++s) {
            mbar_init(&q_full[s], 1);
            mbar_init(&q_empty[s], 1);
            mbar_init(&x_full[s], 1);
        }
        mbar_init(s_full, 1);
        mbar_init(dp_full, 1);
        mbar_init(p_half, 8);
        mbar_init(p_full, 8);
        mbar_init(ds_full, 8);
        mbar_init(o_full, 1);
        mbar_init(db_full, 4);
        for (int t = 0; t < 2; ++t) {
            mbar_init(&u_full[t], 1);
            mbar_init(&u_empty[t], 11);
        }
        mbar_init(fin, 1);
        *s_abort = 0;
        s_steps[0] = s_steps[1] = 0;
        fence_mbar_init();
    }
    if (tid < 64) reinterpret_cast<float*>(smem + SH::TOK_OFF)[tid] = (float)(tid >> lg);
    if (tid < KT) {
        *reinterpret_cast<uint4*>(smem + SH::ONE_OFF + plain16_off(tid, 0)) = make_uint4(0u, 0u, 0u, 0u);
        *reinterpret_cast<uint4*>(smem + SH::ONE_OFF + plain16_off(tid, 1)) = make_uint4(0u, 0u, 0x3f803f80u, 0x3f80u);
    }
    fence_proxy_async_smem();
    if (warp == 9 && lane == 0) {
        prefetch_tensormap(&tmQ);
        prefetch_tensormap(&tmO);
        prefetch_tensormap(&tmK);
        prefetch_tensormap(&tmV);
    }
    if (warp == 8) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tslot)),
                     "r"(SH::TM_COLS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    griddep_wait();
    griddep_launch_dependents();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tslot;
    auto fail = [&]() {
        raise_error(KVB_DERR_TIMEOUT);
        *s_abort = 1;
    };

    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(SH::REG_REST));
        if (warp == 9) {
            // ======================= units and loads =======================
            int done = 1;   // its loads go out together, ahead of the walks' own
            static_assert(kMaxPieces % 32 == 0, "a lane per CTA");
#pragma unroll
            for (int c = 0; c < kMaxPieces; c += 32)
                if (c + lane < p.dq_ctas) done &= p.dq_done[c + lane];
            const StepLine line(p);
            const bool cut = line.cut(gridDim.x);
            const long long piece = line.piece(gridDim.x), x1 = min((blockIdx.x + 1) * piece, line.steps);
            const PrefillWalk walk(p, 7);
            // where a CTA of the kernel by query rows gave up, its deltas are not there: nothing is done
            const bool lost = __any_sync(kFull, done == 0);
            int step = 0, uc = 0;
            bool stop = false;
            long long x = blockIdx.x * piece, round = 0;
            int4 record = make_int4(0, 0, 0, -1);
            for (;; ++uc) {
                bool end;
                int s = 0, len = 0, g = 0, pre = 0, j0 = 0, b0 = 0, b1 = 0, part = 0;
                if (cut) {
                    end = lost || x >= x1;
                    if (!end) {
                        const StepLine::At u = line.find(x);
                        const long long till = min(u.end, x1);
                        s = u.d.s, len = u.d.len, pre = u.d.pre, g = u.g;
                        j0 = u.kb * KT;
                        b0 = u.b0 + (int)(x - u.begin);
                        b1 = u.b0 + (int)(till - u.begin);
                        // a whole key block (0), one that began in an earlier piece (1), one that goes on in the next (2)
                        part = x > u.begin ? 1 : (till < u.end ? 2 : 0);
                        if (part == 2) record = make_int4(s + j0, min(len - j0, KT), g, (int)((u.end - 1) / piece));
                        x = till;
                    }
                } else {
                    long long u = PrefillWalk::nth(round, blockIdx.x, gridDim.x);
                    end = lost || round * gridDim.x >= walk.units;
                    if (!end && u >= walk.units) {
                        end = true;   // a last round without this CTA
                    }
                    if (!end) {
                        const PrefillUnit w = walk.unit(u);
                        s = w.s, len = w.len, pre = w.pre, g = w.g;
                        // the first keys meet the most queries: the heaviest level is block 0
                        j0 = ((len + KT - 1) / KT - 1 - w.blk) * KT;
                        b0 = j0 < pre ? 0 : j0 / bt;
                        b1 = (len + bt - 1) / bt;
                        ++round;
                    }
                }
                const int ub = uc & 1;
                if (uc >= 2 && !warp_wait(&u_empty[ub], (unsigned)((uc >> 1) - 1) & 1u, p.wait_ns)) { stop = true; break; }
                if (__any_sync(kFull, *s_abort != 0)) break;
                if (lane == 0) {
                    int* m = info + ub * 8;
                    m[0] = end ? -1 : s;
                    m[1] = len;
                    m[2] = j0;
                    m[3] = g;
                    m[4] = pre;
                    m[5] = b0;
                    m[6] = b1;
                    m[7] = part;
                    mbar_arrive(&u_full[ub]);
                }
                __syncwarp();
                if (end) break;
                if (uc >= 1 && !warp_wait(k_empty, (unsigned)(uc - 1) & 1u, p.wait_ns)) { stop = true; break; }
                if (lane == 0) {
                    mbar_arrive_expect_tx(k_full, (unsigned)(2 * SH::TILE));
                    for (int h = 0; h < D / 64; ++h) {
                        unsigned char* at = smem + SH::K_OFF + h * SH::HALF;
                        tma_load_3d(at, &tmK, 64 * h, g, s + j0, k_full);
                        tma_load_3d(at + SH::TILE, &tmV, 64 * h, g, s + j0, k_full);
                    }
                    s_steps[1] = uc + 1;
                }
                const int till = p.withhold == blockIdx.x + 1 ? min(b1, b0 + max(1 - step, 0)) : b1;   // test hook
                for (int b = b0; b < till; ++b, ++step) {
                    const int st = step % ST;
                    if (step >= ST && !warp_wait(&q_empty[st], (unsigned)((step / ST) - 1) & 1u, p.wait_ns)) { stop = true; break; }
                    if (lane == 0) {
                        mbar_arrive_expect_tx(&q_full[st], (unsigned)(2 * SH::TILE));
                        for (int h = 0; h < D / 64; ++h) {
                            unsigned char* at = smem + SH::QO_OFF + st * 2 * SH::TILE + h * SH::HALF;
                            tma_load_3d(at, &tmQ, 64 * h, g << lg, s + b * bt, &q_full[st]);
                            tma_load_3d(at + SH::TILE, &tmO, 64 * h, g << lg, s + b * bt, &q_full[st]);
                        }
                        s_steps[0] = step + 1;
                    }
                    if (__any_sync(kFull, *s_abort != 0)) { stop = true; break; }
                }
                if (stop || till < b1) break;
            }
            if (lane == 0) p.records[blockIdx.x] = record;
            if (stop && lane == 0) fail();
        } else if (warp >= 10) {
            // ======================= extra columns, row values, rows past a document's end =======================
            // two warps, a step each in turn; the rows' numbers of a warp's next step load while it writes this one's
            int step = 0;
            bool stop = false;
            for (int uc = 0; !stop; ++uc) {
                const int ub = uc & 1;
                if (!warp_wait(&u_full[ub], (unsigned)(uc >> 1) & 1u, p.wait_ns)) { stop = true; break; }
                const int* m = info + ub * 8;
                const int s = m[0], len = m[1], j0 = m[2], g = m[3], b0 = m[5], b1 = m[6];
                __syncwarp();
                if (lane == 0) mbar_arrive(&u_empty[ub]);
                if (s < 0) break;
                const int last = j0 + KT - 1, n = b1 - b0;
                float lse[4], delta[4];
                auto load = [&](int blk) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int c = lane + 32 * e, i = blk * bt + (c >> lg);
                        lse[e] = 1.2676506e30f;   // no such row (2^100): P = 0
                        delta[e] = 0.f;
                        if (i < len) {
                            const size_t row = (size_t)(s + i) * p.Hq + (g << lg) + (c & (p.G - 1));
                            lse[e] = p.lse[row];
                            delta[e] = p.delta[row];
                        }
                    }
                };
                const int q0 = (step + warp) & 1;   // this warp's first step of the unit
                load(b0 + q0);
                if (BETA && !CAP && warp == 10 + (step & 1)) {   // the warp of the unit's first step
                    float b[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int j = j0 + lane + 32 * e;
                        b[e] = j < len ? clamp_log_beta(p.lb[(long long)(s + j) * p.lb_st + g * p.lb_sh]) / p.scale : 0.f;
                    }
                    if (uc >= 1 && !warp_wait(k_empty, (unsigned)(uc - 1) & 1u, p.wait_ns)) { stop = true; break; }
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int c = lane + 32 * e;
                        uint4 c0, c1;
                        far_key(b[e], last - j0 - c, c0, c1);
                        *reinterpret_cast<uint4*>(smem + SH::KX_OFF + plain16_off(c, 0)) = c0;
                        *reinterpret_cast<uint4*>(smem + SH::KX_OFF + plain16_off(c, 1)) = c1;
                    }
                }
                for (int q = q0; q < n; q += 2) {
                    const int blk = b0 + q, k = step + q, st = k % ST;
                    const unsigned ph = (unsigned)(k / ST) & 1u;
                    float y[4], dl[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        y[e] = lse[e] * (CAP ? kLog2e : -1.f / p.scale);
                        dl[e] = -delta[e];
                    }
                    load(blk + 2);
                    if (k >= ST && !warp_wait(&q_empty[st], ph ^ 1u, p.wait_ns)) { stop = true; break; }
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int c = lane + 32 * e;
                        uint4 c0, c1;
                        unsigned char* at = smem + SH::QX_OFF + st * 2 * QT * 32;
                        if (CAP) {
                            reinterpret_cast<float*>(smem + SH::ROW_OFF)[st * QT + c] = y[e];
                        } else {
                            far_query(BETA ? max(blk * bt + (c >> lg) - last, 0) : 0, y[e], c0, c1);
                            *reinterpret_cast<uint4*>(at + plain16_off(c, 0)) = c0;
                            *reinterpret_cast<uint4*>(at + plain16_off(c, 1)) = c1;
                        }
                        far_query(0, dl[e], c0, c1);
                        *reinterpret_cast<uint4*>(at + QT * 32 + plain16_off(c, 0)) = c0;
                        *reinterpret_cast<uint4*>(at + QT * 32 + plain16_off(c, 1)) = c1;
                    }
                    if ((blk + 1) * bt > len) {
                        if (!warp_wait(&q_full[st], ph, p.wait_ns)) { stop = true; break; }
                        const int rows = (len - blk * bt) << lg;
                        unsigned char* qt = smem + SH::QO_OFF + st * 2 * SH::TILE;
                        for (int x = lane; x < (QT - rows) * 16 * (D / 64); x += 32) {
                            const int row = rows + x / (16 * (D / 64)), c = x % (16 * (D / 64));   // chunks of Q, then of dO
                            *reinterpret_cast<uint4*>(qt + (c >> 3) * SH::HALF + row * 128 + ((c & 7) << 4)) =
                                make_uint4(0u, 0u, 0u, 0u);
                        }
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&x_full[st]);
                    if (__any_sync(kFull, *s_abort != 0)) { stop = true; break; }
                }
                step += n;
            }
            if (stop && lane == 0) fail();
        } else if (warp == 8) {
            // ======================= products =======================
            // the warp stays together (its values are uniform); one lane issues
            constexpr uint32_t idesc_s = umma_idesc_bf16(KT, QT), idesc_o = umma_idesc_bf16_bmn(KT, D);
            int step = 0;
            bool stop = false;
            const uint32_t k_lo = desc_sw128_lo(sbase + SH::K_OFF), q_lo = desc_sw128_lo(sbase + SH::QO_OFF);
            const uint32_t qr_lo = desc_mn_lo(sbase + SH::QO_OFF, SH::HALF);
            const uint32_t kx_lo = desc_plain_lo(sbase + SH::KX_OFF), qx_lo = desc_plain_lo(sbase + SH::QX_OFF);
            const uint32_t one_lo = desc_plain_lo(sbase + SH::ONE_OFF);
            auto scores = [&](int st, bool past) {
                umma_kmajor<D / 16>(tmem + SH::TM_S, k_lo, SH::HALF, q_lo + st * (2 * SH::TILE >> 4), SH::HALF, idesc_s);
                if (!CAP)   // - lse, and the bias where every query is past every key
                    umma_bf16(tmem + SH::TM_S, desc(BETA && past ? kx_lo : one_lo, kDescPlainHi),
                              desc(qx_lo + st * (2 * QT * 32 >> 4), kDescPlainHi), idesc_s, 1u);
                umma_commit(s_full);
            };
            auto pulls = [&](int st) {
                umma_kmajor<D / 16>(tmem + SH::TM_DP, k_lo + (SH::TILE >> 4), SH::HALF, q_lo + (st * 2 + 1) * (SH::TILE >> 4),
                                    SH::HALF, idesc_s);
                umma_bf16(tmem + SH::TM_DP, desc(one_lo, kDescPlainHi), desc(qx_lo + (st * 2 + 1) * (QT * 32 >> 4), kDescPlainHi),
                          idesc_s, 1u);   // - delta
                umma_commit(dp_full);
            };
            // P^T and dS^T: a warpgroup's 64 columns as 32 words at the start of its half; 32 columns of each
            auto grad_half = [&](uint32_t d, uint32_t a, uint32_t b, bool fresh) {
                umma_rows<2>(d, a, b, idesc_o, fresh);
                umma_rows<2>(d, a + 64, b + 64 * 128 / 16, idesc_o, false);
            };
            auto loaded = [&](int k) {
                return warp_wait(&q_full[k % ST], (unsigned)(k / ST) & 1u, p.wait_ns) &&
                       warp_wait(&x_full[k % ST], (unsigned)(k / ST) & 1u, p.wait_ns);
            };
            for (int uc = 0; !stop; ++uc) {
                const int ub = uc & 1;
                if (!warp_wait(&u_full[ub], (unsigned)(uc >> 1) & 1u, p.wait_ns)) { stop = true; break; }
                const int* m = info + ub * 8;
                const int s = __shfl_sync(kFull, m[0], 0), j0 = __shfl_sync(kFull, m[2], 0);
                const int b0 = __shfl_sync(kFull, m[5], 0), b1 = __shfl_sync(kFull, m[6], 0);
                if (lane == 0) mbar_arrive(&u_empty[ub]);
                if (s < 0) break;
                const int n = b1 - b0, last = j0 + KT - 1;
                if (!warp_wait(k_full, (unsigned)uc & 1u, p.wait_ns) || !loaded(step)) { stop = true; break; }
                // S and dP were read before the previous unit's last P and dS
                tc_fence_after();
                if (elect_one()) {
                    scores(step % ST, b0 * bt >= last);
                    pulls(step % ST);
                }
                __syncwarp();
                for (int q = 0; q < n; ++q, ++step) {
                    const int st = step % ST, nst = (step + 1) % ST;
                    const bool more = q + 1 < n;
                    const uint32_t rows = qr_lo + st * (2 * SH::TILE >> 4);
                    if (SH::SPLIT_P) {
                        if (!warp_wait(p_half, (unsigned)step & 1u, p.wait_ns)) { stop = true; break; }
                        tc_fence_after();
                        if (elect_one()) grad_half(tmem + SH::TM_DV, tmem + SH::TM_S, rows + (SH::TILE >> 4), q == 0);
                        __syncwarp();
                    }
                    if (more && !loaded(step + 1)) { stop = true; break; }
                    if (!warp_wait(p_full, (unsigned)step & 1u, p.wait_ns)) { stop = true; break; }
                    tc_fence_after();
                    if (elect_one()) {
                        if (!SH::SPLIT_P) grad_half(tmem + SH::TM_DV, tmem + SH::TM_S, rows + (SH::TILE >> 4), q == 0);
                        grad_half(tmem + SH::TM_DV, tmem + SH::TM_S + 16, rows + (SH::TILE >> 4) + 32 * 128 / 16, false);
                        if (more) scores(nst, (b0 + q + 1) * bt >= last);
                    }
                    __syncwarp();
                    if (!warp_wait(ds_full, (unsigned)step & 1u, p.wait_ns)) { stop = true; break; }
                    tc_fence_after();
                    if (elect_one()) {
                        grad_half(tmem + SH::TM_DK, tmem + SH::TM_DP, rows, q == 0);
                        grad_half(tmem + SH::TM_DK, tmem + SH::TM_DP + 16, rows + 32 * 128 / 16, false);
                        umma_commit(&q_empty[st]);
                        if (more) {
                            pulls(nst);
                        } else {
                            umma_commit(k_empty);
                            umma_commit(o_full);
                        }
                    }
                    __syncwarp();
                }
                if (stop) break;
            }
            if (stop && lane == 0) fail();
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(SH::REG_SOFT));
        // ======================= P^T and dS^T of a key row; dV, dK, d log beta =======================
        const int t = warp >> 2, quarter = warp & 3;        // columns 64 t .. of every step
        const int r = 32 * quarter + lane;
        const uint32_t tl = tmem + ((uint32_t)(32 * quarter) << 16);
        const float C = CAP ? 1.f : p.scale * kLog2e;
        const float cap2 = CAP ? p.softcap * kLog2e : 0.f, per_cap = CAP ? p.scale / p.softcap : 0.f;
        const float inv_cap2 = CAP ? -1.f / (cap2 * cap2) : 0.f;
        const float4* tok4 = reinterpret_cast<const float4*>(smem + SH::TOK_OFF);
        float* s_db = reinterpret_cast<float*>(smem + SH::DB_OFF);
        int step = 0;
        bool stop = false;
        for (int uc = 0; !stop; ++uc) {
            const int ub = uc & 1;
            if (!warp_wait(&u_full[ub], (unsigned)(uc >> 1) & 1u, p.wait_ns)) { stop = true; break; }
            const int* m = info + ub * 8;
            const int s = m[0], len = m[1], j0 = m[2], g = m[3], pre = m[4], b0 = m[5], b1 = m[6], part = m[7];
            __syncwarp();
            if (lane == 0) mbar_arrive(&u_empty[ub]);
            if (s < 0) break;
            const int last = j0 + KT - 1;
            const int j = j0 + r;
            const float slope_b = (BETA && j < len) ? clamp_log_beta(p.lb[(long long)(s + j) * p.lb_st + g * p.lb_sh]) *
                                                          (CAP ? kLog2e : 1.f / p.scale)
                                                    : 0.f;
            float db = 0.f;
            for (int blk = b0; blk < b1; ++blk, ++step) {
                const int st = step % ST, tb = blk * bt + ((64 * t) >> lg);   // this half's first token
                const bool past = blk * bt >= last;
                const float di = (float)(tb - j);
                // ---- P
                if (!warp_wait(s_full, (unsigned)step & 1u, p.wait_ns)) { stop = true; break; }
                tc_fence_after();
                float x[64], th[CAP ? 64 : 1];
                tmem_ld32(tl + SH::TM_S + t * 64, x);
                tmem_ld32(tl + SH::TM_S + t * 64 + 32, x + 32);
                tmem_ld_wait();
                if (CAP) {
                    if (!warp_wait(&x_full[st], (unsigned)(step / ST) & 1u, p.wait_ns)) { stop = true; break; }
                    const float4* l4 = reinterpret_cast<const float4*>(smem + SH::ROW_OFF + (st * QT + 64 * t) * 4);
                    cap_scores<64>(x, per_cap, cap2);
                    // + (di + c >> lg) b where all is past: by blocks of eight columns
                    const float in_block = BETA && past ? slope_b : 0.f, per_block = in_block * (float)(8 >> lg);
                    uint64_t by2[4];
#pragma unroll
                    for (int e = 0; e < 8; e += 2) by2[e / 2] = pk2((float)(e >> lg) * in_block, (float)((e + 1) >> lg) * in_block);
                    float block = di * in_block;
#pragma unroll
                    for (int c = 0; c < 64; c += 4) {
                        const float4 l = l4[c / 4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) th[c + e] = x[c + e];
                        const uint64_t at = same2(block);
                        const uint64_t u = add2(add2(by2[(c / 2) & 3], at), pk2(-l.x, -l.y));
                        const uint64_t w = add2(add2(by2[(c / 2 + 1) & 3], at), pk2(-l.z, -l.w));
                        upk2(add2(pk2(x[c], x[c + 1]), u), x[c], x[c + 1]);
                        upk2(add2(pk2(x[c + 2], x[c + 3]), w), x[c + 2], x[c + 3]);
                        if (c % 8 == 4) block += per_block;
                    }
                }
                if (BETA && !past) {
#pragma unroll
                    for (int c = 0; c < 64; c += 4) {
                        const float4 k4 = tok4[c / 4];
                        x[c] = fmaf(fmaxf(di + k4.x, 0.f), slope_b, x[c]);
                        x[c + 1] = fmaf(fmaxf(di + k4.y, 0.f), slope_b, x[c + 1]);
                        x[c + 2] = fmaf(fmaxf(di + k4.z, 0.f), slope_b, x[c + 2]);
                        x[c + 3] = fmaf(fmaxf(di + k4.w, 0.f), slope_b, x[c + 3]);
                    }
                }
                if (!past) {
                    const int from = j < pre ? 0 : min(max(j - tb, 0) << lg, 64);   // the first row that sees key j
#pragma unroll
                    for (int c = 0; c < 64; ++c) x[c] = c >= from ? x[c] : -INFINITY;
                }
                const uint64_t c2 = pk2(C, C);
#pragma unroll
                for (int c0 = 0; c0 < 64; c0 += 32) {
                    uint32_t w[16];
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        float a, b;
                        upk2(CAP ? pk2(x[c0 + e], x[c0 + e + 1]) : mul2(pk2(x[c0 + e], x[c0 + e + 1]), c2), a, b);
                        if (D == 64 && e % 8 == 6) {   // a quarter of the exponentials on the FMA pipe, as forward
                            exp2_poly2<5>(a, b);
                        } else {
                            a = ex2_approx(a);
                            b = ex2_approx(b);
                        }
                        x[c0 + e] = a;
                        x[c0 + e + 1] = b;
                        w[e / 2] = pack_bf16(a, b);   // P and dS enter the gradients' products as bf16: 2^-8 each
                    }
                    tmem_st16(tl + SH::TM_S + t * 64 + c0 / 2, w);
                    if (SH::SPLIT_P || c0 > 0) {
                        tmem_st_wait();
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(c0 == 0 ? p_half : p_full);
                    }
                }
                // ---- dS
                if (!warp_wait(dp_full, (unsigned)step & 1u, p.wait_ns)) { stop = true; break; }
                tc_fence_after();
                uint64_t ds[32];
#pragma unroll
                for (int c0 = 0; c0 < 64; c0 += 32) {
                    float dp[32];
                    uint32_t w[16];
                    tmem_ld32(tl + SH::TM_DP + t * 64 + c0, dp);
                    tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        const uint64_t d = mul2(pk2(x[c0 + e], x[c0 + e + 1]), pk2(dp[e], dp[e + 1]));
                        ds[(c0 + e) / 2] = d;
                        float a, b;
                        upk2(CAP ? mul2(d, cap_slope2(th[c0 + e], th[c0 + e + 1], inv_cap2)) : d, a, b);
                        w[e / 2] = pack_bf16(a, b);
                    }
                    tmem_st16(tl + SH::TM_DP + t * 64 + c0 / 2, w);
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(ds_full);
                // ---- d log beta, while the products run. Where all is past: sum dS (di + tok(c)), tok(c) =
                // c >> lg, from the eight sums over c = e mod 8 and from sum (c / 8) dS; else one by one
                if (BETA) {
                    if (past) {
                        uint64_t by8[4], up = 0ull;
#pragma unroll
                        for (int e = 0; e < 4; ++e) by8[e] = ds[e];
#pragma unroll
                        for (int c = 4; c < 32; c += 4) {
                            uint64_t four = add2(add2(ds[c], ds[c + 1]), add2(ds[c + 2], ds[c + 3]));
                            up = fma2(four, same2((float)(c / 4)), up);
#pragma unroll
                            for (int e = 0; e < 4; ++e) by8[e] = add2(by8[e], ds[c + e]);
                        }
                        float u0, u1, all = 0.f;
                        upk2(up, u0, u1);
                        float part = (u0 + u1) * (float)(8 >> lg);
#pragma unroll
                        for (int e = 0; e < 8; e += 2) {
                            float a, b;
                            upk2(by8[e / 2], a, b);
                            all += a + b;
                            part = fmaf(a, (float)(e >> lg), part);
                            part = fmaf(b, (float)((e + 1) >> lg), part);
                        }
                        db += fmaf(all, di, part);
                    } else {
                        float u = 0.f, v = 0.f;
#pragma unroll
                        for (int c = 0; c < 64; c += 2) {
                            const float2 k2 = reinterpret_cast<const float2*>(tok4)[c / 2];
                            float a, b;
                            upk2(ds[c / 2], a, b);
                            u = fmaf(a, fmaxf(di + k2.x, 0.f), u);
                            v = fmaf(b, fmaxf(di + k2.y, 0.f), v);
                        }
                        db += u + v;
                    }
                }
            }
            if (stop) break;
            if (!warp_wait(o_full, (unsigned)uc & 1u, p.wait_ns)) { stop = true; break; }
            tc_fence_after();
            uint4* dst = reinterpret_cast<uint4*>((t ? p.dk : p.dv) + ((size_t)(s + j) * p.Hkv + g) * D);
            float* sums = p.parts + ((size_t)blockIdx.x * 2 + (part - 1)) * kPartFloats;   // where part > 0
#pragma unroll 1
            for (int c0 = 0; c0 < D; c0 += 32) {
                float o[32];
                tmem_ld32(tl + (t ? SH::TM_DK : SH::TM_DV) + c0, o);
                tmem_ld_wait();
                if (part) {
#pragma unroll
                    for (int c = 0; c < 32; ++c) sums[(t * 128 + c0 + c) * 128 + r] = o[c];
                } else if (j < len) {
                    store_bf16x32(dst + c0 / 8, o, t ? p.scale : 1.f);
                }
            }
            tc_fence_before();   // the next unit's products follow this thread's next P
            if (BETA) {
                // the next unit's part is posted only after this warpgroup's steps of that unit
                if (t == 1) {
                    s_db[r] = db;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(db_full);
                } else {
                    if (!warp_wait(db_full, (unsigned)uc & 1u, p.wait_ns)) { stop = true; break; }
                    if (part) {
                        sums[2 * 128 * 128 + r] = db + s_db[r];
                    } else if (j < len) {
                        p.dlb[(size_t)(s + j) * p.Hkv + g] = db + s_db[r];
                    }
                }
            }
        }
        if (stop && lane == 0) fail();
    }

    // ---- teardown: copies and products in flight finish (bounded) before the tensor memory goes
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 8) {
        if (elect_one()) umma_commit(fin);   // by the lane that issued the products
        __syncwarp();
        mbar_wait(fin, 0u);
    }
    if (tid == 0 && *s_abort) {
        for (int k = max(0, s_steps[0] - ST); k < s_steps[0]; ++k)
            mbar_wait(&q_full[k % ST], (unsigned)(k / ST) & 1u, 100000000ull);
        if (s_steps[1] > 0) mbar_wait(k_full, (unsigned)(s_steps[1] - 1) & 1u, 100000000ull);
        p.records[blockIdx.x].w = -2;
    }
    __syncthreads();
    if (warp == 8) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(SH::TM_COLS) : "memory");
    }
}

// The key blocks that a cut goes through: the sums of their pieces, in order. blockIdx.x names the piece that
// holds a key block's first step and not its last; a thread sums one key's 8 columns of dV or dK (the parts are
// [column][key], so that a warp's accesses are whole lines). A key block with a piece of a CTA that gave up stays
// as it was.
template <int D, bool BETA>
__global__ void __launch_bounds__(256) prefill_dkv_sum_kernel(const __grid_constant__ PrefillParams p) {
    griddep_wait();
    griddep_launch_dependents();
    const int4 rec = p.records[blockIdx.x];
    static_assert(kMaxPieces <= 256, "a thread per piece");
    const int piece = threadIdx.x, state = piece < gridDim.x ? p.records[piece].w : -1;
    if (rec.w < 0 || __syncthreads_or(piece > blockIdx.x && piece <= rec.w && state == -2)) return;
    const int r = threadIdx.x & 127;
    if (r >= rec.y) return;
    const int col = (blockIdx.y * 2 + (threadIdx.x >> 7)) * 8;   // of dV's D columns, then dK's
    const float* first = p.parts + ((size_t)blockIdx.x * 2 + 1) * kPartFloats;
    const float* others = p.parts + (size_t)blockIdx.x * 2 * kPartFloats;   // + 2 q kPartFloats: the q-th piece after
    const int at = (col < D ? col : 128 + col - D) * 128 + r, more = rec.w - blockIdx.x;
    float sum[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) sum[c] = first[at + c * 128];
#pragma unroll 4
    for (int q = 1; q <= more; ++q)
#pragma unroll
        for (int c = 0; c < 8; ++c) sum[c] += others[(size_t)q * 2 * kPartFloats + at + c * 128];
    const size_t row = (size_t)(rec.x + r) * p.Hkv + rec.z;
    const float f = col < D ? 1.f : p.scale;
    *reinterpret_cast<uint4*>((col < D ? p.dv + row * D + col : p.dk + row * D + col - D)) =
        make_uint4(pack_bf16(sum[0] * f, sum[1] * f), pack_bf16(sum[2] * f, sum[3] * f), pack_bf16(sum[4] * f, sum[5] * f),
                   pack_bf16(sum[6] * f, sum[7] * f));
    if (BETA && col == 0) {
        float b = first[2 * 128 * 128 + r];
        for (int q = 1; q <= more; ++q) b += others[(size_t)q * 2 * kPartFloats + 2 * 128 * 128 + r];
        p.dlb[row] = b;
    }
}

}  // namespace kvb
