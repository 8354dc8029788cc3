// Gradients of the prompt attention (kvb_prefill_attn_bwd) on the 5th-generation tensor cores, as two
// kernels, so that every sum runs in one CTA in a fixed order (no atomics, no fp32 copy of dq):
//
//   prefill_dq_kernel   per block of query rows: S = Q K^T, dP = dO V^T, P = exp2(C S - lse),
//                       dS = P (dP - delta), dQ += dS K; leaves delta for the second kernel
//   prefill_dkv_kernel  per block of keys: S^T, dP^T, then dV += P^T dO, dK += dS^T Q, and
//                       d log beta_j = sum_i dS_ij max(i - j, 0) in fp32
//
// delta_i = sum_j p_ij dP_ij - dlse_i. dO . o would give it from the output, but o is held in bf16
// (2^-9 relative), which d log beta, an fp32 result whose terms cancel, would show. The first kernel
// starts from that estimate e_i = dO . o - dlse_i; its row sums of dS are then sum_j p_ij dP_ij - e_i,
// so e_i + their sum - dlse_i is delta to fp32, for one addition per score. dq, held in bf16 itself,
// keeps the estimate.
//
// In both, key or query steps of 64 give every S and dP a 128 x 64 accumulator, and two of each pair
// are in flight: while a warpgroup turns one pair into P and dS, the products of the other run. The
// bias rides the S product as in prefill_fwd_kernel.
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
    static constexpr int R = 128, KT = 64;
    static constexpr int ST = D == 128 ? 2 : 4;
    static constexpr int NT = 12 * 32;
    static constexpr int REG_SOFT = 208, REG_REST = 88;
    static constexpr int QHALF = R * 128, QTILE = QHALF * (D / 64);
    static constexpr int KHALF = KT * 128, KTILE = KHALF * (D / 64);
    static constexpr int Q_OFF = 0;                      // Q of both tiles, then dO of both
    static constexpr int KV_OFF = Q_OFF + 4 * QTILE;     // [ST] K, V
    static constexpr int QX_OFF = KV_OFF + ST * 2 * KTILE;
    static constexpr int KX_OFF = QX_OFF + 2 * R * 32;
    static constexpr int LB_OFF = KX_OFF + ST * KT * 32;
    static constexpr int INFO_OFF = LB_OFF + ST * KT * 4;
    static constexpr int BAR_OFF = INFO_OFF + 2 * 8 * 4;
    static constexpr int NBAR = 2 + 3 * ST + 8 + 4;
    static constexpr int MISC_OFF = BAR_OFF + NBAR * 8;
    static constexpr size_t SMEM = 1024 + MISC_OFF + 32;
    static constexpr int TM_T = 256, TM_S = 0, TM_DP = 64, TM_DQ = 128, TM_COLS = 512;
    static_assert(SMEM <= 227 * 1024, "shared memory");
};

template <int D, bool BETA, bool CAP>
__global__ void __launch_bounds__(DqShape<D>::NT, 1)
    prefill_dq_kernel(const __grid_constant__ PrefillParams p, const __grid_constant__ CUtensorMap tmQ,
                      const __grid_constant__ CUtensorMap tmO, const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV) {
    using SH = DqShape<D>;
    constexpr int ST = SH::ST, R = SH::R, KT = SH::KT;
    extern __shared__ unsigned char smem_dyn[];
    unsigned char* smem = reinterpret_cast<unsigned char*>(
        (reinterpret_cast<uintptr_t>(smem_dyn) + 1023) & ~static_cast<uintptr_t>(1023));
    const uint32_t sbase = smem_u32(smem);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + SH::BAR_OFF);
    uint64_t* q_full = bars;
    uint64_t* q_empty = bars + 1;
    uint64_t* kv_full = bars + 2;
    uint64_t* kv_empty = kv_full + ST;
    uint64_t* x_full = kv_empty + ST;    // the bias columns and slopes; K's and V's rows past the document cleared
    uint64_t* s_full = x_full + ST;      // [tile] S and dP
    uint64_t* ds_full = s_full + 2;
    uint64_t* o_full = ds_full + 2;      // [tile] dQ
    uint64_t* o_empty = o_full + 2;
    uint64_t* u_full = o_empty + 2;
    uint64_t* u_empty = u_full + 2;
    int* info = reinterpret_cast<int*>(smem + SH::INFO_OFF);
    uint32_t* tslot = reinterpret_cast<uint32_t*>(smem + SH::MISC_OFF);
    volatile int* s_abort = reinterpret_cast<int*>(smem + SH::MISC_OFF) + 1;
    int* s_steps = reinterpret_cast<int*>(smem + SH::MISC_OFF) + 2;
    uint64_t* fin = reinterpret_cast<uint64_t*>(smem + SH::MISC_OFF + 16);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int lg = 31 - __clz(p.G), sh = 8 - lg;
    if (tid == 0) {
        mbar_init(q_full, 1);
        mbar_init(q_empty, 1);
        for (int s = 0; s < ST; ++s) {
            mbar_init(&kv_full[s], 1);
            mbar_init(&kv_empty[s], 1);
            mbar_init(&x_full[s], 1);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(&s_full[t], 1);
            mbar_init(&ds_full[t], 4);
            mbar_init(&o_full[t], 1);
            mbar_init(&o_empty[t], 4);
            mbar_init(&u_full[t], 1);
            mbar_init(&u_empty[t], 10);
        }
        mbar_init(fin, 1);
        *s_abort = 0;
        s_steps[0] = s_steps[1] = 0;
        fence_mbar_init();
    }
    if (warp == 9 && lane == 0) {
        prefetch_tensormap(&tmQ);
        prefetch_tensormap(&tmO);
        prefetch_tensormap(&tmK);
        prefetch_tensormap(&tmV);
    }
    if (BETA && !CAP) {
        for (int x = tid; x < 2 * R; x += SH::NT) {
            unsigned char* at = smem + SH::QX_OFF + (x >> 7) * R * 32;
            *reinterpret_cast<uint4*>(at + plain16_off(x & 127, 0)) = bias_query(x >> lg);
            *reinterpret_cast<uint4*>(at + plain16_off(x & 127, 1)) = make_uint4(0u, 0u, 0u, 0u);
        }
        for (int x = tid; x < ST * KT; x += SH::NT)
            *reinterpret_cast<uint4*>(smem + SH::KX_OFF + (x >> 6) * KT * 32 + plain16_off(x & 63, 1)) =
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
            const bool ok = prefill_docs_ok(p.cu, p.N, p.T);
            const PrefillWalk walk(p, sh);
            const long long units = ok ? walk.units : 0;
            int step = 0, uc = 0;
            bool stop = false;
            for (long long r = 0; !stop; ++r, ++uc) {
                const long long u = PrefillWalk::nth(r, blockIdx.x, gridDim.x);
                const bool end = r * gridDim.x >= units;
                if (!end && u >= units) { --uc; continue; }
                PrefillUnit x{};
                int n0 = 0, n1 = 0;
                if (!end) {
                    x = walk.unit(u);
                    const int bt = 1 << (sh - 1), i0 = x.blk << sh, i1 = i0 + bt;
                    n0 = (max(min(i1, x.len), x.pre) + KT - 1) / KT;
                    n1 = i1 < x.len ? (max(min(i1 + bt, x.len), x.pre) + KT - 1) / KT : 0;
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
                    m[5] = n0;
                    m[6] = n1;
                    mbar_arrive(&u_full[ub]);
                }
                __syncwarp();
                if (end) break;
                if (uc >= 1 && !warp_wait(q_empty, (unsigned)(uc - 1) & 1u, p.wait_ns)) { stop = true; break; }
                if (lane == 0) {
                    mbar_arrive_expect_tx(q_full, (unsigned)(4 * SH::QTILE));
                    for (int t = 0; t < 2; ++t)
                        for (int h = 0; h < D / 64; ++h) {
                            const int i = x.s + (x.blk << sh) + (t << (sh - 1));
                            unsigned char* at = smem + SH::Q_OFF + t * SH::QTILE + h * SH::QHALF;
                            tma_load_3d(at, &tmQ, 64 * h, x.g << lg, i, q_full);
                            tma_load_3d(at + 2 * SH::QTILE, &tmO, 64 * h, x.g << lg, i, q_full);
                        }
                    s_steps[1] = uc + 1;
                }
                for (int tile = max(n0, n1) - 1; tile >= 0; --tile, ++step) {
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
            }
            if (stop && lane == 0) fail();
        } else if (warp == 10) {
            // ======================= bias columns, K and V past a document's end =======================
            const float unit_b = CAP ? kLog2e : 1.f / p.scale;
            int step = 0;
            bool stop = false;
            for (int uc = 0; !stop; ++uc) {
                const int ub = uc & 1;
                if (!warp_wait(&u_full[ub], (unsigned)(uc >> 1) & 1u, p.wait_ns)) { stop = true; break; }
                const int* m = info + ub * 8;
                const int s = m[0], len = m[1], i0 = m[2], g = m[3], n = max(m[5], m[6]);
                __syncwarp();
                if (lane == 0) mbar_arrive(&u_empty[ub]);
                if (s < 0) break;
                for (int tile = n - 1; tile >= 0; --tile, ++step) {
                    const int st = step % ST;
                    const unsigned ph = (unsigned)(step / ST) & 1u;
                    float b[2] = {0.f, 0.f};
                    if (BETA) {
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int j = tile * KT + lane + 32 * e;
                            if (j < len) b[e] = clamp_log_beta(p.lb[(long long)(s + j) * p.lb_st + g * p.lb_sh]) * unit_b;
                        }
                    }
                    if (step >= ST && !warp_wait(&kv_empty[st], ph ^ 1u, p.wait_ns)) { stop = true; break; }
                    if (BETA) {
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
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
            }
            if (stop && lane == 0) fail();
        } else if (warp == 8) {
            // ======================= products =======================
            // the warp stays together (its values are uniform); one lane issues
            constexpr uint32_t idesc_s = umma_idesc_bf16(R, KT), idesc_o = umma_idesc_bf16_bmn(R, D);
            int step = 0;
            unsigned dc = 0;           // bit t: parity of tile t's next dS
            int oc0 = 0, oc1 = 0;
            bool stop = false;
            const uint32_t q_lo = desc_sw128_lo(sbase + SH::Q_OFF), k_lo = desc_sw128_lo(sbase + SH::KV_OFF);
            const uint32_t kr_lo = desc_mn_lo(sbase + SH::KV_OFF, SH::KHALF);
            const uint32_t qx_lo = desc_plain_lo(sbase + SH::QX_OFF), kx_lo = desc_plain_lo(sbase + SH::KX_OFF);
            auto scores = [&](int t, int st, bool past) {
                const uint32_t tm = tmem + t * SH::TM_T, q = q_lo + t * (SH::QTILE >> 4), k = k_lo + st * (2 * SH::KTILE >> 4);
                umma_kmajor<D / 16>(tm + SH::TM_S, q, SH::QHALF, k, SH::KHALF, idesc_s);
                if (BETA && !CAP && past)
                    umma_bf16(tm + SH::TM_S, desc(qx_lo + t * (R * 32 >> 4), kDescPlainHi),
                              desc(kx_lo + st * (KT * 32 >> 4), kDescPlainHi), idesc_s, 1u);
                umma_kmajor<D / 16>(tm + SH::TM_DP, q + (2 * SH::QTILE >> 4), SH::QHALF, k + (SH::KTILE >> 4), SH::KHALF, idesc_s);
                umma_commit(&s_full[t]);
            };
            auto loaded = [&](int k) {
                return warp_wait(&kv_full[k % ST], (unsigned)(k / ST) & 1u, p.wait_ns) &&
                       warp_wait(&x_full[k % ST], (unsigned)(k / ST) & 1u, p.wait_ns);
            };
            for (int uc = 0; !stop; ++uc) {
                const int ub = uc & 1;
                if (!warp_wait(&u_full[ub], (unsigned)(uc >> 1) & 1u, p.wait_ns)) { stop = true; break; }
                const int* m = info + ub * 8;
                const int s = __shfl_sync(kFull, m[0], 0), i0 = __shfl_sync(kFull, m[2], 0);
                const int n0 = __shfl_sync(kFull, m[5], 0), n1 = __shfl_sync(kFull, m[6], 0);
                if (lane == 0) mbar_arrive(&u_empty[ub]);
                if (s < 0) break;
                const int n = max(n0, n1), i1 = i0 + (1 << (sh - 1));
                if (!warp_wait(q_full, (unsigned)uc & 1u, p.wait_ns) || !loaded(step)) { stop = true; break; }
                tc_fence_after();
                if (elect_one()) {
                    if (n - 1 < n0) scores(0, step % ST, n * KT <= i0 + 1);
                    if (n - 1 < n1) scores(1, step % ST, n * KT <= i1 + 1);
                    if (n == 1) umma_commit(q_empty);
                }
                __syncwarp();
                for (int tile = n - 1; tile >= 0; --tile, ++step) {
                    const int st = step % ST;
                    const bool more = tile > 0;
                    if (more && !loaded(step + 1)) { stop = true; break; }
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        const int nt = t ? n1 : n0;
                        const bool have = tile < nt, first = tile == nt - 1;
                        if (have) {
                            if (!warp_wait(&ds_full[t], (dc >> t) & 1u, p.wait_ns)) { stop = true; break; }
                            dc ^= 1u << t;
                            if (first) {
                                int& oc = t ? oc1 : oc0;
                                if (oc > 0 && !warp_wait(&o_empty[t], (unsigned)(oc - 1) & 1u, p.wait_ns)) { stop = true; break; }
                                ++oc;
                            }
                        }
                        tc_fence_after();
                        if (elect_one()) {
                            if (have) {
                                umma_rows<KT / 16>(tmem + t * SH::TM_T + SH::TM_DQ, tmem + t * SH::TM_T + SH::TM_S,
                                                   kr_lo + st * (2 * SH::KTILE >> 4), idesc_o, first);
                                if (tile == 0) umma_commit(&o_full[t]);
                            }
                            if (t == 1) umma_commit(&kv_empty[st]);
                            if (more && tile - 1 < nt) scores(t, (step + 1) % ST, tile * KT <= (t ? i1 : i0) + 1);
                            if (t == 1 && tile == 1) umma_commit(q_empty);
                        }
                        __syncwarp();
                    }
                    if (stop) break;
                }
            }
            if (stop && lane == 0) fail();
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(SH::REG_SOFT));
        // ======================= dS of a tile's rows, dQ and delta =======================
        const int t = warp >> 2, quarter = warp & 3;
        const int r = 32 * quarter + lane;
        const uint32_t tb = tmem + ((uint32_t)(32 * quarter) << 16) + t * SH::TM_T;
        const float C = CAP ? 1.f : p.scale * kLog2e;
        const float cap2 = CAP ? p.softcap * kLog2e : 0.f, per_cap = CAP ? p.scale / p.softcap : 0.f;
        int sc = 0, step = 0, oc = 0;
        bool stop = false;
        for (int uc = 0; !stop; ++uc) {
            const int ub = uc & 1;
            if (!warp_wait(&u_full[ub], (unsigned)(uc >> 1) & 1u, p.wait_ns)) { stop = true; break; }
            const int* m = info + ub * 8;
            const int s = m[0], len = m[1], g = m[3], pre = m[4], n0 = m[5], n1 = m[6];
            const int first = m[2] + (t << (sh - 1));
            __syncwarp();
            if (lane == 0) mbar_arrive(&u_empty[ub]);
            if (s < 0) break;
            const int n = max(n0, n1), nt = t ? n1 : n0;
            const int i = first + (r >> lg);
            const int lim = min(max(i + 1, pre), len);
            const size_t row = (size_t)(s + i) * p.Hq + (g << lg) + (r & (p.G - 1));
            step += n - nt;
            if (nt == 0) continue;
            // the estimate of delta from the output, and lse in log2 units (a row past the document: P = 0)
            float est = 0.f, dlse = 0.f, lse2 = INFINITY;
            if (i < len) {
                const uint4* a = reinterpret_cast<const uint4*>(p.d_o + row * D);
                const uint4* b = reinterpret_cast<const uint4*>(p.o + row * D);
                float e0 = 0.f, e1 = 0.f;
#pragma unroll 4
                for (int c = 0; c < D / 8; ++c) {
                    float fa[8], fb[8];
                    unpack8(a[c], fa);
                    unpack8(b[c], fb);
#pragma unroll
                    for (int e = 0; e < 8; e += 2) {
                        e0 = fmaf(fa[e], fb[e], e0);
                        e1 = fmaf(fa[e + 1], fb[e + 1], e1);
                    }
                }
                if (p.d_lse != nullptr) dlse = p.d_lse[row];
                est = e0 + e1 - dlse;
                lse2 = p.lse[row] * kLog2e;
            }
            float rsum = 0.f;
            for (int tile = nt - 1; tile >= 0; --tile, ++step, ++sc) {
                if (!warp_wait(&s_full[t], (unsigned)sc & 1u, p.wait_ns)) { stop = true; break; }
                tc_fence_after();
                float x[64], th[CAP ? 64 : 1];
                tmem_ld32(tb + SH::TM_S, x);
                tmem_ld32(tb + SH::TM_S + 32, x + 32);
                tmem_ld_wait();
                const int j0 = tile * KT, st = step % ST;
                if (CAP) {
#pragma unroll
                    for (int c = 0; c < 64; ++c) {
                        th[c] = tanh_exp(x[c] * per_cap);
                        x[c] = cap2 * th[c];
                    }
                }
                if (BETA && (CAP || j0 + KT > first + 1)) {
                    if (!warp_wait(&x_full[st], (unsigned)(step / ST) & 1u, p.wait_ns)) { stop = true; break; }
                    const float4* lb = reinterpret_cast<const float4*>(smem + SH::LB_OFF + st * KT * 4);
                    const float di = (float)(i - j0);
#pragma unroll
                    for (int c = 0; c < 64; c += 4) {
                        const float4 b = lb[c / 4];
                        x[c] = fmaf(fmaxf(di - c, 0.f), b.x, x[c]);
                        x[c + 1] = fmaf(fmaxf(di - (c + 1), 0.f), b.y, x[c + 1]);
                        x[c + 2] = fmaf(fmaxf(di - (c + 2), 0.f), b.z, x[c + 2]);
                        x[c + 3] = fmaf(fmaxf(di - (c + 3), 0.f), b.w, x[c + 3]);
                    }
                }
                if (j0 + KT > max(first + 1, pre)) {
#pragma unroll
                    for (int c = 0; c < 64; ++c) x[c] = c < lim - j0 ? x[c] : -INFINITY;
                }
                const uint64_t c2 = pk2(C, C), n2 = pk2(-lse2, -lse2), e2 = pk2(-est, -est);
#pragma unroll
                for (int c = 0; c < 64; c += 2) {
                    float a, b;
                    upk2(fma2(pk2(x[c], x[c + 1]), c2, n2), a, b);
                    x[c] = ex2_approx(a);
                    x[c + 1] = ex2_approx(b);
                }
                uint64_t sum = 0ull;
#pragma unroll
                for (int c0 = 0; c0 < 64; c0 += 32) {
                    float dp[32];
                    tmem_ld32(tb + SH::TM_DP + c0, dp);
                    tmem_ld_wait();
                    uint64_t ds[16];
#pragma unroll
                    for (int e = 0; e < 32; e += 2)
                        ds[e / 2] = mul2(pk2(x[c0 + e], x[c0 + e + 1]), add2(pk2(dp[e], dp[e + 1]), e2));
                    uint32_t w[16];
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        sum = add2(sum, ds[e / 2]);
                        float a, b;
                        upk2(ds[e / 2], a, b);
                        if (CAP) {
                            a *= 1.f - th[c0 + e] * th[c0 + e];
                            b *= 1.f - th[c0 + e + 1] * th[c0 + e + 1];
                        }
                        w[e / 2] = pack_bf16(a, b);   // dS enters dS K as bf16: 2^-9 each, as dq's own rounding
                    }
                    tmem_st16(tb + SH::TM_S + c0 / 2, w);
                }
                float s0, s1;
                upk2(sum, s0, s1);
                rsum += s0 + s1;
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ds_full[t]);
            }
            if (stop) break;
            if (i < len) p.delta[row] = est + (rsum - dlse);
            if (!warp_wait(&o_full[t], (unsigned)oc & 1u, p.wait_ns)) { stop = true; break; }
            ++oc;
            tc_fence_after();
            uint4* dst = reinterpret_cast<uint4*>(p.dq + row * D);
#pragma unroll 1
            for (int c0 = 0; c0 < D; c0 += 32) {
                float o[32];
                tmem_ld32(tb + SH::TM_DQ + c0, o);
                tmem_ld_wait();
                if (i < len) store_bf16x32(dst + c0 / 8, o, p.scale);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&o_empty[t]);   // the next unit's product may overwrite dQ
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
        mbar_wait(fin, 0u, p.wait_ns);
    }
    if (tid == 0 && *s_abort) {
        for (int k = max(0, s_steps[0] - ST); k < s_steps[0]; ++k)
            mbar_wait(&kv_full[k % ST], (unsigned)(k / ST) & 1u, 100000000ull);
        if (s_steps[1] > 0) mbar_wait(q_full, (unsigned)(s_steps[1] - 1) & 1u, 100000000ull);
    }
    __syncthreads();
    if (warp == 8) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(SH::TM_COLS) : "memory");
    }
}

template <int D>
struct DkvShape {
    static constexpr int KT = 128, QT = 64;              // keys of a unit; query rows of a step (QT / G tokens)
    static constexpr int ST = 4;
    static constexpr int NT = 12 * 32;
    static constexpr int REG_SOFT = 208, REG_REST = 88;
    static constexpr int KHALF = KT * 128, KTILE = KHALF * (D / 64);
    static constexpr int QHALF = QT * 128, QTILE = QHALF * (D / 64);
    static constexpr int K_OFF = 0;                      // K, V
    static constexpr int QO_OFF = K_OFF + 2 * KTILE;     // [ST] Q, dO
    static constexpr int KX_OFF = QO_OFF + ST * 2 * QTILE;
    static constexpr int ONE_OFF = KX_OFF + KT * 32;     // key columns without a bias
    static constexpr int QX_OFF = ONE_OFF + KT * 32;     // [ST] extra columns of Q, of dO
    static constexpr int ROW_OFF = QX_OFF + ST * 2 * QT * 32;   // [ST][64] lse in log2 units
    static constexpr int TOK_OFF = ROW_OFF + ST * QT * 4;   // [64] token of a row within the step, as float
    static constexpr int DB_OFF = TOK_OFF + QT * 4;      // [128] d log beta of the second warpgroup's steps
    static constexpr int INFO_OFF = DB_OFF + KT * 4;
    static constexpr int BAR_OFF = INFO_OFF + 2 * 8 * 4;
    static constexpr int NBAR = 2 + 3 * ST + 7 + 4;
    static constexpr int MISC_OFF = BAR_OFF + NBAR * 8;
    static constexpr size_t SMEM = 1024 + MISC_OFF + 32;
    static constexpr int TM_S = 0, TM_DP = 128, TM_DV = 256, TM_DK = 384, TM_COLS = 512;   // S, dP: two of 64
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
    uint64_t* x_full = q_empty + ST;     // bias columns, row values; rows past the document cleared
    uint64_t* s_full = x_full + ST;      // [buffer]
    uint64_t* ds_full = s_full + 2;
    uint64_t* o_full = ds_full + 2;
    uint64_t* o_empty = o_full + 1;
    uint64_t* db_full = o_empty + 1;     // the second warpgroup's part of d log beta
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
        for (int t = 0; t < 2; ++t) {
            mbar_init(&s_full[t], 1);
            mbar_init(&ds_full[t], 4);
            mbar_init(&u_full[t], 1);
            mbar_init(&u_empty[t], 10);
        }
        mbar_init(o_full, 1);
        mbar_init(o_empty, 8);
        mbar_init(db_full, 4);
        mbar_init(fin, 1);
        *s_abort = 0;
        s_steps[0] = s_steps[1] = 0;
        fence_mbar_init();
    }
    if (tid < QT) reinterpret_cast<float*>(smem + SH::TOK_OFF)[tid] = (float)(tid >> lg);
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
            const bool ok = prefill_docs_ok(p.cu, p.N, p.T);
            const PrefillWalk walk(p, 7);
            const long long units = ok ? walk.units : 0;
            int step = 0, uc = 0;
            bool stop = false;
            for (long long r = 0; !stop; ++r, ++uc) {
                const long long u = PrefillWalk::nth(r, blockIdx.x, gridDim.x);
                const bool end = r * gridDim.x >= units;
                if (!end && u >= units) { --uc; continue; }
                PrefillUnit x{};
                int j0 = 0, b0 = 0, b1 = 0;
                if (!end) {
                    x = walk.unit(u);
                    // the first keys meet the most queries: the heaviest level is block 0
                    j0 = ((x.len + KT - 1) / KT - 1 - x.blk) * KT;
                    b0 = j0 < x.pre ? 0 : j0 / bt;
                    b1 = (x.len + bt - 1) / bt;
                }
                const int ub = uc & 1;
                if (uc >= 2 && !warp_wait(&u_empty[ub], (unsigned)((uc >> 1) - 1) & 1u, p.wait_ns)) { stop = true; break; }
                if (__any_sync(kFull, *s_abort != 0)) break;
                if (lane == 0) {
                    int* m = info + ub * 8;
                    m[0] = end ? -1 : x.s;
                    m[1] = x.len;
                    m[2] = j0;
                    m[3] = x.g;
                    m[4] = x.pre;
                    m[5] = b0;
                    m[6] = b1;
                    mbar_arrive(&u_full[ub]);
                }
                __syncwarp();
                if (end) break;
                if (uc >= 1 && !warp_wait(k_empty, (unsigned)(uc - 1) & 1u, p.wait_ns)) { stop = true; break; }
                if (lane == 0) {
                    mbar_arrive_expect_tx(k_full, (unsigned)(2 * SH::KTILE));
                    for (int h = 0; h < D / 64; ++h) {
                        unsigned char* at = smem + SH::K_OFF + h * SH::KHALF;
                        tma_load_3d(at, &tmK, 64 * h, x.g, x.s + j0, k_full);
                        tma_load_3d(at + SH::KTILE, &tmV, 64 * h, x.g, x.s + j0, k_full);
                    }
                    s_steps[1] = uc + 1;
                }
                for (int b = b0; b < b1; ++b, ++step) {
                    const int st = step % ST;
                    if (step >= ST && !warp_wait(&q_empty[st], (unsigned)((step / ST) - 1) & 1u, p.wait_ns)) { stop = true; break; }
                    if (lane == 0) {
                        mbar_arrive_expect_tx(&q_full[st], (unsigned)(2 * SH::QTILE));
                        for (int h = 0; h < D / 64; ++h) {
                            unsigned char* at = smem + SH::QO_OFF + st * 2 * SH::QTILE + h * SH::QHALF;
                            tma_load_3d(at, &tmQ, 64 * h, x.g << lg, x.s + b * bt, &q_full[st]);
                            tma_load_3d(at + SH::QTILE, &tmO, 64 * h, x.g << lg, x.s + b * bt, &q_full[st]);
                        }
                        s_steps[0] = step + 1;
                    }
                    if (__any_sync(kFull, *s_abort != 0)) { stop = true; break; }
                }
            }
            if (stop && lane == 0) fail();
        } else if (warp == 10) {
            // ======================= bias columns, row values, rows past a document's end =======================
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
                const int last = j0 + KT - 1;
                if (BETA && !CAP) {
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
                for (int blk = b0; blk < b1; ++blk, ++step) {
                    const int st = step % ST;
                    const unsigned ph = (unsigned)(step / ST) & 1u;
                    float lse[2], delta[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int c = lane + 32 * e, i = blk * bt + (c >> lg);
                        lse[e] = 1.2676506e30f;   // no such row (2^100): P = 0
                        delta[e] = 0.f;
                        if (i < len) {
                            const size_t row = (size_t)(s + i) * p.Hq + (g << lg) + (c & (p.G - 1));
                            lse[e] = p.lse[row];
                            delta[e] = p.delta[row];
                        }
                    }
                    if (step >= ST && !warp_wait(&q_empty[st], ph ^ 1u, p.wait_ns)) { stop = true; break; }
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int c = lane + 32 * e;
                        uint4 c0, c1;
                        unsigned char* at = smem + SH::QX_OFF + st * 2 * QT * 32;
                        if (CAP) {
                            reinterpret_cast<float*>(smem + SH::ROW_OFF)[st * QT + c] = lse[e] * kLog2e;
                        } else {
                            far_query(BETA ? max(blk * bt + (c >> lg) - last, 0) : 0, lse[e] * (-1.f / p.scale), c0, c1);
                            *reinterpret_cast<uint4*>(at + plain16_off(c, 0)) = c0;
                            *reinterpret_cast<uint4*>(at + plain16_off(c, 1)) = c1;
                        }
                        far_query(0, -delta[e], c0, c1);
                        *reinterpret_cast<uint4*>(at + QT * 32 + plain16_off(c, 0)) = c0;
                        *reinterpret_cast<uint4*>(at + QT * 32 + plain16_off(c, 1)) = c1;
                    }
                    if ((blk + 1) * bt > len) {
                        if (!warp_wait(&q_full[st], ph, p.wait_ns)) { stop = true; break; }
                        const int rows = (len - blk * bt) << lg;
                        unsigned char* qt = smem + SH::QO_OFF + st * 2 * SH::QTILE;
                        for (int x = lane; x < (QT - rows) * 16 * (D / 64); x += 32) {
                            const int row = rows + x / (16 * (D / 64)), c = x % (16 * (D / 64));   // chunks of Q, then of dO
                            *reinterpret_cast<uint4*>(qt + (c >> 3) * SH::QHALF + row * 128 + ((c & 7) << 4)) =
                                make_uint4(0u, 0u, 0u, 0u);
                        }
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&x_full[st]);
                    if (__any_sync(kFull, *s_abort != 0)) { stop = true; break; }
                }
            }
            if (stop && lane == 0) fail();
        } else if (warp == 8) {
            // ======================= products =======================
            // the warp stays together (its values are uniform); one lane issues
            constexpr uint32_t idesc_s = umma_idesc_bf16(KT, QT), idesc_o = umma_idesc_bf16_bmn(KT, D);
            int step = 0;
            unsigned dc = 0;   // bit t: parity of buffer t's next dS
            bool stop = false;
            const uint32_t k_lo = desc_sw128_lo(sbase + SH::K_OFF), q_lo = desc_sw128_lo(sbase + SH::QO_OFF);
            const uint32_t qr_lo = desc_mn_lo(sbase + SH::QO_OFF, SH::QHALF);
            const uint32_t kx_lo = desc_plain_lo(sbase + SH::KX_OFF), qx_lo = desc_plain_lo(sbase + SH::QX_OFF);
            const uint32_t one_lo = desc_plain_lo(sbase + SH::ONE_OFF);
            auto scores = [&](int t, int st, bool past) {
                const uint32_t ts = tmem + SH::TM_S + t * 64, q = q_lo + st * (2 * SH::QTILE >> 4);
                const uint32_t qx = qx_lo + st * (2 * QT * 32 >> 4);
                umma_kmajor<D / 16>(ts, k_lo, SH::KHALF, q, SH::QHALF, idesc_s);
                if (!CAP)   // - lse, and the bias where every query is past every key
                    umma_bf16(ts, desc(BETA && past ? kx_lo : one_lo, kDescPlainHi), desc(qx, kDescPlainHi), idesc_s, 1u);
                umma_kmajor<D / 16>(tmem + SH::TM_DP + t * 64, k_lo + (SH::KTILE >> 4), SH::KHALF, q + (SH::QTILE >> 4),
                                    SH::QHALF, idesc_s);
                umma_bf16(tmem + SH::TM_DP + t * 64, desc(one_lo, kDescPlainHi), desc(qx + (QT * 32 >> 4), kDescPlainHi),
                          idesc_s, 1u);   // - delta
                umma_commit(&s_full[t]);
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
                if (!warp_wait(k_full, (unsigned)uc & 1u, p.wait_ns)) { stop = true; break; }
                for (int q = 0; q < n + 2; ++q) {
                    // step q - 2's gradients free buffer q % 2 for step q's scores
                    const int k = step + q - 2, t = q & 1, st = (k + ST) % ST;
                    if (q >= 2) {
                        if (!warp_wait(&ds_full[t], (dc >> t) & 1u, p.wait_ns)) { stop = true; break; }
                        dc ^= 1u << t;
                        if (q == 2 && uc >= 1 && !warp_wait(o_empty, (unsigned)(uc - 1) & 1u, p.wait_ns)) { stop = true; break; }
                    }
                    if (q < n && !loaded(step + q)) { stop = true; break; }
                    tc_fence_after();
                    if (elect_one()) {
                        if (q >= 2) {
                            const uint32_t q_rows = qr_lo + st * (2 * SH::QTILE >> 4);
                            umma_rows<QT / 16>(tmem + SH::TM_DV, tmem + SH::TM_S + t * 64, q_rows + (SH::QTILE >> 4), idesc_o, q == 2);
                            umma_rows<QT / 16>(tmem + SH::TM_DK, tmem + SH::TM_DP + t * 64, q_rows, idesc_o, q == 2);
                            umma_commit(&q_empty[st]);
                        }
                        if (q < n) scores(t, (step + q) % ST, (b0 + q) * bt >= last);
                        if (q == n - 1) umma_commit(k_empty);
                        if (q == n + 1) umma_commit(o_full);
                    }
                    __syncwarp();
                }
                if (stop) break;
                step += n;
            }
            if (stop && lane == 0) fail();
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(SH::REG_SOFT));
        // ======================= P^T and dS^T of a key row; dV, dK, d log beta =======================
        const int t = warp >> 2, quarter = warp & 3;
        const int r = 32 * quarter + lane;
        const uint32_t tl = tmem + ((uint32_t)(32 * quarter) << 16);
        const float C = CAP ? 1.f : p.scale * kLog2e;
        const float cap2 = CAP ? p.softcap * kLog2e : 0.f, per_cap = CAP ? p.scale / p.softcap : 0.f;
        const float4* tok4 = reinterpret_cast<const float4*>(smem + SH::TOK_OFF);
        float* s_db = reinterpret_cast<float*>(smem + SH::DB_OFF);
        int sc = 0, step = 0;
        bool stop = false;
        for (int uc = 0; !stop; ++uc) {
            const int ub = uc & 1;
            if (!warp_wait(&u_full[ub], (unsigned)(uc >> 1) & 1u, p.wait_ns)) { stop = true; break; }
            const int* m = info + ub * 8;
            const int s = m[0], len = m[1], j0 = m[2], g = m[3], pre = m[4], b0 = m[5], b1 = m[6];
            __syncwarp();
            if (lane == 0) mbar_arrive(&u_empty[ub]);
            if (s < 0) break;
            const int n = b1 - b0, last = j0 + KT - 1;
            const int j = j0 + r;
            const float slope_b = (BETA && j < len) ? clamp_log_beta(p.lb[(long long)(s + j) * p.lb_st + g * p.lb_sh]) *
                                                          (CAP ? kLog2e : 1.f / p.scale)
                                                    : 0.f;
            float db = 0.f;
            for (int q = t; q < n; q += 2, ++sc) {
                const int k = step + q, st = k % ST, tb = (b0 + q) * bt;   // the step's first token
                if (!warp_wait(&s_full[t], (unsigned)sc & 1u, p.wait_ns)) { stop = true; break; }
                if (!warp_wait(&x_full[st], (unsigned)(k / ST) & 1u, p.wait_ns)) { stop = true; break; }
                tc_fence_after();
                float x[64], th[CAP ? 64 : 1];
                tmem_ld32(tl + SH::TM_S + t * 64, x);
                tmem_ld32(tl + SH::TM_S + t * 64 + 32, x + 32);
                tmem_ld_wait();
                const bool past = tb >= last;
                const float di = (float)(tb - j);
                if (CAP) {
                    const float4* l4 = reinterpret_cast<const float4*>(smem + SH::ROW_OFF + st * QT * 4);
#pragma unroll
                    for (int c = 0; c < 64; c += 4) {
                        const float4 l = l4[c / 4];
                        const float ls[4] = {l.x, l.y, l.z, l.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            th[c + e] = tanh_exp(x[c + e] * per_cap);
                            x[c + e] = fmaf(cap2, th[c + e], -ls[e]);
                        }
                    }
                }
                if (BETA && (CAP || !past)) {
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
                    const int from = j < pre ? 0 : min(max(j - tb, 0) << lg, QT);   // the first row that sees key j
#pragma unroll
                    for (int c = 0; c < 64; ++c) x[c] = c >= from ? x[c] : -INFINITY;
                }
                const uint64_t c2 = pk2(C, C);
                // d log beta: where all is past, sum dS (di + tok(c)) with tok(c) = c >> lg, from the eight
                // sums over c = e mod 8 and from sum (c / 8) dS; else the distances one by one
                uint64_t by8[4] = {0ull, 0ull, 0ull, 0ull}, up = 0ull;
#pragma unroll
                for (int c0 = 0; c0 < 64; c0 += 32) {
                    float dp[32];
                    tmem_ld32(tl + SH::TM_DP + t * 64 + c0, dp);
                    uint32_t w[16];
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        float a, b;
                        upk2(mul2(pk2(x[c0 + e], x[c0 + e + 1]), c2), a, b);
                        x[c0 + e] = ex2_approx(a);
                        x[c0 + e + 1] = ex2_approx(b);
                        w[e / 2] = pack_bf16(x[c0 + e], x[c0 + e + 1]);
                    }
                    tmem_st16(tl + SH::TM_S + t * 64 + c0 / 2, w);
                    tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        const uint64_t ds = mul2(pk2(x[c0 + e], x[c0 + e + 1]), pk2(dp[e], dp[e + 1]));
                        if (BETA) {
                            if (past) {
                                by8[(e / 2) & 3] = add2(by8[(e / 2) & 3], ds);
                                up = fma2(ds, pk2((float)((c0 + e) / 8), (float)((c0 + e) / 8)), up);
                            } else {
                                const float2 k2 = reinterpret_cast<const float2*>(tok4)[(c0 + e) / 2];
                                up = fma2(ds, pk2(fmaxf(di + k2.x, 0.f), fmaxf(di + k2.y, 0.f)), up);
                            }
                        }
                        float a, b;
                        upk2(ds, a, b);
                        if (CAP) {
                            a *= 1.f - th[c0 + e] * th[c0 + e];
                            b *= 1.f - th[c0 + e + 1] * th[c0 + e + 1];
                        }
                        w[e / 2] = pack_bf16(a, b);
                    }
                    tmem_st16(tl + SH::TM_DP + t * 64 + c0 / 2, w);
                }
                if (BETA) {
                    float u0, u1;
                    upk2(up, u0, u1);
                    if (past) {
                        float part = (u0 + u1) * (float)(8 >> lg), all = 0.f;
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
                        db += u0 + u1;
                    }
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ds_full[t]);
            }
            if (stop) break;
            step += n;
            if (!warp_wait(o_full, (unsigned)uc & 1u, p.wait_ns)) { stop = true; break; }
            tc_fence_after();
            uint4* dst = reinterpret_cast<uint4*>((t ? p.dk : p.dv) + ((size_t)(s + j) * p.Hkv + g) * D);
#pragma unroll 1
            for (int c0 = 0; c0 < D; c0 += 32) {
                float o[32];
                tmem_ld32(tl + (t ? SH::TM_DK : SH::TM_DV) + c0, o);
                tmem_ld_wait();
                if (j < len) store_bf16x32(dst + c0 / 8, o, t ? p.scale : 1.f);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(o_empty);
            if (BETA) {
                // the next unit's part is posted only after this warpgroup's steps of that unit
                if (t == 1) {
                    s_db[r] = db;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(db_full);
                } else {
                    if (!warp_wait(db_full, (unsigned)uc & 1u, p.wait_ns)) { stop = true; break; }
                    if (j < len) p.dlb[(size_t)(s + j) * p.Hkv + g] = db + s_db[r];
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
        mbar_wait(fin, 0u, p.wait_ns);
    }
    if (tid == 0 && *s_abort) {
        for (int k = max(0, s_steps[0] - ST); k < s_steps[0]; ++k)
            mbar_wait(&q_full[k % ST], (unsigned)(k / ST) & 1u, 100000000ull);
        if (s_steps[1] > 0) mbar_wait(k_full, (unsigned)(s_steps[1] - 1) & 1u, 100000000ull);
    }
    __syncthreads();
    if (warp == 8) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(SH::TM_COLS) : "memory");
    }
}

}  // namespace kvb
