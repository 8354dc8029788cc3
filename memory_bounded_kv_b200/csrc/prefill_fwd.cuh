// Retention-gated attention over packed prompts on the 5th-generation tensor cores
// (kvb_prefill_attn; "Cache What Lasts" section 2.1: the weight of key j for query i is proportional
// to exp(q_i . k_j + (i - j) log beta_j)).
//
// A unit is 256 / G tokens of a document and a kv head, as two tiles of 128 query rows (row r of a
// tile: token r / G, query head r % G of the group), so that a K/V tile read once serves every head
// that shares it. One pass over the visible key tiles (128 keys), from the nearest to the farthest:
// the decay makes near keys large, so the running maximum seldom moves. Per tile
//   S = Q K^T (tcgen05.mma into tensor memory), P = exp2(C S - m) in bf16 over S's columns,
//   O += P V (P from tensor memory, V from shared memory).
// The two tiles alternate: one's softmax runs while the other's products do.
//
// The bias (i - j) log beta_j costs the softmax nothing: it is a product itself. Queries get the
// columns (i', i', i', 1, 1, 1), i' = i - (first token of the unit) <= 255 (exact in bf16), keys the
// three bf16 parts of b_j = log beta_j / scale and of (base - j) b_j, so one more K = 16 step of the
// S product adds (i - j) b_j to fp32 accuracy. That holds where every key lies in every query's
// past; on the tiles of the diagonal and of a prefix the softmax adds max(i - j, 0) b_j itself, and
// the step is left out. With a tanh cap the bias follows the cap, so the softmax always adds it.
//
// Roles (384 threads, one CTA per SM, persistent): warps 0-3 and 4-7 softmax and output of tiles 0
// and 1 (a thread per row), warp 8 issues the products, warp 9 finds the units and issues the TMA
// loads, warps 10 and 11 write the bias columns and clear V's rows past a document's end (their P is 0,
// but 0 times a neighbour's NaN is not).
// Every wait is bounded (wait_ns); a CTA that gives up records KVB_DERR_TIMEOUT and lets its copies
// and products finish (bounded); the rows that it had not written keep what they held.
//
// What bounds it: a K/V step of the pair is 2174 clocks of products (see prefill_bwd.cuh for their rates)
// and takes some 3400, the rest being the hand-over between products and softmax: a tile's next S waits
// for its P V, because two S and two O fill the tensor memory. One document of 8192 tokens, 32/8 heads,
// d 128: 435 us (1.26 PFLOP/s) in short bursts, 501 us at the power cap; d 64 368 us (exponentials); with
// scores capped at 50 765 us. Short documents pay a near tile and 2.5k clocks of output a unit: 6151 tokens in
// 24 documents 59 us. One issuing warp, not one per tile: with two, both tiles' products interleave and
// both finish late (475 -> 537 us). Pairs always: a tile alone takes 0.83 of a pair's step, so units of
// one tile lose even where the longest pair holds up the rest (4000 tokens in 5 documents, 16/2 heads, d 64,
// with a cap: 52.6 -> 69.5 us).
#pragma once

#include "prefill_units.cuh"

namespace kvb {

template <int D>
struct FwdShape {
    static constexpr int R = 128, KT = 128;              // rows of a query tile, keys of a key tile
    static constexpr int ST = D == 128 ? 2 : 4;          // K and V ring stages
    static constexpr int NT = 12 * 32;
    static constexpr int REG_SOFT = 208, REG_REST = 88;  // 2 x 208 + 88 = 3 x 168, the launch's registers
    static constexpr int HALF = 128 * 128;               // 128 rows x 64 dims of bf16
    static constexpr int TILE = HALF * (D / 64);
    static constexpr int XCOL = 128 * 32;                // bias columns of 128 rows
    static constexpr int Q_OFF = 0;
    static constexpr int K_OFF = Q_OFF + 2 * TILE;
    static constexpr int V_OFF = K_OFF + ST * TILE;
    static constexpr int QX_OFF = V_OFF + ST * TILE;
    static constexpr int KX_OFF = QX_OFF + 2 * XCOL;
    static constexpr int LB_OFF = KX_OFF + ST * XCOL;    // [ST][128] f32: the bias slope of each key
    static constexpr int INFO_OFF = LB_OFF + ST * KT * 4;   // [2][8] unit records
    static constexpr int BAR_OFF = INFO_OFF + 2 * 8 * 4;
    static constexpr int NBAR = 2 + 6 * ST + 10 + 4;
    static constexpr int MISC_OFF = BAR_OFF + NBAR * 8;
    static constexpr size_t SMEM = 1024 + MISC_OFF + 32;
    static constexpr int TM_S = 0, TM_O = 256, TM_COLS = 512;
    static_assert(SMEM <= 227 * 1024, "shared memory");
};

template <int D, bool BETA, bool CAP>
__global__ void __launch_bounds__(FwdShape<D>::NT, 1)
    prefill_fwd_kernel(const __grid_constant__ PrefillParams p, const __grid_constant__ CUtensorMap tmQ,
                       const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV) {
    using SH = FwdShape<D>;
    constexpr int ST = SH::ST, R = SH::R, KT = SH::KT;
    extern __shared__ unsigned char smem_dyn[];
    unsigned char* smem = reinterpret_cast<unsigned char*>(
        (reinterpret_cast<uintptr_t>(smem_dyn) + 1023) & ~static_cast<uintptr_t>(1023));
    const uint32_t sbase = smem_u32(smem);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + SH::BAR_OFF);
    uint64_t* q_full = bars;
    uint64_t* q_empty = bars + 1;
    uint64_t* k_full = bars + 2;
    uint64_t* k_empty = k_full + ST;
    uint64_t* v_full = k_empty + ST;
    uint64_t* v_empty = v_full + ST;
    uint64_t* v_fix = v_empty + ST;     // the tile's rows past the document are cleared
    uint64_t* lb_full = v_fix + ST;
    uint64_t* s_full = lb_full + ST;    // [tile]
    uint64_t* p_half = s_full + 2;      // the weights of a tile's first 64 keys, all of them
    uint64_t* p_full = p_half + 2;
    uint64_t* o_full = p_full + 2;
    uint64_t* o_empty = o_full + 2;
    uint64_t* u_full = o_empty + 2;     // [2] unit records
    uint64_t* u_empty = u_full + 2;
    int* info = reinterpret_cast<int*>(smem + SH::INFO_OFF);
    uint32_t* tslot = reinterpret_cast<uint32_t*>(smem + SH::MISC_OFF);
    volatile int* s_abort = reinterpret_cast<int*>(smem + SH::MISC_OFF) + 1;
    int* s_steps = reinterpret_cast<int*>(smem + SH::MISC_OFF) + 2;   // K/V tiles and query blocks loaded
    uint64_t* fin = reinterpret_cast<uint64_t*>(smem + SH::MISC_OFF + 16);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int lg = 31 - __clz(p.G), sh = 8 - lg;       // 2^sh tokens per unit, 2^(sh - 1) per tile
    if (tid == 0) {
        mbar_init(q_full, 1);
        mbar_init(q_empty, 1);
        for (int s = 0; s < ST; ++s) {
            mbar_init(&k_full[s], BETA && !CAP ? 2 : 1);   // the copy, the bias columns
            mbar_init(&k_empty[s], 1);
            mbar_init(&v_full[s], 1);
            mbar_init(&v_empty[s], 1);
            mbar_init(&v_fix[s], 1);
            mbar_init(&lb_full[s], 1);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(&s_full[t], 1);
            mbar_init(&p_half[t], 4);
            mbar_init(&p_full[t], 4);
            mbar_init(&o_full[t], 1);
            mbar_init(&o_empty[t], 4);
            mbar_init(&u_full[t], 1);
            mbar_init(&u_empty[t], 11);   // products, 2 bias warps, 8 softmax warps
        }
        mbar_init(fin, 1);
        *s_abort = 0;
        s_steps[0] = s_steps[1] = 0;
        fence_mbar_init();
    }
    if (warp == 9 && lane == 0) {
        prefetch_tensormap(&tmQ);
        prefetch_tensormap(&tmK);
        prefetch_tensormap(&tmV);
    }
    if (BETA && !CAP) {
        // the queries' bias columns are the same for every unit; the keys' second chunk is 0
        for (int x = tid; x < 2 * R; x += SH::NT) {
            unsigned char* at = smem + SH::QX_OFF + (x >> 7) * SH::XCOL;
            *reinterpret_cast<uint4*>(at + plain16_off(x & 127, 0)) = bias_query(x >> lg);
            *reinterpret_cast<uint4*>(at + plain16_off(x & 127, 1)) = make_uint4(0u, 0u, 0u, 0u);
        }
        for (int x = tid; x < ST * KT; x += SH::NT)
            *reinterpret_cast<uint4*>(smem + SH::KX_OFF + (x >> 7) * SH::XCOL + plain16_off(x & 127, 1)) =
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

    // a row of 128 scores and its packed weights want more than the launch's 168 registers a thread
    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(SH::REG_REST));
        if (warp == 9) {
            // ======================= units and loads =======================
            const PrefillWalk walk(p, sh);
            const long long units = walk.units;
            int step = 0, uc = 0;
            bool stop = false;
            for (long long r = 0; !stop; ++r, ++uc) {
                // rounds of the units: one past the last ends (an odd round may hold this CTA's unit or not)
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
                if (uc >= 2 && !warp_wait(&u_empty[ub], (unsigned)((uc >> 1) - 1) & 1u, p.wait_ns)) {
                    if (lane == 0) fail();
                    break;
                }
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
                if (uc >= 1 && !warp_wait(q_empty, (unsigned)(uc - 1) & 1u, p.wait_ns)) {
                    if (lane == 0) fail();
                    break;
                }
                const int n = max(n0, n1);
                const int loads = p.withhold == blockIdx.x + 1 ? min(n, max(1 - step, 0)) : n;   // test hook: one tile in all
                if (lane == 0) {
                    const int tiles = n1 > 0 ? 2 : 1;
                    mbar_arrive_expect_tx(q_full, (unsigned)(tiles * SH::TILE));
                    for (int t = 0; t < tiles; ++t)
                        for (int h = 0; h < D / 64; ++h)
                            tma_load_3d(smem + SH::Q_OFF + t * SH::TILE + h * SH::HALF, &tmQ, 64 * h, x.g << lg,
                                        x.s + (x.blk << sh) + (t << (sh - 1)), q_full);
                    s_steps[1] = uc + 1;
                }
                for (int tile = n - 1; tile >= n - loads; --tile, ++step) {
                    const int st = step % ST;
                    const unsigned ph = (unsigned)((step / ST) - 1) & 1u;
                    if (step >= ST && !warp_wait(&k_empty[st], ph, p.wait_ns)) { stop = true; break; }
                    if (lane == 0) {
                        mbar_arrive_expect_tx(&k_full[st], (unsigned)SH::TILE);
                        for (int h = 0; h < D / 64; ++h)
                            tma_load_3d(smem + SH::K_OFF + st * SH::TILE + h * SH::HALF, &tmK, 64 * h, x.g, x.s + tile * KT, &k_full[st]);
                        s_steps[0] = step + 1;
                    }
                    if (step >= ST && !warp_wait(&v_empty[st], ph, p.wait_ns)) { stop = true; break; }
                    if (lane == 0) {
                        mbar_arrive_expect_tx(&v_full[st], (unsigned)SH::TILE);
                        for (int h = 0; h < D / 64; ++h)
                            tma_load_3d(smem + SH::V_OFF + st * SH::TILE + h * SH::HALF, &tmV, 64 * h, x.g, x.s + tile * KT, &v_full[st]);
                    }
                    if (__any_sync(kFull, *s_abort != 0)) { stop = true; break; }
                }
                if (stop && lane == 0) fail();
                if (loads < n) break;
            }
        } else if (warp >= 10) {
            // ======================= bias columns, V past a document's end =======================
            // two warps, a step each in turn; the log betas of a warp's next step load while it writes this one's
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
                float nb[4] = {0.f, 0.f, 0.f, 0.f};
                auto load = [&](int tile) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int j = tile * KT + lane + 32 * e;
                        nb[e] = tile >= 0 && j < len ? p.lb[(long long)(s + j) * p.lb_st + g * p.lb_sh] : 0.f;
                    }
                };
                const int q0 = (step + warp) & 1;   // this warp's first step of the unit
                if (BETA) load(n - 1 - q0);
                for (int q = q0; q < n; q += 2) {
                    const int tile = n - 1 - q, k = step + q, st = k % ST;
                    const unsigned ph = (unsigned)(k / ST) & 1u;
                    const bool tail = (tile + 1) * KT > len;   // a document's last tile: the unit's first step
                    float b[4];
                    if (BETA) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) b[e] = clamp_log_beta(nb[e]) * unit_b;
                        load(tile - 2);
                    }
                    // The V stage is free: the slopes of step k - ST were read before the P V product that freed it,
                    // and its V had landed. (Without that v_full could be a phase behind, and the wait on it below
                    // would pass at once. No barrier can be ahead: the step's products wait for its slopes or for its
                    // clearing, and steps with neither do not wait here.)
                    if ((BETA || tail) && k >= ST && !warp_wait(&v_empty[st], ph ^ 1u, p.wait_ns)) { stop = true; break; }
                    if (BETA) {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            reinterpret_cast<float*>(smem + SH::LB_OFF)[st * KT + lane + 32 * e] = b[e];
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&lb_full[st]);
                        if (!CAP) {
                            if (k >= ST && !warp_wait(&k_empty[st], ph ^ 1u, p.wait_ns)) { stop = true; break; }
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const int c = lane + 32 * e;
                                *reinterpret_cast<uint4*>(smem + SH::KX_OFF + st * SH::XCOL + plain16_off(c, 0)) =
                                    bias_columns(b[e], i0 - tile * KT - c);
                            }
                            fence_proxy_async_smem();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(&k_full[st]);
                        }
                    }
                    if (tail) {
                        if (!warp_wait(&v_full[st], ph, p.wait_ns)) { stop = true; break; }
                        const int rows = len - tile * KT;
                        unsigned char* vt = smem + SH::V_OFF + st * SH::TILE;
                        for (int x = lane; x < (KT - rows) * 8 * (D / 64); x += 32) {
                            const int row = rows + x / (8 * (D / 64)), c = x % (8 * (D / 64));
                            *reinterpret_cast<uint4*>(vt + (c >> 3) * SH::HALF + row * 128 + ((c & 7) << 4)) =
                                make_uint4(0u, 0u, 0u, 0u);
                        }
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&v_fix[st]);
                    }
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
            unsigned fixes = 0;           // bit st: parity of the next clearing of stage st
            unsigned pc = 0;              // bit t: parity of tile t's next P
            int oc0 = 0, oc1 = 0;
            bool stop = false;
            const uint32_t q_lo = desc_sw128_lo(sbase + SH::Q_OFF), k_lo = desc_sw128_lo(sbase + SH::K_OFF);
            const uint32_t v_lo = desc_mn_lo(sbase + SH::V_OFF, SH::HALF);
            const uint32_t qx_lo = desc_plain_lo(sbase + SH::QX_OFF), kx_lo = desc_plain_lo(sbase + SH::KX_OFF);
            auto scores = [&](int t, int st, bool past) {
                const uint32_t ts = tmem + SH::TM_S + t * 128;
                umma_kmajor<D / 16>(ts, q_lo + t * (SH::TILE >> 4), SH::HALF, k_lo + st * (SH::TILE >> 4), SH::HALF, idesc_s);
                if (BETA && !CAP && past)
                    umma_bf16(ts, desc(qx_lo + t * (SH::XCOL >> 4), kDescPlainHi), desc(kx_lo + st * (SH::XCOL >> 4), kDescPlainHi),
                              idesc_s, 1u);
                umma_commit(&s_full[t]);
            };
            for (int uc = 0; !stop; ++uc) {
                const int ub = uc & 1;
                if (!warp_wait(&u_full[ub], (unsigned)(uc >> 1) & 1u, p.wait_ns)) { stop = true; break; }
                const int* m = info + ub * 8;
                const int s = __shfl_sync(kFull, m[0], 0), len = __shfl_sync(kFull, m[1], 0), i0 = __shfl_sync(kFull, m[2], 0);
                const int n0 = __shfl_sync(kFull, m[5], 0), n1 = __shfl_sync(kFull, m[6], 0);
                if (lane == 0) mbar_arrive(&u_empty[ub]);
                if (s < 0) break;
                const int n = max(n0, n1), i1 = i0 + (1 << (sh - 1));
                if (!warp_wait(q_full, (unsigned)uc & 1u, p.wait_ns) ||
                    !warp_wait(&k_full[step % ST], (unsigned)(step / ST) & 1u, p.wait_ns)) { stop = true; break; }
                tc_fence_after();
                if (elect_one()) {
                    if (n - 1 < n0) scores(0, step % ST, n * KT <= i0 + 1);
                    if (n - 1 < n1) scores(1, step % ST, n * KT <= i1 + 1);
                    umma_commit(&k_empty[step % ST]);
                    if (n == 1) umma_commit(q_empty);
                }
                __syncwarp();
                for (int tile = n - 1; tile >= 0; --tile, ++step) {
                    const int st = step % ST, nst = (step + 1) % ST;
                    const bool more = tile > 0;
                    if (more && !warp_wait(&k_full[nst], (unsigned)((step + 1) / ST) & 1u, p.wait_ns)) { stop = true; break; }
                    if (!warp_wait(&v_full[st], (unsigned)(step / ST) & 1u, p.wait_ns)) { stop = true; break; }
                    if ((tile + 1) * KT > len) {
                        if (!warp_wait(&v_fix[st], (fixes >> st) & 1u, p.wait_ns)) { stop = true; break; }
                        fixes ^= 1u << st;
                    }
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        const int nt = t ? n1 : n0;
                        const bool have = tile < nt, first = tile == nt - 1;
                        if (have) {
                            if (first) {
                                int& oc = t ? oc1 : oc0;
                                if (oc > 0 && !warp_wait(&o_empty[t], (unsigned)(oc - 1) & 1u, p.wait_ns)) { stop = true; break; }
                                ++oc;
                            }
                            if (!warp_wait(&p_half[t], (pc >> t) & 1u, p.wait_ns)) { stop = true; break; }
                            tc_fence_after();
                            if (elect_one())
                                umma_rows<KT / 32>(tmem + SH::TM_O + t * 128, tmem + SH::TM_S + t * 128,
                                                   v_lo + st * (SH::TILE >> 4), idesc_o, first);
                            __syncwarp();
                            if (!warp_wait(&p_full[t], (pc >> t) & 1u, p.wait_ns)) { stop = true; break; }
                            pc ^= 1u << t;
                        }
                        tc_fence_after();
                        if (elect_one()) {
                            if (have) {
                                umma_rows<KT / 32>(tmem + SH::TM_O + t * 128, tmem + SH::TM_S + t * 128 + 32,
                                                   v_lo + st * (SH::TILE >> 4) + 64 * 128 / 16, idesc_o, false);
                                if (tile == 0) umma_commit(&o_full[t]);
                            }
                            if (t == 1) umma_commit(&v_empty[st]);
                            if (more && tile - 1 < nt) scores(t, nst, tile * KT <= (t ? i1 : i0) + 1);
                            if (t == 1 && more) umma_commit(&k_empty[nst]);
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
        // ======================= softmax and output =======================
        const int t = warp >> 2, quarter = warp & 3;
        const int r = 32 * quarter + lane;
        const uint32_t ts = tmem + ((uint32_t)(32 * quarter) << 16) + SH::TM_S + t * 128;
        const uint32_t to = tmem + ((uint32_t)(32 * quarter) << 16) + SH::TM_O + t * 128;
        const float C = CAP ? 1.f : p.scale * kLog2e;          // S in these units to log2 units
        const float cap2 = CAP ? p.softcap * kLog2e : 0.f, per_cap = CAP ? p.scale / p.softcap : 0.f;
        int sc = 0, step = 0, oc = 0;
        bool stop = false;
        for (int uc = 0; !stop; ++uc) {
            const int ub = uc & 1;
            if (!warp_wait(&u_full[ub], (unsigned)(uc >> 1) & 1u, p.wait_ns)) { stop = true; break; }
            const int* m = info + ub * 8;
            const int s = m[0], len = m[1], g = m[3], pre = m[4], n0 = m[5], n1 = m[6];
            const int first = m[2] + (t << (sh - 1));            // the tile's first token
            __syncwarp();
            if (lane == 0) mbar_arrive(&u_empty[ub]);
            if (s < 0) break;
            const int n = max(n0, n1), nt = t ? n1 : n0;
            const int i = first + (r >> lg);
            const int lim = min(max(i + 1, pre), len);
            const int lo = __shfl_sync(kFull, lim, 0), hi = __shfl_sync(kFull, lim, 31);   // the warp's fewest and most
            step += n - nt;
            if (nt == 0) continue;
            float m_ref = -INFINITY, l_sum = 0.f;
            // 32 scores to their weights (bf16, into tensor memory at dst) and into the sums
            auto weights = [&](float* x, uint64_t c2, uint64_t n2, uint64_t (&sums)[4], uint32_t dst) {
                // in passes, so that independent instructions stand next to each other (d 64: 375 -> 368 us)
                uint32_t w[16];
#pragma unroll
                for (int e = 0; e < 32; e += 2) upk2(fma2(pk2(x[e], x[e + 1]), c2, n2), x[e], x[e + 1]);
#pragma unroll
                for (int e = 0; e < 32; e += 2) {
                    // a quarter of the exponentials on the FMA pipe, where exponentials bound the kernel (d 64: 388 ->
                    // 371 us, with a cap 874 -> 842); at d 128 the products and the power cap hold it and that costs
                    // or changes nothing (454 -> 466 us, with a cap 823 -> 825; 8192 tokens, 32/8 heads)
                    if (D == 64 && e % 8 == 6) {
                        exp2_poly2<4>(x[e], x[e + 1]);
                    } else {
                        x[e] = ex2_approx(x[e]);
                        x[e + 1] = ex2_approx(x[e + 1]);
                    }
                }
#pragma unroll
                for (int e = 0; e < 32; e += 2) {
                    sums[(e / 2) & 3] = add2(sums[(e / 2) & 3], pk2(x[e], x[e + 1]));
                    w[e / 2] = pack_bf16(x[e], x[e + 1]);   // weights enter P V as bf16: 2^-8 each, as the output's own rounding
                }
                tmem_st16(dst, w);
            };
            // the first half's product starts while the second half is computed
            auto half_done = [&] {
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_half[t]);
            };
            auto all_done = [&](const uint64_t (&sums)[4]) {
                float s0, s1;
                upk2(add2(add2(sums[0], sums[1]), add2(sums[2], sums[3])), s0, s1);
                l_sum += s0 + s1;
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[t]);
            };
            for (int tile = nt - 1; tile >= 0; --tile, ++step, ++sc) {
                if (!warp_wait(&s_full[t], (unsigned)sc & 1u, p.wait_ns)) { stop = true; break; }
                tc_fence_after();
                const int j0 = tile * KT, st = step % ST;
                const bool biased = BETA && (CAP || j0 + KT > first + 1), masked = j0 + KT > max(first + 1, pre);
                if (CAP && !masked && tile < nt - 1) {
                    // No score passes the uncapped one's size or the cap, and no bias of a log beta <= 0 raises it: where
                    // that bound stays within 2^16 of the reference, the reference stays, and the tile needs one pass
                    // and no write of the capped scores (8192 tokens, cap 50, d 128: 811 -> 759 us)
                    bool low = true;                             // (not where a log beta is NaN)
                    const float* lbf = reinterpret_cast<const float*>(smem + SH::LB_OFF) + st * KT;
                    if (biased) {
                        if (!warp_wait(&lb_full[st], (unsigned)(step / ST) & 1u, p.wait_ns)) { stop = true; break; }
#pragma unroll
                        for (int e = 0; e < 128; e += 32) low = low && lbf[lane + e] <= 0.f;
                    }
                    float x[128];
#pragma unroll
                    for (int c = 0; c < 128; c += 32) tmem_ld32(ts + c, x + c);
                    tmem_ld_wait();
                    float mx[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int c = 0; c < 128; c += 8)
#pragma unroll
                        for (int e = 0; e < 4; ++e) mx[e] = max3(mx[e], fabsf(x[c + 2 * e]), fabsf(x[c + 2 * e + 1]));
                    const float most = max3(mx[0], mx[1], fmaxf(mx[2], mx[3]));
                    if (__all_sync(kFull, low && fminf(most * p.scale * kLog2e, cap2) - m_ref <= 16.f)) {
                        const bool tiny = cap_tiny(most, per_cap), small = cap_small(most, per_cap);
                        const uint64_t c2 = pk2(C, C), n2 = pk2(-m_ref, -m_ref);
                        uint64_t sums[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll 1
                        for (int c = 0; c < 128; c += 32) {
                            float y[32];
                            tmem_ld32(ts + c, y);
                            tmem_ld_wait();
                            if (tiny)
                                cap_by_2(y, per_cap, cap2);
                            else if (small)
                                cap_by_4(y, per_cap, cap2);
                            else
                                cap_by_exp(y, per_cap, cap2);
                            if (biased) add_bias(y, reinterpret_cast<const float4*>(lbf + c), (float)(i - j0 - c), j0 + KT <= first + 1);
                            weights(y, c2, n2, sums, ts + c / 2);
                            if (c == 32) half_done();
                        }
                        all_done(sums);
                        continue;
                    }
                }
                if (CAP || biased || masked) {
                    // the cap, the bias and the mask of these tiles go into S itself
                    if (biased && !warp_wait(&lb_full[st], (unsigned)(step / ST) & 1u, p.wait_ns)) { stop = true; break; }
                    const float4* lb = reinterpret_cast<const float4*>(smem + SH::LB_OFF + st * KT * 4);
#pragma unroll 1
                    for (int c0 = 0; c0 < KT; c0 += 32) {
                        float y[32];
                        if (masked && c0 >= hi - j0) {
#pragma unroll
                            for (int c = 0; c < 32; ++c) y[c] = -INFINITY;
                        } else {
                            tmem_ld32(ts + c0, y);
                            tmem_ld_wait();
                            if (CAP) cap_scores(y, per_cap, cap2);
                            if (biased) add_bias(y, lb + c0 / 4, (float)(i - j0 - c0), j0 + KT <= first + 1);
                            if (masked && c0 + 32 > lo - j0) {
#pragma unroll
                                for (int c = 0; c < 32; ++c) y[c] = c < lim - j0 - c0 ? y[c] : -INFINITY;
                            }
                        }
                        tmem_st32(ts + c0, reinterpret_cast<const uint32_t*>(y));
                    }
                    tmem_st_wait();
                }
                float x[128];
#pragma unroll
                for (int c = 0; c < 128; c += 32) tmem_ld32(ts + c, x + c);
                tmem_ld_wait();
                float mx[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
                for (int c = 4; c < 124; c += 8)
#pragma unroll
                    for (int e = 0; e < 4; ++e) mx[e] = max3(mx[e], x[c + 2 * e], x[c + 2 * e + 1]);
                const float mt = max3(max3(mx[0], x[124], x[125]), max3(mx[1], x[126], x[127]), fmaxf(mx[2], mx[3]));
                // the reference moves when the row's maximum passes it by more than 2^8: P <= 256, and O is
                // rescaled (read, scaled, written back in tensor memory) only then. P V(tile + 1) is done:
                // its product was issued before this S.
                const bool grow = mt > m_ref && (m_ref == -INFINITY || (mt - m_ref) * C > 8.f);
                const bool resc = grow && m_ref != -INFINITY;
                if (__any_sync(kFull, resc)) {
                    const float alpha = resc ? ex2_approx((m_ref - mt) * C) : 1.f;
#pragma unroll 1
                    for (int c = 0; c < D; c += 32) {
                        float o[32];
                        tmem_ld32(to + c, o);
                        tmem_ld_wait();
                        uint32_t w[32];
#pragma unroll
                        for (int e = 0; e < 32; ++e) w[e] = __float_as_uint(o[e] * alpha);
                        tmem_st32(to + c, w);
                    }
                    l_sum *= alpha;
                }
                if (grow) m_ref = mt;
                const float neg = (m_ref == -INFINITY) ? 0.f : -m_ref * C;
                const uint64_t c2 = pk2(C, C), n2 = pk2(neg, neg);
                uint64_t sums[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
                for (int c = 0; c < 128; c += 32) {
                    weights(x + c, c2, n2, sums, ts + c / 2);
                    if (c == 32) half_done();
                }
                all_done(sums);
            }
            if (stop) break;
            if (!warp_wait(&o_full[t], (unsigned)oc & 1u, p.wait_ns)) { stop = true; break; }
            ++oc;
            tc_fence_after();
            const size_t row = (size_t)(s + i) * p.Hq + (g << lg) + (r & (p.G - 1));
            const float inv = l_sum == 0.f ? 0.f : 1.f / l_sum;
            uint4* dst = reinterpret_cast<uint4*>(p.o + row * D);
#pragma unroll 1
            for (int c0 = 0; c0 < D; c0 += 32) {
                float o[32];
                tmem_ld32(to + c0, o);
                tmem_ld_wait();
                if (i < len) store_bf16x32(dst + c0 / 8, o, inv);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&o_empty[t]);   // the next unit's product may overwrite O
            if (i < len && p.lse != nullptr) p.lse[row] = (m_ref * C + log2f(l_sum)) * kLn2;
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
        for (int k = max(0, s_steps[0] - ST); k < s_steps[0]; ++k) {
            mbar_wait(&k_full[k % ST], (unsigned)(k / ST) & 1u, 100000000ull);
            mbar_wait(&v_full[k % ST], (unsigned)(k / ST) & 1u, 100000000ull);
        }
        if (s_steps[1] > 0) mbar_wait(q_full, (unsigned)(s_steps[1] - 1) & 1u, 100000000ull);
    }
    __syncthreads();
    if (warp == 8) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(SH::TM_COLS) : "memory");
    }
}

}  // namespace kvb
