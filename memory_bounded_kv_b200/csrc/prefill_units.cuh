// Work units and score arithmetic shared by the prompt-attention kernels.
#pragma once

#include "tc5.cuh"

namespace kvb {

struct PrefillParams {
    const uint16_t* q;
    const uint16_t* k;
    const uint16_t* v;
    const float* lb;          // log beta or null
    const int* cu;            // [N + 1]
    const int* prefix;        // [N] or null
    long long q_st, q_sh, kv_st, kv_sh, lb_st, lb_sh;   // element strides of a token and of a head
    int T, N, Hq, Hkv, G;
    float scale, softcap;     // softcap 0: no cap
    uint16_t* o;              // [T, Hq, d] bf16
    float* lse;               // [T, Hq] or null
    unsigned long long wait_ns;
    int withhold;             // test hook: CTA withhold - 1 loads its first tile alone, so its other roles' waits run out (0: off)
    // gradients
    const uint16_t* d_o;      // [T, Hq, d]
    const float* d_lse;       // [T, Hq] or null
    float* delta;             // [T, Hq]: sum_j p_ij (dO_i . v_j) - dlse_i
    uint16_t* dq;             // [T, Hq, d]
    uint16_t* dk;             // [T, Hkv, d]
    uint16_t* dv;             // [T, Hkv, d]
    float* dlb;               // [T, Hkv] or null
    float* parts;             // [pieces][2] sums of key blocks that a cut goes through (kPartFloats each)
    int4* records;            // [pieces] the key block that goes on behind a piece: first row, rows, kv head, last piece
                              // (-1: none; -2: the CTA gave up)
    int* dq_done;             // [dq_ctas] whether a CTA of the kernel by query rows left all its deltas
    int dq_ctas;
};

constexpr int kMaxPieces = 160;                          // CTAs of each gradient kernel, at most
constexpr int kPartFloats = 2 * 128 * 128 + 128;         // dV^T, dK^T [d][128 keys], d log beta [128 keys]

// A unit: block `blk` of 2^sh tokens of a document (rows s .. s + len) and a kv head.
struct PrefillUnit {
    int s, len, blk, g, pre;
};

// The units in an order of falling work, found from cu alone (the host does not know the lengths):
// level b holds block b of every document that has one, for every kv head, and later blocks see more
// keys. A whole warp walks it; document `lane`'s bounds stay in registers. With cu out of order or
// outside [0, T] there are no units (KVB_DERR_RANGE).
struct PrefillWalk {
    const int* cu;
    const int* prefix;
    int N, Hkv, sh, lane, s0, e0, levels;
    long long units;

    __device__ __forceinline__ int blocks_of(int s, int e) const { return (e - s + (1 << sh) - 1) >> sh; }
    __device__ __forceinline__ int blocks(int n) const { return n < N ? blocks_of(cu[n], cu[n + 1]) : 0; }
    // blocks of level >= b, all documents
    __device__ __forceinline__ int count(int b) const {
        int c = max(blocks_of(s0, e0) - b, 0);
        for (int n = lane + 32; n < N; n += 32) c += max(blocks(n) - b, 0);
        return __reduce_add_sync(kFull, c);
    }
    __device__ __forceinline__ PrefillWalk(const PrefillParams& p, int sh_)
        : cu(p.cu), prefix(p.prefix), N(p.N), Hkv(p.Hkv), sh(sh_), lane(threadIdx.x & 31) {
        s0 = lane < N ? cu[lane] : 0;
        e0 = lane < N ? cu[lane + 1] : 0;
        bool bad = s0 < 0 || e0 < s0 || e0 > p.T;
        levels = blocks_of(s0, e0);
        for (int n = lane + 32; n < N; n += 32) {
            const int s = cu[n], e = cu[n + 1];
            bad |= s < 0 || e < s || e > p.T;
            levels = max(levels, blocks_of(s, e));
        }
        if (__any_sync(kFull, bad)) {
            if (lane == 0) raise_error(KVB_DERR_RANGE);
            units = 0;
            return;
        }
        levels = __reduce_max_sync(kFull, levels);
        units = (long long)count(0) * Hkv;
    }
    // unit u of [0, units)
    __device__ __forceinline__ PrefillUnit unit(long long u) const {
        int lo = 0, hi = levels;   // count(lo) * Hkv > u >= count(hi) * Hkv
        int above = 0;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1, c = count(mid);
            if ((long long)c * Hkv > u) {
                lo = mid;
            } else {
                hi = mid;
                above = c;
            }
        }
        const long long at = u - (long long)above * Hkv;
        int rank = (int)(at / Hkv), doc = 0;
        for (int n0 = 0; n0 < N; n0 += 32) {
            const bool has = (n0 == 0 ? blocks_of(s0, e0) : blocks(n0 + lane)) > lo;
            const unsigned m = __ballot_sync(kFull, has);
            const int c = __popc(m);
            if (rank < c) {
                const unsigned pick = __ballot_sync(kFull, has && __popc(m & ((1u << lane) - 1u)) == rank);
                doc = n0 + __ffs(pick) - 1;
                break;
            }
            rank -= c;
        }
        PrefillUnit x;
        int e;
        if (doc < 32) {
            x.s = __shfl_sync(kFull, s0, doc);
            e = __shfl_sync(kFull, e0, doc);
        } else {
            x.s = cu[doc];
            e = cu[doc + 1];
        }
        x.len = e - x.s;
        x.blk = lo;
        x.g = (int)(at % Hkv);
        x.pre = prefix == nullptr ? 0 : min(max(prefix[doc], 0), x.len);
        return x;
    }
    // the r-th unit of CTA `c` of `grid`: rounds run forth and back, so that the CTA with a round's
    // heaviest unit gets the next round's lightest
    __device__ __forceinline__ static long long nth(long long r, int c, int grid) {
        return r * grid + ((r & 1) ? grid - 1 - c : c);
    }
};

// The work of the kernel by keys as one line of steps (128 query rows against 128 keys), in the order
// (document, kv head, key block, query block), to be cut into equal pieces: the first keys of a long
// document meet all its queries, and where there are few key blocks most CTAs would wait for those. A key
// block that a cut goes through is summed from its pieces afterwards, in order.
struct StepLine {
    const int* cu;
    const int* prefix;
    int N, Hkv, lg, lane;
    long long steps;   // 0 with cu out of order or outside [0, T] (KVB_DERR_RANGE)
    int longest;       // steps of the heaviest key block

    struct Doc {
        int s, len, pre, nq, nk, np;   // query blocks, key blocks, key blocks that begin inside the prefix
        // steps of the key blocks before kb, one kv head: the queries of block kb begin at kb 2^lg, or at 0
        __device__ __forceinline__ long long before(int kb, int lg) const {
            const long long k = kb, f = min(kb, np);
            return k * nq - (((k * (k - 1) - f * (f - 1)) / 2) << lg);
        }
    };
    __device__ __forceinline__ Doc doc(int n) const {
        Doc d{};
        if (n < N) {
            d.s = cu[n];
            d.len = cu[n + 1] - d.s;
            d.pre = prefix == nullptr ? 0 : min(max(prefix[n], 0), d.len);
            d.nq = (d.len + (128 >> lg) - 1) >> (7 - lg);
            d.nk = (d.len + 127) >> 7;
            d.np = (d.pre + 127) >> 7;
        }
        return d;
    }
    __device__ __forceinline__ StepLine(const PrefillParams& p)
        : cu(p.cu), prefix(p.prefix), N(p.N), Hkv(p.Hkv), lane(threadIdx.x & 31), steps(0), longest(0) {
        lg = 31 - __clz(p.G);
        bool bad = false;
        for (int n = lane; n < N; n += 32) bad |= cu[n] < 0 || cu[n + 1] < cu[n] || cu[n + 1] > p.T;
        if (__any_sync(kFull, bad)) {
            if (lane == 0) raise_error(KVB_DERR_RANGE);
            return;
        }
        for (int n = lane; n < N; n += 32) {
            const Doc d = doc(n);
            steps += d.before(d.nk, lg);
            longest = max(longest, d.nq);
        }
        longest = __reduce_max_sync(kFull, longest);
#pragma unroll
        for (int m = 16; m >= 1; m >>= 1) steps += __shfl_xor_sync(kFull, steps, m);
        steps *= Hkv;
    }
    __device__ __forceinline__ long long piece(int pieces) const { return (steps + pieces - 1) / pieces; }
    // Whether to cut: where one key block weighs as much as three quarters of a CTA's share. Below that whole
    // key blocks, heaviest first, balance as well, and CTAs that walk the same queries together read them from
    // L2 (8192 tokens, 32/8 heads, d 128: 895 us whole, 972 and the sums cut). 5003 ragged tokens, 16/4 heads,
    // d 128, with a cap, all kernels: 461 us whole, 384 cut; 301 tokens, 8/2 heads, d 64: 44.6 whole, 37.7 cut.
    __device__ __forceinline__ bool cut(int pieces) const { return 4LL * longest > 3 * piece(pieces); }

    struct At {
        Doc d;
        int g, kb, b0;            // kv head, key block, its first query block
        long long begin, end;     // the steps of this (document, head, key block)
    };
    // the key block that step x of [0, steps) belongs to
    __device__ __forceinline__ At find(long long x) const {
        At a{};
        long long base = 0;
        for (int n0 = 0; n0 < N; n0 += 32) {
            Doc d = doc(n0 + lane);
            const long long own = d.before(d.nk, lg) * Hkv;
            long long upto = own;
#pragma unroll
            for (int m = 1; m < 32; m <<= 1) {
                const long long y = __shfl_up_sync(kFull, upto, m);
                if (lane >= m) upto += y;
            }
            const unsigned hit = __ballot_sync(kFull, base + upto > x);
            if (hit) {
                const int l = __ffs(hit) - 1;
                base += __shfl_sync(kFull, upto - own, l);
                a.d.s = __shfl_sync(kFull, d.s, l);
                a.d.len = __shfl_sync(kFull, d.len, l);
                a.d.pre = __shfl_sync(kFull, d.pre, l);
                a.d.nq = __shfl_sync(kFull, d.nq, l);
                a.d.nk = __shfl_sync(kFull, d.nk, l);
                a.d.np = __shfl_sync(kFull, d.np, l);
                break;
            }
            base += __shfl_sync(kFull, upto, 31);
        }
        const long long per_head = a.d.before(a.d.nk, lg);
        a.g = (int)((x - base) / per_head);
        base += a.g * per_head;
        int lo = 0, hi = a.d.nk;   // before(lo) <= x - base < before(hi)
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (a.d.before(mid, lg) <= x - base) {
                lo = mid;
            } else {
                hi = mid;
            }
        }
        a.kb = lo;
        a.b0 = lo < a.d.np ? 0 : lo << lg;
        a.begin = base + a.d.before(lo, lg);
        a.end = base + a.d.before(lo + 1, lg);
        return a;
    }
};

// ---- packed pairs of floats -------------------------------------------------------------------
__device__ __forceinline__ uint64_t pk2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void upk2(uint64_t r, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(r)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

__device__ __forceinline__ uint64_t same2(float a) { return pk2(a, a); }

// the larger of two, NaN where one is
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// 2^x of a pair on the FMA pipe, for x < 128; 0 below -126.5 (-inf too), NaN stays. With n the nearest integer
// (left in the low bits of x + 1.5 2^23) and f = x - n in [-1/2, 1/2], 2^f by the polynomial of degree DEG whose
// largest relative error is smallest (4: 2.6e-6, 5: 7.5e-8; found by a weighted least-squares iteration),
// times 2^n. That is a product and not an addition to the exponent's bits: those of NaN would come out finite,
// and n = -127, where the lower bound of x ends, gives the factor 0.
template <int DEG>
__device__ __forceinline__ void exp2_poly2(float& a, float& b) {
    static_assert(DEG == 4 || DEG == 5, "degree");
    const uint64_t x = pk2(max_nan(a, -127.f), max_nan(b, -127.f));
    const uint64_t t = add2(x, same2(12582912.f));
    const uint64_t f = fma2(add2(t, same2(-12582912.f)), same2(-1.f), x);
    uint64_t r;
    if (DEG == 4) {
        r = fma2(same2(0.009570086374878883f), f, same2(0.055917851626873016f));
        r = fma2(r, f, same2(0.240247443318367f));
        r = fma2(r, f, same2(0.6931217908859253f));
        r = fma2(r, f, same2(0.9999992847442627f));
    } else {
        r = fma2(same2(0.0013276460813358426f), f, same2(0.009675541892647743f));
        r = fma2(r, f, same2(0.05550713464617729f));
        r = fma2(r, f, same2(0.24022120237350464f));
        r = fma2(r, f, same2(0.6931469440460205f));
        r = fma2(r, f, same2(1.0000001192092896f));
    }
    float ta, tb;
    upk2(t, ta, tb);
    upk2(mul2(r, pk2(__uint_as_float((__float_as_uint(ta) << 23) + 0x3f800000u),
                     __uint_as_float((__float_as_uint(tb) << 23) + 0x3f800000u))), a, b);
}

// the larger of three (NaN is passed over, as fmaxf does)
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// 1 / x to about 2^-23 (PTX rcp.approx.ftz)
__device__ __forceinline__ float rcp_approx(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 32 values times f, as bf16, to 64 bytes of a row; a thread writes its own row, so a store touches 32
// lines: in 32 bytes each (whole sectors, half the stores) where the address allows
__device__ __forceinline__ void store_bf16x32(void* dst, const float (&o)[32], float f) {
    uint32_t w[16];
#pragma unroll
    for (int c = 0; c < 16; ++c) w[c] = pack_bf16(o[2 * c] * f, o[2 * c + 1] * f);
    if ((reinterpret_cast<uintptr_t>(dst) & 31) == 0) {
#pragma unroll
        for (int c = 0; c < 16; c += 8)
            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(static_cast<uint32_t*>(dst) + c),
                         "r"(w[c]), "r"(w[c + 1]), "r"(w[c + 2]), "r"(w[c + 3]), "r"(w[c + 4]), "r"(w[c + 5]), "r"(w[c + 6]),
                         "r"(w[c + 7])
                         : "memory");
    } else {
#pragma unroll
        for (int c = 0; c < 16; c += 4) static_cast<uint4*>(dst)[c / 4] = make_uint4(w[c], w[c + 1], w[c + 2], w[c + 3]);
    }
}

// tanh(y) = 1 - 2 / (1 + e^2y): off by about 2^-23 absolute
__device__ __forceinline__ float tanh_exp(float y) { return 1.f - 2.f * rcp_approx(1.f + ex2_approx(2.f * kLog2e * y)); }

// x = amp tanh(per_cap x), N values: where a warp's y = per_cap x are small (scores small beside the cap, the
// common case) by y times the polynomial in y^2 whose largest relative error is smallest, which also keeps
// small values to fp32 accuracy: degree 2 for y^2 <= 1/32 (5e-8; scores of variance 1 beside a cap of 25), with
// per_cap in the coefficients, degree 4 for y^2 <= 1/4 (1.3e-8); else through the exponential.
// `most` is the largest |x| of each thread. One choice for 64 values beats two for 32 in the gradients (8192
// tokens, cap 50, d 128: 1137 -> 1090 and 1291 -> 1240 us).
__device__ __forceinline__ bool cap_tiny(float most, float per_cap) {
    // the coefficients' range: per_cap^4 and x^2 stay normal numbers
    return __all_sync(kFull, most * per_cap <= 0.17677669f) && per_cap >= 1e-6f && per_cap <= 1e6f;
}
__device__ __forceinline__ bool cap_small(float most, float per_cap) { return __all_sync(kFull, most * per_cap <= 0.5f); }

template <int N = 32>
__device__ __forceinline__ void cap_by_2(float* x, float per_cap, float amp) {
    const float k1 = amp * per_cap, k2 = per_cap * per_cap;
    const uint64_t c2 = same2(k1 * k2 * k2 * 0.13083961606025696f), c1 = same2(k1 * k2 * -0.333304226398468f), c0 = same2(k1);
#pragma unroll
    for (int c = 0; c < N; c += 2) {
        const uint64_t z = pk2(x[c], x[c + 1]), u = mul2(z, z);
        upk2(mul2(fma2(fma2(c2, u, c1), u, c0), z), x[c], x[c + 1]);
    }
}

template <int N = 32>
__device__ __forceinline__ void cap_by_4(float* x, float per_cap, float amp) {
    const uint64_t c4 = same2(amp * 0.017135005444288254f), c3 = same2(amp * -0.05298607423901558f),
                   c2 = same2(amp * 0.13324779272079468f), c1 = same2(amp * -0.3333306908607483f), c0 = same2(amp);
#pragma unroll
    for (int c = 0; c < N; c += 2) {
        const uint64_t y = mul2(pk2(x[c], x[c + 1]), same2(per_cap)), u = mul2(y, y);
        const uint64_t r = fma2(fma2(fma2(fma2(c4, u, c3), u, c2), u, c1), u, c0);
        upk2(mul2(r, y), x[c], x[c + 1]);
    }
}

template <int N = 32>
__device__ __forceinline__ void cap_by_exp(float* x, float per_cap, float amp) {
#pragma unroll
    for (int c = 0; c < N; ++c) x[c] = amp * tanh_exp(x[c] * per_cap);
}

template <int N = 32>
__device__ __forceinline__ void cap_scores(float* x, float per_cap, float amp) {
    float most = 0.f;
#pragma unroll
    for (int c = 0; c < N; c += 2) most = max3(most, fabsf(x[c]), fabsf(x[c + 1]));
    if (cap_tiny(most, per_cap))
        cap_by_2<N>(x, per_cap, amp);
    else if (cap_small(most, per_cap))
        cap_by_4<N>(x, per_cap, amp);
    else
        cap_by_exp<N>(x, per_cap, amp);
}

// the derivative 1 - tanh^2 of a pair of capped scores x = amp tanh(.); minus_inv = -1 / amp^2
__device__ __forceinline__ uint64_t cap_slope2(float x, float y, float minus_inv) {
    const uint64_t z = pk2(x, y);
    return fma2(z, mul2(z, same2(minus_inv)), same2(1.f));
}

// x_c += max(dist - c, 0) b_c for 32 keys; without the maximum where all are past
__device__ __forceinline__ void add_bias(float* x, const float4* b4, float dist, bool past) {
    if (past) {
        uint64_t d = pk2(dist, dist - 1.f);
#pragma unroll
        for (int c = 0; c < 32; c += 4) {
            const float4 b = b4[c / 4];
            upk2(fma2(d, pk2(b.x, b.y), pk2(x[c], x[c + 1])), x[c], x[c + 1]);
            d = add2(d, same2(-2.f));
            upk2(fma2(d, pk2(b.z, b.w), pk2(x[c + 2], x[c + 3])), x[c + 2], x[c + 3]);
            d = add2(d, same2(-2.f));
        }
    } else {
#pragma unroll
        for (int c = 0; c < 32; c += 4) {
            const float4 b = b4[c / 4];
            x[c] = fmaf(fmaxf(dist - c, 0.f), b.x, x[c]);
            x[c + 1] = fmaf(fmaxf(dist - (c + 1), 0.f), b.y, x[c + 1]);
            x[c + 2] = fmaf(fmaxf(dist - (c + 2), 0.f), b.z, x[c + 2]);
            x[c + 3] = fmaf(fmaxf(dist - (c + 3), 0.f), b.w, x[c + 3]);
        }
    }
}

// log beta within +-2^60 (NaN stays): -inf times a distance would meet 0 * inf, and its bf16 parts NaN
__device__ __forceinline__ float clamp_log_beta(float x) {
    constexpr float B = 1152921504606846976.f;
    return x < -B ? -B : (x > B ? B : x);
}

// Shared-memory descriptors, low word (address / 16, leading byte offset) and high word apart: one
// thread issues every product, and a product's operands differ in the low word by a constant.
//   sw128: K-major, 128-byte swizzle (rows of 128 bytes, 8-row groups of 1024)
//   mn:    MN-major, 128-byte swizzle, groups of 64 elements `half` bytes apart, 8-row groups of 1024
//   plain: K-major without swizzle, 16 elements of K: 8 rows x 16 bytes are 128 contiguous bytes, the
//          second 16-byte chunk of K 128 bytes on, 8-row groups 256 bytes
constexpr uint32_t kDescSw128Hi = 64u | (1u << 14) | (2u << 29), kDescPlainHi = 16u | (1u << 14);
__device__ __forceinline__ uint32_t desc_sw128_lo(uint32_t saddr) { return (saddr >> 4) | (1u << 16); }
__device__ __forceinline__ uint32_t desc_mn_lo(uint32_t saddr, uint32_t half) { return (saddr >> 4) | ((half >> 4) << 16); }
__device__ __forceinline__ uint32_t desc_plain_lo(uint32_t saddr) { return (saddr >> 4) | (8u << 16); }
__device__ __forceinline__ uint64_t desc(uint32_t lo, uint32_t hi) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(lo), "r"(hi));
    return d;
}
// D (+)= A B^T over K = 16 * STEPS; a, b: low words of K-major 128-byte-swizzled operands whose 64-wide
// halves are `ah`, `bh` bytes apart
template <int STEPS>
__device__ __forceinline__ void umma_kmajor(uint32_t d, uint32_t a, uint32_t ah, uint32_t b, uint32_t bh, uint32_t idesc) {
#pragma unroll
    for (int kk = 0; kk < STEPS; ++kk)
        umma_bf16(d, desc(a + (((kk >> 2) * ah + (kk & 3) * 32) >> 4), kDescSw128Hi),
                  desc(b + (((kk >> 2) * bh + (kk & 3) * 32) >> 4), kDescSw128Hi), idesc, kk > 0 ? 1u : 0u);
}
// the same with A in tensor memory
template <int STEPS>
__device__ __forceinline__ void umma_kmajor_ts(uint32_t d, uint32_t a_tmem, uint32_t b, uint32_t bh, uint32_t idesc) {
#pragma unroll
    for (int kk = 0; kk < STEPS; ++kk)
        umma_bf16_ts(d, a_tmem + kk * 8, desc(b + (((kk >> 2) * bh + (kk & 3) * 32) >> 4), kDescSw128Hi), idesc, kk > 0 ? 1u : 0u);
}
// D (+)= A B over K = 16 * STEPS rows of B (MN-major, 128 bytes a row and half), A in tensor memory
template <int STEPS>
__device__ __forceinline__ void umma_rows(uint32_t d, uint32_t a_tmem, uint32_t b, uint32_t idesc, bool fresh) {
#pragma unroll
    for (int kk = 0; kk < STEPS; ++kk)
        umma_bf16_ts(d, a_tmem + kk * 8, desc(b + kk * 128, kDescSw128Hi), idesc, kk > 0 || !fresh ? 1u : 0u);
}
// byte offset of chunk c (0, 1) of a row in that layout
__host__ __device__ constexpr int plain16_off(int row, int c) { return (row >> 3) * 256 + c * 128 + (row & 7) * 16; }

// Three bf16 parts of an fp32 value (24 bits, so hi + mid + lo = x), each in the low half of a word
__device__ __forceinline__ void split3_bf16(float x, uint32_t& hi, uint32_t& mid, uint32_t& lo) {
    hi = pack_bf16(x, 0.f);
    const float r = x - bf16_lo(hi);
    mid = pack_bf16(r, 0.f);
    lo = pack_bf16(r - bf16_lo(mid), 0.f);
}

// The bias columns of a key: with the query's (i', i', i', 1, 1, 1, 0, 0), i' = i - base, the product is
// i' b + (base - j) b = (i - j) b, b in the units of the raw scores.
__device__ __forceinline__ uint4 bias_columns(float b, int base_minus_j) {
    uint32_t bh, bm, bl, ch, cm, cl;
    split3_bf16(b, bh, bm, bl);
    split3_bf16((float)base_minus_j * b, ch, cm, cl);
    return make_uint4(bh | (bm << 16), bl | (ch << 16), cm | (cl << 16), 0u);
}
// ... and a query's: i' <= 255 is exact in bf16
__device__ __forceinline__ uint4 bias_query(int i) {
    const uint32_t x = pack_bf16((float)i, (float)i), one = 0x3f803f80u;
    return make_uint4(x, (x & 0xffffu) | (one & 0xffff0000u), one, 0u);
}

}  // namespace kvb
