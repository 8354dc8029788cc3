// libkvb: C ABI (include/kvb.h) of the prompt's path: attention over packed prompts and its
// gradients, page planning and page writes. As in kvb.cu, the host code validates, picks the
// kernel and launches it on the caller's stream; it allocates nothing.
#include <algorithm>
#include <atomic>
#include <cmath>

#include "host.cuh"
#include "paged_fill.cuh"
#include "prefill_bwd.cuh"
#include "prefill_fwd.cuh"

kvb_status kvb_prefill_take_error(unsigned* bits) { return take_error_word(bits); }

namespace {

inline size_t round256(size_t x) { return (x + 255) / 256 * 256; }
inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Test hook of kvb_test_withhold_next_prefill: wait limit (ns) | kernel << 32 | (CTA + 1) << 40; 0 = off. Taken
// (and cleared) by the next call that launches the kernel.
std::atomic<unsigned long long> g_withhold_prefill{0};

bool take_withheld(unsigned kernel, kvb::PrefillParams* p) {
    unsigned long long x = g_withhold_prefill.load(std::memory_order_relaxed);
    if (x == 0 || ((x >> 32) & 255) != kernel || !g_withhold_prefill.compare_exchange_strong(x, 0)) return false;
    p->wait_ns = x & 0xffffffffull;
    p->withhold = (int)(x >> 40);
    return true;
}

// The host checks of kvb_prefill_attn and its gradients, and the kernels' parameters.
kvb_status prefill_params(const kvb_prefill_args* a, kvb::PrefillParams* out) {
    if (a == nullptr) return KVB_EINVAL;
    if (a->T < 0 || a->T > KVB_PREFILL_MAX_TOKENS || a->N < 0 || a->N > KVB_PREFILL_MAX_DOCS || a->Hq < 1 || a->Hkv < 1) return KVB_EINVAL;
    if ((a->d != 64 && a->d != 128) || a->Hq % a->Hkv != 0 || a->Hq > 65535) return KVB_EINVAL;
    const int G = a->Hq / a->Hkv;
    if (G != 1 && G != 2 && G != 4 && G != 8) return KVB_EINVAL;
    // the bias rides the score product divided by the scale: both ends keep it in range
    const double scale = a->scale == 0.0f ? 1.0 / std::sqrt((double)a->d) : (double)a->scale;
    if (!(scale >= KVB_PREFILL_MIN_SCALE && scale <= 1.0 / KVB_PREFILL_MIN_SCALE)) return KVB_EINVAL;
    if (a->softcap != 0.0f && !(a->softcap >= KVB_PREFILL_MIN_SCALE && a->softcap <= 1.0f / KVB_PREFILL_MIN_SCALE)) return KVB_EINVAL;
    if (!a->q || !a->k || !a->v || !a->cu || !a->o) return KVB_EINVAL;
    if (!aligned16(a->q) || !aligned16(a->k) || !aligned16(a->v) || !aligned16(a->o)) return KVB_EINVAL;
    if (!aligned4(a->log_beta) || !aligned4(a->cu) || !aligned4(a->prefix_len) || !aligned4(a->lse)) return KVB_EINVAL;
    const long long s[4] = {a->q_stride_t, a->q_stride_h, a->kv_stride_t, a->kv_stride_h};
    for (long long x : s)
        if (x < a->d || x % 8 != 0 || x >= (1LL << 38)) return KVB_EINVAL;
    if (a->log_beta && (a->lb_stride_t < 0 || a->lb_stride_h < 0)) return KVB_EINVAL;
    kvb::PrefillParams& p = *out;
    p = kvb::PrefillParams{};
    p.q = a->q; p.k = a->k; p.v = a->v; p.lb = a->log_beta; p.cu = a->cu; p.prefix = a->prefix_len;
    p.q_st = a->q_stride_t; p.q_sh = a->q_stride_h; p.kv_st = a->kv_stride_t; p.kv_sh = a->kv_stride_h;
    p.lb_st = a->lb_stride_t; p.lb_sh = a->lb_stride_h;
    p.T = a->T; p.N = a->N; p.Hq = a->Hq; p.Hkv = a->Hkv; p.G = G;
    p.scale = (float)scale; p.softcap = a->softcap;
    p.o = a->o; p.lse = a->lse;
    p.wait_ns = 1000000000ull;
    return KVB_OK;
}

// Packed rows x [T][H][d] with strides (elements), in boxes of 64 dims x `bh` heads x `bt` tokens (128-byte
// swizzle; rows past T read zeros).
bool make_rows_map(CUtensorMap* map, const void* x, int d, int H, int T, long long sh, long long st, int bh, int bt) {
    EncodeTiledFn fn = encode_tiled();
    if (fn == nullptr) return false;
    cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)H, (cuuint64_t)T};
    cuuint64_t strides[2] = {(cuuint64_t)sh * 2, (cuuint64_t)st * 2};
    cuuint32_t box[3] = {64, (cuuint32_t)bh, (cuuint32_t)bt};
    cuuint32_t estr[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(x), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The most units of 2^sh tokens that N documents of T tokens in all can have.
long long most_units(const kvb::PrefillParams& p, int sh) { return ((long long)(p.T >> sh) + p.N) * p.Hkv; }

// log2 of the tokens whose 256 query rows are a unit of the kernels by query rows
int unit_shift(const kvb::PrefillParams& p) {
    int sh = 8;
    for (int g = p.G; g > 1; g >>= 1) --sh;
    return sh;
}

template <int D, bool BETA, bool CAP>
kvb_status launch_fwd(const kvb::PrefillParams& p, cudaStream_t st) {
    using SH = kvb::FwdShape<D>;
    auto kern = kvb::prefill_fwd_kernel<D, BETA, CAP>;
    if (set_smem(kern, SH::SMEM) != KVB_OK) return KVB_ECUDA;
    CUtensorMap mq, mk, mv;
    if (!make_rows_map(&mq, p.q, D, p.Hq, p.T, p.q_sh, p.q_st, p.G, 128 / p.G) ||
        !make_rows_map(&mk, p.k, D, p.Hkv, p.T, p.kv_sh, p.kv_st, 1, SH::KT) ||
        !make_rows_map(&mv, p.v, D, p.Hkv, p.T, p.kv_sh, p.kv_st, 1, SH::KT))
        return KVB_EINVAL;
    const int slots = resident_ctas(kern, SH::NT, SH::SMEM);
    if (slots <= 0) return KVB_ECUDA;
    const int grid = (int)std::min<long long>(slots, most_units(p, unit_shift(p)));
    return launch_pdl(kern, dim3(grid), dim3(SH::NT), SH::SMEM, st, p, mq, mk, mv);
}

template <int D>
kvb_status fwd_dispatch(const kvb::PrefillParams& p, cudaStream_t st) {
    const bool beta = p.lb != nullptr, cap = p.softcap > 0.f;
    if (beta) return cap ? launch_fwd<D, true, true>(p, st) : launch_fwd<D, true, false>(p, st);
    return cap ? launch_fwd<D, false, true>(p, st) : launch_fwd<D, false, false>(p, st);
}

template <int D, bool BETA, bool CAP>
kvb_status launch_bwd(kvb::PrefillParams p, cudaStream_t st) {
    using SQ = kvb::DqShape<D>;
    using SK = kvb::DkvShape<D>;
    auto kq = kvb::prefill_dq_kernel<D, BETA, CAP>;
    auto kk = kvb::prefill_dkv_kernel<D, BETA, CAP>;
    if (set_smem(kq, SQ::SMEM) != KVB_OK || set_smem(kk, SK::SMEM) != KVB_OK) return KVB_ECUDA;
    CUtensorMap mq, mo, mk, mv;
    if (!make_rows_map(&mk, p.k, D, p.Hkv, p.T, p.kv_sh, p.kv_st, 1, SQ::KT) ||
        !make_rows_map(&mv, p.v, D, p.Hkv, p.T, p.kv_sh, p.kv_st, 1, SQ::KT))
        return KVB_EINVAL;
    int slots = resident_ctas(kq, SQ::NT, SQ::SMEM);
    if (slots <= 0) return KVB_ECUDA;
    int grid = (int)std::min<long long>(std::min(slots, kvb::kMaxPieces), most_units(p, unit_shift(p) - 1));
    p.dq_ctas = grid;
    kvb::PrefillParams hooked = p;
    take_withheld(1, &hooked);
    if (launch_pdl(kq, dim3(grid), dim3(SQ::NT), SQ::SMEM, st, hooked, mk, mv) != KVB_OK) return KVB_ECUDA;
    if (!make_rows_map(&mq, p.q, D, p.Hq, p.T, p.q_sh, p.q_st, p.G, SK::QT / p.G) ||
        !make_rows_map(&mo, p.d_o, D, p.Hq, p.T, D, (long long)p.Hq * D, p.G, SK::QT / p.G) ||
        !make_rows_map(&mk, p.k, D, p.Hkv, p.T, p.kv_sh, p.kv_st, 1, SK::KT) ||
        !make_rows_map(&mv, p.v, D, p.Hkv, p.T, p.kv_sh, p.kv_st, 1, SK::KT))
        return KVB_EINVAL;
    slots = resident_ctas(kk, SK::NT, SK::SMEM);
    if (slots <= 0) return KVB_ECUDA;
    grid = std::min(slots, kvb::kMaxPieces);
    hooked = p;
    take_withheld(2, &hooked);
    if (launch_pdl(kk, dim3(grid), dim3(SK::NT), SK::SMEM, st, hooked, mq, mo, mk, mv) != KVB_OK) return KVB_ECUDA;
    return launch_pdl(kvb::prefill_dkv_sum_kernel<D, BETA>, dim3(grid, 2 * D / 16), dim3(256), 0, st, p);
}

template <int D>
kvb_status bwd_dispatch(const kvb::PrefillParams& p, cudaStream_t st) {
    const bool beta = p.lb != nullptr, cap = p.softcap > 0.f;
    if (beta) return cap ? launch_bwd<D, true, true>(p, st) : launch_bwd<D, true, false>(p, st);
    return cap ? launch_bwd<D, false, true>(p, st) : launch_bwd<D, false, false>(p, st);
}

}  // namespace

extern "C" {

kvb_status kvb_test_withhold_next_prefill(int32_t kernel, int32_t cta, uint64_t wait_limit_ns) {
    if (kernel < 0 || kernel > 2 || cta < 0 || cta > 65535 || wait_limit_ns < 1000ull || wait_limit_ns > 1000000000ull) return KVB_EINVAL;
    g_withhold_prefill.store(wait_limit_ns | (unsigned long long)kernel << 32 | (unsigned long long)(cta + 1) << 40);
    return KVB_OK;
}

kvb_status kvb_prefill_attn(const kvb_prefill_args* a, kvb_stream stream) {
    kvb::PrefillParams p;
    if (prefill_params(a, &p) != KVB_OK) return KVB_EINVAL;
    if (p.T == 0 || p.N == 0) return KVB_OK;
    take_withheld(0, &p);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return a->d == 128 ? fwd_dispatch<128>(p, st) : fwd_dispatch<64>(p, st);
}

size_t kvb_prefill_attn_bwd_workspace_bytes(int32_t T, int32_t Hq) {
    if (T < 1 || Hq < 1) return 0;
    return round256((size_t)T * Hq * sizeof(float)) + (size_t)kvb::kMaxPieces * (2 * kvb::kPartFloats * sizeof(float) + sizeof(int4) + sizeof(int));
}

kvb_status kvb_prefill_attn_bwd(const kvb_prefill_args* a, const kvb_prefill_grads* g, kvb_stream stream) {
    kvb::PrefillParams p;
    if (g == nullptr || prefill_params(a, &p) != KVB_OK) return KVB_EINVAL;
    if (!a->lse || !g->d_o || !g->dq || !g->dk || !g->dv || (g->d_log_beta != nullptr) != (a->log_beta != nullptr)) return KVB_EINVAL;
    if (!aligned16(g->d_o) || !aligned16(g->dq) || !aligned16(g->dk) || !aligned16(g->dv)) return KVB_EINVAL;
    if (!aligned4(g->d_lse) || !aligned4(g->d_log_beta)) return KVB_EINVAL;
    if (p.T == 0 || p.N == 0) return KVB_OK;
    if (!g->workspace || !aligned16(g->workspace) ||
        g->workspace_bytes < kvb_prefill_attn_bwd_workspace_bytes(a->T, a->Hq))
        return KVB_EINVAL;
    p.d_o = g->d_o; p.d_lse = g->d_lse; p.dq = g->dq; p.dk = g->dk; p.dv = g->dv; p.dlb = g->d_log_beta;
    p.delta = static_cast<float*>(g->workspace);
    p.parts = p.delta + round256((size_t)a->T * a->Hq * sizeof(float)) / sizeof(float);
    p.records = reinterpret_cast<int4*>(p.parts + (size_t)kvb::kMaxPieces * 2 * kvb::kPartFloats);
    p.dq_done = reinterpret_cast<int*>(p.records + kvb::kMaxPieces);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return a->d == 128 ? bwd_dispatch<128>(p, st) : bwd_dispatch<64>(p, st);
}

size_t kvb_paged_plan_workspace_bytes(int32_t B, int32_t Hkv) {
    return B < 1 || Hkv < 1 ? 0 : ((size_t)B * Hkv + 1) * sizeof(int4);
}

kvb_status kvb_paged_plan(const kvb_paged_cache* c, const int32_t* cu, int32_t T, int32_t* slot_map, int32_t empty_only,
                          void* workspace, size_t workspace_bytes, kvb_stream stream) {
    return kvb_paged_plan_within(c, cu, T, slot_map, empty_only, INT32_MAX, workspace, workspace_bytes, stream);
}

kvb_status kvb_paged_plan_within(const kvb_paged_cache* c, const int32_t* cu, int32_t T, int32_t* slot_map,
                                 int32_t empty_only, int32_t max_len, void* workspace, size_t workspace_bytes,
                                 kvb_stream stream) {
    kvb::PagedCache pc;
    if (paged_view(c, &pc) != KVB_OK) return KVB_EINVAL;
    if (max_len < 1 || T < 0 || T > (1 << 30) || !cu || !aligned4(cu) || (T > 0 && !slot_map) || !aligned4(slot_map)) return KVB_EINVAL;
    if (!workspace || !aligned16(workspace) || workspace_bytes < kvb_paged_plan_workspace_bytes(c->B, c->Hkv)) return KVB_EINVAL;
    kvb::PagedPlanParams p{pc, cu, slot_map, c->B, T, empty_only, max_len, static_cast<int4*>(workspace)};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    // few slots: the second launch costs more than it spreads (200 tokens, 2 heads: 7.2 -> 6.2 us with the caller's
    // two copies; 131072 tokens, 8 heads need it)
    if ((long long)T * c->Hkv <= 4096)
        return launch_pdl(kvb::paged_plan_kernel<1024, true>, dim3(1), dim3(1024), 0, st, p);
    if (launch_pdl(kvb::paged_plan_kernel<1024, false>, dim3(1), dim3(1024), 0, st, p) != KVB_OK) return KVB_ECUDA;
    // a block for every 1024 tokens of a row's share (256 tokens: 16.7 us instead of 13 for 131072 tokens in 256 rows)
    const long long share = ((long long)T / c->B + 1023) / 1024;
    const unsigned parts = (unsigned)std::min<long long>(std::max<long long>(share, 1), 64);
    return launch_pdl(kvb::paged_slots_kernel<256>, dim3(c->B * c->Hkv, parts), dim3(256), 0, st, p);
}

kvb_status kvb_paged_write(const kvb_paged_cache* c, const uint16_t* k, const uint16_t* v, int64_t kv_stride_t,
                           int64_t kv_stride_h, const float* log_beta, int64_t lb_stride_t, int64_t lb_stride_h,
                           const int32_t* pos, const int32_t* slot_map, int32_t T, kvb_stream stream) {
    kvb::PagedCache pc;
    if (paged_view(c, &pc) != KVB_OK) return KVB_EINVAL;
    if (T < 0 || T > (1 << 30)) return KVB_EINVAL;
    if (T == 0) return KVB_OK;
    if (!k || !v || !pos || !slot_map || !aligned16(k) || !aligned16(v) || !aligned4(pos) || !aligned4(slot_map)) return KVB_EINVAL;
    if ((c->log_beta_pages != nullptr) != (log_beta != nullptr) || !aligned4(log_beta)) return KVB_EINVAL;
    if (c->Hkv > 65535) return KVB_EINVAL;
    if (kv_stride_t < 0 || kv_stride_h < 0 || kv_stride_t % 8 || kv_stride_h % 8 || lb_stride_t < 0 || lb_stride_h < 0)
        return KVB_EINVAL;
    kvb::PagedWriteParams p{pc, k, v, log_beta, pos, slot_map, kv_stride_t, kv_stride_h, lb_stride_t, lb_stride_h, T};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int groups = 256 / (c->d / 8);
    const long long blocks = ((long long)T + groups - 1) / groups * c->Hkv;
    if (blocks > 0x7fffffffLL) return KVB_EINVAL;
    return launch_pdl(kvb::paged_write_kernel, dim3((unsigned)blocks), dim3(256), 0, st, p);
}

}  // extern "C"
