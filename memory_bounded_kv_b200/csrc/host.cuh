// Host-side helpers of the C ABI's translation units: argument checks, tensor-map encoding, launches.
#pragma once

#include <cuda.h>

#include <cstdint>
#include <map>
#include <mutex>
#include <tuple>
#include <utility>

#include "../../include/kvb.h"
#include "paged_view.cuh"

// The error word of prefill.cu's kernels (every translation unit has one): ORed into *bits and cleared.
__attribute__((visibility("hidden"))) kvb_status kvb_prefill_take_error(unsigned* bits);

namespace {

// This translation unit's device error word: ORed into *bits and cleared.
inline kvb_status take_error_word(unsigned* bits) {
    unsigned w = 0;
    if (cudaMemcpyFromSymbol(&w, kvb::g_error_word, sizeof w) != cudaSuccess) return KVB_ECUDA;
    *bits |= w;
    if (w == 0) return KVB_OK;
    const unsigned zero = 0;
    return cudaMemcpyToSymbol(kvb::g_error_word, &zero, sizeof zero) == cudaSuccess ? KVB_OK : KVB_ECUDA;
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline kvb_status launched() { return cudaGetLastError() == cudaSuccess ? KVB_OK : KVB_ECUDA; }

// Raises a kernel's dynamic shared-memory limit once per (kernel, device):
// later calls (e.g. inside a stream capture) make no runtime call here.
template <typename Kern>
kvb_status set_smem(Kern kern, size_t bytes) {
    if (bytes <= 48 * 1024) return KVB_OK;
    static std::mutex mu;
    static std::map<std::pair<const void*, int>, size_t> granted;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return KVB_ECUDA;
    std::lock_guard<std::mutex> lock(mu);
    size_t& g = granted[{reinterpret_cast<const void*>(kern), dev}];
    if (g >= bytes) return KVB_OK;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) != cudaSuccess)
        return KVB_ECUDA;
    g = bytes;
    return KVB_OK;
}

// ---- tensor maps (driver entry point, no link against libcuda) -------------------
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_tiled() {
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(f);
    });
    return fn;
}

// Resident CTAs the device holds for a kernel (SMs x blocks per SM), once per (kernel, smem, device).
template <typename Kern>
int resident_ctas(Kern kern, int threads, size_t smem) {
    static std::mutex mu;
    static std::map<std::tuple<const void*, size_t, int>, int> cache;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    std::lock_guard<std::mutex> lock(mu);
    auto key = std::make_tuple(reinterpret_cast<const void*>(kern), smem, dev);
    auto it = cache.find(key);
    if (it != cache.end()) return it->second;
    int sms = 0, per_sm = 0;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, threads, smem) != cudaSuccess) return 0;
    const int n = sms * (per_sm > 0 ? per_sm : 1);
    cache[key] = n;
    return n;
}

// Launch with programmatic stream serialization: the kernel may start while the
// previous kernel in the stream drains; its first instruction waits for that
// kernel's completion (griddepcontrol.wait), so only the launch latency overlaps.
template <typename... KArgs, typename... Args>
kvb_status launch_pdl(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t st,
                      Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, args...) == cudaSuccess ? KVB_OK : KVB_ECUDA;
}

// Host checks shared by the paged entry points; fills the kernels' view of the cache.
kvb_status paged_view(const kvb_paged_cache* c, kvb::PagedCache* out) {
    if (c == nullptr) return KVB_EINVAL;
    if (c->B < 1 || c->Hkv < 1 || c->d < 8 || c->d > 1024 || (c->d % 8) || c->max_pages < 1 || c->num_pages < 1)
        return KVB_EINVAL;
    if ((long long)c->B * c->Hkv > 0x7fffffffLL || (long long)c->max_pages * kvb::kPageSlots > 0x7fffffffLL ||
        (long long)c->num_pages * kvb::kPageSlots > 0x7fffffffLL)
        return KVB_EINVAL;
    if (!c->k_pages || !c->v_pages || !c->pos_pages || !c->table || !c->len || !c->free_pages || !c->free_count)
        return KVB_EINVAL;
    if (!aligned16(c->k_pages) || !aligned16(c->v_pages) || !aligned16(c->pos_pages) ||
        (c->log_beta_pages && !aligned16(c->log_beta_pages)))
        return KVB_EINVAL;
    *out = kvb::PagedCache{c->k_pages, c->v_pages, c->log_beta_pages, c->pos_pages, c->table, c->len,
                           c->free_pages, c->free_count, c->Hkv, c->d, c->max_pages, c->num_pages};
    return KVB_OK;
}

}  // namespace
