// Filling a paged cache with the tokens of whole prompts: pages and slots of the new tokens from
// the lengths (kvb_paged_plan), and the copy of their rows into the pages (kvb_paged_write). The
// counterpart, for many tokens at once, of the append of paged_evict_insert_kernel.
#pragma once

#include "paged_view.cuh"

namespace kvb {

struct PagedPlanParams {
    PagedCache c;
    const int* cu;       // [B + 1]
    int* slot_map;       // [Hkv, T]
    int B, T, empty_only;
    int4* rec;           // workspace [B * Hkv + 1]: old length, new tokens, pages taken by the rows ahead,
                         // served; the last one: the free stack's height before the call, cu in order
};

// Pages and records of every (sequence, kv head), in order: one CTA, a running sum over the
// sequences, NT at a time (thread = sequence). A sequence is served when the pages of all
// sequences up to it fit the free stack, or when it needs none; the pages come off the top of the
// stack in the order (sequence, kv head, page).
template <int NT>
__global__ void __launch_bounds__(NT) paged_plan_kernel(const __grid_constant__ PagedPlanParams p) {
    __shared__ int s_warp[NT / 32];
    __shared__ int s_taken;
    griddep_wait();
    griddep_launch_dependents();
    const PagedCache& c = p.c;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int cap = c.max_pages * kPageSlots;
    const int avail = min(max(*c.free_count, 0), c.num_pages);
    const size_t rows = (size_t)p.B * c.Hkv;
    bool bad = false;
    for (int b = tid; b < p.B; b += NT) bad |= p.cu[b] < 0 || p.cu[b + 1] < p.cu[b] || p.cu[b + 1] > p.T;
    bad = __syncthreads_or(bad);
    if (tid == 0) {
        if (bad) raise_error(KVB_DERR_RANGE);
        p.rec[rows] = make_int4(avail, !bad, 0, 0);
        s_taken = 0;
    }
    if (bad) return;
    int ahead = 0;   // pages wanted by the sequences of the earlier rounds
    for (int b0 = 0; b0 < p.B; b0 += NT) {
        const int b = b0 + tid;
        int need = 0, fresh = 0;
        bool ok = b < p.B;
        if (ok) {
            fresh = p.cu[b + 1] - p.cu[b];
            for (int g = 0; g < c.Hkv; ++g) {
                const int n = c.len[(size_t)b * c.Hkv + g];
                if (n < 0 || n > cap || fresh > cap - n || (p.empty_only && n > 0 && fresh > 0)) {
                    ok = false;
                    break;
                }
                need += (n + fresh + kPageSlots - 1) / kPageSlots - (n + kPageSlots - 1) / kPageSlots;
            }
            if (!ok) {
                raise_error(KVB_DERR_LEN);
                need = 0;
            }
        }
        // sums saturate at 2^30 (a batch that wants more pages than that has more than any pool)
        int upto = min(need, 1 << 30);
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int x = __shfl_up_sync(kFull, upto, d);
            if (lane >= d) upto = min(upto + x, 1 << 30);
        }
        if (lane == 31) s_warp[warp] = upto;
        __syncthreads();
        int total = ahead;
        for (int w = 0; w < NT / 32; ++w) {
            if (w == warp) upto = min(upto + total, 1 << 30);
            total = min(total + s_warp[w], 1 << 30);
        }
        ahead = total;
        const bool served = ok && (need == 0 || upto <= avail);
        if (ok && !served) raise_error(KVB_DERR_PAGES);
        if (b < p.B) {
            int first = upto - need;
            for (int g = 0; g < c.Hkv; ++g) {
                const size_t bg = (size_t)b * c.Hkv + g;
                const int n = c.len[bg];
                p.rec[bg] = make_int4(n, fresh, first, served);
                if (served) {
                    first += (n + fresh + kPageSlots - 1) / kPageSlots - (n + kPageSlots - 1) / kPageSlots;
                    c.len[bg] = n + fresh;
                }
            }
            if (served && need > 0) atomicMax(&s_taken, upto);
        }
        __syncthreads();
    }
    if (tid == 0) *c.free_count = avail - s_taken;
}

// Table entries of the new pages and the slots of the new tokens: a CTA per (sequence, kv head).
template <int NT>
__global__ void __launch_bounds__(NT) paged_slots_kernel(const __grid_constant__ PagedPlanParams p) {
    griddep_wait();
    const PagedCache& c = p.c;
    const int bg = blockIdx.x, b = bg / c.Hkv, g = bg % c.Hkv;
    const int4 call = p.rec[(size_t)p.B * c.Hkv];
    if (!call.y) {   // cu out of order: no token gets a slot
        for (long long i = (long long)bg * NT + threadIdx.x; i < (long long)c.Hkv * p.T; i += (long long)gridDim.x * NT)
            p.slot_map[i] = -1;
        return;
    }
    const int4 r = p.rec[bg];
    const int fresh = r.y;
    int* map = p.slot_map + (size_t)g * p.T + p.cu[b];
    if (!r.w) {
        for (int i = threadIdx.x; i < fresh; i += NT) map[i] = -1;
        return;
    }
    int* table = c.table + (size_t)bg * c.max_pages;
    const int old_pages = (r.x + kPageSlots - 1) / kPageSlots;
    const int new_pages = (r.x + fresh + kPageSlots - 1) / kPageSlots;
    const int top = call.x - 1 - r.z;   // the stack's entry of the first new page
    for (int j = old_pages + threadIdx.x; j < new_pages; j += NT) table[j] = c.free_pages[top - (j - old_pages)];
    __syncthreads();
    for (int i = threadIdx.x; i < fresh; i += NT) {
        const int slot = r.x + i, pg = table[slot / kPageSlots];
        int row = -1;
        if (pg >= 0 && pg < c.num_pages)
            row = pg * kPageSlots + slot % kPageSlots;
        else
            raise_error(KVB_DERR_RANGE);
        map[i] = row;
    }
}

struct PagedWriteParams {
    PagedCache c;
    const uint16_t* k;
    const uint16_t* v;
    const float* lb;
    const int* pos;        // [T]
    const int* slot_map;   // [Hkv, T]
    long long kv_st, kv_sh, lb_st, lb_sh;
    int T;
};

// One group of d / 8 threads per (token, kv head): 16 bytes of K and of V per thread.
__global__ void __launch_bounds__(256) paged_write_kernel(const __grid_constant__ PagedWriteParams p) {
    griddep_wait();
    const PagedCache& c = p.c;
    const int per = c.d / 8;
    const long long n = (long long)p.T * c.Hkv * per;
    for (long long x = (long long)blockIdx.x * blockDim.x + threadIdx.x; x < n; x += (long long)gridDim.x * blockDim.x) {
        const int e = (int)(x % per);
        const long long th = x / per;
        const int g = (int)(th % c.Hkv), t = (int)(th / c.Hkv);
        const int row = p.slot_map[(size_t)g * p.T + t];
        if (row < 0) continue;
        if (row >= c.num_pages * kPageSlots) {
            raise_error(KVB_DERR_RANGE);
            continue;
        }
        const long long src = (long long)t * p.kv_st + g * p.kv_sh + 8 * e;
        const size_t dst = (size_t)row * c.d + 8 * e;
        *reinterpret_cast<uint4*>(c.k + dst) = *reinterpret_cast<const uint4*>(p.k + src);
        *reinterpret_cast<uint4*>(c.v + dst) = *reinterpret_cast<const uint4*>(p.v + src);
        if (e == 0) {
            c.pos[row] = p.pos[t];
            if (c.lb != nullptr) c.lb[row] = p.lb[(long long)t * p.lb_st + g * p.lb_sh];
        }
    }
}

}  // namespace kvb
