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
    int most;            // slots that a sequence may hold with its new tokens
    int4* rec;           // workspace [B * Hkv + 1]: old length, new tokens, pages taken by the rows ahead,
                         // served; the last one: the free stack's height before the call, cu in order
};

__device__ __forceinline__ int pages_of(int slots) { return (slots + kPageSlots - 1) / kPageSlots; }

// Table entries of the new pages and the slots of the new tokens of a (sequence, kv head), by threads part,
// part + parts, ... A token's page is read where it stands before the call (the free stack or the table), so
// nothing waits for these writes themselves.
__device__ __forceinline__ void paged_row_slots(const PagedPlanParams& p, int bg, int part, int parts) {
    const PagedCache& c = p.c;
    const int b = bg / c.Hkv, g = bg % c.Hkv;
    const int4 call = p.rec[(size_t)p.B * c.Hkv], r = p.rec[bg];
    const int fresh = r.y;
    int* map = p.slot_map + (size_t)g * p.T + p.cu[b];
    if (!r.w) {
        for (int i = part; i < fresh; i += parts) map[i] = -1;
        return;
    }
    int* table = c.table + (size_t)bg * c.max_pages;
    const int old_pages = pages_of(r.x), new_pages = pages_of(r.x + fresh);
    const int* stack = c.free_pages + call.x - 1 - r.z;   // the first new page; the others lie below it
    for (int j = old_pages + part; j < new_pages; j += parts) table[j] = stack[old_pages - j];
#pragma unroll 4
    for (int i = part; i < fresh; i += parts) {
        const int slot = r.x + i, j = slot / kPageSlots;
        const int pg = j < old_pages ? table[j] : stack[old_pages - j];
        int row = -1;
        if (pg >= 0 && pg < c.num_pages)
            row = pg * kPageSlots + slot % kPageSlots;
        else
            raise_error(KVB_DERR_RANGE);
        map[i] = row;
    }
}

// cu out of order: no token gets a slot
__device__ __forceinline__ void paged_no_slots(const PagedPlanParams& p, long long at, long long threads) {
    for (long long i = at; i < (long long)p.c.Hkv * p.T; i += threads) p.slot_map[i] = -1;
}

// Pages and records of every (sequence, kv head), in order: one CTA, a running sum over the
// sequences, NT at a time (thread = sequence). A sequence is served when the pages of all
// sequences up to it fit the free stack, or when it needs none; the pages come off the top of the
// stack in the order (sequence, kv head, page). Bound by latency: the lengths load eight heads at a time.
// With SLOTS the CTA goes on to the slots itself, a warp per row (few tokens: the second launch would cost
// more than it spreads).
template <int NT, bool SLOTS>
__global__ void __launch_bounds__(NT) paged_plan_kernel(const __grid_constant__ PagedPlanParams p) {
    __shared__ int s_warp[NT / 32];
    __shared__ int s_taken;
    griddep_wait();
    griddep_launch_dependents();
    const PagedCache& c = p.c;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int cap = c.max_pages * kPageSlots, most = min(cap, p.most);
    const int avail = min(max(*c.free_count, 0), c.num_pages);
    const size_t rows = (size_t)p.B * c.Hkv;
    bool bad = false;
    for (int b = tid; b < p.B; b += NT) {
        const int s = p.cu[b], e = p.cu[b + 1];
        bad |= s < 0 || e < s || e > p.T;
    }
    bad = __syncthreads_or(bad);
    if (tid == 0) {
        if (bad) raise_error(KVB_DERR_RANGE);
        p.rec[rows] = make_int4(avail, !bad, 0, 0);
        s_taken = 0;
    }
    if (bad) {
        if (SLOTS) paged_no_slots(p, tid, NT);
        return;
    }
    int ahead = 0;   // pages wanted by the sequences of the earlier rounds
    for (int b0 = 0; b0 < p.B; b0 += NT) {
        const int b = b0 + tid;
        int need = 0, fresh = 0, n[8];
        bool ok = b < p.B;
        const int* len = c.len + (size_t)b * c.Hkv;
        if (ok) {
            fresh = p.cu[b + 1] - p.cu[b];
            for (int g0 = 0; g0 < c.Hkv; g0 += 8) {
#pragma unroll
                for (int g = 0; g < 8; ++g) n[g] = g0 + g < c.Hkv ? len[g0 + g] : 0;
#pragma unroll
                for (int g = 0; g < 8; ++g) {
                    if (g0 + g >= c.Hkv) continue;
                    ok = ok && n[g] >= 0 && n[g] <= cap && (fresh == 0 || (fresh <= most - n[g] && !(p.empty_only && n[g] > 0)));
                    if (ok) need = min(need + pages_of(n[g] + fresh) - pages_of(n[g]), 1 << 30);
                }
            }
            if (!ok) {
                raise_error(KVB_DERR_LEN);
                need = 0;
            }
        }
        // sums saturate at 2^30 (a batch that wants more pages than that has more than any pool)
        int upto = need;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int x = __shfl_up_sync(kFull, upto, d);
            if (lane >= d) upto = min(upto + x, 1 << 30);
        }
        if (lane == 31) s_warp[warp] = upto;
        __syncthreads();
        int before = lane < NT / 32 ? s_warp[lane] : 0;   // every warp scans the warps' sums
        static_assert(NT == 1024, "a lane per warp");
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int x = __shfl_up_sync(kFull, before, d);
            if (lane >= d) before = min(before + x, 1 << 30);
        }
        const int total = __shfl_sync(kFull, before, 31), mine = __shfl_sync(kFull, before, max(warp - 1, 0));
        upto = min(upto + (warp > 0 ? mine : 0), 1 << 30);
        upto = min(upto + ahead, 1 << 30);
        ahead = min(ahead + total, 1 << 30);
        const bool served = ok && (need == 0 || upto <= avail);
        if (ok && !served) raise_error(KVB_DERR_PAGES);
        if (b < p.B) {
            int first = upto - need;
            for (int g0 = 0; g0 < c.Hkv; g0 += 8) {
                if (c.Hkv > 8) {
#pragma unroll
                    for (int g = 0; g < 8; ++g) n[g] = g0 + g < c.Hkv ? len[g0 + g] : 0;
                }
#pragma unroll
                for (int g = 0; g < 8; ++g) {
                    if (g0 + g >= c.Hkv) continue;
                    const size_t bg = (size_t)b * c.Hkv + g0 + g;
                    p.rec[bg] = make_int4(n[g], fresh, first, served);
                    if (served) {
                        first += pages_of(n[g] + fresh) - pages_of(n[g]);
                        c.len[bg] = n[g] + fresh;
                    }
                }
            }
            if (served && need > 0) atomicMax(&s_taken, upto);
        }
        __syncthreads();
    }
    if (tid == 0) *c.free_count = avail - s_taken;
    if (SLOTS)
        for (size_t bg = warp; bg < rows; bg += NT / 32) paged_row_slots(p, (int)bg, lane, 32);
}

// The slots as a launch of their own: blockIdx.x = (sequence, kv head), blockIdx.y strides over its tokens.
template <int NT>
__global__ void __launch_bounds__(NT) paged_slots_kernel(const __grid_constant__ PagedPlanParams p) {
    const int part = blockIdx.y * NT + threadIdx.x, parts = gridDim.y * NT;
    griddep_wait();
    griddep_launch_dependents();
    if (p.rec[(size_t)p.B * p.c.Hkv].y) {
        paged_row_slots(p, blockIdx.x, part, parts);
    } else {
        paged_no_slots(p, (long long)blockIdx.x * parts + part, (long long)gridDim.x * parts);
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

// A block copies the rows of one kv head and 256 / (d / 8) tokens (d / 8 threads move a row of K and of V, 16
// bytes each), and a thread per token writes pos and log beta, so that those writes fill sectors too; blocks
// of the same tokens and other heads are neighbours. Bound by memory: nothing is read twice, and loads and
// stores stream past the cache. 32768 tokens, 8 heads, d 128 (272.6 MB): 43.3 us, 6.3 TB/s (54 us with
// plain stores and 4-byte writes from the rows' first threads; more rows a thread change nothing).
__global__ void __launch_bounds__(256) paged_write_kernel(const __grid_constant__ PagedWriteParams p) {
    const PagedCache& c = p.c;
    const int per = c.d / 8, groups = 256 / per, tid = threadIdx.x;
    const int group = tid / per, e = tid % per;
    const int g = blockIdx.x % c.Hkv, t0 = blockIdx.x / c.Hkv * groups;
    griddep_wait();
    griddep_launch_dependents();
    const int rows = c.num_pages * kPageSlots;
    const int* map = p.slot_map + (size_t)g * p.T;
    int row = -1;
    uint4 kk, vv;
    if (group < groups && t0 + group < p.T) {   // the rows load while their slots do
        row = map[t0 + group];
        const long long src = (long long)(t0 + group) * p.kv_st + (long long)g * p.kv_sh + 8 * e;
        kk = __ldcs(reinterpret_cast<const uint4*>(p.k + src));
        vv = __ldcs(reinterpret_cast<const uint4*>(p.v + src));
    }
    if (tid < groups && t0 + tid < p.T) {
        const int t = t0 + tid, r = map[t];
        if (r >= rows) {
            raise_error(KVB_DERR_RANGE);
        } else if (r >= 0) {
            c.pos[r] = p.pos[t];
            if (c.lb != nullptr) c.lb[r] = p.lb[(long long)t * p.lb_st + (long long)g * p.lb_sh];
        }
    }
    if (row < 0 || row >= rows) return;
    const size_t dst = (size_t)row * c.d + 8 * e;
    __stcs(reinterpret_cast<uint4*>(c.k + dst), kk);
    __stcs(reinterpret_cast<uint4*>(c.v + dst), vv);
}

}  // namespace kvb
