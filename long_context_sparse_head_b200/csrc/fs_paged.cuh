// The paged key-value cache: what its kernels share (fs_paged_append.cu, fs_paged_attend.cu,
// fs_pages.cu).
#pragma once

#include "fs_rotary.cuh"

namespace fs {

// Kernel-side copy of the parameters (passed by value).
struct PagedDev {
    int B, H, Hkv, d, ps, num_pages, max_pages;
    int cap;                           // tokens a table row holds: max_pages * page_size
    unsigned magic;                    // floor(2^32 / page_size), capped at 2^32 - 1
    long long sp, sh, st;              // strides of the pools: page, head, token (elements)

    // token position -> index into the table row, slot within the page.  pos < 2^30, so the
    // product falls short of pos / ps by less than 1/4 + the fraction: at most one too low.
    __host__ __device__ __forceinline__ void locate(int pos, int &idx, int &slot) const {
        unsigned q = (unsigned)((unsigned long long)(unsigned)pos * magic >> 32);
        unsigned r = (unsigned)pos - q * (unsigned)ps;
        if (r >= (unsigned)ps) {
            q++;
            r -= (unsigned)ps;
        }
        idx = (int)q;
        slot = (int)r;
    }
    __host__ __device__ __forceinline__ int pages_of(int tokens) const {
        int q, r;
        locate(tokens, q, r);
        return q + (r != 0);
    }
    __device__ __forceinline__ bool page_ok(int page) const { return (unsigned)page < (unsigned)num_pages; }
};

// Workspace: the error flag, the split rows' arrival counters (zero between calls: the last
// arrival resets its own), then one area that attention uses for partial results and the page
// calls for their lists.  Flag and counters lie at the same place whatever the parameters, so
// a workspace made for the largest batch serves smaller ones.
constexpr size_t kPagedCounters = 256;
constexpr int kPagedCounts = 1536;
constexpr size_t kPagedArea = kPagedCounters + 4 * (size_t)kPagedCounts;

size_t attend_area_bytes(const fs_paged_params *p);
size_t pages_area_bytes(const fs_paged_params *p);

// Checks the parameters and, if `out`, fills the kernel-side copy.
fs_status paged_dev(const fs_paged_params *p, PagedDev *out);
// The same, with the workspace.
fs_status paged_call(const fs_paged_params *p, PagedDev *out, const void *ws, size_t ws_bytes);

__device__ __forceinline__ void raise_check(int *flag) { atomicExch(flag, kFlagCheck); }

}  // namespace fs
