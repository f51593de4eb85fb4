// Management of the paged cache's pages (fs_pages_reserve, _copy, _fork, _free, _compact) and
// the parameter checks of all its calls.
//
// refs is the one record of what is free (refs[page] == 0), and the lowest free pages are taken
// in a stated order, so the result of every call is a function of its inputs: no free list to
// fall out of step with the tables, no atomics whose order shows.
//
// What has to look at all pages (the search for free ones, the packing plan) runs in one cluster:
// a CTA of 512 threads reads 2048 refs a step, one step ahead, and counts them by a block-wide
// prefix sum; eight such CTAs, where there are more pages than that, exchange their counts
// through shared memory.  The search ends with the last page that is wanted.  It is bound by a
// step's latency (load, barriers): the packing plan of 16384 pages takes 7.9 us, in one CTA of 1024 threads 14.4.
// What moves data runs on the whole GPU: a warp copies 4 KB at a time, its eight 16-byte
// loads a lane all in flight before the first store; HBM bounds it.
#include <algorithm>

#include "fs_paged.cuh"
#include "tc_common.cuh"

namespace fs {
namespace {

constexpr int kMaxPages = 2000000;             // kPlanThreads times as many fit an int
constexpr int kPlanThreads = 512, kPerThread = 4, kPlanStep = kPlanThreads * kPerThread;
constexpr int kFreeThreads = 1024;
constexpr int kCopyThreads = 256, kCopyAhead = 8, kSlab = 32 * kCopyAhead;     // vectors a warp copies at once

// ---- lists in the workspace's area, in ints
enum : int { kOk = 0, kMoves = 1, kLive = 2, kHead = 16 };

// Inclusive sum over the block of kPlanThreads; `total` receives the sum.  s: 32 shared ints.
__device__ __forceinline__ int block_scan(int v, int *s, int &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(kFull, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();                           // s is free again
    if (lane == 31) s[warp] = x;
    __syncthreads();
    if (warp == 0) {
        int w = lane < kPlanThreads / 32 ? s[lane] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(kFull, w, o);
            if (lane >= o) w += y;
        }
        s[lane] = w;
    }
    __syncthreads();
    total = s[31];
    return x + (warp ? s[warp - 1] : 0);
}

// The CTAs of the cluster exchange a number: the sum of those before this one, and of all.
// Called by every thread of every CTA, `v` the same in a CTA.  slot: shared ints, two by turns.
struct Cluster {
    int rank, size, turn;
    __device__ __forceinline__ Cluster() : turn(0) {
        asm("mov.u32 %0, %cluster_ctarank;" : "=r"(rank));
        asm("mov.u32 %0, %cluster_nctarank;" : "=r"(size));
    }
    __device__ __forceinline__ void exchange(int v, int *slot, int &before, int &all) {
        before = 0;
        all = v;
        if (size == 1) {
            __syncthreads();
            return;
        }
        int *mine = slot + turn;
        turn ^= 1;                             // a slow reader of this one is past it when it comes round again
        if (threadIdx.x == 0) *mine = v;
        tc::cluster_sync();
        all = 0;
        for (int r = 0; r < size; r++) {
            int x;
            const uint32_t from = tc::cluster_map(tc::smem_u32(mine), r);
            asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(x) : "r"(from) : "memory");
            if (r < rank) before += x;
            all += x;
        }
    }
    // also keeps a CTA's shared memory until all have read it
    __device__ __forceinline__ void sync() const {
        if (size == 1) __syncthreads();
        else tc::cluster_sync();
    }
};

// refs of the pages first .. first + 3; pages past the last read as in use
__device__ __forceinline__ void load_refs(const int32_t *refs, int first, int n, int (&r)[kPerThread]) {
    if (first + kPerThread <= n) {
#pragma unroll
        for (int i = 0; i < kPerThread / 4; i++) {
            const int4 v = *reinterpret_cast<const int4 *>(refs + first + 4 * i);
            r[4 * i] = v.x; r[4 * i + 1] = v.y; r[4 * i + 2] = v.z; r[4 * i + 3] = v.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < kPerThread; i++) r[i] = first + i < n ? refs[first + i] : 1;
    }
}

// The `want` lowest free pages, ascending, to list; returns how many there are (at most want).
// The list is complete for every CTA.
__device__ int find_free(const int32_t *refs, int n, int want, int *list, int *s, int *slot, Cluster &cl) {
    int found = 0;
    int next[kPerThread];
    const int mine = (cl.rank * kPlanThreads + (int)threadIdx.x) * kPerThread, step = cl.size * kPlanStep;
    load_refs(refs, min(mine, n), n, next);
    for (int base = 0; base < n && found < want; base += step) {
        int r[kPerThread], k = 0, total, before, all;
#pragma unroll
        for (int i = 0; i < kPerThread; i++) {
            r[i] = next[i];
            k += r[i] == 0;
        }
        if (base + step < n) load_refs(refs, min(base + step + mine, n), n, next);
        const int incl = block_scan(k, s, total);
        cl.exchange(total, slot, before, all);
        int at = found + before + incl - k;
#pragma unroll
        for (int i = 0; i < kPerThread; i++)
            if (r[i] == 0 && at < want) list[at++] = base + mine + i;
        found += all;
    }
    cl.sync();
    return min(found, want);
}

// n_new[b] more tokens for every sequence.
__global__ void __launch_bounds__(kPlanThreads) reserve_kernel(const __grid_constant__ PagedDev P,
                                                               const int32_t *n_new, int32_t *refs, int32_t *table,
                                                               int32_t *lens, int *area, int *flag) {
    __shared__ int s[32], slot[2];
    Cluster cl;
    griddep_wait();
    int *offs = area + kHead, *list = offs + P.B + 1;
    const int tid = threadIdx.x;
    // the first CTA sums the pages that the sequences before each one need
    bool bad = false;
    long long sum = 0;
    if (cl.rank == 0) {
        for (int base = 0; base < P.B; base += kPlanThreads) {
            const int b = base + tid;
            int need = 0, total;
            if (b < P.B) {
                const int n = n_new[b], len = lens[b];
                if (n < 0 || len < 0 || (long long)len + n > P.cap) bad = true;
                else need = P.pages_of(len + n) - P.pages_of(len);
            }
            need = min(need, P.num_pages + 1); // more than there are; a block's sum fits an int
            const int before = block_scan(need, s, total) - need;
            if (b < P.B) offs[b] = (int)min(sum + before, 0x7fffffffll);
            sum += total;
        }
        bad |= sum > P.num_pages;
        bad = __syncthreads_or(bad);
    }
    int before, want;
    cl.exchange(bad ? -1 : (int)sum, slot, before, want);      // the others add 0
    if (want > 0 && find_free(refs, P.num_pages, want, list, s, slot, cl) < want) want = -1;
    if (want < 0) {
        if (cl.rank == 0 && tid == 0) raise_check(flag);
    } else {
        for (int i = cl.rank * kPlanThreads + tid; i < want; i += cl.size * kPlanThreads) {
            int lo = 0, hi = P.B;              // the last b with offs[b] <= i
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (__ldcg(offs + mid) <= i) lo = mid;
                else hi = mid;
            }
            const int page = __ldcg(list + i);
            table[(long long)lo * P.max_pages + P.pages_of(lens[lo]) + (i - __ldcg(offs + lo))] = page;
            refs[page] = 1;
        }
    }
    cl.sync();                                 // lens has been read
    if (want >= 0 && cl.rank == 0)
        for (int b = tid; b < P.B; b += kPlanThreads) lens[b] += n_new[b];
}

// A page's elements in 16-byte vectors: `outer` x `inner` runs of `run` vectors.
struct PageShape {
    int run, inner, vecs;                      // vectors of a run, runs of an outer step, vectors of a page
    long long so, si;                          // strides of the steps, in vectors
    long long sp;                              // stride of a page
    __device__ __forceinline__ long long at(int x) const {
        if (run == vecs) return x;
        const int k = x / run, o = k / inner;
        return o * so + (k - o * inner) * si + (x - k * run);
    }
};

// One slab of a page: all loads before the first store.
__device__ __forceinline__ void copy_slab(const PageShape &G, uint4 *pool, int src, int dst, int slab, int lane) {
    const uint4 *from = pool + src * G.sp;
    uint4 *to = pool + dst * G.sp;
    uint4 v[kCopyAhead];
    long long at[kCopyAhead];
#pragma unroll
    for (int j = 0; j < kCopyAhead; j++) {
        const int x = slab * kSlab + j * 32 + lane;
        at[j] = x < G.vecs ? G.at(x) : -1;
        if (at[j] >= 0) v[j] = __ldcs(from + at[j]);
    }
#pragma unroll
    for (int j = 0; j < kCopyAhead; j++)
        if (at[j] >= 0) __stcs(to + at[j], v[j]);
}

// The same for pages smaller than a slab: as many of them as fill it, vectors first .. first + 255
// of the 2 n pages (K's and V's by turns) laid end to end.
__device__ __forceinline__ void copy_small(const PagedDev &P, const PageShape &G, uint4 *Kp, uint4 *Vp,
                                           const int32_t *src, const int32_t *dst, int n, long long first, int lane,
                                           int *flag) {
    const long long page0 = (first + lane) / G.vecs;
    const int x0 = (int)(first + lane - page0 * G.vecs);
    uint4 v[kCopyAhead], *to[kCopyAhead];
#pragma unroll
    for (int j = 0; j < kCopyAhead; j++) {
        const int x = x0 + 32 * j, k = x / G.vecs;
        const long long page = page0 + k;
        to[j] = nullptr;
        if (page >= 2ll * n) continue;
        const int a = src[page >> 1], b = dst[page >> 1];
        if (!P.page_ok(a) || !P.page_ok(b)) {
            raise_check(flag);
            continue;
        }
        uint4 *pool = page & 1 ? Vp : Kp;
        const long long at = G.at(x - k * G.vecs);
        to[j] = pool + b * G.sp + at;
        v[j] = __ldcs(pool + a * G.sp + at);
    }
#pragma unroll
    for (int j = 0; j < kCopyAhead; j++)
        if (to[j]) __stcs(to[j], v[j]);
}

// Pages of fewer vectors are copied many to a slab.
constexpr int kSmallPage = kSlab / 2;
// Slabs that the pages src[i] -> dst[i] of both pools, i < n, make.
__host__ __device__ __forceinline__ long long slabs_of(const PageShape &G, long long n) {
    return G.vecs < kSmallPage ? (2 * n * G.vecs + kSlab - 1) / kSlab : 2 * n * ((G.vecs + kSlab - 1) / kSlab);
}

// Pages src[i] -> dst[i] of both pools, i < n.  Small pages share slabs (900,000 of 128 bytes: 104 us, a
// warp each 650; 60,000 of 1 KB: 42, 54); from 2 KB on, where sharing gains nothing, a page is slabs of its own.
template <bool SMALL>
__device__ __forceinline__ void copy_pages(const PagedDev &P, const PageShape &G, uint4 *Kp, uint4 *Vp,
                                           const int32_t *src, const int32_t *dst, int n, int *flag) {
    const int lane = threadIdx.x & 31, slabs = (G.vecs + kSlab - 1) / kSlab;
    const long long tasks = slabs_of(G, n), stride = (long long)gridDim.x * (kCopyThreads / 32);
    for (long long t = (long long)blockIdx.x * (kCopyThreads / 32) + (threadIdx.x >> 5); t < tasks; t += stride) {
        if constexpr (SMALL) {
            copy_small(P, G, Kp, Vp, src, dst, n, t * kSlab, lane, flag);
            continue;
        }
        const long long pair = t / slabs;
        const int slab = (int)(t - pair * slabs), i = (int)(pair >> 1);
        const int a = src[i], b = dst[i];
        if (!P.page_ok(a) || !P.page_ok(b)) {
            raise_check(flag);
            continue;
        }
        copy_slab(G, pair & 1 ? Vp : Kp, a, b, slab, lane);
    }
}

template <bool SMALL>
__global__ void __launch_bounds__(kCopyThreads) copy_kernel(const __grid_constant__ PagedDev P,
                                                            const __grid_constant__ PageShape G, uint4 *Kp, uint4 *Vp,
                                                            const int32_t *src, const int32_t *dst, int n, int *flag) {
    griddep_wait();
    copy_pages<SMALL>(P, G, Kp, Vp, src, dst, n, flag);
}

// Fork, first part: checks everything, finds a page for every part-filled tail, sets lens.
__global__ void __launch_bounds__(kPlanThreads) fork_plan_kernel(const __grid_constant__ PagedDev P, int32_t *refs,
                                                                 int32_t *lens, const int32_t *src, const int32_t *dst,
                                                                 int n, int *area, int *flag) {
    __shared__ int s[32], slot[2];
    Cluster cl;
    griddep_wait();
    int *tail = area + kHead, *list = tail + n, *held = list + P.num_pages;
    const int tid = threadIdx.x;
    bool bad = false;
    int sum = 0;
    if (cl.rank == 0) {                        // the pairs are the first CTA's
        // each dst is claimed by its lens, which has to be 0: neither in use nor listed twice
        for (int i = tid; i < n; i += kPlanThreads) {
            const int a = src[i], d = dst[i];
            held[i] = 0;
            if ((unsigned)a >= (unsigned)P.B || (unsigned)d >= (unsigned)P.B) bad = true;
            else if (atomicCAS(lens + d, 0, -1) != 0) bad = true;
            else held[i] = 1;
        }
        bad = __syncthreads_or(bad);
        // a src that is a dst too has the length -1 now
        for (int base = 0; base < n && !bad; base += kPlanThreads) {
            const int i = base + tid;
            int part = 0, total;
            bool wrong = false;
            if (i < n) {
                const int len = __ldcg(lens + src[i]);
                int q, r = 0;
                wrong = len < 0 || len > P.cap;
                if (!wrong) P.locate(len, q, r);
                part = r > 0;
            }
            bad = __syncthreads_or(wrong);
            const int at = sum + block_scan(part, s, total) - part;
            if (i < n) tail[i] = part ? at : -1;
            sum += total;
        }
    }
    int before, want;
    cl.exchange(bad ? -1 : sum, slot, before, want);           // the others add 0
    if (want > 0 && find_free(refs, P.num_pages, want, list, s, slot, cl) < want) want = -1;
    if (cl.rank == 0) {
        __syncthreads();
        for (int i = tid; i < n; i += kPlanThreads) {
            if (want < 0) {
                if (held[i]) lens[dst[i]] = 0;
            } else {
                lens[dst[i]] = __ldcg(lens + src[i]);
                if (tail[i] >= 0) {
                    const int page = __ldcg(list + tail[i]);
                    tail[i] = page;
                    refs[page] = 1;
                }
            }
        }
        if (tid == 0) {
            area[kOk] = want >= 0;
            if (want < 0) raise_check(flag);
        }
    }
    cl.sync();
}

// Fork, second part: rows, references and the tails' tokens.
__global__ void __launch_bounds__(kCopyThreads) fork_kernel(const __grid_constant__ PagedDev P, int shift, uint4 *Kp,
                                                            uint4 *Vp, int32_t *refs, int32_t *table,
                                                            const int32_t *lens, const int32_t *src, const int32_t *dst,
                                                            const int *area, int *flag) {
    griddep_wait();
    const int i = blockIdx.x, ok = area[kOk], a_row = src[i], b_row = dst[i], b = (area + kHead)[i];
    if (!ok) return;
    const int len = lens[a_row];
    const int32_t *from = table + (long long)a_row * P.max_pages;
    int32_t *to = table + (long long)b_row * P.max_pages;
    int whole, part;
    P.locate(len, whole, part);
    const int a = part ? from[whole] : 0;
    const int t0 = blockIdx.y * kCopyThreads + threadIdx.x, step = gridDim.y * kCopyThreads;
    for (int k = t0; k < whole; k += step) {
        const int page = from[k];
        to[k] = page;
        if (P.page_ok(page)) atomicAdd(refs + page, 1);
        else raise_check(flag);
    }
    if (part == 0) return;
    if (t0 == 0) to[whole] = b;
    if (!P.page_ok(a)) {
        raise_check(flag);
        return;
    }
    // the tokens that the page holds: (head, slot, vector), both pools
    const int cols = P.d >> shift, n = P.Hkv * part * cols;
    const long long sp = P.sp >> shift, sh = P.sh >> shift, st = P.st >> shift;
    for (int x = t0; x < n; x += step) {
        const int row = x / cols, h = row / part;
        const long long at = h * sh + (row - h * part) * st + (x - row * cols);
        const uint4 k = Kp[a * sp + at], v = Vp[a * sp + at];
        Kp[b * sp + at] = k;
        Vp[b * sp + at] = v;
    }
}

// One CTA per listed sequence; the first to take its length frees it.
__global__ void __launch_bounds__(kFreeThreads) free_kernel(const __grid_constant__ PagedDev P, int32_t *refs,
                                                            int32_t *table, int32_t *lens, const int32_t *rows,
                                                            int *flag) {
    __shared__ int s_len;
    griddep_wait();
    const int b = rows[blockIdx.x];
    if ((unsigned)b >= (unsigned)P.B) {
        if (threadIdx.x == 0) raise_check(flag);
        return;
    }
    if (threadIdx.x == 0) {
        int len = atomicExch(lens + b, 0);
        if (len < 0 || len > P.cap) {
            raise_check(flag);
            len = len < 0 ? 0 : P.cap;
        }
        s_len = len;
    }
    __syncthreads();
    const int n = P.pages_of(s_len);
    int32_t *row = table + (long long)b * P.max_pages;
    for (int k = threadIdx.x; k < n; k += kFreeThreads) {
        const int page = row[k];
        row[k] = -1;
        if (!P.page_ok(page)) {
            raise_check(flag);
        } else if (atomicSub(refs + page, 1) <= 0) {           // listed more often than counted
            atomicAdd(refs + page, 1);
            raise_check(flag);
        }
    }
}

// Packing, first part: L, the free pages below it and the used ones from it on, both ascending;
// rank[page] of the latter (-1: a free page there) and their refs.
__global__ void __launch_bounds__(kPlanThreads) compact_plan_kernel(const __grid_constant__ PagedDev P,
                                                                    const int32_t *refs, int32_t *live_out, int *area) {
    __shared__ int s[32], slot[2];
    Cluster cl;
    griddep_wait();
    const int n = P.num_pages, mine = (cl.rank * kPlanThreads + (int)threadIdx.x) * kPerThread;
    const int step = cl.size * kPlanStep;
    int *hole = area + kHead, *mover = hole + n, *count = mover + n, *rank = count + n;
    int used = 0, total, before, live;
    int next[kPerThread];
    for (int base = 0; base < n; base += step) {
        int r[kPerThread];
        load_refs(refs, min(base + mine, n), n, r);
#pragma unroll
        for (int i = 0; i < kPerThread; i++) {
            used += base + mine + i < n && r[i] != 0;
            if (base == 0) next[i] = r[i];     // the first step's are the next loop's first
        }
    }
    block_scan(used, s, total);
    cl.exchange(total, slot, before, live);
    int holes = 0, movers = 0;
    for (int base = 0; base < n; base += step) {
        int r[kPerThread], k = 0;
#pragma unroll
        for (int i = 0; i < kPerThread; i++) {
            const int page = base + mine + i;
            r[i] = next[i];
            if (page < live) k += r[i] == 0 ? 1 : 0;
            else if (page < n) k += r[i] != 0 ? 1 << 16 : 0;        // both counts of a CTA's step fit 16 bits
        }
        if (base + step < n) load_refs(refs, min(base + step + mine, n), n, next);
        const int here = block_scan(k, s, total) - k;
        int hb, ha, mb, ma;
        cl.exchange(total & 0xffff, slot, hb, ha);
        cl.exchange(total >> 16, slot, mb, ma);
        int ah = holes + hb + (here & 0xffff), am = movers + mb + (here >> 16);
#pragma unroll
        for (int i = 0; i < kPerThread; i++) {
            const int page = base + mine + i;
            if (page < live) {
                if (r[i] == 0) hole[ah++] = page;
            } else if (page < n) {
                rank[page] = r[i] != 0 ? am : -1;
                if (r[i] != 0) {
                    mover[am] = page;
                    count[am++] = r[i];
                }
            }
        }
        holes += ha;
        movers += ma;
    }
    if (cl.rank == 0 && threadIdx.x == 0) {
        area[kMoves] = movers;                 // as many as there are holes
        area[kLive] = live;
        if (live_out) *live_out = live;
    }
    cl.sync();
}

// Packing, second part: the pages, the refs, the table.
template <bool SMALL>
__global__ void __launch_bounds__(kCopyThreads) compact_kernel(const __grid_constant__ PagedDev P,
                                                               const __grid_constant__ PageShape G, uint4 *Kp, uint4 *Vp,
                                                               const int32_t *refs, const int32_t *table,
                                                               int32_t *refs_out, int32_t *table_out, const int *area,
                                                               int *flag) {
    griddep_wait();
    const int n = P.num_pages, moves = area[kMoves], live = area[kLive];
    const int *hole = area + kHead, *mover = hole + n, *count = mover + n, *rank = count + n;
    const long long t0 = (long long)blockIdx.x * kCopyThreads + threadIdx.x, step = (long long)gridDim.x * kCopyThreads;
    const long long entries = (long long)P.B * P.max_pages;
    for (long long x = t0; x < entries; x += step) {
        int page = table[x];
        if (page >= live && page < n) {
            const int r = rank[page];
            if (r >= 0) page = hole[r];
        } else if (page >= n) {
            raise_check(flag);
        }
        table_out[x] = page;
    }
    if (refs_out != refs)
        for (long long x = t0; x < n; x += step) {
            const int r = refs[x];
            if (x >= live) refs_out[x] = 0;
            else if (r != 0) refs_out[x] = r;
        }
    for (long long x = t0; x < moves; x += step) {
        refs_out[hole[x]] = count[x];
        if (refs_out == refs) refs_out[mover[x]] = 0;
    }
    copy_pages<SMALL>(P, G, Kp, Vp, mover, hole, moves, flag);
}

// ---- host side
PageShape page_shape(const PagedDev &P, fs_dtype dt) {
    const int v = 16 / (int)dtype_bytes(dt);
    PageShape G;
    G.vecs = P.Hkv * P.ps * (P.d / v);
    G.sp = P.sp / v;
    long long n[2] = {P.Hkv, P.ps}, st[2] = {P.sh, P.st};
    if (st[1] > st[0]) {                       // inner runs are those that lie closer together
        std::swap(n[0], n[1]);
        std::swap(st[0], st[1]);
    }
    long long run = P.d;
    if (n[1] == 1 || st[1] == run) {           // the inner steps continue one another
        run *= n[1];
        n[1] = 1;
        if (n[0] == 1 || st[0] == run) {
            run *= n[0];
            n[0] = 1;
        }
    }
    G.run = (int)(run / v);
    G.inner = (int)n[1];
    G.so = st[0] / v;
    G.si = st[1] / v;
    return G;
}

unsigned copy_grid(const PageShape &G, long long pages) {
    const long long tasks = slabs_of(G, pages), warps = kCopyThreads / 32;
    return (unsigned)std::max(1ll, std::min((tasks + warps - 1) / warps, 148ll * 8));
}

// One cluster: a CTA where it reads all refs in one step, else eight.
template <typename... KArgs, typename... Args>
cudaError_t launch_plan(void (*kern)(KArgs...), int num_pages, cudaStream_t st, Args &&...args) {
    const unsigned n = num_pages <= kPlanStep ? 1 : 8;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(n);
    cfg.blockDim = dim3(kPlanThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = n;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...);
}

int *area_of(void *ws) { return reinterpret_cast<int *>(static_cast<uint8_t *>(ws) + kPagedArea); }
fs_status done(cudaError_t e) { return e == cudaSuccess ? FS_OK : FS_ERR_CUDA; }

}  // namespace

size_t pages_area_bytes(const fs_paged_params *p) {
    return 4 * ((size_t)kHead + 4 * (size_t)p->num_pages + 3 * ((size_t)p->B + 1));
}

fs_status paged_dev(const fs_paged_params *p, PagedDev *out) {
    if (!p) return FS_ERR_INVALID_ARG;
    if (p->B < 1 || p->H < 1 || p->Hkv < 1 || p->d < 1 || p->page_size < 1 || p->num_pages < 1 || p->max_pages < 1)
        return FS_ERR_INVALID_ARG;
    if (!dtype_known(p->dtype) || p->H % p->Hkv) return FS_ERR_INVALID_ARG;
    if (p->d != 64 && p->d != 128 && p->d != 256) return FS_ERR_UNSUPPORTED;
    if ((long long)p->max_pages * p->page_size >= 1ll << 30) return FS_ERR_UNSUPPORTED;
    if (p->H > 65535 || p->num_pages > kMaxPages || (long long)p->Hkv * p->page_size * p->d > 1ll << 30)
        return FS_ERR_UNSUPPORTED;
    const long long v = 16 / (long long)dtype_bytes(p->dtype);
    // the dimensions by stride, each step past everything that the smaller ones span
    struct { long long n, s; } dim[3] = {{p->num_pages, p->page_stride}, {p->Hkv, p->head_stride}, {p->page_size, p->token_stride}};
    std::sort(dim, dim + 3, [](const auto &a, const auto &b) { return a.s < b.s; });
    long long span = p->d;
    for (const auto &x : dim) {
        if (x.n == 1) continue;
        if (x.s < span) return FS_ERR_INVALID_ARG;
        if (x.s % v) return FS_ERR_UNSUPPORTED;
        if (x.s > (1ll << 50) / x.n) return FS_ERR_INVALID_ARG;
        span += (x.n - 1) * x.s;
    }
    if (!out) return FS_OK;
    out->B = p->B; out->H = p->H; out->Hkv = p->Hkv; out->d = p->d;
    out->ps = p->page_size; out->num_pages = p->num_pages; out->max_pages = p->max_pages;
    out->cap = p->max_pages * p->page_size;
    out->magic = (unsigned)std::min(0xffffffffull, 0x100000000ull / (unsigned)p->page_size);
    // a dimension of one has a stride that nothing reads
    out->sp = p->num_pages == 1 ? 0 : p->page_stride;
    out->sh = p->Hkv == 1 ? 0 : p->head_stride;
    out->st = p->page_size == 1 ? 0 : p->token_stride;
    return FS_OK;
}

fs_status paged_call(const fs_paged_params *p, PagedDev *out, const void *ws, size_t ws_bytes) {
    const fs_status s = paged_dev(p, out);
    if (s != FS_OK) return s;
    size_t need;
    fs_paged_workspace_size(p, &need);
    if (!ws || ws_bytes < need) return FS_ERR_WORKSPACE;
    return aligned16(ws) ? FS_OK : FS_ERR_INVALID_ARG;
}

}  // namespace fs

using namespace fs;

extern "C" fs_status fs_paged_workspace_size(const fs_paged_params *p, size_t *bytes) {
    if (!bytes) return FS_ERR_INVALID_ARG;
    const fs_status s = paged_dev(p, nullptr);
    if (s != FS_OK) return s;
    *bytes = (kPagedArea + std::max(attend_area_bytes(p), pages_area_bytes(p)) + 255) / 256 * 256;
    return FS_OK;
}

extern "C" fs_status fs_pages_reserve(const fs_paged_params *p, const int32_t *n_new, int32_t *refs, int32_t *table,
                                      int32_t *lens, void *ws, size_t ws_bytes, void *stream) {
    PagedDev P;
    const fs_status s = paged_call(p, &P, ws, ws_bytes);
    if (s != FS_OK) return s;
    if (!n_new || !refs || !table || !lens || !aligned16(refs)) return FS_ERR_INVALID_ARG;
    const cudaStream_t st = (cudaStream_t)stream;
    LaunchScope scope(kPagesReserve, st);
    return done(launch_plan(reserve_kernel, P.num_pages, st, P, n_new, refs, table, lens, area_of(ws),
                           static_cast<int *>(ws)));
}

extern "C" fs_status fs_pages_copy(const fs_paged_params *p, void *Kp, void *Vp, const int32_t *src, const int32_t *dst,
                                   int n, void *ws, size_t ws_bytes, void *stream) {
    PagedDev P;
    const fs_status s = paged_call(p, &P, ws, ws_bytes);
    if (s != FS_OK) return s;
    if (n < 0) return FS_ERR_INVALID_ARG;
    if (n == 0) return FS_OK;
    if (!Kp || !Vp || !src || !dst || !aligned16(Kp) || !aligned16(Vp)) return FS_ERR_INVALID_ARG;
    const PageShape G = page_shape(P, p->dtype);
    const cudaStream_t st = (cudaStream_t)stream;
    LaunchScope scope(kPagesCopy, st);
    return done(launch_pdl(G.vecs < kSmallPage ? copy_kernel<true> : copy_kernel<false>, dim3(copy_grid(G, n)), dim3(kCopyThreads), 0, st, P, G, (uint4 *)Kp, (uint4 *)Vp,
                           src, dst, n, static_cast<int *>(ws)));
}

extern "C" fs_status fs_pages_fork(const fs_paged_params *p, void *Kp, void *Vp, int32_t *refs, int32_t *table,
                                   int32_t *lens, const int32_t *src, const int32_t *dst, int n, void *ws,
                                   size_t ws_bytes, void *stream) {
    PagedDev P;
    const fs_status s = paged_call(p, &P, ws, ws_bytes);
    if (s != FS_OK) return s;
    if (n < 0 || n > p->B) return FS_ERR_INVALID_ARG;          // the dst are distinct
    if (n == 0) return FS_OK;
    if (!Kp || !Vp || !refs || !table || !lens || !src || !dst) return FS_ERR_INVALID_ARG;
    if (!aligned16(Kp) || !aligned16(Vp) || !aligned16(refs)) return FS_ERR_INVALID_ARG;
    const cudaStream_t st = (cudaStream_t)stream;
    int *flag = static_cast<int *>(ws);
    {
        LaunchScope scope(kPagesForkPlan, st);
        const cudaError_t e = launch_plan(fork_plan_kernel, P.num_pages, st, P, refs, lens, src, dst, n,
                                         area_of(ws), flag);
        if (e != cudaSuccess) return FS_ERR_CUDA;
    }
    const int vec = 16 / (int)dtype_bytes(p->dtype);
    // a tail's vectors and a row's entries over as many CTAs as keep four of either per thread
    const long long work = std::max<long long>((long long)p->Hkv * p->page_size * (p->d / vec), p->max_pages);
    const unsigned gy = (unsigned)std::max(1ll, std::min(std::min(work / (4 * kCopyThreads), 148ll * 8 / n + 1), 64ll));
    LaunchScope scope(kPagesFork, st);
    return done(launch_pdl(fork_kernel, dim3(n, gy), dim3(kCopyThreads), 0, st, P, p->dtype == FS_F32 ? 2 : 3, (uint4 *)Kp, (uint4 *)Vp, refs,
                           table, (const int32_t *)lens, src, dst, (const int *)area_of(ws), flag));
}

extern "C" fs_status fs_pages_free(const fs_paged_params *p, int32_t *refs, int32_t *table, int32_t *lens,
                                   const int32_t *rows, int n, void *ws, size_t ws_bytes, void *stream) {
    PagedDev P;
    const fs_status s = paged_call(p, &P, ws, ws_bytes);
    if (s != FS_OK) return s;
    if (n < 0) return FS_ERR_INVALID_ARG;
    if (n == 0) return FS_OK;
    if (!refs || !table || !lens || !rows) return FS_ERR_INVALID_ARG;
    const cudaStream_t st = (cudaStream_t)stream;
    LaunchScope scope(kPagesFree, st);
    return done(launch_pdl(free_kernel, dim3(n), dim3(kFreeThreads), 0, st, P, refs, table, lens, rows,
                           static_cast<int *>(ws)));
}

extern "C" fs_status fs_pages_compact(const fs_paged_params *p, void *Kp, void *Vp, const int32_t *refs,
                                      const int32_t *table, int32_t *refs_out, int32_t *table_out, int32_t *live,
                                      void *ws, size_t ws_bytes, void *stream) {
    PagedDev P;
    const fs_status s = paged_call(p, &P, ws, ws_bytes);
    if (s != FS_OK) return s;
    if (!Kp || !Vp || !refs || !table || !refs_out || !table_out) return FS_ERR_INVALID_ARG;
    if (!aligned16(Kp) || !aligned16(Vp) || !aligned16(refs)) return FS_ERR_INVALID_ARG;
    const PageShape G = page_shape(P, p->dtype);
    const cudaStream_t st = (cudaStream_t)stream;
    {
        LaunchScope scope(kPagesCompactPlan, st);
        const cudaError_t e = launch_plan(compact_plan_kernel, P.num_pages, st, P, refs, live, area_of(ws));
        if (e != cudaSuccess) return FS_ERR_CUDA;
    }
    const long long rows = std::max<long long>(P.num_pages, (long long)P.B * P.max_pages);
    const unsigned grid = (unsigned)std::max<long long>(copy_grid(G, P.num_pages),
                                                        std::min((rows + kCopyThreads - 1) / kCopyThreads, 148ll * 8));
    LaunchScope scope(kPagesCompact, st);
    return done(launch_pdl(G.vecs < kSmallPage ? compact_kernel<true> : compact_kernel<false>, dim3(grid), dim3(kCopyThreads), 0, st, P, G, (uint4 *)Kp, (uint4 *)Vp, refs,
                           table, refs_out, table_out, (const int *)area_of(ws), static_cast<int *>(ws)));
}
