// Attention of one new token per sequence over the paged cache (fs_paged_attend).
//
//     o = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale q.k_j - m),  one pass with a running m,
//
// for the H / Hkv query heads of a key-value head at once (8 of them in f32, 16 else), so that K
// and V are read once: 4 d flops a head and token against 2 d loads.  HBM bounds it (at 16 heads a
// group, where 82 us of bytes take 94, the tensor cores are still below a tenth of what they
// give), for few tokens the chain of loads lens -> table -> rows.
//
// Split.  The rows of work are (sequence, key-value head, tile of query heads).  Their tokens
// are cut into tiles, the tiles of all rows are laid end to end, and every CTA of one resident
// wave takes an equal share of them, found on the device from lens: ragged batches are spread
// evenly, and the launch does not depend on lens, so a captured graph serves every step.  A row
// that crosses CTAs is joined by the last of them to arrive, in the order of the CTAs, so the
// result does not depend on who that is.  A row counts two tiles more than it has: what
// beginning and ending it costs, without which CTAs with many short rows finish last.
//
// Within a CTA each of four warps streams chunks of its own through a ring of two or three stages
// (cp.async, 16 bytes a lane, the rows found through the page table one stage ahead) and keeps
// its own m, sum and accumulators: no barrier until the row ends.
//
// bf16 and f16: S^T = K Q^T with 16 keys as the M and 8 heads as the N of mma.sync, then
// O^T = V^T P^T, so a group of at most 8 heads wastes no rows of a 16-row tile, and the
// probabilities become the second product's operand by an in-register 8x8 transpose.  The
// tcgen05 form of these products would want 128 keys against at least 8 columns and the scores
// brought back from tensor memory for each; at a tenth of the tensor rate it has nothing to
// win, and its operands could not be read in pages of any size.
// f32: a lane (or two, or four) per key for the scores, lanes over d for the values, fp32 FMA.
#include "fs_paged.cuh"
#include "tc_common.cuh"

namespace fs {
namespace {

constexpr int kSms = 148, kMaxGrid = 3 * kSms;   // three CTAs per SM at most
constexpr int kFlatJoin = 16;                   // most results that one CTA joins in one step
constexpr int kDeep = 4;                        // results in flight in a join
constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;

struct AttendArgs {
    PagedDev P;
    int G, NG, window;                         // heads per group, head tiles per group
    float scale2;                              // scale * log2 e
    long long qs, os;
    const int32_t *table, *lens;
    int *flag, *count;
    float *part;
};

__device__ __forceinline__ uint32_t smem_addr(const void *p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
// 16 bytes to shared memory; zeros where !ok (the source is then not read)
__device__ __forceinline__ void cp16(uint32_t dst, const void *src, bool ok) {
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
template <typename T> struct Half2;
template <> struct Half2<__nv_bfloat16> {
    static constexpr float kRaise = 1.f, kLower = 1.f;
    __device__ __forceinline__ static uint32_t pack(float a, float b) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&v);
    }
    __device__ __forceinline__ static void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                     "{%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    }
};
template <> struct Half2<__half> {
    // Probabilities (at most 1) are raised by 2^15 for the product with V, which still fits under 65504,
    // and the accumulators lowered at the row's end: f16 ends at steps of 2^-24, so that unraised a
    // probability of 2^-16 would lose 2^-9 of itself and one below 2^-25 be gone, while the sum counts it.
    static constexpr float kRaise = 0x1p15f, kLower = 0x1p-15f;
    __device__ __forceinline__ static uint32_t pack(float a, float b) {
        const __half2 v = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&v);
    }
    __device__ __forceinline__ static void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                     "{%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    }
};

// Sizes of one instantiation: HT query heads a tile.
template <typename T, int D, int HT> struct Shape {
    static constexpr bool kTc = sizeof(T) == 2;
    static constexpr int kKeys = kTc ? (D == 64 ? 32 : 16) : (D == 64 ? 16 : 8);   // keys of a warp's chunk
    static constexpr int kTile = kWarps * kKeys;                                   // tokens of a tile
    static constexpr int kRowBytes = D * (int)sizeof(T);
    static constexpr int kChunkBytes = 2 * kKeys * kRowBytes;                      // K and V
    // Stages of a warp's ring and CTAs per SM: three CTAs of two stages where their registers fit
    // (168 a thread), which hide one another's row ends; else two, or one where a chunk is 16 KB.
    static constexpr int kBlocks = D == 256 ? 1 : HT <= 8 || D == 64 ? 3 : 2;
    static constexpr int kStages = kBlocks == 3 ? 2 : 3;
    static constexpr int kWarpBytes = kStages * kChunkBytes;
    static constexpr int kSmem = kWarps * kWarpBytes;
    static constexpr int kPart = HT * D + (HT == 1 ? 4 : 2 * HT);                   // floats of a partial result
    static_assert(kPart % 4 == 0 && kPart <= 16 * (D + 2), "16-byte vectors, attend_area_bytes");
    static_assert(HT * D * 4 <= kChunkBytes, "a warp's result fits in a stage");
    // place of element d of head h in a warp's result: the four head pairs that a warp writes at
    // once go to different banks
    __device__ __forceinline__ static int out(int h, int d) { return h * D + (d ^ (((h >> 1) & 3) << 3)); }
};

// Where a warp's chunk rows are: lane j < kKeys finds row j, one stage ahead of its use.
template <int KEYS> struct Rows {
    int page, slot;
    bool in;
    __device__ __forceinline__ void find(const PagedDev &P, const int32_t *trow, int tok0, int end, int lane) {
        const int tok = tok0 + lane;
        in = lane < KEYS && tok < end;
        page = slot = 0;
        if (in) {
            int pi;
            P.locate(tok, pi, slot);
            page = trow[pi];
        }
    }
};

// The chunk's rows of K and V to shared memory, 16 bytes a lane; 16-byte column c of row j lies
// at column c ^ (j & 7), so eight rows' columns are in different banks.
template <typename T, int D, int HT>
__device__ __forceinline__ void fetch(const Rows<Shape<T, D, HT>::kKeys> &R, const AttendArgs &A, const T *Kh,
                                      const T *Vh, uint32_t stage, int lane) {
    using S = Shape<T, D, HT>;
    constexpr int kCols = S::kRowBytes / 16;
    const bool ok = R.in && A.P.page_ok(R.page);
    if (R.in && !ok) raise_check(A.flag);
    const long long off = ok ? R.page * A.P.sp + R.slot * A.P.st : -1;
#pragma unroll
    for (int i = 0; i < S::kKeys * kCols / 32; i++) {
        const int x = i * 32 + lane, j = x / kCols, c = x % kCols;
        const long long o = __shfl_sync(kFull, off, j);
        const uint32_t dst = stage + j * S::kRowBytes + ((c ^ (j & 7)) << 4);
        const long long e = (o < 0 ? 0 : o) + c * (16 / (int)sizeof(T));
        cp16(dst, Kh + e, o >= 0);
        cp16(dst + S::kKeys * S::kRowBytes, Vh + e, o >= 0);
    }
}

// A warp's running softmax and accumulators, tensor-core form.  Lane l holds, for heads
// 8 n + 2 (l % 4) + {0, 1}, the accumulator rows d = 16 t + l / 4 + {0, 8}.
// The queries are operands held in registers, or, where these and the accumulators would take over
// 190, read from shared memory for every chunk.
template <typename T, int D, int HT> struct TcState {
    static constexpr int NT = HT / 8, DT = D / 16, MT = Shape<T, D, HT>::kKeys / 16;
    static constexpr bool kQShared = HT * D > 2048;
    uint32_t q[kQShared ? 1 : NT][kQShared ? 1 : DT][2];
    float m[NT][2], l[NT][2], o[DT][NT][4];

    // heads past the group's last are zeros and never written out
    __device__ __forceinline__ void start(const T *Q, int heads, uint4 *sq, int lane) {
        if constexpr (kQShared) {              // 16-byte column c of head h at column c ^ (h & 7)
            for (int x = threadIdx.x; x < HT * D / 8; x += kThreads) {
                const int h = x / (D / 8), c = x % (D / 8);
                sq[h * (D / 8) + (c ^ (h & 7))] =
                    h < heads ? reinterpret_cast<const uint4 *>(Q)[x] : make_uint4(0, 0, 0, 0);
            }
            __syncthreads();
        }
#pragma unroll
        for (int n = 0; n < NT; n++) {
            if constexpr (!kQShared) {
                const int h = 8 * n + lane / 4;
                const uint32_t *row = reinterpret_cast<const uint32_t *>(Q + h * D);
#pragma unroll
                for (int t = 0; t < DT; t++)
#pragma unroll
                    for (int e = 0; e < 2; e++) q[n][t][e] = h < heads ? row[8 * t + 4 * e + lane % 4] : 0u;
            }
            m[n][0] = m[n][1] = -INFINITY;
            l[n][0] = l[n][1] = 0.f;
#pragma unroll
            for (int t = 0; t < DT; t++)
#pragma unroll
                for (int e = 0; e < 4; e++) o[t][n][e] = 0.f;
        }
    }
    // `left` keys of the chunk exist
    __device__ __forceinline__ void chunk(uint32_t stage, uint32_t sq, int left, float scale2, int lane) {
        using S = Shape<T, D, HT>;
        float s[MT][NT][4];
#pragma unroll
        for (int i = 0; i < MT; i++) {
#pragma unroll
            for (int n = 0; n < NT; n++)
#pragma unroll
                for (int e = 0; e < 4; e++) s[i][n][e] = 0.f;
            const int row = 16 * i + (lane & 15);
            const uint32_t base = stage + row * S::kRowBytes;
#pragma unroll
            for (int t = 0; t < DT; t += 2) {
                uint32_t a[2][4];
                ldsm4(a[0], base + (((2 * t + (lane >> 4)) ^ (row & 7)) << 4));
                ldsm4(a[1], base + (((2 * t + 2 + (lane >> 4)) ^ (row & 7)) << 4));
#pragma unroll
                for (int n = 0; n < NT; n++) {
                    uint32_t b[4];
                    if constexpr (kQShared) {
                        ldsm4(b, sq + (8 * n + (lane & 7)) * D * 2 + (((2 * t + (lane >> 3)) ^ (lane & 7)) << 4));
                    } else {
                        b[0] = q[n][t][0]; b[1] = q[n][t][1]; b[2] = q[n][t + 1][0]; b[3] = q[n][t + 1][1];
                    }
                    Half2<T>::mma(s[i][n], a[0], b[0], b[1]);
                    Half2<T>::mma(s[i][n], a[1], b[2], b[3]);
                }
            }
        }
        bool up = false;
        float f[NT][2];
#pragma unroll
        for (int n = 0; n < NT; n++) {
#pragma unroll
            for (int e = 0; e < 2; e++) {
                float x = -INFINITY;
#pragma unroll
                for (int i = 0; i < MT; i++)
#pragma unroll
                    for (int k = 0; k < 2; k++) {
                        float &v = s[i][n][2 * k + e];
                        v = 16 * i + 8 * k + lane / 4 < left ? v * scale2 : -INFINITY;
                        x = fmaxf(x, v);
                    }
                x = fmaxf(x, __shfl_xor_sync(kFull, x, 4));
                x = fmaxf(x, __shfl_xor_sync(kFull, x, 8));
                x = fmaxf(x, __shfl_xor_sync(kFull, x, 16));
                const float top = fmaxf(m[n][e], x), ref = top == -INFINITY ? 0.f : top;
                f[n][e] = exp2_fast(m[n][e] - ref);
                up |= top != m[n][e];
                m[n][e] = top;
                l[n][e] *= f[n][e];
#pragma unroll
                for (int i = 0; i < MT; i++)
#pragma unroll
                    for (int k = 0; k < 2; k++) {
                        float &v = s[i][n][2 * k + e];
                        v = exp2_fast(v - ref);
                        l[n][e] += v;
                    }
            }
        }
        if (__any_sync(kFull, up)) {
#pragma unroll
            for (int t = 0; t < DT; t++)
#pragma unroll
                for (int n = 0; n < NT; n++)
#pragma unroll
                    for (int e = 0; e < 4; e++) o[t][n][e] *= f[n][e & 1];
        }
        // For the product with V a probability goes in two parts, T's nearest value and what is left,
        // rounded to T: 2^-16 of it is lost at most (f16: or 2^-40 of the largest, where the second part
        // ends), where one part alone adds as much error as the output's own rounding (262144 tokens
        // in bf16: 2.2e-3 of the output, 1.6e-3 with both).  The second product costs up to 3% at 16
        // heads a group, nothing where HBM bounds it.
        const uint32_t vbase = stage + S::kKeys * S::kRowBytes;
#pragma unroll
        for (int i = 0; i < MT; i++) {
            uint32_t p[2][NT][2];
#pragma unroll
            for (int n = 0; n < NT; n++)
#pragma unroll
                for (int k = 0; k < 2; k++) {
                    const float x = s[i][n][2 * k] * Half2<T>::kRaise, y = s[i][n][2 * k + 1] * Half2<T>::kRaise;
                    const uint32_t near = Half2<T>::pack(x, y);
                    const float2 z = Two<T>::get(near);
                    p[0][n][k] = transpose8(near);
                    p[1][n][k] = transpose8(Half2<T>::pack(x - z.x, y - z.y));
                }
            const int row = 16 * i + (lane & 7) + ((lane >> 4) << 3);
            const uint32_t base = vbase + row * S::kRowBytes;
#pragma unroll
            for (int t = 0; t < DT; t++) {
                uint32_t a[4];
                ldsm4t(a, base + (((2 * t + ((lane >> 3) & 1)) ^ (row & 7)) << 4));
#pragma unroll
                for (int n = 0; n < NT; n++) {
                    Half2<T>::mma(o[t][n], a, p[0][n][0], p[0][n][1]);
                    Half2<T>::mma(o[t][n], a, p[1][n][0], p[1][n][1]);
                }
            }
        }
    }
    // m, l and the accumulators to shared memory
    __device__ __forceinline__ void finish(float *out, float *sm, float *sl, int lane) {
        using S = Shape<T, D, HT>;
#pragma unroll
        for (int n = 0; n < NT; n++)
#pragma unroll
            for (int e = 0; e < 2; e++) {
                float x = l[n][e];
                x += __shfl_xor_sync(kFull, x, 4);
                x += __shfl_xor_sync(kFull, x, 8);
                x += __shfl_xor_sync(kFull, x, 16);
                const int h = 8 * n + 2 * (lane % 4) + e;
                if (lane < 4) {
                    sm[h] = m[n][e];
                    sl[h] = x;
                }
#pragma unroll
                for (int t = 0; t < DT; t++) {
                    out[S::out(h, 16 * t + lane / 4)] = o[t][n][e] * Half2<T>::kLower;
                    out[S::out(h, 16 * t + lane / 4 + 8)] = o[t][n][e + 2] * Half2<T>::kLower;
                }
            }
    }
};

// The same in fp32, two multiply-adds an instruction.  Scores: a lane takes kLane keys (two where
// several heads' q would else be loaded for one key's worth of work) and its share of their 16-byte
// columns; q lies in shared memory, column c of a head at c ^ (c / 8 % 8), so that the lanes'
// columns are in different banks.  The shares are summed by halves that change sides, which leaves
// each lane one to four of the sums and so the softmax of one or two heads, not of all.  Values:
// lane l holds the d's of its 16-byte (D = 64: 8-byte) columns; the probabilities and the factors
// of what is held already come from shared memory, twice each.
template <int D, int HT> struct F32State {
    using S = Shape<float, D, HT>;
    static constexpr int KEYS = S::kKeys, kLane = HT >= 4 ? 2 : 1, kGroups = KEYS / kLane, kParts = 32 / kGroups;
    static constexpr int kCols = D / 4, kOwn = D / 32;
    // A lane's sums after the change of sides: kSums, of kHeads heads and kSums / kHeads keys.  With
    // one head there is nothing to share out: every part has the sum.
    static constexpr int kSums = HT == 1 ? 1 : HT * kLane / kParts, kHeads = kSums > kLane ? kSums / kLane : 1;
    static constexpr int kKeysOwn = kSums / kHeads, kScratch = KEYS * HT + HT;   // float2 of a warp in shared memory
    static_assert(kSums >= 1 && (HT == 1 || kSums * kParts == HT * kLane), "the sums go round");
    float m[kHeads], l[kHeads];
    uint64_t o[HT][kOwn / 2];

    __device__ __forceinline__ void start() {
#pragma unroll
        for (int h = 0; h < kHeads; h++) {
            m[h] = -INFINITY;
            l[h] = 0.f;
        }
#pragma unroll
        for (int h = 0; h < HT; h++)
#pragma unroll
            for (int e = 0; e < kOwn / 2; e++) o[h][e] = 0ull;
    }
    // sum v of a part is of head v / kLane and of the v % kLane-th of its group's keys, v counted
    // over all parts' sums in order
    __device__ __forceinline__ static int head(int part, int i) { return HT == 1 ? 0 : (part * kSums + i) / kLane; }
    __device__ __forceinline__ static int key(int group, int part, int i) {
        return HT == 1 ? group : group + kGroups * ((part * kSums + i) % kLane);
    }
    // over the lanes that hold sums of the same head
    template <typename F> __device__ __forceinline__ static float over_head(float x, F &&f) {
#pragma unroll
        for (int y = kGroups / 2; y >= 1; y >>= 1) x = f(x, __shfl_xor_sync(kFull, x, y));
        if (HT > 1 && kSums < kLane) x = f(x, __shfl_xor_sync(kFull, x, kGroups));
        return x;
    }
    // element offset in a row of the lane's own values (kOwn of them: 2, 4 or two times 4)
    __device__ __forceinline__ static int own(int lane, int e) {
        return kOwn == 2 ? 2 * lane + e : 4 * lane + (e & 3) + (e >> 2) * 128;
    }
    // place of column c of a head in s_q
    __device__ __forceinline__ static int q_col(int c) { return c ^ ((c >> 3) & 7); }
    // the i-th column of part p.  Eight lanes read at once: eight groups read one column of rows that
    // the layout keeps apart, four groups two columns that differ by four.
    __device__ __forceinline__ static int column(int p, int i) {
        if (kGroups >= 8) return p + kParts * i;
        return (i & 3) | ((p & 1) << 2) | (((i >> 2) * (kParts / 2) + (p >> 1)) << 3);
    }
    __device__ __forceinline__ void chunk(const uint8_t *stage, const float *sq, float2 *sp, int left, float scale2,
                                          int lane) {
        const int group = lane % kGroups, part = lane / kGroups;
        uint64_t s2[kLane][HT];
#pragma unroll
        for (int k = 0; k < kLane; k++)
#pragma unroll
            for (int h = 0; h < HT; h++) s2[k][h] = 0ull;
#pragma unroll
        for (int i = 0; i < kCols / kParts; i++) {
            const int c = column(part, i);
            ulonglong2 x[kLane];
#pragma unroll
            for (int k = 0; k < kLane; k++) {
                const int key = group + kGroups * k;
                x[k] = *reinterpret_cast<const ulonglong2 *>(stage + key * S::kRowBytes + ((c ^ (key & 7)) << 4));
            }
#pragma unroll
            for (int h = 0; h < HT; h++) {
                const ulonglong2 q = *reinterpret_cast<const ulonglong2 *>(sq + h * D + 4 * q_col(c));
#pragma unroll
                for (int k = 0; k < kLane; k++) {
                    s2[k][h] = tc::f2_fma(q.x, x[k].x, s2[k][h]);
                    s2[k][h] = tc::f2_fma(q.y, x[k].y, s2[k][h]);
                }
            }
        }
        float v[HT * kLane];
#pragma unroll
        for (int h = 0; h < HT; h++)
#pragma unroll
            for (int k = 0; k < kLane; k++) {
                float a, b;
                tc::f2_unpack(s2[k][h], a, b);
                v[h * kLane + k] = a + b;
            }
        if constexpr (HT == 1) {
#pragma unroll
            for (int y = kGroups; y < 32; y <<= 1) v[0] += __shfl_xor_sync(kFull, v[0], y);
        } else {
#pragma unroll
            for (int bit = kParts / 2, half = HT * kLane / 2; bit >= 1; bit >>= 1, half >>= 1) {
                const bool up = part & bit;
#pragma unroll
                for (int j = 0; j < HT * kLane / 2; j++) {
                    if (j >= half) continue;
                    const float send = up ? v[j] : v[j + half], keep = up ? v[j + half] : v[j];
                    v[j] = keep + __shfl_xor_sync(kFull, send, bit * kGroups);
                }
            }
        }
        bool up = false;
#pragma unroll
        for (int g = 0; g < kHeads; g++) {
            float x = -INFINITY;
#pragma unroll
            for (int k = 0; k < kKeysOwn; k++) {
                float &s = v[g * kKeysOwn + k];
                s = key(group, part, g * kKeysOwn + k) < left ? s * scale2 : -INFINITY;
                x = fmaxf(x, s);
            }
            x = over_head(x, [](float a, float b) { return fmaxf(a, b); });
            const float top = fmaxf(m[g], x), ref = top == -INFINITY ? 0.f : top;
            const float f = exp2f(m[g] - ref);
            up |= top != m[g];
            m[g] = top;
            l[g] *= f;
#pragma unroll
            for (int k = 0; k < kKeysOwn; k++) {
                const int i = g * kKeysOwn + k;
                const float p = exp2f(v[i] - ref);
                l[g] += p;
                if (HT > 1 || part == 0) sp[key(group, part, i) * HT + head(part, i)] = make_float2(p, p);
            }
            if (group == 0) sp[KEYS * HT + head(part, g * kKeysOwn)] = make_float2(f, f);
        }
        up = __any_sync(kFull, up);
        __syncwarp();
        uint64_t w[HT];
        auto read = [&](const float2 *from) {
            if constexpr (HT == 1) {
                w[0] = *reinterpret_cast<const uint64_t *>(from);
            } else {
#pragma unroll
                for (int h = 0; h < HT; h += 2) {
                    const ulonglong2 x = *reinterpret_cast<const ulonglong2 *>(from + h);
                    w[h] = x.x;
                    w[h + 1] = x.y;
                }
            }
        };
        if (up) {
            read(sp + KEYS * HT);
#pragma unroll
            for (int h = 0; h < HT; h++)
#pragma unroll
                for (int e = 0; e < kOwn / 2; e++) o[h][e] = tc::f2_fma(o[h][e], w[h], 0ull);
        }
        const uint8_t *v0 = stage + KEYS * S::kRowBytes;
#pragma unroll
        for (int k = 0; k < KEYS; k++) {
            uint64_t x[kOwn / 2];
            if constexpr (kOwn == 2) {
                x[0] = *reinterpret_cast<const uint64_t *>(v0 + k * S::kRowBytes + (((lane >> 1) ^ (k & 7)) << 4) +
                                                           (lane & 1) * 8);
            } else {
#pragma unroll
                for (int g = 0; g < kOwn / 4; g++) {
                    const ulonglong2 y = *reinterpret_cast<const ulonglong2 *>(v0 + k * S::kRowBytes +
                                                                               (((lane + 32 * g) ^ (k & 7)) << 4));
                    x[2 * g] = y.x;
                    x[2 * g + 1] = y.y;
                }
            }
            read(sp + k * HT);
#pragma unroll
            for (int h = 0; h < HT; h++)
#pragma unroll
                for (int e = 0; e < kOwn / 2; e++) o[h][e] = tc::f2_fma(w[h], x[e], o[h][e]);
        }
        __syncwarp();
    }
    __device__ __forceinline__ void finish(float *out, float *sm, float *sl, int lane) {
        const int group = lane % kGroups, part = lane / kGroups;
#pragma unroll
        for (int g = 0; g < kHeads; g++) {
            const float x = over_head(l[g], [](float a, float b) { return a + b; });
            if (group == 0) {                  // several parts write the same where they share a head
                sm[head(part, g * kKeysOwn)] = m[g];
                sl[head(part, g * kKeysOwn)] = x;
            }
        }
#pragma unroll
        for (int h = 0; h < HT; h++)
#pragma unroll
            for (int e = 0; e < kOwn; e += 2) {
                float a, b;
                tc::f2_unpack(o[h][e / 2], a, b);
                out[S::out(h, own(lane, e))] = a;
                out[S::out(h, own(lane, e + 1))] = b;
            }
    }
};

// Four consecutive outputs, rounded once.
template <typename T> __device__ __forceinline__ void store4(T *p, float4 v, float f) {
    Pack<T, 4> x;
    x.e[0] = from_f<T>(v.x * f); x.e[1] = from_f<T>(v.y * f);
    x.e[2] = from_f<T>(v.z * f); x.e[3] = from_f<T>(v.w * f);
    *reinterpret_cast<Pack<T, 4> *>(p) = x;
}
__device__ __forceinline__ void add4(float4 &a, float f, const float4 &b) {
    a.x = fmaf(f, b.x, a.x); a.y = fmaf(f, b.y, a.y); a.z = fmaf(f, b.z, a.z); a.w = fmaf(f, b.w, a.w);
}

// Tokens [first, n) that sequence b attends to.
__device__ __forceinline__ void span(const AttendArgs &A, int b, int &first, int &n) {
    n = A.lens[b];
    if (n < 0 || n > A.P.cap) {
        raise_check(A.flag);
        n = n < 0 ? 0 : A.P.cap;
    }
    first = A.window >= 0 ? max(0, n - 1 - A.window) : 0;
}
// A row's work in units of a tile's time: what beginning and ending it costs, then its tiles.  An
// empty sequence has one tile, which writes its zeros.
constexpr int kRowCost = 2;
template <int TILE> __device__ __forceinline__ int units_of(int first, int n) {
    return kRowCost + max(1, (n - first + TILE - 1) / TILE);
}

// A place in the CTA's share: `left` units from unit `unit` of row r of sequence b.
struct Place {
    int b, r, unit, left;
};
// One row's part of the share.
struct Segment {
    int b, r, unit, unit1, units;              // units [unit, unit1) of the row's
    int tile, tile1;                           // its tiles
    int t0, t1, hkv;                           // its tokens [t0, t1)
    __device__ __forceinline__ bool whole() const { return tile == 0 && unit1 == units; }
};
template <int TILE> __device__ __forceinline__ Segment open(const AttendArgs &A, int HG, Place &p) {
    Segment s;
    int first, n;
    span(A, p.b, first, n);
    s.b = p.b;
    s.r = p.r;
    s.unit = p.unit;
    s.units = units_of<TILE>(first, n);
    s.unit1 = min(s.units, p.unit + p.left);
    s.tile = max(0, s.unit - kRowCost);
    s.tile1 = max(0, s.unit1 - kRowCost);
    s.t0 = min(n, first + s.tile * TILE);
    s.t1 = min(n, first + s.tile1 * TILE);
    s.hkv = A.NG == 1 ? p.r : p.r / A.NG;
    p.left -= s.unit1 - s.unit;
    p.unit = s.unit1;
    if (p.unit == s.units) {
        p.unit = 0;
        if (++p.r == HG) {
            p.r = 0;
            p.b++;
        }
    }
    return s;
}
// Warp w's chunks of a segment: the w-th of every kWarps.
template <int KEYS> __device__ __forceinline__ int chunks_of(const Segment &s, int warp) {
    const int chunks = max(0, (s.t1 - s.t0 + KEYS - 1) / KEYS);
    return (chunks - warp + kWarps - 1) / kWarps;
}

template <typename T, int D, int HT>
__global__ void __launch_bounds__(kThreads, (Shape<T, D, HT>::kBlocks))
    paged_attend_kernel(const __grid_constant__ AttendArgs A, const T *Q, const T *Kp, const T *Vp, T *O, float *lse) {
    using S = Shape<T, D, HT>;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float s_m[kWarps][HT], s_l[kWarps][HT], s_fac[HT][33];
    // the row's queries: f32, or a group of 16 heads of 256
    __shared__ __align__(16) float s_q[!S::kTc ? HT * D : HT * D > 2048 ? HT * D / 2 : 4];
    __shared__ __align__(16) float2 s_p[S::kTc ? 1 : kWarps * (S::kKeys * HT + HT)];
    __shared__ long long s_sum[kWarps], s_rem;
    __shared__ int s_b, s_last, s_out[kWarps];
    const PagedDev &P = A.P;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int HG = P.Hkv * A.NG;
    griddep_wait();

    // this CTA's share of all rows' units, and where it begins
    auto units_at = [&](int b) {
        int first, n;
        span(A, b, first, n);
        return units_of<S::kTile>(first, n);
    };
    const int seg = (P.B + kThreads - 1) / kThreads, b0 = min(P.B, tid * seg), b1 = min(P.B, b0 + seg);
    long long mine = 0;
    for (int b = b0; b < b1; b++) mine += units_at(b);
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(kFull, incl, o);
        if (lane >= o) incl += x;
    }
    if (lane == 31) s_sum[warp] = incl;
    __syncthreads();
    long long before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; w++) {
        if (w < warp) before += s_sum[w];
        total += s_sum[w];
    }
    total *= HG;
    const long long per = (total + gridDim.x - 1) / gridDim.x;
    const long long begin = blockIdx.x * per, end = min(total, begin + per);
    if (begin >= end) return;
    {
        long long x = (before + incl - mine) * HG;
        if (begin >= x && begin < x + mine * HG)
            for (int b = b0; b < b1; b++) {
                const long long n = (long long)units_at(b) * HG;
                if (begin < x + n) {
                    s_b = b;
                    s_rem = begin - x;
                    break;
                }
                x += n;
            }
    }
    __syncthreads();
    Place at;
    at.b = s_b;
    {
        const int units = units_at(at.b);
        at.r = (int)(s_rem / units);
        at.unit = (int)(s_rem - (long long)at.r * units);
        at.left = (int)(end - begin);          // fits: checked at the call
    }

    // The warp's ring of stages runs on over the rows: `ahead` is the segment whose chunks are
    // being fetched, `next` of its `chunks` chunks are; `rows` has found the one to fetch next.
    uint8_t *wsm = smem + warp * S::kWarpBytes;
    const uint32_t wst = smem_addr(wsm);
    Place fat = at;
    Segment ahead;
    int chunks = 0, next = 0;
    bool more = true;
    Rows<S::kKeys> rows;
    auto find = [&]() {
        while (next >= chunks) {
            if (fat.left <= 0) {
                more = false;
                return;
            }
            ahead = open<S::kTile>(A, HG, fat);
            chunks = chunks_of<S::kKeys>(ahead, warp);
            next = 0;
            // its query rows, to L2: they are read when the row is begun
            const int h0 = ahead.hkv * A.G + (ahead.r - ahead.hkv * A.NG) * HT;
            if (warp == 0 && lane * (128 / (int)sizeof(T)) < min(HT, (ahead.hkv + 1) * A.G - h0) * D)
                asm volatile("prefetch.global.L2 [%0];" ::"l"(Q + ahead.b * A.qs + h0 * D +
                                                              lane * (128 / (int)sizeof(T))));
        }
        rows.find(P, A.table + (long long)ahead.b * P.max_pages, ahead.t0 + (warp + kWarps * next) * S::kKeys, ahead.t1,
                  lane);
        next++;
    };
    auto fill = [&](int slot) {
        if (more) {
            fetch<T, D, HT>(rows, A, Kp + ahead.hkv * P.sh, Vp + ahead.hkv * P.sh, wst + slot * S::kChunkBytes, lane);
            find();
        }
        cp_commit();
    };
    find();
#pragma unroll
    for (int i = 0; i < S::kStages - 1; i++) fill(i);

    int slot = 0, free = S::kStages - 1;          // the stage to work on, the one that is free
    long long done = begin;
    while (at.left > 0) {
        const Segment g = open<S::kTile>(A, HG, at);
        if (g.tile1 == 0) break;               // the row's beginning alone, at the end of the share
        const int h0 = g.hkv * A.G + (g.r - g.hkv * A.NG) * HT;                // first query head
        const int heads = min(HT, (g.hkv + 1) * A.G - h0);
        const T *Qr = Q + g.b * A.qs + h0 * D;
        const int cnt = chunks_of<S::kKeys>(g, warp);
        auto stream = [&](auto &&work) {
            for (int i = 0; i < cnt; i++) {
                cp_wait<S::kStages - 2>();
                __syncwarp();
                fill(free);
                work(slot * S::kChunkBytes, min(S::kKeys, g.t1 - g.t0 - (warp + kWarps * i) * S::kKeys));
                free = slot;
                slot = slot + 1 == S::kStages ? 0 : slot + 1;
            }
            __syncwarp();                      // the free stage takes the result
        };
        if constexpr (S::kTc) {
            TcState<T, D, HT> st;
            st.start(Qr, heads, reinterpret_cast<uint4 *>(s_q), lane);
            stream([&](int off, int left) { st.chunk(wst + off, smem_addr(s_q), left, A.scale2, lane); });
            st.finish(reinterpret_cast<float *>(wsm + free * S::kChunkBytes), s_m[warp], s_l[warp], lane);
        } else {
            for (int x = tid; x < HT * D; x += kThreads)
                s_q[x / D * D + 4 * F32State<D, HT>::q_col(x % D / 4) + x % 4] = x / D < heads ? (float)Qr[x] : 0.f;
            __syncthreads();
            F32State<D, HT> st;
            st.start();
            stream([&](int off, int left) {
                st.chunk(wsm + off, s_q, s_p + warp * F32State<D, HT>::kScratch, left, A.scale2, lane);
            });
            st.finish(reinterpret_cast<float *>(wsm + free * S::kChunkBytes), s_m[warp], s_l[warp], lane);
        }
        if (lane == 0) s_out[warp] = warp * S::kWarpBytes + free * S::kChunkBytes;
        __syncthreads();

        // the four warps' results joined
        const bool whole = g.whole();
        float *part = A.part + ((long long)blockIdx.x * 2 + (g.tile == 0)) * S::kPart;
        for (int x = tid; x < heads * (D / 4); x += kThreads) {
            const int h = x / (D / 4), c = x % (D / 4) * 4;
            float m = s_m[0][h], l = 0.f;
#pragma unroll
            for (int w = 1; w < kWarps; w++) m = fmaxf(m, s_m[w][h]);
            const float ref = m == -INFINITY ? 0.f : m;
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kWarps; w++) {
                const float f = exp2f(s_m[w][h] - ref);
                l = fmaf(f, s_l[w][h], l);
                add4(o, f, *reinterpret_cast<const float4 *>(smem + s_out[w] + S::out(h, c) * 4));
            }
            if (whole) {
                store4(O + g.b * A.os + (h0 + h) * D + c, o, l == 0.f ? 0.f : 1.f / l);
                if (lse && c == 0) lse[(long long)g.b * P.H + h0 + h] = (m + log2f(l)) * kLn2;
            } else {
                *reinterpret_cast<float4 *>(part + h * D + c) = o;
                if (c == 0) {
                    part[HT * D + h] = m;
                    part[HT * D + HT + h] = l;
                }
            }
        }
        if (!whole) {
            const long long row0 = done - g.unit;                              // the row's first unit among all
            const int c0 = (int)((row0 + kRowCost) / per);                     // its CTAs
            const int n = (int)((row0 + g.units - 1) / per) - c0 + 1;
            // c0's result of the row is its second (the row begins there), the others' their first
            auto part_of = [&](int i) { return A.part + ((long long)(c0 + i) * 2 + (i == 0)) * S::kPart; };
            // whether this CTA is the last of `count` to arrive
            auto last = [&](int *counter, int count) {
                __syncthreads();
                if (tid == 0) {
                    // releases what the block wrote before the barrier, acquires what those before it did
                    int before;
                    asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], 1;"
                                 : "=r"(before) : "l"(counter) : "memory");
                    s_last = before == count - 1;
                    if (s_last) *counter = 0;                                  // for the next call
                }
                __syncthreads();
                return s_last != 0;
            };
            // the results i0, i0 + step, ... (count <= 32 of them) joined: to `to`, or as the row's output
            auto join = [&](int i0, int step, int count, float *to) {
                constexpr int kOwn = (HT + kWarps - 1) / kWarps;
                float m[kOwn], l[kOwn];
#pragma unroll
                for (int k = 0; k < kOwn; k++) {
                    const int h = warp + kWarps * k;
                    const bool in = h < heads && lane < count;
                    const float *p = part_of(i0 + (in ? lane : 0) * step) + HT * D;
                    m[k] = in ? __ldcg(p + h) : -INFINITY;
                    l[k] = in ? __ldcg(p + HT + h) : 0.f;
                }
#pragma unroll
                for (int k = 0; k < kOwn; k++) {
                    const int h = warp + kWarps * k;
                    const float top = warp_max(m[k]), f = exp2f(m[k] - (top == -INFINITY ? 0.f : top));
                    const float sum = warp_sum(f * l[k]);
                    if (h < heads) {
                        s_fac[h][lane] = f;
                        if (lane == 0) {
                            s_m[0][h] = top;
                            s_l[0][h] = sum;
                        }
                    }
                }
                __syncthreads();
                const int items = heads * (D / 4);
                for (int x = tid; x < items; x += 2 * kThreads) {              // two float4 a thread at once
                    const int y = x + kThreads < items ? x + kThreads : x;
                    const int hx = x / (D / 4), hy = y / (D / 4);
                    float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
                    // kDeep results in flight at a time; past the last, its again with the factor 0
                    for (int i = 0; i < count; i += kDeep) {
                        float4 u[kDeep], v[kDeep];
#pragma unroll
                        for (int j = 0; j < kDeep; j++) {
                            const float4 *p = reinterpret_cast<const float4 *>(part_of(i0 + min(i + j, count - 1) * step));
                            u[j] = __ldcg(p + x);
                            v[j] = __ldcg(p + y);
                        }
#pragma unroll
                        for (int j = 0; j < kDeep; j++) {
                            add4(a, s_fac[hx][i + j], u[j]);
                            add4(b, s_fac[hy][i + j], v[j]);
                        }
                    }
                    auto put = [&](int z, int h, const float4 &v) {
                        const int c = z % (D / 4) * 4;
                        const float l = s_l[0][h];
                        if (to) {
                            reinterpret_cast<float4 *>(to)[z] = v;
                            if (c == 0) {
                                to[HT * D + h] = s_m[0][h];
                                to[HT * D + HT + h] = l;
                            }
                        } else {
                            store4(O + g.b * A.os + (h0 + h) * D + c, v, l == 0.f ? 0.f : 1.f / l);
                            if (lse && c == 0) lse[(long long)g.b * P.H + h0 + h] = (s_m[0][h] + log2f(l)) * kLn2;
                        }
                    };
                    put(x, hx, a);
                    if (y != x) put(y, hy, b);
                }
            };
            // A row over many CTAs is joined in two steps, groups of about sqrt(n) side by side and
            // then their results: one CTA reads n results no faster than one after the other.
            // Counters: of a group by its first CTA, of rows that begin there and of rows that
            // go on there apart; of the groups by the row's first CTA.
            int size = n;
            if (n > kFlatJoin)
                for (size = kFlatJoin / 2; size * size < n;) size++;
            int i0 = ((int)blockIdx.x - c0) / size * size, step = 1, count = min(size, n - i0);
            int *counter = A.count + (i0 ? kMaxGrid : 0) + c0 + i0;
            while (last(counter, count)) {
                const bool out = step > 1 || size == n;
                join(i0, step, count, out ? nullptr : part_of(i0));
                if (out) break;
                i0 = 0;
                step = size;
                count = (n + size - 1) / size;
                counter = A.count + 2 * kMaxGrid + c0;
            }
        }
        __syncthreads();                       // the results, s_m and s_l are free again
        done += g.unit1 - g.unit;
    }
}


template <typename T, int D, int HT>
cudaError_t launch_as(AttendArgs &A, const void *Q, const void *Kp, const void *Vp, void *O, float *lse,
                      cudaStream_t st) {
    using S = Shape<T, D, HT>;
    A.NG = (A.G + HT - 1) / HT;
    auto *kern = paged_attend_kernel<T, D, HT>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
    if (e != cudaSuccess) return e;
    // one resident wave, or a CTA for every tile that the table could hold
    const long long most = (long long)A.P.B * A.P.Hkv * A.NG *
                           (((A.window >= 0 && A.window < A.P.cap ? A.window + 1 : A.P.cap) + S::kTile - 1) / S::kTile);
    const int grid = (int)(most < kSms * S::kBlocks ? (most < 1 ? 1 : most) : kSms * S::kBlocks);
    static_assert(3 * kMaxGrid <= kPagedCounts, "three counters for every CTA");
    LaunchScope scope(kPagedAttend, st);
    return launch_pdl(kern, dim3(grid), dim3(kThreads), S::kSmem, st, A, (const T *)Q, (const T *)Kp, (const T *)Vp,
                      (T *)O, lse);
}

// Heads per tile: the smallest that holds the group (fewer rows of zeros); larger groups, above 8
// heads in f32 and 16 else, take several tiles, each of which reads K and V again.  262,144 tokens of
// one f32 head of 128 (41 us of bytes) take 64 us for 8 query heads, 102 for 16, 183 for 32; twice
// the tokens in bf16 62 for 16, 171 for 64.
template <typename T>
cudaError_t launch_attend(AttendArgs &A, const void *Q, const void *Kp, const void *Vp, void *O, float *lse,
                          cudaStream_t st) {
    const int d = A.P.d, G = A.G;
    if constexpr (sizeof(T) == 2) {
        if (G <= 8) {
            if (d == 64) return launch_as<T, 64, 8>(A, Q, Kp, Vp, O, lse, st);
            if (d == 128) return launch_as<T, 128, 8>(A, Q, Kp, Vp, O, lse, st);
            return launch_as<T, 256, 8>(A, Q, Kp, Vp, O, lse, st);
        }
        if (d == 64) return launch_as<T, 64, 16>(A, Q, Kp, Vp, O, lse, st);
        if (d == 128) return launch_as<T, 128, 16>(A, Q, Kp, Vp, O, lse, st);
        return launch_as<T, 256, 16>(A, Q, Kp, Vp, O, lse, st);
    } else {
        if (G == 1) {
            if (d == 64) return launch_as<T, 64, 1>(A, Q, Kp, Vp, O, lse, st);
            if (d == 128) return launch_as<T, 128, 1>(A, Q, Kp, Vp, O, lse, st);
            return launch_as<T, 256, 1>(A, Q, Kp, Vp, O, lse, st);
        }
        if (G <= 4) {
            if (d == 64) return launch_as<T, 64, 4>(A, Q, Kp, Vp, O, lse, st);
            if (d == 128) return launch_as<T, 128, 4>(A, Q, Kp, Vp, O, lse, st);
            return launch_as<T, 256, 4>(A, Q, Kp, Vp, O, lse, st);
        }
        if (d == 64) return launch_as<T, 64, 8>(A, Q, Kp, Vp, O, lse, st);
        if (d == 128) return launch_as<T, 128, 8>(A, Q, Kp, Vp, O, lse, st);
        return launch_as<T, 256, 8>(A, Q, Kp, Vp, O, lse, st);
    }
}

}  // namespace

// two partial results for every CTA, of at most 16 heads
size_t attend_area_bytes(const fs_paged_params *p) { return (size_t)kMaxGrid * 2 * 16 * (p->d + 2) * 4; }

}  // namespace fs

using namespace fs;

extern "C" fs_status fs_paged_attend(const fs_paged_params *p, const void *Q, long long q_stride, const void *Kp,
                                     const void *Vp, const int32_t *table, const int32_t *lens, int window,
                                     float scale, void *O, long long o_stride, float *lse, void *ws, size_t ws_bytes,
                                     void *stream) {
    AttendArgs A;
    const fs_status s = paged_call(p, &A.P, ws, ws_bytes);
    if (s != FS_OK) return s;
    if (!Q || !Kp || !Vp || !table || !lens || !O) return FS_ERR_INVALID_ARG;
    if (!(scale > 0.f) || scale > 1e30f) return FS_ERR_INVALID_ARG;
    if (!aligned16(Q) || !aligned16(Kp) || !aligned16(Vp) || !aligned16(O)) return FS_ERR_INVALID_ARG;
    const long long v = 16 / (long long)dtype_bytes(p->dtype);
    if (p->B > 1 && (q_stride % v || o_stride % v)) return FS_ERR_UNSUPPORTED;
    if (p->B > 1 && o_stride < (long long)p->H * p->d) return FS_ERR_INVALID_ARG;        // rows of O would overlap
    // a CTA's share is counted in an int
    const int most = window >= 0 && window < A.P.cap ? window + 1 : A.P.cap;
    if ((double)p->B * p->H * (most / 64 + 1) >= 0x1p36) return FS_ERR_UNSUPPORTED;
    A.G = p->H / p->Hkv;
    A.NG = 1;
    A.window = window;
    A.scale2 = scale * kLog2e;
    A.qs = q_stride;
    A.os = o_stride;
    A.table = table;
    A.lens = lens;
    A.flag = static_cast<int *>(ws);
    A.count = reinterpret_cast<int *>(static_cast<uint8_t *>(ws) + kPagedCounters);
    A.part = reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + kPagedArea);
    const cudaStream_t st = (cudaStream_t)stream;
    cudaError_t e;
    if (p->dtype == FS_BF16) e = launch_attend<__nv_bfloat16>(A, Q, Kp, Vp, O, lse, st);
    else if (p->dtype == FS_F16) e = launch_attend<__half>(A, Q, Kp, Vp, O, lse, st);
    else e = launch_attend<float>(A, Q, Kp, Vp, O, lse, st);
    return e == cudaSuccess ? FS_OK : FS_ERR_CUDA;
}
