// Writing new tokens into the paged cache (fs_paged_append): the queries and keys of a step or
// of prompts are rotated by their positions, and keys and values go to their pages, in one
// launch.  Every element is read once and written once; HBM bounds prompts, the launch and one
// chain of loads (lens, table, rows) bound a decoding step.
//
// One thread holds one unit (16 bytes, 32 in the half layout) of a token's row and goes through
// `hc` of its rows: query heads, key heads, value heads.  The position's sines and the page are
// found once for all of them.
#include "fs_paged.cuh"

namespace fs {
namespace {

struct AppendArgs {
    RotaryDev rot;
    PagedDev P;
    int T, Hq, Htot, units, nrot, hc;
    long long qs, qos, ks, vs;                 // row strides in elements
    const int32_t *cu, *table, *lens;
    int *flag;
};

constexpr int kAppendThreads = 128;

template <typename T, int VE, bool HALF>
__global__ void __launch_bounds__(kAppendThreads, 10) append_kernel(const __grid_constant__ AppendArgs A, const T *Q,
                                                                    T *Qo, const T *Kn, const T *Vn, T *Kp, T *Vp) {
    using Unit = RowUnit<T, VE, HALF>;
    constexpr int kAhead = HALF ? 2 : 4;       // rows in flight per thread: four vectors either way
    __shared__ int s_lo, s_hi;
    griddep_wait();
    const PagedDev &P = A.P;
    const int per = kAppendThreads / A.units;  // tokens per block
    const int lt = threadIdx.x / A.units, u = threadIdx.x - lt * A.units;
    const int t0 = blockIdx.x * per, t = lt < A.T - t0 ? t0 + lt : A.T;      // not past 2^31

    // the sequence of the block's first token: the interval of cu that holds it, cut into 128
    // parts at a time, each thread testing one
    int b = t;
    if (A.cu) {
        const int total = A.cu[P.B];
        if (total > A.T && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0)
            raise_check(A.flag);               // lens counts tokens that were not given
        if (t0 >= total) return;               // padding, the whole block
        if (threadIdx.x == 0) {
            s_lo = 0;
            s_hi = P.B;
        }
        __syncthreads();
        int lo = 0, hi = P.B;
        while (hi - lo > 1) {
            const int step = (hi - lo + kAppendThreads - 1) / kAppendThreads;
            const long long a = lo + (long long)threadIdx.x * step;
            if (a < hi) {
                const int e = (int)min(a + step, (long long)hi);
                if (A.cu[a] <= t0 && t0 < A.cu[e]) {
                    s_lo = (int)a;
                    s_hi = e;
                }
            }
            __syncthreads();
            const int nlo = s_lo, nhi = s_hi;
            __syncthreads();
            // no part holds it: a padding row, or a cu that is not in order
            if (nlo == lo && nhi == hi) break;
            lo = nlo;
            hi = nhi;
        }
        b = lo;
        while (t < total && b + 1 < P.B && t >= A.cu[b + 1]) b++;
    }
    if (lt >= per || t >= A.T) return;

    int len = A.lens[b], pos = len - 1;
    if (A.cu) {
        const int c0 = A.cu[b], c1 = A.cu[b + 1];
        if (t < c0 || t >= c1) return;         // padding
        pos = (int)max((long long)len - c1 + t, -1ll);
    } else if (len == 0) {
        return;
    }
    if (len > P.cap || pos < 0 || pos >= len) {
        raise_check(A.flag);
        return;
    }
    int pi, slot;
    P.locate(pos, pi, slot);
    const int page = A.table[(long long)b * P.max_pages + pi];
    if (!P.page_ok(page)) {
        raise_check(A.flag);
        return;
    }
    const long long at = page * P.sp + slot * P.st;
    float c[Unit::kPairs], s[Unit::kPairs];
    if (u < A.nrot)
#pragma unroll
        for (int m = 0; m < Unit::kPairs; m++)
            rotary_angle(A.rot.turns[Unit::pair(u, m)], pos, A.rot.mscale, 1.f, c[m], s[m]);

    // this block's rows: some of the queries', then of the keys', then of the values'
    const int d = P.d, h0 = blockIdx.y * A.hc, h1 = min(h0 + A.hc, A.Htot);
    auto heads = [&](const T *x, T *y, long long ys, int count, bool turns) {
        for (int g = 0; g < count; g += kAhead) {
            Unit v[kAhead];
#pragma unroll
            for (int j = 0; j < kAhead; j++)
                if (g + j < count) v[j].load(x + j * d, u, d, A.rot.r, A.nrot);
#pragma unroll
            for (int j = 0; j < kAhead; j++) {
                if (g + j >= count) continue;
                if (turns) v[j].turn(c, s);
                v[j].store(y + j * ys, u, d, A.rot.r, A.nrot);
            }
            x += kAhead * d;
            y += kAhead * ys;
        }
    };
    const bool turns = u < A.nrot;
    const int k0 = A.Hq, v0 = k0 + P.Hkv;      // the first of the keys' and of the values' rows
    if (h0 < k0) heads(Q + t * A.qs + h0 * d, Qo + t * A.qos + h0 * d, d, min(h1, k0) - h0, turns);
    if (h0 < v0 && h1 > k0) {
        const int h = max(h0 - k0, 0);
        heads(Kn + t * A.ks + h * d, Kp + at + h * P.sh, P.sh, min(h1, v0) - k0 - h, turns);
    }
    if (h1 > v0) {
        const int h = max(h0 - v0, 0);
        heads(Vn + t * A.vs + h * d, Vp + at + h * P.sh, P.sh, h1 - v0 - h, false);
    }
}

template <typename T, int VE, bool HALF>
cudaError_t launch_as(AppendArgs &A, const void *Q, void *Qo, const void *Kn, const void *Vn, void *Kp, void *Vp,
                      cudaStream_t st) {
    using Unit = RowUnit<T, VE, HALF>;
    A.nrot = Unit::rot_units(A.rot.r);
    A.units = Unit::units(A.P.d, A.rot.r);
    const int per = kAppendThreads / A.units;
    // Rows per thread: the most that leave 2 x 148 x 2048 threads, else one, for latency (and at
    // most 65535 blocks for the rows of a token: the most heads make 196605 rows).  At 48 registers
    // an SM holds 1280 threads, so that is three waves or more.  16 + 4 + 4 heads of 128 in bf16:
    // 16,384 tokens take four (37 us, one a thread 83), 64 tokens one (3.1, four 3.7).  Between the
    // two the rule is not at its best: 2,048 tokens take one, 13.0 us, where four take 7.1.
    A.hc = 32;
    auto blocks = [&](int hc) { return (A.Htot + hc - 1) / hc; };
    while (A.hc > 1 && (long long)A.T * A.units * blocks(A.hc) < 2ll * 148 * 2048 && blocks(A.hc / 2) <= 65535)
        A.hc >>= 1;
    LaunchScope scope(kPagedAppend, st);
    const unsigned gx = (unsigned)(((long long)A.T + per - 1) / per);
    return launch_pdl(append_kernel<T, VE, HALF>, dim3(gx, blocks(A.hc)), dim3(kAppendThreads), 0, st, A,
                      (const T *)Q, (T *)Qo, (const T *)Kn, (const T *)Vn, (T *)Kp, (T *)Vp);
}

template <typename T>
cudaError_t launch_append(AppendArgs &A, bool half, const void *Q, void *Qo, const void *Kn, const void *Vn, void *Kp,
                          void *Vp, cudaStream_t st) {
    constexpr int V = 16 / (int)sizeof(T);
    const bool vec = (half ? A.rot.r / 2 : A.rot.r) % V == 0;      // else a vector would hold parts of two pairs' halves
    if (vec)
        return half ? launch_as<T, V, true>(A, Q, Qo, Kn, Vn, Kp, Vp, st)
                    : launch_as<T, V, false>(A, Q, Qo, Kn, Vn, Kp, Vp, st);
    return half ? launch_as<T, 1, true>(A, Q, Qo, Kn, Vn, Kp, Vp, st)
                : launch_as<T, 1, false>(A, Q, Qo, Kn, Vn, Kp, Vp, st);
}

}  // namespace
}  // namespace fs

using namespace fs;

extern "C" fs_status fs_paged_append(const fs_paged_params *p, const fs_rotary *rot, int T, const void *Q,
                                     long long q_stride, void *Qo, long long qo_stride, const void *K_new,
                                     long long k_stride, const void *V_new, long long v_stride, const int32_t *cu,
                                     void *Kp, void *Vp, const int32_t *table, const int32_t *lens, void *ws,
                                     size_t ws_bytes, void *stream) {
    AppendArgs A;
    const fs_status s = paged_call(p, &A.P, ws, ws_bytes);
    if (s != FS_OK) return s;
    if (T < 0 || (!cu && T != p->B)) return FS_ERR_INVALID_ARG;
    if (Q && (!Qo || !rot)) return FS_ERR_INVALID_ARG;         // without a rotation there is nothing to do to Q
    if (Q && Q == Qo && q_stride != qo_stride) return FS_ERR_INVALID_ARG;
    A.rot.r = 0;
    if (rot) {
        const fs_status r = rotary_dev(rot, p->d, &A.rot);
        if (r != FS_OK) return r;
    }
    if (T == 0) return FS_OK;
    if (!K_new || !V_new || !Kp || !Vp || !table || !lens) return FS_ERR_INVALID_ARG;
    const long long v = 16 / (long long)dtype_bytes(p->dtype);
    if (!aligned16(Q) || !aligned16(Qo) || !aligned16(K_new) || !aligned16(V_new) || !aligned16(Kp) || !aligned16(Vp))
        return FS_ERR_INVALID_ARG;
    if (T > 1 && ((Q && (q_stride % v || qo_stride % v)) || k_stride % v || v_stride % v)) return FS_ERR_UNSUPPORTED;
    if (T > 1 && Q && qo_stride < (long long)p->H * p->d) return FS_ERR_INVALID_ARG;      // rows of Qo would overlap
    A.T = T;
    A.Hq = Q ? p->H : 0;
    A.Htot = A.Hq + 2 * p->Hkv;
    A.qs = q_stride; A.qos = qo_stride; A.ks = k_stride; A.vs = v_stride;
    A.cu = cu; A.table = table; A.lens = lens;
    A.flag = static_cast<int *>(ws);
    const bool half = rot && rot->layout == FS_ROPE_HALF;
    const cudaStream_t st = (cudaStream_t)stream;
    cudaError_t e;
    if (p->dtype == FS_BF16) e = launch_append<__nv_bfloat16>(A, half, Q, Qo, K_new, V_new, Kp, Vp, st);
    else if (p->dtype == FS_F16) e = launch_append<__half>(A, half, Q, Qo, K_new, V_new, Kp, Vp, st);
    else e = launch_append<float>(A, half, Q, Qo, K_new, V_new, Kp, Vp, st);
    return e == cudaSuccess ? FS_OK : FS_ERR_CUDA;
}
