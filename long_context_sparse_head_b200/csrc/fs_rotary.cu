// Rotary positions as an operator of their own (fs_rotary_init, fs_rope, fs_rope_backward).
//
//     (y_1, y_2) = mscale (x_1 cos a - x_2 sin a, x_1 sin a + x_2 cos a),  a = pos theta_m,
//
// on the pairs (2m, 2m+1) or (m, m + r/2) of the first r of d dims; the backward pass is the
// same with -a (the transpose of mscale R(a) is mscale R(-a)).  Every element is read once
// and written once and 3 flops are done on it: HBM bounds it, at small sizes the launch.
//
// One thread holds one unit (16 bytes, 32 in the half layout) of a token's row and goes
// through `hc` of its heads, queries then keys, so the sines are computed once for all of
// them: at one head a thread they cost more than the memory (16,384 tokens of 16 + 4 heads of
// 128 in bf16: 62 us, with four heads a thread 30).  Four heads are loaded before the first is
// turned.
#include <algorithm>
#include <cmath>
#include <cstdlib>
#include <cstring>

#include "fs_rotary.cuh"

namespace fs {
namespace {

struct RopeArgs {
    RotaryDev rot;
    int T, N, H, Htot, d, units, nrot, hc;
    float sign;
    long long qs[3], qos[3], ks[3], kos[3];    // strides over b, h, n in elements
    long long pos_b, pos0;
    const int32_t *pos;
};

constexpr int kRopeThreads = 128;

template <typename T, int VE, bool HALF>
__global__ void __launch_bounds__(kRopeThreads, 10) rope_kernel(const __grid_constant__ RopeArgs A,
                                                            const T *Q, T *Qo, const T *K, T *Ko) {
    using Unit = RowUnit<T, VE, HALF>;
    constexpr int kRopeAhead = HALF ? 2 : 4;   // heads in flight per thread: four vectors either way
    griddep_wait();
    const int per = kRopeThreads / A.units;    // tokens per block
    const int lt = threadIdx.x / A.units, u = threadIdx.x - lt * A.units;
    const int t0 = blockIdx.x * per;
    if (lt >= per || lt >= A.T - t0) return;   // t0 + lt could pass 2^31
    const int t = t0 + lt, b = t / A.N, n = t - b * A.N;
    float c[Unit::kPairs], s[Unit::kPairs];
    if (u < A.nrot) {
        const long long pos = A.pos ? (long long)A.pos[b * A.pos_b + n] : A.pos0 + n;
#pragma unroll
        for (int m = 0; m < Unit::kPairs; m++)
            rotary_angle(A.rot.turns[Unit::pair(u, m)], pos, A.rot.mscale, A.sign, c[m], s[m]);
    }
    // this block's heads: some of Q's, then some of K's
    const int h0 = blockIdx.y * A.hc, h1 = min(h0 + A.hc, A.Htot);
    auto heads = [&](const T *x, T *y, long long xs, long long ys, int count) {
        for (int g = 0; g < count; g += kRopeAhead) {
            Unit v[kRopeAhead];
#pragma unroll
            for (int j = 0; j < kRopeAhead; j++)
                if (g + j < count) v[j].load(x + j * xs, u, A.d, A.rot.r, A.nrot);
#pragma unroll
            for (int j = 0; j < kRopeAhead; j++) {
                if (g + j >= count) continue;
                if (u < A.nrot) v[j].turn(c, s);
                v[j].store(y + j * ys, u, A.d, A.rot.r, A.nrot);
            }
            x += kRopeAhead * xs;
            y += kRopeAhead * ys;
        }
    };
    if (h0 < A.H)
        heads(Q + b * A.qs[0] + n * A.qs[2] + h0 * A.qs[1], Qo + b * A.qos[0] + n * A.qos[2] + h0 * A.qos[1], A.qs[1],
              A.qos[1], min(h1, A.H) - h0);
    if (h1 > A.H) {
        const int k0 = max(h0 - A.H, 0);
        heads(K + b * A.ks[0] + n * A.ks[2] + k0 * A.ks[1], Ko + b * A.kos[0] + n * A.kos[2] + k0 * A.kos[1], A.ks[1],
              A.kos[1], h1 - A.H - k0);
    }
}

template <typename T, int VE, bool HALF>
cudaError_t launch_as(RopeArgs &A, bool in_place, const void *Q, void *Qo, const void *K, void *Ko, cudaStream_t st) {
    using Unit = RowUnit<T, VE, HALF>;
    A.nrot = Unit::rot_units(A.rot.r);
    A.units = in_place ? A.nrot : Unit::units(A.d, A.rot.r);   // in place nothing is copied
    const int per = kRopeThreads / A.units;
    const unsigned gx = (unsigned)(((long long)A.T + per - 1) / per);
    // Heads per thread: the most that leave 2 x 148 x 2048 threads, else one, for latency.  At 48
    // registers an SM holds 1280 of them, so that is three waves or more.  16 + 4 heads of 128 in
    // bf16: 16,384 tokens take four (30 us, one a thread 62), 64 tokens one (2.5, four 3.1).  Between
    // the two the rule is not at its best: 2,048 tokens take one, 9.8 us, where eight take 5.1.
    A.hc = 32;
    while (A.hc > 1 && (long long)A.T * A.units * ((A.Htot + A.hc - 1) / A.hc) < 2ll * 148 * 2048) A.hc >>= 1;
    LaunchScope scope(kRope, st);
    return launch_pdl(rope_kernel<T, VE, HALF>, dim3(gx, (A.Htot + A.hc - 1) / A.hc), dim3(kRopeThreads), 0, st, A,
                      (const T *)Q, (T *)Qo, (const T *)K, (T *)Ko);
}

template <typename T>
cudaError_t launch_rope_op(RopeArgs &A, bool half, bool vec, bool in_place, const void *Q, void *Qo, const void *K,
                           void *Ko, cudaStream_t st) {
    constexpr int V = 16 / (int)sizeof(T);
    if (vec)
        return half ? launch_as<T, V, true>(A, in_place, Q, Qo, K, Ko, st)
                    : launch_as<T, V, false>(A, in_place, Q, Qo, K, Ko, st);
    return half ? launch_as<T, 1, true>(A, in_place, Q, Qo, K, Ko, st)
                : launch_as<T, 1, false>(A, in_place, Q, Qo, K, Ko, st);
}

// The strides of an output must keep its elements apart: taken by size, each reaches past
// everything that the smaller ones span.
bool apart(const long long (&s)[3], int B, int H, int N, int d) {
    struct { long long n, s; } dim[3] = {{B, s[0]}, {H, s[1]}, {N, s[2]}};
    for (auto &x : dim) {
        if (x.n == 1) x.s = 0;
        if (x.s > (1ll << 50) / x.n || x.s < -((1ll << 50) / x.n)) return false;
        x.s = std::abs(x.s);
    }
    std::sort(dim, dim + 3, [](const auto &a, const auto &b) { return a.s < b.s; });
    long long span = d;
    for (const auto &x : dim) {
        if (x.n == 1) continue;
        if (x.s < span) return false;
        span += (x.n - 1) * x.s;
    }
    return true;
}
// every row starts on a 16-byte boundary
bool rows_aligned(const void *p, const long long (&s)[3], int B, int H, int N, size_t es) {
    const long long v = 16 / (long long)es;
    return aligned16(p) && (B == 1 || s[0] % v == 0) && (H == 1 || s[1] % v == 0) && (N == 1 || s[2] % v == 0);
}
bool same(const long long (&a)[3], const long long (&b)[3]) { return a[0] == b[0] && a[1] == b[1] && a[2] == b[2]; }

fs_status rope(const fs_rope_params *p, const fs_rotary *rot, const void *Q, void *Qo, const void *K, void *Ko,
               const int32_t *pos, long long pos_stride, long long pos0, float sign, void *stream) {
    if (!p || !rot) return FS_ERR_INVALID_ARG;
    if (p->B < 0 || p->N < 0 || p->H < 0 || p->Hk < 0 || p->d < 1 || !dtype_known(p->dtype)) return FS_ERR_INVALID_ARG;
    if (p->d > FS_ROPE_MAX_R) return FS_ERR_UNSUPPORTED;
    RopeArgs A;
    const fs_status rs = rotary_dev(rot, p->d, &A.rot);
    if (rs != FS_OK) return rs;
    const long long T = (long long)p->B * p->N, Htot = (long long)p->H + p->Hk;
    if (T > 0x7fffffffll || Htot > 65535) return FS_ERR_UNSUPPORTED;
    if (T == 0 || Htot == 0) return FS_OK;
    if ((p->H > 0 && (!Q || !Qo)) || (p->Hk > 0 && (!K || !Ko))) return FS_ERR_INVALID_ARG;
    if ((p->H > 0 && !apart(p->qo, p->B, p->H, p->N, p->d)) || (p->Hk > 0 && !apart(p->ko, p->B, p->Hk, p->N, p->d)))
        return FS_ERR_INVALID_ARG;
    const size_t es = dtype_bytes(p->dtype);
    const uintptr_t em = es - 1;
    if (((uintptr_t)Q | (uintptr_t)Qo | (uintptr_t)K | (uintptr_t)Ko) & em) return FS_ERR_INVALID_ARG;
    // in place only with the same strides: a thread writes just what it has read
    if ((p->H > 0 && Q == Qo && !same(p->q, p->qo)) || (p->Hk > 0 && K == Ko && !same(p->k, p->ko)))
        return FS_ERR_INVALID_ARG;
    A.T = (int)T; A.N = p->N; A.H = p->H; A.Htot = (int)Htot; A.d = p->d; A.sign = sign;
    std::memcpy(A.qs, p->q, sizeof(A.qs));
    std::memcpy(A.qos, p->qo, sizeof(A.qos));
    std::memcpy(A.ks, p->k, sizeof(A.ks));
    std::memcpy(A.kos, p->ko, sizeof(A.kos));
    A.pos = pos; A.pos_b = pos_stride; A.pos0 = pos0;
    const bool half = rot->layout == FS_ROPE_HALF;
    const int v = 16 / (int)es;
    const bool vec = p->d % v == 0 && (half ? rot->r / 2 : rot->r) % v == 0 && rot->r % v == 0 &&
                     (p->H == 0 || (rows_aligned(Q, p->q, p->B, p->H, p->N, es) && rows_aligned(Qo, p->qo, p->B, p->H, p->N, es))) &&
                     (p->Hk == 0 || (rows_aligned(K, p->k, p->B, p->Hk, p->N, es) && rows_aligned(Ko, p->ko, p->B, p->Hk, p->N, es)));
    const bool in_place = (p->H == 0 || Q == Qo) && (p->Hk == 0 || K == Ko);
    const cudaStream_t st = (cudaStream_t)stream;
    cudaError_t e;
    if (p->dtype == FS_BF16) e = launch_rope_op<__nv_bfloat16>(A, half, vec, in_place, Q, Qo, K, Ko, st);
    else if (p->dtype == FS_F16) e = launch_rope_op<__half>(A, half, vec, in_place, Q, Qo, K, Ko, st);
    else e = launch_rope_op<float>(A, half, vec, in_place, Q, Qo, K, Ko, st);
    return e == cudaSuccess ? FS_OK : FS_ERR_CUDA;
}

}  // namespace

fs_status rotary_dev(const fs_rotary *rot, int d, RotaryDev *out) {
    if (rot->r < 2 || rot->r % 2 || rot->r > d || rot->r > FS_ROPE_MAX_R) return FS_ERR_INVALID_ARG;
    if (rot->layout != FS_ROPE_INTERLEAVED && rot->layout != FS_ROPE_HALF) return FS_ERR_INVALID_ARG;
    if (!std::isfinite(rot->mscale)) return FS_ERR_INVALID_ARG;
    out->r = rot->r;
    out->mscale = rot->mscale;
    static_assert(sizeof(out->turns) == sizeof(rot->turns), "one entry per pair");
    std::memcpy(out->turns, rot->turns, sizeof(out->turns));
    return FS_OK;
}

}  // namespace fs

using namespace fs;

extern "C" fs_status fs_rotary_init(int r, fs_rope_layout layout, double base, fs_rope_scaling scaling, double factor,
                                    double orig_len, double slow, double fast, double mscale, fs_rotary *out) {
    if (!out || r < 2 || r % 2) return FS_ERR_INVALID_ARG;
    if (r > FS_ROPE_MAX_R) return FS_ERR_UNSUPPORTED;
    if (layout != FS_ROPE_INTERLEAVED && layout != FS_ROPE_HALF) return FS_ERR_INVALID_ARG;
    if (!(base >= 1.0) || !std::isfinite(base) || !std::isfinite((float)mscale)) return FS_ERR_INVALID_ARG;
    if (scaling < FS_ROPE_NONE || scaling > FS_ROPE_BY_PARTS) return FS_ERR_INVALID_ARG;
    if (scaling != FS_ROPE_NONE && (!(factor >= 1.0) || !std::isfinite(factor))) return FS_ERR_INVALID_ARG;
    if (scaling == FS_ROPE_NTK && r == 2) return FS_ERR_INVALID_ARG;        // its exponent r / (r - 2)
    if (scaling == FS_ROPE_BY_PARTS &&
        (!(orig_len > 0.0) || !std::isfinite(orig_len) || !(slow >= 0.0) || !(fast > slow) || !std::isfinite(fast)))
        return FS_ERR_INVALID_ARG;
    std::memset(out, 0, sizeof(*out));
    out->r = r;
    out->layout = layout;
    out->mscale = (float)mscale;
    const long double two_pi = 6.283185307179586476925286766559005768L;
    long double lbase = logl((long double)base);
    if (scaling == FS_ROPE_NTK) lbase += logl((long double)factor) * r / (r - 2);
    for (int m = 0; m < r / 2; m++) {
        long double theta = expl(-2.0L * m / r * lbase);
        if (scaling == FS_ROPE_LINEAR) theta /= factor;
        if (scaling == FS_ROPE_BY_PARTS) {
            long double keep = (orig_len * theta / two_pi - slow) / ((long double)fast - slow);
            keep = keep < 0 ? 0 : keep > 1 ? 1 : keep;
            theta *= (1 - keep) / factor + keep;
        }
        out->turns[m] = (uint64_t)(theta / two_pi * 18446744073709551616.0L + 0.5L);   // theta <= 1: below a turn
    }
    return FS_OK;
}

extern "C" fs_status fs_rope(const fs_rope_params *p, const fs_rotary *rot, const void *Q, void *Qo, const void *K,
                             void *Ko, const int32_t *pos, long long pos_stride, long long pos0, void *stream) {
    return rope(p, rot, Q, Qo, K, Ko, pos, pos_stride, pos0, 1.f, stream);
}

extern "C" fs_status fs_rope_backward(const fs_rope_params *p, const fs_rotary *rot, const void *dQo, void *dQ,
                                      const void *dKo, void *dK, const int32_t *pos, long long pos_stride,
                                      long long pos0, void *stream) {
    return rope(p, rot, dQo, dQ, dKo, dK, pos, pos_stride, pos0, -1.f, stream);
}
