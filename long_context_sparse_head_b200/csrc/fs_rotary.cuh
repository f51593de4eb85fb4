// Rotary positions shared by the rope and the page-writing kernels.
//
// Pair m of a row turns by the angle pos * theta_m.  A float product would be off by ~0.03 rad
// at position 2^18, so theta_m / 2 pi is held as a 64-bit fraction of a turn: the 64-bit
// product with the position wraps at whole turns by itself and is off by at most
// |pos| * 2^-65 turns.  Its upper 32 bits are kept (less than 2^-32 turns are cut off) and
// reduced to an eighth of a turn either way, an exact integer step, before they become a float:
// the argument of sincospi is off by 2^-32 turns and by 2^-24 of itself, which moves a product
// by less than 2^-29 of the element beside the fp32 roundings.
#pragma once

#include <cuda_fp16.h>

#include "fs_common.cuh"

namespace fs {

template <> __device__ __forceinline__ float to_f<__half>(__half x) { return __half2float(x); }
template <> __device__ __forceinline__ __half from_f<__half>(float x) { return __float2half_rn(x); }

// Kernel-side copy of an fs_rotary (passed by value).
struct RotaryDev {
    int r;                                 // rotated dims (the first r of d); 0: none
    float mscale;
    unsigned long long turns[FS_ROPE_MAX_R / 2];
};

// (cos, sin)(pos theta) * mscale, the sine times `sign` (-1: the backward rotation).
__device__ __forceinline__ void rotary_angle(unsigned long long turns, long long pos, float mscale, float sign,
                                             float &c, float &s) {
    const unsigned long long frac = turns * (unsigned long long)pos;
    const int t = (int)(unsigned)(frac >> 32);               // a turn is 2^32
    const int quad = (int)(((unsigned)t + 0x20000000u) >> 30);   // nearest quarter turn, 0..3
    const int rest = (int)((unsigned)t - ((unsigned)quad << 30));
    float sn, cs;
    sincospif((float)rest * 0x1p-31f, &sn, &cs);
    float a = quad & 1 ? sn : cs, b = quad & 1 ? cs : sn;
    if (quad == 1 || quad == 2) a = -a;
    if (quad >= 2) b = -b;
    c = a * mscale;
    s = b * (mscale * sign);
}

// Two 16-bit elements of a 32-bit word, widened and rounded together.
template <typename T> struct Two;
template <> struct Two<__nv_bfloat16> {
    __device__ __forceinline__ static float2 get(uint32_t w) {
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    }
    __device__ __forceinline__ static uint32_t put(float a, float b) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&v);
    }
};
template <> struct Two<__half> {
    __device__ __forceinline__ static float2 get(uint32_t w) {
        return __half22float2(*reinterpret_cast<const __half2 *>(&w));
    }
    __device__ __forceinline__ static uint32_t put(float a, float b) {
        const __half2 v = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&v);
    }
};

// N elements in one access of N * sizeof(T) bytes (N = 1: one element).
template <typename T, int N> struct alignas(N * sizeof(T)) Pack {
    T e[N];
};

// A row of d elements is worked on in units, one thread per unit.  VE elements to a vector
// (16 bytes), or the element-wise form VE = 1 for rows that a vector would not fit.  The first
// `rot_units` units turn pairs: vector form, HALF: vector u of the first half with vector u
// of the second (VE pairs); interleaved: vector u (VE / 2 pairs); element-wise form: pair u.
// The others copy what lies behind the first r dims: a vector, or two elements.
template <typename T, int VE, bool HALF> struct RowUnit {
    static constexpr int kPairs = VE == 1 ? 1 : (HALF ? VE : VE / 2);
    static constexpr int kVecs = VE == 1 ? 2 : (HALF ? 2 : 1);     // accesses of a turning unit
    using P = Pack<T, VE>;
    P v[kVecs];

    __host__ __device__ static int rot_units(int r) {
        return VE == 1 ? r / 2 : (HALF ? r / 2 / VE : r / VE);
    }
    __host__ __device__ static int units(int d, int r) {
        return rot_units(r) + (VE == 1 ? (d - r + 1) / 2 : (d - r) / VE);
    }
    // element offset of access i of unit u, and whether it exists
    __device__ __forceinline__ static int offset(int u, int i, int r, int nrot) {
        if (u < nrot) {
            if (VE == 1) return HALF ? u + i * (r / 2) : 2 * u + i;
            return HALF ? u * VE + i * (r / 2) : u * VE;
        }
        return r + (VE == 1 ? 2 * (u - nrot) + i : (u - nrot) * VE);
    }
    __device__ __forceinline__ static bool exists(int u, int i, int d, int r, int nrot) {
        if (u < nrot) return true;
        return VE == 1 ? r + 2 * (u - nrot) + i < d : i == 0;
    }
    __device__ __forceinline__ void load(const T *row, int u, int d, int r, int nrot) {
#pragma unroll
        for (int i = 0; i < kVecs; i++)
            if (exists(u, i, d, r, nrot)) v[i] = *reinterpret_cast<const P *>(row + offset(u, i, r, nrot));
    }
    __device__ __forceinline__ void store(T *row, int u, int d, int r, int nrot) const {
#pragma unroll
        for (int i = 0; i < kVecs; i++)
            if (exists(u, i, d, r, nrot)) *reinterpret_cast<P *>(row + offset(u, i, r, nrot)) = v[i];
    }
    // the pairs turned in fp32 and rounded once to T
    __device__ __forceinline__ void turn(const float (&c)[kPairs], const float (&s)[kPairs]) {
        if constexpr (sizeof(T) == 2 && VE > 1) {              // word by word: one instruction rounds two
            uint32_t *x = reinterpret_cast<uint32_t *>(&v[0]);
            if constexpr (HALF) {
                uint32_t *y = reinterpret_cast<uint32_t *>(&v[1]);
#pragma unroll
                for (int w = 0; w < VE / 2; w++) {
                    const float2 a = Two<T>::get(x[w]), b = Two<T>::get(y[w]);
                    const int m = 2 * w;
                    x[w] = Two<T>::put(fmaf(a.x, c[m], -b.x * s[m]), fmaf(a.y, c[m + 1], -b.y * s[m + 1]));
                    y[w] = Two<T>::put(fmaf(a.x, s[m], b.x * c[m]), fmaf(a.y, s[m + 1], b.y * c[m + 1]));
                }
            } else {
#pragma unroll
                for (int m = 0; m < VE / 2; m++) {
                    const float2 a = Two<T>::get(x[m]);
                    x[m] = Two<T>::put(fmaf(a.x, c[m], -a.y * s[m]), fmaf(a.x, s[m], a.y * c[m]));
                }
            }
        } else {
#pragma unroll
            for (int m = 0; m < kPairs; m++) {
                constexpr bool split = VE == 1 || HALF;        // the pair's elements are in two accesses
                T &x = split ? v[0].e[VE == 1 ? 0 : m] : v[0].e[VE == 1 ? 0 : 2 * m];
                T &y = split ? v[kVecs - 1].e[VE == 1 ? 0 : m] : v[0].e[VE == 1 ? 0 : 2 * m + 1];
                const float a = to_f<T>(x), b = to_f<T>(y);
                x = from_f<T>(fmaf(a, c[m], -b * s[m]));
                y = from_f<T>(fmaf(a, s[m], b * c[m]));
            }
        }
    }
    // index of pair m of a turning unit
    __device__ __forceinline__ static int pair(int u, int m) { return u * kPairs + m; }
};

// fs_rotary -> RotaryDev; checks the fields (defined in fs_rotary.cu)
fs_status rotary_dev(const fs_rotary *rot, int d, RotaryDev *out);
inline size_t dtype_bytes(fs_dtype t) { return t == FS_F32 ? 4 : 2; }
inline bool dtype_known(fs_dtype t) { return t == FS_BF16 || t == FS_F32 || t == FS_F16; }
inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

}  // namespace fs
