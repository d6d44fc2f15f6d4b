// rope.cuh -- rotary positions: angles and the turning of 16 values, and the 16-bit
// conversions around them.
#pragma once

#include "common.cuh"

namespace dsa {

template <typename T>
__device__ __forceinline__ float2 to_float2(uint32_t v);
template <>
__device__ __forceinline__ float2 to_float2<__nv_bfloat16>(uint32_t v) {
    return __bfloat1622float2(*reinterpret_cast<__nv_bfloat162*>(&v));
}
template <>
__device__ __forceinline__ float2 to_float2<__half>(uint32_t v) {
    return __half22float2(*reinterpret_cast<__half2*>(&v));
}

template <typename T>
__device__ __forceinline__ uint32_t from_float2(float x, float y);
template <>
__device__ __forceinline__ uint32_t from_float2<__nv_bfloat16>(float x, float y) {
    __nv_bfloat162 r = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<uint32_t*>(&r);
}
template <>
__device__ __forceinline__ uint32_t from_float2<__half>(float x, float y) {
    __half2 r = __floats2half2_rn(x, y);
    return *reinterpret_cast<uint32_t*>(&r);
}

template <typename T>
__device__ __forceinline__ void unpack8(const uint4& u, float (&x)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = to_float2<T>(w[i]);
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}

template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&x)[8]) {
    uint4 u;
    u.x = from_float2<T>(x[0], x[1]);
    u.y = from_float2<T>(x[2], x[3]);
    u.z = from_float2<T>(x[4], x[5]);
    u.w = from_float2<T>(x[6], x[7]);
    *reinterpret_cast<uint4*>(p) = u;
}

// (cos, sin) of pos * inv_freq.  Positions reach 2^20 and beyond, where a 32-bit angle is
// off by 1/16 of a radian, so the angle is reduced in fixed point: inv_freq / 2 pi as a
// fraction of a turn in 64 bits, times the position, modulo 2^64, is the fraction of the
// turn (the product wraps exactly; the rate is off by less than 2^-53 turns per unit of
// position).  Its upper 32 bits go to sincospi.
// The fraction of a turn per unit of position, in units of 2^-64.
__device__ __forceinline__ unsigned long long turn_rate(double inv_freq) {
    double turns = inv_freq * 0.15915494309189533577;
    turns -= floor(turns);
    return (unsigned long long)(turns * 18446744073709551616.0);
}

// In units of 2^-31 half turns.
__device__ __forceinline__ int turn_angle(unsigned long long rate, int pos) {
    const long long angle = (long long)((unsigned long long)(long long)pos * rate);
    return (int)(angle >> 32);
}

__device__ __forceinline__ float2 turn_of(double inv_freq, int pos) {
    float sn, cs;
    sincospif((float)turn_angle(turn_rate(inv_freq), pos) * 4.656612873077393e-10f, &sn, &cs);  // 2^-31
    return make_float2(cs, sn);
}

// The same from the rate, with what the angle loses as a float (up to 2^-25 half turns) given back, to
// within 2^-31: cos(a + d) = cos a - d sin a, sin(a + d) = sin a + d cos a.
__device__ __forceinline__ float2 fine_turn_of(unsigned long long rate, int pos) {
    const int angle = turn_angle(rate, pos);
    const float rounded = (float)angle;
    const int lost = (int)((unsigned)angle - (unsigned)__float2int_rz(rounded * 0.5f) * 2u);
    const float d = (float)lost * 1.4629180792671596e-9f;  // 2^-31 pi
    float sn, cs;
    sincospif(rounded * 4.656612873077393e-10f, &sn, &cs);
    return make_float2(fmaf(-d, sn, cs), fmaf(d, cs, sn));
}

// A token's (cos, sin) in shared memory as [4][pairs / 8][2]: pair 8 u + 2 p + e at
// [p][u][e], two to a load, neighbouring units in neighbouring banks.
__device__ __forceinline__ int turn_at(int pair, int pairs) {
    return (((pair >> 1 & 3) * (pairs >> 3) + (pair >> 3)) << 1) + (pair & 1);
}

// Turns unit `unit` of a head by the token's `turns`: eight pairs, the values x[i], y[i]
// of the two halves, or (interleaved) neighbours in x and then in y.
__device__ __forceinline__ void turn16(float (&x)[8], float (&y)[8], const float2* turns,
                                       int units, int unit, bool interleaved) {
    const float4* cs = reinterpret_cast<const float4*>(turns) + unit;
    if (interleaved) {
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            const float4 c = cs[p * units], d = cs[(2 + p) * units];
            const float x0 = x[4 * p], x1 = x[4 * p + 1], x2 = x[4 * p + 2], x3 = x[4 * p + 3];
            const float y0 = y[4 * p], y1 = y[4 * p + 1], y2 = y[4 * p + 2], y3 = y[4 * p + 3];
            x[4 * p] = x0 * c.x - x1 * c.y;
            x[4 * p + 1] = x1 * c.x + x0 * c.y;
            x[4 * p + 2] = x2 * c.z - x3 * c.w;
            x[4 * p + 3] = x3 * c.z + x2 * c.w;
            y[4 * p] = y0 * d.x - y1 * d.y;
            y[4 * p + 1] = y1 * d.x + y0 * d.y;
            y[4 * p + 2] = y2 * d.z - y3 * d.w;
            y[4 * p + 3] = y3 * d.z + y2 * d.w;
        }
    } else {
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            const float4 c = cs[p * units];
            const float x0 = x[2 * p], y0 = y[2 * p], x1 = x[2 * p + 1], y1 = y[2 * p + 1];
            x[2 * p] = x0 * c.x - y0 * c.y;
            y[2 * p] = y0 * c.x + x0 * c.y;
            x[2 * p + 1] = x1 * c.z - y1 * c.w;
            y[2 * p + 1] = y1 * c.z + x1 * c.w;
        }
    }
}

}  // namespace dsa
