// Exponentials to about 2^-36, in float32 (of float64 this GPU has little).
#pragma once

#include "obj_device.cuh"

namespace isodev {

// 2^(i / 32) as two floats.
__device__ const float2 kPowers[32] = {
    {0x1.0000000000000p+0f, 0x0.0p+0f}, {0x1.059b0e0000000p+0f, -0x1.9d4f520000000p-25f}, {0x1.0b55860000000p+0f, 0x1.9f31220000000p-25f},
    {0x1.11301e0000000p+0f, -0x1.fdb4960000000p-25f}, {0x1.172b840000000p+0f, -0x1.c157420000000p-27f}, {0x1.1d48740000000p+0f, -0x1.d2e8ca0000000p-25f},
    {0x1.2387a60000000p+0f, 0x1.ceac480000000p-25f}, {0x1.29e9e00000000p+0f, -0x1.5c04240000000p-25f}, {0x1.306fe00000000p+0f, 0x1.4636e20000000p-25f},
    {0x1.371a740000000p+0f, -0x1.18aac60000000p-25f}, {0x1.3dea640000000p+0f, 0x1.8246840000000p-25f}, {0x1.44e0860000000p+0f, 0x1.8624b40000000p-30f},
    {0x1.4bfdae0000000p+0f, -0x1.593abc0000000p-25f}, {0x1.5342b60000000p+0f, -0x1.2c56100000000p-25f}, {0x1.5ab07e0000000p+0f, -0x1.5bd5ec0000000p-27f},
    {0x1.6247ec0000000p+0f, -0x1.f8b5500000000p-25f}, {0x1.6a09e60000000p+0f, 0x1.9fcef40000000p-26f}, {0x1.71f75e0000000p+0f, 0x1.1d8bee0000000p-25f},
    {0x1.7a11480000000p+0f, -0x1.829fd00000000p-25f}, {0x1.82589a0000000p+0f, -0x1.accc7c0000000p-26f}, {0x1.8ace540000000p+0f, 0x1.15506e0000000p-27f},
    {0x1.93737c0000000p+0f, -0x1.e647440000000p-25f}, {0x1.9c49180000000p+0f, 0x1.51f8480000000p-27f}, {0x1.a5503c0000000p+0f, -0x1.b83b540000000p-25f},
    {0x1.ae89fa0000000p+0f, -0x1.a94b140000000p-26f}, {0x1.b7f7700000000p+0f, -0x1.a094380000000p-25f}, {0x1.c199be0000000p+0f, -0x1.3d56b20000000p-27f},
    {0x1.cb720e0000000p+0f, -0x1.8837cc0000000p-27f}, {0x1.d5818e0000000p+0f, -0x1.822dbc0000000p-27f}, {0x1.dfc9740000000p+0f, -0x1.908c940000000p-25f},
    {0x1.ea4afa0000000p+0f, 0x1.52486c0000000p-27f}, {0x1.f507660000000p+0f, -0x1.246eb00000000p-26f},
};

// Adds exp((v - m) / T) to the sum, a_hi + a_lo being log2(e) / T.  The exponent as two floats is split into
// i / 32 and a rest of at most 1 / 64; the rest's exponential is a polynomial (its z^5 / 120 is under
// 1.3e-12).  NaN where v is NaN or m is not finite; v is at most m.
__device__ __forceinline__ void exp_add(Sum& s, float v, float m, float a_hi, float a_lo) {
    constexpr float kLn2Hi = (float)0.693147180559945309417, kLn2Lo = (float)(0.693147180559945309417 - (double)kLn2Hi);
    // v - m = d + d_low
    const float d = __fsub_rn(v, m), back = __fsub_rn(d, v);
    const float d_low = __fsub_rn(__fsub_rn(v, __fsub_rn(d, back)), __fadd_rn(m, back));
    const float y = __fmul_rn(d, a_hi);
    if (!(y > -126.f)) {  // nothing, beside a term of 1 (or NaN)
        s.hi += d == d || v == -INFINITY ? 0.f : NAN;
        return;
    }
    const float y_low = __fmaf_rn(d, a_hi, -y) + (d * a_lo + d_low * a_hi);
    const float i = rintf(y * 32.f);
    const float r = __fmaf_rn(i, -0.03125f, y);  // exact
    // z = (r + y_low) log 2, two floats
    const float z = __fmul_rn(r, kLn2Hi);
    const float z_low = __fmaf_rn(r, kLn2Hi, -z) + __fmaf_rn(r, kLn2Lo, y_low * kLn2Hi);
    const float rest = __fmaf_rn(z * z, __fmaf_rn(z, __fmaf_rn(z, 1.f / 24, 1.f / 6), 0.5f), z_low * (1.f + z));
    const int k = (int)i;
    const float2 t = kPowers[k & 31];
    const float p = __fmul_rn(t.x, z), p_low = __fmaf_rn(t.x, z, -p) + __fmaf_rn(t.x, rest, t.y * (1.f + z));
    const float f = __uint_as_float((uint32_t)(127 + (k >> 5)) << 23);  // 2^(k >> 5); k >= -126 * 32
    s.add(t.x * f);
    s.add(p * f);
    s.lo += p_low * f;
}

}  // namespace isodev
