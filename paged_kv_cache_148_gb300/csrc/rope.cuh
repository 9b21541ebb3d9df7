// Rotary positions shared by the writes that rotate (rope.cu, latent_write.cu).
//
// Pair i of a head is turned by the angle p * f_i.  The frequency is held as
// turns = f_i / 2pi in unsigned 64-bit fixed point (all 64 bits behind the
// point), so p * turns modulo 2^64, one integer product, is the fraction of a
// turn left at position p: whole turns fall off the top exactly, and no
// position is far enough to lose the angle.  A float32 p * f_i would be off by
// 2^-8 rad at p = 131072.  The fraction as a signed number of half turns
// is in [-1, 1), rounded to float32 once (angle error under 2^-23 rad).
#pragma once

#include "common.cuh"

namespace pa {

// Cosine and sine of pair i at position p, times the magnitude.
PA_DEVICE float2 rope_angle(uint64_t turns, int64_t p, float magnitude) {
    const int64_t left = (int64_t)((uint64_t)p * turns);  // signed: (-1/2, 1/2] turn
    float s, c;
    sincospif((float)left * 0x1p-63f, &s, &c);
    return make_float2(c * magnitude, s * magnitude);
}

// (x, y) turned by the angle.
PA_DEVICE void rope_turn(float2 cs, float& x, float& y) {
    const float u = x * cs.x - y * cs.y;
    y = x * cs.y + y * cs.x;
    x = u;
}

PA_DEVICE uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// 16 bytes as floats and back: 4 float32 or 8 bf16 (rounded to nearest even).
template <typename T> struct Vec16;
template <> struct Vec16<float> {
    static constexpr int N = 4;
    static PA_DEVICE void open(const uint4& w, float* f) {
        f[0] = __uint_as_float(w.x);
        f[1] = __uint_as_float(w.y);
        f[2] = __uint_as_float(w.z);
        f[3] = __uint_as_float(w.w);
    }
    static PA_DEVICE uint4 close(const float* f) {
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                          __float_as_uint(f[3]));
    }
};
template <> struct Vec16<uint16_t> {  // bf16
    static constexpr int N = 8;
    static PA_DEVICE void open(const uint4& w, float* f) {
        const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = bf16_lo(a[i]);
            f[2 * i + 1] = bf16_hi(a[i]);
        }
    }
    static PA_DEVICE uint4 close(const float* f) {
        return make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]),
                          pack_bf16(f[6], f[7]));
    }
};

// Two 16-byte vectors of one row turned together.  Half layout: a holds
// elements e.., b elements e + rot/2.., and element j of both is pair e + j
// (cs[j]).  Interleaved: a and b are neighbours, pair j is elements 2j, 2j + 1
// of the 2N.
template <typename T>
PA_DEVICE void rope_turn_vectors(bool interleaved, const float2* cs, float* a, float* b) {
    constexpr int N = Vec16<T>::N;
    if (interleaved) {
#pragma unroll
        for (int j = 0; j < N / 2; ++j) {
            rope_turn(cs[j], a[2 * j], a[2 * j + 1]);
            rope_turn(cs[N / 2 + j], b[2 * j], b[2 * j + 1]);
        }
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j) rope_turn(cs[j], a[j], b[j]);
    }
}

}  // namespace pa
