// dt_cache.cuh -- device helpers of the paged e4m3 cache and its rotation.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "dt_device.cuh"

// Eight elements as they are stored.
template <typename T>
struct DtRaw8;
template <>
struct DtRaw8<uint16_t> {
    uint4 v;
    DT_DI void load(const uint16_t* p) { v = *(const uint4*)p; }
    DT_DI void values(float (&x)[8]) const { dt_vec_vals<uint16_t>(v, x); }
};
template <>
struct DtRaw8<float> {
    float4 v, w;
    DT_DI void load(const float* p) { v = ((const float4*)p)[0], w = ((const float4*)p)[1]; }
    DT_DI void values(float (&x)[8]) const {
        x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w, x[4] = w.x, x[5] = w.y, x[6] = w.z, x[7] = w.w;
    }
};
// Elements 8c .. 8c+7 of a head vector, rotated to position `at` (which must lie in
// the tables): loads (no branch among them, so that several chunks' are in flight
// together) and arithmetic apart.  The partner chunk of the split-halves form is
// read again by the thread that owns it: both reads hit the same cache lines.
template <typename T>
struct DtTurned8 {
    DtRaw8<T> own, other;
    DtRaw8<float> c, s;
    DT_DI void load(const T* row, int ch, const dt_rope& r, int at) {
        const int half = r.rot >> 1;
        const bool turn = 8 * ch < r.rot;
        // where the angles are read: eight of them that lie in the row
        const int i0 = r.interleaved ? min(4 * ch, half - 8) : 8 * ch >= half ? 8 * ch - half : 8 * ch;
        const int mate = !turn || r.interleaved ? 8 * ch : 8 * ch >= half ? 8 * ch - half : 8 * ch + half;
        own.load(row + 8 * ch);
        other.load(row + mate);
        c.load(turn ? r.cos + (size_t)at * half + i0 : (const float*)row);  // else any 32 bytes
        s.load(turn ? r.sin + (size_t)at * half + i0 : (const float*)row);
    }
    DT_DI void values(int ch, const dt_rope& r, float (&x)[8]) const {
        own.values(x);
        if (8 * ch >= r.rot) return;
        float cv[8], sv[8];
        c.values(cv);
        s.values(sv);
        if (r.interleaved) {
            const bool up = 4 * ch > (r.rot >> 1) - 8;  // the angles are the last four read
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float u = x[2 * i], v = x[2 * i + 1], co = up ? cv[4 + i] : cv[i], si = up ? sv[4 + i] : sv[i];
                x[2 * i] = __fsub_rn(__fmul_rn(u, co), __fmul_rn(v, si));
                x[2 * i + 1] = __fadd_rn(__fmul_rn(v, co), __fmul_rn(u, si));
            }
        } else {
            const bool second = 8 * ch >= (r.rot >> 1);
            float y[8];
            other.values(y);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float t = __fmul_rn(y[i], sv[i]);
                x[i] = second ? __fadd_rn(__fmul_rn(x[i], cv[i]), t) : __fsub_rn(__fmul_rn(x[i], cv[i]), t);
            }
        }
    }
};

// Two chunks of 8 elements of a head vector that rotate together, index p of
// D / 16: split halves pair chunk p with chunk p + rot / 16; otherwise, and
// past rot, neighbours.  c0, c1: which chunks they are.
DT_DI void dt_pair_chunks(int p, const dt_rope& r, int& c0, int& c1) {
    const bool halves = !r.interleaved && 16 * p < r.rot;
    c0 = halves ? p : 2 * p;
    c1 = halves ? p + (r.rot >> 4) : 2 * p + 1;
}
// Both chunks and their angles, loads (no branch among them, so that those of
// several rows are in flight together) and arithmetic apart.
template <typename T>
struct DtPair {
    DtRaw8<T> a, b;
    DtRaw8<float> c, s;
    // `at` must lie in the tables.
    DT_DI void load(const T* row, int p, const dt_rope& r, int at) {
        int c0, c1;
        dt_pair_chunks(p, r, c0, c1);
        a.load(row + 8 * c0);
        b.load(row + 8 * c1);
        const bool turn = 16 * p < r.rot;  // else any 32 bytes
        const size_t o = (size_t)at * (r.rot >> 1) + 8 * p;
        c.load(turn ? r.cos + o : (const float*)row);
        s.load(turn ? r.sin + o : (const float*)row);
    }
    // The chunks as fp32, rotated.
    DT_DI void rotated(int p, const dt_rope& r, float (&x)[8], float (&y)[8]) const {
        a.values(x);
        b.values(y);
        if (16 * p >= r.rot) return;
        float cv[8], sv[8];
        c.values(cv);
        s.values(sv);
        if (r.interleaved) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float u0 = x[2 * i], u1 = x[2 * i + 1], v0 = y[2 * i], v1 = y[2 * i + 1];
                x[2 * i] = __fsub_rn(__fmul_rn(u0, cv[i]), __fmul_rn(u1, sv[i]));
                x[2 * i + 1] = __fadd_rn(__fmul_rn(u1, cv[i]), __fmul_rn(u0, sv[i]));
                y[2 * i] = __fsub_rn(__fmul_rn(v0, cv[4 + i]), __fmul_rn(v1, sv[4 + i]));
                y[2 * i + 1] = __fadd_rn(__fmul_rn(v1, cv[4 + i]), __fmul_rn(v0, sv[4 + i]));
            }
        } else {
#pragma unroll
            // products two at a time; the sums are not, or they would be contracted with them
            for (int i = 0; i < 8; i += 2) {
                const unsigned long long u = dt_f2_pack(x[i], x[i + 1]), v = dt_f2_pack(y[i], y[i + 1]);
                const unsigned long long co = dt_f2_pack(cv[i], cv[i + 1]), si = dt_f2_pack(sv[i], sv[i + 1]);
                float a0, a1, b0, b1, c0, c1, d0, d1;
                dt_f2_unpack(dt_f2_mul(u, co), a0, a1);
                dt_f2_unpack(dt_f2_mul(v, si), b0, b1);
                dt_f2_unpack(dt_f2_mul(v, co), c0, c1);
                dt_f2_unpack(dt_f2_mul(u, si), d0, d1);
                x[i] = __fsub_rn(a0, b0), x[i + 1] = __fsub_rn(a1, b1);
                y[i] = __fadd_rn(c0, d0), y[i + 1] = __fadd_rn(c1, d1);
            }
        }
    }
};

// Two e4m3 codes (the low 16 bits) as an exact fp16 pair.
DT_DI uint32_t dt_e4m3x2_to_f16x2(uint32_t codes) {
    uint32_t d;
    asm("{\n .reg .b16 t;\n cvt.u16.u32 t, %1;\n cvt.rn.f16x2.e4m3x2 %0, t;\n}\n" : "=r"(d) : "r"(codes));
    return d;
}
// Four codes as two pairs.
DT_DI void dt_e4m3x4_to_f16x4(uint32_t codes, uint32_t& lo, uint32_t& hi) {
    asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.rn.f16x2.e4m3x2 %0, l;\n cvt.rn.f16x2.e4m3x2 %1, h;\n}\n"
        : "=r"(lo), "=r"(hi)
        : "r"(codes));
}
DT_DI float2 dt_e4m3x2_to_f32x2(uint32_t codes) {
    const uint32_t h = dt_e4m3x2_to_f16x2(codes);
    return __half22float2(*(const __half2*)&h);
}
// Two fp32 values to e4m3 (to nearest, ties to even, saturating): lo in the low byte.
DT_DI uint32_t dt_f32x2_to_e4m3x2(float lo, float hi) {
    uint16_t d;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
    return d;
}

// 2^e for -126 <= e <= 127.
DT_DI float dt_pow2(int e) { return __int_as_float((e + 127) << 23); }
