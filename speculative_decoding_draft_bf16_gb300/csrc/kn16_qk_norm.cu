// kn16_qk_norm.cu -- root-mean-square norms of query and key heads with the position
// rotation in the same pass (dt_qk_norm).
//
// y = R(x / sqrt(mean x^2 + eps) * w): D / 16 lanes hold a head vector, two chunks of 8
// elements each that rotate together, so the sum of squares takes a few shuffles, rotation
// none, and x is read and y written once.  A warp walks the heads of a token, queries'
// first, so that the token's angles and the kind's weights are read once; steps of a few
// heads are loaded while those before them are worked on.
//
// Bound by HBM: eight prompts of up to 4000 rows, 40 heads of 128 in bf16, 504 MB, 86 us, 5.9
// TB/s (87% of a copy's rate); 4112 rows of 32 heads in fp32 with weights of each head, 102
// MB, 23 us.  64 single tokens take 2.4 us, a launch and two dependent reads.  Persistent
// warps that copied rows ahead through shared memory took 91 us: the bookkeeping of such a
// queue costs more instructions (260 a step) than the rows in flight gain.
#include "dt_cache.cuh"
#include "dt_launch.h"

namespace {

constexpr int NT = 128;
constexpr int CTAS = 4;   // per SM: five or six take 91 to 94 us where four take 87
// Units of work per warp from which tokens are cut no further: with fewer units than warps
// the SMs idle, with more the angles are read more often (4112 rows of fp32: 1, 2, 8 units
// 27.8, 23.3, 30.3 us; 3904 short bf16 rows 12.4, 12.6, 20.6).
constexpr int UNITS = 2;

DT_DI uint32_t bf16x2(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *(const uint32_t*)&v;
}
DT_DI void store8(uint16_t* p, const float2 (&x)[4]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = bf16x2(x[i].x, x[i].y);
    *(uint4*)p = make_uint4(w[0], w[1], w[2], w[3]);
}
DT_DI void store8(float* p, const float2 (&x)[4]) {
    ((float4*)p)[0] = make_float4(x[0].x, x[0].y, x[1].x, x[1].y);
    ((float4*)p)[1] = make_float4(x[2].x, x[2].y, x[3].x, x[3].y);
}

typedef float2 f2;
DT_DI f2 mul2(f2 a, f2 b) { return __fmul2_rn(a, b); }
DT_DI f2 fma2(f2 a, f2 b, f2 c) { return __ffma2_rn(a, b, c); }
DT_DI f2 add2(f2 a, f2 b) { return __fadd2_rn(a, b); }

// Eight values as pairs.
DT_DI void pairs(const float (&x)[8], f2 (&p)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = make_float2(x[2 * i], x[2 * i + 1]);
}
// Mean square over a head's PPR lanes, D = 16 PPR elements, of them or (SMALL) of 2^-68 times them.
template <int PPR, bool SMALL>
DT_DI float mean_square(const f2 (&x)[4], const f2 (&y)[4]) {
    const f2 k = make_float2(dt_pow2(-68), dt_pow2(-68));
    f2 s = make_float2(0.f, 0.f), t = s;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const f2 u = SMALL ? mul2(x[i], k) : x[i], v = SMALL ? mul2(y[i], k) : y[i];
        s = fma2(u, u, s);
        t = fma2(v, v, t);
    }
    s = add2(s, t);
    float r = __fadd_rn(s.x, s.y);
#pragma unroll
    for (int d = 1; d < PPR; d <<= 1) r = __fadd_rn(r, __shfl_xor_sync(0xffffffffu, r, d));
    return __fmul_rn(r, 1.f / (16 * PPR));
}
// 1 / sqrt(mean square + eps).  Squares that leave fp32's range upwards are formed again of
// numbers 2^-68 as large, with eps 2^-136 as large.  With an eps below TINY squares may leave it
// downwards, too: the head itself is scaled then, by 2^100, and eps by 2^200, because the root's
// reciprocal of the smallest numbers would leave the range and its product with them does not.
// Only one step at a time does that, and both ends alike: 3904 short rows take 10.7 us with it and
// 10.9 without, but the prompts above, two steps at a time, 86 without and 89 to 92 with it.
constexpr float TINY = 1e-30f;
template <int PPR, int U>
DT_DI float inverse_root(f2 (&x)[4], f2 (&y)[4], float eps) {
    const float s = __fadd_rn(mean_square<PPR, false>(x, y), eps);
    const bool big = s > 3e37f, tiny = U == 1 && s < TINY;
    if (__any_sync(0xffffffffu, big || tiny)) {  // all lanes go on together
        if (U == 1) {
            const float k = big ? dt_pow2(-68) : tiny ? dt_pow2(100) : 1.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[i] = mul2(x[i], make_float2(k, k));
                y[i] = mul2(y[i], make_float2(k, k));
            }
            return rsqrtf(__fadd_rn(mean_square<PPR, false>(x, y), __fmul_rn(__fmul_rn(eps, k), k)));
        }
        const float t = mean_square<PPR, true>(x, y);
        if (big) return __fmul_rn(rsqrtf(__fadd_rn(t, __fmul_rn(__fmul_rn(eps, dt_pow2(-68)), dt_pow2(-68)))), dt_pow2(-68));
    }
    return rsqrtf(s);
}

// A token's angles for a lane's chunk pair; n: minus the sines.
struct Angles {
    f2 c[4], s[4], n[4];
    DT_DI void load(const dt_rope& r, int p, int at) {
        const size_t o = (size_t)at * (r.rot >> 1) + 8 * p;
        DtRaw8<float> raw;
        float x[8];
        raw.load(r.cos + o);
        raw.values(x);
        pairs(x, c);
        raw.load(r.sin + o);
        raw.values(x);
        pairs(x, s);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = -x[i];
        pairs(x, n);
    }
    DT_DI void turn(bool interleaved, f2 (&x)[4], f2 (&y)[4]) const {
        if (!interleaved) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const f2 u = fma2(x[i], c[i], mul2(y[i], n[i]));
                y[i] = fma2(y[i], c[i], mul2(x[i], s[i]));
                x[i] = u;
            }
        } else {  // both elements of a pair in one f2; x has the first four angles
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                f2& z = i < 2 ? x[2 * i] : y[2 * i - 4];
                f2& w = i < 2 ? x[2 * i + 1] : y[2 * i - 3];
                z = make_float2(__fmaf_rn(z.x, c[i].x, -__fmul_rn(z.y, s[i].x)), __fmaf_rn(z.y, c[i].x, __fmul_rn(z.x, s[i].x)));
                w = make_float2(__fmaf_rn(w.x, c[i].y, -__fmul_rn(w.y, s[i].y)), __fmaf_rn(w.y, c[i].y, __fmul_rn(w.x, s[i].y)));
            }
        }
    }
};

template <typename T>
DT_DI void load_pairs(const T* p, f2 (&x)[4]) {
    DtRaw8<T> raw;
    float v[8];
    raw.load(p);
    raw.values(v);
    pairs(v, x);
}

// One kind of heads (queries or keys) of a token: steps [s0, s1) of VPW heads, U of them
// loaded while the U before them are worked on.
template <typename T, int PPR, int U>
DT_DI void run_heads(const T* in, long long in_stride, T* out, long long out_stride, int H, const float* w, int w_stride,
                     int s0, int s1, int sub, int c0, int c1, float eps, const Angles& angles, bool turns, bool interleaved) {
    constexpr int VPW = 32 / PPR;
    DtRaw8<T> a[U], b[U];
    int h = s0 * VPW + sub;
    const T* src = in + h * in_stride;
    auto load = [&](int i) {
        if (h + i * VPW < H) {
            a[i].load(src + i * VPW * in_stride + c0);
            b[i].load(src + i * VPW * in_stride + c1);
        }
    };
#pragma unroll
    for (int i = 0; i < U; ++i)
        if (s0 + i < s1) load(i);
    T* dst = out + h * out_stride;
    f2 g0[4], g1[4];
    const f2 ones = make_float2(1.f, 1.f);
#pragma unroll
    for (int i = 0; i < 4; ++i) g0[i] = g1[i] = ones;
    if (w && !w_stride) {
        load_pairs(w + c0, g0);
        load_pairs(w + c1, g1);
    }
#pragma unroll 1
    for (int s = s0; s < s1; s += U) {  // all lanes walk together
        f2 x[U][4], y[U][4];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            float u[8], v[8];
            a[i].values(u);
            b[i].values(v);
            pairs(u, x[i]);
            pairs(v, y[i]);
        }
        const int now = h;
        h += U * VPW;
        src += U * VPW * in_stride;
#pragma unroll
        for (int i = 0; i < U; ++i)
            if (s + U + i < s1) load(i);
#pragma unroll
        for (int i = 0; i < U; ++i) {
            if (s + i >= s1) break;
            const float f = inverse_root<PPR, U>(x[i], y[i], eps);
            const f2 ff = make_float2(f, f);
            if (w_stride && now + i * VPW < H) {
                load_pairs(w + (now + i * VPW) * w_stride + c0, g0);
                load_pairs(w + (now + i * VPW) * w_stride + c1, g1);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                x[i][e] = mul2(mul2(x[i][e], ff), g0[e]);
                y[i][e] = mul2(mul2(y[i][e], ff), g1[e]);
            }
            if (turns) angles.turn(interleaved, x[i], y[i]);
            if (now + i * VPW < H) {
                store8(dst + c0, x[i]);
                store8(dst + c1, y[i]);
            }
            dst += VPW * out_stride;
        }
    }
}

// U: steps loaded at a time.
template <typename T, int D, int U>
__global__ void __launch_bounds__(NT, CTAS) kn16_kernel(const __grid_constant__ DtNorm a) {
    constexpr int PPR = D / 16;  // lanes of a head
    dt_pdl_trigger();
    dt_pdl_wait();
    const int lane = threadIdx.x & 31, p = lane % PPR, sub = lane / PPR;
    const uint32_t unit = blockIdx.x * (NT / 32) + (threadIdx.x >> 5), token = unit / (uint32_t)a.parts;
    const int part = (int)(unit - token * a.parts), b = (int)(token / (uint32_t)a.M), n = (int)(token - b * (uint32_t)a.M);
    if (b >= a.batch) return;
    const int rows = a.n_nodes ? a.n_nodes[b] : a.M;
    const long long pos = (long long)(a.len ? a.len[b] : 0) + (a.pos ? a.pos[(size_t)b * a.M + n] : n);
    const bool off = rows < 0 || rows > a.M || (n < rows && a.rope.rot && (pos < 0 || pos >= a.rope.max_pos));
    if (off && lane == 0) atomicOr(&a.status[b], DT_DEV_BAD_CACHE);
    if (off || n >= rows) return;
    int c0, c1;
    dt_pair_chunks(p, a.rope, c0, c1);
    c0 *= 8, c1 *= 8;
    const bool turns = 16 * p < a.rope.rot;
    Angles angles;
    if (turns) angles.load(a.rope, p, (int)pos);
    const int s0 = part * a.per, s1 = min(s0 + a.per, a.q_steps + a.k_steps);
    if (s0 < a.q_steps)
        run_heads<T, PPR, U>((const T*)a.q.ptr + b * a.q.stride_b + n * a.q.stride_n, a.q.stride_h,
                             (T*)a.q_out.ptr + b * a.q_out.stride_b + n * a.q_out.stride_n, a.q_out.stride_h, a.Hq, a.q_weight,
                             a.q_weight_stride, s0, min(s1, a.q_steps), sub, c0, c1, a.eps, angles, turns, a.rope.interleaved);
    if (s1 > a.q_steps)
        run_heads<T, PPR, U>((const T*)a.k.ptr + b * a.k.stride_b + n * a.k.stride_n, a.k.stride_h,
                             (T*)a.k_out.ptr + b * a.k_out.stride_b + n * a.k_out.stride_n, a.k_out.stride_h, a.Hk, a.k_weight,
                             a.k_weight_stride, max(s0 - a.q_steps, 0), s1 - a.q_steps, sub, c0, c1, a.eps, angles, turns,
                             a.rope.interleaved);
}

template <typename T, int D, int U>
cudaError_t launch_u(const DtNorm& a, unsigned ctas, cudaStream_t st) {
    DtLaunch lc(dim3(ctas), dim3(NT), 0, st);
    return cudaLaunchKernelEx(&lc.cfg, kn16_kernel<T, D, U>, a);
}

template <typename T, int D>
cudaError_t launch(DtNorm a, int sms, cudaStream_t st) {
    constexpr int VPW = 32 / (D / 16);
    const long long tokens = (long long)a.batch * a.M, warps = CTAS * sms * (NT / 32);
    a.q_steps = (a.Hq + VPW - 1) / VPW;
    a.k_steps = (a.Hk + VPW - 1) / VPW;
    const int most = a.q_steps + a.k_steps;
    a.parts = 1;
    while (a.parts < most && tokens * a.parts < UNITS * warps) a.parts *= 2;
    a.parts = a.parts < most ? a.parts : most;
    a.per = (most + a.parts - 1) / a.parts;
    const long long units = tokens * a.parts, need = (units + NT / 32 - 1) / (NT / 32);
    // whole tokens: two steps at a time (the prompts 86 us, one at a time 89); parts of
    // tokens have few steps (3904 short rows 12.6 us with two, 10.7 with one), and an eps below
    // TINY needs one at a time
    return (a.parts == 1 && a.eps >= TINY ? launch_u<T, D, 2> : launch_u<T, D, 1>)(a, (unsigned)need, st);
}

}  // namespace

cudaError_t dt_kn16_launch(const DtNorm& a, int sms, cudaStream_t st) {
    if (a.dtype == DT_BF16) return a.D == 64 ? launch<uint16_t, 64>(a, sms, st) : launch<uint16_t, 128>(a, sms, st);
    return a.D == 64 ? launch<float, 64>(a, sms, st) : launch<float, 128>(a, sms, st);
}
