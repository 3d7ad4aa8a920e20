// kn16_qk_norm.cu -- root-mean-square norms of query and key heads with the position
// rotation in the same pass (dt_qk_norm).
//
// y = R(x / sqrt(mean x^2 + eps) * w): D / 16 lanes hold a head vector, two chunks of 8
// elements each that rotate together, so the sum of squares takes a few shuffles, rotation
// none, and x is read and y written once.  A warp stays with one token and walks its heads,
// so that the token's angles are read once.
#include "dt_cache.cuh"
#include "dt_launch.h"

namespace {

constexpr int NT = 256;

DT_DI uint32_t bf16x2(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *(const uint32_t*)&v;
}
DT_DI void store8(uint16_t* p, const float (&x)[8]) {
    *(uint4*)p = make_uint4(bf16x2(x[0], x[1]), bf16x2(x[2], x[3]), bf16x2(x[4], x[5]), bf16x2(x[6], x[7]));
}
DT_DI void store8(float* p, const float (&x)[8]) {
    ((float4*)p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    ((float4*)p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}

// 1 / sqrt(mean square + eps) of a head whose lanes hold x, y.  Squares that leave fp32's
// range are formed again of numbers 2^-68 as large; such heads need no eps.
template <int PPR>
DT_DI float inverse_root(const float (&x)[8], const float (&y)[8], float eps) {
    float f = 1.f;
#pragma unroll 1
    for (int pass = 0;; ++pass) {
        float s = 0.f, t = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float u = __fmul_rn(x[i], f), v = __fmul_rn(y[i], f);
            s = __fmaf_rn(u, u, s);
            t = __fmaf_rn(v, v, t);
        }
        s = __fadd_rn(s, t);
#pragma unroll
        for (int d = 1; d < PPR; d <<= 1) s = __fadd_rn(s, __shfl_xor_sync(0xffffffffu, s, d));
        s = __fmul_rn(s, 1.f / (16 * PPR));
        // all lanes go on together
        if (pass || !__any_sync(0xffffffffu, s > 3e37f)) return __fmul_rn(rsqrtf(__fmaf_rn(eps, __fmul_rn(f, f), s)), f);
        f = s > 3e37f ? dt_pow2(-68) : 1.f;
    }
}

template <typename T, int D>
__global__ void __launch_bounds__(NT, 2) kn16_kernel(const __grid_constant__ DtNorm a) {
    constexpr int PPR = D / 16, VPW = 32 / PPR;  // lanes of a head, heads of a warp at a time
    dt_pdl_trigger();
    dt_pdl_wait();
    const int lane = threadIdx.x & 31, p = lane % PPR, sub = lane / PPR;
    const long long w = (long long)blockIdx.x * (NT / 32) + (threadIdx.x >> 5);
    const int part = (int)(w % a.parts);
    const long long token = w / a.parts;
    if (token >= (long long)a.batch * a.M) return;
    const int b = (int)(token / a.M), n = (int)(token % a.M);
    const int rows = a.n_nodes ? a.n_nodes[b] : a.M;
    const long long at = (long long)(a.len ? a.len[b] : 0) + (a.pos ? a.pos[(size_t)b * a.M + n] : n);
    if (rows < 0 || rows > a.M) {
        if (lane == 0) atomicOr(&a.status[b], DT_DEV_BAD_CACHE);
        return;
    }
    if (n >= rows) return;
    if (a.rope.rot && (at < 0 || at >= a.rope.max_pos)) {
        if (lane == 0) atomicOr(&a.status[b], DT_DEV_BAD_CACHE);
        return;
    }
    int c0, c1;
    dt_pair_chunks(p, a.rope, c0, c1);
    const int heads = a.Hq + a.Hk, per = (heads + a.parts - 1) / a.parts, end = min((part + 1) * per, heads);
    // all lanes walk together; those past the last head repeat it
    for (int h0 = part * per; h0 < end; h0 += VPW) {
        const bool live = h0 + sub < end;
        const int hh = min(h0 + sub, end - 1);
        const bool isq = hh < a.Hq;
        const int h = isq ? hh : hh - a.Hq;
        const dt_rows& src = isq ? a.q : a.k;
        const dt_rows& dst = isq ? a.q_out : a.k_out;
        const float* wt = isq ? a.q_weight : a.k_weight;
        const T* row = (const T*)src.ptr + b * src.stride_b + n * src.stride_n + h * src.stride_h;
        DtPair<T> raw;
        raw.load(row, p, a.rope, (int)at);
        float x[8], y[8];
        raw.a.values(x);
        raw.b.values(y);
        const float f = inverse_root<PPR>(x, y, a.eps);
        float g0[8], g1[8];
        if (wt) {
            wt += h * (isq ? a.q_weight_stride : a.k_weight_stride);
            DtRaw8<float> g;
            g.load(wt + 8 * c0);
            g.values(g0);
            g.load(wt + 8 * c1);
            g.values(g1);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            x[e] = __fmul_rn(x[e], f);
            y[e] = __fmul_rn(y[e], f);
            if (wt) x[e] = __fmul_rn(x[e], g0[e]), y[e] = __fmul_rn(y[e], g1[e]);
        }
        raw.turn(p, a.rope, x, y);
        if (live) {
            T* out = (T*)dst.ptr + b * dst.stride_b + n * dst.stride_n + h * dst.stride_h;
            store8(out + 8 * c0, x);
            store8(out + 8 * c1, y);
        }
    }
}

template <typename T, int D>
cudaError_t launch(DtNorm a, cudaStream_t st) {
    constexpr int VPW = 32 / (D / 16);
    const long long tokens = (long long)a.batch * a.M;
    const int most = (a.Hq + a.Hk + VPW - 1) / VPW;  // steps of a token's heads
    a.parts = tokens >= 4096 ? 1 : most;
    const long long ctas = (tokens * a.parts + NT / 32 - 1) / (NT / 32);
    if (ctas > 0x7fffffffll) return cudaErrorInvalidValue;
    DtLaunch lc(dim3((unsigned)ctas), dim3(NT), 0, st);
    return cudaLaunchKernelEx(&lc.cfg, kn16_kernel<T, D>, a);
}

}  // namespace

cudaError_t dt_kn16_launch(const DtNorm& a, cudaStream_t st) {
    if (a.dtype == DT_BF16) return a.D == 64 ? launch<uint16_t, 64>(a, st) : launch<uint16_t, 128>(a, st);
    return a.D == 64 ? launch<float, 64>(a, st) : launch<float, 128>(a, st);
}
