// kn14_append4.cu -- rotation, quantisation to e2m1 and storing of new keys and values in
// the paged 4-bit cache (dt_kv_append4).
//
// Sixteen neighbouring elements of a head share a scale, so rows are independent of each
// other and of what their page holds.  A thread takes two blocks of 16: those that rotate
// together, or neighbours.
//   scale s = the smallest number of five exponent and three fraction bits with the
//             block's largest magnitude within 6 s;
//   codes   x / s to the nearest of e2m1.  The quotient is formed as q = x r with
//             r = 1 / s rounded, then q + (x - s q) r (Markstein's correction step).  A
//             product x r alone would miss ties, which bf16 values over 4-bit numbers hit
//             often; corrected, a quotient lies on the right side of every border: borders
//             have 3 bits and s has 4, so that x / s is either one of them exactly or more
//             than half a step of fp32 away from it.
#include "dt_cache.cuh"
#include "dt_launch.h"

namespace {

constexpr int NT = 256;

// Sixteen values to codes and the byte of their scale.
DT_DI int block4(const float (&x)[8], const float (&y)[8], uint2& codes) {
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(top) : "f"(top), "f"(fabsf(x[i])), "f"(fabsf(y[i])));
    if (!(__float_as_uint(top) < 0x7F800000u)) {  // not finite
        codes = make_uint2(0u, 0u);
        return DT_E5M3_NAN;
    }
    const int b = dt_e5m3_for(top);
    const float s = dt_e5m3_to_f32(b), r = __frcp_rn(s);
    // negative quotients, so that zeros keep their sign: m = -x r, then m - (x + s m) r
    const unsigned long long r2 = dt_f2_pack(-r, -r), s2 = dt_f2_pack(s, s);
    float p[8], q[8];
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        const unsigned long long u = dt_f2_pack(x[i], x[i + 1]), v = dt_f2_pack(y[i], y[i + 1]);
        const unsigned long long m = dt_f2_mul(u, r2), n = dt_f2_mul(v, r2);
        dt_f2_unpack(dt_f2_fma(dt_f2_fma(s2, m, u), r2, m), p[i], p[i + 1]);
        dt_f2_unpack(dt_f2_fma(dt_f2_fma(s2, n, v), r2, n), q[i], q[i + 1]);
    }
    codes = make_uint2(dt_f32x8_to_e2m1x8(p) ^ 0x88888888u, dt_f32x8_to_e2m1x8(q) ^ 0x88888888u);
    return b;
}

template <typename T>
__global__ void __launch_bounds__(NT, 2) kn14_kernel(const __grid_constant__ dt_kv_cache4 c, const __grid_constant__ dt_rope kv_rope,
                                                     int M, const __grid_constant__ dt_rows kr, const __grid_constant__ dt_rows vr,
                                                     const int32_t* rows, int N, const int32_t* count, int count_add,
                                                     int32_t* len_out, int32_t* status) {
    dt_pdl_trigger();
    dt_pdl_wait();
    const int tid = threadIdx.x, b = blockIdx.z, h = blockIdx.y >> 1;
    const bool keys = (blockIdx.y & 1) == 0;
    const int len = c.len[b];
    const long long want = count ? (long long)count[b] + count_add : N;
    const int n = want < 0 || want > N ? -1 : (int)want;
    const int* table = c.table + (size_t)b * c.max_pages;
    const long long cap = (long long)c.max_pages * c.page;
    bool bad = len < 0 || n < 0 || (long long)len + n > cap ||
               (kv_rope.rot && n > 0 && (long long)len + n > kv_rope.max_pos);
    const int lp = 31 - __clz(c.page);
    // every CTA of a request comes to the same verdict on it
    if (!bad && n > 0) {
        if (rows)
            for (int j = tid; j < n; j += NT) bad |= (unsigned)rows[(size_t)b * N + j] >= (unsigned)M;
        const int last = (len + n - 1) >> lp;
        for (int k = (len >> lp) + tid; k <= last; k += NT) bad |= (unsigned)table[k] >= (unsigned)c.n_pages;
    }
    bad = __syncthreads_or(bad);
    if (blockIdx.x == 0 && blockIdx.y == 0 && tid == 0) {
        if (len_out) len_out[b] = bad ? len : len + n;
        if (bad) atomicOr(&status[b], DT_DEV_BAD_CACHE);
    }
    if (bad) return;

    const dt_rows& src = keys ? kr : vr;
    dt_rope rope = kv_rope;
    if (!keys) rope.rot = 0;
    const T* base = (const T*)src.ptr + b * src.stride_b + h * src.stride_h;
    uint8_t* codes = keys ? c.k : c.v;
    uint8_t* scales = keys ? c.k_scale : c.v_scale;
    const int sh = c.D == 128 ? 2 : 1;        // threads per row, as a power of two
    const int p = tid & ((1 << sh) - 1);      // which pair of blocks
    const bool halves = !rope.interleaved && 32 * p < rope.rot;
    // split halves of an odd number of chunks: blocks do not rotate in pairs
    const bool odd = !rope.interleaved && (rope.rot & 31);
    for (int j = (int)blockIdx.x * (NT >> sh) + (tid >> sh); j < n; j += (int)gridDim.x * (NT >> sh)) {
        const T* row = base + (size_t)(rows ? rows[(size_t)b * N + j] : j) * src.stride_n;
        float x[2][8], y[2][8];
        int c0 = 2 * p, c1 = 2 * p + 1;  // blocks
        if (!odd) {
            DtPair<T> raw[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) raw[i].load(row, 2 * p + i, rope, len + j);
            raw[0].rotated(2 * p, rope, x[0], y[0]);
            raw[1].rotated(2 * p + 1, rope, x[1], y[1]);
            if (halves) {  // x: block p, y: its partner
                c0 = p;
                c1 = p + (rope.rot >> 5);
            } else {  // x[i], y[i]: block 2p + i
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float t = y[0][e];
                    y[0][e] = x[1][e];
                    x[1][e] = t;
                }
            }
        } else {
            DtTurned8<T> raw[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) raw[i].load(row, 4 * p + i, rope, len + j);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                raw[i].values(4 * p + i, rope, x[i]);
                raw[2 + i].values(4 * p + 2 + i, rope, y[i]);
            }
        }
        uint2 q0, q1;
        const int s0 = block4(x[0], x[1], q0), s1 = block4(y[0], y[1], q1);
        const int at = len + j;
        const size_t slot = (((size_t)table[at >> lp] * c.Hkv + h) << lp) + (at & (c.page - 1));
        uint8_t* dst = codes + slot * (c.D >> 1);
        uint8_t* sc = scales + slot * (c.D >> 4);
        if (c1 == c0 + 1) {
            *(uint4*)(dst + 8 * c0) = make_uint4(q0.x, q0.y, q1.x, q1.y);
            *(uint16_t*)(sc + c0) = (uint16_t)(s0 | s1 << 8);
        } else {
            *(uint2*)(dst + 8 * c0) = q0;
            *(uint2*)(dst + 8 * c1) = q1;
            sc[c0] = (uint8_t)s0;
            sc[c1] = (uint8_t)s1;
        }
    }
}

template <typename T>
cudaError_t launch(const dt_kv_cache4& c, const dt_rope& rope, int batch, int M, const dt_rows& k, const dt_rows& v,
                   const int32_t* rows, int N, const int32_t* count, int count_add, int32_t* len_out, int32_t* status,
                   cudaStream_t st) {
    const int per = NT * 32 / c.D;  // rows of a pass
    DtLaunch lc(dim3((N + per - 1) / per, 2 * c.Hkv, batch), dim3(NT), 0, st);
    return cudaLaunchKernelEx(&lc.cfg, kn14_kernel<T>, c, rope, M, k, v, rows, N, count, count_add, len_out, status);
}

}  // namespace

cudaError_t dt_kn14_launch(const dt_kv_cache4& c, const dt_rope& rope, int batch, int M, int dtype, const dt_rows& k,
                           const dt_rows& v, const int32_t* rows, int N, const int32_t* count, int count_add,
                           int32_t* len_out, int32_t* status, cudaStream_t st) {
    return (dtype == DT_BF16 ? launch<uint16_t> : launch<float>)(c, rope, batch, M, k, v, rows, N, count, count_add,
                                                                 len_out, status, st);
}
