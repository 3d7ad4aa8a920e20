// kn14_append4.cu -- rotation, quantisation to e2m1 and storing of new keys and values in
// the paged 4-bit cache (dt_kv_append4).
//
// Sixteen neighbouring elements of a head share a scale, so rows are independent of each
// other and of what their page holds.  A thread takes two blocks of 16: those that rotate
// together, or neighbours.
//   scale s = the smallest number of five exponent and three fraction bits with the
//             block's largest magnitude within 6 s;
//   codes   x / s to the nearest of e2m1.  The quotient is formed as q = x r with r near
//             1 / s, then q + (x - s q) r (Markstein's correction step).  A product x r
//             alone would miss ties, which bf16 values over 4-bit numbers hit often;
//             corrected, a quotient lies on the right side of every border: x - s q is
//             exact, so the sum is x / s to nearest up to 2^-21 of a step; borders have 3
//             bits and s has 4, so that x / s is either one of them exactly or more than
//             half a step of fp32 away from it.
//
// Paths take a launch and three dependent reads: 64 paths of up to 17 rows 2.7 us.  Prompts are
// bound by the rows in flight, not by issue (280 instructions for 32 elements, 44% of the
// slots; most stalls wait for loads): 8 prompts of up to
// 4000 bf16 rows, 8 heads of 128, 126 MB in all, 27.8 us, 4.5 TB/s (67% of a copy's rate);
// fp32 45.7.  Four heads to a thread share a token's angles and the checks: with one each
// 55 us.  CTAs of 128 threads start and end more evenly than of 256 (29.5 us); three of 256 to
// an SM spill (44.7); rows copied ahead through shared memory took 45.8.
#include "dt_cache.cuh"
#include "dt_launch.h"

namespace {

constexpr int NT = 128;
// CTAs with a head each from which a thread takes several: 8 prompts of 4000 rows (16128 CTAs)
// 27.8 us with four, 55 with one; fewer CTAs do not fill the GPU twice over.
constexpr int GROUP_FROM = 4096;
typedef unsigned long long f2;    // two fp32

DT_DI float rcp_near(float x) {  // within a step; x normal
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// Sixteen values to codes and the byte of their scale.
DT_DI int block4(const f2 (&x)[8], uint2& codes) {
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float a, b;
        dt_f2_unpack(x[i], a, b);
        asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(top) : "f"(top), "f"(fabsf(a)), "f"(fabsf(b)));
    }
    if (!(__float_as_uint(top) < 0x7F800000u)) {  // not finite
        codes = make_uint2(0u, 0u);
        return DT_E5M3_NAN;
    }
    const int b = dt_e5m3_for(top);
    const float s = dt_e5m3_to_f32(b), r = -rcp_near(s);
    // negative quotients, so that zeros keep their sign: m = -x r, then m - (x + s m) r
    const f2 r2 = dt_f2_pack(r, r), s2 = dt_f2_pack(s, s);
    float p[16];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const f2 m = dt_f2_mul(x[i], r2);
        dt_f2_unpack(dt_f2_fma(dt_f2_fma(s2, m, x[i]), r2, m), p[2 * i], p[2 * i + 1]);
    }
    const float lo[8] = {p[0], p[1], p[2], p[3], p[4], p[5], p[6], p[7]};
    const float hi[8] = {p[8], p[9], p[10], p[11], p[12], p[13], p[14], p[15]};
    codes = make_uint2(dt_f32x8_to_e2m1x8(lo) ^ 0x88888888u, dt_f32x8_to_e2m1x8(hi) ^ 0x88888888u);
    return b;
}

// Sixteen neighbouring elements as they are stored, and as pairs.
template <typename T>
struct Raw16 {
    DtRaw8<T> a, b;
    DT_DI void load(const T* p) {
        a.load(p);
        b.load(p + 8);
    }
    DT_DI void values(f2 (&x)[8]) const {
        float u[8], v[8];
        a.values(u);
        b.values(v);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[i] = dt_f2_pack(u[2 * i], u[2 * i + 1]);
            x[4 + i] = dt_f2_pack(v[2 * i], v[2 * i + 1]);
        }
    }
};

// Rotation of two blocks, every step rounded once: element by element with the sixteen
// angles (split halves), or of neighbours, block x with the first eight angles and y with the
// others.  Sums are fma with a factor of one: sums proper would be contracted with the products.
DT_DI void turn_blocks(f2 (&x)[8], f2 (&y)[8], const f2 (&c)[8], const f2 (&s)[8], bool halves, bool both, float one) {
    if (halves) {
        const f2 one2 = dt_f2_pack(one, one), minus = dt_f2_pack(-one, -one);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const f2 u = dt_f2_fma(dt_f2_mul(y[i], s[i]), minus, dt_f2_mul(x[i], c[i]));
            y[i] = dt_f2_fma(dt_f2_mul(x[i], s[i]), one2, dt_f2_mul(y[i], c[i]));
            x[i] = u;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float c0, c1, s0, s1, a, b;
            dt_f2_unpack(c[i >> 1], c0, c1);
            dt_f2_unpack(s[i >> 1], s0, s1);
            const float co = i & 1 ? c1 : c0, si = i & 1 ? s1 : s0;
            dt_f2_unpack(x[i], a, b);
            x[i] = dt_f2_pack(__fsub_rn(__fmul_rn(a, co), __fmul_rn(b, si)), __fadd_rn(__fmul_rn(b, co), __fmul_rn(a, si)));
        }
        if (!both) return;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float c0, c1, s0, s1, a, b;
            dt_f2_unpack(c[4 + (i >> 1)], c0, c1);
            dt_f2_unpack(s[4 + (i >> 1)], s0, s1);
            const float co = i & 1 ? c1 : c0, si = i & 1 ? s1 : s0;
            dt_f2_unpack(y[i], a, b);
            y[i] = dt_f2_pack(__fsub_rn(__fmul_rn(a, co), __fmul_rn(b, si)), __fadd_rn(__fmul_rn(b, co), __fmul_rn(a, si)));
        }
    }
}

// HG: heads that a thread takes one after the other, the next one's rows on their way.
// ODD: split halves of an odd number of chunks, whose blocks do not rotate in pairs (rare:
// one head, chunk by chunk).  `one` is 1.
template <typename T, int HG, bool ODD>
__global__ void __launch_bounds__(NT, 4) kn14_kernel(const __grid_constant__ dt_kv_cache4 c, const __grid_constant__ dt_rope kv_rope,
                                                     int M, const __grid_constant__ dt_rows kr, const __grid_constant__ dt_rows vr,
                                                     const int32_t* rows, int N, const int32_t* count, int count_add,
                                                     int32_t* len_out, int32_t* status, float one) {
    dt_pdl_trigger();
    dt_pdl_wait();
    const int tid = threadIdx.x, b = blockIdx.z, h0 = (int)(blockIdx.y >> 1) * HG, h1 = min(h0 + HG, c.Hkv);
    const bool keys = (blockIdx.y & 1) == 0;
    const int len = c.len[b];
    const long long want = count ? (long long)count[b] + count_add : N;
    const int n = want < 0 || want > N ? -1 : (int)want;
    const int* table = c.table + (size_t)b * c.max_pages;
    const long long cap = (long long)c.max_pages * c.page;
    bool bad = len < 0 || n < 0 || (long long)len + n > cap ||
               (kv_rope.rot && n > 0 && (long long)len + n > kv_rope.max_pos);
    const int lp = 31 - __clz(c.page);
    const dt_rows& src = keys ? kr : vr;
    dt_rope rope = kv_rope;
    if (!keys) rope.rot = 0;
    const int sh = c.D == 128 ? 2 : 1;        // threads per row, as a power of two
    const int p = tid & ((1 << sh) - 1);
    const bool turns = 32 * p < rope.rot, halves = !ODD && !rope.interleaved && turns;
    const bool both = 32 * p + 16 < rope.rot;
    // blocks: the p-th and its partner, or neighbours
    const int c0 = halves ? p : 2 * p, c1 = halves ? p + (rope.rot >> 5) : 2 * p + 1;
    const int j = (int)blockIdx.x * (NT >> sh) + (tid >> sh);
    // Rows are read before the verdict on the request is known (row numbers clamped), so
    // that their latency and the checks' overlap.
    const bool mine = !bad && j < n;
    const T* row = (const T*)src.ptr + b * src.stride_b + h0 * src.stride_h;
    int id = 0;
    Raw16<T> nx, ny;
    f2 co[8], si[8];
    if (mine) {
        row += (size_t)(rows ? min(max(rows[(size_t)b * N + j], 0), M - 1) : j) * src.stride_n;
        id = table[(len + j) >> lp];
        if (!ODD) {
            nx.load(row + 16 * c0);
            ny.load(row + 16 * c1);
            if (turns) {
                const size_t o = (size_t)(len + j) * (rope.rot >> 1) + 16 * p;
                const int more = halves || both ? 8 : 0;  // else the tables may end there
                Raw16<float> a;
                a.a.load(rope.cos + o);
                a.b.load(rope.cos + o + more);
                a.values(co);
                a.a.load(rope.sin + o);
                a.b.load(rope.sin + o + more);
                a.values(si);
            }
        }
    }
    // every CTA of a request comes to the same verdict on it
    if (!bad && n > 0) {
        if (rows)
            for (int k = tid; k < n; k += NT) bad |= (unsigned)rows[(size_t)b * N + k] >= (unsigned)M;
        const int last = (len + n - 1) >> lp;
        for (int k = (len >> lp) + tid; k <= last; k += NT) bad |= (unsigned)table[k] >= (unsigned)c.n_pages;
    }
    bad = __syncthreads_or(bad);
    if (blockIdx.x == 0 && blockIdx.y == 0 && tid == 0) {
        if (len_out) len_out[b] = bad ? len : len + n;
        if (bad) atomicOr(&status[b], DT_DEV_BAD_CACHE);
    }
    if (bad || !mine) return;

    const size_t slot = (((size_t)id * c.Hkv + h0) << lp) + ((len + j) & (c.page - 1));
    uint8_t* codes = (keys ? c.k : c.v) + slot * (c.D >> 1) + 8 * c0;
    uint8_t* scales = (keys ? c.k_scale : c.v_scale) + slot * (c.D >> 4) + c0;
#pragma unroll 1
    for (int h = h0;;) {
        f2 x[8], y[8];
        if (!ODD) {
            nx.values(x);
            ny.values(y);
            if (HG > 1 && h + 1 < h1) {
                row += src.stride_h;
                nx.load(row + 16 * c0);
                ny.load(row + 16 * c1);
            }
            if (turns) turn_blocks(x, y, co, si, halves, both, one);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                DtTurned8<T> raw;
                float v[8];
                raw.load(row, 4 * p + i, rope, len + j);
                raw.values(4 * p + i, rope, v);
#pragma unroll
                for (int e = 0; e < 4; ++e) (i < 2 ? x : y)[4 * (i & 1) + e] = dt_f2_pack(v[2 * e], v[2 * e + 1]);
            }
        }
        uint2 q0, q1;
        const int s0 = block4(x, q0), s1 = block4(y, q1);
        if (!halves) {
            *(uint4*)codes = make_uint4(q0.x, q0.y, q1.x, q1.y);
            *(uint16_t*)scales = (uint16_t)(s0 | s1 << 8);
        } else {
            *(uint2*)codes = q0;
            *(uint2*)(codes + 8 * (c1 - c0)) = q1;
            scales[0] = (uint8_t)s0;
            scales[c1 - c0] = (uint8_t)s1;
        }
        if (++h >= h1) break;
        codes += (size_t)c.page * (c.D >> 1);
        scales += (size_t)c.page * (c.D >> 4);
    }
}

template <typename T, int HG, bool ODD>
cudaError_t launch_hg(const dt_kv_cache4& c, const dt_rope& rope, int batch, int M, const dt_rows& k, const dt_rows& v,
                      const int32_t* rows, int N, const int32_t* count, int count_add, int32_t* len_out, int32_t* status,
                      cudaStream_t st) {
    const int per = NT * 32 / c.D;  // rows of a CTA
    DtLaunch lc(dim3((N + per - 1) / per, 2 * ((c.Hkv + HG - 1) / HG), batch), dim3(NT), 0, st);
    return cudaLaunchKernelEx(&lc.cfg, kn14_kernel<T, HG, ODD>, c, rope, M, k, v, rows, N, count, count_add, len_out, status, 1.f);
}

template <typename T>
cudaError_t launch(const dt_kv_cache4& c, const dt_rope& rope, int batch, int M, const dt_rows& k, const dt_rows& v,
                   const int32_t* rows, int N, const int32_t* count, int count_add, int32_t* len_out, int32_t* status,
                   cudaStream_t st) {
    const int per = NT * 32 / c.D;
    const long long ctas = (long long)((N + per - 1) / per) * 2 * c.Hkv * batch;
    const bool odd = !rope.interleaved && (rope.rot & 31);
    auto f = odd ? launch_hg<T, 1, true> : ctas >= GROUP_FROM ? launch_hg<T, 4, false> : launch_hg<T, 1, false>;
    return f(c, rope, batch, M, k, v, rows, N, count, count_add, len_out, status, st);
}

}  // namespace

cudaError_t dt_kn14_launch(const dt_kv_cache4& c, const dt_rope& rope, int batch, int M, int dtype, const dt_rows& k,
                           const dt_rows& v, const int32_t* rows, int N, const int32_t* count, int count_add,
                           int32_t* len_out, int32_t* status, cudaStream_t st) {
    return (dtype == DT_BF16 ? launch<uint16_t> : launch<float>)(c, rope, batch, M, k, v, rows, N, count, count_add,
                                                                 len_out, status, st);
}
