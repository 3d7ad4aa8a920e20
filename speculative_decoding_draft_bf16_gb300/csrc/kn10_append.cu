// kn10_append.cu -- rotation, e4m3 quantisation and storing of new keys and
// values in the paged cache (dt_kv_append).
//
// One CTA per (page touched, key head, keys or values, request): the block
// that shares a scale.  Its new rows stay in registers between the two things
// that need them: the largest magnitude, which fixes the scale 2^e, and the
// codes x / 2^e.  Rows read once, codes written once.
//
// A path's few rows cost a launch and the latency of three dependent reads (lengths,
// rows, tables' ids): 2.6 us for 4 paths, 5 us for 64.  Prompts are bound by how many
// rows are in flight: 8 prompts of up to 4000 bf16 rows, 160 MB, 37 us, 4.3 TB/s (64% of
// a copy's rate), instructions issued in three of four clocks.  Rows read before the
// verdict on the request, in pairs of chunks that rotate together, took 66 us to 43, four
// CTAs per SM (64 registers) to 39, steps of two elements to 37; five CTAs spill (50 us),
// 512 threads to a block leave them idle at short pages (50 us).
#include "dt_cache.cuh"
#include "dt_launch.h"

namespace {

constexpr int NT = 256;
constexpr int E_MIN = -48;  // smallest exponent of a block scale

// Exponent of the scale for a block whose largest magnitude has these bits
// (finite): the smallest e >= E_MIN with amax <= 448 * 2^e, 448 = 1.75 * 2^8.
DT_DI int block_exponent(uint32_t amax_bits) {
    const int x = (int)(amax_bits >> 23) - 127;
    const int e = ((amax_bits & 0x7FFFFFu) <= 0x600000u) ? x - 8 : x - 7;
    return max(e, E_MIN);
}

// Smallest e with scale <= 2^e (scale positive, finite, normal).
DT_DI int scale_exponent(float scale) {
    const uint32_t b = __float_as_uint(scale);
    return (int)(b >> 23) - 127 + ((b & 0x7FFFFFu) ? 1 : 0);
}

// The codes of eight values, scaled.
DT_DI uint2 codes8(const float (&x)[8], float inv) {
    const unsigned long long f = dt_f2_pack(inv, inv);
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float lo, hi;
        dt_f2_unpack(dt_f2_mul(dt_f2_pack(x[2 * i], x[2 * i + 1]), f), lo, hi);
        c[i] = dt_f32x2_to_e4m3x2(lo, hi);
    }
    return make_uint2(__byte_perm(c[0], c[1], 0x5410), __byte_perm(c[2], c[3], 0x5410));
}

// The largest of three numbers, NaN if one is.
DT_DI float max3_nan(float a, float b, float c) {
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// CP: pairs of 8-element chunks a thread may own (four, with rows in flight, take 114 registers).
template <typename T, int CP>
__global__ void __launch_bounds__(NT, CP > 2 ? 2 : 4) kn10_kernel(const __grid_constant__ dt_kv_cache c, const __grid_constant__ dt_rope kv_rope,
                                                  int M, const __grid_constant__ dt_rows kr, const __grid_constant__ dt_rows vr,
                                                  const int32_t* rows, int N, const int32_t* count, int count_add,
                                                  int32_t* len_out, int32_t* status) {
    __shared__ uint32_t red[NT / 32];
    dt_pdl_trigger();
    dt_pdl_wait();
    const int tid = threadIdx.x, b = blockIdx.z, h = blockIdx.y;
    const bool keys = (blockIdx.x & 1) == 0;
    const int at = blockIdx.x >> 1;  // page touched, counted from the first one
    const int len = c.len[b];
    const long long want = count ? (long long)count[b] + count_add : N;
    const int n = want < 0 || want > N ? -1 : (int)want;
    const int* table = c.table + (size_t)b * c.max_pages;
    const long long cap = (long long)c.max_pages * c.page;
    bool bad = len < 0 || n < 0 || (long long)len + n > cap ||
               (kv_rope.rot && n > 0 && (long long)len + n > kv_rope.max_pos);
    const int lp = 31 - __clz(c.page), p = bad ? 0 : (len >> lp) + at;
    const int lo = bad ? 0 : max(len, p << lp), hi = bad ? 0 : min(len + n, (p + 1) << lp);  // slots of new rows
    const bool mine = lo < hi;
    const dt_rows& src = keys ? kr : vr;
    dt_rope rope = kv_rope;
    if (!keys) rope.rot = 0;
    // The rows are read before the verdict on the request is known (row numbers
    // clamped), so that their latency and the checks' overlap.
    const int ppr = c.D >> 4, sh = c.D == 128 ? 3 : 2;  // chunk pairs per row
    const int m = mine ? (hi - lo) << sh : 0;
    float x[CP][8], y[CP][8];
    constexpr int U = CP < 2 ? 1 : 2;  // rows in flight
#pragma unroll
    for (int i0 = 0; i0 < CP; i0 += U) {
        DtPair<T> raw[U];
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int q = tid + (i0 + k) * NT, j = lo - len + (q >> sh);
            if (q < m) {
                const int row = rows ? min(max(rows[(size_t)b * N + j], 0), M - 1) : j;
                raw[k].load((const T*)src.ptr + b * src.stride_b + row * src.stride_n + h * src.stride_h, q & (ppr - 1),
                            rope, len + j);
            }
        }
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int q = tid + (i0 + k) * NT;
            if (q < m) raw[k].rotated(q & (ppr - 1), rope, x[i0 + k], y[i0 + k]);
        }
    }
    // every CTA of a request comes to the same verdict on it
    int id = 0;
    if (!bad && n > 0) {
        if (rows)
            for (int j = tid; j < n; j += NT) bad |= (unsigned)rows[(size_t)b * N + j] >= (unsigned)M;
        const int last = (len + n - 1) >> lp;
        for (int k = (len >> lp) + tid; k <= last; k += NT) bad |= (unsigned)table[k] >= (unsigned)c.n_pages;
        if (mine) id = table[p];
    }
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < CP; ++i) {
        if (tid + i * NT < m) {
#pragma unroll
            for (int e = 0; e < 8; ++e) top = max3_nan(top, fabsf(x[i][e]), fabsf(y[i][e]));
        }
    }
    // as bits: NaN above infinity above the rest
    uint32_t amax = __reduce_max_sync(0xffffffffu, __float_as_uint(top));
    if ((tid & 31) == 0) red[tid >> 5] = amax;
    bad = __syncthreads_or(bad);
    if (blockIdx.x == 0 && h == 0 && tid == 0) {
        if (len_out) len_out[b] = bad ? len : len + n;
        if (bad) atomicOr(&status[b], DT_DEV_BAD_CACHE);
    }
    if (bad || !mine) return;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) amax = max(amax, red[w]);

    const size_t blk = (size_t)id * c.Hkv + h;
    float* scale = (keys ? c.k_scale : c.v_scale) + blk;
    uint8_t* codes = (keys ? c.k : c.v) + ((blk << lp) * c.D);
    const int first = lo - (p << lp);  // slot of the first new row
    int e = amax < 0x7F800000u ? block_exponent(amax) : 0;
    bool nan = amax >= 0x7F800000u;
    float old = 1.f;
    if (first > 0) {  // the block holds older tokens
        old = *scale;
        if (old > 0.f && old <= dt_pow2(120)) e = max(e, scale_exponent(old));
        else nan = true;  // also a scale above any that a finite value gives
        __syncthreads();  // every thread has read the scale
    }
    if (tid == 0) *scale = nan ? __int_as_float(0x7FC00000) : dt_pow2(e);
    const float inv = dt_pow2(-e);  // -e in [-120, 48]
#pragma unroll
    for (int i = 0; i < CP; ++i) {
        const int q = tid + i * NT;
        if (q < m) {
            int c0, c1;
            dt_pair_chunks(q & (ppr - 1), rope, c0, c1);
            uint8_t* dst = codes + (first + (q >> sh)) * c.D;
            const uint2 u = codes8(x[i], inv), v = codes8(y[i], inv);
            if (c1 == c0 + 1) {
                *(uint4*)(dst + 8 * c0) = make_uint4(u.x, u.y, v.x, v.y);
            } else {
                *(uint2*)(dst + 8 * c0) = u;
                *(uint2*)(dst + 8 * c1) = v;
            }
        }
    }
    if (first > 0 && !nan && dt_pow2(e) != old) {  // older codes to the larger scale
        const float f = __fmul_rn(old, inv);
        for (int q = tid; q < first * c.D / 4; q += NT) {
            const uint32_t w = ((const uint32_t*)codes)[q];
            const float2 a = dt_e4m3x2_to_f32x2(w & 0xFFFFu), d = dt_e4m3x2_to_f32x2(w >> 16);
            ((uint32_t*)codes)[q] = dt_f32x2_to_e4m3x2(__fmul_rn(a.x, f), __fmul_rn(a.y, f)) |
                                    dt_f32x2_to_e4m3x2(__fmul_rn(d.x, f), __fmul_rn(d.y, f)) << 16;
        }
    }
}

template <typename T, int CP>
cudaError_t launch(const dt_kv_cache& c, const dt_rope& rope, int batch, int M, const dt_rows& k, const dt_rows& v,
                   const int32_t* rows, int N, const int32_t* count, int count_add, int32_t* len_out, int32_t* status,
                   cudaStream_t st) {
    const int touched = (N + c.page - 2) / c.page + 1;  // pages that N rows may touch
    DtLaunch lc(dim3(2 * touched, c.Hkv, batch), dim3(NT), 0, st);
    return cudaLaunchKernelEx(&lc.cfg, kn10_kernel<T, CP>, c, rope, M, k, v, rows, N, count, count_add, len_out,
                              status);
}

template <typename T>
cudaError_t launch_ch(const dt_kv_cache& c, const dt_rope& rope, int batch, int M, const dt_rows& k, const dt_rows& v,
                      const int32_t* rows, int N, const int32_t* count, int count_add, int32_t* len_out,
                      int32_t* status, cudaStream_t st) {
    // chunk pairs of a block that new rows can fill, per thread
    const int most = ((N < c.page ? N : c.page) * (c.D / 16) + NT - 1) / NT;
    auto f = most <= 1 ? launch<T, 1> : most <= 2 ? launch<T, 2> : launch<T, 4>;
    return f(c, rope, batch, M, k, v, rows, N, count, count_add, len_out, status, st);
}

}  // namespace

cudaError_t dt_kn10_launch(const dt_kv_cache& c, const dt_rope& rope, int batch, int M, int dtype, const dt_rows& k,
                           const dt_rows& v, const int32_t* rows, int N, const int32_t* count, int count_add,
                           int32_t* len_out, int32_t* status, cudaStream_t st) {
    return (dtype == DT_BF16 ? launch_ch<uint16_t> : launch_ch<float>)(c, rope, batch, M, k, v, rows, N, count,
                                                                       count_add, len_out, status, st);
}
