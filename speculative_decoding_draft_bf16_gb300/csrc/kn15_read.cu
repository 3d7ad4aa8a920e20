// kn15_read.cu -- reading back tokens of the paged caches, in 4 bits and in e4m3
// (dt_kv_read4, dt_kv_read).
//
// A thread turns runs of 32 elements of a token's head (two scales of the 4-bit cache) into
// bf16 or fp32; a CTA keeps to one head, whose tokens lie together in a page.
//
// Bound by HBM, mostly writes: 8 contexts of 500 to 8000 tokens of 8 heads of 128 to bf16,
// 178 MB, 30 us, 5.9 TB/s (87% of a copy's rate).  Runs of 16 took 31 us and issued in 81% of
// the clocks; one, two, four runs of 32 in flight per thread take
// 32, 30, 30 us.  Picked rows take the latency of four dependent reads: 16 requests' 129 tokens of
// e4m3 4.5 us.
#include "dt_cache.cuh"
#include "dt_launch.h"

namespace {

constexpr int NT = 256;
constexpr int U = 2;  // runs of 32 in flight per thread

DT_DI uint32_t bf16x2(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *(const uint32_t*)&v;
}
DT_DI void store32(void* p, const uint32_t (&w)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}
DT_DI void store16(void* p, const uint32_t (&w)[8]) {
    ((uint4*)p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    ((uint4*)p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
}

template <int BITS>
struct Raw {  // 32 codes and their scales
    uint4 q[BITS / 4];
    uint32_t s;  // two scale bytes, or an fp32 number's bits
    DT_DI void load(const uint8_t* codes, const void* scales, size_t slot, size_t blk, int runs, int at) {
        const uint4* p = (const uint4*)codes + (slot * runs + at) * (BITS / 4);
#pragma unroll
        for (int i = 0; i < BITS / 4; ++i) q[i] = p[i];
        s = BITS == 4 ? ((const uint16_t*)scales)[slot * runs + at] : ((const uint32_t*)scales)[blk];
    }
    // Elements 16 half .. 16 half + 15, as pairs of fp32.
    DT_DI void values(int half, float2 (&x)[8]) const {
        const uint4 w = BITS == 4 ? q[0] : q[half & (BITS / 4 - 1)];
        uint32_t h[8];
        float f;
        if constexpr (BITS == 4) {
            uint32_t lo[4], hi[4];
            dt_e2m1x8_to_f16x8(half ? w.z : w.x, lo);
            dt_e2m1x8_to_f16x8(half ? w.w : w.y, hi);
#pragma unroll
            for (int i = 0; i < 4; ++i) h[i] = lo[i], h[4 + i] = hi[i];
            f = dt_e5m3_to_f32(half ? s >> 8 : s & 255u);
        } else {
            dt_e4m3x4_to_f16x4(w.x, h[0], h[1]);
            dt_e4m3x4_to_f16x4(w.y, h[2], h[3]);
            dt_e4m3x4_to_f16x4(w.z, h[4], h[5]);
            dt_e4m3x4_to_f16x4(w.w, h[6], h[7]);
            f = __uint_as_float(s);
        }
        const float2 f2 = make_float2(f, f);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = __fmul2_rn(__half22float2(*(const __half2*)&h[i]), f2);
    }
};

// OUT: bytes of an output element.  WIDE: outputs start on 32 bytes.
template <int BITS, int OUT, bool WIDE>
__global__ void __launch_bounds__(NT, 6) kn15_kernel(const __grid_constant__ dt_kv_cache c, const int32_t* rows, int N,
                                                     const int32_t* start, const int32_t* count, int count_add,
                                                     const __grid_constant__ dt_rows ko, const __grid_constant__ dt_rows vo,
                                                     int32_t* status) {
    dt_pdl_trigger();
    dt_pdl_wait();
    const int tid = threadIdx.x, b = blockIdx.z, h = blockIdx.y >> 1;
    const bool keys = (blockIdx.y & 1) == 0;
    const int len = c.len[b], s0 = !rows && start ? start[b] : 0;
    const long long want = count ? (long long)count[b] + count_add : rows ? N : (long long)len - s0;
    const bool bad = len < 0 || (long long)len > (long long)c.max_pages * c.page || s0 < 0 || want < 0 || want > N ||
                     (!rows && s0 + want > len);
    if (bad) {
        if (blockIdx.x == 0 && blockIdx.y == 0 && tid == 0) atomicOr(&status[b], DT_DEV_BAD_CACHE);
        return;
    }
    const int n = (int)want;
    const int sh = c.D == 128 ? 2 : 1, runs = 1 << sh, run = tid & (runs - 1);  // runs of a head
    const int lp = 31 - __clz(c.page);
    const int32_t* table = c.table + (size_t)b * c.max_pages;
    const uint8_t* codes = keys ? c.k : c.v;
    const void* scales = keys ? c.k_scale : c.v_scale;
    const dt_rows& dst = keys ? ko : vo;
    char* out = (char*)dst.ptr + (b * dst.stride_b + h * dst.stride_h + run * 32) * OUT;
    const int per = NT >> sh;  // tokens of a pass
    for (int j0 = (int)blockIdx.x * U * per + (tid >> sh); j0 < n; j0 += (int)gridDim.x * U * per) {
        Raw<BITS> raw[U];
        bool off[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int j = j0 + i * per;
            off[i] = false;
            if (j < n) {
                int tok = rows ? rows[(size_t)b * N + j] : s0 + j;
                uint32_t id = 0;
                off[i] = (unsigned)tok >= (unsigned)len;
                if (!off[i]) {
                    id = (uint32_t)table[tok >> lp];
                    off[i] = id >= (uint32_t)c.n_pages;
                }
                if (!off[i]) {
                    const size_t k = (size_t)id * c.Hkv + h;
                    raw[i].load(codes, scales, (k << lp) + (tok & (c.page - 1)), k, runs, run);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int j = j0 + i * per;
            if (j >= n) continue;
            if (off[i]) atomicOr(&status[b], DT_DEV_BAD_CACHE);
            char* o = out + j * dst.stride_n * OUT;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                float2 x[8];
                raw[i].values(half, x);
#pragma unroll
                for (int part = 0; part < OUT / 2; ++part) {
                    uint32_t w[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        if (OUT == 2) w[e] = bf16x2(x[e].x, x[e].y);
                        else w[e] = __float_as_uint(e & 1 ? x[4 * part + e / 2].y : x[4 * part + e / 2].x);
                        if (off[i]) w[e] = 0u;
                    }
                    if (WIDE) store32(o + 16 * OUT * half + 32 * part, w);
                    else store16(o + 16 * OUT * half + 32 * part, w);
                }
            }
        }
    }
}

template <int BITS, int OUT, bool WIDE>
cudaError_t launch(const dt_kv_cache& c, int batch, const int32_t* rows, int N, const int32_t* start, const int32_t* count,
                   int count_add, const dt_rows& k, const dt_rows& v, int32_t* status, cudaStream_t st) {
    const int per = NT * 32 / c.D * U;  // tokens of a CTA
    DtLaunch lc(dim3((N + per - 1) / per, 2 * c.Hkv, batch), dim3(NT), 0, st);
    return cudaLaunchKernelEx(&lc.cfg, kn15_kernel<BITS, OUT, WIDE>, c, rows, N, start, count, count_add, k, v, status);
}

bool aligned32(const dt_rows& r, int size) {
    return (((uintptr_t)r.ptr | (uintptr_t)(r.stride_b * size) | (uintptr_t)(r.stride_n * size) | (uintptr_t)(r.stride_h * size)) & 31) == 0;
}

template <int BITS>
cudaError_t launch_bits(const dt_kv_cache& c, int batch, const int32_t* rows, int N, const int32_t* start, const int32_t* count,
                        int count_add, int dtype, const dt_rows& k, const dt_rows& v, int32_t* status, cudaStream_t st) {
    const int size = dtype == DT_BF16 ? 2 : 4;
    const bool wide = aligned32(k, size) && aligned32(v, size);
    auto f = dtype == DT_BF16 ? (wide ? launch<BITS, 2, true> : launch<BITS, 2, false>)
                              : (wide ? launch<BITS, 4, true> : launch<BITS, 4, false>);
    return f(c, batch, rows, N, start, count, count_add, k, v, status, st);
}

}  // namespace

cudaError_t dt_kn15_launch(const dt_kv_cache& c, int bits, int batch, const int32_t* rows, int N, const int32_t* start,
                           const int32_t* count, int count_add, int dtype, const dt_rows& k, const dt_rows& v,
                           int32_t* status, cudaStream_t st) {
    return (bits == 4 ? launch_bits<4> : launch_bits<8>)(c, batch, rows, N, start, count, count_add, dtype, k, v, status, st);
}
