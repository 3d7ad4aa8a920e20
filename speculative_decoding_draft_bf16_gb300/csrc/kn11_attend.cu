// kn11_attend.cu -- tree attention over the paged e4m3 cache (dt_tree_attention).
//
// One warp per query row: the lanes share the head's elements, keys come one
// at a time, with a running maximum and sum.  fp32 throughout.
#include "dt_cache.cuh"
#include "dt_launch.h"

namespace {

constexpr int NW = 4;  // warps (query rows) per CTA

template <int D>
__global__ void __launch_bounds__(NW * 32) kn11_kernel(DtAttend a) {
    constexpr int E = D / 32;  // elements per lane
    __shared__ float vec[NW][2][D];
    dt_pdl_trigger();
    dt_pdl_wait();
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int b = blockIdx.z, h = blockIdx.y, n = blockIdx.x * NW + w;
    if (n >= a.M) return;
    const dt_kv_cache& c = a.c;
    const int kh = h / (a.G);
    uint16_t* out = (uint16_t*)a.out + (((size_t)b * a.M + n) * a.Hq + h) * D + lane * E;
    int len = c.len[b], rows = a.n_nodes ? a.n_nodes[b] : a.M;
    bool bad = len < 0 || (long long)len > (long long)c.max_pages * c.page || rows < 0 || rows > a.M;
    if (bad) len = rows = 0;
    float acc[E] = {}, m_run = -__int_as_float(0x7F800000), l_run = 0.f;
    float q[E], x[8];

    // a new row's vector (rotated when it is a query or key) by way of shared memory
    auto fetch = [&](const dt_rows& r, int row, int head, bool turn, float (&o)[E]) {
        const uint16_t* p = (const uint16_t*)r.ptr + b * r.stride_b + row * r.stride_n + head * r.stride_h;
        if (lane < D / 8) {
            int at = 0;
            dt_rope rope = a.rope;
            if (!turn) rope.rot = 0;
            if (rope.rot) {
                at = len + (a.pos ? a.pos[(size_t)b * a.M + row] : row);
                if (at < 0 || at >= rope.max_pos) bad = true, at = 0;
            }
            dt_rotated8(p, lane, rope, at, x);
            for (int i = 0; i < 8; ++i) vec[w][turn][lane * 8 + i] = isfinite(x[i]) ? x[i] : __int_as_float(0x7FC00000);
        }
        __syncwarp();
        for (int i = 0; i < E; ++i) o[i] = vec[w][turn][lane * E + i];
        __syncwarp();
    };
    auto add = [&](const float (&k)[E], const float (&v)[E], float ks, float vs) {
        float s = 0.f;
        for (int i = 0; i < E; ++i) s = fmaf(q[i], k[i], s);
        s = dt_warp_sum(s) * ks * a.scale;
        const float m = fmaxf(m_run, s);
        const float f = m_run == m ? 1.f : expf(m_run - m), p = expf(s - m);
        for (int i = 0; i < E; ++i) acc[i] = fmaf(acc[i], f, p * (v[i] * vs));
        l_run = fmaf(l_run, f, p);
        m_run = m;
    };
    if (n < rows) {
        fetch(a.q, n, h, true, q);
        for (int j = 0; j < len; ++j) {
            int page = c.table[(size_t)b * c.max_pages + j / c.page];
            if ((unsigned)page >= (unsigned)c.n_pages) bad = true, page = 0;
            const size_t blk = (size_t)page * c.Hkv + kh;
            const size_t off = (blk * c.page + j % c.page) * D + lane * E;
            float k[E], v[E];
            for (int i = 0; i < E; i += 2) {
                const float2 kf = dt_e4m3x2_to_f32x2(*(const uint16_t*)(c.k + off + i));
                const float2 vf = dt_e4m3x2_to_f32x2(*(const uint16_t*)(c.v + off + i));
                k[i] = kf.x, k[i + 1] = kf.y, v[i] = vf.x, v[i + 1] = vf.y;
            }
            add(k, v, c.k_scale[blk], c.v_scale[blk]);
        }
        const int words = (a.M + 31) / 32;
        for (int m = 0; m < rows; ++m) {
            const bool sees = a.mask ? (a.mask[((size_t)b * a.M + n) * words + m / 32] >> (m % 32)) & 1 : m <= n;
            if (!sees) continue;
            float k[E], v[E];
            fetch(a.k, m, kh, true, k);
            fetch(a.v, m, kh, false, v);
            // a value that is not finite makes the whole row NaN
            bool odd = false;
            for (int i = 0; i < E; ++i) odd |= k[i] != k[i] || v[i] != v[i];
            if (__any_sync(0xffffffffu, odd)) k[0] = __int_as_float(0x7FC00000);
            add(k, v, 1.f, 1.f);
        }
    }
    for (int i = 0; i < E; ++i) {
        const __nv_bfloat16 o = __float2bfloat16_rn(l_run == 0.f ? 0.f : acc[i] / l_run);
        out[i] = *(const uint16_t*)&o;
    }
    if (__any_sync(0xffffffffu, bad) && lane == 0) atomicOr(&a.status[b], DT_DEV_BAD_CACHE);
}

}  // namespace

cudaError_t dt_kn11_launch(const DtAttend& a, cudaStream_t st) {
    DtLaunch lc(dim3((a.M + NW - 1) / NW, a.Hq, a.batch), dim3(NW * 32), 0, st);
    return a.c.D == 64 ? cudaLaunchKernelEx(&lc.cfg, kn11_kernel<64>, a) : cudaLaunchKernelEx(&lc.cfg, kn11_kernel<128>, a);
}
