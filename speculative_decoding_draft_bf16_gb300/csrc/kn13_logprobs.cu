// kn13_logprobs.cu -- log-probability, rank, entropy and best alternatives of
// given tokens (dt_token_logprobs).
//
// One CTA per row, one pass per quantity.
#include "dt_launch.h"
#include "dt_device.cuh"

namespace {

constexpr int NT = 512;

// Order of tokens: larger logit first, then the smaller id; as one key.
template <typename T>
DT_DI unsigned long long order_key(T x, int id) {
    return (unsigned long long)DtElem<T>::key(x) << 32 | (uint32_t)~id;
}

template <typename T>
__global__ void __launch_bounds__(NT) kn13_kernel(DtLogprobs a) {
    using E = DtElem<T>;
    __shared__ float fred[NT / 32];
    __shared__ unsigned long long kred[NT / 32];
    dt_pdl_trigger();
    dt_pdl_wait();
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    const size_t e = blockIdx.x;
    const int b = (int)(e / a.N), j = (int)(e % a.N);
    const int row = a.rows ? a.rows[e] : j, tok = a.tokens[e];
    const float nan = __int_as_float(0x7FC00000);
    if (row < 0 || row >= a.M) {
        const float v = row < 0 ? 0.f : nan;
        if (tid == 0) {
            if (a.logprob) a.logprob[e] = v;
            if (a.entropy) a.entropy[e] = v;
            if (a.rank) a.rank[e] = -1;
        }
        if (tid < a.top) a.top_id[e * a.top + tid] = -1, a.top_logprob[e * a.top + tid] = v;
        return;
    }
    const T* x = (const T*)a.logits + b * a.stride_b + row * a.stride;
    auto total = [&](float v) {
        v = dt_warp_sum(v);
        __syncthreads();
        if (lane == 0) fred[w] = v;
        __syncthreads();
        float t = 0.f;
        for (int i = 0; i < NT / 32; ++i) t += fred[i];
        return t;
    };
    float m = -__int_as_float(0x7F800000);
    for (int i = tid; i < a.V; i += NT) m = fmaxf(m, E::val(x[i]));
    m = dt_warp_max(m);
    if (lane == 0) fred[w] = m;
    __syncthreads();
    for (int i = 0; i < NT / 32; ++i) m = fmaxf(m, fred[i]);
    const bool named = tok >= 0 && tok < a.V;
    const unsigned long long mine = named ? order_key<T>(x[tok], tok) : ~0ull;
    float s = 0.f, t = 0.f;
    int before = 0;
    for (int i = tid; i < a.V; i += NT) {
        const float d = E::val(x[i]) - m, p = expf(d);
        s += p;
        if (p > 0.f) t += d * p;
        before += order_key<T>(x[i], i) > mine;
    }
    s = total(s);
    t = total(t);
    before = (int)total((float)before);
    const float ln = logf(s);
    const float lse = m + ln;
    if (tid == 0) {
        if (a.logprob) a.logprob[e] = named ? E::val(x[tok]) - lse : tok < 0 ? 0.f : nan;
        if (a.entropy) a.entropy[e] = ln - t / s;
        if (a.rank) a.rank[e] = named ? before : -1;
    }
    unsigned long long last = ~0ull;
    for (int k = 0; k < a.top; ++k) {
        unsigned long long best = 0ull;
        for (int i = tid; i < a.V; i += NT) {
            const unsigned long long key = order_key<T>(x[i], i);
            if (key < last && key > best) best = key;
        }
        for (int o = 16; o > 0; o >>= 1) best = max(best, __shfl_xor_sync(0xffffffffu, best, o));
        __syncthreads();
        if (lane == 0) kred[w] = best;
        __syncthreads();
        for (int i = 0; i < NT / 32; ++i) best = max(best, kred[i]);
        last = best;
        if (tid == 0) {
            a.top_id[e * a.top + k] = (int)~(uint32_t)best;
            a.top_logprob[e * a.top + k] = E::key_val((uint32_t)(best >> 32)) - lse;
        }
    }
}

}  // namespace

cudaError_t dt_kn13_launch(const DtLogprobs& a, cudaStream_t st) {
    DtLaunch lc(dim3((unsigned)((size_t)a.batch * a.N)), dim3(NT), 0, st);
    return a.dtype == DT_BF16 ? cudaLaunchKernelEx(&lc.cfg, kn13_kernel<uint16_t>, a)
                              : cudaLaunchKernelEx(&lc.cfg, kn13_kernel<float>, a);
}
