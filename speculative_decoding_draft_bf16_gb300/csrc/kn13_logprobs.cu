// kn13_logprobs.cu -- log-probability, rank, entropy and best alternatives of
// given tokens (dt_token_logprobs).
//
// One pass over a row, by a cluster of S CTAs (S > 1 when there are few rows).
// A thread keeps, for the elements x that it has read, sums relative to a
// reference m of its own, with y = x log2(e) - m: s = sum 2^y and u = sum y 2^y.
// m is its first vectors' maximum (times log2(e), rounded) and moves only when an
// element lies more than 6 above it.  Then lse = m ln(2) + ln s and the entropy is
// ln s - ln(2) u / s, whose terms cancel in a row that is certain: they are at most
// some 6 there, and the difference is off by less than 2e-6.
//
// What concerns few elements is looked at once per 16-byte vector, by its
// maximum: elements at least as large as the token (its rank), and elements at
// least as large as a lower bound of the row's top-th best, which go to a list in
// shared memory.  The bound starts as the top-th best of the threads' maxima and rises
// when the list is cut back to its best; a round that overflows the list is read
// again with a higher bound.
//
// Rows whose largest logit is so large that only ties with it have a weight count those
// instead (see FLAT).
//
// Many rows are bound by instruction issue and HBM together: 10 instructions per bf16
// element, one of them the exponential; with 1, 5, 20 alternatives 11.3, 11.9, 14.1.  4000
// rows of 151936 bf16 logits with the best alternative: 237 us, 5.1 TB/s (76% of a copy's
// rate), fp32 401 us, 6.1 TB/s (89%); ten CTAs of 128 threads on an SM (eight: 242 us
// against 234 then; twelve spill: 276).  Few rows are bound by the latency of their phases,
// on the device: one path of 17 rows 12.8 us, 16 paths of 17 fp32 rows 18.3 us.
#include <type_traits>

#include "dt_device.cuh"
#include "dt_launch.h"

namespace {

constexpr int U = 6;                // vectors in flight per thread
constexpr int ROUND = 6;            // batches between two looks at the list
constexpr int CAP = 1024;           // list entries
// How far above its reference a thread lets an element lie.  Entropy of rows of 151936 normal
// logits with one up to 25 above the others, largest error with 20, 12, 8, 6, 4: 13, 10, 4.6,
// 2.1, 1.7e-6 (in 32 bits from the row's maximum 1.1); 4000 rows: 236.1, 236.0, 236.3, 237.5,
// 239.9 us.
constexpr float FAR = 6.f;
constexpr float LOG2E = 1.44269504088896340736f, LN2 = 0.693147180559945309417f;
// What stands for -infinity, whose exponential has to be zero and its product with it
// too, and the reference of a thread that has read nothing else.
constexpr float LOWEST = -1.7014118346046923e38f, NO_REF = -1.0e38f;  // -2^127
// A reference of this magnitude or more is too coarse: x log2(e) - m of the element it was
// taken from is 2^6 off, and beyond that its exponential underflows.  But logits so large
// lie 32 apart at least, and only ties with the row's largest have a weight: a CTA with such
// a largest reference counts them.
constexpr float FLAT = 536870912.f;  // 2^29, in base 2

typedef unsigned long long u64;

// Order of tokens: larger logit first, then the smaller id; as one key (never 0).
template <typename T>
DT_DI u64 order_key(T x, int id) {
    return (u64)DtElem<T>::key(x) << 32 | (uint32_t)~id;
}
template <typename T>
DT_DI float key_value(u64 k) {
    return DtElem<T>::key_val((uint32_t)(k >> 32));
}

// The vector with LOWEST for -infinity; NaN stays.
DT_DI uint32_t floor2(uint32_t w) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(w), "r"(0xFF00FF00u));
    return r;
}
DT_DI void finite_vals(const uint4& q, float (&x)[8]) {
    const uint4 f = make_uint4(floor2(q.x), floor2(q.y), floor2(q.z), floor2(q.w));
    dt_vec_vals<uint16_t>(f, x);
}
DT_DI void finite_vals(const uint4& q, float (&x)[4]) {
    dt_vec_vals<float>(q, x);
#pragma unroll
    for (int i = 0; i < 4; ++i) asm("max.NaN.f32 %0, %0, %1;" : "+f"(x[i]) : "f"(LOWEST));
}

struct Part {  // of a CTA, in rank 0's shared memory
    float m, s, u;
    float flat;      // beyond FLAT: its largest logit (s counts the ties), else 0
    int before, any;
    u64 top[32];
};

template <int NT>
struct Shared {
    u64 list[CAP];
    u64 scratch[NT];

    u64 bound;
    int count, kept;
    float rm[NT / 32], rs[NT / 32], ru[NT / 32];
    int rb[NT / 32];
    Part part[8];
};

template <typename T, bool TOP>
struct Row {
    using E = DtElem<T>;
    static constexpr int EV = 16 / sizeof(T);  // elements of a vector
    float m, lim;    // reference; what an element must exceed to move it
    u64 s2, u2;      // s and u, two fp32 parts each
    int before;
    float token;     // the token's logit
    typename std::conditional<sizeof(T) == 2, uint32_t, float>::type
        least_pre, least_post;  // what an element must reach to come before it, ahead of the token and
                                // after it (bf16: in both halves)
    uint32_t masks;  // bf16: sum of masks (0xFFFF in each half that comes before), since the last flush

    DT_DI bool any() const { return lim > -__int_as_float(0x7F800000); }  // a value above -infinity
    DT_DI void refer(float to) {  // the reference to `to`, which is not below it (or there are no sums)
        const float d = fminf(fmaxf(__fsub_rn(m, to), -200.f), 0.f), f = dt_ex2_approx(d);  // far: 0, with finite terms
        u2 = dt_f2_mul(dt_f2_fma(s2, dt_f2_pack(d, d), u2), dt_f2_pack(f, f));
        s2 = dt_f2_mul(s2, dt_f2_pack(f, f));
        m = to;
    }
    DT_DI void move(float x) {  // and to the element x
        // above x log2(e) by more than it is rounded, so that no exponential overflows, and
        // not below what stands for -infinity
        refer(__fmaf_rn(fabsf(x), 0x1p-22f, __fmul_rn(fmaxf(x, LOWEST), LOG2E)));
        lim = __fadd_rn(x, FAR);
    }
    DT_DI void add(float x0, float x1) {
        const u64 y = dt_f2_fma(dt_f2_pack(x0, x1), dt_f2_pack(LOG2E, LOG2E), dt_f2_pack(-m, -m));
        float y0, y1;
        dt_f2_unpack(y, y0, y1);
        const u64 e = dt_f2_pack(dt_ex2_approx(y0), dt_ex2_approx(y1));
        s2 = dt_f2_add(s2, e);
        u2 = dt_f2_fma(y, e, u2);
    }
    // A vector's sums, and how many of its elements come before the token: those
    // not smaller when they precede it, the larger ones when they follow.
    DT_DI void sums(const uint4& q, int id, int tok) {
        float x[EV];
        finite_vals(q, x);
#pragma unroll
        for (int i = 0; i < EV; i += 2) add(x[i], x[i + 1]);
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
        if ((uint32_t)(tok - id) < (uint32_t)EV) {
#pragma unroll
            for (int i = 0; i < EV; ++i) {
                const float v = sizeof(T) == 2 ? __uint_as_float((w[i >> 1] >> (16 * (i & 1))) << 16) : __uint_as_float(w[i]);
                before += i < tok - id ? v >= token : v > token;
            }
        } else if constexpr (sizeof(T) == 2) {
            const uint32_t t2 = id < tok ? least_pre : least_post;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                masks += __hge2_mask(*(const __nv_bfloat162*)&w[i], *(const __nv_bfloat162*)&t2);
        } else {
            const float t = id < tok ? least_pre : least_post;
#pragma unroll
            for (int i = 0; i < 4; ++i) before += __uint_as_float(w[i]) >= t;
        }
    }
    DT_DI void flush() {
        if (sizeof(T) == 2) {
            // with a low and b high halves set, masks = 2^16 (a - b) - a (mod 2^32); a, b < 2^16
            const uint32_t a = -masks & 0xFFFFu, b = (a - ((masks + a) >> 16)) & 0xFFFFu;
            before += (int)(a + b);
            masks = 0u;
        }
    }
};

// Lists the elements that may be among the best of the warp's vectors that hold
// such (hit): each of these in turn, an element to a lane.  id: of the vector's
// first element.  All lanes.
template <typename T, int NT>
DT_DI void list_hits(bool hit, const uint4& q, int id, Shared<NT>* sh) {
    constexpr int EV = 16 / sizeof(T);
    const int lane = threadIdx.x & 31;
    const u64 bound = sh->bound;
    for (unsigned m = __ballot_sync(0xffffffffu, hit); m; m &= m - 1) {
        const int src = __ffs(m) - 1;
        const uint32_t x = __shfl_sync(0xffffffffu, q.x, src), y = __shfl_sync(0xffffffffu, q.y, src);
        const uint32_t z = __shfl_sync(0xffffffffu, q.z, src), w = __shfl_sync(0xffffffffu, q.w, src);
        const int i = __shfl_sync(0xffffffffu, id, src) + lane, word = sizeof(T) == 2 ? lane >> 1 : lane;
        const uint32_t v = word < 2 ? (word ? y : x) : (word == 2 ? z : w);
        T t;
        if constexpr (sizeof(T) == 2) t = (T)(v >> (16 * (lane & 1)));
        else t = __uint_as_float(v);
        const u64 k = order_key<T>(t, i);
        if (lane < EV && k >= bound) {
            const int at = atomicAdd(&sh->count, 1);
            if (at < CAP) sh->list[at] = k;
        }
    }
}

// The next larger number (finite or infinite input).
DT_DI uint16_t next_up(uint16_t h) {
    if ((h & 0x7FFFu) == 0) return 1;
    return (h & 0x8000u) ? h - 1 : h + 1;
}
DT_DI float next_up(float x) {
    const uint32_t b = __float_as_uint(x);
    if ((b & 0x7FFFFFFFu) == 0) return __uint_as_float(1);
    return __uint_as_float((b & 0x80000000u) ? b - 1 : b + 1);
}

// The k best keys of the list (k <= 32) to its front, in order; the k-th becomes
// the bound when there are as many.  All threads.
template <int NT>
DT_DI void cut_list(Shared<NT>* sh, int n, int k) {
    u64 best = 0ull;
    if (n <= 128) {
        if (threadIdx.x < 32) {
            for (int i = threadIdx.x; i < n + (int)threadIdx.x; i += 32) {
                const u64 x = dt_warp_sort_reg(i < n ? sh->list[i] : 0ull, true);
                best = i < 32 ? x : dt_warp_top32_merge(best, x);
            }
        }
    } else {
        best = dt_block_top32<NT>(n, [&](int i) { return sh->list[i]; }, sh->scratch);
    }
    __syncthreads();
    if (threadIdx.x < 32) {
        if (threadIdx.x < k && threadIdx.x < n) sh->list[threadIdx.x] = best;
        if (threadIdx.x == k - 1 && n >= k) sh->bound = best;
        if (threadIdx.x == 0) sh->count = min(n, k);
    }
    __syncthreads();
}

template <typename T, bool TOP, int NT>
__global__ void __launch_bounds__(NT, NT == 128 ? 10 : 2) kn13_kernel(const __grid_constant__ DtLogprobs a, int S) {
    using E = DtElem<T>;
    using R = Row<T, TOP>;
    constexpr int EV = R::EV;
    __shared__ Shared<NT> sh;
    const float NEG_INF = -__int_as_float(0x7F800000), NaN = __int_as_float(0x7FC00000);
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    dt_pdl_wait();
    const uint32_t c = blockIdx.x % (uint32_t)S;  // rank in the row's cluster
    const uint32_t e = blockIdx.x / (uint32_t)S;
    const int b = (int)(e / (uint32_t)a.N), j = (int)(e % (uint32_t)a.N);
    const int row = a.rows ? a.rows[e] : j, tok = a.tokens[e];
    if (row < 0 || row >= a.M) {  // the whole cluster
        const float v = row < 0 ? 0.f : NaN;
        if (c == 0) {
            if (tid == 0) {
                if (a.logprob) a.logprob[e] = v;
                if (a.entropy) a.entropy[e] = v;
                if (a.rank) a.rank[e] = -1;
            }
            if (tid < a.top) a.top_id[(size_t)e * a.top + tid] = -1, a.top_logprob[(size_t)e * a.top + tid] = v;
        }
        return;
    }
    const T* x = (const T*)a.logits + b * a.stride_b + row * a.stride;
    // elements before the first 16-byte boundary and after the last vector go one by one
    const int lead = min((int)((16 - ((uintptr_t)x & 15)) & 15) / (int)sizeof(T), a.V);
    const int nvec = (a.V - lead) / EV, tail = lead + nvec * EV;
    const uint4* vec = (const uint4*)(x + lead);
    const int per = (nvec + S - 1) / S, v0 = min((int)c * per, nvec), v1 = min(v0 + per, nvec);
    const bool named = tok >= 0 && tok < a.V;

    R r;
    r.s2 = r.u2 = dt_f2_pack(0.f, 0.f);
    r.before = 0;
    r.masks = 0u;
    uint4 q[U];
    const uint4 none = sizeof(T) == 2 ? make_uint4(0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u)
                                      : make_uint4(0xFF800000u, 0xFF800000u, 0xFF800000u, 0xFF800000u);
    // a batch: vectors base + tid + i * NT
    auto fetch = [&](int base, int i) {
        const int v = base + i * NT + tid;
        q[i] = none;
        if (v < v1) q[i] = vec[v];
    };
#pragma unroll
    for (int i = 0; i < U; ++i) fetch(v0, i);
    T raw_token = (T)0;
    if (named) raw_token = x[tok];
    r.token = named ? E::val(raw_token) : __int_as_float(0x7F800000);
    if constexpr (sizeof(T) == 2) {
        const uint32_t pre = named ? raw_token : 0x7FC0u, post = named ? next_up(raw_token) : 0x7FC0u;
        r.least_pre = pre | pre << 16;  // no number reaches NaN
        r.least_post = post | post << 16;
    } else {
        r.least_pre = named ? raw_token : NaN;
        r.least_post = named ? next_up(raw_token) : NaN;
    }
    float first = NEG_INF;
#pragma unroll
    for (int i = 0; i < U; ++i) first = fmaxf(first, dt_vec_max<T>(q[i]));
    r.m = NO_REF;
    r.lim = NEG_INF;  // the first value that there is moves it
    if (first > NEG_INF) r.move(first);
    float bound_val = __int_as_float(0x7F800000);
    if (TOP) {
        if (tid == 0) sh.count = 0;
        // the bound: the top-th best of the threads' maxima, with the last id (NaN: no
        // number, a lower bound all the same)
        const u64 mine = (r.any() ? (u64)dt_fkey(first) : 0ull) << 32 | (uint32_t)tid;
        __syncthreads();
        const u64 best = dt_block_top32<NT>(NT, [&](int) { return mine; }, sh.scratch);  // asked for tid only
        if (tid == a.top - 1) {
            const uint32_t k = (uint32_t)(best >> 32);
            sh.bound = k ? order_key<T>(dt_to_elem<T>(dt_fkey_val(k)), -1) : 0ull;
        }
        __syncthreads();
        bound_val = sh.bound ? key_value<T>(sh.bound) : NEG_INF;
    }
    for (int round = v0; round < v1; round += ROUND * U * NT) {
        const int rend = min(round + ROUND * U * NT, v1);
#pragma unroll 1
        for (int base = round; base < rend; base += U * NT) {
#pragma unroll
            for (int h = 0; h < U; h += U / 2) {  // half a batch read, the next one's half on its way
#pragma unroll
                for (int i = h; i < h + U / 2; ++i) {
                    // a vector past the end is all -infinity and behind every token; the
                    // warp stays together, or it would do its sums twice
                    const int v = base + i * NT + tid;
                    const int id = v < v1 ? lead + v * EV : 0x7FFFFFFF;
                    const float vm = dt_vec_max<T>(q[i]);
                    const bool far = vm > r.lim, hit = TOP && vm >= bound_val && v < v1;
                    if (__any_sync(0xffffffffu, far || hit)) {
                        if (far) r.move(vm);
                        __syncwarp();
                        if (TOP) list_hits<T, NT>(hit, q[i], id, &sh);
                    }
                    r.sums(q[i], id, tok);
                }
#pragma unroll
                for (int i = h; i < h + U / 2; ++i) fetch(base + U * NT, i);
            }
        }
        r.flush();
        if (TOP) {
            const int kept = round == v0 ? 0 : sh.kept;
            __syncthreads();
            int n = sh.count;
            while (n > CAP) {  // this round again, with a higher bound
                const u64 was = sh.bound;
                __syncthreads();
                // the best of what the list holds bound the rest; entries from earlier rounds stay
                const u64 top = dt_block_top32<NT>(CAP, [&](int i) { return sh.list[i]; }, sh.scratch);
                __syncthreads();
                if (tid == a.top - 1) sh.bound = max(top, was);
                if (tid == 0) sh.count = kept;
                __syncthreads();
#pragma unroll 1
                for (int first_v = round; first_v < rend; first_v += NT) {
                    const int v = first_v + tid;
                    uint4 y = none;
                    if (v < rend) y = vec[v];
                    list_hits<T, NT>(v < rend && dt_vec_max<T>(y) >= key_value<T>(sh.bound), y, lead + v * EV, &sh);
                }
                __syncthreads();
                n = sh.count;
            }
            // after the first round the list's own best are a much better bound
            if (n > CAP / 2 || (round == v0 && n > a.top)) cut_list(&sh, n, a.top);
            if (tid == 0) sh.kept = sh.count;
            __syncthreads();
            bound_val = sh.bound ? key_value<T>(sh.bound) : NEG_INF;
        }
    }
    if (TOP && v0 >= v1) {
        if (tid == 0) sh.kept = 0;
        __syncthreads();
    }
    // Not before: the next grid's CTAs would take their places among this one's, on
    // some SMs more than on others.
    dt_pdl_trigger();
    // the elements outside the vectors (fewer than 2 * EV, rank 0)
    if (c == 0) {
        const int n = lead + a.V - tail;
        if (tid < n) {
            const int id = tid < lead ? tid : tail + tid - lead;
            const T raw = x[id];
            float y = E::val(raw);
            r.before += named && (id < tok ? y >= r.token : y > r.token);
            if (y > r.lim) r.move(y);
            if (y < LOWEST) y = LOWEST;
            const float d = __fmaf_rn(y, LOG2E, -r.m), ex = dt_ex2_approx(d);
            r.s2 = dt_f2_add(r.s2, dt_f2_pack(ex, 0.f));
            r.u2 = dt_f2_add(r.u2, dt_f2_pack(__fmul_rn(d, ex), 0.f));
            if (TOP) sh.list[sh.kept + tid] = order_key<T>(raw, id);  // kept <= CAP / 2
        }
        if (TOP) {
            __syncthreads();
            if (tid == 0) sh.count = sh.kept + n;
        }
    }
    __syncthreads();
    if (TOP) {
        const int n = sh.count;
        cut_list(&sh, n, a.top);
    }
    // the CTA's sums, relative to the largest reference among those with a value
    float M = r.any() ? r.m : NEG_INF;
    M = dt_warp_max(M);
    if (lane == 0) sh.rm[w] = M;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NT / 32; ++i) M = fmaxf(M, sh.rm[i]);
    const float ref = M > NEG_INF ? M : 0.f;
    // a thread without a value has sums of zeros, or NaN
    float sa, sb, ua, ub;
    dt_f2_unpack(r.s2, sa, sb);
    r.refer(r.any() || sa != sa || sb != sb ? ref : r.m);
    dt_f2_unpack(r.s2, sa, sb);
    dt_f2_unpack(r.u2, ua, ub);
    const float s = dt_warp_sum(__fadd_rn(sa, sb)), u = dt_warp_sum(__fadd_rn(ua, ub));
    const int before = dt_warp_sum_i(r.before);
    if (lane == 0) sh.rs[w] = s, sh.ru[w] = u, sh.rb[w] = before;
    __syncthreads();
    cg::cluster_group cluster = cg::this_cluster();
    Part* to = S > 1 ? cluster.map_shared_rank(&sh.part[c], 0) : &sh.part[0];
    if (S > 1) cluster.sync();  // rank 0 runs before others write to it
    if (tid == 0) {
        float ss = 0.f, uu = 0.f;
        int bb = 0;
        for (int i = 0; i < NT / 32; ++i) ss += sh.rs[i], uu += sh.ru[i], bb += sh.rb[i];
        to->m = ref;
        to->s = ss;
        to->u = uu;
        to->flat = 0.f;
        to->before = bb;
        to->any = M > NEG_INF;
    }
    if (fabsf(M) >= FLAT && M > NEG_INF) {  // (all threads) the largest logit, and how many there are of it
        float flat = 0.f, ties = 0.f;
        for (int pass = 0; pass < 2; ++pass) {
            float best = NEG_INF, n = 0.f;
            auto look = [&](T raw) {
                const float y = E::val(raw);
                best = fmaxf(best, y);
                n += y != y || y == __int_as_float(0x7F800000) ? NaN : y == flat ? 1.f : 0.f;  // no figures, as elsewhere
            };
#pragma unroll 1
            for (const T* p = (const T*)(vec + v0) + tid; p < (const T*)(vec + v1); p += NT) look(*p);
            if (c == 0 && tid < lead) look(x[tid]);
            if (c == 0 && tid < a.V - tail) look(x[tail + tid]);
            const float part = pass ? dt_warp_sum(n) : dt_warp_max(best);
            __syncthreads();  // rm has been read
            if (lane == 0) sh.rm[w] = part;
            __syncthreads();
            if (pass == 0) flat = sh.rm[0];
#pragma unroll 1
            for (int i = 0; i < NT / 32; ++i) {
                if (pass) ties += sh.rm[i];
                else flat = fmaxf(flat, sh.rm[i]);
            }
        }
        if (tid == 0) to->s = ties, to->u = 0.f, to->flat = flat;
    }
    if (TOP && tid < 32) to->top[tid] = tid < sh.count ? sh.list[tid] : 0ull;
    if (S > 1) cluster.sync();
    else __syncthreads();
    if (c != 0 || w != 0) return;
    // rank 0's first warp: the CTAs' parts in their order
    float m = NEG_INF, X = NEG_INF;
    bool any = false;
    for (int i = 0; i < S; ++i) {
        if (sh.part[i].any) m = fmaxf(m, sh.part[i].m);
        any |= sh.part[i].any != 0;
    }
    const bool flat_row = any && fabsf(m) >= FLAT;
    if (flat_row) {
        for (int i = 0; i < S; ++i)
            if (sh.part[i].flat != 0.f) X = fmaxf(X, sh.part[i].flat);
    }
    float ts = 0.f, tu = 0.f;
    int tb = 0;
    for (int i = 0; i < S; ++i) {
        const Part& p = sh.part[i];
        tb += p.before;
        const float d = p.any && any ? fmaxf(p.m - m, -200.f) : 0.f;
        const float f = flat_row ? (p.flat == X ? 1.f : 0.f) : dt_ex2_approx(d);
        tu = __fmaf_rn(__fmaf_rn(p.s, d, p.u), f, tu);
        ts = __fmaf_rn(p.s, f, ts);
    }
    const float ln = logf(ts);
    const float lse = any ? __fmaf_rn(m, LN2, ln) : NaN;
    // in a flat row the difference from the largest logit comes first, or it would absorb the logarithm
    auto logprob_of = [&](float y) { return flat_row ? (y - X) - ln : y - lse; };
    if (lane == 0) {
        if (a.logprob) a.logprob[e] = named ? logprob_of(r.token) : tok < 0 ? 0.f : NaN;
        const float h = flat_row ? ln : __fmaf_rn(-LN2, tu / ts, ln);
        if (a.entropy) a.entropy[e] = !any ? NaN : h < 0.f ? 0.f : h;  // rounding alone takes it below 0
        if (a.rank) a.rank[e] = named ? tb : -1;
    }
    if (TOP) {
        u64 best = sh.part[0].top[lane];
        for (int i = 1; i < S; ++i) best = dt_warp_top32_merge(best, sh.part[i].top[lane]);
        if (lane < a.top) {
            a.top_id[(size_t)e * a.top + lane] = (int)~(uint32_t)best;
            a.top_logprob[(size_t)e * a.top + lane] = logprob_of(key_value<T>(best));
        }
    }
}

template <typename T, int NT>
cudaError_t launch(const DtLogprobs& a, int S, cudaStream_t st) {
    const unsigned rows = (unsigned)((size_t)a.batch * a.N);
    DtLaunch lc(dim3(rows * S), dim3(NT), 0, st, S > 1 ? S : 0);
    return a.top > 0 ? cudaLaunchKernelEx(&lc.cfg, kn13_kernel<T, true, NT>, a, S)
                     : cudaLaunchKernelEx(&lc.cfg, kn13_kernel<T, false, NT>, a, S);
}

}  // namespace

cudaError_t dt_kn13_launch(const DtLogprobs& a, cudaStream_t st) {
    // A cluster per row while rows alone leave SMs idle (two CTAs of 512 threads fit an
    // SM), with two vectors at least for every thread (one row of 151936 bf16: 8 CTAs;
    // 17 rows by one CTA each 17.5 us, by 8 each 12.5).
    const long long rows = (long long)a.batch * a.N;
    const long long bytes = (long long)a.V * (a.dtype == DT_BF16 ? 2 : 4);
    int S = 1;
    while (S < 8 && rows * S < 2 * 152 && bytes >= (long long)S * 2 * 512 * 16 * 2) S *= 2;
    // Many rows: few threads to a row, so that what a row costs once is spread over
    // more of its vectors.  Measured, bf16, 128 threads against 512: 304 rows of 32000
    // 13.7 : 13.6 us, 456 rows 15.2 : 19.7; of 151936, 456 rows 48.9 : 44.0, 608 rows
    // 54.7 : 55.2, 2432 rows 151 : 202; of 262144, 760 rows 98 : 95, 912 rows 110 : 111.
    if (rows >= 256 + bytes / 800)
        return a.dtype == DT_BF16 ? launch<uint16_t, 128>(a, S, st) : launch<float, 128>(a, S, st);
    return a.dtype == DT_BF16 ? launch<uint16_t, 512>(a, S, st) : launch<float, 512>(a, S, st);
}
