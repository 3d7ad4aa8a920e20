// kn12_attend_tc.cu -- tree attention on the tensor cores, for many query rows
// per key head (dt_tree_attention).
//
// A CTA works on a block of up to 256 query rows (two slots of 128, the rows of
// an MMA) and a run of 128-token tiles:
//   converter warps  read e4m3 codes (or new rows, which they rotate) into
//                    registers and write exact fp16 tiles, 128-byte swizzled, to
//                    shared memory: keys K-major, values MN-major -- the same
//                    physical layout, so neither is transposed;
//   MMA warp         S = Q K^T (128 x 128 per slot) and O += P V, accumulators
//                    in tensor memory, P read from tensor memory;
//   softmax warps    one thread per row: row maximum, exponentials, P in fp16
//                    over the columns of S it has read, and the rescaling of O.
// While one slot's softmax runs, the other slot's products do.  A block of at
// most 128 rows puts the same rows in both slots, which then take every other
// tile and are joined at the end.
//
// Scales.  A tile has a key scale ks and a value scale vs for each 16 tokens.
// Scores in base 2 are t = s * (row factor * ks); P holds p = 2^(t + log2 vs - m),
// so the products need no scaling, and the row sum adds p / vs.  m is the running
// maximum of t + log2 vs less 5 (fp16 then resolves probabilities down to 2^-29 of
// the largest), moved -- and O rescaled -- only when the maximum has grown by
// more than 8 since.
#include "dt_attend.cuh"
#include "dt_tcgen05.cuh"

namespace {

constexpr int ROWS = 256;       // query rows of a block
constexpr int TQ = 128;         // rows of a slot
constexpr int NS = 256;         // softmax threads
constexpr int NC = 128;         // converter threads
constexpr int NT = NS + NC + 32;
constexpr int STAGES = 2;       // K and V tiles in shared memory, each
constexpr int RING = 4;         // tiles whose scales are kept
constexpr int ATOM = 4;         // tiles of the longest unit that is not split
constexpr int MIN_SHARE = 4;    // least cost worth a CTA: two tiles of a full block
constexpr float LOG2E = 1.44269504088896340736f;
constexpr float HEADROOM = 5.f, LAZY = 8.f;

struct Ring {
    float ks[8], lv[8], iv[8];  // key scale, log2 and inverse of the value scale per 16 tokens
    uint32_t bad[4];            // new rows with a value that is not finite
};

struct Shared {
    uint64_t kfull[STAGES], kfree[STAGES], vfull[STAGES], vfree[STAGES];
    uint64_t sfull[2], pfull[2], ofull[2], qfull, scfull[RING];
    uint32_t tmem;
    int fail, last;
    AtShare share;
    Ring ring[RING];
    float qscale[ROWS];
    float mrg_m[TQ], mrg_l[TQ];
    uint32_t amax[2][NC / 32];
};

template <int D>
struct Lay {
    static constexpr int TILE = AT_TILE * D * 2;  // bytes of an fp16 tile
    static constexpr int HALF = AT_TILE * 128;    // bytes of 64 elements of every row
    static constexpr int Q = 0, K = 2 * TILE, V = K + STAGES * TILE, SH = V + STAGES * TILE;
    static constexpr size_t SMEM = 1024 + SH + sizeof(Shared);
};

// Bounded wait; once one has run out, later ones return at once.
DT_DI void wait(uint64_t* bar, uint32_t phase, int* fail) {
    if (*(volatile int*)fail) return;
    if (!dt_mbar_wait(bar, phase)) *(volatile int*)fail = 1;
}

// 32-bit pair of fp16 from two fp32 (lo in the low half).
DT_DI uint32_t f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
DT_DI float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// Byte offset of the 16-byte chunk c (8 fp16) of row r in a tile of D columns.
DT_DI uint32_t chunk_at(int r, int c) {
    return (uint32_t)((c >> 3) * (AT_TILE * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}
DT_DI void sts16(uint32_t addr, const uint32_t (&w)[4]) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
                 : "memory");
}

// Sixteen e4m3 codes to two fp16 chunks 2 * pc, 2 * pc + 1 of row r.  The lanes
// of the upper 64 columns store their odd chunk first: the eight lanes of a
// store phase then hit eight different 16-byte columns.
template <int D>
DT_DI void store_codes(uint32_t tile, int r, int pc, const uint4& q) {
    uint32_t a[4], b[4];
    a[0] = dt_e4m3x2_to_f16x2(q.x), a[1] = dt_e4m3x2_to_f16x2(q.x >> 16);
    a[2] = dt_e4m3x2_to_f16x2(q.y), a[3] = dt_e4m3x2_to_f16x2(q.y >> 16);
    b[0] = dt_e4m3x2_to_f16x2(q.z), b[1] = dt_e4m3x2_to_f16x2(q.z >> 16);
    b[2] = dt_e4m3x2_to_f16x2(q.w), b[3] = dt_e4m3x2_to_f16x2(q.w >> 16);
    const bool odd = D == 128 && pc >= 4;
    uint32_t f[4], s[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = odd ? b[i] : a[i], s[i] = odd ? a[i] : b[i];
    sts16(tile + chunk_at(r, 2 * pc + odd), f);
    sts16(tile + chunk_at(r, 2 * pc + !odd), s);
}

// log2 of a positive normal number, and its inverse: exact for powers of two.
DT_DI void scale_parts(float s, float& lg, float& inv) {
    lg = log2f(s);
    inv = 1.0f / s;
}

template <int D>
struct Conv {  // the converter warps
    static constexpr int PPT = D / 16;        // 16-byte pieces of a token's codes
    static constexpr int TPI = NC / PPT;      // tokens per iteration
    static constexpr int NI = AT_TILE / TPI;  // iterations per tile
    using L = Lay<D>;

    // page ids of the tokens this thread reads of tile j (-1: none)
    static DT_DI void pages(const DtAttend& a, const AtWalk<ROWS, ATOM>& u, int lp, int j, int ct, int (&id)[NI]) {
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int tok = j * AT_TILE + i * TPI + ct / PPT;
            int p = -1;
            if (tok < u.r.len) {
                p = a.c.table[(size_t)u.b * a.c.max_pages + (tok >> lp)];
                if ((unsigned)p >= (unsigned)a.c.n_pages) {
                    atomicOr(&a.status[u.b], DT_DEV_BAD_CACHE);
                    p = 0;
                }
            }
            id[i] = p;
        }
    }
    static DT_DI void codes(const DtAttend& a, const AtWalk<ROWS, ATOM>& u, const uint8_t* base, int lp, int j, int ct,
                            const int (&id)[NI], uint4 (&q)[NI]) {
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int tok = j * AT_TILE + i * TPI + ct / PPT;
            q[i] = make_uint4(0u, 0u, 0u, 0u);
            if (id[i] >= 0) {
                const size_t row = (((size_t)id[i] * a.c.Hkv + u.h) << lp) + (tok & ((1 << lp) - 1));
                q[i] = *(const uint4*)(base + row * D + (ct % PPT) * 16);
            }
        }
    }
    static DT_DI void store(uint32_t tile, int ct, const uint4 (&q)[NI]) {
#pragma unroll
        for (int i = 0; i < NI; ++i) store_codes<D>(tile, i * TPI + ct / PPT, ct % PPT, q[i]);
        dt_fence_proxy_async_smem();
    }
    // scales of group ct (< 8) of tile j
    static DT_DI void scales(const DtAttend& a, const AtWalk<ROWS, ATOM>& u, int lp, int j, int ct, float& ks, float& vs) {
        const int tok = j * AT_TILE + ct * 16;
        ks = vs = 1.f;
        if (ct < 8 && tok < u.r.len) {
            int p = a.c.table[(size_t)u.b * a.c.max_pages + (tok >> lp)];
            if ((unsigned)p >= (unsigned)a.c.n_pages) p = 0;
            ks = a.c.k_scale[(size_t)p * a.c.Hkv + u.h];
            vs = a.c.v_scale[(size_t)p * a.c.Hkv + u.h];
        }
    }

    // One tile of new rows, from row m0: keys rotated, both scaled by a power of
    // two when their largest magnitude leaves fp16's comfortable range.
    static DT_DI void fresh(const DtAttend& a, const AtWalk<ROWS, ATOM>& u, int m0, int ct, Shared* sh, Ring* ring,
                            uint32_t kt, uint32_t vt, int stage, uint32_t kfree_ph, uint32_t vfree_ph, uint64_t* scfull) {
        constexpr int CPR = D / 8;  // chunks per row
        const int left = min(AT_TILE, u.r.n - m0);
        const uint16_t* kp = (const uint16_t*)a.k.ptr + u.b * a.k.stride_b + u.h * a.k.stride_h;
        const uint16_t* vp = (const uint16_t*)a.v.ptr + u.b * a.v.stride_b + u.h * a.v.stride_h;
        if (ct < 4) ring->bad[ct] = 0u;
        asm volatile("bar.sync 1, 128;" ::: "memory");
        uint32_t big[2] = {0u, 0u};
        float x[8];
        for (int i = ct; i < left * CPR; i += NC) {
            const int m = m0 + i / CPR, c = i % CPR;
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                if (w == 0)
                    dt_rotated8(kp + m * a.k.stride_n, c, a.rope, at_position(a, u.b, u.r.len, m), x);
                else
                    dt_load8(vp + m * a.v.stride_n + 8 * c, x);
                bool bad = false;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const uint32_t v = __float_as_uint(x[e]) & 0x7FFFFFFFu;
                    if (v >= 0x7F800000u) bad = true;
                    else big[w] = max(big[w], v);
                }
                if (bad) atomicOr(&ring->bad[(m - m0) >> 5], 1u << ((m - m0) & 31));
            }
        }
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            big[w] = dt_warp_max_u32(big[w]);
            if ((ct & 31) == 0) sh->amax[w][ct >> 5] = big[w];
        }
        asm volatile("bar.sync 1, 128;" ::: "memory");
        int ex[2];
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            uint32_t v = 0;
            for (int i = 0; i < NC / 32; ++i) v = max(v, sh->amax[w][i]);
            // as they are in [2^-4, 2^15), else scaled to below 2^9; none or very small: 2^-57
            const int e = (int)(v >> 23) - 127;
            ex[w] = e >= -4 && e < 15 ? 0 : max(e - 8, -57);
        }
        if (ct < 8) {
            ring->ks[ct] = dt_pow2(ex[0]);
            ring->lv[ct] = (float)ex[1];
            ring->iv[ct] = dt_pow2(-ex[1]);
        }
        dt_mbar_arrive(scfull);
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            wait(w == 0 ? &sh->kfree[stage] : &sh->vfree[stage], w == 0 ? kfree_ph : vfree_ph, &sh->fail);
            const float f = dt_pow2(-ex[w]);
            for (int i = ct; i < AT_TILE * CPR; i += NC) {
                const int r = i / CPR, c = i % CPR;
                uint32_t o[4] = {0u, 0u, 0u, 0u};
                if (r < left) {
                    if (w == 0)
                        dt_rotated8(kp + (m0 + r) * a.k.stride_n, c, a.rope, at_position(a, u.b, u.r.len, m0 + r), x);
                    else
                        dt_load8(vp + (m0 + r) * a.v.stride_n + 8 * c, x);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        x[e] = (__float_as_uint(x[e]) & 0x7FFFFFFFu) >= 0x7F800000u ? 0.f : __fmul_rn(x[e], f);
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[e] = f16x2(x[2 * e], x[2 * e + 1]);
                }
                sts16((w == 0 ? kt : vt) + chunk_at(r, c), o);
            }
            dt_fence_proxy_async_smem();
            dt_mbar_arrive(w == 0 ? &sh->kfull[stage] : &sh->vfull[stage]);
        }
    }

    static DT_DI void run(const DtAttend& a, unsigned char* sm, Shared* sh, int ct, int cta) {
        const int lp = 31 - __clz(a.c.page);
        const uint32_t kt = dt_smem_addr(sm + L::K), vt = dt_smem_addr(sm + L::V);
        AtWalk<ROWS, ATOM> u;
        u.start(a, sh->share);
        uint32_t g = 0;  // tiles done
        for (; u.next(a, sh->share, cta); u.step(a)) {
            uint4 kq[NI], vq[NI];
            int id[NI];
            float ks, vs;
            const int cend = min(u.t1, u.r.ctx);
            int j = u.t0;
            if (j < cend) {
                pages(a, u, lp, j, ct, id);
                codes(a, u, a.c.k, lp, j, ct, id, kq);
                codes(a, u, a.c.v, lp, j, ct, id, vq);
                scales(a, u, lp, j, ct, ks, vs);
                if (j + 1 < cend) pages(a, u, lp, j + 1, ct, id);
            }
            for (; j < cend; ++j, ++g) {
                const int s = g % STAGES;
                const uint32_t free_ph = (g / STAGES + 1) & 1;
                Ring* ring = &sh->ring[g % RING];
                wait(&sh->kfree[s], free_ph, &sh->fail);
                if (ct < 8) {
                    ring->ks[ct] = ks;
                    scale_parts(vs, ring->lv[ct], ring->iv[ct]);
                }
                dt_mbar_arrive(&sh->scfull[g % RING]);
                store(kt + s * L::TILE, ct, kq);
                dt_mbar_arrive(&sh->kfull[s]);
                const bool more = j + 1 < cend;
                if (more) {
                    codes(a, u, a.c.k, lp, j + 1, ct, id, kq);
                    scales(a, u, lp, j + 1, ct, ks, vs);
                }
                wait(&sh->vfree[s], free_ph, &sh->fail);
                store(vt + s * L::TILE, ct, vq);
                dt_mbar_arrive(&sh->vfull[s]);
                if (more) {
                    codes(a, u, a.c.v, lp, j + 1, ct, id, vq);
                    if (j + 2 < cend) pages(a, u, lp, j + 2, ct, id);
                }
            }
            for (; j < u.t1; ++j, ++g) {
                const int s = g % STAGES;
                const uint32_t free_ph = (g / STAGES + 1) & 1;
                wait(&sh->kfree[s], free_ph, &sh->fail);  // and so the ring's slot
                fresh(a, u, (j - u.r.ctx) * AT_TILE, ct, sh, &sh->ring[g % RING], kt + s * L::TILE, vt + s * L::TILE,
                      s, free_ph, free_ph, &sh->scfull[g % RING]);
            }
        }
    }
};

// The MMA warp's one thread.
template <int D>
DT_DI void issue_all(const DtAttend& a, unsigned char* sm, Shared* sh, uint32_t tmem, int cta) {
    using L = Lay<D>;
    constexpr uint32_t ID_S = dt_idesc_f16_f32(TQ, AT_TILE, false), ID_O = dt_idesc_f16_f32(TQ, D, true);
    const uint32_t qb = dt_smem_addr(sm + L::Q), kb = dt_smem_addr(sm + L::K), vb = dt_smem_addr(sm + L::V);
    AtWalk<ROWS, ATOM> u;
    u.start(a, sh->share);
    uint32_t g0 = 0, seg = 0, pc[2] = {0u, 0u};
    for (; u.next(a, sh->share, cta); u.step(a), ++seg) {
        const bool dual = u.rows > TQ;  // two slots of rows; else two slots of tiles
        const int nt = u.t1 - u.t0;
        wait(&sh->qfull, seg & 1, &sh->fail);
        auto qk = [&](int s, int lt) {
            const uint32_t g = g0 + lt, st = g % STAGES;
            wait(&sh->kfull[st], (g / STAGES) & 1, &sh->fail);
            dt_tc_fence_after();
            const uint32_t q = qb + (dual ? s : 0) * L::TILE, k = kb + st * L::TILE;
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                const uint32_t o = (kk >> 2) * L::HALF + (kk & 3) * 32;
                dt_mma_bf16(tmem + s * AT_TILE, dt_desc_kmajor_sw128(q + o), dt_desc_kmajor_sw128(k + o), ID_S, kk > 0);
            }
            dt_mma_commit(&sh->sfull[s]);
            if (!dual || s == 1) dt_mma_commit(&sh->kfree[st]);
        };
        auto pv = [&](int s, int lt, bool first, bool last) {
            const uint32_t g = g0 + lt, st = g % STAGES;
            wait(&sh->pfull[s], pc[s]++ & 1, &sh->fail);
            wait(&sh->vfull[st], (g / STAGES) & 1, &sh->fail);
            dt_tc_fence_after();
            const uint32_t v = vb + st * L::TILE;
#pragma unroll
            for (int kk = 0; kk < AT_TILE / 16; ++kk)
                dt_mma_f16_ts(tmem + 2 * AT_TILE + s * D, tmem + s * AT_TILE + kk * 8,
                              dt_desc_mnmajor_sw128(v + kk * 2048, L::HALF), ID_O, !first || kk > 0);
            if (!dual || s == 1) dt_mma_commit(&sh->vfree[st]);
            if (last) dt_mma_commit(&sh->ofull[s]);
        };
        const int hop = dual ? 1 : 2;
        qk(0, 0);
        if (dual) qk(1, 0);
        else if (nt > 1) qk(1, 1);
        for (int lt = 0; lt < nt; lt += hop) {
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const int t = dual ? lt : lt + s;
                if (t < nt) {
                    pv(s, t, lt == 0, t + hop >= nt);
                    if (t + hop < nt) qk(s, t + hop);
                }
            }
        }
        g0 += nt;
    }
}

// A slot's softmax: 128 threads, one per row.
template <int D>
struct Soft {
    using L = Lay<D>;

    // The block's rows, rotated, scaled by a power of two and converted.
    static DT_DI void queries(const DtAttend& a, const AtWalk<ROWS, ATOM>& u, unsigned char* sm, Shared* sh, int tid) {
        constexpr int CPR = D / 8, RPI = NS / CPR;
        const int G = a.Hq / a.c.Hkv;
        const int tiles = u.rows > TQ ? 2 : 1;
        const uint32_t qb = dt_smem_addr(sm + L::Q);
        const int c = tid % CPR;
        for (int r = tid / CPR; r < tiles * TQ; r += RPI) {
            float x[8] = {};
            if (r < u.rows) {
                const long long row = (long long)u.qb * ROWS + r;
                const int n = (int)(row / G), h = u.h * G + (int)(row % G);
                const uint16_t* p = (const uint16_t*)a.q.ptr + u.b * a.q.stride_b + n * a.q.stride_n + h * a.q.stride_h;
                dt_rotated8(p, c, a.rope, at_position(a, u.b, u.r.len, n), x);
            }
            uint32_t big = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) big = max(big, __float_as_uint(x[e]) & 0x7FFFFFFFu);
#pragma unroll
            for (int o = CPR / 2; o > 0; o >>= 1) big = max(big, __shfl_xor_sync(0xffffffffu, big, o));
            int ex = (int)(big >> 23) - 127;  // largest magnitude in [2^ex, 2^(ex+1))
            ex = big >= 0x7F800000u ? 0 : max(ex, -100);
            const float f = dt_pow2(-ex);
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = f16x2(__fmul_rn(x[2 * e], f), __fmul_rn(x[2 * e + 1], f));
            sts16(qb + (r / TQ) * L::TILE + chunk_at(r % TQ, c), w);
            if (c == 0) sh->qscale[r] = __fmul_rn(__fmul_rn(a.scale, LOG2E), dt_pow2(ex));
        }
        dt_fence_proxy_async_smem();
        dt_mbar_arrive(&sh->qfull);
    }

    // The row's mask words of a tile that is not wholly visible.
    static DT_DI void mask_words(const DtAttend& a, const AtWalk<ROWS, ATOM>& u, int t, int row, uint32_t (&mk)[4]) {
        const int G = a.Hq / a.c.Hkv;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (t < u.r.ctx) {
                const int left = u.r.len - t * AT_TILE - 32 * i;
                mk[i] = left >= 32 ? 0xFFFFFFFFu : left <= 0 ? 0u : (1u << left) - 1u;
            } else {
                const long long rr = (long long)u.qb * ROWS + row;
                mk[i] = row < u.rows ? at_mask_word(a, u.b, (int)(rr / G), (t - u.r.ctx) * AT_TILE + 32 * i, u.r.n) : 0u;
            }
        }
    }

    static DT_DI void run(const DtAttend& a, unsigned char* sm, Shared* sh, uint32_t tmem, int tid, int cta, int ctas,
                          float* part, int* counters) {
        const int s = tid / TQ, w4 = (tid >> 5) & 3;
        const float NEG_INF = -__int_as_float(0x7F800000);
        const uint32_t lanes = (uint32_t)(w4 * 32) << 16;
        const uint32_t ts = tmem + s * AT_TILE + lanes, to = tmem + 2 * AT_TILE + s * D + lanes;
        AtWalk<ROWS, ATOM> u;
        u.start(a, sh->share);
        uint32_t g0 = 0, seg = 0, sc = 0, oc = 0;
        for (; u.next(a, sh->share, cta); u.step(a), ++seg) {
            const bool dual = u.rows > TQ;
            const int nt = u.t1 - u.t0;
            const int row = dual ? tid : tid % TQ;  // within the block
            // every product of the last segment has read its queries
            asm volatile("bar.sync 2, 256;" ::: "memory");
            queries(a, u, sm, sh, tid);
            asm volatile("bar.sync 2, 256;" ::: "memory");
            const float rowc = sh->qscale[row];
            float m = NEG_INF, l = 0.f;
            bool poison = false;
            for (int lt = dual ? 0 : s; lt < nt; lt += dual ? 1 : 2) {
                const uint32_t g = g0 + lt;
                const Ring* ring = &sh->ring[g % RING];
                wait(&sh->sfull[s], sc++ & 1, &sh->fail);
                wait(&sh->scfull[g % RING], (g / RING) & 1, &sh->fail);
                __syncwarp();
                dt_tc_fence_after();
                const int t = u.t0 + lt;
                const bool masked = (t + 1) * AT_TILE > u.r.len;
                uint32_t mk[4] = {0xFFFFFFFFu, 0xFFFFFFFFu, 0xFFFFFFFFu, 0xFFFFFFFFu};
                if (masked) {
                    mask_words(a, u, t, row, mk);
                    if (t >= u.r.ctx) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) poison |= (mk[i] & ring->bad[i]) != 0u;
                    }
                }
                // pass 1: the largest score
                float mx = NEG_INF;
                uint32_t v[2][32];
                dt_tmem_ld32_async(ts, v[0]);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    dt_tmem_ld_wait(v[c & 1]);
                    if (c < 3) dt_tmem_ld32_async(ts + 32 * (c + 1), v[(c + 1) & 1]);
                    uint32_t(&x)[32] = v[c & 1];
                    if (masked) {
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (!((mk[c] >> i) & 1)) x[i] = __float_as_uint(NEG_INF);
                    }
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float q = __uint_as_float(x[16 * h]);
#pragma unroll
                        for (int i = 1; i < 15; i += 2)
                            q = max3(q, __uint_as_float(x[16 * h + i]), __uint_as_float(x[16 * h + i + 1]));
                        q = fmaxf(q, __uint_as_float(x[16 * h + 15]));
                        mx = fmaxf(mx, __fmaf_rn(q, __fmul_rn(rowc, ring->ks[2 * c + h]), ring->lv[2 * c + h]));
                    }
                }
                // a maximum that has grown moves the reference; rows of a warp do so together
                const bool grown = mx > m + (HEADROOM + LAZY);
                if (__any_sync(0xffffffffu, grown)) {
                    const float to_m = grown ? mx - HEADROOM : m;
                    const float f = grown ? dt_ex2_approx(m - to_m) : 1.f;  // m = -inf: 0
                    m = to_m;
                    l = __fmul_rn(l, f);
                    if (lt >= (dual ? 1 : 2)) {  // there is something in O
#pragma unroll
                        for (int c = 0; c < D / 32; ++c) {
                            dt_tmem_ld32_async(to + 32 * c, v[0]);
                            dt_tmem_ld_wait(v[0]);
#pragma unroll
                            for (int i = 0; i < 32; ++i) v[0][i] = __float_as_uint(__fmul_rn(__uint_as_float(v[0][i]), f));
                            dt_tmem_st32(to + 32 * c, v[0]);
                        }
                    }
                }
                const float mu = m == NEG_INF ? 0.f : m;
                // pass 2: probabilities, over the columns already read
                dt_tmem_ld32_async(ts, v[0]);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    dt_tmem_ld_wait(v[c & 1]);
                    if (c < 3) dt_tmem_ld32_async(ts + 32 * (c + 1), v[(c + 1) & 1]);
                    uint32_t(&x)[32] = v[c & 1];
                    if (masked) {
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (!((mk[c] >> i) & 1)) x[i] = __float_as_uint(NEG_INF);
                    }
                    uint32_t p[16];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float ka = __fmul_rn(rowc, ring->ks[2 * c + h]), kb = __fsub_rn(ring->lv[2 * c + h], mu);
                        const unsigned long long ka2 = dt_f2_pack(ka, ka), kb2 = dt_f2_pack(kb, kb);
                        unsigned long long sum = dt_f2_pack(0.f, 0.f);
#pragma unroll
                        for (int i = 0; i < 16; i += 2) {
                            float e0, e1;
                            dt_f2_unpack(dt_f2_fma(dt_f2_pack(__uint_as_float(x[16 * h + i]), __uint_as_float(x[16 * h + i + 1])),
                                                   ka2, kb2), e0, e1);
                            e0 = dt_ex2_approx(e0);
                            e1 = dt_ex2_approx(e1);
                            sum = dt_f2_add(sum, dt_f2_pack(e0, e1));
                            p[8 * h + i / 2] = f16x2(e0, e1);
                        }
                        float s0, s1;
                        dt_f2_unpack(sum, s0, s1);
                        l = __fmaf_rn(__fadd_rn(s0, s1), ring->iv[2 * c + h], l);
                    }
                    dt_tmem_st16(ts + 16 * c, p);
                }
                dt_tmem_st_wait();
                dt_tc_fence_before();
                dt_mbar_arrive(&sh->pfull[s]);
            }
            if (poison) l = __int_as_float(0x7FC00000);
            // the segment's sums
            const bool any = dual || s < nt;  // the slot had a tile
            if (any) {
                wait(&sh->ofull[s], oc++ & 1, &sh->fail);
                __syncwarp();
                dt_tc_fence_after();
            }
            g0 += nt;
            const bool whole = u.t0 == 0 && u.t1 == u.nt;
            float* my = part + (size_t)(2 * cta + (u.t0 == 0)) * ROWS * (D + 2);
            float f0 = 1.f, f1 = 0.f;  // weights of this slot's and the other slot's sums
            const uint32_t xb = dt_smem_addr(sm + L::Q) + (tid % TQ) * (D * 4);
            if (!dual) {
                // slot 1 hands its rows to slot 0 by way of the query tiles
                if (s == 1) {
                    sh->mrg_m[row] = m;
                    sh->mrg_l[row] = l;
                    if (any) {
#pragma unroll 1
                        for (int c = 0; c < D / 32; ++c) {
                            uint32_t v[32];
                            dt_tmem_ld32_async(to + 32 * c, v);
                            dt_tmem_ld_wait(v);
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                const uint32_t q[4] = {v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]};
                                sts16(xb + (((8 * c + i) ^ (row & 7)) << 4), q);
                            }
                        }
                    }
                }
                asm volatile("bar.sync 2, 256;" ::: "memory");
                if (s == 0 && nt > 1) {
                    const float m1 = sh->mrg_m[row], M = fmaxf(m, m1);
                    f0 = m == NEG_INF ? 0.f : dt_ex2_approx(m - M);
                    f1 = m1 == NEG_INF ? 0.f : dt_ex2_approx(m1 - M);
                    // a row that saw nothing keeps l = 0; NaN stays
                    l = __fadd_rn(__fmul_rn(l, f0), __fmul_rn(sh->mrg_l[row], f1));
                    m = M;
                }
            }
            if (dual || s == 0) {
                const float inv = l == 0.f ? 0.f : 1.0f / l;
                const float w0 = whole ? __fmul_rn(f0, inv) : f0, w1 = whole ? __fmul_rn(f1, inv) : f1;
                const int G = a.Hq / a.c.Hkv;
                const long long rr = (long long)u.qb * ROWS + row;
                uint16_t* out = (uint16_t*)a.out + (((size_t)u.b * a.M + rr / G) * a.Hq + u.h * G + rr % G) * D;
                if (!whole) {
                    my[row] = m;
                    my[ROWS + row] = l;
                }
#pragma unroll 1
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t v[32];
                    dt_tmem_ld32_async(to + 32 * c, v);
                    dt_tmem_ld_wait(v);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
                        if (!dual && nt > 1) {
                            const uint32_t ad = xb + (((8 * c + i) ^ (row & 7)) << 4);
                            asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                                         : "=f"(y.x), "=f"(y.y), "=f"(y.z), "=f"(y.w) : "r"(ad));
                        }
                        float x[4];
                        x[0] = __fmaf_rn(__uint_as_float(v[4 * i]), w0, __fmul_rn(y.x, w1));
                        x[1] = __fmaf_rn(__uint_as_float(v[4 * i + 1]), w0, __fmul_rn(y.y, w1));
                        x[2] = __fmaf_rn(__uint_as_float(v[4 * i + 2]), w0, __fmul_rn(y.z, w1));
                        x[3] = __fmaf_rn(__uint_as_float(v[4 * i + 3]), w0, __fmul_rn(y.w, w1));
#pragma unroll
                        for (int e = 0; e < 4; ++e) v[4 * i + e] = __float_as_uint(x[e]);
                    }
                    if (row < u.rows) {
                        if (whole) {
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                uint32_t o[4];
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    const __nv_bfloat162 b2 = __floats2bfloat162_rn(__uint_as_float(v[8 * i + 2 * e]),
                                                                                    __uint_as_float(v[8 * i + 2 * e + 1]));
                                    o[e] = *(const uint32_t*)&b2;
                                }
                                *(uint4*)(out + 32 * c + 8 * i) = make_uint4(o[0], o[1], o[2], o[3]);
                            }
                        } else {
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                *(uint4*)(my + 2 * ROWS + (size_t)row * D + 32 * c + 4 * i) =
                                    make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
                        }
                    }
                }
                dt_tc_fence_before();
            }
            if (!whole) {
                // the CTA that finishes a unit's last part joins all of them, in their order
                __threadfence();
                asm volatile("bar.sync 2, 256;" ::: "memory");
                if (tid == 0) {
                    const int done = atomicAdd(&counters[u.first], 1) + 1;
                    sh->last = done == u.segs;
                    if (done == u.segs) counters[u.first] = 0;
                    __threadfence();
                }
                asm volatile("bar.sync 2, 256;" ::: "memory");
                if (sh->last) join(a, u, part, tid);
            }
        }
    }

    static DT_DI void join(const DtAttend& a, const AtWalk<ROWS, ATOM>& u, const float* part, int tid) {
        constexpr int CPR = D / 8, RPI = NS / CPR;  // 8 columns per thread
        const float NEG_INF = -__int_as_float(0x7F800000);
        const int G = a.Hq / a.c.Hkv, c = tid % CPR;
        auto slot = [&](int i) { return part + (size_t)(2 * (u.first + i) + (i == 0)) * ROWS * (D + 2); };
        for (int r = tid / CPR; r < u.rows; r += RPI) {
            float M = NEG_INF, l = 0.f, x[8] = {};
            for (int i = 0; i < u.segs; ++i) M = fmaxf(M, __ldcg(slot(i) + r));
            for (int i = 0; i < u.segs; ++i) {
                const float* p = slot(i);
                const float mi = __ldcg(p + r);
                const float f = mi == NEG_INF ? 0.f : dt_ex2_approx(mi - M);
                l = __fmaf_rn(__ldcg(p + ROWS + r), f, l);
                const float4* o = (const float4*)(p + 2 * ROWS + (size_t)r * D + 8 * c);
                const float4 y = __ldcg(o), z = __ldcg(o + 1);
                x[0] = __fmaf_rn(y.x, f, x[0]), x[1] = __fmaf_rn(y.y, f, x[1]);
                x[2] = __fmaf_rn(y.z, f, x[2]), x[3] = __fmaf_rn(y.w, f, x[3]);
                x[4] = __fmaf_rn(z.x, f, x[4]), x[5] = __fmaf_rn(z.y, f, x[5]);
                x[6] = __fmaf_rn(z.z, f, x[6]), x[7] = __fmaf_rn(z.w, f, x[7]);
            }
            const float inv = l == 0.f ? 0.f : 1.0f / l;
            const long long rr = (long long)u.qb * ROWS + r;
            uint16_t* out = (uint16_t*)a.out + (((size_t)u.b * a.M + rr / G) * a.Hq + u.h * G + rr % G) * D + 8 * c;
            uint32_t o[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const __nv_bfloat162 b2 = __floats2bfloat162_rn(__fmul_rn(x[2 * e], inv), __fmul_rn(x[2 * e + 1], inv));
                o[e] = *(const uint32_t*)&b2;
            }
            *(uint4*)out = make_uint4(o[0], o[1], o[2], o[3]);
        }
    }
};

template <int D>
__global__ void __launch_bounds__(NT, 1) kn12_kernel(const __grid_constant__ DtAttend a, float* part, int* counters) {
    using L = Lay<D>;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* sm = (unsigned char*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    Shared* sh = (Shared*)(sm + L::SH);
    const int tid = threadIdx.x, wid = tid >> 5;
    const int cta = blockIdx.x, ctas = gridDim.x;
    if (wid == 0) dt_tmem_alloc(&sh->tmem, 512);
    if (tid == 0) {
        for (int i = 0; i < STAGES; ++i) {
            dt_mbar_init(&sh->kfull[i], NC);
            dt_mbar_init(&sh->vfull[i], NC);
            dt_mbar_init(&sh->kfree[i], 1);
            dt_mbar_init(&sh->vfree[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            dt_mbar_init(&sh->sfull[i], 1);
            dt_mbar_init(&sh->pfull[i], TQ);
            dt_mbar_init(&sh->ofull[i], 1);
        }
        for (int i = 0; i < RING; ++i) dt_mbar_init(&sh->scfull[i], NC);
        dt_mbar_init(&sh->qfull, NS);
        dt_fence_mbar_init();
        sh->fail = 0;
    }
    dt_pdl_trigger();
    dt_pdl_wait();
    if (wid == 1) at_share<ROWS>(a, cta, ctas, MIN_SHARE, &sh->share);
    dt_tc_fence_before();
    __syncthreads();
    dt_tc_fence_after();
    const uint32_t tmem = sh->tmem;
    if (tid < NS) {
        at_zero_rest(a, cta, ctas, tid, NS);
        Soft<D>::run(a, sm, sh, tmem, tid, cta, ctas, part, counters);
    } else if (tid < NS + NC) {
        Conv<D>::run(a, sm, sh, tid - NS, cta);
    } else if (tid == NS + NC) {
        issue_all<D>(a, sm, sh, tmem, cta);
    }
    dt_tc_fence_before();
    __syncthreads();
    if (tid == 0 && sh->fail)
        for (int b = 0; b < a.batch; ++b) atomicOr(&a.status[b], DT_DEV_TIMEOUT);
    if (wid == 0) {
        dt_tc_fence_after();
        dt_tmem_dealloc(tmem, 512);
    }
}

template <int D>
cudaError_t launch(const DtAttend& a, void* workspace, int ctas, cudaStream_t st) {
    constexpr size_t smem = Lay<D>::SMEM;
    static_assert(smem <= 227 * 1024, "shared memory of a CTA");
    // more than half of an SM's shared memory: one CTA per SM, as its 512 TMEM columns need
    static_assert(2 * (smem + 1024) > 233472 || D == 64, "one CTA per SM");
    constexpr size_t ask = smem > 116 * 1024 ? smem : 116 * 1024;
    cudaError_t e = cudaFuncSetAttribute(kn12_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)ask);
    if (e != cudaSuccess) return e;
    DtLaunch lc(dim3(ctas), dim3(NT), ask, st);
    return cudaLaunchKernelEx(&lc.cfg, kn12_kernel<D>, a, (float*)((char*)workspace + AT_MAX_CTAS * sizeof(int)),
                              (int*)workspace);
}

}  // namespace

size_t dt_kn12_workspace(int D, int ctas) {
    return AT_MAX_CTAS * sizeof(int) + (size_t)ctas * 2 * ROWS * (D + 2) * sizeof(float);
}

cudaError_t dt_kn12_launch(const DtAttend& a, void* workspace, int ctas, cudaStream_t st) {
    return a.c.D == 64 ? launch<64>(a, workspace, ctas, st) : launch<128>(a, workspace, ctas, st);
}
