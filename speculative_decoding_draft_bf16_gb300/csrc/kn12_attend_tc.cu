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
// more than 8 since.  A tile of new rows has one scale, or, when the rows'
// magnitudes lie too far apart for fp16, one for each row: such tiles go through
// a short loop of their own, and what a row does not see never matters to it.
//
// Roundings: codes are exact in fp16; q, new k and v are scaled by powers of two into
// fp16's range and rounded to 11 bits (bf16 has 8, rotation gives them more); P to 11
// bits, below the 8 of the output; all sums fp32.
//
// What bounds it.  A tile of 256 rows and 128 tokens takes 2560 clocks of MMAs at D = 128
// (64 clocks for 128 x 128 x 16; 48, not 32, for the 128 x 64 x 16 of the halves, which
// read Q from shared memory each time) and 3200 to 4200 in all: a half's softmax takes
// 1300 to 1500 clocks for 64 elements of 32 rows, in which two softmax and two converter
// warps share an SM quarter's issue slots, and the slots' chains (scores, softmax,
// products) overlap but do not fill each other's gaps.  Sixteen trees of 257 nodes, 64
// heads on 8, contexts of 5000 to 16384: 1.12 ms, 0.98 PFLOP/s (51% of the measured bf16
// rate).  Scores of a whole tile at a time (fewer, wider MMAs, but a slot's softmax then
// waits for all of them): 1.27 ms against 1.10 then.  Short contexts are bound by what a
// unit costs beside its tiles, in thousands of clocks: queries (8), outputs (3 to 5), joins
// (5 to 15), and tiles of new rows, which take 9 in trees and 20 in prompts (cached ones
// 4): one prompt of 4000 rows over an empty cache, 32 heads on 8, 542 us (13% of the rate).
// Code size matters as much: with unrolled tiles the roles' loops overflowed the
// instruction caches (one tree of 257 nodes 125 us instead of 99).
#include <atomic>

#include "dt_attend.cuh"
#include "dt_tcgen05.cuh"

namespace {

constexpr int ROWS = 256;       // query rows of a block
constexpr int TQ = 128;         // rows of a slot
constexpr int NS = 256;         // softmax threads
constexpr int NC = 128;         // converter threads for the keys, and as many for the values
// Five warpgroups; in the last one two warps issue the MMAs of the slots, a thread
// walks the CTA's share of the work and a warp looks up pages.
constexpr int NT = NS + 2 * NC + 128;
// Registers per thread of the warpgroups (softmax, converters, MMA): over the
// CTA they sum to what it is launched with, LAUNCH_REGS each.  No loop of a role may
// spill: the shared memory in use leaves the L1 less than the spills need.
constexpr int LAUNCH_REGS = 65536 / NT / 8 * 8;
constexpr int REG_SOFT = 120, REG_CONV = 96, REG_MMA = 48;
static_assert(NS * REG_SOFT + 2 * NC * REG_CONV + 128 * REG_MMA == NT * LAUNCH_REGS, "register split");
constexpr int STAGES = 2;       // K and V tiles in shared memory, each
constexpr int RING = 8;         // tiles whose page ids and scales are kept
constexpr int SEGS = 4;         // segments the walk may be ahead
constexpr int ATOM = 4;         // tiles of the longest unit that is not split (8: 64 trees of 61 nodes 206 : 183 us)
constexpr uint32_t MIN_SHARE = 36;    // least cost worth a CTA: the start and three tiles of a full block
static_assert(MIN_SHARE >= AtPlan<ROWS>::HEAD + (AtPlan<ROWS>::SNAP + 1) * AtPlan<ROWS>::FULL,
              "every CTA between a unit's ends has a tile of it");
constexpr int OWN_PARTS = 8;    // most parts of a unit that its last CTA joins to its own
constexpr float LOG2E = 1.44269504088896340736f;
constexpr float HEADROOM = 5.f, LAZY = 8.f;

struct Apart {  // of a tile of new rows, keys and values: each row's exponent, and whether rows have their own
    int8_t e[2][AT_TILE];
    int yes[2];
};
struct Scales {  // of four groups of 16 tokens: key scale, log2 and inverse of the value scale
    float4 ks, lv, iv;
};
struct __align__(16) Ring {
    Scales half[2];
    uint32_t id[8];             // their pages
    uint32_t bad[2][4];         // new rows with a key, a value that is not finite
    DT_DI float* ks(int g) { return &half[g >> 2].ks.x + (g & 3); }
    DT_DI float* lv(int g) { return &half[g >> 2].lv.x + (g & 3); }
    DT_DI float* iv(int g) { return &half[g >> 2].iv.x + (g & 3); }
};

// The tiles [t0, t1) of a unit (b, h, qb), from the walk to the roles.
struct Seg {
    int b, h, qb, t0, t1, nt;  // b < 0: no more
    int rows, len, n, ctx;     // rows of the block; cached tokens, new rows, cached tiles
    int first, segs;           // CTA of the unit's first tile, CTAs that share it
};

struct Shared {
    uint64_t kfull[STAGES], kfree[STAGES], vfull[STAGES], vfree[STAGES];
    uint64_t sfull[2][2], pfull[2][2], qfull, scfull[RING], idfull[RING], ringfree[RING];
    uint64_t drain[2], probe;
    uint32_t tmem;
    int fail, drain_fail[2], last;
    AtShare share;
    Ring ring[RING];
    Apart apart[RING];
    float qscale[ROWS];
    int qpos[ROWS], kpos[AT_TILE];
    long long qoff[ROWS];
    float mrg_m[TQ], mrg_l[TQ];
    float wt[OWN_PARTS][ROWS];
    int emax[2][NC / 32], emin[2][NC / 32];
    uint64_t segfull[SEGS], segfree[SEGS];
    Seg seg[SEGS];
};

template <int D>
struct Lay {
    static constexpr int TILE = AT_TILE * D * 2;  // bytes of an fp16 tile
    static constexpr int HALF = AT_TILE * 128;    // bytes of 64 elements of every row
    static constexpr int Q = 0, K = 2 * TILE, V = K + STAGES * TILE, SH = V + STAGES * TILE;
    static constexpr size_t SMEM = 1024 + SH + sizeof(Shared);
};

// Bounded wait: 2^18 tries of 3.8 us (measured, whatever the hint says), a second; once
// one has run out, `fail` is set and later ones give up at their first look.  Short code: it
// stands in every role.
DT_DI void wait(uint64_t* bar, uint32_t phase, int* fail) {
    asm volatile(
        "{\n .reg .pred p;\n .reg .u32 n, f;\n mov.u32 n, 262144;\n"
        "AGAIN:\n mbarrier.try_wait.parity.shared::cta.b64 p, [%0], %1, 1000;\n @p bra DONE;\n"
        " sub.u32 n, n, 1;\n setp.ne.u32 p, n, 0;\n @!p st.volatile.shared.u32 [%2], 1;\n"
        " ld.volatile.shared.u32 f, [%2];\n setp.eq.u32 p, f, 0;\n @p bra AGAIN;\nDONE:\n}\n" ::"r"(dt_smem_addr(bar)),
        "r"(phase), "r"(dt_smem_addr(fail))
        : "memory");
}

// The same, four times as long and whatever has run out elsewhere: for segments, which come
// in the end, because every role then runs on without waiting.  False when it has run out.
DT_DI bool wait_long(uint64_t* bar, uint32_t phase, int* fail) {
    uint32_t n = 1048576;
    asm volatile(
        "{\n .reg .pred p;\n"
        "AGAIN:\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 1000;\n @p bra DONE;\n"
        " sub.u32 %0, %0, 1;\n setp.ne.u32 p, %0, 0;\n @p bra AGAIN;\n st.volatile.shared.u32 [%3], 1;\nDONE:\n}\n"
        : "+r"(n)
        : "r"(dt_smem_addr(bar)), "r"(phase), "r"(dt_smem_addr(fail))
        : "memory");
    return n != 0;
}

DT_DI bool elect_one() {  // one lane of a converged warp
    uint32_t p;
    asm volatile("{\n .reg .pred q;\n elect.sync _|q, 0xFFFFFFFF;\n selp.u32 %0, 1, 0, q;\n}\n" : "=r"(p));
    return p;
}

// This warpgroup's registers per thread, from the LAUNCH_REGS it started with
// (`dec` takes a lower count only, `inc` a higher one).
template <int R>
DT_DI void set_regs() {
    static_assert(R >= 24 && R <= 256 && R % 8 == 0, "register count");
    if constexpr (R > LAUNCH_REGS) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R));
    if constexpr (R < LAUNCH_REGS) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R));
}

DT_DI bool failed(const Shared* sh) { return *(const volatile int*)&sh->fail != 0; }

// The thread that walks the share, up to SEGS segments ahead of the roles.  When a wait
// of a role has run out, it ends the walk.
DT_DI void walk_share(const DtAttend& a, Shared* sh, int cta) {
    AtWalk<ROWS, ATOM> u;
    u.start(a, sh->share);
    uint32_t i = 0;
    for (bool more = true; more; ++i) {
        more = u.next(a, sh->share, cta);
        if (!wait_long(&sh->segfree[i % SEGS], (i / SEGS + 1) & 1, &sh->fail)) return;  // it may still be read
        more = more && !failed(sh);
        Seg* s = &sh->seg[i % SEGS];
        *s = more ? Seg{u.b, u.h, u.qb, u.t0, u.t1, u.nt, u.rows, u.r.len, u.r.n, u.r.ctx, u.first, u.segs} : Seg{-1};
        dt_mbar_arrive(&sh->segfull[i % SEGS]);
        if (more) u.step(a);
    }
}
// Segment i of the share, or null after the last one.  Every thread of a role gets each
// segment and releases it when it has read what it needs.  The threads of a role wait for
// each other within a segment, so all have to come to one answer whatever has run out: it
// depends on what the walk has published alone.
DT_DI const Seg* get_segment(Shared* sh, uint32_t i) {
    const bool there = wait_long(&sh->segfull[i % SEGS], (i / SEGS) & 1, &sh->fail);
    const Seg* s = &sh->seg[i % SEGS];
    return !there || s->b < 0 ? nullptr : s;
}
DT_DI void release_segment(Shared* sh, uint32_t i) { dt_mbar_arrive(&sh->segfree[i % SEGS]); }

// 32-bit pair of fp16 from two fp32 (lo in the low half).
DT_DI uint32_t f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
DT_DI uint32_t bf16x2(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *(const uint32_t*)&v;
}
DT_DI float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

DT_DI float max3_nan(float a, float b, float c) {  // NaN if one is
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// Streamed codes: read once by this CTA, not kept in L1.
DT_DI uint4 ldg16(const void* p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p)
                 : "memory");
    return v;
}

// Byte offset of the 16-byte chunk c (8 fp16) of row r in a tile of D columns.
DT_DI uint32_t chunk_at(int r, int c) {
    return (uint32_t)((c >> 3) * (AT_TILE * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}
DT_DI void sts16(uint32_t addr, const uint32_t (&w)[4]) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
                 : "memory");
}

// Sixteen e4m3 codes to two fp16 chunks at a0 and a1.
DT_DI void store_codes(uint32_t a0, uint32_t a1, const uint4& q) {
    uint32_t w[4];
    dt_e4m3x4_to_f16x4(q.x, w[0], w[1]);
    dt_e4m3x4_to_f16x4(q.y, w[2], w[3]);
    sts16(a0, w);
    dt_e4m3x4_to_f16x4(q.z, w[0], w[1]);
    dt_e4m3x4_to_f16x4(q.w, w[2], w[3]);
    sts16(a1, w);
}

// log2 of a value scale (2^-100 to 2^120), and its inverse: exact for powers of two.
DT_DI void scale_parts(float s, float& lg, float& inv) {
    lg = log2f(s);
    inv = 1.0f / s;
}

// The converter warps: 128 threads for the keys, 128 for the values, one code (the
// instruction caches nearest the SM's quarters hold little more than the loops of
// the roles that run there).
template <int D>
struct Conv {
    // A thread reads 16-byte piece `piece` (of D / 16) of token i * TPI + `tok`
    // in iteration i.  Four lanes read half a row of 128 columns; eight lanes of
    // a store phase then hold two tokens, whose chunks swizzle to eight
    // different 16-byte columns.
    static constexpr int PPT = D / 16;
    static constexpr int TPI = NC / PPT;      // tokens per iteration
    static DT_DI int piece_of(int ct) { return D == 128 ? (ct & 3) + ((ct >> 4) & 1) * 4 : ct & 3; }
    static DT_DI int tok_of(int ct) { return D == 128 ? ((ct >> 2) & 3) + (ct >> 5) * 4 : ct >> 2; }
    static constexpr int NI = AT_TILE / TPI;  // iterations per tile
    using L = Lay<D>;

    static DT_DI void group_sync(bool keys) {
        if (keys) asm volatile("bar.sync 1, 128;" ::: "memory");
        else asm volatile("bar.sync 3, 128;" ::: "memory");
    }

    static constexpr float INF = __builtin_huge_valf();
    static constexpr int8_t NONE = 127;  // in place of the exponent of a row of zeros

    // One tile of new rows, from row m0: keys rotated, and scaled by powers of two when
    // the rows' largest magnitudes are not all in [2^-4, 2^15), where fp16 is exact enough:
    // by one for the tile when that brings them there, else by one for each row, so that
    // what other rows hold does not matter.
    static DT_DI void fresh(const DtAttend& a, const Seg& u, bool keys, int m0, int ct, Shared* sh, uint32_t g,
                            uint32_t tile) {
        Ring* ring = &sh->ring[g % RING];
        Apart* ap = &sh->apart[g % RING];
        const int which = keys ? 0 : 1, b = u.b, n = u.n, len = u.len, left = min(AT_TILE, n - m0);
        const dt_rows& src = keys ? a.k : a.v;
        const uint16_t* p = (const uint16_t*)src.ptr + b * src.stride_b + u.h * src.stride_h;
        const long long stride = src.stride_n;
        dt_rope rope = a.rope;
        if (!keys) rope.rot = 0;
        if (ct < 4) ring->bad[which][ct] = 0u;
        ap->e[which][ct] = NONE;
        if (keys) sh->kpos[ct] = rope.rot && ct < left ? at_position(a, b, len, m0 + ct) : 0;
        group_sync(keys);
        const int pr = ct % PPT;  // this thread's chunk pair of rows ct / PPT + i * TPI
        int c0, c1;
        dt_pair_chunks(pr, rope, c0, c1);
        constexpr int U = D == 64 ? 2 : 1;  // rows in flight (two at D = 128 make the loop over cached tiles spill)
#pragma unroll 1
        for (int pass = 0; pass < 2; ++pass) {  // the second one when the tile needs scales
#pragma unroll 1
            for (int i0 = 0; i0 < NI; i0 += U) {
                if (i0 * TPI >= left) {  // no row of these: zeros, which a weight of zero leaves zero
                    const uint32_t zero[4] = {};
#pragma unroll
                    for (int k = 0; k < U; ++k) {
                        sts16(tile + chunk_at(ct / PPT + (i0 + k) * TPI, c0), zero);
                        sts16(tile + chunk_at(ct / PPT + (i0 + k) * TPI, c1), zero);
                    }
                    continue;
                }
                DtPair<uint16_t> raw[U];
#pragma unroll
                for (int k = 0; k < U; ++k) {
                    const int r = min(ct / PPT + (i0 + k) * TPI, left - 1);
                    raw[k].load(p + (m0 + r) * stride, pr, rope, sh->kpos[r]);
                }
#pragma unroll
                for (int k = 0; k < U; ++k) {
                    const int r = ct / PPT + (i0 + k) * TPI;
                    uint32_t o[4], w[4];
                    float x[8], y[8];
                    raw[k].rotated(pr, rope, x, y);
                    float top = max3_nan(fabsf(x[0]), fabsf(y[0]), 0.f);
#pragma unroll
                    for (int q = 1; q < 8; ++q) top = max3_nan(top, fabsf(x[q]), fabsf(y[q]));
                    if (__float_as_uint(top) >= 0x7F800000u) {  // zeros for what is not finite
                        top = 0.f;
#pragma unroll
                        for (int q = 0; q < 8; ++q) {
                            x[q] = fabsf(x[q]) < INF ? x[q] : 0.f;
                            y[q] = fabsf(y[q]) < INF ? y[q] : 0.f;
                            top = max3_nan(top, fabsf(x[q]), fabsf(y[q]));
                        }
                        if (r < left) atomicOr(&ring->bad[which][r >> 5], 1u << (r & 31));
                    }
                    const float f = r >= left ? 0.f : pass ? dt_pow2(-ap->e[which][r]) : 1.f;
#pragma unroll
                    for (int q = 0; q < 8; ++q) x[q] = __fmul_rn(x[q], f), y[q] = __fmul_rn(y[q], f);
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        o[q] = f16x2(x[2 * q], x[2 * q + 1]);
                        w[q] = f16x2(y[2 * q], y[2 * q + 1]);
                    }
                    sts16(tile + chunk_at(r, c0), o);
                    sts16(tile + chunk_at(r, c1), w);
                    if (pass == 0) {
#pragma unroll
                        for (int d = 1; d < PPT; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
                        if (pr == 0 && top > 0.f && r < left) ap->e[which][r] = (int8_t)at_row_exponent(__float_as_uint(top), keys);
                    }
                }
            }
            if (pass) break;
            group_sync(keys);
            const int own = ap->e[which][ct];
            int hi = __reduce_max_sync(0xffffffffu, own == NONE ? -128 : own), lo = __reduce_min_sync(0xffffffffu, own);
            if ((ct & 31) == 0) sh->emax[which][ct >> 5] = hi, sh->emin[which][ct >> 5] = lo;
            group_sync(keys);
            for (int i = 0; i < NC / 32; ++i) hi = max(hi, sh->emax[which][i]), lo = min(lo, sh->emin[which][i]);
            const bool apart = hi - lo > 18 && hi != -128;
            const int e = apart || hi == -128 || (lo >= -4 && hi < 15) ? 0 : max(hi - 14, keys ? -126 : -57);
            if (!apart) ap->e[which][ct] = (int8_t)e;
            else if (own == NONE) ap->e[which][ct] = 0;
            if (ct == 0) ap->yes[which] = apart;
            if (ct < 8) {
                if (keys) {
                    *ring->ks(ct) = dt_pow2(e);
                } else {
                    *ring->lv(ct) = (float)e;
                    *ring->iv(ct) = dt_pow2(-e);
                }
            }
            group_sync(keys);
            if (e == 0 && !apart) return;
        }
        group_sync(keys);
    }

    static DT_DI void run(const DtAttend& a, unsigned char* sm, Shared* sh, int ct, bool keys) {
        const int lp = 31 - __clz(a.c.page), low = a.c.page - 1;
        const uint32_t base = dt_smem_addr(sm + (keys ? L::K : L::V));
        const uint32_t a0 = base + chunk_at(tok_of(ct), 2 * piece_of(ct)),
                       a1 = base + chunk_at(tok_of(ct), 2 * piece_of(ct) + 1);
        const uint32_t page_bytes = ((uint32_t)a.c.Hkv << lp) * D;
        uint64_t* full = keys ? sh->kfull : sh->vfull;
        uint64_t* free_ = keys ? sh->kfree : sh->vfree;
        uint32_t g = 0, i = 0;  // tiles, segments done
        for (const Seg* sg; (sg = get_segment(sh, i)) != nullptr; release_segment(sh, i++)) {
            const Seg& u = *sg;
            const int t1 = u.t1, cend = min(t1, u.ctx), last = u.len - 1;
            const uint8_t* codes = (keys ? a.c.k : a.c.v) + (((size_t)u.h << lp) * D + piece_of(ct) * 16);
            // The next tile's codes are loaded in two batches, each when this
            // tile's have left its registers.  Page ids come from shared memory:
            // loads that wait for loads would share their scoreboards.  Past len,
            // the last token's.
            uint4 q[NI];
            auto load = [&](int j, uint32_t g, int i0) {
                const Ring* ring = &sh->ring[g % RING];
#pragma unroll
                for (int i = i0; i < i0 + NI / 2; ++i) {
                    const int r = tok_of(ct) + i * TPI, tok = min(j * AT_TILE + r, last);
                    q[i] = ldg16(codes + (size_t)ring->id[r >> 4] * page_bytes + (uint32_t)(tok & low) * D);
                }
            };
            int j = u.t0;
            if (j < cend) {
                wait(&sh->idfull[g % RING], (g / RING) & 1, &sh->fail);
                load(j, g, 0);
                load(j, g, NI / 2);
            }
            auto stored = [&](int s) {
                dt_fence_proxy_async_smem();
                __syncwarp();
                if ((ct & 31) == 0) dt_mbar_arrive(&full[s]);
            };
#pragma unroll 1
            for (; j < cend; ++j, ++g) {
                const int s = g % STAGES;
                wait(&free_[s], (g / STAGES + 1) & 1, &sh->fail);
                if (ct == 0) dt_mbar_arrive(&sh->scfull[g % RING]);
                const uint32_t o = s * L::TILE;
                const bool more = j + 1 < cend;
                if (more) wait(&sh->idfull[(g + 1) % RING], ((g + 1) / RING) & 1, &sh->fail);
#pragma unroll
                for (int i0 = 0; i0 < NI; i0 += NI / 2) {
#pragma unroll
                    for (int i = i0; i < i0 + NI / 2; ++i)  // rows TPI apart, a multiple of 8, swizzle alike
                        store_codes(a0 + o + i * (TPI * 128), a1 + o + i * (TPI * 128), q[i]);
                    if (more) load(j + 1, g + 1, i0);
                }
                stored(s);
            }
#pragma unroll 1
            for (; j < t1; ++j, ++g) {
                const int s = g % STAGES;
                wait(&free_[s], (g / STAGES + 1) & 1, &sh->fail);
                wait(&sh->idfull[g % RING], (g / RING) & 1, &sh->fail);  // the ring's slot is free
                fresh(a, u, keys, (j - u.ctx) * AT_TILE, ct, sh, g, base + s * L::TILE);
                if (ct == 0) dt_mbar_arrive(&sh->scfull[g % RING]);
                stored(s);
            }
        }
    }
};

DT_DI void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// The warp that looks up pages and scales, four tiles at a time (eight lanes,
// of 16 tokens each, to a tile), up to RING tiles ahead of their use, and asks
// L2 for the codes.  A page id out of range is reported and reads another page.
template <int D>
DT_DI void look_up(const DtAttend& a, Shared* sh, int lane) {
    const int lp = 31 - __clz(a.c.page), grp = lane & 7;
    const uint32_t page_bytes = ((uint32_t)a.c.Hkv << lp) * D;
    uint32_t g = 0, i = 0;
    for (const Seg* sg; (sg = get_segment(sh, i)) != nullptr; release_segment(sh, i++)) {
        const int t0 = sg->t0, nt = sg->t1 - t0, ctx = min(sg->t1, sg->ctx) - t0, len = sg->len, b = sg->b, h = sg->h;
        const int* table = a.c.table + (size_t)b * a.c.max_pages;
        for (int k = 0; k < nt; k += 4) {
            const int t = k + (lane >> 3), tok = (t0 + t) * AT_TILE + grp * 16;
            const bool in = t < ctx;
            uint32_t id = 0;
            float ks = 1.f, vs = 1.f;
            if (in) {
                id = (uint32_t)table[min(tok, len - 1) >> lp];
                if (id >= (uint32_t)a.c.n_pages) {
                    atomicOr(&a.status[b], DT_DEV_BAD_CACHE);
                    id = 0;
                }
            }
            if (in && tok < len) {
                ks = a.c.k_scale[(size_t)id * a.c.Hkv + h];
                vs = a.c.v_scale[(size_t)id * a.c.Hkv + h];
                // the 16 tokens' codes: 16 D bytes of keys and of values
                const size_t o = (size_t)id * page_bytes + ((size_t)h << lp) * D + (tok & (a.c.page - 1)) * D;
#pragma unroll 4
                for (int c = 0; c < D / 8; ++c) {
                    prefetch_l2(a.c.k + o + c * 128);
                    prefetch_l2(a.c.v + o + c * 128);
                }
            }
            if (t >= ctx && t < nt) {  // 16 new rows
                const int m0 = (t0 + t - sg->ctx) * AT_TILE + grp * 16;
                for (int m = m0; m < min(m0 + 16, sg->n); ++m) {
                    for (int c = 0; c < D; c += 64) {
                        prefetch_l2((const uint16_t*)a.k.ptr + b * a.k.stride_b + m * a.k.stride_n + h * a.k.stride_h + c);
                        prefetch_l2((const uint16_t*)a.v.ptr + b * a.v.stride_b + m * a.v.stride_n + h * a.v.stride_h + c);
                    }
                }
            }
            if (k == 0) {  // the block's query rows
                const uint32_t G = a.G, r0 = (uint32_t)sg->qb * ROWS;
                const uint16_t* q = (const uint16_t*)a.q.ptr + b * a.q.stride_b + (size_t)h * G * a.q.stride_h;
#pragma unroll 1
                for (uint32_t r = r0 + lane; r < r0 + sg->rows; r += 32)
                    for (int c = 0; c < D; c += 64) prefetch_l2(q + r / G * a.q.stride_n + r % G * a.q.stride_h + c);
            }
            for (int d = 0; d < 4 && k + d < nt; ++d, ++g) {
                wait(&sh->ringfree[g % RING], (g / RING + 1) & 1, &sh->fail);
                if ((lane >> 3) == d && k + d < ctx) {
                    Ring* ring = &sh->ring[g % RING];
                    ring->id[grp] = id;
                    *ring->ks(grp) = ks;
                    scale_parts(vs, *ring->lv(grp), *ring->iv(grp));
                }
                __syncwarp();
                if (lane == 0) dt_mbar_arrive(&sh->idfull[g % RING]);
            }
        }
    }
}

// The MMA warp of slot s.  All its lanes walk along, so that operands stay in
// uniform registers, and an elected one issues (39 clocks for an MMA at most,
// against 52 from a branch of one thread); a warp for each slot, because one for
// both cannot issue as fast as the tensor cores take them.  A tile's scores come
// in two halves of 64 tokens with a buffer each, so that a slot's softmax works on
// one half while the other half's probabilities meet V and its next scores are
// formed.  sfull[s][h] counts, per segment: the first scores, then for each tile
// of the slot its product P V of half h, with the next tile's scores when there
// are any.  A tile's stages are free after two commits: one from each slot's
// warp, or both from the one slot that uses it.
template <int D>
DT_DI void issue_slot(unsigned char* sm, Shared* sh, uint32_t tmem, int s) {
    using L = Lay<D>;
    constexpr uint32_t ID_S = dt_idesc_f16_f32(TQ, 64, false), ID_O = dt_idesc_f16_f32(TQ, D, true);
    const uint32_t qd = dt_desc_lo(dt_smem_addr(sm + L::Q), 16), kd = dt_desc_lo(dt_smem_addr(sm + L::K), 16),
                   vd = dt_desc_lo(dt_smem_addr(sm + L::V), L::HALF);
    const bool el = elect_one();
    const uint32_t ts = tmem + s * AT_TILE, to = tmem + 2 * AT_TILE + s * D;
    uint32_t g0 = 0, seg = 0, pc = 0;  // pc: phase of pfull[s]
    for (const Seg* u; (u = get_segment(sh, seg)) != nullptr; ++seg) {
        const bool dual = __shfl_sync(0xffffffffu, u->rows, 0) > TQ;  // two slots of rows; else two slots of tiles
        const int nt = __shfl_sync(0xffffffffu, u->t1 - u->t0, 0), hop = dual ? 1 : 2;
        if (el) release_segment(sh, seg);
        wait(&sh->qfull, seg & 1, &sh->fail);
        const uint32_t q = qd + (dual ? s : 0) * (L::TILE / 16);
#pragma unroll 1
        for (int t = (dual ? 0 : s) - hop; t < nt; t += hop) {  // before the first tile: its scores only
            const bool here = t >= 0, next = t + hop < nt;
            if (!here && !next) break;
            const uint32_t g = g0 + t, gn = g + hop, st = g % STAGES, sn = gn % STAGES;
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {
                if (here) {
                    wait(&sh->pfull[s][h], pc, &sh->fail);
                    if (h == 0) wait(&sh->vfull[st], (g / STAGES) & 1, &sh->fail);
                    __syncwarp();
                    dt_tc_fence_after();
                    const uint32_t v = vd + st * (L::TILE / 16) + h * (8192 / 16);
                    if (el) {
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            dt_mma_ts_lo(to, ts + 64 * h + kk * 8, v + kk * (2048 / 16), ID_O, t >= hop || h > 0 || kk > 0);
                        if (h == 1) {
                            dt_mma_commit(&sh->vfree[st]);
                            dt_mma_commit(&sh->ringfree[g % RING]);
                            if (!dual) {
                                dt_mma_commit(&sh->vfree[st]);
                                dt_mma_commit(&sh->ringfree[g % RING]);
                            }
                        }
                    }
                    __syncwarp();
                }
                if (next) {
                    if (h == 0) wait(&sh->kfull[sn], (gn / STAGES) & 1, &sh->fail);
                    __syncwarp();
                    dt_tc_fence_after();
                    const uint32_t kt = kd + sn * (L::TILE / 16) + h * (8192 / 16);
                    if (el) {
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk) {
                            const uint32_t o = ((kk >> 2) * L::HALF + (kk & 3) * 32) / 16;
                            dt_mma_ss_lo(ts + 64 * h, q + o, kt + o, ID_S, kk > 0);
                        }
                        if (h == 1) {
                            dt_mma_commit(&sh->kfree[sn]);
                            if (!dual) dt_mma_commit(&sh->kfree[sn]);
                        }
                    }
                    __syncwarp();
                }
                if (el) dt_mma_commit(&sh->sfull[s][h]);
                __syncwarp();
            }
            if (here) pc ^= 1;
        }
        g0 += nt;
    }
    if (el && failed(sh)) {  // otherwise the softmax warps have waited for every product
        dt_mma_commit(&sh->drain[s]);
        wait(&sh->drain[s], 0, &sh->drain_fail[s]);
    }
    __syncwarp();
}

// A slot's softmax: 128 threads, one per row.
template <int D>
struct Soft {
    using L = Lay<D>;

    // The block's rows, rotated, scaled by a power of two and converted.
    static DT_DI void queries(const DtAttend& a, const Seg& u, unsigned char* sm, Shared* sh, int tid) {
        constexpr int PPR = D / 16, RPI = NS / PPR, U = 2;  // chunk pairs per row, rows per pass
        const uint32_t G = a.G;
        const int tiles = u.rows > TQ ? 2 : 1;
        const uint32_t qb = dt_smem_addr(sm + L::Q);
        const int pr = tid % PPR;
        int c0, c1;
        dt_pair_chunks(pr, a.rope, c0, c1);
        {
            const uint32_t row = (uint32_t)u.qb * ROWS + min(tid, u.rows - 1), n = row / G;
            sh->qpos[tid] = a.rope.rot ? at_position(a, u.b, u.len, (int)n) : 0;
            sh->qoff[tid] = n * a.q.stride_n + (row % G) * a.q.stride_h;
        }
        asm volatile("bar.sync 2, 256;" ::: "memory");
        const uint16_t* base = (const uint16_t*)a.q.ptr + u.b * a.q.stride_b + (size_t)u.h * G * a.q.stride_h;
#pragma unroll 1
        for (int r0 = tid / PPR; r0 < tiles * TQ; r0 += U * RPI) {
            DtPair<uint16_t> raw[U];
#pragma unroll
            for (int k = 0; k < U; ++k)  // U rows in flight
                raw[k].load(base + sh->qoff[r0 + k * RPI], pr, a.rope, sh->qpos[r0 + k * RPI]);
#pragma unroll
            for (int k = 0; k < U; ++k) {
                const int r = r0 + k * RPI;
                float x[8], y[8];
                raw[k].rotated(pr, a.rope, x, y);
                // the row's largest magnitude (rows past the block's repeat its last one)
                float top = fmaxf(fabsf(x[0]), fabsf(y[0]));
#pragma unroll
                for (int e = 1; e < 8; ++e) top = max3(top, fabsf(x[e]), fabsf(y[e]));
                uint32_t big = __float_as_uint(top);
#pragma unroll
                for (int o = PPR / 2; o > 0; o >>= 1) big = max(big, __shfl_xor_sync(0xffffffffu, big, o));
                int ex = (int)(big >> 23) - 127;  // largest magnitude in [2^ex, 2^(ex+1))
                ex = big >= 0x7F800000u ? 0 : min(max(ex, -100), 126);  // 2^-ex is a normal number
                const float f = dt_pow2(-ex);
                uint32_t w[4], z[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    w[e] = f16x2(__fmul_rn(x[2 * e], f), __fmul_rn(x[2 * e + 1], f));
                    z[e] = f16x2(__fmul_rn(y[2 * e], f), __fmul_rn(y[2 * e + 1], f));
                }
                sts16(qb + (r / TQ) * L::TILE + chunk_at(r % TQ, c0), w);
                sts16(qb + (r / TQ) * L::TILE + chunk_at(r % TQ, c1), z);
                if (pr == 0) sh->qscale[r] = __fmul_rn(__fmul_rn(a.scale, LOG2E), dt_pow2(ex));
            }
        }
        dt_fence_proxy_async_smem();
        dt_mbar_arrive(&sh->qfull);
    }

    // The row's mask of 64 tokens of a tile that is not wholly visible.
    static DT_DI uint2 mask_words(const DtAttend& a, const Seg& u, int t, int h, int row) {
        if (t < u.ctx) {
            const int left = u.len - t * AT_TILE - 64 * h;
            return make_uint2(left >= 32 ? ~0u : left <= 0 ? 0u : (1u << left) - 1u,
                              left >= 64 ? ~0u : left <= 32 ? 0u : (1u << (left - 32)) - 1u);
        }
        if (row >= u.rows) return make_uint2(0u, 0u);
        const int node = (int)(((uint32_t)u.qb * ROWS + row) / (uint32_t)(a.G));
        const int m0 = (t - u.ctx) * AT_TILE + 64 * h;
        return make_uint2(at_mask_word(a, u.b, node, m0, u.n), at_mask_word(a, u.b, node, m0 + 32, u.n));
    }

    // A maximum that has grown moves the reference, and O when it has sums; rows of a
    // warp do so together.
    static DT_DI void follow(float mx, float& m, float& l, uint32_t to, bool has_o, uint64_t* other, uint32_t other_ph,
                             int* fail) {
        const bool grown = mx > m + (HEADROOM + LAZY);
        if (__any_sync(0xffffffffu, grown)) {
            const float to_m = grown ? mx - HEADROOM : m;
            const float f = grown ? dt_ex2_approx(m - to_m) : 1.f;  // m = -inf: 0
            m = to_m;
            l = __fmul_rn(l, f);
            if (has_o) {
                wait(other, other_ph, fail);
                __syncwarp();
                dt_tc_fence_after();
#pragma unroll 1
                for (int c = 0; c < D / 16; ++c) {
                    uint32_t o[16];
                    dt_tmem_ld16_async(to + 16 * c, o);
                    dt_tmem_ld_wait(o);
#pragma unroll
                    for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__fmul_rn(__uint_as_float(o[i]), f));
                    dt_tmem_st16(to + 16 * c, o);
                }
            }
        }
    }

    // 64 tokens of a row: their scores at ts become probabilities in place, the
    // running reference m and sum l move on, and O is rescaled when it has sums;
    // before that every product of the slot must be done: `other` is the barrier
    // of the other half's.  sc: the scales of the four groups.
    static DT_DI void half(const Scales* sc, uint32_t ts, uint32_t to, bool has_o, float rowc, bool masked, uint2 mk,
                           float& m, float& l, uint64_t* other, uint32_t other_ph, int* fail) {
        const float NEG_INF = -__int_as_float(0x7F800000);
        if (masked && !__any_sync(0xffffffffu, mk.x | mk.y)) {  // none of the warp's rows sees any of them
            const uint32_t z[16] = {};
            dt_tmem_st16(ts, z);
            dt_tmem_st16(ts + 16, z);
            dt_tmem_st_wait();
            return;
        }
        uint32_t x[64];
        const float4 ks = sc->ks, lv = sc->lv, iv = sc->iv;
        dt_tmem_ld64(ts, x);
        const float ka[4] = {at_factor(rowc, ks.x), at_factor(rowc, ks.y), at_factor(rowc, ks.z), at_factor(rowc, ks.w)};
        const float l4[4] = {lv.x, lv.y, lv.z, lv.w}, i4[4] = {iv.x, iv.y, iv.z, iv.w};
        if (masked) {
#pragma unroll
            for (int i = 0; i < 64; ++i)
                if (!(((i < 32 ? mk.x : mk.y) >> (i & 31)) & 1)) x[i] = 0xFF800000u;  // -infinity
        }
        // the largest score + log2 of its value scale
        float tg[4];
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            float q0 = __uint_as_float(x[16 * g]), q1 = __uint_as_float(x[16 * g + 1]);
#pragma unroll
            for (int i = 2; i < 14; i += 4) {
                q0 = max3(q0, __uint_as_float(x[16 * g + i]), __uint_as_float(x[16 * g + i + 1]));
                q1 = max3(q1, __uint_as_float(x[16 * g + i + 2]), __uint_as_float(x[16 * g + i + 3]));
            }
            q0 = max3(q0, __uint_as_float(x[16 * g + 14]), __uint_as_float(x[16 * g + 15]));
            tg[g] = __fmaf_rn(fmaxf(q0, q1), ka[g], l4[g]);
        }
        const float mx = fmaxf(max3(tg[0], tg[1], tg[2]), tg[3]);
        follow(mx, m, l, to, has_o, other, other_ph, fail);
        const float mu = m == NEG_INF ? 0.f : m;
#pragma unroll
        for (int g2 = 0; g2 < 4; g2 += 2) {
            uint32_t p[16];
#pragma unroll
            for (int g = g2; g < g2 + 2; ++g) {
                const float kb = __fsub_rn(l4[g], mu);
                const unsigned long long ka2 = dt_f2_pack(ka[g], ka[g]), kb2 = dt_f2_pack(kb, kb);
                unsigned long long sum = dt_f2_pack(0.f, 0.f);
#pragma unroll
                for (int i = 0; i < 16; i += 2) {
                    float e0, e1;
                    dt_f2_unpack(dt_f2_fma(dt_f2_pack(__uint_as_float(x[16 * g + i]), __uint_as_float(x[16 * g + i + 1])),
                                           ka2, kb2), e0, e1);
                    e0 = dt_ex2_approx(e0);
                    e1 = dt_ex2_approx(e1);
                    sum = dt_f2_add(sum, dt_f2_pack(e0, e1));
                    p[8 * (g - g2) + i / 2] = f16x2(e0, e1);
                }
                float s0, s1;
                dt_f2_unpack(sum, s0, s1);
                l = __fmaf_rn(__fadd_rn(s0, s1), i4[g], l);
            }
            dt_tmem_st16(ts + 8 * g2, p);  // over columns that are in registers
        }
        dt_tmem_st_wait();
    }

    // The same for tokens with scales of their own: key exponents ek, value exponents ev.
    // Rare, so short: 16 tokens at a time, their scores read twice.
    static DT_DI void half_apart(const Apart* ap, int h, uint32_t ts, uint32_t to, bool has_o, float rowc,
                                 uint2 mk, float& m, float& l, uint64_t* other, uint32_t other_ph, int* fail) {
        const float NEG_INF = -__int_as_float(0x7F800000);
        const int8_t *ek = ap->e[0] + 64 * h, *ev = ap->e[1] + 64 * h;
        float mx = NEG_INF, mu = 0.f;
#pragma unroll 1
        for (int pass = 0; pass < 2; ++pass) {
#pragma unroll 1
            for (int g = 0; g < 4; ++g) {
                const uint32_t bits = (g < 2 ? mk.x : mk.y) >> (16 * (g & 1));
                uint32_t x[16], p[8];
                dt_tmem_ld16_async(ts + 16 * g, x);
                dt_tmem_ld_wait(x);
                float y[16];
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    y[i] = (bits >> i) & 1 ? __fmaf_rn(__uint_as_float(x[i]), at_factor(rowc, dt_pow2(ek[16 * g + i])),
                                                       __fsub_rn((float)ev[16 * g + i], mu))
                                           : NEG_INF;
                if (pass == 0) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) mx = fmaxf(mx, y[i]);
                } else {
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        y[i] = dt_ex2_approx(y[i]);
                        l = __fmaf_rn(y[i], dt_pow2(-ev[16 * g + i]), l);
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i) p[i] = f16x2(y[2 * i], y[2 * i + 1]);
                    dt_tmem_st8(ts + 8 * g, p);  // over scores that have been read
                }
            }
            if (pass == 0) {
                follow(mx, m, l, to, has_o, other, other_ph, fail);
                mu = m == NEG_INF ? 0.f : m;
            }
        }
        dt_tmem_st_wait();
    }

    static DT_DI void run(const DtAttend& a, unsigned char* sm, Shared* sh, uint32_t tmem, int tid, int cta,
                          float* part, int* counters) {
        const int s = tid / TQ, w4 = (tid >> 5) & 3;
        const float NEG_INF = -__int_as_float(0x7F800000);
        const uint32_t lanes = (uint32_t)(w4 * 32) << 16;
        const uint32_t ts = tmem + s * AT_TILE + lanes, to = tmem + 2 * AT_TILE + s * D + lanes;
        uint32_t g0 = 0, ph = 0, seg = 0;  // ph: next phase of sfull[s][0] and [1]
        for (const Seg* sg; (sg = get_segment(sh, seg)) != nullptr; release_segment(sh, seg++)) {
            const Seg& u = *sg;
            // every product of the last segment has read its queries
            asm volatile("bar.sync 2, 256;" ::: "memory");
            const bool dual = u.rows > TQ;
            const int nt = u.t1 - u.t0, hop = dual ? 1 : 2, len = u.len;
            const int row = dual ? tid : tid % TQ;  // within the block
            queries(a, u, sm, sh, tid);
            asm volatile("bar.sync 2, 256;" ::: "memory");
            const float rowc = sh->qscale[row];
            float m = NEG_INF, l = 0.f;
            bool poison = false;
            const int clear = len / AT_TILE - u.t0;  // tiles before this one are wholly visible
            uint32_t pa = ph & 1;                    // phase of both halves' scores
            int lt = dual ? 0 : s;
#pragma unroll 1
            for (; lt < nt; lt += hop, pa ^= 1) {
                const uint32_t g = g0 + lt;
                const Ring* ring = &sh->ring[g % RING];
                wait(&sh->scfull[g % RING], (g / RING) & 1, &sh->fail);
                // (under `clear`, known already: without it 16 trees of 257 nodes 1.14 ms instead of 1.13)
                if (lt >= clear && u.t0 + lt >= u.ctx && (sh->apart[g % RING].yes[0] | sh->apart[g % RING].yes[1])) break;
#pragma unroll 1
                for (int h = 0; h < 2; ++h) {
                    uint64_t* other = &sh->sfull[s][h ^ 1];  // of half 0: waited for next; of half 1: of the next tile
                    const uint32_t other_ph = pa ^ h, st = ts + 64 * h;
                    const bool has_o = lt >= hop || h;
                    const bool masked = lt >= clear;
                    uint2 mk = make_uint2(0u, 0u);
                    if (masked) {
                        mk = mask_words(a, u, u.t0 + lt, h, row);
                        if (u.t0 + lt >= u.ctx)
                            poison |= ((mk.x & (ring->bad[0][2 * h] | ring->bad[1][2 * h])) |
                                       (mk.y & (ring->bad[0][2 * h + 1] | ring->bad[1][2 * h + 1]))) != 0u;
                    }
                    wait(&sh->sfull[s][h], pa, &sh->fail);
                    __syncwarp();
                    dt_tc_fence_after();
                    half(&ring->half[h], st, to, has_o, rowc, masked, mk, m, l, other, other_ph, &sh->fail);
                    dt_tc_fence_before();
                    __syncwarp();
                    if ((tid & 31) == 0) dt_mbar_arrive(&sh->pfull[s][h]);
                }
            }
            // new rows from a tile on whose rows have scales of their own (rare: short code, apart
            // from the loop above)
#pragma unroll 1
            for (; lt < nt; lt += hop, pa ^= 1) {
                const uint32_t g = g0 + lt;
                const Ring* ring = &sh->ring[g % RING];
                wait(&sh->scfull[g % RING], (g / RING) & 1, &sh->fail);
#pragma unroll 1
                for (int h = 0; h < 2; ++h) {
                    const uint2 mk = mask_words(a, u, u.t0 + lt, h, row);
                    poison |= ((mk.x & (ring->bad[0][2 * h] | ring->bad[1][2 * h])) |
                               (mk.y & (ring->bad[0][2 * h + 1] | ring->bad[1][2 * h + 1]))) != 0u;
                    wait(&sh->sfull[s][h], pa, &sh->fail);
                    __syncwarp();
                    dt_tc_fence_after();
                    half_apart(&sh->apart[g % RING], h, ts + 64 * h, to, lt >= hop || h, rowc, mk, m, l, &sh->sfull[s][h ^ 1],
                               pa ^ h, &sh->fail);
                    dt_tc_fence_before();
                    __syncwarp();
                    if ((tid & 31) == 0) dt_mbar_arrive(&sh->pfull[s][h]);
                }
            }
            if (poison) l = __int_as_float(0x7FC00000);
            // the segment's sums
            const bool any = dual || s < nt;  // the slot had a tile
            if (any) {
                wait(&sh->sfull[s][0], pa, &sh->fail);
                wait(&sh->sfull[s][1], pa, &sh->fail);
                ph = pa ^ 1;
                __syncwarp();
                dt_tc_fence_after();
            }
            g0 += nt;
            const bool whole = u.t0 == 0 && u.t1 == u.nt;
            if (!whole && dual && u.segs <= OWN_PARTS) {
                if (tid == 0) {  // are all other parts there?
                    int done;
                    asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(done) : "l"(counters + u.first) : "memory");
                    sh->last = done == u.segs - 1;
                    if (done == u.segs - 1) counters[u.first] = 0;
                }
                asm volatile("bar.sync 2, 256;" ::: "memory");
                if (sh->last) {
                    join_own(a, u, sh, part, cta - u.first, to, row, m, l, dt_smem_addr(sm + L::Q) + (tid >> 5) * (32 * D * 2),
                             out_row(a, u, row));
                    continue;
                }
            }
            float* my = part + (size_t)(2 * cta + (u.t0 == 0)) * ROWS * (D + 2);
            float f0 = 1.f, f1 = 0.f;  // weights of this slot's and the other slot's sums
            const uint32_t xb = dt_smem_addr(sm + L::Q) + (tid % TQ) * (D * 4);
            if (!dual) {
                // slot 1 hands its rows to slot 0 by way of the query tiles, which the
                // products of both slots have read
                asm volatile("bar.sync 2, 256;" ::: "memory");
                if (s == 1) {
                    sh->mrg_m[row] = m;
                    sh->mrg_l[row] = l;
                    if (any) {
#pragma unroll 1
                        for (int c = 0; c < D / 16; ++c) {
                            uint32_t v[16];
                            dt_tmem_ld16_async(to + 16 * c, v);
                            dt_tmem_ld_wait(v);
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const uint32_t q[4] = {v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]};
                                sts16(xb + (((4 * c + i) ^ (row & 7)) << 4), q);
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
                uint16_t* out = out_row(a, u, row);
                // a full block's rows go out by way of the query tiles, whole lines at a
                // time: a warp's 32 rows in the place of its own slot's queries
                const bool staged = whole && dual;
                const uint32_t stage = dt_smem_addr(sm + L::Q) + (tid >> 5) * (32 * D * 2);
                const int lane = tid & 31;
                if (!whole) {
                    my[row] = m;
                    my[ROWS + row] = l;
                }
#pragma unroll 1
                for (int c = 0; c < D / 16; ++c) {
                    uint32_t v[16];
                    dt_tmem_ld16_async(to + 16 * c, v);
                    dt_tmem_ld_wait(v);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
                        if (!dual && nt > 1) {
                            const uint32_t ad = xb + (((4 * c + i) ^ (row & 7)) << 4);
                            asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                                         : "=f"(y.x), "=f"(y.y), "=f"(y.z), "=f"(y.w) : "r"(ad));
                        }
                        const float z[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            v[4 * i + e] = __float_as_uint(__fmaf_rn(__uint_as_float(v[4 * i + e]), w0, __fmul_rn(z[e], w1)));
                    }
                    if (whole) {
                        uint32_t o[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) o[e] = bf16x2(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1]));
                        if (staged) {
                            stage_row(stage, lane, c, o);
                        } else if (row < u.rows) {
                            *(uint4*)(out + 16 * c) = make_uint4(o[0], o[1], o[2], o[3]);
                            *(uint4*)(out + 16 * c + 8) = make_uint4(o[4], o[5], o[6], o[7]);
                        }
                    } else if (row < u.rows) {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            *(uint4*)(my + 2 * ROWS + ((4 * c + i) * ROWS + row) * 4) =
                                make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
                    }
                }
                dt_tc_fence_before();
                if (staged) send_rows(stage, lane, out, row & ~31, u.rows);
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
                if (sh->last) join(a, sm, u, part, tid);
            }
        }
    }

    // 16 columns from 16c of the thread's row, in bf16, to its place in the staged rows.
    static DT_DI void stage_row(uint32_t stage, int lane, int c, const uint32_t (&o)[8]) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t q[4] = {o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]};
            sts16(stage + lane * (D * 2) + (((2 * c + i) ^ (lane & 7)) << 4), q);
        }
    }
    // The warp's 32 staged rows (from block row `first`) to memory, whole lines at a time.
    static DT_DI void send_rows(uint32_t stage, int lane, uint16_t* out, int first, int rows) {
        __syncwarp();
        constexpr int CPR = D / 8, RPI = 32 / CPR;  // 16-byte chunks of a row, rows at a time
        const int ch = lane % CPR;
#pragma unroll 4
        for (int r0 = 0; r0 < 32; r0 += RPI) {
            const int r = r0 + lane / CPR;
            uint16_t* dst = (uint16_t*)__shfl_sync(0xffffffffu, (unsigned long long)out, r);
            uint4 q;
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(q.x), "=r"(q.y), "=r"(q.z), "=r"(q.w)
                         : "r"(stage + r * (D * 2) + ((ch ^ (r & 7)) << 4)) : "memory");
            if (first + r < rows) *(uint4*)(dst + ch * 8) = q;
        }
    }

    // The last CTA of a full block's unit: the other parts come from memory, its own
    // straight from tensor memory; same sums in the same order as join(), which writes
    // and reads all of them (64 trees of 61 nodes 174 us, this 166).
    static DT_DI void join_own(const DtAttend& a, const Seg& u, Shared* sh, const float* part, int own, uint32_t to, int row,
                               float m, float l0, uint32_t stage, uint16_t* out) {
        const float NEG_INF = -__int_as_float(0x7F800000);
        const int first = u.first, segs = u.segs, lane = row & 31;
        auto slot = [&](int i) { return part + (size_t)(2 * (first + i) + (i == 0)) * ROWS * (D + 2); };
        float M = NEG_INF, l = 0.f;
#pragma unroll 4
        for (int i = 0; i < segs; ++i) {
            const float mi = i == own ? m : __ldcg(slot(i) + row), li = i == own ? l0 : __ldcg(slot(i) + ROWS + row);
            sh->wt[i][row] = mi;
            const float up = fmaxf(M, mi);
            if (up != NEG_INF) l = __fmaf_rn(li, dt_ex2_approx(mi - up), __fmul_rn(l, dt_ex2_approx(M - up)));
            else l = __fadd_rn(l, li);  // 0, or NaN
            M = up;
        }
        const float inv = l == 0.f ? 0.f : 1.0f / l;
        for (int i = 0; i < segs; ++i) {
            const float mi = sh->wt[i][row];
            sh->wt[i][row] = mi == NEG_INF ? 0.f : __fmul_rn(dt_ex2_approx(mi - M), inv);
        }
#pragma unroll 1
        for (int c = 0; c < D / 16; c += 2) {  // 32 columns
            uint32_t v[2][16];
            dt_tmem_ld16_async(to + 16 * c, v[0]);
            dt_tmem_ld_wait(v[0]);
            dt_tmem_ld16_async(to + 16 * c + 16, v[1]);
            dt_tmem_ld_wait(v[1]);
            float x[32] = {};
#pragma unroll 1
            for (int i = 0; i < segs; ++i) {
                const float f = sh->wt[i][row];
                if (i == own) {
#pragma unroll
                    for (int e = 0; e < 32; ++e) x[e] = __fmaf_rn(__uint_as_float(v[e >> 4][e & 15]), f, x[e]);
                } else {
                    const float4* o = (const float4*)(slot(i) + 2 * ROWS) + 4 * c * ROWS + row;
                    float4 y[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) y[k] = __ldcg(o + k * ROWS);
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        x[4 * k] = __fmaf_rn(y[k].x, f, x[4 * k]), x[4 * k + 1] = __fmaf_rn(y[k].y, f, x[4 * k + 1]);
                        x[4 * k + 2] = __fmaf_rn(y[k].z, f, x[4 * k + 2]), x[4 * k + 3] = __fmaf_rn(y[k].w, f, x[4 * k + 3]);
                    }
                }
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t o[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) o[e] = bf16x2(x[16 * h + 2 * e], x[16 * h + 2 * e + 1]);
                stage_row(stage, lane, c + h, o);
            }
        }
        dt_tc_fence_before();
        send_rows(stage, lane, out, row & ~31, u.rows);
    }

    static DT_DI uint16_t* out_row(const DtAttend& a, const Seg& u, int r) {
        const uint32_t G = a.G, rr = (uint32_t)u.qb * ROWS + r;
        return (uint16_t*)a.out + (((size_t)u.b * a.M + rr / G) * a.Hq + u.h * G + rr % G) * D;
    }

    // Joins the parts of a unit: O = sum O_i 2^(m_i - M), l likewise.  A part's O
    // lies as [D / 4][ROWS][4], so that a warp of rows writes and reads whole
    // lines.  The weights go to shared memory (the query tiles) first, P parts at a
    // time, so that the loads of a row's parts do not wait on each other.
    static DT_DI void join(const DtAttend& a, unsigned char* sm, const Seg& u, float* part, int tid) {
        constexpr int P = 16;
        const float NEG_INF = -__int_as_float(0x7F800000);
        const int first = u.first, segs = u.segs, rows = u.rows;
        float* wt = (float*)(sm + L::Q);  // [P][ROWS]
        auto slot = [&](int i) { return part + (size_t)(2 * (first + i) + (i == 0)) * ROWS * (D + 2); };
        float M = NEG_INF, l = 0.f;  // of row tid
        if (tid < rows) {
#pragma unroll 4
            for (int i = 0; i < segs; ++i) {
                const float mi = __ldcg(slot(i) + tid), li = __ldcg(slot(i) + ROWS + tid), up = fmaxf(M, mi);
                if (up != NEG_INF) l = __fmaf_rn(li, dt_ex2_approx(mi - up), __fmul_rn(l, dt_ex2_approx(M - up)));
                else l = __fadd_rn(l, li);  // 0, or NaN
                M = up;
            }
        }
        const float inv = l == 0.f ? 0.f : 1.0f / l;
        // a thread has two neighbouring chunks of 4 columns of 16 rows apart: lanes
        // 0-15 and 16-31 of a warp take 16 rows each, 32 bytes of output together;
        // U such pieces at a time, so that their loads are in flight together
        constexpr int U = 4;
        const int r0 = tid & 15, c0 = ((tid >> 4) & 1) * 2, w = tid >> 5, pieces = (rows + 15) / 16 * (D / 16);
        for (int i0 = 0; i0 < segs; i0 += P) {
            // weight of part i for each row, 1 / l included
            const int np = min(P, segs - i0);
            asm volatile("bar.sync 2, 256;" ::: "memory");
#pragma unroll 4
            for (int i = 0; i < np; ++i) {
                const float mi = tid < rows ? __ldcg(slot(i0 + i) + tid) : NEG_INF;
                wt[i * ROWS + tid] = mi == NEG_INF ? 0.f : __fmul_rn(dt_ex2_approx(mi - M), inv);
            }
            asm volatile("bar.sync 2, 256;" ::: "memory");
#pragma unroll 1
            for (int k0 = w; k0 < pieces; k0 += U * (NS / 32)) {
                float x[U][8] = {};
                int at[U];  // row + ROWS * chunk of a piece; past the end the first one again
#pragma unroll
                for (int v = 0; v < U; ++v) {
                    const int k = k0 + v * (NS / 32) < pieces ? k0 + v * (NS / 32) : k0;
                    at[v] = k / (D / 16) * 16 + r0 + (k % (D / 16) * 4 + c0) * ROWS;
                }
                if (i0 > 0) {
#pragma unroll
                    for (int v = 0; v < U; ++v) {
                        const float4* acc = (const float4*)(slot(0) + 2 * ROWS) + at[v];  // this thread's, read already
                        const float4 y = acc[0], z = acc[ROWS];
                        x[v][0] = y.x, x[v][1] = y.y, x[v][2] = y.z, x[v][3] = y.w;
                        x[v][4] = z.x, x[v][5] = z.y, x[v][6] = z.z, x[v][7] = z.w;
                    }
                }
#pragma unroll 1
                for (int i = 0; i < np; ++i) {
                    const float4* o = (const float4*)(slot(i0 + i) + 2 * ROWS);
                    float4 y[U], z[U];
#pragma unroll
                    for (int v = 0; v < U; ++v) y[v] = __ldcg(o + at[v]), z[v] = __ldcg(o + at[v] + ROWS);
#pragma unroll
                    for (int v = 0; v < U; ++v) {
                        const float f = wt[i * ROWS + at[v] % ROWS];
                        x[v][0] = __fmaf_rn(y[v].x, f, x[v][0]), x[v][1] = __fmaf_rn(y[v].y, f, x[v][1]);
                        x[v][2] = __fmaf_rn(y[v].z, f, x[v][2]), x[v][3] = __fmaf_rn(y[v].w, f, x[v][3]);
                        x[v][4] = __fmaf_rn(z[v].x, f, x[v][4]), x[v][5] = __fmaf_rn(z[v].y, f, x[v][5]);
                        x[v][6] = __fmaf_rn(z[v].z, f, x[v][6]), x[v][7] = __fmaf_rn(z[v].w, f, x[v][7]);
                    }
                }
#pragma unroll
                for (int v = 0; v < U; ++v) {
                    if (k0 + v * (NS / 32) >= pieces) continue;
                    const int r = at[v] % ROWS;
                    if (i0 + P < segs) {
                        float4* acc = (float4*)(slot(0) + 2 * ROWS) + at[v];
                        acc[0] = make_float4(x[v][0], x[v][1], x[v][2], x[v][3]);
                        acc[ROWS] = make_float4(x[v][4], x[v][5], x[v][6], x[v][7]);
                    } else if (r < rows) {
                        uint32_t o[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) o[e] = bf16x2(x[v][2 * e], x[v][2 * e + 1]);
                        *(uint4*)(out_row(a, u, r) + 4 * (at[v] / ROWS)) = make_uint4(o[0], o[1], o[2], o[3]);
                    }
                }
            }
        }
    }
};

template <int D>
__global__ void __launch_bounds__(NT, 1) kn12_kernel(const __grid_constant__ DtAttend a, float* part, int* counters,
                                                          long long probe) {
    using L = Lay<D>;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* sm = (unsigned char*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    Shared* sh = (Shared*)(sm + L::SH);
    const int tid = threadIdx.x, wid = tid >> 5;
    const int cta = blockIdx.x, ctas = gridDim.x;
    if (wid == 0) dt_tmem_alloc(&sh->tmem, 512);
    if (tid == 0) {
        for (int i = 0; i < STAGES; ++i) {
            dt_mbar_init(&sh->kfull[i], NC / 32);
            dt_mbar_init(&sh->vfull[i], NC / 32);
            dt_mbar_init(&sh->kfree[i], 2);
            dt_mbar_init(&sh->vfree[i], 2);
        }
        for (int i = 0; i < 4; ++i) {
            dt_mbar_init(&sh->sfull[i >> 1][i & 1], 1);
            dt_mbar_init(&sh->pfull[i >> 1][i & 1], TQ / 32);
        }
        for (int i = 0; i < RING; ++i) {
            dt_mbar_init(&sh->scfull[i], 2);
            dt_mbar_init(&sh->idfull[i], 1);
            dt_mbar_init(&sh->ringfree[i], 2);
        }
        for (int i = 0; i < SEGS; ++i) {
            dt_mbar_init(&sh->segfull[i], 1);
            dt_mbar_init(&sh->segfree[i], NS + 2 * NC + 2 + 32);
        }
        dt_mbar_init(&sh->qfull, NS);
        dt_mbar_init(&sh->drain[0], 1);
        dt_mbar_init(&sh->drain[1], 1);
        dt_mbar_init(&sh->probe, 1);
        dt_fence_mbar_init();
        sh->fail = sh->drain_fail[0] = sh->drain_fail[1] = 0;
    }
    if (tid < RING * 8) sh->ring[tid >> 3].id[tid & 7] = 0;  // a page for whoever gives up waiting for one
    dt_pdl_trigger();
    dt_pdl_wait();
    if (wid == 1) at_share<ROWS>(a, cta, ctas, MIN_SHARE, &sh->share);
    dt_tc_fence_before();
    __syncthreads();
    dt_tc_fence_after();
    const uint32_t tmem = sh->tmem;
    if (tid < NS) {
        set_regs<REG_SOFT>();
        Soft<D>::run(a, sm, sh, tmem, tid, cta, part, counters);
    } else if (tid < NS + 2 * NC) {
        set_regs<REG_CONV>();
        Conv<D>::run(a, sm, sh, (tid - NS) % NC, tid < NS + NC);
        at_zero_rest(a, cta, ctas, tid - NS, 2 * NC);
    } else {
        set_regs<REG_MMA>();
        constexpr int W0 = (NS + 2 * NC) / 32;
        if (wid == W0 || wid == W0 + 3)
            issue_slot<D>(sm, sh, __shfl_sync(0xffffffffu, tmem, 0), __shfl_sync(0xffffffffu, wid != W0, 0));
        if (tid == NS + 2 * NC + 32) walk_share(a, sh, cta);
        if (wid == W0 + 2) {
            if ((tid & 31) == 0 && !dt_probe_wait(&sh->probe, probe)) sh->fail = 1;
            __syncwarp();
            look_up<D>(a, sh, tid & 31);
        }
    }
    dt_tc_fence_before();
    __syncthreads();
    // The outputs are undefined then, and so are the counters in the workspace.
    if (tid == 0 && sh->fail)
        for (int b = 0; b < a.batch; ++b) atomicOr(&a.status[b], DT_DEV_TIMEOUT);
    if (wid == 0) {
        dt_tc_fence_after();
        dt_tmem_dealloc(tmem, 512);
    }
}

// Probe budget of the timeout path's test hook (0: off) in the calls made from now on.
std::atomic<long long> g_probe{0};

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
                              (int*)workspace, g_probe.load(std::memory_order_relaxed));
}

}  // namespace

void dt_kn12_set_probe(long long budget) { g_probe.store(budget, std::memory_order_relaxed); }

size_t dt_kn12_workspace(int D, int ctas) {
    return AT_MAX_CTAS * sizeof(int) + (size_t)ctas * 2 * ROWS * (D + 2) * sizeof(float);
}

cudaError_t dt_kn12_launch(const DtAttend& a, void* workspace, int ctas, cudaStream_t st) {
    return a.c.D == 64 ? launch<64>(a, workspace, ctas, st) : launch<128>(a, workspace, ctas, st);
}
