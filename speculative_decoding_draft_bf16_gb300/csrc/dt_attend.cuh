// dt_attend.cuh -- how tree attention is cut into work, shared by its kernels.
//
// Rows of one request and key head share their keys: row r of the M * G query
// rows (G = Hq / Hkv) is node r / G, head h * G + r % G.  A unit is a block of
// ROWS rows over all of its 128-token tiles, first the cached ones, then the
// tree's own.  All units of a call, laid end to end by cost, are divided evenly
// over the CTAs, so that ragged lengths balance and one long request still
// fills the GPU; a unit whose tiles fall to several CTAs is joined from their
// partial sums.  Every CTA derives the division by itself from len and n_nodes.
#pragma once

#include "dt_cache.cuh"
#include "dt_launch.h"

constexpr int AT_TILE = 128;      // tokens per tile
constexpr int AT_MAX_CTAS = 1024; // counters at the head of the workspace

struct AtReq {  // one request
    int len, n;         // cached tokens, rows (0 when something is out of range)
    int ctx;            // cached tiles
    int nqb;            // row blocks
    bool bad;
};

template <int ROWS>
struct AtPlan {
    // Cost of a tile of a block: blocks of more than half the rows cost two.
    static DT_DI int weight(int rows) { return 1; }
    static DT_DI AtReq req(const DtAttend& a, int b) {
        AtReq r;
        const int len = a.c.len[b], n = a.n_nodes ? a.n_nodes[b] : a.M;
        r.bad = len < 0 || (long long)len > (long long)a.c.max_pages * a.c.page || n < 0 || n > a.M;
        r.len = r.bad ? 0 : len;
        r.n = r.bad ? 0 : n;
        r.ctx = (r.len + AT_TILE - 1) / AT_TILE;
        r.nqb = (int)(((long long)r.n * (a.Hq / a.c.Hkv) + ROWS - 1) / ROWS);
        return r;
    }
    static DT_DI int block_rows(const DtAttend& a, const AtReq& r, int qb) {
        const long long left = (long long)r.n * (a.Hq / a.c.Hkv) - (long long)qb * ROWS;
        return left < ROWS ? (int)left : ROWS;
    }
    // New rows that block qb can see: all of them, or up to its last node in a chain.
    static DT_DI int block_new(const DtAttend& a, const AtReq& r, int qb) {
        if (a.mask) return r.n;
        const int G = a.Hq / a.c.Hkv;
        const long long last = ((long long)(qb + 1) * ROWS - 1) / G + 1;
        return last < r.n ? (int)last : r.n;
    }
    static DT_DI int block_tiles(const DtAttend& a, const AtReq& r, int qb) {
        return r.ctx + (block_new(a, r, qb) + AT_TILE - 1) / AT_TILE;
    }
    static DT_DI long long cost(const DtAttend& a, const AtReq& r) {
        if (r.nqb == 0) return 0;
        long long s = 0;
        if (a.mask) {
            const long long t = block_tiles(a, r, 0);
            s = t * (weight(ROWS) * (r.nqb - 1) + weight(block_rows(a, r, r.nqb - 1)));
        } else {
            for (int qb = 0; qb < r.nqb; ++qb) s += (long long)block_tiles(a, r, qb) * weight(block_rows(a, r, qb));
        }
        return s * a.c.Hkv;
    }
};

// The division's result in shared memory: the total cost, the CTAs that work,
// and where this CTA's share begins (request, and that request's first cost).
struct AtShare {
    long long total, beg, end, b0_at;
    int ctas, b0;
};

// One warp: the share of CTA c of grid.  min_share: least cost worth a CTA.
template <int ROWS>
DT_DI void at_share(const DtAttend& a, int c, int grid, int min_share, AtShare* sh) {
    using P = AtPlan<ROWS>;
    const int lane = threadIdx.x & 31;
    long long total = 0;
    for (int b = lane; b < a.batch; b += 32) {
        const AtReq r = P::req(a, b);
        if (r.bad && c == 0) atomicOr(&a.status[b], DT_DEV_BAD_CACHE);
        total += P::cost(a, r);
    }
    total = (long long)dt_warp_sum_u64((unsigned long long)total);
    long long g = total / min_share;
    g = g < 1 ? 1 : g > grid ? grid : g;
    const long long beg = c < g ? total * c / g : total, end = c < g ? total * (c + 1) / g : total;
    // the request that holds position beg
    long long at = 0;
    int b0 = a.batch;
    long long b0_at = total;
    for (int base = 0; base < a.batch && beg < end; base += 32) {
        const int b = base + lane;
        const long long mine = b < a.batch ? P::cost(a, P::req(a, b)) : 0;
        long long inc = mine;
        for (int o = 1; o < 32; o <<= 1) {
            const long long t = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += t;
        }
        const bool hit = at + inc > beg;
        const unsigned m = __ballot_sync(0xffffffffu, hit);
        if (m) {
            const int l = __ffs(m) - 1;
            b0 = base + l;
            b0_at = at + __shfl_sync(0xffffffffu, inc - mine, l);
            break;
        }
        at += __shfl_sync(0xffffffffu, inc, 31);
    }
    if (lane == 0) {
        sh->total = total;
        sh->beg = beg;
        sh->end = end;
        sh->ctas = (int)g;
        sh->b0 = b0;
        sh->b0_at = b0_at;
    }
}

// Walks a CTA's segments: the tiles [t0, t1) of one unit each.
template <int ROWS, int ATOM>
struct AtWalk {
    using P = AtPlan<ROWS>;
    int b, qb, h;       // the unit
    AtReq r;
    int rows, nt, w;    // its rows, tiles and tile cost
    long long at;       // its first cost position
    int t0, t1;         // this CTA's tiles of it
    int first, segs;    // the CTA that holds tile 0, and how many CTAs share it

    DT_DI void unit(const DtAttend& a) {
        rows = P::block_rows(a, r, qb);
        nt = P::block_tiles(a, r, qb);
        w = P::weight(rows);
    }
    DT_DI void start(const DtAttend& a, const AtShare& s) {
        b = s.b0;
        qb = h = 0;
        at = s.b0_at;
        t1 = 0;
        if (b >= a.batch) return;
        r = P::req(a, b);
        unit(a);
        // whole units before the share (blocks hold Hkv units of one cost)
        while (at + (long long)a.c.Hkv * nt * w <= s.beg) {
            at += (long long)a.c.Hkv * nt * w;
            ++qb;
            unit(a);
        }
        h = (int)((s.beg - at) / ((long long)nt * w));
        at += (long long)h * nt * w;
    }
    static DT_DI int owner(const AtShare& s, long long x) { return (int)(((x + 1) * s.ctas - 1) / s.total); }
    // The next segment, or false.  A unit of at most ATOM tiles is not split.
    DT_DI bool next(const DtAttend& a, const AtShare& s, int c) {
        while (b < a.batch && at < s.end) {
            if (nt <= ATOM) {
                first = owner(s, at);
                segs = 1;
                t0 = 0;
                t1 = first == c ? nt : 0;
            } else {
                const long long lo = s.beg - at, hi = s.end - at;
                t0 = lo <= 0 ? 0 : (int)((lo + w - 1) / w);
                t1 = (hi + w - 1) / w < nt ? (int)((hi + w - 1) / w) : nt;
                first = owner(s, at);
                segs = owner(s, at + (long long)w * (nt - 1)) - first + 1;
            }
            if (t1 > t0) return true;
            step(a);
        }
        return false;
    }
    DT_DI void step(const DtAttend& a) {  // to the next unit
        at += (long long)nt * w;
        if (++h < a.c.Hkv) return;
        h = 0;
        ++qb;
        while (qb >= r.nqb) {
            qb = 0;
            if (++b >= a.batch) return;
            r = P::req(a, b);
        }
        unit(a);
    }
};

// The bits of new rows [m0, m0 + 32) that row `node` sees, rows below n only.
DT_DI uint32_t at_mask_word(const DtAttend& a, int b, int node, int m0, int n) {
    uint32_t bits;
    if (a.mask)
        bits = m0 < n ? a.mask[((size_t)b * a.M + node) * ((a.M + 31) / 32) + m0 / 32] : 0u;
    else
        bits = node >= m0 + 31 ? 0xFFFFFFFFu : node < m0 ? 0u : (2u << (node - m0)) - 1u;
    const int left = n - m0;
    return left >= 32 ? bits : left <= 0 ? 0u : bits & ((1u << left) - 1u);
}

// Position of a new row in the rotation tables; out of range: flagged, 0.
DT_DI int at_position(const DtAttend& a, int b, int len, int node) {
    const long long at = (long long)len + (a.pos ? a.pos[(size_t)b * a.M + node] : node);
    if (a.rope.rot && (at < 0 || at >= a.rope.max_pos)) {
        atomicOr(&a.status[b], DT_DEV_BAD_CACHE);
        return 0;
    }
    return (int)at;
}

// Zeros for the output rows past n_nodes (all rows of a request out of range),
// spread over the grid.
DT_DI void at_zero_rest(const DtAttend& a, int cta, int ctas, int tid, int nt) {
    const size_t chunks = (size_t)a.Hq * a.c.D / 8;
    for (int b = 0; b < a.batch; ++b) {
        const int n = AtPlan<16>::req(a, b).n;
        uint4* o = (uint4*)a.out + ((size_t)b * a.M + n) * chunks;
        const size_t m = (size_t)(a.M - n) * chunks;
        for (size_t i = (size_t)cta * nt + tid; i < m; i += (size_t)ctas * nt) o[i] = make_uint4(0u, 0u, 0u, 0u);
    }
}
