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

// BITS: of the cache's codes.
template <int ROWS, int BITS = 8>
struct AtPlan {
    // Cost of a tile of a block; one of at most half of 256 rows costs less (of e4m3 3.5
    // against 4.2 thousand clocks measured, of 4 bits 2.2 against 3.3).
    static constexpr uint32_t FULL = ROWS == 256 ? (BITS == 4 ? 6 : 5) : 1, PART = ROWS == 256 ? 4 : 1;
    // What starting on a unit costs: its queries, its new rows, its sums' way out.  64 trees
    // of 61 nodes with 14, 20, 26: 208, 183, 188 us, over 4 bits with 24, 30, 34: 132, 128,
    // 127; 64 single tokens with 1, 2, 3: 240, 233, 234.
    static constexpr uint32_t HEAD = ROWS == 256 ? (BITS == 4 ? 30 : 20) : 2;
    // The same of 16 rows over 4 bits when every CTA has work (see AtShareLead): a unit's start
    // and end take the time of so many tiles then.  64 single tokens with 2, 5, 6, 7, 8: 144,
    // 129, 129, 130, 136 us; calls that do not fill the GPU need the smaller one (one token
    // 12.5 us, 15 with 6).
    static constexpr uint32_t HEAD_FULL = 6;
    // Pieces of so few tiles at a unit's end are not worth starting on (one tree of 257
    // nodes over 8000 tokens without this 92 us, with 2 77, with 4 81).
    static constexpr int SNAP = ROWS == 256 ? 2 : 1;
    static DT_DI uint32_t weight(int rows) { return rows > ROWS / 2 ? FULL : PART; }
    static DT_DI AtReq req(const DtAttend& a, int b) {
        AtReq r;
        const int len = a.c.len[b], n = a.n_nodes ? a.n_nodes[b] : a.M;
        r.bad = len < 0 || len > a.c.max_pages * a.c.page || n < 0 || n > a.M;
        r.len = r.bad ? 0 : len;
        r.n = r.bad ? 0 : n;
        r.ctx = (r.len + AT_TILE - 1) / AT_TILE;
        r.nqb = (r.n * a.G + ROWS - 1) / ROWS;
        return r;
    }
    static DT_DI int block_rows(const DtAttend& a, const AtReq& r, int qb) { return min(r.n * a.G - qb * ROWS, ROWS); }
    // New rows that block qb can see: all of them, or up to its last node in a chain.
    static DT_DI int block_new(const DtAttend& a, const AtReq& r, int qb) {
        return a.mask ? r.n : min(((qb + 1) * ROWS - 1) / a.G + 1, r.n);
    }
    static DT_DI int block_tiles(const DtAttend& a, const AtReq& r, int qb) {
        return r.ctx + (block_new(a, r, qb) + AT_TILE - 1) / AT_TILE;
    }
    static DT_DI uint32_t cost(const DtAttend& a, const AtReq& r, uint32_t head = HEAD) {
        if (r.nqb == 0) return 0;
        uint32_t s = block_tiles(a, r, r.nqb - 1) * weight(block_rows(a, r, r.nqb - 1)) + r.nqb * head;
        if (a.mask) {
            s += (r.nqb - 1) * block_tiles(a, r, 0) * FULL;
        } else {
#pragma unroll 1
            for (int qb = 0; qb < r.nqb - 1; ++qb) s += block_tiles(a, r, qb) * FULL;
        }
        return s * a.c.Hkv;
    }
};

// The division's result in shared memory: `ctas` CTAs work; the first `rest` of
// them take each + 1, the others `each`; this CTA's share is [beg, end) and
// begins in request b0, whose own cost begins at b0_at.
struct AtShare {
    uint32_t beg, end, b0_at, each, rest;
    int ctas, b0;
    AtReq r0;  // of request b0
    DT_DI uint32_t start_of(uint32_t c) const { return c * each + min(c, rest); }
    DT_DI int owner(uint32_t x) const {  // of cost position x
        const uint32_t wide = rest * (each + 1);
        return (int)(x < wide ? x / (each + 1) : rest + (x - wide) / each);
    }
};

// The cost of starting on a unit that the walk counts with.
template <class Plan>
DT_DI uint32_t at_head(const AtShare&) { return Plan::HEAD; }

// A division with a choice of HEAD, and with LEAD / 256 of a share more for each CTA of the
// first half when all of a grid of two CTAs to an SM work: of two CTAs on an SM the one that
// came first issues first.
template <int LEAD>
struct AtShareLead : AtShare {
    uint32_t half;  // CTAs of the first half; 0: shares are equal
    uint32_t head;
    DT_DI uint32_t more() const { return each * LEAD / 256; }
    DT_DI uint32_t start_of(uint32_t c) const { return AtShare::start_of(c) + (c < half ? c : 2 * half - c) * (half ? more() : 0u); }
    DT_DI int owner(uint32_t x) const {
        if (half == 0) return AtShare::owner(x);
        const uint32_t wide = half * (each + more());
        int c = (int)(x < wide ? x / (each + more() + 1) : half + (x - wide) / (each - more() + 1));  // near it
        c = min(c, ctas - 1);
        while (start_of(c) > x) --c;
        while (c + 1 < ctas && start_of(c + 1) <= x) ++c;
        return c;
    }
};
template <class Plan, int LEAD>
DT_DI uint32_t at_head(const AtShareLead<LEAD>& s) { return s.head; }

// How many CTAs work, and the cost of all units (whose tiles cost `tiles`).  A division with
// a choice takes the larger head when that still gives every CTA of the grid a share.
template <class Plan>
DT_DI void at_choose(AtShare& s, uint32_t tiles, uint32_t units, uint32_t grid, uint32_t min_share, uint32_t& total) {
    total = tiles + units * Plan::HEAD;
    s.ctas = (int)max(1u, min(total / min_share, grid));
}
template <class Plan, int LEAD>
DT_DI void at_choose(AtShareLead<LEAD>& s, uint32_t tiles, uint32_t units, uint32_t grid, uint32_t min_share, uint32_t& total) {
    const uint32_t more = Plan::HEAD_FULL - Plan::HEAD;
    const bool full = tiles + units * Plan::HEAD_FULL >= grid * (min_share + more);
    s.head = full ? Plan::HEAD_FULL : Plan::HEAD;
    total = tiles + units * s.head;
    s.ctas = (int)max(1u, min(total / (min_share + (full ? more : 0u)), grid));
    s.half = full && grid % 2 == 0 ? grid / 2 : 0;
}

// One warp: the share of CTA c of grid.  min_share: least cost worth a CTA.
template <int ROWS, int BITS = 8, class Share>
DT_DI void at_share(const DtAttend& a, uint32_t c, uint32_t grid, uint32_t min_share, Share* sh) {
    using P = AtPlan<ROWS, BITS>;
    const int lane = threadIdx.x & 31;
    uint32_t tiles = 0, units = 0, total;
    AtReq r;
#pragma unroll 1
    for (int b = lane; b < a.batch; b += 32) {
        r = P::req(a, b);
        if (r.bad && c == 0) atomicOr(&a.status[b], DT_DEV_BAD_CACHE);
        tiles += P::cost(a, r, 0);
        units += r.nqb * a.c.Hkv;
    }
    const uint32_t own_tiles = tiles, own_units = units;  // with up to 32 requests, of the lane's only one
    Share s;
    at_choose<P>(s, __reduce_add_sync(0xffffffffu, tiles), __reduce_add_sync(0xffffffffu, units), grid, min_share, total);
    const uint32_t head = at_head<P>(s), own = own_tiles + own_units * head;
    s.each = total / s.ctas;
    s.rest = total % s.ctas;
    s.beg = c < s.ctas ? s.start_of(c) : total;
    s.end = c < s.ctas ? s.start_of(c + 1) : total;
    // the request that holds position beg
    s.b0 = a.batch;
    s.b0_at = total;
    uint32_t at = 0;
#pragma unroll 1
    for (int base = 0; base < a.batch && s.beg < s.end; base += 32) {
        const int b = base + lane;
        uint32_t mine = own;
        if (a.batch > 32) {
            mine = 0;
            if (b < a.batch) {
                r = P::req(a, b);
                mine = P::cost(a, r, head);
            }
        }
        const uint32_t inc = (uint32_t)dt_warp_incl_scan((int)mine);
        const unsigned m = __ballot_sync(0xffffffffu, at + inc > s.beg);
        if (m) {
            const int l = __ffs(m) - 1;
            s.b0 = base + l;
            s.b0_at = at + __shfl_sync(0xffffffffu, inc - mine, l);
            s.r0.len = __shfl_sync(0xffffffffu, r.len, l);
            s.r0.n = __shfl_sync(0xffffffffu, r.n, l);
            s.r0.ctx = __shfl_sync(0xffffffffu, r.ctx, l);
            s.r0.nqb = __shfl_sync(0xffffffffu, r.nqb, l);
            s.r0.bad = false;
            break;
        }
        at += __shfl_sync(0xffffffffu, inc, 31);
    }
    if (lane == 0) *sh = s;
}

// Walks a CTA's segments: the tiles [t0, t1) of one unit each.
template <int ROWS, int ATOM, int BITS = 8>
struct AtWalk {
    using P = AtPlan<ROWS, BITS>;
    int b, qb, h;       // the unit
    AtReq r;
    int rows, nt;       // its rows and tiles
    uint32_t head;      // what starting on a unit costs
    uint32_t w, at;     // its tile cost and first cost position; tile 0 costs `head` more
    int t0, t1;         // this CTA's tiles of it
    int first, segs;    // the CTA that holds tile 0, and how many CTAs share it

    DT_DI void unit(const DtAttend& a) {
        rows = P::block_rows(a, r, qb);
        nt = P::block_tiles(a, r, qb);
        w = P::weight(rows);
    }
    template <class Share>
    DT_DI void start(const DtAttend& a, const Share& s) {
        head = at_head<P>(s);
        b = s.b0;
        qb = h = 0;
        at = s.b0_at;
        if (b >= a.batch) return;
        r = s.r0;
        unit(a);
        // whole blocks before the share (Hkv units of one cost each)
#pragma unroll 1
        while (at + a.c.Hkv * (nt * w + head) <= s.beg) {
            at += a.c.Hkv * (nt * w + head);
            ++qb;
            unit(a);
        }
        h = (int)((s.beg - at) / (nt * w + head));
        at += h * (nt * w + head);
    }
    // The first tile that starts at cost position x or later; no cut leaves a piece
    // of SNAP tiles or fewer at either end of the unit.
    DT_DI int tile_from(uint32_t x) const {
        if (x <= at + head + P::SNAP * w) return 0;
        const int t = (int)((x - at - head + w - 1) / w);
        return t >= nt - P::SNAP ? nt : t;
    }
    // The next segment, or false.  A unit of at most ATOM tiles is not split.
    template <class Share>
    DT_DI bool next(const DtAttend& a, const Share& s, int c) {
        static_assert(ATOM >= 2 * P::SNAP, "a cut is near one end of a unit only");
#pragma unroll 1
        while (b < a.batch && at < s.end) {
            first = s.owner(at);
            if (nt <= ATOM) {
                segs = 1;
                t0 = 0;
                t1 = first == c ? nt : 0;
            } else {
                t0 = tile_from(s.beg);
                t1 = tile_from(s.end);
                int last = s.owner(at + head + w * (nt - 1));
                if (tile_from(s.start_of(first + 1)) == 0) ++first;
                if (tile_from(s.start_of(last)) == nt) --last;
                segs = last - first + 1;
            }
            if (t1 > t0) return true;
            step(a);
        }
        return false;
    }
    DT_DI void step(const DtAttend& a) {  // to the next unit
        at += nt * w + head;
        if (++h < a.c.Hkv) return;
        h = 0;
        ++qb;
#pragma unroll 1
        while (qb >= r.nqb) {
            qb = 0;
            if (++b >= a.batch) return;
            r = P::req(a, b);
        }
        unit(a);
    }
};

// Factor from a product of codes to a score in base 2, as a normal number: a masked
// score is -infinity, which a factor of zero would make NaN.  What the rounding up
// adds to a score is below 2^-100.  NaN (a block that is not finite) stays.
DT_DI float at_factor(float row, float keys) {
    float f;
    asm("max.NaN.f32 %0, %1, 0f00800000;" : "=f"(f) : "f"(__fmul_rn(row, keys)));
    return f;
}

// Exponent of a row from the bits of its largest magnitude; of a row of zeros, 0.  Least: of keys
// down to where a scale is a normal number; of values to 2^-57 (what lies below counts as small
// against 1), so that sums over rows and pages keep their range.
DT_DI int at_row_exponent(uint32_t big, bool keys) {
    return big == 0u ? 0 : min(max((int)(big >> 23) - 127, keys ? -126 : -57), 126);
}

// Over 4 bits the values of new rows are scaled by 2^-e, one e for all that come together, and
// their products join sums that are held 2^-e as large: P, in fp16, follows the weights alone,
// and fp32 sums have the range that P has not.  (With e in P's exponent, tokens whose values need a
// smaller e lose bits of their weights, and beside 2^30 all of them.)
//   at_value_exponent: of rows whose largest magnitudes have the exponents lo to hi.  fp16 holds
// them without a scale from 2^-8 (which keeps 2^-24) up to 2^15; else the largest comes to 2^14.
//   at_value_row: a row's own, where it lies more than 18 octaves below the largest, of 2^15 or
// more: 2^-4 then keeps what lies 2^-20 below its largest, and P takes the difference, not below
// AT_LEAST_SHIFT, so that the weight itself stays a normal number.  Such a row's weight has all
// its bits up to 2^37 below the largest value and some up to 2^48.
//   AT_KEEP: how far a later e may be below an earlier one: sums of 2^20 rows of up to 2^128, with
// weights of up to 2^13, then stay below 2^125.
constexpr int AT_KEEP = 76, AT_LEAST_SHIFT = -60;
DT_DI int at_value_exponent(int hi, int lo) { return hi < 15 && lo >= -8 ? 0 : max(hi - 14, -57); }
DT_DI int at_value_row(int x, int e) { return e > 0 && max(x, -10) < e - 4 ? max(x, -10) + 4 : e; }

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

// Zeros for the output rows past n_nodes, spread over the grid: a warp reads 32
// requests' counts at a time and takes every (nt / 32)th of those.
DT_DI void at_zero_rest(const DtAttend& a, int cta, int ctas, int tid, int nt) {
    if (!a.n_nodes) return;  // a request out of range then has undefined rows
    const int lane = tid & 31, w = tid >> 5;
    const size_t chunks = (size_t)a.Hq * a.c.D / 8;
#pragma unroll 1
    for (int base = 0; base < a.batch; base += 32) {
        const int mine = base + lane < a.batch ? AtPlan<16>::req(a, base + lane).n : a.M;
#pragma unroll 1
        for (int k = w; k < 32; k += nt / 32) {
            const int n = __shfl_sync(0xffffffffu, mine, k);
            uint4* o = (uint4*)a.out + ((size_t)(base + k) * a.M + n) * chunks;
            const size_t m = (size_t)(a.M - n) * chunks;
#pragma unroll 1
            for (size_t i = (size_t)cta * 32 + lane; i < m; i += (size_t)ctas * 32) o[i] = make_uint4(0u, 0u, 0u, 0u);
            __syncwarp();
        }
    }
}
