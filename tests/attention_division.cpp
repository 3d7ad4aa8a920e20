// Host check of tree attention's division of the work (csrc/dt_attend.cuh): over random
// batches every tile of every unit falls to one CTA, in order, the CTAs of a unit are
// neighbours that agree on the first of them and on their number, and no CTA has two parts
// that would share a slot.  Only the share's search for its first request is the test's own.
//   usage: division BATCHES;  -DK_ROWS -DK_ATOM -DK_MIN_SHARE: the constants of the kernel
#include <algorithm>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <map>
#include <random>
#include <tuple>
#include <vector>

#include "dtree.h"

using std::max;
using std::min;
static inline unsigned min(unsigned a, int b) { return a < (unsigned)b ? a : b; }

struct DtAttend {
    dt_kv_cache c;
    dt_rope rope;
    int batch, M, Hq, G;
    dt_rows q, k, v;
    const uint32_t* mask;
    const int32_t* pos;
    const int32_t* n_nodes;
    float scale;
    void* out;
    int32_t* status;
};

#define DT_DI inline
#include "division_body.h"

struct Part {
    int t0, t1, nt, cta, first, segs;
};

static int fail(const char* what, int batch) {
    printf("batch %d: %s\n", batch, what);
    return 1;
}

int main(int, char** argv) {
    using Plan = AtPlan<K_ROWS>;
    std::mt19937 g(1);
    auto rnd = [&](int n) { return (int)(g() % (unsigned)n); };
    for (int it = 0; it < atoi(argv[1]); ++it) {
        const int batch = rnd(10) ? 1 + rnd(6) : 33 + rnd(60);
        std::vector<int> len(batch), n(batch);
        const int page = 16 << rnd(4), M = 1 + rnd(rnd(2) ? 40 : 1100), G = 1 + rnd(16), Hkv = 1 + rnd(5);
        int pages = 1;
        for (int b = 0; b < batch; ++b) {
            len[b] = rnd(40) == 0 ? rnd(70000) : rnd(3) ? rnd(3000) : rnd(5);
            n[b] = rnd(4) ? 1 + rnd(M) : rnd(2) ? M : 0;
            pages = max(pages, len[b] / page + 1);
        }
        if (rnd(5) == 0) len[rnd(batch)] = -1;  // out of range: no work
        uint32_t some;
        DtAttend a{};
        a.c.page = page, a.c.Hkv = Hkv, a.c.max_pages = pages, a.c.len = len.data();
        a.batch = batch, a.M = M, a.G = G, a.Hq = G * Hkv, a.n_nodes = n.data(), a.mask = rnd(2) ? &some : nullptr;
        const int grid = 1 + rnd(310);
        long long total = 0;
        for (int b = 0; b < batch; ++b) total += Plan::cost(a, Plan::req(a, b));
        const int ctas = (int)min<long long>(max<long long>(total / K_MIN_SHARE, 1), grid);
        std::map<std::tuple<int, int, int>, std::vector<Part>> got;
        for (int c = 0; c < grid; ++c) {
            AtShare s;
            s.ctas = ctas, s.each = total / ctas, s.rest = total % ctas;
            s.beg = c < ctas ? s.start_of(c) : total, s.end = c < ctas ? s.start_of(c + 1) : total;
            s.b0 = batch, s.b0_at = total;
            long long at = 0;
            for (int b = 0; b < batch && s.beg < s.end; ++b) {
                const AtReq r = Plan::req(a, b);
                if (at + Plan::cost(a, r) > s.beg) {
                    s.b0 = b, s.b0_at = at, s.r0 = r;
                    break;
                }
                at += Plan::cost(a, r);
            }
            AtWalk<K_ROWS, K_ATOM> u;
            u.start(a, s);
            int slots = 0;
            for (; u.next(a, s, c); u.step(a)) {
                got[{u.b, u.qb, u.h}].push_back({u.t0, u.t1, u.nt, c, u.first, u.segs});
                const int slot = u.t0 == 0 && u.t1 == u.nt ? 0 : 1 << (u.t0 == 0);
                if (slots & slot) return fail("two parts in one slot", it);
                slots |= slot;
            }
        }
        std::map<int, int> counters;
        size_t units = 0;
        for (int b = 0; b < batch; ++b) {
            const AtReq r = Plan::req(a, b);
            for (int qb = 0; qb < r.nqb; ++qb)
                for (int h = 0; h < Hkv; ++h, ++units) {
                    const std::vector<Part>& parts = got[{b, qb, h}];
                    int t = 0, i = 0;
                    for (const Part& p : parts) {
                        if (p.t0 != t || p.nt != Plan::block_tiles(a, r, qb)) return fail("a gap or an overlap", it);
                        if (p.segs != (int)parts.size() || p.first != parts[0].cta || p.cta != p.first + i)
                            return fail("CTAs that do not agree", it);
                        t = p.t1, ++i;
                    }
                    if (t != Plan::block_tiles(a, r, qb)) return fail("tiles left out", it);
                    if (i > 1 && counters[parts[0].first]++) return fail("two units on one counter", it);
                }
        }
        if (units != got.size()) return fail("a unit that is not there", it);
    }
    printf("ok\n");
}
