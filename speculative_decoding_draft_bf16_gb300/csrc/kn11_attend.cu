// kn11_attend.cu -- tree attention for up to 16 query rows per key head (single
// tokens and small trees), bound by the reading of the cache (dt_tree_attention).
//
// A CTA streams runs of 128-token tiles, 16 tokens to each of its 8 warps.  A
// lane copies the bytes that it will need itself to its own places in shared
// memory (cp.async, STAGES tiles ahead: up to 192 KB of an SM's loads are in
// flight, and nothing is waited for but the lane's own copies), turns the e4m3
// codes into fp16 in registers and feeds 16 x 8 x 16 MMAs, tokens and columns on
// the side of 16, NR groups of 8 query rows on the other:
//   S' = K Q'    a lane's 32 bytes of a token serve as the K-fragment of all
//                steps: which elements of the head a step takes is free, as long
//                as Q's fragments are cut alike;
//   O' += V' P'  P's fragments are S's, transposed 8 x 8 at a time; a lane reads 16
//                columns of four tokens and pairs the tokens' bytes before it
//                converts them.
// These narrow products do not fill a tcgen05 tile (16 rows of 128), and the cache's
// bytes are to bound the time; the same calls on 128-row tiles take 364 us against 264 at
// 16 rows (64 requests, contexts to 16000), 31.6 against 22.9 for one request over 4000.
// With the rows on the side of 16, single tokens paid for 12 idle rows in MMAs and
// exponentials, a third of all instructions: 276 us instead of 233.
//   Scales: P holds 2^(t + log2 vs - m) for scores t in base 2, the row sum adds p / vs
// (value scales from 2^-100 on, or the sum leaves fp32), and m moves only when the maximum
// has grown by more than 8.  The warps' sums are joined in shared memory, the CTAs' in the
// workspace.
//
// On the device (calls in a graph): 64 single tokens, 32 heads on 8, over contexts of 1001
// to 16384 (1.14 GB) 228 to 231 us, 4.9 TB/s (73% of a copy's rate).  Equal shares end
// between 165 and 228 us, by where on the chip an SM lies: that spread, not the loop, is
// what is left.  One token over 1000: 15.9 us, the latency of the share, pages, copies, new
// row and join in turn (15.6 before each new row had a scale of its own).
#include "dt_attend.cuh"

namespace {

constexpr int ROWS = 16, NW = 8, NT = NW * 32;
// One token over 1000 with 4 and 4: 16.7 us; 6 and 6: 19.5; 10 and 8: 17.3; 8 and 8: 22.6
// (long contexts do not notice).
constexpr int ATOM = 4;              // tiles of the longest unit that is not split
constexpr uint32_t MIN_SHARE = 4;    // least cost worth a CTA: the start and two tiles
static_assert(MIN_SHARE >= AtPlan<ROWS>::HEAD + (AtPlan<ROWS>::SNAP + 1) * AtPlan<ROWS>::FULL,
              "every CTA between a unit's ends has a tile of it");
constexpr float LOG2E = 1.44269504088896340736f;
constexpr float HEADROOM = 5.f, LAZY = 8.f;

// Three tiles in flight of 4 KB to a warp, two CTAs to an SM; three CTAs with two tiles
// each are slower (246 : 233 us).
template <int D>
struct Lay {
    static constexpr int KC = D / 64;             // 16-byte pieces of a token's keys per lane
    static constexpr int VB = D / 8;              // bytes of a token's values per lane
    static constexpr int STAGES = D == 128 ? 3 : 6;
    static constexpr int KBYTES = 2 * KC * 512, BYTES = KBYTES + 4 * VB * 32;  // per warp and stage
    static constexpr size_t FIFO = (size_t)NW * STAGES * BYTES;
    static constexpr size_t JOIN = (size_t)NW * ROWS * D * 4;
    static constexpr size_t SMEM = FIFO > JOIN ? FIFO : JOIN;
};

struct Shared {
    AtShare share;
    float m[NW][ROWS], l[NW][ROWS], w[NW][ROWS];
    int last;
};

DT_DI uint32_t f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
DT_DI uint32_t bf16x2(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *(const uint32_t*)&v;
}
DT_DI void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
        "%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <int BYTES>
DT_DI void copy_async(uint32_t dst, const void* src) {
    if (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(BYTES) : "memory");
}
template <int WORDS>
DT_DI void lds(uint32_t addr, uint32_t (&w)[WORDS]) {
    if constexpr (WORDS == 4)
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(addr) : "memory");
    else
        asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr) : "memory");
}

// The transpose of an 8 x 8 matrix of 16-bit elements, two of a row to a lane.
DT_DI uint32_t transposed8x8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

template <int D, int NR>
struct Stream {
    using L = Lay<D>;
    using Walk = AtWalk<ROWS, ATOM>;
    static constexpr int KS = D / 16;  // steps of K Q'
    static constexpr int NV = D / 8;   // columns of a lane in V' P': NV * g + j; two to an MMA

    uint32_t qs;  // Q's fragments in shared memory, [KS / 2][NR][32 lanes][4 words]
    // of rows 2t + e + 8i (g, t: the lane's group of 4 and place in it)
    float rowc[NR][2], m[NR][2], l[NR][2];
    float o[NV / 2][NR][4];  // [j / 2][i][2 * (j % 2) + e]

    // 16 elements from 16 * c of a head vector, rotated.
    static DT_DI void pick16(const uint16_t* row, int c, const dt_rope& r, int at, float (&x)[16]) {
        DtTurned8<uint16_t> raw[2];
        float y[8];
#pragma unroll
        for (int i = 0; i < 2; ++i) raw[i].load(row, 2 * c + i, r, at);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            raw[i].values(2 * c + i, r, y);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[8 * i + e] = y[e];
        }
    }

    DT_DI void queries(const DtAttend& a, const Walk& u, int lane) {
        const int g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            const int r = g + 8 * i;
            float x[L::KC][16];
            uint32_t big = 0;
#pragma unroll
            for (int j = 0; j < L::KC; ++j) {
#pragma unroll
                for (int e = 0; e < 16; ++e) x[j][e] = 0.f;
            }
            if (r < u.rows) {
                const int n = r / a.G;
                const uint16_t* p = (const uint16_t*)a.q.ptr + u.b * a.q.stride_b + n * a.q.stride_n +
                                    (u.h * a.G + r % a.G) * a.q.stride_h;
                const int at = a.rope.rot ? at_position(a, u.b, u.r.len, n) : 0;
#pragma unroll
                for (int j = 0; j < L::KC; ++j) {
                    pick16(p, t + 4 * j, a.rope, at, x[j]);
#pragma unroll
                    for (int e = 0; e < 16; ++e) big = max(big, __float_as_uint(x[j][e]) & 0x7FFFFFFFu);
                }
            }
            big = max(big, __shfl_xor_sync(0xffffffffu, big, 1));
            big = max(big, __shfl_xor_sync(0xffffffffu, big, 2));
            int ex = (int)(big >> 23) - 127;  // largest magnitude in [2^ex, 2^(ex+1))
            ex = big >= 0x7F800000u ? 0 : min(max(ex, -100), 126);  // 2^-ex is a normal number
            const float f = dt_pow2(-ex), rc = __fmul_rn(__fmul_rn(a.scale, LOG2E), dt_pow2(ex));
            rowc[i][0] = __shfl_sync(0xffffffffu, rc, 8 * t);
            rowc[i][1] = __shfl_sync(0xffffffffu, rc, 8 * t + 4);
            // every warp writes the same words
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                const float* y = x[s >> 2] + 4 * (s & 3);
                asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(qs + (((s >> 1) * NR + i) * 32 + lane) * 16 + (s & 1) * 8),
                             "r"(f16x2(__fmul_rn(y[0], f), __fmul_rn(y[1], f))),
                             "r"(f16x2(__fmul_rn(y[2], f), __fmul_rn(y[3], f)))
                             : "memory");
            }
        }
    }

    // Scores of 16 tokens, masked (c[i][2k + e]: token g + 8k, row 2t + e + 8i), to
    // probabilities as the fragments of P'; ks, lv, iv: the 16 tokens', or (T = 2) of
    // tokens g and g + 8.
    template <int T>
    DT_DI void weigh(float (&c)[NR][4], const float (&ks)[T], const float (&lv)[T], const float (&iv)[T], uint32_t (&p)[NR][2]) {
        const float NEG_INF = -__int_as_float(0x7F800000);
        float k[NR][2][T], top[NR][2];
        bool grown = false;
#pragma unroll
        for (int i = 0; i < NR; ++i) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int h = 0; h < T; ++h) k[i][e][h] = at_factor(rowc[i][e], ks[h]);
                if constexpr (T == 1) top[i][e] = __fmaf_rn(fmaxf(c[i][e], c[i][2 + e]), k[i][e][0], lv[0]);
                else top[i][e] = fmaxf(__fmaf_rn(c[i][e], k[i][e][0], lv[0]), __fmaf_rn(c[i][2 + e], k[i][e][1], lv[1]));
                grown |= top[i][e] > m[i][e] + (HEADROOM + LAZY);
            }
        }
        if (__any_sync(0xffffffffu, grown)) {
#pragma unroll
            for (int i = 0; i < NR; ++i) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float x = top[i][e];
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
                    const float to = x > m[i][e] + (HEADROOM + LAZY) ? x - HEADROOM : m[i][e];
                    const float f = to == m[i][e] ? 1.f : dt_ex2_approx(m[i][e] - to);  // m = -inf: 0
                    m[i][e] = to;
                    l[i][e] = __fmul_rn(l[i][e], f);
#pragma unroll
                    for (int j = 0; j < NV / 2; ++j) {
                        o[j][i][e] = __fmul_rn(o[j][i][e], f);
                        o[j][i][2 + e] = __fmul_rn(o[j][i][2 + e], f);
                    }
                }
            }
        }
#pragma unroll
        for (int i = 0; i < NR; ++i) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float mu = m[i][e] == NEG_INF ? 0.f : m[i][e];
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    c[i][2 * h + e] = dt_ex2_approx(__fmaf_rn(c[i][2 * h + e], k[i][e][h % T], __fsub_rn(lv[h % T], mu)));
                if constexpr (T == 1) l[i][e] = __fmaf_rn(__fadd_rn(c[i][e], c[i][2 + e]), iv[0], l[i][e]);
                else l[i][e] = __fmaf_rn(c[i][2 + e], iv[1], __fmaf_rn(c[i][e], iv[0], l[i][e]));
            }
            p[i][0] = transposed8x8(f16x2(c[i][0], c[i][1]));
            p[i][1] = transposed8x8(f16x2(c[i][2], c[i][3]));
        }
    }

    // The staged 16 tokens at `st`, of which the first `left` exist.
    DT_DI void tile(uint32_t st, int lane, int left, float ks, float lv, float iv) {
        const int g = lane >> 2;
        const uint32_t my = st + lane * 16;
        float c[NR][4] = {};
#pragma unroll
        for (int j = 0; j < L::KC; ++j) {
            uint32_t w[2][4];
            lds<4>(my + j * 512, w[0]);
            lds<4>(my + (L::KC + j) * 512, w[1]);
#pragma unroll
            for (int s = 0; s < 4; s += 2) {
                uint32_t f[2][4], q[NR][4];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    dt_e4m3x4_to_f16x4(w[0][s + k], f[k][0], f[k][2]);
                    dt_e4m3x4_to_f16x4(w[1][s + k], f[k][1], f[k][3]);
                }
#pragma unroll
                for (int i = 0; i < NR; ++i) {
                    lds<4>(qs + (((4 * j + s) / 2 * NR + i) * 32 + lane) * 16, q[i]);
                    mma(c[i], f[0], q[i][0], q[i][1]);
                    mma(c[i], f[1], q[i][2], q[i][3]);
                }
            }
        }
        if (left < 16) {
#pragma unroll
            for (int i = 0; i < NR; ++i) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (g + 8 * (k >> 1) >= left) c[i][k] = -__int_as_float(0x7F800000);
            }
        }
        uint32_t p[NR][2];
        weigh<1>(c, {ks}, {lv}, {iv}, p);
        // values of tokens 2t, 2t + 1, 2t + 8, 2t + 9
        constexpr int VW = L::VB / 4;
        uint32_t w[4][VW];
#pragma unroll
        for (int k = 0; k < 4; ++k) lds<VW>(st + L::KBYTES + k * (L::VB * 32) + lane * L::VB, w[k]);
#pragma unroll
        for (int j = 0; j < VW; ++j) {
            const uint32_t a0 = __byte_perm(w[0][j], w[1][j], 0x5140), a1 = __byte_perm(w[0][j], w[1][j], 0x7362);
            const uint32_t b0 = __byte_perm(w[2][j], w[3][j], 0x5140), b1 = __byte_perm(w[2][j], w[3][j], 0x7362);
            uint32_t f[2][4];
            dt_e4m3x4_to_f16x4(a0, f[0][0], f[0][1]);
            dt_e4m3x4_to_f16x4(b0, f[0][2], f[0][3]);
            dt_e4m3x4_to_f16x4(a1, f[1][0], f[1][1]);
            dt_e4m3x4_to_f16x4(b1, f[1][2], f[1][3]);
#pragma unroll
            for (int i = 0; i < NR; ++i) {
                mma(o[2 * j][i], f[0], p[i][0], p[i][1]);
                mma(o[2 * j + 1][i], f[1], p[i][0], p[i][1]);
            }
        }
    }

    DT_DI void clear() {
#pragma unroll
        for (int i = 0; i < NR; ++i) {
#pragma unroll
            for (int j = 0; j < NV / 2; ++j) o[j][i][0] = o[j][i][1] = o[j][i][2] = o[j][i][3] = 0.f;
            m[i][0] = m[i][1] = -__int_as_float(0x7F800000);
            l[i][0] = l[i][1] = 0.f;
        }
    }

    // The first of a warp's sums, from up to 16 new rows: rotated, each scaled by a power of
    // two to a largest magnitude below 4 (one of its own, so that what other rows hold does
    // not matter), elements that are not finite replaced by zeros and reported to the rows
    // that see them.
    DT_DI void fresh(const DtAttend& a, const Walk& u, int lane) {
        const int g = lane >> 2, t = lane & 3, n = u.r.n;
        const uint16_t* kp = (const uint16_t*)a.k.ptr + u.b * a.k.stride_b + u.h * a.k.stride_h;
        const uint16_t* vp = (const uint16_t*)a.v.ptr + u.b * a.v.stride_b + u.h * a.v.stride_h;
        uint32_t bad = 0;  // bit per row
        if (lane < n) {
            for (int e = 0; e < D; e += 64) asm volatile("prefetch.global.L2 [%0];" ::"l"(vp + lane * a.v.stride_n + e));
        }
        float c[NR][4] = {};
        float k[2][L::KC][16];
        float ks[2], fk[2];  // of rows g, g + 8
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int row = g + 8 * i;
            ks[i] = fk[i] = 1.f;
#pragma unroll
            for (int j = 0; j < L::KC; ++j) {
#pragma unroll
                for (int e = 0; e < 16; ++e) k[i][j][e] = 0.f;
            }
            if (8 * i >= n) continue;  // short: code that runs once waits for its instructions
            uint32_t big = 0;
            const int at = a.rope.rot && row < n ? at_position(a, u.b, u.r.len, row) : 0;
#pragma unroll
            for (int j = 0; j < L::KC; ++j) {
                if (row < n) pick16(kp + row * a.k.stride_n, t + 4 * j, a.rope, at, k[i][j]);
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const uint32_t w = __float_as_uint(k[i][j][e]) & 0x7FFFFFFFu;
                    if (w >= 0x7F800000u) k[i][j][e] = 0.f, bad |= 1u << row;
                    else big = max(big, w);
                }
            }
            big = max(big, __shfl_xor_sync(0xffffffffu, big, 1));
            big = max(big, __shfl_xor_sync(0xffffffffu, big, 2));
            const int ek = at_row_exponent(big, true);
            ks[i] = dt_pow2(ek), fk[i] = dt_pow2(-ek);
        }
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            const float *y = k[0][s >> 2] + 4 * (s & 3), *z = k[1][s >> 2] + 4 * (s & 3);
            const uint32_t f[4] = {f16x2(__fmul_rn(y[0], fk[0]), __fmul_rn(y[1], fk[0])), f16x2(__fmul_rn(z[0], fk[1]), __fmul_rn(z[1], fk[1])),
                                   f16x2(__fmul_rn(y[2], fk[0]), __fmul_rn(y[3], fk[0])), f16x2(__fmul_rn(z[2], fk[1]), __fmul_rn(z[3], fk[1]))};
#pragma unroll
            for (int i = 0; i < NR; ++i) {
                uint32_t q[2];
                lds<2>(qs + (((s >> 1) * NR + i) * 32 + lane) * 16 + (s & 1) * 8, q);
                mma(c[i], f, q[0], q[1]);
            }
        }
        uint32_t v[4][L::VB / 2];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int row = 2 * t + (k & 1) + 8 * (k >> 1);
#pragma unroll
            for (int e = 0; e < L::VB / 2; e += 4) {
                uint4 y = make_uint4(0u, 0u, 0u, 0u);
                if (row < n && (k < 2 || n > 8)) y = *(const uint4*)(vp + row * a.v.stride_n + L::VB * g + 2 * e);
                v[k][e] = y.x, v[k][e + 1] = y.y, v[k][e + 2] = y.z, v[k][e + 3] = y.w;
            }
        }
        float fv[4];  // of rows as v's
        int ev[4];
#pragma unroll
        for (int k4 = 0; k4 < 4; ++k4) {
            const int row = 2 * t + (k4 & 1) + 8 * (k4 >> 1);
            ev[k4] = 0, fv[k4] = 1.f;
            if (8 * (k4 >> 1) >= n) continue;
            uint32_t big = 0;
#pragma unroll
            for (int e = 0; e < L::VB / 2; ++e) {
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const uint32_t w = half ? v[k4][e] & 0x7FFF0000u : v[k4][e] << 16 & 0x7FFF0000u;  // magnitude as fp32
                    if (w >= 0x7F800000u) v[k4][e] &= half ? 0x0000FFFFu : 0xFFFF0000u, bad |= 1u << row;
                    else big = max(big, w);
                }
            }
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) big = max(big, __shfl_xor_sync(0xffffffffu, big, d));
            ev[k4] = at_row_exponent(big, false);
            fv[k4] = dt_pow2(-ev[k4]);
        }
        float lv[2], iv[2];  // of rows g, g + 8, which lanes with t = g / 2 hold
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int e0 = __shfl_sync(0xffffffffu, ev[2 * i], g >> 1), e1 = __shfl_sync(0xffffffffu, ev[2 * i + 1], g >> 1);
            const int e = g & 1 ? e1 : e0;
            lv[i] = (float)e, iv[i] = dt_pow2(-e);
        }
        bad = __reduce_or_sync(0xffffffffu, bad);
        // what the lane's rows see
        bool poison[NR][2];
#pragma unroll
        for (int i = 0; i < NR; ++i) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = 2 * t + e + 8 * i;
                const uint32_t sees = r < u.rows ? at_mask_word(a, u.b, r / a.G, 0, n) : 0u;
                poison[i][e] = (sees & bad) != 0u;
#pragma unroll
                for (int k8 = 0; k8 < 2; ++k8)
                    if (!((sees >> (g + 8 * k8)) & 1)) c[i][2 * k8 + e] = -__int_as_float(0x7F800000);
            }
        }
        uint32_t p[NR][2];
        clear();
        weigh<2>(c, ks, lv, iv, p);
#pragma unroll
        for (int i = 0; i < NR; ++i) {
#pragma unroll
            for (int e = 0; e < 2; ++e)
                if (poison[i][e]) l[i][e] = __int_as_float(0x7FC00000);
        }
        auto pair = [&](int x, int y, int j) {  // column j of rows v[x], v[y], scaled
            const float lo = __uint_as_float(j & 1 ? v[x][j / 2] & 0xFFFF0000u : v[x][j / 2] << 16);
            const float hi = __uint_as_float(j & 1 ? v[y][j / 2] & 0xFFFF0000u : v[y][j / 2] << 16);
            return f16x2(__fmul_rn(lo, fv[x]), __fmul_rn(hi, fv[y]));
        };
#pragma unroll
        for (int j = 0; j < NV; j += 2) {
            const uint32_t f[4] = {pair(0, 1, j), pair(0, 1, j + 1), pair(2, 3, j), pair(2, 3, j + 1)};
#pragma unroll
            for (int i = 0; i < NR; ++i) mma(o[j / 2][i], f, p[i][0], p[i][1]);
        }
    }
};

template <int D, int NR>
__global__ void __launch_bounds__(NT, 2) kn11_kernel(const __grid_constant__ DtAttend a, float* part, int* counters) {
    using L = Lay<D>;
    using S = Stream<D, NR>;
    constexpr int NV = S::NV;
    extern __shared__ __align__(128) unsigned char fifo[];
    __shared__ Shared sh;
    __shared__ __align__(16) uint32_t qfrag[S::KS * NR * 64];
    const float NEG_INF = -__int_as_float(0x7F800000);
    const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int cta = blockIdx.x, ctas = gridDim.x;
    dt_pdl_trigger();
    dt_pdl_wait();
    if (w == 0) at_share<ROWS>(a, cta, ctas, MIN_SHARE, &sh.share);
    at_zero_rest(a, cta, ctas, tid, NT);
    __syncthreads();
    const AtShare share = sh.share;
    const int lp = 31 - __clz(a.c.page), low = a.c.page - 1;
    const uint32_t page_bytes = ((uint32_t)a.c.Hkv << lp) * D;
    const uint32_t my_fifo = dt_smem_addr(fifo) + w * L::STAGES * L::BYTES;
    AtWalk<ROWS, ATOM> u;
    u.start(a, share);
    S x;
    x.qs = dt_smem_addr(qfrag);
    for (; u.next(a, share, cta); u.step(a)) {
        const int len = u.r.len, cend = min(u.t1, u.r.ctx), n = max(0, cend - u.t0);
        const int* table = a.c.table + (size_t)u.b * a.c.max_pages;
        const uint8_t* kbase = a.c.k + ((size_t)u.h << lp) * D + t * 16;
        const uint8_t* vbase = a.c.v + ((size_t)u.h << lp) * D + g * L::VB;
        // Pages and scales of this warp's 16 tokens of 32 tiles at a time, one
        // tile to a lane; the next batch's pages are loaded a batch ahead.
        auto page_at = [&](int i) {  // of tile t0 + i (past the end: of the last token)
            const int tok = min((u.t0 + i) * AT_TILE + w * 16, len - 1);
            uint32_t id = (uint32_t)table[tok >> lp];
            if (id >= (uint32_t)a.c.n_pages) {
                atomicOr(&a.status[u.b], DT_DEV_BAD_CACHE);
                id = 0;
            }
            return id;
        };
        uint32_t id = 0, id_next = 0;
        float ks[2] = {1.f, 1.f}, vs[2] = {1.f, 1.f};  // of batches, by parity
        auto scales_of = [&](uint32_t page, float& k, float& v) {
            k = a.c.k_scale[(size_t)page * a.c.Hkv + u.h];
            v = a.c.v_scale[(size_t)page * a.c.Hkv + u.h];
        };
        float lv = 0.f, iv = 1.f;  // log2 and inverse of the value scale, of the batch being computed
        int issued = 0, put = 0;
        auto issue = [&]() {  // the next tile's copies (past the last one: none)
            if (issued < n) {
                if ((issued & 31) == 0 && issued > 0) {
                    id = id_next;
                    if ((issued >> 5) & 1) scales_of(id, ks[1], vs[1]);
                    else scales_of(id, ks[0], vs[0]);
                    id_next = page_at(issued + 32 + lane);
                }
                const uint32_t p = __shfl_sync(0xffffffffu, id, issued & 31);
                const int tok0 = (u.t0 + issued) * AT_TILE + w * 16;
                const uint32_t st = my_fifo + put * L::BYTES + lane * 16, sv = my_fifo + put * L::BYTES + L::KBYTES + lane * L::VB;
                const size_t o = (size_t)p * page_bytes + (uint32_t)(tok0 & low) * D;
                if (tok0 + 16 <= len) {  // 16 tokens lie in one page
                    const uint8_t* k = kbase + o + g * D;
                    const uint8_t* v = vbase + o + 2 * t * D;
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
#pragma unroll
                        for (int j = 0; j < L::KC; ++j) copy_async<16>(st + (i * L::KC + j) * 512, k + 8 * i * D + 64 * j);
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) copy_async<L::VB>(sv + i * (L::VB * 32), v + ((i & 1) + 8 * (i >> 1)) * D);
                } else {  // past len: the last token again
                    const int last = max(len - 1 - tok0, 0);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint8_t* k = kbase + o + min(g + 8 * i, last) * D;
#pragma unroll
                        for (int j = 0; j < L::KC; ++j) copy_async<16>(st + (i * L::KC + j) * 512, k + 64 * j);
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        copy_async<L::VB>(sv + i * (L::VB * 32), vbase + o + min(2 * t + (i & 1) + 8 * (i >> 1), last) * D);
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
            ++issued;
            put = put + 1 == L::STAGES ? 0 : put + 1;
        };
        if (n > 0) {
            id = page_at(lane);
            id_next = page_at(32 + lane);
            scales_of(id, ks[0], vs[0]);
        }
        for (int i = 0; i < L::STAGES - 1; ++i) issue();
        x.queries(a, u, lane);
        __syncwarp();
        // new rows while the first copies are on their way
        if (w == 0 && u.t1 > u.r.ctx) x.fresh(a, u, lane);
        else x.clear();
        int slot = 0;  // of tile i
        for (int i = 0; i < n; ++i) {
            issue();
            asm volatile("cp.async.wait_group %0;" ::"n"(L::STAGES - 1) : "memory");
            const bool odd = (i >> 5) & 1;
            if ((i & 31) == 0) {
                const float v = odd ? vs[1] : vs[0];
                lv = log2f(v);
                iv = 1.0f / v;
            }
            const float k = __shfl_sync(0xffffffffu, odd ? ks[1] : ks[0], i & 31);
            const float v = __shfl_sync(0xffffffffu, lv, i & 31), r = __shfl_sync(0xffffffffu, iv, i & 31);
            const int left = len - (u.t0 + i) * AT_TILE - w * 16;
            if (left > 0) x.tile(my_fifo + slot * L::BYTES, lane, left, k, v, r);
            slot = slot + 1 == L::STAGES ? 0 : slot + 1;
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");

        // join the warps
#pragma unroll
        for (int i = 0; i < NR; ++i) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int d = 4; d < 32; d <<= 1)
                    x.l[i][e] = __fadd_rn(x.l[i][e], __shfl_xor_sync(0xffffffffu, x.l[i][e], d));
                if (g == 0) {
                    sh.m[w][2 * t + e + 8 * i] = x.m[i][e];
                    sh.l[w][2 * t + e + 8 * i] = x.l[i][e];
                }
            }
        }
        __syncthreads();  // all copies have been read
        // O as [warp][row][D]
        float* all = (float*)fifo;
#pragma unroll
        for (int i = 0; i < NR; ++i) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = 2 * t + e + 8 * i;
                if (r < u.rows) {
                    float* dst = all + ((size_t)w * ROWS + r) * D + NV * g;
#pragma unroll
                    for (int j = 0; j < NV / 2; j += 2)
                        *(float4*)(dst + 2 * j) = make_float4(x.o[j][i][e], x.o[j][i][2 + e], x.o[j + 1][i][e], x.o[j + 1][i][2 + e]);
                }
            }
        }
        const bool whole = u.t0 == 0 && u.t1 == u.nt;
        if (tid < 8 * NR) {
            float M = NEG_INF, sum = 0.f;
#pragma unroll
            for (int i = 0; i < NW; ++i) M = fmaxf(M, sh.m[i][tid]);
#pragma unroll
            for (int i = 0; i < NW; ++i) {
                const float mi = sh.m[i][tid], f = mi == NEG_INF ? 0.f : dt_ex2_approx(mi - M);
                sh.w[i][tid] = f;
                sum = __fmaf_rn(sh.l[i][tid], f, sum);
            }
            // NaN of a row that saw something not finite passes even with weight 0
            sh.m[0][tid] = M;
            sh.l[0][tid] = sum;
        }
        __syncthreads();
        constexpr int C4 = D / 4;
        float* my = part + (size_t)(2 * cta + (u.t0 == 0)) * ROWS * (D + 2);
        auto out_row = [&](int r) {
            return (uint16_t*)a.out + (((size_t)u.b * a.M + r / a.G) * a.Hq + u.h * a.G + r % a.G) * D;
        };
        for (int i = tid; i < u.rows * C4; i += NT) {
            const int r = i / C4, c = i % C4 * 4;
            float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int k = 0; k < NW; ++k) {
                const float4 z = *(const float4*)(all + ((size_t)k * ROWS + r) * D + c);
                const float f = sh.w[k][r];
                y.x = __fmaf_rn(z.x, f, y.x), y.y = __fmaf_rn(z.y, f, y.y);
                y.z = __fmaf_rn(z.z, f, y.z), y.w = __fmaf_rn(z.w, f, y.w);
            }
            if (whole) {
                const float sum = sh.l[0][r], inv = sum == 0.f ? 0.f : 1.0f / sum;
                *(uint2*)(out_row(r) + c) = make_uint2(bf16x2(__fmul_rn(y.x, inv), __fmul_rn(y.y, inv)),
                                                       bf16x2(__fmul_rn(y.z, inv), __fmul_rn(y.w, inv)));
            } else {
                *(float4*)(my + 2 * ROWS + (size_t)r * D + c) = y;
            }
        }
        if (!whole) {
            if (tid < u.rows) my[tid] = sh.m[0][tid], my[ROWS + tid] = sh.l[0][tid];
            // the CTA that finishes a unit's last part joins all of them, in their order
            __threadfence();
            __syncthreads();
            if (tid == 0) {
                const int done = atomicAdd(&counters[u.first], 1) + 1;
                sh.last = done == u.segs;
                if (done == u.segs) counters[u.first] = 0;
                __threadfence();
            }
            __syncthreads();
            if (sh.last) {
                auto slot = [&](int i) { return part + (size_t)(2 * (u.first + i) + (i == 0)) * ROWS * (D + 2); };
                for (int i = tid; i < u.rows * C4; i += NT) {
                    const int r = i / C4, c = i % C4 * 4;
                    float M = NEG_INF, sum = 0.f;
                    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
                    for (int k = 0; k < u.segs; ++k) M = fmaxf(M, __ldcg(slot(k) + r));
#pragma unroll 4
                    for (int k = 0; k < u.segs; ++k) {
                        const float mk = __ldcg(slot(k) + r), f = mk == NEG_INF ? 0.f : dt_ex2_approx(mk - M);
                        const float4 z = __ldcg((const float4*)(slot(k) + 2 * ROWS + (size_t)r * D + c));
                        sum = __fmaf_rn(__ldcg(slot(k) + ROWS + r), f, sum);
                        y.x = __fmaf_rn(z.x, f, y.x), y.y = __fmaf_rn(z.y, f, y.y);
                        y.z = __fmaf_rn(z.z, f, y.z), y.w = __fmaf_rn(z.w, f, y.w);
                    }
                    const float inv = sum == 0.f ? 0.f : 1.0f / sum;
                    *(uint2*)(out_row(r) + c) = make_uint2(bf16x2(__fmul_rn(y.x, inv), __fmul_rn(y.y, inv)),
                                                           bf16x2(__fmul_rn(y.z, inv), __fmul_rn(y.w, inv)));
                }
            }
        }
        __syncthreads();  // before the next segment's copies
    }
}

template <int D, int NR>
cudaError_t launch(const DtAttend& a, void* workspace, int ctas, cudaStream_t st) {
    constexpr size_t smem = Lay<D>::SMEM;
    static_assert(2 * (smem + sizeof(Shared) + 4096 + 1024) <= 228 * 1024, "two CTAs per SM");
    cudaError_t e = cudaFuncSetAttribute(kn11_kernel<D, NR>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    DtLaunch lc(dim3(ctas), dim3(NT), smem, st);
    return cudaLaunchKernelEx(&lc.cfg, kn11_kernel<D, NR>, a, (float*)((char*)workspace + AT_MAX_CTAS * sizeof(int)),
                              (int*)workspace);
}

}  // namespace

cudaError_t dt_kn11_launch(const DtAttend& a, void* workspace, int ctas, cudaStream_t st) {
    if (a.M * a.G <= 8) return a.c.D == 64 ? launch<64, 1>(a, workspace, ctas, st) : launch<128, 1>(a, workspace, ctas, st);
    return a.c.D == 64 ? launch<64, 2>(a, workspace, ctas, st) : launch<128, 2>(a, workspace, ctas, st);
}
