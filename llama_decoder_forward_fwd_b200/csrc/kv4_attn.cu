// Attention over a paged KV cache held in 4 bits, for ragged new tokens per sequence.
//
// For query row r of a sequence with n new tokens and len keys (the new ones included):
// token t = r / G, head r % G of its KV head's group, position len - n + t;
//   o = sum_j softmax_j(q . k_j / sqrt(d)) v_j over keys j <= position,
// k_j and v_j the bf16 values that the codes stand for.
//
// What bounds it. A key costs 1.25 d bytes and, at one query row per head, 4 d G flops:
// HBM. But each byte of codes also has to become two bf16 values, some two instructions
// a value, so the issue slots come second, close behind. Hence:
//   - The codes go from shared memory into registers in the fragment layout of
//     mma.sync m16n8k16, with no staging of the expanded values. Both products take
//     the cache as the 16-row operand A and the query rows as the 8 columns of B, so a
//     group of up to 8 query rows costs one expansion:
//       S^T[key][row] = K Q^T: lane (g, t) = (lane / 4, lane % 4) holds d values
//         t d/4 .. of keys g and g + 8, one 16-byte load each; which d a slot of the
//         contraction stands for is free, so Q is laid out to match;
//       O^T[d][row] = V^T P^T: the lane takes d/8 values g d/8 .. of its four keys; the
//         codes of two keys are interleaved by a byte permute before they are expanded.
//         P^T in the B layout is the transpose of S^T's layout (movmatrix).
//     tcgen05 would want the expanded values in shared memory: a store and a read of
//     four times the codes' bytes for products that are 8 of 128 rows wide.
//   - Each warp streams its own 32-key units through its own ring of asynchronous copies,
//     with no barrier between the warps.
//   - The running maximum is only raised (and O scaled) when a score passes it by 2^8.
//   - Sixteen warps a CTA, one CTA per SM: 8 warps (more registers each) take 17% longer over
//     32 x 8k-16k keys, 18 and 20 (fewer) 9% and 1%.
//   - The units of all (sequence, KV head, row chunk) items form one line that is cut
//     evenly over all warps of the grid, wherever items begin or end: ragged lengths
//     and short items cost no balance. An item's parts in one CTA are joined through
//     shared memory, those of several CTAs by the second kernel, in a fixed order.
// Measured (32 query heads, 8 KV heads, d = 128, one new token; a few hundred calls back to back): 32 sequences of
// 8k to 16k keys 110 us, 4.9 TB/s, 75% of the copy bandwidth (119-123 us, 67-69%, in loops of a second, which the power
// cap takes from 1965 to 1800 MHz; with the expansion and the products skipped 89 us: the rest is their
// instructions, 690 per 32 keys of which 290 are the expansion's); 16 of 4k to 8k 38 us; one of 2100 keys 10 us,
// of which a launch and the chain lengths -> table -> codes -> join are 8.
#include "../../include/llama_fwd.h"
#include "kernels.cuh"
#include "kv4_attn.cuh"

#include <float.h>
#include <math.h>

namespace lfw {
namespace {

constexpr int KA_SUB = 16;              // keys per operand tile
constexpr int KA_KEYS = 2 * KA_SUB;     // keys per unit

// One CTA per SM: sixteen warps for one tile of 8 rows (128 registers a thread), eight
// for more. The ring takes what shared memory there is: bytes in flight are what
// keeps HBM busy (44 B/ns per SM and about 1 us of latency under load: 45 KB).
constexpr int ka_warps(int nt) { return nt == 1 ? 16 : 8; }
template <int D, int NT> struct Cfg {
    static constexpr int WARPS = ka_warps(NT);
    static constexpr int R = 8 * NT;
    // a stage: K codes, V codes, K pairs and V pairs of 32 keys
    static constexpr int CODES = KA_KEYS * D / 2, PAIRS = KA_KEYS * D / 8, UNIT = 2 * (CODES + PAIRS);
    static constexpr int STAGES = 14 * 1024 / WARPS * 16 / UNIT < 16 ? 14 * 1024 / WARPS * 16 / UNIT : 16;
    static constexpr int PART = R * (D + 2);  // floats of a partial result
    static constexpr int RING = STAGES * UNIT;
    static constexpr int SMEM = WARPS * RING;
    static_assert(PART * 4 <= RING, "the ring becomes the place of the warp's last partial result");
    static_assert(WARPS * 32 * 8 <= SMEM, "and of the scan over the sequences before");
};

struct Seq {
    int q0, n, len, nt, nch;  // first query row's token, tokens, keys, units, row chunks
};

DEVI uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) { return __byte_perm(a, b, sel); }

// v * inv, and NaN for an infinite v: the mark of a row that sees a value that is not finite.
DEVI float scaled(float v, float inv) { return fmaf(v, 0.f, v * inv); }
// As mma_bf16_16816, but free to move: the expansions between the products fill its latency.
DEVI void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
DEVI uint32_t movm_t(uint32_t a) {
    uint32_t d;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}
// 16 bytes from global to shared memory, past L1, unless `on` is false.
DEVI void copy16(uint32_t dst, const void* src, bool on) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %2, 0;\n\t@p cp.async.cg.shared.global [%0], [%1], 16;\n\t}" ::"r"(dst),
                 "l"(src), "r"((int)on)
                 : "memory");
}
DEVI void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All but the last N committed groups of this thread have landed.
template <int N> DEVI void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

template <int R> DEVI Seq seq_of(const Kv4AttnArgs& a, int b) {
    Seq s;
    const int q0 = a.q_start[b], q1 = a.q_start[b + 1], len = a.lens[b];
    s.q0 = min(max(q0, 0), a.N);
    s.n = min(max(q1, s.q0), a.N) - s.q0;
    s.len = min(max(len, 0), a.max_blocks << a.lp);
    s.nt = max(1, (s.len + KA_KEYS - 1) / KA_KEYS);
    const int rows = s.n * a.G;
    s.nch = rows > a.few && !a.odd[b] ? 0 : (rows + R - 1) / R;
    return s;
}

// An item: one KV head's keys for one chunk of a sequence's query rows.
template <int R> struct Item {
    int b, kvh, chunk;
    Seq s;
    // Takes the fields that lane `from` holds: the same in all lanes, which the shuffle tells the compiler.
    DEVI void take(const Seq& x, int from) {
        s.q0 = __shfl_sync(0xffffffffu, x.q0, from);
        s.n = __shfl_sync(0xffffffffu, x.n, from);
        s.len = __shfl_sync(0xffffffffu, x.len, from);
        s.nt = __shfl_sync(0xffffffffu, x.nt, from);
        s.nch = __shfl_sync(0xffffffffu, x.nch, from);
    }
    DEVI void next(const Kv4AttnArgs& a) {
        if (++chunk < s.nch) return;
        chunk = 0;
        if (++kvh < a.Hk) return;
        kvh = 0;
        do {
            if (++b >= a.B) return;
            take(seq_of<R>(a, b), 0);
        } while (s.nch == 0);
    }
};

// I: the type that the line's units are counted in.
template <int D, int NT, typename I>
__global__ void __launch_bounds__(Cfg<D, NT>::WARPS * 32, 1) kv4_attn_kernel(const Kv4AttnArgs a) {
    using C = Cfg<D, NT>;
    constexpr int W = C::WARPS, R = C::R, ST = C::STAGES, T = W * 32;
    constexpr int KW = D / 32;   // code words of a lane per key of K
    constexpr int VW = D / 64;   // and per key of V
    constexpr int MT = D / 16;   // 16-row tiles of O^T
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ I wsum[W];
    constexpr int WL = W > 16 ? 32 : W > 8 ? 16 : 8;  // a row's lanes when partial results are joined
    static_assert(W <= 32 && R * WL <= T, "one lane a warp, one pass over the rows");
    __shared__ float weight[R][WL];
    __shared__ float2 row_ml[R];
    constexpr int NONE = -0x7fffffff - 1;
    __shared__ int piece_id[2 * W];  // first unit of the item that a warp's partial result belongs to, or NONE
    __shared__ int4 piece_item[2 * W][2];  // units, sequence's first token, rows, first row; KV head
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int g = lane >> 2, t = lane & 3;
    uint8_t* ring = smem + warp * C::RING;
    float* head_part = a.warp_part + ((long long)blockIdx.x * W + warp) * C::PART;
    float* tail_part = reinterpret_cast<float*>(ring);

    pdl_wait();
    pdl_trigger();
    if (lane == 0) {
        piece_id[2 * warp] = piece_id[2 * warp + 1] = NONE;
    }

    // ---- the line of units: its length, this warp's share, where the share begins ----
    // Even shares for the CTAs, then for their warps: a short line still spreads over all SMs.
    // What follows the schedule counts from the CTA's first unit.
    int per_cta = 1, cta_n = 0, u0 = 0, u1 = 0, tile = 0;
    Item<R> cur;
    cur.b = 0;
    I total = 0, cta_lo = 0, seq_at = 0;  // units of the line, the CTA's first, the first of sequence cur.b
    auto shares = [&]() {
        per_cta = div_up(total, gridDim.x);
        const int per = (per_cta + W - 1) / W;
        cta_lo = (I)min((long long)total, (long long)blockIdx.x * per_cta);
        cta_n = (int)min(total - cta_lo, (I)per_cta);
        u0 = min(cta_n, warp * per);
        u1 = min(cta_n, u0 + per);
    };
    // Sums stop at the most units of a call: the entry point bounds them, but only for a q_start that does
    // not decrease; with any other, every share still begins inside some sequence's items.
    const I most = sizeof(I) == 4 ? (I)0x7fffffff : (I)kv4_most_units(gridDim.x);
    auto plus = [&](I x, I y) -> I { return x > most - y ? most : x + y; };
    auto units_of = [&](const Seq& x) -> I { return (I)x.nch * a.Hk * x.nt; };
    auto scan = [&](I u) -> I {  // inclusive over the warp
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const I v = __shfl_up_sync(0xffffffffu, u, o);
            if (lane >= o) u = plus(u, v);
        }
        return u;
    };
    if (a.B <= 32) {
        // one sequence a lane: each warp finds its place by itself
        Seq x = {0, 0, 0, 1, 0};
        if (lane < a.B) x = seq_of<R>(a, lane);
        const I u = units_of(x), incl = scan(u);
        total = __shfl_sync(0xffffffffu, incl, 31);
        shares();
        if (u0 < u1) {
            cur.b = 31 - __clz(__ballot_sync(0xffffffffu, u > 0 && incl - u <= cta_lo + u0));
            seq_at = __shfl_sync(0xffffffffu, incl - u, cur.b);
            cur.take(x, cur.b);
        }
    } else {
        // T sequences at a time; twice over them when there are more
        I* pre = reinterpret_cast<I*>(smem);  // first unit of each, before the rings start
        for (int turn = 0; turn < 2; ++turn) {
            I carry = 0;
            for (int c = 0; c < a.B; c += T) {
                const I u = c + tid < a.B ? units_of(seq_of<R>(a, c + tid)) : 0;
                I incl = scan(u);
                __syncthreads();
                if (lane == 31) wsum[warp] = incl;
                __syncthreads();
                I all = 0;
                for (int w = 0; w < W; ++w) {
                    const I v = wsum[w];
                    if (w < warp) incl = plus(incl, v);
                    all = plus(all, v);
                }
                pre[tid] = plus(carry, incl) - u;
                __syncthreads();
                if (turn == 0 && a.B <= T) {
                    total = all;
                    shares();
                }
                const I mine = cta_lo + u0;
                if ((turn == 1 || a.B <= T) && u0 < u1 && pre[0] <= mine) {
                    int lo = 0, hi = min(T, a.B - c) - 1;  // the last sequence that begins at or before this share
                    while (lo < hi) {
                        const int mid = (lo + hi + 1) >> 1;
                        if (pre[mid] <= mine) lo = mid;
                        else hi = mid - 1;
                    }
                    cur.b = c + lo;
                    seq_at = pre[lo];
                }
                carry = plus(carry, all);
            }
            if (a.B <= T) break;
            if (turn == 0) {
                total = carry;
                shares();
            }
        }
        __syncthreads();  // the rings take pre's place
        cur.b = __shfl_sync(0xffffffffu, cur.b, 0);
        if (u0 < u1) cur.take(seq_of<R>(a, cur.b), 0);
    }
    if (u0 < u1) {
        const I into = cta_lo + u0 - seq_at, skip = into / cur.s.nt;  // units and items of the sequence before this share
        tile = (int)(into - skip * cur.s.nt);
        cur.kvh = (int)(skip / cur.s.nch);
        cur.chunk = (int)(skip - (I)cur.kvh * cur.s.nch);
    }
    const int units = u1 - u0;
    const Kv4Rec rec = kv4_rec(1 << a.lp, D);
    const uint32_t page_bytes = a.Hk * rec.bytes;

    if (units > 0) {
        int at = u0 - tile;  // first unit of the current item, below 0 where a CTA before this one began it

        // ---- the ring: copies run ST units ahead, the table entries of the one after them too ----
        Item<R> ld = cur;
        int ld_tile = tile, issued = 0, st_ld = 0;
        uint32_t oks = 0;  // two bits per stage: which of its 16-key halves hold keys
        int page[2];       // of the halves; equal for pages of more than 16 tokens
        const int32_t* ld_row = a.table + (long long)ld.b * a.max_blocks;
        const uint8_t* ld_head = a.pool + ((uint32_t)ld.kvh * rec.bytes + lane * 16);
        auto look_up = [&]() {
            const int key0 = ld_tile * KA_KEYS, blk = key0 >> a.lp;
            page[0] = key0 < ld.s.len ? ld_row[blk] : -1;
            page[1] = a.lp > 4 ? page[0] : key0 + KA_SUB < ld.s.len ? ld_row[blk + 1] : -1;
        };
        look_up();
        // Copies of one unit, 16 bytes a lane each: half of each codes part per 16 keys, then the pairs
        // (of d = 64, only the first 16 lanes have one).
        constexpr int CPL = KA_SUB * (D / 2) / 512;  // copies of 16 bytes a lane, per half of the codes
        const uint32_t dst0 = smem_u32(ring) + lane * 16;
        const uint32_t hi = lane >= (C::PAIRS / 32 < 32 ? C::PAIRS / 32 : 16);  // half of the lane's pairs
        const bool pair_lane = lane * 16 < C::PAIRS;
        auto issue = [&]() {
            if (issued < units) {
                const int key0 = ld_tile * KA_KEYS, pm = (1 << a.lp) - 1;
                const bool there0 = (unsigned)page[0] < (unsigned)a.n_pages;
                const bool there1 = (unsigned)page[1] < (unsigned)a.n_pages && key0 + KA_SUB < ld.s.len;
                oks = (oks & ~(3u << (2 * st_ld))) | ((there0 ? 1u : 0u) | (there1 ? 2u : 0u)) << (2 * st_ld);
                const uint32_t dst = dst0 + st_ld * C::UNIT;
                const uint8_t* r0 = ld_head + (uint64_t)(uint32_t)page[0] * page_bytes;
                if (a.lp > 4) {  // both halves lie side by side
                    const int o = key0 & pm;
                    const uint8_t* c = r0 + (uint32_t)(o * (D / 2));
                    const uint8_t* p = r0 + (uint32_t)(2 * rec.codes + o * (D / 8));
#pragma unroll
                    for (int j = 0; j < 2 * CPL; ++j) {
                        copy16(dst + j * 512, c + j * 512, there0);
                        copy16(dst + C::CODES + j * 512, c + rec.codes + j * 512, there0);
                    }
                    copy16(dst + 2 * C::CODES, p, there0 && pair_lane);
                    copy16(dst + 2 * C::CODES + C::PAIRS, p + rec.pairs, there0 && pair_lane);
                } else {
                    const uint8_t* r1 = ld_head + (uint64_t)(uint32_t)page[1] * page_bytes;
#pragma unroll
                    for (int j = 0; j < CPL; ++j) {
                        copy16(dst + j * 512, r0 + j * 512, there0);
                        copy16(dst + C::CODES + j * 512, r0 + rec.codes + j * 512, there0);
                        copy16(dst + C::CODES / 2 + j * 512, r1 + j * 512, there1);
                        copy16(dst + C::CODES + C::CODES / 2 + j * 512, r1 + rec.codes + j * 512, there1);
                    }
                    const uint8_t* p = (hi ? r1 - C::PAIRS / 2 : r0) + 2 * rec.codes;
                    const bool on = pair_lane && (hi ? there1 : there0);
                    copy16(dst + 2 * C::CODES, p, on);
                    copy16(dst + 2 * C::CODES + C::PAIRS, p + rec.pairs, on);
                }
                if (++st_ld == ST) st_ld = 0;
                if (++issued < units) {
                    if (++ld_tile == ld.s.nt) {
                        ld_tile = 0;
                        ld.next(a);
                        ld_row = a.table + (long long)ld.b * a.max_blocks;
                        ld_head = a.pool + ((uint32_t)ld.kvh * rec.bytes + lane * 16);
                    }
                    look_up();
                }
            }
            copies_commit();  // empty at the end: the count of groups goes on
        };
#pragma unroll 1
        for (int i = 0; i < ST; ++i) issue();

        // The lane's places in a stage. Operand row r of a 16-key tile is key r ^ (r >> 1 & 1): with
        // the odd pairs swapped, the four t of a load of V fall into both halves of the banks (two
        // wavefronts instead of four), and K's rows still pair up to whole 128-byte lines.
        const int sg = g ^ ((g >> 1) & 1), ve = (2 * t) ^ (t & 1);  // keys of rows g and 2t; 2t + 1's is ve ^ 1
        const uint8_t* k_at = ring + sg * (D / 2) + t * (D / 8);
        const uint8_t* kp_at = ring + 2 * C::CODES + sg * (D / 8) + (t * (D / 4) / KV4_GROUP) * 4;
        const uint8_t* v_at = ring + C::CODES + ve * (D / 2) + g * (D / 16);
        const uint8_t* vp_at = ring + 2 * C::CODES + C::PAIRS + ve * (D / 8) + (g * (D / 8) / KV4_GROUP) * 4;
        const int v_odd = (ve & 1 ? -1 : 1) * (D / 2), vp_odd = (ve & 1 ? -1 : 1) * (D / 8);

        int st = 0, done = 0;
        while (done < units) {
            const Seq& s = cur.s;
            const int here = min(s.nt - tile, units - done);
            const int limmin = max(0, s.len - s.n + div_g(a, cur.chunk * R) + 1);  // keys that every row sees
            uint32_t qf[NT][MT][2];
            float o[NT][MT][4], m[NT][2], l[NT][2];
            int lim[NT][2];  // visible keys of the lane's rows
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                // the B operand's columns: row g of this tile, the lane's d/4 values of it
                const int r = cur.chunk * R + nt * 8 + g;
                const int tok = div_g(a, r), h = cur.kvh * a.G + (r - tok * a.G);
                const uint4* src = reinterpret_cast<const uint4*>(a.q + ((long long)(s.q0 + tok) * a.H + h) * D + t * (D / 4));
#pragma unroll
                for (int w = 0; w < KW; ++w) {
                    const uint4 x = tok < s.n ? __ldg(src + w) : make_uint4(0, 0, 0, 0);
                    qf[nt][2 * w][0] = prmt(x.x, x.z, 0x5410);
                    qf[nt][2 * w][1] = prmt(x.x, x.z, 0x7632);
                    qf[nt][2 * w + 1][0] = prmt(x.y, x.w, 0x5410);
                    qf[nt][2 * w + 1][1] = prmt(x.y, x.w, 0x7632);
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int tk = div_g(a, cur.chunk * R + nt * 8 + 2 * t + e);
                    lim[nt][e] = tk < s.n ? min(s.len, s.len - s.n + tk + 1) : 0x7fffffff;
                    m[nt][e] = -FLT_MAX;  // not -inf: differences from it stay defined
                    l[nt][e] = 0.f;
                }
#pragma unroll
                for (int k = 0; k < MT; ++k)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[nt][k][e] = 0.f;
            }
#pragma unroll 1
            for (int i = 0; i < here; ++i) {
                copies_wait<ST - 1>();
                __syncwarp();  // the other lanes' copies as well
                const uint32_t have = oks >> (2 * st) & 3u;
                bool second = false;
                uint32_t pf[NT][2];
                // One tile of 16 keys at a time, not unrolled: the first pass through this code
                // comes from L2, and there are calls whose warps have one unit each.
#pragma unroll 1
                for (int sb = 0; sb < 2;) {
                    if (!(have >> sb & 1)) {
                        ++sb;
                        continue;
                    }
                    const int kb = (tile + i) * KA_KEYS + sb * KA_SUB;
                    const bool edge = kb + KA_SUB > limmin;  // some row does not see some key
                    const int oc = st * C::UNIT + sb * (C::CODES / 2), op = st * C::UNIT + sb * (C::PAIRS / 2);
                    uint32_t vw[4][VW], vp[4];
                    auto load_v = [&]() {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {  // rows 2t, 2t + 1, 2t + 8, 2t + 9
                        const uint8_t* src = v_at + oc + (j & 1 ? v_odd : 0) + (j >> 1) * 8 * (D / 2);
                        if (VW == 2) {
                            const uint2 x = *reinterpret_cast<const uint2*>(src);
                            vw[j][0] = x.x;
                            vw[j][VW - 1] = x.y;
                        } else {
                            vw[j][0] = *reinterpret_cast<const uint32_t*>(src);
                        }
                        vp[j] = kv4_pair(*reinterpret_cast<const uint32_t*>(vp_at + op + (j & 1 ? vp_odd : 0) + (j >> 1) * 8 * (D / 8)));
                    }
                    };
                    if (!second) {
                        // ---- S^T = K Q^T ----
                        float sc[NT][4];
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) sc[nt][0] = sc[nt][1] = sc[nt][2] = sc[nt][3] = 0.f;
                        uint32_t w0[KW], w1[KW];
                        if (KW == 4) {
                            const uint4 x = *reinterpret_cast<const uint4*>(k_at + oc);
                            const uint4 y = *reinterpret_cast<const uint4*>(k_at + oc + 8 * (D / 2));
                            w0[0] = x.x, w0[1] = x.y, w0[2 % KW] = x.z, w0[3 % KW] = x.w;
                            w1[0] = y.x, w1[1] = y.y, w1[2 % KW] = y.z, w1[3 % KW] = y.w;
                        } else {
                            const uint2 x = *reinterpret_cast<const uint2*>(k_at + oc);
                            const uint2 y = *reinterpret_cast<const uint2*>(k_at + oc + 8 * (D / 2));
                            w0[0] = x.x, w0[1] = x.y;
                            w1[0] = y.x, w1[1] = y.y;
                        }
                        const uint32_t p0 = kv4_pair(*reinterpret_cast<const uint32_t*>(kp_at + op));
                        const uint32_t p1 = kv4_pair(*reinterpret_cast<const uint32_t*>(kp_at + op + 8 * (D / 8)));
                        const uint32_t s0 = prmt(p0, 0, 0x1010), z0 = prmt(p0, 0, 0x3232);
                        const uint32_t s1 = prmt(p1, 0, 0x1010), z1 = prmt(p1, 0, 0x3232);
                        const uint32_t s0h = kv4_16th(s0), s1h = kv4_16th(s1);
#pragma unroll
                        for (int w = 0; w < KW; ++w) {
                            uint32_t x[4], y[4];
                            kv4_expand(w0[w], s0, s0h, z0, x);
                            kv4_expand(w1[w], s1, s1h, z1, y);
#pragma unroll
                            for (int hf = 0; hf < 2; ++hf) {
                                const uint32_t af[4] = {x[2 * hf], y[2 * hf], x[2 * hf + 1], y[2 * hf + 1]};
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt)
                                    mma16816(sc[nt], af, qf[nt][2 * w + hf][0], qf[nt][2 * w + hf][1]);
                            }
                        }
                        load_v();  // in front of the votes and branches below, which no load moves across
                        // ---- softmax in the log2 domain; the lane's keys are kb + sg and 8 on ----
                        if (edge) {
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    if (kb + sg + (e >> 1) * 8 >= lim[nt][e & 1]) sc[nt][e] = -INFINITY;
                        }
                        float x[NT][4], top = -INFINITY;
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                x[nt][e] = fmaf(sc[nt][e], a.scale_log2, -m[nt][e & 1]);
                                top = fmaxf(top, x[nt][e]);
                            }
                        if (__any_sync(0xffffffffu, top > 8.f)) {
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                                for (int e = 0; e < 2; ++e) {
                                    float mx = fmaxf(sc[nt][e], sc[nt][e + 2]);
#pragma unroll
                                    for (int d = 4; d < 32; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
                                    const float mn = fmaxf(m[nt][e], mx * a.scale_log2);
                                    const float al = m[nt][e] == mn ? 1.f : ex2(m[nt][e] - mn);
                                    m[nt][e] = mn;
                                    l[nt][e] *= al;
                                    x[nt][e] = fmaf(sc[nt][e], a.scale_log2, -mn);
                                    x[nt][e + 2] = fmaf(sc[nt][e + 2], a.scale_log2, -mn);
#pragma unroll
                                    for (int k = 0; k < MT; ++k) {
                                        o[nt][k][e] *= al;
                                        o[nt][k][e + 2] *= al;
                                    }
                                }
                        }
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            const float p0f = ex2(x[nt][0]), p1f = ex2(x[nt][1]), p2f = ex2(x[nt][2]), p3f = ex2(x[nt][3]);
                            l[nt][0] += p0f + p2f;
                            l[nt][1] += p1f + p3f;
                            // P enters the product in bf16 (2^-8 of each weight at most, over sums that the
                            // output rounds to bf16 as well); the sum l keeps the full weights
                            pf[nt][0] = movm_t(pack_bf16x2(p0f, p1f));
                            pf[nt][1] = movm_t(pack_bf16x2(p2f, p3f));
                        }
                    }
                    // ---- O^T += V^T P^T ----
                    if (second) load_v();
                    // Where some row does not see some key, 0 * NaN must not reach it: a pair that is
                    // not finite counts as 0 in the product, and a second product, of 2^127 in the
                    // place of such pairs and 2^127 for each key that a row sees, makes the rows
                    // that do see it infinite (NaN at the output). Keys behind the last count as 0
                    // whatever the page holds there.
                    bool odd = false;
                    if (edge) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            if (kb + (ve ^ (j & 1)) + (j >> 1) * 8 >= s.len) vp[j] = 0;
                            const bool bad = kv4_odd(vp[j]);
                            odd = odd || bad;
                            if (bad != second) vp[j] = 0;
                            else if (bad) vp[j] = 0x7F000000u;
                        }
                        odd = __any_sync(0xffffffffu, odd);
                    }
                    const uint32_t sa = prmt(vp[0], vp[1], 0x5410), za = prmt(vp[0], vp[1], 0x7632);
                    const uint32_t sb2 = prmt(vp[2], vp[3], 0x5410), zb = prmt(vp[2], vp[3], 0x7632);
                    const uint32_t sah = kv4_16th(sa), sbh = kv4_16th(sb2);
#pragma unroll
                    for (int w = 0; w < VW; ++w)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const uint32_t sel = h ? 0x7632 : 0x5410;
                            uint32_t x[4], y[4];
                            kv4_expand(prmt(vw[0][w], vw[1][w], sel), sa, sah, za, x);
                            kv4_expand(prmt(vw[2][w], vw[3][w], sel), sb2, sbh, zb, y);
#pragma unroll
                            for (int ip = 0; ip < 2; ++ip) {
                                const uint32_t af[4] = {x[2 * ip], x[2 * ip + 1], y[2 * ip], y[2 * ip + 1]};
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt)
                                    mma16816(o[nt][4 * w + 2 * h + ip], af, pf[nt][0], pf[nt][1]);
                            }
                        }
                    second = odd && !second;
                    if (second) {
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int hf = 0; hf < 2; ++hf) {
                                const int k0 = kb + sg + hf * 8;
                                pf[nt][hf] = movm_t((k0 < lim[nt][0] ? 0x7F00u : 0u) | (k0 < lim[nt][1] ? 0x7F000000u : 0u));
                            }
                    } else {
                        ++sb;
                    }
                }
                __syncwarp();  // every lane has read the stage
                issue();
                if (++st == ST) st = 0;
            }

            // ---- the item's end, or the share's ----
            done += here;
            const bool item_end = tile + here == s.nt, whole = item_end && at >= u0, first = item_end && done < units;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], d);
                    const int rl = nt * 8 + 2 * t + e;
                    if (whole) {
                        const int r = cur.chunk * R + rl, tok = div_g(a, r), h = cur.kvh * a.G + (r - tok * a.G);
                        const float inv = l[nt][e] != 0.f ? KV4_BACK / l[nt][e] : 0.f;
                        if (tok < s.n) {
                            uint32_t x[MT];
#pragma unroll
                            for (int k = 0; k < MT; ++k) x[k] = pack_bf16x2(scaled(o[nt][k][e], inv), scaled(o[nt][k][e + 2], inv));
                            uint4* dst = reinterpret_cast<uint4*>(a.out + ((long long)(s.q0 + tok) * a.H + h) * D + g * (D / 8));
#pragma unroll
                            for (int k = 0; k < MT; k += 4) dst[k / 4] = make_uint4(x[k], x[k + 1], x[k + 2], x[k + 3]);
                        }
                    } else {
                        float* pp = first ? head_part : tail_part;
#pragma unroll
                        for (int k = 0; k < MT; ++k)
                            *reinterpret_cast<float2*>(pp + rl * D + g * (D / 8) + 2 * k) = make_float2(o[nt][k][e], o[nt][k][e + 2]);
                        if (g == 0) *reinterpret_cast<float2*>(pp + R * D + rl * 2) = make_float2(m[nt][e], l[nt][e]);
                    }
                }
            if (!whole && lane == 0) {
                const int slot = 2 * warp + (first ? 0 : 1);
                piece_id[slot] = at;
                piece_item[slot][0] = make_int4(s.nt, s.q0, min(R, s.n * a.G - cur.chunk * R), cur.chunk * R);
                piece_item[slot][1].x = cur.kvh;
            }
            at += s.nt;
            tile = 0;
            if (done < units) cur.next(a);
        }
    }
    __syncthreads();

    // ---- join the parts of each item that this CTA's warps hold ----
    // Entry 2w is warp w's result for an item that began before its share and ended in it
    // while the share went on, entry 2w + 1 its last; an item's entries are the last results of
    // consecutive warps and at the end perhaps the first of the next. Lane w looks at warp w's.
    int4 split = make_int4(0, 0, 0, 0);
    int split_kvh = 0;
    const int my_head = lane < W ? piece_id[2 * lane] : NONE, my_tail = lane < W ? piece_id[2 * lane + 1] : NONE;
    const int before = __shfl_up_sync(0xffffffffu, my_tail, 1);
    unsigned leaders = __ballot_sync(0xffffffffu, my_tail != NONE && (lane == 0 || before != my_tail));
    // an item that ends in the first warp's share has no last result here
    bool alone = __shfl_sync(0xffffffffu, my_head, 0) != NONE;
    while (alone || leaders) {
        const int w_lo = alone ? 0 : __ffs(leaders) - 1, p = 2 * w_lo + (alone ? 0 : 1);
        const int id = __shfl_sync(0xffffffffu, alone ? my_head : my_tail, w_lo);
        if (!alone) leaders &= leaders - 1;
        const unsigned tails = __ballot_sync(0xffffffffu, my_tail == id), closes = __ballot_sync(0xffffffffu, my_head == id);
        const bool last_is_head = closes != 0;
        const int w_hi = 31 - __clz(last_is_head ? closes : tails);
        alone = false;
        const int4 it = piece_item[p][0];  // units, first token, rows, first row
        const int kvh = piece_item[p][1].x;
        const bool whole = id >= 0 && id + it.x <= cta_n;
        const int tail = id >= 0 ? 1 : 0;
        if (!whole && tail) {
            split = make_int4((id + it.x - 1) / per_cta + 1, it.y, it.z, it.w);
            split_kvh = kvh;
        }
        // every entry but the last is a last result (in shared memory)
        const float* last = last_is_head ? a.warp_part + ((long long)blockIdx.x * W + w_hi) * C::PART
                                         : reinterpret_cast<const float*>(smem + w_hi * C::RING);
        // weights of a row's entries, by the lanes of the row
        if (tid < R * WL) {
            const int rl = tid / WL, w = tid % WL;
            const bool in = w >= w_lo && w <= w_hi;
            float2 ml = make_float2(-FLT_MAX, 0.f);
            if (in && rl < it.z)
                ml = *reinterpret_cast<const float2*>((w == w_hi ? last : reinterpret_cast<const float*>(smem + w * C::RING)) + R * D + rl * 2);
            float mx = ml.x;
#pragma unroll
            for (int o = 1; o < WL; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            const float wgt = ex2(ml.x - mx);
            float lsum = wgt * ml.y;
#pragma unroll
            for (int o = 1; o < WL; o <<= 1) lsum += __shfl_xor_sync(0xffffffffu, lsum, o);
            weight[rl][w] = wgt;
            if (w == 0) row_ml[rl] = make_float2(mx, lsum);
        }
        __syncthreads();
        constexpr int VEC = NT == 1 ? 2 : 4;
        for (int x = tid; x < R * D / VEC; x += T) {
            const int rl = x / (D / VEC);
            if (rl >= it.z) break;
            float acc[VEC];
            auto add = [&](const float* f, float wgt, bool first) {
                float v[VEC];
                if (VEC == 4) {
                    const float4 u = reinterpret_cast<const float4*>(f)[x];
                    v[0] = u.x, v[1] = u.y, v[2 % VEC] = u.z, v[3 % VEC] = u.w;
                } else {
                    const float2 u = reinterpret_cast<const float2*>(f)[x];
                    v[0] = u.x, v[1] = u.y;
                }
#pragma unroll
                for (int k = 0; k < VEC; ++k) acc[k] = first ? wgt * v[k] : fmaf(wgt, v[k], acc[k]);
            };
            add(last, weight[rl][w_hi], true);
#pragma unroll 8
            for (int w = w_lo; w < w_hi; ++w) add(reinterpret_cast<const float*>(smem + w * C::RING), weight[rl][w], false);
            if (whole) {
                const int r = it.w + rl, tok = div_g(a, r), h = kvh * a.G + (r - tok * a.G);
                const float lsum = row_ml[rl].y, inv = lsum != 0.f ? KV4_BACK / lsum : 0.f;
                uint32_t* dst = reinterpret_cast<uint32_t*>(a.out + ((long long)(it.y + tok) * a.H + h) * D + x % (D / VEC) * VEC);
#pragma unroll
                for (int k = 0; k < VEC; k += 2) dst[k / 2] = pack_bf16x2(scaled(acc[k], inv), scaled(acc[k + 1], inv));
            } else {
                const long long slot = (long long)blockIdx.x * 2 + tail;
                float* dst = a.part + slot * R * D + x * VEC;
#pragma unroll
                for (int k = 0; k < VEC; k += 2) *reinterpret_cast<float2*>(dst + k) = make_float2(acc[k], acc[k + 1]);
                if (x % (D / VEC) == 0) *reinterpret_cast<float2*>(a.part_ml + slot * R * 2 + rl * 2) = row_ml[rl];
            }
        }
        __syncthreads();  // the weights' place is taken by the next item's
    }
    if (tid == 0) {
        a.desc[2 * blockIdx.x] = split;
        a.desc[2 * blockIdx.x + 1].x = split_kvh;
    }
}

// Join the parts of the items that were split between CTAs: four warps a row, two rows a block.
template <int D, int NT> __global__ void __launch_bounds__(256) kv4_attn_join_kernel(const Kv4AttnArgs a) {
    constexpr int R = 8 * NT, VPL = D / 32;
    __shared__ float part[2][4][D + 1];
    const int lane = threadIdx.x & 31, q = threadIdx.x >> 5 & 3, rr = threadIdx.x >> 7, rl = blockIdx.y * 2 + rr;
    pdl_wait();
    pdl_trigger();
    const int4 it = a.desc[2 * blockIdx.x];  // parts, first token, rows, first row
    const int kvh = a.desc[2 * blockIdx.x + 1].x;
    if (it.x <= 1) return;
    // part i lies in CTA blockIdx.x + i: its tail slot for the first, the head slot for the others
    auto slot = [&](int i) -> long long { return ((long long)blockIdx.x + i) * 2 + (i == 0 ? 1 : 0); };
    const bool row = rl < it.z;
    float mx = -FLT_MAX, lsum = 0.f, acc[VPL] = {};
    if (row) {
#pragma unroll 4
        for (int i = lane; i < it.x; i += 32) mx = fmaxf(mx, a.part_ml[slot(i) * R * 2 + rl * 2]);
        mx = warp_max(mx);
#pragma unroll 8
        for (int i = q; i < it.x; i += 4) {
            const float2 ml = *reinterpret_cast<const float2*>(a.part_ml + slot(i) * R * 2 + rl * 2);
            const float wgt = ex2(ml.x - mx);
            lsum = fmaf(wgt, ml.y, lsum);
            const float* f = a.part + slot(i) * R * D + rl * D + lane * VPL;
#pragma unroll
            for (int k = 0; k < VPL; k += 2) {
                const float2 v = *reinterpret_cast<const float2*>(f + k);
                acc[k] = fmaf(wgt, v.x, acc[k]);
                acc[k + 1] = fmaf(wgt, v.y, acc[k + 1]);
            }
        }
#pragma unroll
        for (int k = 0; k < VPL; ++k) part[rr][q][lane * VPL + k] = acc[k];
        if (lane == 0) part[rr][q][D] = lsum;
    }
    __syncthreads();
    if (!row || q) return;
    lsum = part[rr][0][D] + part[rr][1][D] + part[rr][2][D] + part[rr][3][D];
    const float inv = lsum != 0.f ? KV4_BACK / lsum : 0.f;
    const int r = it.w + rl, tok = div_g(a, r), h = kvh * a.G + (r - tok * a.G);
    __nv_bfloat16* dst = a.out + ((long long)(it.y + tok) * a.H + h) * D + lane * VPL;
#pragma unroll
    for (int k = 0; k < VPL; ++k) {
        const float* c = &part[rr][0][lane * VPL + k];
        acc[k] = scaled(c[0] + c[D + 1] + c[2 * (D + 1)] + c[3 * (D + 1)], inv);
    }
#pragma unroll
    for (int k = 0; k < VPL; k += 2) *reinterpret_cast<uint32_t*>(dst + k) = pack_bf16x2(acc[k], acc[k + 1]);
}

// Above this many rows per KV head a sequence is the prompts' kernel's. Measured (us, 8 KV heads,
// streaming kernel / prompts' kernel): 64 rows over 8192 keys 28 / 39, 128 rows 41 / 39; 16
// sequences over 4096 keys, 64 rows 98 / 91, 128 rows 179 / 88.
constexpr int kFewRows = 64;
bool has_prompts(int max_new, int G) { return (long long)max_new * G > kFewRows; }
// Above this many rows of the longest prompt, all of them are expanded before, once. Measured (us, 8 KV heads,
// every row block expanding for itself / before): 512 rows over 8192 keys 49 / 61, 1024 rows 72 / 71, 2048 rows
// 121 / 99, 4096 rows 220 / 161; 16 sequences over 4096 keys, 512 rows 73 / 77, 1024 rows 137 / 119; 4 over 2048 keys
// with one KV head, 1024 rows 31 / 41.
constexpr int kImageRows = 1024;
bool has_images(int max_new, int G) { return (long long)max_new * G > kImageRows; }
// Room for the expanded tiles: at most 1 GiB. The lengths are on the device, so a workspace is asked for
// by the tables' width; where that passes the most, the lengths are likely to be far below it: 64 MiB are asked for
// then (16k keys of 8 KV heads of 128), and what a caller gives beyond is used. Prompts that find no room are
// expanded row block by row block, in a second turn of the kernels: 7 us more where all had room (192 us for 4 prompts of
// 2048 tokens, 8 KV heads, tables of 131k tokens; 185 us with tables that fit).
constexpr long long kMostImageBytes = 1LL << 30, kSomeImageBytes = 1LL << 26;
int images_within(long long images, int d, long long bytes) {
    const long long room = bytes / (512 * d);
    return (int)(images < room ? images : room);
}
// Row tiles of 8 per item: as many as the longest sequence's rows need, at most 4 (the
// accumulators fill the registers). Beside prompts the others mostly decode.
int row_tiles(int max_new, int G) {
    const long long rows = has_prompts(max_new, G) ? G : (long long)max_new * G;
    return rows <= 8 ? 1 : rows <= 16 ? 2 : 4;
}

// Workspace: CTAs' parts | their maxima and sums | warps' parts | split items; with prompts their row blocks and shares |
// marks of odd sequences | what they are expanded to, n_images tiles | their parts.
struct Ws {
    size_t ml, warp, desc, blocks, starts, splits, p_part, p_ml, odd, expanded, holes, images, bytes;
    long long cap;  // row blocks of the prompts' kernel
};
Ws ws_layout(int grid, int nt, int d, int B, int N, int G, bool prompts, int n_images) {
    const size_t slots = (size_t)grid * 2, R = 8 * nt, warps = (size_t)grid * ka_warps(nt);
    auto up16 = [](size_t x) { return (x + 15) & ~size_t(15); };
    Ws w = {};
    w.ml = slots * R * d * 4;
    w.warp = w.ml + slots * R * 8;
    w.desc = w.warp + warps * R * (d + 2) * 4;
    w.blocks = w.desc + (size_t)grid * 32;
    w.cap = 0;
    if (!prompts) {
        w.bytes = w.blocks;
        return w;
    }
    w.cap = kv4_prefill_blocks(B, N, G, kFewRows);
    w.starts = w.blocks + (size_t)w.cap * sizeof(Kv4Block);
    w.splits = w.starts + (size_t)(grid + 1) * 16;
    w.odd = w.splits + (size_t)grid * sizeof(Kv4Split);
    w.p_part = up16(w.odd + (size_t)(B + 2) * 4);
    if (n_images) {
        w.expanded = w.p_part;
        w.holes = w.expanded + (size_t)kv4_expanded_seqs(B, N, G, kFewRows) * sizeof(Kv4Expanded);
        w.images = up16(w.holes + (size_t)n_images * 8);
        w.p_part = w.images + (size_t)n_images * 512 * d;
    }
    const size_t rows = n_images ? 256 : 128;  // of a block
    w.p_ml = w.p_part + slots * rows * d * 4;
    w.bytes = w.p_ml + slots * rows * 8;
    return w;
}
// The tiles that fit into a workspace of so many bytes, `images` at most; fewer than a sequence needs are none.
int images_in(size_t bytes, int images, int grid, int nt, int d, int B, int N, int G, int Hk) {
    auto need = [&](int n) { return ws_layout(grid, nt, d, B, N, G, true, n).bytes; };
    if (images < Hk || bytes < need(Hk)) return 0;
    const size_t more = (bytes - need(Hk)) / (512 * d + 8) + 2;  // one too many at least, but for the padding
    int n = more < (size_t)(images - Hk) ? Hk + (int)more : images;
    while (need(n) > bytes) --n;
    return n;
}

template <int D, int NT> cudaError_t launch_attn(const Kv4AttnArgs& a, bool wide, int grid, cudaStream_t s) {
    using C = Cfg<D, NT>;
    auto* kernel = wide ? kv4_attn_kernel<D, NT, long long> : kv4_attn_kernel<D, NT, int>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    e = launch_k(kernel, dim3(grid), dim3(C::WARPS * 32), C::SMEM, s, true, a);
    if (e != cudaSuccess) return e;
    return launch_k(kv4_attn_join_kernel<D, NT>, dim3(grid, 4 * NT), dim3(256), 0, s, true, a);
}

int check_shape(int B, int N, int max_new, int H, int Hk, int d, int max_blocks, int page_size) {
    if (B < 1 || N < 0 || max_new < 0 || H < 1 || Hk < 1 || H % Hk != 0 || max_blocks < 1 ||
        kv4_page_log2(page_size) < 0 || (long long)max_blocks * page_size > 0x7fffff00LL)
        return set_error(LLM_ERR_BAD_ARG, "need B >= 1, N >= 0, H % Hk == 0, max_blocks >= 1, page_size 16, 32, 64 or 128");
    if (d != 64 && d != 128) return set_error(LLM_ERR_UNSUPPORTED, "the 4-bit cache needs d == 64 or 128");
    return LLM_OK;
}

}  // namespace
}  // namespace lfw

using namespace lfw;

static size_t kv4_workspace(int B, int N, int max_new, int H, int Hk, int d, int max_blocks, int page_size, bool most) {
    if (check_shape(B, N, max_new, H, Hk, d, max_blocks, page_size) != LLM_OK) return 0;
    const int G = H / Hk;
    const long long all = has_images(max_new, G) ? kv4_images(B, N, G, Hk, (long long)max_blocks * page_size, kFewRows) : 0;
    const int fit = images_within(all, d, kMostImageBytes);
    return ws_layout(current_num_sms(), row_tiles(max_new, G), d, B, N, G, has_prompts(max_new, G),
                     most || fit == all ? fit : images_within(all, d, kSomeImageBytes)).bytes;
}

extern "C" size_t llm_op_attention_kv4_workspace(int B, int N, int max_new, int H, int Hk, int d, int max_blocks,
                                                 int page_size) {
    return kv4_workspace(B, N, max_new, H, Hk, d, max_blocks, page_size, false);
}

size_t lfw::attention_kv4_most_workspace(int B, int N, int max_new, int H, int Hk, int d, int max_blocks, int page_size) {
    return kv4_workspace(B, N, max_new, H, Hk, d, max_blocks, page_size, true);
}

extern "C" int llm_op_attention_kv4(const void* q, const void* pool, int n_pages, int page_size, const int32_t* table,
                                    int max_blocks, const int32_t* lens, const int32_t* q_start, int B, int N,
                                    int max_new, int H, int Hk, int d, void* out, void* workspace,
                                    size_t workspace_bytes, void* stream) {
    return attention_kv4(q, pool, n_pages, page_size, table, max_blocks, lens, q_start, B, N, max_new, H, Hk, d, out,
                         workspace, workspace_bytes, nullptr, reinterpret_cast<cudaStream_t>(stream));
}

int lfw::kv4_check_size(int B, int N, int H, int Hk, int max_blocks, int page_size) {
    // a row is divided by G as 32-bit fixed point; units: see kv4_most_units; the prompts' tiles are counted in 32 bits
    const long long G = H / Hk, chunks = (long long)N * G / 8 + B, keys = (long long)max_blocks * page_size;
    if ((long long)N * G * G >= (1LL << 31) || chunks * Hk > kv4_most_units(current_num_sms()) / ((keys + KA_KEYS - 1) / KA_KEYS) ||
        kv4_prefill_blocks(B, N, (int)G, kFewRows) * Hk >= (1LL << 31) / (keys / 128 + 4))
        return set_error(LLM_ERR_UNSUPPORTED, "more query rows over tables this wide than one call takes");
    return LLM_OK;
}

int lfw::attention_kv4(const void* q, const void* pool, int n_pages, int page_size, const int32_t* table, int max_blocks,
                       const int32_t* lens, const int32_t* q_start, int B, int N, int max_new, int H, int Hk, int d,
                       void* out, void* workspace, size_t workspace_bytes, uint32_t* err, cudaStream_t s) {
    const int rc = check_shape(B, N, max_new, H, Hk, d, max_blocks, page_size);
    if (rc) return rc;
    if (N == 0) return LLM_OK;
    if (!q || !pool || !table || !lens || !q_start || !out || !workspace)
        return set_error(LLM_ERR_NULL_PTR, "NULL operand or workspace");
    if (n_pages < 0) return set_error(LLM_ERR_BAD_ARG, "n_pages must not be negative");
    if (const int too_large = kv4_check_size(B, N, H, Hk, max_blocks, page_size)) return too_large;
    if ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(pool) | reinterpret_cast<uintptr_t>(out) |
         reinterpret_cast<uintptr_t>(workspace)) & 15)
        return set_error(LLM_ERR_BAD_ARG, "operands must be 16-byte aligned");
    const int nt = row_tiles(max_new, H / Hk), grid = current_num_sms();
    const bool prompts = has_prompts(max_new, H / Hk);
    const long long all_images =
        has_images(max_new, H / Hk) ? kv4_images(B, N, H / Hk, Hk, (long long)max_blocks * page_size, kFewRows) : 0;
    const int n_images =
        images_in(workspace_bytes, images_within(all_images, d, kMostImageBytes), grid, nt, d, B, N, H / Hk, Hk);
    const Ws w = ws_layout(grid, nt, d, B, N, H / Hk, prompts, n_images);
    if (workspace_bytes < w.bytes) return set_error(LLM_ERR_BAD_ARG, "workspace too small");
    const size_t row = (size_t)H * d * 2;
    const Bytes in[] = {{q, N * row}, {pool, n_pages * llm_kv4_page_bytes(Hk, d, page_size)}, {table, (size_t)B * max_blocks * 4},
                        {lens, (size_t)B * 4}, {q_start, (size_t)B * 4 + 4}}, res[] = {{out, N * row}, {workspace, w.bytes}};
    if (any_overlap(in, res)) return set_error(LLM_ERR_BAD_ARG, "out or the workspace overlaps an input or the other");
    Kv4AttnArgs a;
    a.q = reinterpret_cast<const __nv_bfloat16*>(q);
    a.pool = reinterpret_cast<const uint8_t*>(pool);
    a.table = table;
    a.lens = lens;
    a.q_start = q_start;
    a.out = reinterpret_cast<__nv_bfloat16*>(out);
    a.B = B;
    a.N = N;
    a.n_pages = n_pages;
    a.lp = kv4_page_log2(page_size);
    a.max_blocks = max_blocks;
    a.H = H;
    a.Hk = Hk;
    a.G = H / Hk;
    const bool wide = ((long long)N * a.G / 8 + B) * Hk * (((long long)max_blocks * page_size + KA_KEYS - 1) / KA_KEYS) >= 1LL << 31;
    a.g_mul = a.G > 1 ? (uint32_t)(((1ULL << 32) + a.G - 1) / a.G) : 0;
    a.scale_log2 = (float)(1.4426950408889634 / sqrt((double)d) * KV4_BACK);  // the keys come * 2^-72
    a.part = reinterpret_cast<float*>(workspace);
    a.part_ml = reinterpret_cast<float*>(reinterpret_cast<char*>(workspace) + w.ml);
    a.warp_part = reinterpret_cast<float*>(reinterpret_cast<char*>(workspace) + w.warp);
    a.desc = reinterpret_cast<int4*>(reinterpret_cast<char*>(workspace) + w.desc);
    char* base = reinterpret_cast<char*>(workspace);
    a.few = prompts ? kFewRows : 0x7fffffff;
    a.blocks = reinterpret_cast<Kv4Block*>(base + w.blocks);
    a.blocks_cap = (int)w.cap;
    a.odd = prompts ? reinterpret_cast<int*>(base + w.odd) : nullptr;
    a.counts = prompts ? a.odd + B : nullptr;
    a.splits = reinterpret_cast<Kv4Split*>(base + w.splits);
    a.starts = reinterpret_cast<int4*>(base + w.starts);
    a.expanded = reinterpret_cast<Kv4Expanded*>(base + w.expanded);
    a.holes = reinterpret_cast<uint64_t*>(base + w.holes);
    a.images = reinterpret_cast<uint8_t*>(base + w.images);
    a.images_cap = n_images;
    a.expanded_cap = n_images ? kv4_expanded_seqs(B, N, H / Hk, kFewRows) : 0;
    a.turn = n_images && n_images < all_images ? 1 : 0;
    a.p_part = reinterpret_cast<float*>(base + w.p_part);
    a.p_ml = reinterpret_cast<float*>(base + w.p_ml);
    a.err = err || !prompts ? err : op_err_word();  // only the prompts' kernel waits on barriers
    cudaError_t e;
    if (prompts) {
        e = launch_kv4_prefill(a, d, s);
        if (e != cudaSuccess) return set_error(LLM_ERR_CUDA, cudaGetErrorString(e));
    }
    if (d == 128) e = nt == 1 ? launch_attn<128, 1>(a, wide, grid, s) : nt == 2 ? launch_attn<128, 2>(a, wide, grid, s) : launch_attn<128, 4>(a, wide, grid, s);
    else e = nt == 1 ? launch_attn<64, 1>(a, wide, grid, s) : nt == 2 ? launch_attn<64, 2>(a, wide, grid, s) : launch_attn<64, 4>(a, wide, grid, s);
    return e == cudaSuccess ? LLM_OK : set_error(LLM_ERR_CUDA, cudaGetErrorString(e));
}
