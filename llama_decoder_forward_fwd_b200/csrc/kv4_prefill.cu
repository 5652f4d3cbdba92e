// Attention over the 4-bit paged cache for prompts: sequences with many new tokens, whose
// products belong on the 5th-generation tensor cores.
//
// A work item is a block of query rows (token, head of the KV head's group) of one sequence and KV head, as in the
// bf16 prefill kernel: S = Q K^T and O += P V by tcgen05 with S, P and O in tensor memory, O rescaled only
// when a row's maximum grows by more than 2^8. What differs is where K and V come from, in two variants:
//
// - With few row blocks a sequence, four warps read the codes from the pages (the next tile's into
//   registers while one is worked on), expand them and store the bf16 tiles in the 128-byte
//   swizzle that the tensor cores read: some 1800 instructions a 128-key tile next to the
//   softmax's 16,000 scores, repeated by every block of 128 rows. Two softmax threads a row.
// - With many, a kernel before expands each sequence once, into tiles laid out like that, and one thread
//   copies a tile in one bulk copy. That moves 4 d bytes per key and KV head out and back through L2
//   and takes a workspace of the size of the prompts' bf16 cache. A block has 256 rows, which share a tile, and
//   one softmax thread a row. Prompts for whose tiles the workspace has no room take the first variant, in a
//   second turn.
//
// Two orders inside 8 values: a code word expands to the pairs (0, 4), (1, 5), (2, 6),
// (3, 7), and is stored so. Q is staged in the same order, which the contraction over d
// does not notice; O's columns come in it and are written out straight. Expanded before, they are put in
// plain order, so that Q's rows can be copied.
//
// Measured: 134 GFLOP of prompts over a cached context 177 us in short runs, 760 TFLOP/s, 10 us of it the
// expansion before (185-190 us, 707-725 TFLOP/s, in loops of a second under the power cap); 252 us with the expanding
// warps in the kernel, which share the issue slots with the softmax (a 128-key tile takes 1.8 us so).
//
// A small kernel before lists the row blocks. Their tiles, for each KV head, form one line that
// is cut evenly over the SMs (one CTA each): neither ragged prompts nor few rows over a long
// context leave SMs idle. A kernel after joins what was cut: 256 rows over 8192 keys of 8 KV heads
// take 40 us so, and 126 us with a row block to a CTA.
#include "kv4_attn.cuh"

#include <math.h>

namespace lfw {
namespace {

constexpr int KP_THREADS = 416;
constexpr int KP_MMA = 8, KP_EXPAND = 9;  // warps 0..7 softmax, 8 tcgen05, 9..12 expansion
// With expanded prompts: warps 0..3 and 4..7 the softmax of a row block each, 8 tcgen05, 9 copies
// of K and V, 10 and 11 of a block's Q each, behind the first item (the softmax warps stage that).
constexpr int KQ_THREADS = 384, KQ_LOAD = 9, KQ_Q = 10, KQ_ROWS = 256;
constexpr int KP_ROWS = 128, KP_KT = 128;
constexpr int KP_HALF = 128 * 128;  // [128 rows][64 bf16]
constexpr uint32_t KP_TMEM_COLS = 512, KP_TMEM_O = 256, KP_TMEM_P = 384;
constexpr float KP_RESCALE_LOG2 = 8.f;
constexpr int KP_LIST = 1024;  // threads of the kernel that lists the blocks
// An item's fixed cost in tiles (prompts' case: 304 us with 0, 266 with 1, 263 with 2, 266 with 3).
constexpr int KP_ITEM = 2;
constexpr int KQ_ITEM = 3;  // the same of 256 rows: 200 us with 1, 187 with 2, 179 with 3, 181 with 4
constexpr int KP_SHARE = 4;  // units of a CTA, at least: with fewer the parts' ends cost more than they save

template <int D> constexpr int kp_tile() { return D / 64 * KP_HALF; }
template <int D> constexpr int kq_smem() { return 6 * kp_tile<D>() + 256 + 1024; }
template <int D> constexpr int kp_smem() { return 1024 + 5 * kp_tile<D>() + 256 + 2 * KP_ROWS * 4; }

// A maximum that a NaN does not drop out of.
DEVI float max3(float a, float b, float c) {
    float d;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
// A row's running maximum as it is kept. A NaN or infinite score makes the row NaN by its definition, but a
// quarter of the exponentials (ex2_fma) lose a NaN: so the maximum carries it, to the row's sum and to all its weights.
// An infinite maximum becomes NaN here, a finite one stays (x * 0 + x).
DEVI float kept_max(float x) { return fmaf(x, 0.f, x); }
// 2^x of a pair on the FMA pipe, for a share of the exponentials: x = n + f, n to the
// exponent field, 2^f by a cubic with relative error below 1.5e-4, far below the bf16
// rounding that P gets next. -inf gives the clamp, just under 2^-126, and not 0 (see less_clamp).
DEVI float2 ex2_fma(float2 x) {
    x.x = fmaxf(x.x, -126.f);
    x.y = fmaxf(x.y, -126.f);
    const float2 t = __fadd2_rn(x, make_float2(12582912.f, 12582912.f));
    const float2 n = __fadd2_rn(t, make_float2(-12582912.f, -12582912.f));
    const float2 f = __ffma2_rn(n, make_float2(-1.f, -1.f), x);
    float2 p = __ffma2_rn(make_float2(0.05517166f, 0.05517166f), f, make_float2(0.24261114f, 0.24261114f));
    p = __ffma2_rn(p, f, make_float2(0.69326097f, 0.69326097f));
    p = __ffma2_rn(p, f, make_float2(0.99992806f, 0.99992806f));
    return make_float2(__int_as_float(__float_as_int(p.x) + (__float_as_int(t.x) << 23)),
                       __int_as_float(__float_as_int(p.y) + (__float_as_int(t.y) << 23)));
}
// A pair of weights from ex2_fma, in bf16, less 2^-126, which the clamp has become: a masked key's weight is 0 then,
// however large its value is, and other weights change by nothing that a sum could show.
DEVI uint32_t less_clamp(uint32_t w) {
    const uint32_t least = 0x80808080u;
    const __nv_bfloat162 v = __hadd2(*reinterpret_cast<const __nv_bfloat162*>(&w), *reinterpret_cast<const __nv_bfloat162*>(&least));
    return *reinterpret_cast<const uint32_t*>(&v);
}
// mbar_wait whose polls may sleep in the barrier unit: the waiting warps' polls would otherwise take
// issue slots from the softmax and the expansion.
DEVI bool wait_for(uint64_t* bar, uint32_t parity, uint32_t* err, uint32_t code) {
    uint64_t t0 = 0;
    while (true) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(smem_u32(bar)), "r"(parity), "r"(1000000u)
            : "memory");
        if (ok) return true;
        const uint64_t t = globaltimer();
        if (t0 == 0) t0 = t;
        if (t - t0 > kWaitLimitNs) {
            if (err) atomicCAS(err, 0u, code);
            return false;
        }
    }
}
// A matrix descriptor `bytes` further on: the address is its lowest field, in 16 bytes.
DEVI uint64_t desc_at(uint64_t desc, int bytes) { return desc + (uint32_t)(bytes >> 4); }
// True in one lane, the same one each time. The compiler knows by this instruction, and not by a lane's number,
// that a single thread runs what follows: without, it issues each tcgen05 instruction in a loop over the
// lanes that might be there, 90 clocks instead of 30.
DEVI bool elected() {
    uint32_t yes;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(yes));
    return yes != 0;
}
// 16 bytes from global to shared memory, or zeros.
DEVI void copy_16(void* dst, const void* src, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(there ? 16 : 0) : "memory");
}
// A whole tile from global to shared memory.
DEVI void copy_tile(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)), "l"(src),
                 "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}
// 16 columns of the warp's lanes.
DEVI void tc_ld_x16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
                   "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                 : "r"(taddr));
}
DEVI void tc_st_x16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
                 "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(taddr)
                 : "memory");
}
// D (+)= A B, A in tensor memory, B in shared memory.
DEVI void mma_tmem_a(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// An item is what the CTA's share has of one row block and KV head. Every role walks the same items.
struct Walk {
    int blk, kvh, tile;
};
struct Work {
    int q0, n, len, row0, b, kvh;
    int tile0, nkt, all;  // first tile, tiles here (0: the share has ended), tiles of the row block
    int image;            // with expanded prompts: of the KV head's first tile
};
DEVI Work describe(const Kv4AttnArgs& a, const int4& end, const Walk& w) {
    const bool last = w.blk == end.x && w.kvh == end.y;
    if (w.blk > end.x || (w.blk == end.x && w.kvh > end.y) || (last && w.tile >= end.z)) return Work{};
    const int4* src = reinterpret_cast<const int4*>(a.blocks + w.blk);
    const int4 x = src[0], y = src[1];
    return Work{x.x, x.y, x.z, x.w, y.x, w.kvh, w.tile, (last ? end.z : y.y) - w.tile, y.y,
                y.w + w.kvh * max(1, (x.z + KP_KT - 1) / KP_KT)};
}
DEVI void advance(const Kv4AttnArgs& a, Walk& w) {
    w.tile = 0;
    if (++w.kvh == a.Hk) {
        w.kvh = 0;
        ++w.blk;
    }
}
// How the CTAs whose shares begin inside an item, which this one begins, join it.
DEVI Kv4Split split_of(const Kv4AttnArgs& a, const Walk& at, const Work& it) {
    int parts = 1;
    for (int c = blockIdx.x + 1; c < a.counts[0]; ++c) {
        const int4 x = a.starts[c];
        if (x.x != at.blk || x.y != at.kvh) break;
        ++parts;
    }
    return Kv4Split{parts, it.q0, it.n, it.row0, it.kvh, {}};
}
// Stage 128 query rows of an item, from its row `from` on: 16-byte chunks XOR-swizzled by row, 8 values as
// (0,4),(1,5),(2,6),(3,7).
template <int D> DEVI void stage_q(const Kv4AttnArgs& a, const Work& it, int from, uint8_t* Qs, int tid, int nthr) {
    constexpr int CH = D / 8, QB = 8;
    for (int base = tid; base < KP_ROWS * CH; base += nthr * QB) {
        uint4 v[QB];
#pragma unroll
        for (int i = 0; i < QB; ++i) {
            const int idx = base + i * nthr, r = idx / CH, c = idx % CH;
            const int rg = it.row0 + from + r, t = div_g(a, rg), h = it.kvh * a.G + (rg - t * a.G);
            v[i] = make_uint4(0, 0, 0, 0);
            if (idx < KP_ROWS * CH && t < it.n)
                v[i] = __ldcg(reinterpret_cast<const uint4*>(a.q + ((long long)(it.q0 + t) * a.H + h) * D + c * 8));
        }
#pragma unroll
        for (int i = 0; i < QB; ++i) {
            const int idx = base + i * nthr, r = idx / CH, c = idx % CH;
            if (idx < KP_ROWS * CH)
                *reinterpret_cast<uint4*>(Qs + (c >> 3) * KP_HALF + r * 128 + (((c & 7) ^ (r & 7)) << 4)) =
                    make_uint4(__byte_perm(v[i].x, v[i].z, 0x5410), __byte_perm(v[i].x, v[i].z, 0x7632),
                               __byte_perm(v[i].y, v[i].w, 0x5410), __byte_perm(v[i].y, v[i].w, 0x7632));
        }
    }
}

// The row blocks of all sequences with more than a.few rows that this turn takes, the CTAs' shares of their
// tiles, and the marks of odd sequences cleared. One CTA.
__global__ void __launch_bounds__(KP_LIST) kv4_blocks_kernel(const Kv4AttnArgs a, int sms, int block_rows) {
    __shared__ int wsum[KP_LIST / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_wait();
    pdl_trigger();
    // inclusive scan over the CTA; `all`: the sum
    auto scan = [&](int v, int& all) -> int {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += u;
        }
        __syncthreads();
        if (lane == 31) wsum[warp] = v;
        __syncthreads();
        int x = wsum[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += u;
        }
        all = __shfl_sync(0xffffffffu, x, 31);
        const int before = __shfl_sync(0xffffffffu, x, max(warp - 1, 0));
        return warp ? v + before : v;
    };
    // the blocks, a sequence's shared out over the lanes of a warp
    int blocks = 0, images = 0, listed = 0;
    for (int b0 = 0; b0 < a.B; b0 += KP_LIST) {
        const int b = b0 + tid;
        int q0 = 0, n = 0, len = 0;
        if (b < a.B) {
            const int x0 = a.q_start[b], x1 = a.q_start[b + 1];
            len = min(max(a.lens[b], 0), a.max_blocks << a.lp);
            q0 = min(max(x0, 0), a.N);
            n = min(max(x1, q0), a.N) - q0;
        }
        const int rows = n * a.G;
        int nb = rows > a.few ? (rows + block_rows - 1) / block_rows : 0, all, all_images, all_listed, image = -1;
        if (b < a.B && a.turn == 2 && a.odd[b] != KV4_REST) nb = 0;
        else if (b < a.B) a.odd[b] = 0;
        if (a.images_cap > 0) {
            // A sequence's tiles, or one more than there is room for: those before the first without room are listed.
            const int tiles = max(1, (len + KP_KT - 1) / KP_KT);
            const int ask = nb ? (int)min((long long)tiles * a.Hk, a.images_cap + 1LL) : 0;
            image = images + scan(ask, all_images) - ask;
            bool fits = nb > 0 && image + ask <= a.images_cap;
            const int li = listed + scan(fits, all_listed) - (fits ? 1 : 0);
            fits = fits && li < a.expanded_cap;  // always, unless q_start decreases somewhere
            if (fits) {
                a.expanded[li] = Kv4Expanded{b, len, image, tiles};
            } else if (nb > 0) {
                a.odd[b] = a.turn == 1 ? KV4_REST : 1;
                nb = 0;
            }
            images = min(images + all_images, a.images_cap);
            listed = min(listed + all_listed, a.expanded_cap);
        }
        const int at = blocks + scan(nb, all) - nb;
        unsigned many = __ballot_sync(0xffffffffu, nb > 0);
        while (many) {
            const int src = __ffs(many) - 1;
            many &= many - 1;
            const int sq0 = __shfl_sync(0xffffffffu, q0, src), sn = __shfl_sync(0xffffffffu, n, src),
                      sl = __shfl_sync(0xffffffffu, len, src), sat = __shfl_sync(0xffffffffu, at, src), srows = sn * a.G,
                      simg = __shfl_sync(0xffffffffu, image, src);
            for (int i = lane; i * block_rows < srows; i += 32) {
                const int t_last = div_g(a, min(srows, (i + 1) * block_rows) - 1);
                const int keys = min(sl, sl - sn + t_last + 1);
                if (sat + i < a.blocks_cap)  // always, unless q_start decreases somewhere
                    a.blocks[sat + i] = Kv4Block{sq0, sn, sl, i * block_rows, b0 + warp * 32 + src, max(1, (keys + KP_KT - 1) / KP_KT), 0, simg};
            }
        }
        blocks += all;
    }
    blocks = min(blocks, a.blocks_cap);
    __syncthreads();
    // where each begins on the line of tiles
    const int item = block_rows == KQ_ROWS ? KQ_ITEM : KP_ITEM;
    int tiles = 0;
    for (int i0 = 0; i0 < blocks; i0 += KP_LIST) {
        const int i = i0 + tid, nkt = i < blocks ? a.blocks[i].nkt + item : 0;
        int all;
        const int incl = tiles + scan(nkt, all);
        if (i < blocks) a.blocks[i].start = incl - nkt;
        tiles += all;
    }
    // The CTAs' shares: the item in which one begins says where. A share that would begin in an
    // item's fixed cost begins with its first tile.
    const int units = tiles * a.Hk, per = max(KP_SHARE, div_up(units, sms)), ctas = div_up(units, per);
    if (tid == 0) {
        a.counts[0] = ctas;
        a.counts[1] = listed;
        a.starts[ctas] = make_int4(blocks, 0, 0, 0);
    }
    for (int i = tid; i < blocks; i += KP_LIST) {
        const int len = a.blocks[i].nkt + item, lo = a.blocks[i].start * a.Hk, hi = lo + len * a.Hk;
        for (int c = div_up(lo, per); c < ctas && c * per < hi; ++c) {
            const int off = c * per - lo, kvh = off / len;
            a.starts[c] = make_int4(i, kvh, max(0, off - kvh * len - item), 0);
        }
    }
}

// Expand the listed sequences: a CTA writes one K or V tile as the tensor cores read it (rows of 64
// values, 16-byte chunks XOR-swizzled by row), so that the main kernel takes it in one copy. The tile is
// put together in shared memory, where its threads' 16 bytes fill whole lines: written straight out they
// are half sectors of L2 (15 us against 10 for 7,800 keys of 8 KV heads).
template <int D> __global__ void __launch_bounds__(256) kv4_expand_kernel(const Kv4AttnArgs a) {
    constexpr int WPL = D / 32;
    const int lane = threadIdx.x & 31, key_l = (threadIdx.x >> 5) * 8 + (lane & 7), t = lane >> 3;
    const Kv4Rec rec = kv4_rec(1 << a.lp, D);
    __shared__ alignas(128) uint8_t tile_mem[kp_tile<D>()];
    pdl_wait();
    pdl_trigger();
    const int listed = a.counts[1];
    if (listed == 0) return;
    const Kv4Expanded last = a.expanded[listed - 1];
    const int units = 2 * (last.image + last.tiles * a.Hk);
    for (int u = blockIdx.x; u < units; u += gridDim.x) {
        const int img = u >> 1, is_v = u & 1;
        int lo = 0, hi = listed - 1;  // the last sequence whose images begin at or before this one
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (a.expanded[mid].image <= img) lo = mid;
            else hi = mid - 1;
        }
        const Kv4Expanded e = a.expanded[lo];
        const int kvh = (img - e.image) / e.tiles, tile = img - e.image - kvh * e.tiles;
        if (threadIdx.x == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");  // the last tile has been read
        __syncthreads();
        bool odd = false;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = i * 64 + key_l, key = tile * KP_KT + r, off = r & ((1 << a.lp) - 1);
            const int page = key < e.len ? a.table[(long long)e.b * a.max_blocks + (key >> a.lp)] : 0;
            const bool there = (unsigned)page < (unsigned)a.n_pages;
            if (!is_v && (r & 15) == 0 && t == 0) reinterpret_cast<uint8_t*>(a.holes + img)[r >> 4] = !there;
            uint32_t c[WPL] = {}, q = 0;
            if (there && key < e.len) {
                const uint8_t* src = a.pool + (uint64_t)page * ((uint64_t)a.Hk * rec.bytes) + (uint32_t)(kvh * rec.bytes);
                const uint8_t* cp = src + (is_v ? rec.codes : 0) + off * (D / 2) + t * (D / 8);
                if (WPL == 4) {
                    const uint4 x = __ldcs(reinterpret_cast<const uint4*>(cp));
                    c[0] = x.x, c[1] = x.y, c[2 % WPL] = x.z, c[3 % WPL] = x.w;
                } else {
                    const uint2 x = __ldcs(reinterpret_cast<const uint2*>(cp));
                    c[0] = x.x, c[1] = x.y;
                }
                q = *reinterpret_cast<const uint32_t*>(src + 2 * rec.codes + (is_v ? rec.pairs : 0) + off * (D / 8) + t * (D / 4) / KV4_GROUP * 4);
            }
            q = kv4_pair(q);
            if (kv4_odd(q)) {
                odd = true;
                q = 0;
            }
            const uint32_t s2 = __byte_perm(q, 0, 0x1010), z2 = __byte_perm(q, 0, 0x3232), s2h = kv4_16th(s2);
#pragma unroll
            for (int x = 0; x < WPL; ++x) {
                uint32_t v[4];
                kv4_expand(c[x], s2, s2h, z2, v);
                const int ch = t * WPL + x;
                *reinterpret_cast<uint4*>(tile_mem + (ch >> 3) * KP_HALF + r * 128 + (((ch & 7) ^ (r & 7)) << 4)) =
                    make_uint4(__byte_perm(v[0], v[1], 0x5410), __byte_perm(v[2], v[3], 0x5410), __byte_perm(v[0], v[1], 0x7632),
                               __byte_perm(v[2], v[3], 0x7632));
            }
        }
        if (odd) a.odd[e.b] = 1;
        fence_proxy_async();  // the copy reads shared memory through the async proxy
        __syncthreads();
        if (threadIdx.x == 0)
            asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;\n\tcp.async.bulk.commit_group;" ::"l"(
                             a.images + ((long long)img * 2 + is_v) * kp_tile<D>()),
                         "r"(smem_u32(tile_mem)), "r"(kp_tile<D>())
                         : "memory");
    }
    if (threadIdx.x == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

// Join the parts of split row blocks: a thread per row and 16 values. The parts lie as
// [4 values][row], so that the rows' threads write and read them in whole lines.
template <int D, int ROWS> __global__ void __launch_bounds__(ROWS) kv4_prefill_join_kernel(const Kv4AttnArgs a) {
    const int r = threadIdx.x, c0 = blockIdx.y * 16;
    pdl_wait();
    pdl_trigger();
    if ((int)blockIdx.x >= a.counts[0]) return;  // a CTA without a share
    const Kv4Split sp = a.splits[blockIdx.x];
    const int rg = sp.row0 + r, t = div_g(a, rg), h = sp.kvh * a.G + (rg - t * a.G);
    if (sp.parts <= 1 || t >= sp.n) return;
    // part i lies in CTA blockIdx.x + i: what goes on after it for the first, what began before for the others
    auto slot = [&](int i) -> long long { return ((long long)blockIdx.x + i) * 2 + (i == 0 ? 1 : 0); };
    float mx = -INFINITY;
#pragma unroll 4
    for (int i = 0; i < sp.parts; ++i) mx = fmaxf(mx, a.p_ml[(slot(i) * ROWS + r) * 2]);
    const float mu = mx == -INFINITY ? 0.f : mx;
    float l = 0.f, acc[16] = {};
#pragma unroll 2
    for (int i = 0; i < sp.parts; ++i) {
        const float2 ml = *reinterpret_cast<const float2*>(a.p_ml + (slot(i) * ROWS + r) * 2);
        const float w = ex2(ml.x - mu);
        l = fmaf(w, ml.y, l);
        const float4* f = reinterpret_cast<const float4*>(a.p_part + slot(i) * ROWS * D) + c0 / 4 * ROWS + r;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float4 v = f[k * ROWS];
            acc[4 * k] = fmaf(w, v.x, acc[4 * k]);
            acc[4 * k + 1] = fmaf(w, v.y, acc[4 * k + 1]);
            acc[4 * k + 2] = fmaf(w, v.z, acc[4 * k + 2]);
            acc[4 * k + 3] = fmaf(w, v.w, acc[4 * k + 3]);
        }
    }
    const float inv = mx != -INFINITY ? KV4_BACK / l : 0.f;
    uint4* dst = reinterpret_cast<uint4*>(a.out + ((long long)(sp.q0 + t) * a.H + h) * D + c0);
    auto pk = [&](int x) { return pack_bf16x2(acc[x] * inv, acc[x + 1] * inv); };
    dst[0] = make_uint4(pk(0), pk(2), pk(4), pk(6));
    dst[1] = make_uint4(pk(8), pk(10), pk(12), pk(14));
}

template <int D> __global__ void __launch_bounds__(KP_THREADS, 1) kv4_prefill_kernel(const Kv4AttnArgs a) {
    constexpr int TILE = kp_tile<D>();
    constexpr int WPL = D / 32;   // code words of an expanding lane per key
    constexpr int DPH = D / 2;    // dims of O that a softmax thread writes
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* Ks = smem;              // 2 stages
    uint8_t* Vs = smem + 2 * TILE;   // 2 stages
    uint8_t* Qs = smem + 4 * TILE;
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + 5 * TILE);
    float* lsum = reinterpret_cast<float*>(smem + 5 * TILE + 256);  // [half][row]
    uint64_t *k_full = bars, *k_empty = bars + 2, *v_full = bars + 4, *v_empty = bars + 6, *s_full = bars + 8,
             *p_full = bars + 10, *pv_done = bars + 12, *q_full = bars + 14, *mma_done = bars + 15;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 16);
    __shared__ float red_max[2][2][KP_ROWS];
    // Which 16-key parts of a tile have no page, a byte each. Four tiles deep: the entry of tile g is
    // written again for tile g + 4 after S of tile g + 2 is complete, which was issued after
    // the softmax of tile g.
    __shared__ uint64_t holes[4];

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int G = a.G;
    pdl_wait();
    pdl_trigger();
    uint32_t* err = a.err;
    if ((int)blockIdx.x >= a.counts[0]) return;

    const int4 s0 = a.starts[blockIdx.x], s1 = a.starts[blockIdx.x + 1];
    const Walk start = {s0.x, s0.y, s0.z};

    if (warp == 0 && lane == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&k_full[i], 128);
            mbar_init(&k_empty[i], 1);
            mbar_init(&v_full[i], 128);
            mbar_init(&v_empty[i], 1);
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], 256);
            mbar_init(&pv_done[i], 1);
        }
        mbar_init(q_full, 256);
        mbar_init(mma_done, 1);
        fence_mbar_init();
    }
    if (warp == KP_MMA) {
        tc_alloc(tmem_slot, KP_TMEM_COLS);
        tc_relinquish();
    }
    const Work first = describe(a, s1, start);
    stage_q<D>(a, first, 0, Qs, threadIdx.x, KP_THREADS);
    fence_proxy_async();  // the tensor cores read Q through the async proxy
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;

    if (warp >= KP_EXPAND) {
        // ---------------- expansion: K and V tiles from codes ----------------
        // A warp takes 8 keys at a time, lane (key % 8, quarter of the head): the 8 lanes of a
        // store phase write the same chunk of 8 rows, which the swizzle puts into 8 places.
        const int w = warp - KP_EXPAND, key_l = w * 8 + (lane & 7), t = lane >> 3;
        const Kv4Rec rec = kv4_rec(1 << a.lp, D);
        const long long page_bytes = (long long)a.Hk * rec.bytes;
        // The next tile's codes are in registers while one is worked on; K's are asked for again as
        // soon as K is stored, and so on; the table entries one tile earlier still, and not looked at
        // before their tile is loaded.
        int page[4];  // table entries of the lane's keys i * 32 + key_l
        uint32_t kc[4][WPL], vc[4][WPL], kp[4], vp[4];
        int hole = 0;  // which of the lane's keys have no page
        auto look_up = [&](const Work& it, int j) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int key = (it.tile0 + j) * KP_KT + i * 32 + key_l;
                page[i] = 0;
                if (key < it.len) page[i] = a.table[(long long)it.b * a.max_blocks + (key >> a.lp)];
            }
        };
        auto load = [&](const Work& it, int j, bool is_v, uint32_t (&c)[4][WPL], uint32_t (&pr)[4]) {
            if (!is_v) hole = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int off = (i * 32 + key_l) & ((1 << a.lp) - 1);
                const bool there = (unsigned)page[i] < (unsigned)a.n_pages;
                const bool on = there && (it.tile0 + j) * KP_KT + i * 32 + key_l < it.len;
                if (!is_v && !there) hole |= 1 << i;
                const uint8_t* r = a.pool + page[i] * page_bytes + (uint32_t)(it.kvh * rec.bytes);
                const uint8_t* cp = r + (is_v ? rec.codes : 0) + off * (D / 2) + t * (D / 8);
                const uint8_t* pp = r + 2 * rec.codes + (is_v ? rec.pairs : 0) + off * (D / 8) + t * (D / 4) / KV4_GROUP * 4;
                pr[i] = 0;
                if (WPL == 4) {
                    uint4 x = make_uint4(0, 0, 0, 0);
                    if (on) x = __ldg(reinterpret_cast<const uint4*>(cp));
                    c[i][0] = x.x, c[i][1] = x.y, c[i][2 % WPL] = x.z, c[i][3 % WPL] = x.w;
                } else {
                    uint2 x = make_uint2(0, 0);
                    if (on) x = __ldg(reinterpret_cast<const uint2*>(cp));
                    c[i][0] = x.x, c[i][1] = x.y;
                }
                if (on) pr[i] = __ldg(reinterpret_cast<const uint32_t*>(pp));
            }
        };
        bool odd = false;
        auto store = [&](uint8_t* tile, const uint32_t (&c)[4][WPL], const uint32_t (&pr)[4]) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t q = kv4_pair(pr[i]);
                if (kv4_odd(q)) {
                    odd = true;
                    q = 0;
                }
                const uint32_t s2 = __byte_perm(q, 0, 0x1010), z2 = __byte_perm(q, 0, 0x3232), s2h = kv4_16th(s2);
                const int r = i * 32 + key_l;
#pragma unroll
                for (int x = 0; x < WPL; ++x) {
                    uint32_t v[4];
                    kv4_expand(c[i][x], s2, s2h, z2, v);
                    const int ch = t * WPL + x;
                    *reinterpret_cast<uint4*>(tile + (ch >> 3) * KP_HALF + r * 128 + (((ch & 7) ^ (r & 7)) << 4)) =
                        make_uint4(v[0], v[1], v[2], v[3]);
                }
            }
            fence_proxy_async();
        };
        Walk at = start;
        Work it = first;
        int j = 0, g = 0;  // g: running tile index over this CTA's items
        // the tile after (it, j); false at the share's end
        auto next = [&]() -> bool {
            if (++j < it.nkt) return true;
            j = 0;
            advance(a, at);
            it = describe(a, s1, at);
            return it.nkt > 0;
        };
        bool more = it.nkt > 0;
        if (more) {
            look_up(it, 0);
            load(it, 0, false, kc, kp);
            load(it, 0, true, vc, vp);
        }
        while (more) {
            const int b = it.b, h = hole, st = g & 1;
            more = next();
            if (more) look_up(it, j);
            const uint32_t empty = ((g >> 1) & 1) ^ 1u;
            if (!wait_for(&k_empty[st], empty, err, DERR_ATTN_TMA_WAIT)) break;
            if (!(w & 1) && lane == 0) {
#pragma unroll
                for (int i = 0; i < 4; ++i) reinterpret_cast<uint8_t*>(&holes[g & 3])[i * 2 + (w >> 1)] = h >> i & 1;
            }
            store(Ks + st * TILE, kc, kp);
            mbar_arrive(&k_full[st]);
            if (more) load(it, j, false, kc, kp);
            if (!wait_for(&v_empty[st], empty, err, DERR_ATTN_TMA_WAIT)) break;
            store(Vs + st * TILE, vc, vp);
            mbar_arrive(&v_full[st]);
            if (more) load(it, j, true, vc, vp);
            if (odd) a.odd[b] = 1;
            odd = false;
            ++g;
        }
    } else if (warp == KP_MMA) {
        // ---------------- MMA issuer ----------------
        if (elected()) {
            constexpr uint32_t idS = idesc_bf16_f32(KP_ROWS, KP_KT);
            constexpr uint32_t idO = idesc_bf16_f32_bmn(KP_ROWS, D);
            const uint64_t qd = smem_desc_sw128(smem_u32(Qs)), kd = smem_desc_sw128(smem_u32(Ks)), vd = smem_desc_sw128_mn(smem_u32(Vs), KP_HALF);
            auto issue_s = [&](int gg) -> bool {
                const int st = gg & 1;
                if (!wait_for(&k_full[st], (gg >> 1) & 1, err, DERR_ATTN_MMA_WAIT)) return false;
                tc_fence_after();
                const uint64_t ks = desc_at(kd, st * TILE);
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t off = (kk >> 2) * KP_HALF + (kk & 3) * 32;
                    tc_mma_f16(tmem_base + st * KP_KT, desc_at(qd, off), desc_at(ks, off), idS, kk != 0);
                }
                tc_commit(&k_empty[st]);
                tc_commit(&s_full[st]);
                return true;
            };
            bool ok = true;
            int g = 0;
            Walk at = start;
            for (int ki = 0; ok; ++ki) {
                const int nkt = ki ? describe(a, s1, at).nkt : first.nkt;
                if (nkt == 0) break;
                advance(a, at);
                if (ki > 0 && !wait_for(q_full, (ki - 1) & 1, err, DERR_ATTN_MMA_WAIT)) break;
                tc_fence_after();
                ok = issue_s(g);
                if (ok && nkt > 1) ok = issue_s(g + 1);
                for (int j = 0; j < nkt && ok; ++j) {
                    const int gg = g + j, st = gg & 1;
                    if (!wait_for(&p_full[st], (gg >> 1) & 1, err, DERR_ATTN_MMA_WAIT) ||
                        !wait_for(&v_full[st], (gg >> 1) & 1, err, DERR_ATTN_MMA_WAIT)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t vs = desc_at(vd, st * TILE);
                    const uint32_t pj = tmem_base + KP_TMEM_P + st * 64;
#pragma unroll
                    for (int kk = 0; kk < KP_KT / 16; ++kk)
                        mma_tmem_a(tmem_base + KP_TMEM_O, pj + kk * 8, desc_at(vs, kk * 2048), idO,
                                   (j | kk) != 0);
                    tc_commit(&v_empty[st]);
                    tc_commit(&pv_done[st]);
                    if (j + 2 < nkt) ok = issue_s(gg + 2);
                }
                g += nkt;
            }
            tc_commit(mma_done);  // arrives once every MMA issued above has completed
        }
    } else {
        // ---------------- softmax: two threads per row, 64 keys of each tile and half of O's dims each ----------------
        const int q4 = warp & 3, half = warp >> 2;  // the warp's TMEM lane quarter; its keys
        const int r = q4 * 32 + lane;
        const uint32_t lane_base = tmem_base + ((uint32_t)(q4 * 32) << 16);
        const float sl2 = a.scale_log2;
        bool ok = true;
        int g = 0;
        Kv4Split split = {};
        Walk at = start;
        for (Work it = first, nx; it.nkt > 0; it = nx) {
            const int rg = it.row0 + r, t = div_g(a, rg), h = it.kvh * G + (rg - t * G);
            const bool live = t < it.n;
            const int prow = live ? it.len - it.n + t : -1;  // the last key that the row sees
            const bool whole = it.nkt == it.all;
            if (!whole && it.tile0 == 0) split = split_of(a, at, it);
            advance(a, at);
            nx = describe(a, s1, at);
            float m_used = -INFINITY, l = 0.f;
            for (int j = 0; j < it.nkt; ++j) {
                const int gg = g + j, sb = gg & 1;
                if (ok && !wait_for(&s_full[sb], (gg >> 1) & 1, err, DERR_ATTN_SOFTMAX_WAIT)) ok = false;
                tc_fence_after();
                float s[64];
                {
                    uint32_t u[2][32];
#pragma unroll
                    for (int c = 0; c < 2; ++c) tc_ld_32x32b_x32(lane_base + sb * KP_KT + half * 64 + c * 32, u[c]);
                    tc_wait_ld();
#pragma unroll
                    for (int c = 0; c < 2; ++c)
#pragma unroll
                        for (int i = 0; i < 32; ++i) s[c * 32 + i] = __uint_as_float(u[c][i]);
                }
                const int key0 = (it.tile0 + j) * KP_KT + half * 64;
                const uint32_t hole = reinterpret_cast<const uint32_t*>(&holes[gg & 3])[half];
                if (hole) {
#pragma unroll
                    for (int i = 0; i < 64; ++i)
                        if (hole >> (i / 16 * 8) & 1) s[i] = -INFINITY;
                }
                if (key0 + 63 > prow) {
#pragma unroll
                    for (int i = 0; i < 64; ++i)
                        if (key0 + i > prow) s[i] = -INFINITY;
                }
                float mx4[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
                for (int i = 4; i < 64; i += 2) mx4[(i >> 1) & 3] = max3(mx4[(i >> 1) & 3], s[i], s[i + 1]);
                const float mine = max3(mx4[0], mx4[1], max_nan(mx4[2], mx4[3])) * sl2;
                red_max[sb][half][r] = mine;
                named_bar_sync(1 + q4, 64);
                const float m_new = max3(m_used, mine, red_max[sb][half ^ 1][r]);
                const bool need = !(m_new <= m_used + KP_RESCALE_LOG2);  // false while the row has seen no key; true for NaN
                const float alpha = need ? ex2(m_used - m_new) : 1.f;
                // P buffer sb is free once PV of running tile gg-2 has completed
                if (gg >= 2 && ok && !wait_for(&pv_done[sb], ((gg - 2) >> 1) & 1, err, DERR_ATTN_SOFTMAX_WAIT)) ok = false;
                if (j > 0 && __any_sync(0xffffffffu, need)) {
                    const int pg = gg - 1;
                    if (ok && !wait_for(&pv_done[pg & 1], (pg >> 1) & 1, err, DERR_ATTN_SOFTMAX_WAIT)) ok = false;
                    tc_fence_after();
#pragma unroll 1
                    for (int c = 0; c < DPH / 32; ++c) {
                        uint32_t u[32];
                        tc_ld_32x32b_x32(lane_base + KP_TMEM_O + half * DPH + c * 32, u);
                        tc_wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; i += 2) {
                            const float2 o = __fmul2_rn(make_float2(__uint_as_float(u[i]), __uint_as_float(u[i + 1])),
                                                        make_float2(alpha, alpha));
                            u[i] = __float_as_uint(o.x);
                            u[i + 1] = __float_as_uint(o.y);
                        }
                        tc_st_32x32b_x32(lane_base + KP_TMEM_O + half * DPH + c * 32, u);
                    }
                    tc_wait_st();
                }
                if (need) {
                    l *= alpha;
                    m_used = kept_max(m_new);
                }
                const float muse = m_used == -INFINITY ? 0.f : m_used;
                const float2 sl2x2 = make_float2(sl2, sl2), nmx2 = make_float2(-muse, -muse);
                float2 sum2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                uint32_t pw[32];
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    float2 p[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 x = __ffma2_rn(make_float2(s[c * 8 + 2 * e], s[c * 8 + 2 * e + 1]), sl2x2, nmx2);
                        p[e] = e < 3 ? make_float2(ex2(x.x), ex2(x.y)) : ex2_fma(x);  // a quarter on the FMA pipe
                        sum2[e & 1] = __fadd2_rn(sum2[e & 1], p[e]);
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        pw[c * 4 + e] = pack_bf16x2(p[e].x, p[e].y);
                        if (e == 3) pw[c * 4 + e] = less_clamp(pw[c * 4 + e]);
                    }
                }
                l += (sum2[0].x + sum2[0].y) + (sum2[1].x + sum2[1].y);
                tc_st_32x32b_x32(lane_base + KP_TMEM_P + sb * 64 + half * 32, pw);
                tc_wait_st();
                tc_fence_before();
                mbar_arrive(&p_full[sb]);
            }
            {
                // Q is free (the item's last S product is complete): stage the next item's while PV runs
                if (nx.nkt > 0) {
                    stage_q<D>(a, nx, 0, Qs, threadIdx.x, 256);
                    fence_proxy_async();
                    mbar_arrive(q_full);
                }
            }
            const int gl = g + it.nkt - 1;
            if (ok && !wait_for(&pv_done[gl & 1], (gl >> 1) & 1, err, DERR_ATTN_SOFTMAX_WAIT)) ok = false;
            tc_fence_after();
            lsum[half * KP_ROWS + r] = l;
            named_bar_sync(1 + q4, 64);
            l += lsum[(half ^ 1) * KP_ROWS + r];
            // a row that saw no key: 0
            const float inv = m_used != -INFINITY ? KV4_BACK / l : 0.f;
            __nv_bfloat16* dst = a.out + ((long long)(it.q0 + t) * a.H + h) * D + half * DPH;
            const long long prow_at = ((long long)blockIdx.x * 2 + (it.tile0 ? 0 : 1)) * KP_ROWS + r;  // of a part's result
            float4* part = reinterpret_cast<float4*>(a.p_part + (prow_at - r) * D) + half * DPH / 4 * KP_ROWS + r;
            if (!whole && half == 0) *reinterpret_cast<float2*>(a.p_ml + prow_at * 2) = make_float2(m_used, l);
#pragma unroll 1
            for (int c = 0; c < DPH / 32; ++c) {
                uint32_t u[32];
                tc_ld_32x32b_x32(lane_base + KP_TMEM_O + half * DPH + c * 32, u);
                tc_wait_ld();
                if (!whole) {
#pragma unroll
                    for (int i = 0; i < 32; i += 8) {
                        auto f = [&](int x) { return __uint_as_float(u[i + x]); };
                        part[(c * 8 + i / 4) * KP_ROWS] = make_float4(f(0), f(2), f(4), f(6));
                        part[(c * 8 + i / 4 + 1) * KP_ROWS] = make_float4(f(1), f(3), f(5), f(7));
                    }
                } else if (live) {
                    auto pk = [&](int x, int y) { return pack_bf16x2(__uint_as_float(u[x]) * inv, __uint_as_float(u[y]) * inv); };
#pragma unroll
                    for (int i = 0; i < 32; i += 8)  // columns hold the values 0, 4, 1, 5, 2, 6, 3, 7 of each 8
                        *reinterpret_cast<uint4*>(dst + c * 32 + i) = make_uint4(pk(i, i + 2), pk(i + 4, i + 6), pk(i + 1, i + 3), pk(i + 5, i + 7));
                }
            }
            g += it.nkt;
        }
        if (threadIdx.x == 0) a.splits[blockIdx.x] = split;
    }

    tc_fence_before();
    __syncthreads();
    if (warp == KP_MMA) {
        if (lane == 0) wait_for(mma_done, 0, err, DERR_ATTN_MMA_WAIT);  // before the accumulators are freed
        __syncwarp();
        tc_fence_after();
        tc_dealloc(tmem_base, KP_TMEM_COLS);
    }
}

// Expanded prompts: 256 query rows, as two blocks of 128 that take turns. While the softmax of one
// works on its scores, the tensor cores work for the other. Two blocks' S and O fill the tensor memory, so
// that P lies over S, and S of a block's next tile waits for its P V. A thread has a row: nothing is
// exchanged, and a tile of K and V serves twice the rows that the kernel above has.
//
// What bounds it (134 GFLOP, 177 us): the chain of a block's tile. At 1.7 GHz of 3500 clocks for two
// blocks' tiles the softmax takes 1900 (reading and maximum 600, exponentials 1200), P V behind the
// second half of P 480, S 950; the tensor cores alone would take 2048. Some 11000 clocks of an item's
// 70000 go by at its end, half of them while Q is staged.
// Tried: S by halves of the keys, so that half of it need not wait (N = 64 takes the tensor cores as long
// as 128: 212 us against 185); masks written into S instead of the registers (184 against 180);
// 0, 3/8, 1/2 and 5/8 of the exponentials on the FMA pipe (191, 188, 187, 193 against 184 with 1/4); two
// threads per row, 16 softmax warps at 96 registers (192 against 180); Q of all items staged by the softmax warps
// (182 against 180; of the first item alone, which nothing else could wait for, 176.4 against 177.2).
template <int D> __global__ void __launch_bounds__(KQ_THREADS, 1) kv4_expanded_kernel(const Kv4AttnArgs a) {
    constexpr int TILE = kp_tile<D>();
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* Ks = smem;              // 2 stages
    uint8_t* Vs = smem + 2 * TILE;   // 2 stages
    uint8_t* Qs = smem + 4 * TILE;   // 2 blocks
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + 6 * TILE);
    uint64_t *k_full = bars, *k_empty = bars + 2, *v_full = bars + 4, *v_empty = bars + 6;  // by stage
    uint64_t *s_full = bars + 8, *pv_done = bars + 10, *q_full = bars + 12, *q_empty = bars + 14;  // by block
    uint64_t *p_full = bars + 16, *mma_done = bars + 20;  // p_full: by block and half of the keys
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 21);
    // As above: the entry of tile g is written again for tile g + 4 after both S of tile g + 2 are
    // complete, which were issued after the softmax of tile g.
    __shared__ uint64_t holes[4];

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_wait();
    pdl_trigger();
    uint32_t* err = a.err;
    if ((int)blockIdx.x >= a.counts[0]) return;
    const int4 s0 = a.starts[blockIdx.x], s1 = a.starts[blockIdx.x + 1];
    const Walk start = {s0.x, s0.y, s0.z};
    const Work first = describe(a, s1, start);
    bool ok = true;
    // the loader's thread: K and V of tile j of an item, the CTA's tile g
    int copied = 0;  // copies begun
    auto copy = [&](const Work& it, int j, int g) {
        const int st = g & 1;
        const uint32_t empty = ((g >> 1) & 1) ^ 1u;
        const long long image = it.image + it.tile0 + j;
        const uint8_t* src = a.images + image * 2 * TILE;
        const uint64_t no_page = a.holes[image];
        if (!(ok = wait_for(&k_empty[st], empty, err, DERR_ATTN_TMA_WAIT))) return;
        holes[g & 3] = no_page;
        mbar_arrive_expect_tx(&k_full[st], TILE);
        copy_tile(Ks + st * TILE, src, TILE, &k_full[st]);
        ++copied;
        if (!(ok = wait_for(&v_empty[st], empty, err, DERR_ATTN_TMA_WAIT))) return;
        mbar_arrive_expect_tx(&v_full[st], TILE);
        copy_tile(Vs + st * TILE, src + TILE, TILE, &v_full[st]);
        ++copied;
    };
    if (warp == KQ_LOAD) {
        if (elected()) {
            for (int i = 0; i < 2; ++i) {
                mbar_init(&k_full[i], 1);
                mbar_init(&k_empty[i], 1);
                mbar_init(&v_full[i], 1);
                mbar_init(&v_empty[i], 1);
                mbar_init(&s_full[i], 1);
                for (int half = 0; half < 2; ++half) mbar_init(&p_full[i * 2 + half], 128);
                mbar_init(&pv_done[i], 1);
                mbar_init(&q_full[i], 32);
                mbar_init(&q_empty[i], 1);
            }
            mbar_init(mma_done, 1);
            fence_mbar_init();
            for (int j = 0; j < 2 && j < first.nkt; ++j) copy(first, j, j);  // the first waits pass
        }
        __syncwarp();
    }
    if (warp == KP_MMA) {
        tc_alloc(tmem_slot, KP_TMEM_COLS);
        tc_relinquish();
    }
    // rows `from` to `to` of the 128 query rows of block x of an item, rows behind the last as zeros
    auto stage = [&](const Work& it, int x, int from, int to) {
        constexpr int CH = D / 8, ROWS = 32 / CH;  // 16-byte chunks of a row, rows of a warp's copy
        const int c = lane % CH, r0 = lane / CH, rg0 = it.row0 + x * KP_ROWS + r0;
        // row rg is token t = rg / G and head kvh G + rg - t G
        const __nv_bfloat16* src = a.q + ((long long)it.q0 * a.H + it.kvh * a.G) * D + c * 8;
        const long long token = (long long)(a.H - a.G) * D;
        uint8_t* dst = Qs + x * TILE + (c >> 3) * KP_HALF;
#pragma unroll 8
        for (int i = from; i < to; i += ROWS) {
            const int r = i + r0, rg = rg0 + i, tok = div_g(a, rg);
            const bool live = tok < it.n;
            copy_16(dst + r * 128 + (((c & 7) ^ (r & 7)) << 4), live ? src + tok * token + (long long)rg * D : a.q, live);
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        fence_proxy_async();  // the tensor cores read Q through the async proxy
    };
    if (warp < KP_MMA) stage(first, warp >> 2, (warp & 3) * 32, (warp & 3) * 32 + 32);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;

    if (warp >= KQ_Q) {
        // ---------------- Q of the items ----------------
        const int x = warp - KQ_Q;
        Walk at = start;
        for (int ki = 0;; ++ki) {
            mbar_arrive(&q_full[x]);
            advance(a, at);
            const Work it = describe(a, s1, at);
            if (it.nkt == 0 || !wait_for(&q_empty[x], ki & 1, err, DERR_ATTN_TMA_WAIT)) break;
            __syncwarp();
            stage(it, x, 0, KP_ROWS);
        }
    } else if (warp == KQ_LOAD) {
        // ---------------- copies of K and V ----------------
        if (elected()) {
            int g = 0, j = min(2, first.nkt);
            Walk at = start;
            for (Work it = first; ok && it.nkt > 0; advance(a, at), it = describe(a, s1, at), j = 0) {
                for (; ok && j < it.nkt; ++j) copy(it, j, g + j);
                g += it.nkt;
            }
            if (!ok)  // copies on their way land before the CTA can exit
                for (int x = max(0, copied - 4); x < copied; ++x)
                    wait_for(&(x & 1 ? v_full : k_full)[(x >> 1) & 1], (x >> 2) & 1, nullptr, 0);
        }
    } else if (warp == KP_MMA) {
        // ---------------- MMA issuer ----------------
        if (elected()) {
            constexpr uint32_t idS = idesc_bf16_f32(KP_ROWS, KP_KT);
            constexpr uint32_t idO = idesc_bf16_f32_bmn(KP_ROWS, D);
            auto need = [&](uint64_t* bar, uint32_t parity) {
                if (ok && !mbar_wait(bar, parity, err, DERR_ATTN_MMA_WAIT)) ok = false;
                return ok;
            };
            const uint64_t qd = smem_desc_sw128(smem_u32(Qs)), kd = smem_desc_sw128(smem_u32(Ks)), vd = smem_desc_sw128_mn(smem_u32(Vs), KP_HALF);
            // S of a block's tile gg, over P of tile gg - 1; `last` of the item
            auto issue_s = [&](int x, int gg, bool last) {
                if (!need(&k_full[gg & 1], (gg >> 1) & 1) || (gg > 0 && !need(&pv_done[x], (gg - 1) & 1))) return;
                const uint64_t qs = desc_at(qd, x * TILE), ks = desc_at(kd, (gg & 1) * TILE);
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t off = (kk >> 2) * KP_HALF + (kk & 3) * 32;
                    tc_mma_f16(tmem_base + x * KP_KT, desc_at(qs, off), desc_at(ks, off), idS, kk != 0);
                }
                if (x) tc_commit(&k_empty[gg & 1]);
                tc_commit(&s_full[x]);
                if (last) tc_commit(&q_empty[x]);
            };
            int g = 0;
            Walk at = start;
            for (int x = 0; x < 2 && ok && first.nkt > 0; ++x)
                if (need(&q_full[x], 0)) issue_s(x, 0, first.nkt == 1);
            for (int ki = 0, nkt = first.nkt, nx; ok && nkt > 0; ++ki, nkt = nx) {
                advance(a, at);
                nx = describe(a, s1, at).nkt;
                for (int j = 0; j < nkt && ok; ++j) {
                    const int gg = g + j, st = gg & 1;
                    for (int x = 0; x < 2 && ok; ++x) {
                        const uint64_t vs = desc_at(vd, st * TILE);
                        auto issue_pv = [&](int half) {
#pragma unroll
                            for (int kk = half * 4; kk < half * 4 + 4; ++kk)
                                mma_tmem_a(tmem_base + KP_TMEM_O + x * 128, tmem_base + x * KP_KT + kk * 8,
                                           desc_at(vs, kk * 2048), idO, (j | kk) != 0);
                        };
                        if (!need(&p_full[x * 2], gg & 1) || !need(&v_full[st], (gg >> 1) & 1)) break;
                        tc_fence_after();
                        issue_pv(0);
                        if (!need(&p_full[x * 2 + 1], gg & 1)) break;
                        tc_fence_after();
                        issue_pv(1);
                        if (x) tc_commit(&v_empty[st]);
                        tc_commit(&pv_done[x]);
                        if (j + 1 < nkt) issue_s(x, gg + 1, j + 2 == nkt);
                        else if (nx > 0 && need(&q_full[x], (ki + 1) & 1)) issue_s(x, gg + 1, nx == 1);
                    }
                }
                g += nkt;
            }
            tc_commit(mma_done);  // arrives once every MMA issued above has completed
        }
    } else {
        // ---------------- softmax: a thread per row ----------------
        const int x = warp >> 2, q4 = warp & 3, r = q4 * 32 + lane, row = x * KP_ROWS + r;
        const uint32_t lanes = tmem_base + ((uint32_t)(q4 * 32) << 16), S = lanes + x * KP_KT, O = lanes + KP_TMEM_O + x * 128;
        const float sl2 = a.scale_log2;
        int g = 0;
        Kv4Split split = {};
        Walk at = start;
        for (Work it = first, nx; it.nkt > 0; it = nx) {
            const int rg = it.row0 + row, t = div_g(a, rg), h = it.kvh * a.G + (rg - t * a.G);
            const bool live = t < it.n;
            // the last key that the row sees; rows behind the last are masked nowhere, which costs no time
            const int prow = live ? it.len - it.n + t : 0x7fffffff;
            const bool whole = it.nkt == it.all;
            if (!whole && it.tile0 == 0) split = split_of(a, at, it);
            advance(a, at);
            nx = describe(a, s1, at);
            float m_used = -INFINITY, l = 0.f;
            for (int j = 0; j < it.nkt; ++j) {
                const int gg = g + j;
                const int key0 = (it.tile0 + j) * KP_KT;
                if (ok && !wait_for(&s_full[x], gg & 1, err, DERR_ATTN_SOFTMAX_WAIT)) ok = false;
                tc_fence_after();
                // All scores for the maximum; the upper half is read a second time for the exponentials, which
                // leaves them their registers (168 a thread).
                uint32_t s[4][32];
#pragma unroll
                for (int c = 0; c < 4; ++c) tc_ld_32x32b_x32(S + c * 32, s[c]);
                tc_wait_ld();
                const uint64_t hole = holes[gg & 3];
                const bool masked = __any_sync(0xffffffffu, hole != 0 || key0 + KP_KT - 1 > prow);
                auto f = [&](int i) { return __uint_as_float(s[i >> 5][i & 31]); };
                const int seen = prow - key0;  // the last key of the tile that the row sees
                auto mask = [&](int c) {
                    if (hole)
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if ((uint32_t)(hole >> (c * 16)) >> (i / 16 * 8) & 1) s[c][i] = 0xFF800000u;
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (c * 32 + i > seen) s[c][i] = 0xFF800000u;
                };
                if (masked) {
#pragma unroll
                    for (int c = 0; c < 4; ++c) mask(c);
                }
                float mx[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) mx[e] = max_nan(f(e), f(4 + e));
#pragma unroll
                for (int i = 8; i < 128; i += 8)
#pragma unroll
                    for (int e = 0; e < 4; ++e) mx[e] = max3(mx[e], f(i + e), f(i + 4 + e));
                const float m_new = max_nan(m_used, max3(mx[0], mx[1], max_nan(mx[2], mx[3])) * sl2);
                const bool need = !(m_new <= m_used + KP_RESCALE_LOG2);  // false while the row has seen no key; true for NaN
                if (j > 0 && __any_sync(0xffffffffu, need)) {
                    // P V of the tile before is complete: the scores were issued after it
                    const float alpha = need ? ex2(m_used - m_new) : 1.f;
                    l *= alpha;
#pragma unroll 1
                    for (int c = 0; c < D / 16; ++c) {
                        uint32_t u[16];
                        tc_ld_x16(O + c * 16, u);
                        tc_wait_ld();
#pragma unroll
                        for (int i = 0; i < 16; i += 2) {
                            const float2 o = __fmul2_rn(make_float2(__uint_as_float(u[i]), __uint_as_float(u[i + 1])),
                                                        make_float2(alpha, alpha));
                            u[i] = __float_as_uint(o.x);
                            u[i + 1] = __float_as_uint(o.y);
                        }
                        tc_st_x16(O + c * 16, u);
                    }
                    tc_wait_st();
                }
                if (need) m_used = kept_max(m_new);
                const float muse = m_used == -INFINITY ? 0.f : m_used;
                const float2 sl2x2 = make_float2(sl2, sl2), nmx2 = make_float2(-muse, -muse);
                float2 sum2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    if (c < 2) tc_ld_32x32b_x32(S + (2 + c) * 32, s[2 + c]);
                    uint32_t pw[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const float2 y = __ffma2_rn(make_float2(f(c * 32 + 2 * e), f(c * 32 + 2 * e + 1)), sl2x2, nmx2);
                        const float2 p = (e & 3) < 3 ? make_float2(ex2(y.x), ex2(y.y)) : ex2_fma(y);  // a quarter on the FMA pipe
                        sum2[e & 1] = __fadd2_rn(sum2[e & 1], p);
                        pw[e] = pack_bf16x2(p.x, p.y);
                        if ((e & 3) == 3) pw[e] = less_clamp(pw[e]);
                    }
                    tc_st_x16(S + c * 16, pw);
                    if (c == 1) {
                        tc_wait_ld();
                        tc_wait_st();
                        tc_fence_before();
                        mbar_arrive(&p_full[x * 2]);
                        if (masked) {
                            mask(2);
                            mask(3);
                        }
                    }
                }
                l += (sum2[0].x + sum2[0].y) + (sum2[1].x + sum2[1].y);
                tc_wait_st();
                tc_fence_before();
                mbar_arrive(&p_full[x * 2 + 1]);
            }
            g += it.nkt;
            if (ok && !wait_for(&pv_done[x], (g - 1) & 1, err, DERR_ATTN_SOFTMAX_WAIT)) ok = false;
            tc_fence_after();
            // a row that saw no key: 0
            const float inv = m_used != -INFINITY ? KV4_BACK / l : 0.f;
            __nv_bfloat16* dst = a.out + ((long long)(it.q0 + t) * a.H + h) * D;
            const long long slot = (long long)blockIdx.x * 2 + (it.tile0 ? 0 : 1);  // of a part's result
            float4* part = reinterpret_cast<float4*>(a.p_part + slot * KQ_ROWS * D) + row;
            if (!whole) *reinterpret_cast<float2*>(a.p_ml + (slot * KQ_ROWS + row) * 2) = make_float2(m_used, l);
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
                uint32_t u[32];
                tc_ld_32x32b_x32(O + c * 32, u);
                tc_wait_ld();
                if (!whole) {
#pragma unroll
                    for (int i = 0; i < 32; i += 8) {
                        auto f = [&](int k) { return __uint_as_float(u[i + k]); };
                        part[(c * 8 + i / 4) * KQ_ROWS] = make_float4(f(0), f(1), f(2), f(3));
                        part[(c * 8 + i / 4 + 1) * KQ_ROWS] = make_float4(f(4), f(5), f(6), f(7));
                    }
                } else if (live) {
                    auto pk = [&](int k) { return pack_bf16x2(__uint_as_float(u[k]) * inv, __uint_as_float(u[k + 1]) * inv); };
#pragma unroll
                    for (int i = 0; i < 32; i += 8) *reinterpret_cast<uint4*>(dst + c * 32 + i) = make_uint4(pk(i), pk(i + 2), pk(i + 4), pk(i + 6));
                }
            }
            tc_fence_before();  // the next item's first P V, after this thread's next arrival, writes O anew
        }
        if (threadIdx.x == 0) a.splits[blockIdx.x] = split;
    }

    tc_fence_before();
    __syncthreads();
    if (warp == KP_MMA) {
        if (lane == 0) wait_for(mma_done, 0, err, DERR_ATTN_MMA_WAIT);  // before the accumulators are freed
        __syncwarp();
        tc_fence_after();
        tc_dealloc(tmem_base, KP_TMEM_COLS);
    }
}

template <int D> cudaError_t launch(const Kv4AttnArgs& a, cudaStream_t s) {
    const int sms = current_num_sms();
    const bool images = a.images_cap > 0;
    cudaError_t e = launch_k(kv4_blocks_kernel, dim3(1), dim3(KP_LIST), 0, s, true, a, sms, images ? KQ_ROWS : KP_ROWS);
    if (e != cudaSuccess) return e;
    if (!images) {
        e = cudaFuncSetAttribute(kv4_prefill_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, kp_smem<D>());
        if (e != cudaSuccess) return e;
        e = launch_k(kv4_prefill_kernel<D>, dim3(sms), dim3(KP_THREADS), kp_smem<D>(), s, true, a);
        if (e != cudaSuccess) return e;
        return launch_k(kv4_prefill_join_kernel<D, KP_ROWS>, dim3(sms, D / 16), dim3(KP_ROWS), 0, s, true, a);
    }
    e = launch_k(kv4_expand_kernel<D>, dim3(6 * sms), dim3(256), 0, s, true, a);
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(kv4_expanded_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, kq_smem<D>());
    if (e != cudaSuccess) return e;
    e = launch_k(kv4_expanded_kernel<D>, dim3(sms), dim3(KQ_THREADS), kq_smem<D>(), s, true, a);
    if (e != cudaSuccess) return e;
    e = launch_k(kv4_prefill_join_kernel<D, KQ_ROWS>, dim3(sms, D / 16), dim3(KQ_ROWS), 0, s, true, a);
    if (e != cudaSuccess || a.turn == 0) return e;
    Kv4AttnArgs rest = a;
    rest.images_cap = 0;
    rest.turn = 2;
    return launch<D>(rest, s);
}

}  // namespace

cudaError_t launch_kv4_prefill(const Kv4AttnArgs& a, int d, cudaStream_t s) {
    return d == 128 ? launch<128>(a, s) : launch<64>(a, s);
}

}  // namespace lfw
