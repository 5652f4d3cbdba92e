// Norms of queries and keys per head, the position rotation, and the append of keys and
// values to the 4-bit paged cache, in one pass over a step's projections.
//
// Per token and head of q and k: y = x w / sqrt(mean x^2 + eps) (when w is given), then
// pairs (2i, 2i + 1) turn by the angle whose cosine and sine the tables hold for the
// token's position. q is stored in bf16. k (after that) and v (as it comes) are cut into
// groups of 32 values; in 32-bit floats, each operation rounded by itself,
//   s = bf16((mx - mn) * (1/15)), z = bf16(mn), c = clamp(rint((x - z) * (1/s)), 0, 15),
// with s = 0 and c = 0 where s would be below the smallest normal float. A group that
// holds an infinity or a NaN, or whose range does not fit a float, is stored as NaN: it
// reads back as NaN instead of passing for finite values.
//
// The keys' norm and rotation run in fp64. A code is a rounding decision with steps of a
// fifteenth of the range: in fp32 the order of a sum would decide a code near a border, and
// what a call stores would depend on how its kernel sums. The queries, rounded to bf16 next,
// take fp32, with a second sum for rows whose squares pass its range. (LLM_FLAG_KV4's own path
// does not come through here: its keys are rotated in fp32 by the projection's epilogue and
// rounded to bf16, and kv4_store_kernel codes those.)
//
// Every input element is read once, in 16-byte loads; a lane holds 8 consecutive values, so a
// head row is 16 lanes at d = 128 (8 at 64), a group of 32 is 4 lanes, and the code word of a
// lane is one store. That width and not 4 values a lane: with 32 KV heads the issue slots
// bound the pass, and sums, group minima and scales are per lane and step, not per value.
// Measured: 2048 tokens of 32 + 2 x 8 fp32 heads 17.9 us, 4.4 TB/s (67% of the copy bandwidth; 4
// values a lane 26.7 us); 9070 tokens of 32 + 2 x 32 bf16 heads 118.5 us, 4.2 TB/s (338 us);
// one token 3.0 us.
#include "../../include/llama_fwd.h"
#include "kernels.cuh"
#include "kv4.cuh"

#include <float.h>

#include <type_traits>

namespace lfw {
namespace {

constexpr int AP_WARPS = 8;

struct AppendArgs {
    const void *q, *k, *v;
    long long q_ld, k_ld, v_ld;  // elements from a token to the next
    const void *q_norm, *k_norm;
    float eps;
    const float *cos_t, *sin_t;
    int n_pos;
    const int32_t* positions;
    const int64_t* slots;
    int N, H, Hk;
    __nv_bfloat16 *q_out, *k_out, *v_out;
    uint8_t* pool;
    long long n_slots, page_bytes;
    int lp;
};

constexpr int VPL = 8;     // consecutive values a lane
constexpr int PASSES = 2;  // head rows of a lane in flight

template <typename T> struct Raw;  // VPL values as loaded
template <> struct Raw<float> {
    float4 a, b;
    DEVI void load(const float* p) { a = __ldcs(reinterpret_cast<const float4*>(p)), b = __ldcs(reinterpret_cast<const float4*>(p) + 1); }
    DEVI void get(float (&x)[VPL]) const {
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    }
};
template <> struct Raw<__nv_bfloat16> {
    uint4 a;
    DEVI void load(const __nv_bfloat16* p) { a = __ldcs(reinterpret_cast<const uint4*>(p)); }
    DEVI void get(float (&x)[VPL]) const {
        x[0] = bf16lo(a.x), x[1] = bf16hi(a.x), x[2] = bf16lo(a.y), x[3] = bf16hi(a.y);
        x[4] = bf16lo(a.z), x[5] = bf16hi(a.z), x[6] = bf16lo(a.w), x[7] = bf16hi(a.w);
    }
};
DEVI void store_bf16(__nv_bfloat16* p, const uint32_t (&w)[VPL / 2]) {
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

DEVI float inv_sqrt(float v) { return 1.f / sqrtf(v); }
DEVI double inv_sqrt(double v) { return rsqrt(v); }

// Norm (w: the lane's weights, or none) and rotation of a head row spread over LPR lanes (their
// mask: row), in type A.
template <typename A, int LPR>
DEVI void norm_rotate(A (&y)[VPL], const float (&x)[VPL], bool norm, const float (&w)[VPL], A eps, unsigned row,
                      const float (&cs)[VPL / 2], const float (&sn)[VPL / 2]) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) y[i] = (A)x[i];
    if (norm) {
        A ss = 0;
#pragma unroll
        for (int i = 0; i < VPL; ++i) ss += y[i] * y[i];
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(row, ss, o);
        A r = inv_sqrt(ss * (A)(1.0 / (LPR * VPL)) + eps);
        if (sizeof(A) == 4 && ss > FLT_MAX) {  // squares beyond fp32: the same of x 2^-70 (the row's lanes agree)
            ss = 0;
#pragma unroll
            for (int i = 0; i < VPL; ++i) ss += (y[i] * (A)0x1p-70) * (y[i] * (A)0x1p-70);
#pragma unroll
            for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(row, ss, o);
            r = (A)0x1p-70 * inv_sqrt(ss * (A)(1.0 / (LPR * VPL)) + eps * (A)0x1p-140);
        }
#pragma unroll
        for (int i = 0; i < VPL; ++i) y[i] = y[i] * r * (A)w[i];
    }
#pragma unroll
    for (int i = 0; i < VPL / 2; ++i) {
        const A a = y[2 * i], b = y[2 * i + 1], c = (A)cs[i], s = (A)sn[i];
        y[2 * i] = a * c - b * s;
        y[2 * i + 1] = a * s + b * c;
    }
}

// A minimum that a NaN does not drop out of.
DEVI float min_nan(float a, float b) {
    float d;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}

// The codes of a lane's 8 values (a word), their group's pair, and as bf16 pairs the values that
// they stand for.
DEVI uint32_t quantise(const float (&x)[VPL], unsigned row, uint32_t& pair, uint32_t (&val)[VPL / 2]) {
    float mn = x[0], mx = x[0];
#pragma unroll
    for (int i = 1; i < VPL; ++i) {
        mn = min_nan(mn, x[i]);
        mx = max_nan(mx, x[i]);
    }
#pragma unroll
    for (int o = KV4_GROUP / VPL / 2; o > 0; o >>= 1) {
        mn = min_nan(mn, __shfl_xor_sync(row, mn, o));
        mx = max_nan(mx, __shfl_xor_sync(row, mx, o));
    }
    __nv_bfloat16 s = __float2bfloat16_rn(__fmul_rn(__fsub_rn(mx, mn), 1.0f / 15.0f)), z = __float2bfloat16_rn(mn);
    float sf = __bfloat162float(s);
    const float zf = __bfloat162float(z);
    const bool fine = sf <= FLT_MAX && fabsf(zf) <= FLT_MAX;
    if (sf < FLT_MIN) {
        sf = 0.f;
        s = __float2bfloat16_rn(0.f);
    }
    if (!fine) s = z = __ushort_as_bfloat16(0x7FFF);
    const float inv = sf > 0.f ? __frcp_rn(sf) : 0.f;
    const __nv_bfloat162 s2 = __halves2bfloat162(s, s), z2 = __halves2bfloat162(z, z), sz = __halves2bfloat162(s, z);
    pair = *reinterpret_cast<const uint32_t*>(&sz);
    // 1.5 * 2^23 added: the nearest integer (ties to even) in the low bits of the sum
    float c[VPL];
    uint32_t word = 0;
#pragma unroll
    for (int i = VPL - 1; i >= 0; --i) {
        c[i] = __fadd_rn(fminf(fmaxf(__fmul_rn(__fsub_rn(x[i], zf), inv), 0.f), 15.f), 12582912.f);
        word = word * 16 + __float_as_uint(c[i]);  // the sums' common bits are taken off at the end
    }
    word -= 0x4B400000u * 0x11111111u;
#pragma unroll
    for (int i = 0; i < VPL / 2; ++i) {
        const __nv_bfloat162 v = __hfma2(__floats2bfloat162_rn(c[2 * i] - 12582912.f, c[2 * i + 1] - 12582912.f), s2, z2);
        val[i] = *reinterpret_cast<const uint32_t*>(&v);
    }
    return fine ? word : 0u;
}

// A block takes one group of PASSES x 32 / LPR heads of one kind (blockIdx.y; the queries' groups,
// then the keys', then the values') and a warp every so many tokens of it, the next token's
// loads in flight while one is worked on: weights, head pointers and kind are settled once.
template <typename TIn, typename TW, int D, int KIND> DEVI void append_tokens(const AppendArgs& a, int h0) {
    constexpr int LPR = D / VPL, RPW = 32 / LPR;  // lanes per row, rows at a time
    using A = typename std::conditional<KIND == 1, double, float>::type;
    const int lane = threadIdx.x & 31, sub = lane / LPR, at = lane % LPR * VPL;
    const unsigned row = ((1u << LPR) - 1u) << (sub * LPR);
    const int heads = KIND == 0 ? a.H : a.Hk, h = h0 + sub;
    const TIn* src = reinterpret_cast<const TIn*>(KIND == 0 ? a.q : KIND == 1 ? a.k : a.v) + h * D + at;
    const long long ld = KIND == 0 ? a.q_ld : KIND == 1 ? a.k_ld : a.v_ld;
    __nv_bfloat16* out = KIND == 0 ? a.q_out : KIND == 1 ? a.k_out : a.v_out;
    const TW* wp = reinterpret_cast<const TW*>(KIND == 0 ? a.q_norm : a.k_norm);
    const bool norm = KIND != 2 && wp != nullptr;
    float w[VPL] = {};
    if (norm) {
        Raw<TW> wr;
        wr.load(wp + at);
        wr.get(w);
    }
    const Kv4Rec rec = kv4_rec(1 << a.lp, D);
    Raw<TIn> next[PASSES];
    int next_pos = -1;
    long long next_slot = -1;
    auto fetch = [&](int n) {
#pragma unroll
        for (int j = 0; j < PASSES; ++j)
            if (h + j * RPW < heads) next[j].load(src + n * ld + j * RPW * D);
        next_pos = a.positions[n];
        if (KIND != 0) next_slot = a.slots[n];
    };
    const int step = gridDim.x * AP_WARPS;
    int n = blockIdx.x * AP_WARPS + (threadIdx.x >> 5);
    if (n < a.N) fetch(n);
    for (; n < a.N; n += step) {
        Raw<TIn> raw[PASSES];
#pragma unroll
        for (int j = 0; j < PASSES; ++j) raw[j] = next[j];
        const int pos = next_pos;
        const long long slot = next_slot;
        if (n + step < a.N) fetch(n + step);
        if (pos < 0 || pos >= a.n_pos) continue;  // a padding row, or a position without a table row
        float cs[VPL / 2] = {}, sn[VPL / 2] = {};
        if (KIND != 2) {
            const float4 c = *reinterpret_cast<const float4*>(a.cos_t + (long long)pos * (D / 2) + at / 2);
            const float4 s = *reinterpret_cast<const float4*>(a.sin_t + (long long)pos * (D / 2) + at / 2);
            cs[0] = c.x, cs[1] = c.y, cs[2] = c.z, cs[3] = c.w;
            sn[0] = s.x, sn[1] = s.y, sn[2] = s.z, sn[3] = s.w;
        }
#pragma unroll
        for (int j = 0; j < PASSES; ++j) {
            if (h + j * RPW >= heads) break;
            float x[VPL];
            raw[j].get(x);
            uint32_t v[VPL / 2];
            const long long row_out = ((long long)n * heads + h + j * RPW) * D + at;
            if (KIND != 2) {
                A y[VPL];
                norm_rotate<A, LPR>(y, x, norm, w, (A)a.eps, row, cs, sn);
#pragma unroll
                for (int i = 0; i < VPL; ++i) x[i] = (float)y[i];
            }
            if (KIND == 0) {
#pragma unroll
                for (int i = 0; i < VPL / 2; ++i) v[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
                store_bf16(out + row_out, v);
                continue;
            }
            uint32_t pair;
            const uint32_t word = quantise(x, row, pair, v);
            if (slot >= 0 && slot < a.n_slots) {
                const int off = (int)slot & ((1 << a.lp) - 1);
                uint8_t* r = a.pool + (slot >> a.lp) * a.page_bytes + (uint32_t)((h + j * RPW) * rec.bytes);
                *reinterpret_cast<uint32_t*>(r + (KIND == 2 ? rec.codes : 0) + off * (D / 2) + at / 2) = word;
                if (at % KV4_GROUP == 0)
                    *reinterpret_cast<uint32_t*>(r + 2 * rec.codes + (KIND == 2 ? rec.pairs : 0) + off * (D / 8) + at / KV4_GROUP * 4) = pair;
            }
            if (out) store_bf16(out + row_out, v);
        }
    }
}

template <typename TIn, typename TW, int D>
__global__ void __launch_bounds__(AP_WARPS * 32, 3) qk_norm_rope_kv4_kernel(const AppendArgs a) {
    constexpr int HPB = PASSES * 32 * VPL / D;  // heads of a group
    pdl_wait();
    pdl_trigger();
    const int qg = (a.H + HPB - 1) / HPB, kg = (a.Hk + HPB - 1) / HPB, g = blockIdx.y;
    if (g < qg) append_tokens<TIn, TW, D, 0>(a, g * HPB);
    else if (g < qg + kg) append_tokens<TIn, TW, D, 1>(a, (g - qg) * HPB);
    else append_tokens<TIn, TW, D, 2>(a, (g - qg - kg) * HPB);
}

template <typename TIn, typename TW, int D> cudaError_t launch_append(const AppendArgs& a, cudaStream_t s) {
    constexpr int HPB = PASSES * 32 * VPL / D;
    const int groups = (a.H + HPB - 1) / HPB + 2 * ((a.Hk + HPB - 1) / HPB);
    // 8 blocks per SM where there are tokens enough: the 3 that fit at once and their successors, since the
    // keys' blocks take longer (4 per SM: 126 us for 9070 tokens of 32 + 2 x 32 heads, 8: 122, 24: 123)
    const int want = (a.N + AP_WARPS - 1) / AP_WARPS, most = (current_num_sms() * 8 + groups - 1) / groups;
    return launch_k(qk_norm_rope_kv4_kernel<TIn, TW, D>, dim3(want < most ? want : most, groups), dim3(AP_WARPS * 32), 0, s,
                    true, a);
}
template <typename TIn, typename TW> cudaError_t launch_append(const AppendArgs& a, int d, cudaStream_t s) {
    return d == 128 ? launch_append<TIn, TW, 128>(a, s) : launch_append<TIn, TW, 64>(a, s);
}

// One head row of keys or values per D / 8 lanes.
template <int D> __global__ void __launch_bounds__(AP_WARPS * 32) kv4_store_kernel(const Kv4StoreArgs a) {
    constexpr int LPR = D / VPL, RPB = AP_WARPS * 32 / LPR;  // lanes per row, rows per block
    const int sub = threadIdx.x / LPR, at = threadIdx.x % LPR * VPL;
    const unsigned row = ((1u << LPR) - 1u) << ((threadIdx.x & 31) / LPR * LPR);
    pdl_wait();
    pdl_trigger();
    const int i = blockIdx.x * RPB + sub, n = i / (2 * a.Hk), h = i % (2 * a.Hk), kvh = h % a.Hk;
    if (n >= a.N) return;
    const bool is_v = h >= a.Hk;
    const int pos = a.positions[n];
    const long long slot = a.slots[n];
    if (pos < 0 || pos >= a.S_max || slot < 0 || slot >= a.n_slots) return;
    Raw<__nv_bfloat16> raw;
    raw.load((is_v ? a.v : a.k) + (((long long)(n / a.T) * a.Hk + kvh) * a.S_max + pos) * D + at);
    float x[VPL];
    raw.get(x);
    uint32_t pair, val[VPL / 2];
    const uint32_t word = quantise(x, row, pair, val);
    const Kv4Rec rec = kv4_rec(1 << a.lp, D);
    const int off = (int)slot & ((1 << a.lp) - 1);
    uint8_t* r = a.pool + (slot >> a.lp) * a.page_bytes + (uint32_t)(kvh * rec.bytes);
    *reinterpret_cast<uint32_t*>(r + (is_v ? rec.codes : 0) + off * (D / 2) + at / 2) = word;
    if (at % KV4_GROUP == 0)
        *reinterpret_cast<uint32_t*>(r + 2 * rec.codes + (is_v ? rec.pairs : 0) + off * (D / 8) + at / KV4_GROUP * 4) = pair;
}

}  // namespace

cudaError_t launch_kv4_store(const Kv4StoreArgs& a, int d, cudaStream_t s) {
    const long long rows = (long long)a.N * 2 * a.Hk, per_block = AP_WARPS * 32 * VPL / d;
    const dim3 grid((unsigned)((rows + per_block - 1) / per_block)), block(AP_WARPS * 32);
    return d == 128 ? launch_k(kv4_store_kernel<128>, grid, block, 0, s, true, a) : launch_k(kv4_store_kernel<64>, grid, block, 0, s, true, a);
}

}  // namespace lfw

using namespace lfw;

extern "C" int llm_op_qk_norm_rope_kv4(const void* q, const void* k, const void* v, int64_t q_ld, int64_t k_ld,
                                       int64_t v_ld, int dtype, const void* q_norm, const void* k_norm,
                                       int norm_dtype, float eps, const float* rope_cos, const float* rope_sin,
                                       int n_pos, const int32_t* positions, const int64_t* slots, int N, int H,
                                       int Hk, int d, void* q_out, void* pool, int n_pages, int page_size,
                                       void* k_out, void* v_out, void* stream) {
    if (N == 0) return LLM_OK;
    if (!q || !k || !v || !rope_cos || !rope_sin || !positions || !slots || !q_out || !pool)
        return set_error(LLM_ERR_NULL_PTR, "NULL operand");
    if (N < 0 || H < 1 || Hk < 1 || H % Hk != 0 || n_pos < 1 || n_pages < 0 || kv4_page_log2(page_size) < 0)
        return set_error(LLM_ERR_BAD_ARG, "need N >= 0, H % Hk == 0, n_pos >= 1, page_size 16, 32, 64 or 128");
    if (d != 64 && d != 128) return set_error(LLM_ERR_UNSUPPORTED, "the 4-bit cache needs d == 64 or 128");
    if ((dtype != LLM_F32 && dtype != LLM_BF16) || (norm_dtype != LLM_F32 && norm_dtype != LLM_BF16))
        return set_error(LLM_ERR_BAD_ARG, "bad dtype");
    if (!(eps >= 0.f)) return set_error(LLM_ERR_BAD_ARG, "eps must not be negative");
    const int unit = dtype == LLM_F32 ? 4 : 8;  // elements of 16 bytes
    if (q_ld % unit || k_ld % unit || v_ld % unit)
        return set_error(LLM_ERR_BAD_ARG, "token strides must be multiples of 16 bytes");
    if (N > 1 && (q_ld < (int64_t)H * d || k_ld < (int64_t)Hk * d || v_ld < (int64_t)Hk * d))
        return set_error(LLM_ERR_BAD_ARG, "a token stride is smaller than the token's heads");
    uintptr_t all = 0;
    for (const void* p : {q, k, v, q_norm, k_norm, (const void*)rope_cos, (const void*)rope_sin, (const void*)q_out,
                          (const void*)pool, (const void*)k_out, (const void*)v_out})
        all |= reinterpret_cast<uintptr_t>(p);
    if (all & 15) return set_error(LLM_ERR_BAD_ARG, "operands must be 16-byte aligned");
    if ((long long)H * d > (1 << 20) || N > (1 << 30)) return set_error(LLM_ERR_UNSUPPORTED, "more heads or token rows than one call takes");
    const size_t esz = dtype == LLM_F32 ? 4 : 2, wsz = norm_dtype == LLM_F32 ? 4 : 2, hd = (size_t)H * d, kd = (size_t)Hk * d;
    const Bytes in[] = {{q_norm, d * wsz}, {k_norm, d * wsz}, {rope_cos, (size_t)n_pos * d * 2}, {rope_sin, (size_t)n_pos * d * 2},
                        {positions, (size_t)N * 4}, {slots, (size_t)N * 8}};
    const Bytes out[] = {{pool, n_pages * llm_kv4_page_bytes(Hk, d, page_size)}, {q_out, N * hd * 2}, {k_out, N * kd * 2},
                         {v_out, N * kd * 2}};
    // the rows of q, k and v: a lane reads 16 bytes of a row and writes the same ones of an output that is the row
    const struct {
        const void *rows, *own;
        int64_t ld;
        size_t n;
    } src[] = {{q, q_out, q_ld, hd}, {k, k_out, k_ld, kd}, {v, v_out, v_ld, kd}};
    bool bad = any_overlap(in, out);
    for (const auto& x : src) {
        const bool in_place = x.own == x.rows && dtype == LLM_BF16 && (N == 1 || x.ld == (int64_t)x.n);
        for (const auto& o : out) bad = bad || (!(in_place && o.p == x.own) && overlap_rows(x.rows, x.n * esz, x.ld * (int64_t)esz, N, o));
    }
    if (bad) return set_error(LLM_ERR_BAD_ARG, "an output overlaps an input or another output");
    AppendArgs a{q, k, v, q_ld, k_ld, v_ld, q_norm, k_norm, eps, rope_cos, rope_sin, n_pos, positions, slots, N, H, Hk,
                 reinterpret_cast<__nv_bfloat16*>(q_out), reinterpret_cast<__nv_bfloat16*>(k_out),
                 reinterpret_cast<__nv_bfloat16*>(v_out), reinterpret_cast<uint8_t*>(pool),
                 (long long)n_pages * page_size, (long long)Hk * kv4_rec(page_size, d).bytes, kv4_page_log2(page_size)};
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (dtype == LLM_F32)
        e = norm_dtype == LLM_F32 ? launch_append<float, float>(a, d, s) : launch_append<float, __nv_bfloat16>(a, d, s);
    else
        e = norm_dtype == LLM_F32 ? launch_append<__nv_bfloat16, float>(a, d, s)
                                  : launch_append<__nv_bfloat16, __nv_bfloat16>(a, d, s);
    return e == cudaSuccess ? LLM_OK : set_error(LLM_ERR_CUDA, cudaGetErrorString(e));
}
