// The 4-bit paged KV cache: its format, and what its operators share.
//
// A pool of pages; a page holds P tokens (16, 32, 64 or 128) of every KV head. The
// record of one KV head in one page is contiguous:
//   K codes [P][d/2] | V codes [P][d/2] | K pairs [P][d/32] | V pairs [P][d/32]
// codes: value 2i of a token's head in the low half of byte i; pairs: (scale, zero) of
// 32 consecutive values, two bf16. A code c stands for bf16(scale c + zero), rounded
// once; the scale is bf16((max - min) / 15) and the zero bf16(min) of the 32 values.
// 1.25 d bytes per token and head against 4 d in bf16. Groups of 32 and not of the
// whole head: the pairs cost a quarter of the codes' bytes, and the step between codes
// follows the local range (0.28 of a normal group's deviation instead of 0.36).
// The decode kernels read a 16-token block of a record as four contiguous pieces.
#pragma once
#include "common.cuh"

namespace lfw {

constexpr int KV4_GROUP = 32;

// Sizes in bytes of one KV head's record of a page of P tokens.
struct Kv4Rec {
    int codes, pairs;  // of K (or V)
    int bytes;         // the whole record
};
__host__ __device__ constexpr Kv4Rec kv4_rec(int P, int d) {
    return Kv4Rec{P * d / 2, P * d / 8, P * (d + d / 4)};
}
// log2 of a page size, or -1 when it is not one that the cache has.
__host__ __device__ constexpr int kv4_page_log2(int P) {
    return P == 16 ? 4 : P == 32 ? 5 : P == 64 ? 6 : P == 128 ? 7 : -1;
}

// Codes to values. The bits of a code alone are a subnormal bf16, c * 2^-133 exactly, so one
// fused multiply-add with a scale that is 2^133 too large gives the value, rounded once
// as its definition says, and no conversion comes first. A code in the upper half of the low
// byte needs no shift either: bf16's subnormals and its first normal exponent are one linear
// range of 256 steps, so its bits are 16 c * 2^-133. 2^133 is out of bf16's range: what comes
// out is the value * 2^-72 (scale * 2^61, or * 2^57 for the upper half, zero * 2^-72), the same
// rounding, and the products' results are scaled back in fp32. That holds for scales below
// 2^67 (a group of a larger one reads as NaN) and, to the last bit, for values above 2^-54 (smaller ones
// are off by up to 2^-62).
constexpr float KV4_BACK = 4722366482869645213696.f;  // 2^72
DEVI uint32_t kv4_mul(uint32_t a, uint32_t b) {
    const __nv_bfloat162 v = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&v);
}
// A (scale, zero) pair times (2^61, 2^-72), as kv4_expand takes its parts; and a pair of such scales / 16.
DEVI uint32_t kv4_pair(uint32_t sz) { return kv4_mul(sz, 0x1B805E00u); }
// Whether a pair from kv4_pair holds an infinity or a NaN (a scale of 2^67 or more has become infinite).
DEVI bool kv4_odd(uint32_t sz) { return (sz & 0x7F80u) == 0x7F80u || (sz & 0x7F800000u) == 0x7F800000u; }
DEVI uint32_t kv4_16th(uint32_t s2) { return kv4_mul(s2, 0x3D803D80u); }
// The eight codes of a word as four bf16 pairs, (value i, value i + 4) for i = 0..3, * 2^-72.
DEVI void kv4_expand(uint32_t w, uint32_t s2, uint32_t s2_16th, uint32_t z2, uint32_t (&r)[4]) {
    const __nv_bfloat162 z = *reinterpret_cast<__nv_bfloat162*>(&z2);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t c = (w >> (i / 2 * 8)) & (i & 1 ? 0x00F000F0u : 0x000F000Fu), s = i & 1 ? s2_16th : s2;
        const __nv_bfloat162 v = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&c), *reinterpret_cast<const __nv_bfloat162*>(&s), z);
        r[i] = *reinterpret_cast<const uint32_t*>(&v);
    }
}

// A maximum that a NaN does not drop out of.
DEVI float max_nan(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}

// ---- the entry points' checks ----
struct Bytes {
    const void* p;
    size_t n;  // 0: nothing
};
inline bool overlap(const Bytes& a, const Bytes& b) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return a.p && b.p && a.n && b.n && x < y + b.n && y < x + a.n;
}
// Whether b overlaps one of n rows of `row` bytes, `apart` bytes (row or more) from one to the next.
inline bool overlap_rows(const void* rows, size_t row, long long apart, int n, const Bytes& b) {
    if (n < 1 || !b.p || !b.n) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(rows), y = reinterpret_cast<uintptr_t>(b.p);
    const unsigned long long i = y < x + row ? 0 : n == 1 ? 1 : (y - x - row) / apart + 1;  // the first row that ends behind b's begin
    return i < (unsigned long long)n && x + i * apart < y + b.n;
}
// Whether one of the outputs overlaps an input or another output.
template <int I, int O> bool any_overlap(const Bytes (&in)[I], const Bytes (&out)[O]) {
    for (int o = 0; o < O; ++o) {
        for (int i = 0; i < I; ++i)
            if (overlap(in[i], out[o])) return true;
        for (int i = 0; i < o; ++i)
            if (overlap(out[i], out[o])) return true;
    }
    return false;
}

// ---- what the model's own path uses ----
// llm_op_kv_pages; n_new null: n_each new tokens for every sequence; held > 0: the pages taken already are
// those of the first `held` lengths, whatever became of earlier plans (used_in and used_out null).
cudaError_t launch_kv_pages(const int32_t* lens, const int32_t* n_new, int n_each, int held, int B, int page_size,
                            const int32_t* free_pages, int n_free, const int32_t* used_in, int32_t* table, int max_blocks,
                            int32_t* q_start, int32_t* positions, int64_t* slots, int N, int32_t* new_lens,
                            int32_t* used_out, cudaStream_t s);
// Quantise one layer's new keys (rotated) and values from the contiguous bf16 staging cache
// [B][Hk][S_max][d], row n of B * T being position positions[n] of sequence n / T, into the slots.
struct Kv4StoreArgs {
    const __nv_bfloat16 *k, *v;
    const int32_t* positions;
    const int64_t* slots;
    int N, T, Hk, S_max;
    uint8_t* pool;
    long long n_slots, page_bytes;
    int lp;
};
cudaError_t launch_kv4_store(const Kv4StoreArgs& a, int d, cudaStream_t s);
// LLM_OK, or why a call of these sizes is more than llm_op_attention_kv4 takes.
int kv4_check_size(int B, int N, int H, int Hk, int max_blocks, int page_size);
// Workspace with room for all the expanded tiles that a call of these sizes, or a smaller one, may use.
size_t attention_kv4_most_workspace(int B, int N, int max_new, int H, int Hk, int d, int max_blocks, int page_size);
// llm_op_attention_kv4 with the error word of the caller's model.
int attention_kv4(const void* q, const void* pool, int n_pages, int page_size, const int32_t* table, int max_blocks,
                  const int32_t* lens, const int32_t* q_start, int B, int N, int max_new, int H, int Hk, int d, void* out,
                  void* workspace, size_t workspace_bytes, uint32_t* err, cudaStream_t s);

}  // namespace lfw
