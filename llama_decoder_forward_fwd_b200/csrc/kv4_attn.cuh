// What the two kernels of attention over the 4-bit cache share: the streaming kernel
// (kv4_attn.cu: few query rows per sequence) and the prompts' (kv4_prefill.cu).
#pragma once
#include "kernels.cuh"
#include "kv4.cuh"

namespace lfw {

// A block of 128 query rows of one sequence (256 with expanded prompts), for every KV head.
struct Kv4Block {
    int q0, n, len, row0;   // first token row, new tokens and keys of the sequence; the block's first row
    int b, nkt, start;       // sequence; 128-key tiles that some row sees; the blocks' costs before it
    int image;               // first of its sequence's expanded tiles, or -1
};
// A row block and KV head whose tiles are shared by `parts` CTAs (of the first of them).
struct Kv4Split {
    int parts, q0, n, row0, kvh, pad[3];
};

// A sequence whose keys and values are expanded before: its tiles' images lie [KV head][tile] from `image` on.
struct Kv4Expanded {
    int b, len, image, tiles;
};

struct Kv4AttnArgs {
    const __nv_bfloat16* q;
    const uint8_t* pool;
    const int32_t *table, *lens, *q_start;
    __nv_bfloat16* out;
    int B, N, n_pages, lp, max_blocks, H, Hk, G;
    uint32_t g_mul;  // r / G = mulhi(r, g_mul), see div_g
    float scale_log2;
    float* part;   // [CTA][head, tail][R][d]
    float* part_ml;  // [CTA][head, tail][R][2]
    float* warp_part;  // [CTA][warp]: a warp's result for an item that began before its share, [R][d] then [R][2]
    int4* desc;    // [CTA][2]: the split item that begins in it: parts, sequence's first token, rows, first row; KV head
    // sequences of more than `few` rows per KV head are the prompts' kernel's, unless it marks them
    int few;
    int* odd;          // [B]: nonzero for a sequence that is the streaming kernel's all the same, since it has a pair
                       // that is not finite (KV4_REST between the turns: it had no room); null without that kernel
    Kv4Block* blocks;  // the prompts' row blocks
    int* counts;       // of CTAs with a share, of expanded sequences
    int4* starts;      // [CTAs + 1]: block, KV head and tile that a share begins with
    Kv4Split* splits;  // [CTA]
    int blocks_cap, expanded_cap, images_cap;
    // Where the prompts may ask for more tiles than there is room for, their kernels run twice: 1, for those that
    // have room, then 2, for the others, row block by row block. 0: all have room, or none.
    int turn;
    Kv4Expanded* expanded;
    uint8_t* images;    // [tile][K, V], each as the tensor cores read it
    uint64_t* holes;    // [tile]: which 16-key parts have no page, a byte each
    float* p_part;     // [CTA][began before, goes on after][d/4][rows of a block][4]
    float* p_ml;       // [CTA][began before, goes on after][rows of a block][2]
    uint32_t* err;
};

constexpr int KV4_REST = 2;

// 2^x by the special-function unit, subnormals flushed: a few ulp, far below the bf16 rounding that weights get; 2^-inf = 0.
DEVI float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// r / G for 0 <= r < 2^31: g_mul is ceil(2^32 / G), exact while r * (g_mul G - 2^32) < 2^32,
// that is for r < 2^32 / G, and rows of a call are fewer (the entry point checks).
DEVI int div_g(const Kv4AttnArgs& a, int r) { return a.G == 1 ? r : (int)__umulhi((uint32_t)r, a.g_mul); }

// Units of work lie on one line. Where many rows meet many keys there are more of them than 32 bits count; the
// kernel that counts in 64 is for those calls alone (one sequence of 2100 keys: 10.4 us with it, 10.1 without). A
// CTA's share fits an int, and within it units are counted from its first one. Units of a call, at most:
__host__ __device__ constexpr long long kv4_most_units(int ctas) { return (long long)ctas << 29; }
// ceil(a / b) for 0 <= a, 1 <= b.
DEVI int div_up(int a, int b) { return (int)(((unsigned)a + b - 1) / b); }
DEVI int div_up(long long a, int b) { return (int)((a + b - 1) / b); }

// The prompts' kernel. Blocks of a call, at most:
inline long long kv4_prefill_blocks(int B, int N, int G, int few) {
    const long long rows = (long long)N * G, seqs = rows / (few + 1);
    return rows / 128 + (seqs < B ? seqs : B) + 1;
}
// Where some sequence has many row blocks, the prompts are expanded before, once. Sequences and tiles of
// that, at most (the tiles by the tables' width, the lengths being on the device).
inline int kv4_expanded_seqs(int B, int N, int G, int few) {
    const long long n = (long long)N * G / (few + 1);
    return (int)(n < B ? n : B);
}
inline long long kv4_images(int B, int N, int G, int Hk, long long max_keys, int few) {
    return (long long)kv4_expanded_seqs(B, N, G, few) * ((max_keys + 127) / 128) * Hk;
}
cudaError_t launch_kv4_prefill(const Kv4AttnArgs& a, int d, cudaStream_t s);

}  // namespace lfw
