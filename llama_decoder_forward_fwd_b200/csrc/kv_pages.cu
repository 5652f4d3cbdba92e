// Block tables and slot maps of a paged KV cache, built on the GPU from request lengths.
//
// A sequence of len tokens holds ceil(len / P) pages. n new tokens need the blocks
// ceil(len / P) .. ceil((len + n) / P) - 1 of its table; they take the next ids of the
// free list, sequence by sequence. Token r of sequence b is row q_start[b] + r of the
// step's token rows (q_start: the running sum of n), at position len + r, in the slot
// page * P + position % P.
//
// The work is a scan over the sequences and 12 bytes per token row: latency, not
// bandwidth (16 sequences: 0.5 KB). So there is one launch and no exchange between
// CTAs: each CTA scans all sequences itself, 256 at a time (two warp scans and one
// barrier a chunk), and writes its share of the chunk's token rows, finding a row's
// sequence by bisection in shared memory. The token that opens a page writes the table
// entry, so every entry has one writer, and nothing that the kernel reads is written by
// it: entries below ceil(len / P) are only read, the others only written. Measured: 16
// sequences 2.6 us, 512 sequences with 33k token rows 4.5 us, launch included.
#include "../../include/llama_fwd.h"
#include "kernels.cuh"
#include "kv4.cuh"

namespace lfw {
namespace {

constexpr int PG_THREADS = 256;

struct PagesArgs {
    const int32_t *lens, *n_new, *free_pages, *used_in;
    int32_t *table, *q_start, *positions, *new_lens, *used_out;
    int64_t* slots;
    int B, lp, n_free, max_blocks, N;
    int n_each;  // new tokens of every sequence when n_new is null
    int held;    // sequences of lens, B or more, whose pages are the ones taken already; used_in is null then
};

DEVI int sat32(long long v) { return v > 0x7fffffffLL ? 0x7fffffff : (int)v; }

// Inclusive scan over the CTA of two counts at once.
DEVI void scan2(long long& a, long long& b, long long (&part)[2][PG_THREADS / 32], int tid) {
    const int lane = tid & 31, warp = tid >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long ua = __shfl_up_sync(0xffffffffu, a, o), ub = __shfl_up_sync(0xffffffffu, b, o);
        if (lane >= o) {
            a += ua;
            b += ub;
        }
    }
    if (lane == 31) {
        part[0][warp] = a;
        part[1][warp] = b;
    }
    __syncthreads();
    for (int w = 0; w < warp; ++w) {
        a += part[0][w];
        b += part[1][w];
    }
}

__global__ void __launch_bounds__(PG_THREADS) kv_pages_kernel(const PagesArgs a) {
    __shared__ long long part[2][2][PG_THREADS / 32];  // two buffers: one barrier a chunk is enough for them
    __shared__ long long row0[2][PG_THREADS];          // first token row of a sequence
    __shared__ long long page0[2][PG_THREADS];         // its first new page's place in the free list
    __shared__ int len_s[2][PG_THREADS];
    const int tid = threadIdx.x, P = 1 << a.lp;
    pdl_wait();
    pdl_trigger();
    long long rows = 0, pages = a.used_in ? (long long)*a.used_in : 0;
    for (int i = 0; i < a.held; ++i) pages += ((long long)max(a.lens[i], 0) + P - 1) >> a.lp;
    for (int c = 0, it = 0; c < a.B; c += PG_THREADS, ++it) {
        const int buf = it & 1, b = c + tid;
        long long len = 0, n = 0;
        if (b < a.B) {
            len = max(a.lens[b], 0);
            n = max(a.n_new ? a.n_new[b] : a.n_each, 0);
        }
        const long long take = ((len + n + P - 1) >> a.lp) - ((len + P - 1) >> a.lp);
        long long in = n, ip = take;
        scan2(in, ip, part[buf], tid);
        row0[buf][tid] = rows + in - n;
        page0[buf][tid] = pages + ip - take;
        len_s[buf][tid] = (int)len;
        __syncthreads();
        long long chunk_rows = 0, chunk_pages = 0;
#pragma unroll
        for (int w = 0; w < PG_THREADS / 32; ++w) {
            chunk_rows += part[buf][0][w];
            chunk_pages += part[buf][1][w];
        }
        if (b < a.B && it % gridDim.x == blockIdx.x) {
            a.q_start[b] = sat32(row0[buf][tid]);
            a.new_lens[b] = sat32(len + n);
        }
        const long long end = min(rows + chunk_rows, (long long)a.N);
        const int live = min(PG_THREADS, a.B - c);
        for (long long i = rows + (long long)blockIdx.x * PG_THREADS + tid; i < end; i += (long long)gridDim.x * PG_THREADS) {
            int lo = 0, hi = live - 1;  // the last sequence that starts at or before row i
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (row0[buf][mid] <= i) lo = mid;
                else hi = mid - 1;
            }
            const long long l = len_s[buf][lo], pos = l + (i - row0[buf][lo]);
            const long long blk = pos >> a.lp, held = (l + P - 1) >> a.lp;
            int page = -1;
            if (blk < a.max_blocks) {
                int32_t* entry = a.table + (long long)(c + lo) * a.max_blocks + blk;
                if (blk < held) {
                    page = *entry;
                } else {
                    const long long k = page0[buf][lo] + (blk - held);
                    if (k >= 0 && k < a.n_free) page = a.free_pages[k];
                    if ((pos & (P - 1)) == 0) *entry = page;
                }
            }
            a.positions[i] = sat32(pos);
            a.slots[i] = page < 0 ? -1 : (long long)page * P + (pos & (P - 1));
        }
        rows += chunk_rows;
        pages += chunk_pages;
    }
    // padding rows behind the last sequence's
    for (long long i = rows + (long long)blockIdx.x * PG_THREADS + tid; i < a.N; i += (long long)gridDim.x * PG_THREADS) {
        a.positions[i] = -1;
        a.slots[i] = -1;
    }
    if (blockIdx.x == 0 && tid == 0) {
        a.q_start[a.B] = sat32(rows);
        if (a.used_out) *a.used_out = sat32(pages);
    }
}

}  // namespace
}  // namespace lfw

using namespace lfw;

extern "C" size_t llm_kv4_page_bytes(int Hk, int d, int page_size) {
    if (Hk < 1 || (d != 64 && d != 128) || kv4_page_log2(page_size) < 0) return 0;
    return (size_t)Hk * kv4_rec(page_size, d).bytes;
}

extern "C" int llm_op_kv_pages(const int32_t* lens, const int32_t* n_new, int B, int page_size,
                               const int32_t* free_pages, int n_free, const int32_t* used_in, int32_t* table,
                               int max_blocks, int32_t* q_start, int32_t* positions, int64_t* slots, int N,
                               int32_t* new_lens, int32_t* used_out, void* stream) {
    if (!lens || !n_new || !free_pages || !table || !q_start || !positions || !slots || !new_lens || !used_out)
        return set_error(LLM_ERR_NULL_PTR, "NULL operand");
    if (B < 1 || N < 0 || n_free < 0 || max_blocks < 1 || kv4_page_log2(page_size) < 0)
        return set_error(LLM_ERR_BAD_ARG, "need B >= 1, N >= 0, n_free >= 0, max_blocks >= 1, page_size 16, 32, 64 or 128");
    // every CTA reads the inputs while others already write
    const size_t nb = (size_t)B * 4;
    const Bytes in[] = {{lens, nb}, {n_new, nb}, {free_pages, (size_t)n_free * 4}, {used_in, 4}};
    const Bytes out[] = {{table, nb * max_blocks}, {q_start, nb + 4}, {positions, (size_t)N * 4},
                         {slots, (size_t)N * 8},   {new_lens, nb},    {used_out, 4}};
    if (any_overlap(in, out))
        return set_error(LLM_ERR_BAD_ARG, "an output overlaps an input (lens, n_new, free_pages, used_in) or another output");
    const cudaError_t e = lfw::launch_kv_pages(lens, n_new, 0, 0, B, page_size, free_pages, n_free, used_in, table, max_blocks, q_start,
                                               positions, slots, N, new_lens, used_out, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? LLM_OK : set_error(LLM_ERR_CUDA, cudaGetErrorString(e));
}

cudaError_t lfw::launch_kv_pages(const int32_t* lens, const int32_t* n_new, int n_each, int held, int B, int page_size,
                                 const int32_t* free_pages, int n_free, const int32_t* used_in, int32_t* table,
                                 int max_blocks, int32_t* q_start, int32_t* positions, int64_t* slots, int N,
                                 int32_t* new_lens, int32_t* used_out, cudaStream_t s) {
    PagesArgs a{lens, n_new, free_pages, used_in, table, q_start, positions, new_lens, used_out, slots, B,
                kv4_page_log2(page_size), n_free, max_blocks, N, n_each, held};
    // one CTA per 256 token rows, at most one per SM: a CTA more repeats the scan
    const int sms = current_num_sms();
    int grid = (N + PG_THREADS - 1) / PG_THREADS;
    grid = grid < 1 ? 1 : grid > sms ? sms : grid;
    return launch_k(kv_pages_kernel, dim3(grid), dim3(PG_THREADS), 0, s, true, a);
}
