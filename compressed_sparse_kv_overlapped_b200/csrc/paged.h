// paged.h -- the paged key/value operators (csa_kv_append, csa_window_attn, csa_prefix_attn): launch
// interface between their C entry points (paged.cu) and kernels, and the device code both attention
// kernels share: which keys a block of queries sees, and where they lie.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <cuda.h>

#include "common.cuh"

namespace csa {

struct PagedAppendParams {
    csa_kv_cache kv;
    int64_t rows, max_n;
    const uint16_t* k;
    const uint16_t* v;
    const uint16_t* q;  // nullable
    uint16_t* q_out;
    int64_t k_stride, v_stride, q_stride, q_out_stride;
    const float* inv_freq;
    int rot, interleaved;
    int* status;
};
cudaError_t launch_paged_append(const PagedAppendParams& p, cudaStream_t stream);

// Partial results: o [slots][rows][H][d] (normalized, fp32), lse [slots][rows][H] (base 2; -inf: an empty
// partial, its o is not written).  The row of token i of sequence b is that of the token arrays, or
// b * per_seq + i where only sequences with up to per_seq tokens have partials.
struct PagedPartials {
    float* o;
    float* lse;
    int64_t rows;
    int per_seq;
    int slots;
};

// One launch of an attention kernel over keys [key_begin, key_end of the mode) of every query.
struct PagedAttnParams {
    csa_kv_cache kv;
    int64_t rows;
    int max_n;
    // the rows of a block of queries: 0 = one sequence's new tokens, each seeing its window and first
    // tokens from key_begin on; 1 = all rows of the token arrays, each seeing the prefix
    // [0, prefix_len) through row 0 of the table
    int prefix_mode;
    int prefix_len;     // sequences need len - n >= prefix_len (0: no prefix)
    int key_begin;      // first key (the suffix of csa_prefix_attn: prefix_len)
    int W, S;           // window (2^31 - 1: none) and first tokens
    float scale_log2;   // scale * log2(e)
    const uint16_t* q;
    uint16_t* out;
    float* lse;         // nullable
    int64_t q_stride, out_stride;
    // sequences with n G <= few_rows query rows per key head belong to the stream kernel, the others to
    // the tile kernel (without prefix_mode)
    int64_t few_rows;
    // splits of the keys of a block: split s writes slot s of the partials, or without any (part.o =
    // nullptr, one split) out / lse
    int splits;
    PagedPartials part;
    int* status;
    uint64_t wait_ns;
    int debug_fault;    // 1 (tests of the bounded waits): the first wait for keys counts as run out
};

// Few query rows per key (decode): mma.sync tiles of 16 or 32 rows, each warp streaming its own keys.
// One launch takes up to two parts, the rows of all sequences on the prefix and each sequence's own keys;
// these fields stand in the place of PagedAttnParams'.
struct PagedStreamPart {
    int prefix_mode, key_begin;
    int splits;
    int split_groups;   // 16-key groups of a split (split s: [s, s + 1) times these, as far as there are)
    int row_tiles;      // (filled in by the launch)
    PagedPartials part;
};
struct PagedStreamParts {
    PagedStreamPart part[2];
    int n;
    unsigned blocks0;   // blocks of part 0 (filled in by the launch)
};
cudaError_t launch_paged_stream(const PagedAttnParams& p, PagedStreamParts parts, cudaStream_t stream);
// Many query rows per key: tcgen05 tiles of 128 rows.  pdl: it may start before the launch in front of it,
// one of the same call, ends (it ends after it).
cudaError_t launch_paged_tile(const PagedAttnParams& p, cudaStream_t stream, bool pdl);
// Tensor maps of the pools: boxes of 16 slots x 64 channels of one head and page, 128-byte swizzle.
cudaError_t paged_kv_maps(const csa_kv_cache& kv, CUtensorMap* k, CUtensorMap* v);
// Merge of the partials of each (row, head) into out / lse: those of the prefix, and those of a sequence with
// few rows or of another.  A sequence without any was written directly and is left alone.
struct PagedMerge {
    PagedPartials prefix, few, many;
};
cudaError_t launch_paged_combine(const PagedAttnParams& p, const PagedMerge& m, cudaStream_t stream, bool pdl);

// ---------------------------------------------------------------------------------------------

// Sequence b of the table, checked; false: it is skipped (and reported by the thread with `say`).
__device__ __forceinline__ bool paged_seq(const csa_kv_cache& kv, int b, int64_t rows, int64_t max_n, int prefix_len,
                                          int* status, bool say, csa_kv_seq* out) {
    const csa_kv_seq s = kv.seqs[b];
    *out = s;
    if (s.n == 0) return false;
    const bool ok = s.n > 0 && s.n <= max_n && s.len >= s.n && s.len <= kv.max_pages * kv.page_size &&
                    s.row >= 0 && s.n <= rows && s.row <= rows - s.n && s.len - s.n >= prefix_len;
    if (!ok && say) report(status, CSA_ERR_INDEX);
    return ok;
}

// The keys that a block of queries with positions [p0, p0 + cnt) sees, as two runs of tokens: the first
// tokens [0, s1) and the window part [lo, hi), s1 <= lo.  Every query of the block sees all of the
// first run; the second needs a mask per query.
struct KeySpan {
    int s1, lo, hi;
};
__device__ __forceinline__ KeySpan key_span(const PagedAttnParams& p, int64_t p0, int64_t cnt) {
    KeySpan k;
    if (p.prefix_mode) {
        k.s1 = k.lo = 0;
        k.hi = p.prefix_len;
        return k;
    }
    const int64_t lo = p0 - (int64_t)p.W + 1;
    k.lo = (int)(lo > p.key_begin ? lo : p.key_begin);
    k.hi = (int)(p0 + cnt);
    k.s1 = p.S < k.lo ? p.S : k.lo;
    if (k.s1 < p.key_begin) k.s1 = 0;  // (key_begin > 0 only without first tokens)
    return k;
}

// Bits [from, to) of a 16-key group that starts at token t0: the tokens of [a, b) in it.
__device__ __forceinline__ uint32_t span16(int t0, int a, int b) {
    int f = a - t0, e = b - t0;
    f = f < 0 ? 0 : (f > 16 ? 16 : f);
    e = e < 0 ? 0 : (e > 16 ? 16 : e);
    return ((1u << e) - 1u) & ~((1u << f) - 1u);
}

// log2 of the page size (a power of two).
__device__ __forceinline__ int page_shift(const csa_kv_cache& kv) { return 31 - __clz(kv.page_size); }

// The page of token t through `table`, or -1 (reported) when its number is out of range.
__device__ __forceinline__ int page_of(const csa_kv_cache& kv, const int32_t* table, int shift, int t, int* status) {
    const int pg = __ldg(table + (t >> shift));
    if (pg < 0 || pg >= kv.num_pages) {
        report(status, CSA_ERR_INDEX);
        return -1;
    }
    return pg;
}

}  // namespace csa
