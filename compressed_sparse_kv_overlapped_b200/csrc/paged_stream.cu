// paged_stream.cu -- attention of few query rows over a paged cache (decode steps, proposed tokens),
// and the merge of partial results.
//
// With G = H / H_kv query heads per key head a decode step does 4 G d operations per 4 d bytes of key
// and value, so the kernel is a read of the cache: what matters is bytes in flight and how few
// instructions a key costs on the way.  A block takes one (sequence, 16 or 32 query rows, key head) and
// a share of its keys; rows are (token, head of the group) pairs.  Its four warps are independent streams:
// warp w takes the 16-key groups w, w + 4, ... of the block's share through a ring of its own (one lane
// issues a TMA box per 64 channels of K and of V, kStages groups ahead, no barrier among warps) and
// keeps its own running maximum, sum and output, in the online softmax form
//     m' = max(m, max_t x_t),  l' = l 2^(m - m') + sum_t 2^(x_t - m'),  o' = o 2^(m - m') + sum_t 2^(x_t - m') V_t
// with x in base-2 units.  The four results meet once, in shared memory at the end.  Two blocks share an
// SM, so that one's start and end overlap the other's stream; the key heads of the same tokens are
// neighbours in the grid, since their rows are neighbours in memory.
//
// A 16-key group never crosses a page (pages are multiples of 16 and groups are aligned to 16 tokens),
// so it costs one page lookup, made one group ahead of its copy.  A group that straddles the end of a
// visible run is copied whole; its dead rows of V are zeroed before use (a freed page or an unwritten
// slot may hold anything, and a weight of zero does not remove a NaN), its dead scores replaced.  A page
// number out of range becomes a coordinate past the last page, which the copy fills with zeros.  The
// two products run on mma.sync m16n8k16: the tensor pipe is far from a limit here (32 of them per
// 8 KiB at d = 128, 19 % busy) and tcgen05 would want 128 rows.
//
// Measured (d = 128, 8 key heads): five sequences with a window of 65,536, 1.24 GB in 206 us = 6.0 TB/s
// (0.92 of the copy rate) and 221 us with the merge; 32 sequences with a window of 4,096, 538 MB in 92 us
// = 5.8 TB/s; one short row 8.2 us a call, a chain of latencies (tables, copy, merge of the warps).
// Copies by cp.async from eight warps of one block an SM took 324, 115 and 6.2 us: some 700 instructions a
// group, most of them addresses, but a shorter start.
#include "paged.h"
#include "tma.h"

namespace csa {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kCombineThreads = 256;
// What the weights are multiplied by for the product with V: fp16 has no normal numbers below 2^-14, and a row's
// weights reach 1 at most.  With 2^15 one of 2^-29 of the largest is still normal and only those under 2^-40 are
// lost; unscaled, 131,072 keys of 2^-25.2 behind one strong first token lose all of their 0.3 %.  bf16 has the
// range of fp32.  A power of two: O is that much larger, without a further rounding, until it is divided by the sum.
template <bool F16>
constexpr float kWeightScale = F16 ? 32768.f : 1.f;

struct StreamMaps {
    CUtensorMap k, v;
};

template <int D, int MT>
struct StreamCfg {
    static constexpr int kRows = 16 * MT;
    static constexpr int kHalves = D / 64;         // boxes of 16 rows x 64 channels (2 KB, 128-byte swizzle)
    static constexpr int kGroup = 16 * D * 2;      // bytes of one group's keys (or values)
    static constexpr int kStages = D == 128 ? 3 : 5;
    static constexpr int kWarpBytes = kStages * 2 * kGroup;
    static constexpr int kOStride = D + 4;         // floats; the padding spreads the rows over the banks
    static constexpr int kOBytes = kRows * kOStride * 4;  // a warp's result, in its own ring
    static_assert(kOBytes <= kWarpBytes, "the result fits the ring");
    static constexpr int kML = kWarps * kWarpBytes;  // float2 [kWarps][kRows]: maximum and sum
    static constexpr int kBars = kML + kWarps * kRows * 8;
    static constexpr int kTotal = kBars + kWarps * kStages * 8;
    static_assert(2 * (kTotal + 1024) <= 227 * 1024, "two blocks on an SM");
};

__device__ __forceinline__ void ldmatrix4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldmatrix4t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
template <bool F16>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if (F16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <bool F16>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
    if (F16) {
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    return pack_bf16x2(lo, hi);
}

// grid: for each part, x = ((b * row_tiles + row tile) * splits + split) * H_kv + key head
template <int D, int MT, bool F16>
__global__ void __launch_bounds__(kThreads)
    paged_stream_kernel(const __grid_constant__ StreamMaps maps, const __grid_constant__ PagedAttnParams params,
                        const __grid_constant__ PagedStreamParts parts) {
    using C = StreamCfg<D, MT>;
    extern __shared__ __align__(1024) unsigned char smem[];
    grid_dep_launch();
    unsigned u = blockIdx.x;
    const bool second = u >= parts.blocks0;
    if (second) u -= parts.blocks0;
    const PagedStreamPart& part = parts.part[second ? 1 : 0];
    PagedAttnParams p = params;
    p.prefix_mode = part.prefix_mode;
    p.key_begin = part.key_begin;
    p.splits = part.splits;
    p.part = part.part;
    const int row_tiles = part.row_tiles, split_groups = part.split_groups;
    const csa_kv_cache& kv = params.kv;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {  // (fetched while the tables are read)
        tma_prefetch_map(&maps.k);
        tma_prefetch_map(&maps.v);
    }
    if (smem_u32(smem) & 1023u) {  // (the swizzled boxes need it; the launch gives it)
        if (threadIdx.x == 0) report(p.status, CSA_ERR_CUDA);
        return;
    }
    const int hk = (int)(u % (unsigned)kv.H_kv);
    u /= (unsigned)kv.H_kv;
    const int split = (int)(u % (unsigned)p.splits);
    u /= (unsigned)p.splits;
    const int rt = (int)(u % (unsigned)row_tiles), b = (int)(u / (unsigned)row_tiles);
    const int G = kv.H / kv.H_kv;

    // the block's rows r in [0, R): new token (r0 + r) / G of the sequence, head (r0 + r) % G of the group
    csa_kv_seq seq;
    const int64_t r0 = (int64_t)rt * C::kRows;
    int64_t pos0;  // position of the sequence's new token 0
    if (p.prefix_mode) {
        seq.row = 0;
        seq.n = p.rows;
        pos0 = p.prefix_len;
    } else {
        if (!paged_seq(kv, b, p.rows, p.max_n, p.prefix_len, p.status,
                       threadIdx.x == 0 && rt == 0 && hk == 0 && split == 0, &seq))
            return;
        if (seq.n * G > p.few_rows) return;
        pos0 = seq.len - seq.n;
    }
    const int64_t left = seq.n * G - r0;
    if (left <= 0) return;
    const int R = (int)(left < C::kRows ? left : C::kRows);
    const int64_t tok0 = r0 / G, tok1 = (r0 + R - 1) / G;
    const KeySpan span = key_span(p, pos0 + tok0, tok1 - tok0 + 1);
    const int p_first = (int)(pos0 + tok0), p_last = (int)(pos0 + tok1);
    const int32_t* table = kv.page_table + (p.prefix_mode ? 0 : (int64_t)b * kv.max_pages);

    // 16-key groups: those of the first tokens, then those of the window from lo rounded down
    const int n_first = (span.s1 + 15) >> 4, win0 = span.lo & ~15;
    const int n_groups = n_first + (span.hi > span.lo ? (span.hi - win0 + 15) >> 4 : 0);
    const int g_begin = split * split_groups < n_groups ? split * split_groups : n_groups;
    // (the last split takes the rest, should a sequence be longer than the host's bound)
    const int g_end = split + 1 < p.splits && g_begin + split_groups < n_groups ? g_begin + split_groups : n_groups;
    const int my = g_end - g_begin > warp ? (g_end - g_begin - warp + kWarps - 1) / kWarps : 0;
    if (g_begin == g_end && p.part.o) {  // nothing in this split: empty partials
        if ((int)threadIdx.x < R) {
            const int64_t f = r0 + threadIdx.x, tok = f / G;
            const int64_t row = (int64_t)split * p.part.rows + (p.part.per_seq ? (int64_t)b * p.part.per_seq : seq.row) + tok;
            p.part.lse[row * kv.H + hk * G + (f - tok * G)] = -INFINITY;
        }
        return;
    }

    const uint32_t ring = smem_u32(smem) + warp * C::kWarpBytes;
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kBars) + warp * C::kStages;
    if (lane == 0) {
        for (int i = 0; i < C::kStages; ++i) mbar_init(full + i, 1);
        fence_mbar_init();
    }
    __syncwarp();

    auto group_start = [&](int g, int* a, int* e) {
        const bool first = g < n_first;
        *a = first ? 0 : span.lo;
        *e = first ? span.s1 : span.hi;
        return first ? g * 16 : win0 + (g - n_first) * 16;
    };
    const int shift = page_shift(kv);
    auto lookup = [&](int i) {  // page of the warp's group i (past the last: zeros)
        if (i >= my) return -1;
        int a, e;
        const int pg = page_of(kv, table, shift, group_start(g_begin + warp + i * kWarps, &a, &e), p.status);
        return pg < 0 ? (int)kv.num_pages : pg;
    };
    auto copy = [&](int i, int page) {  // by lane 0
        if (i >= my) return;
        int a, e;
        const int slot = group_start(g_begin + warp + i * kWarps, &a, &e) & (kv.page_size - 1), st = i % C::kStages;
        const uint32_t dst = ring + st * (2 * C::kGroup), bar = smem_u32(full + st);
        mbar_arrive_expect_tx(full + st, 2 * C::kGroup);
#pragma unroll
        for (int h = 0; h < C::kHalves; ++h) {
            tma_load_4d(dst + h * 2048, &maps.k, h * 64, slot, hk, page, bar);
            tma_load_4d(dst + C::kGroup + h * 2048, &maps.v, h * 64, slot, hk, page, bar);
        }
    };

    int page_next = -1;
    if (lane == 0) {
        int pages[C::kStages];
#pragma unroll
        for (int i = 0; i < C::kStages; ++i) pages[i] = lookup(i);
#pragma unroll
        for (int i = 0; i < C::kStages; ++i) copy(i, pages[i]);
        page_next = lookup(C::kStages);
    }

    // Q as the A operand: rows lane / 4 (+ 8) of each 16-row tile
    const int ra = lane >> 2, cq = (lane & 3) * 2;
    uint32_t qf[MT][D / 16][4];
    int pr[2 * MT];  // positions of this thread's rows
#pragma unroll
    for (int i = 0; i < 2 * MT; ++i) {
        const int r = i * 8 + ra;
        const int64_t f = r0 + (r < R ? r : 0);
        const int64_t tok = f / G;
        const uint16_t* src = p.q + (seq.row + tok) * p.q_stride + (hk * G + (f - tok * G)) * D + cq;
        pr[i] = (int)(pos0 + tok);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
            qf[i >> 1][k][i & 1] = r < R ? *reinterpret_cast<const uint32_t*>(src + k * 16) : 0u;
            qf[i >> 1][k][(i & 1) + 2] = r < R ? *reinterpret_cast<const uint32_t*>(src + k * 16 + 8) : 0u;
        }
    }

    float o[MT][D / 8][4];
    float m[2 * MT], l[2 * MT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < D / 8; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[i][j][e] = 0.f;
#pragma unroll
    for (int i = 0; i < 2 * MT; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.f;
    }

    const int km = lane >> 3, kr = lane & 7;  // ldmatrix: this lane addresses row kr of matrix km
    int stage = 0;
    uint32_t phase = 0;
    int done = 0;
    const int run = p.debug_fault == 1 ? 0 : my;
    if (run < my) report(p.status, CSA_ERR_TIMEOUT);
    for (; done < run; ++done) {
        const int i = done;
        if (!__all_sync(0xffffffffu, mbar_wait(full + stage, phase, p.status, nullptr, p.wait_ns))) break;
        const uint32_t kb = ring + stage * (2 * C::kGroup), vb = kb + C::kGroup;
        int a, e;
        const bool first = g_begin + warp + i * kWarps < n_first;
        const int t0 = group_start(g_begin + warp + i * kWarps, &a, &e);
        if (t0 < a || t0 + 16 > e) {
            for (int c = lane; c < 16 * 8 * C::kHalves; c += 32) {
                const int r = (c >> 3) & 15;
                if (t0 + r < a || t0 + r >= e) st_shared_v4(vb + (c >> 7) * 2048 + r * 128 + (c & 7) * 16, make_uint4(0, 0, 0, 0));
            }
            fence_proxy_async_smem();  // (the next copy into this stage comes after these stores)
            __syncwarp();
        }
        float s[MT][2][4];
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[t][n][e] = 0.f;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
            uint32_t kf[4];
            const int key = (km >> 1) * 8 + kr;
            ldmatrix4(kb + (k >> 2) * 2048 + key * 128 + (((2 * (k & 3) + (km & 1)) ^ (key & 7)) << 4), kf);
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                mma16816<F16>(s[t][0], qf[t][k], kf[0], kf[1]);
                mma16816<F16>(s[t][1], qf[t][k], kf[2], kf[3]);
            }
        }
        const bool whole = t0 >= a && t0 + 16 <= e &&
                           (first || (t0 + 15 <= p_first && (t0 > p_last - p.W || t0 + 16 <= p.S)));
#pragma unroll
        for (int t = 0; t < MT; ++t) {
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
                float x[4] = {s[t][0][2 * hh] * p.scale_log2, s[t][0][2 * hh + 1] * p.scale_log2,
                              s[t][1][2 * hh] * p.scale_log2, s[t][1][2 * hh + 1] * p.scale_log2};
                if (!whole) {
                    const int pos = pr[2 * t + hh];
                    uint32_t see;
                    if (first) {
                        see = span16(t0, 0, span.s1);
                    } else {  // (a prefix: pos lies behind hi, so all of it)
                        const int up = pos + 1 < span.hi ? pos + 1 : span.hi;
                        const int w0 = pos - p.W + 1 > span.lo ? pos - p.W + 1 : span.lo;
                        see = span16(t0, w0, up) | span16(t0, span.lo, p.S < up ? p.S : up);
                    }
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        if (!((see >> (cq + (c & 1) + (c >> 1) * 8)) & 1u)) x[c] = -INFINITY;
                }
                float mx = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                const int ri = 2 * t + hh;
                if (__any_sync(0xffffffffu, mx > m[ri])) {
                    const float mn = fmaxf(m[ri], mx);
                    const float f = mn == -INFINITY ? 1.f : fast_exp2(m[ri] - mn);
                    m[ri] = mn;
                    l[ri] *= f;
#pragma unroll
                    for (int j = 0; j < D / 8; ++j) {
                        o[t][j][2 * hh] *= f;
                        o[t][j][2 * hh + 1] *= f;
                    }
                }
                const float mu = m[ri] == -INFINITY ? 0.f : m[ri];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const float w = fast_exp2(x[c] - mu);
                    l[ri] += w;
                    s[t][c >> 1][2 * hh + (c & 1)] = w * kWeightScale<F16>;
                }
            }
        }
        // the weights, rounded to the cache's type, as the A operand of the product with V: at most half a step
        // of each weight, 2^-40 of the row's largest for fp16's smallest ones; the sum l keeps the unrounded
        // ones (the errors of the keys are independent, and one pass over V in the cache's type is what the
        // tensor pipe takes)
        uint32_t pf[MT][4];
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            pf[t][0] = pack16<F16>(s[t][0][0], s[t][0][1]);
            pf[t][1] = pack16<F16>(s[t][0][2], s[t][0][3]);
            pf[t][2] = pack16<F16>(s[t][1][0], s[t][1][1]);
            pf[t][3] = pack16<F16>(s[t][1][2], s[t][1][3]);
        }
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
            uint32_t vf[4];
            const int key = (km & 1) * 8 + kr;
            ldmatrix4t(vb + (j >> 2) * 2048 + key * 128 + (((2 * (j & 3) + (km >> 1)) ^ (key & 7)) << 4), vf);
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                mma16816<F16>(o[t][2 * j], pf[t], vf[0], vf[1]);
                mma16816<F16>(o[t][2 * j + 1], pf[t], vf[2], vf[3]);
            }
        }
        __syncwarp();
        if (lane == 0) {
            const int pg = page_next;
            page_next = lookup(i + C::kStages + 1);
            copy(i + C::kStages, pg);
        }
        if (++stage == C::kStages) {
            stage = 0;
            phase ^= 1u;
        }
    }
    // After a wait that ran out the copies in flight, that one's among them, land before the block ends: a wait of
    // its own, whatever limit ran out.
    for (int i = done; i < my && i < done + C::kStages; ++i)
        mbar_wait(full + i % C::kStages, (i / C::kStages) & 1, nullptr, nullptr);

    // the warps' results meet: each in its own ring
    float* so = reinterpret_cast<float*>(smem + warp * C::kWarpBytes);
    float2* ml = reinterpret_cast<float2*>(smem + C::kML);
#pragma unroll
    for (int t = 0; t < MT; ++t) {
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
            const int ri = 2 * t + hh, r = t * 16 + hh * 8 + ra;
            l[ri] += __shfl_xor_sync(0xffffffffu, l[ri], 1);
            l[ri] += __shfl_xor_sync(0xffffffffu, l[ri], 2);
            if ((lane & 3) == 0) ml[warp * C::kRows + r] = make_float2(m[ri], l[ri]);
#pragma unroll
            for (int j = 0; j < D / 8; ++j)
                *reinterpret_cast<float2*>(so + r * C::kOStride + j * 8 + cq) =
                    make_float2(o[t][j][2 * hh], o[t][j][2 * hh + 1]);
        }
    }
    if (__syncthreads_or(done < my)) return;  // (reported; nothing is written)
    for (int i = threadIdx.x; i < R * (D / 4); i += kThreads) {
        const int r = i / (D / 4), c = (i % (D / 4)) * 4;
        float top = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) top = fmaxf(top, ml[w * C::kRows + r].x);
        const float mu = top == -INFINITY ? 0.f : top;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float2 v = ml[w * C::kRows + r];
            const float f = fast_exp2(v.x - mu);  // 0 for a warp without keys
            const float4 x = *reinterpret_cast<const float4*>(smem + w * C::kWarpBytes + (r * C::kOStride + c) * 4);
            sum = fmaf(v.y, f, sum);
            acc.x = fmaf(x.x, f, acc.x);
            acc.y = fmaf(x.y, f, acc.y);
            acc.z = fmaf(x.z, f, acc.z);
            acc.w = fmaf(x.w, f, acc.w);
        }
        const float inv = sum != 0.f ? 1.f / kWeightScale<F16> / sum : 0.f;  // (a NaN sum stays NaN)
        acc.x *= inv;
        acc.y *= inv;
        acc.z *= inv;
        acc.w *= inv;
        const int64_t f = r0 + r, tok = f / G;
        const int64_t row = seq.row + tok;
        const int h = hk * G + (int)(f - tok * G);
        if (p.part.o) {
            const int64_t at =
                ((int64_t)split * p.part.rows + (p.part.per_seq ? (int64_t)b * p.part.per_seq : seq.row) + tok) * kv.H + h;
            *reinterpret_cast<float4*>(p.part.o + at * D + c) = acc;
            if (c == 0) p.part.lse[at] = sum == 0.f ? -INFINITY : mu + log2f(sum);
        } else {
            *reinterpret_cast<uint2*>(p.out + row * p.out_stride + h * D + c) =
                make_uint2(pack16<F16>(acc.x, acc.y), pack16<F16>(acc.z, acc.w));
            if (c == 0 && p.lse)
                p.lse[row * kv.H + h] = sum == 0.f ? -INFINITY : (mu + log2f(sum)) * 0.69314718055994530942f;
        }
    }
}

// The merge, a few us that move the partials once through L2 (bound by the latency of three dependent reads):
// out = sum_s 2^(lse_s - lse) part_s, lse = log2 sum_s 2^(lse_s), over the slots of one (row, head):
// D / 4 threads each take four channels.  grid: x = ((b * row blocks) + block)
template <int D, bool F16>
__global__ void __launch_bounds__(kCombineThreads) paged_combine_kernel(const PagedAttnParams p, const PagedMerge m,
                                                                int blocks) {
    constexpr int kLanes = D / 4, kHeads = kCombineThreads / kLanes;
    const csa_kv_cache& kv = p.kv;
    const int b = (int)(blockIdx.x / (unsigned)blocks);
    csa_kv_seq seq;
    bool live = paged_seq(kv, b, p.rows, p.max_n, p.prefix_len, nullptr, false, &seq);
    const int64_t f = (int64_t)(blockIdx.x % (unsigned)blocks) * kHeads + threadIdx.x / kLanes;
    const PagedPartials& own = seq.n * (kv.H / kv.H_kv) <= p.few_rows ? m.few : m.many;
    const int first = m.prefix.slots, slots = own.slots ? first + own.slots : 0;  // the prefix's slots come first
    live = live && f < seq.n * kv.H && slots > 0;
    // (the tables above are older than the launches that wrote the partials; every block waits for these,
    // so that this grid never ends before them)
    grid_dep_wait();
    if (!live) return;
    const int ln = threadIdx.x % kLanes, c = ln * 4;
    const int64_t at = seq.row * kv.H + f;
    const int64_t at_own = own.per_seq ? (int64_t)b * own.per_seq * kv.H + f : at;
    auto sum_at = [&](int s) {
        return s < first ? m.prefix.lse[at + s * m.prefix.rows * kv.H] : own.lse[at_own + (s - first) * own.rows * kv.H];
    };
    // a head's lanes read the sums of kLanes slots at once and pass them round
    const unsigned mask = kLanes == 32 ? 0xffffffffu : 0xffffu << (threadIdx.x & 16);
    float top = -INFINITY;
    for (int s = ln; s < slots; s += kLanes) top = fmaxf(top, sum_at(s));
#pragma unroll
    for (int o = kLanes / 2; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(mask, top, o, kLanes));
    const float mu = top == -INFINITY ? 0.f : top;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float sum = 0.f;
    for (int base = 0; base < slots; base += kLanes) {
        const float mine = base + ln < slots ? fast_exp2(sum_at(base + ln) - mu) : 0.f;
        const int cnt = slots - base < kLanes ? slots - base : kLanes;
        for (int j0 = 0; j0 < cnt; j0 += 8) {  // eight loads in flight
            float w[8];
            float4 x[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int slot = base + j0 + j;
                w[j] = __shfl_sync(mask, mine, j0 + j, kLanes);
                // (0 past the last, or of an empty partial, whose output was not written: not read either)
                x[j] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (w[j] != 0.f)
                    x[j] = *reinterpret_cast<const float4*>(
                        (slot < first ? m.prefix.o + (at + slot * m.prefix.rows * kv.H) * D
                                      : own.o + (at_own + (slot - first) * own.rows * kv.H) * D) + c);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                sum += w[j];
                acc.x = fmaf(x[j].x, w[j], acc.x);
                acc.y = fmaf(x[j].y, w[j], acc.y);
                acc.z = fmaf(x[j].z, w[j], acc.z);
                acc.w = fmaf(x[j].w, w[j], acc.w);
            }
        }
    }
    const float inv = sum != 0.f ? 1.f / sum : 0.f;
    const int64_t row = seq.row + f / kv.H;
    const int h = (int)(f % kv.H);
    *reinterpret_cast<uint2*>(p.out + row * p.out_stride + h * D + c) =
        make_uint2(pack16<F16>(acc.x * inv, acc.y * inv), pack16<F16>(acc.z * inv, acc.w * inv));
    if (c == 0 && p.lse) p.lse[at] = sum == 0.f ? -INFINITY : (mu + log2f(sum)) * 0.69314718055994530942f;
}

// Query rows of one key head, at most.
int64_t most_rows(const PagedAttnParams& p, const PagedStreamPart& part) {
    const int64_t G = p.kv.H / p.kv.H_kv;
    if (part.prefix_mode) return p.rows * G;
    return p.max_n * G < p.few_rows ? p.max_n * G : p.few_rows;
}

template <int D, int MT, bool F16>
cudaError_t launch_stream(const PagedAttnParams& p, PagedStreamParts& parts, cudaStream_t stream) {
    using C = StreamCfg<D, MT>;
    static PerDeviceOnce once;
    cudaError_t e = once.run([] {
        return cudaFuncSetAttribute(paged_stream_kernel<D, MT, F16>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    C::kTotal);
    });
    if (e != cudaSuccess) return e;
    int64_t grid = 0;
    for (int i = 0; i < parts.n; ++i) {
        PagedStreamPart& part = parts.part[i];
        const int64_t row_tiles = (most_rows(p, part) + C::kRows - 1) / C::kRows;
        part.row_tiles = (int)row_tiles;
        grid += (part.prefix_mode ? 1 : p.kv.B) * row_tiles * p.kv.H_kv * part.splits;
        if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
        if (i == 0) parts.blocks0 = (unsigned)grid;
    }
    StreamMaps maps;
    if ((e = paged_kv_maps(p.kv, &maps.k, &maps.v)) != cudaSuccess) return e;
    return launch_kernel(paged_stream_kernel<D, MT, F16>, dim3((unsigned)grid), dim3(kThreads), C::kTotal, stream,
                         false, maps, p, parts);
}

template <int D>
cudaError_t launch_stream_d(const PagedAttnParams& p, PagedStreamParts& parts, cudaStream_t stream) {
    const bool f16 = p.kv.type == CSA_KV_F16;
    int64_t rows = 0;
    for (int i = 0; i < parts.n; ++i) rows = most_rows(p, parts.part[i]) > rows ? most_rows(p, parts.part[i]) : rows;
    if (rows <= 16) return f16 ? launch_stream<D, 1, true>(p, parts, stream) : launch_stream<D, 1, false>(p, parts, stream);
    return f16 ? launch_stream<D, 2, true>(p, parts, stream) : launch_stream<D, 2, false>(p, parts, stream);
}

}  // namespace

cudaError_t launch_paged_stream(const PagedAttnParams& p, PagedStreamParts parts, cudaStream_t stream) {
    return p.kv.d == 128 ? launch_stream_d<128>(p, parts, stream) : launch_stream_d<64>(p, parts, stream);
}

cudaError_t launch_paged_combine(const PagedAttnParams& p, const PagedMerge& m, cudaStream_t stream, bool pdl) {
    const int heads = kCombineThreads / (p.kv.d / 4);
    // rows of a sequence that has partials
    const int64_t few = p.few_rows / (p.kv.H / p.kv.H_kv), n = m.many.slots || p.max_n < few ? p.max_n : few;
    const int64_t blocks = (n * p.kv.H + heads - 1) / heads;
    const int64_t grid = blocks * p.kv.B;
    if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
    const bool f16 = p.kv.type == CSA_KV_F16;
    auto k = p.kv.d == 128 ? (f16 ? paged_combine_kernel<128, true> : paged_combine_kernel<128, false>)
                           : (f16 ? paged_combine_kernel<64, true> : paged_combine_kernel<64, false>);
    return launch_kernel(k, dim3((unsigned)grid), dim3(kCombineThreads), 0, stream, pdl, p, m, (int)blocks);
}

}  // namespace csa
