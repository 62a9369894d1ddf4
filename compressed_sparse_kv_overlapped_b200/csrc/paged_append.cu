// paged_append.cu -- csa_kv_append: new keys and values into their pages, keys and queries turned by
// position on the way.
//
// A turn needs cos and sin of t * inv_freq[j]: the product is formed in double and reduced to
// (-1, 1] half-turns there (position 2^20 times a frequency near 1 leaves fp32 with an error of a
// sixteenth of a radian), then one sincospif in fp32 (error below 2^-23, far under the 16-bit
// rounding of the result).  A block takes up to kTok consecutive tokens of one sequence and computes
// their rot / 2 pairs of cos and sin once, in shared memory, for all heads of q and k.
//
// The work is a copy: 4 d (H + 2 H_kv) bytes per token, bound by HBM for prompts and by one launch's
// latency for decode steps.  The unit of a thread is 16 channels of one head as two 16-byte vectors:
// channels 8 j and rot / 2 + 8 j (pairs half a rotation apart) or 16 j and 16 j + 8 (pairs side by
// side, and channels behind rot), which always hold the pairs of frequencies 8 j .. 8 j + 7, so both
// pairings share one loop.  Each thread loads kBatch units before it turns and stores the first, to
// keep enough bytes in flight.  Measured: ragged prompts of 28,000 tokens, 1.16 GB in 195 us = 5.9 TB/s
// (0.91 of the copy rate); a step of 128 sequences 6.0 us, of four 2.7 us on the device.
#include "paged.h"

namespace csa {

namespace {

constexpr int kTok = 8;
constexpr int kThreads = 256;
constexpr int kBatch = 4;

template <bool F16>
__device__ __forceinline__ float2 unpack2(uint32_t v) {
    if (F16) return __half22float2(*reinterpret_cast<const __half2*>(&v));
    return make_float2(bf16lo(v), bf16hi(v));
}
template <bool F16>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    if (F16) {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    return pack_bf16x2(a, b);
}

// Pairs (x, y) of eight frequencies, turned in place.  Interleaved: a and b hold x, y side by side;
// else a holds the eight x and b the eight y.
template <bool F16>
__device__ __forceinline__ void turn(uint4& a, uint4& b, const float* cs, bool interleaved) {
    uint32_t va[4] = {a.x, a.y, a.z, a.w}, vb[4] = {b.x, b.y, b.z, b.w};
    if (interleaved) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            uint32_t& w = i < 4 ? va[i] : vb[i - 4];
            const float2 v = unpack2<F16>(w);
            const float c = cs[2 * i], s = cs[2 * i + 1];
            w = pack2<F16>(v.x * c - v.y * s, v.x * s + v.y * c);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 x = unpack2<F16>(va[i]), y = unpack2<F16>(vb[i]);
            const float c0 = cs[4 * i], s0 = cs[4 * i + 1], c1 = cs[4 * i + 2], s1 = cs[4 * i + 3];
            va[i] = pack2<F16>(x.x * c0 - y.x * s0, x.y * c1 - y.y * s1);
            vb[i] = pack2<F16>(x.x * s0 + y.x * c0, x.y * s1 + y.y * c1);
        }
    }
    a = make_uint4(va[0], va[1], va[2], va[3]);
    b = make_uint4(vb[0], vb[1], vb[2], vb[3]);
}

template <bool F16>
__global__ void __launch_bounds__(kThreads) paged_append_kernel(const PagedAppendParams p, int tok, int tiles) {
    __shared__ __align__(16) float cs[kTok][64][2];  // cos, sin of each token and frequency
    __shared__ int64_t slot[kTok];                   // element offset of each token's slot, -1: no page
    const int b = (int)(blockIdx.x / (unsigned)tiles);
    const int64_t i0 = (int64_t)(blockIdx.x % (unsigned)tiles) * tok;
    csa_kv_seq s;
    if (!paged_seq(p.kv, b, p.rows, p.max_n, 0, p.status, threadIdx.x == 0 && i0 == 0, &s) || i0 >= s.n) return;
    const int cnt = (int)(s.n - i0 < tok ? s.n - i0 : tok);
    const int64_t t0 = s.len - s.n + i0, r0 = s.row + i0;
    const int half = p.rot / 2;
    for (int i = threadIdx.x; i < cnt * half; i += kThreads) {
        const int t = i / half, j = i % half;
        double u = (double)(t0 + t) * (double)p.inv_freq[j] * 0.31830988618379067154;  // angle / pi
        u -= 2.0 * rint(0.5 * u);
        float sn, c;
        sincospif((float)u, &sn, &c);
        cs[t][j][0] = c;
        cs[t][j][1] = sn;
    }
    if ((int)threadIdx.x < cnt) {
        const int64_t t = t0 + threadIdx.x;
        const int pg = page_of(p.kv, p.kv.page_table + (int64_t)b * p.kv.max_pages, page_shift(p.kv), (int)t,
                               p.status);
        slot[threadIdx.x] =
            pg < 0 ? -1 : pg * p.kv.page_stride + (t & (p.kv.page_size - 1)) * p.kv.slot_stride;
    }
    __syncthreads();

    const int H = p.q ? p.kv.H : 0, Hk = p.kv.H_kv, d = p.kv.d;
    const int lu = d == 128 ? 3 : 2, nrot = p.rot / 16;  // log2 of a head's units; units that turn
    const int heads = H + 2 * Hk, per_tok = heads << lu, total = cnt * per_tok;
    for (int base = threadIdx.x; base < total; base += kThreads * kBatch) {
        uint4 a[kBatch], c[kBatch];
        uint16_t* dst[kBatch];
        const float* f[kBatch];
        int second[kBatch];  // offset of the second vector
#pragma unroll
        for (int m = 0; m < kBatch; ++m) {
            const int i = base + m * kThreads;
            dst[m] = nullptr;
            f[m] = nullptr;
            second[m] = 8;
            if (i < total) {
                const int t = i / per_tok, r = i - t * per_tok, h = r >> lu, j = r & ((1 << lu) - 1);
                const uint16_t* src;
                if (h < H) {
                    src = p.q + (r0 + t) * p.q_stride + h * d;
                    dst[m] = p.q_out + (r0 + t) * p.q_out_stride + h * d;
                } else {
                    const bool key = h < H + Hk;
                    const int hk = h - H - (key ? 0 : Hk);
                    src = (key ? p.k + (r0 + t) * p.k_stride : p.v + (r0 + t) * p.v_stride) + hk * d;
                    if (slot[t] >= 0)
                        dst[m] = static_cast<uint16_t*>(key ? p.kv.k_pages : p.kv.v_pages) + slot[t] +
                                 hk * p.kv.head_stride;
                }
                int off = 16 * j;
                if (j < nrot && h < H + Hk) {
                    f[m] = &cs[t][8 * j][0];
                    if (!p.interleaved) {
                        off = 8 * j;
                        second[m] = half;
                    }
                }
                src += off;
                if (dst[m]) dst[m] += off;
                a[m] = *reinterpret_cast<const uint4*>(src);
                c[m] = *reinterpret_cast<const uint4*>(src + second[m]);
            }
        }
#pragma unroll
        for (int m = 0; m < kBatch; ++m) {
            if (!dst[m]) continue;
            if (f[m]) turn<F16>(a[m], c[m], f[m], p.interleaved != 0);
            *reinterpret_cast<uint4*>(dst[m]) = a[m];
            *reinterpret_cast<uint4*>(dst[m] + second[m]) = c[m];
        }
    }
}

}  // namespace

cudaError_t launch_paged_append(const PagedAppendParams& p, cudaStream_t stream) {
    const int tok = (int)(p.max_n < kTok ? p.max_n : kTok);
    const int64_t tiles = (p.max_n + tok - 1) / tok;
    const int64_t grid = tiles * p.kv.B;
    if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
    return launch_kernel(p.kv.type == CSA_KV_F16 ? paged_append_kernel<true> : paged_append_kernel<false>,
                         dim3((unsigned)grid), dim3(kThreads), 0, stream, false, p, tok, (int)tiles);
}

}  // namespace csa
