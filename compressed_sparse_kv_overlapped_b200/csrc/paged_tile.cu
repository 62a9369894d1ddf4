// paged_tile.cu -- attention of many query rows over a paged cache (prompts, chunks of prompts, wide
// batches on a shared prefix) on tcgen05.
//
// A block is one key head and up to two tiles of 128 query rows; row r of a tile is head r % G of the
// group of token r / G, so all G heads of a token share each key that is loaded.  Its keys are the
// 16-key groups of its visible runs (first tokens, then window), eight groups to a key tile:
//     S = Q K^T     (128 x 128, over d)      tcgen05, Q and K from shared memory, S in TMEM
//     P = 2^(scale S - m)                    one thread per row, P back into the columns of its S
//     O += P V      (128 x d, over 128 keys) tcgen05, P from TMEM, V from shared memory, O in TMEM
// The reference m of a row is not its running maximum but a maximum that is moved (and O and the sum
// rescaled) only when the true one passes it by 2^8: weights then reach 2^8 at most, far from either
// type's range, and O is hardly ever touched between products.  One tile's softmax runs while the
// tensor pipe works for the other tile.
//
// A 16-key group never crosses a page, so it is one TMA box per 64 channels: a warp's lanes each look
// up and issue one box.  A group behind the last and a page number out of range become a coordinate
// past the last page, which the copy fills with zeros.  Groups that straddle the end of a run are
// loaded whole; their dead rows of V are zeroed in shared memory before the product (a weight of zero
// does not remove a NaN), their dead scores by selection.
//
// CTAs are persistent, one per SM, and all rings run on across blocks: the next block's Q, keys and
// first scores overlap this one's last product and its epilogue.  Blocks are taken longest first, in
// alternating order, so that the CTAs' sums stay close for causal prompts.
//
// Warps: 0-3 / 4-7 softmax of tile 0 / 1, 8-11 epilogue, 12 MMA issuer, 13 key loader, 14 query
// loader, 15 zeroing of dead V rows.  Every wait is bounded and winds the CTA down.
#include <cfloat>

#include "paged.h"
#include "tma.h"

namespace csa {

namespace {

constexpr int kThreads = 512;
constexpr int kTile = 128;             // query rows and keys of a tile
constexpr int kBlk = kTile * 128;      // bytes of 128 rows x 64 channels
constexpr float kSlack = 8.f;          // base-2 units by which the maximum may pass its reference

struct TileMaps {
    CUtensorMap q, k, v;
};

template <int D>
struct TileCfg {
    static constexpr int kHalves = D / 64;
    static constexpr int kOperand = kHalves * kBlk;         // a tile of Q, K or V
    static constexpr int kStages = D == 128 ? 4 : 8;        // K and V tiles in flight
    static constexpr int kQ = 0;
    static constexpr int kKV = 2 * kOperand;
    static constexpr int kOut = kKV + kStages * kOperand;   // epilogue: 32 rows of each warp
    static constexpr int kOutWarp = 32 * D * 2;
    static constexpr int kMl = kOut + 4 * kOutWarp;         // float2 [2][128]: reference and sum
    static constexpr int kBars = kMl + 2 * kTile * 8;
    static constexpr int kMisc = kBars + 40 * 8;            // tmem base, abort, block counts of 32 chunks
    static constexpr int kTotal = kMisc + 8 + 32 * 4;
    static_assert(kTotal <= 227 * 1024, "shared memory of a CTA");
};

template <int ST>
struct TileBars {
    uint64_t kv_full[ST];   // TMA: the stage holds its tile
    uint64_t kv_empty[ST];  // MMA commit: its products are done
    uint64_t v_ready[ST];   // dead rows of the V tile are zero
    uint64_t q_full[2], q_empty[2];
    uint64_t s_full[2];     // MMA commit: S of the tile is complete (and every product before it)
    uint64_t p_full[2];     // softmax: P is in TMEM, O is rescaled
    uint64_t ml_full[2];    // softmax: reference and sum of the block's rows
    uint64_t o_full[2];     // MMA commit: O is complete
    uint64_t o_free[2];     // epilogue: O and the sums are read
    uint64_t fin;
};

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w,
                                            uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
        "[%6];" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar))
        : "memory");
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
        "[%5];" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
        : "memory");
}

// 32 lanes x 32 bits, 32 consecutive columns.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
        "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,"
        "%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}

// Instruction descriptor of kind::f16, fp32 accumulation, both operands of the cache's type.
template <bool F16>
__host__ __device__ constexpr uint32_t idesc_16(int M, int N, bool b_mn_major) {
    return idesc_bf16(M, N, false, b_mn_major) & (F16 ? ~((1u << 7) | (1u << 10)) : ~0u);
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ uint64_t pair2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpair2(uint64_t v, float* a, float* b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(*a), "=f"(*b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

template <bool F16>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
    if (F16) {
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    return pack_bf16x2(lo, hi);
}

// Bits [from, to) of a 32-bit word that starts at `base`.
__device__ __forceinline__ uint32_t bits32(int from, int to, int base) {
    int f = from - base, e = to - base;
    f = f < 0 ? 0 : (f > 32 ? 32 : f);
    e = e < 0 ? 0 : (e > 32 ? 32 : e);
    return (uint32_t)((1ull << e) - 1ull) & ~(uint32_t)((1ull << f) - 1ull);
}

// One block: the tokens [tok0, tok0 + ntok) of a sequence, one key head, key tiles [t0, t1).
struct TileWork {
    int b, hk, split;
    int64_t row0;       // row of the first token
    int p0, ntok;       // its position; tokens (up to 2 tpt)
    int s1, lo, hi;     // visible runs (KeySpan)
    int n_first, win0;  // groups of the first tokens; token where the window's groups start
    int n_groups;
    int t0, t1;
};

struct TileGrid {
    int G, tpt;    // heads of a group; tokens of a 128-row tile
    int chunk;     // sequences of one of the 32 chunks of the table of block counts
    int total;     // blocks x key heads x splits
};

// Sequence b as this launch takes it: its blocks (0: none).
__device__ __forceinline__ int seq_blocks(const PagedAttnParams& p, const TileGrid& g, int b, bool say, csa_kv_seq* s) {
    if (!paged_seq(p.kv, b, p.rows, p.max_n, p.prefix_len, p.status, say, s)) return 0;
    if (s->n * g.G <= p.few_rows) return 0;
    return (int)((s->n + 2 * g.tpt - 1) / (2 * g.tpt));
}

// The CTA's k-th block: whole warps call it.  False: there is none.
__device__ __forceinline__ bool tile_work(const PagedAttnParams& p, const TileGrid& g, const int* counts, int k,
                                          TileWork& w) {
    const int64_t at = (int64_t)k * gridDim.x + ((k & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
    if (at >= g.total) return false;
    int u = (int)at;
    w.split = u % p.splits;
    u /= p.splits;
    w.hk = u % p.kv.H_kv;
    u /= p.kv.H_kv;
    int x = g.total / (p.splits * p.kv.H_kv) - 1 - u;  // the last block of a sequence sees most keys
    int64_t n, row, pos0;
    if (p.prefix_mode) {
        w.b = 0;
        n = p.rows;
        row = 0;
        pos0 = p.prefix_len;
    } else {
        const int lane = threadIdx.x & 31;
        const int c = __popc(__ballot_sync(0xffffffffu, counts[lane] <= x));
        if (c) x -= counts[c - 1];
        csa_kv_seq s;
        int b = c * g.chunk;
        for (;; ++b) {
            if (b >= p.kv.B) return false;  // (the table of sequences changed under the launch)
            const int nb = seq_blocks(p, g, b, false, &s);
            if (x < nb) break;
            x -= nb;
        }
        w.b = b;
        n = s.n;
        row = s.row;
        pos0 = s.len - s.n;
    }
    const int64_t tok0 = (int64_t)x * 2 * g.tpt;
    w.ntok = (int)(n - tok0 < 2 * g.tpt ? n - tok0 : 2 * g.tpt);
    w.row0 = row + tok0;
    w.p0 = (int)(pos0 + tok0);
    const KeySpan sp = key_span(p, w.p0, w.ntok);
    w.s1 = sp.s1;
    w.lo = sp.lo;
    w.hi = sp.hi;
    w.n_first = (sp.s1 + 15) >> 4;
    w.win0 = sp.lo & ~15;
    w.n_groups = w.n_first + (sp.hi > sp.lo ? (sp.hi - w.win0 + 15) >> 4 : 0);
    const int T = (w.n_groups + 7) >> 3;
    w.t0 = (int)((int64_t)T * w.split / p.splits);
    w.t1 = (int)((int64_t)T * (w.split + 1) / p.splits);
    return true;
}

template <int D, bool F16>
__global__ void __launch_bounds__(kThreads, 1)
    paged_tile_kernel(const __grid_constant__ TileMaps maps, const PagedAttnParams p) {
    using C = TileCfg<D>;
    extern __shared__ __align__(1024) unsigned char smem[];
    const uint32_t sbase = smem_u32(smem);
    TileBars<C::kStages>* bars = reinterpret_cast<TileBars<C::kStages>*>(smem + C::kBars);
    static_assert(sizeof(*bars) <= 40 * 8, "room for the barriers");
    uint32_t* misc = reinterpret_cast<uint32_t*>(smem + C::kMisc);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + 1);
    int* counts = reinterpret_cast<int*>(misc + 2);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const csa_kv_cache& kv = p.kv;
    if (sbase & 1023u) {  // (the swizzled layout needs it; the launch gives it)
        if (threadIdx.x == 0) report(p.status, CSA_ERR_CUDA);
        return;
    }
    TileGrid g;
    g.G = kv.H / kv.H_kv;
    g.tpt = kTile / g.G;
    g.chunk = (kv.B + 31) / 32;

    if (warp == 0) {
        if (lane == 0) {
            for (int i = 0; i < C::kStages; ++i) {
                mbar_init(&bars->kv_full[i], 1);
                mbar_init(&bars->kv_empty[i], 1);
                mbar_init(&bars->v_ready[i], 1);
            }
            for (int i = 0; i < 2; ++i) {
                mbar_init(&bars->q_full[i], 1);
                mbar_init(&bars->q_empty[i], 1);
                mbar_init(&bars->s_full[i], 1);
                mbar_init(&bars->p_full[i], 4);
                mbar_init(&bars->ml_full[i], 4);
                mbar_init(&bars->o_full[i], 1);
                mbar_init(&bars->o_free[i], 4);
            }
            mbar_init(&bars->fin, 1);
            misc[1] = 0;
            fence_mbar_init();
        }
    } else if (warp == 1) {
        // blocks of each of 32 chunks of the sequences, as running totals
        int sum = 0;
        if (p.prefix_mode) {
            sum = lane == 0 ? (int)((p.rows + 2 * g.tpt - 1) / (2 * g.tpt)) : 0;
        } else {
            for (int b = lane * g.chunk; b < kv.B && b < (lane + 1) * g.chunk; ++b) {
                csa_kv_seq s;
                sum += seq_blocks(p, g, b, blockIdx.x == 0, &s);
            }
        }
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += v;
        }
        counts[lane] = sum;
    } else if (warp == 12) {
        tmem_alloc(misc, 512);
        tmem_relinquish();
    } else if (warp == 13 && lane == 0) {
        tma_prefetch_map(&maps.q);
        tma_prefetch_map(&maps.k);
        tma_prefetch_map(&maps.v);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = misc[0];
    g.total = counts[31] * kv.H_kv * p.splits;
    const uint32_t tS[2] = {tmem, tmem + 128}, tO[2] = {tmem + 256, tmem + 384};

    auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
        return __all_sync(0xffffffffu, mbar_wait(bar, parity & 1u, p.status, abort_flag, p.wait_ns));
    };
    TileWork w;

    if (warp >= 12) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
        if (warp == 12) {
            // ---------------------------------------------------------------- MMA issuer
            constexpr uint32_t id_s = idesc_16<F16>(kTile, kTile, false), id_o = idesc_16<F16>(kTile, D, true);
            uint32_t unit = 0, nb[2] = {0, 0}, nt[2] = {0, 0};
            bool ok = true;
            auto stage = [&](uint32_t u) { return u % C::kStages; };
            auto phase = [&](uint32_t u) { return u / C::kStages; };
            auto scores = [&](int q, uint32_t u) {
                const uint64_t qd = sdesc_kmajor(sbase + C::kQ + q * C::kOperand);
                const uint64_t kd = sdesc_kmajor(sbase + C::kKV + stage(u) * C::kOperand);
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    const uint64_t off = (uint64_t)(((i >> 2) * kBlk + (i & 3) * 32) >> 4);
                    umma_bf16(tS[q], qd + off, kd + off, id_s, i != 0);
                }
                umma_commit(&bars->s_full[q]);
            };
            for (int k = 0; ok && tile_work(p, g, counts, k, w); ++k) {
                const int T = w.t1 - w.t0, nq = w.ntok > g.tpt ? 2 : 1;
                if (T == 0) continue;
                const uint32_t u0 = unit;
                unit += 2 * T;
                ok = wait(&bars->kv_full[stage(u0)], phase(u0));
                for (int q = 0; ok && q < nq; ++q) {
                    ok = wait(&bars->q_full[q], nb[q]);
                    if (!ok) break;
                    tc_fence_after();
                    scores(q, u0);
                    if (T == 1) umma_commit(&bars->q_empty[q]);
                }
                if (ok) umma_commit(&bars->kv_empty[stage(u0)]);
                for (int t = 0; ok && t < T; ++t) {
                    const uint32_t uv = u0 + 2 * t + 1, uk = uv + 1;
                    const bool more = t + 1 < T;
                    ok = wait(&bars->kv_full[stage(uv)], phase(uv)) && wait(&bars->v_ready[stage(uv)], phase(uv));
                    for (int q = 0; ok && q < nq; ++q) {
                        ok = wait(&bars->p_full[q], nt[q] + t);
                        if (ok && t == 0 && nb[q] > 0) ok = wait(&bars->o_free[q], nb[q] - 1);
                        if (!ok) break;
                        tc_fence_after();
                        const uint64_t vd = sdesc_mnmajor(sbase + C::kKV + stage(uv) * C::kOperand, kBlk);
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            umma_bf16_ts(tO[q], tS[q] + i * 8, vd + (uint64_t)((i * 16 * 128) >> 4), id_o, t > 0 || i > 0);
                        if (q == nq - 1) umma_commit(&bars->kv_empty[stage(uv)]);
                        if (more) {
                            // S takes the columns of P: products run in the order of their issue
                            if (q == 0) ok = wait(&bars->kv_full[stage(uk)], phase(uk));
                            if (!ok) break;
                            tc_fence_after();
                            scores(q, uk);
                            if (t + 2 == T) umma_commit(&bars->q_empty[q]);
                        } else {
                            umma_commit(&bars->o_full[q]);
                        }
                    }
                    if (ok && more) umma_commit(&bars->kv_empty[stage(uk)]);
                }
                for (int q = 0; q < nq; ++q) {
                    ++nb[q];
                    nt[q] += T;
                }
            }
            umma_commit(&bars->fin);
            mbar_wait(&bars->fin, 0, p.status, nullptr, p.wait_ns);
        } else if (warp == 13) {
            // ---------------------------------------------------------------- keys and values
            const int shift = page_shift(kv), grp = lane & 7, half = (lane >> 3) & 1, val = lane >> 4;
            const bool issue = half < C::kHalves;
            uint32_t unit = 0;
            bool ok = true;
            for (int k = 0; ok && tile_work(p, g, counts, k, w); ++k) {
                const int32_t* table = kv.page_table + (int64_t)w.b * kv.max_pages;
                auto find = [&](int t, int* slot) {  // page and slot of this lane's group of tile t
                    const int gi = t * 8 + grp;
                    if (gi >= w.n_groups || t >= w.t1) {
                        *slot = 0;
                        return -1;
                    }
                    const int tok = gi < w.n_first ? gi * 16 : w.win0 + (gi - w.n_first) * 16;
                    *slot = tok & (kv.page_size - 1);
                    return page_of(kv, table, shift, tok, p.status);
                };
                int slot, next_slot, next = find(w.t0, &next_slot);
                for (int t = w.t0; ok && t < w.t1; ++t) {
                    const int page = next < 0 ? (int)kv.num_pages : next;
                    slot = next_slot;
                    next = find(t + 1, &next_slot);
                    for (int e = 0; ok && e < 2; ++e, ++unit) {  // K, then V
                        const uint32_t st = unit % C::kStages;
                        if (unit >= C::kStages) ok = wait(&bars->kv_empty[st], unit / C::kStages - 1);
                        if (!ok) break;
                        if (lane == 0) mbar_arrive_expect_tx(&bars->kv_full[st], C::kOperand);
                        __syncwarp();
                        if (issue && val == e)
                            tma_load_4d(sbase + C::kKV + st * C::kOperand + half * kBlk + grp * 16 * 128,
                                        e ? &maps.v : &maps.k, half * 64, slot, w.hk, page, &bars->kv_full[st]);
                    }
                }
            }
            __syncwarp();
            if (!ok)  // the CTA gives up: its copies in flight land before it ends
                for (uint32_t u = unit > C::kStages ? unit - C::kStages : 0; u < unit; ++u)
                    mbar_wait(&bars->kv_full[u % C::kStages], (u / C::kStages) & 1, nullptr, nullptr, p.wait_ns);
        } else if (warp == 14) {
            // ---------------------------------------------------------------- queries
            uint32_t nb[2] = {0, 0};
            bool ok = true;
            for (int k = 0; ok && tile_work(p, g, counts, k, w); ++k) {
                if (w.t1 == w.t0) continue;
                const int nq = w.ntok > g.tpt ? 2 : 1;
                for (int q = 0; ok && q < nq; ++q) {
                    if (nb[q] > 0) ok = wait(&bars->q_empty[q], nb[q] - 1);
                    if (!ok) break;
                    if (lane == 0) {
                        mbar_arrive_expect_tx(&bars->q_full[q], g.G * g.tpt * 128 * C::kHalves);
#pragma unroll
                        for (int h = 0; h < C::kHalves; ++h)
                            tma_load_3d(sbase + C::kQ + q * C::kOperand + h * kBlk, &maps.q, h * 64, w.hk * g.G,
                                        (int)(w.row0 + q * g.tpt), &bars->q_full[q]);
                    }
                    __syncwarp();
                    ++nb[q];
                }
            }
            if (!ok)
                for (int q = 0; q < 2; ++q)
                    if (nb[q]) mbar_wait(&bars->q_full[q], (nb[q] - 1) & 1, nullptr, nullptr, p.wait_ns);
        } else {
            // ---------------------------------------------------------------- dead rows of V
            uint32_t unit = 0;
            bool ok = true;
            for (int k = 0; ok && tile_work(p, g, counts, k, w); ++k) {
                for (int t = w.t0; ok && t < w.t1; ++t, unit += 2) {
                    const uint32_t u = unit + 1, st = u % C::kStages;
                    ok = wait(&bars->kv_full[st], u / C::kStages);
                    if (!ok) break;
                    const uint32_t vb = sbase + C::kKV + st * C::kOperand;
                    bool wrote = false;
                    for (int j = 0; j < 8; ++j) {
                        const int gi = t * 8 + j;
                        if (gi >= w.n_groups) break;
                        const bool first = gi < w.n_first;
                        const int tok = first ? gi * 16 : w.win0 + (gi - w.n_first) * 16;
                        const int a = first ? 0 : w.lo, e = first ? w.s1 : w.hi;
                        if (tok >= a && tok + 16 <= e) continue;
                        wrote = true;
                        for (int i = lane; i < 16 * 8 * C::kHalves; i += 32) {
                            const int r = (i >> 3) & 15, key = tok + r;
                            if (key < a || key >= e)
                                st_shared_v4(vb + (i >> 7) * kBlk + (j * 16 + r) * 128 + (i & 7) * 16, make_uint4(0, 0, 0, 0));
                        }
                    }
                    if (wrote) fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bars->v_ready[st]);
                }
            }
        }
    } else if (warp >= 8) {
        // -------------------------------------------------------------------- epilogue
        asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
        const int ew = warp - 8, er = ew * 32;  // this warp's rows of a tile
        const uint32_t so = sbase + C::kOut + ew * C::kOutWarp;
        const unsigned char* sp = smem + C::kOut + ew * C::kOutWarp;
        const float2* ml = reinterpret_cast<const float2*>(smem + C::kMl);
        const uint32_t rcp = (65536u + g.G - 1) / g.G;  // r / G = r * rcp >> 16 for r < 128, G <= 64
        uint32_t nb[2] = {0, 0};
        bool ok = true;
        for (int k = 0; ok && tile_work(p, g, counts, k, w); ++k) {
            const int nq = w.ntok > g.tpt ? 2 : 1;
            for (int q = 0; ok && q < nq; ++q) {
                const int nrow = (w.ntok - q * g.tpt < g.tpt ? w.ntok - q * g.tpt : g.tpt) * g.G;
                const int64_t row0 = w.row0 + q * g.tpt;
                const int r = er + lane, rt = (int)((uint32_t)r * rcp >> 16);
                float m = -INFINITY, l = 0.f;
                if (w.t1 > w.t0) {
                    ok = wait(&bars->ml_full[q], nb[q]);
                    if (ok) ok = wait(&bars->o_full[q], nb[q]);
                    if (!ok) break;
                    const float2 v = ml[q * kTile + r];
                    m = v.x;
                    l = v.y;
                }
                const float lse = l == 0.f ? -INFINITY : m + log2f(l);  // base 2
                const float inv = l != 0.f ? 1.f / l : 0.f;             // (a NaN sum stays NaN)
                const int64_t part = (int64_t)(p.part_base + w.split) * p.rows;
                if (r < nrow) {
                    const int64_t at = (row0 + rt) * kv.H + w.hk * g.G + (r - rt * g.G);
                    if (p.part_o) p.part_lse[part * kv.H + at] = lse;
                    else if (p.lse) p.lse[at] = lse * 0.69314718055994530942f;
                }
                if (w.t1 == w.t0) continue;
                tc_fence_after();
                const uint32_t to = tO[q] + ((uint32_t)er << 16);
                // rows of D 16-bit values, or of D / 2 floats in two passes, through shared memory, so
                // that whole rows go out as contiguous 16-byte vectors
                constexpr int kRow = D * 2, kVec = kRow / 16, kRowsAt = 32 / kVec;
                const int passes = p.part_o ? 2 : 1;
                for (int s = 0; s < passes; ++s) {
#pragma unroll
                    for (int c = 0; c < D / 32; ++c) {
                        if (passes == 2 && c / (D / 64) != s) continue;
                        uint32_t x[32];
                        tmem_ld32(to + c * 32, x);
                        tmem_ld_wait();
                        if (passes == 1) {
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                uint32_t y[4];
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    y[e] = pack16<F16>(__uint_as_float(x[8 * i + 2 * e]) * inv,
                                                       __uint_as_float(x[8 * i + 2 * e + 1]) * inv);
                                st_shared_v4(so + lane * kRow + (((c * 4 + i) ^ (lane & 7)) << 4),
                                             make_uint4(y[0], y[1], y[2], y[3]));
                            }
                        } else {
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                st_shared_v4(so + lane * kRow + ((((c % (D / 64)) * 8 + i) ^ (lane & 7)) << 4),
                                             make_uint4(__float_as_uint(__uint_as_float(x[4 * i]) * inv),
                                                        __float_as_uint(__uint_as_float(x[4 * i + 1]) * inv),
                                                        __float_as_uint(__uint_as_float(x[4 * i + 2]) * inv),
                                                        __float_as_uint(__uint_as_float(x[4 * i + 3]) * inv)));
                        }
                    }
                    if (s == passes - 1) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&bars->o_free[q]);
                    } else {
                        __syncwarp();
                    }
#pragma unroll 4
                    for (int i = 0; i < 32; i += kRowsAt) {
                        const int lr = i + lane / kVec, v = lane % kVec, tr = er + lr;
                        const uint4 y = *reinterpret_cast<const uint4*>(sp + lr * kRow + ((v ^ (lr & 7)) << 4));
                        if (tr < nrow) {
                            const int tt = (int)((uint32_t)tr * rcp >> 16), h = w.hk * g.G + (tr - tt * g.G);
                            if (passes == 1)
                                *reinterpret_cast<uint4*>(p.out + (row0 + tt) * p.out_stride + h * D + v * 8) = y;
                            else
                                *reinterpret_cast<uint4*>(p.part_o + ((part + row0 + tt) * kv.H + h) * D + s * (D / 2) + v * 4) = y;
                        }
                    }
                    __syncwarp();
                }
                ++nb[q];
            }
        }
    } else {
        // -------------------------------------------------------------------- softmax
        asm volatile("setmaxnreg.inc.sync.aligned.u32 192;");
        const int q = warp >> 2, r = threadIdx.x & 127;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t ts = tS[q] + lanes, to = tO[q] + lanes;
        float2* ml = reinterpret_cast<float2*>(smem + C::kMl) + q * kTile;
        const int rt = r / g.G;
        const float sc = p.scale_log2;
        uint32_t nb = 0, nt = 0;
        bool ok = true;
        for (int k = 0; ok && tile_work(p, g, counts, k, w); ++k) {
            const int T = w.t1 - w.t0;
            if (T == 0 || w.ntok <= q * g.tpt) continue;
            const int p_first = w.p0 + q * g.tpt, p_last = w.p0 + (w.ntok < (q + 1) * g.tpt ? w.ntok : (q + 1) * g.tpt) - 1;
            const int pos = p_first + rt;
            const int wb = 16 * w.n_first - w.win0;  // index in the list of groups of a window token
            const int up = pos + 1 < w.hi ? pos + 1 : w.hi;
            const int low = pos - p.W + 1 > w.lo ? pos - p.W + 1 : w.lo;
            const int first_up = p.S < up ? p.S : up;
            const int all_up = p_first + 1 < w.hi ? p_first + 1 : w.hi;  // tokens every row sees, but for the window
            float m = -INFINITY;
            uint64_t l2[2] = {0, 0};
            for (int t = 0; t < T; ++t) {
                ok = wait(&bars->s_full[q], nt + t);
                if (!ok) break;
                tc_fence_after();
                uint32_t s[128];
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_ld32(ts + c * 32, s + c * 32);
                tmem_ld_wait();
                const int i0 = (w.t0 + t) * kTile, tok0 = i0 - wb;
                const bool whole = i0 + kTile <= w.s1 ||
                                   (i0 >= 16 * w.n_first && tok0 >= w.lo && tok0 + kTile <= all_up &&
                                    (tok0 > p_last - p.W || tok0 + kTile <= p.S));
                if (!whole) {
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const int base = i0 + c * 32;
                        const uint32_t see = bits32(0, w.s1, base) | bits32(wb + low, wb + up, base) |
                                             bits32(wb + w.lo, wb + first_up, base);
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (!((see >> i) & 1u)) s[c * 32 + i] = 0xff800000u;  // -inf
                    }
                }
                float mx[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) mx[c] = fmaxf(__uint_as_float(s[c]), __uint_as_float(s[4 + c]));
#pragma unroll
                for (int i = 8; i < 128; i += 4) {
#pragma unroll
                    for (int c = 0; c < 4; ++c) mx[c] = fmaxf(mx[c], __uint_as_float(s[i + c]));
                }
                const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                if (t == 0) {
                    m = top;
                } else {
                    const bool move = (top - m) * sc > kSlack;
                    if (__any_sync(0xffffffffu, move)) {
                        // every product so far came before this S: O can be changed
                        const float f = move ? fast_exp2((m - top) * sc) : 1.f;
                        if (move) m = top;
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            float a, b;
                            unpair2(l2[i], &a, &b);
                            l2[i] = pair2(a * f, b * f);
                        }
#pragma unroll 1
                        for (int c = 0; c < D; c += 16) {
                            uint32_t x[16];
                            tmem_ld16(to + c, x);
                            tmem_ld_wait();
#pragma unroll
                            for (int i = 0; i < 16; ++i) x[i] = __float_as_uint(__uint_as_float(x[i]) * f);
                            tmem_st16(to + c, x);
                        }
                    }
                }
                const float neg = m == -INFINITY ? 0.f : -m * sc;
                const uint64_t sc2 = pair2(sc, sc), neg2 = pair2(neg, neg);
                // the weights, rounded to the cache's type for the product with V: the sum keeps the
                // unrounded ones (the rounding errors of the keys average out, half a step each at most)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t pk[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        const int e = h * 64 + i * 2;
                        float a, b;
                        unpair2(fma2(pair2(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), sc2, neg2), &a, &b);
                        a = fast_exp2(a);
                        b = fast_exp2(b);
                        l2[i & 1] = add2(l2[i & 1], pair2(a, b));
                        pk[i] = pack16<F16>(a, b);
                    }
                    tmem_st32(ts + h * 32, pk);
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars->p_full[q]);
            }
            if (!ok) break;
            // (the sums of the block before are read once its O is)
            if (nb > 0) ok = wait(&bars->o_free[q], nb - 1);
            if (!ok) break;
            float a, b, c, d;
            unpair2(l2[0], &a, &b);
            unpair2(l2[1], &c, &d);
            ml[r] = make_float2(m == -INFINITY ? 0.f : m * sc, (a + b) + (c + d));
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->ml_full[q]);
            ++nb;
            nt += T;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 12) tmem_dealloc(tmem, 512);
}

template <int D, bool F16>
cudaError_t launch_tile(const PagedAttnParams& p, cudaStream_t stream) {
    using C = TileCfg<D>;
    static PerDeviceOnce once;
    cudaError_t e = once.run([] {
        return cudaFuncSetAttribute(paged_tile_kernel<D, F16>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kTotal);
    });
    if (e != cudaSuccess) return e;
    const csa_kv_cache& kv = p.kv;
    const int G = kv.H / kv.H_kv, tpt = kTile / G;
    TileMaps maps;
    const uint64_t row = (uint64_t)kv.slot_stride * 2;
    const uint64_t qd[3] = {(uint64_t)D, (uint64_t)kv.H, (uint64_t)p.rows}, qs[2] = {(uint64_t)D * 2, (uint64_t)p.q_stride * 2};
    const uint32_t qb[3] = {64, (uint32_t)G, (uint32_t)tpt};
    const uint64_t kd[4] = {(uint64_t)D, (uint64_t)kv.page_size, (uint64_t)kv.H_kv, (uint64_t)kv.num_pages};
    const uint64_t ks[3] = {row, kv.H_kv > 1 ? (uint64_t)kv.head_stride * 2 : row,
                            kv.num_pages > 1 ? (uint64_t)kv.page_stride * 2 : row};
    const uint32_t kb[4] = {64, 16, 1, 1};
    if ((e = tensor_map_16bit(&maps.q, F16, p.q, 3, qd, qs, qb)) != cudaSuccess) return e;
    if ((e = tensor_map_16bit(&maps.k, F16, kv.k_pages, 4, kd, ks, kb)) != cudaSuccess) return e;
    if ((e = tensor_map_16bit(&maps.v, F16, kv.v_pages, 4, kd, ks, kb)) != cudaSuccess) return e;
    int dev = 0, sms = 0;
    if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
    if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
    const int64_t n = p.prefix_mode ? p.rows : p.max_n;
    const int64_t most = (p.prefix_mode ? 1 : kv.B) * ((n + 2 * tpt - 1) / (2 * tpt)) * kv.H_kv * p.splits;
    if (most > 0x7fffffff) return cudaErrorInvalidConfiguration;
    return launch_kernel(paged_tile_kernel<D, F16>, dim3((unsigned)(most < sms ? most : sms)), dim3(kThreads), C::kTotal,
                         stream, false, maps, p);
}

}  // namespace

cudaError_t launch_paged_tile(const PagedAttnParams& p, cudaStream_t stream) {
    const bool f16 = p.kv.type == CSA_KV_F16;
    if (p.kv.d == 128) return f16 ? launch_tile<128, true>(p, stream) : launch_tile<128, false>(p, stream);
    return f16 ? launch_tile<64, true>(p, stream) : launch_tile<64, false>(p, stream);
}

}  // namespace csa
