// paged_tile.cu -- attention of many query rows over a paged cache (prompts, chunks of prompts, wide
// batches on a shared prefix) on tcgen05.
//
// A block is one key head and up to two tiles of 128 query rows; row r of a tile is head r % G of the
// group of token r / G, so all G heads of a token share each key that is loaded.  Its keys are the
// 16-key groups of its visible runs (first tokens, then window), up to eight groups to a key tile (tiles
// of equal width: twelve groups are two tiles of 96 keys, not of 128 and 64):
//     S = Q K^T     (128 x 128, over d)      tcgen05, Q and K from shared memory, S in TMEM
//     P = 2^(scale S - m)                    one thread per row, P back into the columns of its S (fp16: 2^7 P)
//     O += P V      (128 x d, over 128 keys) tcgen05, P from TMEM, V from shared memory, O in TMEM
// The reference m of a row is not its running maximum but a maximum that is moved (and O and the sum
// rescaled) only when the true one passes it by 2^8: weights then reach 2^8 at most, far from either
// type's range, and O is hardly ever touched between products.  One tile's softmax runs while the
// tensor pipe works for the other tile; the product of the first 64 keys starts when their weights are
// stored (8 % on causal prompts).
//
// A 16-key group never crosses a page, so it is one TMA box per 64 channels: a warp's lanes each look
// up and issue one box.  A group behind the last and a page number out of range become a coordinate
// past the last page, which the copy fills with zeros.  Groups that straddle the end of a run are
// loaded whole; their dead rows of V are zeroed in shared memory before the product (a weight of zero
// does not remove a NaN), their dead scores by selection.
//
// CTAs are persistent, one per SM, and all rings run on across blocks: the next block's Q and keys arrive
// during this one's last products, behind which its first scores are issued (those of both row tiles, so
// that the tiles start a block together), and both overlap this one's epilogue.  Blocks are taken longest
// first, in alternating order, so that the CTAs' sums stay close for causal prompts.
//
// Warps: 0-3 / 4-7 softmax of tile 0 / 1, 8-11 epilogue, 12 MMA issuer, 13 key loader, 14 look-up of
// the blocks and query loader, 15 zeroing of dead V rows.  Every wait is bounded and winds the CTA down.
//
// Measured (bf16, d = 128): causal prompts of 77 to 8,191 tokens, 32 heads on 8, 0.85 ms = 0.96 PFLOP/s
// (0.58 of a cuBLAS GEMM); the tensor pipe is 53 % busy and issue slots 41 %.  Bound by the chain of one
// tile: of its period of about 3,700 clocks the softmax of a row tile takes about 2,500 (512 clocks of
// loads and maximum, the rest exponentials at 16 a clock and SM, shared with the other tile's) and the
// products 1,000.  A prompt of 32,768 with a window of 128: 0.44 ms for 1.2 GB (0.42 of the copy rate),
// two key tiles a block, so every latency of the chain shows.  Measured and not taken: a share of the
// exponentials as a polynomial on the FMA pipe (5 % slower: that unit is no limit), two threads per row
// (768 threads; 15 % slower on causal prompts, 3 % faster at d = 64), scores read twice from TMEM in
// short loops (10 % slower with a window of 128), P handed over after 32 or 96 keys (1 % slower).
// What helped most after the first form was short code: the roles share the instruction cache, and a
// warp-uniform role index, 32-bit barrier addresses and products issued several per block of code took
// causal prompts from 1.01 to 0.93 ms.
#include <cstddef>

#include "paged.h"
#include "tma.h"

namespace csa {

namespace {

constexpr int kThreads = 512;
// Registers of a thread: at launch, and of the softmax, epilogue and last four warps after the exchange
// between them, which waits until they are there.
constexpr int kRegs = 128, kRegsSoftmax = 192, kRegsEpilogue = 80, kRegsLast = 48;
static_assert(256 * kRegsSoftmax + 128 * kRegsEpilogue + 128 * kRegsLast <= kThreads * kRegs, "registers of a block");
constexpr int kTile = 128;             // query rows and keys of a tile
constexpr int kBlk = kTile * 128;      // bytes of 128 rows x 64 channels
constexpr int kWorks = 4;              // blocks looked up ahead
constexpr int kReaders = 15;           // warps that read them
constexpr float kSlack = 8.f;          // base-2 units by which the maximum may pass its reference
// Base-2 units added to the exponent of every weight: fp16 has no normal numbers below 2^-14, and weights reach
// 2^(kSlack + kShift) = 2^15 at most.  So one of 2^-21 of the row's largest is still normal and only those under
// 2^-32 are lost (2^-12 of the output with a million of them); unshifted, 131,072 keys of 2^-25.2 behind one strong
// first token lose all of their 0.3 %.  bf16 has the range of fp32.  Sum and O grow alike.
template <bool F16>
constexpr float kShift = F16 ? 7.f : 0.f;

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
    static constexpr int kWork = kBars + 52 * 8;            // TileWork [kWorks]
    static constexpr int kMisc = kWork + kWorks * 64;       // tmem base, abort, block counts of 32 chunks
    static constexpr int kTotal = kMisc + 8 + 32 * 4;
    static_assert(kTotal <= 227 * 1024, "shared memory of a CTA");
};

// Barriers by their 32-bit address: an operation is one or two instructions.
__device__ __forceinline__ bool try_wait(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity & 1u)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ void arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void arrive_expect_tx(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.release.cta.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}

template <int ST>
struct TileBars {
    uint64_t kv_full[ST];   // TMA: the stage holds its tile
    uint64_t kv_empty[ST];  // MMA commit: its products are done
    uint64_t v_ready[ST];   // dead rows of the V tile are zero
    uint64_t q_full[2], q_empty[2];
    uint64_t s_full[2];     // MMA commit: S of the tile is complete (and every product before it)
    uint64_t p_half[2];     // softmax: O is rescaled, P of the first 64 keys of a full tile is in TMEM
    uint64_t p_full[2];     // softmax: all of P is
    uint64_t ml_full[2];    // softmax: reference and sum of the block's rows
    uint64_t o_full[2];     // MMA commit: O is complete
    uint64_t o_free[2];     // epilogue: O and the sums are read
    uint64_t work_full[kWorks], work_empty[kWorks];
    uint64_t fin;
};

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
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// The issue of a product costs more instructions than it has operands if the compiler must move each
// into uniform registers on its own.  So a warp issues several from one block of code: the operands'
// descriptors differ in their low words only (addresses below 256 KB: no carry into the other fields),
// the high word is a constant, TMEM addresses are constants (an allocation of all 512 columns starts
// at column 0), and the electing predicate is made once per block.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);  // 8-row groups 1024 bytes apart, 128-byte swizzle
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lbo) { return (saddr >> 4) | ((lbo >> 4) << 16); }

#define CSA_MMA_SS(OFF, P)                                                                     \
    "add.u32 x, %1, " OFF ";\n\tmov.b64 a, {x, %4};\n\tadd.u32 x, %2, " OFF ";\n\tmov.b64 b, {x, %4};\n\t" \
    "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, " P ";\n\t"
// True in one lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred e;\n\t.reg .b32 l;\n\telect.sync l|e, 0xffffffff;\n\tselp.u32 %0, 1, 0, e;\n\t}" : "=r"(r));
    return r != 0;
}
__device__ __forceinline__ void commit(uint32_t bar) {
    if (elect_one())
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
// D (+)= A B over 64 channels: K-major operands in shared memory, low descriptor words a and b.
__device__ __forceinline__ void umma_64ch(uint32_t d_tmem, uint32_t a, uint32_t b, uint32_t idesc, bool accumulate) {
    if (!elect_one()) return;
    asm volatile(
        "{\n\t.reg .pred p, t;\n\t.reg .b32 x;\n\t.reg .b64 a, b;\n\t"
        "setp.ne.b32 p, %5, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
        CSA_MMA_SS("0", "p") CSA_MMA_SS("2", "t") CSA_MMA_SS("4", "t") CSA_MMA_SS("6", "t") "}" ::"r"(d_tmem),
        "r"(a), "r"(b), "r"(idesc), "n"(kDescHi), "r"((uint32_t)accumulate)
        : "memory");
}
#define CSA_MMA_TS(I, J, P)                                                                    \
    "add.u32 x, %1, " I ";\n\tadd.u32 y, %2, " J ";\n\tmov.b64 b, {y, %4};\n\t"                    \
    "tcgen05.mma.cta_group::1.kind::f16 [%0], [x], b, %3, " P ";\n\t"
// D (+)= A B over 32 keys: A in TMEM (8 columns for 16 keys), B MN-major (2048 bytes for 16 keys).
__device__ __forceinline__ void umma_32keys(uint32_t d_tmem, uint32_t a, uint32_t b, uint32_t idesc, bool accumulate) {
    if (!elect_one()) return;
    asm volatile(
        "{\n\t.reg .pred p, t;\n\t.reg .b32 x, y;\n\t.reg .b64 b;\n\t"
        "setp.ne.b32 p, %5, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
        CSA_MMA_TS("0", "0", "p") CSA_MMA_TS("8", "128", "t") "}" ::"r"(d_tmem),
        "r"(a), "r"(b), "r"(idesc), "n"(kDescHi), "r"((uint32_t)accumulate)
        : "memory");
}
// The same over 64 keys.
__device__ __forceinline__ void umma_64keys(uint32_t d_tmem, uint32_t a, uint32_t b, uint32_t idesc, bool accumulate) {
    if (!elect_one()) return;
    asm volatile(
        "{\n\t.reg .pred p, t;\n\t.reg .b32 x, y;\n\t.reg .b64 b;\n\t"
        "setp.ne.b32 p, %5, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
        CSA_MMA_TS("0", "0", "p") CSA_MMA_TS("8", "128", "t") CSA_MMA_TS("16", "256", "t") CSA_MMA_TS("24", "384", "t")
        "}" ::"r"(d_tmem),
        "r"(a), "r"(b), "r"(idesc), "n"(kDescHi), "r"((uint32_t)accumulate)
        : "memory");
}
#undef CSA_MMA_SS
#undef CSA_MMA_TS

template <bool F16>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
    if (F16) {
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    return pack_bf16x2(lo, hi);
}

// The weight of a score s is 2^(s sc + weight_ref(m)): kShift - m sc, rounded so that no weight of a score up to m
// passes 2^kShift, however large m is (0 while no key was seen, whose m is -inf).
template <bool F16>
__device__ __forceinline__ float weight_ref(float m, float sc) {
    return m == -INFINITY ? 0.f : F16 ? __fmaf_rd(-m, sc, kShift<F16>) : -m * sc;
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
    int b, hk, split;   // b < 0: there are no more
    int row0;           // row of the first token
    int p0, ntok;       // its position; tokens (up to 2 tpt)
    int s1, lo, hi;     // visible runs (KeySpan)
    int n_first, win0;  // groups of the first tokens; token where the window's groups start
    int n_groups, gw;   // groups; of them in a key tile (an even number up to 8)
    int t0, t1;
};
static_assert(sizeof(TileWork) <= 64, "an entry of the ring");

struct TileGrid {
    int G, tpt;    // heads of a group; tokens of a 128-row tile
    int chunk;     // sequences of one of the 32 chunks of the table of block counts
    int total;     // blocks x key heads x splits
};

// Sequence b as this launch takes it: its blocks (0: none).
__device__ __forceinline__ int seq_blocks(const PagedAttnParams& p, const TileGrid& g, int b, bool say, csa_kv_seq* s) {
    if (!paged_seq(p.kv, b, p.rows, p.max_n, p.prefix_len, p.status, say, s)) return 0;
    if (s->n * g.G <= p.few_rows) return 0;
    return (int)(((uint32_t)s->n + 2u * g.tpt - 1u) / (2u * g.tpt));  // (n <= rows < 2^30)
}

// The CTA's k-th block: whole warps call it.  False: there is none.
__device__ __forceinline__ bool tile_work(const PagedAttnParams& p, const TileGrid& g, const int* counts, int k,
                                          TileWork& w) {
    const int64_t at = (int64_t)k * gridDim.x + ((k & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
    if (at >= g.total) return false;
    uint32_t u = (uint32_t)at;
    w.split = 0;
    if (p.splits > 1) {
        w.split = (int)(u % (uint32_t)p.splits);
        u /= (uint32_t)p.splits;
    }
    w.hk = (int)(u % (uint32_t)p.kv.H_kv);
    u /= (uint32_t)p.kv.H_kv;
    int x = counts[31] - 1 - (int)u;  // the last block of a sequence sees most keys
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
    w.row0 = (int)(row + tok0);
    w.p0 = (int)(pos0 + tok0);
    const KeySpan sp = key_span(p, w.p0, w.ntok);
    w.s1 = sp.s1;
    w.lo = sp.lo;
    w.hi = sp.hi;
    w.n_first = (sp.s1 + 15) >> 4;
    w.win0 = sp.lo & ~15;
    w.n_groups = w.n_first + (sp.hi > sp.lo ? (sp.hi - w.win0 + 15) >> 4 : 0);
    // key tiles of equal width: 12 groups are two tiles of 6, not of 8 and 4 zero ones
    const int T = (w.n_groups + 7) >> 3;
    w.gw = T > 1 ? (((w.n_groups + T - 1) / T) + 1) & ~1 : (w.n_groups + 1) & ~1;
    w.t0 = 0;
    w.t1 = T;
    if (p.splits > 1) {  // (T < 2^23, at most 256 splits)
        w.t0 = (int)((uint32_t)T * (uint32_t)w.split / (uint32_t)p.splits);
        w.t1 = (int)((uint32_t)T * (uint32_t)(w.split + 1) / (uint32_t)p.splits);
    }
    return true;
}

template <int D, bool F16>
__global__ void __launch_bounds__(kThreads, 1)
    paged_tile_kernel(const __grid_constant__ TileMaps maps, const __grid_constant__ PagedAttnParams p) {
    using C = TileCfg<D>;
    extern __shared__ __align__(1024) unsigned char smem[];
    const uint32_t sbase = smem_u32(smem);
    TileBars<C::kStages>* bars = reinterpret_cast<TileBars<C::kStages>*>(smem + C::kBars);
    static_assert(sizeof(*bars) <= 52 * 8, "room for the barriers");
    uint32_t* misc = reinterpret_cast<uint32_t*>(smem + C::kMisc);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + 1);
    int* counts = reinterpret_cast<int*>(misc + 2);
    // (the shuffle tells the compiler that a warp's threads take the same branches)
    const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    const csa_kv_cache& kv = p.kv;
    grid_dep_launch();
    if (sbase & 1023u) {  // (the swizzled layout needs it; the launch gives it)
        if (threadIdx.x == 0) report(p.status, CSA_ERR_CUDA);
        grid_dep_wait();
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
                mbar_init(&bars->p_half[i], 4);
                mbar_init(&bars->p_full[i], 4);
                mbar_init(&bars->ml_full[i], 4);
                mbar_init(&bars->o_full[i], 1);
                mbar_init(&bars->o_free[i], 4);
            }
            for (int i = 0; i < kWorks; ++i) {
                mbar_init(&bars->work_full[i], 1);
                mbar_init(&bars->work_empty[i], kReaders);
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
    if (misc[0] != 0) {  // (an allocation of every column starts at the first)
        if (threadIdx.x == 0) report(p.status, CSA_ERR_CUDA);
        if (warp == 12) tmem_dealloc(misc[0], 512);
        grid_dep_wait();
        return;
    }
    g.total = counts[31] * kv.H_kv * p.splits;
    // S (and P) of tile q in columns 128 q, O in columns 256 + 128 q
    auto tS = [&](int q) { return (uint32_t)q * 128u; };
    auto tO = [&](int q) { return 256u + (uint32_t)q * 128u; };

    // A bounded wait of a whole warp, kept small: the kernel's roles share the instruction cache.  Time in
    // clocks (two a nanosecond: at least the limit; 2.1 seconds at most); the first to give up makes every
    // role stop, and the end of the kernel reports it.
    const uint32_t limit = p.wait_ns < 2100000000ull ? (uint32_t)(p.wait_ns * 2) : 4200000000u;
    using Bars = TileBars<C::kStages>;
#define BAR(field, i) (sbase + (uint32_t)(C::kBars + offsetof(Bars, field)) + 8u * (uint32_t)(i))
    auto wait = [&](uint32_t bar, uint32_t parity) -> bool {
        bool done = try_wait(bar, parity);
        if (__builtin_expect(!done, 0)) {
            const uint32_t t0 = (uint32_t)clock();
#pragma unroll 1
            while (!(done = try_wait(bar, parity))) {
                if (*abort_flag) break;
                if ((uint32_t)clock() - t0 > limit) *abort_flag = 2;
            }
        }
        return __all_sync(0xffffffffu, done);
    };
    // Copies or products in flight: each role that issues some waits for its last ones before it ends, since any
    // role may have given up on them.  A limit of its own, 2.1 seconds, whatever limit ran out.
    auto drain = [&](uint32_t bar, uint32_t parity) {
        const uint32_t t0 = (uint32_t)clock();
#pragma unroll 1
        while (!try_wait(bar, parity))
            if ((uint32_t)clock() - t0 > 4200000000u) break;
    };
    // the CTA's k-th block, looked up by warp 14 for all roles
    const TileWork* works = reinterpret_cast<const TileWork*>(smem + C::kWork);
    TileWork w;
    auto next_work = [&](int k) -> bool {
        if (!wait(BAR(work_full, k % kWorks), k / kWorks)) return false;
        w = *reinterpret_cast<const TileWork*>(reinterpret_cast<const unsigned char*>(works) + (k % kWorks) * 64);
        __syncwarp();
        if (lane == 0) arrive(BAR(work_empty, k % kWorks));
        return w.b >= 0;
    };

    if (warp >= 12) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsLast));
        if (warp == 12) {
            // ---------------------------------------------------------------- MMA issuer
            constexpr uint32_t id_o = idesc_16<F16>(kTile, D, true);
            // blocks and key tiles that ran on the two row tiles; tile 1 may be left out of a block
            uint32_t unit = 0, nb0 = 0, nb1 = 0, nt0 = 0, nt1 = 0;
            bool ok = p.debug_fault != 1;
            if (!ok) *abort_flag = 2;
            for (int k = 0; ok && next_work(k); ++k) {
                const int T = w.t1 - w.t0, nq = w.ntok > g.tpt ? 2 : 1;
                if (T == 0) continue;
                const uint32_t id_s = idesc_16<F16>(kTile, w.gw * 16, false);
                // step t: for each row tile the product P V of key tile t - 1, then the scores of tile t,
                // which take the columns of that P: products run in the order of their issue
#pragma unroll 1
                for (int t = 0; ok && t <= T; ++t) {
                    const uint32_t uk = unit + 2 * t, uv = uk - 1;  // ring units of K(t) and V(t - 1)
                    const uint32_t ks = uk % C::kStages, vs = uv % C::kStages;
                    if (t > 0) ok = wait(BAR(kv_full, vs), uv / C::kStages) && wait(BAR(v_ready, vs), uv / C::kStages);
                    if (ok && t < T) ok = wait(BAR(kv_full, ks), uk / C::kStages);
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        if (!ok || q >= nq) break;
                        const uint32_t nb = q ? nb1 : nb0;
                        if (t > 0) {
                            const uint32_t turn = (q ? nt1 : nt0) + t - 1;
                            const bool full = w.gw == 8;
                            ok = wait(full ? BAR(p_half, q) : BAR(p_full, q), turn);
                            if (ok && t == 1 && nb > 0) ok = wait(BAR(o_free, q), nb - 1);
                            if (!ok) break;
                            tc_fence_after();
                            const uint32_t vd = desc_lo(sbase + C::kKV + vs * C::kOperand, kBlk);
                            if (full) {
                                umma_64keys(tO(q), tS(q), vd, id_o, t > 1);
                                ok = wait(BAR(p_full, q), turn);
                                if (!ok) break;
                                tc_fence_after();
                                umma_64keys(tO(q), tS(q) + 32, vd + 512, id_o, true);
                            } else {
#pragma unroll 1
                                for (int i = 0; i < w.gw; i += 2)
                                    umma_32keys(tO(q), tS(q) + i * 8, vd + i * 128, id_o, t > 1 || i > 0);
                            }
                            if (q == nq - 1) commit(BAR(kv_empty, vs));
                            if (t == T) commit(BAR(o_full, q));
                        } else {
                            ok = wait(BAR(q_full, q), nb);
                            if (!ok) break;
                        }
                        if (t < T) {
                            const uint32_t qd = desc_lo(sbase + C::kQ + q * C::kOperand, 16);
                            const uint32_t kd = desc_lo(sbase + C::kKV + ks * C::kOperand, 16);
#pragma unroll
                            for (int i = 0; i < C::kHalves; ++i)
                                umma_64ch(tS(q), qd + i * (kBlk >> 4), kd + i * (kBlk >> 4), id_s, i > 0);
                            commit(BAR(s_full, q));
                            if (q == nq - 1) commit(BAR(kv_empty, ks));
                            if (t == T - 1) commit(BAR(q_empty, q));
                        }
                    }
                }
                unit += 2 * T;
                ++nb0;
                nt0 += T;
                if (nq == 2) {
                    ++nb1;
                    nt1 += T;
                }
            }
            commit(BAR(fin, 0));
            drain(BAR(fin, 0), 0);  // (all products are done: TMEM may go)
        } else if (warp == 13) {
            // ---------------------------------------------------------------- keys and values
            const int shift = page_shift(kv), grp = lane & 7, half = (lane >> 3) & 1, val = lane >> 4;
            const bool issue = half < C::kHalves;
            uint32_t unit = 0;
            bool ok = true;
            for (int k = 0; ok && next_work(k); ++k) {
                const int32_t* table = kv.page_table + (int64_t)w.b * kv.max_pages;
                auto find = [&](int t, int* slot) {  // page and slot of this lane's group of tile t
                    const int gi = t * w.gw + grp;
                    if (gi >= w.n_groups || grp >= w.gw || t >= w.t1) {
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
                        if (unit >= C::kStages) ok = wait(BAR(kv_empty, st), unit / C::kStages - 1);
                        if (!ok) break;
                        if (lane == 0) arrive_expect_tx(BAR(kv_full, st), w.gw * 16 * D * 2);
                        __syncwarp();
                        if (issue && val == e && grp < w.gw)
                            tma_load_4d(sbase + C::kKV + st * C::kOperand + half * kBlk + grp * 16 * 128,
                                        e ? &maps.v : &maps.k, half * 64, slot, w.hk, page, BAR(kv_full, st));
                    }
                }
            }
            __syncwarp();
            for (uint32_t u = unit > C::kStages ? unit - C::kStages : 0; u < unit; ++u)
                drain(BAR(kv_full, u % C::kStages), u / C::kStages);
        } else if (warp == 14) {
            // ---------------------------------------------------------------- blocks and queries
            uint32_t nb0 = 0, nb1 = 0;
            bool ok = true, last = false;
            int made = 0;
            for (int k = 0; ok; ++k) {
                // two blocks ahead of their queries: the key loader runs on with them
                for (; ok && !last && made <= k + 2; ++made) {
                    if (made >= kWorks) ok = wait(BAR(work_empty, made % kWorks), made / kWorks - 1);
                    if (!ok) break;
                    last = !tile_work(p, g, counts, made, w);
                    if (last) w.b = -1;
                    if (lane == 0) {
                        *reinterpret_cast<TileWork*>(smem + C::kWork + (made % kWorks) * 64) = w;
                        arrive(BAR(work_full, made % kWorks));
                    }
                    __syncwarp();
                }
                if (!ok) break;
                w = *reinterpret_cast<const TileWork*>(smem + C::kWork + (k % kWorks) * 64);
                if (w.b < 0) break;
                if (w.t1 == w.t0) continue;
                const int nq = w.ntok > g.tpt ? 2 : 1;
                for (int q = 0; ok && q < nq; ++q) {
                    const uint32_t before = q ? nb1 : nb0;
                    if (before > 0) ok = wait(BAR(q_empty, q), before - 1);
                    if (!ok) break;
                    if (lane == 0) {
                        arrive_expect_tx(BAR(q_full, q), g.G * g.tpt * 128 * C::kHalves);
#pragma unroll
                        for (int h = 0; h < C::kHalves; ++h)
                            tma_load_3d(sbase + C::kQ + q * C::kOperand + h * kBlk, &maps.q, h * 64, w.hk * g.G,
                                        (int)(w.row0 + q * g.tpt), BAR(q_full, q));
                    }
                    __syncwarp();
                    if (q) ++nb1; else ++nb0;
                }
            }
            if (nb0) drain(BAR(q_full, 0), nb0 - 1);
            if (nb1) drain(BAR(q_full, 1), nb1 - 1);
        } else {
            // ---------------------------------------------------------------- dead rows of V
            uint32_t unit = 0;
            bool ok = true;
            for (int k = 0; ok && next_work(k); ++k) {
                for (int t = w.t0; ok && t < w.t1; ++t, unit += 2) {
                    const uint32_t u = unit + 1, st = u % C::kStages;
                    ok = wait(BAR(kv_full, st), u / C::kStages);
                    if (!ok) break;
                    const uint32_t vb = sbase + C::kKV + st * C::kOperand;
                    bool wrote = false;
#pragma unroll 1
                    for (int j = 0; j < w.gw; ++j) {
                        const int gi = t * w.gw + j;
                        if (gi >= w.n_groups) break;
                        const bool first = gi < w.n_first;
                        const int tok = first ? gi * 16 : w.win0 + (gi - w.n_first) * 16;
                        const int a = first ? 0 : w.lo, e = first ? w.s1 : w.hi;
                        if (tok >= a && tok + 16 <= e) continue;
                        wrote = true;
#pragma unroll 1
                        for (int i = lane; i < 16 * 8 * C::kHalves; i += 32) {
                            const int r = (i >> 3) & 15, key = tok + r;
                            if (key < a || key >= e)
                                st_shared_v4(vb + (i >> 7) * kBlk + (j * 16 + r) * 128 + (i & 7) * 16, make_uint4(0, 0, 0, 0));
                        }
                    }
                    if (wrote) fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) arrive(BAR(v_ready, st));
                }
            }
        }
    } else if (warp >= 8) {
        // -------------------------------------------------------------------- epilogue
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsEpilogue));
        const int ew = warp - 8, er = ew * 32;  // this warp's rows of a tile
        const uint32_t so = sbase + C::kOut + ew * C::kOutWarp;
        const unsigned char* sp = smem + C::kOut + ew * C::kOutWarp;
        const float2* ml = reinterpret_cast<const float2*>(smem + C::kMl);
        constexpr int kRow = D * 2, kVec = kRow / 16, kRowsAt = 32 / kVec;
        const int step_t = kRowsAt / g.G, step_h = kRowsAt % g.G;
        const uint32_t rcp = (65536u + g.G - 1) / g.G;  // r / G = r * rcp >> 16 for r < 128, G <= 64
        uint32_t nb0 = 0, nb1 = 0;
        bool ok = true;
        for (int k = 0; ok && next_work(k); ++k) {
            const int nq = w.ntok > g.tpt ? 2 : 1;
            for (int q = 0; ok && q < nq; ++q) {
                const int nrow = (w.ntok - q * g.tpt < g.tpt ? w.ntok - q * g.tpt : g.tpt) * g.G;
                const int64_t row0 = w.row0 + q * g.tpt;
                const int r = er + lane, rt = (int)((uint32_t)r * rcp >> 16);
                float m = -INFINITY, l = 0.f;
                if (w.t1 > w.t0) {
                    const uint32_t before = q ? nb1 : nb0;
                    ok = wait(BAR(ml_full, q), before) && wait(BAR(o_full, q), before);
                    if (!ok) break;
                    const float2 v = ml[q * kTile + r];
                    m = v.x;
                    l = v.y;
                }
                const float lse = l == 0.f ? -INFINITY : m + log2f(l);  // base 2
                const float inv = l != 0.f ? 1.f / l : 0.f;             // (a NaN sum stays NaN)
                const int64_t part = (int64_t)w.split * p.part.rows;  // (by row)
                if (r < nrow) {
                    const int64_t at = (row0 + rt) * kv.H + w.hk * g.G + (r - rt * g.G);
                    if (p.part.o) p.part.lse[part * kv.H + at] = lse;
                    else if (p.lse) p.lse[at] = lse * 0.69314718055994530942f;
                }
                if (w.t1 == w.t0) continue;
                tc_fence_after();
                const uint32_t to = tO(q) + ((uint32_t)er << 16);
                // rows of D 16-bit values, or of D / 2 floats in two passes, through shared memory, so
                // that whole rows go out as contiguous 16-byte vectors
                const int passes = p.part.o ? 2 : 1;
                const uint64_t inv2 = pair2(inv, inv);
#pragma unroll 1
                for (int s = 0; s < passes; ++s) {
#pragma unroll 1
                    for (int c = 0; c < D / 32; ++c) {
                        if (passes == 2 && c / (D / 64) != s) continue;
                        uint32_t x[32];
                        tmem_ld32(to + c * 32, x);
                        tmem_ld_wait();
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            float a, b;
                            unpair2(mul2(pair2(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1])), inv2), &a, &b);
                            x[2 * i] = __float_as_uint(a);
                            x[2 * i + 1] = __float_as_uint(b);
                        }
                        if (passes == 1) {
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                uint32_t y[4];
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    y[e] = pack16<F16>(__uint_as_float(x[8 * i + 2 * e]), __uint_as_float(x[8 * i + 2 * e + 1]));
                                st_shared_v4(so + lane * kRow + (((c * 4 + i) ^ (lane & 7)) << 4),
                                             make_uint4(y[0], y[1], y[2], y[3]));
                            }
                        } else {
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                st_shared_v4(so + lane * kRow + ((((c % (D / 64)) * 8 + i) ^ (lane & 7)) << 4),
                                             make_uint4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]));
                        }
                    }
                    if (s == passes - 1) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) arrive(BAR(o_free, q));
                    } else {
                        __syncwarp();
                    }
                    // the lane's vector of rows er + lane / kVec, + kRowsAt, ...: a step of kRowsAt heads, or on
                    // to the next token
                    const int v = lane % kVec;
                    int lr = lane / kVec, tt = (int)((uint32_t)(er + lr) * rcp >> 16), h = er + lr - tt * g.G;
                    const int64_t row_bytes = passes == 1 ? p.out_stride * 2 : (int64_t)kv.H * D * 4;
                    const int head_bytes = passes == 1 ? D * 2 : D * 4;
                    unsigned char* dst = passes == 1 ? reinterpret_cast<unsigned char*>(p.out) + v * 16
                                                     : reinterpret_cast<unsigned char*>(p.part.o + part * kv.H * D + s * (D / 2)) + v * 16;
                    dst += (row0 + tt) * row_bytes + (int64_t)(w.hk * g.G + h) * head_bytes;
                    const int64_t step = step_t * row_bytes + step_h * head_bytes, wrap = row_bytes - g.G * head_bytes;
#pragma unroll 4
                    for (int i = 0; i < 32; i += kRowsAt, lr += kRowsAt) {
                        const uint4 y = *reinterpret_cast<const uint4*>(sp + lr * kRow + ((v ^ (lr & 7)) << 4));
                        if (er + lr < nrow) *reinterpret_cast<uint4*>(dst) = y;
                        dst += step;
                        h += step_h;
                        if (h >= g.G) {
                            h -= g.G;
                            dst += wrap;
                        }
                    }
                    __syncwarp();
                }
                if (q) ++nb1; else ++nb0;
            }
        }
    } else {
        // -------------------------------------------------------------------- softmax
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
        const int q = warp >> 2, r = threadIdx.x & 127;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t ts = tS(q) + lanes, to = tO(q) + lanes;
        float2* ml = reinterpret_cast<float2*>(smem + C::kMl) + q * kTile;
        auto stored = [&](uint32_t bar) {  // this warp's TMEM stores so far are complete
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive(bar);
        };
        const int rt = r / g.G;
        const float sc = p.scale_log2;
        uint32_t nb = 0, nt = 0;
        bool ok = true;
        for (int k = 0; ok && next_work(k); ++k) {
            const int T = w.t1 - w.t0;
            if (T == 0 || w.ntok <= q * g.tpt) continue;
            const int p_first = w.p0 + q * g.tpt, p_last = w.p0 + (w.ntok < (q + 1) * g.tpt ? w.ntok : (q + 1) * g.tpt) - 1;
            const int pos = p_first + rt;
            const int wb = 16 * w.n_first - w.win0;  // index in the list of groups of a window token
            const int up = pos + 1 < w.hi ? pos + 1 : w.hi;
            const int low = pos - p.W + 1 > w.lo ? pos - p.W + 1 : w.lo;
            const int first_up = p.S < up ? p.S : up;
            const int all_up = p_first + 1 < w.hi ? p_first + 1 : w.hi;  // tokens every row sees, but for the window
            const int width = 16 * w.gw;
            float m = -INFINITY;
            uint64_t l2[2] = {0, 0};
            for (int t = 0; t < T; ++t) {
                ok = wait(BAR(s_full, q), nt + t);
                if (!ok) break;
                tc_fence_after();
                uint32_t s[128];  // (chunks of 32 keys; those behind the tile's width stay out)
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    if (c * 32 < width) tmem_ld32(ts + c * 32, s + c * 32);
                tmem_ld_wait();
                const bool wide = width == kTile;
                const int i0 = (w.t0 + t) * width, tok0 = i0 - wb;
                const bool whole = i0 + width <= w.s1 ||
                                   (i0 >= 16 * w.n_first && tok0 >= w.lo && tok0 + width <= all_up &&
                                    (tok0 > p_last - p.W || tok0 + width <= p.S));
                if (!whole) {
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const int base = i0 + c * 32;
                        const uint32_t see = bits32(0, w.s1, base) | bits32(wb + low, wb + up, base) |
                                             bits32(wb + w.lo, wb + first_up, base);
                        if (c * 32 < width && __any_sync(0xffffffffu, see != 0xffffffffu)) {
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (!((see >> i) & 1u)) s[c * 32 + i] = 0xff800000u;  // -inf
                        }
                    }
                }
                float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                auto chunk_max = [&](int c) {
#pragma unroll
                    for (int i = 0; i < 32; i += 8) {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            mx[e] = max3(mx[e], __uint_as_float(s[c * 32 + i + e]), __uint_as_float(s[c * 32 + i + e + 4]));
                    }
                };
                if (wide) {
#pragma unroll
                    for (int c = 0; c < 4; ++c) chunk_max(c);
                } else {
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        if (c * 32 < width) chunk_max(c);
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
                const float neg = weight_ref<F16>(m, sc);
                const uint64_t sc2 = pair2(sc, sc), neg2 = pair2(neg, neg);
                // the weights, rounded to the cache's type for the product with V: at most half a step of each
                // weight, 2^-32 of the row's reference for fp16's smallest ones; the sum keeps the unrounded
                // ones (the errors of the keys are independent, and P in the cache's type is what the tensor
                // pipe takes beside V)
                auto chunk_exp = [&](int c) {
                    uint32_t pk[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const int e = c * 32 + i * 2;
                        float a, b;
                        const uint64_t x2 = fma2(pair2(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), sc2, neg2);
                        unpair2(x2, &a, &b);
                        a = fast_exp2(a);
                        b = fast_exp2(b);
                        l2[i & 1] = add2(l2[i & 1], pair2(a, b));
                        pk[i] = pack16<F16>(a, b);
                    }
                    tmem_st16(ts + c * 16, pk);
                };
                if (wide) {
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        chunk_exp(c);
                        if (c == 1) stored(BAR(p_half, q));  // the product of the first 64 keys can start
                    }
                } else {
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        if (c * 32 < width) chunk_exp(c);
                    if (lane == 0) arrive(BAR(p_half, q));
                }
                stored(BAR(p_full, q));
            }
            if (!ok) break;
            // (the sums of the block before are read once its O is)
            if (nb > 0) ok = wait(BAR(o_free, q), nb - 1);
            if (!ok) break;
            float a, b, c, d;
            unpair2(l2[0], &a, &b);
            unpair2(l2[1], &c, &d);
            ml[r] = make_float2(-weight_ref<F16>(m, sc), (a + b) + (c + d));
            __syncwarp();
            if (lane == 0) arrive(BAR(ml_full, q));
            ++nb;
            nt += T;
        }
    }
    grid_dep_wait();  // (a launch that this one overlapped: whatever waits for this grid waits for that one too)
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0 && *abort_flag == 2) report(p.status, CSA_ERR_TIMEOUT);
    if (warp == 12) tmem_dealloc(misc[0], 512);
}

#undef BAR

template <int D, bool F16>
cudaError_t launch_tile(const PagedAttnParams& p, cudaStream_t stream, bool pdl) {
    using C = TileCfg<D>;
    static PerDeviceOnce once;
    cudaError_t e = once.run([] {
        // (the exchange of registers would wait for ever in a block that starts with fewer than it counts on)
        cudaFuncAttributes attr;
        const cudaError_t err = cudaFuncGetAttributes(&attr, paged_tile_kernel<D, F16>);
        if (err != cudaSuccess) return err;
        if (attr.numRegs < kRegs) return cudaErrorInvalidConfiguration;
        return cudaFuncSetAttribute(paged_tile_kernel<D, F16>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kTotal);
    });
    if (e != cudaSuccess) return e;
    const csa_kv_cache& kv = p.kv;
    const int G = kv.H / kv.H_kv, tpt = kTile / G;
    TileMaps maps;
    const uint64_t qd[3] = {(uint64_t)D, (uint64_t)kv.H, (uint64_t)p.rows}, qs[2] = {(uint64_t)D * 2, (uint64_t)p.q_stride * 2};
    const uint32_t qb[3] = {64, (uint32_t)G, (uint32_t)tpt};
    if ((e = tensor_map_16bit(&maps.q, F16, p.q, 3, qd, qs, qb)) != cudaSuccess) return e;
    if ((e = paged_kv_maps(kv, &maps.k, &maps.v)) != cudaSuccess) return e;
    int dev = 0, sms = 0;
    if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
    if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
    const int64_t n = p.prefix_mode ? p.rows : p.max_n;
    const int64_t most = (p.prefix_mode ? 1 : kv.B) * ((n + 2 * tpt - 1) / (2 * tpt)) * kv.H_kv * p.splits;
    if (most > 0x7fffffff) return cudaErrorInvalidConfiguration;
    return launch_kernel(paged_tile_kernel<D, F16>, dim3((unsigned)(most < sms ? most : sms)), dim3(kThreads), C::kTotal,
                         stream, pdl, maps, p);
}

}  // namespace

cudaError_t paged_kv_maps(const csa_kv_cache& kv, CUtensorMap* k, CUtensorMap* v) {
    const uint64_t row = (uint64_t)kv.slot_stride * 2;
    const uint64_t dims[4] = {(uint64_t)kv.d, (uint64_t)kv.page_size, (uint64_t)kv.H_kv, (uint64_t)kv.num_pages};
    const uint64_t strides[3] = {row, kv.H_kv > 1 ? (uint64_t)kv.head_stride * 2 : row,
                                 kv.num_pages > 1 ? (uint64_t)kv.page_stride * 2 : row};
    const uint32_t box[4] = {64, 16, 1, 1};
    const bool f16 = kv.type == CSA_KV_F16;
    const cudaError_t e = tensor_map_16bit(k, f16, kv.k_pages, 4, dims, strides, box);
    return e != cudaSuccess ? e : tensor_map_16bit(v, f16, kv.v_pages, 4, dims, strides, box);
}

cudaError_t launch_paged_tile(const PagedAttnParams& p, cudaStream_t stream, bool pdl) {
    const bool f16 = p.kv.type == CSA_KV_F16;
    if (p.kv.d == 128) return f16 ? launch_tile<128, true>(p, stream, pdl) : launch_tile<128, false>(p, stream, pdl);
    return f16 ? launch_tile<64, true>(p, stream, pdl) : launch_tile<64, false>(p, stream, pdl);
}

}  // namespace csa
