// paged.cu -- C entry points of the paged key/value operators (declared in include/csa.h): host-side
// checks, the split of long rows, workspace layout and launches.
#include <cmath>

#include "kernels.h"
#include "paged.h"

namespace csa {

namespace {

constexpr int64_t kMaxTokens = (int64_t)1 << 30;  // token positions and counts fit 32 bits on the device
constexpr size_t align256(size_t v) { return (v + 255) & ~(size_t)255; }
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool stride_ok(int64_t v, int64_t least) { return v >= least && v % 8 == 0 && v < (int64_t)1 << 36; }

// Checks of the cache's shape (`pointers`: and of its pointers).
int check_cache(const csa_kv_cache& kv, bool pointers) {
    if (kv.d != 64 && kv.d != 128) return set_error(CSA_ERR_UNSUPPORTED, "d = %d (supported: 64, 128)", kv.d);
    if (kv.type != CSA_KV_BF16 && kv.type != CSA_KV_F16)
        return set_error(CSA_ERR_UNSUPPORTED, "type = %d (CSA_KV_BF16 or CSA_KV_F16)", kv.type);
    if (kv.H < 1 || kv.H > 256) return set_error(CSA_ERR_UNSUPPORTED, "H = %d (supported: 1..256)", kv.H);
    if (kv.H_kv < 1 || kv.H % kv.H_kv) return set_error(CSA_ERR_ARG, "H_kv = %d does not divide H = %d", kv.H_kv, kv.H);
    if (kv.H / kv.H_kv > 64)
        return set_error(CSA_ERR_UNSUPPORTED, "%d query heads on a key head (supported: 1..64)", kv.H / kv.H_kv);
    if (kv.page_size < 16 || kv.page_size > 256 || (kv.page_size & (kv.page_size - 1)))
        return set_error(CSA_ERR_UNSUPPORTED, "page_size = %d (supported: powers of two from 16 to 256)", kv.page_size);
    if (kv.B < 1 || kv.num_pages < 1 || kv.max_pages < 1)
        return set_error(CSA_ERR_ARG, "B = %d, num_pages = %lld, max_pages = %lld", kv.B, (long long)kv.num_pages,
                         (long long)kv.max_pages);
    if (kv.max_pages > kMaxTokens / kv.page_size || kv.num_pages > 0x7fffffff)
        return set_error(CSA_ERR_UNSUPPORTED, "max_pages = %lld of %d tokens, num_pages = %lld", (long long)kv.max_pages,
                         kv.page_size, (long long)kv.num_pages);
    if (!stride_ok(kv.page_stride, kv.num_pages > 1 ? 8 : 0) || !stride_ok(kv.slot_stride, 8) ||
        !stride_ok(kv.head_stride, kv.H_kv > 1 ? 8 : 0))
        return set_error(CSA_ERR_ARG, "page_stride = %lld, slot_stride = %lld, head_stride = %lld (multiples of 8)",
                         (long long)kv.page_stride, (long long)kv.slot_stride, (long long)kv.head_stride);
    if (!pointers) return CSA_OK;
    if (!kv.k_pages || !kv.v_pages || !kv.page_table || !kv.seqs) return set_error(CSA_ERR_ARG, "NULL pointer argument");
    if (!aligned16(kv.k_pages) || !aligned16(kv.v_pages))
        return set_error(CSA_ERR_ARG, "pages must be 16-byte aligned");
    if ((reinterpret_cast<uintptr_t>(kv.page_table) & 3u) || (reinterpret_cast<uintptr_t>(kv.seqs) & 7u))
        return set_error(CSA_ERR_ARG, "page_table must be 4-byte, seqs 8-byte aligned");
    return CSA_OK;
}

int check_rows(int64_t rows, int64_t max_n) {
    if (rows < 0 || rows >= kMaxTokens || max_n < 0)
        return set_error(CSA_ERR_ARG, "rows = %lld, max_n = %lld", (long long)rows, (long long)max_n);
    return CSA_OK;
}

// No query anywhere by the host's bounds: the call does nothing.
bool no_rows(const csa_kv_attn_args& a) { return a.rows == 0 || a.max_n == 0 || a.max_len == 0; }

// Shape checks of an attention call; op: CSA_OP_WINDOW_ATTN or CSA_OP_PREFIX_ATTN.
int check_attn(const csa_kv_attn_args& a, int op) {
    int rc = check_cache(a.kv, false);
    if (rc) return rc;
    if ((rc = check_rows(a.rows, a.max_n))) return rc;
    if (a.max_len < 0) return set_error(CSA_ERR_ARG, "max_len = %lld", (long long)a.max_len);
    if (!(a.scale > 0.f) || !std::isfinite(a.scale)) return set_error(CSA_ERR_ARG, "scale = %g", (double)a.scale);
    if (a.reserved != 0) return set_error(CSA_ERR_ARG, "reserved must be 0");
    if (op == CSA_OP_WINDOW_ATTN) {
        if (a.W < 1 || a.S < 0 || a.prefix_len != 0)
            return set_error(CSA_ERR_ARG, "W = %lld (>= 1), S = %lld (>= 0), prefix_len = %lld (0)", (long long)a.W,
                             (long long)a.S, (long long)a.prefix_len);
    } else {
        if (a.W != 0 || a.S != 0 || a.prefix_len < 0)
            return set_error(CSA_ERR_ARG, "W = %lld (0), S = %lld (0), prefix_len = %lld (>= 0)", (long long)a.W,
                             (long long)a.S, (long long)a.prefix_len);
        if (a.prefix_len > a.kv.max_pages * a.kv.page_size)
            return set_error(CSA_ERR_ARG, "prefix_len = %lld exceeds a row of the page table", (long long)a.prefix_len);
    }
    return CSA_OK;
}

// How a call is cut.  Sequences with few query rows per key head go through the stream kernel, those
// with more through the tile kernel; so do the rows of all sequences on a shared prefix.
struct PagedPlan {
    bool few, many;              // classes of sequences that may be there
    int splits_few, splits_many; // key splits of their windows / suffixes
    bool prefix_tile;
    int splits_prefix;           // 0: no prefix
    int few_groups, prefix_groups;  // 16-key groups of a split of the stream kernel
    PagedMerge merge;            // partials, their pointers offsets into the workspace
    bool any;                    // there are some
    size_t total;
};

// Rows of one key head up to which the stream kernel is used.  It reads a block's keys once per 32 rows,
// the tile kernel once per 256 but with at least a tile's time (2 us) per 128 keys: 128 rows on a prefix of
// 8,192 take 37 us here through the tile kernel and 92 through the stream kernel; up to 64 rows, where
// long rows are split over all SMs, the stream kernel's launch is the shorter one.
constexpr int64_t kFewRows = 64;
constexpr int64_t kFewPrefixRows = 64;  // the same for the rows of all sequences on the prefix

int sm_count_or(int dflt) {
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        cudaGetLastError();  // no device here: the plan of a full-size part
        return dflt;
    }
    return n;
}

// The tile kernel's cut of `items` blocks over up to `keys` keys each: while there are fewer blocks than SMs
// each is cut so that every SM has one, of 256 keys at least (128 rows on a prefix of 8,192: 43 us, uncut 127;
// 128 tokens behind 30,000: 72 us, uncut 410).  More blocks than that are never cut to even out the last
// round: partials of many rows cost more than it wins (prompts of 4,096 tokens, 3.5 rounds: 125 us uncut,
// 260 cut in two).
int tile_splits(int64_t items, int64_t keys, int sms) {
    int64_t s = items > 0 ? sms / items : 1;
    if (s > keys / 256) s = keys / 256;
    s = s < 1 ? 1 : (s < 64 ? s : 64);
    // no more than the longest split's key tiles ask for: 64 tiles in 18 are four each, as in 16
    const int64_t tiles = (keys + 127) / 128, each = (tiles + s - 1) / s;
    return tiles > 0 ? (int)((tiles + each - 1) / each) : 1;
}

// What the host knows of the keys that the sequences of a launch see: all the same (a shared prefix), bounded by a
// window that most of them fill, or only that none has more than the bound.
enum class Lengths { same, window, bound };

// The stream kernel's cut: splits of `groups` 16-key groups each, for `items` blocks that see up to `keys`
// keys.  Lengths are known on the device only, so a split is a fixed number of keys: a shorter sequence
// has fewer.  The number is the one with the least estimated time, in us: blocks run in rounds of two an
// SM; a round takes its bytes at 6.4 TB/s, but no less than a block alone needs, 60 keys a us, and 1.5 to
// start; a merge that would not be there otherwise costs 6, each split of a row 0.5 (0.25 beside a prefix).
// A tenth of the estimate under a window is that of a batch with half of the keys, whose time ends with one long
// row's last block.
// A split has at most 2,048 keys (8,192 where lengths are the same or bounded by a window), lest one long sequence
// outlast the rest.  That asks for no more than `asked` splits, nor than 2^14 blocks, of 4 ns each where they are
// empty, lest a loose bound fill the grid and the workspace with nothing.  Beyond it there are never more than `most`.
// Measured with 8 key heads of 128, in us.
//   Windows of 4,096, 80 / 128 / 256 / 320 / 384 / 512 blocks: 47 / 68 / 107 / 141 / 154 / 188; uncut 78 / 78 / 107 /
//     182 / 184 / 188.
//   Five windows of 65,536: 14 splits 230 (6: 222, 7: 232, 15: 271); one of them of 40,000: 220 (7: 212, 15: 214).
//   Windows of 16,384, 31 sequences of 1,000 and one of 131,072: 8 splits 73 (2: 161, uncut 283).
//   Windows of 12,000, 32 full ones, where the cap costs: 2 splits 265 (uncut 244).
//   Causal, 31 sequences of 1,000 and one of 131,072: 32 splits 160 (64: 194, 8: 323, 3: 599).
//   Causal, 32 sequences of 1,000 to 32,768: 15 splits 339 (7: 353, 3: 392).
//   Causal, 128 sequences of 8,000: 4 splits 645; with a bound of 2^20: 16 splits 695 (32: 729, 256: 1,592).
//   Beside a prompt of 512, 64 sequences of 1,000, bound 131,072: 16 splits 158 (32: 206, uncut 95); one of them of
//     131,072: 249 (32: 302, uncut 3,110).
constexpr int64_t kAsked = 32;
int stream_splits(int64_t items, int64_t keys, Lengths lengths, bool merged, int d, int sms, int64_t asked, int64_t most,
                  int* groups) {
    constexpr int64_t kLongest = 2048, kLongestEven = 8192;
    constexpr double kBytesUs = 6.4e6, kKeysUs = 60.0, kStartUs = 1.5, kShortShare = 0.1;
    const int64_t places = 2 * (int64_t)sms;
    const int64_t least = items * (keys / 128) <= places ? 128 : 256;  // keys of a split
    const int64_t longest = lengths == Lengths::bound ? kLongest : kLongestEven;
    int64_t from = keys > longest ? (keys + longest - 1) / longest : 1;
    const int64_t blocks = items < 16384 ? 16384 / items : 1;
    if (from > asked) from = asked;
    if (from > blocks) from = blocks;
    const int64_t fill = (places + items - 1) / items, upto = fill > 64 ? fill : 64;
    int64_t s = from;
    double best = 1e30;
    for (int64_t i = from; i == from || (i <= upto && i * least <= keys); ++i) {
        const double share = (double)keys / (double)i, alone = share / kKeysUs, us = share * 4.0 * d / kBytesUs;
        const int64_t full = items * i / places, rest = items * i % places;
        double t = (double)full * (((double)places * us > alone ? (double)places * us : alone) + kStartUs);
        if (rest) t += ((double)rest * us > alone ? (double)rest * us : alone) + kStartUs;
        if (lengths == Lengths::window)
            t += kShortShare * (0.5 * (double)(items * i) * us + alone + kStartUs - t);
        if (i > 1) t = 1.05 * t + (merged ? 0.25 * (double)i : 6.0 + 0.5 * (double)i);  // (a cut has to be worth it)
        if (t < best) {
            best = t;
            s = i;
        }
    }
    if (s > most) s = most > from ? most : from;
    const int64_t n = keys / 16 + 2;  // (both runs of keys may begin and end inside a group)
    *groups = (int)((n + s - 1) / s);
    return (int)((n + *groups - 1) / *groups);
}

PagedPlan make_plan(const csa_kv_attn_args& a, int op) {
    PagedPlan pl{};
    if (no_rows(a)) {
        pl.total = 256;
        return pl;
    }
    const int64_t G = a.kv.H / a.kv.H_kv, cap = a.kv.max_pages * a.kv.page_size, B = a.kv.B;
    const int64_t max_len = a.max_len < cap ? a.max_len : cap;
    const int64_t n = a.max_n < a.rows ? a.max_n : a.rows;  // (what the kernels bound a sequence's n by)
    const int64_t n_few = n * G > kFewRows ? kFewRows / G : n, tpb = 2 * (128 / G);
    const bool by_seq = B * n_few <= a.rows;  // how partials of few rows are held: whichever is less
    const int64_t few_rows = by_seq ? B * n_few : a.rows;
    const int sms = sm_count_or(148);
    auto stream_items = [&](int64_t seqs, int64_t rows) { return seqs * a.kv.H_kv * ((rows * G + 31) / 32); };
    pl.many = n * G > kFewRows;
    pl.few = !pl.many || B > 1;
    auto keys = [&](int64_t q) {  // that a block of q queries of one sequence sees
        if (op == CSA_OP_PREFIX_ATTN) return max_len > a.prefix_len ? max_len - a.prefix_len : (int64_t)0;
        const int64_t win = a.W < max_len ? a.W + q - 1 + (a.S < max_len ? a.S : max_len) : max_len;
        return win < max_len ? win : max_len;
    };
    const bool prefix = op == CSA_OP_PREFIX_ATTN && a.prefix_len > 0;
    if (pl.few) {
        // (beside prompts most sequences may have none of these rows: no more than one round of blocks but for the cap
        // on a split's keys, which asks for a gigabyte of partials at most)
        const int64_t items = stream_items(B, n_few), one_round = 2 * (int64_t)sms / items;
        const int64_t fit = ((int64_t)1 << 30) / (few_rows * a.kv.H * (a.kv.d + 1) * 4), room = fit > 1 ? fit : 1;
        const Lengths lengths = op == CSA_OP_WINDOW_ATTN && a.W < max_len ? Lengths::window : Lengths::bound;
        pl.splits_few = stream_splits(items, keys(n_few), lengths, prefix, a.kv.d, sms, pl.many && room < kAsked ? room : kAsked,
                                      pl.many ? one_round : 256, &pl.few_groups);
    }
    if (pl.many) {
        int64_t blocks = B * ((n + tpb - 1) / tpb);
        if (blocks > a.rows / tpb + B) blocks = a.rows / tpb + B;
        pl.splits_many = tile_splits(blocks * a.kv.H_kv, keys(tpb), sms);
    }
    if (prefix) {
        pl.prefix_tile = a.rows * G > kFewPrefixRows;
        pl.splits_prefix = pl.prefix_tile
                               ? tile_splits(a.kv.H_kv * ((a.rows + tpb - 1) / tpb), a.prefix_len, sms)
                               : stream_splits(stream_items(1, a.rows), a.prefix_len, Lengths::same, true, a.kv.d, sms, kAsked,
                                               256, &pl.prefix_groups);
    }
    // partials of the prefix for all rows; of a class of sequences where it is split or has a prefix, those of
    // few rows by sequence (the rows of a prompt beside them need none) unless the call has fewer rows than that
    auto partials = [&](int splits, int64_t rows, int64_t per_seq) {
        PagedPartials q{};
        q.rows = rows;
        q.per_seq = (int)per_seq;
        q.slots = splits;
        return q;
    };
    if (pl.splits_prefix) pl.merge.prefix = partials(pl.splits_prefix, a.rows, 0);
    if (pl.few && (pl.splits_prefix || pl.splits_few > 1)) pl.merge.few = partials(pl.splits_few, few_rows, by_seq ? n_few : 0);
    if (pl.many && (pl.splits_prefix || pl.splits_many > 1)) pl.merge.many = partials(pl.splits_many, a.rows, 0);
    for (PagedPartials* q : {&pl.merge.prefix, &pl.merge.few, &pl.merge.many}) {
        const size_t heads = (size_t)q->rows * a.kv.H * q->slots;
        pl.any = pl.any || q->slots;
        q->o = reinterpret_cast<float*>(pl.total);
        pl.total += align256(heads * a.kv.d * 4);
        q->lse = reinterpret_cast<float*>(pl.total);
        pl.total += align256(heads * 4);
    }
    if (pl.total < 256) pl.total = 256;
    return pl;
}

int run_attn(const csa_kv_attn_args* a, int op, void* ws, size_t ws_bytes, cudaStream_t stream) {
    if (!a) return set_error(CSA_ERR_ARG, "args is NULL");
    int rc = check_attn(*a, op);
    if (rc) return rc;
    if (no_rows(*a)) return CSA_OK;
    if ((rc = check_cache(a->kv, true))) return rc;
    if (!a->q || !a->out) return set_error(CSA_ERR_ARG, "NULL pointer argument");
    if (!aligned16(a->q) || !aligned16(a->out) || (reinterpret_cast<uintptr_t>(a->lse) & 3u))
        return set_error(CSA_ERR_ARG, "q and out must be 16-byte, lse 4-byte aligned");
    const int64_t width = (int64_t)a->kv.H * a->kv.d;
    if (!stride_ok(a->q_stride, width) || !stride_ok(a->out_stride, width))
        return set_error(CSA_ERR_ARG, "q_stride = %lld, out_stride = %lld (multiples of 8, >= H d = %lld)",
                         (long long)a->q_stride, (long long)a->out_stride, (long long)width);
    PagedPlan pl = make_plan(*a, op);
    if (pl.any && (!ws || ws_bytes < pl.total || (reinterpret_cast<uintptr_t>(ws) & 255u)))
        return set_error(CSA_ERR_ARG, "workspace: %zu bytes at a 256-byte aligned address needed, %zu given", pl.total,
                         ws ? ws_bytes : (size_t)0);
    PagedAttnParams p{};
    p.kv = a->kv;
    p.rows = a->rows;
    p.max_n = (int)(a->max_n < a->rows ? a->max_n : a->rows);
    p.prefix_len = (int)a->prefix_len;
    p.key_begin = (int)a->prefix_len;
    p.W = op == CSA_OP_WINDOW_ATTN && a->W < 0x7fffffff ? (int)a->W : 0x7fffffff;
    p.S = (int)(a->S < kMaxTokens ? a->S : kMaxTokens);
    p.scale_log2 = a->scale * 1.44269504088896340736f;
    p.q = static_cast<const uint16_t*>(a->q);
    p.out = static_cast<uint16_t*>(a->out);
    p.lse = a->lse;
    p.q_stride = a->q_stride;
    p.out_stride = a->out_stride;
    // (without a stream launch the tile kernel takes every sequence, also one far shorter than max_n)
    p.few_rows = !pl.many ? (int64_t)1 << 40 : pl.few ? kFewRows : 0;
    for (PagedPartials* q : {&pl.merge.prefix, &pl.merge.few, &pl.merge.many}) {
        unsigned char* const base = static_cast<unsigned char*>(ws);
        q->o = q->slots ? reinterpret_cast<float*>(base + reinterpret_cast<size_t>(q->o)) : nullptr;
        q->lse = q->slots ? reinterpret_cast<float*>(base + reinterpret_cast<size_t>(q->lse)) : nullptr;
    }
    if ((rc = device_status(&p.status))) return rc;
    debug_fault_state(&p.debug_fault, &p.wait_ns);
    auto tile = [&](bool prefix, int splits, const PagedPartials& partials, bool pdl) {
        PagedAttnParams f = p;
        f.prefix_mode = prefix ? 1 : 0;
        if (prefix) f.key_begin = 0;
        f.splits = splits;
        f.part = partials;
        return launch_paged_tile(f, stream, pdl);
    };
    cudaError_t e = cudaSuccess;
    PagedStreamParts parts{};
    auto stream_part = [&](bool prefix, int splits, int groups, const PagedPartials& partials) {
        parts.part[parts.n++] = PagedStreamPart{prefix ? 1 : 0, prefix ? 0 : p.key_begin, splits, groups, 0, partials};
    };
    if (pl.splits_prefix && !pl.prefix_tile) stream_part(true, pl.splits_prefix, pl.prefix_groups, pl.merge.prefix);
    if (pl.few) stream_part(false, pl.splits_few, pl.few_groups, pl.merge.few);
    // the first launch starts when all work before it is done; the others, on the same inputs and with
    // partials and rows of their own, may overlap it
    int launched = 0;
    if (parts.n) {
        e = launch_paged_stream(p, parts, stream);
        ++launched;
    }
    if (e == cudaSuccess && pl.prefix_tile) e = tile(true, pl.splits_prefix, pl.merge.prefix, launched++ > 0);
    if (e == cudaSuccess && pl.many) e = tile(false, pl.splits_many, pl.merge.many, launched++ > 0);
    if (e == cudaSuccess && pl.any) e = launch_paged_combine(p, pl.merge, stream, true);
    if (e != cudaSuccess) return set_error(CSA_ERR_CUDA, "paged attention launch: %s", cudaGetErrorString(e));
    return CSA_OK;
}

}  // namespace

size_t paged_workspace_size(const csa_kv_attn_args* a, int op) {
    return check_attn(*a, op) ? 0 : make_plan(*a, op).total;
}

}  // namespace csa

using namespace csa;

extern "C" {

int csa_kv_append(const csa_kv_append_args* a, csa_stream_t stream) {
    if (!a) return set_error(CSA_ERR_ARG, "args is NULL");
    int rc = check_cache(a->kv, false);
    if (rc) return rc;
    if ((rc = check_rows(a->rows, a->max_n))) return rc;
    const csa_kv_cache& kv = a->kv;
    if (a->rot < 0 || a->rot > kv.d || a->rot % 16)
        return set_error(CSA_ERR_UNSUPPORTED, "rot = %d (supported: multiples of 16 from 0 to d)", a->rot);
    if (a->interleaved != 0 && a->interleaved != 1) return set_error(CSA_ERR_ARG, "interleaved = %d", a->interleaved);
    if (a->rows == 0 || a->max_n == 0) return CSA_OK;
    if ((rc = check_cache(kv, true))) return rc;
    if (!a->k || !a->v || (a->rot && !a->inv_freq)) return set_error(CSA_ERR_ARG, "NULL pointer argument");
    if ((a->q == nullptr) != (a->q_out == nullptr)) return set_error(CSA_ERR_ARG, "q and q_out go together");
    if (!aligned16(a->k) || !aligned16(a->v) || !aligned16(a->q) || !aligned16(a->q_out) ||
        (reinterpret_cast<uintptr_t>(a->inv_freq) & 3u))
        return set_error(CSA_ERR_ARG, "token arrays must be 16-byte, inv_freq 4-byte aligned");
    const int64_t wk = (int64_t)kv.H_kv * kv.d, wq = (int64_t)kv.H * kv.d;
    if (!stride_ok(a->k_stride, wk) || !stride_ok(a->v_stride, wk) ||
        (a->q && (!stride_ok(a->q_stride, wq) || !stride_ok(a->q_out_stride, wq))))
        return set_error(CSA_ERR_ARG, "row strides must be multiples of 8 and hold all heads");
    PagedAppendParams p{};
    p.kv = kv;
    p.rows = a->rows;
    p.max_n = a->max_n < a->rows ? a->max_n : a->rows;
    p.k = static_cast<const uint16_t*>(a->k);
    p.v = static_cast<const uint16_t*>(a->v);
    p.q = static_cast<const uint16_t*>(a->q);
    p.q_out = static_cast<uint16_t*>(a->q_out);
    p.k_stride = a->k_stride;
    p.v_stride = a->v_stride;
    p.q_stride = a->q_stride;
    p.q_out_stride = a->q_out_stride;
    p.inv_freq = a->inv_freq;
    p.rot = a->rot;
    p.interleaved = a->interleaved;
    if ((rc = device_status(&p.status))) return rc;
    const cudaError_t e = launch_paged_append(p, stream);
    return e == cudaSuccess ? CSA_OK : set_error(CSA_ERR_CUDA, "append launch: %s", cudaGetErrorString(e));
}

int csa_window_attn(const csa_kv_attn_args* args, void* ws, size_t ws_bytes, csa_stream_t stream) {
    return run_attn(args, CSA_OP_WINDOW_ATTN, ws, ws_bytes, stream);
}

int csa_prefix_attn(const csa_kv_attn_args* args, void* ws, size_t ws_bytes, csa_stream_t stream) {
    return run_attn(args, CSA_OP_PREFIX_ATTN, ws, ws_bytes, stream);
}

}  // extern "C"
