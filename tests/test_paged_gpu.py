"""The paged key/value operators against a plain 64-bit implementation: appends with rotation, windowed
attention with first tokens, shared-prefix attention, and the three together."""
import math

import pytest
import torch

import compressed_sparse_kv_overlapped_b200 as csa
from tests.paged_harness import SENTINEL, Case, World, rotated

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


def run(c, **kw):
    w = World(c, **kw)
    w.attend()
    assert csa.csa_sync_status() == csa.CSA_OK
    w.check()
    return w


# ------------------------------------------------------------------------------------- window

STEPS = [(1, 1), (1, 2), (1, 15), (1, 16), (1, 17), (1, 128), (1, 129), (1, 133), (1, 500), (0, 40), (1, 1000)]


@pytest.mark.parametrize("dtype,d", [(BF, 64), (BF, 128), (HF, 64), (HF, 128)])
@pytest.mark.parametrize("page,W,S", [(16, 128, 4), (64, 1, 0), (256, 37, 16), (32, 1 << 20, 0), (128, 100, 130)])
def test_window_single_tokens(dtype, d, page, W, S):
    run(Case(STEPS, H=8, H_kv=2, d=d, page=page, dtype=dtype, W=W, S=S))


@pytest.mark.parametrize("H,H_kv", [(1, 1), (3, 1), (5, 5), (12, 2), (16, 1), (20, 1), (32, 1), (40, 2), (64, 1), (128, 2)])
def test_window_head_layouts(H, H_kv):
    run(Case([(1, 70), (2, 300), (1, 31)], H=H, H_kv=H_kv, d=128, page=32, W=150, S=3, heads_first=True))


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("seqs", [[(2, 2), (3, 130), (4, 555), (1, 700)], [(5, 5), (7, 64), (16, 200)], [(1, 1), (33, 40), (17, 300)]])
@pytest.mark.parametrize("W,S", [(1, 0), (2, 1), (64, 4), (1 << 30, 0), (100, 1000)])
def test_window_few_tokens(dtype, seqs, W, S):
    run(Case(seqs, H=8, H_kv=2, d=64, page=16, dtype=dtype, W=W, S=S, gap=2, pad_cols=16))


PROMPTS = [[(1, 1), (65, 65), (300, 300)], [(128, 128), (129, 1000), (0, 0), (255, 256)], [(513, 900)]]


@pytest.mark.parametrize("dtype,d,H,H_kv", [(BF, 128, 8, 1), (HF, 128, 4, 4), (BF, 64, 14, 2), (HF, 64, 6, 2), (BF, 128, 3, 1)])
@pytest.mark.parametrize("seqs", PROMPTS, ids=["short", "mixed", "chunk"])
@pytest.mark.parametrize("page,W,S", [(16, 128, 4), (64, 1 << 20, 0), (256, 50, 20), (128, 400, 300)])
def test_window_prompts(dtype, d, H, H_kv, seqs, page, W, S):
    run(Case(seqs, H=H, H_kv=H_kv, d=d, page=page, dtype=dtype, W=W, S=S, gap=1))


@pytest.mark.parametrize("n", [1, 2, 40])
def test_window_long_rows_are_split(n):
    """Few blocks over many keys: the keys are split and the partials merged."""
    w = run(Case([(n, 9001), (n, 4000)], H=8, H_kv=1, d=128, page=64, W=1 << 20, S=0))
    assert w.kv.workspace(w.args()).numel() > 256


def test_window_large_scores():
    """Scores far apart (one key takes all the weight) and far from zero."""
    run(Case([(1, 300), (40, 333)], H=4, H_kv=2, d=128, W=200, S=2, q_std=30.0))
    run(Case([(1, 300), (40, 333)], H=4, H_kv=2, d=128, dtype=HF, W=200, S=2, q_std=30.0))


def test_window_without_lse_and_default_scale():
    w = World(Case([(1, 50), (9, 90)], W=20, S=1))
    a = w.kv.window_args(w.q, w.out, W=20, S=1, max_n=9)
    w.kv.window_attn(a, w.kv.workspace(a))
    w2 = World(Case([(1, 50), (9, 90)], W=20, S=1))
    w2.attend()
    assert torch.equal(w.out, w2.out) and (w.lse == SENTINEL).all()


# ------------------------------------------------------------------------------------- prefix

@pytest.mark.parametrize("dtype,d,H,H_kv", [(BF, 64, 8, 2), (HF, 128, 8, 1), (BF, 128, 32, 2), (HF, 64, 5, 5)])
@pytest.mark.parametrize("prefix,page", [(1, 16), (16, 16), (100, 32), (1000, 64), (2049, 256)])
def test_prefix(dtype, d, H, H_kv, prefix, page):
    seqs = [(1, prefix + 1), (2, prefix + 2), (1, prefix + 40), (0, prefix), (3, prefix + 333), (1, prefix + 64)]
    run(Case(seqs, H=H, H_kv=H_kv, d=d, page=page, dtype=dtype, prefix=prefix, gap=1))


def test_prefix_wide_batch():
    run(Case([(1 + b % 2, 700 + 2 + b % 19) for b in range(70)], H=16, H_kv=2, d=128, page=64, prefix=700))


def test_prefix_with_prompts_behind_it():
    run(Case([(150, 500 + 150), (40, 500 + 300)], H=8, H_kv=2, d=128, page=16, prefix=500))


def test_prefix_zero_is_causal_attention():
    c = Case([(1, 90), (5, 400)], H=8, H_kv=2, d=64)
    w = World(c)
    a = w.kv.prefix_args(w.q, w.out, prefix_len=0, max_n=5, max_len=400, lse=w.lse)
    w.kv.prefix_attn(a, w.kv.workspace(a))
    assert csa.csa_sync_status() == csa.CSA_OK
    w.check()


# ------------------------------------------------------------------------------------- append

def append_world(c, rot, interleaved, with_q=True, in_place=False, device="cuda"):
    """Runs an append into empty (sentinel) pools and checks every element of pools and queries."""
    w = World(c, device=device, all_live=True)
    w.kp.fill_(SENTINEL)
    w.vp.fill_(SENTINEL)
    g = torch.Generator().manual_seed(c.seed + 5)
    width = (c.H + 2 * c.H_kv) * c.d
    qkv = torch.randn(w.rows, width, generator=g).to(c.dtype).to(device)
    src = qkv.clone()
    q, k, v = (x.unflatten(1, (-1, c.d)) for x in qkv.split([c.H * c.d, c.H_kv * c.d, c.H_kv * c.d], dim=1))
    q_out = q if in_place else torch.full((w.rows, c.H, c.d), SENTINEL, dtype=c.dtype, device=device)
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float32) / max(rot, 1))
    a = w.kv.append_args(k, v, q if with_q else None, q_out if with_q else None, max_n=w.max_n,
                         inv_freq=inv.to(device), interleaved=interleaved)
    w.kv.append(a)
    assert csa.csa_sync_status() == csa.CSA_OK
    sq, sk, sv = (x.unflatten(1, (-1, c.d)).cpu() for x in src.split([c.H * c.d, c.H_kv * c.d, c.H_kv * c.d], dim=1))
    kp, vp = w.kp.cpu(), w.vp.cpu()
    want_k, want_v = torch.full_like(kp, SENTINEL).double(), torch.full_like(vp, SENTINEL)
    want_q = sq.double() if in_place else torch.full_like(sq, SENTINEL).double()
    for b, (row, n, m) in enumerate(w.seq_rows):
        pos = torch.arange(m - n, m)
        pg, sl = w.table_cpu[b, pos // c.page].long(), pos % c.page
        want_k[pg, sl] = rotated(sk[row:row + n], pos, inv, interleaved)
        want_v[pg, sl] = sv[row:row + n]
        want_q[row:row + n] = rotated(sq[row:row + n], pos, inv, interleaved)
    assert torch.equal(vp, want_v)
    # one rounding of the result, and products and sums in fp32 of cos and sin good to 2^-22
    h = torch.finfo(c.dtype).eps / 2
    pairs = [(kp.double(), want_k, sk.abs().max())] + ([(q_out.double().cpu(), want_q, sq.abs().max())] if with_q else [])
    for got, want, src_max in pairs:
        sub = 2.0 ** -25 if c.dtype == HF else 0.0
        assert ((got - want).abs() <= h * want.abs() + 2.0 ** -20 * src_max.double() + sub).all()
    if not with_q:
        assert (q_out == SENTINEL).all()
    return w


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("d,rot,interleaved", [(64, 64, False), (64, 32, True), (128, 128, True), (128, 48, False), (128, 0, False)])
@pytest.mark.parametrize("seqs", [[(1, 1)], [(1, 77), (0, 5), (1, 1000), (1, 16)], [(40, 40), (9, 300), (3, 16)]], ids=["one", "step", "prompts"])
def test_append(dtype, d, rot, interleaved, seqs):
    append_world(Case(seqs, H=6, H_kv=3, d=d, page=16, dtype=dtype, gap=1), rot, interleaved)


@pytest.mark.parametrize("heads_first", [False, True])
def test_append_layouts_in_place_and_without_queries(heads_first):
    c = Case([(5, 200), (1, 64), (33, 33)], H=4, H_kv=4, d=128, page=64, heads_first=heads_first)
    append_world(c, 64, False, in_place=True)
    append_world(c, 64, True, with_q=False)


def test_append_at_far_positions():
    """Positions near 2^20: the angle needs more than 32 bits."""
    page, m = 256, (1 << 20) - 3
    dev = "cuda"
    kp = torch.zeros(2, page, 1, 64, dtype=BF, device=dev)
    vp = torch.zeros_like(kp)
    table = torch.full((1, (m + page - 1) // page), -1, dtype=torch.int32, device=dev)
    table[0, -1] = 1
    seqs = torch.tensor([[0, 4, m]], dtype=torch.int64, device=dev)
    kv = csa.PagedKV(kp, vp, table, seqs, 2)
    k, q = torch.randn(4, 1, 64, device=dev).to(BF), torch.randn(4, 2, 64, device=dev).to(BF)
    inv = (10000.0 ** (-torch.arange(0, 64, 2) / 64)).float().to(dev)
    q_out = torch.empty_like(q)
    kv.append(kv.append_args(k, k.clone(), q, q_out, max_n=4, inv_freq=inv))
    assert csa.csa_sync_status() == csa.CSA_OK
    pos = torch.arange(m - 4, m)
    want = rotated(q.cpu(), pos, inv.cpu(), False)
    assert ((q_out.double().cpu() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -20 * 8).all()
    want = rotated(k.cpu(), pos, inv.cpu(), False)
    at = pos % page
    assert ((kp[1, at].double().cpu() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -20 * 8).all()


# ------------------------------------------------------------------------------------- errors on the device

def test_bad_tables_are_reported_and_skipped():
    c = Case([(1, 40), (1, 60), (1, 50), (1, 70)], W=1 << 20)
    w = World(c)
    w.seqs[1, 2] = w.kv.kv.max_pages * c.page + 1   # longer than its row of the table
    w.seqs[2, 0] = w.rows                           # rows outside the token arrays
    w.attend()
    assert csa.csa_sync_status() == csa.CSA_ERR_INDEX
    w.check(skip=(1, 2))
    w = World(c)
    w.seqs[0, 1] = -1
    w.seqs[3, 1] = 71                               # more new tokens than tokens, and than max_n
    w.attend()
    assert csa.csa_sync_status() == csa.CSA_ERR_INDEX
    w.check(skip=(0, 3))


def test_bad_page_is_reported_and_the_other_sequences_are_right():
    c = Case([(1, 40), (33, 60)], W=1 << 20)
    for bad in (-1, 1 << 20):
        w = World(c)
        w.table[0, 1] = bad
        w.attend()
        assert csa.csa_sync_status() == csa.CSA_ERR_INDEX
        w.out[:1] = SENTINEL
        w.lse[:1] = SENTINEL
        w.check(skip=(0,))


def test_prefix_behind_a_sequences_tokens_is_reported():
    c = Case([(1, 300), (1, 257), (1, 280)], prefix=256)
    w = World(c)
    w.seqs[1, 2] = 256  # its new token would lie inside the prefix
    w.attend()
    assert csa.csa_sync_status() == csa.CSA_ERR_INDEX
    w.check(skip=(1,))


def test_append_skips_a_missing_page():
    c = Case([(1, 40), (1, 20)], H=2, H_kv=1, d=64)
    w = World(c, all_live=True)
    w.table[0, 2] = -1
    before = w.kp.clone()
    k = torch.ones(2, 1, 64, dtype=BF, device="cuda")
    w.kv.append(w.kv.append_args(k, k, max_n=1))
    assert csa.csa_sync_status() == csa.CSA_ERR_INDEX
    changed = (w.kp != before) & ~(w.kp.isnan() & before.isnan())
    assert changed.any(-1).sum() <= 1 and (w.kp[w.table_cpu[1, 1].item(), 19 - 16] == 1).all()


# ------------------------------------------------------------------------------------- together

def test_decode_loop_append_then_window():
    """A prompt and then single tokens through append and window attention, in one captured graph that
    is replayed, against the definition over the whole history."""
    H, H_kv, d, page, W, S, n0, steps = 8, 2, 64, 16, 48, 3, 37, 30
    dev, g = "cuda", torch.Generator().manual_seed(3)
    total = n0 + steps
    inv = (10000.0 ** (-torch.arange(0, d, 2) / d)).float().to(dev)
    pages = (total + page - 1) // page
    kp = torch.full((pages, page, H_kv, d), math.nan, dtype=BF, device=dev)
    vp = kp.clone()
    table = torch.randperm(pages, generator=g).to(torch.int32)[None].to(dev)
    seqs = torch.tensor([[0, n0, n0]], dtype=torch.int64, device=dev)
    kv = csa.PagedKV(kp, vp, table, seqs, H)
    q, k, v = (torch.randn(total, h, d, generator=g).to(BF).to(dev) for h in (H, H_kv, H_kv))
    q_rot, out = torch.empty_like(q), torch.empty_like(q)
    a = kv.append_args(k[:n0], v[:n0], q[:n0], q_rot[:n0], max_n=n0, inv_freq=inv)
    kv.append(a)
    b = kv.window_args(q_rot[:n0], out[:n0], W=W, S=S, max_n=n0, max_len=n0)
    kv.window_attn(b, kv.workspace(b))
    qs, ks, vs, qr, o = (torch.empty_like(x[:1]) for x in (q, k, v, q, q))
    a = kv.append_args(ks, vs, qs, qr, max_n=1, inv_freq=inv)
    b = kv.window_args(qr, o, W=W, S=S, max_n=1, max_len=total)
    ws = kv.workspace(b)
    seqs.copy_(torch.tensor([[0, 1, n0]]))
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        seqs[:, 2] += 1
        kv.append(a)
        kv.window_attn(b, ws)
    for t in range(n0, total):
        qs.copy_(q[t:t + 1]), ks.copy_(k[t:t + 1]), vs.copy_(v[t:t + 1])
        graph.replay()
        out[t:t + 1].copy_(o)
        q_rot[t:t + 1].copy_(qr)
    assert csa.csa_sync_status() == csa.CSA_OK
    # the definition over the stored (rounded) keys and queries
    from tests.paged_harness import reference
    pos = torch.arange(total)
    at = table[0, pos // page].long().cpu(), pos % page
    K, V = kp.cpu()[at].double(), vp.cpu()[at].double()
    h = 2.0 ** -8
    want = rotated(k.cpu(), pos, inv.cpu(), False)
    assert ((K - want).abs() <= h * want.abs() + 2.0 ** -17).all()
    ref, _, tol, _ = reference(Case([(total, total)], H=H, H_kv=H_kv, d=d, W=W, S=S), q_rot.double().cpu(), K, V, 0, d ** -0.5)
    assert ((out.double().cpu() - ref).abs() <= tol).all()


def test_prefix_equals_plain_causal_attention():
    """The same batch through csa_prefix_attn and through csa_window_attn without a window."""
    c = Case([(1, 600 + i) for i in range(1, 40)], H=16, H_kv=2, d=128, page=32, prefix=600)
    w = run(c, all_live=True)
    out, lse = w.out.clone(), w.lse.clone()
    a = w.kv.window_args(w.q, w.out, W=1 << 20, max_n=1, max_len=w.max_len, lse=w.lse, scale=w.scale)
    w.kv.window_attn(a, w.kv.workspace(a))
    assert csa.csa_sync_status() == csa.CSA_OK
    w.check()
    assert (lse - w.lse).abs().max() < 1e-5 and (out.float() - w.out.float()).abs().max() < 0.05


def test_another_stream_and_two_calls_at_once():
    """Calls on two streams with a workspace each."""
    cs = [Case([(1, 5000), (1, 3000)], H=8, H_kv=1, d=128, page=64, W=1 << 20, seed=s) for s in (1, 2)]
    ws = [World(c) for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    args = [w.args() for w in ws]
    spaces = [w.kv.workspace(a) for w, a in zip(ws, args)]
    torch.cuda.synchronize()
    for _ in range(5):
        for w, s, a, sp in zip(ws, streams, args, spaces):
            w.attend(a, sp, s)
    torch.cuda.synchronize()
    assert csa.csa_sync_status() == csa.CSA_OK
    for w in ws:
        w.check()


def test_results_do_not_change_from_call_to_call():
    c = Case([(1, 9000), (2, 700)], H=8, H_kv=2, d=128, page=64, W=1 << 20)
    w = run(c)
    out, lse = w.out.clone(), w.lse.clone()
    for _ in range(3):
        w.attend()
        assert torch.equal(out, w.out) and torch.equal(lse, w.lse)


# ------------------------------------------------------------------------------------- calls off the usual path

@pytest.mark.parametrize("n,m", [(1, 300), (5, 40), (8, 8)])
def test_one_sequence_far_below_the_bound_of_n(n, m):
    """max_n only bounds: a captured call is made for the longest prompt and replayed for a short one."""
    w = World(Case([(n, m)], H=8, H_kv=1, d=128, page=32, W=100, S=2))
    w.max_n, w.max_len = 500, 2000
    w.attend()
    assert csa.csa_sync_status() == csa.CSA_OK
    w.check()


@pytest.mark.parametrize("dtype,d", [(BF, 128), (HF, 64)])
@pytest.mark.parametrize("W,S,prefix", [(1 << 20, 0, 0), (3000, 40, 0), (0, 0, 700)])
def test_single_tokens_and_prompts_in_one_call(dtype, d, W, S, prefix):
    seqs = [(1, 9000), (300, 1100), (0, 800), (2, 5000), (130, 6000), (1, 701), (64, 900)]
    run(Case(seqs, H=8, H_kv=1, d=d, page=64, dtype=dtype, W=W or 1 << 20, S=S, prefix=prefix, gap=1))


@pytest.mark.parametrize("prefix", [0, 300])
def test_lengths_beyond_their_bound(prefix):
    """max_len sizes the split of long rows; the keys come from the sequences' own lengths."""
    for seqs in ([(1, 3000), (1, 700)], [(200, 3000), (1, 900)]):
        w = World(Case(seqs, H=8, H_kv=2, d=128, page=64, W=1 << 20, prefix=prefix))
        w.max_len = 1000
        w.attend()
        assert csa.csa_sync_status() == csa.CSA_OK
        w.check()


@pytest.mark.parametrize("prefix", [0, 1000])
def test_captured_calls_share_a_workspace(prefix):
    """Two graphs over one workspace, replayed in turn with changed queries, lengths and tables."""
    cs = [Case([(1, 4000), (1, 1500), (140, 2500)], H=16, H_kv=2, d=128, page=64, W=1 << 20, prefix=prefix, seed=s)
          for s in (3, 4)]
    ws = [World(c) for c in cs]
    args = [w.args() for w in ws]
    space = max((w.kv.workspace(a) for w, a in zip(ws, args)), key=lambda t: t.numel())
    graphs = []
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    for w, a in zip(ws, args):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            w.attend(a, space)
        graphs.append(g)
    for _ in range(3):
        for w, g in zip(ws, graphs):
            w.q_full.copy_(w.q_full.roll(1, 0))
            w.out_full.fill_(SENTINEL), w.lse.fill_(SENTINEL)
            g.replay()
    torch.cuda.synchronize()
    assert csa.csa_sync_status() == csa.CSA_OK
    for w in ws:
        w.check()


def test_pages_four_gigabytes_apart():
    """Offsets in the pools pass 32 bits: pages 2^31 elements apart, appended to and attended."""
    dev, H, H_kv, d, page, n, m = "cuda", 8, 2, 128, 16, 40, 40
    step = 1 << 31
    size = 2 * step + page * H_kv * d
    pools = []
    for _ in range(2):
        flat = torch.empty(size, dtype=BF, device=dev)
        pools.append(flat.as_strided((3, page, H_kv, d), (step, H_kv * d, d, 1)))
    table = torch.tensor([[2, 0, 1]], dtype=torch.int32, device=dev)
    seqs = torch.tensor([[0, n, m]], dtype=torch.int64, device=dev)
    kv = csa.PagedKV(*pools, table, seqs, H)
    g = torch.Generator().manual_seed(9)
    q, k, v = (torch.randn(n, h, d, generator=g).to(BF).to(dev) for h in (H, H_kv, H_kv))
    kv.append(kv.append_args(k, v, max_n=n))
    from tests.paged_harness import reference
    for max_n in (n, 8):
        rows = slice(n - max_n, n)
        seqs.copy_(torch.tensor([[0, max_n, m]]))
        out = torch.zeros(max_n, H, d, dtype=BF, device=dev)
        a = kv.window_args(q[rows], out, W=1 << 20, max_n=max_n, max_len=m)
        kv.window_attn(a, kv.workspace(a))
        assert csa.csa_sync_status() == csa.CSA_OK
        ref, _, tol, _ = reference(Case([(max_n, m)], H=H, H_kv=H_kv, d=d), q[rows].double().cpu(), k.double().cpu(),
                                   v.double().cpu(), m - max_n, d ** -0.5)
        assert ((out.double().cpu() - ref).abs() <= tol).all()


def test_a_workspace_too_small_and_a_wrong_stream_are_refused():
    w = World(Case([(1, 9001)], H=8, H_kv=1, d=128, page=64, W=1 << 20))
    a = w.args()
    ws = w.kv.workspace(a)
    with pytest.raises(RuntimeError, match="workspace"):
        w.kv.window_attn(a, ws[:ws.numel() - 256])
    assert (w.out == SENTINEL).all()


@pytest.mark.parametrize("n", [1, 90])
def test_a_missing_page_counts_as_zeros(n):
    """Keys and values of a page number out of range are zeros: score 0, no value (few rows and many)."""
    c = Case([(n, 300), (n, 280)], H=8, H_kv=2, d=64, page=32, W=1 << 20)
    w = World(c)
    w.table[0, 2] = w.kp.shape[0] + 5
    w.K[0][64:96] = 0
    w.V[0][64:96] = 0
    w.attend()
    assert csa.csa_sync_status() == csa.CSA_ERR_INDEX
    w.check()


@pytest.mark.parametrize("n", [3, 90])
def test_a_query_of_nan_stays_alone(n):
    c = Case([(n, 300), (n, 280)], H=8, H_kv=2, d=128, page=32, W=100, S=3)
    w = World(c)
    w.q[1, 3] = math.nan
    w.attend()
    assert csa.csa_sync_status() == csa.CSA_OK
    assert w.out[1, 3].isnan().all() and w.lse[1, 3].isnan()
    w.q[1, 3] = 1.0
    out, lse = w.out.clone(), w.lse.clone()
    w.attend()
    keep = torch.ones(w.rows, c.H, dtype=torch.bool, device="cuda")
    keep[1, 3] = False
    assert torch.equal(out[keep], w.out[keep]) and torch.equal(lse[keep], w.lse[keep])
    w.check()


@pytest.mark.parametrize("seed", range(4))
def test_split_plans_of_many_batches(seed):
    """Batches of many widths and lengths, so that every cut of long rows meets short and empty sequences."""
    g = torch.Generator().manual_seed(50 + seed)
    def pick(*a):
        return a[int(torch.randint(len(a), (1,), generator=g))]
    for _ in range(6):
        B, top = pick(1, 3, 9, 40), pick(40, 700, 5000)
        seqs = []
        for _ in range(B):
            n = pick(0, 1, 1, 1, 2, 4)
            m = max(n, int(torch.randint(1, top + 1, (1,), generator=g)))
            seqs.append((n, m))
        seqs[0] = (1, top)
        H_kv = pick(1, 2)
        prefix = pick(0, 0, 17, 600)
        seqs = [(n, m + prefix) for n, m in seqs]
        run(Case(seqs, H=H_kv * pick(1, 3, 8), H_kv=H_kv, d=pick(64, 128), page=pick(16, 64), dtype=pick(BF, HF),
                 W=1 << 20 if prefix else pick(30, 2000, 1 << 20), S=0 if prefix else pick(0, 5), prefix=prefix, seed=seed))
