"""Cases of the paged key/value operators at the edges of their contracts: softmax weights far below a row's
largest one, waits that run out, queries of rows that no sequence has."""
import pytest
import torch

import compressed_sparse_kv_overlapped_b200 as csa
from tests.paged_harness import SENTINEL, Case, World

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


# Half a step of fp16's subnormal numbers, 2^-25, below the largest weight that the format holds at the kernel's
# scale: 2^15 (one that a weight never passes) in the stream kernel, 2^7 in the tile kernel, whose largest weight
# is 2^8 times that of the row's reference.
LOST = {"stream": 2.0 ** -40, "tile": 2.0 ** -32}


@pytest.mark.parametrize("dtype", [HF, BF])
@pytest.mark.parametrize("kernel", ["stream", "tile"])
@pytest.mark.parametrize("a,keys", [(2.1875, 65536), (2.1875, 8000), (1.640625, 4096)])
def test_weights_far_below_the_first_tokens(dtype, kernel, a, keys):
    """A first token that takes nearly all the weight and has no value, before a long uniform rest: each of the
    rest's weights is 2^-25.2 (2^-18.9) of the first one's, their sum is the whole output.

    Bound: relative h = eps / 2 for each rounding (weights, output), the fp32 errors of scores and sums, and an
    absolute LOST for a weight below the type's normal numbers (bf16 has the range of fp32)."""
    d, page, dev = 64, 256, "cuda"
    if kernel == "tile":  # 80 blocks of 64 tokens: the keys are not split
        B, H, H_kv, n, W, S = 1, 32, 8, 640, 1 << 20, 0
    else:                 # 512 blocks of one row; the window and the first token
        B, H, H_kv, n, W, S = 64, 8, 8, 1, min(keys, 8000), 1
    m = keys + 1
    pages = -(-m // page)
    g = torch.Generator(device=dev).manual_seed(11)
    kp = torch.zeros(pages, page, H_kv, d, dtype=dtype, device=dev)
    vp = (1 + 0.25 * torch.randn(pages, page, H_kv, d, generator=g, device=dev)).to(dtype)
    kp[0, 0], vp[0, 0] = a, 0
    table = torch.arange(pages, dtype=torch.int32, device=dev).expand(B, -1).contiguous()
    seqs = torch.tensor([[b * n, n, m] for b in range(B)], dtype=torch.int64, device=dev)
    kv = csa.PagedKV(kp, vp, table, seqs, H)
    q = torch.ones(B * n, H, d, dtype=dtype, device=dev)
    out, lse = torch.zeros_like(q), torch.zeros(B * n, H, dtype=torch.float32, device=dev)
    args = kv.window_args(q, out, W=W, S=S, max_n=n, max_len=m, lse=lse)
    kv.window_attn(args, kv.workspace(args))
    assert csa.csa_sync_status() == csa.CSA_OK

    # in 64 bits: every key of the rest has score 0, the first one d a scale
    first = torch.tensor(d * a * d ** -0.5, dtype=torch.float64, device=dev).exp()
    V = vp.double().flatten(0, 1)
    total = torch.cat((torch.zeros_like(V[:1]), V[1:m].cumsum(0)))        # [t]: V_1 + .. + V_t
    mag = torch.cat((torch.zeros_like(V[:1]), V[1:m].abs().cumsum(0)))
    pos = torch.arange(m - n, m, device=dev)
    before = (pos - W).clamp(min=0)                                       # tokens 1 .. before are out of the window
    rest = (pos - before).double()[:, None, None]
    sums = first + rest
    ref = (total[pos] - total[before]) / sums                             # [n, H_kv, d]
    A = (mag[pos] - mag[before]) / sums
    h, u = torch.finfo(dtype).eps / 2, 2.0 ** -24
    rel = 2 * ((d + 8) * 2 * u * (d * a * d ** -0.5) + 2.0 ** -20) + 4 * (rest + 1) * u
    lost = LOST[kernel] * rest * V.abs().max() if dtype == HF else 0.0
    tol = (h + rel) * A + h * ref.abs() + lost + (2.0 ** -25 if dtype == HF else 0.0)
    ref, tol = (x.repeat_interleave(H // H_kv, 1).repeat(B, 1, 1) for x in (ref, tol))
    e = (out.double() - ref).abs()
    assert (e <= tol).all(), f"off by {(e / tol).max():.1f} of the bound, {(e / ref.abs()).mean():.4f} of the value"
    ref_lse = sums.log()[..., 0].repeat(B, 1)
    assert ((lse.double() - ref_lse).abs() <= rel[..., 0].repeat(B, 1) + 2.0 ** -22 * ref_lse).all()


@pytest.mark.parametrize("seqs,prefix,direct", [
    ([(1, 300), (2, 90)], 0, True), ([(1, 9001)], 0, False), ([(90, 300), (64, 64)], 0, True), ([(130, 9001)], 0, False),
    ([(1, 200), (100, 250)], 0, True), ([(1, 700), (3, 612), (1, 650)], 600, False), ([(90, 900), (1, 700)], 600, False)])
@pytest.mark.parametrize("dtype,d", [(BF, 128), (HF, 64)])
def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_right(seqs, prefix, direct, dtype, d):
    """Every CTA's first wait for keys counts as run out while its copies are in flight: the kernels wind down and
    report it, blocks that write their rows directly leave them alone, and the same call is right afterwards."""
    w = World(Case(seqs, H=8, H_kv=2, d=d, page=32, dtype=dtype, W=1 << 20, prefix=prefix))
    args = w.args()
    ws = w.kv.workspace(args)
    try:
        csa.csa_debug_inject(1, 1_000_000)  # 1 ms limit
        for _ in range(3):
            w.attend(args, ws)
        assert csa.csa_sync_status() == csa.CSA_ERR_TIMEOUT
        if direct:
            assert (w.out == SENTINEL).all() and (w.lse == SENTINEL).all()
    finally:
        csa.csa_debug_inject(0, 0)
    w.attend(args, ws)
    assert csa.csa_sync_status() == csa.CSA_OK
    w.check()


@pytest.mark.parametrize("seqs,prefix", [([(1, 300), (2, 90), (0, 40)], 0), ([(90, 300), (64, 64)], 0), ([(1, 700), (3, 612), (0, 650)], 600),
                                         ([(90, 900), (1, 700)], 600)])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_queries_of_no_sequence_change_nothing(seqs, prefix, value):
    """Rows between the sequences, and those of a sequence that is left out, hold no numbers."""
    w = World(Case(seqs, H=8, H_kv=2, d=64, page=32, W=1 << 20, prefix=prefix, gap=3))
    mine = torch.zeros(w.rows, dtype=torch.bool)
    for row, n, _ in w.seq_rows:
        mine[row:row + n] = True
    w.q[~mine.to(w.q.device)] = value
    w.attend()
    assert csa.csa_sync_status() == csa.CSA_OK
    w.check()


@pytest.mark.parametrize("prefix", [0, 600])
def test_empty_partials_are_not_used(prefix):
    """Sequences far below the bound on lengths leave most splits empty: the workspace holds NaN there, which is neither
    read nor weighed."""
    w = World(Case([(1, 700), (2, 950), (1, 601), (1, 640)], H=8, H_kv=1, d=128, page=64, W=1 << 20, prefix=prefix))
    args = w.kv.prefix_args(w.q, w.out, prefix_len=prefix, max_n=2, lse=w.lse, scale=w.scale) if prefix else \
        w.kv.window_args(w.q, w.out, W=1 << 20, max_n=2, lse=w.lse, scale=w.scale)
    args.max_len = 60000
    args.kv.max_pages = 1024
    w.table = torch.nn.functional.pad(w.table, (0, 1024 - w.table.shape[1]), value=-1)
    args.kv.page_table = w.table.data_ptr()
    ws = w.kv.workspace(args)
    assert ws.numel() > 4 * 8 * 129 * 4 * 8, "at least eight splits"
    ws.fill_(255)  # NaN in fp32
    w.attend(args, ws)
    assert csa.csa_sync_status() == csa.CSA_OK
    w.check()


@pytest.mark.parametrize("dtype,d", [(BF, 128), (HF, 64)])
@pytest.mark.parametrize("chunk", [300, 1300])
def test_one_long_row_in_a_wide_batch_beside_a_prompt(dtype, d, chunk):
    """The long row's keys are cut, the prompt's rows are written directly.  Partials are held by the rows of the call
    (399, fewer than eight of each sequence) or by sequence (1,399)."""
    c = Case([(1, 50 + i) for i in range(98)] + [(1, 9000), (chunk, chunk + 100)], H=8, H_kv=1, d=d, page=64, dtype=dtype, W=1 << 20)
    w = World(c)
    args = w.args()
    ws = w.kv.workspace(args)
    assert ws.numel() >= 4 * min(w.rows, 100 * 8) * 8 * (d + 1) * 4, "four splits"
    w.attend(args, ws)
    assert csa.csa_sync_status() == csa.CSA_OK
    w.check()


@pytest.mark.parametrize("prefix", [0, 100])
def test_module_functions_make_the_same_calls(prefix):
    """csa_kv_append, csa_window_attn and csa_prefix_attn of the module, beside the methods of PagedKV."""
    c = Case([(2, 3000), (70, 300)], H=8, H_kv=2, d=64, page=32, W=1 << 20, prefix=prefix)
    results = []
    for methods in (True, False):
        w = World(c, all_live=True)
        g = torch.Generator().manual_seed(2)
        k, v = (torch.randn(w.rows, c.H_kv, c.d, generator=g).to(c.dtype).cuda() for _ in range(2))
        turned = torch.empty_like(w.q)
        inv = (10000.0 ** (-torch.arange(0, c.d, 2) / c.d)).float().cuda()
        a = w.kv.append_args(k, v, w.q, turned, max_n=w.max_n, inv_freq=inv)
        kw = dict(max_n=w.max_n, max_len=w.max_len, lse=w.lse, scale=w.scale)
        b = w.kv.prefix_args(turned, w.out, prefix_len=prefix, **kw) if prefix else w.kv.window_args(turned, w.out, W=c.W, **kw)
        ws = w.kv.workspace(b)
        if methods:
            w.kv.append(a)
            w.attend(b, ws)
        else:
            csa.csa_kv_append(a)
            (csa.csa_prefix_attn if prefix else csa.csa_window_attn)(b, ws)
        assert csa.csa_sync_status() == csa.CSA_OK
        results.append([w.kp, w.vp, turned, w.out, w.lse])
    for x, y in zip(*results):
        assert torch.equal(x.nan_to_num(9.0), y.nan_to_num(9.0))
    assert not results[0][3].isnan().any()
