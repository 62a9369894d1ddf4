"""The paged key/value operators on a machine without a GPU: struct layouts, refusals before any launch,
workspace sizes, and the plain visibility rule against a literal loop."""
import ctypes
import os
import subprocess

import pytest
import torch

import compressed_sparse_kv_overlapped_b200 as csa

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(csa.LIB_PATH):
        csa.build()
    return csa.lib()


def cache(**kw):
    kv = csa.csa_kv_cache()
    for k, v in dict(H=8, H_kv=2, d=64, type=csa.CSA_KV_BF16, page_size=16, B=2, num_pages=10, max_pages=5,
                     page_stride=16 * 2 * 64, slot_stride=128, head_stride=64, k_pages=256, v_pages=256, page_table=256,
                     seqs=256, **{}).items():
        setattr(kv, k, kw.get(k, v))
    return kv


def append_args(kv=None, **kw):
    a = csa.csa_kv_append_args()
    a.kv = kv or cache()
    for k, v in dict(rows=4, max_n=2, k=256, v=256, q=256, q_out=256, k_stride=128, v_stride=128, q_stride=512,
                     q_out_stride=512, inv_freq=256, rot=64, interleaved=0).items():
        setattr(a, k, kw.get(k, v))
    return a


def attn_args(kv=None, **kw):
    a = csa.csa_kv_attn_args()
    a.kv = kv or cache()
    for k, v in dict(rows=4, max_n=2, max_len=80, W=16, S=4, prefix_len=0, scale=0.125, reserved=0, q=256, out=256,
                     lse=None, q_stride=512, out_stride=512).items():
        setattr(a, k, kw.get(k, v))
    return a


def test_struct_layouts_match_header(tmp_path):
    prog = tmp_path / "sizes.c"
    fields = [("csa_kv_cache", "num_pages"), ("csa_kv_cache", "seqs"), ("csa_kv_append_args", "inv_freq"),
              ("csa_kv_append_args", "interleaved"), ("csa_kv_attn_args", "scale"), ("csa_kv_attn_args", "out_stride")]
    types = ["csa_kv_cache", "csa_kv_append_args", "csa_kv_attn_args", "csa_kv_seq"]
    exprs = [f"sizeof({t})" for t in types] + [f"offsetof({t}, {f})" for t, f in fields]
    prog.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "csa.h"\nint main(void){'
                    + "".join(f'printf("%zu ", {e});' for e in exprs) + "return 0;}\n")
    exe = tmp_path / "sizes"
    subprocess.run(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), str(prog), "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True).stdout.split()]
    assert got == [ctypes.sizeof(csa.csa_kv_cache), ctypes.sizeof(csa.csa_kv_append_args),
                   ctypes.sizeof(csa.csa_kv_attn_args), 24] + [getattr(getattr(csa, t), f).offset for t, f in fields]


ARG, UNS = csa.CSA_ERR_ARG, csa.CSA_ERR_UNSUPPORTED
BAD_CACHES = [
    (dict(d=96), UNS, "d = 96"), (dict(type=2), UNS, "type = 2"), (dict(H=0), UNS, "H = 0"), (dict(H=300, H_kv=300), UNS, "H = 300"),
    (dict(H_kv=3), ARG, "does not divide"), (dict(H_kv=0), ARG, "does not divide"), (dict(H=130, H_kv=1), UNS, "on a key head"),
    (dict(page_size=8), UNS, "page_size"), (dict(page_size=48), UNS, "page_size"), (dict(page_size=512), UNS, "page_size"),
    (dict(B=0), ARG, "B = 0"), (dict(num_pages=0), ARG, "num_pages"), (dict(max_pages=1 << 27), UNS, "max_pages"),
    (dict(page_stride=12), ARG, "page_stride"), (dict(slot_stride=0), ARG, "slot_stride"), (dict(head_stride=-64), ARG, "head_stride"),
]
BAD_POINTERS = [(dict(k_pages=None), ARG, "NULL"), (dict(seqs=None), ARG, "NULL"), (dict(page_table=None), ARG, "NULL"),
                (dict(v_pages=264), ARG, "aligned"), (dict(page_table=258), ARG, "aligned"), (dict(seqs=260), ARG, "aligned")]


@pytest.mark.parametrize("kw,code,word", BAD_CACHES + BAD_POINTERS)
def test_every_call_checks_the_cache(lib, kw, code, word):
    kv = cache(**kw)
    assert lib.csa_kv_append(ctypes.byref(append_args(kv)), None) == code and word in csa.csa_last_error()
    assert lib.csa_window_attn(ctypes.byref(attn_args(kv)), 256, 1 << 30, None) == code and word in csa.csa_last_error()
    a = attn_args(kv, W=0, S=0, prefix_len=8)
    assert lib.csa_prefix_attn(ctypes.byref(a), 256, 1 << 30, None) == code and word in csa.csa_last_error()
    if (kw, code, word) in BAD_CACHES:
        assert csa.csa_workspace_size(csa.CSA_OP_PREFIX_ATTN, a) == 0


@pytest.mark.parametrize("kw,code,word", [
    (dict(rot=8), UNS, "rot = 8"), (dict(rot=80), UNS, "rot = 80"), (dict(rot=-16), UNS, "rot"), (dict(interleaved=2), ARG, "interleaved"),
    (dict(rows=-1), ARG, "rows"), (dict(rows=1 << 30), ARG, "rows"), (dict(max_n=-1), ARG, "max_n"), (dict(k=None), ARG, "NULL"),
    (dict(inv_freq=None), ARG, "NULL"), (dict(q_out=None), ARG, "go together"), (dict(q=None), ARG, "go together"),
    (dict(v=264), ARG, "aligned"), (dict(inv_freq=258), ARG, "aligned"), (dict(k_stride=120), ARG, "strides"),
    (dict(q_stride=516), ARG, "strides"), (dict(q_out_stride=504), ARG, "strides")])
def test_append_refusals(lib, kw, code, word):
    assert lib.csa_kv_append(ctypes.byref(append_args(**kw)), None) == code and word in csa.csa_last_error()
    assert lib.csa_kv_append(None, None) == ARG


@pytest.mark.parametrize("kw,code,word", [
    (dict(W=0), ARG, "W = 0"), (dict(S=-1), ARG, "S = -1"), (dict(prefix_len=16), ARG, "prefix_len"), (dict(scale=0.0), ARG, "scale"),
    (dict(scale=-1.0), ARG, "scale"), (dict(scale=float("nan")), ARG, "scale"), (dict(scale=float("inf")), ARG, "scale"),
    (dict(reserved=1), ARG, "reserved"), (dict(max_len=-1), ARG, "max_len"), (dict(rows=-1), ARG, "rows"), (dict(q=None), ARG, "NULL"),
    (dict(out=None), ARG, "NULL"), (dict(q=264), ARG, "aligned"), (dict(lse=258), ARG, "aligned"), (dict(q_stride=504), ARG, "q_stride"),
    (dict(out_stride=513), ARG, "out_stride")])
def test_window_refusals(lib, kw, code, word):
    assert lib.csa_window_attn(ctypes.byref(attn_args(**kw)), 256, 1 << 30, None) == code and word in csa.csa_last_error()
    assert lib.csa_window_attn(None, None, 0, None) == ARG


@pytest.mark.parametrize("kw,code,word", [
    (dict(W=16), ARG, "W = 16"), (dict(S=1), ARG, "S = 1"), (dict(prefix_len=-1), ARG, "prefix_len"), (dict(prefix_len=81), ARG, "exceeds")])
def test_prefix_refusals(lib, kw, code, word):
    a = attn_args(**{**dict(W=0, S=0, prefix_len=32), **kw})
    assert lib.csa_prefix_attn(ctypes.byref(a), 256, 1 << 30, None) == code and word in csa.csa_last_error()


def test_empty_calls_do_nothing(lib):
    assert lib.csa_kv_append(ctypes.byref(append_args(rows=0)), None) == csa.CSA_OK
    assert lib.csa_kv_append(ctypes.byref(append_args(max_n=0)), None) == csa.CSA_OK
    assert lib.csa_window_attn(ctypes.byref(attn_args(rows=0)), None, 0, None) == csa.CSA_OK
    assert lib.csa_window_attn(ctypes.byref(attn_args(max_n=0)), None, 0, None) == csa.CSA_OK
    assert lib.csa_prefix_attn(ctypes.byref(attn_args(W=0, S=0, max_len=0)), None, 0, None) == csa.CSA_OK


def test_workspace(lib):
    kv = cache(H=64, H_kv=8, d=128, page_size=64, max_pages=2048, page_stride=64 * 8 * 128, slot_stride=1024, head_stride=128)
    a = attn_args(kv, rows=2, max_n=1, max_len=131072, W=1 << 40, q_stride=8192, out_stride=8192)
    n = csa.csa_workspace_size(csa.CSA_OP_WINDOW_ATTN, a)
    assert n > 2 * 64 * 128 * 4  # few queries over many keys: partials of at least two splits
    assert lib.csa_window_attn(ctypes.byref(a), 256, n - 1, None) == ARG and "workspace" in csa.csa_last_error()
    assert lib.csa_window_attn(ctypes.byref(a), None, 0, None) == ARG and "workspace" in csa.csa_last_error()
    assert lib.csa_window_attn(ctypes.byref(a), 264, n, None) == ARG and "workspace" in csa.csa_last_error()
    a.W = 0
    assert csa.csa_workspace_size(csa.CSA_OP_WINDOW_ATTN, a) == 0
    a.S, a.prefix_len = 0, 100000
    assert csa.csa_workspace_size(csa.CSA_OP_PREFIX_ATTN, a) > 2 * 64 * 128 * 4


def test_binding_refuses_cpu_tensors():
    pages = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="cpu"):
        csa.PagedKV(pages, pages.clone(), torch.zeros(1, 4, dtype=torch.int32), torch.zeros(1, 3, dtype=torch.int64), 4)
    with pytest.raises(ValueError, match="int32"):
        csa.PagedKV(pages, pages.clone(), torch.zeros(1, 4), torch.zeros(1, 3, dtype=torch.int64), 4)
    with pytest.raises(ValueError, match="same strides"):
        csa.PagedKV(pages, pages.transpose(1, 2).contiguous().transpose(1, 2), torch.zeros(1, 4, dtype=torch.int32),
                    torch.zeros(1, 3, dtype=torch.int64), 4)


def test_visibility_of_the_reference():
    from tests.paged_harness import Case, sees
    c = Case([(5, 30)], W=7, S=3)
    see = sees(c, torch.arange(25, 30), torch.arange(30))
    for i, p in enumerate(range(25, 30)):
        for t in range(30):
            assert bool(see[i, t]) == (t <= p and (t > p - 7 or t < 3))


def test_workspace_of_prompts_beside_long_single_rows(lib):
    """Rows of prompts are written directly: only the short rows of a mixed batch have partials."""
    kv = cache(H=32, H_kv=8, d=128, B=3, page_size=64, max_pages=2048, page_stride=64 * 8 * 128, slot_stride=1024, head_stride=128)
    a = attn_args(kv, rows=16384, max_n=8191, max_len=131072, W=1 << 40, q_stride=4096, out_stride=4096)
    n = csa.csa_workspace_size(csa.CSA_OP_WINDOW_ATTN, a)
    # at most 64 query rows of each key head of each sequence, at most 256 splits, 516 bytes a row
    assert 256 < n <= 3 * 64 * 8 * 256 * 516 + 4096


@pytest.mark.parametrize("kw", [dict(rows=0), dict(max_n=0), dict(rows=0, max_n=0), dict(max_len=0)])
def test_workspace_of_empty_calls(lib, kw):
    """A call without rows plans nothing: the least workspace, which the call then takes."""
    for op, more in ((csa.CSA_OP_WINDOW_ATTN, {}), (csa.CSA_OP_PREFIX_ATTN, dict(W=0, S=0)),
                     (csa.CSA_OP_PREFIX_ATTN, dict(W=0, S=0, prefix_len=40))):
        a = attn_args(**{**more, **kw})
        n = csa.csa_workspace_size(op, a)
        assert n == 256
        call = lib.csa_window_attn if op == csa.CSA_OP_WINDOW_ATTN else lib.csa_prefix_attn
        assert call(ctypes.byref(a), 256, n, None) == csa.CSA_OK


def splits_of(a, op=csa.CSA_OP_WINDOW_ATTN):
    """Key splits of the rows of a batch of single tokens, from the workspace: d + 1 floats a row, head and split."""
    per = a.kv.B * a.kv.H * (a.kv.d + 1) * 4
    n = csa.csa_workspace_size(op, a)
    return 1 if n <= per else round(n / per)


def decode(B, max_len, W=1 << 40, H_kv=8, d=128):
    kv = cache(H=8 * H_kv, H_kv=H_kv, d=d, B=B, page_size=64, max_pages=1 << 15, num_pages=1 << 20, page_stride=64 * H_kv * d,
               slot_stride=H_kv * d, head_stride=d)
    return attn_args(kv, rows=B, max_n=1, max_len=max_len, W=W, S=0, q_stride=8 * H_kv * d, out_stride=8 * H_kv * d)


@pytest.mark.parametrize("B", [1, 3, 5, 8, 16, 31, 32, 33, 64, 128, 300])
@pytest.mark.parametrize("H_kv,d", [(8, 128), (2, 128), (8, 64), (1, 64)])
def test_no_split_outlasts_the_batch(lib, B, H_kv, d):
    """Keys of a split: at most 2,048, or 8,192 under a window, or a 32nd of the bound on the keys (less often cut where
    there are more than 512 blocks already); and never so many splits that a loose bound fills the workspace."""
    asked = min(32, 16384 // (B * H_kv))
    for keys in (100, 1000, 2048, 2049, 6000, 6200, 8192, 10000, 16384, 40000, 65536, 70000, 131072, 1 << 20):
        for window in (False, True):
            s = splits_of(decode(B, 1 << 21 if window else keys, keys if window else 1 << 40, H_kv, d))
            longest = max(8192 if window else 2048, -(-keys // asked))
            assert s * (longest + 32) >= keys, (keys, window, s)
            # (what fills two blocks on each of 148 SMs may be more)
            assert s <= max(64, -(-296 // (B * H_kv))) and s <= 256, (keys, window, s)


def test_few_long_rows_beside_prompts_are_split(lib):
    """The same cap where prompts are in the call: a continuous batch of 64 sequences, one of them long."""
    a = decode(64, 131072)
    a.rows, a.max_n = 64 + 512, 512
    # 8 tokens of each sequence belong to the kernel of few rows, 1,024 blocks before the cut
    per = 64 * 8 * 64 * 129 * 4
    assert csa.csa_workspace_size(csa.CSA_OP_WINDOW_ATTN, a) >= 16 * per


@pytest.mark.parametrize("B", [2, 16, 64, 256, 1024])
@pytest.mark.parametrize("H,H_kv", [(64, 8), (64, 64), (32, 1)])
@pytest.mark.parametrize("chunk", [100, 512, 8192])
def test_partials_beside_prompts_stay_small(lib, B, H, H_kv, chunk):
    """A continuous batch of B sequences and a chunk of a prompt: partials are held for the rows of the call or for the
    short rows of each sequence, whichever is less, and for few splits where even that is much."""
    d = 128
    kv = cache(H=H, H_kv=H_kv, d=d, B=B, page_size=64, max_pages=1 << 15, num_pages=1 << 20, page_stride=64 * H_kv * d,
               slot_stride=H_kv * d, head_stride=d)
    rows = B - 1 + chunk
    one = min(rows, B * (64 // (H // H_kv))) * H * (d + 1) * 4  # bytes of a split of the short rows
    for max_len in (5000, 131072, 1 << 20):
        a = attn_args(kv, rows=rows, max_n=chunk, max_len=max_len, W=1 << 40, S=0, q_stride=H * d, out_stride=H * d)
        n = csa.csa_workspace_size(csa.CSA_OP_WINDOW_ATTN, a)
        # the chunk itself is cut while its blocks are fewer than SMs (each of up to 2 * 128 / G tokens)
        tpb = 2 * (128 // (H // H_kv))
        blocks = min(B * -(-chunk // tpb), rows // tpb + B) * H_kv
        many = rows * H * (d + 1) * 4 * min(64, 148 // blocks) if 2 * blocks <= 148 else 0
        assert n - many <= max((1 << 30) + 4096, 296 // (B * H_kv) * one + 4096), (max_len, n)
