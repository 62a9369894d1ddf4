"""PagedKV on a machine without a GPU: what its arguments keep alive, and what it refuses before a launch.  The
handles of these tests are filled in by hand, over CPU tensors that no kernel ever sees."""
import gc
import weakref

import pytest
import torch

import compressed_sparse_kv_overlapped_b200 as csa

H, H_KV, D = 8, 2, 64


def handle(device=torch.device("cpu")):
    kv = csa.PagedKV.__new__(csa.PagedKV)
    kv.device, kv.dtype, kv.H, kv.H_kv, kv.d = device, torch.bfloat16, H, H_KV, D
    c = kv.kv = csa.csa_kv_cache()
    c.H, c.H_kv, c.d, c.page_size, c.B, c.num_pages, c.max_pages = H, H_KV, D, 16, 1, 4, 4
    c.page_stride, c.slot_stride, c.head_stride = 16 * H_KV * D, H_KV * D, D
    return kv


def tokens(heads, rows=3):
    return torch.zeros(rows, heads, D, dtype=torch.bfloat16)


@pytest.mark.parametrize("call", ["append", "window", "prefix"])
def test_dropped_arguments_free_their_tensors_at_once(call):
    """Device memory is freed when the arguments go, not when the cycle collector runs."""
    kv = handle()
    held = [tokens(H), tokens(H), tokens(H_KV), tokens(H_KV), torch.zeros(D // 2), torch.zeros(3, H)]
    if call == "append":
        args = kv.append_args(held[2], held[3], held[0], held[1], max_n=3, inv_freq=held[4])
        used = held[:5]
    elif call == "window":
        args = kv.window_args(held[0], held[1], W=8, max_n=3, lse=held[5])
        used = [held[0], held[1], held[5]]
    else:
        args = kv.prefix_args(held[0], held[1], prefix_len=8, max_n=3, lse=held[5])
        used = [held[0], held[1], held[5]]
    refs = [weakref.ref(kv)] + [weakref.ref(t) for t in used]
    enabled = gc.isenabled()
    gc.disable()
    try:
        del kv, held, used
        assert all(r() is not None for r in refs), "the arguments keep their tensors and the cache alive"
        del args
        assert all(r() is None for r in refs)
    finally:
        if enabled:
            gc.enable()


class Refused(Exception):
    pass


def no_call(*a):
    raise Refused("the library was called")


@pytest.mark.parametrize("call", ["window_attn", "prefix_attn"])
def test_a_workspace_elsewhere_is_refused(call):
    """A workspace that the kernels cannot reach, or that is not one run of bytes, never gets to a launch."""
    kv = handle()
    q, out = tokens(H), tokens(H)
    args = kv.window_args(q, out, W=8, max_n=3) if call == "window_attn" else kv.prefix_args(q, out, prefix_len=8, max_n=3)
    kv._device_index, kv._window_fn, kv._prefix_fn = 0, no_call, no_call
    kv._current_stream, kv._current_device = (lambda i: 0), (lambda: 0)
    kv.device = torch.device("cuda", 0)
    run = getattr(kv, call)
    with pytest.raises(ValueError, match="workspace"):
        run(args, torch.empty(1 << 20, dtype=torch.uint8))
    with pytest.raises(ValueError, match="workspace"):
        run(args, torch.empty(1, dtype=torch.uint8).expand(1 << 20))
    with pytest.raises(ValueError, match="workspace"):
        run(args, torch.empty(1 << 20, dtype=torch.uint8, device="meta"))
    with pytest.raises(Refused):  # (none at all is the library's to judge)
        run(args, None)
