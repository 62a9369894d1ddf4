"""Paged key/value operators: their cases, inputs and plain forms.

Three operators that serve attention layers with separate keys and values beside the compressed
ones: csa_kv_append (new tokens into a paged cache, rotated by position on the way, with the queries'
rotation), csa_window_attn (causal attention over a sliding window and the first tokens, read from the
pages; a window as long as the sequence is plain causal attention) and csa_prefix_attn (a batch whose
sequences share a long prefix, attended once for all of them).

A cache holds pages [num_pages, page, H_kv, d] of keys and of values; sequence b's token t lies at slot
t % page of page table[b, t // page].  Sequence b has `len` tokens, the newest `n` of which are the rows
`row .. row + n` of the token arrays (q, k, v, out).
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
BLOCK = 256  # queries of one block of the plain window form


def listed():
    return [
        # a decode step of a small draft model: four short sequences, where the call's own latency counts
        dict(name="append_step_small", op="append", type="bf16", B=4, n_lo=1, n_hi=1, len_lo=3, len_hi=700, H=8, H_kv=2,
             d=64, page=16, rot=64, interleaved=False),
        # a decode step of a wide batch, positions up to a million (the long-context workload's length)
        dict(name="append_step_b128", op="append", type="bf16", B=128, n_lo=1, n_hi=1, len_lo=1000, len_hi=1 << 20, H=64,
             H_kv=8, d=128, page=64, rot=128, interleaved=False),
        # ragged prompts in one call; half of each head is rotated, pairs side by side
        dict(name="append_prompts", op="append", type="f16", B=6, n_lo=511, n_hi=9001, len_lo=511, len_hi=20000, H=64,
             H_kv=8, d=128, page=32, rot=64, interleaved=True),
        # one short sequence of a small layer, one new token: latency
        dict(name="window_step_small", op="window", type="bf16", B=1, n_lo=1, n_hi=1, len_lo=1023, len_hi=1023, H=8, H_kv=1,
             d=64, page=16, W=128, S=4),
        # the ragged decode workload (32 sequences of 32,768 to 131,072 tokens) with a window of 4,096
        dict(name="window_step_b32", op="window", type="bf16", B=32, n_lo=1, n_hi=1, len_lo=32768, len_hi=131072, H=64,
             H_kv=8, d=128, page=64, W=4096, S=4),
        # long windows and few sequences, three proposed tokens each to check at once
        dict(name="window_step_long", op="window", type="f16", B=5, n_lo=1, n_hi=3, len_lo=40000, len_hi=131072, H=32,
             H_kv=8, d=128, page=16, W=65536, S=16),
        # a long prompt through a local layer: window of 128 as in the compressed layers
        dict(name="window_prompt", op="window", type="bf16", B=1, n_lo=32768, n_hi=32768, len_lo=32768, len_hi=32768, H=64,
             H_kv=8, d=128, page=64, W=128, S=4),
        # ragged prompts, plain causal attention (the window covers everything)
        dict(name="window_causal", op="window", type="bf16", B=3, n_lo=77, n_hi=8191, len_lo=77, len_hi=8191, H=32, H_kv=8,
             d=128, page=128, W=1 << 20, S=0),
        # a chunk of a prompt behind a long history, as many key heads as query heads, narrow heads
        dict(name="window_chunk", op="window", type="f16", B=2, n_lo=1000, n_hi=2000, len_lo=20001, len_hi=30001, H=16,
             H_kv=16, d=64, page=16, W=4096, S=64),
        # a handful of sequences behind a short common prompt
        dict(name="prefix_small", op="prefix", type="bf16", B=5, n_lo=1, n_hi=1, prefix=1000, suf_lo=1, suf_hi=37, H=8,
             H_kv=2, d=64, page=16),
        # a serving batch behind a common system prompt
        dict(name="prefix_b32", op="prefix", type="bf16", B=32, n_lo=1, n_hi=1, prefix=8192, suf_lo=1, suf_hi=512, H=32,
             H_kv=8, d=128, page=64),
        # many samples of one long document, two proposed tokens in some of them
        dict(name="prefix_b128", op="prefix", type="f16", B=128, n_lo=1, n_hi=2, prefix=32768, suf_lo=2, suf_hi=1024, H=64,
             H_kv=8, d=128, page=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("append", "window", "window", "prefix"))
    H_kv = rng.choice((1, 2, 4, 8))
    H = H_kv * rng.choice((1, 2, 3, 4, 5, 7, 8))
    c = dict(op=op, type=rng.choice(("bf16", "f16")), H=H, H_kv=H_kv, d=rng.choice((64, 128)),
             page=rng.choice((16, 32, 64, 128, 256)))
    if op == "append":
        c["rot"] = rng.choice([r for r in (0, 32, 64, 96, 128) if r <= c["d"]])
        c["interleaved"] = rng.random() < 0.5
        if rng.random() < 0.5:
            c.update(B=_log(rng, 1, 256), n_lo=1, n_hi=rng.choice((1, 1, 4)), len_lo=4, len_hi=_log(rng, 100, 1 << 20))
        else:
            n = _log(rng, 16, 8000)
            c.update(B=rng.randint(1, 5), n_lo=rng.randint(1, n), n_hi=n, len_lo=n, len_hi=n + _log(rng, 1, 100000))
    elif op == "window":
        c["S"] = rng.choice((0, 1, 4, 16, 100))
        if rng.random() < 0.5:
            hi = _log(rng, 16, 60000)
            c.update(B=_log(rng, 1, 64), n_lo=1, n_hi=rng.choice((1, 1, 4)), len_lo=rng.randint(4, hi), len_hi=hi,
                     W=_log(rng, 16, 16384))
        else:
            n = _log(rng, 16, 4000)
            c.update(B=rng.randint(1, 3), n_lo=rng.randint(1, n), n_hi=n, len_lo=n, len_hi=n + _log(rng, 1, 8000),
                     W=_log(rng, 16, 16384))
    else:
        c.update(B=_log(rng, 2, 100), n_lo=1, n_hi=rng.choice((1, 1, 3)), prefix=_log(rng, 50, 20000), suf_lo=3,
                 suf_hi=_log(rng, 4, 1000))
    return c


def _lengths(c):
    """[(n, len)] of the case's sequences: spread over their ranges in an order without a pattern."""
    f = [(b * 0.6180339887498949) % 1.0 for b in range(1, c["B"] + 1)]
    g = [(b * 0.7548776662466927) % 1.0 for b in range(1, c["B"] + 1)]
    if c["B"] == 1:
        f, g = [1.0], [1.0]
    ns = [c["n_lo"] + int(x * (c["n_hi"] - c["n_lo"]) + 0.5) for x in f]
    if c["op"] == "prefix":
        lens = [c["prefix"] + c["suf_lo"] + int(x * (c["suf_hi"] - c["suf_lo"]) + 0.5) for x in g]
    else:
        lens = [c["len_lo"] + int(x * (c["len_hi"] - c["len_lo"]) + 0.5) for x in g]
    return [(n, max(n, m)) for n, m in zip(ns, lens)]


def _held(c):
    """Pages in use: [(sequence, page of the sequence)], and pages of the shared prefix."""
    P, held, shared = c["page"], [], 0
    if c["op"] == "prefix":
        shared = c["prefix"] // P
    for b, (n, m) in enumerate(_lengths(c)):
        last = (m - 1) // P
        if c["op"] == "append":
            first, head = (m - n) // P, -1
        elif c["op"] == "window":
            first, head = max(0, m - n - c["W"] + 1) // P, (min(c["S"], m) - 1) // P if c["S"] else -1
        else:
            first, head = shared, -1
        held += [(b, j) for j in range(0, min(head, first - 1) + 1)] + [(b, j) for j in range(first, last + 1)]
    return held, shared


def prepare(case, seed):
    c, dev, dt = case, "cuda", TYPES[case["type"]]
    gen = torch.Generator(device=dev).manual_seed(seed)
    seqs = _lengths(c)
    rows, table_rows = 0, []
    for n, m in seqs:
        table_rows.append([rows, n, m])
        rows += n
    held, shared = _held(c)
    num_pages = len(held) + shared + 3
    order = torch.randperm(num_pages, generator=gen, device=dev).to(torch.int32)
    max_pages = max((m + c["page"] - 1) // c["page"] for _, m in seqs)
    # a page that no query sees any more has been given back: its entry of the table says -1
    table = torch.full((c["B"], max_pages), -1, dtype=torch.int32, device=dev)
    at = torch.tensor(held, dtype=torch.int64).reshape(-1, 2).to(dev)
    table[at[:, 0], at[:, 1]] = order[shared:shared + len(held)]
    if shared:
        table[:, :shared] = order[:shared]
    part = c["prefix"] % c["page"] if c["op"] == "prefix" else 0

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=gen, dtype=dt, device=dev).mul_(std)

    s = dict(c=c, rows=rows, seqs=torch.tensor(table_rows, dtype=torch.int64, device=dev), table=table,
             k_pages=normal(num_pages, c["page"], c["H_kv"], c["d"]),
             v_pages=normal(num_pages, c["page"], c["H_kv"], c["d"]), scale=c["d"] ** -0.5)
    if part:  # a prefix that ends inside a page: every sequence holds its own copy of that page
        for x in (s["k_pages"], s["v_pages"]):
            x[table[:, shared].long(), :part] = x[table[0, shared].long(), :part].clone()
    if c["op"] == "append":
        # q, k and v are the parts of one projection's output, as a layer hands them over
        qkv = normal(rows, (c["H"] + 2 * c["H_kv"]) * c["d"])
        q, k, v = qkv.split([c["H"] * c["d"], c["H_kv"] * c["d"], c["H_kv"] * c["d"]], dim=1)
        s.update(q=q.unflatten(1, (c["H"], c["d"])), k=k.unflatten(1, (c["H_kv"], c["d"])),
                 v=v.unflatten(1, (c["H_kv"], c["d"])), q_out=torch.empty(rows, c["H"], c["d"], dtype=dt, device=dev),
                 inv_freq=10000.0 ** (-torch.arange(0, c["rot"], 2, dtype=torch.float32, device=dev) / max(c["rot"], 1)))
    else:
        s.update(q=normal(rows, c["H"], c["d"], std=1.5), out=torch.zeros(rows, c["H"], c["d"], dtype=dt, device=dev),
                 lse=torch.zeros(rows, c["H"], dtype=torch.float32, device=dev))
    if own:
        import compressed_sparse_kv_overlapped_b200 as csa
        kv = s["kv"] = csa.PagedKV(s["k_pages"], s["v_pages"], s["table"], s["seqs"], c["H"])
        max_n, max_len = max(n for n, _ in seqs), max(m for _, m in seqs)
        if c["op"] == "append":
            s["args"] = kv.append_args(s["k"], s["v"], s["q"], s["q_out"], max_n=max_n, inv_freq=s["inv_freq"],
                                       interleaved=c["interleaved"])
        elif c["op"] == "window":
            s["args"] = kv.window_args(s["q"], s["out"], W=c["W"], S=c["S"], max_n=max_n, max_len=max_len, lse=s["lse"],
                                       scale=s["scale"])
            s["ws"] = kv.workspace(s["args"])
        else:
            s["args"] = kv.prefix_args(s["q"], s["out"], prefix_len=c["prefix"], max_n=max_n, max_len=max_len,
                                       lse=s["lse"], scale=s["scale"])
            s["ws"] = kv.workspace(s["args"])
    return s


def run(s):
    op = s["c"]["op"]
    if own:
        if op == "append":
            s["kv"].append(s["args"])
            return s["q_out"], s["k_pages"], s["v_pages"]
        if op == "window":
            s["kv"].window_attn(s["args"], s["ws"])
        else:
            s["kv"].prefix_attn(s["args"], s["ws"])
        return s["out"], s["lse"]
    return {"append": _append, "window": _window, "prefix": _prefix}[op](s)


# ------------------------------------------------------------------------------- the plain forms

def _tokens(s):
    """Sequence and position of every row of the token arrays."""
    row, n, m = s["seqs"].unbind(1)
    b = torch.repeat_interleave(torch.arange(len(n), device=n.device), n, output_size=s["rows"])
    return b, m[b] - n[b] + torch.arange(s["rows"], device=n.device) - row[b]


def _rotated(x, pos, inv_freq, rot, interleaved):
    x = x.float()
    if not rot:
        return x
    angle = pos.double()[:, None, None] * inv_freq.double()
    cos, sin = angle.cos().float(), angle.sin().float()
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack((a * cos - b * sin, a * sin + b * cos), dim=-1).flatten(-2)
    else:
        a, b = x[..., : rot // 2], x[..., rot // 2: rot]
        turned = torch.cat((a * cos - b * sin, a * sin + b * cos), dim=-1)
    return torch.cat((turned, x[..., rot:]), dim=-1)


def _append(s):
    c, dt = s["c"], s["k_pages"].dtype
    b, pos = _tokens(s)
    page, slot = s["table"][b, pos // c["page"]].long(), pos % c["page"]
    s["k_pages"][page, slot] = _rotated(s["k"], pos, s["inv_freq"], c["rot"], c["interleaved"]).to(dt)
    s["v_pages"][page, slot] = s["v"]
    s["q_out"].copy_(_rotated(s["q"], pos, s["inv_freq"], c["rot"], c["interleaved"]).to(dt))
    return s["q_out"], s["k_pages"], s["v_pages"]


def _gather(pages, table_rows, t, page):
    """[.., H_kv, len(t), d] in 32 bits: the vectors of tokens t (clamped; the caller masks)."""
    at = torch.gather(table_rows, 1, (t // page).clamp(max=table_rows.shape[1] - 1)).long().clamp(min=0)
    return pages[at, t % page].float().transpose(1, 2)


def _window(s):
    c, dt = s["c"], s["q"].dtype
    P, G, dev = c["page"], c["H"] // c["H_kv"], s["q"].device
    seqs = _lengths(c)
    step = min(BLOCK, max(n for n, _ in seqs))
    blocks = torch.tensor([(b, i) for b, (n, _) in enumerate(seqs) for i in range(0, n, step)], device=dev)
    row, n, m = s["seqs"][blocks[:, 0]].unbind(1)
    i = blocks[:, 1:] + torch.arange(step, device=dev)                        # [N, step] new tokens of the blocks
    p = (m - n)[:, None] + i                                                  # their positions
    W, S = min(c["W"], 1 << 31), c["S"]
    base = (p[:, :1] - W + 1).clamp(min=0)
    span = min(W + step - 1, max(m for _, m in seqs))
    t = torch.cat((torch.arange(S, device=dev).expand(len(p), S), base + torch.arange(span, device=dev)), dim=1)
    first = torch.arange(S + span, device=dev) < S                            # a first token counts once
    see = (t[:, None] <= p[..., None]) & ((t[:, None] > p[..., None] - W) | (t[:, None] < S))
    see &= ~(first & (t >= base))[:, None]
    table = s["table"][blocks[:, 0]]
    K, V = _gather(s["k_pages"], table, t, P), _gather(s["v_pages"], table, t, P)
    at = (row[:, None] + i).clamp(max=s["rows"] - 1)
    q = s["q"][at].float().unflatten(2, (c["H_kv"], G)).permute(0, 2, 3, 1, 4)   # [N, H_kv, G, step, d]
    x = (q.flatten(2, 3) @ K.transpose(2, 3)).unflatten(2, (G, step)) * s["scale"]
    x = x.masked_fill(~see[:, None, None], -math.inf)
    top = x.amax(dim=-1, keepdim=True).clamp(min=-1e30)
    w = torch.exp(x - top)
    total = w.sum(dim=-1, keepdim=True)
    o = (w.flatten(2, 3) @ V).unflatten(2, (G, step)) / total
    lse = (total.log() + top).squeeze(-1)
    new = i < n[:, None]
    s["out"][at[new]] = o.permute(0, 3, 1, 2, 4).flatten(2, 3)[new].to(dt)
    s["lse"][at[new]] = lse.permute(0, 3, 1, 2).flatten(2, 3)[new]
    return s["out"], s["lse"]


def _prefix(s):
    c, dt = s["c"], s["q"].dtype
    P, G, dev, L = c["page"], c["H"] // c["H_kv"], s["q"].device, c["prefix"]
    b, p = _tokens(s)
    R = s["rows"]
    q = s["q"].float().unflatten(1, (c["H_kv"], G))                            # [R, H_kv, G, d]
    K = _gather(s["k_pages"], s["table"][:1], torch.arange(L, device=dev)[None], P)[0]
    V = _gather(s["v_pages"], s["table"][:1], torch.arange(L, device=dev)[None], P)[0]
    x = q.permute(1, 0, 2, 3).flatten(1, 2) @ K.transpose(1, 2) * s["scale"]    # [H_kv, R G, L]
    t = L + torch.arange(max(m for _, m in _lengths(c)) - L, device=dev)
    Ks = _gather(s["k_pages"], s["table"], t.expand(c["B"], -1), P)[b]          # [R, H_kv, suffix, d]
    Vs = _gather(s["v_pages"], s["table"], t.expand(c["B"], -1), P)[b]
    y = (q @ Ks.transpose(2, 3) * s["scale"]).masked_fill((t > p[:, None])[:, None, None], -math.inf)
    top = torch.maximum(x.amax(dim=-1).unflatten(1, (R, G)).transpose(0, 1), y.amax(dim=-1))   # [R, H_kv, G]
    w = torch.exp(x - top.transpose(0, 1).flatten(1)[..., None])
    z = torch.exp(y - top[..., None])
    total = w.sum(dim=-1).unflatten(1, (R, G)).transpose(0, 1) + z.sum(dim=-1)
    o = ((w @ V).unflatten(1, (R, G)).transpose(0, 1) + z @ Vs) / total[..., None]
    s["out"].copy_(o.flatten(1, 2).to(dt))
    s["lse"].copy_((total.log() + top).flatten(1, 2))
    return s["out"], s["lse"]


# --------------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    c = case
    if work(c)["flops"] > 4e13:
        return None
    s = prepare(case, seed)
    table, seqs = s["table"].cpu(), _lengths(c)

    def places(b, t):  # pool row of token t of sequence b, slots of all pages counted through
        return table[b].long()[t // c["page"]] * c["page"] + t % c["page"]

    pools = [s[x].flatten(0, 1) for x in ("k_pages", "v_pages")]
    if c["op"] == "append":
        pools = [x.double() for x in pools]
        q_out = s["q"].double()
        row = 0
        for b, (n, m) in enumerate(seqs):
            pos = torch.arange(m - n, m)
            turn = torch.polar(torch.ones((), dtype=torch.float64),
                               pos.double()[:, None] * s["inv_freq"].cpu().double()).cuda()[:, None]
            at = places(b, pos).cuda()
            pools[0][at] = _turned(s["k"][row:row + n].double(), turn, c)
            pools[1][at] = s["v"][row:row + n].double()
            q_out[row:row + n] = _turned(s["q"][row:row + n].double(), turn, c)
            row += n
        return q_out, *(x.reshape(s["k_pages"].shape) for x in pools)
    out, lse = (torch.zeros(x.shape, dtype=torch.float64, device="cuda") for x in (s["out"], s["lse"]))
    G, row = c["H"] // c["H_kv"], 0
    for b, (n, m) in enumerate(seqs):
        for i in range(0, n, 128):
            p = torch.arange(m - n + i, m - n + min(n, i + 128))
            t = torch.arange(int(p[-1]) + 1)
            see = torch.ones(len(p), len(t), dtype=torch.bool).tril(int(p[0]))
            if c["op"] == "window":
                lo = max(0, int(p[0]) - c["W"] + 1)
                t = torch.cat((t[: min(c["S"], lo)], t[lo:]))
                far = p[:, None] - t[None]
                see = (far >= 0) & ((far < c["W"]) | (t < c["S"]))
            at = places(b, t).cuda()
            bias = torch.zeros(see.shape, dtype=torch.float64).masked_fill_(~see, -math.inf).cuda()
            for h in range(c["H_kv"]):
                K, V = (x[at, h].double() for x in pools)
                q = s["q"][row + i:row + i + len(p), h * G:(h + 1) * G].double()
                x = torch.einsum("pgd,td->gpt", q, K) * s["scale"] + bias
                lse[row + i:row + i + len(p), h * G:(h + 1) * G] = torch.logsumexp(x, dim=-1).T
                out[row + i:row + i + len(p), h * G:(h + 1) * G] = torch.einsum("gpt,td->pgd", torch.softmax(x, dim=-1), V)
        row += n
    return out, lse


def _turned(x, turn, c):
    """x with its first `rot` channels as complex numbers times `turn`."""
    r = c["rot"]
    if not r:
        return x
    pairs = x[..., :r].unflatten(-1, (r // 2, 2) if c["interleaved"] else (2, r // 2))
    if not c["interleaved"]:
        pairs = pairs.transpose(-1, -2)
    z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
    if not c["interleaved"]:
        z = z.transpose(-1, -2)
    return torch.cat((z.flatten(-2), x[..., r:]), dim=-1)


def work(case):
    c, seqs, e = case, _lengths(case), 2
    rows, kv_row = sum(n for n, _ in seqs), 2 * case["H_kv"] * case["d"] * e
    if c["op"] == "append":
        return {"bytes": rows * (2 * kv_row + 2 * c["H"] * c["d"] * e), "flops": rows * 3 * (c["H"] + c["H_kv"]) * c["rot"]}
    tokens = c["prefix"] if c["op"] == "prefix" else 0  # key/value rows read
    pairs = 0                                            # (query, visible token) pairs
    for n, m in seqs:
        if c["op"] == "prefix":
            tokens += m - c["prefix"]
            pairs += n * m - n * (n - 1) // 2
            continue
        lo = max(0, m - n - c["W"] + 1)
        tokens += m - lo + min(c["S"], lo)
        full = min(n, max(0, m - c["W"]))                # queries whose window does not reach token 0
        rest = n - full
        pairs += rest * (m - n + 1) + rest * (rest - 1) // 2 + full * c["W"]
        first = m - full + 1                             # visible tokens of the first of them
        few = min(full, max(0, c["W"] + c["S"] - first)) # of those, the ones whose window reaches the first tokens
        pairs += few * (first - c["W"]) + few * (few - 1) // 2 + (full - few) * c["S"]
    return {"bytes": tokens * kv_row + rows * c["H"] * (2 * c["d"] * e + 4), "flops": pairs * c["H"] * c["d"] * 4}
