"""Cases of the paged cache's attention with a sliding window and sinks, and of batches that share a
long prefix: packed chunks and decoded tokens, and the verification of draft trees.

Every case is a dict of plain values.  `prepare` makes the inputs of a case from a seed, `run` is
one call of the operator (its plain form in torch, or the library's kernels where `own` is set),
`exact` the same outputs from the definition in 64 bits, `work` the bytes and operations that the
call cannot do without.  Sequence lengths, groups and trees belong to the case; values and page
order come from the seed.
"""
import math
import random

import numpy as np
import torch

own = False

PAGE = 16
E4M3_MAX = 448.0


# ------------------------------------------------------------------------------ cases

def _case(name, op, **kw):
    # own_lo .. own_hi: cached tokens of a sequence beside the shared ones; new_lo .. new_hi: its new tokens or tree nodes
    c = dict(name=name, op=op, batch=1, own_lo=0, own_hi=0, new_lo=1, new_hi=1, q_heads=32, kv_heads=8, dim=128,
             dtype="bf16", cache="same", lens=1, window=0, sinks=0, groups=0, shared_lo=0, shared_hi=0)
    c.update(kw)
    return c


def listed():
    return [
        # one sequence, one decoded token of a window layer: the smallest call, where only latency counts
        _case("window token", "window", own_lo=2500, own_hi=2500, window=1024, sinks=4),
        # one decoded token of each of 64 sequences of very different lengths, most longer than the window
        _case("window decode", "window", batch=64, own_lo=512, own_hi=32767, window=4096, sinks=4, lens=2),
        # decoding over an 8-bit cache, an odd window
        _case("window decode e4m3", "window", batch=32, own_lo=300, own_hi=9000, q_heads=64, cache="e4m3", window=2047,
              sinks=16, lens=3),
        # whole prompts of different lengths through a window layer, packed
        _case("window prompts", "window", batch=4, new_lo=900, new_hi=5000, window=1024, sinks=4, lens=4),
        # float32, small heads, a few short odd chunks
        _case("window chunk f32", "window", batch=5, own_hi=700, new_hi=130, q_heads=4, kv_heads=1, dim=64, dtype="f32",
              window=100, sinks=3, lens=5),
        # one small draft tree over an 8-bit cache
        _case("window tree e4m3 small", "window tree", own_lo=2048, own_hi=2048, new_lo=8, new_hi=8, cache="e4m3",
              window=512, sinks=4, lens=6),
        # a batch of draft trees of up to 64 nodes, eight query heads to a kv head
        _case("window tree", "window tree", batch=32, own_lo=6000, own_hi=8192, new_lo=40, new_hi=64, q_heads=64,
              window=4096, sinks=4, lens=7),
        # 64 requests behind one system prompt, a decoded token of each
        _case("shared decode", "shared", batch=64, own_lo=20, own_hi=600, groups=1, shared_lo=8192, shared_hi=8192, lens=8),
        # samples of three prompts over an 8-bit cache, a few odd new tokens of each
        _case("shared groups e4m3", "shared", batch=47, own_lo=0, own_hi=900, new_lo=1, new_hi=5, q_heads=64, cache="e4m3",
              groups=3, shared_lo=2000, shared_hi=6000, lens=9),
        # float32, small heads, four short chunks behind one prompt
        _case("shared chunk f32", "shared", batch=4, own_hi=60, new_hi=7, q_heads=4, kv_heads=1, dim=64, dtype="f32",
              groups=1, shared_lo=800, shared_hi=800, lens=10),
        # four small draft trees, the samples of one prompt, over an 8-bit cache
        _case("shared tree e4m3 small", "shared tree", batch=4, own_lo=10, own_hi=200, new_lo=8, new_hi=8, cache="e4m3",
              groups=1, shared_lo=2048, shared_hi=2048, lens=11),
        # 32 draft trees of up to 16 nodes behind one long document
        _case("shared tree", "shared tree", batch=32, own_lo=100, own_hi=1500, new_lo=9, new_hi=16, groups=1,
              shared_lo=16384, shared_hi=16384, lens=12),
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], even over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("window", "window", "window tree", "shared", "shared", "shared tree"))
    hq, hkv = rng.choice(((4, 1), (8, 2), (12, 4), (28, 4), (32, 8), (32, 32), (64, 8)))
    dim = rng.choice((64, 128, 128))
    if dim == 64:
        hq, hkv = rng.choice(((4, 1), (16, 4), (32, 32), (20, 4)))
    f32 = rng.random() < 0.25
    c = _case(None, op, q_heads=hq, kv_heads=hkv, dim=dim, lens=rng.randrange(1 << 30), dtype="f32" if f32 else "bf16",
              cache=rng.choice(("same", "e4m3")))
    del c["name"]
    if op.endswith("tree"):
        new = _log(rng, 2, 64)
        batch = _log(rng, 1, max(1, min(32, 1500 // new)))
    else:
        kind = rng.choice(("decode", "chunk", "prompt" if op == "window" else "few"))
        new = {"decode": 1, "chunk": _log(rng, 2, 512), "few": _log(rng, 2, 16), "prompt": _log(rng, 16, 4000)}[kind]
        if f32:
            new = min(new, 300)
        batch = _log(rng, 1, 64 if new <= 16 else 6)
    if op.startswith("window"):
        pre = 0 if new > 512 else _log(rng, 16, 2000 if f32 else 20000)
        batch = max(1, min(batch, 600_000 // (pre + new)))
        c.update(own_lo=pre // 4, own_hi=pre, window=_log(rng, 16, 6000), sinks=rng.choice((0, 1, 4, 4, 16, 37, 128)))
    else:
        shared, pre = _log(rng, 16, 1500 if f32 else 16000) // 16 * 16, _log(rng, 1, 1500)
        batch = max(1, min(batch, 500_000 // (shared + pre + new)))
        c.update(own_lo=pre // 8, own_hi=pre, groups=rng.choice((1, 1, 1, 2, 4)), shared_lo=shared // 2, shared_hi=shared)
    c.update(batch=batch, new_lo=(new + 1) // 2, new_hi=new)
    return c


def _lengths(c):
    """Cached and new-token counts of each sequence, its group's first sequence and the tokens it shares; the same for
    every seed.  Groups are runs of consecutive sequences, as even as they come."""
    r = random.Random(c["lens"])
    B = c["batch"]
    pre = [r.randint(c["own_lo"], c["own_hi"]) for _ in range(B)]
    new = [r.randint(c["new_lo"], c["new_hi"]) for _ in range(B)]
    new[r.randrange(B)] = c["new_hi"]
    n = min(c["groups"], B)
    starts = [B * g // n for g in range(n)] + [B] if n else []
    shared = [r.randint(c["shared_lo"], c["shared_hi"]) // PAGE * PAGE for _ in range(n)]
    for g in range(n):
        for b in range(starts[g], starts[g + 1]):
            pre[b] += shared[g]
    return pre, new, starts, shared


def _trees(c, new, width):
    """A random tree of new[b] nodes for each sequence, rows padded with -2 to `width`."""
    r = random.Random(c["lens"] + 1)
    rows = np.full((len(new), width), -2, dtype=np.int32)
    for b, n in enumerate(new):
        rows[b, :n] = [-1] + [max(0, i - 1 - int(r.random() ** 2 * 8)) for i in range(1, n)]
    return rows


def _is_tree(c):
    return c["op"].endswith("tree")


# ------------------------------------------------------------------------------ inputs

def prepare(case, seed):
    c, dev = case, torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed * 7919 + 29)
    B, Hq, Hkv, D = c["batch"], c["q_heads"], c["kv_heads"], c["dim"]
    dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
    pre, new, starts, shared = _lengths(c)
    tree = _is_tree(c)
    width = max(new)
    # the pages that hold what some row sees: of a window layer the others are given back, and their entries are -1
    held = []
    for b in range(B):
        last = (pre[b] + new[b] + PAGE - 1) // PAGE
        if c["window"]:
            low = max(0, pre[b] - c["window"] + 1) // PAGE
            sinks = (min(c["sinks"], pre[b] + new[b]) + PAGE - 1) // PAGE
            held.append([i for i in range(last) if i >= low or i < sinks])
        else:
            first = next((b == starts[k] for k in range(len(shared)) if starts[k] <= b < starts[k + 1]), True)
            skip = 0 if first else next(shared[k] for k in range(len(shared)) if starts[k] <= b < starts[k + 1]) // PAGE
            held.append(list(range(skip, last)))
    pool = sum(map(len, held)) + 2
    order = torch.randperm(pool, generator=g, device=dev).to(torch.int32)
    columns = max((p + n + PAGE - 1) // PAGE for p, n in zip(pre, new))
    table = torch.full((B, columns), -1, dtype=torch.int32, device=dev)
    at = 0
    for b in range(B):
        table[b, torch.tensor(held[b], device=dev)] = order[at:at + len(held[b])]
        at += len(held[b])
    for k in range(len(shared)):
        table[starts[k]:starts[k + 1], :shared[k] // PAGE] = table[starts[k], :shared[k] // PAGE].clone()
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    s = dict(case=c, page_table=table, prefix_lens=ints(pre), k_scales=None, v_scales=None, pre=pre, new=new,
             group_offsets=ints(starts), shared_lens=ints(shared))
    for name in ("k", "v"):
        x = torch.empty((pool, PAGE, Hkv, D), dtype=torch.float8_e4m3fn if c["cache"] == "e4m3" else dt, device=dev)
        scales = torch.empty((pool, Hkv, PAGE), device=dev)
        for a in range(0, pool, 4096):                      # a few pages at a time: the cache may be large
            y = torch.randn((min(4096, pool - a), PAGE, Hkv, D), generator=g, device=dev)
            if c["cache"] == "e4m3":                        # a scale for each token and head, as the append writes it
                scale = y.abs().amax(-1) / E4M3_MAX
                y = y / scale[..., None]
                scales[a:a + 4096] = scale.transpose(1, 2)
            x[a:a + 4096] = y.to(x.dtype)
        s[name + "_pages"] = x
        if c["cache"] == "e4m3":
            s[name + "_scales"] = scales
    if tree:
        s["q"] = torch.randn((B, width, Hq, D), generator=g, device=dev).to(dt)
        s["tree_parents"] = ints(_trees(c, new, width).tolist())
    else:
        offsets = [0]
        for n in new:
            offsets.append(offsets[-1] + n)
        s["q"] = torch.randn((offsets[-1], Hq, D), generator=g, device=dev).to(dt)
        s["chunk_offsets"] = ints(offsets)
    return s


# ------------------------------------------------------------------------------ plain forms

def _cached(s, name, pos, live):
    """K or V at the logical positions pos [B, L] in 32 bits, [B, Hkv, L, D]; zero where not live."""
    B = pos.shape[0]
    pos = torch.where(live, pos, 0)
    page = s["page_table"].long()[torch.arange(B, device=pos.device)[:, None], pos // PAGE]
    page, at = torch.where(live, page, 0), pos % PAGE
    pages = s[name + "_pages"]
    if pages.dtype == torch.float8_e4m3fn:
        x = pages.view(torch.uint8)[page, at].view(torch.float8_e4m3fn).float()
        x = x * s[name + "_scales"][page, :, at][..., None]
    else:
        x = pages[page, at].float()
    return torch.where(live[..., None, None], x, 0.0).transpose(1, 2)


def _softmax_product(q, k, v, seen):
    """q [B, N, Hq, D], k and v [B, Hkv, L, D], seen [B, N, L] -> [B, N, Hq, D], all in 32 bits."""
    B, N, Hq, D = q.shape
    Hkv = k.shape[1]
    q = q.view(B, N, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, D)
    w = q @ k.transpose(-1, -2) * (1 / math.sqrt(D))
    w = w.view(B, Hkv, Hq // Hkv, N, -1).masked_fill_(~seen[:, None, None], -math.inf)
    w = w - w.amax(-1, keepdim=True).clamp(min=-1e30)
    w = w.exp_()
    w = w / w.sum(-1, keepdim=True).clamp(min=1e-30)
    return (w.view(B, Hkv, -1, w.shape[-1]) @ v).view(B, Hkv, -1, N, D).permute(0, 3, 1, 2, 4).reshape(B, N, Hq, D)


def _plain(s):
    c = s["case"]
    dev = s["page_table"].device
    pre = s["prefix_lens"].long()
    N = max(s["new"])
    i = torch.arange(N, device=dev)
    if _is_tree(c):
        parents = s["tree_parents"]
        live_rows = parents >= -1
        step = (parents[..., None] == i).double() + torch.eye(N, device=dev, dtype=torch.float64)
        family = torch.linalg.matrix_power(step, 128) > 0           # node j is node i or above it
        depth = torch.where(live_rows, family.sum(-1) - 1, 0)
        q = s["q"].float()
    else:
        off = s["chunk_offsets"].long()
        live_rows = i[None] < (off[1:] - off[:-1])[:, None]
        family = (i[:, None] >= i)[None].expand(len(s["new"]), N, N)
        depth = i[None].expand(len(s["new"]), N)
        q = s["q"].float()[torch.where(live_rows, off[:-1, None] + i, 0)]
    used = pre + live_rows.sum(1)
    # the positions that some row sees: the sinks, and from the first row's window on
    low = [max(c["sinks"], p - c["window"] + 1) if c["window"] else 0 for p in s["pre"]]
    sinks = c["sinks"] if c["window"] else 0
    reach = sinks + max(max(0, p + n - a) for p, n, a in zip(s["pre"], s["new"], low))
    u = torch.arange(reach, device=dev)
    first = torch.clamp(pre - c["window"] + 1, min=sinks) if c["window"] else torch.zeros_like(pre)
    pos = torch.where(u[None] < sinks, u[None], first[:, None] + u[None] - sinks)
    live = pos < used[:, None]
    j = pos - pre[:, None]                                          # new token or node when >= 0
    jn = j.clamp(0, N - 1)[:, None].expand(-1, N, -1)
    seen = ((j < 0)[:, None] | family.gather(2, jn)) & live[:, None]
    if c["window"]:
        at = torch.where(j >= 0, pre[:, None] + depth.gather(1, j.clamp(0, N - 1)), pos)
        seen = seen & ((at < sinks)[:, None] | (at[:, None] > (pre[:, None] + depth)[..., None] - c["window"]))
    out = _softmax_product(q, _cached(s, "k", pos, live), _cached(s, "v", pos, live), seen)
    if _is_tree(c):
        return torch.where(live_rows[..., None, None], out, 0.0).to(s["q"].dtype)
    t = torch.arange(s["q"].shape[0], device=dev)
    seq = (t[:, None] >= off[None, 1:]).sum(1)
    return out[seq, t - off[seq]].to(s["q"].dtype)


# ------------------------------------------------------------------------------ one pass

def _workspace(s, size):
    if "workspace" not in s:                                # kept with the inputs, as a program would
        s["workspace"] = torch.empty(size(), dtype=torch.uint8, device=s["page_table"].device)
    return s["workspace"]


def _own(s):
    import eagle_speculative_tree_gb300 as ts
    c = s["case"]
    kv = ts.DTYPE_E4M3 if c["cache"] == "e4m3" else ts.DTYPE_BF16 if c["dtype"] == "bf16" else ts.DTYPE_F32
    pools = (s["q"], s["k_pages"], s["v_pages"], s["page_table"], s["prefix_lens"])
    scales = dict(k_scales=s["k_scales"], v_scales=s["v_scales"])
    if _is_tree(c):
        prob = lambda: ts.attn_problem(s["q"], s["k_pages"], s["page_table"])  # noqa: E731
        if c["op"] == "window tree":
            ws = _workspace(s, lambda: ts.attn_window_workspace_bytes(prob(), kv, c["window"], c["sinks"]))
            return ts.tree_attn_verify_window(*pools, s["tree_parents"], c["window"], c["sinks"], workspace=ws, **scales)
        ws = _workspace(s, lambda: ts.attn_shared_workspace_bytes(prob(), kv, s["shared_lens"].shape[0]))
        return ts.tree_attn_verify_shared(*pools, s["tree_parents"], s["group_offsets"], s["shared_lens"], workspace=ws,
                                          **scales)
    prob = lambda: ts.chunk_problem(s["q"], s["k_pages"], s["page_table"], s["chunk_offsets"])  # noqa: E731
    if c["op"] == "window":
        ws = _workspace(s, lambda: ts.chunk_window_workspace_bytes(prob(), c["window"], c["sinks"]))
        return ts.tree_chunk_attn_window(*pools, s["chunk_offsets"], c["window"], c["sinks"], workspace=ws, **scales)
    ws = _workspace(s, lambda: ts.chunk_shared_workspace_bytes(prob(), s["shared_lens"].shape[0]))
    return ts.tree_chunk_attn_shared(*pools, s["chunk_offsets"], s["group_offsets"], s["shared_lens"], workspace=ws, **scales)


def run(state):
    return (_own if own else _plain)(state)


# ------------------------------------------------------------------------------ work

def work(case):
    c = case
    Hq, Hkv, D, W, sinks = c["q_heads"], c["kv_heads"], c["dim"], c["window"], c["sinks"]
    e = 2 if c["dtype"] == "bf16" else 4
    row = Hkv * (D + 4) if c["cache"] == "e4m3" else Hkv * D * e     # K or V of one cached token
    pre, new, starts, shared = _lengths(c)
    parents = _trees(c, new, max(new)) if _is_tree(c) else None
    pairs, tokens = 0, -sum((starts[k + 1] - starts[k] - 1) * shared[k] for k in range(len(shared)))
    for b, (S, n) in enumerate(zip(pre, new)):
        tokens += S + n if not W else min(sinks, S + n) + max(0, S + n - max(sinks, S - W + 1))
        depth = list(range(n))
        if parents is not None:
            depth = [0] * n
            for i in range(1, n):
                depth[i] = depth[parents[b, i]] + 1
        for d in depth:                                     # visible tokens of a row: those of a causal one at its position
            p = S + d
            pairs += p + 1 if not W else min(sinks, p + 1) + max(0, p + 1 - max(sinks, p - W + 1))
    return {"bytes": 2 * sum(new) * Hq * D * e + 2 * row * tokens, "flops": 4 * D * Hq * pairs}


# ------------------------------------------------------------------------------ 64 bits

def _exact_kv(s, b, pos):
    page, at = s["page_table"].long()[b, pos // PAGE], pos % PAGE
    got = []
    for name in ("k", "v"):
        pages = s[name + "_pages"]
        x = pages.view(torch.uint8)[page, at].view(pages.dtype).double() if pages.dtype == torch.float8_e4m3fn \
            else pages[page, at].double()
        if s[name + "_scales"] is not None:
            x = x * s[name + "_scales"].double()[page, :, at][..., None]
        got.append(x)
    return got


def _exact_rows(q, k, v, hidden):
    """One sequence: q [N, Hq, D]; hidden [N, L] marks what a row may not see."""
    G = q.shape[1] // k.shape[1]
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    for h in range(q.shape[1]):
        w = torch.exp((q[:, h].double() @ k[:, h // G].T / q.shape[2] ** 0.5).masked_fill_(hidden, -math.inf))
        out[:, h] = (w @ v[:, h // G]) / w.sum(1, keepdim=True)
    return out


def exact(case, seed):
    c, s = case, prepare(case, seed)
    dev = s["page_table"].device
    W, sinks = c["window"] or 1 << 30, c["sinks"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=dev)
    parents = s["tree_parents"].tolist() if _is_tree(c) else None
    start = 0
    for b, (S, n) in enumerate(zip(s["pre"], s["new"])):
        if parents is None:
            for a in range(0, n, 512):                      # rows a .. z - 1 over the tokens that one of them sees
                z = min(n, a + 512)
                keep = [t for t in range(S + z) if t < sinks or t > S + a - W]
                t = torch.tensor(keep, device=dev)
                p = S + torch.arange(a, z, device=dev)[:, None]
                hidden = (t > p) | ((t >= sinks) & (t <= p - W))
                out[start + a:start + z] = _exact_rows(s["q"][start + a:start + z], *_exact_kv(s, b, t), hidden)
            start += n
            continue
        depth, above = [0] * n, [[0]] + [None] * (n - 1)
        for i in range(1, n):
            depth[i] = depth[parents[b][i]] + 1
            above[i] = above[parents[b][i]] + [i]
        keep = [t for t in range(S) if t < sinks or t > S - W]
        hidden = np.ones((n, len(keep) + n), dtype=bool)
        prefix = np.array(keep)
        for i in range(n):
            p = S + depth[i]
            hidden[i, :len(keep)] = (prefix >= sinks) & (prefix <= p - W)
            for j in above[i]:
                hidden[i, len(keep) + j] = S + depth[j] >= sinks and depth[i] - depth[j] >= W
        t = torch.tensor(keep + [S + j for j in range(n)], device=dev)
        out[b, :n] = _exact_rows(s["q"][b, :n], *_exact_kv(s, b, t), torch.from_numpy(hidden).to(dev))
    return out
