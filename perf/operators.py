"""Cases of the paged cache's operators: appending new tokens, attention of chunks and prompts,
and the tree verification and commit over an 8-bit cache.

Every case is a dict of plain values.  `prepare` makes the inputs of a case from a seed, `run` is
one call of the operator (its plain form in torch, or the library's kernels where `own` is set),
`exact` the same outputs from the definition in 64 bits, `work` the bytes and operations that the
call cannot do without.  Sequence lengths and trees belong to the case; values, page order and
accepted paths come from the seed.
"""
import math
import random

import numpy as np
import torch

own = False

PAGE = 16
EPS = 1e-6
E4M3_MAX = 448.0
SCALE_MIN = 2.0 ** -100      # of an all-zero row


# ------------------------------------------------------------------------------ cases

def _case(name, op, **kw):
    c = dict(name=name, op=op, batch=1, pre_lo=0, pre_hi=0, new_lo=1, new_hi=1, q_heads=32, kv_heads=8, dim=128,
             dtype="bf16", cache="same", lens=1)
    c.update(kw)
    return c


def listed():
    return [
        # one sequence, one decoded token: the smallest append, where only latency counts
        _case("append token", "append", pre_lo=2048, pre_hi=2048, rope="half", rot=128, norm=False, tree=False),
        # 32 draft trees of up to 64 nodes before verification: positions by depth, padded rows
        _case("append trees", "append", batch=32, pre_lo=1500, pre_hi=2500, new_lo=33, new_hi=64, q_heads=64, rope="half",
              rot=128, norm=True, tree=True, lens=2),
        # ragged chunks of prompts into an 8-bit cache, half of each head rotated
        _case("append prompts e4m3", "append", batch=7, pre_lo=0, pre_hi=1500, new_lo=700, new_hi=2900, rope="half", rot=64,
              norm=True, tree=False, cache="e4m3", lens=3),
        # one decoded token of each of 64 sequences of very different lengths
        _case("decode ragged", "attend", batch=64, pre_lo=512, pre_hi=32767, lens=4),
        # decoding over an 8-bit cache
        _case("decode e4m3", "attend", batch=8, pre_lo=3000, pre_hi=8191, q_heads=64, cache="e4m3", lens=5),
        # a chunk of a long prompt, after its first part
        _case("chunk", "attend", batch=4, pre_lo=6000, pre_hi=12000, new_lo=500, new_hi=512, q_heads=64, lens=6),
        # whole prompts of different lengths, packed
        _case("prompts", "attend", batch=6, new_lo=300, new_hi=4096, lens=7),
        # float32, small heads, a few short odd chunks
        _case("chunk f32", "attend", batch=5, pre_lo=0, pre_hi=700, new_lo=1, new_hi=130, q_heads=4, kv_heads=1, dim=64,
              dtype="f32", lens=8),
        # one small draft tree over an 8-bit cache
        _case("verify e4m3 small", "verify", pre_lo=2048, pre_hi=2048, new_lo=8, new_hi=8, cache="e4m3", lens=9),
        # a batch of 64-node draft trees over an 8-bit cache, one query head group of eight
        _case("verify e4m3", "verify", batch=32, pre_lo=8192, pre_hi=8192, new_lo=64, new_hi=64, q_heads=64, cache="e4m3",
              lens=10),
        # the accepted path of one small tree
        _case("commit e4m3 small", "commit", pre_lo=2048, pre_hi=2048, new_lo=8, new_hi=8, cache="e4m3", lens=11),
        # the accepted paths of a large batch of trees
        _case("commit e4m3", "commit", batch=64, pre_lo=200, pre_hi=2000, new_lo=16, new_hi=64, kv_heads=32, cache="e4m3",
              lens=12),
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], even over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("append", "append", "attend", "attend", "attend", "verify", "verify", "commit"))
    hq, hkv = rng.choice(((4, 1), (8, 2), (12, 4), (28, 4), (32, 8), (32, 32), (64, 8)))
    dim = rng.choice((64, 128, 128))
    if dim == 64:
        hq, hkv = rng.choice(((4, 1), (16, 4), (32, 32), (20, 4)))
    c = dict(op=op, q_heads=hq, kv_heads=hkv, dim=dim, lens=rng.randrange(1 << 30),
             dtype=rng.choice(("bf16", "bf16", "bf16", "f32")), cache=rng.choice(("same", "e4m3")))
    if op == "append":
        tree = rng.random() < 0.4
        new = _log(rng, 2, 64) if tree else _log(rng, 1, 2900)
        batch = _log(rng, 1, max(1, min(64, 12000 // new)))
        pre = _log(rng, 1, 4000)
        rot = rng.choice((16, 32, 48, 64) if c["dim"] == 64 else (32, 64, 80, 128))
        c.update(batch=batch, pre_lo=pre // 3, pre_hi=pre, new_lo=(new + 1) // 2, new_hi=new, tree=tree, rot=rot,
                 rope=rng.choice(("half", "interleaved")), norm=rng.random() < 0.6)
    elif op == "attend":
        f32 = c["dtype"] == "f32"
        kind = rng.choice(("decode", "chunk", "prompt"))
        if kind == "decode":
            new, pre = 1, _log(rng, 16, 4000 if f32 else 30000)
            batch = _log(rng, 1, max(1, min(64, (300_000 if f32 else 900_000) // pre)))
        elif kind == "chunk":
            new, pre = _log(rng, 2, 200 if f32 else 512), _log(rng, 16, 1500 if f32 else 11000)
            batch = _log(rng, 1, 4)
        else:
            new, pre = _log(rng, 16, 600 if f32 else 4000), 0
            batch = _log(rng, 1, 6)
        c.update(batch=batch, pre_lo=pre // 4, pre_hi=pre, new_lo=(new + 1) // 2, new_hi=new)
    elif op == "verify":
        nodes = _log(rng, 2, 64)
        pre = _log(rng, 16, 2000 if c["dtype"] == "f32" else 8192)
        c.update(cache="e4m3", batch=_log(rng, 1, max(1, min(24, 1500 // nodes))), pre_lo=pre // 2, pre_hi=pre,
                 new_lo=(nodes + 1) // 2, new_hi=nodes)
    else:
        nodes = _log(rng, 2, 127)
        pre = _log(rng, 16, 2000)
        c.update(cache="e4m3", batch=_log(rng, 1, 64), pre_lo=pre // 2, pre_hi=pre, new_lo=(nodes + 1) // 2, new_hi=nodes)
    return c


def _lengths(c):
    """Prefix and new-token counts of each sequence, the same for every seed."""
    r = random.Random(c["lens"])
    pre = [r.randint(c["pre_lo"], c["pre_hi"]) for _ in range(c["batch"])]
    new = [r.randint(c["new_lo"], c["new_hi"]) for _ in range(c["batch"])]
    new[r.randrange(c["batch"])] = c["new_hi"]
    return pre, new


def _trees(c, new, width):
    """A random tree of new[b] nodes for each sequence, rows padded with -2 to `width`."""
    r = random.Random(c["lens"] + 1)
    rows = np.full((len(new), width), -2, dtype=np.int32)
    for b, n in enumerate(new):
        rows[b, :n] = [-1] + [max(0, i - 1 - int(r.random() ** 2 * 8)) for i in range(1, n)]
    return rows


def _is_tree(c):
    return c["op"] in ("verify", "commit") or c.get("tree", False)


# ------------------------------------------------------------------------------ inputs

def _quantise(x):
    """Codes and scales of rows of 32-bit values: scale = max |x| / 448, at least 2^-100."""
    scale = (x.abs().amax(-1) / E4M3_MAX).clamp(min=SCALE_MIN)
    return (x / scale[..., None]).to(torch.float8_e4m3fn), scale


def prepare(case, seed):
    c, dev = case, torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed * 7919 + 13)
    B, Hq, Hkv, D = c["batch"], c["q_heads"], c["kv_heads"], c["dim"]
    dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
    pre, new = _lengths(c)
    tree = _is_tree(c)
    width = max(new)
    rows = [width] * B if tree else new                     # rows of q of each sequence
    need = [(p + n + PAGE - 1) // PAGE for p, n in zip(pre, rows)]
    pool = sum(need) + 2
    order = torch.randperm(pool, generator=g, device=dev).to(torch.int32)
    table = torch.zeros((B, max(need)), dtype=torch.int32, device=dev)
    at = 0
    for b in range(B):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    normal = lambda *s: torch.randn(s, generator=g, device=dev)  # noqa: E731
    offsets = [0]
    for n in rows:
        offsets.append(offsets[-1] + n)
    T = offsets[-1]
    s = dict(case=c, page_table=table, prefix_lens=ints(pre), chunk_offsets=ints(offsets), longest=max(rows),
             reach=max(p + n for p, n in zip(pre, rows)), k_scales=None, v_scales=None)
    for name in ("k", "v"):
        if c["cache"] == "e4m3":
            codes = torch.empty((pool, PAGE, Hkv, D), dtype=torch.float8_e4m3fn, device=dev)
            scales = torch.empty((pool, Hkv, PAGE), device=dev)
            for a in range(0, pool, 4096):                  # a few pages at a time: the cache may be large
                x, y = _quantise(normal(min(4096, pool - a), PAGE, Hkv, D))
                codes[a:a + 4096], scales[a:a + 4096] = x, y.transpose(1, 2)
            s[name + "_pages"], s[name + "_scales"] = codes, scales
        else:
            s[name + "_pages"] = torch.randn((pool, PAGE, Hkv, D), generator=g, device=dev, dtype=dt)
    if tree:
        parents = _trees(c, new, width)
        s["tree_parents"] = ints(parents.tolist())
    if c["op"] == "append":
        qkv = normal(T, (Hq + 2 * Hkv) * D).to(dt)           # one projection's output; q, k and v are views of it
        s["q"] = qkv[:, :Hq * D].unflatten(1, (Hq, D))
        s["k"] = qkv[:, Hq * D:(Hq + Hkv) * D].unflatten(1, (Hkv, D))
        s["v"] = qkv[:, (Hq + Hkv) * D:].unflatten(1, (Hkv, D))
        s["q_out"] = torch.zeros((T, Hq, D), dtype=dt, device=dev)
        s["q_norm"] = 1 + 0.1 * normal(D) if c["norm"] else None
        s["k_norm"] = 1 + 0.1 * normal(D) if c["norm"] else None
        j = torch.arange(0, c["rot"], 2, dtype=torch.float64, device=dev)
        s["inv_freq"] = (500000.0 ** (-j / c["rot"])).float()
        if tree:                                            # a node's position is the prefix and its depth
            depth = np.full(parents.shape, -1, dtype=np.int64)
            for b in range(B):
                for i in range(new[b]):
                    depth[b, i] = pre[b] if i == 0 else depth[b, parents[b, i]] + 1
            s["positions"] = ints(depth.reshape(-1).tolist())
        else:
            s["positions"] = ints([p + i for p, n in zip(pre, rows) for i in range(n)])
    elif c["op"] == "attend":
        s["q"] = normal(T, Hq, D).to(dt)
    elif c["op"] == "verify":
        s["q"] = normal(B, width, Hq, D).to(dt)
    else:
        path = np.full((B, width), -1, dtype=np.int32)      # a path from the root, in node order
        length = np.zeros(B, dtype=np.int32)
        r = random.Random(seed)
        for b in range(B):
            node = r.randrange(new[b])
            chain = []
            while node > 0:
                chain.append(node)
                node = int(parents[b, node])
            path[b, :len(chain)] = chain[::-1]
            length[b] = len(chain)
        s["accept_path"], s["accept_len"] = ints(path.tolist()), ints(length.tolist())
    return s


# ------------------------------------------------------------------------------ plain forms

def _rows(s, T):
    """Sequence and index in it of each of T packed rows."""
    t = torch.arange(T, device=s["chunk_offsets"].device)
    seq = (t[:, None] >= s["chunk_offsets"][None, 1:]).sum(1)
    return seq, t - s["chunk_offsets"].long()[seq]


def _slots(s, seq, pos):
    """Rows of the flattened pools that hold the logical positions `pos` of the sequences `seq`."""
    return s["page_table"].long()[seq, pos // PAGE] * PAGE + pos % PAGE


def _rotated(x, s, weight):
    """Heads x [T, H, D] in 32 bits, normed and turned by their positions."""
    if weight is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight
    angle = s["positions"].double()[:, None] * s["inv_freq"].double()
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    rot = 2 * s["inv_freq"].numel()
    part, rest = x[..., :rot], x[..., rot:]
    if s["case"]["rope"] == "half":
        a, b = part[..., :rot // 2], part[..., rot // 2:]
        return torch.cat((a * cos - b * sin, b * cos + a * sin, rest), -1)
    a, b = part[..., 0::2], part[..., 1::2]
    return torch.cat((torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2), rest), -1)


def _store(s, name, x, slots, live):
    """Rows x [T, Hkv, D] in 32 bits into the pool at `slots`, where `live`; other rows keep what they hold."""
    pages = s[name + "_pages"]
    Hkv, D = pages.shape[2:]
    if s["case"]["cache"] == "e4m3":
        codes, scale = _quantise(x)
        scales = s[name + "_scales"]
        page, at = slots // PAGE, slots % PAGE
        scales[page, :, at] = torch.where(live[:, None], scale, scales[page, :, at])
        pages, x, live = pages.view(torch.uint8), codes.view(torch.uint8), live[:, None, None]
    else:
        x, live = x.to(pages.dtype), live[:, None, None]
    flat = pages.view(-1, Hkv, D)
    flat[slots] = torch.where(live, x, flat[slots])


def _plain_append(s):
    q = _rotated(s["q"].float(), s, s["q_norm"])
    k = _rotated(s["k"].float(), s, s["k_norm"])
    live = s["positions"] >= 0
    s["q_out"].copy_(torch.where(live[:, None, None], q.to(s["q_out"].dtype), s["q_out"]))
    seq, i = _rows(s, q.shape[0])
    slots = _slots(s, seq, s["prefix_lens"].long()[seq] + i)
    _store(s, "k", k, slots, live)
    _store(s, "v", s["v"].float(), slots, live)


def _cached(s, name, used):
    """K or V of every sequence in 32 bits, [B, Hkv, L, D]; zero past a sequence's last token."""
    B, pos = used.shape[0], torch.arange(s["reach"], device=used.device)
    live = pos[None] < used[:, None]
    slots = _slots(s, torch.arange(B, device=used.device)[:, None], torch.where(live, pos[None], 0))
    pages = s[name + "_pages"]
    x = pages.view(-1, *pages.shape[2:])[slots] if pages.dtype != torch.float8_e4m3fn else \
        pages.view(torch.uint8).view(-1, *pages.shape[2:])[slots].view(torch.float8_e4m3fn)
    x = x.float()
    if s[name + "_scales"] is not None:
        x = x * s[name + "_scales"][slots // PAGE, :, slots % PAGE][..., None]
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


def _plain_attend(s):
    off, pre = s["chunk_offsets"].long(), s["prefix_lens"].long()
    n = off[1:] - off[:-1]
    i = torch.arange(s["longest"], device=off.device)
    live = i[None] < n[:, None]
    q = s["q"].float()[torch.where(live, off[:-1, None] + i, 0)]
    t = torch.arange(s["reach"], device=off.device)
    seen = t[None, None] <= (pre[:, None] + i)[..., None]
    used = pre + n
    out = _softmax_product(q, _cached(s, "k", used), _cached(s, "v", used), seen)
    seq, at = _rows(s, s["q"].shape[0])
    return out[seq, at].to(s["q"].dtype)


def _ancestry(parents):
    """[B, N, N]: whether node j is node i or an ancestor of it (powers of the parent relation)."""
    N = parents.shape[1]
    j = torch.arange(N, device=parents.device)
    step = (parents[..., None] == j).double() + torch.eye(N, device=parents.device, dtype=torch.float64)
    return torch.linalg.matrix_power(step, 128) > 0


def _plain_verify(s):
    pre, parents = s["prefix_lens"].long(), s["tree_parents"]
    node = parents >= -1
    used = pre + node.sum(1)
    t = torch.arange(s["reach"], device=pre.device)
    j = t[None] - pre[:, None]
    inside = (j >= 0) & (j < parents.shape[1])
    tree = _ancestry(parents).gather(2, torch.where(inside, j, 0)[:, None].expand(-1, parents.shape[1], -1))
    seen = (j < 0)[:, None] | (tree & inside[:, None])
    out = _softmax_product(s["q"].float(), _cached(s, "k", used), _cached(s, "v", used), seen)
    return torch.where(node[..., None, None], out, 0.0).to(s["q"].dtype)


def _plain_commit(s):
    pre, n, path = s["prefix_lens"].long(), s["accept_len"].long(), s["accept_path"].long()
    k = torch.arange(path.shape[1], device=path.device)
    live = k[None] < n[:, None]
    seq = torch.arange(path.shape[0], device=path.device)[:, None].expand_as(path)
    last = pre[:, None] + path.shape[1] - 1
    to = _slots(s, seq, torch.minimum(pre[:, None] + 1 + k, last))
    source = _slots(s, seq, torch.where(live, pre[:, None] + path, pre[:, None]))
    to, source = to[live], source[live]
    for_pages = lambda x: x.view(torch.uint8).view(-1, *x.shape[2:])  # noqa: E731
    kp, vp = for_pages(s["k_pages"]), for_pages(s["v_pages"])
    kp[to], vp[to] = kp[source], vp[source]
    ks, vs = s["k_scales"], s["v_scales"]
    ks[to // PAGE, :, to % PAGE] = ks[source // PAGE, :, source % PAGE]
    vs[to // PAGE, :, to % PAGE] = vs[source // PAGE, :, source % PAGE]
    return (pre + 1 + n).to(torch.int32)


# ------------------------------------------------------------------------------ one pass

def _cache_outputs(s):
    out = {"k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    if s["k_scales"] is not None:
        out.update(k_scales=s["k_scales"], v_scales=s["v_scales"])
    return out


def _workspace(s, size):
    if "workspace" not in s:                                # kept with the inputs, as a program would
        s["workspace"] = torch.empty(size, dtype=torch.uint8, device=s["page_table"].device)
    return s["workspace"]


def _own_append(s):
    import eagle_speculative_tree_gb300 as ts
    ts.tree_chunk_append(s["q"], s["k"], s["v"], s["k_pages"], s["v_pages"], s["page_table"], s["prefix_lens"],
                         s["chunk_offsets"], s["q_out"], positions=s["positions"], q_norm=s["q_norm"],
                         k_norm=s["k_norm"], norm_eps=EPS, inv_freq=s["inv_freq"],
                         rope=ts.ROPE_HALF if s["case"]["rope"] == "half" else ts.ROPE_INTERLEAVED,
                         k_scales=s["k_scales"], v_scales=s["v_scales"],
                         workspace=_workspace(s, ts.append_workspace_bytes()))


def _own_attend(s):
    import eagle_speculative_tree_gb300 as ts
    if "workspace" not in s:
        _workspace(s, ts.chunk_attn_workspace_bytes(ts.chunk_problem(s["q"], s["k_pages"], s["page_table"],
                                                                     s["chunk_offsets"])))
    return ts.tree_chunk_attn(s["q"], s["k_pages"], s["v_pages"], s["page_table"], s["prefix_lens"],
                              s["chunk_offsets"], k_scales=s["k_scales"], v_scales=s["v_scales"],
                              workspace=s["workspace"])


def _own_verify(s):
    import eagle_speculative_tree_gb300 as ts
    if "workspace" not in s:
        _workspace(s, ts.attn_e4m3_workspace_bytes(ts.attn_problem(s["q"], s["k_pages"], s["page_table"])))
    return ts.tree_attn_verify_e4m3(s["q"], s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"], s["page_table"],
                                    s["prefix_lens"], s["tree_parents"], workspace=s["workspace"])


def _own_commit(s):
    import eagle_speculative_tree_gb300 as ts
    return ts.tree_kv_commit_e4m3(s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"], s["page_table"],
                                  s["prefix_lens"], s["accept_path"], s["accept_len"],
                                  workspace=_workspace(s, ts.commit_workspace_bytes()))


def run(state):
    s, op = state, state["case"]["op"]
    if op == "append":
        (_own_append if own else _plain_append)(s)
        return {"q_out": s["q_out"], **_cache_outputs(s)}
    if op == "attend":
        return (_own_attend if own else _plain_attend)(s)
    if op == "verify":
        return (_own_verify if own else _plain_verify)(s)
    new = (_own_commit if own else _plain_commit)(s)
    return {"new_prefix_lens": new, **_cache_outputs(s)}


# ------------------------------------------------------------------------------ work

def work(case):
    c = case
    Hq, Hkv, D = c["q_heads"], c["kv_heads"], c["dim"]
    e = 2 if c["dtype"] == "bf16" else 4
    row = Hkv * (D + 4) if c["cache"] == "e4m3" else Hkv * D * e     # K or V of one cached token
    pre, new = _lengths(c)
    T = sum(new)
    if c["op"] == "append":
        return {"bytes": T * (2 * Hq * D * e + 2 * Hkv * D * e + 2 * row), "flops": T * (Hq + Hkv) * D * 8}
    if c["op"] == "commit":
        moved = sum(max(0, int(0.3 * n)) for n in new)                # about a path's length
        return {"bytes": 4 * moved * row + 64 * len(new), "flops": 0}
    pairs = 0
    if c["op"] == "attend":
        pairs = sum(n * p + n * (n + 1) // 2 for p, n in zip(pre, new))
    else:
        parents = _trees(c, new, max(new))
        for b, n in enumerate(new):
            depth = [1] * n
            for i in range(1, n):
                depth[i] = depth[parents[b, i]] + 1
            pairs += n * pre[b] + sum(depth)
    return {"bytes": 2 * T * Hq * D * e + 2 * row * sum(p + n for p, n in zip(pre, new)), "flops": 4 * D * Hq * pairs}


# ------------------------------------------------------------------------------ 64 bits

def _exact_heads(x, w, pos, inv_freq, layout):
    x = x.double().clone()
    if w is not None:
        x = x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt() * w.double()
    half = inv_freq.numel()
    for j in range(half):
        a, b = (j, j + half) if layout == "half" else (2 * j, 2 * j + 1)
        z = torch.polar(torch.ones_like(pos, dtype=torch.float64), pos.double() * inv_freq[j].double())
        y = torch.complex(x[..., a], x[..., b]) * z[:, None]
        x[..., a], x[..., b] = y.real, y.imag
    return x


def _exact_append(c, s):
    live = torch.nonzero(s["positions"] >= 0).flatten()
    pos = s["positions"][live]
    out = {"q_out": s["q_out"].double()}
    out["q_out"][live] = _exact_heads(s["q"][live], s["q_norm"], pos, s["inv_freq"], c["rope"])
    new = {"k": _exact_heads(s["k"][live], s["k_norm"], pos, s["inv_freq"], c["rope"]), "v": s["v"][live].double()}
    offsets, pre = s["chunk_offsets"].tolist(), s["prefix_lens"].tolist()
    slots = [pre[b] + i for b in range(c["batch"]) for i in range(offsets[b + 1] - offsets[b])]
    seqs = [b for b in range(c["batch"]) for _ in range(offsets[b + 1] - offsets[b])]
    slot = torch.tensor(slots, device=live.device)[live]
    page = s["page_table"].long()[torch.tensor(seqs, device=live.device)[live], slot // PAGE]
    for name in ("k", "v"):
        pages, x = s[name + "_pages"].double(), new[name]
        if c["cache"] == "e4m3":
            scale = (x.abs().amax(-1) / E4M3_MAX).clamp(min=SCALE_MIN)
            x = x / scale[..., None]
            scales = s[name + "_scales"].double()
            scales[page, :, slot % PAGE] = scale
            out[name + "_scales"] = scales
        pages[page, slot % PAGE] = x
        out[name + "_pages"] = pages
    return {k: out[k] for k in ("q_out", "k_pages", "v_pages", "k_scales", "v_scales") if k in out}


def _exact_kv(s, b, n):
    pos = torch.arange(n, device=s["page_table"].device)
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
    N, Hq, D = q.shape
    G = Hq // k.shape[1]
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    for h in range(Hq):
        w = torch.exp((q[:, h].double() @ k[:, h // G].T / D ** 0.5).masked_fill_(hidden, -math.inf))
        out[:, h] = (w @ v[:, h // G]) / w.sum(1, keepdim=True)
    return out


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "append":
        return _exact_append(c, s)
    pre, new = _lengths(c)
    dev = s["page_table"].device
    if c["op"] == "commit":
        path, length = s["accept_path"].tolist(), s["accept_len"].tolist()
        table = s["page_table"].tolist()
        place = lambda b, p: (table[b][p // PAGE], p % PAGE)  # noqa: E731
        moves = [(place(b, pre[b] + path[b][i]), place(b, pre[b] + 1 + i)) for b in range(c["batch"])
                 for i in range(length[b])]
        out = {"new_prefix_lens": torch.tensor([p + 1 + n for p, n in zip(pre, length)], dtype=torch.int32, device=dev)}
        for name in ("k_pages", "v_pages", "k_scales", "v_scales"):
            was = s[name].double()
            x = was.clone()
            for (p0, a0), (p1, a1) in moves:
                if name.endswith("pages"):
                    x[p1, a1] = was[p0, a0]
                else:
                    x[p1, :, a1] = was[p0, :, a0]
            out[name] = x
        return out
    if c["op"] == "attend":
        parts, at = [], 0
        for b in range(c["batch"]):
            k, v = _exact_kv(s, b, pre[b] + new[b])
            t = torch.arange(pre[b] + new[b], device=dev)
            i = torch.arange(new[b], device=dev)
            parts.append(_exact_rows(s["q"][at:at + new[b]], k, v, t[None] > pre[b] + i[:, None]))
            at += new[b]
        return torch.cat(parts)
    parents = s["tree_parents"].tolist()
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=dev)
    for b in range(c["batch"]):
        hidden = np.zeros((new[b], pre[b] + new[b]), dtype=bool)
        hidden[:, pre[b]:] = True
        for i in range(new[b]):
            j = i
            while j >= 0:
                hidden[i, pre[b] + j] = False
                j = parents[b][j]
        k, v = _exact_kv(s, b, pre[b] + new[b])
        out[b, :new[b]] = _exact_rows(s["q"][b, :new[b]], k, v, torch.from_numpy(hidden).to(dev))
    return out
