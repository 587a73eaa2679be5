"""Problems and float64 results of the tests of sliding windows and shared prefixes."""
from __future__ import annotations

import math

import numpy as np
import torch

from oracle import window as ow

from chunk_util import Problem, make


def drop_pages(p: Problem, window: int, sinks: int) -> int:
    """Take the pages that no row sees out of the page table (an id that no pool has) and fill them
    with NaN, as of a sequence that gave them back; returns how many."""
    table = p.page_table.cpu().numpy()
    gone = 0
    for b, (S, n) in enumerate(zip(p.prefix, p.new)):
        for i in range((S + n + 15) // 16):
            lo, hi = 16 * i, min(16 * i + 16, S + n)
            if hi <= S - window + 1 and lo >= sinks:
                page = int(table[b, i])
                for pages in (p.k_pages, p.v_pages):
                    if pages.element_size() == 1:
                        pages.view(torch.uint8)[page] = 0x7f
                    else:
                        pages[page] = math.nan
                table[b, i] = -1 - i
                gone += 1
    p.page_table.copy_(torch.from_numpy(table))
    return gone


def make_shared(device, groups, new, hq, hkv, dim, dtype, e4m3=False, seed=0, lead=0, tail=0, rows=None, copies=False):
    """groups: for each, its shared length and its sequences' own cached lengths (behind the shared
    tokens).  Page tables name the same pages for a group's whole shared pages, and pages of equal
    content where the shared length ends inside one (everywhere, with `copies`).  Returns the problem,
    group_offsets and shared_lens."""
    prefix = [s + o for s, own in groups for o in own]
    p = make(device, prefix, new, hq, hkv, dim, dtype, e4m3, seed=seed, lead=lead, tail=tail, rows=rows)
    table = p.page_table.cpu().numpy()
    starts, b = [0], 0
    raw = lambda t: t.view(torch.uint8) if t.element_size() == 1 else t  # noqa: E731
    for s, own in groups:
        first = b
        for k in range(1, len(own)):
            for i in range((s + 15) // 16):
                n = min(16, s - 16 * i)
                if n == 16 and not copies:
                    table[first + k, i] = table[first, i]
                    continue
                a, z = int(table[first, i]), int(table[first + k, i])
                for pages, scales in ((p.k_pages, p.k_scales), (p.v_pages, p.v_scales)):
                    raw(pages)[z, :n] = raw(pages)[a, :n]
                    if scales is not None:
                        scales[z, :, :n] = scales[a, :, :n]
        b += len(own)
        starts.append(b)
    p.page_table.copy_(torch.from_numpy(table))
    ints = lambda a: torch.tensor(a, dtype=torch.int32, device=device)  # noqa: E731
    return p, ints(starts), ints([s for s, _ in groups])


def rows64(p: Problem, q, b, seen):
    """Sequence b in 64 bits: q [n][Hq][D], seen [n][L] (numpy) -> (out, spread, reach) of
    oracle.chunk.attend; only tokens that some row sees are looked at.  NaN where a row sees a NaN or
    an infinity in V."""
    n, H, D = q.shape
    t = torch.from_numpy(np.flatnonzero(seen.any(0))).to(q.device)
    seen = torch.from_numpy(seen).to(q.device)[:, t]
    page, at = p.page_table[b].long()[t // 16], t % 16
    kv = []
    for pages, scales in ((p.k_pages, p.k_scales), (p.v_pages, p.v_scales)):
        x = pages.view(torch.uint8)[page, at].view(pages.dtype) if pages.element_size() == 1 else pages[page, at]
        x = x.double()
        kv.append(x if scales is None else x * scales.transpose(1, 2)[page, at].double()[..., None])
    out, spread = (torch.empty((n, H, D), dtype=torch.float64, device=q.device) for _ in "os")
    reach = torch.empty((n, H), dtype=torch.float64, device=q.device)
    G = H // kv[0].shape[1]
    for h in range(H):
        k, v, x = kv[0][:, h // G], kv[1][:, h // G], q[:, h].double()
        s = (x @ torch.where(k.isfinite(), k, 0.0).T / math.sqrt(D)).masked_fill(~seen, -math.inf)
        key = seen.double() @ (~k.isfinite()).any(1).double()[:, None] > 0       # such a row is NaN throughout
        w = torch.softmax(s, -1)
        # a value that is not finite reaches the rows that see it, and no product with a weight of 0 may bring it to others
        odd = seen.double() @ (~v.isfinite()).double() > 0
        plain = torch.where(v.isfinite(), v, 0.0)
        out[:, h], spread[:, h] = (w @ plain).masked_fill(odd | key, math.nan), w @ plain.abs()
        reach[:, h] = (x.abs() @ torch.where(k.isfinite(), k, 0.0).abs().T / math.sqrt(D)).masked_fill(~seen, 0).amax(-1)
    return out, spread, reach


def chunk64(p: Problem, window: int = 1 << 30, sinks: int = 0):
    """(out, spread, reach) of every packed row, as numpy arrays."""
    parts = []
    offsets = p.chunk_offsets.tolist()
    for b, (S, n) in enumerate(zip(p.prefix, p.new)):
        if n:
            parts.append(rows64(p, p.q[offsets[b]:offsets[b] + n], b, ow.seen_by_chunk(S, n, window, sinks)))
    return tuple(torch.cat(x).cpu().numpy() for x in zip(*parts))


def tree64(p: Problem, q, parents, window: int = 1 << 30, sinks: int = 0):
    """The same for padded trees q [B][N][Hq][D]; rows of padding slots are zeros."""
    res = [torch.zeros(s, dtype=torch.float64) for s in (q.shape, q.shape, q.shape[:3])]
    for b, (S, n) in enumerate(zip(p.prefix, p.new)):
        seen = ow.seen_by_tree(S, [int(x) for x in parents[b][:n]], window, sinks)
        for whole, part in zip(res, rows64(p, q[b, :n], b, seen)):
            whole[b, :n] = part.cpu()
    return tuple(x.numpy() for x in res)
