"""Problems and error bounds of the chunk and 8-bit cache tests."""
from __future__ import annotations

import math
from dataclasses import dataclass

import numpy as np
import torch

from oracle import chunk as och

U_BF16 = 2.0 ** -8            # a rounding to bf16 is off by at most this share of the value
U_F32 = 2.0 ** -24
U_E4M3 = 2.0 ** -4


@dataclass
class Problem:
    """Inputs of one batch on the device, and their float64 values."""
    prefix: list
    new: list
    q: torch.Tensor              # [T][Hq][D]
    k_pages: torch.Tensor
    v_pages: torch.Tensor
    k_scales: torch.Tensor | None
    v_scales: torch.Tensor | None
    page_table: torch.Tensor
    prefix_lens: torch.Tensor
    chunk_offsets: torch.Tensor

    def pools64(self):
        if self.k_scales is None:
            return self.k_pages.double().cpu().numpy(), self.v_pages.double().cpu().numpy()
        return tuple(och.dequantise(p.view(torch.uint8).cpu().numpy(), s.cpu().numpy())
                     for p, s in ((self.k_pages, self.k_scales), (self.v_pages, self.v_scales)))

    def scales(self):
        return {} if self.k_scales is None else {"k_scales": self.k_scales, "v_scales": self.v_scales}


def make(device, prefix, new, hq, hkv, dim, dtype, e4m3=False, seed=0, spare=3, lead=0, tail=0, rows=None,
         extra_pages=0):
    """Random pools and queries.  Slots past a sequence's last token and the spare pages hold
    NaN.  `lead` / `tail`: rows of q before the first and behind the last sequence."""
    rng = np.random.default_rng([seed, 77])
    B = len(prefix)
    rows = rows or new
    need = [(p + n + 15) // 16 for p, n in zip(prefix, rows)]
    pool = sum(need) + spare
    order = rng.permutation(pool).astype(np.int32)
    table = np.full((B, max(max(need), 1) + extra_pages), pool + 5, dtype=np.int32)   # unused entries: no page
    used = np.zeros((pool, 16), dtype=bool)
    at = 0
    for b in range(B):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
        t = np.arange(prefix[b] + new[b])
        used[table[b][t // 16], t % 16] = True
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    T = lead + sum(rows) + tail
    q = torch.from_numpy(rng.standard_normal((T, hq, dim)).astype(np.float32)).to(device).to(dt)
    pools, scales = [], []
    for _ in range(2):
        x = rng.standard_normal((pool, 16, hkv, dim)) * np.exp(rng.normal(size=(pool, 16, hkv, 1)) * 0.5 * e4m3)
        if e4m3:
            codes, sc = och.quantise(x)
            codes[~used] = 0x7f
            sc = sc.transpose(0, 2, 1).astype(np.float32)
            sc[~used[:, None, :].repeat(hkv, 1)] = np.nan
            pools.append(torch.from_numpy(codes).to(device).view(torch.float8_e4m3fn))
            scales.append(torch.from_numpy(np.ascontiguousarray(sc)).to(device))
        else:
            x[~used] = np.nan
            pools.append(torch.from_numpy(x.astype(np.float32)).to(device).to(dt))
            scales.append(None)
    ints = lambda a: torch.from_numpy(np.asarray(a, dtype=np.int32)).to(device)  # noqa: E731
    offsets = lead + np.concatenate(([0], np.cumsum(rows)))
    return Problem(list(prefix), list(new), q, pools[0], pools[1], scales[0], scales[1], ints(table), ints(prefix),
                   ints(offsets))


def attention_bound(ref, spread, reach, tokens, dim, dtype, tensor_cores):
    """How far a kernel's rows may be from the float64 ones: [.., H, D].

    A score is a sum of `dim` products in 32 bits (tensor cores may truncate: 2^-23 a step)
    and two scalings: it is off by ds <= (dim + 8) 2^-23 reach.  Every weight is then off by
    exp(2 ds) - 1 and by 2^-21 of exp2 and the running rescales; on tensor cores the weight
    (times V's scale, over 8-bit V) is rounded once to bf16 before it meets V, half a step of
    which is 2^-8 of the value, while the sum that divides it is not: w + 2^-8.  Over 8-bit
    V the codes themselves are exact in bf16.  A sum of `tokens` terms in 32 bits adds
    tokens 2^-23.  The result is rounded once."""
    ds = (dim + 8) * 2.0 ** -23 * reach[..., None]
    w = np.expm1(2 * ds) + 2.0 ** -21 + tokens * 2.0 ** -23
    if tensor_cores:
        w = w + U_BF16
    out = U_BF16 if dtype == "bf16" else U_F32
    return w * spread * 1.0001 + out * (np.abs(ref) + w * spread) + 1e-30


def check_attention(got, ref, spread, reach, tokens, dim, dtype, tensor_cores):
    g = got.double().cpu().numpy()
    assert np.array_equal(np.isnan(g), np.isnan(ref)), "NaN in other places than the definition's"
    live = ~np.isnan(ref)
    bound = attention_bound(ref, spread, reach, tokens, dim, dtype, tensor_cores)
    err = np.abs(g - ref)
    bad = live & ~(err <= bound)
    assert not bad.any(), f"{bad.sum()} of {live.sum()} elements out of bounds, worst {np.nanmax(err / bound):.3g} times"


def make_8bit(device, prefix, new, hq, hkv, dim, seed=0, rows=None, spread=1.0):
    """As make(), for larger problems over 8-bit pools, drawn on the device: codes of normal
    values, scales 0.01 x 10^u with u even in [-spread, spread] for each token and kv head, so that a
    scale of another token is far from the right one."""
    gen = torch.Generator(device=device)
    gen.manual_seed(seed)
    rows = rows or new
    need = [(p + n + 15) // 16 for p, n in zip(prefix, rows)]
    pool = sum(need) + 3
    order = torch.randperm(pool, generator=gen, device=device).to(torch.int32)
    table = torch.full((len(prefix), max(need)), pool + 5, dtype=torch.int32, device=device)
    used = torch.zeros((pool, 16), dtype=torch.bool, device=device)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
        t = torch.arange(prefix[b] + new[b], device=device)
        used[table[b].long()[t // 16], t % 16] = True
    pools, scales = [], []
    for _ in range(2):
        x = torch.randn((pool, 16, hkv, dim), generator=gen, device=device) * 100
        codes = x.clamp(-448, 448).to(torch.float8_e4m3fn)
        codes.view(torch.uint8)[~used] = 0x7f
        u = 2 * torch.rand((pool, hkv, 16), generator=gen, device=device) - 1
        sc = 0.01 * 10.0 ** (spread * u)
        sc.transpose(1, 2)[~used] = math.nan
        pools.append(codes)
        scales.append(sc)
    scales[0] *= 0.1                                           # scores of a few units
    q = torch.randn((sum(rows), hq, dim), generator=gen, device=device).to(torch.bfloat16)
    ints = lambda a: torch.tensor(a, dtype=torch.int32, device=device)  # noqa: E731
    offsets = np.concatenate(([0], np.cumsum(rows))).tolist()
    return Problem(list(prefix), list(new), q, pools[0], pools[1], scales[0], scales[1], table, ints(prefix), ints(offsets))


def attend64(p, q, b, seen):
    """Sequence b in 64 bits, all of its rows at once: q [n][Hq][D], seen [n][L] -> (out, spread, reach)
    of oracle.chunk.attend as tensors; NaN where a row sees a NaN or an infinity in V."""
    n, H, D = q.shape
    t = torch.arange(seen.shape[1], device=q.device)
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
        s = (x @ k.T / math.sqrt(D)).masked_fill(~seen, -math.inf)
        w = torch.softmax(s, -1)
        # a value that is not finite reaches the rows that see it, and no product with a weight of 0 may bring it to others
        odd = seen.double() @ (~v.isfinite()).double() > 0
        plain = torch.where(v.isfinite(), v, 0.0)
        out[:, h], spread[:, h] = (w @ plain).masked_fill(odd, math.nan), w @ plain.abs()
        reach[:, h] = (x.abs() @ k.abs().T / math.sqrt(D)).masked_fill(~seen, 0).amax(-1)
    return out, spread, reach


def causal64(p):
    """(out, spread, reach) of every packed row, as numpy arrays."""
    parts = []
    offsets = p.chunk_offsets.tolist()
    for b, (S, n) in enumerate(zip(p.prefix, p.new)):
        if n == 0:
            continue
        t = torch.arange(S + n, device=p.q.device)
        i = torch.arange(n, device=p.q.device)
        parts.append(attend64(p, p.q[offsets[b]:offsets[b] + n], b, t[None] <= S + i[:, None]))
    return tuple(torch.cat(x).cpu().numpy() for x in zip(*parts))


def tree64(p, q, parents):
    """The same for padded trees q [B][N][Hq][D]; rows of padding slots are zeros."""
    out, spread, reach = (torch.zeros(s, dtype=torch.float64) for s in (q.shape, q.shape, q.shape[:3]))
    for b, (S, n) in enumerate(zip(p.prefix, p.new)):
        seen = torch.zeros((n, S + n), dtype=torch.bool)
        seen[:, :S] = True
        for i in range(n):
            j = i
            while j >= 0:
                seen[i, S + j] = True
                j = int(parents[b, j])
        for whole, part in zip((out, spread, reach), attend64(p, q[b, :n], b, seen.to(q.device))):
            whole[b, :n] = part.cpu()
    return out.numpy(), spread.numpy(), reach.numpy()
