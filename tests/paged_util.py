"""Helpers of the paged-cache tests: random paged caches, and attention, rotation and e4m3
rounding in 64 bits, without the library."""
from __future__ import annotations

import math

import torch


def pages_of(n, ps):
    return -(-n // ps)


class Cache:
    """A paged cache whose rows are known in 64 bits. Unused page rows hold NaN (bf16) or codes
    with a NaN scale (e4m3), unused table entries are out of range."""

    def __init__(self, G, kind, hkv, d, page, dtype, kv_lens, seed=0, extra_pages=2, device="cuda", keep=None,
                 scale=1.0):
        """keep[b]: first position of sequence b that is held (earlier pages are dropped)."""
        self.G, self.kind, self.hkv, self.d, self.ps, self.dtype, self.device = G, kind, hkv, d, page, dtype, device
        gen = torch.Generator().manual_seed(seed)
        self.lens = list(kv_lens)
        B = len(self.lens)
        keep = keep or [0] * B
        blocks = [pages_of(n, page) for n in self.lens]
        self.num_pages = sum(blocks) + extra_pages
        order = torch.randperm(self.num_pages, generator=gen).tolist()
        self.max_blocks = max(max(blocks), 1) + 1
        table = torch.full((B, self.max_blocks), 1 << 30, dtype=torch.int32)
        at = 0
        for b, n in enumerate(blocks):
            for i in range(keep[b] // page, n):
                table[b, i] = order[at]
                at += 1
        self.table = table.to(device)
        self.rows, self.pages, self.scales = {}, {}, {}
        for t in ("k", "v")[: 1 if kind == G.GLOBAL else 2]:
            pool = torch.full((self.num_pages, hkv, page, d), math.nan, dtype=torch.float32)
            sc = torch.full((self.num_pages, hkv, page), math.nan)
            self.rows[t] = []
            for b, n in enumerate(self.lens):
                x = (torch.randn(n, hkv, d, generator=gen) * scale).to(torch.bfloat16).float()
                if dtype == "e4m3":
                    x, s = quantise64(x.double())
                    codes = (x / s).float()
                for i in range(keep[b] // page, blocks[b]):
                    lo, hi = max(i * page, keep[b]), min(n, (i + 1) * page)
                    dst = pool[int(table[b, i]), :, lo - i * page: hi - i * page]
                    dst.copy_((codes if dtype == "e4m3" else x)[lo:hi].transpose(0, 1))
                    if dtype == "e4m3":
                        sc[int(table[b, i]), :, lo - i * page: hi - i * page] = s[lo:hi, :, 0].float().T
                self.rows[t].append(x.double().to(device))
            if dtype == "e4m3":
                self.pages[t] = pool.to(torch.float8_e4m3fn).to(device)
                self.scales[t] = sc.to(device)
            else:
                self.pages[t] = pool.to(torch.bfloat16).to(device)
        self.handle = G.paged_cache(self.pages["k"], self.pages.get("v"), self.table, k_scales=self.scales.get("k"),
                                    v_scales=self.scales.get("v"))


def quantise64(x):
    """(values held, scales [..., 1]) of rows of x in e4m3 with a power-of-two scale per row."""
    amax = x.abs().amax(-1, keepdim=True)
    m, e = torch.frexp(amax)
    k = torch.where(m <= 0.875, e - 9, e - 8).clamp(min=-126)
    s = torch.where(amax > 0, torch.ldexp(torch.ones_like(x[..., :1]), k), torch.ones_like(amax))
    y = x / s
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    y = torch.round(y / step) * step
    y = torch.where(s == 2.0 ** 120, y.clamp(-240.0, 240.0), y)  # 256 * 2^120 is no fp32 number
    return y * s, s


def turn64(x, pos, r, base):
    """Rows x [n, h, d] with their first r pairs (j, j + d/2) turned by pos * base^(-2j/d)."""
    d = x.shape[-1]
    y = x.double().clone()
    if r:
        theta = torch.pow(torch.tensor(float(base), dtype=torch.float64, device=x.device),
                          -2.0 * torch.arange(r, dtype=torch.float64, device=x.device) / d)
        a = pos.double()[:, None, None] * theta
        c, s = torch.cos(a), torch.sin(a)
        x0, x1 = y[..., :r].clone(), y[..., d // 2: d // 2 + r].clone()
        y[..., :r], y[..., d // 2: d // 2 + r] = x0 * c - x1 * s, x0 * s + x1 * c
    return y


def attend64(q, k, v, ctx, window, r, base, scale, turn_keys):
    """q [n, Hq, d] un-rotated at positions ctx.., k / v [ctx + n, Hkv, d]: output and log-sum-exp."""
    n, hq, d = q.shape
    g = hq // k.shape[1]
    pq = torch.arange(ctx, ctx + n, device=q.device)
    pk = torch.arange(k.shape[0], device=q.device)
    q = turn64(q, pq, r, base)
    kk = turn64(k, pk, r, base) if turn_keys else k
    s = torch.einsum("nhd,khd->hnk", q, kk.repeat_interleave(g, 1)) * scale
    hide = pk[None] > pq[:, None]
    if window:
        hide = hide | (pk[None] <= pq[:, None] - window)
    s = s.masked_fill(hide, -math.inf)
    out = torch.einsum("hnk,khd->nhd", torch.softmax(s, -1), v.repeat_interleave(g, 1))
    return out, torch.logsumexp(s, -1).T


def run_attend(G, cache, p, q, nq, ctx, out_f32=True, pad_rows=0, lse=True, stream=None, max_q=None, max_len=None):
    """One call; returns (out, lse), whose rows past the last sequence were filled with 7."""
    import itertools
    B, T = len(nq), sum(nq) + pad_rows
    cu = torch.tensor([0] + list(itertools.accumulate(nq)), dtype=torch.int32, device="cuda")
    lens = torch.tensor(ctx, dtype=torch.int32, device="cuda")
    pp = G.GemmaAttnParams.from_buffer_copy(p)
    pp.out_dtype = G.OUT_F32 if out_f32 else G.OUT_BF16
    out = torch.full((T, pp.num_q_heads, pp.head_dim), 7.0, dtype=torch.float32 if out_f32 else torch.bfloat16, device="cuda")
    ls = torch.full((T, pp.num_q_heads), 7.0, device="cuda") if lse else None
    mq, ml = max(nq) if max_q is None else max_q, max(ctx) if max_len is None else max_len
    nb = G.gemma_attn_paged_workspace_size(pp, cache.handle, B, T, mq, ml)
    # scratch that holds NaN: nothing in it may be relied on
    ws = torch.full((max(nb, 256) // 4 + 64,), math.nan, device="cuda")
    G.gemma_attn_paged_attend(pp, cache.handle, q, cu, lens, out, ls, B, T, mq, ml, ws, nb, stream=stream)
    return out, ls
