"""Cases of the paged-cache operators and of the draft verification, with their plain forms.

Three operators of serving:

- ``attend``: attention of a chunk of new tokens (one token to thousands, ragged over the
  batch) over a paged key/value cache that already holds the chunk's own rows. Sliding-window
  layers keep rotated keys and separate values; global layers keep one un-rotated K=V row
  that is rotated (the first pairs only) for the scores.
- ``write``: new rows written into the pages (keys of sliding-window layers rotated at their
  positions), in bf16 or quantised to e4m3 with one power-of-two scale per row and KV head,
  and the rows read back; ``read``: whole sequences read back from the pages.
- ``draft``: verification of drafted tokens against the target's probabilities from given
  random numbers, with the next token drawn by an exponential race.

``run`` computes them with elementary torch operations in 32 bits, or, where ``own`` is set,
through the framework's calls.
"""
import math
import random

import torch

own = False

# Head layouts (query heads, KV heads, head dim) of the framework's workloads and a few
# others of its supported range.
LOCAL_HEADS = [(8, 4, 256), (32, 16, 256), (4, 2, 128), (6, 2, 64), (12, 1, 128), (16, 16, 64)]
GLOBAL_HEADS = [(8, 1, 512), (32, 4, 512), (16, 2, 256), (8, 1, 64), (20, 4, 128)]
PAGES = [16, 32, 64, 128, 256]


def _attend(name, kind, heads, page, dtype, batch, nq, ctx, window=0, mixed=False, lens_seed=7):
    hq, hkv, d = heads
    return {"name": name, "op": "attend", "kind": kind, "hq": hq, "hkv": hkv, "d": d, "page": page, "dtype": dtype,
            "batch": batch, "nq_lo": nq[0], "nq_hi": nq[1], "ctx_lo": ctx[0], "ctx_hi": ctx[1], "window": window,
            "mixed": mixed, "lens_seed": lens_seed}


def _rows(name, op, kind, heads, page, dtype, batch, nq, ctx, window=0, lens_seed=7):
    return dict(_attend(name, kind, heads, page, dtype, batch, nq, ctx, window, False, lens_seed), op=op)


def _draft(name, batch, draft, vocab, dtype, onehot=False):
    return {"name": name, "op": "draft", "batch": batch, "draft": draft, "vocab": vocab, "dtype": dtype, "onehot": onehot}


def listed():
    return [
        # one user's next token on a small sliding-window layer: nothing but latency
        _attend("decode_one_local", "local", (8, 4, 256), 16, "bf16", 1, (1, 1), (100, 100), 512),
        # a small batch far into long documents, on the layer kind that reads the whole history
        _attend("decode_global_32k", "global", (32, 4, 512), 64, "bf16", 8, (1, 1), (30000, 32768)),
        # a full serving batch at mixed ages on a sliding-window layer with an 8-bit cache
        _attend("decode_local_e4m3", "local", (32, 16, 256), 32, "e4m3", 64, (1, 1), (500, 8000), 1024),
        # four drafted tokens per sequence verified against ragged 8-bit histories
        _attend("verify_global_e4m3", "global", (32, 4, 512), 64, "e4m3", 16, (5, 5), (1024, 32768)),
        # a long prompt's chunk late in its prefill: products, not bytes
        _attend("chunk_global_bf16", "global", (32, 4, 512), 64, "bf16", 1, (2048, 2048), (29777, 29777)),
        # the same on a sliding-window layer, three prompts at once
        _attend("chunk_local_bf16", "local", (32, 16, 256), 16, "bf16", 3, (700, 2100), (1, 9000), 1024),
        # a scheduler's step: some sequences decode, others run a prompt chunk, 8-bit cache
        _attend("mixed_global_e4m3", "global", (32, 4, 512), 128, "e4m3", 12, (20, 256), (17, 16000), 0, True),
        # one decode step's rows of a full batch quantised into the pages, and read back
        _rows("write_step_e4m3", "write", "local", (32, 16, 256), 16, "e4m3", 64, (1, 1), (30, 9000), 1024),
        # prompt chunks quantised into the pages of a global layer, and read back
        _rows("write_chunk_e4m3", "write", "global", (32, 4, 512), 64, "e4m3", 6, (1000, 8191), (0, 5000)),
        # whole sequences read back in bf16 from an 8-bit cache (to move them to another replica)
        _rows("read_e4m3", "read", "local", (32, 16, 256), 64, "e4m3", 3, (0, 0), (9000, 33333), 1024),
        # one user's four drafted tokens
        _draft("draft_one", 1, 4, 262144, "f32"),
        # a full batch's drafted tokens, probabilities kept in 16 bits
        _draft("draft_batch", 64, 7, 262144, "bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    cap = {op: max(work(c)["flops"] + work(c)["bytes"] * 100 for c in listed() if c["op"] == op) for op in ("attend", "write", "read", "draft")}
    while True:
        op = rng.choice(["attend", "attend", "attend", "write", "read", "draft"])
        if op == "draft":
            case = _draft("", _log(rng, 1, 64), rng.randint(1, 9), _log(rng, 1000, 262144), rng.choice(["f32", "bf16"]), rng.random() < 0.3)
        else:
            kind = rng.choice(["local", "global"])
            heads = rng.choice(LOCAL_HEADS if kind == "local" else GLOBAL_HEADS)
            page, dtype, window = rng.choice(PAGES), rng.choice(["bf16", "e4m3"]), _log(rng, 16, 1024)
            if kind == "global":
                window = 0
            batch, hi = _log(rng, 1, 32), _log(rng, 8, 24000)
            ctx = (_log(rng, 1, hi), hi)
            lens_seed = rng.randrange(1 << 30)
            if op == "attend":
                mode = rng.choice(["decode", "verify", "chunk", "mixed"])
                n = {"decode": 1, "verify": rng.randint(2, 9), "chunk": _log(rng, 20, 2048), "mixed": _log(rng, 4, 600)}[mode]
                nq = (n, n) if mode in ("decode", "verify") else (max(1, n // rng.randint(1, 9)), n)
                case = _attend("", kind, heads, page, dtype, batch, nq, ctx, window, mode == "mixed", lens_seed)
                # the plain form holds every score of the padded batch
                if batch * heads[0] * n * (hi + n if not window else window + n) > 2.2e9 or batch * heads[1] * heads[2] * hi > 1.0e9:
                    continue
            else:
                n = _log(rng, 1, 8192)
                nq = (max(1, n // rng.randint(1, 5)), n) if op == "write" else (0, 0)
                case = _rows("", op, kind, heads, page, dtype, batch, nq, ctx, window, lens_seed)
                if batch * heads[1] * heads[2] * (hi + n) > 1.0e9:
                    continue
        del case["name"]
        w = work(case)
        if w["flops"] + w["bytes"] * 100 <= cap[op]:
            return case


def _lens(case):
    """New tokens and tokens before them, per sequence: of the case alone."""
    r = random.Random(case["lens_seed"])
    pick = lambda lo, hi: lo if hi <= lo else _log(r, max(lo, 1), hi)  # noqa: E731
    ctx = [pick(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["batch"])]
    nq = [pick(case["nq_lo"], case["nq_hi"]) for _ in range(case["batch"])]
    if case["mixed"]:
        nq = [1 if i % 2 else n for i, n in enumerate(nq)]
    return nq, ctx


def _rope(case):
    return (0.25, 1e6) if case["kind"] == "global" else (1.0, 1e4)


def _pairs(case):
    return int(_rope(case)[0] * case["d"] / 2)


def work(case):
    if case["op"] == "draft":
        e = 4 if case["dtype"] == "f32" else 2
        rows = (1 if case["onehot"] else 2) * e + 4  # the stopping position's rows and the noise
        return {"bytes": case["batch"] * (case["vocab"] * rows + 16 * case["draft"]), "flops": 4 * case["batch"] * case["vocab"]}
    nq, ctx = _lens(case)
    d, hq, hkv, w = case["d"], case["hq"], case["hkv"], case["window"]
    tensors = 1 if case["kind"] == "global" else 2
    row = hkv * d * (2 if case["dtype"] == "bf16" else 1) + (0 if case["dtype"] == "bf16" else 4 * hkv)
    if case["op"] == "write":  # bf16 rows in, cache rows out, cache rows in, bf16 rows out
        n = sum(nq)
        back = row + hkv * d * 2 if case["dtype"] == "e4m3" else 0
        return {"bytes": tensors * n * (hkv * d * 2 + row + back), "flops": 8 * tensors * n * hkv * d}
    if case["op"] == "read":
        return {"bytes": tensors * sum(ctx) * (row + hkv * d * 2), "flops": tensors * sum(ctx) * hkv * d}
    flops, rows = 0, 0
    for n, c in zip(nq, ctx):
        if w:
            rows += n + min(c, w - 1)
            flops += 4 * d * hq * sum(min(c + i + 1, w) for i in range(n))
        else:
            rows += n + c
            flops += 4 * d * hq * (n * c + n * (n + 1) // 2)
    return {"bytes": tensors * rows * row + sum(nq) * hq * d * 4, "flops": flops}


def _quantise(x):
    """e4m3 codes and the power-of-two scale of each row (last dimension): the smallest one
    with |x| <= 448 * scale; a row with a non-finite value gets a NaN scale."""
    amax = x.abs().amax(-1, keepdim=True)
    m, e = torch.frexp(amax)
    k = torch.where(m <= 0.875, e - 9, e - 8).clamp(min=-126)
    scale = torch.ldexp(torch.ones_like(amax), torch.where(amax > 0, k, torch.zeros_like(k)))
    scale = torch.where(torch.isfinite(amax), scale, torch.full_like(scale, math.nan))
    codes = torch.where(torch.isfinite(scale), x / scale, torch.zeros_like(x)).to(torch.float8_e4m3fn)
    return codes, scale.squeeze(-1)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    randn = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    if case["op"] == "draft":
        b, n, v = case["batch"], case["draft"], case["vocab"]
        dt = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
        expo = lambda *s: torch.empty(*s, device="cuda").exponential_(generator=gen)  # noqa: E731
        logits = randn(b, n + 1, v) * 3
        target = torch.softmax(logits, -1)
        near = torch.softmax(logits[:, :n] + 0.4 * randn(b, n, v), -1)
        del logits
        tokens = (near / expo(b, n, v)).argmax(-1).to(torch.int32)
        return {"case": dict(case), "target": target.to(dt), "draft": None if case["onehot"] else near.to(dt), "tokens": tokens,
                "lens": torch.randint(0, n + 1, (b,), generator=gen, device="cuda", dtype=torch.int32).clamp(min=min(n, 1)),
                "uniforms": torch.rand(b, n, generator=gen, device="cuda"), "noise": expo(b, v)}
    nq, ctx = _lens(case)
    d, hq, hkv, ps, b = case["d"], case["hq"], case["hkv"], case["page"], case["batch"]
    blocks = [max(1, -(-(n + c) // ps)) for n, c in zip(nq, ctx)]
    num = sum(blocks) + 3
    order = torch.randperm(num, generator=gen, device="cuda").to(torch.int32)
    table = torch.zeros(b, max(blocks), dtype=torch.int32, device="cuda")
    at = 0
    for i, n in enumerate(blocks):
        table[i, :n] = order[at:at + n]
        at += n
    s = {"case": dict(case), "nq": nq, "ctx": ctx, "total": sum(nq), "table": table}
    for t in ("k", "v")[: 1 if case["kind"] == "global" else 2]:
        pages = randn(num, hkv, ps, d).to(torch.bfloat16)
        if case["dtype"] == "e4m3":
            pages, s[t + "_scales"] = _quantise(pages.float())
        s[t + "_pages"] = pages
        if case["op"] == "write":
            s["new_" + t] = randn(s["total"], hkv, d).to(torch.bfloat16)
    if case["op"] == "attend":
        s["q"] = randn(s["total"], hq, d).to(torch.bfloat16)
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    s["cu"] = ints([0] + [sum(nq[: i + 1]) for i in range(b)])
    s["lens"] = ints(ctx)
    s["cu_ctx"] = ints([0] + [sum(ctx[: i + 1]) for i in range(b)])
    s["zeros"] = ints([0] * b)
    return s


# ---------------------------------------------------------------------- plain forms

def _turn(x, pos, pairs, base):
    """The first `pairs` pairs (j, j + d/2) of the last dimension turned by pos * base^(-2j/d); `pos` has x's leading dimensions."""
    d = x.shape[-1]
    if pairs == 0:
        return x
    freq = torch.pow(torch.tensor(base, dtype=torch.float64, device=x.device), -2.0 * torch.arange(pairs, device=x.device, dtype=torch.float64) / d)
    angle = torch.remainder(pos.double().unsqueeze(-1) * freq, 2 * math.pi)
    c, s = torch.cos(angle).to(x.dtype), torch.sin(angle).to(x.dtype)
    x0, x1 = x[..., :pairs], x[..., d // 2: d // 2 + pairs]
    return torch.cat([x0 * c - x1 * s, x[..., pairs: d // 2], x0 * s + x1 * c, x[..., d // 2 + pairs:]], -1)


def _tokens(s):
    """Sequence and place in the sequence of each new token."""
    t = torch.arange(s["total"], device="cuda")
    seq = torch.searchsorted(s["cu"][1:].long(), t, right=True)
    return seq, t - s["cu"].long()[seq]


def _paged(s, name, pos):
    """Rows [batch, n, kv_heads, d] at positions pos [batch, n], in 32 bits."""
    ps = s["case"]["page"]
    page = torch.gather(s["table"].long(), 1, (pos // ps).clamp(0, s["table"].shape[1] - 1))
    rows = s[name + "_pages"][page, :, pos % ps].float()
    if name + "_scales" in s:
        rows = rows * s[name + "_scales"][page, :, pos % ps].unsqueeze(-1)
    return rows


def _plain_attend(s):
    c = s["case"]
    hq, hkv, d, w, nmax = c["hq"], c["hkv"], c["d"], c["window"], max(s["nq"])
    g = hq // hkv
    lens, nq = s["lens"].long(), torch.diff(s["cu"].long())
    first = (lens - w + 1).clamp(min=0) if w else torch.zeros_like(lens)
    width = max((min(k, w - 1) if w else k) + n for k, n in zip(s["ctx"], s["nq"]))
    pos_k = first[:, None] + torch.arange(width, device="cuda")
    held = pos_k < (lens + nq)[:, None]
    k = torch.where(held[:, :, None, None], _paged(s, "k", pos_k), 0.0)
    v = k if c["kind"] == "global" else torch.where(held[:, :, None, None], _paged(s, "v", pos_k), 0.0)
    i = torch.arange(nmax, device="cuda")
    pos_q = lens[:, None] + i
    q = s["q"].float()[(s["cu"].long()[:-1, None] + i).clamp(max=s["total"] - 1)]  # [batch, nmax, hq, d]
    base = _rope(c)[1]
    q = _turn(q, pos_q[:, :, None], _pairs(c), base)
    if c["kind"] == "global":
        k = _turn(k, pos_k[:, :, None], _pairs(c), base)
    q = q.reshape(-1, nmax, hkv, g, d).permute(0, 2, 1, 3, 4).reshape(-1, hkv, nmax * g, d)
    scores = (torch.matmul(q, k.permute(0, 2, 3, 1)) * d ** -0.5).reshape(-1, hkv, nmax, g, width)
    seen = held[:, None] & (pos_k[:, None] <= pos_q[:, :, None])
    if w:
        seen = seen & (pos_k[:, None] > pos_q[:, :, None] - w)
    scores.masked_fill_(~seen[:, None, :, None, :], -math.inf)
    top = scores.amax(-1, keepdim=True)
    scores.sub_(torch.where(torch.isfinite(top), top, 0.0)).exp_()
    total = scores.sum(-1, keepdim=True)
    out = torch.matmul(scores.reshape(-1, hkv, nmax * g, width), v.transpose(1, 2)).reshape(-1, hkv, nmax, g, d)
    out = torch.where(total > 0, out / total, 0.0).permute(0, 2, 1, 3, 4).reshape(-1, nmax, hq, d)
    seq, at = _tokens(s)
    return out[seq, at].to(torch.bfloat16)


def _plain_write(s):
    c = s["case"]
    names = ("k",) if c["kind"] == "global" else ("k", "v")
    seq, at = _tokens(s)
    pos = s["lens"].long()[seq] + at
    page = s["table"].long()[seq, pos // c["page"]]
    slot = pos % c["page"]
    found = []
    new = {n: s["new_" + n].float() for n in names}
    if c["kind"] == "local":
        new["k"] = _turn(new["k"], pos[:, None], _pairs(c), _rope(c)[1])
    if c["dtype"] == "bf16":
        s["k_pages"][page, :, slot] = new["k"].to(torch.bfloat16)
        if "v" in new:
            s["v_pages"][page, :, slot] = new["v"].to(torch.bfloat16)
        return [s[n + "_pages"] for n in names]
    codes, scale = _quantise(new["k"])
    s["k_pages"].view(torch.uint8)[page, :, slot] = codes.view(torch.uint8)
    s["k_scales"][page, :, slot] = scale
    found.append((s["k_pages"][page, :, slot].float() * s["k_scales"][page, :, slot].unsqueeze(-1)).to(torch.bfloat16))
    if "v" in new:
        codes, scale = _quantise(new["v"])
        s["v_pages"].view(torch.uint8)[page, :, slot] = codes.view(torch.uint8)
        s["v_scales"][page, :, slot] = scale
        found.append((s["v_pages"][page, :, slot].float() * s["v_scales"][page, :, slot].unsqueeze(-1)).to(torch.bfloat16))
    return found


def _plain_read(s):
    c = s["case"]
    t = torch.arange(sum(s["ctx"]), device="cuda")
    seq = torch.searchsorted(s["cu_ctx"][1:].long(), t, right=True)
    pos = t - s["cu_ctx"].long()[seq]
    page, slot = s["table"].long()[seq, pos // c["page"]], pos % c["page"]
    rows = lambda n: (s[n + "_pages"][page, :, slot].float() * s[n + "_scales"][page, :, slot].unsqueeze(-1)  # noqa: E731
                      if n + "_scales" in s else s[n + "_pages"][page, :, slot].float()).to(torch.bfloat16)
    return [rows("k")] if c["kind"] == "global" else [rows("k"), rows("v")]


def _plain_draft(s):
    b, n, v = s["case"]["batch"], s["case"]["draft"], s["case"]["vocab"]
    row, place = torch.arange(b, device="cuda"), torch.arange(n, device="cuda")
    x, lens = s["tokens"].long(), s["lens"].long()
    p_x = torch.gather(s["target"][:, :n], 2, x[:, :, None]).squeeze(-1).float()
    q_x = torch.ones_like(p_x) if s["draft"] is None else torch.gather(s["draft"], 2, x[:, :, None]).squeeze(-1).float()
    good = (s["uniforms"] * q_x < p_x) & (place < lens[:, None])
    accepted = torch.cumprod(good.long(), 1).sum(1)
    p = s["target"][row, accepted].float()
    stop = accepted.clamp(max=n - 1)
    if s["draft"] is None:
        q = torch.zeros_like(p).scatter_(1, x[row, stop][:, None], 1.0)
        left = torch.where(q > 0, 0.0, p)
    else:
        left = (p - s["draft"][row, stop].float()).clamp(min=0)
    left = torch.where((accepted < lens)[:, None], left, p)
    left = torch.where((left > 0).any(1, keepdim=True), left, p)
    race = torch.where(left > 0, left / s["noise"], -1.0)
    best = race.amax(1, keepdim=True)
    token = torch.where(race == best, torch.arange(v, device="cuda"), v).amin(1)  # the lowest index of a tie
    place = torch.arange(n + 1, device="cuda")
    padded = torch.cat([x, x[:, :1]], 1)
    tokens = torch.where(place < accepted[:, None], padded, torch.where(place == accepted[:, None], token[:, None], -1))
    return [accepted.to(torch.int32), tokens.to(torch.int32)]


# ---------------------------------------------------------------------- the framework's calls

def _setup(s):
    """What a user's program keeps beside the inputs: parameters, the cache's handle, outputs and the workspace."""
    import global_interleaved_layers_b200 as G
    c = s["case"]
    new = lambda *sh, dt=torch.bfloat16: torch.empty(*sh, dtype=dt, device="cuda")  # noqa: E731
    h = {}
    if c["op"] == "draft":
        h["accepted"], h["tokens"] = new(c["batch"], dt=torch.int32), new(c["batch"], c["draft"] + 1, dt=torch.int32)
        return h
    glob = c["kind"] == "global"
    p, base = _rope(c)
    h["params"] = G.params(G.GLOBAL if glob else G.LOCAL, c["hq"], c["hkv"], c["d"], window=c["window"], rope_p=p, rope_base=base)
    h["cache"] = G.paged_cache(s["k_pages"], s.get("v_pages"), s["table"], k_scales=s.get("k_scales"), v_scales=s.get("v_scales"))
    if c["op"] == "attend":
        h["out"] = new(s["total"], c["hq"], c["d"])
        h["bytes"] = G.gemma_attn_paged_workspace_size(h["params"], h["cache"], c["batch"], s["total"], max(s["nq"]), max(s["ctx"]))
        h["ws"] = new(max(h["bytes"], 256), dt=torch.uint8)
    else:
        n = s["total"] if c["op"] == "write" else sum(s["ctx"])
        h["back"] = [new(n, c["hkv"], c["d"]) for _ in range(1 if glob else 2)]
    return h


def _own(s):
    import global_interleaved_layers_b200 as G
    c = s["case"]
    if "handle" not in s:
        s["handle"] = _setup(s)
    h = s["handle"]
    if c["op"] == "draft":
        G.gemma_attn_draft_verify(s["target"], s["draft"], s["tokens"], s["lens"], s["uniforms"], s["noise"], h["accepted"], h["tokens"])
        return [h["accepted"], h["tokens"]]
    if c["op"] == "attend":
        G.gemma_attn_paged_attend(h["params"], h["cache"], s["q"], s["cu"], s["lens"], h["out"], None, c["batch"], s["total"],
                                  max(s["nq"]), max(s["ctx"]), h["ws"], h["bytes"])
        return h["out"]
    back = h["back"] + [None]
    if c["op"] == "read":
        G.gemma_attn_paged_gather(h["params"], h["cache"], s["zeros"], s["cu_ctx"], back[0], back[1], c["batch"], sum(s["ctx"]))
        return h["back"]
    G.gemma_attn_paged_append(h["params"], h["cache"], s["new_k"], s.get("new_v"), s["cu"], s["lens"], c["batch"], s["total"])
    if c["dtype"] == "bf16":
        return [s["k_pages"], s["v_pages"]] if "v_pages" in s else [s["k_pages"]]
    G.gemma_attn_paged_gather(h["params"], h["cache"], s["lens"], s["cu"], back[0], back[1], c["batch"], s["total"])
    return h["back"]


def run(state):
    if own:
        return _own(state)
    return {"attend": _plain_attend, "write": _plain_write, "read": _plain_read, "draft": _plain_draft}[state["case"]["op"]](state)


# ---------------------------------------------------------------------- 64 bits, from the definition

def _exact_rotation(x, pos, pairs, base):
    """Rows x [n, ..., d] as complex pairs times exp(i pos theta)."""
    d = x.shape[-1]
    y = x.clone()
    if pairs:
        theta = torch.exp(torch.arange(pairs, device=x.device, dtype=torch.float64) * (-2.0 / d * math.log(base)))
        turn = torch.polar(torch.ones(len(pos), pairs, dtype=torch.float64, device=x.device), pos.double()[:, None] * theta)
        turn = turn.reshape([len(pos)] + [1] * (x.dim() - 2) + [pairs])
        z = torch.complex(x[..., :pairs], x[..., d // 2: d // 2 + pairs]) * turn
        y[..., :pairs], y[..., d // 2: d // 2 + pairs] = z.real, z.imag
    return y


def _exact_rows(s, name, seq, lo, hi):
    """Rows [hi - lo, kv_heads, d] of one sequence, page by page."""
    ps, parts = s["case"]["page"], []
    for blk in range(lo // ps, -(-hi // ps)):
        page = int(s["host_table"][seq][blk])
        a, b = max(lo - blk * ps, 0), min(hi - blk * ps, ps)
        rows = s[name + "_pages"][page, :, a:b].double()
        if name + "_scales" in s:
            rows = rows * s[name + "_scales"][page, :, a:b, None].double()
        parts.append(rows.transpose(0, 1))
    return torch.cat(parts)


def _exact_e4m3(x):
    """Values that rows of x have once they are held in e4m3 with a power-of-two scale per row."""
    amax = x.abs().amax(-1, keepdim=True)
    k = torch.ceil(torch.log2(amax / 448.0))
    k = torch.where(448.0 * torch.exp2(k - 1) >= amax, k - 1, torch.where(448.0 * torch.exp2(k) < amax, k + 1, k))
    y = x / torch.exp2(k)
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(y / step) * step * torch.exp2(k)


def exact(case, seed):
    if case["op"] == "draft":
        return None  # whole numbers
    if work(case)["flops"] > 6e12:
        return None
    s = prepare(case, seed)
    s["host_table"] = s["table"].tolist()
    nq, ctx, w = s["nq"], s["ctx"], case["window"]
    names = ("k",) if case["kind"] == "global" else ("k", "v")
    pairs, base = _pairs(case), _rope(case)[1]
    if case["op"] == "read":
        return [torch.cat([_exact_rows(s, n, b, 0, ctx[b]) for b in range(case["batch"])]) for n in names]
    pos = torch.cat([torch.arange(c, c + n, device="cuda") for c, n in zip(ctx, nq)])
    if case["op"] == "write":
        new = {n: s["new_" + n].double() for n in names}
        if case["kind"] == "local":
            new["k"] = _exact_rotation(new["k"], pos, pairs, base)
        if case["dtype"] == "e4m3":
            return [_exact_e4m3(new[n]) for n in names]
        for n in names:
            pool, at = s[n + "_pages"].double(), 0
            for b in range(case["batch"]):
                for blk in range(ctx[b] // case["page"], -(-(ctx[b] + nq[b]) // case["page"])):
                    lo = max(ctx[b], blk * case["page"])
                    hi = min(ctx[b] + nq[b], (blk + 1) * case["page"])
                    pool[s["host_table"][b][blk], :, lo - blk * case["page"]: hi - blk * case["page"]] = new[n][at: at + hi - lo].transpose(0, 1)
                    at += hi - lo
            s[n + "_exact"] = pool
        return [s[n + "_exact"] for n in names]
    g, out, at = case["hq"] // case["hkv"], [], 0
    for b in range(case["batch"]):
        q = _exact_rotation(s["q"][at: at + nq[b]].double(), pos[at: at + nq[b]], pairs, base)
        lo, hi = (max(0, ctx[b] - w + 1) if w else 0), ctx[b] + nq[b]
        kpos = torch.arange(lo, hi, device="cuda")
        k = _exact_rows(s, "k", b, lo, hi)
        v = k if case["kind"] == "global" else _exact_rows(s, "v", b, lo, hi)
        if case["kind"] == "global":
            k = _exact_rotation(k, kpos, pairs, base)
        hide = kpos[None] > pos[at: at + nq[b], None]
        if w:
            hide = hide | (kpos[None] <= pos[at: at + nq[b], None] - w)
        o = torch.empty_like(q)
        for h in range(case["hq"]):
            logits = (q[:, h] @ k[:, h // g].T) / math.sqrt(case["d"])
            o[:, h] = torch.softmax(logits.masked_fill(hide, -math.inf), -1) @ v[:, h // g]
        out.append(o)
        at += nq[b]
    return torch.cat(out)
