"""The sequence operators' measured cases: attention over packed sequences, the
paged key-value cache (written, read back, attended to one token at a time)
and the gated residual with the norms around it.

`listed()` names the cases, `draw()` makes more of the same ranges, `prepare()`
builds what a program holds before the call, `run()` makes one pass: in plain
fp32 torch operations, or, where `own` is true, through the library.
`exact()` computes the same outputs in 64 bits from the definitions.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
EXP_MIN, EXP_MAX = -100, 120  # exponents a cache row's power-of-two scale may take


# ------------------------------------------------------------------ cases
def _text(lens):
    return ",".join(str(n) for n in lens)


def _lens(case, key="lens"):
    return [int(n) for n in case[key].split(",")]


def _ragged(n, lo, hi, step):
    """n lengths spread over [lo, hi], in an order that is not sorted."""
    return [lo + (hi - lo) * ((i * step) % n) // max(1, n - 1) for i in range(n)]


def listed():
    return [
        # A handful of short prompts at once: latency of a nearly empty GPU.
        dict(name="attn_short", op="attention", lens=_text([7, 64, 33, 129]), kv_heads=1, group=3,
             head_dim=128, causal=True),
        # Prompts of different lengths packed into one batch, grouped heads.
        dict(name="attn_packed", op="attention", lens=_text([8192, 5003, 188, 3001]), kv_heads=4,
             group=4, head_dim=128, causal=True),
        # Every frame of the latent clip (21 frames of 60 x 104) attending to itself,
        # 384 channels as 6 heads of 64.
        dict(name="attn_frames", op="attention", lens=_text([6240] * 21), kv_heads=6, group=1,
             head_dim=64, causal=False),
        # Prompts enter the cache.
        dict(name="append_prompts", op="append", lens=_text([8192, 5003, 188, 3001]), before=0,
             kv_heads=8, head_dim=128, page=64, dtype="e4m3"),
        # One new token of each of 64 sequences enters the cache.
        dict(name="append_tokens", op="append", lens=_text([1] * 64), before=1000, kv_heads=8,
             head_dim=128, page=64, dtype="e4m3"),
        # The cache of a batch read back for a pass over many new tokens.
        dict(name="gather_batch", op="gather", lens=_text(_ragged(16, 999, 8191, 7)), kv_heads=8,
             head_dim=128, page=64, dtype="e4m3"),
        # A few short sequences in small pages read back.
        dict(name="gather_short", op="gather", lens=_text([1, 300, 77, 16]), kv_heads=2,
             head_dim=64, page=16, dtype="e4m3"),
        # One token for each of a few sequences, 16-bit cache: latency.
        dict(name="decode_short", op="decode", lens=_text([5, 300, 77, 128]), kv_heads=2, group=4,
             head_dim=64, page=16, dtype="bf16"),
        # A serving batch of ragged lengths over the 8-bit cache.
        dict(name="decode_batch", op="decode", lens=_text(_ragged(64, 17, 8192, 37)), kv_heads=8,
             group=4, head_dim=128, page=64, dtype="e4m3"),
        # One sequence as long as the latent clip has positions (21 x 60 x 104).
        dict(name="decode_long", op="decode", lens=_text([131040]), kv_heads=8, group=8,
             head_dim=128, page=64, dtype="e4m3"),
        # The latent clip's positions at 384 channels, one gate per frame.
        dict(name="norm_clip", op="norm", tokens=131040, channels=384, per_gate=6240,
             dtype="bf16"),
        # The tokens of one decoding step.
        dict(name="norm_tokens", op="norm", tokens=64, channels=4096, per_gate=1, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attention", "attention", "append", "gather", "decode", "decode", "norm"])
    head_dim = rng.choice([64, 128])
    if op == "attention":
        kv_heads, group = rng.choice([1, 2, 4, 6]), rng.choice([1, 2, 3, 4, 8])
        n = _log_int(rng, 1, 24)
        top = min(8192, int(4e4 / math.sqrt(n * kv_heads * group)))
        return dict(op=op, lens=_text([_log_int(rng, 1, top) for _ in range(n)]),
                    kv_heads=kv_heads, group=group, head_dim=head_dim,
                    causal=rng.random() < 0.7)
    if op == "norm":
        channels = 16 * _log_int(rng, 1, 256)
        return dict(op=op, tokens=_log_int(rng, 1, min(131040, 131040 * 384 // channels)),
                    channels=channels, per_gate=_log_int(rng, 1, 8192),
                    dtype=rng.choice(["bf16", "bf16", "f32"]))
    case = dict(op=op, kv_heads=rng.choice([1, 2, 4, 8]), head_dim=head_dim,
                page=rng.choice([16, 32, 64, 128]), dtype=rng.choice(["e4m3", "e4m3", "bf16"]))
    if op == "decode":
        n = _log_int(rng, 1, 64)
        case["group"] = rng.choice([1, 2, 3, 4, 8, 16])
    else:
        n = _log_int(rng, 1, 24)
    if op == "append":
        case["before"] = rng.choice([0, 0, 1, 100, 1000])
    top = (131040 if op == "decode" else 65536) // n
    case["lens"] = _text([_log_int(rng, 1, max(2, top)) for _ in range(n)])
    return case


# ------------------------------------------------------------------ inputs
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, shape, dtype=torch.bfloat16):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _starts(lens):
    starts = [0]
    for n in lens:
        starts.append(starts[-1] + n)
    return _ints(starts)


def _pages(g, lens, page):
    """A page table whose sequences' pages lie anywhere in the cache, and the
    number of pages of the cache (a few stay unused)."""
    need = [-(-n // page) for n in lens]
    n_pages = sum(need) + 3
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros((len(lens), max(1, max(need))), dtype=torch.int32, device="cuda")
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = order[at:at + n]
        at += n
    return table, n_pages


def _row_exponent(x):
    """The exponent of a row's scale: the smallest power of two that brings the
    row's largest magnitude to 448 or below (0 for a row of zeros)."""
    amax = x.abs().amax(-1)
    m, e = torch.frexp(amax / E4M3_MAX)  # amax / 448 = m 2^e, m in [0.5, 1)
    e = torch.where(m == 0.5, e - 1, e)
    return torch.where(amax == 0, torch.zeros_like(e), e.clamp(EXP_MIN, EXP_MAX))


def _power(e):
    """2^e in fp32, exactly, for e in [-126, 127]."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _quantise(x):
    """x [..., D] -> e4m3 elements and the rows' scales, E8M0."""
    x = x.float()
    e = _row_exponent(x)
    q = (x * _power(-e)[..., None]).to(torch.float8_e4m3fn)
    return q, (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _cache_values(pages, scales):
    """A cache's elements as fp32 values."""
    if scales is None:
        return pages.float()
    return pages.float() * _power(scales.view(torch.uint8).to(torch.int32) - 127)[..., None]


def prepare(case, seed):
    g = _generator(seed)
    st = {"case": case}
    op = case["op"]
    if op == "attention":
        lens, D = _lens(case), case["head_dim"]
        hq, hk, total = case["kv_heads"] * case["group"], case["kv_heads"], sum(_lens(case))
        # q, k and v side by side, as one projection writes them
        qkv = _normal(g, (total, hq + 2 * hk, D))
        st["q"], st["k"], st["v"] = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
        st["cu"] = _starts(lens)
        st["longest"] = max(lens)
        st["out"] = torch.empty((total, hq, D), dtype=torch.bfloat16, device="cuda")
        return st
    if op == "norm":
        n, C = case["tokens"], case["channels"]
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        st["x"], st["f"] = _normal(g, (n, C), dt), _normal(g, (n, C), dt)
        st["gate"] = _normal(g, (-(-n // case["per_gate"]), C), torch.float32)
        for name in ("gamma_post", "gamma_pre"):
            st[name] = torch.rand((C,), generator=g, device="cuda") + 0.5
        st["scale"] = 0.7071
        st["y"], st["n"] = torch.empty_like(st["x"]), torch.empty_like(st["x"])
        return st
    lens, D, H, page = _lens(case), case["head_dim"], case["kv_heads"], case["page"]
    before = case.get("before", 0)
    after = [before + n for n in lens]
    st["lens"], st["cu"] = _ints(after), _starts(lens)
    st["table"], n_pages = _pages(g, after, page)
    shape = (n_pages, H, page, D)
    if op == "append":
        st["k"], st["v"] = _normal(g, (sum(lens), H, D)), _normal(g, (sum(lens), H, D))
        quant = case["dtype"] == "e4m3"
        dt = torch.float8_e4m3fn if quant else torch.bfloat16
        st["pages"] = [torch.zeros(shape, dtype=torch.uint8 if quant else dt,
                                   device="cuda").view(dt) for _ in range(2)]
        st["scales"] = [torch.full(shape[:3], 127, dtype=torch.uint8, device="cuda")
                        .view(torch.float8_e8m0fnu) if quant else None for _ in range(2)]
        st["new_seq"] = torch.repeat_interleave(
            torch.arange(len(lens), device="cuda"), torch.tensor(lens, device="cuda"))
    else:
        st["pages"], st["scales"] = [], []
        for _ in range(2):  # keys, values; a row's magnitude varies from token to token
            x = _normal(g, shape, torch.float32)
            x = x * torch.exp(0.5 * _normal(g, shape[:3] + (1,), torch.float32))
            if case["dtype"] == "e4m3":
                q, s = _quantise(x)
            else:
                q, s = x.to(torch.bfloat16), None
            st["pages"].append(q)
            st["scales"].append(s)
    if op == "gather":
        st["k"], st["v"] = (torch.empty((sum(lens), H, D), dtype=torch.bfloat16, device="cuda")
                            for _ in range(2))
        st["seq"] = torch.repeat_interleave(torch.arange(len(lens), device="cuda"),
                                            torch.tensor(lens, device="cuda"))
    if op == "decode":
        hq = H * case["group"]
        st["q"] = _normal(g, (len(lens), hq, D))
        st["out"] = torch.empty_like(st["q"])
        st["longest"] = max(lens)
    if own:
        from video_vae_causal_gb300 import wanvae
        st["cache"] = wanvae.KVCache(st["pages"][0], st["pages"][1], st["scales"][0],
                                     st["scales"][1])
        if op == "decode":
            st["workspace"] = wanvae.make_paged_attention_workspace(st["q"], st["cache"])
    return st


# ------------------------------------------------------------------ one pass
def run(st):
    if own:
        return _run_own(st)
    return {"attention": _attention, "append": _append, "gather": _gather, "decode": _decode,
            "norm": _norm}[st["case"]["op"]](st)


def _run_own(st):
    from video_vae_causal_gb300 import wanvae
    op = st["case"]["op"]
    if op == "attention":
        return wanvae.packed_attention(st["q"], st["k"], st["v"], st["cu"], out=st["out"],
                                       causal=st["case"]["causal"])
    if op == "norm":
        return wanvae.gated_residual_norm(st["x"], st["f"], st["gamma_post"], st["gate"],
                                          st["gamma_pre"], tokens_per_gate=st["case"]["per_gate"],
                                          residual_scale=st["scale"], y=st["y"], n=st["n"])
    if op == "append":
        wanvae.kv_cache_append(st["cache"], st["k"], st["v"], st["lens"], st["table"], st["cu"])
        return [st["pages"], st["scales"]]
    if op == "gather":
        return wanvae.kv_cache_gather(st["cache"], st["table"], st["cu"], k=st["k"], v=st["v"])
    return wanvae.paged_attention(st["q"], st["cache"], st["lens"], st["table"], out=st["out"],
                                  workspace=st["workspace"])


def _softmax_product(scores, seen, v):
    """Rows of softmax(scores) v over the places that are seen; a row that
    sees nothing is zero."""
    scores = torch.where(seen, scores, -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(scores - top)
    total = p.sum(-1, keepdim=True)
    return torch.where(total > 0, p @ v / total, 0.0)


def _attention(st):
    case, cu = st["case"], st["cu"].long()
    D, hk, group = case["head_dim"], case["kv_heads"], case["group"]
    n, L = cu.numel() - 1, st["longest"]
    lens = cu[1:] - cu[:-1]
    at = torch.arange(L, device="cuda")
    there = at[None] < lens[:, None]                      # [n, L]
    row = torch.where(there, cu[:-1, None] + at[None], 0)
    q = st["q"].float()[row].view(n, L, hk, group, D).permute(0, 2, 3, 1, 4)
    k = st["k"].float()[row].permute(0, 2, 3, 1)[:, :, None]   # [n, hk, 1, D, L]
    v = st["v"].float()[row].permute(0, 2, 1, 3)[:, :, None]
    seen = there[:, None, None, None, :]
    if case["causal"]:
        seen = seen & (at[None, :] <= at[:, None])
    o = _softmax_product(q @ k / math.sqrt(D), seen, v)   # [n, hk, group, L, D]
    o = o.permute(0, 3, 1, 2, 4).reshape(n, L, hk * group, D)
    return o[there].to(torch.bfloat16)


def _append(st):
    case, seq = st["case"], st["new_seq"]
    cu, lens, page = st["cu"].long(), st["lens"].long(), case["page"]
    i = torch.arange(seq.numel(), device="cuda")
    pos = lens[seq] - (cu[seq + 1] - i)
    where, slot = st["table"].long()[seq, pos // page], pos % page
    for x, pages, scales in zip((st["k"], st["v"]), st["pages"], st["scales"]):
        if scales is None:
            pages[where, :, slot] = x
        else:
            q, s = _quantise(x)
            pages.view(torch.uint8)[where, :, slot] = q.view(torch.uint8)
            scales.view(torch.uint8)[where, :, slot] = s.view(torch.uint8)
    return [st["pages"], st["scales"]]


def _rows(st, seq, pos):
    """The cache's key and value rows of positions `pos` of sequences `seq`."""
    page = st["case"]["page"]
    where, slot = st["table"].long()[seq, pos // page], pos % page
    got = []
    for pages, scales in zip(st["pages"], st["scales"]):
        if scales is None:
            got.append(pages[where, :, slot].float())
        else:
            got.append(_cache_values(
                pages.view(torch.uint8)[where, :, slot].view(torch.float8_e4m3fn),
                scales.view(torch.uint8)[where, :, slot]))
    return got


def _gather(st):
    seq, cu = st["seq"], st["cu"].long()
    pos = torch.arange(seq.numel(), device="cuda") - cu[seq]
    return [x.to(torch.bfloat16) for x in _rows(st, seq, pos)]


def _decode(st):
    case, lens = st["case"], st["lens"].long()
    D, hk, group, n = case["head_dim"], case["kv_heads"], case["group"], lens.numel()
    at = torch.arange(st["longest"], device="cuda")
    there = at[None] < lens[:, None]
    pos = torch.where(there, at[None], 0)
    seq = torch.arange(n, device="cuda")[:, None].expand_as(pos)
    k, v = _rows(st, seq, pos)                            # [n, L, hk, D]
    q = st["q"].float().view(n, hk, group, D)
    scores = q @ k.permute(0, 2, 3, 1) / math.sqrt(D)
    o = _softmax_product(scores, there[:, None, None], v.permute(0, 2, 1, 3))
    return o.reshape(n, hk * group, D).to(torch.bfloat16)


def _rms(x, gamma, eps=1e-12):
    norm = x.square().sum(-1, keepdim=True).sqrt().clamp_min(eps)
    return x / norm * math.sqrt(x.shape[-1]) * gamma


def _norm(st):
    x, f = st["x"].float(), st["f"].float()
    gate = st["gate"].repeat_interleave(st["case"]["per_gate"], 0)[:x.shape[0]]
    y = x + st["scale"] * gate * _rms(f, st["gamma_post"])
    return [y.to(st["x"].dtype), _rms(y, st["gamma_pre"]).to(st["x"].dtype)]


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op = case["op"]
    if op == "norm":
        size = 2 if case["dtype"] == "bf16" else 4
        n, C = case["tokens"], case["channels"]
        return {"bytes": 4 * n * C * size + -(-n // case["per_gate"]) * C * 4 + 8 * C,
                "flops": 10 * n * C}
    lens, D, hk = _lens(case), case["head_dim"], case["kv_heads"]
    total = sum(lens)
    if op == "attention":
        hq = hk * case["group"]
        pairs = sum(n * (n + 1) // 2 if case["causal"] else n * n for n in lens)
        return {"bytes": 2 * total * D * (2 * hq + 2 * hk), "flops": 4 * D * hq * pairs}
    row = D + 1 if case["dtype"] == "e4m3" else 2 * D     # a cache row
    if op in ("append", "gather"):
        return {"bytes": total * hk * 2 * (2 * D + row), "flops": 4 * total * hk * D}
    hq = hk * case["group"]
    return {"bytes": total * hk * 2 * row + len(lens) * hq * D * 4, "flops": 4 * D * hq * total}


# ------------------------------------------------------------------ the definitions in 64 bits
def _two_to(e):
    """2^e in 64 bits, exactly, from the bits of its exponent."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _e4m3_grid(x):
    """x (64 bits, magnitudes up to 448) rounded to the nearest e4m3 value, ties to even."""
    step = _two_to((torch.frexp(x)[1] - 1).clamp_min(-6) - 3)
    return torch.round(x / step) * step


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        x, f, gate = st["x"].double(), st["f"].double(), st["gate"].double()
        C = x.shape[1]
        which = torch.arange(x.shape[0], device="cuda") // case["per_gate"]
        post = f * (C / (f * f).sum(1)).sqrt()[:, None] * st["gamma_post"].double()
        y = x + st["scale"] * gate[which] * post
        return [y, y * (C / (y * y).sum(1)).sqrt()[:, None] * st["gamma_pre"].double()]
    lens, D, hk = _lens(case), case["head_dim"], case["kv_heads"]
    if op == "attention":
        hq, group = hk * case["group"], case["group"]
        if sum(n * n for n in lens) * hq * D > 1.5e12:
            return None
        out = torch.zeros((sum(lens), hq, D), dtype=torch.float64, device="cuda")
        at = 0
        for n in lens:
            rows = slice(at, at + n)
            for h in range(hq):
                s = st["q"][rows, h].double() @ st["k"][rows, h // group].double().T
                s *= D ** -0.5
                if case["causal"]:
                    s.masked_fill_(torch.ones_like(s, dtype=torch.bool).triu(1), -math.inf)
                out[rows, h] = torch.softmax(s, -1) @ st["v"][rows, h // group].double()
            at += n
        return out
    page, table = case["page"], st["table"].tolist()
    if op == "append":
        before, found = case["before"], [[], []]
        for which, x in enumerate((st["k"].double(), st["v"].double())):
            pages = torch.zeros(st["pages"][which].shape, dtype=torch.float64, device="cuda")
            scales = torch.ones(pages.shape[:3], dtype=torch.float64, device="cuda")
            if case["dtype"] == "e4m3":
                amax = x.abs().amax(-1)
                e = torch.ceil(torch.log2(amax / E4M3_MAX))
                e = torch.where(amax == 0, 0.0, e).clamp(EXP_MIN, EXP_MAX)
                e += ((_two_to(e) * E4M3_MAX < amax) & (e < EXP_MAX)).double()  # log2 rounds,
                low = (_two_to(e - 1) * E4M3_MAX >= amax) & (amax > 0)          # up or down
                e -= (low & (e > EXP_MIN)).double()
                x = _e4m3_grid(x / _two_to(e)[..., None])
            at = 0
            for s, n in enumerate(lens):
                for p in range(before // page, -(-(before + n) // page)):
                    lo, hi = max(before, p * page), min(before + n, (p + 1) * page)
                    rows = slice(at + lo - before, at + hi - before)
                    cells = slice(lo - p * page, hi - p * page)
                    pages[table[s][p], :, cells] = x[rows].transpose(0, 1)
                    if case["dtype"] == "e4m3":
                        scales[table[s][p], :, cells] = _two_to(e[rows]).transpose(0, 1)
                at += n
            found[0].append(pages)
            found[1].append(scales if case["dtype"] == "e4m3" else None)
        return found
    values = []
    for pages, scales in zip(st["pages"], st["scales"]):
        x = pages.double()
        if scales is not None:
            x = x * _two_to(scales.view(torch.uint8).to(torch.int64) - 127)[..., None]
        values.append(x)

    def sequence(which, s, n):  # [hk, n, D]
        need = -(-n // page)
        x = values[which][st["table"][s, :need].long()]
        return x.transpose(0, 1).reshape(hk, need * page, D)[:, :n]

    if op == "gather":
        return [torch.cat([sequence(w, s, n).transpose(0, 1) for s, n in enumerate(lens)])
                for w in (0, 1)]
    out = []
    for s, n in enumerate(lens):
        q = st["q"][s].double().view(hk, case["group"], D)
        p = torch.softmax(q @ sequence(0, s, n).transpose(1, 2) * D ** -0.5, -1)
        out.append((p @ sequence(1, s, n)).reshape(-1, D))
    return torch.stack(out)
