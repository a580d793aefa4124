"""The paged KV-cache operators as measured cases: append, gather, decode and importance.

Every case is one call (or, for an append to a 4-bit cache, the call and the read-back of the rows it
wrote) on a paged cache whose pages lie in shuffled order in one pool.  With `own` false, run() computes
the operators from elementary torch operations in 32 bits; with `own` true it calls the library.
"""
import math
import random

import torch

own = False

D = 128
BLOCK = 16                      # values that share one scale in a 4-bit row
LN2 = math.log(2.0)
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one decoding step of eight sequences of a document reader: the smallest call, latency only
        dict(name="append_step_bf16", op="append", fmt="bf16", B=8, Hkv=8, G=2, T=4864, page=16, new=1, rot=128,
             inter=False),
        # one decoding step of a serving batch far into long contexts, half of each head rotated in pairs
        dict(name="append_step_e2m1", op="append", fmt="e2m1", B=64, Hkv=8, G=4, T=32768, page=64, new=1, rot=64,
             inter=True),
        # ragged prompts of four sequences written in one call
        dict(name="append_prompt_e2m1", op="append", fmt="e2m1", B=4, Hkv=8, G=4, T=8191, page=64, new=8191,
             rot=128, inter=False),
        # whole ragged sequences read back into a contiguous cache
        dict(name="gather_all_e2m1", op="gather", fmt="e2m1", B=4, Hkv=8, G=4, T=32768, page=64, k=0),
        # the rows a selection kept, read back per head
        dict(name="gather_rows_bf16", op="gather", fmt="bf16", B=8, Hkv=8, G=2, T=4864, page=16, k=205),
        # dense decoding of the document reader's batch: short enough that start-up counts
        dict(name="decode_e2m1", op="decode", fmt="e2m1", B=8, Hkv=8, G=2, T=4864, page=16, Mq=1, k=0, tail=0),
        # dense decoding over long ragged contexts: bound by the cache's bytes
        dict(name="decode_long_e2m1", op="decode", fmt="e2m1", B=16, Hkv=8, G=4, T=32768, page=64, Mq=1, k=0, tail=0),
        dict(name="decode_long_bf16", op="decode", fmt="bf16", B=8, Hkv=8, G=4, T=32768, page=64, Mq=1, k=0, tail=0),
        # decoding over the selected rows of a long context and its most recent tokens
        dict(name="decode_listed_e2m1", op="decode", fmt="e2m1", B=8, Hkv=8, G=4, T=131072, page=128, Mq=1, k=2048,
             tail=512),
        # verification of seven drafted tokens a sequence
        dict(name="verify_e2m1", op="decode", fmt="e2m1", B=64, Hkv=8, G=2, T=3335, page=32, Mq=7, k=0, tail=0),
        # token importance from a window of eight queries before a retention
        dict(name="importance_e2m1", op="importance", fmt="e2m1", B=4, Hkv=8, G=4, T=32768, page=64, Mq=8),
        # token importance of one decoding step on a focal layer
        dict(name="importance_bf16", op="importance", fmt="bf16", B=8, Hkv=8, G=2, T=4864, page=16, Mq=1),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "append", "gather", "decode", "decode", "decode", "importance"])
    fmt = rng.choice(["bf16", "e2m1", "e2m1"])
    c = dict(op=op, fmt=fmt, Hkv=rng.choice([1, 2, 4, 8]), G=rng.choice([1, 2, 3, 4, 8]),
             page=rng.choice([16, 32, 64, 128, 256]))
    Mq = 1 if op in ("append", "gather") else rng.choice([1, 8]) if op == "importance" else \
        rng.choice([1, 1, 1, rng.randint(2, 8)])
    # rows of all heads: the bytes and products of a drawn case stay below the largest listed one's
    rows = (1 << 20 if fmt == "bf16" else 1 << 21) >> (op == "gather")
    rows = min(rows, (1 << 24) // (c["G"] * Mq))
    T = _log_int(rng, 17, 65536)
    B = max(1, min(_log_int(rng, 1, 128), rows // (T * c["Hkv"])))
    c.update(B=B, T=T)
    if op == "append":
        new = rng.choice([1, 1, rng.randint(2, 8), T])
        c.update(new=max(1, min(new, T, 131072 // (B * c["Hkv"]))), rot=rng.choice([0, 32, 64, 96, 128]),
                 inter=rng.random() < 0.5)
    elif op == "gather":
        c.update(k=rng.choice([0, rng.randint(1, T)]))
    elif op == "decode":
        k = rng.choice([0, 0, rng.randint(1, max(1, min(T // 2, 4096)))])
        c.update(Mq=Mq, k=k, tail=0 if k == 0 else min(T, _log_int(rng, 1, 1024)))
    else:
        c.update(Mq=Mq)
    return c


def _lengths(c):
    """Ragged lengths of a case: the first sequence is the longest, the others reach down to a third of it."""
    r = random.Random(c["T"] * 1000003 + c["B"])
    return [c["T"]] + [r.randint(max(1, c["T"] // 3), c["T"]) for _ in range(c["B"] - 1)]


def _new(c):
    """Rows that an append adds to each sequence: the end of it, one, or up to c["new"] (ragged for prompts)."""
    r = random.Random(c["T"] * 7919 + c["B"])
    return [min(n, c["new"] if c["new"] <= 8 else r.randint(c["new"] // 2 + 1, c["new"])) for n in _lengths(c)]


def _keys(c):
    """Cache rows that one KV head of each sequence reads."""
    if c["op"] == "decode" and c["k"]:
        return [min(c["k"], max(0, n - c["tail"])) + min(n, c["tail"]) for n in _lengths(c)]
    if c["op"] == "gather" and c["k"]:
        return [min(c["k"], n) for n in _lengths(c)]
    return _lengths(c)


def work(c):
    row = 2 * D if c["fmt"] == "bf16" else D // 2 + D // BLOCK       # one K or V row
    Hq, B, H = c["Hkv"] * c["G"], c["B"], c["Hkv"]
    if c["op"] == "append":
        n = sum(_new(c))
        b = n * (2 * H + Hq) * 2 * D + n * Hq * 2 * D + n * 2 * H * row + n * (8 + 4 * c["rot"])
        if c["fmt"] == "e2m1":
            b += n * 2 * H * (row + 2 * D)                           # the rows read back
        return {"bytes": b, "flops": 3 * n * (Hq + H) * c["rot"]}
    if c["op"] == "gather":
        n = sum(_keys(c)) * H
        return {"bytes": n * 2 * (row + 2 * D) + (4 * n if c["k"] else 0), "flops": 0}
    keys = sum(_keys(c))
    q = B * Hq * c["Mq"] * D * 2
    if c["op"] == "decode":
        return {"bytes": keys * H * 2 * row + q + 2 * q + B * Hq * c["Mq"] * 4 + (4 * B * H * c["k"]),
                "flops": 4 * D * keys * Hq * c["Mq"]}
    return {"bytes": keys * H * row + q + B * H * c["T"] * 4, "flops": 2 * D * keys * Hq * c["Mq"]}


# ---------------------------------------------------------------------------------------- inputs
def _quantize(x):
    """Codes [..., 64] and scale bytes [..., 8] of rows x [..., 128] (bf16 values): blocks of 16 share an e4m3
    scale, the block's largest magnitude over 6 (at least 2^-9); values round to the nearest of +-E2M1, ties to
    the even code.  fp32 decides every border exactly: values have 8 significant bits, scales 4."""
    y = x.float().unflatten(-1, (D // BLOCK, BLOCK))
    a = y.abs().amax(-1, keepdim=True)
    s = (a / 6).clamp(min=2.0 ** -9, max=448.0).to(torch.float8_e4m3fn)
    sf = s.float()
    m = y.abs()
    code = torch.zeros_like(m, dtype=torch.uint8)
    for i, t in enumerate((0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)):
        code += (m > t * sf) if i % 2 == 0 else (m >= t * sf)
    code = (code | (torch.signbit(y).to(torch.uint8) << 3)).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), s.view(torch.uint8).squeeze(-1)


def _dequantize(codes, scales):
    """fp32 rows [..., 128] that codes [..., 64] and scale bytes [..., 8] stand for."""
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    idx = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    v = lut[idx.int()].unflatten(-1, (D // BLOCK, BLOCK))
    return (v * scales.view(torch.float8_e4m3fn).float().unsqueeze(-1)).flatten(-2)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    randn = lambda *s, **kw: torch.randn(*s, generator=g, device=dev, **kw)  # noqa: E731
    c = dict(case)
    B, H, G, T, page, op = c["B"], c["Hkv"], c["G"], c["T"], c["page"], c["op"]
    Hq = H * G
    lens = _lengths(c)
    pages = [-(-n // page) for n in lens]
    n_pages = sum(pages) + 3
    order = torch.randperm(n_pages, generator=g, device=dev, dtype=torch.int64)
    table = torch.full((B, max(pages)), -1, dtype=torch.int32)
    first = 0
    owned = []
    for b, n in enumerate(pages):
        owned.append((b, first, n))
        first += n
    order = order.to(torch.int32).cpu()
    for b, at, n in owned:
        table[b, :n] = order[at:at + n]
    s = {"case": c, "table": table.to(dev), "len": torch.tensor(lens, dtype=torch.int32, device=dev)}
    Mq = c.get("Mq", 1)
    # channels of unequal size, as keys have them, and queries that some tokens answer to
    chan = torch.exp(0.5 * randn(H, 1, D))
    kind = torch.bfloat16 if c["fmt"] == "bf16" else torch.uint8
    width = D if c["fmt"] == "bf16" else D // 2
    pools = {n: torch.zeros(n_pages, H, page, width, dtype=kind, device=dev) for n in ("k", "v")}
    if c["fmt"] == "e2m1":
        pools |= {n: torch.zeros(n_pages, H, page, D // BLOCK, dtype=torch.uint8, device=dev)
                  for n in ("k_scale", "v_scale")}
    if op != "append":
        step = max(1, (1 << 17) // (H * page))
        for at in range(0, n_pages, step):
            shape = (min(step, n_pages - at), H, page, D)
            for n in ("k", "v"):
                x = (randn(*shape) * (chan if n == "k" else 1.0)).to(torch.bfloat16)
                if c["fmt"] == "bf16":
                    pools[n][at:at + step] = x
                else:
                    pools[n][at:at + step], pools[n + "_scale"][at:at + step] = _quantize(x)
    s.update(pools)
    for n in ("k_scale", "v_scale"):
        s.setdefault(n, None)
    if op == "append":
        new = _new(c)
        s["seq"] = torch.repeat_interleave(torch.arange(B), torch.tensor(new)).to(torch.int32).to(dev)
        s["pos"] = torch.cat([torch.arange(n - m, n) for n, m in zip(lens, new)]).to(torch.int32).to(dev)
        s["lo"] = torch.tensor([n - m for n, m in zip(lens, new)], dtype=torch.int32, device=dev)
        s["rows"] = max(new)
        n = sum(new)
        qkv = randn(n, Hq + 2 * H, D, dtype=torch.bfloat16)          # the fused projection's output
        s["q"], s["k_new"], s["v_new"] = qkv[:, :Hq], qkv[:, Hq:Hq + H], qkv[:, Hq + H:]
        s["q_out"] = torch.empty(n, Hq, D, dtype=torch.bfloat16, device=dev)
        s["cos_sin"] = None
        if c["rot"]:
            half = c["rot"] // 2
            f = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device=dev) / half)
            ang = torch.arange(T, dtype=torch.float64, device=dev)[:, None] * f
            s["cos_sin"] = torch.cat((ang.cos(), ang.sin()), -1).float()
        if c["fmt"] == "e2m1":
            s["k_rows"], s["v_rows"] = (torch.zeros(B, H, s["rows"], D, dtype=torch.bfloat16, device=dev)
                                        for _ in range(2))
    elif op == "gather":
        n = c["k"] or T
        s["idx"] = _some(c, lens, n, T, g, dev) if c["k"] else None
        s["k_rows"], s["v_rows"] = (torch.zeros(B, H, n, D, dtype=torch.bfloat16, device=dev) for _ in range(2))
        s["rows"], s["lo"] = n, None
    else:
        s["q"] = (2.0 * randn(B, Mq, Hq, D)).to(torch.bfloat16).transpose(1, 2)    # a projection's layout
        s["idx"], s["tail_lo"], s["scale"] = None, None, 1.0 / math.sqrt(D)
        if op == "decode":
            if c["k"]:
                older = [max(0, n - c["tail"]) for n in lens]
                s["tail_lo"] = torch.tensor(older, dtype=torch.int32, device=dev)
                s["idx"] = _some(c, older, c["k"], T, g, dev)
            s["out"] = torch.empty(B, Hq, Mq, D, device=dev)
            s["lse"] = torch.empty(B, Hq, Mq, device=dev)
        else:
            s["scores"] = torch.empty(B, H, T, device=dev)
            s["lse"] = _decode(s)[1]
    if own:
        import kv_cache_token_fx_gb300 as fx
        s["cache"] = fx.PagedKV(s["k"], s["v"], s["table"], s["len"], k_scale=s["k_scale"], v_scale=s["v_scale"])
        if op == "decode":
            s["ws"] = fx.Workspace(nbytes=fx.fx_paged_decode_workspace_bytes(B, H, Hq, Mq))
    return s


def _some(c, lens, k, cap, g, dev):
    """[B, Hkv, k] ascending distinct rows below each length; a list longer than its sequence repeats the last row."""
    r = torch.rand(c["B"], c["Hkv"], max(cap, k), generator=g, device=dev)
    n = torch.tensor(lens, device=dev)[:, None, None]
    r = r.masked_fill(torch.arange(r.shape[-1], device=dev) >= n, 2.0)
    idx = r.topk(k, largest=False).indices.sort(-1).values
    return torch.minimum(idx, (n - 1).clamp(min=0)).to(torch.int32).contiguous()


# ---------------------------------------------------------------------------------------- plain forms
def _read(s, at):
    """fp32 K and V rows at positions `at` [B, Hkv, n] (clamped into the sequence; callers mask the rest)."""
    c = s["case"]
    at = at.clamp(min=0).minimum((s["len"].long() - 1).clamp(min=0)[:, None, None])
    b = torch.arange(c["B"], device=at.device)[:, None, None]
    h = torch.arange(c["Hkv"], device=at.device)[None, :, None]
    pg, row = s["table"].long()[b, at // c["page"]], at % c["page"]
    if c["fmt"] == "bf16":
        return tuple(s[n][pg, h, row].float() for n in ("k", "v"))
    return tuple(_dequantize(s[n][pg, h, row], s[n + "_scale"][pg, h, row]) for n in ("k", "v"))


def _rotate(x, cs, inter):
    """Rows x [n, heads, 128] with their first dimensions rotated by cs [n, rot]: each product and each sum is
    rounded to fp32, the result to bf16."""
    rot = cs.shape[-1]
    half = rot // 2
    cos, sin = cs[:, None, :half], cs[:, None, half:]
    y = x.float().clone()
    one, two = (slice(0, rot, 2), slice(1, rot, 2)) if inter else (slice(0, half), slice(half, rot))
    a, b = y[..., one], y[..., two]
    y[..., one], y[..., two] = a * cos - b * sin, b * cos + a * sin
    return y.to(torch.bfloat16)


def _append(s):
    c = s["case"]
    seq, pos = s["seq"].long(), s["pos"].long()
    q, k, v = s["q"], s["k_new"], s["v_new"]
    if s["cos_sin"] is not None:
        cs = s["cos_sin"][pos]
        q, k = _rotate(q, cs, c["inter"]), _rotate(k, cs, c["inter"])
    s["q_out"].copy_(q)
    pg, row = s["table"].long()[seq, pos // c["page"]], pos % c["page"]
    for n, x in (("k", k), ("v", v)):
        if c["fmt"] == "bf16":
            s[n][pg, :, row] = x
        else:
            s[n][pg, :, row], s[n + "_scale"][pg, :, row] = _quantize(x)
    if c["fmt"] == "bf16":
        return s["k"], s["v"], s["q_out"]
    return _gather(s) + (s["q_out"],)


def _gather(s):
    c = s["case"]
    if s.get("idx") is not None:
        at = s["idx"].long()
    else:
        at = torch.arange(s["rows"], device=s["len"].device).expand(c["B"], c["Hkv"], -1)
        if s["lo"] is not None:
            at = at + s["lo"].long()[:, None, None]
    inside = (at < s["len"].long()[:, None, None])[..., None]
    rows = _read(s, at)
    return tuple(torch.where(inside, x.to(torch.bfloat16), s[n]) for n, x in zip(("k_rows", "v_rows"), rows))


def _logits(s, at):
    """fp32 logits [B, Hkv, G, Mq, n] of the rows at `at` [B, Hkv, n] (-inf where a query does not see one), and V."""
    c = s["case"]
    B, H, G, Mq = c["B"], c["Hkv"], c["G"], c["Mq"]
    k, v = _read(s, at)
    q = s["q"].float().reshape(B, H, G * Mq, D)
    x = (q @ k.transpose(-1, -2) * s["scale"]).unflatten(2, (G, Mq))
    last = s["len"].long()[:, None] - Mq + torch.arange(Mq, device=at.device)      # the position of query i
    see = at[:, :, None, None] <= last[:, None, None, :, None]
    return x.masked_fill(~see, -math.inf), v


def _decode(s):
    c = s["case"]
    B, H, G, Mq = c["B"], c["Hkv"], c["G"], c["Mq"]
    dev = s["len"].device
    if s["idx"] is None:
        at = torch.arange(c["T"], device=dev).expand(B, H, -1)
    else:
        at = s["tail_lo"].long()[:, None] + torch.arange(c["tail"], device=dev)
        at = torch.cat((s["idx"].long(), at[:, None].expand(B, H, -1)), -1)
    x, v = _logits(s, at)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(m == -math.inf, 0.0, m))
    z = p.sum(-1, keepdim=True)
    p = torch.where(z > 0, p / z, 0.0)
    out = p.flatten(2, 3) @ v
    lse = torch.where(z > 0, m + torch.log(z), -math.inf)
    return out.reshape(B, H * G, Mq, D), lse.reshape(B, H * G, Mq)


def _importance(s):
    c = s["case"]
    at = torch.arange(c["T"], device=s["len"].device).expand(c["B"], c["Hkv"], -1)
    x, _ = _logits(s, at)
    lse = s["lse"].reshape(c["B"], c["Hkv"], c["G"], c["Mq"], 1)
    return torch.where(x == -math.inf, 0.0, torch.exp(x - lse)).sum((2, 3))


def run(s):
    op = s["case"]["op"]
    if not own:
        return {"append": _append, "gather": _gather, "decode": _decode, "importance": _importance}[op](s)
    import kv_cache_token_fx_gb300 as fx
    cache = s["cache"]
    if op == "append":
        fx.fx_paged_append(cache, s["k_new"], s["v_new"], s["seq"], s["pos"], cos_sin=s["cos_sin"],
                           interleaved=s["case"]["inter"], q=s["q"], q_out=s["q_out"])
        if s["case"]["fmt"] == "bf16":
            return s["k"], s["v"], s["q_out"]
        fx.fx_paged_gather(cache, s["rows"], lo=s["lo"], k_out=s["k_rows"], v_out=s["v_rows"])
        return s["k_rows"], s["v_rows"], s["q_out"]
    if op == "gather":
        fx.fx_paged_gather(cache, s["rows"], idx=s["idx"], k_out=s["k_rows"], v_out=s["v_rows"])
        return s["k_rows"], s["v_rows"]
    if op == "decode":
        fx.fx_paged_decode(cache, s["q"], s["idx"], s["tail_lo"], scale=s["scale"], out=s["out"], lse=s["lse"],
                           ws=s["ws"])
        return s["out"], s["lse"]
    return fx.fx_paged_importance(cache, s["q"], s["lse"], scale=s["scale"], scores=s["scores"])


# ---------------------------------------------------------------------------------------- 64 bits
def _value64(pool, scale, page, head, row):
    """One head's rows of a pool as 64-bit values, straight from what the bytes mean."""
    x = pool[page, head, row]
    if scale is None:
        return x.double()
    e = torch.empty(x.shape[0], D, dtype=torch.float64, device=x.device)
    for half in (0, 1):
        nib = (x.int() >> (4 * half)) & 15
        ex, man = (nib >> 1) & 3, (nib & 1).double()
        mag = torch.where(ex == 0, 0.5 * man, torch.ldexp(1.0 + 0.5 * man, (ex - 1).double()))
        e[:, half::2] = torch.where(nib >= 8, -mag, mag)
    return e * scale[page, head, row].view(torch.float8_e4m3fn).double().repeat_interleave(BLOCK, -1)


def _spot(s, b, at):
    return s["table"][b].long()[at // s["case"]["page"]], at % s["case"]["page"]


def _stored64(x, fmt):
    """What a cache of that format holds for 64-bit rows x."""
    x = x.to(torch.bfloat16).double()
    if fmt == "bf16":
        return x
    y = x.unflatten(-1, (D // BLOCK, BLOCK))
    sc = (y.abs().amax(-1, keepdim=True) / 6).clamp(2.0 ** -9, 448.0).to(torch.float8_e4m3fn).double()
    grid = torch.tensor(E2M1, dtype=torch.float64, device=x.device)
    r = (y / sc).abs().clamp(max=6.0)
    up = torch.bucketize(r, grid).clamp(1, 7)
    lo, hi = grid[up - 1], grid[up]
    high = (r - lo > hi - r) | ((r - lo == hi - r) & (up % 2 == 0))
    return (torch.where(high, hi, lo) * torch.sign(y) * sc).flatten(-2)


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    B, H, G, op = c["B"], c["Hkv"], c["G"], c["op"]
    dev = s["len"].device
    lens = _lengths(c)
    if op == "append":
        def turned(x):
            y = x.double()
            if s["cos_sin"] is not None:
                half = c["rot"] // 2
                t = s["cos_sin"].double()[s["pos"].long()][:, None]
                z = torch.complex(t[..., :half], t[..., half:])
                pair = (y[..., :c["rot"]].unflatten(-1, (half, 2)) if c["inter"] else
                        y[..., :c["rot"]].unflatten(-1, (2, half)).transpose(-1, -2))
                w = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * z)
                y = torch.cat(((w if c["inter"] else w.transpose(-1, -2)).flatten(-2), y[..., c["rot"]:]), -1)
            return y
        k, v = _stored64(turned(s["k_new"]), c["fmt"]), _stored64(s["v_new"].double(), c["fmt"])
        q = turned(s["q"]).to(torch.bfloat16).double()
        if c["fmt"] == "bf16":
            kk, vv = s["k"].double(), s["v"].double()
        else:
            kk, vv = s["k_rows"].double(), s["v_rows"].double()
        first = 0
        for b, m in enumerate(_new(c)):
            rows = slice(first, first + m)
            first += m
            if c["fmt"] == "bf16":
                pg, row = _spot(s, b, s["pos"][rows].long())
                kk[pg, :, row], vv[pg, :, row] = k[rows], v[rows]
            else:
                kk[b, :, :m], vv[b, :, :m] = k[rows].transpose(0, 1), v[rows].transpose(0, 1)
        return kk, vv, q
    if op == "gather":
        kk, vv = s["k_rows"].double(), s["v_rows"].double()
        for b in range(B):
            for h in range(H):
                at = torch.arange(lens[b], device=dev) if s["idx"] is None else s["idx"][b, h].long()
                pg, row = _spot(s, b, at)
                kk[b, h, :len(at)] = _value64(s["k"], s["k_scale"], pg, h, row)
                vv[b, h, :len(at)] = _value64(s["v"], s["v_scale"], pg, h, row)
        return kk, vv
    Mq = c["Mq"]
    out = torch.zeros(B, H, G, Mq, D, dtype=torch.float64, device=dev)
    lse = torch.full((B, H, G, Mq), -math.inf, dtype=torch.float64, device=dev)
    scores = torch.zeros(B, H, c["T"], dtype=torch.float64, device=dev)
    q = s["q"].double().reshape(B, H, G, Mq, D)
    for b in range(B):
        for h in range(H):
            if s["idx"] is None:
                at = torch.arange(lens[b], device=dev)
            else:
                at = torch.cat((s["idx"][b, h].long(), torch.arange(max(0, lens[b] - c["tail"]), lens[b], device=dev)))
            if not len(at):
                continue
            pg, row = _spot(s, b, at)
            k = _value64(s["k"], s["k_scale"], pg, h, row)
            x = torch.einsum("gic,tc->git", q[b, h], k) * s["scale"]
            hidden = at[None, :] > lens[b] - Mq + torch.arange(Mq, device=dev)[:, None]
            x = x.masked_fill(hidden, -math.inf)
            if op == "decode":
                lse[b, h] = torch.logsumexp(x, -1)
                p = torch.exp(x - torch.where(lse[b, h] == -math.inf, 0.0, lse[b, h])[..., None])
                out[b, h] = p @ _value64(s["v"], s["v_scale"], pg, h, row)
            else:
                p = torch.exp(x - s["lse"].double().reshape(B, H, G, Mq)[b, h][..., None])
                scores[b, h, :lens[b]] = p.nan_to_num(0.0).sum((0, 1))
    if op == "decode":
        return out.reshape(B, H * G, Mq, D), lse.reshape(B, H * G, Mq)
    return scores
