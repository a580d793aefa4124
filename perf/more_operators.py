"""Operators around a prompt in the paged KV cache as measured cases: attention of ragged new tokens, append with
positions of several axes, compaction of retained rows, copies of pages.

Every case is one call (or, where a call leaves 4-bit rows, the call and their read-back) on a paged cache whose pages
lie in shuffled order in one pool.  With `own` false, run() computes the operators from elementary torch operations in
32 bits; with `own` true it calls the library.
"""
import math
import random

import torch

own = False

D = 128
BLOCK = 16                      # values that share one scale in a 4-bit row
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
CHUNK = 1 << 28                 # logits that the plain form holds at a time


# ---------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one decoding step of a document reader whose layers cap their scores: the smallest call, latency only
        dict(name="step_cap_bf16", op="attend", fmt="bf16", B=8, Hkv=8, G=2, T=4864, page=16, new=1, cap=50.0,
             slope=False, window=0, mask="none"),
        # one decoding step over long ragged contexts, scores with a bias by distance
        dict(name="step_bias_e2m1", op="attend", fmt="e2m1", B=16, Hkv=8, G=4, T=32768, page=64, new=1, cap=0.0,
             slope=True, window=0, mask="none"),
        # the same with capped scores on bf16 pages: bound by the cache's bytes
        dict(name="step_cap_long_bf16", op="attend", fmt="bf16", B=8, Hkv=8, G=4, T=32768, page=64, new=1, cap=50.0,
             slope=False, window=0, mask="none"),
        # whole ragged prompts of pages with pictures, whose tokens see their picture's both ways
        dict(name="prompt_images_bf16", op="attend", fmt="bf16", B=4, Hkv=8, G=4, T=8191, page=64, new=8191, cap=0.0,
             slope=False, window=0, mask="images"),
        # a layer with a window and capped scores, over a prompt of the document reader in 4 bits
        dict(name="prompt_window_e2m1", op="attend", fmt="e2m1", B=8, Hkv=8, G=2, T=4608, page=32, new=4608, cap=50.0,
             slope=False, window=1024, mask="none"),
        # a chunk of a prompt far into a context that packs several documents
        dict(name="chunk_docs_bf16", op="attend", fmt="bf16", B=2, Hkv=8, G=4, T=32768, page=128, new=512, cap=0.0,
             slope=True, window=0, mask="docs"),
        # one decoding step of a serving batch, positions of time, height and width in sections of the head
        dict(name="append_axes_step_e2m1", op="append", fmt="e2m1", B=64, Hkv=8, G=4, T=3335, page=64, new=1, rot=128,
             inter=False, sections="16 24 24", cyclic=False),
        # ragged prompts with pictures, the axes taking turns over the pairs
        dict(name="append_axes_prompt_bf16", op="append", fmt="bf16", B=4, Hkv=8, G=4, T=8191, page=64, new=8191,
             rot=128, inter=False, sections="24 20 20", cyclic=True),
        # the retention of one layer: selected rows of each head and the last window, into pages of their own
        dict(name="compact_rows_e2m1", op="compact", fmt="e2m1", B=4, Hkv=8, G=4, T=32768, page=64, k=2040, tail=8,
             to=16),
        # whole sequences into other pages, of another size
        dict(name="compact_all_bf16", op="compact", fmt="bf16", B=4, Hkv=8, G=4, T=32768, page=16, k=0, tail=32768,
             to=128),
        # the last pages of 64 branches that have just been forked
        dict(name="copy_forks_bf16", op="copy", fmt="bf16", Hkv=8, page=16, n=64),
        # a prefix of long contexts duplicated, in 4 bits
        dict(name="copy_many_e2m1", op="copy", fmt="e2m1", Hkv=8, page=64, n=2048),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "attend", "append", "compact", "copy"])
    fmt = rng.choice(["bf16", "e2m1"])
    c = dict(op=op, fmt=fmt, Hkv=rng.choice([1, 2, 4, 8]), page=rng.choice([16, 32, 64, 128, 256]))
    if op == "copy":
        rows = 1 << 18 if fmt == "bf16" else 1 << 20
        return c | dict(n=max(1, min(_log_int(rng, 1, 4096), rows // (c["page"] * c["Hkv"]))))
    G = rng.choice([1, 2, 3, 4, 8])
    T = _log_int(rng, 17, 65536)
    # rows of all heads: the bytes and products of a drawn case stay below the largest listed one's
    B = max(1, min(_log_int(rng, 1, 128), (1 << 20 if fmt == "bf16" else 1 << 21) // (2 * T * c["Hkv"])))
    c |= dict(B=B, G=G, T=T)
    if op == "attend":
        new = rng.choice([1, 1, rng.randint(2, 8), _log_int(rng, 9, 4096), T])
        new = max(1, min(new, T, (1 << 32) // (B * T * G * c["Hkv"])))
        c.update(new=new, cap=rng.choice([0.0, 0.0, 30.0, 50.0]), slope=rng.random() < 0.4,
                 window=rng.choice([0, 0, _log_int(rng, 1, T)]), mask=rng.choice(["none", "none", "docs", "images"]))
    elif op == "append":
        new = rng.choice([1, 1, rng.randint(2, 8), T])
        rot = rng.choice([32, 64, 96, 128])
        parts = sorted(rng.randint(0, rot // 2) for _ in range(2))
        sections = rng.choice([(parts[0], parts[1] - parts[0], rot // 2 - parts[1]), (rot // 4, rot // 8, rot // 8),
                               (rot // 4, rot // 4)])
        c.update(new=max(1, min(new, T, 65536 // (B * c["Hkv"]))), rot=rot, inter=rng.random() < 0.5,
                 sections=" ".join(map(str, sections)), cyclic=rng.random() < 0.5)
    else:
        k = rng.choice([0, rng.randint(1, T)])
        c.update(k=k, tail=_log_int(rng, 1, T), to=rng.choice([16, 32, 64, 128, 256]))
    return c


def _lengths(c):
    """Ragged lengths of a case: the first sequence is the longest, the others reach down to a third of it."""
    r = random.Random(c["T"] * 1000003 + c["B"])
    return [c["T"]] + [r.randint(max(1, c["T"] // 3), c["T"]) for _ in range(c["B"] - 1)]


def _new(c):
    """New rows of each sequence: the end of it, one, or up to c["new"] (ragged where there are many)."""
    r = random.Random(c["T"] * 7919 + c["B"])
    return [min(n, c["new"] if c["new"] <= 8 else r.randint(c["new"] // 2 + 1, c["new"])) for n in _lengths(c)]


def _spans(c, b):
    """[(start, end)] of the documents (or pictures) of sequence b; pictures leave text between them."""
    r = random.Random(c["T"] * 31 + b)
    T, at, out = _lengths(c)[b], 0, []
    while at < T:
        n = _log_int(r, max(1, T // 24), max(2, T // 3))
        if c["mask"] == "docs" or r.random() < 0.6:
            out.append((at, min(T, at + n)))
        at += n
    return out


def _sections(c):
    return tuple(map(int, c["sections"].split()))


def _seen(c):
    """(first, last) of every query, lists over all sequences: it sees rows first <= t < last."""
    first, last = [], []
    for b, (n, m) in enumerate(zip(_lengths(c), _new(c))):
        lo, hi = [0] * n, list(range(1, n + 1))
        if c["mask"] != "none":
            for a, e in _spans(c, b):
                if c["mask"] == "docs":
                    lo[a:e] = [a] * (e - a)
                else:
                    hi[a:e] = [e] * (e - a)
        if c["window"]:
            lo = [max(x, t - c["window"] + 1) for t, x in enumerate(lo)]
        first += lo[n - m:]
        last += hi[n - m:]
    return first, last


def _kept(c):
    """Rows that a compaction keeps of each sequence: (listed, tail)."""
    return [(c["k"], min(n, c["tail"])) for n in _lengths(c)]


def work(c):
    row = 2 * D if c["fmt"] == "bf16" else D // 2 + D // BLOCK       # one K or V row
    H = c["Hkv"]
    if c["op"] == "copy":
        return {"bytes": c["n"] * H * c["page"] * 2 * (2 * row + (2 * D + row if c["fmt"] == "e2m1" else 0)), "flops": 0}
    Hq, B = H * c["G"], c["B"]
    n = sum(_new(c)) if c["op"] != "compact" else 0
    if c["op"] == "append":
        b = n * (2 * H + Hq) * 2 * D + n * Hq * 2 * D + n * 2 * H * row + n * (8 + 4 * len(_sections(c)) + 4 * c["rot"])
        if c["fmt"] == "e2m1":
            b += n * 2 * H * (row + 2 * D)                           # the rows read back
        return {"bytes": b, "flops": 3 * n * (Hq + H) * c["rot"]}
    if c["op"] == "compact":
        rows = sum(k + t for k, t in _kept(c)) * H
        return {"bytes": rows * 2 * (2 * row + (2 * D + row if c["fmt"] == "e2m1" else 0)) + 4 * B * H * c["k"], "flops": 0}
    first, last = _seen(c)
    keys, at = 0, 0                                                  # rows that some query of their sequence sees
    for m in _new(c):
        edge = 0
        for a, e in sorted(set(zip(first[at:at + m], last[at:at + m]))):
            keys += max(0, e - max(a, edge))
            edge = max(edge, e)
        at += m
    return {"bytes": keys * H * 2 * row + 2 * n * Hq * 2 * D + 4 * n * Hq,
            "flops": 4 * D * Hq * sum(e - a for a, e in zip(first, last))}


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


def _parts(fmt):
    """(name, width, type) of the tensors of a pool."""
    if fmt == "bf16":
        return [(n, D, torch.bfloat16) for n in ("k", "v")]
    return [(n, D // 2, torch.uint8) for n in ("k", "v")] + [(n + "_scale", D // BLOCK, torch.uint8) for n in ("k", "v")]


def _pool(s, fmt, n_pages, H, page, prefix=""):
    for n, w, t in _parts(fmt):
        s[prefix + n] = torch.zeros(n_pages, H, page, w, dtype=t, device="cuda")
    for n in ("k_scale", "v_scale"):
        s.setdefault(prefix + n, None)


def _fill(s, fmt, randn):
    """Channels of unequal size, as keys have them."""
    n_pages, H, page = s["k"].shape[:3]
    chan = torch.exp(0.5 * randn(H, 1, D))
    step = max(1, (1 << 17) // (H * page))
    for at in range(0, n_pages, step):
        shape = (min(step, n_pages - at), H, page, D)
        for n in ("k", "v"):
            x = (randn(*shape) * (chan if n == "k" else 1.0)).to(torch.bfloat16)
            if fmt == "bf16":
                s[n][at:at + step] = x
            else:
                s[n][at:at + step], s[n + "_scale"][at:at + step] = _quantize(x)


def _table(lens, page, g):
    """Shuffled pages for sequences of those lengths: (table [B, most], pages in the pool)."""
    pages = [-(-n // page) for n in lens]
    n_pages = sum(pages) + 3
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32).cpu()
    table = torch.full((len(lens), max(pages)), -1, dtype=torch.int32)
    first = 0
    for b, n in enumerate(pages):
        table[b, :n] = order[first:first + n]
        first += n
    return table.to("cuda"), n_pages


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    randn = lambda *a, **kw: torch.randn(*a, generator=g, device=dev, **kw)  # noqa: E731
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    c = dict(case)
    H, page, op, fmt = c["Hkv"], c["page"], c["op"], c["fmt"]
    s = {"case": c}
    if op == "copy":
        n = c["n"]
        _pool(s, fmt, 2 * n + 1, H, page)
        _fill(s, fmt, randn)
        order = torch.randperm(2 * n + 1, generator=g, device=dev).to(torch.int32)
        s["src"], s["dst"] = order[:n].contiguous(), order[n:2 * n].contiguous()
        # the copies as one sequence, for the read-back
        s["table"], s["len"], s["rows"] = s["dst"][None], ints([n * page]), n * page
    else:
        B, T = c["B"], c["T"]
        lens = _lengths(c)
        s["table"], n_pages = _table(lens, page, g)
        s["len"] = ints(lens)
        _pool(s, fmt, n_pages, H, page)
        if op != "append":
            _fill(s, fmt, randn)
    if op in ("attend", "append"):
        new = _new(c)
        n, Hq = sum(new), H * c["G"]
        qkv = randn(n, Hq + 2 * H, D)                                # the fused projection's output
        if op == "attend":
            qkv *= 8.0 if c["cap"] else 2.0                          # queries that some tokens answer to
        qkv = qkv.to(torch.bfloat16)
        s["q"], s["k_new"], s["v_new"] = qkv[:, :Hq], qkv[:, Hq:Hq + H], qkv[:, Hq + H:]
    if op == "attend":
        s["start"] = ints([sum(new[:b]) for b in range(B + 1)])
        first, last = _seen(c | dict(window=0))
        s["first"] = ints(first) if c["mask"] == "docs" else None
        s["last"] = ints(last) if c["mask"] == "images" else None
        s["slope"] = None
        if c["slope"]:
            s["slope"] = 2.0 ** (-8.0 * torch.arange(1, Hq + 1, device=dev) / Hq).float()
        s["scale"], s["most"] = 1.0 / math.sqrt(D), max(new)
        s["out"] = torch.zeros(n, Hq, D, dtype=torch.bfloat16, device=dev)
        s["lse"] = torch.zeros(n, Hq, device=dev)
    elif op == "append":
        s["seq"] = torch.repeat_interleave(torch.arange(B), torch.tensor(new)).to(torch.int32).to(dev)
        s["pos"] = torch.cat([torch.arange(m - k, m) for m, k in zip(lens, new)]).to(torch.int32).to(dev)
        s["lo"] = ints([m - k for m, k in zip(lens, new)])
        s["rows"] = max(new)
        axes = len(_sections(c))
        # time runs with the tokens, the other axes over a picture's rows and columns
        s["rope_pos"] = torch.stack([s["pos"]] + [torch.randint(0, min(T, 96), (n,), generator=g, device=dev,
                                                                dtype=torch.int32) for _ in range(axes - 1)])
        half = c["rot"] // 2
        f = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device=dev) / half)
        ang = torch.arange(T, dtype=torch.float64, device=dev)[:, None] * f
        s["cos_sin"] = torch.cat((ang.cos(), ang.sin()), -1).float()
        s["axis"] = _axes(_sections(c), c["cyclic"])
        s["q_out"] = torch.empty(n, Hq, D, dtype=torch.bfloat16, device=dev)
        if fmt == "e2m1":
            s["k_rows"], s["v_rows"] = (torch.zeros(B, H, s["rows"], D, dtype=torch.bfloat16, device=dev)
                                        for _ in range(2))
    elif op == "compact":
        kept = _kept(c)
        s["to_table"], to_pages = _table([k + t for k, t in kept], c["to"], g)
        _pool(s, fmt, to_pages, H, c["to"], "to_")
        s["to_len"] = torch.zeros_like(s["len"])
        s["tail_lo"] = ints([m - t for m, (_, t) in zip(lens, kept)])
        s["idx"] = _some(lens, H, c["k"], T, g) if c["k"] else None
        s["rows"] = max(k + t for k, t in kept)
    if fmt == "e2m1" and op in ("copy", "compact"):
        s["k_rows"], s["v_rows"] = (torch.zeros(c.get("B", 1), H, s["rows"], D, dtype=torch.bfloat16, device=dev)
                                    for _ in range(2))
    if own:
        import kv_cache_token_fx_gb300 as fx
        s["cache"] = fx.PagedKV(s["k"], s["v"], s["table"], s["len"], k_scale=s["k_scale"], v_scale=s["v_scale"])
        if op == "attend":
            s["ws"] = fx.Workspace(nbytes=fx.fx_paged_attend_workspace_bytes(B, H, Hq, max(new)))
        elif op == "append":
            s["axes"] = fx.fx_rope_axes(_sections(c), cyclic=c["cyclic"])
        elif op == "compact":
            s["to_cache"] = fx.PagedKV(s["to_k"], s["to_v"], s["to_table"], s["to_len"], k_scale=s["to_k_scale"],
                                       v_scale=s["to_v_scale"])
    return s


def _axes(sections, cyclic):
    """The axis of every pair: sections one after the other, or in turns until an axis has had its share."""
    if not cyclic:
        return [a for a, n in enumerate(sections) for _ in range(n)]
    left, out = list(sections), []
    while any(left):
        for a in range(len(left)):
            if left[a]:
                left[a] -= 1
                out.append(a)
    return out


def _some(lens, H, k, cap, g):
    """[B, H, k] ascending distinct rows below each length; a list longer than its sequence repeats the last row."""
    r = torch.rand(len(lens), H, max(cap, k), generator=g, device="cuda")
    n = torch.tensor(lens, device="cuda")[:, None, None]
    r = r.masked_fill(torch.arange(r.shape[-1], device="cuda") >= n, 2.0)
    idx = r.topk(k, largest=False).indices.sort(-1).values
    return torch.minimum(idx, (n - 1).clamp(min=0)).to(torch.int32).contiguous()


# ---------------------------------------------------------------------------------------- plain forms
def _raw(s, at, b=None):
    """The pool's tensors at rows `at` [B, H, n] of every sequence (or of those numbered b), by name; rows past the
    length are clamped (callers leave them out)."""
    c = s["case"]
    b = torch.arange(at.shape[0], device=at.device) if b is None else b
    at = at.clamp(min=0).minimum((s["len"].long()[b] - 1).clamp(min=0)[:, None, None])
    h = torch.arange(c["Hkv"], device=at.device)[None, :, None]
    pg, row = s["table"].long()[b[:, None, None], at // c["page"]], at % c["page"]
    return {n: s[n][pg, h, row] for n, _, _ in _parts(c["fmt"])}


def _values(r):
    """fp32 K and V rows of what _raw gives."""
    if "k_scale" not in r:
        return r["k"].float(), r["v"].float()
    return tuple(_dequantize(r[n], r[n + "_scale"]) for n in ("k", "v"))


def _attend(s):
    """Logits cap tanh(scale q k / cap) - slope |distance| over the rows that a query sees, their softmax, the mean
    of V: sequences together where each has few queries, else one after the other, queries in chunks."""
    c = s["case"]
    H, G, T = c["Hkv"], c["G"], c["T"]
    dev, lens, new = s["len"].device, _lengths(c), _new(c)

    def some(q, pos, lo, hi, k, v):
        """q [B, H, G, m, D]; pos, lo, hi [B, m]; k, v [B, H, n, D] -> out and lse of the queries."""
        x = (q.flatten(2, 3) @ k.transpose(-1, -2)).unflatten(2, (G, -1)) * s["scale"]
        if c["cap"]:
            x = c["cap"] * torch.tanh(x / c["cap"])
        t = torch.arange(k.shape[2], device=dev)
        if s["slope"] is not None:
            x = x - s["slope"].view(H, G, 1, 1) * (pos[..., None] - t).abs().float()[:, None, None]
        see = (t >= lo[..., None]) & (t < hi[..., None])
        x = x.masked_fill(~see[:, None, None], -math.inf)
        m = x.amax(-1, keepdim=True)
        p = torch.exp(x - torch.where(m == -math.inf, 0.0, m))
        z = p.sum(-1, keepdim=True)
        o = (p.flatten(2, 3) @ v).unflatten(2, (G, -1))
        return torch.where(z > 0, o / z, 0.0), torch.where(z > 0, m + torch.log(z), -math.inf).squeeze(-1)

    start, length = s["start"].long(), s["len"].long()
    q = s["q"].float().unflatten(1, (H, G))
    for b0 in range(0, c["B"], c["B"] if c["new"] == 1 else 1):
        ids = torch.arange(b0, c["B"] if c["new"] == 1 else b0 + 1, device=dev)
        m, n = max(new[b0:b0 + len(ids)]), max(lens[b0:b0 + len(ids)])
        k, v = _values(_raw(s, torch.arange(n, device=dev).expand(len(ids), H, n), ids))
        step = max(1, CHUNK // (len(ids) * H * G * n))
        for j in range(0, m, step):
            own_rows = start[ids][:, None] + torch.arange(j, min(m, j + step), device=dev)     # [ids, m]
            pos = (length[ids] - (start[ids + 1] - start[ids]))[:, None] + (own_rows - start[ids][:, None])
            lo = torch.zeros_like(pos) if s["first"] is None else s["first"].long()[own_rows]
            hi = pos + 1 if s["last"] is None else s["last"].long()[own_rows]
            if c["window"]:
                lo = torch.maximum(lo, pos - c["window"] + 1)
            o, z = some(q[own_rows].permute(0, 2, 3, 1, 4), pos, lo, hi, k, v)
            s["out"][own_rows] = o.permute(0, 3, 1, 2, 4).flatten(2, 3).to(torch.bfloat16)
            s["lse"][own_rows] = z.permute(0, 3, 1, 2).flatten(2, 3)
    return s["out"], s["lse"]


def _append(s):
    c = s["case"]
    half = c["rot"] // 2
    at = s["rope_pos"].long()[torch.tensor(s["axis"], device=s["len"].device)].T              # [n, half]
    j = torch.arange(half, device=at.device)
    cos, sin = s["cos_sin"][at, j][:, None], s["cos_sin"][at, j + half][:, None]

    def turned(x):
        """The first rot dimensions rotated: each product and each sum rounded to fp32, the result to bf16."""
        y = x.float().clone()
        one, two = ((slice(0, c["rot"], 2), slice(1, c["rot"], 2)) if c["inter"] else
                    (slice(0, half), slice(half, c["rot"])))
        a, b = y[..., one], y[..., two]
        y[..., one], y[..., two] = a * cos - b * sin, b * cos + a * sin
        return y.to(torch.bfloat16)

    s["q_out"].copy_(turned(s["q"]))
    seq, pos = s["seq"].long(), s["pos"].long()
    pg, row = s["table"].long()[seq, pos // c["page"]], pos % c["page"]
    for n, x in (("k", turned(s["k_new"])), ("v", s["v_new"])):
        if c["fmt"] == "bf16":
            s[n][pg, :, row] = x
        else:
            s[n][pg, :, row], s[n + "_scale"][pg, :, row] = _quantize(x)
    if c["fmt"] == "bf16":
        return s["k"], s["v"], s["q_out"]
    at = s["lo"].long()[:, None, None] + torch.arange(s["rows"], device=pos.device).expand(c["B"], c["Hkv"], -1)
    _back(s, at, _raw(s, at), s["len"])
    return s["k_rows"], s["v_rows"], s["q_out"]


def _back(s, at, raw, length):
    """4-bit rows back as bf16, where they lie below the length."""
    inside = (at < length.long()[:, None, None])[..., None]
    for n, x in zip(("k_rows", "v_rows"), _values(raw)):
        s[n].copy_(torch.where(inside, x.to(torch.bfloat16), s[n]))


def _compact(s):
    c = s["case"]
    B, H, dev = c["B"], c["Hkv"], s["len"].device
    n = s["rows"]
    at = torch.arange(n, device=dev).expand(B, H, n)
    src = s["tail_lo"].long()[:, None, None] + at - c["k"]
    if c["k"]:
        src = torch.cat((s["idx"].long(), src[..., c["k"]:]), -1)
    length = c["k"] + s["len"].long() - s["tail_lo"].long()
    raw = _raw(s, src)
    b, h, i = torch.nonzero(at < length[:, None, None], as_tuple=True)
    pg, row = s["to_table"].long()[b, i // c["to"]], i % c["to"]
    for name, x in raw.items():
        s["to_" + name][pg, h, row] = x[b, h, i]
    s["to_len"].copy_(length)
    if c["fmt"] == "bf16":
        return s["to_k"], s["to_v"], s["to_len"]
    _back(s, at, raw, s["to_len"])
    return s["k_rows"], s["v_rows"], s["to_len"]


def _copy(s):
    c = s["case"]
    src, dst = s["src"].long(), s["dst"].long()
    for n, _, _ in _parts(c["fmt"]):
        s[n][dst] = s[n][src]
    if c["fmt"] == "bf16":
        return s["k"], s["v"]
    at = torch.arange(s["rows"], device=src.device).expand(1, c["Hkv"], -1)
    _back(s, at, _raw(s, at), s["len"])
    return s["k_rows"], s["v_rows"]


def run(s):
    c = s["case"]
    op = c["op"]
    if not own:
        return {"attend": _attend, "append": _append, "compact": _compact, "copy": _copy}[op](s)
    import kv_cache_token_fx_gb300 as fx
    cache = s["cache"]
    if op == "attend":
        fx.fx_paged_attend(cache, s["q"], s["start"], max_new=s["most"], first=s["first"], last=s["last"],
                           window=c["window"], cap=c["cap"], slope=s["slope"], scale=s["scale"], out=s["out"],
                           lse=s["lse"], ws=s["ws"])
        return s["out"], s["lse"]
    bf16 = c["fmt"] == "bf16"
    if op == "append":
        fx.fx_paged_append(cache, s["k_new"], s["v_new"], s["seq"], s["pos"], cos_sin=s["cos_sin"],
                           rope_pos=s["rope_pos"], axes=s["axes"], interleaved=c["inter"], q=s["q"], q_out=s["q_out"])
        if bf16:
            return s["k"], s["v"], s["q_out"]
        fx.fx_paged_gather(cache, s["rows"], lo=s["lo"], k_out=s["k_rows"], v_out=s["v_rows"])
        return s["k_rows"], s["v_rows"], s["q_out"]
    if op == "compact":
        fx.fx_paged_compact(cache, s["to_cache"], idx=s["idx"], tail_lo=s["tail_lo"])
        if bf16:
            return s["to_k"], s["to_v"], s["to_len"]
        fx.fx_paged_gather(s["to_cache"], s["rows"], k_out=s["k_rows"], v_out=s["v_rows"])
        return s["k_rows"], s["v_rows"], s["to_len"]
    fx.fx_paged_copy(cache, s["src"], s["dst"])
    if bf16:
        return s["k"], s["v"]
    fx.fx_paged_gather(cache, s["rows"], k_out=s["k_rows"], v_out=s["v_rows"])
    return s["k_rows"], s["v_rows"]


# ---------------------------------------------------------------------------------------- 64 bits
def _value64(s, name, page, head, row):
    """One head's rows of a pool as 64-bit values, straight from what the bytes mean."""
    x = s[name][page, head, row]
    if s["case"]["fmt"] == "bf16":
        return x.double()
    e = torch.empty(x.shape[0], D, dtype=torch.float64, device=x.device)
    for half in (0, 1):
        nib = (x.int() >> (4 * half)) & 15
        ex, man = (nib >> 1) & 3, (nib & 1).double()
        mag = torch.where(ex == 0, 0.5 * man, torch.ldexp(1.0 + 0.5 * man, (ex - 1).double()))
        e[:, half::2] = torch.where(nib >= 8, -mag, mag)
    return e * s[name + "_scale"][page, head, row].view(torch.float8_e4m3fn).double().repeat_interleave(BLOCK, -1)


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
    H, op, bf16 = c["Hkv"], c["op"], c["fmt"] == "bf16"
    dev = s["len"].device
    if op == "copy":
        if bf16:
            out = [s[n].double() for n in ("k", "v")]
            for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
                for x in out:
                    x[b] = x[a]
            return tuple(out)
        every = torch.arange(c["page"], device=dev)
        out = [torch.stack([torch.cat([_value64(s, n, torch.full_like(every, a), h, every) for a in s["src"].tolist()])
                            for h in range(H)])[None] for n in ("k", "v")]
        return tuple(out)
    B, G, lens = c["B"], c["G"], _lengths(c)
    if op == "compact":
        out = [(s["to_" + n] if bf16 else s[n + "_rows"]).double() for n in ("k", "v")]
        sizes = []
        for b, (k, t) in enumerate(_kept(c)):
            sizes.append(k + t)
            for h in range(H):
                at = torch.arange(lens[b] - t, lens[b], device=dev)
                if k:
                    at = torch.cat((s["idx"][b, h].long(), at))
                pg, row = _spot(s, b, at)
                i = torch.arange(len(at), device=dev)
                for x, n in zip(out, ("k", "v")):
                    if bf16:
                        x[s["to_table"][b].long()[i // c["to"]], h, i % c["to"]] = _value64(s, n, pg, h, row)
                    else:
                        x[b, h, :len(at)] = _value64(s, n, pg, h, row)
        return (*out, torch.tensor(sizes, dtype=torch.int32, device=dev))
    new = _new(c)
    if op == "append":
        half = c["rot"] // 2

        def turned(x):
            y = x.double()
            t = torch.stack([s["cos_sin"].double()[s["rope_pos"][a].long()][:, [p, half + p]]
                             for p, a in enumerate(s["axis"])], 1)[:, None]
            z = torch.view_as_complex(t.contiguous())
            pair = (y[..., :c["rot"]].unflatten(-1, (half, 2)) if c["inter"] else
                    y[..., :c["rot"]].unflatten(-1, (2, half)).transpose(-1, -2))
            w = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * z)
            return torch.cat(((w if c["inter"] else w.transpose(-1, -2)).flatten(-2), y[..., c["rot"]:]), -1)

        k, v = _stored64(turned(s["k_new"]), c["fmt"]), _stored64(s["v_new"].double(), c["fmt"])
        kk, vv = ((s[n] if bf16 else s[n + "_rows"]).double() for n in ("k", "v"))
        first = 0
        for b, m in enumerate(new):
            rows = slice(first, first + m)
            first += m
            if bf16:
                pg, row = _spot(s, b, s["pos"][rows].long())
                kk[pg, :, row], vv[pg, :, row] = k[rows], v[rows]
            else:
                kk[b, :, :m], vv[b, :, :m] = k[rows].transpose(0, 1), v[rows].transpose(0, 1)
        return kk, vv, turned(s["q"]).to(torch.bfloat16).double()
    if sum(m * n for m, n in zip(new, lens)) * H * G > 1 << 33:
        return None
    first, last = (torch.tensor(x, device=dev) for x in _seen(c))
    out = torch.zeros(sum(new), H * G, D, dtype=torch.float64, device=dev)
    lse = torch.full((sum(new), H * G), -math.inf, dtype=torch.float64, device=dev)
    at = 0
    for b, m in enumerate(new):
        t = torch.arange(lens[b], device=dev)
        pg, row = _spot(s, b, t)
        for h in range(H):
            k, v = (_value64(s, n, pg, h, row) for n in ("k", "v"))
            step = max(1, (1 << 26) // (lens[b] * G))
            for j in range(at, at + m, step):
                rows = slice(j, min(j + step, at + m))
                x = torch.einsum("igc,tc->igt", s["q"][rows, h * G:(h + 1) * G].double(), k) * s["scale"]
                if c["cap"]:
                    x = torch.tanh(x.div_(c["cap"])).mul_(c["cap"])
                pos = torch.arange(rows.start, rows.stop, device=dev) - at + lens[b] - m
                if s["slope"] is not None:
                    far = (pos[:, None, None] - t).abs().double()
                    x -= far * s["slope"][h * G:(h + 1) * G].double()[None, :, None]
                hidden = (t < first[rows, None]) | (t >= last[rows, None])
                x.masked_fill_(hidden[:, None], -math.inf)
                z = torch.logsumexp(x, -1)
                lse[rows, h * G:(h + 1) * G] = z
                x.sub_(torch.where(z == -math.inf, 0.0, z)[..., None]).exp_()
                out[rows, h * G:(h + 1) * G] = x @ v
        at += m
    return out, lse
