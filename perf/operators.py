"""What is measured of the key/value cache and the attention over it.

Three operators of a decoder layer next to its feed-forward half:

- "rope": rotary positions for the queries and keys of a step, with the write of
  the new keys and values into the pages of the cache (`pi_rope_append`);
- "attention": a chunk of new tokens of every sequence, single tokens included,
  over the paged cache (`pi_paged_attention`);
- "pages": what a server does with the pages: beams forked and extended with
  copy on write (`pi_pages_fork`, `pi_pages_extend`), finished sequences freed
  and others extended (`pi_pages_free`, `pi_pages_extend`), a fragmented cache
  compacted (`pi_pages_compact`).

`own` false computes them in elementary torch operations, true calls the
library.  Widths (1024, 7168, 8192 = heads x head size) are those of the
workloads in workload/synth.py; the other sizes are generic.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
DT = {"f16": torch.float16, "f32": torch.float32}


# ---- cases -------------------------------------------------------------------

def _attention(name, dtype, seqs, new, min_len, max_len, q_heads, kv_heads, head_dim, page,
               cap=0.0, bias=False, window=0, doc=0, prefix=0.0):
    c = dict(op="attention", dtype=dtype, seqs=seqs, new=new, min_len=min_len, max_len=max_len,
             q_heads=q_heads, kv_heads=kv_heads, head_dim=head_dim, page=page, cap=cap, bias=bias,
             window=window, doc=doc, prefix=prefix)
    return dict(c, name=name) if name else c


def _rope(name, dtype, seqs, new, max_len, q_heads, kv_heads, head_dim, page, rotary, pairs):
    c = dict(op="rope", dtype=dtype, seqs=seqs, new=new, min_len=new, max_len=max_len,
             q_heads=q_heads, kv_heads=kv_heads, head_dim=head_dim, page=page, rotary=rotary,
             pairs=pairs)
    return dict(c, name=name) if name else c


def _pages(name, kind, seqs, max_len, layers, kv_heads, head_dim, page, pool):
    c = dict(op="pages", kind=kind, dtype="f16", seqs=seqs, max_len=max_len, layers=layers,
             kv_heads=kv_heads, head_dim=head_dim, page=page, pool=pool)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one user's next token on a small model: nothing but latency
        _attention("token-1x16h64", "f16", 1, 1, 511, 511, 16, 16, 64, 16),
        # a served batch's next tokens, lengths as a server sees them, grouped heads
        _attention("tokens-48x64h128", "f16", 48, 1, 300, 8191, 64, 8, 128, 16),
        # two users far into long documents: few rows, the whole time goes into reading the cache
        _attention("tokens-2x131072", "f16", 2, 1, 100001, 131072, 64, 8, 128, 64),
        # a chunk of a long prompt, every head with keys of its own: matrix products
        _attention("chunk-2048x56h128", "f16", 1, 2048, 10001, 10001, 56, 56, 128, 16),
        # chunks and single tokens in one call, packed documents, a window, capped scores
        _attention("mixed-8x128h64", "f16", 8, 512, 40, 4095, 128, 8, 64, 32, cap=30.0, window=1500, doc=701),
        # the 32-bit model with a bias by distance and a prefix that is seen from both sides
        _attention("chunk-f32-3x16h64", "f32", 3, 160, 200, 1500, 16, 16, 64, 16, bias=True, prefix=0.3),
        # a served batch's next tokens go into the cache: latency again
        _rope("rope-64x64h128", "f16", 64, 1, 8191, 64, 8, 128, 16, 128, False),
        # prompts go into the cache: half of each head turns, pairs of neighbours
        _rope("rope-8192x128h64", "f16", 4, 2048, 10001, 128, 8, 64, 16, 32, True),
        # the 32-bit model, odd lengths
        _rope("rope-f32-5x16h64", "f32", 5, 203, 1009, 16, 16, 64, 16, 64, False),
        # one step of a beam search: 16 prompts of 8 beams change parents, then grow by a token
        _pages("beams-128", "beams", 128, 2047, 4, 8, 128, 16, 16384),
        # between two steps of a server: some sequences end, the others grow
        _pages("turnover-256", "turnover", 256, 2047, 1, 8, 64, 32, 10007),
        # a cache after hours of that, half of its pages in use: the pages move together
        _pages("compact-4096", "compact", 64, 1023, 4, 8, 128, 16, 4096),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attention", "attention", "attention", "rope", "pages"])
    if op == "attention":
        while True:
            kv, g = rng.choice([1, 2, 8, 16, 56]), rng.choice([1, 1, 2, 3, 5, 8, 16])
            d = rng.choice([64, 64, 80, 96, 128, 128, 256])
            if kv * g * d > 8192:
                continue
            new = 1 if rng.random() < 0.5 else _log(rng, 2, 2048)
            max_len = max(new, _log(rng, 1 if rng.random() < 0.1 else 256, 131072))
            seqs = _log(rng, 1, 64)
            c = _attention(None, rng.choice(["f16", "f16", "f16", "f32"]), seqs, new,
                           _log(rng, 1, max_len), max_len, kv * g, kv, d, rng.choice([8, 16, 32, 64, 128]),
                           rng.choice([0.0, 0.0, 20.0, 50.0]), rng.random() < 0.25,
                           rng.choice([0, 0, 0, 129, 1000]), rng.choice([0, 0, 0, 257]),
                           rng.choice([0.0, 0.0, 0.0, 0.5]))
            size = 2 if c["dtype"] == "f16" else 4
            if seqs * kv * g * new * max_len <= 1.1e9 and seqs * max_len * kv * d * size <= 2.6e8 and \
                    seqs * new * kv * g * d <= 2e7 and (size == 2 or seqs * kv * g * new * max_len <= 3e8):
                return c
    if op == "rope":
        kv, g = rng.choice([1, 2, 8, 16]), rng.choice([1, 2, 3, 5, 8])
        d = rng.choice([64, 80, 128, 256])
        new = 1 if rng.random() < 0.4 else _log(rng, 2, 4096)
        seqs = _log(rng, 1, max(1, min(96, 8192 // new)))
        return _rope(None, rng.choice(["f16", "f16", "f32"]), seqs, new, new + _log(rng, 1, 4000), kv * g, kv, d,
                     rng.choice([8, 16, 32, 64]), rng.choice([d, d // 2, d - 6]), rng.random() < 0.5)
    page = rng.choice([16, 32, 64])
    seqs = _log(rng, 8, 256)
    max_len = _log(rng, 40, 4095)
    d = rng.choice([64, 128])
    kv = rng.choice([2, 8])
    kind = rng.choice(["beams", "turnover", "compact"])
    pool = seqs * (-(-max_len // page) + 2) + rng.randrange(1, 999)
    layers = max(1, min(4, int(2.5e8 // (pool * page * kv * d))))
    while pool * layers * page * kv * d > 2.7e8:
        seqs //= 2
        pool = seqs * (-(-max_len // page) + 2) + 7
    return _pages(None, kind, seqs, max_len, layers, kv, d, page, pool)


# ---- what a case's sequences are (of the case alone) ----------------------------

def _lengths(c):
    """New tokens and lengths of the sequences: spread evenly over the logarithm, one at each end."""
    n, rng = c["seqs"], random.Random(7)
    if c["op"] == "attention":
        new = [c["new"] if n == 1 else max(1, round(c["new"] ** (1 - i / (n - 1)))) for i in range(n)]
    else:
        new = [max(1, c["new"] - i) for i in range(n)]
    lo, hi = c["min_len"], c["max_len"]
    lens = [hi if n == 1 else round(hi * (lo / hi) ** (i / (n - 1))) for i in range(n)]
    rng.shuffle(lens)
    return new, [max(a, b) for a, b in zip(new, lens)]


def _bounds(c):
    """For every new token its position and the keys it sees, [lo, hi)."""
    new, lens = _lengths(c)
    pos = np.concatenate([np.arange(b - a, b, dtype=np.int64) for a, b in zip(new, lens)])
    owner = np.repeat(np.arange(len(new)), new)
    first = pos // c["doc"] * c["doc"] if c["doc"] else np.zeros_like(pos)
    lo = np.maximum(first, pos - c["window"] + 1) if c["window"] else first
    pre = np.array([int(c["prefix"] * x) for x in lens], dtype=np.int64)
    hi = np.minimum(np.array(lens)[owner], np.maximum(pos + 1, pre[owner]))
    return pos, owner, first, pre, lo, hi


def _turns(rotary):
    """Turns per position of each pair, base 10000, every second half slowed by four (a long context)."""
    i = np.arange(rotary // 2, dtype=np.float64)
    t = 10000.0 ** (-2.0 * i / max(rotary, 1)) / (2.0 * math.pi)
    return np.where(i * 2 >= rotary // 2, t / 4, t)


def work(c):
    size = 2 if c["dtype"] == "f16" else 4
    if c["op"] == "attention":
        new, lens = _lengths(c)
        _, owner, _, _, lo, hi = _bounds(c)
        seen = int(np.maximum(hi - lo, 0).sum())
        keys = 0                                            # keys that some token of their sequence sees
        at = 0
        for n in new:
            keys += int(hi[at:at + n].max() - min(lo[at:at + n].min(), hi[at:at + n].max()))
            at += n
        t, hd = sum(new), c["q_heads"] * c["head_dim"]
        return {"bytes": 2 * keys * c["kv_heads"] * c["head_dim"] * size + 2 * t * hd * size + 4 * t * c["q_heads"],
                "flops": 4 * seen * hd}
    if c["op"] == "rope":
        t = sum(_lengths(c)[0])
        moved = (c["q_heads"] + 2 * c["kv_heads"]) * c["head_dim"] * t * size * 2
        return {"bytes": moved, "flops": 3 * (c["q_heads"] + c["kv_heads"]) * c["rotary"] * t}
    stride = -(-c["max_len"] // c["page"]) + 1
    page = 2 * c["layers"] * c["kv_heads"] * c["page"] * c["head_dim"] * size
    s = _pool(c, 0)
    table = c["seqs"] * stride * 4
    if c["kind"] == "compact":
        return {"bytes": 2 * page * s["moves"] + 2 * table + 12 * c["pool"], "flops": 0}
    return {"bytes": 2 * page * s["copies"] + 2 * table + 8 * c["pool"], "flops": 0}


# ---- inputs --------------------------------------------------------------------

def _pool(c, seed):
    """The pages of a server's sequences, on the host: reference counts, tables, lengths and the step's lists."""
    rng = np.random.default_rng([seed, 3])
    n, page, pool = c["seqs"], c["page"], c["pool"]
    stride = -(-c["max_len"] // page) + 1
    table = np.full((n, stride), -1, dtype=np.int32)
    refs = np.zeros(pool, dtype=np.int32)
    out = {"copies": 0, "moves": 0}
    if c["kind"] == "beams":
        # the beams of one prompt share its full pages and each its own last one
        lens = np.zeros(n, dtype=np.int32)
        ids, at = rng.permutation(pool).astype(np.int32), 0
        parent = np.arange(n, dtype=np.int32)
        for b in range(0, n, 8):
            ln = int(c["max_len"] * (b + 8) / (n + 8))
            full = ln // page
            for k in range(b, min(n, b + 8)):
                lens[k] = ln
                table[k, :full] = ids[at:at + full]
                refs[ids[at:at + full]] += 1
            at += full
            for k in range(b, min(n, b + 8)):
                parent[k] = b + (k - b) * 3 % 5 % (min(n, b + 8) - b)
                if ln % page:
                    table[k, full] = ids[at]
                    refs[ids[at]] += 1
                    at += 1
            if ln % page:
                used = [int(p) for p in parent[b:min(n, b + 8)]]
                out["copies"] += sum(used.count(p) for p in set(used) if used.count(p) > 1)
        out |= {"src": parent, "dst": np.arange(n, dtype=np.int32)}
    else:
        lens = np.array([1 + (k * 977 + 13) % c["max_len"] for k in range(n)], dtype=np.int32)
        need = -(-lens // page)
        if c["kind"] == "compact":                          # half of the pages in use, all over the pool
            while need.sum() > pool // 2:
                lens = np.maximum(1, lens // 2)
                need = -(-lens // page)
        ids, at = rng.permutation(pool).astype(np.int32), 0
        for k in range(n):
            table[k, :need[k]] = ids[at:at + need[k]]
            at += need[k]
        refs[ids[:at]] = 1
        out["moves"] = int(at) * (pool - int(at)) // pool if seed == 0 else int((refs[at:] > 0).sum())
        gone = np.arange(n) % 5 == 2
        out |= {"gone": np.flatnonzero(gone).astype(np.int32), "grow": np.flatnonzero(~gone).astype(np.int32)}
        out["add"] = np.array([1 if k % 3 else 1 + k % 40 for k in out["grow"]], dtype=np.int32)
        out["add"] = np.minimum(out["add"], c["max_len"] - lens[out["grow"]] + 1).astype(np.int32)
    return out | {"refs": refs, "table": table, "lens": lens, "stride": stride}


def _dev(a, dtype=torch.int32):
    return torch.from_numpy(np.ascontiguousarray(a)).to(device=DEV, dtype=dtype)


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    dt = DT[c["dtype"]]
    s = {"case": c}

    def normal(*shape):
        return torch.randn(shape, generator=g, device=DEV, dtype=dt if dt == torch.float32 else torch.float16)

    if c["op"] == "pages":
        p = _pool(c, seed)
        n, stride, pool = c["seqs"], p["stride"], c["pool"]
        # counts, tables and lengths in one buffer, so that a pass begins with one small copy of the same step's
        s["meta0"] = torch.cat([_dev(p["refs"]), _dev(p["table"]).reshape(-1), _dev(p["lens"])])
        s["meta"] = s["meta0"].clone()
        s["refs"], s["lens"] = s["meta"][:pool], s["meta"][pool + n * stride:]
        s["table"] = s["meta"][pool:pool + n * stride].view(n, stride)
        shape = (c["layers"], pool, c["kv_heads"], c["page"], c["head_dim"])
        s["k"], s["v"] = normal(*shape), normal(*shape)
        if c["kind"] == "beams":
            s["src"], s["dst"] = _dev(p["src"]), _dev(p["dst"])
            s["grow"], s["add"] = s["dst"], torch.ones(n, dtype=torch.int32, device=DEV)
        else:
            s["gone"], s["grow"], s["add"] = _dev(p["gone"]), _dev(p["grow"]), _dev(p["add"])
        if own:
            from sparse_activation_ffn_amd import binding as pb
            s["cache"] = pb.make_kv_cache(s["k"], s["v"])
            s["state"] = pb.make_page_state(s["refs"], s["table"], s["lens"], c["page"])
            s["ws"] = torch.empty(pb.pi_pages_workspace_bytes(s["state"], n), dtype=torch.uint8, device=DEV)
            s["granted"] = torch.empty(s["grow"].numel(), dtype=torch.int32, device=DEV)
            s["copies"] = torch.empty((2, s["grow"].numel()), dtype=torch.int32, device=DEV)
            s["moved"] = torch.empty(pool, dtype=torch.int32, device=DEV)
        return s

    new, lens = _lengths(c)
    n, t = len(new), sum(new)
    hq, hk, d, page = c["q_heads"], c["kv_heads"], c["head_dim"], c["page"]
    need = [-(-x // page) for x in lens]
    pool = sum(need) + 3
    # the pages of a cache that has been in use lie in no order; places after a sequence's last page hold -1
    ids = torch.randperm(pool, generator=g, device=DEV).to(torch.int32)
    table = torch.full((n, max(need) + 1), -1, dtype=torch.int32, device=DEV)
    at = torch.from_numpy(np.concatenate([[0], np.cumsum(need)])).to(DEV)
    col = torch.arange(table.shape[1], device=DEV)
    inside = col[None, :] < (at[1:] - at[:-1])[:, None]
    table[inside] = ids[(at[:-1, None] + col[None, :])[inside]]
    s["k"], s["v"] = normal(1, pool, hk, page, d), normal(1, pool, hk, page, d)
    # queries, keys and values of a step come out of one product: rows with strides
    fused = normal(t, (hq + 2 * hk) * d)
    s["q"] = fused[:, :hq * d].view(t, hq, d)
    s["new_k"] = fused[:, hq * d:(hq + hk) * d].view(t, hk, d)
    s["new_v"] = fused[:, (hq + hk) * d:].view(t, hk, d)
    s["table"], s["new"], s["lens"] = table, new, lens
    s["q_start"] = _dev(np.concatenate([[0], np.cumsum(new)]))
    s["kv_len"] = _dev(np.array(lens))
    s["out"] = torch.empty((t, hq, d), dtype=dt, device=DEV)
    if c["op"] == "attention":
        # heads look as sharply as trained ones do: some over everything, some at few keys
        s["q"].mul_((1 + torch.arange(hq, device=DEV) % 4).to(dt)[None, :, None])
        _, _, first, pre, _, _ = _bounds(c)
        s["lse"] = torch.empty((t, hq), dtype=torch.float32, device=DEV)
        s["scale"] = 1.0 / math.sqrt(d)
        s["slopes"] = _dev(2.0 ** (-8.0 * (np.arange(hq) + 1) / hq), torch.float32) if c["bias"] else None
        s["first"] = _dev(first) if c["doc"] else None
        s["pre"] = _dev(pre) if c["prefix"] else None
    else:
        s["turns"] = _dev(_turns(c["rotary"]), torch.float64)
    if own:
        from sparse_activation_ffn_amd import binding as pb
        s["cache"] = pb.make_kv_cache(s["k"], s["v"])
        s["batch"] = pb.make_seq_batch(s["q_start"], s["kv_len"], table, t, max(new), max(lens))
        if c["op"] == "attention":
            s["rule"] = pb.make_score_rule(s["scale"], c["cap"], s["slopes"], c["window"], s["pre"], s["first"])
            s["ws"] = torch.empty(pb.pi_attention_workspace_bytes(s["cache"], s["batch"], hq), dtype=torch.uint8,
                                  device=DEV)
        else:
            s["rope"] = pb.make_rope(s["turns"], c["pairs"])
    return s


# ---- one pass --------------------------------------------------------------------

def run(state):
    c = state["case"]
    if c["op"] == "attention":
        return _run_attention(state)
    if c["op"] == "rope":
        return _run_rope(state)
    return _run_pages(state)


def _run_attention(s):
    if own:
        from sparse_activation_ffn_amd import binding as pb
        pb.pi_paged_attention(s["cache"], 0, s["batch"], s["rule"], s["q"], s["out"], s["lse"], s["ws"])
        return {"out": s["out"], "lse": s["lse"]}
    c = s["case"]
    hq, hk, d, page = c["q_heads"], c["kv_heads"], c["head_dim"], c["page"]
    n, width, most, g = c["seqs"], s["table"].shape[1], max(s["new"]), c["q_heads"] // c["kv_heads"]
    start, lens = s["q_start"].long(), s["kv_len"].long()
    new = start[1:] - start[:-1]
    # keys and values of every sequence, to the longest: [seq, head, key, d]
    pages = s["table"].long().clamp_min(0)
    k = s["k"][0][pages].transpose(1, 2).reshape(n, hk, width * page, d).float()
    v = s["v"][0][pages].transpose(1, 2).reshape(n, hk, width * page, d).float()
    j = torch.arange(width * page, device=DEV)
    v = torch.where((j < lens[:, None])[:, None, :, None], v, 0.0)
    # queries padded to the most new tokens: [seq, kv head, token, head of the group, d]
    i = torch.arange(most, device=DEV)
    row = (start[:-1, None] + i).clamp_max(s["q"].shape[0] - 1)
    q = s["q"][row].float().view(n, most, hk, g, d).permute(0, 2, 1, 3, 4).reshape(n, hk, most * g, d)
    p = torch.matmul(q, k.transpose(2, 3).contiguous()).view(n, hk, most, g, width * page)
    p.mul_(s["scale"])
    if c["cap"]:
        p.div_(c["cap"]).tanh_().mul_(c["cap"])
    pos = (lens - new)[:, None] + i                                     # [seq, token]
    if s["slopes"] is not None:
        p.sub_(s["slopes"].view(1, hk, 1, g, 1) * (pos[:, :, None] - j).abs().float()[:, None, :, None, :])
    lo = torch.zeros_like(pos) if s["first"] is None else s["first"].long()[row]
    if c["window"]:
        lo = torch.maximum(lo, pos - c["window"] + 1)
    hi = pos + 1 if s["pre"] is None else torch.maximum(pos + 1, s["pre"].long()[:, None])
    hi = torch.minimum(hi, lens[:, None])
    seen = (j >= lo[:, :, None]) & (j < hi[:, :, None])                  # [seq, token, key]
    p.masked_fill_(~seen[:, None, :, None, :], -math.inf)
    m = p.amax(dim=-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p.sub_(m).exp_()
    total = p.sum(dim=-1, keepdim=True)
    o = torch.matmul(p.view(n, hk, most * g, width * page), v).view(n, hk, most, g, d)
    o = torch.where(total > 0, o / total, 0.0)
    lse = (m + total.log()).squeeze(-1)
    real = i < new[:, None]
    o = o.permute(0, 2, 1, 3, 4).reshape(n, most, hq, d)[real]
    return {"out": o.to(s["q"].dtype), "lse": lse.permute(0, 2, 1, 3).reshape(n, most, hq)[real]}


def _run_rope(s):
    if own:
        from sparse_activation_ffn_amd import binding as pb
        pb.pi_rope_append(s["cache"], 0, s["batch"], s["rope"], s["q"], s["out"], s["new_k"], s["new_v"])
        return {"q": s["out"], "k": s["k"], "v": s["v"]}
    c = s["case"]
    page, r = c["page"], c["rotary"]
    t = torch.arange(s["q"].shape[0], device=DEV)
    owner = torch.searchsorted(s["q_start"][1:].long(), t, right=True)
    pos = s["kv_len"].long()[owner] - s["q_start"].long()[owner + 1] + t
    # the angles are kept in 64 bits: at position 100000 a 32-bit product is already off by a hundredth
    a = pos.double()[:, None] * s["turns"][None, :]
    a = (a - a.round()) * (2.0 * math.pi)
    cos, sin = a.cos().float()[:, None, :], a.sin().float()[:, None, :]

    def turned(x):
        x = x.float()
        x0, x1 = (x[..., 0:r:2], x[..., 1:r:2]) if c["pairs"] else (x[..., :r // 2], x[..., r // 2:r])
        y0, y1 = x0 * cos - x1 * sin, x1 * cos + x0 * sin
        y = torch.stack([y0, y1], dim=-1).flatten(-2) if c["pairs"] else torch.cat([y0, y1], dim=-1)
        return torch.cat([y, x[..., r:]], dim=-1)

    dt = s["q"].dtype
    at = s["table"][owner, pos // page].long()
    s["k"][0, at, :, pos % page] = turned(s["new_k"]).to(dt)
    s["v"][0, at, :, pos % page] = s["new_v"]
    return {"q": turned(s["q"]).to(dt), "k": s["k"], "v": s["v"]}


def _run_pages(s):
    c = s["case"]
    s["meta"].copy_(s["meta0"])
    out = {"refs": s["refs"], "table": s["table"], "lens": s["lens"], "k": s["k"], "v": s["v"]}
    if own:
        from sparse_activation_ffn_amd import binding as pb
        if c["kind"] == "compact":
            pb.pi_pages_compact(s["state"], s["cache"], s["moved"], s["ws"])
            return out | {"moved": s["moved"]}
        if c["kind"] == "beams":
            pb.pi_pages_fork(s["state"], s["src"], s["dst"], s["ws"])
        else:
            pb.pi_pages_free(s["state"], s["gone"])
        pb.pi_pages_extend(s["state"], s["cache"], s["grow"], s["add"], s["granted"], s["copies"], s["ws"])
        return out | {"granted": s["granted"], "copies": s["copies"]}
    if c["kind"] == "compact":
        return out | {"moved": _compact(s)}
    if c["kind"] == "beams":
        _fork(s)
    else:
        _free(s, s["gone"].long())
    granted, copies = _extend(s, c["page"])
    return out | {"granted": granted, "copies": copies}


def _count(refs, ids, by):
    """refs[id] += by for every id that is one (not -1)."""
    ids = ids.reshape(-1).long()
    refs.scatter_add_(0, ids.clamp_min(0), torch.where(ids >= 0, by, 0).to(torch.int32))


def _fork(s):
    src, dst = s["src"].long(), s["dst"].long()
    rows, lens, old = s["table"][src], s["lens"][src], s["table"][dst]
    _count(s["refs"], rows, 1)
    _count(s["refs"], old, -1)
    s["table"][dst] = rows
    s["lens"][dst] = lens


def _free(s, gone):
    _count(s["refs"], s["table"][gone], -1)
    s["table"][gone] = -1
    s["lens"][gone] = 0


def _extend(s, page):
    refs, table, lens, seqs, add = s["refs"], s["table"], s["lens"], s["grow"].long(), s["add"]
    stride, now = table.shape[1], lens[seqs]
    have, want = (now + page - 1) // page, (now + add + page - 1) // page
    rows = table[seqs]
    last = rows.gather(1, (have - 1).clamp_min(0).long()[:, None])[:, 0].long()
    shared = (now % page != 0) & (add > 0) & (refs[last.clamp_min(0)] > 1)
    fits = want <= stride
    need = torch.where(fits, want - have + shared.int(), 0)
    total = need.cumsum(0)
    free = torch.argsort((refs != 0).int(), stable=True)
    ok = fits & (total <= (refs == 0).sum())
    # the pages a sequence takes, from the lowest: the copy of its last one first, then the new ones
    begin = have - shared.int()
    col = torch.arange(stride, device=DEV, dtype=torch.int32)
    takes = ok[:, None] & (col >= begin[:, None]) & (col < want[:, None])
    got = free[((total - need)[:, None] + col - begin[:, None]).clamp(0, refs.numel() - 1).long()].int()
    copied = ok & shared
    src = torch.where(copied, last.int(), -1)
    dst = torch.where(copied, got.gather(1, begin.clamp(0, stride - 1).long()[:, None])[:, 0], -1)
    _count(refs, src, -1)
    _count(refs, torch.where(takes, got, -1), 1)
    table[seqs] = torch.where(takes, got, rows)
    lens[seqs] = torch.where(ok, now + add, now)
    at = copied.nonzero()[:, 0]
    a, b = src[at].long(), dst[at].long()
    s["k"][:, b] = s["k"][:, a]
    s["v"][:, b] = s["v"][:, a]
    return ok.int(), torch.stack([src, dst])


def _compact(s):
    refs, table = s["refs"], s["table"]
    ids = torch.arange(refs.numel(), device=DEV)
    live = refs > 0
    count = live.sum()
    hole, mover = ~live & (ids < count), live & (ids >= count)
    holes = torch.argsort((~hole).int(), stable=True)
    to = torch.where(mover, holes[(mover.cumsum(0) - 1).clamp_min(0)], ids)
    moved = torch.where(live, to, -1).int()
    at = mover.nonzero()[:, 0]
    refs[to[at]] = refs[at]
    refs[at] = 0
    table.copy_(torch.where(table >= 0, moved[table.long().clamp_min(0)], -1))
    s["k"][:, to[at]] = s["k"][:, at]
    s["v"][:, to[at]] = s["v"][:, at]
    return moved


# ---- the definition in 64 bits ------------------------------------------------------

def exact(case, seed):
    c = case
    s = prepare(c, seed)
    if c["op"] == "attention":
        return _exact_attention(c, s)
    if c["op"] == "rope":
        return _exact_rope(c, s)
    return _exact_pages(c, s)


def _exact_attention(c, s):
    pos, owner, _, pre, lo, hi = _bounds(c)
    page, g, d = c["page"], c["q_heads"] // c["kv_heads"], c["head_dim"]
    out = torch.zeros((len(pos), c["q_heads"], d), dtype=torch.float64, device=DEV)
    lse = torch.full((len(pos), c["q_heads"]), -math.inf, dtype=torch.float64, device=DEV)
    at = 0
    for b, (new, length) in enumerate(zip(s["new"], s["lens"])):
        ids = s["table"][b, :-(-length // page)].long()
        p64 = torch.from_numpy(pos[at:at + new]).to(DEV)[:, None]
        j = torch.arange(length, device=DEV)[None, :]
        seen = (j >= torch.from_numpy(lo[at:at + new]).to(DEV)[:, None]) & (j < torch.from_numpy(hi[at:at + new]).to(DEV)[:, None])
        for h in range(c["q_heads"]):
            if h % g == 0:
                k = s["k"][0, ids, h // g].reshape(-1, d)[:length].double()
                v = s["v"][0, ids, h // g].reshape(-1, d)[:length].double()
            x = s["q"][at:at + new, h].double() @ k.t() / math.sqrt(d)
            if c["cap"]:
                x = c["cap"] * torch.tanh(x / c["cap"])
            if c["bias"]:
                x = x - float(s["slopes"][h]) * (p64 - j).abs().double()
            x = torch.where(seen, x, -math.inf)
            l = torch.logsumexp(x, dim=1)
            w = torch.where(seen, torch.exp(x - torch.where(l > -math.inf, l, 0.0)[:, None]), 0.0)
            out[at:at + new, h], lse[at:at + new, h] = w @ v, l
        at += new
    return {"out": out, "lse": lse}


def _exact_rope(c, s):
    r, page = c["rotary"], c["page"]
    x, y = s["q"].double(), s["new_k"].double()
    k, v = s["k"].double(), s["v"].double()
    freq = torch.from_numpy(_turns(r)).to(DEV) * (2.0 * math.pi)
    at = 0
    for b, (new, length) in enumerate(zip(s["new"], s["lens"])):
        pos = torch.arange(length - new, length, device=DEV)
        z = torch.polar(torch.ones((), dtype=torch.float64, device=DEV), pos.double()[:, None] * freq)[:, None, :]
        for w in (x, y):
            part = w[at:at + new, :, :r]
            two = part.unflatten(-1, (r // 2, 2)) if c["pairs"] else part.unflatten(-1, (2, r // 2)).transpose(-1, -2)
            turned = torch.view_as_real(torch.view_as_complex(two.contiguous()) * z)
            w[at:at + new, :, :r] = turned.flatten(-2) if c["pairs"] else turned.transpose(-1, -2).flatten(-2)
        where = s["table"][b].long()[pos // page]
        k[0, where, :, pos % page] = y[at:at + new]
        v[0, where, :, pos % page] = s["new_v"][at:at + new].double()
        at += new
    return {"q": x, "k": k, "v": v}


def _exact_pages(c, s):
    refs, lens = s["refs"].cpu().numpy().copy(), s["lens"].cpu().numpy().copy()
    table, page = s["table"].cpu().numpy().copy(), c["page"]
    rows = lambda r: [int(p) for p in r if p >= 0]  # noqa: E731
    more, pairs = {}, []
    if c["kind"] == "compact":
        live = [p for p in range(len(refs)) if refs[p]]
        holes = [p for p in range(len(live)) if not refs[p]]
        pairs = list(zip([p for p in live if p >= len(live)], holes))
        to = {p: p for p in live} | dict(pairs)
        for a, b in pairs:
            refs[b], refs[a] = refs[a], 0
        table = np.array([[to[int(p)] if p >= 0 else -1 for p in r] for r in table], dtype=np.int32)
        more["moved"] = np.array([to.get(p, -1) for p in range(len(refs))], dtype=np.int32)
    else:
        if c["kind"] == "beams":
            before, old = table.copy(), lens.copy()
            for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
                for p in rows(before[a]):
                    refs[p] += 1
                for p in rows(before[b]):
                    refs[p] -= 1
                table[b], lens[b] = before[a], old[a]
        else:
            for b in s["gone"].tolist():
                for p in rows(table[b]):
                    refs[p] -= 1
                table[b], lens[b] = -1, 0
        at_start = refs.copy()
        free, granted, copies, open_ = [p for p in range(len(refs)) if not refs[p]], [], [], True
        for b, add in zip(s["grow"].tolist(), s["add"].tolist()):
            have, want = -(-int(lens[b]) // page), -(-(int(lens[b]) + add) // page)
            last = int(table[b, have - 1]) if have else -1
            copy = bool(lens[b] % page and add > 0 and at_start[last] > 1)
            fits = want <= table.shape[1]
            open_ = open_ and (not fits or want - have + copy <= len(free))
            pair = (-1, -1)
            if fits and open_:
                if copy:
                    pair = (last, free.pop(0))
                    refs[last] -= 1
                    refs[pair[1]] = 1
                    table[b, have - 1] = pair[1]
                    pairs.append(pair)
                for e in range(have, want):
                    table[b, e] = free.pop(0)
                    refs[table[b, e]] = 1
                lens[b] += add
            granted.append(int(fits and open_))
            copies.append(pair)
        more = {"granted": np.array(granted, dtype=np.int32), "copies": np.array(copies, dtype=np.int32).T.copy()}
    k, v = s["k"].double(), s["v"].double()
    for a, b in pairs:
        k[:, b], v[:, b] = k[:, a].clone(), v[:, a].clone()
    return {"refs": refs, "table": table, "lens": lens, "k": k, "v": v} | more
