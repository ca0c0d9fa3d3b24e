"""Measured cases of the paged key-value cache operators.

Three operators serve the attention branch of a decode loop whose sequences share a pool of
pages instead of owning one contiguous cache each:

  append   the new tokens' keys (rotated to their positions) and values go into their
           sequences' pages; the queries are rotated on the way; each page keeps the smallest
           and the largest key value per channel (its bounds)
  select   per sequence and key-value head, the pages that a decode query should read: the
           first ones (meta tokens), the last ones, and those with the largest upper bound on
           the query heads' summed scores, computed from the page bounds
  attend   attention of one new token per sequence over its pages: all of them, the meta
           tokens and a sliding window, or the selected ones

`run` computes them in plain torch operations, or calls the library where `own` is true.
A pool is [n_pages, n_kv_heads, page_size, head_dim]; a block table row lists a sequence's
pages in order; a sequence of length n holds positions 0 .. n - 1.
"""
import math

import torch

own = False

_DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------
def _case(name, op, batch, length, hq, hkv, dim, page, dtype, **kw):
    c = {"name": name, "op": op, "batch": batch, "length": length, "hq": hq, "hkv": hkv, "dim": dim, "page": page,
         "dtype": dtype, "ragged": False, "src": "f32", "new": 1, "rope_base": 10000.0, "bounds": False, "first": 0,
         "last": 1, "top": 0, "meta": 0, "window": 0, "idle": 0, "out": dtype, "lse": False}
    c.update(kw)
    return c


def listed():
    return [
        # one chat's decode step at the mixer's heads: only latency counts
        _case("append_step_1", "append", 1, 4129, 25, 5, 64, 64, "f16", bounds=True),
        # the decode batch of the mixer's decode workload, from the fp32 projection
        _case("append_step_64", "append", 64, 4129, 25, 5, 64, 64, "f16", bounds=True, ragged=True),
        # ragged prompt pieces with odd starts, 16-token pages, wide heads, bf16 activations
        _case("append_prompts_ragged", "append", 7, 2047, 32, 8, 128, 16, "bf16", src="bf16", new=1500, ragged=True,
              bounds=True),
        # four whole prompts of the full-attention workload
        _case("append_prompts_8320", "append", 4, 8320, 25, 5, 64, 64, "f16", src="bf16", new=8320),
        # page choice for one very long context
        _case("select_131073_1", "select", 1, 131073, 25, 5, 64, 64, "f16", first=2, last=2, top=64),
        # page choice for a full batch of mixed lengths
        _case("select_16384_64", "select", 64, 16384, 25, 5, 64, 32, "f16", ragged=True, first=4, last=2, top=48),
        # a short chat's step at the smallest heads: launch latency
        _case("attend_37_1", "attend", 1, 37, 4, 2, 64, 16, "f16", lse=True),
        # a sliding-window layer of the decode workload: 128 meta tokens and 1024 keys each
        _case("attend_window_64", "attend", 64, 4129, 25, 5, 64, 64, "f16", meta=128, window=1024, out="f32"),
        # a full-attention layer, mixed lengths, every seventh slot idle
        _case("attend_8320_64", "attend", 64, 8320, 25, 5, 64, 64, "f16", ragged=True, idle=7),
        # wide heads in bf16 on small pages, long and short contexts together
        _case("attend_65537_8", "attend", 8, 65537, 32, 4, 128, 16, "bf16", ragged=True, lse=True),
        # one very long context, split over the whole GPU and joined
        _case("attend_131073_1", "attend", 1, 131073, 25, 5, 64, 64, "f16", out="f32", lse=True),
        # the selected pages of a full batch
        _case("attend_selected_64", "attend", 64, 16384, 25, 5, 64, 32, "f16", ragged=True, top=48, first=4, last=2),
    ]


def draw(rng):
    log = lambda lo, hi: int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    op = rng.choice(["append", "select", "attend", "attend"])
    hq, hkv = rng.choice([(25, 5), (4, 2), (32, 8), (32, 4), (6, 6), (15, 3), (16, 1), (9, 1)])
    dim = rng.choice([64, 64, 128])
    page = rng.choice([16, 32, 64, 128])
    dtype = rng.choice(["f16", "bf16"])
    batch = log(1, 64)
    room = 260000 * 320 // (hkv * dim)            # tokens of all sequences, as in the largest listed case
    length = log(1, min(131073, max(2, room // batch)))
    kw = {"ragged": rng.random() < 0.7}
    if op == "append":
        kw["src"] = rng.choice(["f32", "bf16", "f16"])
        kw["new"] = 1 if rng.random() < 0.5 else log(1, max(1, min(length, 33280 // batch)))
        kw["bounds"] = rng.random() < 0.5
        kw["rope_base"] = rng.choice([10000.0, 500000.0])
        length = max(length, kw["new"])
    elif op == "select":
        kw["first"] = rng.choice([0, 1, 3])
        kw["last"] = rng.choice([1, 2])
        length = max(length, 32 * page)           # enough pages to choose among
        kw["top"] = kw["first"] + kw["last"] + log(4, min(96, length // page - 8))
    else:
        kw["out"] = rng.choice([dtype, "f32"])
        kw["idle"] = rng.choice([0, 5])
        kw["lse"] = kw["idle"] == 0
        mode = rng.choice(["all", "all", "window", "selected"])
        if mode == "window":
            kw["window"] = log(1, 2048)
            kw["meta"] = rng.choice([0, 8, 128])
        elif mode == "selected":
            kw["first"], kw["last"] = rng.choice([(0, 1), (2, 1)])
            kw["top"] = kw["first"] + kw["last"] + log(1, 96)
    c = _case("", op, batch, length, hq, hkv, dim, page, dtype, **kw)
    del c["name"]
    return c


# ---------------------------------------------------------------------------------------
# sizes that follow from a case
# ---------------------------------------------------------------------------------------
def _lengths(c):
    """Keys of each sequence after this step (0 for an idle slot)."""
    out = []
    for b in range(c["batch"]):
        n = c["length"]
        if c["ragged"] and b > 0:
            n = 1 + int((n - 1) * math.modf(b * 0.6180339887498949)[0])
        if c["idle"] and b % c["idle"] == c["idle"] - 1:
            n = 0
        out.append(n)
    return out


def _new(c):
    """New tokens of each sequence (append): the last ones of its length."""
    return [min(n, 1 + (c["new"] - 1) * (b % 3 + 1) // 3 if c["ragged"] else c["new"])
            for b, n in enumerate(_lengths(c))]


def _pages(c):
    return [-(-n // c["page"]) for n in _lengths(c)]


def _visible(c, n, pages):
    """Keys that one query reads."""
    if c["top"]:
        return n - max(0, pages - c["top"]) * c["page"]
    if c["window"]:
        w = min(n, c["window"])
        return w + min(c["meta"], n - w)
    return n


def work(case):
    c = case
    lens, pages = _lengths(c), _pages(c)
    esz = 2
    kvw, qw = c["hkv"] * c["dim"], c["hq"] * c["dim"]
    if c["op"] == "append":
        t = sum(_new(c))
        src = 4 if c["src"] == "f32" else 2
        touched = sum((n - 1) // c["page"] - (n - m) // c["page"] + 1 for n, m in zip(lens, _new(c)) if m)
        nbytes = t * (qw + 2 * kvw) * (src + esz) + touched * (4 + (2 * kvw * esz if c["bounds"] else 0)) + 8 * c["batch"]
        return {"bytes": nbytes, "flops": t * 3 * (qw + kvw)}
    if c["op"] == "select":
        n = sum(pages)
        return {"bytes": n * (2 * kvw * esz + 4) + c["batch"] * (qw * esz + 4 + c["hkv"] * c["top"] * 4),
                "flops": n * 4 * kvw}
    seen = sum(_visible(c, n, p) for n, p in zip(lens, pages))
    osz = 4 if c["out"] == "f32" else 2
    ids = seen // c["page"] * 4 * (1 + (c["hkv"] if c["top"] else 0))
    return {"bytes": seen * 2 * kvw * esz + ids + c["batch"] * (qw * (esz + osz) + 4),
            "flops": seen * 4 * qw}


# ---------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------
def _inputs(c, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    dt, D, Hq, Hkv, ps, B = _DT[c["dtype"]], c["dim"], c["hq"], c["hkv"], c["page"], c["batch"]
    randn = lambda *s: torch.randn(*s, generator=g, device=dev)
    lens, pages, new = _lengths(c), _pages(c), _new(c)
    used = sum(pages)
    n_pages = used + max(1, used // 16)           # some pages of the pool are free
    width = max(1, max(pages))
    perm = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)
    table = torch.full((B, width), -1, dtype=torch.int32, device=dev)
    at = 0
    for b in range(B):
        table[b, :pages[b]] = perm[at:at + pages[b]]
        at += pages[b]
    s = {"case": c, "table": table, "lens": torch.tensor(lens, dtype=torch.int32, device=dev)}
    # pages hold the earlier tokens, and behind a sequence's end what their last user left
    s["k"] = randn(n_pages, Hkv, ps, D).to(dt)
    s["v"] = randn(n_pages, Hkv, ps, D).to(dt)
    if c["op"] == "append":
        t = sum(new)
        proj = (randn(t, (Hq + 2 * Hkv) * D) * 1.3).to(_DT[c["src"]])     # one fused projection's rows
        s["q_new"] = proj[:, :Hq * D].view(t, Hq, D)
        s["k_new"] = proj[:, Hq * D:(Hq + Hkv) * D].view(t, Hkv, D)
        s["v_new"] = proj[:, (Hq + Hkv) * D:].view(t, Hkv, D)
        s["q_out"] = torch.zeros(t, Hq, D, dtype=dt, device=dev)
        s["start"] = torch.tensor([n - m for n, m in zip(lens, new)], dtype=torch.int32, device=dev)
        cu = [0]
        for m in new:
            cu.append(cu[-1] + m)
        s["cu_new"] = torch.tensor(cu, dtype=torch.int32, device=dev)
        if c["bounds"]:
            s["k_lo"], s["k_hi"] = s["k"].amin(2), s["k"].amax(2)
        return s
    s["q"] = (randn(B, Hq, D) * 1.5).to(dt)
    if c["op"] == "select":
        # the extremes of a page's normal keys: about sqrt(2 ln page_size) either way
        mid = math.sqrt(2 * math.log(ps))
        s["k_hi"] = (mid + 0.4 * randn(n_pages, Hkv, D)).to(dt)
        s["k_lo"] = (-mid + 0.4 * randn(n_pages, Hkv, D)).to(dt)
        s["page_idx"] = torch.zeros(B, Hkv, c["top"], dtype=torch.int32, device=dev)
        return s
    if c["top"]:
        # a choice of pages as `select` makes it: ascending, the first and last among them
        sc = torch.rand(B, Hkv, width, generator=g, device=dev)
        j = torch.arange(width, device=dev)
        n = torch.tensor(pages, device=dev)[:, None, None]
        sc = torch.where((j < c["first"]) | (j >= n - c["last"]), 2.0, sc)
        sc = torch.where(j < n, sc, -1.0)
        k = min(c["top"], width)
        best = sc.topk(k, dim=-1)
        idx = torch.where(best.values < 0, width, best.indices).sort(dim=-1).values
        idx = torch.where(idx == width, -1, idx)
        s["page_idx"] = torch.full((B, Hkv, c["top"]), -1, dtype=torch.int32, device=dev)
        s["page_idx"][..., :k] = idx.to(torch.int32)
    s["out"] = torch.zeros(B, Hq, D, dtype=_DT[c["out"]], device=dev)
    s["lse"] = torch.zeros(B, Hq, dtype=torch.float32, device=dev) if c["lse"] else None
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        # what a serving program makes once: the cache's handle and a workspace
        from hybrid_attention_ssm_b200 import hymba as H
        s["cache"] = H.PagedCache(s["k"], s["v"], s.get("k_lo"), s.get("k_hi"))
        s["ws"] = H.alloc_workspace(H.paged_workspace_size(s["cache"], case["batch"], case["hq"], s["table"].shape[1]))
    return s


# ---------------------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------------------
def _rotate(x, pos, base):
    """Half-split rotation: the pair (j, j + D/2) turns by pos * base^(-2j/D)."""
    h = x.shape[-1] // 2
    theta = base ** (-torch.arange(h, dtype=torch.float64, device=x.device) / h)
    ang = pos.double()[:, None] * theta
    cs, sn = ang.cos().float()[:, None], ang.sin().float()[:, None]
    a, b = x[..., :h], x[..., h:]
    return torch.cat([a * cs - b * sn, b * cs + a * sn], dim=-1)


def _append(s):
    c = s["case"]
    ps, Hkv, D = c["page"], c["hkv"], c["dim"]
    dt = s["k"].dtype
    t = s["k_new"].shape[0]
    i = torch.arange(t, device=s["k"].device)
    b = torch.bucketize(i, s["cu_new"][1:], right=True)
    pos = s["start"].long()[b] + i - s["cu_new"].long()[b]
    page, row = s["table"].long()[b, pos // ps], pos % ps
    k = _rotate(s["k_new"].float(), pos, c["rope_base"]).to(dt)
    s["q_out"].copy_(_rotate(s["q_new"].float(), pos, c["rope_base"]).to(dt))
    s["k"][page, :, row] = k
    s["v"][page, :, row] = s["v_new"].to(dt)
    out = {"q": s["q_out"], "k": s["k"], "v": s["v"]}
    if c["bounds"]:
        lo, hi = s["k_lo"].float(), s["k_hi"].float()
        fresh = page[row == 0]                     # a page begun in this call starts over
        lo[fresh], hi[fresh] = math.inf, -math.inf
        at = page[:, None, None].expand(t, Hkv, D)
        s["k_lo"].copy_(lo.scatter_reduce(0, at, k.float(), "amin"))
        s["k_hi"].copy_(hi.scatter_reduce(0, at, k.float(), "amax"))
        out["k_lo"], out["k_hi"] = s["k_lo"], s["k_hi"]
    return out


def _select(s):
    c = s["case"]
    B, Hkv, D, K = c["batch"], c["hkv"], c["dim"], c["top"]
    q = s["q"].double().view(B, Hkv, -1, D)
    up, dn = q.clamp(min=0).sum(2), q.clamp(max=0).sum(2)                  # [B, Hkv, D]
    table = s["table"].long().clamp(min=0)
    hi, lo = s["k_hi"][table].double(), s["k_lo"][table].double()          # [B, W, Hkv, D]
    score = (hi * up[:, None]).sum(-1) + (lo * dn[:, None]).sum(-1)        # [B, W, Hkv]
    score = score.transpose(1, 2)
    W = score.shape[-1]
    j = torch.arange(W, device=score.device)
    n = ((s["lens"].long() + c["page"] - 1) // c["page"])[:, None, None]
    score = torch.where((j < c["first"]) | (j >= n - c["last"]), math.inf, score)
    score = torch.where(j < n, score, -math.inf)
    order = score.sort(dim=-1, descending=True, stable=True).indices[..., :K]
    order = torch.where(order < n, order, W).sort(dim=-1).values
    k = order.shape[-1]
    s["page_idx"].fill_(-1)
    s["page_idx"][..., :k] = torch.where(order == W, -1, order).to(torch.int32)
    return s["page_idx"]


def _attend(s):
    c = s["case"]
    B, Hkv, D, ps = c["batch"], c["hkv"], c["dim"], c["page"]
    G = c["hq"] // Hkv
    r = torch.arange(ps, device=s["q"].device)
    lens = s["lens"].long()
    if c["top"]:
        idx = s["page_idx"].long()                                         # [B, Hkv, P]
        ids = s["table"].long().gather(1, idx.clamp(min=0).view(B, -1)).view_as(idx)
        heads = torch.arange(Hkv, device=idx.device)[None, :, None]
        k, v = s["k"][ids.clamp(min=0), heads], s["v"][ids.clamp(min=0), heads]
        pos = idx[..., None] * ps + r
        seen = (idx[..., None] >= 0) & (pos < lens[:, None, None, None])
    else:
        ids = s["table"].long().clamp(min=0)                               # [B, W]
        k, v = s["k"][ids].transpose(1, 2), s["v"][ids].transpose(1, 2)    # [B, Hkv, W, ps, D]
        pos = torch.arange(ids.shape[1], device=ids.device)[:, None] * ps + r
        seen = pos < lens[:, None, None]
        if c["window"]:
            seen = seen & ((pos < c["meta"]) | (pos >= lens[:, None, None] - c["window"]))
        seen = seen[:, None].expand(B, Hkv, -1, -1)
    k, v, seen = k.reshape(B, Hkv, -1, D).float(), v.reshape(B, Hkv, -1, D).float(), seen.reshape(B, Hkv, 1, -1)
    x = torch.matmul(s["q"].float().view(B, Hkv, G, D), k.transpose(-1, -2)) * D ** -0.5
    x = torch.where(seen, x, -math.inf)
    m = x.amax(-1, keepdim=True)
    e = torch.where(seen, (x - torch.where(m == -math.inf, 0.0, m)).exp(), 0.0)
    z = e.sum(-1, keepdim=True)
    o = torch.matmul(e, v) / torch.where(z == 0, 1.0, z)
    s["out"].copy_(o.view(B, c["hq"], D).to(s["out"].dtype))
    if s["lse"] is None:
        return s["out"]
    s["lse"].copy_((m + z.log()).view(B, c["hq"]))
    return s["out"], s["lse"]


def run(state):
    s = state
    c = s["case"]
    if own:
        from hybrid_attention_ssm_b200 import hymba as H
        if c["op"] == "append":
            H.paged_append(s["cache"], s["table"], s["start"], s["k_new"], s["v_new"], s["ws"], q=s["q_new"],
                           q_out=s["q_out"], cu_new=s["cu_new"], rope_base=c["rope_base"])
            out = {"q": s["q_out"], "k": s["k"], "v": s["v"]}
            if c["bounds"]:
                out["k_lo"], out["k_hi"] = s["k_lo"], s["k_hi"]
            return out
        if c["op"] == "select":
            H.paged_select(s["cache"], s["q"], s["table"], s["lens"], s["page_idx"], s["ws"], n_first=c["first"],
                           n_last=c["last"])
            return s["page_idx"]
        H.paged_attention(s["cache"], s["q"], s["table"], s["lens"], s["out"], s["ws"], n_meta=c["meta"],
                          window=c["window"], page_idx=s.get("page_idx"), lse=s["lse"])
        return s["out"] if s["lse"] is None else (s["out"], s["lse"])
    return {"append": _append, "select": _select, "attend": _attend}[c["op"]](s)


# ---------------------------------------------------------------------------------------
# the definitions in 64 bits, sequence by sequence
# ---------------------------------------------------------------------------------------
def exact(case, seed):
    c = case
    s = _inputs(c, seed)
    ps, D, Hq, Hkv = c["page"], c["dim"], c["hq"], c["hkv"]
    G = Hq // Hkv
    lens, table = _lengths(c), s["table"].tolist()
    if c["op"] == "append":
        return _exact_append(c, s, table)
    if c["op"] == "select":
        res = torch.full((c["batch"], Hkv, c["top"]), -1, dtype=torch.int32)
        for b, n in enumerate(_pages(c)):
            if n == 0:
                continue
            rows = torch.tensor(table[b][:n], device="cuda")
            lo, hi = s["k_lo"][rows].double(), s["k_hi"][rows].double()
            q = s["q"][b].double().view(Hkv, G, D)
            # per head the largest value of q.k over keys inside the page's box, summed over the group
            sc = [torch.maximum(q[g][:, None] * lo[:, g], q[g][:, None] * hi[:, g]).sum((0, 2)).tolist()
                  for g in range(Hkv)]
            forced = [j for j in range(n) if j < c["first"] or j >= n - c["last"]]
            for g in range(Hkv):
                rest = sorted((j for j in range(n) if j not in set(forced)), key=lambda j: (-sc[g][j], j))
                pick = sorted(forced + rest[:max(0, c["top"] - len(forced))])[:c["top"]]
                res[b, g, :len(pick)] = torch.tensor(pick, dtype=torch.int32)
        return res.cuda()
    out = torch.zeros(c["batch"], Hq, D, dtype=torch.float64, device="cuda")   # an idle slot's row is zero
    lse = torch.full((c["batch"], Hq), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(lens):
        if n == 0:
            continue
        for g in range(Hkv):
            if c["top"]:
                pages = [j for j in s["page_idx"][b, g].tolist() if j >= 0]
                pos = torch.cat([torch.arange(j * ps, min(n, (j + 1) * ps)) for j in pages]).cuda()
            else:
                pos = torch.arange(n, device="cuda")
                if c["window"]:
                    pos = pos[(pos < c["meta"]) | (pos >= n - c["window"])]
            page = torch.tensor(table[b], device="cuda")[pos // ps]
            k, v = s["k"][page, g, pos % ps].double(), s["v"][page, g, pos % ps].double()
            x = s["q"][b, g * G:(g + 1) * G].double() @ k.T / math.sqrt(D)
            lse[b, g * G:(g + 1) * G] = torch.logsumexp(x, -1)
            out[b, g * G:(g + 1) * G] = torch.softmax(x, -1) @ v
    return out if s["lse"] is None else (out, lse)


def _exact_append(c, s, table):
    ps, D = c["page"], c["dim"]
    k, v = s["k"].double(), s["v"].double()
    q = torch.zeros_like(s["q_out"], dtype=torch.float64)
    bounds = [s["k_lo"].double(), s["k_hi"].double()] if c["bounds"] else None
    at = 0
    for b, (n, m) in enumerate(zip(_lengths(c), _new(c))):
        if m == 0:
            continue
        pos = torch.arange(n - m, n, dtype=torch.float64, device="cuda")
        j = torch.arange(D // 2, dtype=torch.float64, device="cuda")
        turn = torch.polar(torch.ones(m, D // 2, dtype=torch.float64, device="cuda"),
                           torch.outer(pos, torch.exp(j * (-2.0 * math.log(c["rope_base"]) / D))))[:, None]

        def rotated(x):
            z = torch.complex(x[..., :D // 2].double(), x[..., D // 2:].double()) * turn
            return torch.cat([z.real, z.imag], -1)

        kb, qb = rotated(s["k_new"][at:at + m]), rotated(s["q_new"][at:at + m])
        q[at:at + m] = qb
        p = pos.long()
        page = torch.tensor(table[b], device="cuda")[p // ps]
        k[page, :, p % ps] = kb
        v[page, :, p % ps] = s["v_new"][at:at + m].double()
        if bounds:
            for pg in range((n - m) // ps, (n - 1) // ps + 1):
                rows = kb[max(0, pg * ps - (n - m)):(pg + 1) * ps - (n - m)]
                old = pg * ps < n - m              # the page was begun by an earlier call
                for t, f in zip(bounds, (torch.amin, torch.amax)):
                    x = f(rows, 0)
                    t[table[b][pg]] = f(torch.stack([x, t[table[b][pg]]]), 0) if old else x
        at += m
    out = {"q": q, "k": k, "v": v}
    if bounds:
        out["k_lo"], out["k_hi"] = bounds
    return out
