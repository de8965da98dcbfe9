"""The serving-step operators on the paged KV pool: what is measured, and their plain forms.

  append   new tokens: per-head norm of queries and keys, position rotation, K/V rows into the pool's pages
  attend   attention over the pool for requests that share a prefix (read once) and own a suffix each
  pages    page copies inside the pool: forks of tail pages, compaction, reordering

`own` selects the framework's kernels; otherwise `run` computes the same with elementary torch
operations in 32 bits (angles in 64).
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------------------ cases
def _gqa(heads, kv_heads, head_dim):
    return {"family": "gqa", "dtype": "bf16", "heads": heads, "kv_heads": kv_heads, "head_dim": head_dim}


def _mla(heads):
    return {"family": "mla", "dtype": "bf16", "heads": heads, "latent": 512, "rope": 64}


def listed():
    vl7b, deque, mha = _gqa(28, 4, 128), _gqa(32, 8, 128), _gqa(32, 32, 128)
    return [
        # a handful of chat turns on one cached image: latency
        dict(vl7b, name="attend_few", op="attend", layers=2, page=16, requests=4, prefix=1000, own_lo=1, own_hi=64, q_lo=1, q_hi=1),
        # a serving batch on one video of eight 1024-token segments, one token each
        dict(deque, name="attend_decode", op="attend", layers=4, page=16, requests=64, prefix=8192, own_lo=17, own_hi=1500, q_lo=1, q_hi=1),
        # the longest shared context
        dict(deque, name="attend_long", op="attend", layers=2, page=16, requests=16, prefix=131072, own_lo=1, own_hi=4096, q_lo=1, q_hi=1),
        # one KV head per query head, four 2048-token document chunks
        dict(mha, name="attend_mha", op="attend", layers=2, page=16, requests=32, prefix=8192, own_lo=1, own_hi=256, q_lo=1, q_hi=1),
        # questions of several hundred tokens on the shared video, all at once (the first pass of each request)
        dict(vl7b, name="attend_extend", op="attend", layers=1, page=16, requests=8, prefix=8192, own_lo=0, own_hi=700, q_lo=33, q_hi=731),
        # latent rows: 16 heads read one 576-wide row a token
        dict(_mla(16), name="attend_mla", op="attend", layers=4, page=16, requests=32, prefix=4096, own_lo=1, own_hi=1024, q_lo=1, q_hi=1),
        # the single-precision layout, a few tokens a request (speculated ones)
        dict(_gqa(8, 2, 64), name="attend_f32", dtype="f32", op="attend", layers=1, page=16, requests=5, prefix=300, own_lo=0, own_hi=40, q_lo=1, q_hi=9),
        # one token of 64 requests
        dict(vl7b, name="append_decode", op="append", layers=4, page=16, requests=64, prefix=0, own_lo=1, own_hi=1024, q_lo=1, q_hi=1, norm=True, sections=False),
        # prompts with (t, h, w) positions, ragged
        dict(deque, name="append_prompt", op="append", layers=1, page=16, requests=7, prefix=0, own_lo=0, own_hi=300, q_lo=257, q_hi=2048, norm=True, sections=True),
        # latent rows of a prompt
        dict(_mla(16), name="append_mla", op="append", layers=2, page=16, requests=3, prefix=0, own_lo=0, own_hi=64, q_lo=100, q_hi=1024, norm=True, sections=False),
        # 64 requests fork the partly filled last page of what they share
        dict(vl7b, name="pages_fork", op="pages", kind="fork", layers=28, page=16, pages=2048, moves=64),
        # a quarter of a deque's pool has been evicted: the rest moves together
        dict(deque, name="pages_compact", op="pages", kind="compact", layers=12, page=16, pages=4096, moves=768),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "append", "append", "pages"])
    shape = rng.choice([_gqa(28, 4, 128), _gqa(32, 8, 128), _gqa(32, 32, 128), _gqa(16, 2, 128), _gqa(16, 4, 64), _gqa(12, 12, 64),
                        _mla(16), _mla(32), dict(_gqa(8, 2, 64), dtype="f32")])
    page = rng.choice([8, 16, 16, 32, 64])
    small = shape["dtype"] == "f32"
    if op == "pages":
        pages = _log(rng, 300, 4096)
        return dict(shape, op=op, kind=rng.choice(["fork", "compact", "permute"]), layers=rng.randint(1, 8), page=min(page, 32), pages=pages,
                    moves=_log(rng, 1, pages // 4))
    if op == "append":
        decode = rng.random() < 0.5
        return dict(shape, op=op, layers=rng.randint(1, 4), page=page, requests=_log(rng, 1, 200) if decode else rng.randint(1, 4), prefix=0,
                    own_lo=0, own_hi=_log(rng, 1, 1000), q_lo=1, q_hi=1 if decode else _log(rng, 2, 1024), norm=rng.random() < 0.7,
                    sections=rng.random() < 0.5)
    for _ in range(1000):
        c = dict(shape, op=op, layers=rng.randint(1, 2), page=page, requests=_log(rng, 1, 20 if small else 100),
                 prefix=_log(rng, 16, 600 if small else 131072), own_lo=rng.choice([0, 1, 16]), own_hi=_log(rng, 17, 100 if small else 4096), q_lo=1,
                 q_hi=1 if rng.random() < 0.6 else _log(rng, 2, 9 if small else 700))
        w, most = work(c), work(listed()[4])
        if w["flops"] <= most["flops"] and w["bytes"] <= 1.2e9 and c["layers"] * sum(_lengths(c)[1]) * c["heads"] * (c["prefix"] + max(_lengths(c)[0])) < 1.2e9:
            return c
    return dict(shape, op=op, layers=1, page=page, requests=_log(rng, 1, 9), prefix=_log(rng, 16, 600), own_lo=0, own_hi=_log(rng, 17, 60), q_lo=1, q_hi=1)


def _lengths(c):
    """(own tokens, query tokens) of every request; a request's last query tokens are among its own."""
    r = np.arange(c["requests"], dtype=np.int64)
    q = c["q_lo"] + (r * 2654435761 % (1 << 32) >> 7) % (c["q_hi"] - c["q_lo"] + 1)
    old = c["own_lo"] + (r * 40503 + 977) * 2246822519 % (1 << 32) % (c["own_hi"] - c["own_lo"] + 1)
    return old + q, q


def _widths(c):
    """(KV heads, key width, value width, row width F)."""
    if c["family"] == "mla":
        f = c["latent"] + c["rope"]
        return 1, f, c["latent"], f
    return c["kv_heads"], c["head_dim"], c["head_dim"], c["kv_heads"] * c["head_dim"]


def work(case):
    c = case
    hkv, dk, dv, f = _widths(c)
    e = 4 if c["dtype"] == "f32" else 2
    tensors = 1 if c["family"] == "mla" else 2
    if c["op"] == "pages":
        return {"bytes": 2 * c["moves"] * c["page"] * f * e * tensors * c["layers"], "flops": 0}
    own_len, q_len = _lengths(c)
    n = int(q_len.sum())
    if c["op"] == "append":
        row = c["heads"] * dk + tensors * f
        return {"bytes": 2 * c["layers"] * n * row * e, "flops": 10 * c["layers"] * n * row}
    pairs = n * c["prefix"] + int((q_len * own_len - q_len * (q_len - 1) // 2).sum())
    rows = c["prefix"] + int(own_len.sum())
    return {"bytes": c["layers"] * (rows * f * e * tensors + n * c["heads"] * ((dk + dv) * e + 4)),
            "flops": 2 * c["layers"] * pairs * c["heads"] * (dk + dv)}


# ------------------------------------------------------------------------------------------ inputs
def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device=DEV, dtype=torch.float32)


def _pool(gen, c, pages, f):
    """Keys with a few large channels, as trained keys have them; values without."""
    shape, t = (c["layers"], pages, c["page"], f), TYPES[c["dtype"]]
    k = torch.empty(shape, device=DEV, dtype=t)
    k.normal_(generator=gen)
    k[..., 5::64] *= 4.0
    if c["family"] == "mla":
        return k, None
    v = torch.empty(shape, device=DEV, dtype=t)
    v.normal_(generator=gen)
    return k, v


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    host = np.random.default_rng([seed, 77])
    hkv, dk, dv, f = _widths(c)
    t = TYPES[c["dtype"]]
    s = {"case": c}
    if c["op"] == "pages":
        s["k"], s["v"] = _pool(gen, c, c["pages"], f)
        order = host.permutation(c["pages"]).astype(np.int32)
        n = c["moves"]
        if c["kind"] == "fork":  # a few shared tails, each into pages of their own
            s["src"], s["dst"] = order[:max(1, n // 16)][np.arange(n) % max(1, n // 16)].copy(), order[n:2 * n].copy()
        elif c["kind"] == "permute":  # pages of one sequence into the order of its tokens
            s["src"], s["dst"] = order[:n].copy(), np.sort(order[:n])
        else:  # tables of what stays: `moves` of its pages lie beyond their number
            live = c["pages"] - n - c["pages"] // 8
            high = live + host.permutation(c["pages"] - live)[:n]
            low = host.permutation(live)[:live - n]
            s["table"] = host.permutation(np.concatenate([low, high])).astype(np.int32)
        if "src" in s:
            s["src_dev"], s["dst_dev"] = (torch.from_numpy(s[k].astype(np.int64)).to(DEV) for k in ("src", "dst"))
        else:
            s["table_dev"] = torch.from_numpy(s["table"].astype(np.int64)).to(DEV)
        return s

    own_len, q_len = _lengths(c)
    n, p, r = int(q_len.sum()), c["page"], c["requests"]
    slot0 = c["prefix"] % p  # a request's first page is its copy of the prefix's last one
    own_pages = (slot0 + own_len + p - 1) // p
    prefix_pages = -(-c["prefix"] // p)
    pages = int(own_pages.sum()) + prefix_pages + 3
    order = host.permutation(pages).astype(np.int32)
    s["k"], s["v"] = _pool(gen, c, pages, f)
    s["pages"], s["slot0"], s["own_len"], s["q_len"] = pages, slot0, own_len, q_len
    s["prefix_table"] = order[:prefix_pages].copy()
    s["tables"] = np.zeros((r, int(own_pages.max())), np.int32)
    s["tables"][np.arange(s["tables"].shape[1])[None] < own_pages[:, None]] = order[prefix_pages:prefix_pages + int(own_pages.sum())]
    for name in ("prefix_table", "tables", "own_len", "q_len"):
        s[name + "_dev"] = torch.from_numpy(s[name].astype(np.int64)).to(DEV)
    s["request_dev"] = torch.from_numpy(np.repeat(np.arange(r), q_len)).to(DEV)  # of every query token
    s["index_dev"] = torch.from_numpy(np.concatenate([np.arange(m) for m in q_len])).to(DEV)  # its number in its request
    heads = c["heads"]
    if c["op"] == "attend":
        s["q"] = (_normal(gen, c["layers"], n, heads, dk) * 1.5).to(t)
        s["out"] = torch.empty(c["layers"], n, heads, dv, device=DEV, dtype=t)
        s["lse"] = torch.empty(c["layers"], n, heads, device=DEV, dtype=torch.float32)
        s["scale"] = 1.0 / math.sqrt(192.0 if c["family"] == "mla" else dk)
        return s
    # the projections' output: one row a token, queries, keys and values side by side
    s["rows"] = (_normal(gen, c["layers"], n, heads * dk + f * (1 if c["family"] == "mla" else 2)) * 2.0).to(t)
    s["q_out"] = torch.empty(c["layers"], n, heads * dk, device=DEV, dtype=t)
    s["q_weight"] = (1.0 + 0.2 * _normal(gen, dk)).to(t) if c["norm"] and c["family"] == "gqa" else None
    s["k_weight"] = (1.0 + 0.2 * _normal(gen, dk if c["family"] == "gqa" else dv)).to(t) if c["norm"] else None
    s["start"] = 40000 + 7 * np.arange(r)  # where a request's own tokens begin
    s["start_dev"] = torch.from_numpy(s["start"]).to(DEV)
    s["positions"] = None
    if c["sections"]:
        i = np.concatenate([np.arange(m) for m in q_len])
        s["positions"] = torch.from_numpy((np.stack([i // 64, i % 64 // 8, i % 8], 1) + 30011).astype(np.int32)).to(DEV)
    return s


def _sections(c):
    d = (c["head_dim"] if c["family"] == "gqa" else c["rope"]) // 2
    a, b = d // 4, (d - d // 4) // 2
    return (a, b, d - a - b) if c.get("sections") else (0, 0, 0)


BASE, EPS = 1e6, 1e-6


# ------------------------------------------------------------------------------------------ the framework's calls
def _handle(s):
    """What a user's program keeps between steps: the layout, the pool, the step's description and a workspace."""
    from position_free_kv_amd import abi, step
    c = s["case"]
    if "own" in s:
        return s["own"]
    kind = dict(num_kv_heads=c["kv_heads"], head_dim=c["head_dim"]) if c["family"] == "gqa" else dict(latent_dim=c["latent"], rope_dim=c["rope"])
    lay = abi.make_layout(abi.GQA if c["family"] == "gqa" else abi.MLA, abi.BF16 if c["dtype"] == "bf16" else abi.F32, c["layers"],
                          rope_base=BASE, page_size=c["page"], mrope_section=_sections(c), **kind)
    pool = abi.make_pool(s["k"], s["v"], s["k"].shape[1])
    if c["op"] == "pages":
        desc, size = None, step.copy_pages_workspace_bytes(c["pages"])
    else:
        prefixes = [dict(block_table=s["prefix_table"], num_tokens=c["prefix"])] if c["op"] == "attend" else []
        desc = step.Step(num_q_heads=c["heads"], block_tables=s["tables"], slot0=s["slot0"], num_tokens=s["own_len"], num_queries=s["q_len"],
                         prefix=0 if prefixes else -1, prefixes=prefixes, position0=s.get("start", 0), positions=s.get("positions"),
                         flags=step.APPEND if c["op"] == "append" else step.ATTEND)
        size = step.workspace_bytes(lay, desc)
    s["own"] = (step, lay, pool, desc, torch.empty(size, dtype=torch.uint8, device=DEV))
    return s["own"]


def _own_run(s):
    c = s["case"]
    step, lay, pool, desc, ws = _handle(s)
    if c["op"] == "pages":
        if c["kind"] == "compact":
            table = s["table"].copy()
            live = step.compact_pages(lay, pool, [table], ws)
            return {"k": s["k"], "v": s["v"], "table": table, "live": live}
        step.copy_pages(lay, pool, s["src"], s["dst"], ws)
        return {"k": s["k"], "v": s["v"]}
    plan = step.upload(lay, desc, pool, ws)  # once a step, for all layers
    if c["op"] == "attend":
        for layer in range(c["layers"]):
            step.attend(plan, layer, s["q"][layer], s["out"][layer], s["scale"], lse=s["lse"][layer])
        return {"out": s["out"], "lse": s["lse"]}
    f, nq = _widths(c)[3], s["q_out"].shape[2]
    for layer in range(c["layers"]):
        rows = s["rows"][layer]
        step.append(plan, layer, q=rows[:, :nq], k=rows[:, nq:nq + f], v=rows[:, nq + f:] if c["family"] == "gqa" else None,
                    q_out=s["q_out"][layer], q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS)
    return {"q": s["q_out"], "k": s["k"], "v": s["v"]}


# ------------------------------------------------------------------------------------------ the plain forms
def _slots(table, first, tokens, page):
    """Pool slots of tokens `tokens` (any shape) of the table rows beside them."""
    at = first + tokens
    return torch.gather(table, -1, (at // page).clamp(max=table.shape[-1] - 1)) * page + at % page


def _plain_pages(s):
    c, k, v = s["case"], s["k"], s["v"]
    more = {}
    if c["kind"] == "compact":
        table = s["table_dev"]
        used = torch.zeros(c["pages"], dtype=torch.bool, device=DEV)
        used[table] = True
        live = table.numel()
        src = torch.nonzero(used[live:])[:, 0] + live
        dst = torch.nonzero(~used[:live])[:, 0]
        to = torch.arange(c["pages"], device=DEV)
        to[src] = dst
        more = {"table": to[table].to(torch.int32), "live": live}
    else:
        src, dst = s["src_dev"], s["dst_dev"]
    k[:, dst] = k[:, src]
    if v is not None:
        v[:, dst] = v[:, src]
    return {"k": k, "v": v, **more}


def _plain_append(s):
    c = s["case"]
    hkv, dk, dv, f = _widths(c)
    heads, layers, n = c["heads"], c["layers"], s["rows"].shape[1]
    mla = c["family"] == "mla"
    rows = s["rows"].float()
    q = rows[..., :heads * dk].reshape(layers, n, heads, dk)
    k = rows[..., heads * dk:heads * dk + f].reshape(layers, n, hkv, dk)

    def norm(x, w):
        return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.float()

    if s["q_weight"] is not None:
        q = norm(q, s["q_weight"])
    if s["k_weight"] is not None:
        k = torch.cat([norm(k[..., :dv], s["k_weight"]), k[..., dv:]], -1) if mla else norm(k, s["k_weight"])
    d = c["rope"] if mla else dk
    place = (s["own_len_dev"] - s["q_len_dev"])[s["request_dev"]] + s["index_dev"]
    if s["positions"] is None:
        at = (s["start_dev"][s["request_dev"]] + place)[:, None].expand(n, d // 2)
    else:
        a, b, e = _sections(c)
        which = torch.arange(3, device=DEV).repeat_interleave(torch.tensor([a, b, e], device=DEV), output_size=d // 2)
        at = s["positions"].long()[:, which]
    theta = BASE ** (-2.0 * torch.arange(d // 2, device=DEV, dtype=torch.float64) / d)
    angle = at.double() * theta
    cos, sin = angle.cos().float()[None, :, None], angle.sin().float()[None, :, None]

    def rotate(x):
        a, b = x[..., -d:-d // 2], x[..., -d // 2:]
        return torch.cat([x[..., :-d], a * cos - b * sin, a * sin + b * cos], -1)

    s["q_out"].copy_(rotate(q).reshape(layers, n, heads * dk))
    slots = _slots(s["tables_dev"][s["request_dev"]], s["slot0"], place[:, None], c["page"])[:, 0]
    s["k"].view(layers, -1, f)[:, slots] = rotate(k).reshape(layers, n, f).to(s["k"].dtype)
    if not mla:
        s["v"].view(layers, -1, f)[:, slots] = s["rows"][..., heads * dk + f:]
    return {"q": s["q_out"], "k": s["k"], "v": s["v"]}


def _plain_attend(s):
    c = s["case"]
    hkv, dk, dv, f = _widths(c)
    g, layers, n, r = c["heads"] // hkv, c["layers"], s["q"].shape[1], c["requests"]
    req, idx = s["request_dev"], s["index_dev"]
    to, tq, tp = int(s["own_len"].max()), int(s["q_len"].max()), c["prefix"]
    kr = s["k"].view(layers, -1, f)
    vr = kr if s["v"] is None else s["v"].view(layers, -1, f)
    q = (s["q"].float() * s["scale"]).view(layers, n, hkv, g, dk)
    # the shared prefix: every query against the same rows
    shared = _slots(s["prefix_table_dev"], 0, torch.arange(tp, device=DEV), c["page"])
    kp = kr[:, shared].float().view(layers, tp, hkv, dk).permute(0, 2, 3, 1).contiguous()
    qp = q.permute(0, 2, 1, 3, 4).reshape(layers, hkv, n * g, dk)
    sp = torch.matmul(qp, kp).view(layers, hkv, n, g, tp)
    # each request's own rows, padded to the longest
    t = torch.arange(to, device=DEV)[None].expand(r, to)
    at = _slots(s["tables_dev"], s["slot0"], t, c["page"])
    ko = kr[:, at].float().view(layers, r, to, hkv, dk).permute(0, 1, 3, 4, 2).contiguous()
    qo = torch.zeros(layers, r, hkv, tq, g, dk, device=DEV)
    qo[:, req, :, idx] = q.permute(1, 0, 2, 3, 4)
    so = torch.matmul(qo.view(layers, r, hkv, tq * g, dk), ko).view(layers, r, hkv, tq, g, to)
    so = so[:, req, :, idx].permute(1, 2, 0, 3, 4)
    last = (s["own_len_dev"] - s["q_len_dev"])[req] + idx
    hidden = torch.arange(to, device=DEV)[None] > last[:, None]
    so = so.masked_fill(hidden[None, None, :, None], float("-inf"))
    m = torch.maximum(sp.amax(-1), so.amax(-1))[..., None]
    sp, so = torch.exp(sp - m), torch.exp(so - m)
    total = sp.sum(-1, keepdim=True) + so.sum(-1, keepdim=True)
    vp = vr[:, shared].view(layers, tp, hkv, -1)[..., :dv].float().permute(0, 2, 1, 3).contiguous()
    o = torch.matmul(sp.view(layers, hkv, n * g, tp), vp).view(layers, hkv, n, g, dv)
    vo = vr[:, at].view(layers, r, to, hkv, -1)[..., :dv].float().permute(0, 1, 3, 2, 4).contiguous()
    po = torch.zeros(layers, r, hkv, tq, g, to, device=DEV)
    po[:, req, :, idx] = so.permute(2, 0, 1, 3, 4)
    oo = torch.matmul(po.view(layers, r, hkv, tq * g, to), vo).view(layers, r, hkv, tq, g, dv)
    o = (o + oo[:, req, :, idx].permute(1, 2, 0, 3, 4)) / total
    s["out"].copy_(o.permute(0, 2, 1, 3, 4).reshape(layers, n, hkv * g, dv))
    s["lse"].copy_((m + total.log())[..., 0].permute(0, 2, 1, 3).reshape(layers, n, hkv * g))
    return {"out": s["out"], "lse": s["lse"]}


def run(state):
    if own:
        return _own_run(state)
    return {"pages": _plain_pages, "append": _plain_append, "attend": _plain_attend}[state["case"]["op"]](state)


# ------------------------------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    hkv, dk, dv, f = _widths(c)
    page, layers, heads = c["page"], c["layers"], c["heads"]
    if c["op"] == "pages":
        take, more = np.arange(c["pages"]), {}
        if c["kind"] == "compact":
            table, live = s["table"], len(s["table"])
            holes = sorted(set(range(live)) - set(table.tolist()))
            beyond = sorted(x for x in table.tolist() if x >= live)
            new = dict(zip(beyond, holes))
            for a, b in new.items():
                take[b] = a
            more = {"table": np.array([new.get(x, x) for x in table.tolist()], np.int32), "live": live}
        else:
            for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
                take[b] = a
        take = torch.from_numpy(take).to(DEV)
        return {"k": s["k"].index_select(1, take), "v": None if s["v"] is None else s["v"].index_select(1, take), **more}

    first = np.concatenate([[0], np.cumsum(s["q_len"])])

    def where(table, slot0, tokens):
        at = slot0 + np.asarray(tokens)
        return torch.from_numpy(table[at // page].astype(np.int64) * page + at % page).to(DEV)

    if c["op"] == "append":
        q_out, k_out = s["q_out"].double(), s["k"].double().view(layers, -1, f)
        v_out = None if s["v"] is None else s["v"].double().view(layers, -1, f)
        d = c["rope"] if c["family"] == "mla" else dk
        theta = np.exp(np.arange(d // 2) * (-2.0 / d) * math.log(BASE))
        part = np.repeat(np.arange(3), _sections(c))
        for i in range(c["requests"]):
            m, have = int(s["q_len"][i]), int(s["own_len"][i])
            rows = s["rows"][:, first[i]:first[i] + m].double()
            if s["positions"] is not None:
                pos = s["positions"][first[i]:first[i] + m].cpu().numpy().astype(np.float64)[:, part]
            else:
                pos = (int(s["start"][i]) + have - m + np.arange(m, dtype=np.float64))[:, None]
            turn = torch.from_numpy(np.exp(1j * (pos * theta))).to(DEV)[None, :, None]

            def turned(x):  # the last d of a head's columns, as complex numbers
                z = torch.complex(x[..., -d:-d + d // 2], x[..., -d + d // 2:]) * turn
                return torch.cat([x[..., :x.shape[-1] - d], z.real, z.imag], -1)

            def normed(x, w):
                return x / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + EPS) * w.double()

            qi = rows[..., :heads * dk].reshape(layers, m, heads, dk)
            ki = rows[..., heads * dk:heads * dk + f].reshape(layers, m, hkv, dk)
            qi = qi if s["q_weight"] is None else normed(qi, s["q_weight"])
            if s["k_weight"] is not None:
                w = s["k_weight"]
                ki = torch.cat([normed(ki[..., :w.numel()], w), ki[..., w.numel():]], -1)
            to = where(s["tables"][i], s["slot0"], np.arange(have - m, have))
            q_out[:, first[i]:first[i] + m] = turned(qi).reshape(layers, m, -1)
            k_out[:, to] = turned(ki).reshape(layers, m, f)
            if v_out is not None:
                v_out[:, to] = rows[..., heads * dk + f:]
        return {"q": q_out, "k": k_out.view(s["k"].shape), "v": None if v_out is None else v_out.view(s["v"].shape)}

    out = torch.empty(s["out"].shape, dtype=torch.float64, device=DEV)
    lse = torch.empty(s["lse"].shape, dtype=torch.float64, device=DEV)
    g = heads // hkv
    shared = where(s["prefix_table"], 0, np.arange(c["prefix"]))
    for layer in range(layers):
        keys = s["k"][layer].view(-1, f)
        values = keys if s["v"] is None else s["v"][layer].view(-1, f)
        for i in range(c["requests"]):
            m, have = int(s["q_len"][i]), int(s["own_len"][i])
            at = torch.cat([shared, where(s["tables"][i], s["slot0"], np.arange(have))])
            seen = torch.arange(at.numel(), device=DEV)[None] <= (c["prefix"] + have - m + torch.arange(m, device=DEV))[:, None]
            qi = s["q"][layer, first[i]:first[i] + m].double()
            for h in range(hkv):
                kh = keys[at, h * dk:(h + 1) * dk].double().t().contiguous()
                vh = values[at, h * dk:h * dk + dv].double()
                z = (qi[:, h * g:(h + 1) * g].reshape(m * g, dk) @ kh * s["scale"]).view(m, g, -1)
                z = z.masked_fill(~seen[:, None], -math.inf)
                total = torch.logsumexp(z, -1)
                w = torch.exp(z - total[..., None])
                out[layer, first[i]:first[i] + m, h * g:(h + 1) * g] = (w.view(m * g, -1) @ vh).view(m, g, dv)
                lse[layer, first[i]:first[i] + m, h * g:(h + 1) * g] = total
    return {"out": out, "lse": lse}
