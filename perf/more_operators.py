"""More serving operators on the paged KV pool: what is measured, and their plain forms.

  diff    differential attention over the pool: the difference of two softmax maps with learned weights, normed per head
  weigh   attention weight that the cached tokens receive from a step's queries, accumulated beside the pool
  evict   the tokens of least accumulated weight leave the cache: selection per layer and KV head, survivors moved
          together in order (and, where asked for, their keys turned to their new positions)

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
    vl7b, deque, small = _gqa(28, 4, 128), _gqa(32, 8, 128), _gqa(16, 4, 64)
    return [
        # a handful of chat turns on one cached image: latency
        dict(vl7b, name="diff_few", op="diff", layers=2, page=16, requests=4, prefix=1000, own_lo=1, own_hi=64, q_lo=1, q_hi=1),
        # a serving batch on one video of eight 1024-token segments, one token each
        dict(deque, name="diff_decode", op="diff", layers=4, page=16, requests=64, prefix=8192, own_lo=17, own_hi=1500, q_lo=1, q_hi=1),
        # narrow heads over a long shared context
        dict(small, name="diff_long", op="diff", layers=2, page=16, requests=12, prefix=65536, own_lo=1, own_hi=4096, q_lo=1, q_hi=1),
        # questions of several hundred tokens on the shared video, all at once
        dict(vl7b, name="diff_extend", op="diff", layers=1, page=16, requests=8, prefix=8192, own_lo=0, own_hi=700, q_lo=33, q_hi=731),
        # the single-precision layout, a few tokens a request (speculated ones)
        dict(_gqa(8, 2, 64), name="diff_f32", dtype="f32", op="diff", layers=1, page=16, requests=5, prefix=300, own_lo=0, own_hi=40, q_lo=1, q_hi=9),
        # the same chat turns: what their one token each adds to the weights
        dict(vl7b, name="weigh_few", op="weigh", layers=2, page=16, requests=4, prefix=1000, own_lo=1, own_hi=64, q_lo=1, q_hi=1, decay=1.0),
        # the serving batch: every step of a decode loop that evicts by accumulated weight makes this call
        dict(deque, name="weigh_decode", op="weigh", layers=4, page=16, requests=64, prefix=8192, own_lo=17, own_hi=1500, q_lo=1, q_hi=1, decay=1.0),
        # questions as observation windows: all of their tokens weigh the shared video, the weights before them fade
        dict(vl7b, name="weigh_window", op="weigh", layers=1, page=16, requests=8, prefix=8192, own_lo=0, own_hi=700, q_lo=33, q_hi=731, decay=0.5),
        # latent rows: 16 heads weigh one row a token
        dict(_mla(16), name="weigh_mla", op="weigh", layers=4, page=16, requests=32, prefix=4096, own_lo=1, own_hi=1024, q_lo=1, q_hi=1, decay=1.0),
        # one conversation has outgrown its budget: all 28 layers
        dict(vl7b, name="evict_turn", op="evict", layers=28, page=16, seqs=1, n_lo=1500, n_hi=1500, keep=0.75, first=4, last=128, together=1, reanchor=False),
        # a deque's batch, to half its tokens
        dict(deque, name="evict_batch", op="evict", layers=12, page=16, seqs=16, n_lo=1000, n_hi=8000, keep=0.5, first=4, last=64, together=1, reanchor=False),
        # latent rows of long documents, survivors at consecutive positions again
        dict(_mla(16), name="evict_mla", op="evict", layers=27, page=16, seqs=8, n_lo=2048, n_hi=6000, keep=0.5, first=16, last=256, together=1, reanchor=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["diff", "diff", "diff", "weigh", "weigh", "weigh", "evict", "evict"])
    heads = [_gqa(28, 4, 128), _gqa(32, 8, 128), _gqa(32, 32, 128), _gqa(16, 2, 128), _gqa(16, 4, 64), _gqa(12, 12, 64),
             dict(_gqa(8, 2, 64), dtype="f32")]
    shape = rng.choice(heads if op == "diff" else heads + [_mla(16), _mla(32)])
    page = rng.choice([8, 16, 16, 32, 64])
    small, mla = shape["dtype"] == "f32", shape["family"] == "mla"
    if op == "evict":
        hkv = 1 if mla else shape["kv_heads"]
        for _ in range(1000):
            lo = _log(rng, 1, 8000)
            c = dict(shape, op=op, layers=rng.randint(1, 28), page=page, seqs=_log(rng, 1, 32), n_lo=lo, n_hi=rng.choice([lo, min(8000, 3 * lo)]),
                     keep=round(rng.uniform(0.1, 0.95), 2), first=rng.choice([0, 1, 4, 16]), last=rng.choice([0, 1, 64, 256]),
                     together=rng.choice([x for x in (1, 1, 2, hkv) if hkv % x == 0]), reanchor=rng.random() < 0.4)
            if work(c)["bytes"] <= 0.9 * work(listed()[10])["bytes"]:
                return c
    decay = dict(decay=rng.choice([1.0, 1.0, 0.9, 0.0])) if op == "weigh" else {}
    most = work(listed()[3 if op == "diff" else 7])
    for _ in range(1000):
        c = dict(shape, op=op, layers=rng.randint(1, 2), page=page, requests=_log(rng, 1, 20 if small else 100),
                 prefix=_log(rng, 16, 600 if small else 65536), own_lo=rng.choice([0, 1, 16]), own_hi=_log(rng, 17, 100 if small else 4096), q_lo=1,
                 q_hi=1 if rng.random() < 0.6 else _log(rng, 2, 9 if small else 700), **decay)
        w = work(c)
        if w["flops"] <= most["flops"] and w["bytes"] <= 1.2e9 and c["layers"] * sum(_lengths(c)[1]) * c["heads"] * (c["prefix"] + max(_lengths(c)[0])) < 1.2e9:
            return c
    return dict(shape, op=op, layers=1, page=page, requests=_log(rng, 1, 9), prefix=_log(rng, 16, 600), own_lo=0, own_hi=_log(rng, 17, 60), q_lo=1, q_hi=1,
                **decay)


def _lengths(c):
    """(own tokens, query tokens) of every request; a request's last query tokens are among its own."""
    r = np.arange(c["requests"], dtype=np.int64)
    q = c["q_lo"] + (r * 2654435761 % (1 << 32) >> 7) % (c["q_hi"] - c["q_lo"] + 1)
    old = c["own_lo"] + (r * 40503 + 977) * 2246822519 % (1 << 32) % (c["own_hi"] - c["own_lo"] + 1)
    return old + q, q


def _evictions(c):
    """(tokens, tokens to keep, of them the first, the last) of every sequence."""
    r = np.arange(c["seqs"], dtype=np.int64)
    n = c["n_lo"] + (r * 2654435761 % (1 << 32) >> 5) % (c["n_hi"] - c["n_lo"] + 1)
    keep = np.maximum((n * c["keep"]).astype(np.int64), 1)
    first = np.minimum(c["first"], keep)
    return n, keep, first, np.minimum(c["last"], keep - first)


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
    if c["op"] == "evict":
        n, keep, first, _ = _evictions(c)
        moved = int((keep - first).sum())
        groups = hkv // c["together"]
        # all scores read, those of the kept written; kept rows behind the first ones read and written
        return {"bytes": c["layers"] * (4 * hkv * int((n + keep).sum()) + 4 * groups * int(keep.sum()) + 2 * moved * f * e * tensors),
                "flops": c["layers"] * moved * hkv * 6 * (c.get("head_dim") or c["rope"]) // 2 if c["reanchor"] else 0}
    own_len, q_len = _lengths(c)
    n = int(q_len.sum())
    pairs = n * c["prefix"] + int((q_len * own_len - q_len * (q_len - 1) // 2).sum())
    rows = c["prefix"] + int(own_len.sum())
    if c["op"] == "weigh":  # keys, queries, their statistics; weights added
        return {"bytes": c["layers"] * (rows * f * e + n * c["heads"] * (dk * e + 4) + rows * hkv * (8 if c["decay"] else 4)),
                "flops": 2 * c["layers"] * pairs * c["heads"] * dk}
    # a query head's scores of its key head, and its weights with the values of two heads
    return {"bytes": c["layers"] * (rows * f * e * 2 + n * c["heads"] * ((dk + dv) * e + 4)), "flops": 2 * c["layers"] * pairs * c["heads"] * 3 * dk}


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


def _lambda_init(layer):
    return 0.8 - 0.6 * math.exp(-0.3 * layer)


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    host = np.random.default_rng([seed, 78])
    hkv, dk, dv, f = _widths(c)
    t, p = TYPES[c["dtype"]], c["page"]
    s = {"case": c}
    if c["op"] == "evict":
        n, keep, first, last = _evictions(c)
        slot0 = (7 * np.arange(c["seqs"]) + 3) % p  # sequences begin inside a page, behind what they share with others
        need = (slot0 + n + p - 1) // p
        pages = int(need.sum()) + 5
        order = host.permutation(pages).astype(np.int32)
        s["k"], s["v"] = _pool(gen, c, pages, f)
        s["tables"] = np.zeros((c["seqs"], int(need.max())), np.int32)
        s["tables"][np.arange(s["tables"].shape[1])[None] < need[:, None]] = order[:int(need.sum())]
        # weights accumulated over many queries: a few tokens have received most
        s["scores"] = torch.exp(2.0 * _normal(gen, c["layers"], pages, hkv, p))
        s["n"], s["keep"], s["first"], s["last"], s["slot0"] = n, keep, first, last, slot0
        s["kept"] = torch.empty(c["layers"], hkv // c["together"], int(keep.sum()), device=DEV, dtype=torch.int32)
        for name in ("tables", "n", "keep", "first", "last", "slot0"):
            s[name + "_dev"] = torch.from_numpy(s[name].astype(np.int64)).to(DEV)
        return s

    own_len, q_len = _lengths(c)
    n, r = int(q_len.sum()), c["requests"]
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
    s["scale"] = 1.0 / math.sqrt(192.0 if c["family"] == "mla" else dk)
    s["q"] = (_normal(gen, c["layers"], n, heads, dk) * 1.5).to(t)
    s["lse"] = torch.empty(c["layers"], n, heads, device=DEV, dtype=torch.float32)
    if c["op"] == "weigh":
        # what the attention before it left: the logarithm of every query's sum; and the weights of earlier steps
        for layer in range(c["layers"]):
            sp, so = _scores(s, layer)
            flat = torch.logaddexp(torch.logsumexp(sp, -1), torch.logsumexp(_of_tokens(s, so), -1))
            s["lse"][layer] = flat.permute(1, 0, 2).reshape(n, heads)
        s["scores"] = torch.exp(2.0 * _normal(gen, c["layers"], pages, hkv, p))
        return s
    s["out"] = torch.empty(c["layers"], n, heads // 2, 2 * dv, device=DEV, dtype=t)
    s["lambdas"] = 0.1 * _normal(gen, c["layers"], 4, dk)  # lambda_q1, lambda_k1, lambda_q2, lambda_k2 of each layer
    s["norm_weight"] = (1.0 + 0.2 * _normal(gen, c["layers"], 2 * dv)).to(t)
    return s


BASE, EPS = 1e6, 1e-5


# ------------------------------------------------------------------------------------------ the framework's calls
def _handle(s):
    """What a user's program keeps between steps: the layout, the pool, the description and a workspace."""
    from position_free_kv_amd import abi, step
    c = s["case"]
    if "own" in s:
        return s["own"]
    kind = dict(num_kv_heads=c["kv_heads"], head_dim=c["head_dim"]) if c["family"] == "gqa" else dict(latent_dim=c["latent"], rope_dim=c["rope"])
    lay = abi.make_layout(abi.GQA if c["family"] == "gqa" else abi.MLA, abi.BF16 if c["dtype"] == "bf16" else abi.F32, c["layers"],
                          rope_base=BASE, page_size=c["page"], **kind)
    pool = abi.make_pool(s["k"], s["v"], s["k"].shape[1])
    if c["op"] == "evict":
        desc = step.Eviction(block_tables=s["tables"], slot0=s["slot0"], num_tokens=s["n"], keep=s["keep"], first=s["first"], last=s["last"],
                             heads_together=c["together"], flags=step.REANCHOR if c["reanchor"] else 0)
        size = step.evict_workspace_bytes(lay, desc)
    else:
        desc = step.Step(num_q_heads=c["heads"], block_tables=s["tables"], slot0=s["slot0"], num_tokens=s["own_len"], num_queries=s["q_len"],
                         prefix=0, prefixes=[dict(block_table=s["prefix_table"], num_tokens=c["prefix"])],
                         flags=step.WEIGH if c["op"] == "weigh" else step.ATTEND | step.DIFFERENTIAL)
        size = step.workspace_bytes(lay, desc)
    s["own"] = (step, lay, pool, desc, torch.empty(size, dtype=torch.uint8, device=DEV))
    return s["own"]


def _own_run(s):
    c = s["case"]
    step, lay, pool, desc, ws = _handle(s)
    if c["op"] == "evict":
        step.evict(lay, pool, desc, s["scores"], ws, kept=s["kept"])
        return {"k": s["k"], "v": s["v"], "scores": s["scores"], "kept": s["kept"]}
    plan = step.upload(lay, desc, pool, ws)  # once a step, for all layers
    for layer in range(c["layers"]):
        if c["op"] == "weigh":
            step.weigh(plan, layer, s["q"][layer], s["lse"][layer], s["scores"][layer], s["scale"], decay=c["decay"])
        else:
            step.attend_diff(plan, layer, s["q"][layer], s["out"][layer], s["scale"], lambdas=s["lambdas"][layer], lambda_init=_lambda_init(layer),
                             norm_weight=s["norm_weight"][layer], eps=EPS, lse=s["lse"][layer])
    return {"scores": s["scores"]} if c["op"] == "weigh" else {"out": s["out"], "lse": s["lse"]}


# ------------------------------------------------------------------------------------------ the plain forms
def _slots(table, first, tokens, page):
    """Pool slots of tokens `tokens` (any shape) of the table rows beside them."""
    at = first + tokens
    return torch.gather(table, -1, (at // page).clamp(max=table.shape[-1] - 1)) * page + at % page


def _by_key_head(s, x):
    """Query rows [n][heads][d] as [KV heads][n][G][d]: differential heads 2 i and 2 i + 1 of a pair of KV heads read one each."""
    c = s["case"]
    hkv, n = _widths(c)[0], x.shape[0]
    if c["op"] == "diff":
        return x.view(n, hkv // 2, -1, 2, x.shape[-1]).permute(1, 3, 0, 2, 4).reshape(hkv, n, -1, x.shape[-1])
    return x.view(n, hkv, -1, x.shape[-1]).permute(1, 0, 2, 3)


def _own_slots(s):
    to, r = int(s["own_len"].max()), s["case"]["requests"]
    t = torch.arange(to, device=DEV)[None].expand(r, to)
    return t, _slots(s["tables_dev"], s["slot0"], t, s["case"]["page"])


def _scores(s, layer):
    """Scaled scores of a layer: [KV heads][n][G][prefix], and [requests][KV heads][q][G][own], padded and -inf where unseen."""
    c = s["case"]
    hkv, dk, _, f = _widths(c)
    r, tp = c["requests"], c["prefix"]
    kr = s["k"][layer].view(-1, f)
    q = _by_key_head(s, s["q"][layer].float()) * s["scale"]
    n, g = q.shape[1:3]
    shared = _slots(s["prefix_table_dev"], 0, torch.arange(tp, device=DEV), c["page"])
    kp = kr[shared].float().view(tp, hkv, dk).permute(1, 2, 0).contiguous()
    sp = torch.matmul(q.reshape(hkv, n * g, dk), kp).view(hkv, n, g, tp)
    t, at = _own_slots(s)
    to, tq = t.shape[1], int(s["q_len"].max())
    ko = kr[at].float().view(r, to, hkv, dk).permute(0, 2, 3, 1).contiguous()
    qo = torch.zeros(r, hkv, tq, g, dk, device=DEV)
    qo[s["request_dev"], :, s["index_dev"]] = q.permute(1, 0, 2, 3)
    so = torch.matmul(qo.view(r, hkv, tq * g, dk), ko).view(r, hkv, tq, g, to)
    i = torch.arange(tq, device=DEV)[None]
    last = torch.where(i < s["q_len_dev"][:, None], (s["own_len_dev"] - s["q_len_dev"])[:, None] + i, -1)
    return sp, so.masked_fill(t[:, None, None, None] > last[:, None, :, None, None], float("-inf"))


def _of_tokens(s, x):
    """[requests][KV heads][q][...] as [KV heads][n][...]."""
    return x[s["request_dev"], :, s["index_dev"]].transpose(0, 1)


def _plain_diff(s):
    c = s["case"]
    hkv, dk, dv, f = _widths(c)
    tp, r = c["prefix"], c["requests"]
    shared = _slots(s["prefix_table_dev"], 0, torch.arange(tp, device=DEV), c["page"])
    _, at = _own_slots(s)
    for layer in range(c["layers"]):
        sp, so = _scores(s, layer)
        n, g = sp.shape[1:3]
        tq, to = so.shape[2], so.shape[4]
        m = torch.maximum(sp.amax(-1), _of_tokens(s, so).amax(-1))[..., None]
        padded = torch.zeros(r, hkv, tq, g, 1, device=DEV)
        padded[s["request_dev"], :, s["index_dev"]] = m.transpose(0, 1)
        sp, so = torch.exp(sp - m), torch.exp(so - padded)
        total = sp.sum(-1, keepdim=True) + _of_tokens(s, so).sum(-1, keepdim=True)
        vr = s["v"][layer].view(-1, f)
        vp = vr[shared].float().view(tp, hkv // 2, 2 * dv).permute(1, 0, 2)[:, None].expand(-1, 2, -1, -1).reshape(hkv, tp, 2 * dv)
        vo = vr[at].float().view(r, to, hkv // 2, 2 * dv).permute(0, 2, 1, 3)[:, :, None].expand(-1, -1, 2, -1, -1).reshape(r, hkv, to, 2 * dv)
        o = torch.matmul(sp.view(hkv, n * g, tp), vp).view(hkv, n, g, 2 * dv)
        o = (o + _of_tokens(s, torch.matmul(so.view(r, hkv, tq * g, to), vo).view(r, hkv, tq, g, 2 * dv))) / total
        o = o.view(hkv // 2, 2, n, g, 2 * dv)
        q1, k1, q2, k2 = s["lambdas"][layer]
        lam = torch.exp((q1 * k1).sum()) - torch.exp((q2 * k2).sum()) + _lambda_init(layer)
        x = o[:, 0] - lam * o[:, 1]
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * s["norm_weight"][layer].float() * (1.0 - _lambda_init(layer))
        s["out"][layer] = x.permute(1, 0, 2, 3).reshape(n, -1, 2 * dv)
        z = (m + total.log())[..., 0].view(hkv // 2, 2, n, g)
        s["lse"][layer] = z.permute(2, 0, 3, 1).reshape(n, -1)
    return {"out": s["out"], "lse": s["lse"]}


def _plain_weigh(s):
    c = s["case"]
    hkv, p, r = _widths(c)[0], c["page"], c["requests"]
    shared = _slots(s["prefix_table_dev"], 0, torch.arange(c["prefix"], device=DEV), p)
    t, at = _own_slots(s)
    real = t < s["own_len_dev"][:, None]
    for layer in range(c["layers"]):
        sp, so = _scores(s, layer)
        n, g = sp.shape[1:3]
        z = s["lse"][layer].view(n, hkv, g).transpose(0, 1)[..., None]
        padded = torch.zeros(r, hkv, so.shape[2], g, 1, device=DEV)
        padded[s["request_dev"], :, s["index_dev"]] = z.transpose(0, 1)
        wp = torch.exp(sp - z).sum((1, 2)).t()  # [prefix][KV heads]
        wo = torch.exp(so - padded).sum((2, 3)).transpose(1, 2)[real]  # [own tokens][KV heads]
        slots = torch.cat([shared, at[real]])
        page, place = slots // p, slots % p
        before = s["scores"][layer]
        before[page, :, place] = before[page, :, place] * c["decay"] + torch.cat([wp, wo])
    return {"scores": s["scores"]}


def _plain_evict(s):
    c = s["case"]
    hkv, dk, _, f = _widths(c)
    p, layers, tog = c["page"], c["layers"], c["together"]
    groups, most = hkv // tog, int(s["n"].max())
    t = torch.arange(most, device=DEV)[None].expand(c["seqs"], most)
    slots = _slots(s["tables_dev"], s["slot0_dev"][:, None], t, p)
    each = s["scores"][:, slots // p, :, slots % p].permute(2, 3, 0, 1).view(layers, groups, tog, c["seqs"], most)
    rank = each[:, :, 0]
    for h in range(1, tog):
        rank = rank + each[:, :, h]
    n, keep = s["n_dev"][:, None], s["keep_dev"][:, None]
    rank = rank.masked_fill((t < s["first_dev"][:, None]) | ((t >= n - s["last_dev"][:, None]) & (t < n)), float("inf"))
    rank = rank.masked_fill(t >= n, float("-inf"))
    order = torch.sort(rank, dim=-1, descending=True, stable=True).indices
    stays = torch.zeros_like(rank, dtype=torch.bool).scatter_(-1, order, (t < keep).expand(layers, groups, -1, -1))
    layer, group, seq, old = stays.nonzero(as_tuple=True)
    new = (torch.cumsum(stays, -1) - 1)[layer, group, seq, old]
    src, dst = slots[seq, old], slots[seq, new]
    s["kept"].copy_(old.view(layers, groups, -1))
    k = s["k"].view(layers, -1, groups, tog * dk)
    rows = k[layer, src, group]
    if c["reanchor"]:
        d = c["rope"] if c["family"] == "mla" else dk
        theta = BASE ** (-2.0 * torch.arange(d // 2, device=DEV, dtype=torch.float64) / d)
        angle = (new - old).double()[:, None] * theta
        cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
        x = rows.view(-1, tog, dk).float()
        a, b = x[..., -d:-d // 2], x[..., -d // 2:]
        rows = torch.cat([x[..., :-d], a * cos - b * sin, a * sin + b * cos], -1).to(rows.dtype).view(rows.shape)
    k[layer, dst, group] = rows
    if s["v"] is not None:
        v = s["v"].view(layers, -1, groups, tog * dk)
        v[layer, dst, group] = v[layer, src, group]
    w = s["scores"].view(layers, -1, groups, tog, p)
    w[layer, dst // p, group, :, dst % p] = w[layer, src // p, group, :, src % p]
    return {"k": s["k"], "v": s["v"], "scores": s["scores"], "kept": s["kept"]}


def run(state):
    if own:
        return _own_run(state)
    return {"diff": _plain_diff, "weigh": _plain_weigh, "evict": _plain_evict}[state["case"]["op"]](state)


# ------------------------------------------------------------------------------------------ in 64 bits
def _exact_evict(s):
    c = s["case"]
    hkv, dk, _, f = _widths(c)
    p, tog, layers = c["page"], c["together"], c["layers"]
    scores = s["scores"].cpu().numpy()
    new_scores = scores.copy()
    d = c["rope"] if c["family"] == "mla" else dk
    turn = c["reanchor"]
    k_out = s["k"].double() if turn else s["k"].clone()
    v_out = None if s["v"] is None else s["v"].clone()
    kept = np.zeros((layers, hkv // tog, int(s["keep"].sum())), np.int32)
    theta = torch.from_numpy(np.exp(np.arange(d // 2) * (-2.0 / d) * math.log(BASE))).to(DEV)
    done = 0
    for i in range(c["seqs"]):
        n, keep, first, last = (int(s[x][i]) for x in ("n", "keep", "first", "last"))
        at = int(s["slot0"][i]) + np.arange(n)
        page, place = s["tables"][i][at // p].astype(np.int64), at % p
        slot = page * p + place
        for layer in range(layers):
            for h in range(0, hkv, tog):
                w = scores[layer, page, h, place]
                for e in range(h + 1, h + tog):
                    w = w + scores[layer, page, e, place]  # in 32 bits, one head after the other: what the choice goes by
                middle = np.arange(first, n - last)
                order = middle[np.argsort(-w[middle].astype(np.float64), kind="stable")]
                stay = np.sort(np.concatenate([np.arange(first), order[:keep - first - last], np.arange(n - last, n)]))
                kept[layer, h // tog, done:done + keep] = stay
                for e in range(h, h + tog):
                    new_scores[layer, page[:keep], e, place[:keep]] = scores[layer, page[stay], e, place[stay]]
                src, dst = (torch.from_numpy(x).to(DEV) for x in (slot[stay], slot[:keep]))
                cols = slice(h * dk, (h + tog) * dk)
                rows = s["k"][layer].view(-1, f)[src, cols]
                if turn:
                    z = rows.double().view(keep, tog, dk)
                    delta = torch.from_numpy((np.arange(keep) - stay).astype(np.float64)).to(DEV)
                    spin = torch.exp(1j * (delta[:, None] * theta))[:, None]
                    y = torch.complex(z[..., dk - d:dk - d // 2], z[..., dk - d // 2:]) * spin
                    rows = torch.cat([z[..., :dk - d], y.real, y.imag], -1).reshape(keep, -1)
                k_out[layer].view(-1, f)[dst, cols] = rows
                if v_out is not None:
                    v_out[layer].view(-1, f)[dst, cols] = s["v"][layer].view(-1, f)[src, cols]
        done += keep
    return {"k": k_out, "v": v_out, "scores": torch.from_numpy(new_scores).to(DEV), "kept": torch.from_numpy(kept).to(DEV)}


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "evict":
        return _exact_evict(s)
    hkv, dk, dv, f = _widths(c)
    p, layers, heads, diff = c["page"], c["layers"], c["heads"], c["op"] == "diff"
    first = np.concatenate([[0], np.cumsum(s["q_len"])])

    def where(table, slot0, tokens):
        at = slot0 + np.asarray(tokens)
        return torch.from_numpy(table[at // p].astype(np.int64) * p + at % p).to(DEV)

    shared = where(s["prefix_table"], 0, np.arange(c["prefix"]))
    out = torch.empty(s["out"].shape, dtype=torch.float64, device=DEV) if diff else None
    lse = s["lse"].double()
    weights = None if diff else s["scores"].double()
    for layer in range(layers):
        keys = s["k"][layer].view(-1, f)
        values = None if not diff else s["v"][layer].view(-1, f)
        gained = torch.zeros(keys.shape[0], hkv, dtype=torch.float64, device=DEV)
        met = torch.zeros(keys.shape[0], dtype=torch.bool, device=DEV)
        for i in range(c["requests"]):
            m, have = int(s["q_len"][i]), int(s["own_len"][i])
            at = torch.cat([shared, where(s["tables"][i], s["slot0"], np.arange(have))])
            met[at] = True
            unseen = torch.arange(at.numel(), device=DEV)[None] > (c["prefix"] + have - m + torch.arange(m, device=DEV))[:, None]
            rows = slice(int(first[i]), int(first[i]) + m)
            qi = s["q"][layer, rows].double()
            maps = {}
            for h in range(hkv):
                if diff:  # query heads of this key head: every other one of the pair's
                    per = 2 * heads // hkv
                    mine = [h // 2 * per + 2 * j + h % 2 for j in range(per // 2)]
                else:
                    mine = list(range(h * heads // hkv, (h + 1) * heads // hkv))
                kh = keys[at, h * dk:(h + 1) * dk].double().t().contiguous()
                z = (qi[:, mine].reshape(m * len(mine), dk) @ kh * s["scale"]).view(m, len(mine), -1)
                z = z.masked_fill(unseen[:, None], -math.inf)
                if not diff:
                    gained[:, h].index_add_(0, at, torch.exp(z - lse[layer, rows][:, mine, None]).sum((0, 1)))
                    continue
                total = torch.logsumexp(z, -1)
                lse[layer, rows, mine[0]:mine[-1] + 1:2] = total
                w = torch.exp(z - total[..., None]).view(m * len(mine), -1)
                pair = h // 2 * 2 * dv
                maps[h % 2] = (w @ values[at, pair:pair + 2 * dv].double()).view(m, len(mine), 2 * dv)
                if h % 2 == 0:
                    continue
                a = s["lambdas"][layer].double()
                lam = math.exp(float(a[0] @ a[1])) - math.exp(float(a[2] @ a[3])) + _lambda_init(layer)
                x = maps[0] - lam * maps[1]
                x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / (2 * dv) + EPS) * s["norm_weight"][layer].double()
                out[layer, rows, mine[0] // 2:mine[-1] // 2 + 1] = x * (1.0 - _lambda_init(layer))
        if not diff:
            at = torch.nonzero(met)[:, 0]
            w = weights[layer]
            w[at // p, :, at % p] = w[at // p, :, at % p] * c["decay"] + gained[at]
    return {"out": out, "lse": lse} if diff else {"scores": weights}
