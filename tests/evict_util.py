"""Expectations of differential attention, weighing and eviction for the cases of step_util.py."""
from __future__ import annotations

import numpy as np
import torch

from oracle import evict_oracle as eo
from oracle import step_oracle as so
from position_free_kv_amd import abi, step
from tests.step_util import E32, HALF, TYPES


def host(x):
    return x.double().cpu().numpy()


def visible(c):
    """Per request: (rows of its queries, pool rows of the tokens it may see, last seen of each query)."""
    n0, np_ = 0, len(c.prefix_tokens)
    for r, (pre, own, nq, flags) in enumerate(c.requests):
        head = c.rows[pre] if pre >= 0 else np.zeros(0, np.int64)
        at = np.concatenate([head, c.rows[np_ + r]])
        last = np.full(nq, at.size - 1) if flags else np.maximum(head.size + own - nq + np.arange(nq), head.size - 1)
        yield slice(n0, n0 + nq), at, last
        n0 += nq


# ------------------------------------------------------------------------------------------ differential attention
class Params:
    def __init__(self, c, *, lambdas=True, weight=True, norm=True, lambda_init=0.35, out_scale=None, eps=1e-5, seed=1):
        rng = np.random.default_rng(seed)
        self.norm, self.lambda_init, self.eps = norm, lambda_init, eps
        self.out_scale = 1.0 - lambda_init if out_scale is None else out_scale
        self.lambdas = torch.from_numpy((0.3 * rng.standard_normal((4, c.dk))).astype(np.float32)).to(c.device) if lambdas else None
        self.weight = torch.from_numpy((1 + 0.2 * rng.standard_normal(2 * c.dk)).astype(np.float32)).to(TYPES[c.dtype]).to(c.device) if weight else None

    def kwargs(self):
        return dict(lambdas=self.lambdas, lambda_init=self.lambda_init, norm_weight=self.weight, norm=self.norm, eps=self.eps, out_scale=self.out_scale)


def attend_diff(c, p, scale, stream=None, flags=0):
    s = c.step(step.ATTEND | step.DIFFERENTIAL | flags)
    plan = step.upload(c.lay, s, c.pool, c.workspace(s), stream=stream)
    out = torch.full((c.layers, c.n, c.heads * c.dk), 7.0, dtype=TYPES[c.dtype], device=c.device)
    lse = torch.full((c.layers, c.n, c.heads), 7.0, device=c.device)
    for layer in range(c.layers):
        step.attend_diff(plan, layer, c.q[layer], out[layer], scale, lse=lse[layer], stream=stream, **p.kwargs())
    return out, lse


def expect_diff(c, p, layer, scale):
    """(out, tolerance, lse, tolerance) in 64 bits."""
    k, v = (host(x[layer]) for x in c.pools)
    q = host(c.q[layer]).reshape(c.n, c.heads, c.dk)
    d, pairs = c.dk, c.hkv // 2
    per = c.heads // pairs  # query heads of a pair
    maps = np.zeros((2, c.n, c.heads // 2, 2 * d))
    mtol = np.zeros_like(maps)
    lse, ltol = np.zeros((c.n, c.heads)), np.zeros((c.n, c.heads))
    for rows, at, last in visible(c):
        for h in range(c.hkv):
            heads = h // 2 * per + h % 2 + 2 * np.arange(per // 2)
            vals = v[at, h // 2 * 2 * d:(h // 2 + 1) * 2 * d]
            o, z, a, terms = so.attend(q[rows][:, heads], k[at, h * d:(h + 1) * d], vals, scale, last)
            # as in the attention's bounds (step_util.py): scores off by ds, probabilities by 2 ds and their roundings
            ds = (d + 8) * E32 * terms[..., None]
            rel = 2 * ds + (2 * at.size + 128) * E32 + (HALF[abi.BF16] if c.dtype == abi.BF16 else 0.0)
            maps[h % 2][rows, heads[0] // 2:heads[-1] // 2 + 1] = o
            mtol[h % 2][rows, heads[0] // 2:heads[-1] // 2 + 1] = rel * (a + np.abs(o)) + 1e-38
            lse[rows, heads[0]:heads[-1] + 1:2] = z
            seen = np.isfinite(z)
            ltol[rows, heads[0]:heads[-1] + 1:2] = ds[..., 0] + (at.size + 128) * E32 + 8 * E32 * np.where(seen, np.abs(np.where(seen, z, 0)), 0)
    value, terms = eo.lam(None if p.lambdas is None else host(p.lambdas), p.lambda_init)
    x = eo.combine(maps[0], maps[1], value)
    # lambda: dot products of d terms in fp32, two exponentials, sums; then the difference's own roundings
    off = (d + 16) * E32 * terms
    tx = mtol[0] + abs(value) * mtol[1] + off * np.abs(maps[1]) + 4 * E32 * (np.abs(maps[0]) + abs(value) * np.abs(maps[1]))
    w = np.ones(2 * d) if p.weight is None or not p.norm else host(p.weight)
    if p.norm:
        # N = |(x, sqrt(eps))| / sqrt(2 d) moves by at most T = rms(tx) (triangle inequality), so
        # |x'/N' - x/N| <= (tx + |x| T / N) / (N - T); the sum of squares and what follows: 2 d + 16 roundings
        size = np.sqrt((x * x).mean(-1, keepdims=True) + p.eps)
        t = np.sqrt((tx * tx).mean(-1, keepdims=True))
        room = np.where(size > t, size - t, np.nan)
        with np.errstate(invalid="ignore"):
            bound = (tx + np.abs(x) * t / np.where(size > 0, size, 1)) / room
        bound = np.where(np.isnan(bound), np.inf, bound)
        y = eo.head_norm(x, w, p.eps, p.out_scale)
        tol = bound * np.abs(w * p.out_scale) + (2 * d + 16) * E32 * np.abs(y)
        zero = (np.abs(x).max(-1, keepdims=True) == 0) & (tx.max(-1, keepdims=True) <= 1e-30)
        tol = np.where(zero, 0.0, tol)
    else:
        y = x * p.out_scale
        tol = tx * abs(p.out_scale) + 4 * E32 * np.abs(y)
    tol = tol + HALF[c.dtype] * np.abs(y) * (1 + 2 ** -6) + 1e-37
    return y.reshape(c.n, -1), tol.reshape(c.n, -1), lse, ltol


def check_diff(c, p, scale, stream=None, flags=0):
    out, lse = attend_diff(c, p, scale, stream, flags)
    torch.cuda.synchronize()
    for layer in range(c.layers):
        o, tol, z, ltol = expect_diff(c, p, layer, scale)
        got, gz = host(out[layer]), host(lse[layer])
        assert np.isfinite(got).all(), f"layer {layer}: {np.argwhere(~np.isfinite(got))[:4]}"
        assert np.isfinite(tol).mean() > 0.95  # (the bound says something about nearly every element)
        bad = np.abs(got - o) > tol
        assert not bad.any(), (layer, np.argwhere(bad)[:4].tolist(), got[bad][:4], o[bad][:4], tol[bad][:4], int(bad.sum()))
        empty = np.isneginf(z)
        assert (np.isneginf(gz) == empty).all()
        off = np.abs(np.where(empty, 0, gz) - np.where(empty, 0, z))
        assert (off <= ltol).all(), (layer, float((off - ltol).max()))
    return out, lse


# ------------------------------------------------------------------------------------------ weighing
def own_lse(c, layer, scale, diff=False):
    """Statistics of the attention (fp32, as it leaves them) in 64 bits, rounded once."""
    k = host(c.pools[0][layer])
    q = host(c.q[layer]).reshape(c.n, c.heads, c.dk)
    lse = np.full((c.n, c.heads), -np.inf)
    for rows, at, last in visible(c):
        for h in range(c.hkv):
            heads = heads_of(c, h, diff)
            keys = k[at, h * c.dk:(h + 1) * c.dk]
            lse[rows, heads[0]:heads[-1] + 1:2 if diff else 1] = so.attend(q[rows][:, heads], keys, keys[:, :1], scale, last)[1]
    return torch.from_numpy(lse.astype(np.float32)).to(c.device)


def heads_of(c, h, diff):
    per = c.heads // c.hkv
    return h // 2 * 2 * per + h % 2 + 2 * np.arange(per) if diff else h * per + np.arange(per)


def new_scores(c, seed=3):
    gen = torch.Generator().manual_seed(seed)
    return torch.randn(c.layers, c.pages, c.hkv, c.page, generator=gen).exp().to(c.device)


def expect_weigh(c, layer, lse, before, scale, decay, diff=False):
    """(scores, tolerance) [pages, heads, page]."""
    k = host(c.pools[0][layer])
    q = host(c.q[layer]).reshape(c.n, c.heads, c.dk)
    z = host(lse)
    gain, terms, met, count = (np.zeros((c.pages * c.page, c.hkv)) for _ in range(4))
    for rows, at, last in visible(c):
        if rows.stop == rows.start:
            continue
        met[at] = 1
        for h in range(c.hkv):
            heads = heads_of(c, h, diff)
            g, t = eo.weights(q[rows][:, heads], k[at, h * c.dk:(h + 1) * c.dk], z[rows][:, heads], scale, last)
            np.add.at(gain[:, h], at, g)
            np.add.at(terms[:, h], at, t)
            np.add.at(count[:, h], at, (rows.stop - rows.start) * len(heads))
    by_page = lambda x: x.reshape(c.pages, c.page, c.hkv).transpose(0, 2, 1)  # noqa: E731
    gain, terms, met, count = (by_page(x) for x in (gain, terms, met, count))
    old = host(before)
    want = np.where(met > 0, np.where(decay == 0, 0.0, decay * old) + gain, old)
    # a score: dk products in fp32 and a few more roundings of scores and statistics; a weight: that, in its
    # exponent, and the exponential's own; sums of `count` weights; the old score's product and the sum
    tol = (c.dk + 16) * E32 * terms + (count + 16) * E32 * gain + 4 * E32 * np.abs(decay * old) * (met > 0) + 1e-36 * met
    return want, tol


def weigh(c, lse, scores, scale, decay=1.0, diff=False, stream=None, flags=0):
    s = c.step(step.WEIGH | flags | (step.DIFFERENTIAL if diff else 0))
    plan = step.upload(c.lay, s, c.pool, c.workspace(s), stream=stream)
    for layer in range(c.layers):
        step.weigh(plan, layer, c.q[layer], lse[layer], scores[layer], scale, decay, stream=stream)


def check_weigh(c, scale, decay=1.0, diff=False, stream=None, flags=0):
    lse = torch.stack([own_lse(c, layer, scale, diff) for layer in range(c.layers)])
    before = new_scores(c)
    after = before.clone()
    weigh(c, lse, after, scale, decay, diff, stream, flags)
    torch.cuda.synchronize()
    for layer in range(c.layers):
        want, tol = expect_weigh(c, layer, lse[layer], before[layer], scale, decay, diff)
        got = host(after[layer])
        bad = ~(np.abs(got - want) <= tol)
        assert not bad.any(), (layer, np.argwhere(bad)[:4].tolist(), got[bad][:4], want[bad][:4], tol[bad][:4], int(bad.sum()))
    return lse, before, after


# ------------------------------------------------------------------------------------------ eviction
class Cache:
    """A pool, its scores and sequences on pages of their own. seqs: (tokens, keep, first, last)."""

    def __init__(self, *, seqs, family=abi.GQA, dtype=abi.BF16, kv_heads=2, head_dim=64, latent=0, rope=0, layers=2, page=16, together=1, reanchor=False,
                 seed=0, spare=3, pad_layer=0, pad_scores=0, base=1e4, pairing=abi.NEOX, offset=0, ties=False, device="cuda"):
        rng = np.random.default_rng([seed, 6])
        self.seqs, self.page, self.layers, self.together, self.reanchor, self.base, self.dtype = list(seqs), page, layers, together, reanchor, base, dtype
        self.hkv, self.dk = (kv_heads, head_dim) if family == abi.GQA else (1, latent + rope)
        self.band0 = 0 if family == abi.GQA else latent
        self.F, self.pairing, self.device = self.hkv * self.dk, pairing, device
        self.lay = abi.make_layout(family, dtype, layers, num_kv_heads=kv_heads if family == abi.GQA else 0, head_dim=head_dim if family == abi.GQA else 0,
                                   latent_dim=latent, rope_dim=rope, pairing=pairing, rope_base=base, page_size=page)
        self.slot0 = [int(rng.integers(0, page)) for _ in seqs]
        need = [-(-(s + n[0]) // page) if n[0] else 0 for s, n in zip(self.slot0, seqs)]
        self.pages = sum(need) + spare
        order = rng.permutation(self.pages).astype(np.int32)
        cut = np.cumsum([0] + need)
        self.tables = [order[a:b].copy() for a, b in zip(cut[:-1], cut[1:])]
        self.rows = [so.slots(t, s, n[0], page) if n[0] else np.zeros(0, np.int64) for t, s, n in zip(self.tables, self.slot0, seqs)]
        per = self.pages * page * self.F + pad_layer
        tensors = 2 if family == abi.GQA else 1
        self.flat = [torch.from_numpy(rng.standard_normal(layers * per + offset).astype(np.float32)).to(TYPES[dtype]).to(device) for _ in range(tensors)]
        self.pools = [f[offset:].as_strided((layers, self.pages * page, self.F), (per, self.F, 1)) for f in self.flat]
        self.pool = abi.make_pool(self.pools[0], self.pools[-1] if tensors == 2 else None, self.pages, per)
        self.layer_scores = self.pages * page * self.hkv
        values = rng.integers(-3, 4, layers * (self.layer_scores + pad_scores)) if ties else np.exp(2 * rng.standard_normal(layers * (self.layer_scores + pad_scores)))
        self.scores_flat = torch.from_numpy(values.astype(np.float32)).to(device)
        self.scores_stride = self.layer_scores + pad_scores
        self.total = sum(min(n, k) for n, k, _, _ in seqs)
        self.kept = torch.full((layers, self.hkv // together, self.total), -1, dtype=torch.int32, device=device)

    def scores(self, layer):
        return self.scores_flat[layer * self.scores_stride:layer * self.scores_stride + self.layer_scores].view(self.pages, self.hkv, self.page)

    def eviction(self):
        n, keep, first, last = (list(x) for x in zip(*self.seqs)) if self.seqs else ([], [], [], [])
        return step.Eviction(block_tables=[t if t.size else None for t in self.tables], slot0=self.slot0, num_tokens=n, keep=keep, first=first, last=last,
                             heads_together=self.together, flags=step.REANCHOR if self.reanchor else 0)

    def run(self, kept=True, stream=None, workspace=None):
        e = self.eviction()
        ws = torch.empty(step.evict_workspace_bytes(self.lay, e), dtype=torch.uint8, device=self.device) if workspace is None else workspace
        step.evict(self.lay, self.pool, e, self.scores_flat, ws, kept=self.kept if kept else None, scores_stride=self.scores_stride, stream=stream)

    def check(self, kept=True, stream=None):
        was = [f.clone() for f in self.flat]
        was_scores = self.scores_flat.clone()
        offset = self.pools[0].storage_offset()
        self.run(kept, stream)
        torch.cuda.synchronize()
        want = [w.clone() for w in was]
        want_scores = was_scores.clone()
        views = [w[offset:].as_strided(p.shape, p.stride()) for w, p in zip(want, self.pools)]
        old = [w[offset:].as_strided(p.shape, p.stride()) for w, p in zip(was, self.pools)]
        turned = []
        done = 0
        for i, (n, keep, first, last) in enumerate(self.seqs):
            m = min(n, keep)
            at = self.rows[i]
            page, place = at // self.page, at % self.page
            for layer in range(self.layers):
                s0 = was_scores[layer * self.scores_stride:layer * self.scores_stride + self.layer_scores].view(self.pages, self.hkv, self.page).cpu().numpy()
                s1 = want_scores[layer * self.scores_stride:layer * self.scores_stride + self.layer_scores].view(self.pages, self.hkv, self.page)
                for g in range(self.hkv // self.together):
                    heads = range(g * self.together, (g + 1) * self.together)
                    stay = eo.stays(eo.group_scores([s0[page, h, place] for h in heads]), keep, first, last) if n else np.zeros(0, np.int64)
                    if kept:
                        assert self.kept[layer, g, done:done + m].tolist() == stay.tolist(), (i, layer, g)
                    if m == 0 or m == n:
                        continue
                    src, dst = (torch.from_numpy(x).to(self.device) for x in (at[stay], at[:m]))
                    for h in heads:
                        s1[torch.from_numpy(page[:m]), h, torch.from_numpy(place[:m])] = torch.from_numpy(s0[page[stay], h, place[stay]]).to(self.device)
                        cols = slice(h * self.dk, (h + 1) * self.dk)
                        for x, (to, frm) in enumerate(zip(views, old)):
                            to[layer][dst, cols] = frm[layer][src, cols]
                            if x == 0 and self.reanchor:
                                turned.append((layer, cols, at[:m], host(frm[layer][src, cols]), stay - np.arange(m)))
            done += m
        torch.cuda.synchronize()
        for layer, cols, dst, rows, back in turned:
            y, terms = eo.turned(rows, back, self.base, self.band0, self.pairing == abi.GPTJ)
            got = host(self.pools[0][layer][torch.from_numpy(dst).to(self.device), cols])
            # cos and sin rounded once, two products and a sum in fp32, one rounding; the angle in 64 bits
            assert (np.abs(got - y) <= 4 * E32 * terms + HALF[self.dtype] * np.abs(y) * (1 + 2 ** -6) + 1e-38).all(), float(np.abs(got - y).max())
            views[0][layer][torch.from_numpy(dst).to(self.device), cols] = self.pools[0][layer][torch.from_numpy(dst).to(self.device), cols]
        same = lambda a, b: torch.equal(a.view(torch.int16 if a.dtype == torch.bfloat16 else torch.int32), b.view(torch.int16 if b.dtype == torch.bfloat16 else torch.int32))  # noqa: E731
        assert all(same(a, b) for a, b in zip(self.flat, want))  # what moves, and everything else as it was
        assert same(self.scores_flat, want_scores)
