"""Limits of the serving step on the GPU: what may be recorded in a graph."""
import numpy as np
import pytest
import torch

from position_free_kv_amd import abi, step
from tests.step_util import E32, HALF, Case
from tests.test_gpu_step import page_pool

pytestmark = pytest.mark.gpu

GQA, MLA, BF16, F32 = abi.GQA, abi.MLA, abi.BF16, abi.F32


# ------------------------------------------------------------------ graph capture
def test_staged_calls_are_refused_while_capturing():
    """A replay would read a staging slot that later calls fill: uploads and ordered page copies are refused,
    and the capture goes on."""
    c = Case(head_dim=128, prefixes=[40], requests=[(0, 5, 1), (0, 3, 2)])
    s = c.step(step.ATTEND)
    ws = c.workspace(s)
    want, _ = c.attend(0.1)
    plan = step.upload(c.lay, s, c.pool, ws)
    lay, pool, views, _ = page_pool(GQA, BF16, 2, 600, 4, kv_heads=1, head_dim=16)
    copies = torch.empty(step.copy_pages_workspace_bytes(500), dtype=torch.uint8, device="cuda")
    other = c.workspace(s)
    out = torch.zeros_like(want[0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step.attend(plan, 0, c.q[0], out, 0.1)
        for call in (lambda: step.upload(c.lay, s, c.pool, other), lambda: step.copy_pages(lay, pool, [1, 2], [2, 3], copies),
                     lambda: step.copy_pages(lay, pool, np.arange(300).repeat(2)[:401] % 100, np.arange(401) + 150, copies)):
            with pytest.raises(abi.KameraError) as e:
                call()
            assert e.value.name == "KAMERA_E_UNSUPPORTED"
        step.copy_pages(lay, pool, np.arange(0, 100), np.arange(200, 300), copies)  # as arguments
    for i in range(3):
        out.zero_()
        views[0][:, :100] = float(i + 1)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0])
        assert (views[0][:, 200:300] == i + 1).all()
        step.upload(c.lay, s, c.pool, other)  # eager calls take the staging slots in between
        step.copy_pages(lay, pool, [401, 402], [402, 401], copies)
        torch.cuda.synchronize()


# ------------------------------------------------------------------ one workspace for many steps
def check(c, out, lse, scale):
    """Outputs of every layer against the 64-bit expectation, within Case's bounds."""
    torch.cuda.synchronize()
    for layer in range(c.layers):
        o, tol, z, ltol = c.expect_attend(layer, scale)
        got, gz = out[layer].double().cpu().numpy(), lse[layer].double().cpu().numpy()
        assert (np.abs(got - o) <= tol).all(), layer
        empty = np.isneginf(z)
        assert (np.isneginf(gz) == empty).all()
        assert (np.abs(np.where(empty, 0, gz) - np.where(empty, 0, z)) <= ltol).all(), layer


def attend(c, s, ws, scale):
    plan = step.upload(c.lay, s, c.pool, ws)
    out = torch.full((c.layers, c.n, c.heads * c.dv), 7.0, dtype=c.q.dtype, device="cuda")
    lse = torch.full((c.layers, c.n, c.heads), 7.0, device="cuda")
    for layer in range(c.layers):
        step.attend(plan, layer, c.q[layer], out[layer], scale, lse=lse[layer])
    return out, lse


KINDS = [dict(heads=8, kv_heads=2, head_dim=128), dict(heads=3, kv_heads=3, head_dim=64), dict(dtype=F32, heads=4, kv_heads=2, head_dim=64),
         dict(heads=4, kv_heads=2, head_dim=80), dict(family=MLA, heads=16, latent=512, rope=64), dict(family=MLA, heads=3, latent=20, rope=6)]


@pytest.mark.parametrize("kind", KINDS)
def test_a_step_uploaded_again_with_other_lengths_into_one_workspace(kind):
    """A loop that changes a Step in place: longer, shorter, empty, and back, in the buffer of the longest."""
    longest = [700, 33, 260, 64]
    c = Case(layers=1, prefixes=[1100], requests=[(0, n, 1) for n in longest] + [(-1, 300, 2)], seed=5, **kind)
    rows = list(c.rows)
    s = c.step(step.ATTEND | step.FIT)
    ws = c.workspace(s)
    for lengths in (longest, [1, 1, 1, 1], [0, 33, 17, 5], [700, 0, 0, 64], [129, 32, 128, 63], [0, 0, 0, 0], longest):
        c.requests = [(0, n, 1, 0) for n in lengths] + [(-1, 300 if lengths[0] else 1, 2, 0)]
        c.rows = [r[:r.size if i == 0 else c.requests[i - 1][1]] for i, r in enumerate(rows)]
        s.requests["num_tokens"] = [r[1] for r in c.requests]
        check(c, *attend(c, s, ws, 0.2), 0.2)


@pytest.mark.parametrize("kind", KINDS)
def test_attend_in_less_workspace(kind):
    """Fewer ranges, then no sharing of the prefix, down to no partial rows; then a refusal."""
    c = Case(layers=1, prefixes=[2500], requests=[(0, 400, 1), (0, 1, 1), (0, 0, 2), (0, 90, 3), (-1, 900, 1), (-1, 0, 2), (0, 130, 130)], seed=6, **kind)
    s = c.step(step.ATTEND | step.FIT)
    ws = c.workspace(s)
    sizes, results = ws.numel(), set()
    while True:
        try:
            out, lse = attend(c, s, (ws.data_ptr(), sizes), 0.2)
        except abi.KameraError as e:
            assert e.name == "KAMERA_E_WORKSPACE"
            break
        check(c, out, lse, 0.2)
        again, _ = attend(c, s, (ws.data_ptr(), sizes), 0.2)
        assert torch.equal(out, again)
        results.add(out.view(torch.int16 if out.dtype == torch.bfloat16 else torch.int32).cpu().numpy().tobytes())
        sizes = sizes * 2 // 3
    assert len(results) > 1  # other plans, other roundings
    exact = c.step(step.ATTEND)
    with pytest.raises(abi.KameraError) as e:
        step.upload(c.lay, exact, c.pool, (ws.data_ptr(), sizes * 3 // 2))
    assert e.value.name == "KAMERA_E_WORKSPACE"


# ------------------------------------------------------------------ numbers that are not finite, where they are seen
def formula(q, k, v, scale, last):
    """softmax(scale q k^T) v as it stands, 0 * inf = NaN included, for queries [n][G][dk] over keys [T][dk]; keys of score
    -inf weigh nothing, and where all do the sum of weights is 0: output 0 (NaN where 0 * inf), lse -inf. Also the sums
    that Case's bounds are made of, over what is finite."""
    n, g, _ = q.shape
    out, absv = np.zeros((n, g, v.shape[1])), np.zeros((n, g, v.shape[1]))
    lse, terms = np.full((n, g), -np.inf), np.zeros((n, g))
    for i in range(n):
        t = int(last[i]) + 1
        for h in range(g if t > 0 else 0):
            prods = scale * q[i, h] * k[:t]
            s = prods.sum(1)
            m = np.nan if np.isnan(s).any() else s.max()
            p = np.zeros(t) if m == -np.inf else np.exp(s - m)
            total = p.sum()
            out[i, h] = (p[:, None] * v[:t]).sum(0) / (total if total != 0 else 1.0)
            absv[i, h] = (p[:, None] * np.abs(np.where(np.isfinite(v[:t]), v[:t], 0))).sum(0) / (total if total != 0 else 1.0)
            lse[i, h] = m + np.log(total) if total != 0 else -np.inf
            live = np.isfinite(s) & (p > 0)
            if live.any():
                terms[i, h] = np.abs(prods[live]).sum(1).max()
    return out, lse, absv, terms


def check_formula(c, s, ws, scale, rounded=True):
    """One layer's outputs against formula(): the same infinities and NaN, the rest within Case's bounds (rounded: with the
    probabilities' rounding to bf16)."""
    got, gz = attend(c, s, ws, scale)
    torch.cuda.synchronize()
    got, gz = got[0].double().cpu().numpy().reshape(c.n, c.heads, c.dv), gz[0].double().cpu().numpy()
    f64 = [p[0].double().cpu().numpy() for p in c.pools]
    q = c.q[0].double().cpu().numpy().reshape(c.n, c.heads, c.dk)
    n0, np_ = 0, len(c.prefix_tokens)
    with np.errstate(all="ignore"):
        for r, (pre, own, nq, flags) in enumerate(c.requests):
            head = c.rows[pre] if pre >= 0 else np.zeros(0, np.int64)
            at = np.concatenate([head, c.rows[np_ + r]])
            last = np.maximum(head.size + own - nq + np.arange(nq), head.size - 1)
            for h in range(c.hkv):
                k, v = f64[0][at, h * c.dk:(h + 1) * c.dk], f64[-1][at, h * c.dk:h * c.dk + c.dv]
                sl = slice(h * c.g, (h + 1) * c.g)
                o, z, a, terms = formula(q[n0:n0 + nq, sl], k, v, scale, last)
                x, y = got[n0:n0 + nq, sl], gz[n0:n0 + nq, sl]
                where = (r, h)
                assert (np.isnan(x) == np.isnan(o)).all(), (where, np.argwhere(np.isnan(x) != np.isnan(o))[:4].tolist(), int(np.isnan(o).sum()))
                assert (np.isinf(x) == np.isinf(o)).all() and (x[np.isinf(o)] == o[np.isinf(o)]).all(), where
                assert (np.isnan(y) == np.isnan(z)).all() and (np.isneginf(y) == np.isneginf(z)).all(), where
                # as in Case.expect_attend; a weight too small for fp32 may be 0: 2^-126 of a value
                ds = (c.dk + 8) * E32 * terms[..., None]
                rel = 2 * ds + (2 * at.size + 128) * E32 + (HALF[BF16] if c.dtype == BF16 and rounded else 0.0)
                fin = np.isfinite(o)
                assert (np.abs(x - o) <= rel * (a + np.abs(o)) + HALF[c.dtype] * np.abs(o) + 1e-37)[fin].all(), where
                fin = np.isfinite(z)
                assert (np.abs(y - z) <= ds[..., 0] + (at.size + 128) * E32 + 8 * E32 * np.abs(z))[fin].all(), where
            n0 += nq


SPOILS = ["inf under no weight", "inf", "nan", "inf and -inf", "key -inf", "key inf", "key nan", "all keys -inf"]


def spoil(c, what, slots, col):
    """Puts what is not finite into key and value rows; queries are positive, so a key column of -inf is a score of -inf."""
    k, v = c.pools[0][0], c.pools[-1][0]
    at = torch.from_numpy(np.asarray(slots)).cuda()
    inf = float("inf")
    for h in range(c.hkv):
        if what == "inf under no weight":
            k[at, h * c.dk:(h + 1) * c.dk] = -200.0
            v[at, h * c.dk + col] = -inf if c.family == MLA else inf
        elif what in ("inf", "nan"):
            v[at, h * c.dk + col] = float(what)
        elif what == "inf and -inf":
            v[at[::2], h * c.dk + col] = inf
            v[at[1::2], h * c.dk + col] = -inf
        elif what.startswith("key"):
            k[at, h * c.dk + (c.dk - 1 if c.family == MLA else col)] = float(what[4:])  # (MLA: in the rope band)
        else:
            k[at, h * c.dk + col] = -inf


@pytest.mark.parametrize("what", SPOILS)
@pytest.mark.parametrize("kind", KINDS)
def test_seen_numbers_that_are_not_finite_act_as_in_the_formula(kind, what):
    """Whatever the plan: keys in the middle of a range, at its masked end, alone in a part, in shared and own tokens."""
    for seed, (prefix, own, nq) in enumerate([(300, 70, 2), (2100, 45, 1), (0, 150, 40), (40, 3, 3)]):
        c = Case(layers=1, prefixes=[prefix], requests=[(0, own, nq), (0, 33, 1), (0, own + 9, 1), (-1, 40, 2)], seed=seed, **kind)
        c.q.abs_()
        for r, rows in enumerate(c.rows):
            if rows.size == 0:
                continue
            n = rows.size
            some = rows if what == "all keys -inf" and r == 3 else rows[sorted({n // 3, max(n - 3, 0), n - 1})] if r % 2 == 0 else rows[:1]
            spoil(c, what, some, (5 * r + 1) % c.dv)
        s = c.step(step.ATTEND | step.FIT)
        ws = c.workspace(s)
        for part in (1.0, 0.5, 0.05, 0.0):
            least = (int(ws.numel() * part) + 255) // 256 * 256
            while True:  # the first size from there on that is taken
                try:
                    check_formula(c, s, (ws.data_ptr(), least), 0.25)
                    break
                except abi.KameraError as e:
                    assert e.name == "KAMERA_E_WORKSPACE"
                    least = least * 5 // 4 + 256


# ------------------------------------------------------------------ launches of more than 2^32 threads
def small_pages(layers, pages, tensors):
    """Pools of 4-byte pages, every page of every layer with bits of its own."""
    family = GQA if tensors == 2 else MLA
    lay = abi.make_layout(family, BF16, layers, num_kv_heads=1, head_dim=2, latent_dim=0, rope_dim=2, page_size=1)
    pools = [torch.arange(layers * pages, dtype=torch.int32, device="cuda").mul_(2654435761 % 2 ** 31).add_(t).view(layers, pages) for t in range(tensors)]
    return lay, abi.make_pool(pools[0], pools[1] if tensors == 2 else None, pages), pools


@pytest.mark.parametrize("layers,pages,n,chained,tensors", [
    (520, 33000, 16384, False, 2),       # 17.0M workgroups, one a page and layer
    (700, 33000, 16384, True, 2),        # pairs of pages change places: 11.5M, two copies and a kept page each
    (1100, 33000, 16384, True, 2),       # 18.0M
    ((1 << 24) + 70000, 66, 65, True, 1),  # a ring in each of 16.8M layers
])
def test_page_copies_of_more_than_2_24_workgroups(layers, pages, n, chained, tensors):
    rng = np.random.default_rng(n)
    order = rng.permutation(pages).astype(np.int32)
    if n < 1000:
        src, dst = np.roll(order[:n], -1), order[:n]
    elif chained:
        src, dst = order[:n], order[:n].reshape(-1, 2)[:, ::-1].reshape(-1)
    else:
        src, dst = order[:n], order[n:2 * n]
    lay, pool, pools = small_pages(layers, pages, tensors)
    want = [p.clone() for p in pools]
    s, d = (torch.from_numpy(x.astype(np.int64)).cuda() for x in (src, dst))
    for w, p in zip(want, pools):
        w[:, d] = p[:, s]
    ws = torch.empty(step.copy_pages_workspace_bytes(n), dtype=torch.uint8, device="cuda")
    step.copy_pages(lay, pool, src, dst, ws)
    torch.cuda.synchronize()
    assert all(torch.equal(p, w) for p, w in zip(pools, want))


def test_append_and_attend_of_more_than_2_24_workgroups():
    """65536 heads of two columns: 17.0M and 34.1M workgroups; position 0 turns nothing, and one key is its value."""
    heads, n = 65536, 520
    f = 2 * heads
    lay = abi.make_layout(GQA, BF16, 1, num_kv_heads=heads, head_dim=2, page_size=1)
    pools = [torch.zeros(1, n, f, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    pool = abi.make_pool(*pools, n)
    table = np.random.default_rng(0).permutation(n).astype(np.int32)
    rows = [torch.randint(-100, 100, (n, f), dtype=torch.int16, device="cuda").bfloat16() for _ in range(3)]
    positions = torch.zeros(n, 3, dtype=torch.int32, device="cuda")
    s = step.Step(num_q_heads=heads, block_tables=table.reshape(n, 1), num_tokens=1, num_queries=1, positions=positions)
    ws = torch.empty(step.workspace_bytes(lay, s), dtype=torch.uint8, device="cuda")
    plan = step.upload(lay, s, pool, ws)
    q, out = torch.empty_like(rows[0]), torch.empty_like(rows[0])
    step.append(plan, 0, q=rows[0], k=rows[1], v=rows[2], q_out=q)
    step.attend(plan, 0, q, out, 1.0)
    torch.cuda.synchronize()
    at = torch.from_numpy(table.astype(np.int64)).cuda()
    assert torch.equal(q, rows[0])
    assert torch.equal(pools[0][0, at], rows[1]) and torch.equal(pools[1][0, at], rows[2])
    assert torch.equal(out, rows[2])


# ------------------------------------------------------------------ the plain kernel's roundings
@pytest.mark.parametrize("kind", [dict(heads=4, kv_heads=2, head_dim=80), dict(heads=3, kv_heads=1, head_dim=10), dict(family=MLA, heads=3, latent=20, rope=6),
                                  dict(heads=4, kv_heads=2, head_dim=128, offset=1)])
def test_plain_attention_rounds_bf16_once(kind):
    """Outside the matrix cores no probability is rounded: all that is left is fp32 arithmetic and the output's own rounding."""
    c = Case(layers=1, prefixes=[300], requests=[(0, 40, 1), (0, 9, 3), (-1, 70, 2), (-1, 2, 1), (-1, 3, 2)], seed=8, **kind)
    s = c.step(step.ATTEND)
    check_formula(c, s, c.workspace(s), 0.2, rounded=False)
