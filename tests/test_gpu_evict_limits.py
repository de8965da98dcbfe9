"""Limits of eviction, weighing and differential attention on the GPU."""
import numpy as np
import pytest
import torch

from oracle import evict_oracle as eo
from position_free_kv_amd import abi, step
from tests import evict_util as eu
from tests.evict_util import Params
from tests.step_util import E32, HALF, Case
from tests.test_gpu_step_limits import SPOILS, formula, spoil

pytestmark = pytest.mark.gpu

GQA, MLA, BF16, F32 = abi.GQA, abi.MLA, abi.BF16, abi.F32


def test_evict_more_than_2_22_workgroups():
    """466 layers of 1001 sequences, 9 slices of a latent row: 3890 workgroups more than a row of the grid, whose second
    row has 4.2 million without work. Two tokens each, of which one stays."""
    layers, seqs, latent, rope, base = 466, 1001, 512, 64, 1e4
    pages, F = seqs + 1, latent + rope
    lay = abi.make_layout(MLA, BF16, layers, latent_dim=latent, rope_dim=rope, rope_base=base, page_size=2)
    gen = torch.Generator(device="cuda").manual_seed(0)
    rows = torch.empty(layers, pages, 2, F, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    scores = torch.rand(layers, pages, 1, 2, generator=gen, device="cuda")
    was, old = rows.clone(), scores.clone()
    order = np.random.default_rng(0).permutation(pages)[:seqs].astype(np.int32)
    e = step.Eviction(block_tables=order.reshape(seqs, 1), num_tokens=2, keep=1, flags=step.REANCHOR)
    kept = torch.full((layers, 1, seqs), -1, dtype=torch.int32, device="cuda")
    ws = torch.empty(step.evict_workspace_bytes(lay, e), dtype=torch.uint8, device="cuda")
    step.evict(lay, abi.make_pool(rows, None, pages), e, scores, ws, kept=kept)
    torch.cuda.synchronize()
    at = torch.from_numpy(order.astype(np.int64)).cuda()
    stays = (old[:, at, 0, 1] > old[:, at, 0, 0]).int()
    assert torch.equal(kept[:, 0], stays)
    want = old.clone()
    want[:, at, 0, 0] = old[:, at, 0].amax(-1)
    assert torch.equal(scores, want)
    spare = torch.ones(pages, dtype=torch.bool, device="cuda")
    spare[at] = False
    assert torch.equal(rows[:, spare].view(torch.int16), was[:, spare].view(torch.int16))
    assert torch.equal(rows[:, at, 1].view(torch.int16), was[:, at, 1].view(torch.int16))
    theta = base ** (-torch.arange(rope // 2, dtype=torch.float64, device="cuda") * 2 / rope)
    c, s = theta.cos(), (-theta).sin()
    for part in range(0, layers, 50):
        l = slice(part, part + 50)
        moved = stays[l].bool()
        got, stay, from1 = rows[l, at, 0], was[l, at, 0], was[l, at, 1]
        assert torch.equal(got[~moved].view(torch.int16), stay[~moved].view(torch.int16))
        got, from1 = got[moved], from1[moved]
        assert torch.equal(got[:, :latent].view(torch.int16), from1[:, :latent].view(torch.int16))
        a, b = (from1[:, latent + i * rope // 2:latent + (i + 1) * rope // 2].double() for i in range(2))
        y = torch.cat([a * c - b * s, a * s + b * c], 1)
        terms = torch.cat([(a * c).abs() + (b * s).abs(), (a * s).abs() + (b * c).abs()], 1)
        # cos and sin rounded once, two products and a sum in fp32, one rounding
        assert ((got[:, latent:].double() - y).abs() <= 4 * E32 * terms + HALF[BF16] * y.abs() * (1 + 2 ** -6) + 1e-38).all()


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("place", [0, 7])
def test_diff_of_a_long_request_among_short_ones(dim, place):
    """More wide tiles than places, whose keys are cut into ranges throughout."""
    requests = [(0, 150, 130)] * 8
    requests[place] = (0, 4000, 130)
    c = Case(layers=1, heads=128, kv_heads=8, head_dim=dim, prefixes=[60], requests=requests, seed=place)
    eu.check_diff(c, Params(c), 1.0 / float(np.sqrt(dim)))


@pytest.mark.parametrize("kind", [dict(heads=14, kv_heads=1, head_dim=64), dict(heads=14, kv_heads=1, head_dim=80), dict(dtype=F32, heads=14, kv_heads=1, head_dim=64),
                                  dict(family=MLA, heads=16, latent=512, rope=64), dict(family=MLA, dtype=F32, heads=16, latent=512, rope=64)])
def test_weigh_in_less_workspace(kind):
    """Rows in ranges, and whole in the least workspace that is taken: within the same bounds."""
    c = Case(layers=1, prefixes=[300], requests=[(0, 200, 180), (0, 700, 120), (-1, 30, 90)], **kind)
    scale = 1.0 / float(np.sqrt(c.dk))
    s = c.step(step.WEIGH | step.FIT)
    ws = c.workspace(s)
    lse, before = eu.own_lse(c, 0, scale), eu.new_scores(c)
    want, tol = eu.expect_weigh(c, 0, lse, before[0], scale, 1.0)
    results, least = [], 0
    for part in (1.0, 0.5, 0.0):
        least = max(int(ws.numel() * part) // 256 * 256, 256)
        while True:  # the first size from there on that is taken
            try:
                plan = step.upload(c.lay, s, c.pool, (ws.data_ptr(), least))
                break
            except abi.KameraError as e:
                assert e.name == "KAMERA_E_WORKSPACE"
                least += 256
        assert least <= ws.numel()
        scores = before.clone()
        step.weigh(plan, 0, c.q[0], lse, scores[0], scale)
        torch.cuda.synchronize()
        assert (np.abs(eu.host(scores[0]) - want) <= tol).all()
        results.append(scores)
    assert least < ws.numel() and not torch.equal(results[0], results[-1])  # other sums, other roundings


# ------------------------------------------------------------------ numbers that are not finite, where they are seen
DIFF_KINDS = [dict(heads=8, kv_heads=2, head_dim=128), dict(heads=4, kv_heads=4, head_dim=64), dict(dtype=F32, heads=4, kv_heads=2, head_dim=64),
              dict(heads=4, kv_heads=2, head_dim=80)]


def check_diff_formula(c, s, ws, p, scale):
    """One layer's outputs against the formula: the same infinities and NaN, the rest within the bounds of eu.expect_diff."""
    plan = step.upload(c.lay, s, c.pool, ws)
    out = torch.full((c.n, c.heads * c.dk), 7.0, dtype=c.q.dtype, device="cuda")
    lse = torch.full((c.n, c.heads), 7.0, device="cuda")
    step.attend_diff(plan, 0, c.q[0], out, scale, lse=lse, **p.kwargs())
    torch.cuda.synchronize()
    d, pairs = c.dk, c.hkv // 2
    per = c.heads // pairs
    k, v = (eu.host(x[0]) for x in c.pools)
    q = eu.host(c.q[0]).reshape(c.n, c.heads, d)
    maps, mtol = np.zeros((2, c.n, c.heads // 2, 2 * d)), np.zeros((2, c.n, c.heads // 2, 2 * d))
    z = np.zeros((c.n, c.heads))
    with np.errstate(all="ignore"):
        for rows, at, last in eu.visible(c):
            for h in range(c.hkv):
                heads = h // 2 * per + h % 2 + 2 * np.arange(per // 2)
                o, l, a, terms = formula(q[rows][:, heads], k[at, h * d:(h + 1) * d], v[at, h // 2 * 2 * d:(h // 2 + 1) * 2 * d], scale, last)
                ds = (d + 8) * E32 * terms[..., None]
                rel = 2 * ds + (2 * at.size + 128) * E32 + (HALF[BF16] if c.dtype == BF16 else 0.0)
                where = slice(heads[0] // 2, heads[-1] // 2 + 1)
                maps[h % 2][rows, where] = o
                mtol[h % 2][rows, where] = rel * (a + np.abs(np.where(np.isfinite(o), o, 0))) + 1e-37
                z[rows, heads[0]:heads[-1] + 1:2] = l
        value, terms = eo.lam(eu.host(p.lambdas), p.lambda_init)
        x = maps[0] - value * maps[1]
        size = [np.abs(np.where(np.isfinite(m), m, 0)) for m in maps]
        tx = mtol[0] + abs(value) * mtol[1] + (d + 16) * E32 * terms * size[1] + 4 * E32 * (size[0] + abs(value) * size[1])
        y = x
        if p.norm:  # a row with an infinity has an infinite norm: its finite numbers become 0, the infinite ones NaN
            y = x / np.sqrt((x * x).mean(-1, keepdims=True) + p.eps) * eu.host(p.weight)
        y = y * p.out_scale
    got, want = eu.host(out).reshape(x.shape), y
    assert (np.isnan(got) == np.isnan(want)).all(), np.argwhere(np.isnan(got) != np.isnan(want))[:4].tolist()
    assert (np.isinf(got) == np.isinf(want)).all() and (got[np.isinf(want)] == want[np.isinf(want)]).all()
    if p.norm:
        rows = np.isinf(x).any(-1, keepdims=True) & np.isfinite(want)
        assert (got[rows] == 0).all()
    else:
        fin = np.isfinite(want)
        tol, off = (tx * abs(p.out_scale) + (4 * E32 + HALF[c.dtype]) * np.abs(want) + 1e-37)[fin], np.abs(got[fin] - want[fin])
        assert (off <= tol).all(), float((off / tol).max())
    gz = eu.host(lse)
    assert (np.isnan(gz) == np.isnan(z)).all() and (np.isneginf(gz) == np.isneginf(z)).all()


@pytest.mark.parametrize("what", SPOILS)
@pytest.mark.parametrize("kind", DIFF_KINDS)
def test_diff_seen_numbers_that_are_not_finite_act_as_in_the_formula(kind, what):
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
        s = c.step(step.ATTEND | step.DIFFERENTIAL | step.FIT)
        ws = c.workspace(s)
        for part, norm in ((1.0, False), (0.5, True), (0.05, False), (0.0, True)):
            least = (int(ws.numel() * part) + 255) // 256 * 256
            while True:  # the first size from there on that is taken
                try:
                    check_diff_formula(c, s, (ws.data_ptr(), least), Params(c, norm=norm), 0.25)
                    break
                except abi.KameraError as e:
                    assert e.name == "KAMERA_E_WORKSPACE"
                    least = least * 5 // 4 + 256


@pytest.mark.parametrize("queries", [1, 40])
@pytest.mark.parametrize("kind", [dict(heads=4, kv_heads=2, head_dim=128), dict(heads=4, kv_heads=2, head_dim=64), dict(dtype=F32, heads=4, kv_heads=2, head_dim=64),
                                  dict(heads=4, kv_heads=2, head_dim=80), dict(family=MLA, heads=4, latent=512, rope=64)])
def test_weigh_seen_numbers_that_are_not_finite_act_as_in_the_formula(kind, queries):
    """Keys and statistics of every kind: exp(scale q.k - lse) as it stands, rows of lse -inf left out."""
    c = Case(layers=1, prefixes=[200], requests=[(0, queries + 30, queries), (0, 9, 1), (-1, 70, queries)], seed=queries, **kind)
    c.q.abs_()
    scale, inf = 0.25 if c.dk < 500 else 0.05, float("inf")
    lse = eu.own_lse(c, 0, scale)
    lse[0, 0], lse[0, 1], lse[c.n // 2, 2], lse[-1, 3] = -inf, inf, float("nan"), inf
    keys = c.pools[0][0]
    for r, rows in enumerate(c.rows):
        for i, bad in enumerate((inf, -inf, float("nan"))):
            keys[int(rows[(3 + 2 * i + r) % rows.size]), ((7 * i + r) % c.hkv) * c.dk + c.dk - 1 - i] = bad
    before = eu.new_scores(c)
    after = before.clone()
    eu.weigh(c, lse[None], after, scale, 0.5)
    torch.cuda.synchronize()
    with np.errstate(all="ignore"):
        want, tol = eu.expect_weigh(c, 0, lse, before[0], scale, 0.5)
    got = eu.host(after[0])
    assert (np.isnan(got) == np.isnan(want)).all(), np.argwhere(np.isnan(got) != np.isnan(want))[:4].tolist()
    assert (np.isinf(got) == np.isinf(want)).all() and (got[np.isinf(want)] > 0).all()
    fin = np.isfinite(want) & np.isfinite(tol)
    assert fin.any() and (np.abs(got[fin] - want[fin]) <= tol[fin]).all()
