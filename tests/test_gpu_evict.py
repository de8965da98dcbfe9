"""Differential attention, weighing and eviction on the GPU against their 64-bit oracle."""
import numpy as np
import pytest
import torch

from position_free_kv_amd import abi, step
from tests import evict_util as eu
from tests.evict_util import Cache, Params
from tests.step_util import TYPES, Case

pytestmark = pytest.mark.gpu

ALL = step.REQUEST_ALL
GQA, MLA, BF16, F32 = abi.GQA, abi.MLA, abi.BF16, abi.F32
HEADS = [(8, 2, 64), (8, 2, 128), (28, 4, 128), (4, 4, 128), (6, 6, 64), (40, 2, 64), (36, 2, 128), (6, 2, 80), (4, 2, 10), (4, 2, 256), (2, 2, 512)]


def scale_of(c):
    return 1.0 / float(np.sqrt(c.dk))


# ------------------------------------------------------------------ differential attention
@pytest.mark.parametrize("heads,kv,dim", HEADS)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_diff_layouts(heads, kv, dim, dtype):
    c = Case(dtype=dtype, heads=heads, kv_heads=kv, head_dim=dim, prefixes=[77], seed=heads + dim,
             requests=[(0, 1, 1), (0, 33, 1), (0, 16, 5), (-1, 40, 3), (0, 0, 1)])
    eu.check_diff(c, Params(c), scale_of(c))


@pytest.mark.parametrize("page", [1, 3, 8, 64])
@pytest.mark.parametrize("dim", [64, 128])
def test_diff_page_sizes(page, dim):
    c = Case(head_dim=dim, page=page, prefixes=[130], requests=[(0, 21, 1), (0, 64, 2), (0, 5, 1)], seed=page)
    eu.check_diff(c, Params(c), scale_of(c))


@pytest.mark.parametrize("tokens", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 257, 1000, 4097])
@pytest.mark.parametrize("dim", [64, 128])
def test_diff_lengths(tokens, dim):
    c = Case(layers=1, heads=8, kv_heads=2, head_dim=dim, prefixes=[tokens], requests=[(-1, tokens, 1), (0, 3, 1), (0, 2, 1)], seed=tokens)
    eu.check_diff(c, Params(c), scale_of(c))


@pytest.mark.parametrize("queries", [2, 7, 16, 33, 65, 129])
@pytest.mark.parametrize("dim,dtype", [(128, BF16), (64, BF16), (64, F32), (48, BF16)])
def test_diff_many_queries(queries, dim, dtype):
    """Causal edges inside and between tiles; requests that share and that read the prefix themselves."""
    c = Case(dtype=dtype, layers=1, heads=4, kv_heads=2, head_dim=dim, prefixes=[150, 40], seed=queries,
             requests=[(0, queries, queries), (0, queries + 37, queries), (1, queries + 1, 3), (0, 9, 2), (-1, queries, queries)])
    eu.check_diff(c, Params(c), scale_of(c))


@pytest.mark.parametrize("members", [2, 5, 9, 17, 40])
@pytest.mark.parametrize("dim", [64, 128])
def test_diff_tiles_of_every_size_over_long_prefixes(members, dim):
    c = Case(layers=1, heads=4, kv_heads=2, head_dim=dim, prefixes=[9000], requests=[(0, 1 + i % 3, 1) for i in range(members)], seed=members)
    c.q *= 4  # a few keys stand out: a lost or doubled stage shows
    eu.check_diff(c, Params(c), scale_of(c))


@pytest.mark.parametrize("kw", [dict(lambdas=False), dict(weight=False), dict(norm=False), dict(norm=False, out_scale=1.0, lambda_init=0.0), dict(eps=0.0),
                                dict(lambda_init=-1.5, out_scale=-2.0), dict(lambdas=False, lambda_init=0.0)])
@pytest.mark.parametrize("dim,dtype", [(128, BF16), (64, F32)])
def test_diff_parameters(kw, dim, dtype):
    c = Case(dtype=dtype, head_dim=dim, prefixes=[60], requests=[(0, 40, 2), (-1, 33, 12, ALL), (0, 20, 1, ALL)])
    eu.check_diff(c, Params(c, **kw), scale_of(c))
    eu.check_diff(c, Params(c, **kw), -scale_of(c))


@pytest.mark.parametrize("dim,dtype", [(128, BF16), (64, BF16), (64, F32), (80, BF16)])
@pytest.mark.parametrize("eps", [1e-5, 0.0])
def test_diff_rows_that_see_nothing(dim, dtype, eps):
    c = Case(dtype=dtype, head_dim=dim, prefixes=[0, 30], seed=3,
             requests=[(-1, 0, 2), (-1, 3, 5), (0, 0, 1), (0, 4, 1), (1, 2, 6), (1, 0, 3), (1, 10, 0), (-1, 0, 0), (-1, 17, 60), (1, 1, 1)])
    out, lse = eu.check_diff(c, Params(c, eps=eps), scale_of(c))
    assert (out[:, :2] == 0).all() and torch.isneginf(lse[:, :2]).all()


@pytest.mark.parametrize("dim,dtype", [(128, BF16), (64, BF16), (64, F32), (80, BF16)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_diff_ignores_what_is_unseen(dim, dtype, bad):
    c = Case(dtype=dtype, head_dim=dim, garbage=bad, prefixes=[35], requests=[(0, 20, 4), (-1, 70, 40), (0, 3, 1), (0, 150, 130)], seed=9)
    p = Params(c)
    o0, z0 = eu.check_diff(c, p, scale_of(c))
    for r in range(len(c.requests)):  # each request's last token: only its last query sees it
        for x in c.pools:
            x[:, int(c.rows[1 + r][-1])] = bad
    o1, z1 = eu.attend_diff(c, p, scale_of(c))
    torch.cuda.synchronize()
    keep = torch.ones(c.n, dtype=torch.bool, device="cuda")
    keep[torch.cumsum(torch.tensor([r[2] for r in c.requests]), 0) - 1] = False
    assert torch.equal(o0[:, keep], o1[:, keep]) and torch.equal(z0[:, keep], z1[:, keep])


@pytest.mark.parametrize("dim,dtype", [(128, BF16), (64, BF16), (64, F32)])
def test_diff_a_map_without_a_finite_score(dim, dtype):
    """Keys of -inf in one map's head leave that map 0 and the other as it is."""
    c = Case(dtype=dtype, layers=1, heads=2, kv_heads=2, head_dim=dim, requests=[(-1, 50, 1), (-1, 200, 3)])
    c.q.abs_()
    c.pools[0][:, :, dim:] = float("-inf")
    p = Params(c, norm=False)
    out, lse = eu.attend_diff(c, p, scale_of(c))
    torch.cuda.synchronize()
    assert torch.isneginf(lse[..., 1]).all() and torch.isfinite(lse[..., 0]).all() and torch.isfinite(out.float()).all()
    c.pools[0][:, :, dim:] = 0
    o, tol, _, _ = eu.expect_diff(c, Params(c, norm=False, lambdas=False, lambda_init=0.0, out_scale=p.out_scale), 0, scale_of(c))
    assert (np.abs(eu.host(out[0]) - o) <= tol).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_diff_strides_and_alignment(dtype):
    """Queries and outputs as slices of wider rows, on and off the 16-byte grid; pools off it; no lse."""
    for shift, offset, pad in ((8, 0, 0), (1, 0, 0), (0, 1, 0), (0, 0, 5)):
        c = Case(dtype=dtype, head_dim=64, heads=8, kv_heads=4, prefixes=[50], requests=[(0, 30, 2), (-1, 60, 33)], offset=offset, pad_layer=pad, seed=shift)
        p = Params(c)
        want, _ = eu.check_diff(c, p, scale_of(c))
        s = c.step(step.ATTEND | step.DIFFERENTIAL)
        plan = step.upload(c.lay, s, c.pool, c.workspace(s))
        q = torch.full((c.n, 8 * 64 + 40), 9.0, dtype=TYPES[dtype], device="cuda")
        out = torch.full((c.n, 8 * 64 + 24), 5.0, dtype=TYPES[dtype], device="cuda")
        q[:, shift:shift + 512] = c.q[1]
        step.attend_diff(plan, 1, q[:, shift:shift + 512], out[:, shift:shift + 512], scale_of(c), **p.kwargs())
        torch.cuda.synchronize()
        if dtype == BF16:
            assert torch.equal(out[:, shift:shift + 512], want[1])
        o, tol, _, _ = eu.expect_diff(c, p, 1, scale_of(c))  # (fp32 rows off the grid are read, and so summed, in other pieces)
        assert (np.abs(eu.host(out[:, shift:shift + 512]) - o) <= tol).all()
        assert (out[:, :shift] == 5).all() and (out[:, shift + 512:] == 5).all()


# ------------------------------------------------------------------ weighing
@pytest.mark.parametrize("heads,kv,dim", HEADS + [(7, 1, 128), (3, 3, 64), (20, 1, 64)])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("diff", [False, True])
def test_weigh_layouts(heads, kv, dim, dtype, diff):
    if diff and kv % 2:
        pytest.skip("pairs of KV heads")
    c = Case(dtype=dtype, heads=heads, kv_heads=kv, head_dim=dim, prefixes=[77], seed=heads + dim,
             requests=[(0, 1, 1), (0, 33, 1), (0, 16, 5), (-1, 40, 3), (0, 0, 1)])
    eu.check_weigh(c, scale_of(c), diff=diff)


@pytest.mark.parametrize("heads,latent,rope", [(16, 512, 64), (3, 20, 6), (1, 64, 64), (40, 512, 64), (2, 512, 512)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_weigh_latent_rows(heads, latent, rope, dtype):
    c = Case(family=MLA, dtype=dtype, heads=heads, latent=latent, rope=rope, prefixes=[50], seed=latent + heads,
             requests=[(0, 1, 1), (0, 70, 2), (0, 16, 1), (-1, 19, 3)])
    eu.check_weigh(c, scale_of(c))


@pytest.mark.parametrize("page", [1, 3, 8, 64])
@pytest.mark.parametrize("family,dim", [(GQA, 128), (GQA, 64), (MLA, 64)])
def test_weigh_page_sizes(page, family, dim):
    more = dict(heads=8, kv_heads=2, head_dim=dim) if family == GQA else dict(family=MLA, heads=4, latent=512, rope=dim)
    c = Case(page=page, prefixes=[130], requests=[(0, 21, 1), (0, 64, 2), (0, 5, 1)], seed=page, **more)
    eu.check_weigh(c, scale_of(c))


@pytest.mark.parametrize("tokens", [1, 15, 16, 17, 63, 64, 65, 127, 129, 255, 256, 257, 1000, 4097])
@pytest.mark.parametrize("family,dim", [(GQA, 128), (GQA, 64), (MLA, 64)])
def test_weigh_lengths(tokens, family, dim):
    more = dict(heads=8, kv_heads=2, head_dim=dim) if family == GQA else dict(family=MLA, heads=4, latent=512, rope=dim)
    c = Case(layers=1, prefixes=[tokens], requests=[(-1, tokens, 1), (0, 3, 1), (0, 2, 1)], seed=tokens, **more)
    eu.check_weigh(c, scale_of(c))


@pytest.mark.parametrize("queries", [2, 7, 16, 33, 65, 129, 300])
@pytest.mark.parametrize("dim,dtype", [(128, BF16), (64, BF16), (64, F32), (48, BF16)])
def test_weigh_many_queries(queries, dim, dtype):
    c = Case(dtype=dtype, layers=1, heads=6, kv_heads=2, head_dim=dim, prefixes=[150, 40], seed=queries,
             requests=[(0, queries, queries), (0, queries + 37, queries), (1, queries + 1, 3), (0, 9, 2), (-1, queries, queries), (0, 5, 4, ALL)])
    eu.check_weigh(c, scale_of(c))


@pytest.mark.parametrize("family", [GQA, MLA])
def test_weigh_rows_cut_into_ranges(family):
    """More rows than a range takes, some of which see none of the first keys."""
    more = dict(heads=14, kv_heads=1, head_dim=64) if family == GQA else dict(family=MLA, heads=16, latent=512, rope=64)
    c = Case(layers=1, prefixes=[300], requests=[(0, 200, 180), (0, 700, 120), (-1, 30, 90)], **more)
    _, _, a = eu.check_weigh(c, scale_of(c))
    lse, before, b = eu.check_weigh(c, scale_of(c), flags=step.FIT)
    assert torch.equal(a, b)


@pytest.mark.parametrize("decay", [0.0, 0.5, -1.0])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_weigh_decay_and_scale(decay, dtype):
    c = Case(dtype=dtype, prefixes=[60], requests=[(0, 40, 2), (-1, 33, 12, ALL), (0, 20, 0), (-1, 9, 0)])
    eu.check_weigh(c, scale_of(c), decay)
    eu.check_weigh(c, -scale_of(c), decay)
    eu.check_weigh(c, 0.0, decay)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_weigh_decay_of_zero_reads_no_scores(dtype):
    c = Case(dtype=dtype, requests=[(-1, 40, 2)])
    lse = torch.stack([eu.own_lse(c, layer, scale_of(c)) for layer in range(c.layers)])
    scores = torch.full_like(eu.new_scores(c), float("nan"))
    eu.weigh(c, lse, scores, scale_of(c), 0.0)
    torch.cuda.synchronize()
    at = torch.from_numpy(c.rows[0]).cuda()
    met = scores[:, at // c.page, :, at % c.page]
    assert torch.isfinite(met).all() and torch.isnan(scores).sum() == scores.numel() - met.numel()
    # a query head's weights over all tokens sum to one
    assert abs(float(met.double().sum()) - c.layers * c.n * c.heads) < 1e-3


@pytest.mark.parametrize("dim,dtype", [(128, BF16), (64, BF16), (64, F32), (80, BF16)])
def test_weigh_rows_that_see_nothing(dim, dtype):
    c = Case(dtype=dtype, head_dim=dim, prefixes=[0, 30], seed=3,
             requests=[(-1, 0, 2), (-1, 3, 5), (0, 0, 1), (0, 4, 1), (1, 2, 6), (1, 0, 3), (1, 10, 0), (-1, 0, 0), (-1, 17, 60), (1, 1, 1)])
    eu.check_weigh(c, scale_of(c))


@pytest.mark.parametrize("family,dim,dtype", [(GQA, 128, BF16), (GQA, 64, F32), (MLA, 64, BF16)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_weigh_ignores_what_is_unseen(family, dim, dtype, bad):
    more = dict(heads=4, kv_heads=2, head_dim=dim) if family == GQA else dict(family=MLA, heads=4, latent=512, rope=dim)
    c = Case(dtype=dtype, garbage=bad, prefixes=[35], requests=[(0, 20, 4), (-1, 70, 40), (0, 3, 1), (0, 150, 130)], seed=9, **more)
    lse, before, a = eu.check_weigh(c, scale_of(c))
    # a query that is not finite spoils the keys it sees and no others
    c.q[:, 3] = bad  # (request 0's last; with an lse of NaN)
    lse[:, 3] = float("nan")
    b = before.clone()
    eu.weigh(c, lse, b, scale_of(c))
    torch.cuda.synchronize()
    seen = torch.zeros(c.pages * c.page, dtype=torch.bool, device="cuda")
    seen[torch.from_numpy(np.concatenate([c.rows[0], c.rows[1]])).cuda()] = True
    seen = seen.view(c.pages, 1, c.page).expand(-1, c.hkv, -1)
    assert torch.isnan(b[:, seen]).all() and torch.equal(b[:, ~seen], a[:, ~seen])


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_weigh_strides_and_alignment(dtype):
    for shift, offset, pad in ((8, 0, 0), (1, 0, 0), (0, 1, 0), (0, 0, 5)):
        c = Case(dtype=dtype, head_dim=64, heads=8, kv_heads=4, prefixes=[50], requests=[(0, 30, 2), (-1, 60, 33)], offset=offset, pad_layer=pad, seed=shift)
        lse, before, want = eu.check_weigh(c, scale_of(c))
        s = c.step(step.WEIGH)
        plan = step.upload(c.lay, s, c.pool, c.workspace(s))
        q = torch.full((c.n, 8 * 64 + 40), 9.0, dtype=TYPES[dtype], device="cuda")
        q[:, shift:shift + 512] = c.q[1]
        got = before[1].clone()
        step.weigh(plan, 1, q[:, shift:shift + 512], lse[1], got, scale_of(c))
        torch.cuda.synchronize()
        assert torch.equal(got, want[1])


# ------------------------------------------------------------------ eviction
LAYOUTS = [dict(kv_heads=2, head_dim=64), dict(kv_heads=4, head_dim=128), dict(kv_heads=1, head_dim=10), dict(kv_heads=3, head_dim=2),
           dict(family=MLA, latent=512, rope=64), dict(family=MLA, latent=0, rope=2), dict(family=MLA, latent=20, rope=6), dict(kv_heads=1, head_dim=512)]
SEQS = [(100, 40, 4, 10), (5, 3, 0, 0), (0, 0, 0, 0), (33, 33, 9, 9), (17, 0, 0, 0), (1, 4, 3, 3), (64, 63, 0, 1), (200, 20, 20, 0), (200, 20, 0, 20), (130, 129, 50, 79), (2, 1, 0, 0)]


@pytest.mark.parametrize("kw", LAYOUTS)
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("reanchor", [False, True])
def test_evict_layouts(kw, dtype, reanchor):
    Cache(seqs=SEQS, dtype=dtype, reanchor=reanchor, **kw).check()


@pytest.mark.parametrize("together", [1, 2, 4])
@pytest.mark.parametrize("reanchor", [False, True])
def test_evict_heads_together(together, reanchor):
    Cache(seqs=SEQS, kv_heads=4, head_dim=64, together=together, reanchor=reanchor, seed=together).check()


@pytest.mark.parametrize("page", [1, 3, 8, 64, 256])
def test_evict_page_sizes(page):
    Cache(seqs=SEQS, page=page, seed=page).check()


@pytest.mark.parametrize("n", [2, 63, 64, 65, 511, 512, 513, 2047, 2048, 2049, 5000])
@pytest.mark.parametrize("share", [0.02, 0.5, 0.97])
def test_evict_lengths(n, share):
    keep = max(1, int(n * share))
    Cache(seqs=[(n, keep, min(keep, 2), 0), (n, keep, 0, min(keep, 7))], layers=1, reanchor=n % 2 == 1, seed=n).check()


def test_evict_a_long_sequence():
    Cache(seqs=[(70000, 30000, 4, 64)], layers=1, kv_heads=1, head_dim=64, reanchor=True).check()


@pytest.mark.parametrize("together", [1, 2])
def test_evict_ties_go_to_the_lowest_tokens(together):
    Cache(seqs=SEQS + [(3000, 1000, 0, 0)], ties=True, together=together).check()


def test_evict_scores_of_every_kind():
    """Infinities, NaN (lowest), zeros of both signs, denormal numbers, equal scores throughout."""
    c = Cache(seqs=[(600, 250, 3, 5), (300, 100, 0, 0), (300, 100, 0, 0)], layers=1)
    values = torch.tensor([0.0, -0.0, float("inf"), float("-inf"), float("nan"), 1e-42, -1e-42, 1.0, -1.0, 3e38], device="cuda")
    for h in range(c.hkv):
        s = c.scores(0)
        at = torch.from_numpy(c.rows[0]).cuda()
        s[at // 16, h, at % 16] = values[torch.randint(0, 10, (600,), generator=torch.Generator().manual_seed(h)).cuda()]
        for i, x in ((1, float("nan")), (2, 0.25)):
            at = torch.from_numpy(c.rows[i]).cuda()
            s[at // 16, h, at % 16] = x
    c.check()


def test_evict_without_a_list_and_off_the_grid():
    Cache(seqs=SEQS, pad_layer=5, pad_scores=3, offset=1).check(kept=False)
    Cache(seqs=SEQS, pad_layer=8, pad_scores=1, dtype=F32, pairing=abi.GPTJ, reanchor=True).check(kept=False)
    Cache(seqs=SEQS, pad_layer=64, pairing=abi.GPTJ, reanchor=True, kv_heads=2, head_dim=128).check()
    Cache(seqs=[]).check()
    Cache(seqs=[(30, 30, 0, 0)]).check()


def test_evict_moves_rows_of_every_layer_of_a_deep_pool():
    Cache(seqs=[(300, 100, 4, 32), (1000, 500, 0, 0)], layers=30, kv_heads=4, head_dim=128, reanchor=True).check()
