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


@pytest.mark.parametrize("queries", [1, 17, 300])
@pytest.mark.parametrize("family,dim,dtype", [(GQA, 128, BF16), (GQA, 64, F32), (MLA, 64, BF16)])
def test_weigh_scores_of_appended_tokens_start_at_zero(queries, family, dim, dtype):
    more = dict(heads=14, kv_heads=2, head_dim=dim) if family == GQA else dict(family=MLA, heads=16, latent=512, rope=dim)
    c = Case(dtype=dtype, layers=1, prefixes=[100], requests=[(0, queries + 40, queries), (0, 300, 1), (-1, queries, queries)], **more)
    lse = torch.stack([eu.own_lse(c, 0, scale_of(c))])
    before = eu.new_scores(c)
    after, zeroed = before.clone(), before.clone()
    for r, (_, own, nq, _) in enumerate(c.requests):
        at = torch.from_numpy(c.rows[1 + r][own - nq:]).cuda()
        zeroed[0, at // c.page, :, at % c.page] = 0
        before[0, at // c.page, :, at % c.page] = float("nan")
        after[0, at // c.page, :, at % c.page] = float("nan")
    eu.weigh(c, lse, after, scale_of(c), 0.5, flags=step.APPEND)
    eu.weigh(c, lse, zeroed, scale_of(c), 0.5)
    torch.cuda.synchronize()
    assert torch.equal(after, zeroed)


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


# ------------------------------------------------------------------ together, and as programs use them
@pytest.mark.parametrize("diff", [False, True])
def test_a_cache_that_stays_within_its_budget(diff):
    """Decode steps that append, attend and weigh; evictions between them; the rest goes on at consecutive positions."""
    from oracle import evict_oracle as eo
    from oracle import step_oracle as so
    from tests.step_util import HALF
    torch.manual_seed(1)
    rng = np.random.default_rng(1)
    layers, heads, hkv, d, page, pages, base, n = 2, 8, 4, 64, 16, 64, 1e4, 3
    F, together = hkv * d, 2 if diff else 1
    lay = abi.make_layout(GQA, BF16, layers, num_kv_heads=hkv, head_dim=d, rope_base=base, page_size=page)
    k, v = (torch.zeros(layers, pages, page, F, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    scores = torch.zeros(layers, pages, hkv, page, device="cuda")
    pool = abi.make_pool(k, v, pages)
    tables = rng.permutation(pages)[:n * 8].astype(np.int32).reshape(n, 8)
    start = 100 * np.arange(n)
    flags = step.APPEND | step.ATTEND | step.WEIGH | (step.DIFFERENTIAL if diff else 0)
    s = step.Step(num_q_heads=heads, block_tables=tables, num_tokens=0, num_queries=0, slot0=[3, 0, 15], position0=start, flags=flags)
    raw = [[[] for _ in range(n)] for _ in range(layers)]  # keys as they came: [layer][request][token]
    alive = [[[list() for _ in range(hkv // together)] for _ in range(n)] for _ in range(layers)]  # raw numbers of the tokens that a group holds
    weights = [[np.zeros((hkv, 0)) for _ in range(n)] for _ in range(layers)]
    scale, budget = d ** -0.5, 40

    def rows_of(r):
        return so.slots(tables[r], int(s.requests["slot0"][r]), int(s.requests["num_tokens"][r]), page)

    def decode(queries):
        s.requests["num_tokens"] += queries
        s.requests["num_queries"] = queries
        ws = torch.empty(step.workspace_bytes(lay, s), dtype=torch.uint8, device="cuda")
        plan = step.upload(lay, s, pool, ws)
        total = plan.num_tokens
        for layer in range(layers):
            q, kk, vv = (torch.randn(total, w, device="cuda").bfloat16() for w in (heads * d, F, F))
            out, lse = torch.empty(total, heads * d, dtype=torch.bfloat16, device="cuda"), torch.empty(total, heads, device="cuda")
            step.append(plan, layer, q=q, q_out=q, k=kk, v=vv)
            if diff:
                step.attend_diff(plan, layer, q, out, scale, lambda_init=0.4, lse=lse, norm=False)
            else:
                step.attend(plan, layer, q, out, scale, lse=lse)
            step.weigh(plan, layer, q, lse, scores[layer], scale)
            torch.cuda.synchronize()
            at0, ks, vs, qs, zs, got = 0, eu.host(k[layer]).reshape(-1, F), eu.host(v[layer]).reshape(-1, F), eu.host(q), eu.host(lse), eu.host(out)
            for r in range(n):
                m, at = int(queries[r]), rows_of(r)
                mine = slice(at0, at0 + m)
                last = at.size - m + np.arange(m)
                raw[layer][r] += list(eu.host(kk[mine]))
                weights[layer][r] = np.concatenate([weights[layer][r], np.zeros((hkv, m))], 1)
                for g in alive[layer][r]:
                    g += range(len(raw[layer][r]) - m, len(raw[layer][r]))
                for h in range(hkv):
                    hs = h // 2 * 4 + h % 2 + 2 * np.arange(2) if diff else h * 2 + np.arange(2)
                    qh = qs[mine].reshape(m, heads, d)[:, hs]
                    keys, pair = ks[at, h * d:(h + 1) * d], h // 2 * 2 * d
                    o, z, a, _ = so.attend(qh, keys, vs[at, pair:pair + 2 * d] if diff else vs[at, h * d:(h + 1) * d], scale, last)
                    assert np.abs(zs[mine][:, hs] - z).max() < 1e-4
                    if not diff:
                        assert (np.abs(got[mine].reshape(m, heads, d)[:, hs] - o) <= 2 ** -7 * (a + np.abs(o)) + 1e-6).all()
                    weights[layer][r][h] += eo.weights(qh, keys, zs[mine][:, hs], scale, last)[0]
                    # keys stand at consecutive positions, whatever was evicted before them: the raw key turned there at once,
                    # but for the append's and (at most three) evictions' roundings. Each moves a pair by at most half a
                    # step of its length, which turns keep; fp32's own errors are far below a tenth of that.
                    came = np.array(raw[layer][r])[alive[layer][r][h // together], h * d:(h + 1) * d]
                    y, _ = so.rotate(came, so.phases(start[r] + np.arange(at.size), d, base))
                    length = np.tile(np.hypot(y[:, :d // 2], y[:, d // 2:]), 2)
                    assert (np.abs(keys - y) <= 4 * HALF[BF16] * 1.1 * length + 1e-6).all()
                at0 += m

    def evict():
        had = s.requests["num_tokens"].copy()
        keep = np.minimum(had, budget)
        e = step.Eviction(block_tables=tables, slot0=s.requests["slot0"], num_tokens=had, keep=keep, first=2, last=8, heads_together=together,
                          flags=step.REANCHOR)
        kept = torch.empty(layers, hkv // together, int(keep.sum()), dtype=torch.int32, device="cuda")
        step.evict(lay, pool, e, scores, torch.empty(step.evict_workspace_bytes(lay, e), dtype=torch.uint8, device="cuda"), kept=kept)
        before = scores.clone()
        torch.cuda.synchronize()
        at0 = 0
        for r in range(n):
            for layer in range(layers):
                for g in range(hkv // together):
                    stay = kept[layer, g, at0:at0 + keep[r]].cpu().numpy()
                    w = weights[layer][r][g * together:(g + 1) * together]
                    if had[r] > budget:  # the choice, within the weights' own errors
                        total = w.sum(0)
                        gone = np.setdiff1d(np.arange(had[r]), stay)
                        middle = stay[(stay >= 2) & (stay < had[r] - 8)]
                        assert set(range(2)) | set(range(had[r] - 8, had[r])) <= set(stay.tolist()) and total[middle].min() >= total[gone].max() - 1e-4
                    alive[layer][r][g] = [alive[layer][r][g][t] for t in stay]
                    if g == 0:
                        new = np.zeros((hkv, keep[r]))
                    new[g * together:(g + 1) * together] = w[:, stay]
                    if g == hkv // together - 1:
                        weights[layer][r] = new
                at = torch.from_numpy(so.slots(tables[r], int(s.requests["slot0"][r]), int(keep[r]), page)).cuda()
                off = np.abs(eu.host(before[layer, at // page, :, at % page]).T - weights[layer][r])
                assert off.max() < 1e-4, np.argwhere(off >= 1e-4)[:5]
            at0 += keep[r]
        s.requests["num_tokens"] = keep

    decode(np.array([50, 33, 1]))
    evict()
    for _ in range(3):
        decode(np.array([1, 1, 1]))
    evict()
    decode(np.array([9, 20, 45]))
    evict()
    decode(np.array([1, 2, 1]))


@pytest.mark.parametrize("family,dim", [(GQA, 128), (GQA, 64), (MLA, 64)])
def test_launches_in_a_captured_graph(family, dim):
    """Weighing (ranges of rows joined) and differential attention (parts joined), replayed between eager work."""
    more = dict(heads=8, kv_heads=2, head_dim=dim) if family == GQA else dict(family=MLA, heads=8, latent=512, rope=dim)
    c = Case(layers=1, prefixes=[3000], requests=[(0, 200, 190), (0, 40, 1), (0, 3, 1)], **more)
    diff, scale = family == GQA, scale_of(c)
    flags = step.WEIGH | ((step.ATTEND | step.DIFFERENTIAL) if diff else 0)
    s = c.step(flags)
    ws = c.workspace(s)
    p = Params(c) if diff else None
    lse = eu.own_lse(c, 0, scale, diff)
    first = eu.new_scores(c)
    scores = first.clone()
    out = torch.zeros(c.n, c.heads * c.dk, dtype=torch.bfloat16, device="cuda")
    z = torch.zeros_like(lse)
    plan = step.upload(c.lay, s, c.pool, ws)

    def launch():
        step.weigh(plan, 0, c.q[0], lse, scores[0], scale, 0.5)
        if diff:
            step.attend_diff(plan, 0, c.q[0], out, scale, lse=z, **p.kwargs())
    launch()
    torch.cuda.synchronize()
    want = (scores.clone(), out.clone(), z.clone())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            launch()
    for _ in range(4):
        scores.copy_(first)
        if diff:
            out.fill_(3)
            z.fill_(3)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(scores, want[0]) and torch.equal(out, want[1]) and torch.equal(z, want[2])
        scores.copy_(first)
        launch()  # eager, in the same workspace
        torch.cuda.synchronize()
        assert torch.equal(scores, want[0]) and torch.equal(out, want[1])


def test_evictions_from_a_capturing_stream_are_refused():
    c = Cache(seqs=[(100, 40, 0, 0)])
    e = c.eviction()
    ws = torch.empty(step.evict_workspace_bytes(c.lay, e), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    x = torch.zeros(4, device="cuda")
    with torch.cuda.graph(graph):
        x.add_(1)
        with pytest.raises(abi.KameraError) as err:
            step.evict(c.lay, c.pool, e, c.scores_flat, ws, scores_stride=c.scores_stride)
    assert err.value.name == "KAMERA_E_UNSUPPORTED"
    torch.cuda.synchronize()
    c.check()


def test_on_another_stream():
    side = torch.cuda.Stream()
    c = Case(head_dim=128, heads=8, kv_heads=2, prefixes=[200], requests=[(0, 60, 40), (0, 9, 1)])
    torch.cuda.synchronize()
    eu.check_diff(c, Params(c), scale_of(c), stream=side)
    with torch.cuda.stream(side):
        eu.check_weigh(c, scale_of(c))
        Cache(seqs=SEQS, reanchor=True).check()


@pytest.mark.parametrize("heads,kv,dim,dtype", [(16, 2, 128, BF16), (8, 2, 64, BF16), (8, 2, 64, F32)])
def test_plans_that_fit_a_smaller_workspace(heads, kv, dim, dtype):
    """Fewer ranges, prefixes unshared, rows uncut: within the same bounds, and the same on every run."""
    c = Case(dtype=dtype, layers=1, heads=heads, kv_heads=kv, head_dim=dim, prefixes=[2500], requests=[(0, 100 + i, 1 + 30 * (i % 3 == 0)) for i in range(9)])
    p, scale = Params(c), scale_of(c)
    s = c.step(step.ATTEND | step.DIFFERENTIAL | step.WEIGH | step.FIT)
    full = step.workspace_bytes(c.lay, s)
    o, tol, z, ltol = eu.expect_diff(c, p, 0, scale)
    lse = eu.own_lse(c, 0, scale, True)
    before = eu.new_scores(c)
    want, wtol = eu.expect_weigh(c, 0, lse, before[0], scale, 1.0, True)
    size, sizes = full, 0
    while size > 1024:
        ws = torch.empty(size, dtype=torch.uint8, device="cuda")
        try:
            plan = step.upload(c.lay, s, c.pool, ws)
        except abi.KameraError as e:
            assert e.name == "KAMERA_E_WORKSPACE"
            break
        again = []
        for _ in range(2):
            out, stats, scores = torch.empty(c.n, heads * dim, dtype=TYPES[dtype], device="cuda"), torch.empty(c.n, heads, device="cuda"), before.clone()
            step.attend_diff(plan, 0, c.q[0], out, scale, lse=stats, **p.kwargs())
            step.weigh(plan, 0, c.q[0], lse, scores[0], scale)
            torch.cuda.synchronize()
            assert (np.abs(eu.host(out) - o) <= tol).all() and (np.abs(eu.host(stats) - z) <= ltol).all()
            assert (np.abs(eu.host(scores[0]) - want) <= wtol).all()
            again.append((out, stats, scores))
        assert all(torch.equal(a, b) for a, b in zip(*again))
        sizes += 1
        size = size // 2 // 256 * 256
    assert sizes >= 2


def test_scores_move_with_their_pages():
    """copy_pages and compact_pages under the scores' layout."""
    for kw in (dict(kv_heads=3, head_dim=64), dict(family=MLA, latent=512, rope=64)):
        c = Cache(seqs=[(100, 1, 0, 0), (70, 1, 0, 0)], page=8, **kw)
        lay = step.scores_layout(c.lay)
        scores = c.scores_flat.view(c.layers, c.pages, c.hkv, c.page)
        pool = abi.make_pool(scores, None, c.pages)
        ws = torch.empty(step.copy_pages_workspace_bytes(c.pages), dtype=torch.uint8, device="cuda")
        was = scores.clone()
        step.copy_pages(lay, pool, [0, 1, 2], [1, 2, 0], ws)
        torch.cuda.synchronize()
        assert torch.equal(scores[:, [1, 2, 0]], was[:, [0, 1, 2]]) and torch.equal(scores[:, 3:], was[:, 3:])
        was = scores.clone()
        tables = [t.copy() for t in c.tables]
        moved, live = [t.copy() for t in tables], step.compact_pages(lay, pool, tables, ws)
        assert live == step.compact_pages(c.lay, c.pool, moved, ws) and all((a == b).all() for a, b in zip(tables, moved))
        torch.cuda.synchronize()
        for new, old in zip(tables, c.tables):
            assert torch.equal(scores[:, torch.from_numpy(new).long().cuda()], was[:, torch.from_numpy(old).long().cuda()])


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_pools_beyond_32_bits(dtype):
    """Layers that start, and rows that lie, beyond 2^32 bytes of the pool."""
    pages, page, heads, kv, d, layers = 140000 if dtype == BF16 else 70000, 16, 8, 4, 128, 2
    F = kv * d
    lay = abi.make_layout(GQA, dtype, layers, num_kv_heads=kv, head_dim=d, page_size=page, rope_base=1e4)
    k, v = (torch.empty(layers, pages, page, F, dtype=TYPES[dtype], device="cuda") for _ in range(2))
    assert k[0].numel() * k.element_size() > 2 ** 31 and k.numel() * k.element_size() > 2 ** 32
    rng = np.random.default_rng(0)
    n = 300
    table = (pages - 1 - rng.permutation(100)[:19]).astype(np.int32)
    small = abi.make_layout(GQA, dtype, layers, num_kv_heads=kv, head_dim=d, page_size=page, rope_base=1e4)
    ks, vs = (torch.randn(layers, 19, page, F, device="cuda").to(TYPES[dtype]) for _ in range(2))
    at = torch.from_numpy(table.astype(np.int64)).cuda()
    k[:, at], v[:, at] = ks, vs
    scores = torch.empty(layers, pages, kv, page, device="cuda")
    scores[:, at] = torch.rand(layers, 19, kv, page, device="cuda")
    few = scores[:, at].clone()
    q = torch.randn(layers, 40, heads * d, device="cuda").to(TYPES[dtype])
    results = []
    for lay_, k_, v_, s_, t_, np_ in ((lay, k, v, scores, table, pages), (small, ks, vs, few, np.arange(19, dtype=np.int32), 19)):
        pool = abi.make_pool(k_, v_, np_)
        s = step.Step(num_q_heads=heads, block_tables=[t_], num_tokens=n, num_queries=40, slot0=1, flags=step.ATTEND | step.DIFFERENTIAL | step.WEIGH)
        plan = step.upload(lay_, s, pool, torch.empty(step.workspace_bytes(lay_, s), dtype=torch.uint8, device="cuda"))
        out, lse = torch.empty(layers, 40, heads * d, dtype=TYPES[dtype], device="cuda"), torch.empty(layers, 40, heads, device="cuda")
        for layer in range(layers):
            step.attend_diff(plan, layer, q[layer], out[layer], d ** -0.5, lambda_init=0.3, lse=lse[layer])
            step.weigh(plan, layer, q[layer], lse[layer], s_[layer], d ** -0.5)
        e = step.Eviction(block_tables=[t_], num_tokens=n, keep=100, slot0=1, last=7, flags=step.REANCHOR)
        kept = torch.empty(layers, kv, 100, dtype=torch.int32, device="cuda")
        step.evict(lay_, pool, e, s_, torch.empty(step.evict_workspace_bytes(lay_, e), dtype=torch.uint8, device="cuda"), kept=kept)
        torch.cuda.synchronize()
        rows = torch.from_numpy(t_.astype(np.int64)).cuda()
        results.append((out, lse, kept, k_[:, rows], v_[:, rows], s_[:, rows]))
    assert all(torch.equal(a, b) for a, b in zip(*results))


@pytest.mark.parametrize("dim,dtype", [(128, BF16), (64, BF16), (64, F32)])
def test_results_are_the_same_bits_on_every_run(dim, dtype):
    c = Case(dtype=dtype, head_dim=dim, heads=8, kv_heads=2, prefixes=[1500], requests=[(0, 5 + i, 1) for i in range(7)] + [(0, 300, 200)])
    p = Params(c)
    runs = [eu.attend_diff(c, p, scale_of(c)) for _ in range(3)]
    lse = torch.stack([eu.own_lse(c, layer, scale_of(c), True) for layer in range(c.layers)])
    for _ in range(3):
        scores = eu.new_scores(c)
        eu.weigh(c, lse, scores, scale_of(c), diff=True)
        runs.append((scores,))
    torch.cuda.synchronize()
    for a, b in ((runs[0], runs[1]), (runs[0], runs[2]), (runs[3], runs[4]), (runs[3], runs[5])):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_diff_of_more_tiles_than_places():
    """Whole tiles for whole rounds of workgroups and the last queries in pieces: runs that write their output
    themselves, runs that are joined, and a request that is both."""
    c = Case(layers=1, heads=128, kv_heads=8, head_dim=64, prefixes=[300], requests=[(0, 200, 200), (0, 333, 333), (0, 5, 1)])
    eu.check_diff(c, Params(c), scale_of(c))


@pytest.mark.parametrize("heads,dim,dtype", [(400, 64, BF16), (300, 128, BF16), (400, 64, F32)])
def test_more_heads_of_a_pair_than_rows_of_a_tile(heads, dim, dtype):
    """A token's rows fill several tiles; whole rounds of them do not end between tokens."""
    c = Case(dtype=dtype, layers=1, heads=heads, kv_heads=2, head_dim=dim, prefixes=[70], requests=[(0, 30, 1), (0, 150, 130), (0, 60, 59), (-1, 9, 9)])
    eu.check_diff(c, Params(c), scale_of(c))
    eu.check_weigh(c, scale_of(c), diff=True)


@pytest.mark.parametrize("family,heads,kv,dim", [(GQA, 1, 1, 64), (GQA, 1, 1, 128), (GQA, 2, 2, 64), (MLA, 1, 1, 64)])
def test_weigh_ranges_that_end_in_a_few_rows(family, heads, kv, dim):
    """4100 rows in ranges of 512 (latent ones: 128) leave a last range of 4, whose sums are joined like the others'."""
    more = dict(heads=heads, kv_heads=kv, head_dim=dim) if family == GQA else dict(family=MLA, heads=heads, latent=512, rope=dim)
    c = Case(layers=1, prefixes=[300], requests=[(0, 4100, 4100)], **more)
    eu.check_weigh(c, scale_of(c))


def test_two_callers_at_once():
    """Threads with a stream, workspaces and pools of their own."""
    import threading
    cases = [Case(head_dim=128, heads=8, kv_heads=2, prefixes=[500], requests=[(0, 30 + i, 1) for i in range(9)] + [(0, 200, 150)], seed=i) for i in range(3)]
    params = [Params(c, seed=i) for i, c in enumerate(cases)]
    lse = [torch.stack([eu.own_lse(c, layer, scale_of(c)) for layer in range(c.layers)]) for c in cases]
    caches = [[Cache(seqs=SEQS + [(3000, 1000 + i, 5, 7)], reanchor=True, seed=i) for _ in range(4)] for i in range(3)]

    def work(i, turn, stream):
        scores = eu.new_scores(cases[i])
        with torch.cuda.stream(stream):
            out = eu.attend_diff(cases[i], params[i], scale_of(cases[i]), stream=stream)
            eu.weigh(cases[i], lse[i], scores, scale_of(cases[i]), 0.5, stream=stream)
            cache = caches[i][turn]
            cache.run(stream=stream)
            stream.synchronize()
        return (*out, scores, cache.kept, cache.scores_flat, *cache.flat)

    alone = [work(i, 0, torch.cuda.Stream()) for i in range(3)]
    got, failed = {}, []

    def caller(i, stream):
        try:
            for turn in range(1, 4):
                got[i, turn] = work(i, turn, stream)
        except BaseException as e:  # (shown by the test's own thread)
            failed.append(e)

    torch.cuda.synchronize()
    threads = [threading.Thread(target=caller, args=(i, torch.cuda.Stream())) for i in range(3)]
    for x in threads:
        x.start()
    for x in threads:
        x.join()
    torch.cuda.synchronize()
    assert not failed, failed
    for (i, _), results in got.items():
        assert all(torch.equal(a, b) for a, b in zip(alone[i], results))
