"""The serving step on the GPU against its 64-bit oracle: append, attention, page copies."""
import numpy as np
import pytest
import torch

from oracle import step_oracle as so
from position_free_kv_amd import abi, step
from tests.step_util import E32, HALF, TYPES, Case

pytestmark = pytest.mark.gpu

ALL = step.REQUEST_ALL
GQA, MLA, BF16, F32 = abi.GQA, abi.MLA, abi.BF16, abi.F32

HEADS = [  # query heads, KV heads, head width
    (8, 2, 64), (8, 2, 128), (7, 1, 128), (4, 4, 128), (3, 3, 64), (40, 2, 64), (6, 2, 80), (2, 2, 10), (4, 2, 256), (2, 1, 512)]


def scale_of(c):
    return 1.0 / float(np.sqrt(c.dk))


# ------------------------------------------------------------------ attention
@pytest.mark.parametrize("heads,kv,dim", HEADS)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_attend_layouts(heads, kv, dim, dtype):
    """A shared prefix, own tokens of several lengths, one and several queries."""
    c = Case(dtype=dtype, heads=heads, kv_heads=kv, head_dim=dim, prefixes=[77], seed=heads + dim,
             requests=[(0, 1, 1), (0, 33, 1), (0, 16, 5), (-1, 40, 3), (0, 0, 1)])
    c.check_attend(scale_of(c))


@pytest.mark.parametrize("heads,latent,rope", [(16, 512, 64), (3, 20, 6), (1, 64, 64), (40, 512, 64), (5, 128, 64), (2, 512, 512)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_attend_latent_rows(heads, latent, rope, dtype):
    c = Case(family=MLA, dtype=dtype, heads=heads, latent=latent, rope=rope, prefixes=[50], seed=latent + heads,
             requests=[(0, 1, 1), (0, 70, 2), (0, 16, 1), (-1, 19, 3)])
    c.check_attend(scale_of(c))


@pytest.mark.parametrize("page", [1, 3, 8, 16, 64, 256])
@pytest.mark.parametrize("dim", [64, 128])
def test_attend_page_sizes(page, dim):
    c = Case(head_dim=dim, page=page, prefixes=[130], requests=[(0, 21, 1), (0, 64, 2), (0, 5, 1)], seed=page)
    c.check_attend(scale_of(c))


@pytest.mark.parametrize("tokens", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 257, 1000, 4097])
@pytest.mark.parametrize("family,dim", [(GQA, 128), (GQA, 64), (MLA, 64)])
def test_attend_lengths(tokens, family, dim):
    """Every length around a tile's end, as own tokens and as prefix."""
    more = dict(heads=8, kv_heads=2, head_dim=dim) if family == GQA else dict(family=MLA, heads=4, latent=512, rope=dim)
    c = Case(layers=1, prefixes=[tokens], requests=[(-1, tokens, 1), (0, 3, 1), (0, 2, 1)], seed=tokens, **more)
    c.check_attend(scale_of(c))


@pytest.mark.parametrize("queries", [2, 7, 16, 33, 64, 65, 128, 129, 300])
@pytest.mark.parametrize("dim,dtype", [(128, BF16), (64, BF16), (64, F32), (48, BF16)])
def test_attend_many_queries(queries, dim, dtype):
    """Causal edges inside and between tiles; requests that share and that read the prefix themselves."""
    c = Case(dtype=dtype, layers=1, heads=6, kv_heads=2, head_dim=dim, prefixes=[150, 40], seed=queries,
             requests=[(0, queries, queries), (0, queries + 37, queries), (1, queries + 1, 3), (0, 9, 2), (-1, queries, queries)])
    c.check_attend(scale_of(c))


def test_attend_many_queries_on_latent_rows():
    c = Case(family=MLA, layers=1, heads=16, latent=512, rope=64, prefixes=[90], requests=[(0, 50, 33), (0, 70, 70), (-1, 20, 20), (0, 1, 1)])
    c.check_attend(scale_of(c))


@pytest.mark.parametrize("dim,dtype", [(128, BF16), (64, F32)])
def test_attend_requests_that_see_all(dim, dtype):
    c = Case(dtype=dtype, head_dim=dim, prefixes=[60], requests=[(0, 40, 40, ALL), (-1, 33, 12, ALL), (0, 20, 1, ALL), (0, 90, 50)])
    c.check_attend(scale_of(c))


@pytest.mark.parametrize("dim,dtype", [(128, BF16), (64, BF16), (64, F32), (80, BF16)])
def test_attend_rows_that_see_nothing(dim, dtype):
    """No keys at all, more queries than own tokens, empty prefixes, requests without queries: zeros, -inf."""
    c = Case(dtype=dtype, head_dim=dim, prefixes=[0, 30], seed=3,
             requests=[(-1, 0, 2), (-1, 3, 5), (0, 0, 1), (0, 4, 1), (1, 2, 6), (1, 0, 3), (1, 10, 0), (-1, 0, 0), (-1, 17, 60), (1, 1, 1)])
    out, lse = c.check_attend(scale_of(c))
    assert (out[:, :2] == 0).all() and torch.isneginf(lse[:, :2]).all()


@pytest.mark.parametrize("dim,dtype", [(128, BF16), (64, BF16), (64, F32), (80, BF16)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_attend_ignores_what_is_unseen(dim, dtype, bad):
    """Unused slots, and tokens later than a query, may hold anything, in keys and in values."""
    c = Case(dtype=dtype, head_dim=dim, garbage=bad, prefixes=[35], requests=[(0, 20, 4), (-1, 70, 40), (0, 3, 1), (0, 150, 130)], seed=9)
    o0, z0 = c.check_attend(scale_of(c))
    first = 0
    for r, (pre, own, nq, _) in enumerate(c.requests):  # spoil each request's last token: only its last query sees it
        for p in c.pools:
            p[:, int(c.rows[1 + r][-1])] = bad
        first += nq
    o1, z1 = c.attend(scale_of(c))
    torch.cuda.synchronize()
    keep = torch.ones(c.n, dtype=torch.bool, device="cuda")
    keep[torch.cumsum(torch.tensor([r[2] for r in c.requests]), 0) - 1] = False
    assert torch.equal(o0[:, keep], o1[:, keep]) and torch.equal(z0[:, keep], z1[:, keep])


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("heads", [4, 16, 40])
def test_attend_on_latent_rows_ignores_what_is_unseen(heads, bad):
    c = Case(family=MLA, heads=heads, latent=512, rope=64, garbage=bad, prefixes=[35], seed=9,
             requests=[(0, 20, 4), (-1, 70, 40), (0, 3, 1), (0, 50, 30), (-1, 3, 5)])
    o0, z0 = c.check_attend(scale_of(c))
    for r in range(len(c.requests)):  # each request's last token: only its last query sees it
        c.pools[0][:, int(c.rows[1 + r][-1])] = bad
    o1, z1 = c.attend(scale_of(c))
    torch.cuda.synchronize()
    keep = torch.ones(c.n, dtype=torch.bool, device="cuda")
    keep[torch.cumsum(torch.tensor([r[2] for r in c.requests]), 0) - 1] = False
    assert torch.equal(o0[:, keep], o1[:, keep]) and torch.equal(z0[:, keep], z1[:, keep])


@pytest.mark.parametrize("heads,dim,family", [(8, 128, GQA), (8, 64, GQA), (16, 64, MLA), (48, 64, MLA)])
def test_attend_splits_long_keys(heads, dim, family):
    """Few rows over many keys: split over workgroups and joined, own tokens and prefix alike."""
    more = dict(heads=heads, kv_heads=1, head_dim=dim) if family == GQA else dict(family=MLA, heads=heads, latent=512, rope=dim)
    c = Case(layers=1, prefixes=[9000, 700], requests=[(0, 1, 1), (0, 5000, 1), (1, 20, 1), (-1, 7001, 3), (1, 3, 2)], seed=dim, **more)
    c.check_attend(scale_of(c))
    c.check_attend(-scale_of(c))
    c.check_attend(0.0)


@pytest.mark.parametrize("heads,dim,family", [(4, 128, GQA), (4, 64, GQA), (16, 64, MLA)])
@pytest.mark.parametrize("members", [2, 5, 8, 9, 16, 17, 40])
def test_attend_tiles_of_every_size_over_long_prefixes(heads, dim, family, members):
    """A prefix of many stages a workgroup, its members' rows filling each kind of tile."""
    more = dict(heads=heads, kv_heads=1, head_dim=dim) if family == GQA else dict(family=MLA, heads=heads, latent=512, rope=dim)
    c = Case(layers=1, prefixes=[20000], requests=[(0, 1 + i % 3, 1) for i in range(members)], seed=members, **more)
    c.q *= 4  # a few keys stand out: a lost or doubled stage shows
    c.check_attend(scale_of(c))


@pytest.mark.parametrize("latent,rope", [(260, 4), (300, 8), (512, 64), (516, 4), (1000, 24)])
@pytest.mark.parametrize("tokens", [150, 400, 900, 6000])
def test_attend_joins_rows_wider_than_a_workgroups_share(latent, rope, tokens):
    """Rows of 65 to 250 pieces of 16 bytes, joined from few parts and from many."""
    for dtype in (BF16, F32):
        c = Case(family=MLA, dtype=dtype, heads=3, latent=latent, rope=rope, layers=1, prefixes=[tokens, tokens // 2], seed=latent + tokens,
                 requests=[(0, 1, 1), (0, tokens, 1), (1, 5, 1), (-1, tokens + 1, 2)])
        c.check_attend(scale_of(c))


@pytest.mark.parametrize("heads,queries", [(8, 11), (8, 12), (5, 19), (5, 20), (97, 1)])
@pytest.mark.parametrize("family", [GQA, MLA])
def test_attend_rows_around_the_limit_of_sharing(heads, queries, family):
    """Requests that just share their prefix's reads beside ones that just do not."""
    more = dict(heads=heads, kv_heads=1, head_dim=128) if family == GQA else dict(family=MLA, heads=heads, latent=512, rope=64)
    c = Case(layers=1, prefixes=[1500], seed=heads + queries, **more,
             requests=[(0, queries, queries), (0, queries + 40, queries), (0, queries + 3, queries + 1), (0, 200, max(queries - 1, 1))])
    c.check_attend(scale_of(c))


@pytest.mark.parametrize("dim,dtype", [(128, BF16), (64, F32), (10, BF16)])
def test_attend_scores_of_every_size(dim, dtype):
    """Scores of thousands, equal scores, scores of the type's lowest value."""
    c = Case(dtype=dtype, layers=1, head_dim=dim, prefixes=[100], requests=[(0, 30, 2), (0, 1, 1)], seed=21)
    c.q *= 30
    c.check_attend(scale_of(c) * 4)
    c.q.zero_()
    c.check_attend(scale_of(c))
    c.pools[0].nan_to_num_(0.0)
    c.pools[0][...] = -1.0
    c.q.fill_(torch.finfo(TYPES[dtype]).max / 4)
    out, lse = c.attend(1.0)  # every score is -inf: nothing to weigh
    torch.cuda.synchronize()
    assert (out == 0).all() and torch.isneginf(lse).all()


def test_attend_strides_offsets_and_null_lse():
    """Queries and outputs inside wider rows, pools off the 16-byte grid, layers padded apart."""
    for off, pad in ((0, 64), (1, 0), (8, 24), (4, 3)):
        c = Case(head_dim=128, heads=4, kv_heads=2, prefixes=[50], requests=[(0, 20, 3), (0, 5, 1)], offset=off, pad_layer=pad, seed=off)
        want, _ = c.check_attend(scale_of(c))
        s = c.step(step.ATTEND)
        plan = step.upload(c.lay, s, c.pool, c.workspace(s))
        for shift in (0, 1, 8):
            wide = torch.zeros(c.n, c.heads * c.dk + 40, dtype=torch.bfloat16, device="cuda")
            wide[:, shift:shift + c.heads * c.dk] = c.q[1]
            out = torch.full((c.n, c.heads * c.dv + 24), 5.0, dtype=torch.bfloat16, device="cuda")
            step.attend(plan, 1, wide[:, shift:shift + c.heads * c.dk], out[:, 8:], scale_of(c), out_stride=out.stride(0))
            torch.cuda.synchronize()
            assert (out[:, :8] == 5).all() and (out[:, 8 + c.heads * c.dv:] == 5).all()
            got = out[:, 8:8 + c.heads * c.dv].double().cpu().numpy()
            o, tol, _, _ = c.expect_attend(1, scale_of(c))
            assert (np.abs(got - o) <= tol).all()


def test_attend_offsets_beyond_32_bits():
    """Pool layers of more than 2^31 elements and byte offsets beyond 2^32, the rows in use at their end."""
    P, F, pages = 16, 1024, 140000
    lay = abi.make_layout(GQA, BF16, 1, num_kv_heads=8, head_dim=128, page_size=P)
    pools = [torch.empty(pages, P, F, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    table = np.array([139999, 5, 139000, 131072], np.int32)
    for p in pools:
        p[torch.from_numpy(table).long().cuda()] = torch.randn(4, P, F, device="cuda").bfloat16()
    q = torch.randn(2, 8 * 128, device="cuda").bfloat16()
    out = torch.empty_like(q)
    s = step.Step(num_q_heads=8, block_tables=[table[:2], table[2:]], num_tokens=[30, 31], num_queries=1, flags=step.ATTEND)
    ws = torch.empty(step.workspace_bytes(lay, s), dtype=torch.uint8, device="cuda")
    plan = step.upload(lay, s, abi.make_pool(*pools, pages), ws)
    step.attend(plan, 0, q, out, 0.1)
    for i, n in enumerate((30, 31)):
        k, v = (p[torch.from_numpy(table[2 * i:2 * i + 2]).long().cuda()].double().cpu().numpy().reshape(32, 8, 128)[:n] for p in pools)
        for h in range(8):
            qi = q[i, h * 128:(h + 1) * 128].double().cpu().numpy()[None, None]
            o, _, a, terms = so.attend(qi, k[:, h], v[:, h], 0.1, [n - 1])
            tol = (2 * 136 * E32 * terms[..., None] + 200 * E32 + HALF[BF16]) * (a + np.abs(o)) + HALF[BF16] * np.abs(o)
            assert (np.abs(out[i, h * 128:(h + 1) * 128].double().cpu().numpy() - o[0, 0]) <= tol[0, 0]).all()


def test_attend_is_the_same_on_every_run_stream_and_in_a_graph():
    c = Case(head_dim=128, heads=8, kv_heads=2, prefixes=[900], requests=[(0, 40, 1), (0, 3, 2), (0, 100, 30), (-1, 300, 1)], seed=2)
    want, z = c.check_attend(scale_of(c))
    for _ in range(3):
        out, lse = c.attend(scale_of(c))
        assert torch.equal(out, want) and torch.equal(lse, z)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out, lse = c.attend(scale_of(c), stream=side)
    side.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, z)
    s = c.step(step.ATTEND)
    ws = c.workspace(s)
    plan = step.upload(c.lay, s, c.pool, ws)
    out = torch.zeros_like(want)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for layer in range(c.layers):
            step.attend(plan, layer, c.q[layer], out[layer], scale_of(c))
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        c.attend(scale_of(c))  # eager work in between
        torch.cuda.synchronize()


# ------------------------------------------------------------------ append
def expect_append(c, q, k, v, qw, kw, eps, positions):
    """Per layer: (q, tolerance, K rows, tolerance, V rows) in 64 bits."""
    phi = so.phases(positions, c.d_rot, c.base, c.sections)
    gptj = c.pairing == abi.GPTJ
    band = c.latent

    def run(x, heads, w):
        x = x.double().cpu().numpy().reshape(c.n, heads, c.dk)
        # A norm's factor: dk squares and their sum, a quotient and a root, two products; each
        # term of a rotation: cos/sin rounded, a product, a sum: fp32 roundings of the terms.
        steps = 16.0
        if w is not None:
            w = w.double().cpu().numpy()
            steps += c.dk / 2 + 8
            x = np.concatenate([so.norm(x[..., :w.size], w, eps), x[..., w.size:]], -1)
        y, terms = x.copy(), np.abs(x)
        y[..., band:], terms[..., band:] = so.rotate(x[..., band:], phi, gptj)
        tol = HALF[c.dtype] * np.abs(y) + steps * E32 * terms * 1.01 + 1e-38
        return y.reshape(c.n, -1), tol.reshape(c.n, -1)

    return (*(run(q, c.heads, qw) if q is not None else (None, None)), *run(k, c.hkv, kw), v)


def check_append(c, norm, sections=False, slack=0, inplace=False, with_q=True, stream=None, fused=True, eps=1e-6):
    width = (c.heads * c.dk if with_q else 0) + c.F * len(c.pools)
    rows = c.draw(c.layers, c.n, width + slack).cuda()
    nq = c.heads * c.dk if with_q else 0
    parts = [rows[:, :, :nq], rows[:, :, nq:nq + c.F], rows[:, :, nq + c.F:nq + 2 * c.F]]
    if not fused:
        parts = [p.contiguous() for p in parts]
    wn = c.latent if c.family == MLA else c.dk
    qw = (1 + 0.3 * c.draw(c.dk).float()).to(rows.dtype).cuda() if norm and c.family == GQA and with_q else None
    kw = (1 + 0.3 * c.draw(wn).float()).to(rows.dtype).cuda() if norm and wn else None
    pos3 = torch.from_numpy(c.rng.integers(-70000, 70000, (c.n, 3)).astype(np.int32)).cuda() if sections else None
    start = c.rng.integers(-1000, 100000, len(c.requests))
    s = c.step(step.APPEND, position0=start, positions=pos3)
    flat = np.concatenate([st + own - nq_ + np.arange(nq_) for st, (_, own, nq_, _) in zip(start, c.requests)])
    positions = pos3.cpu().numpy() if sections else flat
    before = [f.clone() for f in c.flat]
    plan = step.upload(c.lay, s, c.pool, c.workspace(s), stream=stream)
    qin = parts[0].clone()
    q_out = torch.full((c.layers, c.n, nq + 8), 3.0, dtype=rows.dtype, device="cuda")[:, :, :nq]
    keep = [p.clone() for p in parts]
    for layer in range(c.layers):
        qo = parts[0][layer] if inplace else q_out[layer]
        step.append(plan, layer, q=parts[0][layer] if with_q else None, q_out=qo if with_q else None, k=parts[1][layer],
                    v=parts[2][layer] if c.family == GQA else None, q_weight=qw, k_weight=kw, eps=eps, stream=stream)
    torch.cuda.synchronize()
    np_ = len(c.prefix_tokens)
    slots = np.concatenate([c.rows[np_ + r][own - nq_:own] for r, (_, own, nq_, _) in enumerate(c.requests)])
    at = torch.from_numpy(slots).cuda()
    for layer in range(c.layers):
        q, qt, k, kt, v = expect_append(c, keep[0][layer] if with_q else None, keep[1][layer], keep[2][layer], qw, kw, eps, positions)
        if with_q:
            got = (parts[0] if inplace else q_out)[layer].double().cpu().numpy()
            assert (np.abs(got - q) <= qt).all(), (layer, np.argwhere(np.abs(got - q) > qt)[:3])
        got = c.pools[0][layer, at].double().cpu().numpy()
        assert (np.abs(got - k) <= kt).all(), (layer, np.argwhere(np.abs(got - k) > kt)[:3])
        if c.family == GQA:
            assert torch.equal(c.pools[1][layer, at], v)
    for p, f, b in zip(c.pools, c.flat, before):  # nothing else in the pool changed
        p[:, at] = 0
        b[p.storage_offset():].as_strided(p.shape, p.stride())[:, at] = 0
        bits = torch.int16 if f.dtype == torch.bfloat16 else torch.int32
        assert torch.equal(f.view(bits), b.view(bits))
    if with_q and not inplace:
        assert torch.equal(parts[0], qin)


REQ = [(-1, 1, 1), (-1, 40, 7), (-1, 33, 33), (-1, 9, 0), (-1, 100, 1)]


@pytest.mark.parametrize("heads,kv,dim", HEADS)
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("norm", [True, False])
def test_append_layouts(heads, kv, dim, dtype, norm):
    c = Case(dtype=dtype, heads=heads, kv_heads=kv, head_dim=dim, requests=REQ, seed=dim)
    check_append(c, norm)


@pytest.mark.parametrize("heads,latent,rope", [(16, 512, 64), (3, 20, 6), (1, 0, 64), (5, 128, 64), (2, 512, 512)])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("inplace", [False, True])
def test_append_latent_rows(heads, latent, rope, dtype, inplace):
    c = Case(family=MLA, dtype=dtype, heads=heads, latent=latent, rope=rope, requests=REQ, seed=latent)
    check_append(c, True, inplace=inplace)


@pytest.mark.parametrize("pairing", [abi.NEOX, abi.GPTJ])
@pytest.mark.parametrize("dim,sections", [(128, (16, 24, 24)), (64, (8, 12, 12)), (80, (10, 13, 17))])
def test_append_sections_and_pairings(pairing, dim, sections):
    c = Case(head_dim=dim, pairing=pairing, sections=sections, requests=REQ, base=1e6)
    check_append(c, True, sections=True)
    c = Case(head_dim=dim, pairing=pairing, requests=REQ, base=1e6)
    check_append(c, True, sections=True)  # no sections in the layout: every pair follows t
    c = Case(family=MLA, heads=4, latent=512, rope=64, pairing=pairing, requests=REQ)
    check_append(c, True, sections=True)


def test_append_strides_alignment_and_parts():
    for off, pad, slack in ((0, 0, 8), (1, 5, 3), (8, 16, 1), (0, 4, 4)):
        for fused in (True, False):
            check_append(Case(head_dim=128, heads=4, requests=REQ, offset=off, pad_layer=pad), True, slack=slack, fused=fused)
    check_append(Case(head_dim=128, heads=4, requests=REQ), True, inplace=True)
    check_append(Case(head_dim=64, heads=4, requests=REQ), False, inplace=True)
    check_append(Case(head_dim=128, heads=0, requests=REQ), True, with_q=False)
    check_append(Case(head_dim=128, heads=4, requests=REQ), True, with_q=False)
    for page in (1, 3, 64):
        check_append(Case(head_dim=64, heads=4, page=page, requests=REQ), True)
    check_append(Case(head_dim=128, heads=4, kv_heads=2, requests=[(-1, 2000, 1500), (-1, 77, 77)], layers=1), True)


def test_append_zero_rows_and_eps():
    """A head of zeros: 0 / sqrt(eps); eps 0 and a head of zeros gives NaN as the formula does."""
    c = Case(head_dim=128, heads=2, kv_heads=2, requests=[(-1, 3, 3)], layers=1)
    s = c.step(step.APPEND)
    plan = step.upload(c.lay, s, c.pool, c.workspace(s))
    z = torch.zeros(3, 256, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(128, dtype=torch.bfloat16, device="cuda")
    for eps, nan in ((1e-6, False), (0.0, True)):
        out = torch.full_like(z, 2.0)
        step.append(plan, 0, q=z, q_out=out, k=z, v=z, q_weight=w, k_weight=w, eps=eps)
        torch.cuda.synchronize()
        assert torch.isnan(out).all() if nan else (out == 0).all()


def test_append_then_attend_one_plan():
    """Append writes what attend reads, layer after layer, and in a captured graph."""
    c = Case(head_dim=128, heads=8, kv_heads=2, prefixes=[64], requests=[(0, 5, 1), (0, 30, 12), (-1, 3, 3)], seed=4)
    rows = c.draw(c.layers, c.n, c.heads * c.dk + 2 * c.F).cuda()
    nq = c.heads * c.dk
    s = c.step(step.APPEND | step.ATTEND, position0=64)
    ws = c.workspace(s)
    plan = step.upload(c.lay, s, c.pool, ws)
    out = torch.zeros(c.layers, c.n, c.heads * c.dv, dtype=torch.bfloat16, device="cuda")

    def layers():
        for layer in range(c.layers):
            r = rows[layer]
            step.append(plan, layer, q=r[:, :nq], q_out=c.q[layer], k=r[:, nq:nq + c.F], v=r[:, nq + c.F:])
            step.attend(plan, layer, c.q[layer], out[layer], scale_of(c))

    layers()
    torch.cuda.synchronize()
    for layer in range(c.layers):
        o, tol, _, _ = c.expect_attend(layer, scale_of(c))
        assert (np.abs(out[layer].double().cpu().numpy() - o) <= tol).all()
    want, pools = out.clone(), [f.clone() for f in c.flat]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layers()
    for _ in range(3):
        out.zero_()
        c.q.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        assert all(torch.equal(f.view(torch.int16), p.view(torch.int16)) for f, p in zip(c.flat, pools))


# ------------------------------------------------------------------ pages
def page_pool(family, dtype, layers, pages, page, kv_heads=2, head_dim=64, latent=20, rope=6, pad=0, off=0):
    f = kv_heads * head_dim if family == GQA else latent + rope
    t = TYPES[dtype]
    per = pages * page * f + pad
    flats = [torch.randn(layers * per + off, device="cuda").to(t) for _ in range(2 if family == GQA else 1)]
    views = [x[off:].as_strided((layers, pages, page * f), (per, page * f, 1)) for x in flats]
    lay = abi.make_layout(family, dtype, layers, num_kv_heads=kv_heads, head_dim=head_dim, latent_dim=latent, rope_dim=rope, page_size=page)
    return lay, abi.make_pool(views[0], views[1] if family == GQA else None, pages, per), views, flats


def check_copies(src, dst, stream=None, **kw):
    lay, pool, views, flats = page_pool(**kw)
    before = [f.clone() for f in flats]
    want = []
    for v, f, b in zip(views, flats, before):
        w = b[v.storage_offset():].as_strided(v.shape, v.stride())
        w[...] = torch.from_numpy(so.copy_pages(w.float().cpu().numpy(), src, dst)).to(w.dtype).cuda()
        want.append(b)
    ws = torch.empty(step.copy_pages_workspace_bytes(len(src)), dtype=torch.uint8, device="cuda")
    step.copy_pages(lay, pool, src, dst, ws, stream=stream)
    torch.cuda.synchronize()
    assert all(torch.equal(f, w) for f, w in zip(flats, want))


SMALL = dict(family=GQA, dtype=BF16, layers=3, pages=40, page=16)


@pytest.mark.parametrize("family,dtype,page,kw", [
    (GQA, BF16, 16, {}), (GQA, F32, 16, {}), (MLA, BF16, 16, dict(latent=512, rope=64)), (MLA, BF16, 1, {}), (MLA, F32, 3, {}),
    (GQA, BF16, 1, dict(kv_heads=1, head_dim=2)), (GQA, BF16, 7, dict(kv_heads=3, head_dim=10)), (GQA, BF16, 16, dict(pad=5, off=1)),
    (GQA, BF16, 16, dict(pad=8, off=8)), (GQA, F32, 5, dict(kv_heads=1, head_dim=6, pad=1)), (GQA, BF16, 16, dict(pad=2, off=2))])
def test_copy_pages_layouts(family, dtype, page, kw):
    rng = np.random.default_rng(page)
    order = rng.permutation(40)
    check_copies(order[:9], order[20:29], **dict(SMALL, family=family, dtype=dtype, page=page, **kw))
    check_copies(order[:30], rng.permutation(order[:30]), **dict(SMALL, family=family, dtype=dtype, page=page, **kw))


@pytest.mark.parametrize("src,dst", [
    ([], []), ([3], [3]), ([0], [39]), ([5, 5, 5], [1, 2, 3]), ([1, 2, 3], [2, 3, 4]), ([2, 3, 4], [1, 2, 3]), ([1, 2], [2, 1]),
    ([0, 1, 2, 7], [1, 2, 0, 7]), ([1, 1, 2, 3, 2, 0], [2, 9, 3, 1, 8, 0]),  # a cycle that also feeds pages outside it
    ([1, 2, 2, 4, 5], [2, 3, 4, 6, 7]), (list(range(39)), list(range(1, 40))), (list(range(1, 40)) + [0], list(range(40))),
    ([10, 11, 12, 13, 20, 21], [11, 10, 13, 12, 21, 22])])
def test_copy_pages_orders(src, dst):
    """Chains, fans, cycles: every copy reads what was there before the call."""
    check_copies(np.array(src, np.int64), np.array(dst, np.int64), **SMALL)


@pytest.mark.parametrize("seed", range(12))
def test_copy_pages_random(seed):
    rng = np.random.default_rng(seed)
    pages = int(rng.integers(2, 900))
    n = int(rng.integers(1, pages + 1))
    src = rng.integers(0, pages, n) if seed % 2 else rng.permutation(pages)[:n]
    check_copies(src, rng.permutation(pages)[:n], family=GQA, dtype=BF16, layers=2, pages=pages, page=4, kv_heads=1, head_dim=16)


@pytest.mark.parametrize("n", [63, 64, 65, 79, 80, 81, 127, 255, 256, 257, 300, 900])
@pytest.mark.parametrize("closed", [False, True])
def test_copy_pages_long_paths_and_cycles(n, closed):
    """Paths and cycles around the length from which they are shared out, alone and beside other copies."""
    order = np.random.default_rng(n).permutation(1000)
    ring = order[:n]
    src, dst = (np.roll(ring, -1), ring) if closed else (ring[1:], ring[:-1])
    for more in (0, 5):
        s, d = np.concatenate([src, order[n:n + more]]), np.concatenate([dst, order[n + more:n + 2 * more]])
        check_copies(s, d, family=GQA, dtype=BF16, layers=2, pages=1000, page=4, kv_heads=1, head_dim=16 if n % 2 else 10)
    if not closed:  # a page of the path read twice: no ring any more
        s, d = np.concatenate([src, src[5:6]]), np.concatenate([dst, order[-1:]])
        check_copies(s, d, family=MLA, dtype=F32, layers=2, pages=1000, page=3)


@pytest.mark.parametrize("seed", range(6))
def test_compact_pages(seed):
    rng = np.random.default_rng(seed)
    pages = 300
    live = rng.permutation(pages)[:int(rng.integers(0, pages + 1))].astype(np.int32)
    tables = [live[:5].copy(), live.copy(), live[3:].copy(), np.zeros(0, np.int32)]  # pages shared between tables
    lay, pool, views, flats = page_pool(GQA, BF16, 2, pages, 4, kv_heads=1, head_dim=16)
    before = [v.clone() for v in views]
    src, dst, want, n = so.compact(tables, pages)
    mine = [t.copy() for t in tables]
    ws = torch.empty(step.copy_pages_workspace_bytes(pages), dtype=torch.uint8, device="cuda")
    assert step.compact_pages(lay, pool, mine, ws) == n
    torch.cuda.synchronize()
    for a, b, old in zip(mine, want, tables):
        assert np.array_equal(a, b) and (a.size == 0 or a.max() < n)
        for v, o in zip(views, before):
            assert torch.equal(v[:, torch.from_numpy(a).long().cuda()], o[:, torch.from_numpy(old).long().cuda()])


def test_copy_pages_on_another_stream_and_far_offsets():
    side = torch.cuda.Stream()
    check_copies(np.arange(20), np.arange(20) + 20, stream=side, **SMALL)
    check_copies(np.arange(39), np.arange(39) + 1, stream=side, **SMALL)
    lay = abi.make_layout(GQA, BF16, 1, num_kv_heads=8, head_dim=128, page_size=16)  # byte offsets beyond 2^32
    pools = [torch.empty(140000, 16384, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    for p in pools:
        p[139998] = 1.5
        p[3] = -2.0
    ws = torch.empty(step.copy_pages_workspace_bytes(2), dtype=torch.uint8, device="cuda")
    step.copy_pages(lay, abi.make_pool(*pools, 140000), [139998, 3], [139999, 139998], ws)
    torch.cuda.synchronize()
    for p in pools:
        assert (p[139999] == 1.5).all() and (p[139998] == -2.0).all()


def test_example_serves_a_shared_chunk():
    """Rehydrate, fork, append, attend, compact together, as examples/serve_step.py does it."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "serve_step.py")
    spec = importlib.util.spec_from_file_location("serve_step", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    mod.main()
