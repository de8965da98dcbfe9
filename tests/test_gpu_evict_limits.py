"""Limits of eviction, weighing and differential attention on the GPU."""
import numpy as np
import pytest
import torch

from position_free_kv_amd import abi, step
from tests import evict_util as eu
from tests.evict_util import Params
from tests.step_util import E32, HALF, Case

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
