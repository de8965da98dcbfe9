"""Limits of the serving step on the GPU: what may be recorded in a graph."""
import numpy as np
import pytest
import torch

from position_free_kv_amd import abi, step
from tests.step_util import Case
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
