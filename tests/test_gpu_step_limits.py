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
