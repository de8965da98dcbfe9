"""What the serving step's Python binding refuses before the library is called. No GPU is needed: device pointers
are fake addresses that nothing dereferences."""

import numpy as np
import pytest

from position_free_kv_amd import abi, step


def _gpu_present() -> bool:
    try:
        import torch
        return torch.cuda.device_count() > 0
    except Exception:  # noqa: BLE001
        return False


pytestmark = pytest.mark.skipif(_gpu_present(), reason="fake device addresses")

FAKE = 0x10_0000_0000
PAGE = 16


def layout(**kw):
    return abi.make_layout(abi.GQA, kw.pop("dtype", abi.BF16), 2, **{**dict(num_kv_heads=2, head_dim=64, page_size=PAGE), **kw})


def upload(s, lay=None):
    return step.upload(lay or layout(), s, abi.make_pool(FAKE, FAKE, 100), (FAKE, 1 << 30))


def accepted(s):
    """All checks passed: what is left is the first call of the GPU."""
    with pytest.raises(abi.KameraError) as e:
        upload(s)
    assert e.value.name == "KAMERA_E_HIP"


def refused(s):
    with pytest.raises(ValueError):
        upload(s)


# ------------------------------------------------------------------ tables as long as their tokens
@pytest.mark.parametrize("rows", [False, True])
@pytest.mark.parametrize("slot0,tokens,entries", [(0, 16, 1), (0, 17, 2), (5, 11, 1), (5, 12, 2), (15, 1, 1), (15, 2, 2), (3, 160, 11)])
def test_tables_shorter_than_their_tokens_are_refused(rows, slot0, tokens, entries):
    """One entry less would be read from the next request's table, or past the array's end."""
    def make(n):
        t = np.arange(2 * n, dtype=np.int32).reshape(2, n)
        return step.Step(num_q_heads=4, block_tables=t if rows else list(t), slot0=slot0, num_tokens=[tokens, 1], num_queries=1)
    accepted(make(entries))
    refused(make(entries - 1))


def test_a_step_that_outgrows_its_tables_in_place_is_refused():
    s = step.Step(num_q_heads=4, block_tables=np.array([[1], [2]], np.int32), num_tokens=[16, 3], num_queries=1)
    accepted(s)
    s.requests["num_tokens"] += 1
    refused(s)


def test_prefix_tables_shorter_than_their_tokens_are_refused():
    def make(tokens, slot0):
        return step.Step(num_q_heads=4, block_tables=[np.array([1], np.int32)], num_tokens=1, num_queries=1, prefix=0,
                         prefixes=[dict(block_table=np.array([3, 4], np.int32), num_tokens=tokens, slot0=slot0)])
    accepted(make(32, 0))
    accepted(make(28, 4))
    refused(make(33, 0))
    refused(make(29, 4))


def test_requests_without_a_table_have_no_tokens():
    with pytest.raises(abi.KameraError) as e:
        upload(step.Step(num_q_heads=4, block_tables=[None], num_tokens=1, num_queries=1))
    assert e.value.name == "KAMERA_E_NULL"
    refused(step.Step(num_q_heads=4, block_tables=[np.zeros(0, np.int32)], num_tokens=1, num_queries=1))
    accepted(step.Step(num_q_heads=4, block_tables=[None, np.zeros(0, np.int32)], num_tokens=0, num_queries=[1, 0], flags=step.ATTEND))


# ------------------------------------------------------------------ tables read in place
def entry(s, record, i):
    """The page id that the library would read as entry i of a record's table."""
    import ctypes
    return ctypes.cast(int(record["block_table"]), ctypes.POINTER(ctypes.c_int32))[i]


@pytest.mark.parametrize("of", [lambda b: b[:, :4], lambda b: b, lambda b: b[::-1], lambda b: b[::2, 3:], lambda b: b[:, 2:3], list,
                                lambda b: [r[1:3] for r in b]])
def test_tables_follow_changes_in_place(of):
    """Column slices, rows in another order and single columns are read where they lie."""
    big = np.zeros((4, 8), np.int32)
    tables = of(big)
    s = step.Step(num_q_heads=4, block_tables=tables, num_tokens=1, num_queries=1)
    big[:] = np.arange(32).reshape(4, 8)
    for r, t in zip(s.requests, tables):
        assert [entry(s, r, i) for i in range(len(t))] == t.tolist()


def test_prefix_tables_follow_changes_in_place():
    pages = np.zeros(6, np.int32)
    s = step.Step(num_q_heads=4, block_tables=[np.array([1], np.int32)], num_tokens=1, num_queries=1, prefix=0,
                  prefixes=[dict(block_table=pages[1:], num_tokens=80)])
    pages[:] = np.arange(6) + 40
    assert [entry(s, s.prefixes[0], i) for i in range(5)] == [41, 42, 43, 44, 45]


@pytest.mark.parametrize("table", [np.zeros((2, 4), np.int64), np.zeros((4, 2), np.int32).T, np.zeros((2, 8), np.int32)[:, ::2],
                                   np.zeros((2, 4), np.uint32), [np.zeros(4, np.int64)] * 2, [np.zeros(8, np.int32)[::2]] * 2,
                                   [[0, 1], [2, 3]], [np.zeros((2, 2), np.int32)] * 2])
def test_tables_that_would_have_to_be_copied_are_refused(table):
    with pytest.raises(ValueError):
        step.Step(num_q_heads=4, block_tables=table, num_tokens=1, num_queries=1)
    for t in table if not isinstance(table, np.ndarray) else []:
        with pytest.raises(ValueError):
            step.Step(num_q_heads=4, block_tables=[], num_tokens=1, num_queries=1, prefixes=[dict(block_table=t, num_tokens=1)])


# ------------------------------------------------------------------ page ids
@pytest.mark.parametrize("bad", [np.array([2 ** 32 + 1]), np.array([2 ** 31], np.uint32), np.array([-2 ** 32]), np.array([1.0]), [1.5], ["1"],
                                 np.array([True])])
def test_page_ids_that_would_become_others_are_refused(bad):
    ws = (FAKE, 1 << 20)
    for src, dst in ((bad, [1]), ([1], bad)):
        with pytest.raises((ValueError, OverflowError)):
            step.copy_pages(layout(), abi.make_pool(FAKE, FAKE, 100), src, dst, ws)
    for good in ([4], np.array([4], np.int64), np.array([4], np.uint8), np.array([4, 0], np.int32)[::2]):
        step.copy_pages(layout(), abi.make_pool(FAKE, FAKE, 100), good, [4], ws)  # (nothing to do)


@pytest.mark.parametrize("kw", [dict(num_tokens=np.array([2 ** 32 + 5])), dict(num_queries=np.array([2 ** 32 + 1])), dict(slot0=np.array([2 ** 32])),
                                dict(prefix=np.array([2 ** 32 - 1])), dict(num_tokens=5.5), dict(position0=0.5), dict(request_flags=np.array([2 ** 32])),
                                dict(num_tokens=2 ** 32 + 5)])
def test_request_fields_that_would_become_others_are_refused(kw):
    with pytest.raises((ValueError, OverflowError)):
        step.Step(num_q_heads=4, block_tables=[np.array([1], np.int32)], **{**dict(num_tokens=5, num_queries=1), **kw})


# ------------------------------------------------------------------ tensors of the launches
@pytest.fixture
def tensors(monkeypatch):
    """Tensors of the host stand for the GPU's: what is left of the checks are types, shapes and strides."""
    torch = pytest.importorskip("torch")
    monkeypatch.setattr(step, "_on_gpu", lambda what, x: None, raising=False)
    return torch


def a_plan(tokens=3, family=abi.GQA, dtype=abi.BF16, heads=4, flags=step.APPEND | step.ATTEND):
    lay = layout(dtype=dtype) if family == abi.GQA else abi.make_layout(abi.MLA, dtype, 2, latent_dim=64, rope_dim=16)
    plan = step.upload(lay, step.Step(num_q_heads=heads, block_tables=[np.array([1], np.int32)], num_tokens=1, num_queries=0, flags=flags),
                       abi.make_pool(FAKE, FAKE, 100), (FAKE, 1 << 30))  # no tokens: nothing is enqueued
    plan.num_tokens = tokens
    return plan


def launched(fn, *args, **kw):
    """Every check passed: what is left is the launch, for which there is no GPU (or nothing to launch)."""
    try:
        fn(*args, **kw)
    except abi.KameraError as e:
        assert e.name == "KAMERA_E_HIP", str(e)


def good_rows(torch, n=3):
    fused = torch.zeros(n, 4 * 64 + 2 * 128, dtype=torch.bfloat16)
    return dict(q=fused[:, :256], k=fused[:, 256:384], v=fused[:, 384:], q_out=torch.zeros(n, 4, 64, dtype=torch.bfloat16),
                q_weight=torch.ones(64, dtype=torch.bfloat16), k_weight=torch.ones(64, dtype=torch.bfloat16))


def test_append_takes_rows_as_they_lie(tensors):
    torch, plan = tensors, a_plan()
    launched(step.append, plan, 0, **good_rows(torch))
    launched(step.append, plan, 0, **good_rows(torch, 5))  # buffers for more tokens than the step has
    wide = torch.zeros(3, 8, 64, dtype=torch.bfloat16)
    launched(step.append, plan, 0, **dict(good_rows(torch), q=wide[:, 2:6], k=wide[:, :2], v=wide[:, 6:]))
    flat = torch.zeros(3 * 256, dtype=torch.bfloat16)  # where rows begin, their stride given
    launched(step.append, plan, 0, **dict(good_rows(torch), q=flat, q_stride=256))
    launched(step.append, a_plan(1), 0, **{k: v[:1] if v.dim() > 1 else v for k, v in good_rows(torch).items()})
    one = torch.zeros(1, 128, dtype=torch.bfloat16)
    launched(step.append, a_plan(1), 0, **dict(good_rows(torch), k=one.expand(4, 128)))
    mla = torch.zeros(3, 4, 80, dtype=torch.bfloat16)
    launched(step.append, a_plan(family=abi.MLA), 0, q=mla, q_out=mla, k=torch.zeros(3, 80, dtype=torch.bfloat16),
             k_weight=torch.ones(64, dtype=torch.bfloat16), v=flat.float())  # (no V rows here)


def bad_rows(torch):
    z = dict(dtype=torch.bfloat16)
    yield "q", torch.zeros(3, 256)                                            # another type
    yield "q", torch.zeros(3, 256, dtype=torch.float16)
    yield "k", torch.zeros(3, 2, 96, **z)[:, :, :64]                          # the first columns of wider heads
    yield "k", torch.zeros(2, 3, 64, **z).transpose(0, 1)                     # heads before tokens
    yield "v", torch.zeros(128, 3, **z).t()
    yield "v", torch.zeros(3, 256, **z)[:, ::2]
    yield "k", torch.zeros(2, 128, **z)                                       # fewer rows than tokens
    yield "k", torch.zeros(3, 120, **z)                                       # narrower
    yield "k", torch.zeros(3, 200, **z)[:, :100]
    yield "q_out", torch.zeros(1, 256, **z).expand(3, 256)                    # one row for all tokens
    yield "v", torch.zeros(1, 128, **z).expand(3, 128)
    yield "q", torch.zeros(256, **z)
    yield "q", torch.zeros((), **z)
    yield "q_weight", torch.ones(64)
    yield "q_weight", torch.ones(256, **z)
    yield "k_weight", torch.ones(128, **z)[::2]
    yield "k_weight", torch.ones(32, **z)


def test_append_refuses_rows_it_would_misread(tensors):
    plan = a_plan()
    for name, x in bad_rows(tensors):
        with pytest.raises(ValueError) as e:
            step.append(plan, 0, **dict(good_rows(tensors), **{name: x}))
        assert str(e.value).startswith(name + ":")
    with pytest.raises(ValueError):  # the last row would end past the buffer
        step.append(plan, 0, **dict(good_rows(tensors), q=tensors.zeros(3 * 256, dtype=tensors.bfloat16)[1:], q_stride=256))
    with pytest.raises(ValueError):
        step.append(a_plan(dtype=abi.F32), 0, **good_rows(tensors))


def test_attend_checks_queries_outputs_and_statistics(tensors):
    torch, plan = tensors, a_plan()
    q, out = torch.zeros(3, 4, 64, dtype=torch.bfloat16), torch.zeros(3, 256, dtype=torch.bfloat16)
    launched(step.attend, plan, 0, q, out, 1.0)
    launched(step.attend, plan, 0, q, out, 1.0, lse=torch.zeros(3, 4))
    launched(step.attend, plan, 0, q, torch.zeros(3, 300, dtype=torch.bfloat16)[:, 8:], 1.0, out_stride=300)
    launched(step.attend, a_plan(family=abi.MLA), 0, torch.zeros(3, 4, 80, dtype=torch.bfloat16), out, 1.0)
    for bad in (dict(q=q.float()), dict(q=q[:2]), dict(q=torch.zeros(3, 4, 80, dtype=torch.bfloat16)[:, :, :64]), dict(out=out.float()),
                dict(out=out[:, :255]), dict(lse=torch.zeros(3, 4, dtype=torch.float64)), dict(lse=torch.zeros(4, 3).t()), dict(lse=torch.zeros(3, 3)),
                dict(lse=torch.zeros(3, 4, dtype=torch.bfloat16)), dict(out=torch.zeros(3 * 300 - 45, dtype=torch.bfloat16), out_stride=300)):
        args = dict(q=q, out=out, lse=None, **{k: v for k, v in bad.items() if k.endswith("stride")})
        args.update(bad)
        with pytest.raises(ValueError):
            step.attend(plan, 0, args.pop("q"), args.pop("out"), 1.0, **args)


def test_positions_are_packed_int32(tensors):
    torch = tensors

    def make(positions):
        return step.Step(num_q_heads=4, block_tables=[np.array([1], np.int32)], num_tokens=5, num_queries=4, positions=positions)
    accepted(make(torch.zeros(4, 3, dtype=torch.int32)))
    for bad in (torch.zeros(4, 3, dtype=torch.int64), torch.zeros(3, 4, dtype=torch.int32).t(), torch.zeros(3, 3, dtype=torch.int32)):
        refused(make(bad))


def test_tensors_of_the_host_are_refused():
    torch = pytest.importorskip("torch")
    for name in good_rows(torch):
        rows = {k: (v if k == name else FAKE) for k, v in good_rows(torch).items()}
        with pytest.raises(ValueError):
            step.append(a_plan(), 0, **rows)
    with pytest.raises(ValueError):
        step.attend(a_plan(), 0, torch.zeros(3, 256, dtype=torch.bfloat16), FAKE, 1.0)
