"""Rehydration at the size of one launch: a grid of 2^32 threads and more would run in part."""
import numpy as np
import pytest

from position_free_kv_amd import abi

FAKE = 0x10_0000_0000


def _gpu_present() -> bool:
    try:
        import torch
        return torch.cuda.device_count() > 0
    except Exception:  # noqa: BLE001
        return False


@pytest.mark.skipif(_gpu_present(), reason="fake device addresses")
@pytest.mark.parametrize("dtype,layers,fits", [(abi.F32, (1 << 23) - 16, True), (abi.F32, 1 << 23, False),
                                               (abi.BF16, (1 << 25) - 16, True), (abi.BF16, 1 << 25, False)])
def test_batches_of_more_than_one_launch_are_refused(dtype, layers, fits):
    """K and V of every layer are a task each: of a workgroup in the plain kernel, of a wave in the matrix-core one."""
    lay = abi.make_layout(abi.GQA, dtype, layers, num_kv_heads=1, head_dim=64)
    ch = abi.ChunkDesc(num_tokens=1, delta=1, flags=0, k_src=FAKE, v_src=FAKE + (1 << 36), k_dst=FAKE + (2 << 36), v_dst=FAKE + (3 << 36))
    with pytest.raises(abi.KameraError) as e:
        abi.rehydrate_batched(lay, [ch], None, (FAKE, 1 << 20))
    assert e.value.name == ("KAMERA_E_HIP" if fits else "KAMERA_E_SHAPE")


@pytest.mark.gpu
def test_cos_sin_tables_of_many_chunks_beside_a_long_one():
    """Tables are laid out by the longest chunk's: 520 chunks of 32768 workgroups each."""
    import torch
    rng = np.random.default_rng(0)
    lay = abi.make_layout(abi.GQA, abi.BF16, 1, num_kv_heads=1, head_dim=128, rope_base=1e6)
    lengths = [131072] + [3] * 519
    total = sum(lengths)
    src = torch.randn(2, total, 128, device="cuda").bfloat16()
    pos = torch.from_numpy(rng.integers(0, 100000, (total, 3)).astype(np.int32)).cuda()

    def chunks(dst, which):
        first = np.concatenate([[0], np.cumsum(lengths)])
        return [abi.ChunkDesc(num_tokens=lengths[i], delta=0, flags=abi.POSITIONS, k_src=src[0, first[i]:], v_src=src[1, first[i]:],
                              k_dst=dst[0, first[i]:], v_dst=dst[1, first[i]:], positions=pos[first[i]:]) for i in which]

    def run(dst, which):
        batch = chunks(dst, which)
        ws = torch.empty(abi.batch_workspace_bytes(lay, batch), dtype=torch.uint8, device="cuda")
        abi.rehydrate_batched(lay, batch, None, ws)
        torch.cuda.synchronize()
    whole, parts = torch.zeros_like(src), torch.zeros_like(src)
    run(whole, range(520))
    for i in range(0, 520, 100):
        run(parts, range(i, min(i + 100, 520)))
    assert torch.equal(whole, parts) and not torch.equal(whole[0, -1], src[0, -1])
