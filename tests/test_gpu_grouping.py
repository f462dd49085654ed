"""Grouping with CTAs that have little or nothing to do: ranges of pairs that are empty or end
early let some CTAs of a cluster finish while others still read their counts."""
import numpy as np
import pytest
import torch

from gpu_common import dev, require_gpu
from oracle import experts

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("pairs", [4097, 4128, 5000, 8193, 20000, 65536, 65537])
@pytest.mark.parametrize("e", [1, 7, 256])
def test_ranges_of_clusters_that_are_empty_or_short(pairs, e):
    """4096 pairs are one CTA's; from 4097 on 8 clusters of 8 share them, the first 32 to a warp,
    so that 5000 pairs leave 59 of 64 CTAs without any.  Two streams at once, many times over: the
    result is a function of the indices alone."""
    sa = require_gpu()
    sa.sink_attn_device_status(True)
    rng = np.random.default_rng(pairs + e)
    sets = []
    for skew in (0.0, 3.0):
        idx = np.minimum((e * rng.random((pairs, 1)) ** (1 + skew)).astype(np.int32), e - 1)
        idx[rng.random((pairs, 1)) < 0.05] = -1
        sets.append((dev(idx), [dev(v) for v in experts.group_rows(idx, e)]))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[sa.moe_group_rows(idx, e) for _ in range(40)] for idx, _ in sets]
    torch.cuda.synchronize()
    for i in range(40):
        for (idx, _), outs, s in zip(sets, got, streams):
            for o in outs[i]:
                o.fill_(-9)
    torch.cuda.synchronize()
    for i in range(40):
        for (idx, _), outs, s in zip(sets, got, streams):
            sa.moe_group_rows(idx, e, *outs[i], stream=s)
    torch.cuda.synchronize()
    for (_, ref), outs in zip(sets, got):
        for out in outs:
            assert all(torch.equal(g, r) for g, r in zip(out, ref))
    assert sa.sink_attn_device_status(True) == 0


def test_refused_numbers_of_experts_allocate_nothing():
    """An argument that the library refuses is refused before memory is asked for in its size."""
    sa = require_gpu()
    idx = torch.zeros((4, 2), dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    for e in (257, 2 ** 20, 2 ** 31 - 1, 0, -1, -2 ** 31 + 1):
        with pytest.raises(sa.SinkAttnError):
            sa.moe_group_rows(idx, e)
    assert torch.cuda.max_memory_allocated() - before < 2 ** 16
    offsets, _, _ = sa.moe_group_rows(idx, 256)
    assert offsets.tolist() == [0] + [8] * 256
