"""Calls of the paged-cache operators at the edges of what their documentation
allows: arguments that share memory, infinite scores, rows behind a sequence in
its last page, pool tensors replaced by others, waits that run out."""
import numpy as np
import pytest
import torch

import mla_latent_kv_07_gb300 as mla

from paged_cases import Pool, evict_reference

pytestmark = pytest.mark.gpu
SM = 0.1352


@pytest.fixture(scope="module", autouse=True)
def _built():
    from mla_latent_kv_07_gb300 import build
    build.build()
    mla.lib()


# ---------------------------------------------------------- eviction in place

@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("ends,keep,sinks,recent", [
    ([4000, 33, 32, 31, 0, 1, 2500], 32, 4, 8), ([300] * 64, 130, 2, 100), ([9001, 17], 9000, 0, 1), ([70], 64, 0, 0)])
def test_eviction_replaces_the_lengths_in_place(fmt, ends, keep, sinks, recent):
    # new_end_pos is end_pos: every CTA of a sequence's cluster has read its
    # length before the new one is stored
    pool = Pool(fmt, ends, 32, seed=60, spare=len(ends) * -(-keep // 32))
    cache, e = pool.device(), pool.dev_ends()
    need = -(-keep // 32)
    new = torch.tensor(pool.free[:len(ends) * need], dtype=torch.int32).view(len(ends), need).cuda()
    ref, rend = evict_reference(pool, keep, sinks, recent)
    for _ in range(20):
        e.copy_(pool.dev_ends())
        kept, end = mla.paged_evict(cache, pool.dev_table(), e, max(ends), keep, new, sinks=sinks, recent=recent, new_end_pos=e)
        assert end is e
        assert np.array_equal(kept.cpu().numpy(), ref) and np.array_equal(e.cpu().numpy(), rend)


def test_a_captured_eviction_in_place_replays():
    pool = Pool(1, [900, 400, 64], 64, seed=61, spare=6)
    cache, tb, e = pool.device(), pool.dev_table(), pool.dev_ends()
    new = torch.tensor(pool.free[:6], dtype=torch.int32).view(3, 2).cuda()
    kept = torch.empty((3, 100), dtype=torch.int32, device="cuda")
    mla.paged_evict(cache, tb, e, 900, 100, new, recent=10, kept=kept, new_end_pos=e)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mla.paged_evict(cache, tb, e, 900, 100, new, recent=10, kept=kept, new_end_pos=e)
    for ends in ([900, 400, 64], [101, 100, 64], [0, 400, 5]):
        e.copy_(torch.tensor(ends, dtype=torch.int32))
        g.replay()
        pool.ends = np.array(ends, np.int32)
        ref, rend = evict_reference(pool, 100, 0, 10)
        assert np.array_equal(kept.cpu().numpy(), ref) and np.array_equal(e.cpu().numpy(), rend)
