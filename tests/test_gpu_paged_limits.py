"""The paged cache's write, reading and windowed attention at the ends of their
ranges, against fp64 references."""
import numpy as np
import pytest
import torch

import mla_latent_kv_07_gb300 as mla

from paged_cases import Pool

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from mla_latent_kv_07_gb300 import build
    build.build()
    mla.native()


@pytest.mark.parametrize("fmt", [1, 2])
def test_blocks_too_small_for_a_scale_are_zeros(fmt):
    # row i's first block holds a few values of 2^-(138 + i) among zeros, its others values
    # of 1/2.  448 times the smallest fp32 number is 2^-140.2: from 2^-142 on the scale is 0
    n = 12
    x = torch.zeros(1, n, 576)
    x[..., 128:512] = 0.5
    x[0, :, [0, 5, 127]] = 2.0 ** -(18 + torch.arange(n)).float()[:, None]
    x[0, :, 5] *= -1
    w = torch.ones(512)
    w[:128] = 2.0 ** -120
    pool = Pool(fmt, [n], 16, seed=60)
    cache = pool.device()
    rot, pos = mla.Rotary(mla.rotary_frequencies()), torch.zeros(1, n, dtype=torch.int32, device="cuda")
    mla.paged_append_rotary(cache, pool.dev_table(), x.to(torch.bfloat16).cuda(), w.cuda(), 1.0, rot, pos, pool.dev_ends())
    rows = pool.rows(0).astype(np.int64)
    codes = cache.kv.cpu().numpy().reshape(-1, 512)[rows]
    scale = cache.kv_scale.cpu().numpy().reshape(-1, 4)[rows].astype(np.float64)
    y = x[0, :, :512].double().numpy()
    y = y / np.sqrt((y ** 2).mean(-1, keepdims=True) + 1.0) * w.double().numpy()
    amax = np.abs(y[:, :128]).max(-1)
    assert (scale[amax < 2.0 ** -150 * 448, 0] == 0).all() and (scale[amax > 2.0 ** -150 * 449, 0] > 0).all()
    assert (codes[scale[:, 0] == 0, :128] == 0).all() and (codes[:, 1:127][:, [0, 60]] == 0).all()
    val = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy() * np.repeat(scale, 128, 1)
    # a code is off by 2^-4 of its value or 2^-10 of the scale; a scale by half of the smallest
    # fp32 number, which is 448 halves at the block's largest value, and so may y be by one half
    bound = 2.0 ** -4 * np.abs(y) + 2.0 ** -10 * np.repeat(scale, 128, 1) + 450 * 2.0 ** -150 + 2.0 ** -19 * np.abs(y)
    assert np.isfinite(val).all() and (np.abs(val - y) <= bound).all()
    # and read back they are finite
    kv, _ = mla.paged_read(cache, pool.dev_table(), torch.tensor([0, n], dtype=torch.int32).cuda(), n)
    assert bool(kv.isfinite().all())
