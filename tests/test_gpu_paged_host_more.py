"""More of the host path of the paged calls: arguments of odd types and layouts are
answered the same way through the extension and without it."""
import pytest
import torch

import mla_latent_kv_07_gb300 as mla

from paged_cases import Pool
from test_gpu_paged_host import _window

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from mla_latent_kv_07_gb300 import build
    build.build()
    mla.native()


class _Undecided:
    def __bool__(self):
        raise KeyError("neither")


@pytest.mark.parametrize("named", [False, True])
def test_a_wish_that_has_no_truth_value_is_refused(named):
    pool = Pool(0, [60, 33], 16, seed=70)
    st = torch.cuda.current_stream() if named else None
    with pytest.raises(KeyError):
        _window(pool.device(), pool, stream=st, want_lse=_Undecided())
    with pytest.raises(RuntimeError, match="ambiguous"):
        _window(pool.device(), pool, stream=st, want_lse=torch.zeros(2))
    assert _window(pool.device(), pool, stream=st, want_lse=torch.ones(1))[1] is not None


@pytest.mark.parametrize("named", [False, True])
def test_one_row_may_have_any_stride(named):
    pool = Pool(1, [60, 33], 16, seed=71)
    cache, off = pool.device(), torch.tensor([0, 1, 1], dtype=torch.int32, device="cuda")
    st = torch.cuda.current_stream() if named else None
    want = mla.paged_read(cache, pool.dev_table(), off, 1)
    kv, pe = torch.zeros(512, dtype=torch.bfloat16, device="cuda"), torch.zeros(64, dtype=torch.bfloat16, device="cuda")
    got = mla.paged_read(cache, pool.dev_table(), off, 1, kv=kv.as_strided((1, 512), (3, 1)), pe=pe.expand(1, 64), stream=st)
    assert got[0].data_ptr() == kv.data_ptr() and torch.equal(kv, want[0][0]) and torch.equal(pe, want[1][0])
    with pytest.raises(mla.MLAError):    # (two rows: looked at)
        mla.paged_read(cache, pool.dev_table(), off, 2, kv=torch.zeros(2, 516, dtype=torch.bfloat16, device="cuda")[:, :512], stream=st)
