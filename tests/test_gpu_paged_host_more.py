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
