"""Refusals of the paged-cache calls on the host (no GPU: fake, aligned device
addresses are never dereferenced on these paths), and of the binding."""
import ctypes

import pytest
import torch

import mla_latent_kv_07_gb300 as mla
from mla_latent_kv_07_gb300 import build as mbuild

FAKE = 0x7F0000000000
INVALID, RANGE, UNSUPPORTED, WORKSPACE = 1, 2, 3, 4


@pytest.fixture(scope="module")
def L():
    mbuild.build()
    return mla.lib()


def at(off=0):
    return ctypes.c_void_p(FAKE + off)


def pool(fmt=0, pages=8, page=64, scale=True, weight=True, kv=FAKE):
    return mla._CPagedCache(fmt, pages, page, kv, FAKE if (fmt and scale) else None, FAKE,
                            FAKE if weight else None)


POOLS = [  # what every paged call refuses in its pool and table
    (dict(kv=None), INVALID), (dict(kv=FAKE + 8), INVALID), (dict(fmt=7), UNSUPPORTED),
    (dict(fmt=1, scale=False), INVALID), (dict(fmt=2, scale=False), INVALID),
    (dict(page=0), INVALID), (dict(page=24), UNSUPPORTED), (dict(page=8), UNSUPPORTED),
    (dict(page=1 << 21), UNSUPPORTED), (dict(pages=0), INVALID), (dict(pages=1 << 15, page=1 << 16), UNSUPPORTED),
]


def call(L, op, cache, **kw):
    a = dict(table=at(), max_pages=4, q=at(), qp=at(), end=at(), max_end=256, B=2, H=128, scale=0.1, kv=None,
             pe=None, out=at(), lse=at(), ws=at(), ws_bytes=1 << 40, s=1, keep=64, sinks=4, recent=8,
             new_table=at(256), new_pages=2, kept=at(), new_end=at(), status=None)
    if op == "append":
        a.update(kv=at(), pe=at())
    a.update(kw)
    c = None if cache is None else ctypes.byref(cache)
    if op == "append":
        return L.mla_paged_append(c, a["table"], a["max_pages"], a["kv"], a["pe"], a["end"], a["B"], a["s"], a["status"], None)
    if op == "decode":
        return L.mla_paged_decode(c, a["table"], a["max_pages"], a["q"], a["qp"], a["end"], a["max_end"], a["B"], a["H"],
                                  a["scale"], a["kv"], a["pe"], a["out"], a["lse"], a["ws"], a["ws_bytes"], None)
    if op == "weights":
        return L.mla_paged_weights(c, a["table"], a["max_pages"], a["q"], a["qp"], a["lse"], a["end"], a["max_end"], a["B"],
                                   a["H"], a["scale"], a["status"], None)
    return L.mla_paged_evict(c, a["table"], a["max_pages"], a["end"], a["max_end"], a["B"], a["keep"], a["sinks"], a["recent"],
                             a["new_table"], a["new_pages"], a["kept"], a["new_end"], a["status"], None)


@pytest.mark.parametrize("op", ["append", "decode", "weights", "evict"])
def test_bad_pools_and_tables_are_refused(L, op):
    assert call(L, op, None) == INVALID
    for kw, code in POOLS:
        assert call(L, op, pool(**kw)) == code, kw
    assert call(L, op, pool(), table=None) == INVALID
    assert call(L, op, pool(), table=at(2)) == INVALID
    assert call(L, op, pool(), max_pages=0) == INVALID
    assert call(L, op, pool(), end=None) == INVALID
    assert call(L, op, pool(), end=at(2)) == INVALID
    assert call(L, op, pool(), B=0) == INVALID


@pytest.mark.parametrize("op", ["decode", "weights", "evict"])
def test_lengths_past_the_table_are_refused(L, op):
    assert call(L, op, pool(), max_end=257) == RANGE          # 4 pages of 64
    assert call(L, op, pool(), max_end=0) == RANGE
    assert call(L, op, pool(), max_end=-5) == RANGE
    assert call(L, op, pool(page=1 << 20), max_pages=2000, max_end=(1 << 30) + 1) == RANGE
    assert call(L, op, pool(), B=65536) == INVALID


@pytest.mark.parametrize("op", ["decode", "weights"])
def test_queries_are_checked(L, op):
    assert call(L, op, pool(), H=48) == UNSUPPORTED
    assert call(L, op, pool(), q=None) == INVALID
    assert call(L, op, pool(), qp=at(8)) == INVALID
    assert call(L, op, pool(), scale=float("nan")) == INVALID
    assert call(L, op, pool(), lse=at(2)) == INVALID


def test_append_rejects_bad_arguments(L):
    assert call(L, "append", pool(), kv=None) == INVALID
    assert call(L, "append", pool(), pe=at(8)) == INVALID
    assert call(L, "append", pool(), s=0) == INVALID
    assert call(L, "append", pool(), B=1 << 16, s=1 << 15) == INVALID       # more than 2^30 rows
    assert call(L, "append", pool(), status=at(2)) == INVALID


def test_decode_rejects_bad_arguments(L):
    assert call(L, "decode", pool(), out=None) == INVALID
    assert call(L, "decode", pool(), out=at(8)) == INVALID
    assert call(L, "decode", pool(), kv=at()) == INVALID                    # one of the pair only
    assert call(L, "decode", pool(), pe=at()) == INVALID
    assert call(L, "decode", pool(), kv=at(8), pe=at()) == INVALID


def test_weights_rejects_bad_arguments(L):
    assert call(L, "weights", pool(weight=False)) == INVALID
    assert call(L, "weights", pool(), lse=None) == INVALID
    assert call(L, "weights", pool(), status=at(1)) == INVALID


def test_evict_rejects_bad_arguments(L):
    assert call(L, "evict", pool(weight=False)) == INVALID
    assert call(L, "evict", pool(), keep=0) == INVALID
    assert call(L, "evict", pool(), sinks=-1) == INVALID
    assert call(L, "evict", pool(), recent=-1) == INVALID
    assert call(L, "evict", pool(), sinks=32, recent=33) == INVALID         # more than keep
    assert call(L, "evict", pool(), sinks=2 ** 31 - 1, recent=2 ** 31 - 1) == INVALID
    assert call(L, "evict", pool(), keep=129) == RANGE                      # two new pages of 64
    assert call(L, "evict", pool(page=1 << 20), new_pages=2000, keep=(1 << 30) + 1) == RANGE
    assert call(L, "evict", pool(), new_table=None) == INVALID
    assert call(L, "evict", pool(), new_table=at()) == INVALID              # the old one
    assert call(L, "evict", pool(), new_pages=0) == INVALID
    assert call(L, "evict", pool(), kept=None) == INVALID
    assert call(L, "evict", pool(), new_end=at(2)) == INVALID


def test_workspace_size_rejects_bad_arguments(L):
    assert L.mla_paged_workspace_size(0, 128) == 0
    assert L.mla_paged_workspace_size(65536, 128) == 0
    assert L.mla_paged_workspace_size(4, 24) == 0


def test_the_binding_refuses_host_tensors():
    with pytest.raises(ValueError):
        mla.PagedCache(2, 64, device="cpu")


@pytest.mark.parametrize("big", [2 ** 31, 2 ** 32 + 100, -2 ** 31 - 1, -2 ** 32 + 100])
def test_the_binding_refuses_numbers_past_32_bits(big):
    # (ctypes would pass on the low 32 bits: 100)
    class Host:   # host tensors are on device -1, so the checks before the call pass
        _dev, device = -1, torch.device("cpu")

    table, end = torch.zeros(1, 4, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    ql, qp = torch.zeros(1, 16, 512, dtype=torch.bfloat16), torch.zeros(1, 16, 64, dtype=torch.bfloat16)
    lse, new = torch.zeros(1, 16), torch.zeros(1, 4, dtype=torch.int32)
    calls = [lambda: mla.paged_decode(Host, table, ql, qp, end, big, 0.1, workspace=torch.zeros(1, dtype=torch.uint8)),
             lambda: mla.paged_weights(Host, table, ql, qp, lse, end, big, 0.1),
             lambda: mla.paged_evict(Host, table, end, big, 10, new),
             lambda: mla.paged_evict(Host, table, end, 100, big, new),
             lambda: mla.paged_evict(Host, table, end, 100, 10, new, sinks=big),
             lambda: mla.paged_evict(Host, table, end, 100, 10, new, recent=big)]
    for call in calls:
        with pytest.raises(mla.MLAError) as err:
            call()
        assert err.value.code == RANGE


def test_the_self_tests_refuse_what_their_calls_refuse(L):
    def decode(c, max_end=256, out=at(), ws=at()):
        return L.mla_selftest_paged_decode_timeout(ctypes.byref(c), at(), 4, at(), at(), at(), max_end, 2, 64, 0.1, out, at(), ws, 1 << 40, None)

    def weights(c, max_end=256, H=64, status=at()):
        return L.mla_selftest_paged_weights_timeout(ctypes.byref(c), at(), 4, at(), at(), at(), at(), max_end, 2, H, 0.1, status, None)

    assert decode(pool(page=24)) == UNSUPPORTED and weights(pool(page=24)) == UNSUPPORTED
    assert decode(pool(), max_end=257) == RANGE and weights(pool(), max_end=257) == RANGE
    assert decode(pool(), out=None) == INVALID and weights(pool(), status=at(2)) == INVALID
    assert weights(pool(weight=False)) == INVALID and weights(pool(), H=48) == UNSUPPORTED
