"""Refusals of the calls that write a paged cache from the projections' outputs,
read it back and attend over a window of it, on the host (fake, aligned device
addresses are never dereferenced on these paths), and the frequencies' fractions
of a turn against exact arithmetic."""
import ctypes
import math
from fractions import Fraction

import pytest
import torch

import mla_latent_kv_07_gb300 as mla
from mla_latent_kv_07_gb300 import build as mbuild

from test_abi_paged import FAKE, INVALID, POOLS, RANGE, UNSUPPORTED, at, pool

PI = Fraction("3.14159265358979323846264338327950288419716939937510582097494459")


@pytest.fixture(scope="module")
def L():
    mbuild.build()
    return mla.lib()


# ------------------------------------------------------------------ turns

@pytest.mark.parametrize("freq", [mla.rotary_frequencies(), mla.rotary_frequencies(factor=40.0), mla.rotary_frequencies(base=5e5),
                                  [0.0, -1.0, -1e-30, 6.283185307179586, 1e6, -1e6, 1e-300, 3.0] * 4])
def test_frequencies_become_fractions_of_a_turn(L, freq):
    # 1 / (2 pi) is held to 2^-109 of itself and the product with its first part is
    # exact, so what is left is one rounding to 2^-64 and 2^-53 of the second part's
    # product, below 2^-64 up to 10^6
    r = mla.Rotary(freq, device="cpu")
    for f, t in zip(freq, r.turns.tolist()):
        want = round(Fraction(f) / (2 * PI) * 2 ** 64)
        d = (t - want) % 2 ** 64
        assert min(d, 2 ** 64 - d) <= 2, f


def test_yarn_keeps_fast_columns_and_slows_slow_ones():
    plain, yarn = mla.rotary_frequencies(), mla.rotary_frequencies(factor=40.0)
    assert yarn[:10] == plain[:10] and all(abs(y * 40 / p - 1) < 1e-12 for y, p in zip(yarn[23:], plain[23:]))
    assert all(p / 40 <= y <= p for y, p in zip(yarn, plain))


def test_rotary_refuses_bad_frequencies(L):
    for bad in (float("nan"), float("inf"), 2e6):
        with pytest.raises(mla.MLAError):
            mla.Rotary([bad] * 32, device="cpu")
    with pytest.raises(ValueError):
        mla.Rotary([1.0] * 31, device="cpu")
    with pytest.raises(ValueError):
        mla.Rotary([1.0] * 32, gain=math.nan, device="cpu")
    out = (ctypes.c_uint64 * 1)()
    assert L.mla_rotary_turns(None, 1, out) == INVALID
    assert L.mla_rotary_turns((ctypes.c_double * 1)(1.0), 0, out) == INVALID


# ---------------------------------------------------------------- refusals

def write(L, cache, **kw):
    a = dict(table=at(), max_pages=4, kv=at(), kv_b=576, kv_s=576, norm=at(), f32=0, eps=1e-6, turns=FAKE, gain=1.0, halves=0,
             pos=at(), end=at(), B=2, s=3, q=at(), q_b=3 * 16 * 192, q_s=16 * 192, q_h=192, H=16, nope=at(), qpe=at(), status=None)
    a.update(kw)
    rot = None if a["turns"] is None else ctypes.byref(mla._CRotary(a["turns"], a["gain"], a["halves"]))
    return L.mla_paged_append_rotary(None if cache is None else ctypes.byref(cache), a["table"], a["max_pages"], a["kv"], a["kv_b"],
                                     a["kv_s"], a["norm"], a["f32"], a["eps"], rot, a["pos"], a["end"], a["B"], a["s"], a["q"],
                                     a["q_b"], a["q_s"], a["q_h"], a["H"], a["nope"], a["qpe"], a["status"], None)


def read(L, cache, **kw):
    a = dict(table=at(), max_pages=4, offsets=at(), first=None, B=2, total=100, kv=at(), kv_n=512, pe=at(), pe_n=64, status=None)
    a.update(kw)
    return L.mla_paged_read(None if cache is None else ctypes.byref(cache), a["table"], a["max_pages"], a["offsets"], a["first"],
                            a["B"], a["total"], a["kv"], a["kv_n"], a["pe"], a["pe_n"], a["status"], None)


@pytest.mark.parametrize("call", [write, read])
def test_bad_pools_and_tables_are_refused(L, call):
    assert call(L, None) == INVALID
    for kw, code in POOLS:
        assert call(L, pool(**kw)) == code, kw
    assert call(L, pool(), table=None) == INVALID
    assert call(L, pool(), table=at(2)) == INVALID
    assert call(L, pool(), max_pages=0) == INVALID
    assert call(L, pool(), B=0) == INVALID
    assert call(L, pool(), status=at(2)) == INVALID


@pytest.mark.parametrize("kw", [
    dict(kv=None), dict(kv=at(8)), dict(norm=None), dict(norm=at(8)), dict(turns=None), dict(turns=FAKE + 4), dict(pos=None),
    dict(pos=at(2)), dict(end=None), dict(end=at(1)), dict(kv_b=4), dict(kv_s=-576), dict(kv_s=577), dict(eps=-1e-6),
    dict(eps=math.nan), dict(eps=math.inf), dict(gain=math.nan), dict(gain=math.inf), dict(halves=2), dict(f32=2), dict(s=0),
    dict(B=1 << 16, s=1 << 15), dict(nope=None), dict(qpe=None), dict(q=None), dict(q=at(8)), dict(nope=at(8)), dict(qpe=at(8)),
    dict(q_h=196), dict(q_s=-192), dict(q_b=1), dict(B=1 << 13, s=1 << 11, H=128)])
def test_append_rotary_rejects_bad_arguments(L, kw):
    assert write(L, pool(), **kw) == INVALID


def test_append_rotary_rejects_other_heads(L):
    assert write(L, pool(), H=48) == UNSUPPORTED
    assert write(L, pool(), H=0) == UNSUPPORTED


@pytest.mark.parametrize("kw", [
    dict(offsets=None), dict(offsets=at(2)), dict(first=at(2)), dict(total=-1), dict(total=(1 << 30) + 1), dict(B=(1 << 30) + 1),
    dict(kv=None), dict(pe=None), dict(kv=at(8)), dict(pe=at(8)), dict(kv_n=511), dict(kv_n=504), dict(kv_n=516), dict(pe_n=56),
    dict(pe_n=68), dict(kv_n=-512)])
def test_read_rejects_bad_arguments(L, kw):
    assert read(L, pool(), **kw) == INVALID


def test_read_of_nothing_is_a_call(L):
    assert read(L, pool(), total=0, kv=None, pe=None) == 0


class Host:   # host tensors are on device -1, so the binding's own checks pass
    _dev, device = -1, torch.device("cpu")


def _host_write(**kw):
    a = dict(table=torch.zeros(2, 4, dtype=torch.int32), kv_a=torch.zeros(2, 3, 576, dtype=torch.bfloat16),
             norm_weight=torch.ones(512), eps=1e-6, rotary=mla.Rotary([1.0] * 32, device="cpu"),
             pos=torch.zeros(2, 3, dtype=torch.int32), end_pos=torch.zeros(2, dtype=torch.int32))
    a.update(kw)
    return mla.paged_append_rotary(Host, **a)


@pytest.mark.parametrize("kw", [
    dict(kv_a=torch.zeros(2, 3, 575, dtype=torch.bfloat16)), dict(kv_a=torch.zeros(2, 3, 576)),
    dict(kv_a=torch.zeros(2, 3, 1152, dtype=torch.bfloat16)[..., ::2]), dict(kv_a=torch.zeros(3, 3, 576, dtype=torch.bfloat16)),
    dict(norm_weight=torch.ones(511)), dict(norm_weight=torch.ones(512, dtype=torch.float64)),
    dict(norm_weight=torch.ones(1024)[::2]), dict(pos=torch.zeros(2, 3, dtype=torch.int64)), dict(end_pos=torch.zeros(3, dtype=torch.int32)),
    dict(table=torch.zeros(3, 4, dtype=torch.int32)), dict(table=torch.zeros(4, dtype=torch.int32)),
    dict(q=torch.zeros(2, 3, 16, 191, dtype=torch.bfloat16)), dict(q=torch.zeros(2, 3, 192, dtype=torch.bfloat16)),
    dict(q_pe=torch.zeros(2, 3, 16, 64, dtype=torch.bfloat16)), dict(status=torch.zeros(2, dtype=torch.int32)),
    dict(q=torch.zeros(2, 3, 16, 192, dtype=torch.bfloat16), q_nope=torch.zeros(2, 3, 16, 64, dtype=torch.bfloat16))])
def test_the_binding_refuses_other_tensors_to_write(L, kw):
    with pytest.raises(ValueError):
        _host_write(**kw)


def _host_read(**kw):
    a = dict(table=torch.zeros(2, 4, dtype=torch.int32), offsets=torch.zeros(3, dtype=torch.int32), total=10)
    a.update(kw)
    return mla.paged_read(Host, **a)


@pytest.mark.parametrize("kw", [
    dict(offsets=torch.zeros(3, dtype=torch.int64)), dict(offsets=torch.zeros(4, dtype=torch.int32)),
    dict(first=torch.zeros(3, dtype=torch.int32)), dict(kv=torch.zeros(9, 512, dtype=torch.bfloat16)),
    dict(kv=torch.zeros(10, 512)), dict(pe=torch.zeros(10, 128, dtype=torch.bfloat16)[:, ::2])])
def test_the_binding_refuses_other_tensors_to_read(L, kw):
    with pytest.raises(ValueError):
        _host_read(**kw)


@pytest.mark.parametrize("total", [-1, 2 ** 31, -2 ** 32 + 5])
def test_the_binding_refuses_other_totals(L, total):
    with pytest.raises(mla.MLAError) as err:
        _host_read(total=total)
    assert err.value.code in (INVALID, RANGE)


# ------------------------------------------------------------------ window

def window(L, cache, **kw):
    a = dict(table=at(), max_pages=4, q=at(), qp=at(), end=at(), max_end=256, B=2, s=3, H=128, scale=0.1, window=100, sinks=4,
             out=at(), lse=at(), ws=at(), ws_bytes=1 << 40)
    a.update(kw)
    return L.mla_paged_decode_window(None if cache is None else ctypes.byref(cache), a["table"], a["max_pages"], a["q"], a["qp"],
                                     a["end"], a["max_end"], a["B"], a["s"], a["H"], a["scale"], a["window"], a["sinks"], a["out"],
                                     a["lse"], a["ws"], a["ws_bytes"], None)


def test_window_refuses_bad_pools_and_tables(L):
    assert window(L, None) == INVALID
    for kw, code in POOLS:
        assert window(L, pool(**kw)) == code, kw


@pytest.mark.parametrize("kw,code", [
    (dict(table=None), INVALID), (dict(max_pages=0), INVALID), (dict(H=48), UNSUPPORTED), (dict(B=0), INVALID), (dict(B=65536), INVALID),
    (dict(s=0), INVALID), (dict(s=1025), INVALID), (dict(B=8192, s=1000), INVALID), (dict(max_end=257), RANGE), (dict(max_end=0), RANGE),
    (dict(window=0), INVALID), (dict(window=-1), INVALID), (dict(sinks=-1), INVALID), (dict(q=None), INVALID), (dict(qp=at(8)), INVALID),
    (dict(end=None), INVALID), (dict(end=at(2)), INVALID), (dict(out=at(8)), INVALID), (dict(lse=at(2)), INVALID),
    (dict(scale=math.nan), INVALID)])
def test_window_rejects_bad_arguments(L, kw, code):
    assert window(L, pool(), **kw) == code


def test_the_windows_self_test_refuses_what_its_call_refuses(L):
    def run(c, **kw):
        a = dict(max_end=256, window=10, out=at(), H=64)
        a.update(kw)
        return L.mla_selftest_paged_window_timeout(ctypes.byref(c), at(), 4, at(), at(), at(), a["max_end"], 2, 3, a["H"], 0.1, a["window"],
                                                   0, a["out"], at(), at(), 1 << 40, None)

    assert run(pool(page=24)) == UNSUPPORTED and run(pool(), H=48) == UNSUPPORTED
    assert run(pool(), max_end=257) == RANGE and run(pool(), window=0) == INVALID and run(pool(), out=None) == INVALID


def test_window_workspace_rejects_bad_arguments(L):
    for a in ((0, 1, 128), (65536, 1, 128), (1, 0, 128), (1, 1025, 128), (8192, 1000, 128), (4, 1, 24)):
        assert L.mla_paged_window_workspace_size(*a) == 0


@pytest.mark.parametrize("name", ["max_end_pos", "window", "sinks"])
@pytest.mark.parametrize("big", [2 ** 31, 2 ** 32 + 100, -2 ** 32 + 100])
def test_the_binding_refuses_window_numbers_past_32_bits(L, name, big):
    a = dict(max_end_pos=100, softmax_scale=0.1, window=10, sinks=2)
    a[name] = big
    with pytest.raises(mla.MLAError) as err:
        mla.paged_decode_window(Host, torch.zeros(1, 4, dtype=torch.int32), torch.zeros(1, 1, 16, 512, dtype=torch.bfloat16),
                                torch.zeros(1, 1, 16, 64, dtype=torch.bfloat16), torch.zeros(1, dtype=torch.int32),
                                workspace=torch.zeros(1, dtype=torch.uint8), **a)
    assert err.value.code == RANGE


@pytest.mark.parametrize("kw", [
    dict(q_latent=torch.zeros(1, 16, 512, dtype=torch.bfloat16)), dict(q_pe=torch.zeros(1, 2, 16, 64, dtype=torch.bfloat16)),
    dict(end_pos=torch.zeros(2, dtype=torch.int32)), dict(table=torch.zeros(2, 4, dtype=torch.int32)),
    dict(out=torch.zeros(1, 16, 512, dtype=torch.bfloat16)), dict(lse=torch.zeros(1, 16)), dict(workspace=torch.zeros(4))])
def test_the_binding_refuses_other_tensors_to_the_window(L, kw):
    a = dict(table=torch.zeros(1, 4, dtype=torch.int32), q_latent=torch.zeros(1, 1, 16, 512, dtype=torch.bfloat16),
             q_pe=torch.zeros(1, 1, 16, 64, dtype=torch.bfloat16), end_pos=torch.zeros(1, dtype=torch.int32))
    a.update({k: v for k, v in kw.items() if k in a})
    rest = {k: v for k, v in kw.items() if k not in a}
    with pytest.raises((ValueError, IndexError)):
        mla.paged_decode_window(Host, a["table"], a["q_latent"], a["q_pe"], a["end_pos"], 100, 0.1, 10,
                                **{**dict(workspace=torch.zeros(1, dtype=torch.uint8)), **rest})
