"""The host path of the paged calls: what the extension answers is what the
written-out way does (the same call with its stream named takes that), and what is
not as it should be is refused in the same words on either."""
import pytest
import torch

import mla_latent_kv_07_gb300 as mla

from paged_cases import Pool, randn_bf16

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from mla_latent_kv_07_gb300 import build
    build.build()
    mla.native()


def _write(cache, pool, stream=None, **kw):
    a = dict(kv_a=randn_bf16((2, 5, 576), 1).cuda(), norm_weight=torch.linspace(0.5, 1.5, 512, device="cuda"), eps=1e-6,
             rotary=mla.Rotary(mla.rotary_frequencies()), pos=torch.arange(10, dtype=torch.int32, device="cuda").view(2, 5),
             end_pos=pool.dev_ends(), q=randn_bf16((2, 5, 16, 192), 2).cuda())
    a.update(kw)
    return mla.paged_append_rotary(cache, pool.dev_table(), stream=stream, **a)


def _read(cache, pool, stream=None, **kw):
    a = dict(offsets=torch.tensor([0, 7, 20], dtype=torch.int32, device="cuda"), total=20,
             first=torch.tensor([3, 0], dtype=torch.int32, device="cuda"))
    a.update(kw)
    return mla.paged_read(cache, pool.dev_table(), stream=stream, **a)


def _window(cache, pool, stream=None, **kw):
    a = dict(q_latent=randn_bf16((2, 3, 16, 512), 3).cuda(), q_pe=randn_bf16((2, 3, 16, 64), 4).cuda(), end_pos=pool.dev_ends(),
             max_end_pos=60, softmax_scale=0.13, window=20, sinks=2)
    a.update(kw)
    return mla.paged_decode_window(cache, pool.dev_table(), stream=stream, **a)


CALLS = {"write": _write, "read": _read, "window": _window}


def same(x, y):
    return (x is None and y is None) or (x.dtype == y.dtype and x.shape == y.shape and torch.equal(x.view(torch.uint8), y.view(torch.uint8)))


@pytest.mark.parametrize("name", CALLS)
def test_both_ways_give_the_same(name):
    pool = Pool(1, [60, 33], 16, seed=50)
    c0, c1 = pool.device(), pool.device()
    a, b = CALLS[name](c0, pool), CALLS[name](c1, pool, stream=torch.cuda.current_stream())
    assert all(same(x, y) for x, y in zip(a, b))
    assert all(same(x, y) for x, y in ((c0.kv, c1.kv), (c0.kv_scale, c1.kv_scale), (c0.pe, c1.pe), (c0.weight, c1.weight)))


def test_the_plain_calls_go_through_the_extension(monkeypatch):
    took = []

    class Spy:
        def __getattr__(self, name):
            f = getattr(host, name)

            def call(*a):
                r = f(*a)
                took.append((name, type(r)))
                return r
            return call

    host = mla.native()
    monkeypatch.setattr(mla, "_host", Spy())
    pool = Pool(0, [60, 33], 16, seed=51)
    cache = pool.device()
    _write(cache, pool)
    _write(cache, pool, q=None)
    _read(cache, pool)
    _read(cache, pool, first=None)
    _window(cache, pool)
    _window(cache, pool, want_lse=False, workspace=mla.alloc_paged_window_workspace(2, 3, 16))
    assert took == [("append_rotary", tuple)] * 2 + [("read", tuple)] * 2 + [("decode_window", tuple)] * 2


@pytest.mark.parametrize("want", [True, False, 1, 0])
def test_the_sums_are_there_when_wanted(want):
    pool = Pool(0, [60, 33], 16, seed=52)
    out, lse = _window(pool.device(), pool, want_lse=want)
    assert (lse is not None) == bool(want)
    given = torch.empty(2, 3, 16, device="cuda")
    assert _window(pool.device(), pool, want_lse=False, lse=given)[1] is given


def test_given_outputs_are_used():
    pool = Pool(0, [60, 33], 16, seed=53)
    cache = pool.device()
    out, lse = torch.empty(2, 3, 16, 512, dtype=torch.bfloat16, device="cuda"), torch.empty(2, 3, 16, device="cuda")
    r = _window(cache, pool, out=out, lse=lse)
    assert r[0] is out and r[1] is lse and all(same(x, y) for x, y in zip(r, _window(cache, pool)))
    both = torch.zeros(20, 640, dtype=torch.bfloat16, device="cuda")
    r = _read(cache, pool, kv=both[:, :512], pe=both[:, 576:])
    want = _read(cache, pool)
    assert torch.equal(both[:, :512].view(torch.int16), want[0].view(torch.int16)) and torch.equal(both[:, 576:], want[1])
    assert bool((both[:, 512:576] == 0).all())


BAD = [  # (call, arguments, error)
    ("write", lambda: dict(kv_a=torch.zeros(2, 5, 576, device="cuda")), ValueError),
    ("write", lambda: dict(kv_a=torch.zeros(2, 5, 576, dtype=torch.bfloat16)), ValueError),
    ("write", lambda: dict(kv_a=torch.zeros(2, 5, 1152, dtype=torch.bfloat16, device="cuda")[..., ::2]), ValueError),
    ("write", lambda: dict(kv_a=torch.zeros(2, 5, 577, dtype=torch.bfloat16, device="cuda")[..., 1:]), mla.MLAError),
    ("write", lambda: dict(kv_a=torch.zeros(2, 5, 580, dtype=torch.bfloat16, device="cuda")[..., :576]), mla.MLAError),
    ("write", lambda: dict(norm_weight=torch.ones(512, dtype=torch.float16, device="cuda")), ValueError),
    ("write", lambda: dict(pos=torch.zeros(2, 5, dtype=torch.int64, device="cuda")), ValueError),
    ("write", lambda: dict(eps=-1.0), mla.MLAError),
    ("write", lambda: dict(end_pos=torch.zeros(3, dtype=torch.int32, device="cuda")), ValueError),
    ("write", lambda: dict(q=torch.zeros(2, 5, 24, 192, dtype=torch.bfloat16, device="cuda")), mla.MLAError),
    ("write", lambda: dict(q=None, q_pe=torch.zeros(2, 5, 16, 64, dtype=torch.bfloat16, device="cuda")), ValueError),
    ("write", lambda: dict(q_nope=torch.zeros(2, 5, 16, 64, dtype=torch.bfloat16, device="cuda")), ValueError),
    ("write", lambda: dict(rotary=mla.Rotary([1.0] * 32, device="cpu")), ValueError),
    ("read", lambda: dict(offsets=torch.zeros(4, dtype=torch.int32, device="cuda")), ValueError),
    ("read", lambda: dict(offsets=torch.zeros(3, dtype=torch.int64, device="cuda")), ValueError),
    ("read", lambda: dict(total=-1), mla.MLAError),
    ("read", lambda: dict(kv=torch.zeros(20, 516, dtype=torch.bfloat16, device="cuda")[:, :512]), mla.MLAError),
    ("read", lambda: dict(pe=torch.zeros(20, 64, device="cuda")), ValueError),
    ("read", lambda: dict(first=torch.zeros(2, device="cuda")), ValueError),
    ("window", lambda: dict(window=0), mla.MLAError),
    ("window", lambda: dict(sinks=-1), mla.MLAError),
    ("window", lambda: dict(sinks=2 ** 31), mla.MLAError),
    ("window", lambda: dict(max_end_pos=10 ** 6), mla.MLAError),
    ("window", lambda: dict(softmax_scale=float("nan")), mla.MLAError),
    ("window", lambda: dict(q_pe=torch.zeros(2, 3, 16, 64, device="cuda")), ValueError),
    ("window", lambda: dict(q_latent=torch.zeros(2, 3, 24, 512, dtype=torch.bfloat16, device="cuda"),
                            q_pe=torch.zeros(2, 3, 24, 64, dtype=torch.bfloat16, device="cuda"),
                            workspace=torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")), mla.MLAError),
    ("window", lambda: dict(workspace=torch.zeros(64, dtype=torch.uint8, device="cuda")), mla.MLAError),
    ("window", lambda: dict(out=torch.zeros(2, 3, 16, 1024, dtype=torch.bfloat16, device="cuda")[..., ::2]), ValueError),
    ("window", lambda: dict(end_pos=torch.zeros(2, dtype=torch.int32)), ValueError),
]


@pytest.mark.parametrize("named", [False, True])
@pytest.mark.parametrize("k", range(len(BAD)))
def test_refusals(k, named):
    name, make, error = BAD[k]
    pool = Pool(0, [60, 33], 16, seed=54)
    with pytest.raises(error):
        CALLS[name](pool.device(), pool, stream=torch.cuda.current_stream() if named else None, **make())
    torch.cuda.synchronize()


def test_a_dimension_of_one_may_have_any_stride():
    pool = Pool(0, [60], 16, seed=55)
    kv, q = randn_bf16((1, 1, 576), 5).cuda(), randn_bf16((1, 1, 16, 192), 6).cuda()
    args = dict(norm_weight=torch.ones(512, device="cuda"), pos=torch.ones(1, 1, dtype=torch.int32, device="cuda"), end_pos=pool.dev_ends())
    c0, c1 = pool.device(), pool.device()
    a = _write(c0, pool, kv_a=kv, q=q, **args)
    b = _write(c1, pool, kv_a=kv.as_strided((1, 1, 576), (3, 5, 1)), q=q.as_strided((1, 1, 16, 192), (7, 1, 192, 1)), **args)
    assert all(same(x, y) for x, y in zip(a, b)) and same(c0.kv, c1.kv) and same(c0.pe, c1.pe)


def test_a_pool_whose_tensors_are_replaced():
    pool = Pool(0, [60, 33], 16, seed=56)
    cache = pool.device()
    old = cache.kv
    cache.kv = old.clone()
    before = old.clone()
    _write(cache, pool)
    assert same(old, before) and not same(cache.kv, old)


def test_two_streams_at_once():
    pool = Pool(1, [60, 33], 16, seed=57)
    cache = pool.device()
    want = _window(cache, pool), _read(cache, pool)
    torch.cuda.synchronize()
    got = []
    for _ in range(8):
        for st in (torch.cuda.Stream(), torch.cuda.Stream()):
            with torch.cuda.stream(st):
                got.append((_window(cache, pool), _read(cache, pool)))
    torch.cuda.synchronize()
    for w, r in got:
        assert all(same(x, y) for x, y in zip(w, want[0])) and all(same(x, y) for x, y in zip(r, want[1]))


def test_write_and_read_captured_and_replayed():
    pool = Pool(1, [60, 33], 16, seed=58)
    cache, eager = pool.device(), pool.device()
    kv, q = randn_bf16((2, 5, 576), 7).cuda(), randn_bf16((2, 5, 16, 192), 8).cuda()
    pos, end = torch.arange(10, dtype=torch.int32, device="cuda").view(2, 5), pool.dev_ends()
    args = dict(kv_a=kv, q=q, pos=pos, end_pos=end, rotary=mla.Rotary(mla.rotary_frequencies()),
                norm_weight=torch.linspace(0.5, 1.5, 512, device="cuda"))
    table, off = pool.dev_table(), torch.tensor([0, 7, 20], dtype=torch.int32, device="cuda")
    call = lambda c: mla.paged_append_rotary(c, table, eps=1e-6, **args) + mla.paged_read(c, table, off, 20)
    call(pool.device())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = call(cache)
    for d in (0, 3):
        kv.copy_(randn_bf16((2, 5, 576), 9 + d))
        pos.add_(d)
        end.sub_(d)
        g.replay()
        want = call(eager)
        assert all(same(x, y) for x, y in zip(out, want)) and same(cache.kv, eager.kv) and same(cache.kv_scale, eager.kv_scale)
