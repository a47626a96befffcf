"""The paged cache's write from the projections' outputs and the reading of cached
rows, against fp64 references.

Bounds.  A rounding is off by half a step: u(bf16) = 2^-8, u(fp32) = 2^-24, e4m3
2^-4 of a normal value and 2^-10 of the scale below 2^-6 of it.
  latent   y = x r w: the sum of squares takes 11 roundings on its longest way (4 in
           a lane, 2 joins, 5 shuffles), the mean 1, eps 1, half of which the root
           keeps, then root, x r and w: 6.5 + 3 < 2^4 roundings of 2^-24: 2^-20 of y
  scale    amax / 448: 2^-20 + 2^-24 of it
  rotary   cos and sin: the angle in 2^-24 half turns, rounded from 32 bits to 24
           (2^-24 pi) and sincospif's last place (2^-23), the two products and their
           difference 3 u(fp32): below 2^-21 gain (|u| + |v|), then u(bf16) of the result
"""
import math

import numpy as np
import pytest
import torch

import mla_latent_kv_07_gb300 as mla
from oracle import oracle as orc

from mla_cases import bits, f64
from paged_cases import Pool, randn_bf16, within

pytestmark = pytest.mark.gpu
EPS = 1e-6
U_BF16 = 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def _built():
    from mla_latent_kv_07_gb300 import build
    build.build()
    mla.lib()


def rotate64(x, pos, freq, gain, halves):
    """x [..., 64] fp64 at pos (x's leading shape): (result, bound)."""
    a = pos.astype(np.float64)[..., None] * np.asarray(freq)
    c, s = gain * np.cos(a), gain * np.sin(a)
    u, v = (x[..., :32], x[..., 32:]) if halves else (x[..., 0::2], x[..., 1::2])
    p, q = u * c - v * s, v * c + u * s
    b = 2.0 ** -21 * abs(gain) * (np.abs(u) + np.abs(v))
    z, bz = np.empty_like(x), np.empty_like(x)
    if halves:
        z[..., :32], z[..., 32:], bz[..., :32], bz[..., 32:] = p, q, b, b
    else:
        z[..., 0::2], z[..., 1::2], bz[..., 0::2], bz[..., 1::2] = p, q, b, b
    return z, bz + U_BF16 * np.abs(z)


def norm64(x, w, eps):
    return x / np.sqrt((x ** 2).mean(-1, keepdims=True) + eps) * w


def check_rows(pool, cache, written, y):
    """Pool rows `written` hold y (fp64 [n, 512]); every other row is as it was."""
    n = pool.num_pages * pool.page
    keep = np.ones(n, bool)
    keep[written] = False
    if pool.fmt == 0:
        got = bits(cache.kv).reshape(-1, 512)
        assert np.array_equal(got[keep], pool.kv[keep])
        within(orc.bf16_bits_to_f64(got[written]), y, (U_BF16 + 2.0 ** -20) * np.abs(y), "latent")
    else:
        codes = cache.kv.cpu().numpy().reshape(-1, 512)
        scale = cache.kv_scale.cpu().numpy().reshape(-1, 4)
        assert np.array_equal(codes[keep], pool.kv[keep]) and np.array_equal(scale[keep].view(np.uint32), pool.scale[keep].view(np.uint32))
        amax = np.abs(y.reshape(-1, 4, 128)).max(-1)
        s = amax / 448.0
        if pool.fmt == 2:
            e = np.log2(np.where(amax > 0, s, 0.7))
            assert (np.abs(e - np.round(e)) > 2.0 ** -16).all(), "a scale next to a border: another seed"
            s = np.where(amax > 0, 2.0 ** np.ceil(e), 0.0)
            assert np.array_equal(scale[written], s)
        else:
            within(scale[written], s, (2.0 ** -20 + 2.0 ** -24) * s, "scale")
        sc = np.repeat(scale[written].astype(np.float64), 128, 1)
        val = torch.from_numpy(codes[written]).view(torch.float8_e4m3fn).float().numpy().astype(np.float64) * sc
        within(val, y, np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** -10 * sc) * (1 + 2.0 ** -10) + 2.0 ** -19 * np.abs(y), "codes")
    pe = bits(cache.pe).reshape(-1, 64)
    assert np.array_equal(pe[keep], pool.pe[keep])
    w = cache.weight.cpu().numpy().reshape(-1)
    assert np.array_equal(w[keep].view(np.uint32), pool.weight[keep].view(np.uint32)) and (w[written] == 0).all()
    return orc.bf16_bits_to_f64(pe[written])


def inputs_of(B, s, H, seed, spread=1.0, wide=0):
    g = torch.Generator().manual_seed(seed)
    kv = torch.randn(B, s, 576 + wide, generator=g) * (spread * torch.randn(B, s, 1, generator=g)).exp()
    kv = kv.to(torch.bfloat16)[..., wide:]
    w = (1 + 0.3 * torch.randn(512, generator=g))
    pos = torch.randint(0, 200000, (B, s), generator=g, dtype=torch.int32)
    q = None if H is None else torch.randn(B, s, H, 192, generator=g).to(torch.bfloat16)
    return kv, w, pos, q


def run_write(pool, B, s, H, seed, halves=False, gain=1.0, bf16_norm=True, freq=None, kv=None, pos=None, eps=EPS, **kw):
    kv_a, w, p, q = inputs_of(B, s, H, seed, **kw)
    kv_a, pos = (kv_a if kv is None else kv), (p if pos is None else pos)
    w = w.to(torch.bfloat16) if bf16_norm else w
    freq = mla.rotary_frequencies() if freq is None else freq
    cache = pool.device()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    rot = mla.Rotary(freq, interleaved=not halves, gain=gain)
    qn, qp = mla.paged_append_rotary(cache, pool.dev_table(), kv_a.cuda() if kv_a.is_contiguous() else _strided(kv_a), w.cuda(), eps,
                                     rot, pos.cuda(), pool.dev_ends(), q=None if q is None else q.cuda(), status=status)
    at, src = [], []
    for b in range(B):
        for j in range(s):
            t = int(pool.ends[b]) - s + j
            if 0 <= t < pool.max_pages * pool.page and 0 <= pool.table[b, t // pool.page] < pool.num_pages:
                at.append(int(pool.table[b, t // pool.page]) * pool.page + t % pool.page)
                src.append((b, j))
    at, ib, ij = np.array(at, np.int64), np.array([x[0] for x in src], np.int64), np.array([x[1] for x in src], np.int64)
    x = f64(kv_a)[ib, ij]
    y = norm64(x[:, :512], f64(w), eps)
    got = check_rows(pool, cache, at, y)
    z, bz = rotate64(x[:, 512:], pos.numpy()[ib, ij], freq, gain, halves)
    within(got, z, bz, "key")
    if q is not None:
        assert np.array_equal(bits(qn), bits(q[..., :128].contiguous()))
        z, bz = rotate64(f64(q[..., 128:]), np.repeat(pos.numpy()[..., None], q.shape[2], 2), freq, gain, halves)
        within(f64(qp), z, bz, "query")
    return cache, qn, qp, int(status), len(at)


def _strided(t):
    """t on the device, with the strides it has here."""
    base = torch.zeros(t.untyped_storage().nbytes() // t.element_size(), dtype=t.dtype)
    view = torch.as_strided(base, t.shape, t.stride(), t.storage_offset())
    view.copy_(t)
    return torch.as_strided(base.cuda(), t.shape, t.stride(), t.storage_offset())


WRITES = [  # (fmt, H, page, ends, s)
    (0, 16, 16, [1], 1), (0, 128, 64, [64, 65, 1, 300], 1), (1, 128, 64, [64, 65, 1, 300], 1), (2, 64, 48, [47, 48, 49], 1),
    (0, 32, 32, [33, 70], 33), (1, 16, 16, [100, 90, 97], 37), (0, 64, 80, [301], 301), (1, 128, 128, [129, 200], 129),
    (1, 32, 64, [7] * 9, 7), (0, 128, 16, [40] * 3, 5), (0, None, 64, [70, 64], 3), (1, None, 64, [70, 64], 3),
    (0, 16, 16, [500, 600, 700], 400), (1, 128, 64, [700] * 3, 211),
]


@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("fmt,H,page,ends,s", WRITES)
def test_rows_and_queries(fmt, H, page, ends, s, halves):
    pool = Pool(fmt, ends, page, seed=3 * s + page)
    _, _, _, status, n = run_write(pool, len(ends), s, H, seed=s + page, halves=halves, bf16_norm=not halves)
    assert status == 0 and n == len(ends) * s


@pytest.mark.parametrize("fmt", [0, 1])
def test_padded_and_overlong_sequences_leave_rows_out(fmt):
    # sequences of fewer positions than new rows (and one of none), and one past its table
    pool = Pool(fmt, [3, 0, 20, 64, -5], 16, seed=9, extra_pages=0)
    pool.ends[3] = 66                       # two positions behind the table's four pages
    _, _, _, status, n = run_write(pool, 5, 8, 16, seed=4)
    assert status == mla.DEV_APPEND_SKIPPED and n == 3 + 0 + 8 + 6


@pytest.mark.parametrize("fmt", [0, 1])
def test_rows_on_bad_pages_are_left_out(fmt):
    pool = Pool(fmt, [40, 33], 16, seed=10)
    pool.table[0, 1], pool.table[1, 2] = -1, pool.num_pages
    _, _, _, status, n = run_write(pool, 2, 30, 32, seed=5)
    assert status == mla.DEV_APPEND_SKIPPED | mla.DEV_BAD_PAGE and n == 60 - 16 - 1


@pytest.mark.parametrize("halves", [False, True])
def test_far_negative_and_extreme_positions(halves):
    pos = torch.tensor([[0, 1, -1, 2 ** 31 - 1, -2 ** 31, 1000003, 16777217, 99999999]], dtype=torch.int32)
    run_write(Pool(0, [8], 16, seed=11), 1, 8, 16, seed=6, pos=pos, halves=halves, gain=1.25,
              freq=mla.rotary_frequencies(factor=40.0))


def test_frequencies_past_a_turn_and_below_zero():
    freq = [100.0, -7.5, 0.0, 6.283185307179586] + [3.0 ** -i for i in range(28)]
    run_write(Pool(0, [40], 16, seed=12), 1, 40, 16, seed=7, freq=freq, gain=-0.5)


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("eps", [0.0, 1e-6, 3.0])
def test_rows_of_every_size(fmt, eps):
    # from rows whose squares leave 32 bits to rows far below eps
    size = 2.0 ** torch.tensor([0., 60., 63., 64., 66., 100., 119., -10., -20., -46., -50., -60., -90., -100.])
    kv = (torch.randn(1, size.numel(), 576, generator=torch.Generator().manual_seed(8)) * size[None, :, None]).to(torch.bfloat16)
    kv[..., 512:] = 1.0
    if eps == 1e-6 and fmt == 1:
        kv = kv[:, :10].contiguous()        # (an FP8 scale below 2^-126 has fewer bits)
    pool = Pool(fmt, [kv.shape[1]], 16, seed=13)
    run_write(pool, 1, kv.shape[1], None, seed=8, kv=kv, eps=eps)


def test_a_row_of_zeros_is_zeros():
    for fmt in (0, 1, 2):
        run_write(Pool(fmt, [2], 16, seed=14), 1, 2, None, seed=9, kv=torch.zeros(1, 2, 576, dtype=torch.bfloat16))


def test_nan_and_infinities_stay_in_their_rows():
    for fmt in (0, 1):
        pool = Pool(fmt, [6, 6], 16, seed=15)
        kv, w, pos, q = inputs_of(2, 6, 16, 10)
        bad = kv.clone()
        bad[0, 1, 7], bad[0, 3, 500], bad[1, 2, 520] = math.nan, math.inf, -math.inf
        qb = q.clone()
        qb[1, 4, 3, 150] = math.nan
        rot = mla.Rotary(mla.rotary_frequencies())
        got = []
        for a, qq in ((kv, q), (bad, qb)):
            cache = pool.device()
            got.append((cache, *mla.paged_append_rotary(cache, pool.dev_table(), a.cuda(), w.cuda(), EPS, rot, pos.cuda(),
                                                        pool.dev_ends(), q=qq.cuda())))
        (c0, n0, p0), (c1, n1, p1) = got
        clean = [r for b in range(2) for j, r in enumerate(pool.rows(b)) if (b, j) not in ((0, 1), (0, 3), (1, 2))]
        for x, y in ((c0.kv, c1.kv), (c0.pe, c1.pe)):
            assert torch.equal(x.flatten(0, 1)[clean].view(torch.uint8), y.flatten(0, 1)[clean].view(torch.uint8))
        m = torch.ones(2, 6, 16, dtype=torch.bool)
        m[1, 4, 3] = False
        assert torch.equal(p0[m.cuda()].view(torch.int16), p1[m.cuda()].view(torch.int16)) and bool(p1[1, 4, 3].isnan().any())
        if fmt == 0:
            assert bool(c1.kv.flatten(0, 1)[pool.rows(0)[1]].isnan().all())
            assert bool(c1.pe.flatten(0, 1)[pool.rows(1)[2]].isfinite().logical_not().any())


@pytest.mark.parametrize("wide", [8, 1024])
def test_strided_inputs(wide):
    pool = Pool(1, [30, 40], 16, seed=16)
    run_write(pool, 2, 12, 16, seed=11, wide=wide)
    # queries whose heads lie apart, and sequences that share one token's row (stride 0)
    kv, w, pos, q = inputs_of(2, 12, 32, 12)
    rot = mla.Rotary(mla.rotary_frequencies())
    qt = q.cuda().transpose(1, 2).contiguous().transpose(1, 2)
    c0, c1 = pool.device(), pool.device()
    one = kv[:, :1].expand(2, 12, 576)
    a = mla.paged_append_rotary(c0, pool.dev_table(), one.contiguous().cuda(), w.cuda(), EPS, rot, pos.cuda(), pool.dev_ends(), q=q.cuda())
    b = mla.paged_append_rotary(c1, pool.dev_table(), kv[:, :1].cuda().expand(2, 12, 576), w.cuda(), EPS, rot, pos.cuda(),
                                pool.dev_ends(), q=qt)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert torch.equal(c0.kv, c1.kv) and torch.equal(c0.pe.view(torch.int16), c1.pe.view(torch.int16))


def test_a_pool_without_weights_and_outputs_given():
    pool = Pool(0, [20, 20], 16, seed=17)
    kv, w, pos, q = inputs_of(2, 4, 16, 13)
    rot = mla.Rotary(mla.rotary_frequencies())
    c0, c1 = pool.device(), pool.device()
    c1.weight = None
    qn, qp = torch.empty(2, 4, 16, 128, dtype=torch.bfloat16, device="cuda"), torch.empty(2, 4, 16, 64, dtype=torch.bfloat16, device="cuda")
    a = mla.paged_append_rotary(c0, pool.dev_table(), kv.cuda(), w.cuda(), EPS, rot, pos.cuda(), pool.dev_ends(), q=q.cuda())
    b = mla.paged_append_rotary(c1, pool.dev_table(), kv.cuda(), w.cuda(), EPS, rot, pos.cuda(), pool.dev_ends(), q=q.cuda(),
                                q_nope=qn, q_pe=qp)
    assert b[0] is qn and b[1] is qp and torch.equal(a[0], qn) and torch.equal(a[1], qp)
    assert torch.equal(c0.kv.view(torch.int16), c1.kv.view(torch.int16))


@pytest.mark.parametrize("fmt", [0, 1])
def test_tokens_one_at_a_time_or_together_are_the_same(fmt):
    B, s, H = 3, 9, 16
    pool = Pool(fmt, [20, 9, 33], 16, seed=18)
    kv, w, pos, q = inputs_of(B, s, H, 14)
    rot = mla.Rotary(mla.rotary_frequencies(), gain=0.9)
    c0, c1 = pool.device(), pool.device()
    qn, qp = mla.paged_append_rotary(c0, pool.dev_table(), kv.cuda(), w.cuda(), EPS, rot, pos.cuda(), pool.dev_ends(), q=q.cuda())
    for j in range(s):
        n, p = mla.paged_append_rotary(c1, pool.dev_table(), kv[:, j:j + 1].cuda(), w.cuda(), EPS, rot, pos[:, j:j + 1].contiguous().cuda(),
                                       pool.dev_ends() - s + 1 + j, q=q[:, j:j + 1].cuda())
        assert torch.equal(n[:, 0], qn[:, j]) and torch.equal(p[:, 0], qp[:, j])
    for x, y in ((c0.kv, c1.kv), (c0.pe, c1.pe)):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


# -------------------------------------------------------------------- read

def expected_rows(pool, b, first, n):
    """bf16 bits of positions first .. first + n - 1 of sequence b (zeros where there is none)."""
    kv, pe, bad = np.zeros((n, 512), np.uint16), np.zeros((n, 64), np.uint16), False
    for i in range(n):
        t = first + i
        pg = pool.table[b, t // pool.page] if 0 <= t < pool.max_pages * pool.page else -1
        if not 0 <= pg < pool.num_pages:
            bad = True
            continue
        r = int(pg) * pool.page + t % pool.page
        kv[i] = pool.kv[r] if pool.fmt == 0 else orc.dequant_rows(pool.kv[r:r + 1], pool.scale[r:r + 1])[0]
        pe[i] = pool.pe[r]
    return kv, pe, bad


READS = [  # (fmt, page, ends, first)
    (0, 16, [1], None), (1, 16, [17, 0, 33, 16], None), (2, 48, [129, 48, 1], [100, 0, 0]), (0, 64, [300, 0, 0, 65], [13, 0, 0, 64]),
    (1, 80, [333, 200], [5, 199]), (0, 128, [500] * 3, None), (1, 16, [3] * 70, [0, 1, 2, 3, 2] * 14), (1, 64, [0, 0, 5, 0], None),
]


@pytest.mark.parametrize("together", [False, True])
@pytest.mark.parametrize("fmt,page,ends,first", READS)
def test_read_back(fmt, page, ends, first, together):
    pool = Pool(fmt, ends, page, seed=21 + page)
    f = [0] * len(ends) if first is None else first
    count = [e - x for e, x in zip(ends, f)]
    off = np.concatenate([[0], np.cumsum(count)]).astype(np.int32)
    n = int(off[-1])
    want = [expected_rows(pool, b, f[b], count[b]) for b in range(len(ends))]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kv = pe = None
    if together:
        both = torch.zeros(n, 576, dtype=torch.bfloat16, device="cuda")
        kv, pe = both[:, :512], both[:, 512:]
    kv, pe = mla.paged_read(pool.device(), pool.dev_table(), torch.from_numpy(off).cuda(), n,
                            first=None if first is None else torch.tensor(first, dtype=torch.int32).cuda(), kv=kv, pe=pe, status=status)
    assert np.array_equal(bits(kv.contiguous()), np.concatenate([w[0] for w in want]))
    assert np.array_equal(bits(pe.contiguous()), np.concatenate([w[1] for w in want])) and int(status) == 0


@pytest.mark.parametrize("fmt", [0, 1])
def test_rows_outside_the_offsets_stay_and_bad_pages_are_zeros(fmt):
    pool = Pool(fmt, [60, 40], 16, seed=22)
    pool.table[0, 2] = -3
    off = torch.tensor([5, 55, 70], dtype=torch.int32).cuda()
    first = torch.tensor([10, -4], dtype=torch.int32).cuda()      # the second starts before its first position
    kv, pe = torch.full((100, 512), 7.0, dtype=torch.bfloat16, device="cuda"), torch.full((100, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    mla.paged_read(pool.device(), pool.dev_table(), off, 100, first=first, kv=kv, pe=pe, status=status)
    a, b = expected_rows(pool, 0, 10, 50), expected_rows(pool, 1, -4, 15)
    assert np.array_equal(bits(kv[5:70]), np.concatenate([a[0], b[0]])) and np.array_equal(bits(pe[5:70]), np.concatenate([a[1], b[1]]))
    assert bool((kv[:5] == 7).all() and (kv[70:] == 7).all() and (pe[:5] == 7).all() and (pe[70:] == 7).all())
    assert int(status) == mla.DEV_BAD_PAGE


def test_offsets_past_the_total_are_cut():
    pool = Pool(1, [60, 40], 16, seed=23)
    off = torch.tensor([0, 60, 100], dtype=torch.int32).cuda()
    kv, _ = mla.paged_read(pool.device(), pool.dev_table(), off, 65)
    a, b = expected_rows(pool, 0, 0, 60), expected_rows(pool, 1, 0, 5)
    assert np.array_equal(bits(kv), np.concatenate([a[0], b[0]]))
    kv, pe = mla.paged_read(pool.device(), pool.dev_table(), off, 0)
    assert kv.shape == (0, 512) and pe.shape == (0, 64)


def test_many_short_sequences():
    rng = np.random.default_rng(5)
    ends = rng.integers(0, 4, 3000)
    pool = Pool(0, ends, 16, seed=24)
    off = np.concatenate([[0], np.cumsum(ends)]).astype(np.int32)
    kv, _ = mla.paged_read(pool.device(), pool.dev_table(), torch.from_numpy(off).cuda(), int(off[-1]))
    rows = np.concatenate([pool.rows(b) for b in range(len(ends))]).astype(np.int64)
    assert np.array_equal(bits(kv), pool.kv[rows])


def test_what_was_written_is_read():
    # a bf16 pool gives back the bits that the write rounded; an FP8 one the values its rows stand for
    for fmt in (0, 1, 2):
        pool = Pool(fmt, [50, 31], 16, seed=25)
        cache, _, _, _, _ = run_write(pool, 2, 31, None, seed=15)
        off = torch.tensor([0, 31, 62], dtype=torch.int32).cuda()
        kv, pe = mla.paged_read(cache, pool.dev_table(), off, 62, first=(pool.dev_ends() - 31))
        rows = np.concatenate([pool.rows(0)[19:], pool.rows(1)]).astype(np.int64)
        raw = cache.kv.flatten(0, 1).cpu()[rows]
        want = bits(raw) if fmt == 0 else orc.dequant_rows(raw.numpy(), cache.kv_scale.flatten(0, 1).cpu().numpy()[rows])
        assert np.array_equal(bits(kv), want) and np.array_equal(bits(pe), bits(cache.pe.flatten(0, 1).cpu()[rows]))
