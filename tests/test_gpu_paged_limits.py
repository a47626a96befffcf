"""The paged cache's write, reading and windowed attention at the ends of their
ranges, against fp64 references."""
import numpy as np
import pytest
import torch

import mla_latent_kv_07_gb300 as mla

from oracle import oracle as orc

from mla_cases import bits, f64
from paged_cases import Pool, randn_bf16, reference, within

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


SM = 0.1352


def _windowed(pool, ql, qp, window, sinks, few=0):
    """paged_decode_window against fp64, where a weight's rounding to bf16 changes the
    output by no more than normalised weights allow.  P_i = p_i (1 + d_i), |d_i| <= 2^-8, and the
    output is sum P_i c_i / sum P_i: to first order it is off by sum w_i d_i (c_i - out), so by
    2^-8 sum w_i |c_i - out| (a token that sees up to `few` positions: without the largest
    weight's, which bf16 holds), with (1 + 2^-6) for what is beyond first order.  The scores' part is that of paged_cases.py:
    |dw_i| <= 2 ds w_i; fp32 sums 2^-16.  The output is rounded once, 2^-8."""
    s, H = ql.shape[1:3]
    e = int(pool.ends[0])
    out, lse = mla.paged_decode_window(pool.device(), pool.dev_table(), ql.cuda(), qp.cuda(), pool.dev_ends(),
                                       pool.max_pages * pool.page, SM, window, sinks=sinks)
    rows = pool.rows(0)
    c = orc.bf16_bits_to_f64(pool.kv[rows] if pool.scale is None else orc.dequant_rows(pool.kv[rows], pool.scale[rows]))
    k = np.concatenate([c, orc.bf16_bits_to_f64(pool.pe[rows])], -1)
    q = np.concatenate([f64(ql), f64(qp)], -1)[0]
    worst = 0.0
    for j in range(s):
        t = e - s + j
        seen = np.array([p for p in range(t + 1) if p < sinks or p > t - window])
        sc = SM * q[j] @ k[seen].T
        top = sc.max(1, keepdims=True)
        w = np.exp(sc - top)
        norm = w.sum(1, keepdims=True)
        w /= norm
        ref, x = w @ c[seen], c[seen]
        ds = (64 * 2.0 ** -23 * SM * np.abs(q[j]) @ np.abs(k[seen]).T + 2.0 ** -16).max(1, keepdims=True)
        r = w.copy()
        if seen.size <= few:
            np.put_along_axis(r, w.argmax(1)[:, None], 0.0, 1)
        apart = np.stack([r[h] @ np.abs(x - ref[h]) for h in range(H)])
        bound = 2.0 ** -8 * (np.abs(ref) + (1 + 2.0 ** -6) * apart) + (2 * ds + 2.0 ** -16) * (w @ np.abs(x))
        worst = max(worst, float((np.abs(f64(out[0, j]) - ref) / bound).max()))
        within(f64(lse[0, j]), (top + np.log(norm))[:, 0], ds[:, 0], "lse")
    assert worst <= 1, f"{worst:.3f} of its bound"


@pytest.mark.parametrize("fmt,H,s", [(0, 16, 1), (1, 32, 2), (0, 64, 1), (0, 128, 1), (0, 16, 161), (1, 16, 163), (0, 32, 150),
                                     (1, 32, 141), (0, 64, 140), (1, 64, 150), (0, 128, 70), (1, 128, 65), (1, 128, 1), (1, 128, 3), (2, 128, 6)])
def test_a_dominant_position_leaves_no_rounding_of_its_weight(fmt, H, s):
    # position 0, which all tokens see, outweighs the others by e^8 to e^14, other
    # amounts per head; its weight is rounded, which the division takes out again
    e = s + 90
    g = np.random.default_rng(H + s)
    u = np.sign(g.standard_normal(512))
    base = Pool(fmt, [e], 16, seed=61)
    x = g.standard_normal((base.num_pages * 16, 512)) * 0.5
    x[base.rows(0)[0]] = u * np.exp(0.3 * g.standard_normal(512))
    pool = Pool(fmt, [e], 16, seed=61, kv=bits(torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16)))
    amount = np.linspace(10.0, 16.0, H) / (SM * 512 * 1.05)
    ql = torch.from_numpy(np.outer(amount, u) + 0.02 * g.standard_normal((1, s, H, 512))).to(torch.bfloat16)
    _windowed(pool, ql, randn_bf16((1, s, H, 64), 62) * 0.1, 33, 1)


@pytest.mark.parametrize("fmt,H,s", [(0, 16, 8), (1, 64, 8), (0, 128, 8), (1, 128, 8), (2, 128, 9), (0, 64, 130), (1, 128, 64)])
def test_a_dominant_position_behind_the_first_tile(fmt, H, s):
    # position 620 outweighs the others, by less than would move the reference that position 540
    # sets in an earlier tile; position 540 is e^6.5 and more above the rest
    e = 992 + s
    g = np.random.default_rng(H + s)
    u = np.sign(g.standard_normal(512))
    base = Pool(fmt, [e], 16, seed=65)
    x = 0.02 * g.standard_normal((base.num_pages * 16, 512))
    x[base.rows(0)] -= u
    x[base.rows(0)[540]] += u
    x[base.rows(0)[620]] += 1.6 * u * np.exp(0.05 * g.standard_normal(512))
    pool = Pool(fmt, [e], 16, seed=65, kv=bits(torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16)))
    amount = np.linspace(6.5, 8.6, H) / (SM * 512)
    ql = torch.from_numpy(np.outer(amount, u) + 0.001 * g.standard_normal((1, s, H, 512))).to(torch.bfloat16)
    _windowed(pool, ql, randn_bf16((1, s, H, 64), 66) * 0.05, 900, 0)


@pytest.mark.parametrize("fmt,H,s", [(0, 16, 1), (1, 64, 3), (0, 32, 15), (0, 16, 165), (1, 16, 166), (0, 32, 161), (1, 32, 162), (0, 64, 133), (1, 128, 2),
                                     (1, 128, 15)])
def test_the_largest_weight_of_few_positions_is_exact(fmt, H, s):
    # token j sees j + 2 positions; among the units' tokens some see up to 16 and some
    # more.  Positions 0 and 1, of about equal weight, outweigh the others
    g = np.random.default_rng(H + s)
    u, v = np.sign(g.standard_normal((2, 512)))
    base = Pool(fmt, [s + 1], 16, seed=63)
    x = g.standard_normal((base.num_pages * 16, 512)) * 0.3
    x[base.rows(0)[0]], x[base.rows(0)[1]] = u + 0.5 * v, u - 0.5 * v
    pool = Pool(fmt, [s + 1], 16, seed=63, kv=bits(torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16)))
    amount = np.linspace(4.0, 16.0, H) / (SM * 512)
    ql = torch.from_numpy(np.outer(amount, u) + 0.02 * g.standard_normal((1, s, H, 512))).to(torch.bfloat16)
    _windowed(pool, ql, randn_bf16((1, s, H, 64), 64) * 0.1, 1000, 0, few=16)


@pytest.mark.parametrize("empty", [0, 1, 3, 4, 5, 6, 100, 1 << 21])
def test_empty_sequences_between_rows_of_one_block(empty):
    # rows of three sequences, with so many empty ones before, between and behind them, in
    # two blocks of 16: what is found by a walk over them would take tens of milliseconds
    pool = Pool(0, [7, 9, 5], 16, seed=67)
    at = [empty, 2 * empty + 1, 3 * empty + 2]
    B = 4 * empty + 3
    count, table = np.zeros(B, np.int64), np.full((B, pool.max_pages), -1, np.int32)
    count[at], table[at] = [7, 9, 5], pool.table
    off = np.concatenate([[0], np.cumsum(count)]).astype(np.int32)
    args = (pool.device(), torch.from_numpy(table).cuda(), torch.from_numpy(off).cuda(), 21)
    kv, pe = mla.paged_read(*args)
    rows = np.concatenate([pool.rows(b) for b in range(3)]).astype(np.int64)
    assert np.array_equal(bits(kv), pool.kv[rows]) and np.array_equal(bits(pe), pool.pe[rows])
    ms = []
    for _ in range(5):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        mla.paged_read(*args)
        b.record()
        b.synchronize()
        ms.append(a.elapsed_time(b))
    assert min(ms) < 2.0


@pytest.mark.parametrize("fmt,H,s,window", [(0, 16, 1, 60), (1, 64, 1, 60), (0, 128, 1, 60), (1, 128, 1, 60), (0, 16, 170, 9), (1, 32, 170, 9),
                                            (0, 64, 150, 120), (1, 64, 150, 120), (0, 128, 70, 300), (1, 128, 70, 300)])
def test_infinite_values_are_nan_or_weigh_nothing(fmt, H, s, window):
    # the row's score is -infinity for some heads, NaN or infinity for others: a token that
    # sees the row gives NaN or what it gives without it, value by value; the others the same bits
    e = max(s + 10, 80)
    hit = e - s + s // 2 if s > 1 else e - 20
    pool = Pool(fmt, [e], 16, seed=68)
    ql, qp = randn_bf16((1, s, H, 512), 69), randn_bf16((1, s, H, 64), 70)
    ql[0, :, ::3, :128] = -ql[0, :, ::3, :128].abs()
    args = lambda: (pool.dev_table(), ql.cuda(), qp.cuda(), pool.dev_ends(), e, SM, window)
    good = mla.paged_decode_window(pool.device(), *args(), sinks=2)
    rows = pool.rows(0).astype(np.int64)
    if fmt == 0:
        pool.kv[rows[hit], 5:128:40] = 0x7F80
    else:
        pool.scale[rows[hit], 0] = np.inf
        pool.kv[rows[hit], :128] &= 0x7F          # (positive codes)
        pool.kv[rows[hit], :128] |= 0x08
        pool.kv[rows[hit], :128] &= 0x7E
    bad = mla.paged_decode_window(pool.device(), *args(), sinks=2)
    t = np.arange(e - s, e)
    sees = (t >= hit) & (t < hit + window)
    assert sees.any() and (s == 1 or not sees.all())
    for x, y in zip(good, bad):
        assert torch.equal(x[0, torch.from_numpy(~sees).cuda()], y[0, torch.from_numpy(~sees).cuda()])
    q = np.concatenate([f64(ql), f64(qp)], -1)[0]
    c = orc.bf16_bits_to_f64(pool.kv[rows] if fmt == 0 else orc.dequant_rows(pool.kv[rows], pool.scale[rows]))
    k = np.concatenate([c, orc.bf16_bits_to_f64(pool.pe[rows])], -1)
    for j in np.flatnonzero(sees):
        seen = np.array([p for p in range(t[j] + 1) if (p < 2 or p > t[j] - window) and p != hit])
        sc = SM * q[j] @ k[seen].T
        top = sc.max(1, keepdims=True)
        w = np.exp(sc - top)
        norm = w.sum(1, keepdims=True)
        w /= norm
        ref, lse = w @ c[seen], (top + np.log(norm))[:, 0]
        wc = w @ np.abs(c[seen])
        ds = (64 * 2.0 ** -23 * SM * np.abs(q[j]) @ np.abs(k[seen]).T + 2.0 ** -16).max(1, keepdims=True)
        got, gl = f64(bad[0][0, j]), f64(bad[1][0, j])
        # (bounds of paged_cases.py)
        near = np.abs(got - ref) <= 2.0 ** -8 * (np.abs(ref) + wc) + (2 * ds + 2.0 ** -16) * wc
        assert (np.isnan(got) | near).all() and (np.isnan(gl) | (np.abs(gl - lse) <= ds[:, 0] + 2.0 ** -16)).all()
        lost = np.isnan(got).all(1) & np.isnan(gl)
        with np.errstate(invalid="ignore"):
            weighs = np.isneginf(SM * np.where(np.isinf(k[hit]), q[j] * k[hit], 0.0).sum(1))
        assert (lost | weighs).all() and not weighs.all()


@pytest.mark.parametrize("fmt,H", [(0, 16), (1, 64), (1, 128)])
def test_several_tokens_over_everything_and_their_weights(fmt, H):
    # a window of at least the length: several tokens in one call, and the weight that they
    # gave the rows, each token as a sequence of its own
    B, s, ends = 2, 3, np.array([150, 70], np.int32)
    pool = Pool(fmt, ends, 16, seed=73)
    cache, table, T = pool.device(), pool.dev_table(), 160
    ql, qp = randn_bf16((B, s, H, 512), 74), randn_bf16((B, s, H, 64), 75)
    out, lse = mla.paged_decode_window(cache, table, ql.cuda(), qp.cuda(), pool.dev_ends(), T, SM, window=T)
    each = (pool.dev_ends()[:, None] - s + 1 + torch.arange(s, dtype=torch.int32, device="cuda")).view(-1)
    mla.paged_weights(cache, table.repeat_interleave(s, 0), ql.view(B * s, H, 512).cuda(), qp.view(B * s, H, 64).cuda(),
                      lse.view(B * s, H), each, T, SM)
    total, bound = pool.weight.astype(np.float64), np.zeros(pool.weight.shape)
    for j in range(s):
        o, l, w, bo, bl, bw = reference(pool, ql[:, j].contiguous(), qp[:, j].contiguous(), SM, ends=ends - s + 1 + j)
        within(f64(out[:, j]), o, bo, "out")
        within(f64(lse[:, j]), l, bl, "lse")
        for b in range(B):
            at = pool.rows(b, ends[b] - s + 1 + j)
            total[at] += w[b]
            bound[at] += bw[b]
    got = cache.weight.cpu().numpy().reshape(-1)
    live = pool.live
    # (the additions to the running weight are rounded, once a token; a sum over heads, H 2^-24,
    # lies within the scores' part, which is 2^-15 and more)
    within(got[live], total[live], bound[live] + s * 2.0 ** -23 * total[live], "weight")
