"""Attention with a sliding window and sinks over a paged cache against the fp64
oracle on the positions that each token sees, with the bounds of paged_cases.py.
Rows that no token sees hold NaN, and pages without a seen row are out of range
in the table (given back)."""
import numpy as np
import pytest
import torch

import mla_latent_kv_07_gb300 as mla

from oracle import oracle as orc

from mla_cases import bits, f64
from paged_cases import Pool, randn_bf16, reference, within

pytestmark = pytest.mark.gpu
SM = 0.1352


@pytest.fixture(scope="module", autouse=True)
def _built():
    from mla_latent_kv_07_gb300 import build
    build.build()
    mla.lib()


def seen(end, s, j, window, sinks):
    """Positions that token j of s sees, in order."""
    t = end - s + j
    return np.array([p for p in range(t + 1) if p < sinks or p > t - window], np.int64)


def hide(pool, s, window, sinks, pages=True):
    """NaN in the rows that no token sees, and out-of-range entries for their pages."""
    for b, e in enumerate(pool.ends):
        rows = pool.rows(b).astype(np.int64)
        m = np.zeros(rows.size, bool)
        for j in range(s):
            m[seen(int(e), s, j, window, sinks)] = True
        off = rows[~m]
        pool.kv[off] = 0x7FC0 if pool.fmt == 0 else 0x7F
        if pool.scale is not None:
            pool.scale[off] = np.nan
        pool.pe[off] = 0x7FC0
        if pages:
            for k in range(-(-rows.size // pool.page)):
                if not m[k * pool.page:(k + 1) * pool.page].any():
                    pool.table[b, k] = -1 - k


def expected(pool, ql, qp, window, sinks, scale=SM, rows=None, bad=None):
    """(out, lse, bounds) [B, s, ...] in fp64; tokens before a sequence's first position: 0, -inf.
    bad: per sequence, positions that are left out."""
    B, s, H = ql.shape[:3]
    keep = pool.rows
    all_rows = [keep(b) if rows is None else rows[b] for b in range(B)]
    parts = []
    for j in range(s):
        idx = [seen(int(e), s, j, window, sinks) for e in pool.ends]
        if bad is not None:
            idx = [i[~np.isin(i, bad[b])] for b, i in enumerate(idx)]
        pool.rows = lambda b, n=None: all_rows[b][idx[b]]
        o, l, _, bo, bl, _ = reference(pool, ql[:, j].contiguous(), qp[:, j].contiguous(), scale, ends=[i.size for i in idx])
        parts.append((o, l, bo, bl))
    pool.rows = keep
    return [np.stack([p[k] for p in parts], 1) for k in range(4)]


def run(pool, s, H, window, sinks, seed, scale=SM, max_end=None, cache=None, status=0, rows=None, **kw):
    B = len(pool.ends)
    ql, qp = randn_bf16((B, s, H, 512), seed), randn_bf16((B, s, H, 64), seed + 1)
    cache = pool.device() if cache is None else cache
    ws = mla.alloc_paged_window_workspace(B, s, H)
    out, lse = mla.paged_decode_window(cache, pool.dev_table(), ql.cuda(), qp.cuda(), pool.dev_ends(),
                                       pool.max_pages * pool.page if max_end is None else max_end, scale, window, sinks=sinks,
                                       workspace=ws, **kw)
    ref, rl, bo, bl = expected(pool, ql, qp, window, sinks, scale, rows)
    within(f64(out), ref, bo, "out")
    within(f64(lse), rl, bl, "lse")
    assert mla.workspace_status(ws) == status
    return out, lse, ws


WINDOWS = [  # (fmt, H, page, ends, s, window, sinks)
    (0, 16, 16, [1], 1, 1, 0), (0, 16, 16, [100, 16, 17, 0], 1, 16, 4), (1, 16, 48, [100, 300], 1, 33, 0),
    (0, 32, 32, [200, 77], 1, 64, 20), (1, 32, 16, [500, 31, 1], 1, 100, 1), (0, 64, 64, [513, 129, 0], 1, 128, 16),
    (1, 64, 80, [400, 81], 1, 17, 17), (2, 64, 16, [640, 31], 1, 300, 100), (0, 128, 64, [300, 33, 1], 1, 47, 4),
    (1, 128, 64, [1000, 513, 2, 64], 1, 96, 3), (0, 128, 16, [257, 400], 1, 1, 1), (2, 128, 256, [511, 0, 513], 1, 200, 33),
    (0, 128, 1024, [2000, 5], 1, 700, 50), (1, 16, 64, [3000], 1, 2000, 4), (0, 16, 64, [3000], 1, 2000, 4),
    (0, 64, 112, [1501, 800], 1, 777, 31), (1, 128, 48, [640, 97, 47], 1, 500, 16),
    # several tokens: of sequences longer and shorter than their number
    (0, 16, 16, [40, 3, 0], 5, 16, 2), (1, 16, 32, [400, 7], 8, 100, 4), (0, 32, 64, [300, 65], 3, 64, 0),
    (1, 32, 32, [900, 2], 6, 512, 16), (0, 64, 16, [77, 200], 4, 31, 1), (1, 64, 48, [130, 4], 7, 48, 5),
    (0, 128, 64, [300, 5], 6, 100, 4), (1, 128, 16, [129, 1], 9, 33, 17), (2, 128, 64, [200], 2, 64, 64),
    # more tokens than a warp schedules
    (0, 16, 64, [200, 90, 10], 50, 40, 4), (1, 32, 16, [150, 300], 70, 100, 0), (0, 64, 32, [333], 130, 64, 8),
    (0, 128, 64, [160, 20], 67, 50, 4), (1, 128, 64, [140, 333], 65, 90, 1),
    # 64 columns (token, head) at a time: units of four, two and one tokens, some not
    # full, of sequences with fewer positions than tokens, and half tokens
    (0, 16, 64, [200, 90, 10], 61, 40, 4), (1, 16, 48, [300, 77, 0], 77, 100, 17), (0, 32, 16, [150, 300, 39, 41], 41, 33, 0),
    (1, 32, 32, [150, 300, 39, 41], 43, 128, 5), (0, 64, 32, [333], 150, 64, 8), (1, 64, 80, [200, 63], 80, 1, 3),
    (0, 128, 64, [500, 30], 31, 200, 4), (1, 128, 16, [90, 400], 33, 70, 40), (2, 16, 16, [400], 400, 64, 1),
    (0, 16, 128, [700], 640, 1000, 0), (0, 128, 16, [257], 60, 1, 0), (1, 64, 64, [130] * 130, 1, 40, 4),
    # windows and sinks that cover everything
    (0, 16, 16, [100, 50], 2, 1000, 0), (1, 128, 64, [100, 50], 2, 2 ** 31 - 1, 2 ** 31 - 1), (0, 64, 64, [100, 50], 1, 1, 1000),
]


@pytest.mark.parametrize("fmt,H,page,ends,s,window,sinks", WINDOWS)
def test_all_outputs(fmt, H, page, ends, s, window, sinks):
    pool = Pool(fmt, ends, page, seed=7 * H + page)
    rows = [pool.rows(b).astype(np.int64) for b in range(len(ends))]
    hide(pool, s, window, sinks)
    run(pool, s, H, window, sinks, seed=H + page, rows=rows)


@pytest.mark.parametrize("fmt,H", [(0, 16), (1, 32), (0, 64), (1, 64), (0, 128), (1, 128)])
def test_long_windows_are_split_over_the_gpu(fmt, H):
    pool = Pool(fmt, [9001, 20, 6097], 64, seed=H)
    rows = [pool.rows(b).astype(np.int64) for b in range(3)]
    hide(pool, 1, 5003, 37)
    run(pool, 1, H, 5003, 37, seed=H + 5, rows=rows)


@pytest.mark.parametrize("fmt,H", [(0, 16), (1, 64), (0, 128), (1, 128)])
def test_more_sequences_than_a_warp_schedules(fmt, H):
    rng = np.random.default_rng(H)
    run(Pool(fmt, rng.integers(0, 200, 333), 16, seed=H + 1), 1, H, 50, 3, seed=H + 2)


@pytest.mark.parametrize("fmt,H,B,window", [(0, 16, 80, 1100), (1, 64, 77, 1100), (0, 128, 40, 900), (1, 128, 40, 900)])
def test_long_windows_of_many_sequences_are_balanced(fmt, H, B, window):
    # (too long for equal parts of a few tiles: the schedule of the plain decode)
    rng = np.random.default_rng(B)
    ends = rng.integers(0, 1300, B)
    ends[:3] = 1300, 0, 1
    run(Pool(fmt, ends, 64, seed=H + 2), 1, H, window, 20, seed=H + 3)


@pytest.mark.parametrize("fmt,H,B", [(0, 16, 80), (1, 32, 80), (0, 64, 80), (1, 64, 80), (0, 128, 45), (1, 128, 45)])
@pytest.mark.parametrize("window", [400, 2400])
def test_long_windows_of_sequences_of_many_lengths(fmt, H, B, window):
    # (2400: longer than any equal part; 128 heads, bf16: as twice the tokens of 64)
    rng = np.random.default_rng(H)
    ends = rng.integers(0, 150, B)
    ends[:4], ends[-1] = [2600, 0, 1, 2499], 2433
    pool = Pool(fmt, ends, 64, seed=H + 4)
    rows = [pool.rows(b).astype(np.int64) for b in range(B)]
    hide(pool, 1, window, 20)
    run(pool, 1, H, window, 20, seed=H + 6, rows=rows)


@pytest.mark.parametrize("window", range(1, 34))
@pytest.mark.parametrize("fmt,H", [(0, 16), (1, 128)])
def test_every_alignment_of_the_window(fmt, H, window):
    ends = list(range(60, 78))
    pool = Pool(fmt, ends, 16, seed=31)
    rows = [pool.rows(b).astype(np.int64) for b in range(len(ends))]
    hide(pool, 1, window, window % 7)
    run(pool, 1, H, window, window % 7, seed=window, rows=rows)


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("H", [16, 32, 64, 128])
def test_a_window_of_everything_is_the_decode(fmt, H):
    pool = Pool(fmt, [300, 1, 77, 0, 1000], 64, seed=32)
    B = len(pool.ends)
    ql, qp = randn_bf16((B, 1, H, 512), 1), randn_bf16((B, 1, H, 64), 2)
    cache, T = pool.device(), pool.max_pages * 64
    a = mla.paged_decode_window(cache, pool.dev_table(), ql.cuda(), qp.cuda(), pool.dev_ends(), T, SM, T)
    b = mla.paged_decode(cache, pool.dev_table(), ql[:, 0].contiguous().cuda(), qp[:, 0].contiguous().cuda(), pool.dev_ends(), T, SM)
    # (their references may differ, so the last bits may: each is within its bounds)
    _, _, bo, bl = expected(pool, ql, qp, T, 0)
    within(f64(a[0]), f64(b[0])[:, None], 2 * bo, "out")
    within(f64(a[1]), f64(b[1])[:, None], 2 * bl, "lse")


@pytest.mark.parametrize("fmt,H,s", [(0, 16, 7), (1, 32, 7), (0, 128, 7), (1, 128, 7), (1, 16, 161), (0, 16, 163), (0, 32, 101),
                                     (1, 32, 102), (1, 64, 120), (0, 128, 140)])
def test_later_tokens_rows_do_not_reach_earlier_tokens(fmt, H, s):
    # the last token's own row is NaN: its output is, and no other's
    pool = Pool(fmt, [s + 20, s], 16, seed=33)
    B = 2
    ql, qp = randn_bf16((B, s, H, 512), 3), randn_bf16((B, s, H, 64), 4)
    args = (pool.dev_table(), ql.cuda(), qp.cuda(), pool.dev_ends(), pool.max_pages * 16, SM, 12)
    good = mla.paged_decode_window(pool.device(), *args, sinks=2)
    for b in range(B):
        r = pool.rows(b)[-1]
        pool.kv[r] = 0x7FC0 if fmt == 0 else 0x7F
        pool.pe[r] = 0x7F80
    bad = mla.paged_decode_window(pool.device(), *args, sinks=2)
    assert torch.equal(good[0][:, :-1], bad[0][:, :-1]) and torch.equal(good[1][:, :-1], bad[1][:, :-1])
    assert bool(bad[0][:, -1].isnan().all())


@pytest.mark.parametrize("fmt,H", [(0, 16), (1, 32), (0, 64), (0, 128), (1, 128)])
@pytest.mark.parametrize("s", [1, 60])
def test_positions_on_bad_pages_are_left_out(fmt, H, s):
    pool = Pool(fmt, [700, 64, 200], 64, seed=34)
    rows = [pool.rows(b).astype(np.int64) for b in range(3)]
    pool.table[0, 9] = -1                       # positions 576 .. 639
    ql, qp = randn_bf16((3, s, H, 512), 5), randn_bf16((3, s, H, 64), 6)
    ws = mla.alloc_paged_window_workspace(3, s, H)
    out, lse = mla.paged_decode_window(pool.device(), pool.dev_table(), ql.cuda(), qp.cuda(), pool.dev_ends(), 700, SM, 200, sinks=4,
                                       workspace=ws)
    ref, rl, bo, bl = expected(pool, ql, qp, 200, 4, rows=rows, bad=[np.arange(576, 640), [], []])
    within(f64(out), ref, bo, "out")
    within(f64(lse), rl, bl, "lse")
    assert mla.workspace_status(ws) == mla.DEV_BAD_PAGE


@pytest.mark.parametrize("H", [16, 128])
@pytest.mark.parametrize("s", [1, 3, 70])
def test_lengths_are_clamped_and_flagged(H, s):
    pool = Pool(0, [100, 200, 50], 16, seed=35)
    ql, qp = randn_bf16((3, s, H, 512), 7), randn_bf16((3, s, H, 64), 8)
    ws = mla.alloc_paged_window_workspace(3, s, H)
    e = torch.tensor([100, 500, -3], dtype=torch.int32)
    out, lse = mla.paged_decode_window(pool.device(), pool.dev_table(), ql.cuda(), qp.cuda(), e.cuda(), 200, SM, 60, sinks=1, workspace=ws)
    rows = [pool.rows(b).astype(np.int64) for b in range(3)]
    pool.ends = np.array([100, 200, 0], np.int32)
    ref, rl, bo, bl = expected(pool, ql, qp, 60, 1, rows=rows)
    within(f64(out), ref, bo, "out")
    within(f64(lse), rl, bl, "lse")
    assert mla.workspace_status(ws) == mla.DEV_END_POS_CLAMPED


@pytest.mark.parametrize("fmt,H", [(0, 16), (1, 16), (0, 32), (1, 64), (0, 128)])
@pytest.mark.parametrize("kind", ["nan", "inf", "query"])
def test_what_is_not_finite_stays_with_the_tokens_that_see_it(fmt, H, kind):
    # tokens share tiles: row 50's values, or one token's query, are not finite
    s, w, e = 170, 9, 180
    pool = Pool(fmt, [e], 16, seed=40)
    ql, qp = randn_bf16((1, s, H, 512), 17), randn_bf16((1, s, H, 64), 18)
    args = lambda: (pool.dev_table(), ql.cuda(), qp.cuda(), pool.dev_ends(), e, SM, w)
    good = mla.paged_decode_window(pool.device(), *args(), sinks=3)
    r = pool.rows(0)[50]
    t = np.arange(e - s, e)
    hit = (t >= 50) & (t < 50 + w)
    if kind == "query":
        hit = t == 50
        ql[0, 50 - (e - s), :, 7] = float("nan")
    elif fmt == 0:
        pool.kv[r, 100:300:40] = 0x7FC0 if kind == "nan" else 0x7F80
    elif kind == "nan":
        pool.kv[r, 100:300:40] = 0x7F
    else:
        pool.scale[r, 1] = np.inf
    bad = mla.paged_decode_window(pool.device(), *args(), sinks=3)
    keep = torch.from_numpy(~hit).cuda()
    assert torch.equal(good[0][0, keep], bad[0][0, keep]) and torch.equal(good[1][0, keep], bad[1][0, keep])
    assert not bool(bad[0][0, ~keep].isfinite().all(-1).any()) or kind == "inf"
    assert bool(bad[0][0, ~keep].isnan().any())


@pytest.mark.parametrize("fmt,H,s", [(0, 16, 3), (1, 64, 2), (0, 128, 2), (1, 128, 1), (0, 16, 200), (1, 32, 180), (0, 64, 160), (0, 128, 90)])
@pytest.mark.parametrize("slope", [0.35, -0.35])
def test_drifting_scores_move_the_references(fmt, H, s, slope):
    # the rows drift along a direction, so scores climb (or fall) by far more than any
    # threshold within a window, by other amounts per head
    T, scale = 900, 0.5
    g = np.random.default_rng(5)
    u = g.standard_normal(512)
    u /= np.linalg.norm(u)
    p0 = Pool(fmt, [T], 64, seed=3)
    x = g.standard_normal((p0.num_pages * 64, 512)) * 0.2
    x[p0.rows(0)] += np.outer((np.arange(T) - (0 if slope > 0 else T)) * slope, u)
    pool = Pool(fmt, [T], 64, seed=3, kv=bits(torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16)))
    ql, qp = randn_bf16((1, s, H, 512), 19), randn_bf16((1, s, H, 64), 20)
    ql = (ql.float() + torch.from_numpy(np.outer(np.linspace(-1, 4, H), u)).float()[None, None]).to(torch.bfloat16)
    out, lse = mla.paged_decode_window(pool.device(), pool.dev_table(), ql.cuda(), qp.cuda(), pool.dev_ends(), T, scale, 500, sinks=4)
    ref, rl, bo, bl = expected(pool, ql, qp, 500, 4, scale)
    # scores reach 10^3: their reference value is off by u(fp32) of that, 2^-13
    smax = float(np.abs(rl).max())
    within(f64(out), ref, bo * (1 + 64 * smax * 2.0 ** -24) + 8 * smax * 2.0 ** -24, "out")
    within(f64(lse), rl, bl + 8 * smax * 2.0 ** -24, "lse")


@pytest.mark.parametrize("fmt,H,s", [(0, 16, 1000), (1, 64, 800), (0, 64, 800), (0, 128, 400), (1, 32, 900), (0, 64, 20), (1, 128, 3)])
def test_references_that_rise_in_every_tile_give_the_same_each_time(fmt, H, s):
    # (a unit's last tile among them: what the warps share for it must hold until
    # the last of them has used it)
    T, scale = 1000, 0.5
    u = np.zeros(512)
    u[::2] = 1 / 16
    p0 = Pool(fmt, [T], 64, seed=3)
    x = np.random.default_rng(6).standard_normal((p0.num_pages * 64, 512)) * 0.2
    x[p0.rows(0)] += np.outer(np.arange(T) * 0.5, u)
    pool = Pool(fmt, [T], 64, seed=3, kv=bits(torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16)))
    ql, qp = (randn_bf16((1, s, H, 512), 28) * 0.1), randn_bf16((1, s, H, 64), 29)
    ql = (ql.float() + torch.from_numpy(np.outer(np.linspace(1, 4, H), u)).float()[None, None]).to(torch.bfloat16)
    cache, table, end = pool.device(), pool.dev_table(), pool.dev_ends()
    ql, qp = ql.cuda(), qp.cuda()
    ws = mla.alloc_paged_window_workspace(1, s, H)
    first = mla.paged_decode_window(cache, table, ql, qp, end, T, scale, 200, sinks=4, workspace=ws)
    # one row in the first direction: the weights are those of a few last positions
    rows = torch.from_numpy(orc.bf16_bits_to_f64(pool.kv[pool.rows(0)] if fmt == 0 else orc.dequant_rows(pool.kv[pool.rows(0)], pool.scale[pool.rows(0)]))).cuda()
    keys = torch.from_numpy(orc.bf16_bits_to_f64(pool.pe[pool.rows(0)])).cuda()
    t = torch.arange(T - s, T, device="cuda")
    p = torch.arange(T, device="cuda")
    seen = (p <= t[:, None]) & ((p < 4) | (p > t[:, None] - 200))
    sc = (ql[0].double() @ rows.T + qp[0].double() @ keys.T) * scale
    w = torch.softmax(sc.masked_fill(~seen[:, None], -np.inf), -1)
    ref, mag = w @ rows, w @ rows.abs()
    smax = float(sc.abs().max())
    # (bounds of paged_cases.py; a score's reference value is off by u(fp32) of it, its sum by 64 places of the products')
    ds = 64 * 2.0 ** -23 * scale * float((ql[0].double().abs() @ rows.abs().T).max()) + 8 * smax * 2.0 ** -24 + 2.0 ** -16
    worst = float(((first[0][0].double() - ref).abs() / (2.0 ** -8 * (ref.abs() + mag) + 3 * ds * mag)).max())
    assert worst <= 1, f"{worst:.3g} of its bound"
    for _ in range(40):
        again = mla.paged_decode_window(cache, table, ql, qp, end, T, scale, 200, sinks=4, workspace=ws)
        off = int((first[0] != again[0]).sum()) + int((first[1] != again[1]).sum())
        assert off == 0, f"{off} values differ from one call to the next"


@pytest.mark.parametrize("fmt,H,s", [(0, 16, 200), (1, 16, 160), (0, 128, 70)])
def test_scores_far_from_zero(fmt, H, s):
    # every score of a head is some hundred below (or above) 0: the references go there
    e = 230
    pool = Pool(fmt, [e], 16, seed=41)
    pool.pe[pool.rows(0)] = bits(torch.ones(e, 64, dtype=torch.bfloat16))
    ql, qp = randn_bf16((1, s, H, 512), 21), torch.full((1, s, H, 64), -30.0, dtype=torch.bfloat16)
    qp[:, :, ::2] = 30.0
    out, lse = mla.paged_decode_window(pool.device(), pool.dev_table(), ql.cuda(), qp.cuda(), pool.dev_ends(), e, SM, 33, sinks=2)
    ref, rl, bo, bl = expected(pool, ql, qp, 33, 2)
    smax = float(np.abs(rl).max())
    assert smax > 200
    within(f64(out), ref, bo + 8 * smax * 2.0 ** -24, "out")
    within(f64(lse), rl, bl + 8 * smax * 2.0 ** -24, "lse")


@pytest.mark.parametrize("scale", [0.0, -0.11])
@pytest.mark.parametrize("fmt,H", [(0, 64), (1, 128), (0, 16)])
def test_other_softmax_scales(fmt, H, scale):
    run(Pool(fmt, [200, 333], 64, seed=36), 2, H, 90, 5, seed=9, scale=scale)
    run(Pool(fmt, [200], 64, seed=36), 160, H, 40, 5, seed=9, scale=scale)


@pytest.mark.parametrize("fmt,H", [(0, 16), (1, 64), (0, 128), (1, 128)])
def test_an_infinite_score_of_a_hidden_row_changes_nothing(fmt, H):
    # rows beside the seen ones in the same boxes of 16, with values that give infinite scores and products
    pool = Pool(fmt, [90, 61], 16, seed=37)
    B = 2
    ql, qp = randn_bf16((B, 1, H, 512), 11), randn_bf16((B, 1, H, 64), 12)
    args = (pool.dev_table(), ql.cuda(), qp.cuda(), pool.dev_ends(), 90, SM, 21)
    good = mla.paged_decode_window(pool.device(), *args, sinks=3)
    for b, e in enumerate(pool.ends):
        for p in (3, 15, int(e) - 22, (int(e) - 21) & ~15):
            if not (p < 3 or p > e - 1 - 21):
                r = pool.rows(b)[p]
                if fmt == 0:
                    pool.kv[r] = 0x7F80
                else:
                    pool.scale[r] = np.inf
                pool.pe[r] = 0xFF80
    bad = mla.paged_decode_window(pool.device(), *args, sinks=3)
    assert torch.equal(good[0], bad[0]) and torch.equal(good[1], bad[1])


@pytest.mark.parametrize("fmt,H,s", [(0, 16, 1), (1, 64, 3), (0, 128, 1), (1, 128, 2), (0, 32, 150), (1, 128, 150), (0, 16, 170)])
def test_captured_and_replayed(fmt, H, s):
    pool = Pool(fmt, [300, 200], 64, seed=38)
    B = 2
    ql, qp = randn_bf16((B, s, H, 512), 13).cuda(), randn_bf16((B, s, H, 64), 14).cuda()
    cache, table, end = pool.device(), pool.dev_table(), pool.dev_ends()
    ws = mla.alloc_paged_window_workspace(B, s, H)
    out, lse = torch.empty(B, s, H, 512, dtype=torch.bfloat16, device="cuda"), torch.empty(B, s, H, device="cuda")
    call = lambda: mla.paged_decode_window(cache, table, ql, qp, end, 300, SM, 100, sinks=4, out=out, lse=lse, workspace=ws)
    call()
    want = []
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for d in (0, 1, 57):
        end.copy_(pool.dev_ends() - d)
        out.fill_(7.0)
        g.replay()
        got = out.clone(), lse.clone()
        fresh = mla.paged_decode_window(cache, table, ql, qp, end, 300, SM, 100, sinks=4)
        want.append(torch.equal(got[0], fresh[0]) and torch.equal(got[1], fresh[1]))
    assert all(want)


@pytest.mark.parametrize("fmt,H,s", [(0, 16, 1), (1, 64, 2), (0, 128, 1), (1, 128, 1), (0, 16, 170), (1, 32, 100), (1, 64, 130), (0, 128, 70)])
def test_waits_that_run_out_are_reported_and_leave_the_device_usable(fmt, H, s):
    pool = Pool(fmt, [300, 280], 64, seed=42)
    ql, qp = randn_bf16((2, s, H, 512), 23).cuda(), randn_bf16((2, s, H, 64), 24).cuda()
    cache, ws = pool.device(), mla.alloc_paged_window_workspace(2, s, H)
    args = (cache, pool.dev_table(), ql, qp, pool.dev_ends(), 300, SM, 250)
    good = mla.paged_decode_window(*args, sinks=4)
    for _ in range(2):
        assert mla.selftest_paged_window_timeout(*args, 4, ws) & mla.DEV_PIPELINE_TIMEOUT
    again = mla.paged_decode_window(*args, sinks=4, workspace=ws)
    assert torch.equal(good[0], again[0]) and torch.equal(good[1], again[1]) and mla.workspace_status(ws) == 0


def test_rows_past_32_bit_byte_offsets():
    # the sequences' pages are the last of a pool of 4.6 GB of latents
    pages, page, n = 70000, 64, 200
    kv = torch.zeros(pages, page, 512, dtype=torch.bfloat16, device="cuda")
    pe = torch.zeros(pages, page, 64, dtype=torch.bfloat16, device="cuda")
    cache = mla.PagedCache(pages, page, kv=kv, pe=pe, weight=False)
    table = torch.arange(pages - 8, pages, dtype=torch.int32, device="cuda").flip(0).view(2, 4).contiguous()
    small = mla.PagedCache(8, page)
    near = torch.arange(8, dtype=torch.int32, device="cuda").flip(0).view(2, 4).contiguous()
    end = torch.tensor([n, n], dtype=torch.int32, device="cuda")
    kva, pos = randn_bf16((2, n, 576), 25).cuda(), torch.arange(n, dtype=torch.int32).repeat(2, 1).cuda()
    rot, w = mla.Rotary(mla.rotary_frequencies()), torch.ones(512, device="cuda")
    off = torch.tensor([0, n, 2 * n], dtype=torch.int32, device="cuda")
    got = []
    for c, t in ((cache, table), (small, near)):
        mla.paged_append_rotary(c, t, kva, w, 1e-6, rot, pos, end)
        r = list(mla.paged_read(c, t, off, 2 * n))
        for H, s in ((16, 1), (128, 1), (16, 170), (128, 70)):
            ql, qp = randn_bf16((2, s, H, 512), 26).cuda(), randn_bf16((2, s, H, 64), 27).cuda()
            r += mla.paged_decode_window(c, t, ql, qp, end, 256, SM, 90, sinks=4)
        got.append(r)
    assert all(torch.equal(x, y) for x, y in zip(*got))
    assert bool((kv[:pages - 8] == 0).all())


def test_on_another_stream_without_outputs_or_sums():
    pool = Pool(1, [300, 200], 64, seed=39)
    ql, qp = randn_bf16((2, 2, 128, 512), 15).cuda(), randn_bf16((2, 2, 128, 64), 16).cuda()
    cache, table, end = pool.device(), pool.dev_table(), pool.dev_ends()
    a = mla.paged_decode_window(cache, table, ql, qp, end, 300, SM, 100)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    b = mla.paged_decode_window(cache, table, ql, qp, end, 300, SM, 100, stream=st, want_lse=False)
    st.synchronize()
    assert b[1] is None and torch.equal(a[0], b[0])


@pytest.mark.parametrize("fmt", [0, 1])
def test_a_serving_step_of_all_of_them(fmt):
    # a prompt written from the projections' outputs, a windowed step of three tokens over
    # it, and the prompt read back; each piece against the calls it stands beside
    B, H, n, s, page = 2, 16, 45, 3, 16
    cache = mla.PagedCache(20, page, fmt)
    other = mla.PagedCache(20, page, fmt)
    table = torch.randperm(20, generator=torch.Generator().manual_seed(1)).to(torch.int32).view(2, 10).cuda()
    rot = mla.Rotary(mla.rotary_frequencies(factor=40.0))
    w = (1 + 0.1 * torch.randn(512, generator=torch.Generator().manual_seed(2))).cuda()
    kv, q = randn_bf16((B, n, 576), 21).cuda(), randn_bf16((B, n, H, 192), 22).cuda()
    wkv = (randn_bf16((H, 256, 512), 23).float() * 0.05).to(torch.bfloat16).cuda()
    end = torch.tensor([n, n], dtype=torch.int32).cuda()
    pos = torch.arange(n, dtype=torch.int32).repeat(B, 1).cuda()
    qn, qp = mla.paged_append_rotary(cache, table, kv, w, 1e-6, rot, pos, end, q=q)
    ql = mla.absorb_q(qn.view(B * n, H, 128), wkv).view(B, n, H, 512)
    out, lse = mla.paged_decode_window(cache, table, ql[:, -s:].contiguous(), qp[:, -s:].contiguous(), end, 160, SM, 20, sinks=4)
    # the rows read back are what a second pool gets as plain new rows (bf16: the same bits)
    off = torch.tensor([0, n, 2 * n], dtype=torch.int32).cuda()
    c, k = mla.paged_read(cache, table, off, 2 * n)
    for j in range(s):
        t = n - s + j
        low = max(0, t - 19)
        for b in range(B):
            rows = torch.cat([torch.arange(0, min(4, low)), torch.arange(low, t + 1)]).cuda() + b * n
            x, y = c[rows].double(), k[rows].double()
            sc = (ql[b, t].double() @ x.T + qp[b, t].double() @ y.T) * SM
            p = torch.softmax(sc, -1)
            ref = (p @ x).cpu().numpy()
            # (bounds of paged_cases.py: p and out rounded to bf16 once)
            wc = (p @ x.abs()).cpu().numpy()
            mag = (ql[b, t].double().abs() @ x.abs().T + qp[b, t].double().abs() @ y.abs().T).amax(-1, keepdim=True).cpu().numpy()
            ds = 64 * 2.0 ** -23 * SM * mag + 2.0 ** -16
            within(f64(out[b, j]), ref, 2.0 ** -8 * (np.abs(ref) + wc) + (2 * ds + 2.0 ** -16) * wc, "out")
            within(f64(lse[b, j]), torch.logsumexp(sc, -1).cpu().numpy(), ds[:, 0] + 2.0 ** -16, "lse")
    if fmt == 0:
        mla.paged_append(other, table, c.view(B, n, 512), k.view(B, n, 64), end)
        assert torch.equal(cache.kv.view(torch.int16), other.kv.view(torch.int16)) and torch.equal(cache.pe.view(torch.int16), other.pe.view(torch.int16))
