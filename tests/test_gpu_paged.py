"""GPU parity of the paged-cache operators against fp64 references (the oracle
on each sequence's rows), with bounds derived in paged_cases.py.  Every pool
holds NaN in the rows no sequence uses and out-of-range entries past the used
part of the tables."""
import numpy as np
import pytest
import torch

import mla_latent_kv_07_gb300 as mla

from mla_cases import bits, f64
from paged_cases import Pool, U_F32, evict_reference, randn_bf16, reference, within

pytestmark = pytest.mark.gpu
SM = 0.1352


@pytest.fixture(scope="module", autouse=True)
def _built():
    from mla_latent_kv_07_gb300 import build
    build.build()
    mla.lib()


def queries(B, H, seed):
    return randn_bf16((B, H, 512), seed), randn_bf16((B, H, 64), seed + 1)


def check_decode(pool, H, seed, scale=SM, cache=None, **kw):
    ql, qp = queries(len(pool.ends), H, seed)
    cache = pool.device() if cache is None else cache
    ws = mla.alloc_paged_workspace(len(pool.ends), H)
    out, lse = mla.paged_decode(cache, pool.dev_table(), ql.cuda(), qp.cuda(), pool.dev_ends(),
                                pool.max_pages * pool.page, scale, workspace=ws)
    ref, rl, _, bo, bl, _ = reference(pool, ql, qp, scale, **kw)
    within(f64(out), ref, bo, "out")
    within(f64(lse), rl, bl, "lse")
    assert mla.workspace_status(ws) & mla.DEV_PIPELINE_TIMEOUT == 0
    return out, lse, ws


# ------------------------------------------------------------------ decode

DECODE = [  # (fmt, H, page, ends)
    (0, 16, 16, [1]), (0, 16, 16, [15, 16, 17, 0]), (1, 16, 16, [100, 257, 5]), (2, 16, 48, [129, 48]),
    (0, 32, 32, [64, 1, 200]), (1, 32, 128, [127, 128, 129]), (0, 64, 64, [129, 77, 0, 513]),
    (1, 64, 80, [81, 400]), (2, 64, 16, [640, 31]), (0, 128, 64, [300, 33, 1]), (0, 128, 16, [255, 256, 257]),
    (1, 128, 64, [1000, 513, 2, 64]), (2, 128, 256, [511, 0, 513]), (0, 128, 1024, [2000, 5]),
    (1, 128, 48, [47, 48, 49, 97, 640]), (0, 16, 64, [3000]), (1, 16, 64, [2999]), (0, 64, 112, [1501, 800]),
]


@pytest.mark.parametrize("fmt,H,page,ends", DECODE)
def test_decode_all_outputs(fmt, H, page, ends):
    check_decode(Pool(fmt, ends, page, seed=7 * H + page), H, seed=H + page)


@pytest.mark.parametrize("fmt,H", [(0, 16), (1, 32), (0, 64), (1, 64), (0, 128), (1, 128)])
def test_decode_long_sequences_split_over_the_gpu(fmt, H):
    check_decode(Pool(fmt, [9001, 20, 4097], 64, seed=H), H, seed=H + 5)


@pytest.mark.parametrize("fmt,H", [(0, 16), (1, 64), (0, 128), (1, 128)])
def test_decode_more_sequences_than_units(fmt, H):
    rng = np.random.default_rng(H)
    check_decode(Pool(fmt, rng.integers(0, 200, 333), 16, seed=H + 1), H, seed=H + 2)


@pytest.mark.parametrize("fmt,H", [(0, 16), (1, 32), (0, 64), (1, 128), (0, 128)])
def test_rising_scores_rescale_in_a_unit(fmt, H):
    # the rows drift along a fixed direction, so the running maximum climbs by
    # far more than any threshold within every unit, and by other amounts per head
    T = 1500
    g = np.random.default_rng(5)
    u = g.standard_normal(512)
    u /= np.linalg.norm(u)
    p0 = Pool(fmt, [T], 64, seed=3)
    x = g.standard_normal((p0.num_pages * 64, 512)) * 0.2
    x[p0.rows(0)] += np.outer(np.arange(T) * 0.35, u)
    kv = bits(torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16))
    pool = Pool(fmt, [T], 64, seed=3, kv=kv)
    ql, qp = queries(1, H, 9)
    ql = (ql.float() + torch.from_numpy(np.outer(np.linspace(-1, 4, H), u)).float()[None]).to(torch.bfloat16)
    out, lse = mla.paged_decode(pool.device(), pool.dev_table(), ql.cuda(), qp.cuda(), pool.dev_ends(), T, 0.5)
    ref, rl, _, bo, bl, _ = reference(pool, ql, qp, 0.5)
    # scores reach 10^3: their reference value is off by u(fp32) of that, 2^-13
    smax = float(np.abs(rl).max())
    within(f64(out), ref, bo * (1 + 64 * smax * U_F32) + 8 * smax * U_F32, "out")
    within(f64(lse), rl, bl + 8 * smax * U_F32, "lse")


@pytest.mark.parametrize("scale", [0.0, -0.11, 1e-3])
@pytest.mark.parametrize("fmt,H", [(0, 64), (1, 128), (0, 16)])
def test_other_softmax_scales(fmt, H, scale):
    check_decode(Pool(fmt, [200, 333], 64, seed=8), H, seed=2, scale=scale)


@pytest.mark.parametrize("fmt,H", [(0, 16), (1, 64), (0, 128), (1, 128)])
def test_shared_pages_are_read_by_all(fmt, H):
    check_decode(Pool(fmt, [300, 500, 65], 64, seed=11, shared=3), H, seed=4)


@pytest.mark.parametrize("fmt,H", [(0, 16), (1, 32), (0, 64), (0, 128), (1, 128)])
def test_positions_on_bad_pages_are_left_out(fmt, H):
    pool = Pool(fmt, [700, 64, 200, 130], 64, seed=12)
    pool.table[0, 3], pool.table[0, 10], pool.table[1, 0], pool.table[3, 2] = -1, pool.num_pages, -7, 2 ** 31 - 1
    skip = [np.r_[192:256, 640:700], np.arange(64), [], np.arange(128, 130)]
    rows0 = pool.rows
    pool.rows = lambda b, n=None: np.where(np.isin(np.arange(rows0(b, n).size), skip[b]), 0, rows0(b, n))
    out, lse, ws = check_decode(pool, H, seed=6, leave_out=skip)
    assert mla.workspace_status(ws) == mla.DEV_BAD_PAGE
    assert (out[1] == 0).all() and torch.isneginf(lse[1]).all()


def test_lengths_are_clamped_and_flagged():
    pool = Pool(0, [100, 200, 50], 16, seed=13)
    ql, qp = queries(3, 128, 1)
    ws = mla.alloc_paged_workspace(3, 128)
    e = torch.tensor([100, 500, -3], dtype=torch.int32)
    out, lse = mla.paged_decode(pool.device(), pool.dev_table(), ql.cuda(), qp.cuda(), e.cuda(), 200, SM, workspace=ws)
    ref, rl, _, bo, bl, _ = reference(pool, ql, qp, SM, ends=[100, 200, 0])
    within(f64(out), ref, bo, "out")
    within(f64(lse), rl, bl, "lse")
    assert mla.workspace_status(ws) == mla.DEV_END_POS_CLAMPED


@pytest.mark.parametrize("fmt,H", [(0, 16), (1, 16), (2, 64), (0, 128), (1, 128), (2, 128)])
def test_decode_writes_the_new_rows_first(fmt, H):
    ends = [1, 64, 65, 300, 0, 129]
    pool = Pool(fmt, ends, 64, seed=14)
    cache = pool.device()
    B = len(ends)
    kvn, pen = randn_bf16((B, 512), 30), randn_bf16((B, 64), 31)
    ql, qp = queries(B, H, 3)
    ws = mla.alloc_paged_workspace(B, H)
    out, lse = mla.paged_decode(cache, pool.dev_table(), ql.cuda(), qp.cuda(), pool.dev_ends(), 300, SM,
                                kv_new=kvn.cuda(), pe_new=pen.cuda(), workspace=ws)
    pool.append(kvn, pen, 1)
    pool.same_as(cache)
    ref, rl, _, bo, bl, _ = reference(pool, ql, qp, SM)
    within(f64(out), ref, bo, "out")
    within(f64(lse), rl, bl, "lse")
    assert mla.workspace_status(ws) == mla.DEV_APPEND_SKIPPED      # the empty sequence
    again, _ = mla.paged_decode(cache, pool.dev_table(), ql.cuda(), qp.cuda(), pool.dev_ends(), 300, SM)
    assert torch.equal(again, out)


@pytest.mark.parametrize("H", [16, 128])
def test_results_repeat_bit_for_bit(H):
    pool = Pool(1, [5000, 100, 777], 64, seed=15)
    cache, tb, e = pool.device(), pool.dev_table(), pool.dev_ends()
    ql, qp = [x.cuda() for x in queries(3, H, 3)]
    first = mla.paged_decode(cache, tb, ql, qp, e, 5000, SM)
    for _ in range(5):
        again = mla.paged_decode(cache, tb, ql, qp, e, 5000, SM)
        assert torch.equal(again[0], first[0]) and torch.equal(again[1], first[1])


@pytest.mark.parametrize("fmt", [0, 1])
def test_a_pool_past_32_bit_offsets(fmt):
    # rows near the end of a pool whose latents pass 2^32 bytes (bf16) / 2^32 codes
    page = 64
    pages = (2 ** 32 // (1024 if fmt == 0 else 512)) // page + 40
    pool = Pool(fmt, [333, 64], page, seed=16)
    far = np.arange(pages - pool.num_pages, pages)
    kv = torch.empty((pages, page, 512), dtype=torch.bfloat16 if fmt == 0 else torch.uint8, device="cuda")
    sc = torch.empty((pages, page, 4), device="cuda") if fmt else None
    pe = torch.empty((pages, page, 64), dtype=torch.bfloat16, device="cuda")
    w = torch.empty((pages, page), device="cuda")
    small = pool.device()
    kv[far[0]:], pe[far[0]:], w[far[0]:] = small.kv, small.pe, small.weight
    if fmt:
        sc[far[0]:] = small.kv_scale
    cache = mla.PagedCache(pages, page, fmt, kv=kv, kv_scale=sc, pe=pe, weight=w)
    used = (pool.table >= 0) & (pool.table < pool.num_pages)
    tb = torch.from_numpy(np.where(used, pool.table + far[0], -1).astype(np.int32)).cuda()
    for H in (16, 128):
        ql, qp = queries(2, H, 3)
        out, lse = mla.paged_decode(cache, tb, ql.cuda(), qp.cuda(), pool.dev_ends(), 333, SM)
        ref, rl, wr, bo, bl, bw = reference(pool, ql, qp, SM)
        within(f64(out), ref, bo, "out")
        w[far[0]:] = 0.0
        mla.paged_weights(cache, tb, ql.cuda(), qp.cuda(), lse, pool.dev_ends(), 333, SM)
        got = w[far[0]:].cpu().numpy().reshape(-1)
        for b in range(2):
            within(got[pool.rows(b)], wr[b], bw[b] + 2 ** -20 * wr[b], "weights")


# ------------------------------------------------------------------ append

@pytest.mark.parametrize("fmt", [0, 1, 2])
@pytest.mark.parametrize("page,s", [(16, 1), (48, 7), (64, 130), (128, 300)])
def test_append_bit_exact(fmt, page, s):
    ends = [s, s + 17, 4 * page, s + 200, 1]        # some shorter than their new rows
    pool = Pool(fmt, ends, page, seed=17 + s)
    cache = pool.device()
    g = torch.Generator().manual_seed(3)
    kvn = (torch.randn(len(ends), s, 512, generator=g) * torch.exp(torch.randn(len(ends), s, 1, generator=g) * 4)).to(torch.bfloat16)
    kvn[0, 0, :128] = 0.0
    kvn[1, 0, 128:256] = 448.0
    pen = randn_bf16((len(ends), s, 64), 32)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    mla.paged_append(cache, pool.dev_table(), kvn.cuda(), pen.cuda(), pool.dev_ends(), status=status)
    pool.append(kvn, pen, s)
    pool.same_as(cache)
    short = any(e < s for e in ends)
    assert int(status) == (mla.DEV_APPEND_SKIPPED if short else 0)


def test_append_leaves_out_what_the_table_does_not_name():
    pool = Pool(0, [100, 40], 16, seed=18)
    cache = pool.device()
    pool.ends = np.array([pool.max_pages * 16 + 5, 40], np.int32)       # past the table
    pool.table[0, -1] = 0 if 0 not in pool.table[:, :7] else pool.free[0]
    pool.table[1, 2] = -1                                               # a bad page
    s = 12
    kvn, pen = randn_bf16((2, s, 512), 1), randn_bf16((2, s, 64), 2)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    mla.paged_append(cache, pool.dev_table(), kvn.cuda(), pen.cuda(), pool.dev_ends(), status=status)
    pool.append(kvn, pen, s)
    pool.same_as(cache)
    assert int(status) == mla.DEV_APPEND_SKIPPED | mla.DEV_BAD_PAGE


# ----------------------------------------------------------------- weights

def weights_once(pool, cache, H, seed, ends=None):
    ql, qp = queries(len(pool.ends), H, seed)
    out, rl, wr, _, _, bw = reference(pool, ql, qp, SM, ends=ends)
    lse = torch.from_numpy(rl.astype(np.float32)).cuda()
    mla.paged_weights(cache, pool.dev_table(), ql.cuda(), qp.cuda(), lse, pool.dev_ends(), pool.max_pages * pool.page, SM)
    return wr, bw


@pytest.mark.parametrize("fmt,H,page,ends", DECODE)
def test_weights_all_rows(fmt, H, page, ends):
    pool = Pool(fmt, ends, page, seed=7 * H + page)
    cache = pool.device()
    wr, bw = weights_once(pool, cache, H, seed=H)
    got = cache.weight.cpu().numpy().reshape(-1)
    for b in range(len(ends)):
        r = pool.rows(b)
        # the lse went in rounded to fp32 (2^-24 of it, below 2^-19 for |lse| < 32)
        # and the sum over heads and the total are rounded H + 1 times
        ref = pool.weight[r] + wr[b]
        within(got[r], ref, bw[b] + 2 ** -18 * wr[b] + (H + 1) * U_F32 * wr[b] + 2 * U_F32 * np.abs(ref), f"weights of {b}")
    assert np.array_equal(got[~pool.live].view(np.uint32), pool.weight[~pool.live].view(np.uint32))


@pytest.mark.parametrize("fmt,H", [(0, 16), (1, 64), (0, 128), (1, 128)])
def test_weights_of_shared_rows_add_up(fmt, H):
    pool = Pool(fmt, [300, 500, 65, 9001], 64, seed=19, shared=3)
    cache = pool.device()
    total = pool.weight.astype(np.float64)
    bound = np.zeros_like(total)
    for k in range(2):
        wr, bw = weights_once(pool, cache, H, seed=H + k)
        for b in range(4):
            np.add.at(total, pool.rows(b), wr[b])
            np.add.at(bound, pool.rows(b), bw[b] + (2 ** -18 + (H + 1) * U_F32) * wr[b])
    got = cache.weight.cpu().numpy().reshape(-1)
    live = np.unique(np.concatenate([pool.rows(b) for b in range(4)]))
    within(got[live], total[live], bound[live] + 10 * U_F32 * total[live], "weights")


def test_weights_skip_heads_without_a_sum_and_bad_pages():
    for fmt in (0, 1):
        pool = Pool(fmt, [300, 130], 64, seed=20)
        pool.table[0, 1] = -1
        rows0 = pool.rows
        bad = np.arange(64, 128)
        pool.rows = lambda b, n=None: np.where((b == 0) & np.isin(np.arange(rows0(b, n).size), bad), 0, rows0(b, n))
        cache = pool.device()
        ql, qp = queries(2, 32, 3)
        _, rl, wr, _, _, bw = reference(pool, ql[:, :31], qp[:, :31], SM, leave_out=[bad, []])
        rl = np.concatenate([rl, np.full((2, 1), -np.inf)], 1)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        before = cache.weight.clone()
        mla.paged_weights(cache, pool.dev_table(), ql.cuda(), qp.cuda(), torch.from_numpy(rl.astype(np.float32)).cuda(),
                          pool.dev_ends(), 300, SM, status=status)
        assert int(status) == mla.DEV_BAD_PAGE
        got = cache.weight.cpu().numpy().reshape(-1)
        touched = np.zeros(got.size, bool)
        for b in range(2):
            r = pool.rows(b)
            r = r if b else r[~np.isin(np.arange(r.size), bad)]
            touched[r] = True
            ref = pool.weight[r] + wr[b]
            within(got[r], ref, bw[b] + (2 ** -18 + 33 * U_F32) * wr[b] + 2 * U_F32 * ref, "weights")
        was = before.cpu().numpy().reshape(-1)
        assert np.array_equal(got[~touched].view(np.uint32), was[~touched].view(np.uint32))


# ------------------------------------------------------------------- evict

EVICT = [  # (fmt, page, ends, keep, sinks, recent)
    (0, 16, [100, 33, 32, 31, 0, 1], 32, 4, 8), (1, 64, [1000, 64, 65], 64, 0, 0), (2, 48, [500, 49], 48, 48, 0),
    (0, 64, [777, 2000], 700, 0, 700), (1, 16, [300], 1, 0, 0), (1, 16, [300], 1, 1, 0), (1, 128, [5000, 4097, 10], 2048, 4, 512),
    (0, 80, [900, 901], 900, 10, 20), (1, 64, [9001], 9000, 0, 1), (0, 32, [257], 130, 65, 65),
    (1, 48, [5000, 4097, 3999, 0, 4003], 4001, 4, 100), (2, 16, [17000], 16400, 0, 9),
]


def evict(pool, cache, keep, sinks, recent, max_end=None, **kw):
    need = -(-keep // pool.page)
    B = len(pool.ends)
    new = torch.tensor(pool.free[:B * need], dtype=torch.int32).view(B, need)
    kept, end = mla.paged_evict(cache, pool.dev_table(), pool.dev_ends(), max_end or pool.max_pages * pool.page, keep, new.cuda(),
                                sinks=sinks, recent=recent, **kw)
    return new.numpy(), kept.cpu().numpy(), end.cpu().numpy()


def apply_evict(pool, new, kept, end):
    """The host pool after the copy."""
    old = [None if a is None else a.copy() for a in (pool.kv, pool.scale, pool.pe, pool.weight)]
    for b in range(len(end)):
        n = int(end[b])
        src = pool.rows(b)[kept[b, :n]]
        i = np.arange(n)
        dst = new[b, i // pool.page].astype(np.int64) * pool.page + i % pool.page
        for a, o in zip((pool.kv, pool.scale, pool.pe, pool.weight), old):
            if a is not None:
                a[dst] = o[src]


@pytest.mark.parametrize("fmt,page,ends,keep,sinks,recent", EVICT)
def test_evict_keeps_the_heaviest_rows(fmt, page, ends, keep, sinks, recent):
    pool = Pool(fmt, ends, page, seed=21, spare=len(ends) * -(-keep // page) + 2)
    cache = pool.device()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    new, kept, end = evict(pool, cache, keep, sinks, recent, status=status)
    ref, rend = evict_reference(pool, keep, sinks, recent)
    assert np.array_equal(kept, ref) and np.array_equal(end, rend)
    apply_evict(pool, new, ref, rend)
    pool.same_as(cache)
    assert int(status) == 0


def test_evict_ties_and_strange_weights():
    pool = Pool(0, [600, 400, 300], 16, seed=22, spare=60)
    r0, r1, r2 = pool.rows(0), pool.rows(1), pool.rows(2)
    pool.weight[r0] = np.random.default_rng(1).integers(0, 3, 600)       # many ties
    pool.weight[r1] = 0.0                                                # all tie
    pool.weight[r1[::2]] = -0.0
    pool.weight[r2[:100]] = np.nan
    pool.weight[r2[100:120]] = np.inf
    pool.weight[r2[120:200]] = -1.0
    cache = pool.device()
    new, kept, end = evict(pool, cache, 250, 3, 20)
    ref, rend = evict_reference(pool, 250, 3, 20)
    assert np.array_equal(kept, ref) and np.array_equal(end, rend)
    apply_evict(pool, new, ref, rend)
    pool.same_as(cache)


def test_evict_sequences_with_bad_pages_keep_nothing():
    pool = Pool(1, [300, 300, 300, 20], 64, seed=23, spare=12)
    good = pool.table.copy()
    cache = pool.device()
    pool.table[0, 2] = -1
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    new = torch.tensor(pool.free[:8], dtype=torch.int32).view(4, 2)
    new[1, 1] = pool.num_pages
    new[3, 1] = -5                                                       # not needed: 20 rows
    kept, end = mla.paged_evict(cache, pool.dev_table(), pool.dev_ends(), 300, 100, new.cuda(), status=status)
    kept, end = kept.cpu().numpy(), end.cpu().numpy()
    assert int(status) == mla.DEV_BAD_PAGE
    pool.table = good
    ref, rend = evict_reference(pool, 100, 0, 0)
    ref[:2], rend[:2] = -1, 0
    assert np.array_equal(kept, ref) and np.array_equal(end, rend)
    apply_evict(pool, new.numpy(), ref, rend)
    pool.same_as(cache)


def test_evict_clamps_lengths():
    pool = Pool(0, [300, 200, 100], 16, seed=24, spare=20)
    cache = pool.device()
    true = pool.ends
    pool.ends = np.array([1000, -4, 100], np.int32)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    new, kept, end = evict(pool, cache, 64, 0, 4, max_end=300, status=status)
    pool.ends = np.array([300, 0, 100], np.int32)
    ref, rend = evict_reference(pool, 64, 0, 4)
    assert np.array_equal(kept, ref) and np.array_equal(end, rend) and true[0] == 300
    assert int(status) == mla.DEV_END_POS_CLAMPED


def test_evict_of_a_sequence_past_the_staged_length():
    # longer than the keys a cluster stages in shared memory
    T, page = 8 * 55296 + 1000, 1024
    pages = -(-T // page)
    g = torch.Generator().manual_seed(1)
    cache = mla.PagedCache(pages + 2, page, mla.MLA_KV_FP8_E4M3_B128)
    cache.kv.random_(0, 127)
    cache.pe.normal_()
    perm = torch.randperm(pages + 2, generator=g)
    cache.weight.copy_(torch.randint(0, 1 << 20, cache.weight.shape, generator=g).float())
    table, new = perm[:pages].int()[None], perm[pages:].int()[None]
    kept, end = mla.paged_evict(cache, table.cuda(), torch.tensor([T], dtype=torch.int32, device="cuda"), T, 1500, new.cuda(), recent=7)
    t = torch.arange(T)
    rows = table[0].long()[t // page] * page + t % page
    w = cache.weight.cpu().view(-1)[rows].numpy().astype(np.float64)
    w[T - 7:] = np.inf
    ref = np.sort(np.lexsort((np.arange(T), -w))[:1500])
    assert np.array_equal(kept.cpu().numpy()[0], ref) and int(end) == 1500
    i = torch.arange(1500)
    dst = new[0].long()[i // page] * page + i % page
    for x in (cache.kv.view(-1, 512), cache.pe.view(-1, 64), cache.kv_scale.view(-1, 4)):
        x = x.cpu()
        assert torch.equal(x[dst], x[rows[ref]])


# ------------------------------------------------------- the set together

@pytest.mark.parametrize("fmt,H", [(0, 16), (1, 64), (0, 128), (1, 128)])
def test_serving_with_a_budget(fmt, H):
    # prompts written, steps that write, attend and weigh, one eviction, more
    # steps on the new pages: every step against the references
    page, keep, B = 16, 90, 3
    lens = np.array([150, 91, 40], np.int32)
    grown = lens + 3
    pool = Pool(fmt, grown, page, seed=25, spare=30)
    live = pool.live
    pool.ends = lens.copy()
    pool.weight[:] = np.nan
    cache = pool.device()
    tb = pool.dev_table()
    for b in range(B):                                       # prompts of each length
        n = int(lens[b])
        kvn, pen = randn_bf16((1, n, 512), 40 + b), randn_bf16((1, n, 64), 50 + b)
        mla.paged_append(cache, tb[b:b + 1].contiguous(), kvn.cuda(), pen.cuda(), torch.tensor([n], dtype=torch.int32).cuda())
        for j in range(n):
            r = pool.rows(b)[j]
            one = Pool.__new__(Pool)
            one.__dict__.update(pool.__dict__, ends=np.array([j + 1], np.int32), table=pool.table[b:b + 1])
            one.append(kvn[:, j], pen[:, j], 1)
            pool.weight[r] = 0.0
    pool.same_as(cache, "after the prompts")
    ws = mla.alloc_paged_workspace(B, H)
    limit = pool.max_pages * page

    def step(k):
        pool.ends = pool.ends + 1
        kvn, pen = randn_bf16((B, 512), 60 + k), randn_bf16((B, 64), 70 + k)
        ql, qp = queries(B, H, 80 + k)
        e, t = pool.dev_ends(), pool.dev_table()
        out, lse = mla.paged_decode(cache, t, ql.cuda(), qp.cuda(), e, limit, SM, kv_new=kvn.cuda(), pe_new=pen.cuda(), workspace=ws)
        mla.paged_weights(cache, t, ql.cuda(), qp.cuda(), lse, e, limit, SM)
        pool.append(kvn, pen, 1)
        ref, rl, wr, bo, bl, bw = reference(pool, ql, qp, SM)
        within(f64(out), ref, bo, f"out of step {k}")
        within(f64(lse), rl, bl, f"lse of step {k}")
        got = cache.weight.cpu().numpy().reshape(-1)
        for b in range(B):
            r = pool.rows(b)
            total = pool.weight[r] + wr[b]
            # (the lse is the kernel's own: off by bl)
            within(got[r], total, bw[b] + np.expm1(2 * bl[b].max()) * wr[b] + 2 ** -18 * wr[b] + 4 * U_F32 * total, f"weights of step {k}")
        pool.weight[:] = got                                 # the next comparison starts from the device's totals

    for k in range(3):
        step(k)
    new, kept, end = evict(pool, cache, keep, 2, 16)
    ref, rend = evict_reference(pool, keep, 2, 16)
    assert np.array_equal(kept, ref) and np.array_equal(end, rend)
    apply_evict(pool, new, ref, rend)
    pool.same_as(cache, "after the eviction")
    pool.table = np.concatenate([new, np.array(pool.free[-B:], np.int32)[:, None]], 1).astype(np.int32)   # and a page to grow into
    pool.ends, pool.max_pages = rend, pool.table.shape[1]
    limit = pool.max_pages * page
    for k in range(3, 5):
        step(k)


# -------------------------------------------------- streams and graphs

def test_a_captured_step_replays_with_new_lengths():
    for fmt, H in ((0, 128), (1, 16)):
        pool = Pool(fmt, [700, 300], 64, seed=26)
        cache, tb = pool.device(), pool.dev_table()
        e = torch.tensor([700, 300], dtype=torch.int32).cuda()
        ql, qp = queries(2, H, 3)
        qld, qpd = ql.cuda(), qp.cuda()
        kvn, pen = randn_bf16((2, 512), 5).cuda(), randn_bf16((2, 64), 6).cuda()
        ws = mla.alloc_paged_workspace(2, H)
        out, lse = torch.empty(2, H, 512, dtype=torch.bfloat16, device="cuda"), torch.empty(2, H, device="cuda")

        def step():
            mla.paged_decode(cache, tb, qld, qpd, e, 704, SM, kv_new=kvn, pe_new=pen, out=out, lse=lse, workspace=ws)
            mla.paged_weights(cache, tb, qld, qpd, lse, e, 704, SM)

        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            step()
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        cache.weight.copy_(torch.from_numpy(pool.weight).view_as(cache.weight))
        cache.kv.copy_(pool.device().kv)
        if fmt:
            cache.kv_scale.copy_(pool.device().kv_scale)
        cache.pe.copy_(pool.device().pe)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        host = Pool.__new__(Pool)
        for ends in ([700, 300], [65, 299], [0, 1]):
            e.copy_(torch.tensor(ends, dtype=torch.int32))
            graph.replay()
            torch.cuda.synchronize()
            host.__dict__.update(pool.__dict__, ends=np.array(ends, np.int32))
            host.append(kvn.cpu(), pen.cpu(), 1)
            ref, rl, _, bo, bl, _ = reference(host, ql, qp, SM)
            within(f64(out), ref, bo, f"out at {ends}")
            within(f64(lse), rl, bl, f"lse at {ends}")


def test_calls_on_two_streams_with_workspaces_of_their_own():
    pools = [Pool(0, [900, 20], 64, seed=27), Pool(1, [1500], 16, seed=28)]
    H = [128, 16]
    caches, want, args = [], [], []
    for p, h in zip(pools, H):
        ql, qp = queries(len(p.ends), h, 3)
        want.append(reference(p, ql, qp, SM))
        caches.append(p.device())
        args.append((p.dev_table(), ql.cuda(), qp.cuda(), p.dev_ends(), p.max_pages * p.page, SM))
    ws = [mla.alloc_paged_workspace(len(p.ends), h) for p, h in zip(pools, H)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [None, None]
    for _ in range(10):
        for i in (0, 1):
            with torch.cuda.stream(streams[i]):
                got[i] = mla.paged_decode(caches[i], *args[i], workspace=ws[i])
    torch.cuda.synchronize()
    for i in (0, 1):
        within(f64(got[i][0]), want[i][0], want[i][3], "out")
        within(f64(got[i][1]), want[i][1], want[i][4], "lse")


def test_the_binding_refuses_other_shapes_and_types():
    pool = Pool(0, [100], 16, seed=29)
    cache, tb, e = pool.device(), pool.dev_table(), pool.dev_ends()
    ql, qp = [x.cuda() for x in queries(1, 16, 3)]
    for bad in (dict(table=tb.long()), dict(table=tb[0]), dict(table=tb.repeat(2, 1)), dict(table=tb.cpu()), dict(ql=ql.float()),
                dict(qp=qp[:, :8]), dict(e=e.long()), dict(ql=torch.cat([ql, ql], -1)[..., :512]), dict(e=e.cpu())):
        a = {"table": tb, "ql": ql, "qp": qp, "e": e, **bad}
        with pytest.raises(ValueError):
            mla.paged_decode(cache, a["table"], a["ql"], a["qp"], a["e"], 100, SM)
    with pytest.raises(mla.MLAError) as err:
        mla.paged_decode(cache, tb, ql, qp, e, 16 * tb.shape[1] + 1, SM)
    assert err.value.code == 2
    with pytest.raises(mla.MLAError) as err:
        mla.paged_decode(cache, tb, ql, qp, e, 100, SM, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    assert err.value.code == 4
    with pytest.raises(ValueError):
        mla.paged_evict(cache, tb, e, 100, 10, tb[0])
    bare = mla.PagedCache(cache.num_pages, 16, 0, kv=cache.kv, pe=cache.pe, weight=False)
    with pytest.raises(mla.MLAError) as err:
        mla.paged_evict(bare, tb, e, 100, 10, tb)
    assert err.value.code == 1


# ------------------------------------------ short sequences, taken whole

@pytest.mark.parametrize("fmt,H", [(0, 16), (1, 16), (0, 32), (2, 32), (0, 64), (1, 64)])
def test_short_sequences_with_new_rows_bad_pages_and_none(fmt, H):
    # max_end_pos small enough that sequences are not split: the status word,
    # the empty sequences' outputs and the new rows come from the same kernel
    ends = [0, 1, 16, 17, 63, 64, 65, 128, 150, 200, 0, 255]
    pool = Pool(fmt, ends, 16, seed=31)
    B = len(ends)
    kvn, pen = randn_bf16((B, 512), 33), randn_bf16((B, 64), 34)
    ql, qp = queries(B, H, 35)
    for bad in (False, True):
        skip = [[] for _ in ends]
        if bad:                               # a page in the middle, and the last one of a sequence
            pool.table[8, 3] = -1
            pool.table[9, 12] = pool.num_pages
            skip[8], skip[9] = np.arange(48, 64), np.arange(192, 200)
        rows0 = Pool.rows
        pool.rows = lambda b, n=None: np.where(np.isin(np.arange(rows0(pool, b, n).size), skip[b]), 0, rows0(pool, b, n))
        cache = pool.device()
        ws = mla.alloc_paged_workspace(B, H)
        out, lse = mla.paged_decode(cache, pool.dev_table(), ql.cuda(), qp.cuda(), pool.dev_ends(), 256, SM,
                                    kv_new=kvn.cuda(), pe_new=pen.cuda(), workspace=ws)
        pool.append(kvn, pen, 1)
        pool.same_as(cache)
        ref, rl, _, bo, bl, _ = reference(pool, ql, qp, SM, leave_out=skip)
        within(f64(out), ref, bo, "out")
        within(f64(lse), rl, bl, "lse")
        assert mla.workspace_status(ws) == mla.DEV_APPEND_SKIPPED | (mla.DEV_BAD_PAGE if bad else 0)


def test_short_sequences_are_clamped_and_flagged():
    pool = Pool(1, [100, 200, 50], 16, seed=36)
    ql, qp = queries(3, 64, 1)
    ws = mla.alloc_paged_workspace(3, 64)
    e = torch.tensor([100, 500, -3], dtype=torch.int32)
    out, lse = mla.paged_decode(pool.device(), pool.dev_table(), ql.cuda(), qp.cuda(), e.cuda(), 200, SM, workspace=ws)
    ref, rl, _, bo, bl, _ = reference(pool, ql, qp, SM, ends=[100, 200, 0])
    within(f64(out), ref, bo, "out")
    within(f64(lse), rl, bl, "lse")
    assert mla.workspace_status(ws) == mla.DEV_END_POS_CLAMPED


@pytest.mark.parametrize("fmt,H,T", [(0, 64, 1000), (1, 64, 1000), (1, 16, 64 * 7 + 1), (0, 32, 64 * 5), (2, 16, 641)])
def test_new_rows_at_tile_borders_of_split_sequences(fmt, H, T):
    ends = [T, T - 1, T + 63, 64, 65]
    pool = Pool(fmt, ends, 48, seed=37)
    B = len(ends)
    cache = pool.device()
    kvn, pen = randn_bf16((B, 512), 38), randn_bf16((B, 64), 39)
    ql, qp = queries(B, H, 40)
    out, lse = mla.paged_decode(cache, pool.dev_table(), ql.cuda(), qp.cuda(), pool.dev_ends(), T + 63, SM,
                                kv_new=kvn.cuda(), pe_new=pen.cuda())
    pool.append(kvn, pen, 1)
    pool.same_as(cache)
    ref, rl, _, bo, bl, _ = reference(pool, ql, qp, SM)
    within(f64(out), ref, bo, "out")
    within(f64(lse), rl, bl, "lse")


# ------------------------------------- many sequences, streams, graphs, values

@pytest.mark.parametrize("fmt,H", [(0, 16), (1, 64), (0, 128), (1, 128)])
def test_new_rows_of_more_sequences_than_a_warp_schedules(fmt, H):
    # 130 sequences: the schedule kernel says which unit writes which row
    ends = [int(x) for x in np.random.default_rng(41).integers(0, 300, 130)]
    pool = Pool(fmt, ends, 64, seed=41)
    B = len(ends)
    cache = pool.device()
    kvn, pen = randn_bf16((B, 512), 42), randn_bf16((B, 64), 43)
    ql, qp = queries(B, H, 44)
    ws = mla.alloc_paged_workspace(B, H)
    for bound in (max(ends), pool.max_pages * pool.page):
        out, lse = mla.paged_decode(cache, pool.dev_table(), ql.cuda(), qp.cuda(), pool.dev_ends(), bound, SM,
                                    kv_new=kvn.cuda(), pe_new=pen.cuda(), workspace=ws)
        pool.append(kvn, pen, 1)
        pool.same_as(cache)
        ref, rl, _, bo, bl, _ = reference(pool, ql, qp, SM)
        within(f64(out), ref, bo, "out")
        within(f64(lse), rl, bl, "lse")
        assert mla.workspace_status(ws) == (mla.DEV_APPEND_SKIPPED if 0 in ends else 0)


def test_two_captured_graphs_share_a_workspace():
    # a split call and one whose sequences stay whole, replayed in turn
    pools = [Pool(1, [1500, 700], 64, seed=45), Pool(0, [200, 0, 77, 64], 16, seed=46)]
    heads, bounds = (64, 16), (1536, 208)
    ws = torch.empty(max(mla.paged_workspace_size(len(p.ends), h) for p, h in zip(pools, heads)), dtype=torch.uint8, device="cuda")
    graphs, outs, want, keep = [], [], [], []
    for p, h, bound in zip(pools, heads, bounds):
        ql, qp = queries(len(p.ends), h, 3)
        a = (p.device(), p.dev_table(), ql.cuda(), qp.cuda(), p.dev_ends(), bound, SM)
        want.append(reference(p, ql, qp, SM))
        out, lse = mla.paged_decode(*a, workspace=ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            mla.paged_decode(*a, out=out, lse=lse, workspace=ws)
        graphs.append(g)
        outs.append((out, lse))
        keep.append(a)
    for i in (0, 1, 0, 1, 1, 0):
        for x in outs[i]:
            x.fill_(float("nan"))
        graphs[i].replay()
        torch.cuda.synchronize()
        within(f64(outs[i][0]), want[i][0], want[i][3], "out")
        within(f64(outs[i][1]), want[i][1], want[i][4], "lse")
        assert mla.workspace_status(ws) == 0


def test_outputs_of_a_call_on_another_stream_are_that_streams():
    # the current stream still has work for the block it gave back last: the
    # outputs of a call on a second stream must not lie in it
    pool = Pool(0, [200, 100], 64, seed=47)
    ql, qp = queries(2, 16, 3)
    a = (pool.device(), pool.dev_table(), ql.cuda(), qp.cuda(), pool.dev_ends(), 256, SM)
    ref, rl, _, bo, bl, _ = reference(pool, ql, qp, SM)
    ws = mla.alloc_paged_workspace(2, 16)
    side = torch.cuda.Stream()
    mla.paged_decode(*a, workspace=ws)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    out = torch.empty((2, 16, 512), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((2, 16), dtype=torch.float32, device="cuda")
    out.fill_(0)                  # (its kernel is loaded before the wait)
    lse.fill_(0)
    torch.cuda._sleep(200_000_000)
    out.fill_(1)
    lse.fill_(1)
    del out, lse
    out, lse = mla.paged_decode(*a, workspace=ws, stream=side)
    torch.cuda.synchronize()
    within(f64(out), ref, bo, "out")
    within(f64(lse), rl, bl, "lse")


@pytest.mark.parametrize("fmt", [1, 2])
def test_appended_codes_of_all_bit_patterns(fmt):
    # rows of random bf16 bit patterns (NaN, infinities, subnormals, every
    # exponent): the block's largest magnitude among its numbers (NaN if it has
    # none), scale = fp32(amax / 448), codes of fp32(x / scale) saturated
    rng = np.random.default_rng(48)
    n = 600
    x = rng.integers(0, 1 << 16, (n, 512), dtype=np.uint16)
    x[100:300] = (x[100:300] & 0x80FF) | (rng.integers(0, 0x7F, (200, 1), dtype=np.uint16) << 8)   # few exponents a row
    x[300:400] &= 0x807F                                                        # subnormals
    x[400:500, :128] = 0x7FC1                                                   # blocks without a number
    kvn = torch.from_numpy(x.view(np.int16)).view(torch.bfloat16)
    pen = randn_bf16((n, 64), 49)
    cache = mla.PagedCache(n // 16 + 1, 16, fmt)
    tb = torch.arange(n // 16 + 1, dtype=torch.int32, device="cuda")[None]
    mla.paged_append(cache, tb, kvn[None].cuda(), pen[None].cuda(), torch.tensor([n], dtype=torch.int32, device="cuda"))
    f = (x.astype(np.uint32) << 16).view(np.float32).reshape(n, 4, 128)
    with np.errstate(all="ignore"):
        amax = np.where(np.isnan(f).all(-1), np.float32(np.nan), np.nanmax(np.where(np.isnan(f), -1.0, np.abs(f)), -1)).astype(np.float32)
        scale = (amax / np.float32(448.0)).astype(np.float32)
        if fmt == 2:
            m, e = np.frexp(scale.astype(np.float64))     # scale = m 2^e, m in [0.5, 1)
            up = np.ldexp(1.0, np.where(m == 0.5, e - 1, e)).astype(np.float32)
            scale = np.where((scale > 0) & np.isfinite(scale), up, scale)
        q = (f / scale[..., None]).astype(np.float32)
    codes = torch.from_numpy(np.clip(q, -448.0, 448.0)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    codes = np.where(np.isnan(q), 0x7F, codes)
    codes = np.where((amax > 0)[..., None], codes, 0)     # all-zero blocks, and blocks without a number
    got = cache.kv.cpu().numpy().reshape(-1, 4, 128)[:n]
    got_scale = cache.kv_scale.cpu().numpy().reshape(-1, 4)[:n]
    assert np.array_equal(np.isnan(got_scale), np.isnan(scale))
    assert np.array_equal(got_scale[~np.isnan(scale)], scale[~np.isnan(scale)])
    assert np.array_equal(got, codes)


@pytest.mark.parametrize("ends", [[100, 70, 200], [2000, 700, 3000]])   # whole, and split
@pytest.mark.parametrize("fmt,H", [(0, 16), (1, 16), (0, 64), (1, 64), (0, 128), (1, 128)])
def test_nan_of_attended_rows_and_queries_is_passed_on(fmt, H, ends):
    pool = Pool(fmt, ends, 64, seed=50)
    ql, qp = queries(3, H, 51)
    ref, rl, _, bo, bl, _ = reference(pool, ql, qp, SM)
    cache = pool.device()
    kv, pe = cache.kv.view(-1, 512), cache.pe.view(-1, 64)
    kv[int(pool.rows(0)[37]), 300] = 0x7F if fmt else float("nan")
    pe[int(pool.rows(1)[5]), 40] = float("nan")
    ql[2, 3, 10] = ql[2, H - 1, 400] = float("nan")
    out, lse = mla.paged_decode(cache, pool.dev_table(), ql.cuda(), qp.cuda(), pool.dev_ends(), max(ends), SM)
    out, lse = f64(out), f64(lse)
    assert np.isnan(out[:2]).all() and np.isnan(lse[:2]).all()
    sick = [3, H - 1]
    well = [h for h in range(H) if h not in sick]
    assert np.isnan(out[2, sick]).all() and np.isnan(lse[2, sick]).all()
    within(out[2, well], ref[2, well], bo[2, well], "out")
    within(lse[2, well], rl[2, well], bl[2, well], "lse")


@pytest.mark.parametrize("fmt,H,B", [(0, 16, 100), (1, 64, 100), (0, 128, 60), (1, 128, 60), (1, 128, 30), (0, 32, 128)])
def test_ragged_batches_with_more_units_than_places(fmt, H, B):
    # lengths spread so that short last units share CTAs: every unit's part
    # reaches the place of its sequence, its new row and its flags too
    rng = np.random.default_rng(52 + B)
    ends = [int(x) for x in rng.integers(1, 2500, B)]
    ends[3], ends[B - 1], ends[7] = 0, 2500, 1
    pool = Pool(fmt, ends, 32, seed=52)
    cache = pool.device()
    kvn, pen = randn_bf16((B, 512), 53), randn_bf16((B, 64), 54)
    ql, qp = queries(B, H, 55)
    ws = mla.alloc_paged_workspace(B, H)
    args = (cache, pool.dev_table(), ql.cuda(), qp.cuda(), pool.dev_ends(), 2500, SM)
    out, lse = mla.paged_decode(*args, kv_new=kvn.cuda(), pe_new=pen.cuda(), workspace=ws)
    assert mla.workspace_status(ws) == mla.DEV_APPEND_SKIPPED      # the empty sequence
    pool.append(kvn, pen, 1)
    pool.same_as(cache)
    ref, rl, _, bo, bl, _ = reference(pool, ql, qp, SM)
    within(f64(out), ref, bo, "out")
    within(f64(lse), rl, bl, "lse")
    again, lse2 = mla.paged_decode(*args, workspace=ws)
    assert torch.equal(again, out) and torch.equal(lse2, lse)
    assert mla.workspace_status(ws) == 0
