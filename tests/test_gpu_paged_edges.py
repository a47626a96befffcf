"""Calls of the paged-cache operators at the edges of what their documentation
allows: arguments that share memory, infinite scores, rows behind a sequence in
its last page, pool tensors replaced by others, waits that run out."""
import numpy as np
import pytest
import torch

import mla_latent_kv_07_gb300 as mla

from mla_cases import f64
from paged_cases import Pool, U_F32, evict_reference, randn_bf16, reference, within

pytestmark = pytest.mark.gpu
SM = 0.1352


@pytest.fixture(scope="module", autouse=True)
def _built():
    from mla_latent_kv_07_gb300 import build
    build.build()
    mla.lib()


# ---------------------------------------------------------- eviction in place

@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("ends,keep,sinks,recent", [
    ([4000, 33, 32, 31, 0, 1, 2500], 32, 4, 8), ([300] * 64, 130, 2, 100), ([9001, 17], 9000, 0, 1), ([70], 64, 0, 0)])
def test_eviction_replaces_the_lengths_in_place(fmt, ends, keep, sinks, recent):
    # new_end_pos is end_pos: every CTA of a sequence's cluster has read its
    # length before the new one is stored
    pool = Pool(fmt, ends, 32, seed=60, spare=len(ends) * -(-keep // 32))
    cache, e = pool.device(), pool.dev_ends()
    need = -(-keep // 32)
    new = torch.tensor(pool.free[:len(ends) * need], dtype=torch.int32).view(len(ends), need).cuda()
    ref, rend = evict_reference(pool, keep, sinks, recent)
    for _ in range(20):
        e.copy_(pool.dev_ends())
        kept, end = mla.paged_evict(cache, pool.dev_table(), e, max(ends), keep, new, sinks=sinks, recent=recent, new_end_pos=e)
        assert end is e
        assert np.array_equal(kept.cpu().numpy(), ref) and np.array_equal(e.cpu().numpy(), rend)


def test_a_captured_eviction_in_place_replays():
    pool = Pool(1, [900, 400, 64], 64, seed=61, spare=6)
    cache, tb, e = pool.device(), pool.dev_table(), pool.dev_ends()
    new = torch.tensor(pool.free[:6], dtype=torch.int32).view(3, 2).cuda()
    kept = torch.empty((3, 100), dtype=torch.int32, device="cuda")
    mla.paged_evict(cache, tb, e, 900, 100, new, recent=10, kept=kept, new_end_pos=e)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mla.paged_evict(cache, tb, e, 900, 100, new, recent=10, kept=kept, new_end_pos=e)
    for ends in ([900, 400, 64], [101, 100, 64], [0, 400, 5]):
        e.copy_(torch.tensor(ends, dtype=torch.int32))
        g.replay()
        pool.ends = np.array(ends, np.int32)
        ref, rend = evict_reference(pool, 100, 0, 10)
        assert np.array_equal(kept.cpu().numpy(), ref) and np.array_equal(e.cpu().numpy(), rend)


# --------------------------------------- infinite scores, rows behind the end

@pytest.mark.parametrize("ends", [[100, 70, 200], [2000, 700, 3000]])   # whole, and split
@pytest.mark.parametrize("fmt,H", [(0, 16), (1, 16), (0, 64), (1, 64), (0, 128), (1, 128), (2, 128)])
def test_infinite_rotary_keys(fmt, H, ends):
    # the score of such a row is an infinity of the sign of its product with
    # the query: weight 0 below, no distribution above.  (Sixteen rows, so that
    # every place of a tile is among them; columns of either half.)
    pool = Pool(fmt, ends, 64, seed=62)
    ql, qp = randn_bf16((3, H, 512), 63), randn_bf16((3, H, 64), 64)
    rows = [np.arange(37, 53), np.arange(ends[1] - 16, ends[1]), np.arange(0)]
    cols, signs = [40, 5, 0], [1.0, -1.0, 1.0]
    ref, rl, _, bo, bl, _ = reference(pool, ql, qp, SM, leave_out=rows)
    cache = pool.device()
    for b in range(2):
        cache.pe.view(-1, 64)[torch.from_numpy(pool.rows(b)[rows[b]]).cuda(), cols[b]] = signs[b] * float("inf")
    ws = mla.alloc_paged_workspace(3, H)
    out, lse = mla.paged_decode(cache, pool.dev_table(), ql.cuda(), qp.cuda(), pool.dev_ends(), max(ends), SM, workspace=ws)
    out, lse = f64(out), f64(lse)
    assert mla.workspace_status(ws) == 0
    for b in range(3):
        q = f64(qp)[b, :, cols[b]] * signs[b]
        up = (q > 0) if len(rows[b]) else np.zeros(H, bool)
        assert (q != 0).all()
        assert np.isnan(out[b, up]).all() and np.isnan(lse[b, up]).all()
        within(out[b, ~up], ref[b, ~up], bo[b, ~up], f"out {b}")
        within(lse[b, ~up], rl[b, ~up], bl[b, ~up], f"lse {b}")


@pytest.mark.parametrize("fmt,H", [(0, 16), (1, 32), (0, 64), (1, 128), (0, 128)])
def test_weights_of_rows_with_a_score_of_minus_infinity(fmt, H):
    pool = Pool(fmt, [700, 90], 48, seed=65)
    ql, qp = randn_bf16((2, H, 512), 66), randn_bf16((2, H, 64), 67)
    qp[:, :, 9] = -qp[:, :, 9].abs()
    rows = [np.arange(100, 130), np.array([89])]
    _, rl, wr, _, _, bw = reference(pool, ql, qp, SM, leave_out=rows)
    cache = pool.device()
    for b in range(2):
        cache.pe.view(-1, 64)[torch.from_numpy(pool.rows(b)[rows[b]]).cuda(), 9] = float("inf")
    mla.paged_weights(cache, pool.dev_table(), ql.cuda(), qp.cuda(), torch.from_numpy(rl.astype(np.float32)).cuda(),
                      pool.dev_ends(), 700, SM)
    got = cache.weight.cpu().numpy().reshape(-1)
    for b in range(2):
        r = pool.rows(b)
        out = np.isin(np.arange(r.size), rows[b])
        assert np.array_equal(got[r[out]], pool.weight[r[out]])
        ref = pool.weight[r[~out]] + wr[b]
        within(got[r[~out]], ref, bw[b] + (2 ** -18 + (H + 2) * U_F32) * wr[b] + 2 * U_F32 * ref, "weights")


@pytest.mark.parametrize("ends", [[100, 65, 200, 3], [2000, 700, 3001, 17]])
@pytest.mark.parametrize("fmt,H", [(0, 16), (1, 32), (0, 64), (1, 64), (0, 128), (1, 128), (2, 128)])
def test_rows_behind_the_last_position_change_no_bit(fmt, H, ends):
    # equal inputs, other contents of the rows that no sequence uses
    pool = Pool(fmt, ends, 64, seed=68)
    ql, qp = randn_bf16((4, H, 512), 69).cuda(), randn_bf16((4, H, 64), 70).cuda()
    spare = torch.from_numpy(~pool.live).cuda()
    got = []
    for k in range(4):
        cache = pool.device()
        if k:
            n = int(spare.sum())
            kv, pe = randn_bf16((n, 512), 71 + k).cuda() * 3 ** k, randn_bf16((n, 64), 75 + k).cuda() * 3 ** k
            if fmt:
                cache.kv.view(-1, 512)[spare] = (kv.view(torch.int16) & 0x7F).to(torch.uint8)
                cache.kv_scale.view(-1, 4)[spare] = 0.01 * k
            else:
                cache.kv.view(-1, 512)[spare] = kv
            cache.pe.view(-1, 64)[spare] = pe
        out, lse = mla.paged_decode(cache, pool.dev_table(), ql, qp, pool.dev_ends(), max(ends), SM)
        mla.paged_weights(cache, pool.dev_table(), ql, qp, lse, pool.dev_ends(), max(ends), SM)
        got.append((out, lse, cache.weight.view(-1)[~spare]))
    for x in got[1:]:
        for a, b in zip(x, got[0]):
            assert torch.equal(a, b)


# ------------------------------------------------ the pool's tensors replaced

@pytest.mark.parametrize("fmt", [0, 1])
def test_tensors_assigned_to_a_pool_take_effect(fmt):
    pool = Pool(fmt, [300, 77], 16, seed=80)
    other = Pool(fmt, [300, 77], 16, seed=81)
    other.table = pool.table
    cache, old = pool.device(), pool.device()
    for name in ("kv", "kv_scale", "pe", "weight"):
        setattr(cache, name, getattr(other.device(), name))
    kvn, pen = randn_bf16((2, 512), 82), randn_bf16((2, 64), 83)
    was = cache.weight.clone()
    mla.paged_append(cache, pool.dev_table(), kvn[:, None].contiguous().cuda(), pen[:, None].contiguous().cuda(), pool.dev_ends())
    other.append(kvn, pen, 1)
    other.same_as(cache)
    cache.weight = torch.zeros_like(cache.weight)
    assert (cache.weight == 0).all()
    ql, qp = randn_bf16((2, 16, 512), 84).cuda(), randn_bf16((2, 16, 64), 85).cuda()
    cache.kv, cache.kv_scale, cache.pe = old.kv, old.kv_scale, old.pe      # rows in use, all finite
    out, lse = mla.paged_decode(cache, pool.dev_table(), ql, qp, pool.dev_ends(), 300, SM)
    mla.paged_weights(cache, pool.dev_table(), ql, qp, lse, pool.dev_ends(), 300, SM)
    ref, rl, wr, bo, bl, bw = reference(pool, ql.cpu(), qp.cpu(), SM)
    within(f64(out), ref, bo, "out")
    got = cache.weight.cpu().numpy().reshape(-1)
    for b in range(2):
        within(got[pool.rows(b)], wr[b], bw[b] + np.expm1(2 * bl[b].max()) * wr[b] + (2 ** -18 + 18 * U_F32) * wr[b], "weights")
    assert was.data_ptr() != cache.weight.data_ptr()
    cache.weight = None
    with pytest.raises(mla.MLAError) as err:
        mla.paged_weights(cache, pool.dev_table(), ql, qp, lse, pool.dev_ends(), 300, SM)
    assert err.value.code == 1


@pytest.mark.parametrize("fmt", [0, 1])
def test_other_tensors_are_refused_on_assignment(fmt):
    cache = mla.PagedCache(3, 16, fmt)
    kept = {n: getattr(cache, n) for n in ("kv", "kv_scale", "pe", "weight")}
    for name, t in (("kv", cache.kv.float()), ("kv", cache.kv[:2]), ("kv", None), ("kv", cache.kv.cpu()), ("pe", None),
                    ("pe", cache.pe.transpose(0, 1)), ("weight", cache.weight.double()), ("weight", cache.weight[:, :8]),
                    ("kv_scale", None if fmt else torch.zeros(3, 16, 4, device="cuda"))):
        with pytest.raises(ValueError):
            setattr(cache, name, t)
    for name in ("fmt", "num_pages", "page_size"):
        with pytest.raises(AttributeError):
            setattr(cache, name, 1)
    assert all(getattr(cache, n) is t for n, t in kept.items())


# ------------------------------------------------------- waits that run out

@pytest.mark.parametrize("ends", [[200, 0, 256], [40000, 700, 4097]])   # whole, and split
@pytest.mark.parametrize("fmt,H", [(0, 16), (1, 16), (0, 32), (1, 32), (0, 64), (1, 64), (0, 128), (1, 128)])
def test_a_decode_whose_waits_run_out_reports_it(fmt, H, ends):
    # the next call on the same device and workspace is right again
    pool = Pool(fmt, ends, 32, seed=90)
    ql, qp = randn_bf16((3, H, 512), 91), randn_bf16((3, H, 64), 92)
    ref, rl, _, bo, bl, _ = reference(pool, ql, qp, SM)
    a = (pool.device(), pool.dev_table(), ql.cuda(), qp.cuda(), pool.dev_ends(), max(ends), SM)
    ws = mla.alloc_paged_workspace(3, H)
    for _ in range(3):
        assert mla.selftest_paged_decode_timeout(*a, ws) == mla.DEV_PIPELINE_TIMEOUT
        out, lse = mla.paged_decode(*a, workspace=ws)
        assert mla.workspace_status(ws) == 0
        within(f64(out), ref, bo, "out")
        within(f64(lse), rl, bl, "lse")
    pool.same_as(a[0])


@pytest.mark.parametrize("ends", [[9000, 700, 4097], [40000, 0, 77]])
@pytest.mark.parametrize("fmt,H", [(0, 16), (1, 16), (0, 64), (1, 64), (0, 128), (1, 128)])
def test_weights_whose_waits_run_out_report_it(fmt, H, ends):
    pool = Pool(fmt, ends, 32, seed=93)
    ql, qp = randn_bf16((3, H, 512), 94), randn_bf16((3, H, 64), 95)
    _, rl, wr, _, _, bw = reference(pool, ql, qp, SM)
    cache, status = pool.device(), torch.zeros(1, dtype=torch.int32, device="cuda")
    a = (pool.dev_table(), ql.cuda(), qp.cuda(), torch.from_numpy(rl.astype(np.float32)).cuda(), pool.dev_ends(), max(ends), SM)
    for _ in range(3):
        status.zero_()
        mla.selftest_paged_weights_timeout(cache, *a, status)
        assert int(status) == mla.DEV_PIPELINE_TIMEOUT
        cache.weight.copy_(torch.from_numpy(pool.weight).view_as(cache.weight))
        status.zero_()
        mla.paged_weights(cache, *a, status=status)
        assert int(status) == 0
        got = cache.weight.cpu().numpy().reshape(-1)
        for b in range(3):
            r = pool.rows(b)
            tot = pool.weight[r] + wr[b]
            within(got[r], tot, bw[b] + (2 ** -18 + (H + 2) * U_F32) * wr[b] + 2 * U_F32 * tot, "weights")


# ---------------------------------------------------- several tokens a sequence

@pytest.mark.parametrize("fmt,H", [(0, 16), (1, 64), (0, 128), (1, 128)])
def test_tokens_of_a_chunk_as_sequences_that_share_a_table_row(fmt, H):
    # s new tokens per sequence: the table's row repeated, end_pos one further
    # for each; every token attends to the rows up to its own
    s, ends = 5, [700, 64, 5]
    pool = Pool(fmt, ends, 32, seed=96)
    ql, qp = randn_bf16((3 * s, H, 512), 97), randn_bf16((3 * s, H, 64), 98)
    kvn, pen = randn_bf16((3, s, 512), 99), randn_bf16((3, s, 64), 100)
    cache = pool.device()
    mla.paged_append(cache, pool.dev_table(), kvn.cuda(), pen.cuda(), pool.dev_ends())
    pool.append(kvn, pen, s)
    pool.same_as(cache)
    table = pool.dev_table().repeat_interleave(s, 0)
    each = (pool.dev_ends()[:, None] - s + 1 + torch.arange(s, dtype=torch.int32, device="cuda")).view(-1).to(torch.int32)
    out, lse = mla.paged_decode(cache, table, ql.cuda(), qp.cuda(), each, max(ends), SM)
    mla.paged_weights(cache, table, ql.cuda(), qp.cuda(), lse, each, max(ends), SM)
    wide = Pool.__new__(Pool)
    wide.__dict__.update(pool.__dict__, ends=each.cpu().numpy(), table=table.cpu().numpy())
    ref, rl, wr, bo, bl, bw = reference(wide, ql, qp, SM)
    within(f64(out), ref, bo, "out")
    within(f64(lse), rl, bl, "lse")
    got = cache.weight.cpu().numpy().reshape(-1)
    for b in range(3):
        n = ends[b]
        add, bound = np.zeros(n), np.zeros(n)
        for j in range(s):
            w, e = wr[b * s + j], each[b * s + j].item()
            add[:e] += w
            bound[:e] += bw[b * s + j] + np.expm1(2 * bl[b * s + j].max()) * w + (2 ** -18 + (H + 2) * U_F32) * w
        tot = pool.weight[pool.rows(b)] + add
        within(got[pool.rows(b)], tot, bound + 2 * s * U_F32 * tot, "weights")
