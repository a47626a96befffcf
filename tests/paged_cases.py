"""Shared helpers of the paged-cache tests: pools with poisoned unused rows and
page tables in a random order, the fp64 reference of a paged decode and of the
attention weights (the oracle on each sequence's rows laid side by side), and
error bounds derived from the formats.

Bounds.  u(t) = eps(t) / 2 is the largest relative error of a rounding:
u(bf16) = 2^-8, u(fp32) = 2^-24.
  score   a sum of 576 exact products in fp32, added at most 64 at a time with
          each partial sum off by 2 u(fp32): |ds| <= 64 * 2^-23 * sigma * sum |q c|
          (sum |q c| over the 576 columns), then scaled and referred to a
          maximum in fp32, both off by u(fp32) of a number below 2^7: + 2^-16.
  weight  w = exp(s - lse): |dw| <= w (exp(2 max ds) - 1)  (its own score, and the sum's)
  lse     |dlse| <= max ds + 2^-16
  out     p is rounded to bf16 once and out once, the sum is taken in fp32:
          |dout| <= u(bf16) (|out| + sum w|c|) + 2 max ds sum w|c| + 2^-16 sum w|c|
"""
from __future__ import annotations

import numpy as np
import torch

import mla_latent_kv_07_gb300 as mla
from mla_latent_kv_07_gb300 import inputs
from oracle import oracle as orc

from mla_cases import bits, f64

U_BF16, U_F32 = 2.0 ** -8, 2.0 ** -24


def randn_bf16(shape, seed):
    return inputs.randn_bf16(shape, seed)


class Pool:
    """A pool on the host (numpy, oracle conventions) and the page tables of
    its sequences.  Rows no sequence uses hold NaN (codes 0x7f and infinite
    scales for FP8); table entries past a sequence's pages are out of range."""

    def __init__(self, fmt, ends, page, seed, spare=4, extra_pages=2, kv=None, shared=0):
        self.fmt, self.page, self.ends = fmt, page, np.asarray(ends, np.int32)
        rng = np.random.default_rng(seed)
        used = [-(-int(max(e, 0)) // page) for e in ends]
        self.max_pages = max(max(used), 1) + extra_pages
        self.num_pages = sum(used) + spare
        perm = rng.permutation(self.num_pages)
        self.table = rng.choice(np.array([-1, -2 ** 31, self.num_pages, 2 ** 31 - 1]), (len(ends), self.max_pages)).astype(np.int32)
        at = 0
        for b, n in enumerate(used):
            self.table[b, :n] = perm[at:at + n]
            at += n
        self.free = [int(x) for x in perm[at:]]
        for b in range(1, len(ends)):           # the first `shared` pages of every sequence are sequence 0's
            n = min(shared, used[0], used[b])
            self.table[b, :n] = self.table[0, :n]
        rows = self.num_pages * page
        kvb = bits(randn_bf16((rows, 512), seed + 1)) if kv is None else np.array(kv)
        self.pe = bits(randn_bf16((rows, 64), seed + 2)).copy()
        self.weight = np.exp(1.5 * rng.standard_normal(rows)).astype(np.float32)
        live = np.zeros(rows, bool)
        for b, e in enumerate(ends):
            live[self.rows(b, e)] = True
        self.live = live
        if fmt == 0:
            self.kv, self.scale = kvb.copy(), None
            self.kv[~live] = 0x7FC0
        else:
            self.kv, self.scale = orc.quantize_rows(kvb, pow2=fmt == 2)
            self.kv[~live] = 0x7F
            self.scale[~live] = np.inf
        self.pe[~live] = 0x7FC0
        self.weight[~live] = np.nan

    def rows(self, b, n=None):
        n = int(max(self.ends[b] if n is None else n, 0))
        t = np.arange(n)
        return self.table[b, t // self.page].astype(np.int64) * self.page + t % self.page

    def device(self):
        sh = (self.num_pages, self.page)
        if self.fmt == 0:
            kv = torch.from_numpy(self.kv.view(np.int16)).view(torch.bfloat16).view(sh + (512,)).cuda()
        else:
            kv = torch.from_numpy(self.kv).view(sh + (512,)).cuda()
        sc = None if self.scale is None else torch.from_numpy(self.scale).view(sh + (4,)).cuda()
        pe = torch.from_numpy(self.pe.view(np.int16)).view(torch.bfloat16).view(sh + (64,)).cuda()
        w = torch.from_numpy(self.weight).view(sh).cuda()
        return mla.PagedCache(self.num_pages, self.page, self.fmt, kv=kv, kv_scale=sc, pe=pe, weight=w)

    def dev_table(self):
        return torch.from_numpy(self.table).cuda()

    def dev_ends(self):
        return torch.from_numpy(self.ends).cuda()

    def same_as(self, cache, what="pool"):
        """The device pool equals the host pool, bit for bit."""
        flat = lambda t: t.cpu().contiguous()
        if self.fmt == 0:
            assert np.array_equal(bits(cache.kv).reshape(-1, 512), self.kv), what
        else:
            assert np.array_equal(flat(cache.kv).numpy().reshape(-1, 512), self.kv), what
            assert np.array_equal(flat(cache.kv_scale).numpy().reshape(-1, 4).view(np.uint32), self.scale.view(np.uint32)), what
        assert np.array_equal(bits(cache.pe).reshape(-1, 64), self.pe), what
        assert np.array_equal(flat(cache.weight).numpy().reshape(-1).view(np.uint32), self.weight.view(np.uint32)), what

    def append(self, kv_new, pe_new, s):
        """Host counterpart of paged_append: new row j of sequence b at end - s + j."""
        kvb, peb = bits(kv_new).reshape(-1, 512), bits(pe_new).reshape(-1, 64)
        for b, e in enumerate(self.ends):
            for j in range(s):
                t = int(e) - s + j
                if t < 0 or t >= self.max_pages * self.page:
                    continue
                pg = self.table[b, t // self.page]
                if pg < 0 or pg >= self.num_pages:
                    continue
                r = int(pg) * self.page + t % self.page
                x = kvb[b * s + j]
                if self.fmt == 0:
                    self.kv[r] = x
                else:
                    q, sc = orc.quantize_rows(x[None], pow2=self.fmt == 2)
                    self.kv[r], self.scale[r] = q[0], sc[0]
                self.pe[r] = peb[b * s + j]
                self.weight[r] = 0.0


def reference(pool, ql, qp, scale, ends=None, leave_out=None):
    """fp64 (out [B,H,512], lse [B,H], weights: list of [n_b] summed over heads,
    bounds of out, lse and weights).  leave_out: per sequence, positions that are not attended to."""
    ends = pool.ends if ends is None else ends
    B, H = ql.shape[:2]
    q = np.concatenate([f64(ql), f64(qp)], -1)
    out, lse = np.zeros((B, H, 512)), np.full((B, H), -np.inf)
    b_out, b_lse, w_all, b_w = np.zeros_like(out), np.zeros((B, H)), [], []
    for b in range(B):
        rows = pool.rows(b, ends[b])
        if leave_out is not None:
            rows = rows[~np.isin(np.arange(rows.size), leave_out[b])]
        n = rows.size
        if n == 0:
            w_all.append(np.zeros(0))
            b_w.append(np.zeros(0))
            continue
        oc = {"fmt": pool.fmt, "kv": pool.kv[rows][None], "pe": pool.pe[rows][None]}
        if pool.scale is not None:
            oc["kv_scale"] = pool.scale[rows][None]
        o, l, w = orc.decode_absorbed(oc, bits(ql[b:b + 1]), bits(qp[b:b + 1]), np.array([n], np.int32), scale, weights_upto=n)
        out[b], lse[b] = o, l
        lat = pool.kv[rows] if pool.scale is None else orc.dequant_rows(pool.kv[rows], pool.scale[rows])
        c = np.abs(orc.bf16_bits_to_f64(lat))
        k = np.concatenate([c, np.abs(orc.bf16_bits_to_f64(pool.pe[rows]))], -1)
        ds = 64 * 2.0 ** -23 * abs(scale) * (np.abs(q[b]) @ k.T) + 2.0 ** -16      # [H, n]
        dmax = ds.max(1, keepdims=True)
        wc = w @ c
        b_out[b] = U_BF16 * (np.abs(o) + wc) + (2 * dmax + 2.0 ** -16) * wc
        b_lse[b] = dmax[:, 0] + 2.0 ** -16
        w_all.append(w.sum(0))
        b_w.append((w * np.expm1(2 * dmax)).sum(0))
    return out, lse, w_all, b_out, b_lse, b_w


def within(got, ref, bound, what):
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    ninf = np.isneginf(ref)
    assert np.array_equal(np.isneginf(got), ninf), f"{what}: -inf pattern differs"
    d = np.abs(got[~ninf] - ref[~ninf])
    b = np.broadcast_to(bound, ref.shape)[~ninf]
    assert np.isfinite(d).all(), f"{what}: non-finite values"
    assert (d <= b).all(), f"{what}: {(d > b).sum()} of {d.size} outside, worst {np.max(d / np.maximum(b, 1e-300)):.3f} of its bound"


def evict_reference(pool, keep, sinks, recent):
    """(kept [B, keep], new ends) by sorting (plain Python)."""
    kept = np.full((len(pool.ends), keep), -1, np.int32)
    for b, e in enumerate(pool.ends):
        n = int(max(e, 0))
        w = pool.weight[pool.rows(b)]
        must = [t for t in range(n) if t < sinks or t >= n - recent]
        rest = [t for t in range(n) if not (t < sinks or t >= n - recent)]
        rest.sort(key=lambda t: (np.isnan(w[t]), -w[t] if not np.isnan(w[t]) else 0.0, t))
        pick = sorted((must + rest)[:keep]) if n > keep else list(range(n))
        kept[b, :len(pick)] = pick
    return kept, np.minimum(np.maximum(pool.ends, 0), keep).astype(np.int32)
