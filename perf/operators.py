"""The paged-cache operators, as cases that can be measured: attention of one new
token per sequence over a paged latent cache (decode), the attention weight each
cached row received, summed over heads and added to a running total (weights),
eviction by that total into fresh pages (evict), and the cache write (append).

Each case runs in a plain form (elementary torch operations in 32 bits) or, with
`own` true, through the framework's entry points, on the same inputs.

A pool of pages holds the rows: kv [pages, page, 512] (bf16, or e4m3 codes with one
fp32 scale per 128 values), pe [pages, page, 64] bf16, weight [pages, page] fp32.
Position t of sequence b is row t % page of page table[b, t // page].
"""
import math

import torch

own = False

DC, DR, BLK = 512, 64, 128
E4M3_MAX = 448.0
# softmax scale of a 128 + 64 wide head with the YaRN correction for a factor of 40
SCALE = 192.0 ** -0.5 * (0.1 * math.log(40.0) + 1.0) ** 2


# ------------------------------------------------------------------- cases

def listed():
    return [
        # the smallest call: one sequence, one layer of a small model, where latency counts
        _case("decode_b1_h16_t256_bf16", "decode", fmt=0, H=16, B=1, lo=256, hi=256, page=16),
        # a decode step of a large model, with its cache write: bf16 cache, medium context
        _case("decode_b8_h128_t4096_bf16_write", "decode", fmt=0, H=128, B=8, lo=4096, hi=4096, page=64, new=1),
        # a serving batch of mixed lengths over an FP8 cache
        _case("decode_b32_h128_t1k-16k_fp8", "decode", fmt=1, H=128, B=32, lo=1024, hi=16384, page=64),
        # the heads of one of two devices (64), long ragged documents, bf16 cache, large pages
        _case("decode_b4_h64_t20k-60k_bf16", "decode", fmt=0, H=64, B=4, lo=20001, hi=60001, page=128),
        # the longest context: few sequences, FP8 cache
        _case("decode_b4_h128_t131072_fp8", "decode", fmt=1, H=128, B=4, lo=131072, hi=131072, page=64),
        # weights after a small step: an odd length in pages of 48 rows
        _case("weights_b2_h16_t1001_bf16", "weights", fmt=0, H=16, B=2, lo=1001, hi=1001, page=48),
        # weights of the large model's step
        _case("weights_b8_h128_t4096_bf16", "weights", fmt=0, H=128, B=8, lo=4096, hi=4096, page=64),
        # weights of the serving batch, power-of-two scales
        _case("weights_b32_h128_t1k-16k_fp8", "weights", fmt=2, H=128, B=32, lo=1024, hi=16384, page=64),
        # one conversation cut to half its rows
        _case("evict_b1_t4096_keep2048_bf16", "evict", fmt=0, B=1, lo=4096, hi=4096, page=64, keep=2048, sinks=4, recent=512),
        # a serving batch cut to a common budget; some sequences are shorter than it
        _case("evict_b32_t1k-16k_keep4096_fp8", "evict", fmt=1, B=32, lo=1024, hi=16384, page=64, keep=4096, sinks=4, recent=1024),
        # the cache write of one step
        _case("append_b32_s1_fp8", "append", fmt=1, B=32, lo=1024, hi=16384, page=64, new=1),
        # the cache write of prompts
        _case("append_b8_s2000_fp8", "append", fmt=1, B=8, lo=2000, hi=6000, page=64, new=2000),
    ]


def _case(name, op, fmt, B, lo, hi, page, H=0, keep=0, sinks=0, recent=0, new=0):
    c = dict(op=op, fmt=fmt, H=H, B=B, lo=lo, hi=hi, page=page, keep=keep, sinks=sinks, recent=recent, new=new)
    return dict(c, name=name) if name else c


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["decode", "decode", "weights", "evict", "append"])
    fmt = rng.choice([0, 1, 2])
    page = 16 * _log_int(rng, 1, 16)
    B = _log_int(rng, 1, 32)
    hi = _log_int(rng, 1, min(100000, 400000 // B))
    lo = rng.choice([hi, 0, hi // 2])
    H = rng.choice([16, 32, 64, 128])
    if op in ("decode", "weights"):
        return _case("", op, fmt, B, lo, hi, page, H=H, new=rng.choice([0, 1]) if op == "decode" else 0)
    if op == "evict":
        hi, lo = max(hi, 32), max(lo, 16)
        keep = rng.randint(hi // 4, hi)
        sinks = rng.choice([0, 1, 4])
        return _case("", op, fmt, B, lo, hi, page, keep=keep, sinks=sinks, recent=rng.randint(0, keep - sinks))
    new = _log_int(rng, 1, min(hi, 4096))
    return _case("", op, fmt, B, max(lo, new), hi, page, new=new)


def _row_bytes(fmt):
    return DC * 2 + DR * 2 if fmt == 0 else DC + DC // BLK * 4 + DR * 2


def work(case):
    """Bytes and operations one pass cannot do without; lengths at their mean."""
    c, rb = case, _row_bytes(case["fmt"])
    rows = c["B"] * (c["lo"] + c["hi"]) / 2
    tbl = 4 * rows / c["page"] + 4 * c["B"]
    q = c["B"] * c["H"] * (DC + DR) * 2
    if c["op"] == "decode":
        new = c["B"] * c["new"] * (DC + DR) * 2
        return {"bytes": rows * rb + tbl + q + c["B"] * c["H"] * (DC * 2 + 4) + new,
                "flops": 2 * rows * c["H"] * (2 * DC + DR)}
    if c["op"] == "weights":
        return {"bytes": rows * (rb + 8) + tbl + q + c["B"] * c["H"] * 4, "flops": 2 * rows * c["H"] * (DC + DR)}
    if c["op"] == "evict":
        span = c["hi"] - c["lo"]
        below = 0.0 if c["keep"] <= c["lo"] else min(1.0, (c["keep"] - c["lo"]) / span) if span else float(c["hi"] <= c["keep"])
        kept = c["B"] * (below * (c["lo"] + min(c["keep"], c["hi"])) / 2 + (1 - below) * c["keep"])
        return {"bytes": rows * 4 + tbl + kept * (2 * (rb + 4) + 4), "flops": rows}
    return {"bytes": c["B"] * c["new"] * ((DC + DR) * 2 + rb + 4) + tbl, "flops": c["B"] * c["new"] * DC * 2}


# ------------------------------------------------------------------ inputs

def _quantize(x, fmt):
    """fp32 [..., 512] -> (codes uint8, scales fp32 [..., 4])."""
    y = x.view(x.shape[:-1] + (DC // BLK, BLK))
    amax = y.abs().amax(-1)
    scale = amax / torch.full_like(amax, E4M3_MAX)
    if fmt == 2:
        m, e = torch.frexp(scale)
        scale = torch.where(amax > 0, torch.ldexp(torch.ones_like(m), torch.where(m == 0.5, e - 1, e)), scale)
    z = y / torch.where(scale > 0, scale, torch.ones_like(scale))[..., None]
    codes = z.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return codes.view(torch.uint8).view(x.shape), scale


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    h = torch.Generator()
    h.manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(torch.bfloat16)

    B, page, fmt = c["B"], c["page"], c["fmt"]
    ends = torch.randint(c["lo"], c["hi"] + 1, (B,), generator=h, dtype=torch.int32)
    if B > 1:
        ends[-1] = c["hi"]
    width = -(-c["hi"] // page) + 2                      # a table has room for the rows to come
    used = (ends.long() + page - 1) // page
    new_width = -(-c["keep"] // page)
    pages = B * (-(-c["hi"] // page) + new_width) + 3    # and the pool some free pages
    perm = torch.randperm(pages, generator=h).to(torch.int32)
    table = torch.full((B, width), -1, dtype=torch.int32)
    at = 0
    for b in range(B):
        n = int(used[b])
        table[b, :n] = perm[at:at + n]
        at += n
    s = {"case": c, "end": ends.cuda(), "table": table.cuda()}
    x = randn(pages, page, DC)
    if fmt == 0:
        s["kv"], s["scale"] = x, None
    else:
        s["kv"], s["scale"] = torch.empty(pages, page, DC, dtype=torch.uint8, device="cuda"), torch.empty(pages, page, DC // BLK, device="cuda")
        step = max(1, (1 << 18) // page)
        for i in range(0, pages, step):
            s["kv"][i:i + step], s["scale"][i:i + step] = _quantize(x[i:i + step].float(), fmt)
    del x
    s["pe"] = randn(pages, page, DR)
    # totals of some hundred earlier steps: a few rows draw much of the weight
    mean = 100.0 * max(c["H"], 16) / max(c["hi"], 1)
    s["weight"] = mean * torch.randn(pages, page, generator=g, device="cuda").mul(1.5).exp()
    if c["H"]:
        s["ql"], s["qp"] = randn(B, c["H"], DC), randn(B, c["H"], DR)
    if c["new"]:
        s["kv_new"], s["pe_new"] = randn(B, c["new"], DC), randn(B, c["new"], DR)
    if c["op"] == "weights":                             # from the step's decode
        s["lse"] = _attend(s)[1]
    if c["op"] == "evict":
        s["new_table"] = perm[at:at + B * new_width].view(B, new_width).cuda()
    return s


# -------------------------------------------------------------- plain form

def _rows(table, page, T):
    """Pool row of positions 0 .. T-1 of every sequence: [B, T] (0 where the table has none)."""
    t = torch.arange(T, device=table.device)
    return (table[:, t // page].long() * page + t % page).clamp(min=0)


def _latent(s, rows):
    """Rows of the pool as fp32 [..., 512]: the value an FP8 row stands for is bf16(fp32(code * scale))."""
    x = s["kv"].view(-1, DC)[rows]
    if s["scale"] is None:
        return x.float()
    sc = s["scale"].view(-1, DC // BLK)[rows]
    y = x.view(torch.float8_e4m3fn).float().view(x.shape[:-1] + (DC // BLK, BLK)) * sc[..., None]
    return y.to(torch.bfloat16).float().view(x.shape)


def _scores(s):
    """Masked scores fp32 [B, H, T] and the latent rows [B, T, 512]."""
    T = s["case"]["hi"]
    rows = _rows(s["table"], s["case"]["page"], T)
    k = _latent(s, rows)
    k.masked_fill_((torch.arange(T, device=rows.device) >= s["end"][:, None])[..., None], 0.0)
    sc = s["ql"].float() @ k.transpose(1, 2)
    sc += s["qp"].float() @ s["pe"].view(-1, DR)[rows].float().transpose(1, 2)
    sc *= SCALE
    sc.masked_fill_((torch.arange(T, device=rows.device) >= s["end"][:, None])[:, None], -math.inf)
    return sc, k, rows


def _attend(s):
    sc, k, _ = _scores(s)
    m = sc.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = torch.exp(sc - m)
    l = p.sum(-1, keepdim=True)
    out = (p @ k) / torch.where(l > 0, l, torch.ones_like(l))
    return out.to(torch.bfloat16), (m + torch.log(l)).squeeze(-1)


def _write(s):
    """Rows end - new .. end - 1 of every sequence from kv_new, pe_new; their weight starts at 0.
    A position before 0 (a sequence shorter than its new rows) is left out."""
    c = s["case"]
    pos = s["end"].long()[:, None] - c["new"] + torch.arange(c["new"], device=s["end"].device)
    ok = pos >= 0
    at = (s["table"].long().gather(1, pos.clamp(min=0) // c["page"]) * c["page"] + pos.clamp(min=0) % c["page"])[ok]
    x = s["kv_new"][ok]
    if s["scale"] is None:
        s["kv"].view(-1, DC)[at] = x
    else:
        codes, scale = _quantize(x.float(), c["fmt"])
        s["kv"].view(-1, DC)[at] = codes
        s["scale"].view(-1, DC // BLK)[at] = scale
    s["pe"].view(-1, DR)[at] = s["pe_new"][ok]
    s["weight"].view(-1)[at] = 0.0


def _add_weights(s):
    sc, _, rows = _scores(s)
    lse = s["lse"][..., None]
    p = torch.exp(sc - torch.where(lse == -math.inf, torch.zeros_like(lse), lse))
    w = torch.where(lse == -math.inf, torch.zeros_like(p), p).sum(1)
    live = torch.arange(rows.shape[1], device=rows.device) < s["end"][:, None]
    s["weight"].view(-1).index_add_(0, torch.where(live, rows, torch.zeros_like(rows)).view(-1), torch.where(live, w, torch.zeros_like(w)).view(-1))


def _evict(s):
    c = s["case"]
    T, keep = c["hi"], c["keep"]
    rows = _rows(s["table"], c["page"], T)
    t = torch.arange(T, device=rows.device)
    end = s["end"].long()[:, None]
    key = s["weight"].view(-1)[rows]
    key = torch.where((t < c["sinks"]) | (t >= end - c["recent"]), torch.full_like(key, math.inf), key)
    key = torch.where(t < end, key, torch.full_like(key, -math.inf))
    pick = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :keep]
    pick = torch.where(pick < end, pick, torch.full_like(pick, T))
    pick = torch.sort(pick, dim=1).values                 # positions in order, the empty places last
    if pick.shape[1] < keep:
        pick = torch.cat([pick, torch.full((pick.shape[0], keep - pick.shape[1]), T, device=pick.device)], 1)
    ok = pick < T
    src = rows.gather(1, pick.clamp(max=T - 1))[ok]
    dst = _rows(s["new_table"], c["page"], keep)[ok]
    for name, width in (("kv", DC), ("scale", DC // BLK), ("pe", DR), ("weight", 1)):
        if s[name] is not None:
            flat = s[name].view(-1, width)
            flat[dst] = flat[src]
    kept = torch.where(ok, pick, torch.full_like(pick, -1)).to(torch.int32)
    return kept, torch.minimum(s["end"], torch.full_like(s["end"], keep))


def _pool(s):
    """The pool as what it stands for (views; nothing is copied)."""
    return [s["kv"] if s["scale"] is None else s["kv"].view(torch.float8_e4m3fn)] + ([] if s["scale"] is None else [s["scale"]]) + [s["pe"], s["weight"]]


# ---------------------------------------------------------- framework form

def _own(s):
    import mla_latent_kv_07_gb300 as mla

    c = s["case"]
    if "cache" not in s:                                  # what a serving program sets up once
        s["cache"] = mla.PagedCache(s["kv"].shape[0], c["page"], c["fmt"], kv=s["kv"], kv_scale=s["scale"], pe=s["pe"], weight=s["weight"])
        if c["op"] == "decode":
            s["ws"] = mla.alloc_paged_workspace(c["B"], c["H"])
    cache = s["cache"]
    if c["op"] == "decode":
        if c["new"]:
            out = mla.paged_decode(cache, s["table"], s["ql"], s["qp"], s["end"], c["hi"], SCALE, kv_new=s["kv_new"][:, 0], pe_new=s["pe_new"][:, 0], workspace=s["ws"])
            return list(out) + _pool(s)
        return list(mla.paged_decode(cache, s["table"], s["ql"], s["qp"], s["end"], c["hi"], SCALE, workspace=s["ws"]))
    if c["op"] == "weights":
        mla.paged_weights(cache, s["table"], s["ql"], s["qp"], s["lse"], s["end"], c["hi"], SCALE)
        return [s["weight"]]
    if c["op"] == "evict":
        kept, end = mla.paged_evict(cache, s["table"], s["end"], c["hi"], c["keep"], s["new_table"], sinks=c["sinks"], recent=c["recent"])
        return [kept, end] + _pool(s)
    mla.paged_append(cache, s["table"], s["kv_new"], s["pe_new"], s["end"])
    return _pool(s)


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "decode":
        if state["case"]["new"]:
            _write(state)
            return list(_attend(state)) + _pool(state)
        return list(_attend(state))
    if op == "weights":
        _add_weights(state)
        return [state["weight"]]
    if op == "evict":
        return list(_evict(state)) + _pool(state)
    _write(state)
    return _pool(state)


# ------------------------------------------------------------------- exact

def _nearest_e4m3(y):
    """Nearest e4m3 value of fp64 y in [-448, 448], ties to the even code."""
    codes = torch.arange(127, device=y.device)
    e, m = codes >> 3, (codes & 7).double()
    vals = torch.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * torch.pow(2.0, e.double() - 7))
    a = y.abs().clamp(max=E4M3_MAX)
    hi = torch.searchsorted(vals, a).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    up = vals[hi] - a < a - vals[lo]
    tie = (vals[hi] - a == a - vals[lo]) & (hi % 2 == 0)
    return torch.where(up | tie, vals[hi], vals[lo]) * torch.where(y < 0, -1.0, 1.0)


def _row64(s, rows):
    """Latent rows in fp64."""
    if s["scale"] is None:
        return s["kv"].reshape(-1, DC)[rows].double()
    code = s["kv"].reshape(-1, DC)[rows].view(torch.float8_e4m3fn).float()
    scale = s["scale"].reshape(-1, DC // BLK)[rows].repeat_interleave(BLK, -1)
    return (code * scale).bfloat16().double()


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    page, ends, table = c["page"], s["end"].tolist(), s["table"]

    def where(b, n):
        p = torch.arange(n, device="cuda")
        return table[b].long()[p // page] * page + p % page

    kv = None
    if c["new"]:                                          # the written rows, from the quantiser's definition
        kv = s["kv"].view(torch.float8_e4m3fn).float() if s["scale"] is not None else s["kv"].clone()
        for b in range(c["B"]):
            first = max(0, c["new"] - ends[b])
            at = where(b, ends[b])[ends[b] - c["new"] + first:] if ends[b] else torch.empty(0, dtype=torch.long, device="cuda")
            x = s["kv_new"][b, first:] if ends[b] else s["kv_new"][b, :0]
            if s["scale"] is None:
                kv.view(-1, DC)[at] = x
                s["kv"].view(-1, DC)[at] = x
            elif at.numel():
                y = x.double().view(-1, DC // BLK, BLK)
                amax = y.abs().amax(-1)
                sc = (amax / E4M3_MAX).float().double()
                if c["fmt"] == 2:
                    up = torch.pow(2.0, torch.ceil(torch.log2(sc)))
                    up = torch.where(up / 2 >= sc, up / 2, torch.where(up < sc, up * 2, up))
                    sc = torch.where(amax > 0, up, sc)
                z = (y / torch.where(sc > 0, sc, torch.ones_like(sc))[..., None]).float().double()
                v = _nearest_e4m3(z).view(-1, DC)
                kv.view(-1, DC)[at] = v.float()
                s["kv"].view(-1, DC)[at] = v.float().to(torch.float8_e4m3fn).view(torch.uint8)
                s["scale"].view(-1, DC // BLK)[at] = sc.float()
            s["pe"].view(-1, DR)[at] = s["pe_new"][b, first:] if ends[b] else s["pe_new"][b, :0]
            s["weight"].view(-1)[at] = 0.0
    pool = [] if kv is None else [kv] + ([] if s["scale"] is None else [s["scale"].double()]) + [s["pe"].double(), s["weight"].double()]
    if c["op"] == "append":
        return pool
    if c["op"] in ("decode", "weights"):
        out = torch.zeros(c["B"], c["H"], DC, dtype=torch.float64, device="cuda")
        lse = torch.full((c["B"], c["H"]), -math.inf, dtype=torch.float64, device="cuda")
        total = s["weight"].double().reshape(-1)
        for b in range(c["B"]):
            if not ends[b]:
                continue
            rows = where(b, ends[b])
            q = torch.cat([s["ql"][b], s["qp"][b]], -1).double()
            k = torch.cat([_row64(s, rows), s["pe"].reshape(-1, DR)[rows].double()], -1)
            sc = (q @ k.T) * SCALE
            if c["op"] == "weights":
                total[rows] += torch.exp(sc - s["lse"][b].double()[:, None]).sum(0)
            else:
                lse[b] = torch.logsumexp(sc, -1)
                out[b] = torch.softmax(sc, -1) @ k[:, :DC]
            del k, sc
        return [total.view(s["weight"].shape)] if c["op"] == "weights" else [out, lse] + pool
    kept = torch.full((c["B"], c["keep"]), -1, dtype=torch.int32, device="cuda")
    for b in range(c["B"]):
        n = ends[b]
        rows = where(b, n)
        w = s["weight"].reshape(-1)[rows].double()
        must = [p for p in range(n) if p < c["sinks"] or p >= n - c["recent"]]
        rest = sorted(set(range(n)) - set(must), key=lambda p, v=w.tolist(): (-v[p], p))
        pick = sorted((must + rest)[:c["keep"]])
        p = torch.tensor(pick, device="cuda", dtype=torch.long)
        kept[b, :len(pick)] = p.int()
        i = torch.arange(len(pick), device="cuda")
        dst = s["new_table"][b].long()[i // page] * page + i % page
        for name, width in (("kv", DC), ("scale", DC // BLK), ("pe", DR), ("weight", 1)):
            if s[name] is not None:
                flat = s[name].view(-1, width)
                flat[dst] = flat[rows[p]]
    end = torch.tensor([min(n, c["keep"]) for n in ends], dtype=torch.int32, device="cuda")
    kv = s["kv"] if s["scale"] is None else s["kv"].view(torch.float8_e4m3fn).float()
    return [kept, end, kv] + ([] if s["scale"] is None else [s["scale"].double()]) + [s["pe"].double(), s["weight"].double()]
