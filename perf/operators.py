"""What is measured of the paged 8-bit key/value cache of the attention layers
beside the GatedDeltaNet layers: attention of a transaction's rows over it
(``attend``), the commit that quantises accepted rows into it (``append``) and
the moves of whole pages (``copy``).

Cache: page p of layer l holds e4m3 codes [2 (K, V)][h_kv][page_tokens][d] and
one fp32 power-of-two scale per (kv head, K or V); a request's pages are named
by its row of the page table.  Each case is one call on one layer (``attend``,
``append``) or on every layer (``copy``).
"""
import math
import random

import numpy as np
import torch

own = False

LAYER, E4M3_MAX = 1, 448.0


# --- cases ------------------------------------------------------------------

def listed():
    return [
        # the second token of a short chat turn, alone on the card: latency
        dict(name="attend_one_token", op="attend", reqs=1, rows_lo=1, rows_hi=1, len_lo=37, len_hi=37, h_q=16,
             h_kv=2, d=256, page=64, window=0, pick=1),
        # batch-1 verification, three drafts, a prompt of a few hundred tokens
        dict(name="attend_batch1", op="attend", reqs=1, rows_lo=4, rows_hi=4, len_lo=422, len_hi=422, h_q=16, h_kv=2,
             d=256, page=64, window=0, pick=2),
        # batch-1 verification at 256K tokens of context
        dict(name="attend_batch1_256k", op="attend", reqs=1, rows_lo=4, rows_hi=4, len_lo=262144, len_hi=262144,
             h_q=16, h_kv=2, d=256, page=64, window=0, pick=3),
        # continuous batching, 16 requests with 0 to 3 drafts, ragged contexts
        dict(name="attend_cb16", op="attend", reqs=16, rows_lo=1, rows_hi=4, len_lo=512, len_hi=32768, h_q=32, h_kv=8,
             d=128, page=64, window=0, pick=4),
        # 256 paged requests with three drafts each
        dict(name="attend_paged256", op="attend", reqs=256, rows_lo=4, rows_hi=4, len_lo=512, len_hi=8192, h_q=16,
             h_kv=2, d=256, page=64, window=0, pick=5),
        # plain decode without grouped heads, small heads and pages, a sliding window, odd lengths
        dict(name="attend_window_mha", op="attend", reqs=24, rows_lo=1, rows_hi=1, len_lo=1, len_hi=4097, h_q=12,
             h_kv=12, d=64, page=16, window=1000, pick=6),
        # the most drafts a request may carry: the products weigh as much as the bytes
        dict(name="attend_rows16", op="attend", reqs=32, rows_lo=16, rows_hi=16, len_lo=1000, len_hi=16000, h_q=32,
             h_kv=4, d=128, page=128, window=0, pick=7),
        # the commit of a continuous batch: 1 to 4 accepted rows a request
        dict(name="append_cb16", op="append", reqs=16, rows_lo=1, rows_hi=4, len_lo=512, len_hi=4096, h_q=32, h_kv=8,
             d=128, page=64, accept=True, pick=8),
        # the commit of 256 requests
        dict(name="append_paged256", op="append", reqs=256, rows_lo=4, rows_hi=4, len_lo=1, len_hi=1000, h_q=16,
             h_kv=2, d=256, page=64, accept=True, pick=9),
        # eight prompts of 512 to 32,768 tokens written by their prefill, some behind a shared prefix
        dict(name="append_prefill", op="append", reqs=8, rows_lo=512, rows_hi=32768, len_lo=0, len_hi=300, h_q=32,
             h_kv=8, d=128, page=64, accept=False, pick=10),
        # sixteen requests forked from one prefix: their unfinished last pages, all layers
        dict(name="copy_fork16", op="copy", pages=16, pool=256, layers=10, h_q=16, h_kv=2, d=256, page=64, shared=True,
             pick=11),
        # a fragmented pool packed to its low end
        dict(name="copy_compact", op="copy", pages=1500, pool=4000, layers=10, h_q=32, h_kv=8, d=128, page=32,
             shared=False, pick=12),
    ]


def _spread(rng, lo, hi):
    return lo if lo >= hi else min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "append", "copy"])
    d = rng.choice([64, 128, 256])
    h_kv = rng.choice([1, 2, 4, 8]) if d > 64 else rng.choice([2, 5, 8, 12])
    group = rng.choice([1, 2, 4, 6, 8]) if d > 64 else rng.choice([1, 3, 4])
    case = dict(op=op, h_q=h_kv * group, h_kv=h_kv, d=d, page=rng.choice([16, 32, 64, 128]),
                pick=rng.randrange(1, 1 << 30))
    if op == "copy":
        page_bytes = 2 * h_kv * case["page"] * d
        layers = rng.randrange(1, 13)
        most = max(2, min(2000, (1 << 29) // (page_bytes * layers)))
        n = _spread(rng, 1, most)
        return dict(case, pages=n, pool=2 * n + rng.randrange(2, 40), layers=layers, shared=rng.random() < 0.5)
    reqs = _spread(rng, 1, 256)
    if op == "append":
        prompt = rng.random() < 0.4
        hi = _spread(rng, 17, max(18, (1 << 15) // reqs)) if prompt else rng.randrange(1, 17)
        return dict(case, reqs=reqs, rows_lo=1, rows_hi=hi, len_lo=0, len_hi=_spread(rng, 1, 1000),
                    accept=not prompt)
    most = max(40, min(262144, (1 << 29) // (reqs * h_kv * 2 * d)))
    hi = _spread(rng, 30, most)
    rows = rng.choice([1, 1, 2, 4, 4, 5, 8, 16]) if reqs <= 64 else rng.choice([1, 2, 4])
    return dict(case, reqs=reqs, rows_lo=rng.choice([1, rows]), rows_hi=rows, len_lo=max(0, hi // 8 - 4), len_hi=hi,
                window=rng.choice([0, 0, 0, _spread(rng, 8, hi + 8)]))


def _shape(case):
    """Lengths and row counts of the case's requests (the case's own, whatever the seed)."""
    rng = random.Random(case["pick"])
    n = case["reqs"]
    lens = [case["len_lo"] if case["len_lo"] >= case["len_hi"]
            else _spread(rng, max(1, case["len_lo"]), case["len_hi"]) - (case["len_lo"] == 0) for _ in range(n)]
    rows = [_spread(rng, case["rows_lo"], case["rows_hi"]) for _ in range(n)]
    if n > 1:
        lens[rng.randrange(n)] = case["len_hi"]
    return lens, rows


def _copy_pairs(case):
    rng = random.Random(case["pick"])
    ids = list(range(case["pool"]))
    rng.shuffle(ids)
    n = case["pages"]
    if case["shared"]:
        return [ids[0]] * n, ids[1:n + 1]
    live = sorted(ids[:n])
    return live, sorted(ids[n:2 * n])


def work(case):
    d, h_q, h_kv, page = case["d"], case["h_q"], case["h_kv"], case["page"]
    if case["op"] == "copy":
        one = case["layers"] * (2 * h_kv * page * d + 8 * h_kv)
        src, dst = _copy_pairs(case)
        return {"bytes": float((len(set(src)) + len(dst)) * one), "flops": 0.0}
    lens, rows = _shape(case)
    total = sum(rows)
    if case["op"] == "append":
        touched = sum((a + n - 1) // page - a // page + 1 for a, n in zip(lens, rows))
        old = sum(a % page for a in lens)
        return {"bytes": float(total * h_kv * d * 2 * 3 + old * h_kv * d * 2 + touched * h_kv * 8),
                "flops": float(total * h_kv * d * 2 * 3)}
    w = case["window"]
    seen = [min(a, w + n) if w else a for a, n in zip(lens, rows)]
    pairs = sum(n * (min(a, w) if w else a) + n * (n + 1) // 2 for a, n in zip(lens, rows))
    cache = sum(seen) * h_kv * 2 * d + sum(-(-a // page) for a in seen) * (8 * h_kv + 4)
    return {"bytes": float(cache + total * (h_q * d * 4 + h_kv * d * 4 + h_q * 4)), "flops": 4.0 * pairs * h_q * d}


# --- inputs -----------------------------------------------------------------

def _power(e):
    """2.0 ** e exactly, for fp32's normal exponents."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _quantised(x):
    """e4m3 codes and power-of-two scales of blocks [..., T, d] (how the cache came to hold what it holds)."""
    amax = x.abs().amax(dim=(-2, -1))
    m, e = torch.frexp(amax)
    s = _power((e - 9 + (m > 0.875).int()).clamp(min=-100))
    return (x / s[..., None, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8), s


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    d, h_q, h_kv, T = case["d"], case["h_q"], case["h_kv"], case["page"]

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev)

    s = dict(case=case, T=T, status=torch.zeros(1, dtype=torch.int32, device=dev))
    if case["op"] == "copy":
        n, L = case["pool"], case["layers"]
        codes = torch.randint(0, 254, (n, L, 2, h_kv, T, d), generator=g, device=dev, dtype=torch.uint8)
        codes += (codes >= 127).to(torch.uint8)                          # every code but the two NaNs
        s["kv"] = codes
        s["scale"] = torch.exp2(torch.randint(-9, -4, (n, L, h_kv, 2), generator=g, device=dev).float())
        src, dst = _copy_pairs(case)
        s["src"] = torch.tensor(src, dtype=torch.int32, device=dev)
        s["dst"] = torch.tensor(dst, dtype=torch.int32, device=dev)
        s["src64"], s["dst64"] = s["src"].long(), s["dst"].long()
        return s

    lens, rows = _shape(case)
    B, R = len(lens), sum(rows)
    room = [a + (n if case["op"] == "append" else 0) for a, n in zip(lens, rows)]
    need = [-(-a // T) for a in room]
    P, num_pages, L = max(1, max(need)), sum(need) + 3, 2
    perm = torch.randperm(num_pages, generator=torch.Generator().manual_seed(seed)).tolist()
    table = torch.full((B, P), -1, dtype=torch.int32)
    at = 0
    for r, n in enumerate(need):
        table[r, :n] = torch.tensor(perm[at:at + n], dtype=torch.int32)
        at += n
    # keys with channels of unequal size, values of unit size; only the measured layer's pages are filled
    chan = torch.exp(0.5 * normal(h_kv, 1, d))
    kv = torch.zeros((num_pages, L, 2, h_kv, T, d), dtype=torch.uint8, device=dev)
    scale = torch.full((num_pages, L, h_kv, 2), 0.0, device=dev)
    for a in range(0, num_pages, 4096):
        b = min(num_pages, a + 4096)
        blocks = normal(b - a, 2, h_kv, T, d)
        blocks[:, 0] *= chan
        codes, sc = _quantised(blocks)
        kv[a:b, LAYER] = codes
        scale[a:b, LAYER] = sc.transpose(1, 2)
    cu = [0]
    for n in rows:
        cu.append(cu[-1] + n)
    s.update(kv=kv, scale=scale, table=table.to(dev), B=B, R=R, max_len=max(lens), max_rows=max(rows),
             cache_len=torch.tensor(lens, dtype=torch.int32, device=dev),
             cu_rows=torch.tensor(cu, dtype=torch.int32, device=dev))
    # the layer's projections come as one row: queries, keys, values
    qkv = torch.empty((R, (h_q + 2 * h_kv) * d), dtype=torch.bfloat16, device=dev)
    qkv[:, :h_q * d] = (normal(R, h_q * d) * 1.5).to(torch.bfloat16)
    qkv[:, h_q * d:(h_q + h_kv) * d] = (normal(R, h_kv, d) * chan[:, 0]).reshape(R, -1).to(torch.bfloat16)
    qkv[:, (h_q + h_kv) * d:] = normal(R, h_kv * d).to(torch.bfloat16)
    s["q"] = qkv[:, :h_q * d].unflatten(1, (h_q, d))
    s["k"] = qkv[:, h_q * d:(h_q + h_kv) * d].unflatten(1, (h_kv, d))
    s["v"] = qkv[:, (h_q + h_kv) * d:].unflatten(1, (h_kv, d))
    # the host's own tables, from which the plain forms index
    row_req = torch.repeat_interleave(torch.arange(B), torch.tensor(rows))
    s["row_req"] = row_req.to(dev)
    s["row_at"] = (torch.arange(R) - torch.tensor(cu)[row_req]).to(dev)
    if case["op"] == "append":
        keep = [int(x) for x in np.random.RandomState(seed % (1 << 31)).randint(0, 1 << 30, B)]
        s["accept_len"] = (torch.tensor([k % n for k, n in zip(keep, rows)], dtype=torch.int32, device=dev)
                           if case["accept"] else None)
        req, page = [], []
        for r, (a, n) in enumerate(zip(lens, rows)):
            for j in range(a // T, (a + n - 1) // T + 1):
                req.append(r)
                page.append(j)
        s["page_req"] = torch.tensor(req, device=dev)
        s["page_at"] = torch.tensor(page, device=dev)
        s["page_id"] = s["table"].long()[s["page_req"], s["page_at"]]
    else:
        pad = torch.full((B, max(rows)), 0)
        for r in range(B):
            pad[r, :rows[r]] = torch.arange(cu[r], cu[r + 1])
        s["pad_row"] = pad.to(dev)
        s["n_rows"] = torch.tensor(rows, device=dev)
    return s


# --- the plain forms --------------------------------------------------------

def _plain_attend(s):
    c = s["case"]
    d, h_q, h_kv, T, w = c["d"], c["h_q"], c["h_kv"], s["T"], c["window"]
    B, n, g = s["B"], s["max_rows"], c["h_q"] // c["h_kv"]
    dev = s["q"].device
    page = s["table"].long().clamp(min=0)                                        # [B, P]
    x = s["kv"][page, LAYER].view(torch.float8_e4m3fn).float()                   # [B, P, 2, h, T, d]
    x = x * s["scale"][page, LAYER].transpose(2, 3)[..., None, None]
    x = x.permute(2, 0, 3, 1, 4, 5).reshape(2, B, h_kv, -1, d)                   # [2, B, h, P*T, d]
    rows = s["pad_row"]
    kn, vn = (s[t].float()[rows].permute(0, 2, 1, 3) for t in ("k", "v"))        # [B, h, n, d]
    k, v = torch.cat([x[0], kn], 2), torch.cat([x[1], vn], 2)
    length = s["cache_len"].long()
    slots = x.shape[3]
    t = torch.arange(slots, device=dev)
    i = torch.arange(n, device=dev)
    old = t[None, None, :] < length[:, None, None]                               # [B, 1, P*T]
    new = (i[None, :] <= i[:, None])[None].expand(B, n, n) & (i[None, None, :] < s["n_rows"][:, None, None])
    if w:
        old = old & (t[None, None, :] > (length[:, None] + i[None, :])[:, :, None] - w)
        new = new & (i[None, None, :] > i[None, :, None] - w)
    see = torch.cat([old.expand(B, n, slots), new], 2)                           # [B, n, keys]
    v = torch.where(see.any(1)[:, None, :, None], v, torch.zeros((), device=dev))
    q = s["q"].float()[rows].reshape(B, n, h_kv, g, d).permute(0, 2, 1, 3, 4).reshape(B, h_kv, n * g, d)
    a = torch.matmul(q, k.transpose(2, 3)).reshape(B, h_kv, n, g, -1) * (1.0 / math.sqrt(d))
    a = torch.where(see[:, None, :, None, :], a, torch.full((), -math.inf, device=dev))
    top = a.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    p = torch.exp(a - top)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.reshape(B, h_kv, n * g, -1), v).reshape(B, h_kv, n, g, d)
    o = o / torch.where(total > 0, total, torch.ones_like(total))
    lse = (top + torch.log(total))[..., 0]
    at = (s["row_req"], s["row_at"])
    o = o.permute(0, 2, 1, 3, 4).reshape(B, n, h_q, d)[at].to(torch.bfloat16)
    return {"o": o, "lse": lse.permute(0, 2, 1, 3).reshape(B, n, h_q)[at]}


def _plain_append(s):
    T, kv, scale = s["T"], s["kv"], s["scale"]
    length = s["cache_len"].long()
    cu = s["cu_rows"].long()
    count = cu[1:] - cu[:-1] if s["accept_len"] is None else s["accept_len"].long() + 1
    req, page = s["page_req"], s["page_id"]
    pos = s["page_at"][:, None] * T + torch.arange(T, device=kv.device)          # [N, T]
    first = length[req][:, None]
    is_new = (pos >= first) & (pos < first + count[req][:, None])
    is_old = pos < first
    row = (cu[req][:, None] + pos - first).clamp(0, s["R"] - 1)
    x = torch.stack([s["k"], s["v"]]).float()[:, row].permute(1, 0, 3, 2, 4)     # [N, 2, h, T, d]
    new = is_new[:, None, None, :, None]
    finite = torch.where(new & torch.isfinite(x), x.abs(), torch.zeros((), device=x.device))
    amax = finite.amax(dim=(-2, -1))                                             # [N, 2, h]
    m, e = torch.frexp(amax)
    least = torch.full_like(e, -100)
    fit = _power(torch.where(amax > 0, e - 9 + (m > 0.875).int(), least).clamp(min=-100))
    was = scale[page, LAYER].transpose(1, 2)                                     # [N, 2, h]
    had = torch.where(is_old[:, :1, None], was, torch.zeros_like(was))
    now = torch.maximum(had, fit)
    codes = kv[page, LAYER].view(torch.float8_e4m3fn).float()
    held = (codes * (had / now)[..., None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    put = (x / now[..., None, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
    out = torch.where(new, put, torch.where(is_old[:, None, None, :, None], held, kv[page, LAYER]))
    any_new = is_new.any(1)
    kv[page, LAYER] = torch.where(any_new[:, None, None, None, None], out, kv[page, LAYER])
    scale[page, LAYER] = torch.where(any_new[:, None, None], now, was).transpose(1, 2)
    return {"kv": kv[:, LAYER].view(torch.float8_e4m3fn), "scale": scale}


def _plain_copy(s):
    s["kv"].index_copy_(0, s["dst64"], s["kv"].index_select(0, s["src64"]))
    s["scale"].index_copy_(0, s["dst64"], s["scale"].index_select(0, s["src64"]))
    return {"kv": s["kv"].view(torch.float8_e4m3fn), "scale": s["scale"]}


# --- the framework's calls --------------------------------------------------

def _cache(s):
    """The handle a user's program keeps: the cache's tensors and its head layout."""
    if "cache" not in s:
        from speculative_decoding_hybrid_gb300.kvcache import Kv8Cache
        c = s["case"]
        s["cache"] = Kv8Cache(s["kv"], s["scale"], h_q=c["h_q"], window=c.get("window", 0), status=s["status"])
    return s["cache"]


def _own_attend(s):
    o, lse = _cache(s).attend(LAYER, s["table"], s["cache_len"], s["cu_rows"], s["q"], s["k"], s["v"],
                              max_len=s["max_len"], max_rows=s["max_rows"], want_lse=True)
    return {"o": o, "lse": lse}


def _own_append(s):
    _cache(s).append(LAYER, s["table"], s["cache_len"], s["cu_rows"], s["k"], s["v"], accept_len=s["accept_len"],
                     max_rows=s["max_rows"])
    return {"kv": s["kv"][:, LAYER].view(torch.float8_e4m3fn), "scale": s["scale"]}


def _own_copy(s):
    _cache(s).copy_pages(s["src"], s["dst"])
    return {"kv": s["kv"].view(torch.float8_e4m3fn), "scale": s["scale"]}


def run(state):
    return globals()[("_own_" if own else "_plain_") + state["case"]["op"]](state)


# --- the definition in 64 bits ----------------------------------------------

def _e4m3_values():
    """The value of each of the 256 e4m3 codes: sign, 4 exponent bits (bias 7), 3 mantissa bits; 0x7f is NaN."""
    code = np.arange(256)
    ex, man = (code >> 3) & 15, code & 7
    mag = np.where(ex == 0, man / 8.0 * 2.0 ** -6, (1 + man / 8.0) * 2.0 ** (ex - 7.0))
    mag[(code & 127) == 127] = np.nan
    return np.where(code & 128, -mag, mag)


def _nearest_e4m3(x):
    """The e4m3 value nearest to each fp64 value within +-448, ties to the even code."""
    mag = x.abs()
    _, e = torch.frexp(mag)
    step = _power((e - 1).clamp(min=-6) - 3).double()
    return torch.copysign(torch.round(mag / step) * step, x)


def exact(case, seed):
    if case["op"] == "copy":
        return None
    s = prepare(case, seed)
    val = torch.from_numpy(_e4m3_values()).cuda()
    lens, rows = _shape(case)
    d, h_q, h_kv, T = case["d"], case["h_q"], case["h_kv"], case["page"]
    q, k, v = s["q"].double(), s["k"].double(), s["v"].double()
    sc = s["scale"].double()
    if case["op"] == "attend":
        w, g = case["window"], h_q // h_kv
        outs, lses = [], []
        a = 0
        for r, (length, n) in enumerate(zip(lens, rows)):
            ids = s["table"][r, :-(-length // T)].long()
            x = val[s["kv"][ids, LAYER].int()] * sc[ids, LAYER].transpose(1, 2)[..., None, None]
            x = x.permute(1, 2, 0, 3, 4).reshape(2, h_kv, -1, d)[:, :, :length]
            kk = torch.cat([x[0], k[a:a + n].transpose(0, 1)], 1)                # [h, length + n, d]
            vv = torch.cat([x[1], v[a:a + n].transpose(0, 1)], 1)
            z = torch.einsum("ihgd,htd->ihgt", q[a:a + n].reshape(n, h_kv, g, d), kk) / math.sqrt(d)
            t = torch.arange(length + n, device=z.device)
            i = length + torch.arange(n, device=z.device)
            hide = t[None, :] > i[:, None]
            if w:
                hide |= t[None, :] <= i[:, None] - w
            z.masked_fill_(hide[:, None, None, :], -math.inf)
            l = torch.logsumexp(z, -1)
            outs.append(torch.einsum("ihgt,htd->ihgd", torch.exp(z - l[..., None]), vv).reshape(n, h_q, d))
            lses.append(l.reshape(n, h_q))
            a += n
        return {"o": torch.cat(outs), "lse": torch.cat(lses)}
    held = val[s["kv"][:, LAYER].int()]                                          # [pages, 2, h, T, d]
    new_scale = sc.clone()
    acc = s["accept_len"].tolist() if case["accept"] else [n - 1 for n in rows]
    table = s["table"].tolist()
    a = 0
    for r, (length, n) in enumerate(zip(lens, rows)):
        count = acc[r] + 1
        x = torch.stack([k[a:a + count], v[a:a + count]]).transpose(1, 2)        # [2, h, count, d]
        at = 0
        while at < count:
            j, t0 = divmod(length + at, T)
            m = min(T - t0, count - at)
            p = table[r][j]
            part = x[:, :, at:at + m]
            top = part.abs().amax((2, 3))
            half, e = torch.frexp(top / 448.0)                                   # 2 ** e, or 2 ** (e-1) at one half
            e = torch.where(top > 0, e - (half == 0.5).int(), torch.full_like(e, -100))
            fit = _power(e.clamp(min=-100)).double()
            had = sc[p, LAYER].T if t0 else torch.zeros_like(fit)
            now = torch.maximum(had, fit)
            if t0:
                held[p, :, :, :t0] = _nearest_e4m3(held[p, :, :, :t0] * (had / now)[..., None, None])
            held[p, :, :, t0:t0 + m] = _nearest_e4m3((part / now[..., None, None]).clamp(-448, 448))
            new_scale[p, LAYER] = now.T
            at += m
        a += n
    return {"kv": held, "scale": new_scale}
