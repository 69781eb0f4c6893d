"""What is measured of the attention layers' prompt side: rotary positions of
packed rows (``rope``), causal attention over whole prompts (``prompts``) and
attention of a chunk of new tokens over the paged 8-bit cache and themselves
(``chunk``).  Each case is one call on one layer.

Rows are packed: request r has rows[r] new rows behind lens[r] tokens that it
has already (none in ``prompts``); its row i is at position lens[r] + i.
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
        # a decode step's new token, alone on the card, a quarter of the head rotated: latency
        dict(name="rope_one_token", op="rope", reqs=1, rows_lo=1, rows_hi=1, len_lo=421, len_hi=421, h_q=16, h_kv=2,
             d=256, rot=64, inter=False, base=1e7, scaling="none", factor=1.0, pick=1),
        # verification of 256 requests at far positions, interleaved pairs, a context stretched by parts
        dict(name="rope_verify256", op="rope", reqs=256, rows_lo=4, rows_hi=4, len_lo=512, len_hi=1000000, h_q=32,
             h_kv=8, d=128, rot=128, inter=True, base=1e6, scaling="parts", factor=8.0, pick=2),
        # eight prompts of a prefill transaction, some behind a shared prefix
        dict(name="rope_prefill", op="rope", reqs=8, rows_lo=512, rows_hi=32768, len_lo=0, len_hi=300, h_q=32, h_kv=8,
             d=128, rot=128, inter=False, base=1e4, scaling="linear", factor=4.0, pick=3),
        # a short chat turn: latency
        dict(name="prompt_short", op="prompts", reqs=1, rows_lo=37, rows_hi=37, h_q=16, h_kv=2, d=256, window=0,
             pick=4),
        # sixteen prompts of a batch, ragged
        dict(name="prompt_batch16", op="prompts", reqs=16, rows_lo=100, rows_hi=4000, h_q=32, h_kv=8, d=128, window=0,
             pick=5),
        # one long document
        dict(name="prompt_long", op="prompts", reqs=1, rows_lo=20011, rows_hi=20011, h_q=16, h_kv=2, d=256, window=0,
             pick=6),
        # a long prompt beside short ones
        dict(name="prompt_mixed8", op="prompts", reqs=8, rows_lo=512, rows_hi=12000, h_q=32, h_kv=4, d=128, window=0,
             pick=7),
        # small heads without groups, a sliding window, odd lengths
        dict(name="prompt_window_mha", op="prompts", reqs=24, rows_lo=1, rows_hi=4097, h_q=12, h_kv=12, d=64,
             window=1000, pick=8),
        # the second turn of a chat: a few new tokens behind a short cache, latency
        dict(name="chunk_turn", op="chunk", reqs=1, rows_lo=40, rows_hi=40, len_lo=422, len_hi=422, h_q=16, h_kv=2,
             d=256, page=64, window=0, pick=9),
        # eight requests' next turns behind ragged contexts
        dict(name="chunk_batch8", op="chunk", reqs=8, rows_lo=60, rows_hi=2048, len_lo=512, len_hi=32768, h_q=32,
             h_kv=8, d=128, page=64, window=0, pick=10),
        # a chunk of a prompt split into chunks, 256K tokens in
        dict(name="chunk_256k", op="chunk", reqs=1, rows_lo=512, rows_hi=512, len_lo=262144, len_hi=262144, h_q=16,
             h_kv=2, d=256, page=64, window=0, pick=11),
        # small pages and heads under a sliding window
        dict(name="chunk_window", op="chunk", reqs=12, rows_lo=17, rows_hi=700, len_lo=1, len_hi=9000, h_q=12, h_kv=4,
             d=64, page=16, window=1000, pick=12),
    ]


def _spread(rng, lo, hi):
    return lo if lo >= hi else min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["rope", "prompts", "prompts", "chunk", "chunk"])
    d = rng.choice([64, 128, 256])
    h_kv = rng.choice([1, 2, 4, 8]) if d > 64 else rng.choice([2, 5, 8, 12])
    group = rng.choice([1, 2, 4, 6, 8]) if d > 64 else rng.choice([1, 3, 4])
    if d == 256 and h_kv * group > 32:
        group = 4
    case = dict(op=op, h_q=h_kv * group, h_kv=h_kv, d=d, pick=rng.randrange(1, 1 << 30))
    if op == "rope":
        reqs = _spread(rng, 1, 256)
        hi = _spread(rng, 1, max(2, 16384 // reqs))
        kind = rng.choice(["none", "linear", "base", "parts"])
        return dict(case, reqs=reqs, rows_lo=1, rows_hi=hi, len_lo=0, len_hi=_spread(rng, 8, 1000000),
                    rot=rng.choice([d, d // 2, d // 4, d // 2 + 6]), inter=rng.random() < 0.5,
                    base=rng.choice([1e4, 5e5, 1e6]), scaling=kind,
                    factor=1.0 if kind == "none" else rng.choice([2.0, 4.0, 8.0, 32.0]))
    pairs = 1.2e12 / (4 * h_kv * group * d)                     # of a query row and a position, over all requests
    if op == "prompts":
        reqs = _spread(rng, 1, 64)
        hi = _spread(rng, 2, max(3, min(20000, int(math.sqrt(2 * pairs / reqs)))))
        return dict(case, reqs=reqs, rows_lo=max(1, hi // 16), rows_hi=hi,
                    window=rng.choice([0, 0, 0, _spread(rng, 8, hi + 8)]))
    reqs = _spread(rng, 1, 32)
    rows = _spread(rng, 17, max(18, min(4096, int(math.sqrt(pairs / reqs)))))
    most = min(262144, int(pairs / (reqs * rows)), (1 << 28) // (reqs * h_kv * d))
    hi = _spread(rng, 30, max(40, most))
    return dict(case, reqs=reqs, rows_lo=max(1, rows // 8), rows_hi=rows, len_lo=max(0, hi // 8 - 4), len_hi=hi,
                page=rng.choice([16, 32, 64, 128]), window=rng.choice([0, 0, 0, _spread(rng, 8, hi + 8)]))


def _shape(case):
    """Lengths and row counts of the case's requests (the case's own, whatever the seed)."""
    rng = random.Random(case["pick"])
    n, lo, hi = case["reqs"], case.get("len_lo", 0), case.get("len_hi", 0)
    lens = [lo if lo >= hi else _spread(rng, max(1, lo), hi) - (lo == 0) for _ in range(n)]
    rows = [_spread(rng, case["rows_lo"], case["rows_hi"]) for _ in range(n)]
    if n > 1 and hi:
        lens[rng.randrange(n)] = hi
    if n > 1 and case["op"] == "prompts":
        rows[rng.randrange(n)] = case["rows_hi"]
    return lens, rows


def _pairs(length, n, w):
    """Pairs of a row and a position that it sees."""
    if not w:
        return n * length + n * (n + 1) // 2
    full = max(0, min(n, w - length))                           # rows that see everything before them
    return full * length + full * (full + 1) // 2 + (n - full) * w


def work(case):
    d, h_q, h_kv = case["d"], case["h_q"], case["h_kv"]
    lens, rows = _shape(case)
    total = sum(rows)
    if case["op"] == "rope":
        return {"bytes": 4.0 * total * (h_q + h_kv) * d, "flops": 3.0 * total * (h_q + h_kv) * case["rot"]}
    w = case["window"]
    size = total * (h_q * d * 4 + h_kv * d * 4 + h_q * 4)
    if case["op"] == "chunk":
        seen = [min(a, max(0, w - 1)) if w else a for a in lens]
        size += sum(seen) * h_kv * 2 * d + sum(-(-a // case["page"]) for a in seen) * (8 * h_kv + 4)
    return {"bytes": float(size), "flops": 4.0 * sum(_pairs(a, n, w) for a, n in zip(lens, rows)) * h_q * d}


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


TRAINED = 8192  # the context that a stretched model was trained on


def _frequencies(case):
    """fp64 [rot / 2] angular frequencies and the factor on cosine and sine."""
    rot, base, factor = case["rot"], case["base"], case["factor"]
    j = np.arange(rot // 2, dtype=np.float64)
    if case["scaling"] == "base":
        base = base * factor ** (rot / (rot - 2.0))
    f = base ** (-2.0 * j / rot)
    if case["scaling"] == "linear":
        f = f / factor
    if case["scaling"] == "parts":
        turns = TRAINED * f / (2 * math.pi)
        keep = np.clip((turns - 1.0) / (32.0 - 1.0), 0.0, 1.0)
        return f * keep + f / factor * (1.0 - keep), 0.1 * math.log(factor) + 1.0
    return f, 1.0


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    d, h_q, h_kv = case["d"], case["h_q"], case["h_kv"]

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev)

    s = dict(case=case, status=torch.zeros(1, dtype=torch.int32, device=dev))
    lens, rows = _shape(case)
    B, R = len(lens), sum(rows)
    cu = [0]
    for n in rows:
        cu.append(cu[-1] + n)
    chan = torch.exp(0.5 * normal(h_kv, 1, d))                   # keys have channels of unequal size
    # the layer's projections come as one row: queries, keys, values
    qkv = torch.empty((R, (h_q + 2 * h_kv) * d), dtype=torch.bfloat16, device=dev)
    for a in range(0, R, 8192):
        b = min(R, a + 8192)
        qkv[a:b, :h_q * d] = normal(b - a, h_q * d).to(torch.bfloat16)
        qkv[a:b, h_q * d:(h_q + h_kv) * d] = (normal(b - a, h_kv, d) * chan[:, 0]).reshape(b - a, -1).to(torch.bfloat16)
        qkv[a:b, (h_q + h_kv) * d:] = normal(b - a, h_kv * d).to(torch.bfloat16)
    s["q"] = qkv[:, :h_q * d].unflatten(1, (h_q, d))
    s["k"] = qkv[:, h_q * d:(h_q + h_kv) * d].unflatten(1, (h_kv, d))
    s["v"] = qkv[:, (h_q + h_kv) * d:].unflatten(1, (h_kv, d))
    s.update(lens=lens, rows=rows, cu=cu, B=B, R=R, max_len=max(lens), max_rows=max(rows), total_len=sum(lens),
             cache_len=torch.tensor(lens, dtype=torch.int32, device=dev),
             cu_rows=torch.tensor(cu, dtype=torch.int32, device=dev))
    if case["op"] == "rope":
        f, s["magnitude"] = _frequencies(case)
        s["freq"] = torch.from_numpy(f).to(dev)
    if case["op"] != "chunk":
        return s
    T, L = case["page"], 2
    need = [-(-(a + n) // T) for a, n in zip(lens, rows)]        # room for the new rows too, as their commit wants
    num_pages = sum(need) + 3
    perm = torch.randperm(num_pages, generator=torch.Generator().manual_seed(seed)).tolist()
    table = torch.full((B, max(need)), -1, dtype=torch.int32)
    at = 0
    for r, n in enumerate(need):
        table[r, :n] = torch.tensor(perm[at:at + n], dtype=torch.int32)
        at += n
    kv = torch.zeros((num_pages, L, 2, h_kv, T, d), dtype=torch.uint8, device=dev)
    scale = torch.full((num_pages, L, h_kv, 2), 0.0, device=dev)
    for a in range(0, num_pages, 4096):                          # only the measured layer's pages are filled
        b = min(num_pages, a + 4096)
        blocks = normal(b - a, 2, h_kv, T, d)
        blocks[:, 0] *= chan
        codes, sc = _quantised(blocks)
        kv[a:b, LAYER] = codes
        scale[a:b, LAYER] = sc.transpose(1, 2)
    s.update(kv=kv, scale=scale, table=table.to(dev), T=T)
    return s


# --- the plain forms --------------------------------------------------------

def _plain_rope(s):
    c = s["case"]
    rot, half = c["rot"], c["rot"] // 2
    at = torch.arange(s["R"], device="cuda")
    r = torch.searchsorted(s["cu_rows"].long(), at, right=True) - 1
    pos = s["cache_len"].long()[r] + at - s["cu_rows"].long()[r]
    angle = pos.double()[:, None] * s["freq"]                    # 32 bits would lose far positions' angles
    cos, sin = (torch.cos(angle) * s["magnitude"]).float()[:, None], (torch.sin(angle) * s["magnitude"]).float()[:, None]

    def turn(x):
        y = x[..., :rot].float()
        a, b = (y[..., 0::2], y[..., 1::2]) if c["inter"] else (y[..., :half], y[..., half:])
        p, q = a * cos - b * sin, a * sin + b * cos
        y = torch.stack([p, q], -1).flatten(-2) if c["inter"] else torch.cat([p, q], -1)
        return torch.cat([y.to(torch.bfloat16), x[..., rot:]], -1)

    return {"q": turn(s["q"]), "k": turn(s["k"])}


def _attention(q, k, v, first, w):
    """Rows q [n, h_q, d] at positions first + i of keys and values k, v [h, keys, d] (fp32), those of a block of rows
    at a time that a few GB hold."""
    n, h_q, d = q.shape
    h, keys = k.shape[:2]
    g = h_q // h
    step = max(1, (1 << 30) // (h_q * keys))
    out = torch.empty_like(q)
    lse = torch.empty((n, h_q), device=q.device, dtype=torch.float32)
    for a in range(0, n, step):
        b = min(n, a + step)
        lo, hi = max(0, first + a + 1 - w) if w else 0, first + b
        t = torch.arange(lo, hi, device=q.device)
        i = first + torch.arange(a, b, device=q.device)
        hide = t[None, :] > i[:, None]
        if w:
            hide = hide | (t[None, :] <= i[:, None] - w)
        x = q[a:b].float().reshape(b - a, h, g, d).permute(1, 0, 2, 3).reshape(h, -1, d)
        z = torch.matmul(x, k[:, lo:hi].transpose(1, 2)).mul_(1.0 / math.sqrt(d)).reshape(h, b - a, g, -1)
        z.masked_fill_(hide[None, :, None, :], -math.inf)
        top = z.amax(-1, keepdim=True)
        p = z.sub_(top).exp_()
        total = p.sum(-1, keepdim=True)
        o = torch.matmul(p.reshape(h, (b - a) * g, -1), v[:, lo:hi]).reshape(h, b - a, g, d) / total
        out[a:b] = o.permute(1, 0, 2, 3).reshape(b - a, h_q, d).to(torch.bfloat16)
        lse[a:b] = (top + torch.log(total))[..., 0].permute(1, 0, 2).reshape(b - a, h_q)
    return out, lse


def _plain_prompts(s):
    o, lse = [], []
    for a, b in zip(s["cu"], s["cu"][1:]):
        x = _attention(s["q"][a:b], s["k"][a:b].float().transpose(0, 1), s["v"][a:b].float().transpose(0, 1), 0,
                       s["case"]["window"])
        o.append(x[0])
        lse.append(x[1])
    return {"o": torch.cat(o), "lse": torch.cat(lse)}


def _plain_chunk(s):
    c = s["case"]
    h_kv, d, T = c["h_kv"], c["d"], s["T"]
    o, lse = [], []
    for r, (a, b) in enumerate(zip(s["cu"], s["cu"][1:])):
        length = s["lens"][r]
        page = s["table"][r, :-(-length // T)].long()
        x = s["kv"][page, LAYER].view(torch.float8_e4m3fn).float() * s["scale"][page, LAYER].transpose(1, 2)[..., None, None]
        x = x.permute(1, 2, 0, 3, 4).reshape(2, h_kv, -1, d)[:, :, :length]
        k, v = (torch.cat([x[i], s[t][a:b].float().transpose(0, 1)], 1) for i, t in ((0, "k"), (1, "v")))
        x = _attention(s["q"][a:b], k, v, length, c["window"])
        o.append(x[0])
        lse.append(x[1])
    return {"o": torch.cat(o), "lse": torch.cat(lse)}


# --- the framework's calls --------------------------------------------------

def _own_rope(s):
    if "rope" not in s:  # the handle that a user's program keeps
        from speculative_decoding_hybrid_gb300.prefill import Rope
        c = s["case"]
        s["rope"] = Rope(c["d"], c["rot"], c["base"], interleaved=c["inter"], scaling=c["scaling"], factor=c["factor"],
                         trained=TRAINED, device="cuda")
    q, k = s["rope"].rotate(s["q"], s["k"], s["cu_rows"], s["cache_len"], s["status"])
    return {"q": q, "k": k}


def _own_prompts(s):
    from speculative_decoding_hybrid_gb300.prefill import attend_prompts
    o, lse = attend_prompts(s["q"], s["k"], s["v"], s["cu_rows"], s["max_rows"], s["status"],
                            window=s["case"]["window"], want_lse=True)
    return {"o": o, "lse": lse}


def _own_chunk(s):
    if "cache" not in s:  # the handle that a user's program keeps
        from speculative_decoding_hybrid_gb300.kvcache import Kv8Cache
        c = s["case"]
        s["cache"] = Kv8Cache(s["kv"], s["scale"], h_q=c["h_q"], window=c["window"], status=s["status"])
    o, lse = s["cache"].attend_chunk(LAYER, s["table"], s["cache_len"], s["cu_rows"], s["q"], s["k"], s["v"],
                                     max_len=s["max_len"], max_rows=s["max_rows"], total_len=s["total_len"],
                                     want_lse=True)
    return {"o": o, "lse": lse}


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


def _exact_rope(case, s, lens, rows):
    rot, factor = case["rot"], case["factor"]
    base = case["base"] * (factor ** (rot / (rot - 2)) if case["scaling"] == "base" else 1.0)
    m, f = 1.0, []
    for j in range(rot // 2):
        x = base ** (-2 * j / rot)
        if case["scaling"] == "linear":
            x /= factor
        elif case["scaling"] == "parts":
            ramp = min(1.0, max(0.0, (TRAINED * x / (2 * math.pi) - 1) / 31))
            x = ramp * x + (1 - ramp) * x / factor
            m = 1 + 0.1 * math.log(factor)
        f.append(x)
    pos = torch.cat([torch.arange(a, a + n, dtype=torch.float64) for a, n in zip(lens, rows)]).cuda()
    w = torch.polar(torch.full((len(pos), rot // 2), m, dtype=torch.float64, device="cuda"),
                    torch.outer(pos, torch.tensor(f, dtype=torch.float64, device="cuda")))
    first = torch.arange(rot // 2, device="cuda") * (2 if case["inter"] else 1)
    second = first + (1 if case["inter"] else rot // 2)
    out = {}
    for name in ("q", "k"):
        y = s[name].double()
        z = torch.complex(y[..., first], y[..., second]) * w[:, None]
        y[..., first], y[..., second] = z.real, z.imag
        out[name] = y
    return out


def exact(case, seed):
    lens, rows = _shape(case)
    if case["op"] != "rope" and work(case)["flops"] > 5e12:
        return None
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rope(case, s, lens, rows)
    d, h_q, h_kv, w = case["d"], case["h_q"], case["h_kv"], case["window"]
    g = h_q // h_kv
    val = torch.from_numpy(_e4m3_values()).cuda()
    outs, lses, a = [], [], 0
    for r, (length, n) in enumerate(zip(lens, rows)):
        q, k, v = (s[t][a:a + n].double() for t in ("q", "k", "v"))
        k, v = k.transpose(0, 1), v.transpose(0, 1)
        if case["op"] == "chunk":
            ids = s["table"][r, :-(-length // case["page"])].long()
            x = val[s["kv"][ids, LAYER].int()] * s["scale"][ids, LAYER].double().transpose(1, 2)[..., None, None]
            x = x.permute(1, 2, 0, 3, 4).reshape(2, h_kv, -1, d)[:, :, :length]
            k, v = torch.cat([x[0], k], 1), torch.cat([x[1], v], 1)
        o, lse = torch.empty_like(q), torch.empty((n, h_q), dtype=torch.float64, device="cuda")
        step = max(1, (1 << 29) // (g * (length + n)))
        for h in range(h_kv):
            for i in range(0, n, step):
                j = min(n, i + step)
                top, low = length + j, max(0, length + i + 1 - w) if w else 0
                z = torch.einsum("igd,td->igt", q[i:j, h * g:(h + 1) * g], k[h, low:top]) / math.sqrt(d)
                t = torch.arange(low, top, device="cuda")
                at = length + torch.arange(i, j, device="cuda")
                see = t[None] <= at[:, None]
                if w:
                    see &= t[None] + w > at[:, None]
                z.masked_fill_(~see[:, None], -math.inf)
                l = torch.logsumexp(z, -1)
                lse[i:j, h * g:(h + 1) * g] = l
                o[i:j, h * g:(h + 1) * g] = torch.einsum("igt,td->igd", torch.exp_(z.sub_(l[..., None])), v[h, low:top])
        outs.append(o)
        lses.append(lse)
        a += n
    return {"o": torch.cat(outs), "lse": torch.cat(lses)}
