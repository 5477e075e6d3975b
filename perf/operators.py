"""The cache operators as workloads: keys and values held in 4 bits on pages (written, read back, attended
over by one query per sequence) and the pages of a cache (freed, forked, given out, compacted, copied).

`run` computes each in plain torch (32 bits; the routing in 64), or, where `own` is set, through the package.
The 4-bit format is the package's: groups of 32 consecutive elements of a head share one e4m3 scale,
scale = e4m3(max|x| 2^-exp / 7), code = round(x 2^-exp / scale) + 8 (4 bits, 1..15), a group that holds a NaN or
an infinity has a NaN scale.  Pools are [pages, h_kv, page_size, d / 2] codes and [pages, h_kv, page_size, d / 32]
scales.  A row of codes is d / 8 words of 8 codes, element i of a word in bits 4i..4i+3; values keep the words
in order, keys store word (group G, quarter j) at place j * (d / 32) + G.
"""
import math

import torch

own = False

# exponents of the caches' common scales: keys of unit size with a few large channels, small values
K_EXP, V_EXP = 0, -4
Q_SIZE, V_SIZE = 2.0, 2.0 ** -4
KEY_MS = (31 + 16) / 32   # mean square of a key channel: one channel in 32 is four times larger


# ---- cases ----------------------------------------------------------------------------------------------
def listed():
    return [
        # a short chat of three sequences on small heads: latency of one decoded token
        {"name": "attend_short", "kind": "attend", "batch": 3, "length": 777, "ragged": 150, "h_q": 8, "h_kv": 2, "d": 64,
         "chunk": 32, "page": 64, "alpha": 2.0, "gamma": 2.0},
        # the decode_128k shape: 8 long sequences, about a quarter of the chunks routed
        {"name": "attend_128k_routed", "kind": "attend", "batch": 8, "length": 131072, "ragged": 0, "h_q": 32, "h_kv": 2,
         "d": 128, "chunk": 64, "page": 128, "alpha": 1.5, "gamma": 1.9},
        # dense attention (gamma 0) of a ragged batch of odd lengths
        {"name": "attend_ragged_dense", "kind": "attend", "batch": 12, "length": 50021, "ragged": 1231, "h_q": 32,
         "h_kv": 4, "d": 128, "chunk": 128, "page": 256, "alpha": 1.5, "gamma": 0.0},
        # one token of 8 sequences in the middle of a chunk, as a decode step writes it
        {"name": "store_token", "kind": "store", "batch": 8, "n": 1, "start": 4133, "ragged": 0, "h_kv": 2, "d": 128,
         "chunk": 64, "page": 128},
        # a turn of up to 517 tokens that starts and ends inside chunks, each sequence another number
        {"name": "store_turn", "kind": "store", "batch": 5, "n": 517, "start": 1111, "ragged": 61, "h_kv": 4, "d": 64,
         "chunk": 32, "page": 64},
        # a prompt of 64K tokens of two sequences
        {"name": "store_prompt", "kind": "store", "batch": 2, "n": 65536, "start": 0, "ragged": 0, "h_kv": 2, "d": 128,
         "chunk": 64, "page": 128},
        # 4 beams with two candidates each, short contexts
        {"name": "fork_beams", "kind": "fork", "parents": 4, "children": 8, "length": 1437, "room": 1, "layers": 2,
         "h_kv": 2, "d": 128, "chunk": 64, "page": 128},
        # 32 samples drawn from 8 prompts of 32K tokens
        {"name": "fork_samples", "kind": "fork", "parents": 8, "children": 32, "length": 32768 - 37, "room": 300,
         "layers": 2, "h_kv": 2, "d": 128, "chunk": 64, "page": 128},
        # a small pool after some sequences left
        {"name": "compact_small", "kind": "compact", "pages": 200, "used": 0.4, "batch": 5, "layers": 1, "h_kv": 2,
         "d": 64, "page": 64},
        # half a GB of pages scattered over a GB
        {"name": "compact_large", "kind": "compact", "pages": 8192, "used": 0.5, "batch": 24, "layers": 1, "h_kv": 2,
         "d": 128, "page": 128},
        # a few pages made private
        {"name": "copy_few", "kind": "copy", "pages": 300, "n": 3, "layers": 1, "h_kv": 2, "d": 128, "page": 64},
        # a long context moved aside, all layers at once
        {"name": "copy_many", "kind": "copy", "pages": 2600, "n": 1111, "layers": 4, "h_kv": 2, "d": 128, "page": 128},
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    kind = rng.choice(["attend", "attend", "store", "fork", "compact", "copy"])
    c = {"kind": kind, "h_kv": rng.choice([1, 2, 4, 8]), "d": rng.choice([64, 128]), "page": rng.choice([64, 128, 256])}
    token = c["h_kv"] * c["d"]
    if kind in ("attend", "store", "fork"):
        c["chunk"] = rng.choice([b for b in (16, 32, 64, 128) if b <= c["page"]])
    if kind == "attend":
        c["batch"] = log(1, 24)
        c["h_q"] = c["h_kv"] * rng.choice([1, 2, 4, 8, 16])
        room = min(131072, 8 * 131072 * 256 // (token * c["batch"]), c["chunk"] * 50000 * c["h_kv"] // c["h_q"])
        c["length"] = log(1, max(1, room))
        c["ragged"] = rng.randrange(0, max(1, c["length"] // c["batch"]))
        c["alpha"] = rng.choice([1.5, 2.0])
        c["gamma"] = rng.choice([0.0, round(math.exp(rng.uniform(math.log(0.5), math.log(6.0))), 3)])
    elif kind == "store":
        c["batch"] = log(1, 16)
        c["n"] = log(1, min(65536, 2 * 65536 * 256 // (token * c["batch"])))
        c["start"] = rng.choice([0, log(1, 5000)])
        c["ragged"] = rng.randrange(0, max(1, c["n"] // c["batch"]))
    elif kind == "fork":
        c["parents"], c["children"], c["layers"] = log(1, 8), log(1, 32), rng.choice([1, 2, 3])
        c["length"], c["room"] = log(1, 32768), log(1, 300)
        c["length"] = min(c["length"], 2 * 8 * 32768 * 256 // (token * c["parents"] * c["layers"]))
    else:
        c["layers"] = rng.choice([1, 2, 4])
        most = (1 << 30) // (4 * token * c["page"] * c["layers"])
        c["pages"] = log(8, min(8192, most))
        if kind == "compact":
            c["used"] = round(rng.uniform(0.05, 0.98), 2)
            c["batch"] = log(1, 24)
        else:
            c["n"] = log(1, c["pages"] // 2)
    return c


# ---- what a case takes at least -------------------------------------------------------------------------
def _lengths(c):
    return [max(1, c["length"] - i * c["ragged"]) for i in range(c["batch"])]


def _routed_share(c, chunks):
    """The expected share of `chunks` that some head of a group routes: the logits are normal with a known deviation."""
    if c["gamma"] == 0 or chunks == 0:
        return 1.0
    p = 1 / (c["alpha"] - 1)
    dev = (c["alpha"] - 1) * c["gamma"] * Q_SIZE * math.sqrt(KEY_MS / c["chunk"])
    grid = [-8 + 16 * (i + 0.5) / 2000 for i in range(2000)]
    mass = [math.exp(-z * z / 2) / math.sqrt(2 * math.pi) * 16 / 2000 for z in grid]
    lo, hi = -8 * dev - 1, 8 * dev
    for _ in range(60):
        tau = (lo + hi) / 2
        total = chunks * sum(m * (dev * z - tau) ** p for z, m in zip(grid, mass) if dev * z > tau)
        lo, hi = (tau, hi) if total > 1 else (lo, tau)
    share = sum(m for z, m in zip(grid, mass) if dev * z > lo)
    return 1 - (1 - min(1.0, share)) ** (c["h_q"] // c["h_kv"])


def work(case):
    c, bytes_, flops = case, 0.0, 0.0
    if c["kind"] == "attend":
        g, token = c["h_q"] // c["h_kv"], 2 * (c["d"] // 2 + c["d"] // 32)
        for n in _lengths(c):
            chunks = (n - 1) // c["chunk"]
            keys = _routed_share(c, chunks) * chunks * c["chunk"] + n - chunks * c["chunk"]
            bytes_ += c["h_kv"] * keys * token + 4 * c["h_q"] * c["d"]
            flops += 4 * c["h_q"] * keys * c["d"]
            if c["gamma"] > 0:
                bytes_ += c["h_kv"] * chunks * c["d"] * 4
                flops += 2 * c["h_q"] * chunks * c["d"]
    elif c["kind"] == "store":
        tokens = sum(_counts(c)) * c["h_kv"]
        # written from and read back to bf16, the 4-bit form written and read once; two sums over each key
        bytes_ = tokens * 2 * (4 * c["d"] + 2 * (c["d"] // 2 + c["d"] // 32)) + tokens / c["chunk"] * c["d"] * 4
        flops = tokens * 4 * c["d"]
    else:
        page = 2 * 2 * c["h_kv"] * c["d"] * c["page"] * c["layers"]
        if c["kind"] == "copy":
            bytes_ = 2 * page * c["n"]
        elif c["kind"] == "compact":
            used = max(1, round(c["pages"] * c["used"]))
            slots = -(-used // c["batch"])
            used -= slots // 2 if c["batch"] > 1 else 0   # the shared prefix
            bytes_ = 2 * page * used * (1 - used / c["pages"]) + 12 * c["pages"]
        else:
            n, kids = c["length"], c["children"]
            slots = -(-n // c["page"])
            bytes_ = kids * slots * 16
            if n % c["page"]:
                bytes_ += 2 * kids * page
            bytes_ += 2 * kids * c["layers"] * c["h_kv"] * 4 * ((n // c["chunk"]) * c["d"] + c["d"] + 2)
    return {"bytes": bytes_, "flops": flops}


# ---- the 4-bit form in torch ----------------------------------------------------------------------------
def _quantise(x, exp):
    """Codes (0..15) [..., d] and scales (e4m3) [..., d / 32] of x [..., d]."""
    x = x.float() * 2.0 ** -exp
    g = x.unflatten(-1, (-1, 32))
    top = g.abs().amax(-1)
    scale = (top / torch.full_like(top, 7)).clamp(max=448)   # a true division: torch multiplies by 1 / 7 for a number
    scale = torch.where(torch.isfinite(top), scale, torch.full_like(scale, math.nan)).to(torch.float8_e4m3fn)
    s = scale.float()[..., None]
    q = torch.where(s > 0, torch.round(g / s).clamp(-7, 7), torch.zeros_like(g))
    return (q.flatten(-2) + 8).to(torch.uint8), scale


def _words(rows, back=False):
    """Rows of codes [..., d / 2] from word order to the keys' order (or back)."""
    groups = rows.shape[-1] // 16
    a, b = (4, groups) if back else (groups, 4)
    return rows.unflatten(-1, (a, b, 4)).transpose(-3, -2).flatten(-3)


def _pack(codes):
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def _values(rows, scales, exp):
    """fp32 values of rows of codes in word order."""
    q = torch.stack([rows & 15, rows >> 4], -1).flatten(-2).float() - 8
    s = scales.view(torch.float8_e4m3fn).float() * 2.0 ** exp
    return (q.unflatten(-1, (-1, 32)) * s[..., None]).flatten(-2)


def _cached(pool, s):
    """(keys, values) of every page slot of the tables: [batch, h_kv, slots * page, d] in fp32."""
    table = s["page_table"].long()

    def rows(t):   # [batch, slots, h_kv, page, e] -> [batch, h_kv, slots * page, e]
        return t[table].permute(0, 2, 1, 3, 4).flatten(2, 3)

    k = _values(_words(rows(pool["k_codes"]), back=True), rows(pool["k_scales"]), K_EXP)
    v = _values(rows(pool["v_codes"]), rows(pool["v_scales"]), V_EXP)
    return k, v


# ---- inputs ---------------------------------------------------------------------------------------------
def _rng(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(*shape, device="cuda", generator=g)


def _keys(g, n, h, d):
    size = torch.ones(d, device="cuda")
    size[5::32] = 4.0
    return (_randn(g, n, h, d) * size).bfloat16()


def _new_values(g, n, h, d):
    return (_randn(g, n, h, d) * V_SIZE).bfloat16()


def _summary(k, qbar):
    """Stage 0 of chunks k [chunks, B, h, d]: softmax-weighted mean of the keys, [h, chunks, d]."""
    k = k.float()
    a = torch.softmax((k * qbar).sum(-1) / math.sqrt(k.shape[-1]), 1)
    return (a[..., None] * k).sum(1).transpose(0, 1)


def _table(g, rows, slots, pages):
    return torch.randperm(pages, device="cuda", generator=g)[: rows * slots].view(rows, slots).int()


def _pools(pages, h, page, d):
    def e(n):
        return torch.zeros(pages, h, page, n, dtype=torch.uint8, device="cuda")

    return {"k_codes": e(d // 2), "k_scales": e(d // 32), "v_codes": e(d // 2), "v_scales": e(d // 32)}


def _fill(pool, table, page, k, v):
    """Writes one sequence's keys and values [n, h, d] into its pages (its table row), from position 0."""
    n = k.shape[0]
    slots = -(-n // page)
    for t, exp, name in ((k, K_EXP, "k"), (v, V_EXP, "v")):
        t = torch.nn.functional.pad(t, (0, 0, 0, 0, 0, slots * page - n))
        codes, scales = _quantise(t, exp)
        rows = _pack(codes)
        rows = _words(rows) if name == "k" else rows
        at = table[:slots].long()
        pool[name + "_codes"][at] = rows.unflatten(0, (slots, page)).transpose(1, 2)
        pool[name + "_scales"][at] = scales.view(torch.uint8).unflatten(0, (slots, page)).transpose(1, 2)


def _counts(c):
    return [max(1, c["n"] - i * c["ragged"]) for i in range(c["batch"])]


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    c, g = case, _rng(seed)
    h, d, page = c["h_kv"], c["d"], c["page"]
    s = {"case": dict(c)}
    if c["kind"] in ("attend", "store"):
        B, b = c["chunk"], c["batch"]
        if c["kind"] == "attend":
            held, most = _lengths(c), c["length"]
        else:
            held, most = [c["start"] + 3 * i if c["start"] else 0 for i in range(b)], c["start"] + 3 * b + c["n"]
        slots = -(-most // page)
        s["capacity"] = slots * page
        s["page_table"] = _table(g, b, slots, b * slots + 5)
        s["pool"] = _pools(b * slots + 5, h, page, d)
        s["qbar"] = _randn(g, h, d) * 0.1
        T = s["capacity"] // B
        s["kbar"] = torch.zeros(b, h, T, d, device="cuda")
        s["state"] = torch.zeros(b, h, d + 2, device="cuda")
        s["state"][..., d] = -math.inf
        s["seqlens"] = _ints(held)
        for i, n in enumerate(held):
            if n == 0:
                continue
            k, v = _keys(g, n, h, d), _new_values(g, n, h, d)
            _fill(s["pool"], s["page_table"][i], page, k, v)
            full = n // B
            s["kbar"][i, :, :full] = _summary(k[: full * B].unflatten(0, (full, B)), s["qbar"])
            if n % B:
                rest = k[full * B:].float()
                a = (rest * s["qbar"]).sum(-1) / math.sqrt(d) * math.log2(math.e)
                m = a.amax(0)
                w = torch.exp2(a - m)
                s["state"][i] = torch.cat([(w[..., None] * rest).sum(0), m[:, None], w.sum(0)[:, None]], 1)
        if c["kind"] == "attend":
            s["q"] = (_randn(g, b, c["h_q"], d) * Q_SIZE).bfloat16()
            alpha, gamma, h_q = c["alpha"], c["gamma"], c["h_q"]
        else:
            s["k_new"] = _keys(g, b * c["n"], h, d).unflatten(0, (b, c["n"]))
            s["v_new"] = _new_values(g, b * c["n"], h, d).unflatten(0, (b, c["n"]))
            s["counts"] = _ints(_counts(c))
            s["start"], s["state0"] = s["seqlens"].clone(), s["state"].clone()
            alpha, gamma, h_q = 1.5, 1.0, h
        if own:
            import adaptive_sparse_hierarchical_b200 as D
            st = D.Q4DecodeState(b, s["capacity"], h_q, h, d, chunk=B, alpha=alpha, gamma=gamma, page_size=page,
                                 num_pages=b * slots + 5, page_table=s["page_table"], k_exp=K_EXP, v_exp=V_EXP,
                                 qbar=s["qbar"])
            for name, t in s.pop("pool").items():
                getattr(st, name).copy_(t)
            for name in ("kbar", "state", "seqlens"):
                getattr(st, name).copy_(s[name])
            s["cache"] = st
        return s
    # pages of bf16 caches, one pair of pools for each layer
    if c["kind"] == "fork":
        rows, slots = c["parents"] + c["children"], -(-(c["length"] + c["room"]) // page)
        held = -(-c["length"] // page)
        pages = c["parents"] * held + c["children"] * (slots - held + 2) + 3
        s["page_table"] = torch.full((rows, slots), -1, dtype=torch.int32, device="cuda")
        s["page_table"][: c["parents"], :held] = _table(g, c["parents"], held, pages)
        s["seqlens"] = _ints([max(1, c["length"] - 5 * i) for i in range(c["parents"])] + [0] * c["children"])
        over = torch.arange(slots, device="cuda") >= -(-s["seqlens"] // page)[:, None]
        s["page_table"][over] = -1
        s["src"] = torch.randint(0, c["parents"], (c["children"],), device="cuda", generator=g).int()
        s["dst"] = (c["parents"] + torch.randperm(c["children"], device="cuda", generator=g)).int()
        s["add"] = _ints([0] * c["parents"] + [c["room"]] * c["children"])
        T = slots * page // c["chunk"]
        s["kbar"], s["state"] = [], []
        done = torch.arange(T, device="cuda") < (s["seqlens"] // c["chunk"])[:, None]
        for _ in range(c["layers"]):
            s["kbar"].append(_randn(g, rows, h, T, d) * done[:, None, :, None])
            s["state"].append(_randn(g, rows, h, d + 2) * (s["seqlens"] > 0)[:, None, None])
    else:
        pages = c["pages"]
        if c["kind"] == "copy":
            at = torch.randperm(pages, device="cuda", generator=g)
            s["dst"], rest = at[: c["n"]].int(), at[c["n"]:].int()
            s["src"] = rest[torch.randint(0, rest.numel(), (c["n"],), device="cuda", generator=g)].contiguous()
            s["page_table"] = torch.full((1, 1), -1, dtype=torch.int32, device="cuda")
        else:
            used = max(1, round(pages * c["used"]))
            slots = -(-used // c["batch"])
            s["page_table"] = torch.full((c["batch"] * slots,), -1, dtype=torch.int32, device="cuda")
            s["page_table"][:used] = torch.randperm(pages, device="cuda", generator=g)[:used].int()
            s["page_table"] = s["page_table"].view(c["batch"], slots)
            if slots > 1 and c["batch"] > 1:   # a shared prefix of the first two sequences
                s["page_table"][1, : slots // 2] = s["page_table"][0, : slots // 2]
        s["seqlens"] = ((s["page_table"] >= 0).sum(1) * page).int()
    s["refs"] = torch.zeros(pages, dtype=torch.int32, device="cuda")
    held = s["page_table"][s["page_table"] >= 0].long()
    s["refs"].scatter_add_(0, held, torch.ones_like(held, dtype=torch.int32))
    s["K"] = [torch.randn(pages, page, h, d, device="cuda", dtype=torch.bfloat16, generator=g) for _ in range(c["layers"])]
    s["V"] = [torch.randn(pages, page, h, d, device="cuda", dtype=torch.bfloat16, generator=g) for _ in range(c["layers"])]
    s["refs0"], s["page_table0"] = s["refs"].clone(), s["page_table"].clone()
    if own:
        import adaptive_sparse_hierarchical_b200 as D
        s["pages"] = D.PagePool(s["page_table"], s["refs"], s["seqlens"], page_size=page)
        for t in s["K"] + s["V"]:
            s["pages"].add_pages(t)
        if c["kind"] == "fork":
            for t in s["kbar"]:
                s["pages"].add_rows(t, unit_tokens=c["chunk"])
            for t in s["state"]:
                s["pages"].add_rows(t)
    return s


# ---- the plain forms ------------------------------------------------------------------------------------
def _thresholds(x, alpha, seen):
    """Entmax thresholds of rows x [..., T] (alpha 2 or 1.5; entries that are not `seen` do not count): the support is
    the longest prefix of the sorted row that its own threshold leaves above it."""
    x = torch.where(seen, x, -torch.inf).sort(-1, descending=True).values
    k = torch.arange(1, x.shape[-1] + 1, device=x.device, dtype=x.dtype)
    there = torch.isfinite(x)
    y = torch.where(there, x, 0)
    if alpha == 2.0:
        tau = (y.cumsum(-1) - 1) / k
    else:
        mean, square = y.cumsum(-1) / k, (y * y).cumsum(-1) / k
        tau = mean - ((1 - k * (square - mean * mean)) / k).clamp(min=0).sqrt()
    size = (there & (tau < x)).sum(-1, keepdim=True)
    return tau.gather(-1, (size - 1).clamp(min=0))


def _attend(s):
    c = s["case"]
    h, g, B, d = c["h_kv"], c["h_q"] // c["h_kv"], c["chunk"], c["d"]
    q, last = s["q"].view(-1, h, g, d), s["seqlens"].long() - 1
    k, v = _cached(s["pool"], s)
    at = torch.arange(k.shape[2], device=k.device)
    own_chunk = last // B
    # routing: bias of each complete chunk before the query's own, -inf where it is not routed
    T = s["kbar"].shape[2]
    before = (torch.arange(T, device=k.device) < own_chunk[:, None])[:, None, None]
    if c["gamma"] == 0:
        bias = torch.where(before[:, :, 0], 0.0, -torch.inf).expand(-1, h, T).float()
    else:
        x = torch.matmul(q.double(), s["kbar"].double().transpose(-1, -2)) * ((c["alpha"] - 1) * c["gamma"] / math.sqrt(d))
        tau = _thresholds(x, c["alpha"], before)
        w = torch.where(before, (x - tau).clamp(min=0) ** (1 / (c["alpha"] - 1)), 0).mean(2)
        on = w > 0
        lw = torch.where(on, w, 1).log()
        mu = lw.sum(-1, keepdim=True) / on.sum(-1, keepdim=True).clamp(min=1)
        bias = torch.where(on, lw - mu, -torch.inf).float()
    bias = torch.nn.functional.pad(bias.repeat_interleave(B, -1), (0, at.numel() - T * B), value=-torch.inf)
    near = (at >= (own_chunk * B)[:, None]) & (at <= last[:, None])
    bias = torch.where(near[:, None], 0.0, bias)
    z = torch.matmul(q.float(), k.transpose(-1, -2)) / math.sqrt(d) + bias[:, :, None]
    p = torch.exp(z - z.amax(-1, keepdim=True))
    return {"O": (torch.matmul(p, v) / p.sum(-1, keepdim=True)).flatten(1, 2).bfloat16()}


def _store(s):
    """Appends the first counts[b] new tokens and reads them back."""
    c = s["case"]
    B, d, page, n = c["chunk"], c["d"], c["page"], c["n"]
    pool, b, h = s["pool"], c["batch"], c["h_kv"]
    s["seqlens"].copy_(s["start"])
    s["state"].copy_(s["state0"])
    new = torch.arange(n, device="cuda") < s["counts"][:, None]
    at = s["start"][:, None] + torch.arange(n, device="cuda")
    pg, row = s["page_table"].long().gather(1, (at // page).clamp(max=s["page_table"].shape[1] - 1)), at % page
    back = []
    for t, exp, name in ((s["k_new"], K_EXP, "k"), (s["v_new"], V_EXP, "v")):
        codes, scales = _quantise(t, exp)
        rows = _words(_pack(codes)) if name == "k" else _pack(codes)
        pool[name + "_codes"][pg[new], :, row[new]] = rows[new]
        pool[name + "_scales"][pg[new], :, row[new]] = scales.view(torch.uint8)[new]
        rows, scales = pool[name + "_codes"][pg, :, row], pool[name + "_scales"][pg, :, row]
        got = _values(_words(rows, back=True) if name == "k" else rows, scales, exp)
        back.append(torch.where(new[..., None, None], got, 0.0).bfloat16())
    # summaries: online softmax of the chunk that was open, then whole chunks, then the chunk left open
    first = (s["start"] // B).long()
    chunks = (n + B - 1) // B + 1
    slot = torch.where(new, at // B - first[:, None], chunks)   # chunk of each new token, from the first touched
    a = (s["k_new"].float() * s["qbar"]).sum(-1) * (math.log2(math.e) / math.sqrt(d))
    k = s["k_new"].float()
    m = torch.full((b, chunks + 1, h), -torch.inf, device="cuda")
    m[:, 0] = torch.where((s["start"] % B > 0)[:, None], s["state0"][..., d], -torch.inf)
    m0 = m[:, 0].clone()
    where = slot[..., None].expand(-1, -1, h).long()
    m.scatter_reduce_(1, where, a, "amax")
    ref = torch.where(torch.isfinite(m), m, 0)
    w = torch.exp2(a - ref.gather(1, where))
    keep = torch.exp2(m0 - ref[:, 0])
    l = torch.zeros_like(m)
    acc = torch.zeros(b, chunks + 1, h, d, device="cuda")
    l[:, 0] = keep * s["state0"][..., d + 1]
    acc[:, 0] = keep[..., None] * s["state0"][..., :d]
    l.scatter_add_(1, where, w)
    acc.scatter_add_(1, where[..., None].expand(-1, -1, -1, d), w[..., None] * k)
    end = s["start"] + s["counts"]
    idx = first[:, None] + torch.arange(chunks, device="cuda")
    whole = idx < (end // B)[:, None]
    row_of = torch.arange(b, device="cuda")[:, None].expand_as(idx)
    s["kbar"][row_of[whole], :, idx[whole]] = (acc / l[..., None])[:, :chunks][whole]
    last = (end // B - first).long()
    one = torch.arange(b, device="cuda")
    open_ = (end % B > 0)[:, None, None]
    state = torch.cat([acc[one, last], m[one, last][..., None], l[one, last][..., None]], -1)
    empty = torch.zeros_like(state)
    empty[..., d] = -torch.inf
    s["state"].copy_(torch.where(open_, state, empty))
    s["seqlens"].copy_(end)
    return {"K": back[0], "V": back[1], "kbar": s["kbar"], "state": s["state"], "seqlens": s["seqlens"]}


def _free(s, rows):
    rows = rows.long()
    held = s["page_table"][rows]
    s["refs"].scatter_add_(0, held[held >= 0].long(), torch.full_like(held[held >= 0], -1))
    s["page_table"][rows] = -1
    s["seqlens"][rows] = 0


def _fork(s, src, dst):
    page, src, dst = s["case"]["page"], src.long(), dst.long()
    n = s["seqlens"][src].long()
    whole, part = n // page, n % page > 0
    slot = torch.arange(s["page_table"].shape[1], device="cuda")
    parent = s["page_table"][src]
    shared = slot < whole[:, None]
    child = torch.where(shared, parent, -1)
    s["refs"].scatter_add_(0, child[shared].long(), torch.ones_like(child[shared]))
    fresh = torch.nonzero(s["refs"] == 0).flatten()[: int(part.sum())]
    from_ = parent[part, whole[part]].long()
    child[part, whole[part]] = fresh.int()
    s["refs"][fresh] = 1
    for t in s["K"] + s["V"]:
        t[fresh] = t[from_]
    for t in s["kbar"] + s["state"]:
        t[dst] = t[src]
    s["page_table"][dst] = child
    s["seqlens"][dst] = n.int()


def _reserve(s, add):
    page = s["case"]["page"]
    need = -(-(s["seqlens"] + add) // page)
    slot = torch.arange(s["page_table"].shape[1], device="cuda")
    want = (slot < need[:, None]) & (s["page_table"] < 0) & (add > 0)[:, None]
    fresh = torch.nonzero(s["refs"] == 0).flatten()[: int(want.sum())]
    s["page_table"][want] = fresh.int()
    s["refs"][fresh] = 1


def _compact(s):
    used = s["refs"] > 0
    count = int(used.sum())
    holes = torch.nonzero(~used[:count]).flatten()
    moved = torch.nonzero(used[count:]).flatten() + count
    for t in s["K"] + s["V"]:
        t[holes] = t[moved]
    to = torch.arange(used.numel(), device="cuda")
    to[moved] = holes
    s["refs"][holes] = s["refs"][moved]
    s["refs"][moved] = 0
    s["page_table"].copy_(torch.where(s["page_table"] >= 0, to[s["page_table"].long()].int(), s["page_table"]))


def _copy(s, src, dst):
    for t in s["K"] + s["V"]:
        t[dst.long()] = t[src.long()]


def run(state):
    s = state
    kind = s["case"]["kind"]
    if kind == "attend":
        if own:
            return {"O": s["cache"].decode(s["q"])}
        return _attend(s)
    if kind == "store":
        if own:
            st = s["cache"]
            st.seqlens.copy_(s["start"])
            st.state.copy_(s["state0"])
            st.append(s["k_new"], s["v_new"], s["counts"])
            K, V = st.load(s["start"], s["case"]["n"])
            return {"K": K, "V": V, "kbar": st.kbar, "state": st.state, "seqlens": st.seqlens}
        return _store(s)
    if kind == "fork":   # the last round's candidates leave, the next ones take their rows and get room to grow
        if own:
            s["pages"].free(s["dst"])
            s["pages"].fork(s["src"], s["dst"])
            s["pages"].reserve(s["add"])
        else:
            _free(s, s["dst"])
            _fork(s, s["src"], s["dst"])
            _reserve(s, s["add"])
    elif kind == "compact":
        s["refs"].copy_(s["refs0"])
        s["page_table"].copy_(s["page_table0"])
        if own:
            s["pages"].compact()
        else:
            _compact(s)
    elif own:
        s["pages"].copy(s["src"], s["dst"])
    else:
        _copy(s, s["src"], s["dst"])
    return {k: s[k] for k in ("page_table", "refs", "seqlens", "K", "V", "kbar", "state") if k in s}


# ---- the definitions in 64 bits -------------------------------------------------------------------------
def _e4m3(x):
    """x >= 0 rounded to e4m3 (nearest, ties to even, at most 448) in float64."""
    step = torch.exp2((torch.floor(torch.log2(x.clamp(min=2.0 ** -6))) - 3).clamp(min=-9))
    return (torch.round(x / step) * step).clamp(max=448)


def _exact_values(x, exp):
    g = x.double().unflatten(-1, (-1, 32)) / 2.0 ** exp
    s = _e4m3(g.abs().amax(-1, keepdim=True) / 7)
    return (torch.where(s > 0, torch.round(g / s.clamp(min=2.0 ** -20)).clamp(-7, 7) * s, 0) * 2.0 ** exp).flatten(-2)


def _exact_attend(s):
    c, out = s["case"], []
    h, g, B, d, page = c["h_kv"], c["h_q"] // c["h_kv"], c["chunk"], c["d"], c["page"]
    for i, n in enumerate(_lengths(c)):
        at = s["page_table"][i, : -(-n // page)].long()
        q = s["q"][i].double().view(h, g, d) / math.sqrt(d)

        def rows(name):
            return s["pool"][name][at].transpose(0, 1).flatten(1, 2)[:, :n]

        def scale(name, exp):
            return (rows(name).view(torch.float8_e4m3fn).double() * 2.0 ** exp).repeat_interleave(32, -1)

        def code(r):
            return torch.stack([r.int() % 16, r.int() // 16], -1).flatten(-2).double() - 8

        keys = rows("k_codes").unflatten(-1, (4, d // 32, 4)).permute(0, 1, 3, 2, 4).flatten(2)
        keys = code(keys) * scale("k_scales", K_EXP)
        values = code(rows("v_codes")) * scale("v_scales", V_EXP)
        chunks = (n - 1) // B
        z = q @ keys.transpose(-1, -2)
        if chunks and c["gamma"] > 0:
            x = (c["alpha"] - 1) * c["gamma"] * (q @ s["kbar"][i, :, :chunks].double().transpose(-1, -2))
            p = 1 / (c["alpha"] - 1)
            hi = x.amax(-1, keepdim=True)
            lo = hi - 1
            for _ in range(100):
                mid = (lo + hi) / 2
                over = ((x - mid).clamp(min=0) ** p).sum(-1, keepdim=True) > 1
                lo, hi = torch.where(over, mid, lo), torch.where(over, hi, mid)
            w = ((x - (lo + hi) / 2).clamp(min=0) ** p).mean(1)
            lw = torch.log(w)
            on = w > 0
            mu = torch.where(on, lw, 0).sum(-1, keepdim=True) / on.sum(-1, keepdim=True)
            z[..., : chunks * B] += (lw - mu).repeat_interleave(B, -1)[:, None]
        out.append((torch.softmax(z, -1) @ values).flatten(0, 1))
    return {"O": torch.stack(out)}


def _exact_store(s):
    c = s["case"]
    B, d, n = c["chunk"], c["d"], c["n"]
    K, V = _exact_values(s["k_new"], K_EXP), _exact_values(s["v_new"], V_EXP)
    kbar, state = s["kbar"].double(), s["state0"].double()
    for i, (start, count) in enumerate(zip(s["start"].tolist(), _counts(c))):
        K[i, count:], V[i, count:] = 0, 0
        k = s["k_new"][i, :count].double()
        a = (k * s["qbar"].double()).sum(-1) / math.sqrt(d) * math.log2(math.e)
        if start % B:   # the open chunk's state as one more key of weight l
            old = state[i]
            k = torch.cat([(old[:, :d] / old[:, d + 1:])[None], k])
            a = torch.cat([(old[:, d] + torch.log2(old[:, d + 1]))[None], a])
            cuts = [0, min(1 + B - start % B, a.shape[0])]
        else:
            cuts = [0, min(B, a.shape[0])]
        state[i], state[i, :, d] = 0, -math.inf
        chunk, left = start // B, B - start % B
        whole = max(0, count - left) // B if count >= left else 0
        if whole:   # the complete chunks between, all at once
            kk, aa = (t[cuts[1]: cuts[1] + whole * B].unflatten(0, (whole, B)) for t in (k, a))
            kbar[i, :, chunk + 1: chunk + 1 + whole] = (torch.softmax(aa * math.log(2), 1)[..., None] * kk).sum(1).transpose(0, 1)
        tail = cuts[1] + whole * B
        spans = [(cuts[0], cuts[1], chunk, count >= left)]
        if count > left + whole * B:
            spans.append((tail, a.shape[0], chunk + 1 + whole, False))
        for lo, hi, at, closed in spans:
            if closed:
                kbar[i, :, at] = (torch.softmax(a[lo:hi] * math.log(2), 0)[..., None] * k[lo:hi]).sum(0)
                continue
            tokens, logits = s["k_new"][i, :count].double(), a[lo:hi]
            first = at == chunk and start % B > 0
            m = logits.amax(0)
            if first:   # the running maximum is over the keys, not over the summed weight
                m = torch.maximum(s["state0"][i, :, d].double(), a[lo + 1: hi].amax(0))
            w = torch.exp2(logits - m)
            state[i, :, :d] = (w[..., None] * k[lo:hi]).sum(0)
            state[i, :, d], state[i, :, d + 1] = m, w.sum(0)
            del tokens
    return {"K": K, "V": V, "kbar": kbar, "state": state, "seqlens": s["start"] + s["counts"]}


def exact(case, seed):
    if case["kind"] not in ("attend", "store"):
        return None   # copies: nothing is computed
    s = prepare(case, seed)
    return _exact_attend(s) if case["kind"] == "attend" else _exact_store(s)
