"""The paged K/V cache operators: measured cases, their plain forms and their 64-bit definitions.

Three operators that belong together.  A serving step writes the keys and values of its new
tokens into pages (quantising them where the cache holds 8 bits), lets the new tokens' queries
attend to everything cached so far, and a caller that wants rows of the cache back (to run a
whole-sequence operator on them) reads them.

A cache is k and v [pages, Hkv, page_size, D] in bf16, fp32, e4m3 or int8, the 8-bit ones with one
fp32 scale per row, [pages, Hkv, page_size].  Sequence b's position p lives in page
table[b, p // page_size], row p % page_size; kv_len[b] counts its tokens, the new ones included,
and its new token i of new_len[b] sits at position kv_len[b] - new_len[b] + i.
"""
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn,
          "i8": torch.int8}
SIZE = {"bf16": 2, "f32": 4, "e4m3": 1, "i8": 1}


def _attend(name, B, n, Hq, Hkv, D, kv, page, dtype, cache, causal=True, window=0, ragged=False,
            lse=False):
    return dict(name=name, op="attend", B=B, n=n, Hq=Hq, Hkv=Hkv, D=D, kv=kv, page=page,
                dtype=dtype, cache=cache, causal=causal, window=window, ragged=ragged, lse=lse)


def _write(name, B, n, Hkv, D, kv, page, dtype, cache, ragged=False):
    return dict(name=name, op="write", B=B, n=n, Hq=Hkv, Hkv=Hkv, D=D, kv=kv, page=page,
                dtype=dtype, cache=cache, ragged=ragged)


def _read(name, B, n, Hkv, D, kv, page, dtype, cache, ragged=False):
    return dict(name=name, op="read", B=B, n=n, Hq=Hkv, Hkv=Hkv, D=D, kv=kv, page=page,
                dtype=dtype, cache=cache, ragged=ragged)


def listed():
    return [
        # one user's next token after a short conversation: latency alone
        _attend("attend-one", 1, 1, 8, 8, 64, 1000, 16, "bf16", "bf16"),
        # a full batch's next tokens, every conversation of another length
        _attend("attend-step", 64, 1, 32, 8, 128, 16384, 16, "bf16", "bf16", ragged=True),
        # a few long documents, the cache in 8 bits to hold them
        _attend("attend-step-e4m3", 8, 1, 32, 8, 64, 65536, 64, "bf16", "e4m3", ragged=True),
        # five drafted tokens of every user checked at once, in a page size that is no power of two
        _attend("attend-draft-i8", 16, 5, 32, 8, 128, 8192, 24, "bf16", "i8", ragged=True, lse=True),
        # a long prompt taken in chunks: the last chunk sees all that came before it
        _attend("attend-chunk", 1, 2048, 32, 8, 128, 32768, 64, "bf16", "bf16"),
        # several prompts' chunks of other lengths in one call, a sliding window, an 8-bit cache
        _attend("attend-chunk-e4m3", 6, 777, 8, 8, 64, 9000, 16, "bf16", "e4m3", window=4096,
                ragged=True),
        # a decoder's tokens over an encoder's states, which every query sees whole
        _attend("attend-cross", 4, 448, 16, 16, 64, 1500, 32, "bf16", "bf16", causal=False),
        # an evaluation in fp32, a chunk against a middle-sized context
        _attend("attend-f32", 2, 130, 8, 2, 64, 2100, 16, "f32", "f32", ragged=True, lse=True),
        # a batch's next tokens quantised into their pages, and their stored values read back
        _write("write-step-i8", 64, 1, 8, 128, 16384, 16, "bf16", "i8", ragged=True),
        # two whole prompts quantised into an 8-bit cache, and their stored values read back
        _write("write-prompt-e4m3", 2, 16384, 8, 64, 16384, 64, "bf16", "e4m3"),
        # a few sequences' tails, ragged, read back wide
        _read("read-e4m3-f32", 5, 1001, 8, 64, 3001, 16, "f32", "e4m3", ragged=True),
        # a whole 32k context of one layer read back for a whole-sequence operator
        _read("read-i8", 1, 32768, 8, 128, 32768, 32, "bf16", "i8"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["attend"] * 4 + ["write", "read"])
    D = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8, 8, 16])
    G = rng.choice([1, 1, 2, 3, 4, 4, 7, 8])
    page = rng.choice([8, 16, 16, 24, 32, 64, 128, 256])
    cache = rng.choice(["bf16", "bf16", "e4m3", "i8"])
    if op != "attend":
        dtype = rng.choice(["bf16", "bf16", "f32"])
        cache = rng.choice([cache, cache, cache, "f32"])
        B, n = _log(rng, 1, 64), _log(rng, 1, 16384)
        while B * n * Hkv * D > 1 << 26:
            B, n = max(1, B // 2), max(1, n // 2)
        kv = n + _log(rng, 1, 4096)
        f = _write if op == "write" else _read
        case = f("", B, n, Hkv, D, kv, page, dtype, cache, ragged=rng.random() < 0.5)
    else:
        dtype = "bf16"
        kv = _log(rng, 1, 65536)
        n = min(kv, rng.choice([1, 1, 1, _log(rng, 2, 16), _log(rng, 16, 2048), _log(rng, 16, 2048)]))
        B = _log(rng, 1, 64)
        Hq = Hkv * G
        if rng.random() < 0.12:
            dtype = "f32"
            cache = rng.choice(["f32", "f32", "e4m3", "i8"])
            n, kv = min(n, 300), min(kv, 6000)
        causal = rng.random() < 0.8
        window = _log(rng, 16, 8192) if causal and rng.random() < 0.25 else 0
        # no dearer than the largest listed cases, in products and in cached values
        while B > 1 and (B * n * kv * Hq * D > 1 << 37 or B * kv * Hkv * D > 1 << 29):
            B //= 2
        while n > 1 and B * n * kv * Hq * D > 1 << (37 if dtype == "bf16" else 32):
            n //= 2
        while B * kv * Hkv * D > 1 << 29:
            kv //= 2
        n = min(n, kv)
        case = _attend("", B, n, Hq, Hkv, D, kv, page, dtype, cache, causal, window,
                       rng.random() < 0.6, rng.random() < 0.3)
    del case["name"]
    return case


def _lengths(case):
    """(kv_len, new_len, start) of every sequence, from the case alone."""
    r = random.Random("%(op)s %(B)d %(n)d %(kv)d %(D)d" % case)
    kv, new = [case["kv"]], [case["n"]]
    while len(kv) < case["B"]:
        kv.append(r.randint(1, case["kv"]) if case["ragged"] else case["kv"])
        new.append(r.randint(0, case["n"]) if case["ragged"] and case["n"] > 1 else case["n"])
    new = [min(a, b) for a, b in zip(new, kv)]
    start = [max(0, a - case["n"]) for a in kv]
    return kv, new, start


def _scales(x, cache):
    """Per-row scales of an 8-bit cache.  e4m3: the smallest power of two that brings the row's
    largest magnitude to 448 or less (a finer scale would buy a floating type nothing), 2^-126 at
    the least.  int8: the largest magnitude over 127.  A row of zeros has scale 1."""
    top = x.abs().amax(-1)
    if cache == "e4m3":
        m, e = torch.frexp(top)
        e = torch.where(m <= 0.875, e - 9, e - 8).clamp(min=-126)
        s = ((e + 127) << 23).view(torch.float32)
    else:
        s = top / 127
    return torch.where(top == 0, torch.ones_like(s), s)


def _quantise(x, cache):
    """(stored values, scales or None) of rows x (fp32)."""
    if SIZE[cache] > 1:
        return x.to(DTYPES[cache]), None
    s = _scales(x, cache)
    if cache == "e4m3":
        return (x / s[..., None]).to(DTYPES[cache]), s
    top = x.abs().amax(-1, keepdim=True).double()  # 64 bits: a quotient next to a half step
    y = x.double() * 127 / torch.where(top == 0, 1.0, top)
    return y.round().to(torch.int8), s


def _values(t, s, dtype=torch.float32):
    return t.to(dtype) if s is None else t.to(dtype) * s[..., None].to(dtype)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    B, n, Hq, Hkv, D, page = (case[x] for x in ("B", "n", "Hq", "Hkv", "D", "page"))
    kv, new, start = _lengths(case)
    wide = -(-case["kv"] // page)
    need = [-(-a // page) for a in kv]
    pages = sum(need) + 2
    order = torch.randperm(pages, device=dev, generator=g).tolist()
    table = torch.full((B, wide), -1, dtype=torch.int32)
    at = 0
    for b in range(B):
        table[b, :need[b]] = torch.tensor(order[at:at + need[b]], dtype=torch.int32)
        at += need[b]
    i32 = dict(dtype=torch.int32, device=dev)
    channel = 1 + 3 * (torch.rand(D, device=dev, generator=g) < 0.05)  # a few loud channels, as keys have

    def rows(*shape, loud=True):
        x = torch.randn(*shape, D, device=dev, generator=g)
        return x * channel if loud else x

    s = dict(case=case, table=table.to(dev), kv_len=torch.tensor(kv, **i32),
             new_len=torch.tensor(new, **i32), start=torch.tensor(start, **i32))
    for x in ("k", "v"):
        s[x + "_cache"], s[x + "_scale"] = _quantise(rows(pages, Hkv, page, loud=x == "k"),
                                                     case["cache"])
    # the projections' output, all heads of a token side by side, as a layer has it
    dtype = DTYPES[case["dtype"]]
    if case["op"] == "attend":
        qkv = rows(B, n, Hq + 2 * Hkv, loud=False).to(dtype)
        s["q"] = qkv[:, :, :Hq].transpose(1, 2)
        s["out"] = torch.zeros(B, n, Hq, D, dtype=dtype, device=dev).transpose(1, 2)
        s["lse"] = torch.zeros(B, Hq, n, device=dev) if case["lse"] else None
    elif case["op"] == "write":
        s["k"] = rows(B, n, Hkv).to(dtype).transpose(1, 2)
        s["v"] = rows(B, n, Hkv, loud=False).to(dtype).transpose(1, 2)
    return s


def _positions(s, n):
    """Positions of the new tokens [B, n] and which of them there are."""
    i = torch.arange(n, device=s["kv_len"].device)
    pos = (s["kv_len"] - s["new_len"])[:, None] + i
    return pos, (i < s["new_len"][:, None]) & (pos >= 0)


def _at(s, pos):
    """Page and row of positions [B, m] (those of no page: page 0)."""
    page = s["case"]["page"]
    p = (pos.clamp(min=0) // page).clamp(max=s["table"].shape[1] - 1)
    return s["table"].gather(1, p).long().clamp(min=0), pos.clamp(min=0) % page


def _plain_attend(s):
    c, t = s["case"], s["table"].long().clamp(min=0)
    B, n, Hq, Hkv, D = (c[x] for x in ("B", "n", "Hq", "Hkv", "D"))
    S, G = t.shape[1] * c["page"], Hq // Hkv

    def gathered(x):
        sc = s[x + "_scale"]
        y = _values(s[x + "_cache"][t], None if sc is None else sc[t])
        return y.permute(0, 2, 1, 3, 4).reshape(B, Hkv, S, D)

    q = s["q"].float().reshape(B, Hkv, G * n, D)
    logits = (q @ gathered("k").transpose(-1, -2)).reshape(B, Hkv, G, n, S) * D ** -0.5
    pos, there = _positions(s, n)
    key = torch.arange(S, device=t.device)
    see = (key < s["kv_len"][:, None])[:, None].expand(B, n, S)
    if c["causal"]:
        see = see & (key <= pos[..., None])
        if c["window"]:
            see = see & (key > pos[..., None] - c["window"])
    logits.masked_fill_(~see[:, None, None], float("-inf"))
    m = logits.amax(-1, keepdim=True)
    p = logits.sub_(torch.where(m > float("-inf"), m, 0.0)).exp_()
    total = p.sum(-1, keepdim=True)
    o = p.reshape(B, Hkv, G * n, S) @ gathered("v")
    o = (o.reshape(B, Hkv, G, n, D) / torch.where(total > 0, total, 1.0)).reshape(B, Hq, n, D)
    lse = (m + total.log()).reshape(B, Hq, n)
    there = (torch.arange(n, device=t.device) < s["new_len"][:, None])[:, None]
    o = torch.where(there[..., None], o.to(s["q"].dtype), s["out"])
    return o if s["lse"] is None else (o, torch.where(there, lse, s["lse"]))


def _plain_write(s):
    c = s["case"]
    pos, there = _positions(s, c["n"])
    page, row = _at(s, pos)
    page, row = page[there], row[there]
    for x in ("k", "v"):
        new, sc = _quantise(s[x].transpose(1, 2).float()[there], c["cache"])
        s[x + "_cache"][page, :, row] = new
        if sc is not None:
            s[x + "_scale"][page, :, row] = sc


def _plain_read(s):
    c = s["case"]
    pos = s["start"][:, None] + torch.arange(c["n"], device=s["start"].device)
    page, row = _at(s, pos)
    there = (pos < s["kv_len"][:, None])[..., None, None]

    def back(x):
        sc = s[x + "_scale"]
        y = _values(s[x + "_cache"][page, :, row], None if sc is None else sc[page, :, row])
        return torch.where(there, y, 0.0).transpose(1, 2).contiguous().to(DTYPES[c["dtype"]])

    return back("k"), back("v")


def run(s):
    c = s["case"]
    if own:
        import clustered_multipole_approximation_b200 as muse
        cache = dict(k_scale=s["k_scale"], v_scale=s["v_scale"])
        where = (s["k_cache"], s["v_cache"], s["table"], s["kv_len"])
        if c["op"] == "attend":
            return muse.muse_attn_cache(s["q"], *where, new_len=s["new_len"], scale=c["D"] ** -0.5,
                                        causal=c["causal"], window=c["window"], out=s["out"],
                                        lse=s["lse"], **cache)
        if c["op"] == "write":
            muse.muse_cache_write(s["k"], s["v"], *where, new_len=s["new_len"], **cache)
    else:
        if c["op"] == "attend":
            return _plain_attend(s)
        if c["op"] == "write":
            _plain_write(s)
    if c["op"] == "write" and SIZE[c["cache"]] > 1:
        return s["k_cache"], s["v_cache"]  # the updated pages themselves
    # what a read answers with, or what the written 8-bit rows stand for
    if own:
        return muse.muse_cache_read(*where, c["n"], start=s["start"], dtype=DTYPES[c["dtype"]],
                                    **cache)
    return _plain_read(s)


def _pairs(c, a, m):
    """(query, key) pairs of one head, and the keys that any query sees."""
    if not c["causal"]:
        return m * a, a if m else 0
    w = c["window"] or a
    pairs = sum(min(w, max(0, a - m + i + 1)) for i in range(m))
    return pairs, min(a, w + m - 1) if m else 0


def work(case):
    c = case
    kv, new, start = _lengths(c)
    size, wide = SIZE[c["cache"]], SIZE[c["dtype"]]
    row = 2 * c["Hkv"] * (c["D"] * size + (4 if size == 1 else 0))  # one cached token, K and V
    loose = 2 * c["Hkv"] * c["D"] * wide
    if c["op"] == "attend":
        both = [_pairs(c, a, m) for a, m in zip(kv, new)]
        q = 2 * sum(new) * c["Hq"] * c["D"] * wide
        return {"bytes": q + row * sum(k for _, k in both),
                "flops": 4 * c["Hq"] * c["D"] * sum(p for p, _ in both)}
    there = sum(min(c["n"], a - b) for a, b in zip(kv, start))
    back = row * there + loose * c["B"] * c["n"]
    if c["op"] == "read":
        return {"bytes": back, "flops": 0}
    put = (loose + row) * sum(new)
    return {"bytes": put + (back if size == 1 else 0), "flops": 0}


def _stands_for(x, cache):
    """What a row in 64 bits is stored as, from the definition of its type."""
    top = x.abs().amax(-1, keepdim=True)
    if cache == "i8":
        y = torch.round(x * 127 / torch.where(top == 0, 1.0, top))
        return y * top / 127
    if cache == "e4m3":
        scale = torch.exp2(torch.ceil(torch.log2(torch.where(top == 0, 448.0, top) / 448)).clamp(min=-126))
        y = x / scale
        # three bits behind the leading one; below 2^-6 the steps stay as they are there
        step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
        return torch.round(y / step) * step * scale
    return x.to(DTYPES[cache]).double()


def exact(case, seed):
    c, s = case, prepare(case, seed)
    kv, new, start = _lengths(c)
    page, n = c["page"], c["n"]
    f64 = dict(dtype=torch.float64, device=s["table"].device)

    def cached(x, b, lo, hi):
        """Positions lo to hi of sequence b, [Hkv, hi - lo, D]."""
        p = torch.arange(lo, hi, device=s["table"].device)
        at, r = s["table"][b, p // page].long(), p % page
        y = s[x + "_cache"][at, :, r].to(torch.float64)
        if s[x + "_scale"] is not None:
            y = y * s[x + "_scale"][at, :, r].double()[..., None]
        return y.transpose(0, 1)

    if c["op"] == "attend":
        o = s["out"].double()
        lse = None if s["lse"] is None else s["lse"].double()
        G = c["Hq"] // c["Hkv"]
        for b in range(c["B"]):
            if not new[b]:
                continue
            K, V = cached("k", b, 0, kv[b]), cached("v", b, 0, kv[b])
            seen = torch.ones(new[b], kv[b], dtype=torch.bool, device=K.device)
            if c["causal"]:
                seen = seen.tril(kv[b] - new[b])
                if c["window"]:
                    seen = seen.triu(kv[b] - new[b] - c["window"] + 1)
            for h in range(c["Hq"]):
                x = s["q"][b, h, :new[b]].double() @ K[h // G].T / c["D"] ** 0.5
                x = torch.where(seen, x, -torch.inf)
                z = torch.logsumexp(x, -1)
                o[b, h, :new[b]] = torch.exp(x - z[:, None]) @ V[h // G]
                if lse is not None:
                    lse[b, h, :new[b]] = z
        return o if lse is None else (o, lse)
    if c["op"] == "read" or SIZE[c["cache"]] == 1:
        outs = []
        for x in ("k", "v"):
            out = torch.zeros(c["B"], c["Hkv"], n, c["D"], **f64)
            for b in range(c["B"]):
                out[b, :, :kv[b] - start[b]][:, :n] = cached(x, b, start[b], min(kv[b], start[b] + n))
                if c["op"] == "write":
                    at = kv[b] - new[b] - start[b]
                    out[b, :, at:at + new[b]] = _stands_for(s[x][b, :, :new[b]].double(), c["cache"])
            outs.append(out)
        return tuple(outs)
    outs = []
    for x in ("k", "v"):
        out = s[x + "_cache"].double()
        for b in range(c["B"]):
            p = torch.arange(kv[b] - new[b], kv[b], device=out.device)
            at, r = s["table"][b, p // page].long(), p % page
            out[at, :, r] = _stands_for(s[x][b, :, :new[b]].double(), c["cache"]).transpose(0, 1)
        outs.append(out)
    return tuple(outs)
