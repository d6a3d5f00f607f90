"""The operators around the LLM.int8() linear in a decoder block, as cases that can be measured.

Three families: the residual addition + RMS norm + int8 quantization before a linear, the paged int8 key/value cache
(appending tokens, reading them back), and attention over that cache. `run` makes the calls of
`int8_mixed_precision_rowwise_b200` where `own` is true, and computes the same outputs with elementary torch operations
where it is false. `exact` states the definitions once more, in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
THRESHOLD = 6.0
EPS = 1e-5


# ---------------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # One token of a 4096-wide model before its qkv linear: nothing but latency.
        dict(name="norm_1x4096", op="norm", rows=1, cols=4096, dtype="fp16", threshold=THRESHOLD, y=True),
        # A decode batch at BLOOM-176B width, with the outlier columns the mixed linear looks for.
        dict(name="norm_32x14336", op="norm", rows=32, cols=14336, dtype="fp16", threshold=THRESHOLD, y=True),
        # A prompt of a bf16 model whose linears run without outlier columns, and so need the codes alone.
        dict(name="norm_2048x4096_codes", op="norm", rows=2048, cols=4096, dtype="bf16", threshold=0.0, y=False),
        # A long prompt at BLOOM-176B width.
        dict(name="norm_4001x14336", op="norm", rows=4001, cols=14336, dtype="fp16", threshold=THRESHOLD, y=True),
        # A decode step's cache write for a small batch, read back over the whole (short) sequences.
        dict(name="cache_decode", op="cache", batch=16, len_min=17, len_max=300, new_min=1, new_max=1, kv_heads=8,
             dim=128, page=16, dtype="fp16"),
        # Ragged chunks of prompts that start and end inside pages; a small head.
        dict(name="cache_chunks", op="cache", batch=5, len_min=700, len_max=2500, new_min=33, new_max=700, kv_heads=16,
             dim=64, page=64, dtype="bf16"),
        # The prompt of the BLOOM block benchmark (2048 tokens, 112 heads) written to the cache and read back.
        dict(name="cache_prompt", op="cache", batch=1, len_min=2048, len_max=2048, new_min=2048, new_max=2048,
             kv_heads=112, dim=128, page=16, dtype="fp16"),
        # One sequence, one token: the latency of a decode step's attention.
        dict(name="attend_1x1000", op="attend", batch=1, len_min=1000, len_max=1000, new_min=1, new_max=1, heads=32,
             kv_heads=8, dim=128, page=16, dtype="fp16", alibi=False),
        # A serving batch with ragged lengths and grouped heads.
        dict(name="attend_batch64", op="attend", batch=64, len_min=100, len_max=8000, new_min=1, new_max=1, heads=32,
             kv_heads=8, dim=128, page=16, dtype="fp16", alibi=False),
        # A decode batch of the BLOOM-176B block: 112 heads of their own keys, linear position biases.
        dict(name="attend_bloom16", op="attend", batch=16, len_min=500, len_max=2048, new_min=1, new_max=1, heads=112,
             kv_heads=112, dim=128, page=16, dtype="fp16", alibi=True),
        # Two long contexts, a few drafted tokens each.
        dict(name="attend_long", op="attend", batch=2, len_min=100000, len_max=131072, new_min=2, new_max=2, heads=64,
             kv_heads=8, dim=128, page=64, dtype="bf16", alibi=False),
        # A chunk of two prompts over what is already in the cache.
        dict(name="attend_chunk", op="attend", batch=2, len_min=6000, len_max=8192, new_min=1500, new_max=2048,
             heads=32, kv_heads=8, dim=128, page=32, dtype="bf16", alibi=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "cache", "attend", "attend"])
    dtype = rng.choice(["fp16", "bf16"])
    if op == "norm":
        cols = 16 * _log(rng, 16, 896)
        rows = _log(rng, 1, min(16384, 4001 * 14336 // cols))
        threshold = rng.choice([0.0, THRESHOLD, THRESHOLD])
        return dict(op=op, rows=rows, cols=cols, dtype=dtype, threshold=threshold, y=threshold > 0 or rng.random() < 0.5)
    dim, page = rng.choice([64, 128, 128]), rng.choice([16, 32, 64, 128])
    kv_heads = rng.choice([1, 2, 4, 8, 8, 12, 16, 32, 112])
    if op == "cache":
        budget = 2048 * 112 * 128 // (kv_heads * dim)  # tokens of all sequences
        batch = _log(rng, 1, 64)
        len_max = _log(rng, 2, max(2, min(16384, budget // batch)))
        new_max = rng.choice([1, _log(rng, 1, len_max)])
        return dict(op=op, batch=batch, len_min=max(1, len_max // 3, new_max), len_max=len_max,
                    new_min=max(1, new_max // 2), new_max=new_max, kv_heads=kv_heads, dim=dim, page=page, dtype=dtype)
    group = rng.choice([1, 2, 4, 5, 8, 16])
    heads = kv_heads * group
    budget = 16 * 2048 * 112 * 128 // (kv_heads * dim)
    batch = _log(rng, 1, 128)
    len_max = _log(rng, 2, max(2, min(131072, budget // batch)))
    kind = rng.choice(["one", "one", "few", "chunk"])
    new_max = 1 if kind == "one" else min(len_max, _log(rng, 2, 8) if kind == "few" else _log(rng, 16, 2048))
    if kind != "one":  # scores of the plain form: at most what the largest listed case has
        pairs = 2 * 2048 * 8192 * 32
        batch = max(1, min(batch, pairs // (heads * new_max * len_max)))
        new_max = max(1, min(new_max, pairs // (heads * len_max)))
    return dict(op=op, batch=batch, len_min=max(1, len_max // 4, new_max), len_max=len_max, new_min=max(1, new_max // 2),
                new_max=new_max, heads=heads, kv_heads=kv_heads, dim=dim, page=page, dtype=dtype,
                alibi=rng.random() < 0.25)


def _lengths(case):
    """Lengths and new tokens of the sequences, the same for every seed (work() goes by them): spread evenly over
    their range in an order that mixes short and long ones."""
    b = case["batch"]
    lens, news = [], []
    for i in range(b):
        f = ((i * 7 + 3) % b) / max(1, b - 1) if b > 1 else 1.0
        g = ((i * 5 + 1) % b) / max(1, b - 1) if b > 1 else 1.0
        n = case["new_min"] + round(g * (case["new_max"] - case["new_min"]))
        lens.append(max(n, case["len_min"] + round(f * (case["len_max"] - case["len_min"]))))
        news.append(n)
    return lens, news


def work(case):
    if case["op"] == "norm":
        n, out = case["rows"] * case["cols"], 2 if case["y"] else 0
        # x, residual, new residual; Y; codes written and their values returned; absmax and weight
        return {"bytes": n * (2 + 2 + 2 + out + 1 + 2) + 4 * case["rows"] + 2 * case["cols"], "flops": 10 * n}
    lens, news = _lengths(case)
    hd = case["kv_heads"] * case["dim"]
    if case["op"] == "cache":
        # new tokens in, their codes out; then all codes in and all values out (keys and values each)
        return {"bytes": 2 * hd * (3 * sum(news) + 3 * sum(lens)), "flops": 2 * hd * (3 * sum(news) + sum(lens))}
    pairs = sum(n * (l - n) + n * (n + 1) // 2 for l, n in zip(lens, news))
    pages = sum(-(-l // case["page"]) for l in lens)
    q = sum(news) * case["heads"] * case["dim"]
    return {"bytes": 2 * hd * sum(lens) + 8 * pages * case["kv_heads"] + 4 * q,
            "flops": 4 * case["heads"] * case["dim"] * pairs}


# ---------------------------------------------------------------------------------------------------- inputs

def _codes(x, axes):
    """int8 codes and fp32 absmax of x over `axes`."""
    a = x.abs().amax(dim=axes, keepdim=True)
    return torch.round(x * (127.0 / a.clamp_min(1e-30))).to(torch.int8), a


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def rnd(*shape):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32)

    if case["op"] == "norm":
        rows, cols = case["rows"], case["cols"]
        x, res, w = rnd(rows, cols), rnd(rows, cols), 1 + 0.1 * rnd(cols)
        # hidden states carry a few systematic columns of large magnitude, about 0.05% of them
        big = torch.randperm(cols, generator=g, device=dev)[: max(1, cols // 2048)]
        res[:, big] *= 40.0
        return dict(case=case, x=x.to(dt), res=res.to(dt), w=w.to(dt))
    lens, news = _lengths(case)
    b, h, p, d = case["batch"], case["kv_heads"], case["page"], case["dim"]
    per = [-(-n // p) for n in lens]
    width = max(per) + 1
    pages = sum(per) + 3
    order = torch.randperm(pages, generator=g, device=dev)
    counts = torch.tensor(per, device=dev)
    first = torch.cumsum(counts, 0) - counts
    col = torch.arange(width, device=dev)
    at = (first[:, None] + col[None, :]).clamp_max(pages - 1)
    table = torch.where(col[None, :] < counts[:, None], order[at], -1).to(torch.int32)
    cu = [0]
    for n in news:
        cu.append(cu[-1] + n)
    cu_all = [0]
    for n in lens:
        cu_all.append(cu_all[-1] + n)
    s = dict(case=case, table=table, lens=torch.tensor(lens, dtype=torch.int32, device=dev),
             cu=torch.tensor(cu, dtype=torch.int32, device=dev), cu_all=torch.tensor(cu_all, dtype=torch.int32, device=dev),
             total=cu_all[-1], new_max=max(news))
    # what earlier calls left in the cache: codes of values whose size differs from page to page and head to head
    for name in ("k", "v"):
        codes = torch.empty((pages, h, p, d), dtype=torch.int8, device=dev)
        absmax = torch.empty((pages, h), dtype=torch.float32, device=dev)
        step = max(1, (1 << 26) // (h * p * d))
        for i in range(0, pages, step):
            x = rnd(min(step, pages - i), h, p, d)
            x *= 0.5 + torch.rand((x.shape[0], h, 1, 1), generator=g, device=dev)
            c, a = _codes(x.to(dt).float(), (2, 3))
            codes[i:i + step], absmax[i:i + step] = c, a[:, :, 0, 0]
        s[name], s[name + "a"] = codes, absmax
    if case["op"] == "cache":
        # keys and values are parts of one projection's output, as a fused qkv linear leaves them
        kv = rnd(cu[-1], 2, h, d).to(dt)
        s["K"], s["V"] = kv[:, 0], kv[:, 1]
    else:
        heads = case["heads"]
        s["Q"] = (2.0 * rnd(cu[-1], heads, d)).to(dt)
        s["slopes"] = None
        if case["alibi"]:  # the geometric sequence of linear position biases
            s["slopes"] = torch.exp2(-8.0 * torch.arange(1, heads + 1, device=dev, dtype=torch.float32) / heads)
    return s


# ---------------------------------------------------------------------------------------------------- the calls

def run(s):
    op = s["case"]["op"]
    if own:
        import int8_mixed_precision_rowwise_b200 as llmint8
        if op == "norm":
            codes, absmax, bitmap, y, res = llmint8.add_rmsnorm_quantize(
                s["x"], s["w"], s["res"], eps=EPS, threshold=s["case"]["threshold"], Y=None if s["case"]["y"] else False)
            return {"residual": res, "y": y, "values": llmint8.dequantize_rowwise(codes, absmax), "bitmap": bitmap}
        cache = (s["k"], s["v"], s["ka"], s["va"])
        if op == "cache":
            llmint8.kv_append(s["K"], s["V"], *cache, s["table"], s["lens"], s["cu"])
            k, v = llmint8.kv_read(*cache, s["table"], s["lens"], s["cu_all"], s["total"], dtype=s["K"].dtype)
            return {"k": k, "v": v}
        return {"out": llmint8.kv_attention(s["Q"], *cache, s["table"], s["lens"], s["cu"], alibi_slopes=s["slopes"],
                                            max_new=s["new_max"])}
    return {"norm": _norm, "cache": _cache, "attend": _attend}[op](s)


# ---------------------------------------------------------------------------------------------------- plain forms

def _norm(s):
    case, x, w = s["case"], s["x"], s["w"]
    t = case["threshold"]
    h = (x.float() + s["res"].float()).to(x.dtype)
    hd = h.double()  # y decides which columns reach the threshold
    y = (hd * torch.rsqrt((hd * hd).mean(dim=1, keepdim=True) + EPS) * w.double()).half()
    yf = y.float()
    bitmap = None
    if t > 0:
        out = (yf.abs() >= t).any(dim=0)
        yf = yf.masked_fill(out[None, :], 0.0)
        bits = torch.zeros(-(-case["cols"] // 32) * 32, dtype=torch.int64, device=x.device)
        bits[: case["cols"]] = out.long()
        words = (bits.view(-1, 32) << torch.arange(32, device=x.device)).sum(dim=1)
        bitmap = torch.where(words >= 1 << 31, words - (1 << 32), words).to(torch.int32)
    a = yf.abs().amax(dim=1, keepdim=True)
    codes = torch.round(yf * torch.where(a > 0, 127.0 / a, torch.zeros_like(a)))
    return {"residual": h, "y": y if case["y"] else None, "values": (codes * a / 127.0).half(), "bitmap": bitmap}


def _sequence_of(cu, total):
    """For each packed row its sequence."""
    return torch.searchsorted(cu[1:].long(), torch.arange(total, device=cu.device), right=True)


def _cache(s):
    case, table, cu, lens = s["case"], s["table"].long(), s["cu"].long(), s["lens"].long()
    p = case["page"]
    new = s["K"].shape[0]
    seq = _sequence_of(s["cu"], new)
    start = lens - (cu[1:] - cu[:-1])
    pos = start[seq] + torch.arange(new, device=cu.device) - cu[seq]
    page, slot = table[seq, pos // p], pos % p
    first = table.gather(1, (start // p)[:, None])[:, 0].clamp_min(0)  # the one page that may hold earlier tokens
    held = (start % p > 0)[:, None]
    for x, codes, absmax in ((s["K"], s["k"], s["ka"]), (s["V"], s["v"], s["va"])):
        xf = x.float()
        old = absmax[first]
        top = torch.zeros_like(absmax)
        top.index_reduce_(0, page, xf.abs().amax(dim=2), "amax")
        top.index_reduce_(0, first, torch.where(held, old, torch.zeros_like(old)), "amax")
        ratio = torch.where(held & (top[first] > 0), old / top[first].clamp_min(1e-30), torch.ones_like(old))
        codes[first] = torch.round(codes[first].float() * ratio[:, :, None, None]).to(torch.int8)
        a = top[page]
        mult = torch.where(a > 0, 127.0 / a, torch.zeros_like(a))
        codes[page, :, slot] = torch.round(xf * mult[:, :, None]).to(torch.int8)
        absmax[page] = a
    seq = _sequence_of(s["cu_all"], s["total"])
    pos = torch.arange(s["total"], device=cu.device) - s["cu_all"].long()[seq]
    page, slot = table[seq, pos // p], pos % p
    return {n: (s[n][page, :, slot].float() * (s[n + "a"][page] / 127.0)[:, :, None]).to(s["K"].dtype) for n in ("k", "v")}


def _attend(s):
    case, q = s["case"], s["Q"]
    b, h, p, d = case["batch"], case["kv_heads"], case["page"], case["dim"]
    group = case["heads"] // h
    lens, cu = s["lens"].long(), s["cu"].long()
    width = -(-case["len_max"] // p)
    table = s["table"][:, :width].long().clamp_min(0)
    n = s["new_max"]
    # keys and values of every sequence side by side, up to the longest one's length
    k = s["k"][table].float() * (s["ka"][table] / 127.0)[..., None, None]
    k = k.transpose(1, 2).reshape(b, h, width * p, d)
    news = cu[1:] - cu[:-1]
    row = torch.arange(n, device=q.device)
    at = (cu[:-1, None] + row[None, :]).clamp_max(q.shape[0] - 1)
    qs = q[at].float().view(b, n, h, group, d).permute(0, 2, 3, 1, 4).reshape(b, h, group * n, d)
    scores = torch.matmul(qs, k.transpose(2, 3)).view(b, h, group, n, width * p)
    del k
    scores *= 1.0 / math.sqrt(d)
    pos = (lens - news)[:, None] + row[None, :]
    key = torch.arange(width * p, device=q.device)
    if s["slopes"] is not None:
        away = (key[None, None, :] - pos[:, :, None]).float()
        scores += s["slopes"].view(1, h, group, 1, 1) * away[:, None, None]
    seen = (key[None, None, :] <= pos[:, :, None]) & (key[None, None, :] < lens[:, None, None])
    scores.masked_fill_(~seen[:, None, None], -math.inf)
    scores -= scores.amax(dim=-1, keepdim=True)
    scores.exp_()
    scores /= scores.sum(dim=-1, keepdim=True)
    v = s["v"][table].float() * (s["va"][table] / 127.0)[..., None, None]
    v = v.transpose(1, 2).reshape(b, h, width * p, d)
    out = torch.matmul(scores.view(b, h, group * n, width * p), v)
    out = out.view(b, h, group, n, d).permute(0, 3, 1, 2, 4).reshape(b, n, case["heads"], d)
    seq = _sequence_of(s["cu"], q.shape[0])
    return {"out": out[seq, torch.arange(q.shape[0], device=q.device) - cu[seq]].to(q.dtype)}


# ---------------------------------------------------------------------------------------------------- definitions

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        hidden = (s["x"].double() + s["res"].double()).to(s["x"].dtype).double()
        scale = hidden.pow(2).sum(1).div(case["cols"]).add(EPS).pow(-0.5)
        y = torch.einsum("rc,r,c->rc", hidden, scale, s["w"].double())
        y16 = y.half().double()
        t, bitmap = case["threshold"], None
        if t > 0:
            columns = torch.nonzero(y16.abs().max(0).values >= t).flatten().tolist()
            y16[:, columns] = 0
            words = [0] * -(-case["cols"] // 32)
            for c in columns:
                words[c // 32] |= 1 << (c % 32)
            bitmap = torch.tensor([w - (1 << 32) if w >> 31 else w for w in words], dtype=torch.int32)
        step = y16.abs().max(1).values / 127
        values = torch.where(step[:, None] > 0, (y16 / step[:, None]).round() * step[:, None], 0.0)
        return {"residual": hidden, "y": y if case["y"] else None, "values": values, "bitmap": bitmap}
    lens, news = _lengths(case)
    p, h = case["page"], case["kv_heads"]
    table = s["table"].tolist()
    if case["op"] == "cache":
        out = {}
        for name, x in (("k", s["K"].double()), ("v", s["V"].double())):
            held = s[name].double() * (s[name + "a"].double() / 127)[:, :, None, None]
            rows, done = [], 0
            for i in range(case["batch"]):
                fresh = x[done:done + news[i]]
                done += news[i]
                before = lens[i] - news[i]
                pages = [held[j].transpose(0, 1) for j in table[i][: -(-before // p)]]
                if before % p:  # the page that the new tokens share with earlier ones
                    j = table[i][before // p]
                    mine = fresh[: p - before % p]
                    old = s[name + "a"][j].double()
                    top = torch.maximum(old, mine.abs().amax((0, 2)))
                    step = (top / 127)[None, :, None]
                    kept = s[name][j].double().transpose(0, 1)[: before % p] * (old / top)[None, :, None]
                    pages[-1] = torch.cat([kept.round() * step, (mine / step).round() * step])
                    fresh = fresh[mine.shape[0]:]
                for at in range(0, fresh.shape[0], p):
                    mine = fresh[at:at + p]
                    step = mine.abs().amax((0, 2))[None, :, None] / 127
                    pages.append((mine / step).round() * step)
                rows.append(torch.cat(pages))
            out[name] = torch.cat(rows)
        return out
    group, d = case["heads"] // h, case["dim"]
    cost = sum(n * l for n, l in zip(news, lens)) * case["heads"] * d * 4
    if cost > 1e13:
        return None
    out = torch.empty(s["Q"].shape, dtype=torch.float64, device=s["Q"].device)
    done = 0
    for i in range(case["batch"]):
        n, l = news[i], lens[i]
        pages = s["table"][i, : -(-l // p)].long()
        position = torch.arange(l - n, l, device=out.device, dtype=torch.float64)
        key = torch.arange(l, device=out.device, dtype=torch.float64)
        for j in range(h):
            keys = (s["k"][pages, j].double() * s["ka"][pages, j].double()[:, None, None] / 127).reshape(-1, d)[:l]
            values = (s["v"][pages, j].double() * s["va"][pages, j].double()[:, None, None] / 127).reshape(-1, d)[:l]
            for head in range(j * group, (j + 1) * group):
                z = s["Q"][done:done + n, head].double() @ keys.T / d ** 0.5
                if s["slopes"] is not None:
                    z = z + s["slopes"][head].double() * (key[None, :] - position[:, None])
                z = z.masked_fill(key[None, :] > position[:, None], -math.inf)
                out[done:done + n, head] = torch.softmax(z, dim=1) @ values
        done += n
    return {"out": out}
