"""Plain forms of the paged int8 key/value cache and the attention over it, written from the definitions in
llmint8.h, for the tests. The append's codes are defined by fp32 steps, taken one by one here with numpy; attention is
in 64 bits, with a bound of the error that a kernel of fp32 statistics and fp16 weights may have."""
import numpy as np
import torch


def page_table(lens, page, generator, device, spare=2, width=None, stride_extra=0):
    """Pages in random order; entries that no position uses are -1."""
    per = [-(-n // page) for n in lens]
    pages = sum(per) + spare
    order = torch.randperm(pages, generator=generator).tolist()
    width = width or max(per + [1])
    table = torch.full((len(lens), width + stride_extra), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(per):
        table[b, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
        at += n
    return table.to(device)[:, :width], pages


def cu(news, device):
    return torch.tensor([0] + list(np.cumsum(news)), dtype=torch.int32, device=device)


def random_cache(pages, heads, page, dim, generator, device):
    """Codes and absmax as a cache holds them: sizes that differ by page and head, one page of zeros."""
    out = []
    for _ in range(2):
        codes = torch.randint(-127, 128, (pages, heads, page, dim), generator=generator, dtype=torch.int8)
        absmax = 0.5 + 3 * torch.rand((pages, heads), generator=generator)
        if pages > 3:
            absmax[pages // 2] = 0
            codes[pages // 2] = 0
        out += [codes.to(device), absmax.to(device)]
    return out[0], out[2], out[1], out[3]


def append_reference(x, codes, absmax, table, lens, news):
    """The append's definition for keys or values, in numpy fp32 steps. x fp32 [tokens, H, D] (exact 16-bit values);
    codes int8 [pages, H, P, D] and absmax fp32 [pages, H] are changed in place."""
    page = codes.shape[2]
    f = np.float32
    t0 = 0
    for b, n in enumerate(news):
        first = lens[b] - n
        i = 0
        while i < n:
            pos = first + i
            if pos < 0:
                i += 1
                continue
            slot = pos % page
            m = min(page - slot, n - i)
            pg = int(table[b, pos // page])
            for h in range(x.shape[1]):
                new = x[t0 + i:t0 + i + m, h]
                old = absmax[pg, h] if slot else f(0)
                s = max(old, np.abs(new).max())
                if slot and s > old:
                    ratio = f(old / s)
                    codes[pg, h, :slot] = np.rint(codes[pg, h, :slot].astype(f) * ratio)
                mult = f(f(127) / s) if s > f(4e-37) else f(0)
                codes[pg, h, slot:slot + m] = np.rint(new * mult)
                absmax[pg, h] = s
            i += m
        t0 += n


def sequence_values(codes, absmax, table_row, length, head):
    """float64 [length, D] of one sequence and head; rows of pages that do not exist are None-masked."""
    page = codes.shape[2]
    n = -(-length // page)
    ids = table_row[:n].long()
    ok = (ids >= 0) & (ids < codes.shape[0])
    ids = ids.clamp(0, codes.shape[0] - 1)
    v = codes[ids, head].double() * (absmax[ids, head].double() / 127)[:, None, None]
    return v.reshape(-1, v.shape[-1])[:length], ok.repeat_interleave(page)[:length], \
        (absmax[ids, head].double() / 127).repeat_interleave(page)[:length]


def attention_reference(Q, k, v, ka, va, table, lens, news, scale, causal=True, slopes=None, weight=2.0 ** -11,
                        least=2.0 ** -25):
    """(out, lse, bound of |out's error| before its own rounding) in float64, for packed rows Q. A weight enters the
    value product off by ``weight`` of itself or ``least`` of the row's largest."""
    T, H, D = Q.shape
    group = H // k.shape[1]
    out = torch.zeros((T, H, D), dtype=torch.float64, device=Q.device)
    lse = torch.full((T, H), -float("inf"), dtype=torch.float64, device=Q.device)
    tol = torch.zeros_like(out)
    t0 = 0
    for b, n in enumerate(news):
        length = lens[b]
        pos = torch.arange(length - n, length, device=Q.device, dtype=torch.float64)
        key = torch.arange(max(length, 0), device=Q.device, dtype=torch.float64)
        for h in range(H):
            if n == 0 or length <= 0:
                continue
            K, ok, _ = sequence_values(k, ka, table[b], length, h // group)
            V, _, vs = sequence_values(v, va, table[b], length, h // group)
            q = Q[t0:t0 + n, h].double()
            s = q @ K.T * scale
            # fp32: products and sums of D terms, the scale's and the position term's roundings
            ds = (q.abs() @ K.abs().T) * abs(scale) * 2.0 ** -17
            if slopes is not None:
                away = key[None] - pos[:, None]
                s = s + slopes[h].double() * away
                ds = ds + (slopes[h].double() * away).abs() * 2.0 ** -21
            seen = ok[None] & (pos[:, None] >= 0)
            if causal:
                seen = seen & (key[None] <= pos[:, None])
            s = s.masked_fill(~seen, -float("inf"))
            some = seen.any(1)
            p = torch.where(some[:, None], torch.softmax(s, 1), 0.0).nan_to_num(0.0)
            ds = torch.where(seen, ds, 0.0)
            # a weight is off by its score's error, the exponential's and the score scaling's few units of 2^-24 of
            # |s|, half a step of fp16 (`weight`); weights below fp16's range relative to the row's largest lose 2^-25
            # of it (`least`)
            mag = torch.where(seen, s.abs(), 0.0).amax(1, keepdim=True)
            rel = weight + 2 * (ds.amax(1, keepdim=True) + mag * 2.0 ** -21 + 2.0 ** -19)
            w = (p * vs[None]).amax(1, keepdim=True)
            o = p @ V
            out[t0:t0 + n, h] = o
            tol[t0:t0 + n, h] = rel * (p @ V.abs()) + rel * o.abs() + least * 127 * length * w
            lse[t0:t0 + n, h] = torch.where(some, torch.logsumexp(s, 1), -float("inf"))
        t0 += n
    return out, lse, tol


def check_attention(got, ref, tol, dtype):
    """Every value within its bound and half a step of its type (or of the smallest subnormal)."""
    half = torch.finfo(dtype).eps / 2
    lim = tol * (1 + half) + ref.abs() * half + 2.0 ** -25
    err = (got.double() - ref).abs()
    assert not torch.isnan(got).any()
    assert bool((err <= lim).all()), f"worst excess {float((err - lim).max()):.3g} at bound {float(lim.max()):.3g}"
