"""GPU checks of how exactly the attention's weights enter the value product: as two fp16 values where at most 8 rows
share a head (by the bound max_new), as one elsewhere; and of what max_new may change."""
import math

import pytest
import torch

from kv_support import attention_reference, check_attention, cu, page_table, random_cache

pytestmark = pytest.mark.gpu

F16, BF16 = torch.float16, torch.bfloat16
# Tiles of 8 rows: hi + lo is off by half a step of lo, 2^-22 of the weight, or half of fp16's smallest value, with
# the row's largest weight at 2^8 or above. One value: half a step of fp16, or the same part of the largest.
TWO = dict(weight=2.0 ** -22, least=2.0 ** -33)
ONE = dict(weight=2.0 ** -11, least=2.0 ** -33)


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import int8_mixed_precision_rowwise_b200 as m
    return m


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def cancelling_cache(pages, kv_heads, page, dim, g):
    """Random keys; values of one size whose signs cancel over the keys of a page, apart for each dimension."""
    k, v, ka, va = random_cache(pages, kv_heads, page, dim, g, "cuda")
    signs = torch.rand((pages, kv_heads, page, dim), generator=g).argsort(2).argsort(2) < page // 2
    v.copy_(torch.where(signs, 127, -127).to(torch.int8))
    va.fill_(1.0)
    return k, v, ka, va


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("dim,heads,kv_heads,news", [(128, 8, 1, 1), (64, 6, 2, 2), (128, 3, 3, 1), (64, 8, 8, 5)])
def test_weights_of_few_rows_are_exact_to_22_bits(lib, dtype, dim, heads, kv_heads, news):
    """Nearly flat scores over values that cancel: what is left of them is small, and shows the weights' rounding.
    Weights rounded to fp16 alone would be outside the bound."""
    g = torch.Generator().manual_seed(dim + heads)
    lens, scale = [32, 160], 3e-4
    table, pages = page_table(lens, 16, g, "cuda")
    bufs = cancelling_cache(pages, kv_heads, 16, dim, g)
    assert news * heads // kv_heads <= 8
    Q = torch.randn((2 * news, heads, dim), generator=g).to("cuda").to(dtype)
    for causal in (False, True):
        ref, _, tol = attention_reference(Q, *bufs, table, lens, [news] * 2, scale, causal, **TWO)
        out = lib.kv_attention(Q, *bufs, table, ints(lens), cu([news] * 2, "cuda"), scale=scale, causal=causal,
                               max_new=news)
        check_attention(out, ref, tol, dtype)
    # the first sequence again (all keys seen) with its weights rounded to fp16
    ids = table[0, :2].long()
    ref, _, tol = attention_reference(Q, *bufs, table, lens, [news] * 2, scale, False, **TWO)
    worst = 0.0
    for h in range(heads):
        K, V = (c[ids, h // (heads // kv_heads)].double() * (a[ids, h // (heads // kv_heads)].double() / 127)[:, None, None]
                for c, a in ((bufs[0], bufs[2]), (bufs[1], bufs[3])))
        s = Q[:news, h].double() @ K.reshape(32, dim).T * scale
        w = torch.exp(s - s.amax(1, keepdim=True)) * 256
        rough = (w.half().double() @ V.reshape(32, dim)) / w.sum(1, keepdim=True)
        lim = tol[:news, h] * 1.01 + ref[:news, h].abs() * torch.finfo(dtype).eps / 2 + 2.0 ** -25
        worst = max(worst, float(((rough - ref[:news, h]).abs() / lim).max()))
    assert worst > 2


@pytest.mark.parametrize("heads,news", [(64, 1), (128, 4), (64, 12)])
def test_light_keys_beside_a_heavy_one(lib, heads, news):
    """The first key of every sequence and head has nearly all the weight and a value of 0; the others, 13.5 * 2^-24 of
    it each, make up the result. As fp16 that starts at 1 they would be 13 or 14 * 2^-24, 3.7% off. Enough items that a
    CTA has whole sequences."""
    g = torch.Generator().manual_seed(heads)
    batch, kv_heads, page, dim, length = 8, 64, 64, 64, 2048
    lens = [length] * batch
    table, pages = page_table(lens, page, g, "cuda")
    shape = (pages, kv_heads, page, dim)
    k, v = torch.zeros(shape, dtype=torch.int8, device="cuda"), torch.full(shape, 127, dtype=torch.int8, device="cuda")
    ka, va = torch.ones((pages, kv_heads), device="cuda"), torch.ones((pages, kv_heads), device="cuda")
    first = table[:, 0].long()
    k[first, :, 0], v[first, :, 0] = 127, 0
    Q = torch.ones((batch * news, heads, dim), dtype=F16, device="cuda")
    scale = math.log(2.0 ** 24 / 13.5) / dim
    kind = TWO if news * heads // kv_heads <= 8 else ONE
    ref, _, tol = attention_reference(Q, k, v, ka, va, table, lens, [news] * batch, scale, **kind)
    out = lib.kv_attention(Q, k, v, ka, va, table, ints(lens), cu([news] * batch, "cuda"), scale=scale, max_new=news)
    lim = tol * 1.01 + ref.abs() * 2.0 ** -11 + 2.0 ** -25
    assert float((lim / ref.abs()).max()) < 0.004  # a quarter of the light keys 3.7% off is 0.009
    check_attention(out, ref, tol, F16)


@pytest.mark.parametrize("heads,kv_heads,news", [(8, 2, [1, 1, 1]), (4, 4, [1, 8, 3]), (8, 1, [1, 2, 1]),
                                                 (16, 2, [1, 20, 2])])
def test_max_new_changes_no_more_than_the_rounding(lib, heads, kv_heads, news):
    """Bounds that are right, too high, too low or missing: every result is within the bound of weights in fp16, with
    tiles of 8 rows (max_new, or else all tokens, times the heads of a group) within that of two fp16 values, and
    the same call gives the same bits."""
    g = torch.Generator().manual_seed(heads)
    lens, total, group = [300, 40, 77], sum(news), heads // kv_heads
    table, pages = page_table(lens, 16, g, "cuda")
    bufs = cancelling_cache(pages, kv_heads, 16, 128, g)
    Q = torch.randn((total, heads, 128), generator=g).to("cuda").half()
    args = (table, ints(lens), cu(news, "cuda"))
    for max_new in (0, 1, 2, max(news), 8, 5000):
        few = min(max_new or total, total) * group <= 8
        ref, ref_lse, tol = attention_reference(Q, *bufs, table, lens, news, 1e-3,
                                                **(TWO if few else dict(weight=2.0 ** -11, least=2.0 ** -25)))
        lse = torch.empty((total, heads), device="cuda")
        out = lib.kv_attention(Q, *bufs, *args, scale=1e-3, max_new=max_new, lse=lse)
        check_attention(out, ref, tol, F16)
        assert bool(((lse - ref_lse).abs() <= 2.0 ** -17 * (1 + ref_lse.abs())).all())
        assert torch.equal(out, lib.kv_attention(Q, *bufs, *args, scale=1e-3, max_new=max_new))
