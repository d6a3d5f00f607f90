"""GPU checks of the paged int8 key/value cache (appending, reading back) and of the attention over it."""
import numpy as np
import pytest
import torch

from kv_support import (append_reference, attention_reference, check_attention, cu, page_table, random_cache,
                        sequence_values)

pytestmark = pytest.mark.gpu

F16, BF16 = torch.float16, torch.bfloat16


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import int8_mixed_precision_rowwise_b200 as m
    return m


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def rows(shape, g, dtype, scale=1.0):
    return (scale * torch.randn(shape, generator=g)).to("cuda").to(dtype)


def same_codes(cache, ref, table, lens, page):
    """Codes and absmax of every token that the sequences have."""
    for b, n in enumerate(lens):
        for j in range(-(-n // page)):
            pg, m = int(table[b, j]), min(page, n - j * page)
            assert np.array_equal(cache[0][pg, :, :m], ref[0][pg, :, :m])
            assert np.array_equal(cache[1][pg].view(np.uint32), ref[1][pg].view(np.uint32))


@pytest.mark.parametrize("page,dim,heads,dtype,steps", [
    (16, 128, 3, F16, [[1], [1], [14], [1], [33]]),
    (16, 64, 2, BF16, [[40, 1, 0, 7], [1, 1, 1, 1], [0, 15, 16, 17], [5, 0, 3, 100]]),
    (32, 128, 1, BF16, [[31, 32, 33], [1, 1, 1], [64, 3, 2]]),
    (64, 64, 5, F16, [[130, 2], [1, 200], [1, 1]]),
    (128, 128, 2, F16, [[1, 127, 128, 129, 300], [1, 1, 1, 1, 1], [2, 2, 2, 2, 2]]),
])
def test_append_and_read(lib, page, dim, heads, dtype, steps):
    """Several appends in a row, each from where the last one ended, growing and shrinking values: codes and absmax
    bit-exact after each; then the values read back."""
    g = torch.Generator().manual_seed(page + dim)
    batch = len(steps[0])
    total = [sum(s[b] for s in steps) for b in range(batch)]
    table, pages = page_table(total, page, g, "cuda", stride_extra=3)
    cache = lib.Int8KVCache.empty(pages, heads, page, dim)
    for t in (cache.k_codes, cache.v_codes):
        t.fill_(77)
    for t in (cache.k_absmax, cache.v_absmax):
        t.fill_(float("inf"))  # what a page held before does not matter
    tab = table.cpu()
    ref = [[t.cpu().numpy().copy() for t in p] for p in ((cache.k_codes, cache.k_absmax), (cache.v_codes, cache.v_absmax))]
    lens = [0] * batch
    for i, news in enumerate(steps):
        lens = [a + n for a, n in zip(lens, news)]
        T = sum(news)
        kv = rows((T + 2, heads, 2, dim), g, dtype, scale=[1.0, 3.0, 0.5, 8.0, 1.0][i])  # two rows behind the last
        kv[1 % (T + 2), 0] = 0
        K, V = kv[:, :, 0], kv[:, :, 1]
        cache.append(K, V, table, ints(lens), cu(news, "cuda"))
        for x, (codes, absmax) in zip((K, V), ref):
            append_reference(x[:T].float().cpu().numpy(), codes, absmax, tab, lens, news)
        got = [(cache.k_codes.cpu().numpy(), cache.k_absmax.cpu().numpy()),
               (cache.v_codes.cpu().numpy(), cache.v_absmax.cpu().numpy())]
        for a, b in zip(got, ref):
            same_codes(a, b, tab, lens, page)
    for part in (lens, [min(n, 20) for n in lens]):
        T = sum(part)
        out = [torch.full((T + 1, heads, dim), 7.0, dtype=dtype, device="cuda") for _ in range(2)]
        lib.kv_read(cache.k_codes, cache.v_codes, cache.k_absmax, cache.v_absmax, table, ints(lens), cu(part, "cuda"),
                    T + 1, K=out[0], V=out[1])
        half = torch.finfo(dtype).eps / 2
        for got, codes, absmax in ((out[0], cache.k_codes, cache.k_absmax), (out[1], cache.v_codes, cache.v_absmax)):
            assert bool((got[T] == 7.0).all())  # the row behind the last sequence
            at = 0
            for b, n in enumerate(part):
                for h in range(heads):
                    v = sequence_values(codes, absmax, table[b], lens[b], h)[0][lens[b] - n:]
                    err = (got[at:at + n, h].double() - v).abs()
                    assert bool((err <= v.abs() * (half + 2.0 ** -22) + 2.0 ** -25).all())
                at += n
    assert all(lib.read_status(ws, clear=False) == 0 for ws in lib.workspaces(0))


def test_append_quantizes_within_half_a_step(lib):
    """A page written at once: |value - x| at most half of absmax / 127, with the roundings of the multiplier, of
    the product (up to 127) and of the step: 3 * 127 * 2^-24 of a step each."""
    g = torch.Generator().manual_seed(1)
    table, pages = page_table([100], 32, g, "cuda")
    cache = lib.Int8KVCache.empty(pages, 4, 32, 128)
    K, V = rows((100, 4, 128), g, F16), rows((100, 4, 128), g, F16, 100.0)
    cache.append(K, V, table, ints([100]), ints([0, 100]))
    for x, codes, absmax in ((K, cache.k_codes, cache.k_absmax), (V, cache.v_codes, cache.v_absmax)):
        for h in range(4):
            v, _, step = sequence_values(codes, absmax, table[0], 100, h)
            assert bool(((v - x[:, h].double()).abs() <= step[:, None] * (0.5 + 9 * 127 * 2.0 ** -24)).all())


def test_append_of_tiny_huge_and_zero_values(lib):
    g = torch.Generator().manual_seed(2)
    table, pages = page_table([16] * 4, 16, g, "cuda")
    cache = lib.Int8KVCache.empty(pages, 1, 16, 64)
    K = torch.randn((64, 1, 64), generator=g).to("cuda").to(BF16)
    K[:16] = 0
    K[16:32] *= 1e-38
    K[32:48] *= 1e37
    cache.append(K, -K, table, ints([16] * 4), cu([16] * 4, "cuda"))
    assert not cache.k_codes[table[0, 0].long()].any() and cache.k_absmax[table[0, 0].long(), 0] == 0
    assert not cache.k_codes[table[1, 0].long()].any()  # below what 127 / absmax can express
    k, v = cache.read(table, ints([16] * 4), cu([16] * 4, "cuda"), 64, dtype=BF16)
    assert bool(torch.isfinite(k).all())
    big = K[32:].double()
    step = big.abs().view(2, -1).amax(1) / 127
    assert bool(((k[32:].double() - big).abs() <= step.repeat_interleave(16)[:, None, None] * 0.51 + big.abs() * 2.0 ** -8).all())


def test_pages_outside_the_cache_are_left_out(lib):
    """A page number of -1, one past the cache, and positions past the table: nothing is written there, the status
    bit is set, the other tokens are as ever."""
    g = torch.Generator().manual_seed(3)
    page, heads, dim = 16, 2, 64
    lens, news = [60, 40], [60, 40]
    table, pages = page_table(lens, page, g, "cuda", width=4)
    cache = lib.Int8KVCache.empty(pages, heads, page, dim)
    bad = table.clone()
    bad[0, 1], bad[1, 0] = -1, pages
    narrow = bad[:, :3]  # sequence 0 needs four
    ws = torch.zeros(lib.kv_attention_workspace_size(heads, heads, dim), dtype=torch.uint8, device="cuda")
    K, V = rows((100, heads, dim), g, F16), rows((100, heads, dim), g, F16)
    for t in (cache.k_codes, cache.v_codes):
        t.fill_(5)
    bufs = (cache.k_codes, cache.v_codes, cache.k_absmax, cache.v_absmax)
    lib.kv_append(K, V, *bufs, narrow, ints(lens), cu(news, "cuda"), workspace=ws)
    assert lib.read_status(ws) == 0x20 and lib.read_status(ws) == 0
    for pg in (int(table[0, 1]), int(table[0, 3]), int(table[1, 0])):
        assert bool((cache.k_codes[pg] == 5).all())
    k, v = [torch.full((100, heads, dim), 9.0, dtype=F16, device="cuda") for _ in range(2)]
    lib.kv_read(*bufs, narrow, ints(lens), cu(news, "cuda"), 100, K=k, V=v, workspace=ws)
    assert lib.read_status(ws) == 0x20
    left = torch.zeros(100, dtype=torch.bool, device="cuda")
    left[16:32] = left[48:60] = left[60:76] = True
    assert bool((k[left] == 9.0).all()) and bool(((k[~left] - K[~left]).abs() < 0.05).all())
    Q = rows((2, heads, dim), g, F16)
    lse = torch.empty((2, heads), device="cuda")
    out = lib.kv_attention(Q, *bufs, narrow, ints(lens), ints([0, 1, 2]), lse=lse, workspace=ws)
    assert lib.read_status(ws) == 0x20
    full = torch.full((2, 4), -1, dtype=torch.int32, device="cuda")
    full[:, :3] = narrow
    ref, ref_lse, tol = attention_reference(Q, *bufs, full, lens, [1, 1], dim ** -0.5)
    check_attention(out, ref, tol, F16)
    assert bool(((lse - ref_lse).abs() <= 1e-4).all())


@pytest.mark.parametrize("news,heads,kv_heads", [(1, 4, 1), (40, 4, 1), (1, 112, 112), (40, 112, 112)])
def test_the_first_keys_missing_and_the_others_far_below(lib, news, heads, kv_heads):
    """The first 160 positions without pages, and scores of the others near -600: the rows' maximum is far below zero
    when it is first known, in a unit of keys that is not the first (with 112 heads, of one CTA's)."""
    g = torch.Generator().manual_seed(4)
    lens = [500]
    table, pages = page_table(lens, 16, g, "cuda")
    k, v, ka, va = random_cache(pages, kv_heads, 16, 128, g, "cuda")
    table[0, :10] = -1
    k.copy_(torch.randint(100, 128, k.shape, generator=g, dtype=torch.int8))
    ka.fill_(1.0)
    Q = (-60 - rows((news, heads, 128), g, F16).abs())
    ws = torch.zeros(lib.kv_attention_workspace_size(heads, kv_heads, 128), dtype=torch.uint8, device="cuda")
    ref, _, tol = attention_reference(Q, k, v, ka, va, table, lens, [news], 128 ** -0.5)
    out = lib.kv_attention(Q, k, v, ka, va, table, ints(lens), ints([0, news]), workspace=ws)
    assert lib.read_status(ws) == 0x20
    assert ref.abs().max() > 0.1
    check_attention(out, ref, tol, F16)


@pytest.mark.parametrize("news", [1, 12, 40, 300])
@pytest.mark.parametrize("dim,dtype,alibi", [(128, F16, False), (64, BF16, False), (128, BF16, True)])
def test_scores_that_grow_along_the_sequence(lib, news, dim, dtype, alibi):
    """Enough heads and keys that a CTA runs through several units of an item, with scores that grow from page to
    page, by little, by much and by leaps: the running maximum moves in the middle of it, for some rows."""
    g = torch.Generator().manual_seed(news + dim)
    lens, kv_heads = [1500, 1400, 1450], 40
    table, pages = page_table(lens, 32, g, "cuda")
    k, v, ka, va = random_cache(pages, kv_heads, 32, dim, g, "cuda")
    for b in range(3):
        for j in range(lens[b] // 32):
            ka[table[b, j].long()] *= (1 + j / 10) if b == 0 else 1.3 ** j * 1e-3 if b == 1 else (40.0 if j % 11 == 10 else 0.1)
    Q = rows((3 * news, kv_heads, dim), g, dtype, 2.0)
    slopes = torch.linspace(0.001, 2.0, kv_heads, device="cuda") if alibi else None
    ref, ref_lse, tol = attention_reference(Q, k, v, ka, va, table, lens, [news] * 3, dim ** -0.5, slopes=slopes)
    lse = torch.empty((3 * news, kv_heads), device="cuda")
    out = lib.kv_attention(Q, k, v, ka, va, table, ints(lens), cu([news] * 3, "cuda"), alibi_slopes=slopes, lse=lse)
    check_attention(out, ref, tol, dtype)
    assert bool(((lse - ref_lse).abs() <= 2.0 ** -10 + 2.0 ** -17 * ref_lse.abs()).all())


@pytest.mark.parametrize("news", [1, 40])
@pytest.mark.parametrize("scale", [-0.2, 0.0, 3.0])
def test_attention_scales(lib, news, scale):
    g = torch.Generator().manual_seed(5)
    table, pages = page_table([300], 32, g, "cuda")
    bufs = random_cache(pages, 2, 32, 64, g, "cuda")
    for dtype in (F16, BF16):
        Q = rows((news, 4, 64), g, dtype)
        ref, _, tol = attention_reference(Q, *bufs, table, [300], [news], scale)
        check_attention(lib.kv_attention(Q, *bufs, table, ints([300]), ints([0, news]), scale=scale), ref, tol, dtype)


def run_attention(lib, page, dim, heads, kv_heads, dtype, lens, news, causal=True, alibi=False, seed=0, q_scale=1.0,
                  max_new=None, extra_rows=1, cache=None, **more):
    g = torch.Generator().manual_seed(seed)
    table, pages = page_table(lens, page, g, "cuda", stride_extra=seed % 2)
    bufs = random_cache(pages, kv_heads, page, dim, g, "cuda")
    T = sum(news)
    fused = rows((T + extra_rows, heads + 2 * kv_heads, dim), g, dtype, q_scale)
    Q = fused[:, :heads]  # a part of a fused projection's output
    slopes = torch.exp2(-8 * torch.arange(1, heads + 1, device="cuda") / heads) if alibi else None
    scale = dim ** -0.5
    ref, ref_lse, tol = attention_reference(Q[:T], *bufs, table, lens, news, scale, causal, slopes)
    out = torch.full((T + extra_rows, heads, dim), 3.0, dtype=dtype, device="cuda")
    lse = torch.full((T + extra_rows, heads), 3.0, device="cuda")
    lib.kv_attention(Q, *bufs, table, ints(lens), cu(news, "cuda"), causal=causal, alibi_slopes=slopes, out=out,
                     lse=lse, max_new=max(news) if max_new is None else max_new, **more)
    check_attention(out[:T], ref, tol, dtype)
    assert bool((out[T:] == 3.0).all()) and bool((lse[T:] == 3.0).all())  # rows of no sequence
    fine = torch.isfinite(ref_lse)
    assert torch.equal(fine, torch.isfinite(lse[:T]))
    # scores reach a few hundred: D products' roundings (2^-17 of the sum of magnitudes) and the logarithm's
    assert bool(((lse[:T] - ref_lse)[fine].abs() <= 2.0 ** -10 + 2.0 ** -18 * ref_lse[fine].abs()).all())
    assert all(lib.read_status(ws, clear=False) == 0 for ws in lib.workspaces(0))
    return out


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("page,heads,kv_heads", [(16, 8, 1), (16, 6, 6), (32, 10, 2), (64, 16, 1), (128, 8, 4),
                                                 (16, 24, 1), (32, 40, 1)])
def test_attention_of_single_tokens(lib, page, dim, heads, kv_heads, dtype):
    lens = [1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 100, 127, 128, 129, 200, 257, 0, 511, 700]
    run_attention(lib, page, dim, heads, kv_heads, dtype, lens, [min(n, 1) for n in lens], seed=page + heads)


@pytest.mark.parametrize("dtype,dim", [(F16, 128), (BF16, 64)])
def test_many_short_sequences_one_after_the_other_in_a_cta(lib, dtype, dim):
    """Each CTA ends items and begins the next ones several times over, its warps at their own pace; twice the same."""
    g = torch.Generator().manual_seed(29)
    news = torch.randint(5, 40, (160,), generator=g).tolist()
    lens = [n + e for n, e in zip(news, torch.randint(0, 90, (160,), generator=g).tolist())]
    first, again = (run_attention(lib, 16, dim, 32, 4, dtype, lens, news, seed=31) for _ in range(2))
    assert torch.equal(first, again)


@pytest.mark.parametrize("dtype,dim", [(F16, 128), (BF16, 64)])
@pytest.mark.parametrize("page,heads,kv_heads,alibi", [(16, 8, 2, False), (16, 5, 5, True), (32, 8, 1, True),
                                                       (64, 32, 2, False), (128, 3, 3, False)])
@pytest.mark.parametrize("causal", [True, False])
def test_attention_of_several_tokens(lib, page, dim, heads, kv_heads, dtype, alibi, causal):
    lens = [1, 9, 16, 40, 64, 130, 300, 5, 0, 77]
    news = [1, 4, 16, 3, 64, 129, 17, 5, 0, 2]
    run_attention(lib, page, dim, heads, kv_heads, dtype, lens, news, causal, alibi, seed=page + 2 * heads)


@pytest.mark.parametrize("heads,kv_heads,lens,news", [
    (4, 1, [5000], [1]), (8, 8, [3000, 12], [1, 1]), (4, 2, [2500, 2500], [2, 1]), (2, 1, [1500], [700]),
    (1, 1, [1100], [1100]), (8, 1, [900, 1, 640], [300, 1, 640]), (16, 2, [4097], [33])])
@pytest.mark.parametrize("dim,dtype", [(128, F16), (128, BF16), (64, F16)])
def test_attention_of_longer_sequences(lib, heads, kv_heads, lens, news, dim, dtype):
    run_attention(lib, 32, dim, heads, kv_heads, dtype, lens, news, seed=heads + lens[0], alibi=heads == 8)


@pytest.mark.parametrize("max_new", [0, 1, 5, 5000])
def test_attention_max_new_only_helps(lib, max_new):
    """Bounds that are too low, too high or missing give the same values."""
    run_attention(lib, 16, 128, 8, 2, F16, [300, 40, 7], [150, 1, 7], seed=5, max_new=max_new)


def test_attention_rows_before_the_sequence(lib):
    """More rows than the sequence has tokens: those at negative positions see nothing."""
    g = torch.Generator().manual_seed(8)
    table, pages = page_table([20, 8], 16, g, "cuda")
    bufs = random_cache(pages, 2, 16, 128, g, "cuda")
    for news in ([25, 8], [22, 10]):
        Q = rows((sum(news), 4, 128), g, F16)
        lse = torch.empty((sum(news), 4), device="cuda")
        out = lib.kv_attention(Q, *bufs, table, ints([20, 8]), cu(news, "cuda"), lse=lse)
        n = news[0] - 20
        assert not out[:n].any() and bool((lse[:n] == -float("inf")).all())
        ref, _, tol = attention_reference(Q, *bufs, table, [20, 8], news, 128 ** -0.5)
        check_attention(out, ref, tol, F16)


def test_attention_of_empty_sequences_and_batches(lib):
    g = torch.Generator().manual_seed(9)
    bufs = random_cache(4, 2, 16, 64, g, "cuda")
    table = torch.full((2, 3), -1, dtype=torch.int32, device="cuda")
    Q = rows((3, 2, 64), g, F16)
    out = lib.kv_attention(Q, *bufs, table, ints([0, 0]), ints([0, 1, 3]))
    assert not out.any()  # rows without keys
    out.fill_(2.0)
    lib.kv_attention(Q, *bufs, table, ints([0, 0]), ints([0, 0, 0]), out=out)
    assert bool((out == 2.0).all())
    assert lib.kv_attention(Q[:0], *bufs, table, ints([0, 0]), ints([0, 0, 0])).shape == (0, 2, 64)
    assert lib.kv_attention(Q[:0], *bufs, table[:0], ints([]), ints([0])).numel() == 0
    lib.kv_append(Q[:0], Q[:0], *bufs, table, ints([0, 0]), ints([0, 0, 0]))


@pytest.mark.parametrize("dim,news", [(128, 1), (64, 3), (128, 70)])
def test_attention_sharp_and_flat_scores(lib, dim, news):
    """Queries large enough that one key takes nearly all weight, and zero ones: the mean of the values."""
    for q_scale in (50.0, 0.0):
        run_attention(lib, 16, dim, 4, 2, F16, [400, 90], [news, news], seed=dim, q_scale=q_scale)


@pytest.mark.parametrize("news", [1, 40])
def test_attention_over_pages_of_very_different_size(lib, news):
    """Pages whose values differ by many orders of magnitude; the largest keys get all the weight in some rows and
    the smallest values all of it in others."""
    g = torch.Generator().manual_seed(12)
    lens = [330]
    table, pages = page_table(lens, 16, g, "cuda")
    k, v, ka, va = random_cache(pages, 2, 16, 128, g, "cuda")
    va *= torch.exp2(torch.randint(-40, 10, va.shape, generator=g).float()).to("cuda")
    ka *= torch.exp2(torch.randint(-6, 3, ka.shape, generator=g).float()).to("cuda")
    for dtype in (F16, BF16):
        Q = rows((news, 8, 128), g, dtype, 2.0)
        ref, _, tol = attention_reference(Q, k, v, ka, va, table, lens, [news], 128 ** -0.5)
        out = lib.kv_attention(Q, k, v, ka, va, table, ints(lens), ints([0, news]))
        check_attention(out, ref, tol, dtype)


def test_attention_bf16_queries_beyond_fp16(lib):
    """bf16 queries larger than fp16 can hold, with keys small enough that the scores stay moderate."""
    g = torch.Generator().manual_seed(13)
    table, pages = page_table([200, 200], 16, g, "cuda")
    k, v, ka, va = random_cache(pages, 1, 16, 128, g, "cuda")
    for news in (1, 50):
        Q = rows((2 * news, 4, 128), g, BF16, 1e20)
        ref, _, tol = attention_reference(Q, k, v, ka * 1e-20, va, table, [200, 200], [news, news], 128 ** -0.5)
        out = lib.kv_attention(Q, k, v, ka * 1e-20, va, table, ints([200, 200]), cu([news, news], "cuda"))
        check_attention(out, ref, tol, BF16)


def test_attention_in_a_cache_past_2_gib(lib):
    """Pages whose offset does not fit 31 bits."""
    g = torch.Generator().manual_seed(14)
    page, heads, dim, pages = 128, 8, 128, 17000
    k = torch.zeros((pages, heads, page, dim), dtype=torch.int8, device="cuda")
    v = torch.zeros_like(k)
    ka, va = torch.ones((pages, heads), device="cuda"), torch.ones((pages, heads), device="cuda")
    lens = [400, 300]
    table = ints([[pages - 1, pages - 2, pages - 3, pages - 4], [16500, 16400, 0, -1]])
    K, V = rows((700, heads, dim), g, F16), rows((700, heads, dim), g, F16)
    lib.kv_append(K, V, k, v, ka, va, table, ints(lens), cu(lens, "cuda"))
    rk, rv = lib.kv_read(k, v, ka, va, table, ints(lens), cu(lens, "cuda"), 700)
    assert bool(((rk - K).abs() < 0.03).all()) and bool(((rv - V).abs() < 0.03).all())
    for news in ([1, 1], [200, 130]):
        Q = rows((sum(news), heads, dim), g, F16)
        ref, _, tol = attention_reference(Q, k, v, ka, va, table, lens, news, dim ** -0.5)
        check_attention(lib.kv_attention(Q, k, v, ka, va, table, ints(lens), cu(news, "cuda")), ref, tol, F16)


def test_attention_is_the_same_every_time(lib):
    """No order of summation that changes from run to run."""
    for news in ([1, 1, 1], [2, 300, 1]):
        a = run_attention(lib, 16, 128, 8, 2, F16, [3000, 1000, 50], news, seed=4)
        for _ in range(3):
            assert torch.equal(a, run_attention(lib, 16, 128, 8, 2, F16, [3000, 1000, 50], news, seed=4))


def test_decode_steps_captured_and_replayed(lib):
    """One captured step (append, then attention) replayed with the lengths, tables and tokens of each step, on a
    stream of its own; two such graphs share a workspace and run in turn."""
    g = torch.Generator().manual_seed(15)
    page, heads, kv_heads, dim, batch, steps = 16, 8, 2, 128, 3, 20
    start = [30, 5, 1000]
    total = [n + steps for n in start]
    table, pages = page_table(total, page, g, "cuda")
    cache = lib.Int8KVCache.empty(pages, kv_heads, page, dim)
    bufs = (cache.k_codes, cache.v_codes, cache.k_absmax, cache.v_absmax)
    K0, V0 = rows((sum(start), kv_heads, dim), g, F16), rows((sum(start), kv_heads, dim), g, F16)
    cache.append(K0, V0, table, ints(start), cu(start, "cuda"))
    lens = ints(start)
    q, k, v = (torch.zeros((batch, h, dim), dtype=F16, device="cuda") for h in (heads, kv_heads, kv_heads))
    rows_at = ints(list(range(batch + 1)))
    ws = torch.zeros(max(4096, lib.kv_attention_workspace_size(heads, kv_heads, dim)), dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graphs, outs = [], []
    with torch.cuda.stream(s):
        lib.kv_attention(q, *bufs, table, lens, rows_at, workspace=ws)
        for _ in range(2):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=s):
                lib.kv_append(k, v, *bufs, table, lens, rows_at, workspace=ws)
                outs.append(lib.kv_attention(q, *bufs, table, lens, rows_at, max_new=1, workspace=ws))
            graphs.append(graph)
        for step in range(steps):
            now = [n + step + 1 for n in start]
            lens.copy_(ints(now))
            for x, h in ((q, heads), (k, kv_heads), (v, kv_heads)):
                x.copy_(rows((batch, h, dim), g, F16))
            graphs[step % 2].replay()
            s.synchronize()
            ref, _, tol = attention_reference(q, *bufs, table, now, [1] * batch, dim ** -0.5)
            check_attention(outs[step % 2], ref, tol, F16)
    assert lib.read_status(ws) == 0


def test_first_use_inside_a_capture(lib):
    """Graphs that are captured on streams where these calls were never made before: each replay starts from a clean
    workspace of its own, whatever the memory held; eager calls in between are not disturbed."""
    g = torch.Generator().manual_seed(17)
    lens = [700, 333]
    table, pages = page_table(lens, 16, g, "cuda")
    bufs = random_cache(pages, 2, 16, 128, g, "cuda")
    Q = rows((2, 8, 128), g, F16)
    n, at = ints(lens), ints([0, 1, 2])
    ref, _, tol = attention_reference(Q, *bufs, table, lens, [1, 1], 128 ** -0.5)
    x = rows((3, 512), g, F16)
    w = torch.ones(512, dtype=F16, device="cuda")
    dirt = torch.full((64 << 20,), 255, dtype=torch.uint8, device="cuda")
    del dirt  # what the allocator hands out next is not zeros
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
            a = lib.kv_attention(Q, *bufs, table, n, at)
            b = lib.add_rmsnorm_quantize(x, w, threshold=1.5)
        graphs.append((graph, a, b))
    want = lib.add_rmsnorm_quantize(x, w, threshold=1.5)
    for _ in range(3):
        for graph, a, b in graphs:
            a.zero_()
            graph.replay()
            torch.cuda.synchronize()
            check_attention(a, ref, tol, F16)
            assert all(torch.equal(p, q) for p, q in zip(b[:4], want[:4]))
            check_attention(lib.kv_attention(Q, *bufs, table, n, at), ref, tol, F16)


def test_graphs_captured_on_a_used_stream_run_at_once(lib):
    """Two graphs captured on a stream where these calls were made before have workspaces of their own, one each,
    apart from the stream's: replayed on two streams at once, next to calls on the one they were captured on, all
    give what each gives alone."""
    g = torch.Generator().manual_seed(23)
    lens = [5000, 3000, 900]
    table, pages = page_table(lens, 16, g, "cuda")
    bufs = random_cache(pages, 4, 16, 128, g, "cuda")
    n, at = ints(lens), ints([0, 1, 2, 3])
    q = [rows((3, 16, 128), g, F16) for _ in range(3)]
    want = [lib.kv_attention(x, *bufs, table, n, at, max_new=1) for x in q]
    out = [torch.zeros_like(x) for x in q]
    torch.cuda.synchronize()
    s, others = torch.cuda.Stream(), [torch.cuda.Stream(), torch.cuda.Stream()]
    used, graphs = [], []
    with torch.cuda.stream(s):
        lib.kv_attention(q[2], *bufs, table, n, at, max_new=1, out=out[2])
        used.append(lib._workspace(None, s.device_index)[0])
        for i in range(2):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=s):
                for _ in range(3):
                    lib.kv_attention(q[i], *bufs, table, n, at, max_new=1, out=out[i])
                    used.append(lib._workspace(None, s.device_index)[0])
            graphs.append(graph)
    torch.cuda.synchronize()
    assert used[1] == used[2] == used[3] and used[4] == used[5] == used[6] and len(set(used)) == 3
    for _ in range(5):
        for graph, o in zip(graphs, others):
            with torch.cuda.stream(o):
                graph.replay()
        with torch.cuda.stream(s):
            lib.kv_attention(q[2], *bufs, table, n, at, max_new=1, out=out[2])
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
        for x in out:
            x.zero_()
        torch.cuda.synchronize()


def test_calls_on_two_streams_at_once(lib):
    """The same calls on two streams, each with a workspace of its own, give what one after the other does."""
    g = torch.Generator().manual_seed(18)
    lens = [2000, 1500, 900]
    table, pages = page_table(lens, 32, g, "cuda")
    bufs = random_cache(pages, 4, 32, 128, g, "cuda")
    n = ints(lens)
    cases = [(rows((3, 16, 128), g, F16), ints([0, 1, 2, 3])), (rows((600, 16, 128), g, F16), ints([0, 250, 500, 600]))]
    want = [lib.kv_attention(q, *bufs, table, n, at) for q, at in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[] for _ in cases]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(lib.kv_attention(*(cases[i][0],), *bufs, table, n, cases[i][1]))
    torch.cuda.synchronize()
    for i, outs in enumerate(got):
        assert all(torch.equal(o, want[i]) for o in outs)


def test_a_block_of_operators_together(lib):
    """A prompt and two decode steps through one attention block as it would be served: norm and quantization, the
    int8 qkv linear, the cache, attention, the int8 output linear. Each stage against its definition on the inputs
    it was given."""
    g = torch.Generator().manual_seed(16)
    hidden, heads, kv_heads, dim, page = 512, 8, 2, 64, 16
    width = (heads + 2 * kv_heads) * dim
    w_norm = (1 + 0.1 * torch.randn(hidden, generator=g)).cuda().half()
    w_qkv = (0.05 * torch.randn((width, hidden), generator=g)).cuda().half()
    w_out = (0.05 * torch.randn((hidden, heads * dim), generator=g)).cuda().half()
    CB, SCB, _ = lib.quantize_rowwise(w_qkv)
    out_linear = lib.Int8MixedLinear.from_fp16(w_out)
    prompt, steps = [37, 64, 5], 2
    table, pages = page_table([n + steps for n in prompt], page, g, "cuda")
    cache = lib.Int8KVCache.empty(pages, kv_heads, page, dim)
    bufs = (cache.k_codes, cache.v_codes, cache.k_absmax, cache.v_absmax)
    lens = [0] * 3
    for news in (prompt, [1] * 3, [1] * 3):
        lens = [a + n for a, n in zip(lens, news)]
        T = sum(news)
        x, stream = rows((T, hidden), g, F16), rows((T, hidden), g, F16)
        stream[:, 7] = 40.0
        codes, absmax, bitmap, y, stream = lib.add_rmsnorm_quantize(x, w_norm, stream, threshold=6.0,
                                                                    residual_out=stream)
        col, count, _ = lib.find_outlier_cols(bitmap, hidden, sync_count=False)
        qkv = lib.matmul_codes(codes, absmax, y, CB, SCB, col, count, W_f16=w_qkv)
        ref = lib.matmul_mixed(y, CB, SCB, w_qkv, 6.0)
        assert bool(((qkv - ref).abs() <= 1e-2 + 2e-3 * ref.abs()).all())  # the linear's own bound
        qkv = qkv.view(T, heads + 2 * kv_heads, dim)
        q, k, v = qkv[:, :heads], qkv[:, heads:heads + kv_heads], qkv[:, heads + kv_heads:]
        cache.append(k, v, table, ints(lens), cu(news, "cuda"))
        a = cache.attend(q, table, ints(lens), cu(news, "cuda"))
        ref, _, tol = attention_reference(q, *bufs, table, lens, news, dim ** -0.5)
        check_attention(a, ref, tol, F16)
        kr, _ = cache.read(table, ints(lens), cu(news, "cuda"), T)
        # a new token's step is its page's absmax / 127 at that time, and later appends round once more
        assert bool(((kr - k).abs() <= k.abs().amax() / 127 + 2.0 ** -10 * k.abs()).all())
        out = out_linear(a.reshape(T, heads * dim))
        assert out.shape == (T, hidden) and bool(torch.isfinite(out).all())
