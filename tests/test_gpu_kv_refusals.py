"""What the binding of the norm, cache and attention calls refuses, with tensors on the GPU: nothing is launched."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import int8_mixed_precision_rowwise_b200 as m
    return m


def cache():
    codes = torch.zeros((4, 2, 16, 64), dtype=torch.int8, device="cuda")
    absmax = torch.ones((4, 2), device="cuda")
    table = torch.zeros((3, 2), dtype=torch.int32, device="cuda")
    lens = torch.ones(3, dtype=torch.int32, device="cuda")
    return [codes, codes.clone(), absmax, absmax.clone(), table, lens,
            torch.arange(4, dtype=torch.int32, device="cuda")]


def changes():
    c = cache()
    half = torch.float16
    yield 0, c[0].to(torch.uint8)
    yield 0, c[0][:, :, :8]
    yield 0, c[0].cpu()
    yield 0, c[0].view(4, 2, -1)
    yield 0, None
    yield 1, c[1][:3]
    yield 1, c[1].float()
    yield 2, c[2].to(half)
    yield 2, c[2].T
    yield 3, c[3][:, :1]
    yield 3, c[3].cpu()
    yield 4, c[4].long()
    yield 4, c[4].view(-1)
    yield 4, c[4].T.contiguous().T
    yield 4, c[4][:1].expand(3, 2)
    yield 4, c[4].cpu()
    yield 5, c[5][:2]
    yield 5, c[5].long()
    yield 5, torch.ones(6, dtype=torch.int32, device="cuda")[::2]
    yield 6, c[6][:3]
    yield 6, c[6].cpu()


@pytest.mark.parametrize("n", range(21))
def test_caches_that_do_not_fit_are_refused(lib, n):
    at, bad = list(changes())[n]
    c = cache()
    c[at] = bad
    rows = torch.zeros((3, 2, 64), dtype=torch.float16, device="cuda")
    for call in (lambda: lib.kv_append(rows, rows, *c), lambda: lib.kv_read(*c, 3), lambda: lib.kv_attention(rows, *c)):
        with pytest.raises((TypeError, ValueError)):
            call()


def test_rows_that_do_not_fit_are_refused(lib):
    c = cache()
    rows = torch.zeros((3, 2, 64), dtype=torch.float16, device="cuda")
    for bad in (rows.float(), rows.cpu(), rows[:, :1], rows[..., :32], rows[0], rows.transpose(0, 2).contiguous().transpose(0, 2)):
        with pytest.raises((TypeError, ValueError)):
            lib.kv_append(bad, rows, *c)
        with pytest.raises((TypeError, ValueError)):
            lib.kv_append(rows, bad, *c)
    for bad in (rows.float(), rows.cpu(), rows[..., :32], rows[0]):
        with pytest.raises((TypeError, ValueError)):
            lib.kv_attention(bad, *c)
    with pytest.raises(ValueError):
        lib.kv_append(rows, rows.bfloat16(), *c)
    for bad in (dict(out=rows.bfloat16()), dict(out=rows[:2]), dict(lse=torch.zeros((3, 2), dtype=torch.float64, device="cuda")),
                dict(alibi_slopes=torch.zeros(3, device="cuda"))):
        with pytest.raises((TypeError, ValueError)):
            lib.kv_attention(rows, *c, **bad)
    with pytest.raises(lib.LLMInt8Error):
        lib.kv_attention(torch.zeros((3, 3, 64), dtype=torch.float16, device="cuda"), *c)  # heads % kv heads
    with pytest.raises(lib.LLMInt8Error):
        lib.kv_attention(rows, *c, scale=float("nan"))
    with pytest.raises(lib.LLMInt8Error):
        lib.kv_attention(rows, *c, workspace=torch.zeros(4096, dtype=torch.uint8, device="cuda"))
    odd = torch.zeros(3 * 2 * 64 + 8, dtype=torch.float16, device="cuda")[4:4 + 384].view(3, 2, 64)
    with pytest.raises(lib.LLMInt8Error):
        lib.kv_attention(odd, *c)  # not on a 16-byte boundary
    with pytest.raises(TypeError):
        lib.kv_read(*c, 3, dtype=torch.float32)


def test_norm_arguments_that_do_not_fit_are_refused(lib):
    x = torch.zeros((4, 64), dtype=torch.float16, device="cuda")
    w = torch.ones(64, dtype=torch.float16, device="cuda")
    for args, more in (((x.float(), w), {}), ((x.T, w), {}), ((x[0], w), {}), ((x, w[:32]), {}), ((x, w.bfloat16()), {}),
                       ((x, w.cpu()), {}), ((x, w, x[:2]), {}), ((x, w, x.bfloat16()), {}),
                       ((x, w), dict(threshold=6.0, Y=False)), ((x, w), dict(codes=x)),
                       ((x, w), dict(Y=x.bfloat16())), ((x, w), dict(row_absmax=torch.zeros(3, device="cuda"))),
                       ((x, w), dict(residual_out=x[:2]))):
        with pytest.raises((TypeError, ValueError)):
            lib.add_rmsnorm_quantize(*args, **more)
    with pytest.raises(lib.LLMInt8Error):
        lib.add_rmsnorm_quantize(x, w, eps=-1.0)
    with pytest.raises(lib.LLMInt8Error):
        lib.add_rmsnorm_quantize(torch.zeros((4, 60), dtype=torch.float16, device="cuda"), w[:60])
    codes = torch.zeros((4, 64), dtype=torch.int8, device="cuda")
    for args, more in (((x, w[:4]), {}), ((codes, w[:4]), {}), ((codes[:, :32], torch.ones(4, device="cuda")), {}),
                       ((codes, torch.ones(4, device="cuda")), dict(dtype=torch.float32))):
        with pytest.raises((TypeError, ValueError)):
            lib.dequantize_rowwise(*args, **more)
