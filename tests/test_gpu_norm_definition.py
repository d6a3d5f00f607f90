"""GPU checks of the norm's codes against the definition, value by value."""
import pytest
import torch

pytestmark = pytest.mark.gpu

EPS = 1e-5


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import int8_mixed_precision_rowwise_b200 as m
    return m


def draw(rows, cols, dtype, seed):
    """Hidden states with a few columns of large magnitude: a row's step is then near half of its values' rms."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x, res = (torch.randn((rows, cols), generator=g, device="cuda") for _ in range(2))
    w = 1 + 0.1 * torch.randn(cols, generator=g, device="cuda")
    at = torch.randperm(cols, generator=g, device="cuda")[:max(1, cols // 2048)]
    res[:, at] *= 40
    return x.to(dtype), res.to(dtype), w.to(dtype)


def codes_of(y, reciprocal_first):
    """(codes, absmax) of fp16 values, each step in fp32."""
    a = y.abs().amax(1).float()
    m = a.reciprocal() * 127 if reciprocal_first else torch.full_like(a, 127.0) / a
    m = torch.where(a > 0, m, torch.zeros_like(a))
    return torch.round(y.float() * m[:, None]).to(torch.int8), a


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("rows,cols", [(2048, 4096), (40, 40000)])
def test_codes_alone_take_the_reciprocal_first(lib, rows, cols, dtype):
    """Without Y the codes are torch.round(y * (127.0 / absmax)), which takes the reciprocal of absmax first. Values
    exactly between two codes tell it from 127 / absmax, the multiplier of the form with Y; the larger input holds
    some."""
    X, R, W = draw(rows, cols, dtype, seed=rows)
    full = lib.add_rmsnorm_quantize(X, W, R, eps=EPS)
    bare = lib.add_rmsnorm_quantize(X, W, R, eps=EPS, Y=False)
    want, absmax = codes_of(full[3], True)
    other, _ = codes_of(full[3], False)
    assert rows < 1000 or not torch.equal(want, other)
    assert torch.equal(bare[0], want) and torch.equal(bare[1], absmax)
    assert torch.equal(full[0], other) and torch.equal(full[1], absmax)
