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


def y_of(X, W, R=None, eps=EPS):
    """Y from the definition in 64 bits, rounded to fp32 and then to fp16. eps is an fp32 argument of the call."""
    h = X if R is None else (X.float() + R.float()).to(X.dtype)
    hd = h.double()
    eps = float(torch.tensor(eps, dtype=torch.float32))
    return (hd / torch.sqrt((hd * hd).mean(1, keepdim=True) + eps) * W.double()).float().half()


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("rows,cols", [(1, 16), (1, 4096), (3, 48), (2048, 4096), (700, 1040), (200, 14336),
                                       (300, 32768), (90, 32784), (20, 133136), (5000, 272)])
def test_y_and_codes_are_those_of_64_bits(lib, rows, cols, dtype):
    """Not one value of Y, and not one code of either form, is another than that of a norm in 64 bits. (The kernel's
    scale is off by about 2^-40 of itself: one value in 2^30 lies that near to where the rounding turns.)"""
    X, R, W = draw(rows, cols, dtype, seed=rows + cols)
    y = y_of(X, W, R)
    full = lib.add_rmsnorm_quantize(X, W, R, eps=EPS)
    assert torch.equal(full[3], y)
    assert torch.equal(full[0], codes_of(y, False)[0])
    bare = lib.add_rmsnorm_quantize(X, W, R, eps=EPS, Y=False)
    want, absmax = codes_of(y, True)
    assert torch.equal(bare[0], want) and torch.equal(bare[1], absmax)
    masked = lib.add_rmsnorm_quantize(X, W, R, eps=EPS, threshold=6.0)
    assert torch.equal(masked[3], y)
    out = (y.abs() >= 6.0).any(0)
    assert torch.equal(masked[0], codes_of(y.masked_fill(out[None], 0.0), False)[0])


@pytest.mark.parametrize("cols", [4096, 40000])
def test_y_of_rows_whose_squares_leave_fp32(lib, cols):
    """bf16 rows up to 1e37 and down to 1e-30 (with eps 0 all of them come out near 1), one of both sizes, and one
    that ends in a single value; then weights beyond 2^60 among ordinary ones, finite and not."""
    g = torch.Generator(device="cuda").manual_seed(cols)
    X = torch.randn((9, cols), generator=g, device="cuda").double()
    X = (X * 10.0 ** torch.tensor([37, 20, 18, 9, 0, -9, -20, -30, 0], device="cuda").double()[:, None]).to(torch.bfloat16)
    X[4, ::2] *= 1e15
    X[8] = 0
    X[8, -1] = 3e-30
    W = (1 + 0.1 * torch.randn(cols, generator=g, device="cuda")).to(torch.bfloat16)
    assert torch.isfinite(X).all()
    Y = lib.add_rmsnorm_quantize(X, W, eps=0.0)[3]
    assert torch.equal(Y, y_of(X, W, eps=0.0))
    assert bool((Y[:8].float().pow(2).mean(1) > 0.5).all())
    assert torch.equal(lib.add_rmsnorm_quantize(X, W, eps=EPS)[3], y_of(X, W))
    V = W.clone()
    V[5], V[6], V[cols - 9] = 1e30, 3e38, float("inf")
    Y = lib.add_rmsnorm_quantize(X[:8], V, eps=0.0)[3]
    want = y_of(X[:8], V, eps=0.0)
    assert torch.equal(torch.isnan(Y), torch.isnan(want)) and torch.equal(Y.nan_to_num(7.0), want.nan_to_num(7.0))


def test_y_of_fp16_rows_of_all_sizes(lib):
    """fp16 from its smallest subnormals to its largest values, with eps 0, and weights that are not finite."""
    g = torch.Generator(device="cuda").manual_seed(3)
    X = torch.randn((6, 4096), generator=g, device="cuda")
    X = (X * torch.tensor([2.0 ** -24, 2.0 ** -18, 2.0 ** -9, 1.0, 2.0 ** 9, 12000.0], device="cuda")[:, None]).half()
    W = (1 + 0.1 * torch.randn(4096, generator=g, device="cuda")).half()
    assert torch.equal(lib.add_rmsnorm_quantize(X, W, eps=0.0)[3], y_of(X, W, eps=0.0))
    W[8], W[4000], X[:, 8] = float("inf"), -60000.0, 1.0
    assert torch.equal(lib.add_rmsnorm_quantize(X, W, eps=EPS)[3], y_of(X, W))
