"""GPU checks of the residual + RMS norm + int8 quantization before a linear, and of the values of row codes."""
import numpy as np
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


def draw(rows, cols, dtype, seed, big=2):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rnd(*s):
        return torch.randn(s, generator=g, device="cuda")

    x, res, w = rnd(rows, cols), rnd(rows, cols), 1 + 0.2 * rnd(cols)
    at = torch.randperm(cols, generator=g, device="cuda")[:big]
    res[:, at] *= 30
    return x.to(dtype), res.to(dtype), w.to(dtype)


def check(lib, oracle_mod, X, W, R, t, out, residual=True):
    """h exact; Y within half a step of fp16 of the 64-bit norm of h, with the fp32 sum of squares (chains of at most
    100 additions, 100 * 2^-24 < 2^-17, of which the root halves) and three more roundings; codes, absmax and bitmap
    bit-exact for the Y that was stored."""
    codes, absmax, bitmap, Y, h = out
    h_ref = (X.float() + R.float()).to(X.dtype) if residual else X
    assert torch.equal(h, h_ref)
    hd = h_ref.double()
    y = hd * torch.rsqrt((hd * hd).mean(1, keepdim=True) + EPS) * W.double()
    if Y is not None:
        assert Y.dtype == torch.float16
        assert bool(((Y.double() - y).abs() <= y.abs() * (2.0 ** -11 + 2.0 ** -17) + 2.0 ** -25).all())
        y16 = Y.cpu().numpy()
        mask = oracle_mod.outlier_mask(y16, t) if t > 0 else np.zeros(y16.shape[1], np.uint8)
        c_ref, a_ref = oracle_mod.quantize_rowwise(y16, mask)
        assert np.array_equal(absmax.cpu().numpy().view(np.uint32), a_ref.view(np.uint32))
        assert np.array_equal(codes.cpu().numpy(), c_ref)
        if bitmap is not None:
            bits = np.unpackbits(bitmap.cpu().numpy().astype("<u4").view(np.uint8), bitorder="little")
            assert np.array_equal(bits[:y16.shape[1]], mask) and not bits[y16.shape[1]:].any()
        return int(mask.sum())
    a = y.abs().amax(1)
    assert bool(((absmax.double() - a).abs() <= a * (2.0 ** -11 + 2.0 ** -17)).all())
    return 0


@pytest.mark.parametrize("rows,cols", [(1, 16), (1, 4096), (2, 48), (7, 1040), (33, 4096), (32, 14336), (300, 2064),
                                       (149, 8192), (5, 32768), (3, 32784), (2, 133136), (1000, 256), (600, 4112)])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("t", [6.0, 0.0])
def test_norm_matches_definition(lib, oracle_mod, rows, cols, dtype, t):
    X, R, W = draw(rows, cols, dtype, seed=rows + cols)
    out = lib.add_rmsnorm_quantize(X, W, R, eps=EPS, threshold=t)
    n = check(lib, oracle_mod, X, W, R, t, out)
    assert t == 0 or rows < 30 or n > 0  # with many rows, surely
    ref = lib.quantize_rowwise(out[3], t)
    assert torch.equal(out[0], ref[0]) and torch.equal(out[1], ref[1])
    assert t == 0 or torch.equal(out[2], ref[2])


def test_norm_without_residual_and_without_y(lib, oracle_mod):
    X, R, W = draw(77, 1024, torch.float16, seed=3)
    out = lib.add_rmsnorm_quantize(X, W, eps=EPS, threshold=6.0)
    check(lib, oracle_mod, X, W, R, 6.0, out, residual=False)
    assert out[4] is X
    full = lib.add_rmsnorm_quantize(X, W, R, eps=EPS)
    bare = lib.add_rmsnorm_quantize(X, W, R, eps=EPS, Y=False)
    assert bare[3] is None and bare[2] is None
    assert torch.equal(full[0], bare[0]) and torch.equal(full[1], bare[1]) and torch.equal(full[4], bare[4])
    bitmap = torch.full((32,), -1, dtype=torch.int32, device="cuda")
    lib.add_rmsnorm_quantize(X, W, R, eps=EPS, outlier_bitmap=bitmap)
    assert not bitmap.any()  # no threshold: the bitmap is cleared


def test_norm_of_no_rows(lib):
    x = torch.empty((0, 64), dtype=torch.float16, device="cuda")
    codes, absmax, bitmap, Y, h = lib.add_rmsnorm_quantize(x, torch.ones(64, dtype=torch.float16, device="cuda"), x,
                                                           threshold=6.0)
    assert codes.shape == Y.shape == h.shape == (0, 64) and absmax.shape == (0,) and not bitmap.any()


@pytest.mark.parametrize("cols", [1024, 40000])
@pytest.mark.parametrize("into", ["X", "residual"])
def test_norm_in_place(lib, oracle_mod, cols, into):
    X, R, W = draw(50, cols, torch.bfloat16, seed=cols)
    a, b = X.clone(), R.clone()
    out = lib.add_rmsnorm_quantize(a, W, b, eps=EPS, threshold=6.0, residual_out=a if into == "X" else b)
    check(lib, oracle_mod, X, W, R, 6.0, out)


@pytest.mark.parametrize("rows", [4, 120, 900])
def test_rows_whose_largest_value_is_anothers_outlier_column(lib, oracle_mod, rows):
    """Columns that only one row takes over the threshold, while most rows have their maximum in them: those rows are
    coded again against the complete set. Every column of one band reaches it somewhere (more columns than one list
    holds), in the second shape."""
    for cols, width in ((512, 3), (8192, 1500)):
        g = torch.Generator(device="cuda").manual_seed(rows)
        X = torch.randn((rows, cols), generator=g, device="cuda") * 0.5
        X[:, :width] = 5.5 * torch.sign(X[:, :width])
        scale = torch.sqrt((X * X).mean(1, keepdim=True) + EPS)
        X = X * scale / scale.mean()
        for c in range(width):
            X[(c * 7) % rows, c] = 60.0
        X[rows // 2] = 0
        X = X.half()
        W, R = torch.ones(cols, device="cuda", dtype=torch.float16), torch.zeros_like(X)
        for _ in range(3):  # the workspace's sets are used in turn
            out = lib.add_rmsnorm_quantize(X, W, R, eps=EPS, threshold=3.0)
            assert check(lib, oracle_mod, X, W, R, 3.0, out) >= width // 2  # the zeroed row's are none
        assert not out[0][rows // 2].any() and out[1][rows // 2] == 0


def test_norm_shares_its_workspace_with_the_quantizer(lib, oracle_mod):
    """Calls of both, of several shapes, in turn on one workspace."""
    ws = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    for i, (rows, cols) in enumerate([(100, 4096), (3, 512), (64, 1024), (1, 4096), (200, 4096)]):
        X, R, W = draw(rows, cols, torch.float16, seed=i)
        out = lib.add_rmsnorm_quantize(X, W, R, eps=EPS, threshold=6.0, workspace=ws)
        check(lib, oracle_mod, X, W, R, 6.0, out)
        ref = lib.quantize_rowwise(out[3], 6.0, workspace=ws)
        assert torch.equal(out[0], ref[0]) and torch.equal(out[2], ref[2])
    assert lib.read_status(ws) == 0


def test_norm_captured_and_replayed(lib, oracle_mod):
    X, R, W = draw(40, 4096, torch.float16, seed=11)
    x, r = X.clone(), R.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        ws = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
        lib.add_rmsnorm_quantize(x, W, r, eps=EPS, threshold=6.0, workspace=ws)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = lib.add_rmsnorm_quantize(x, W, r, eps=EPS, threshold=6.0, workspace=ws)
        out2 = lib.add_rmsnorm_quantize(r, W, x, eps=EPS, threshold=6.0, workspace=ws)
    for seed in (12, 13, 14):
        X2, R2, _ = draw(40, 4096, torch.float16, seed=seed)
        x.copy_(X2)
        r.copy_(R2)
        graph.replay()
        torch.cuda.synchronize()
        check(lib, oracle_mod, X2, W, R2, 6.0, out)
        assert torch.equal(out[0], out2[0]) and torch.equal(out[2], out2[2])


def test_norm_of_large_and_small_values(lib):
    """Rows whose squares leave fp16's range, and rows that eps decides."""
    X = torch.full((3, 4096), 60000.0, device="cuda", dtype=torch.float16)
    X[1] = 1e-4
    X[2] = 0
    W = torch.ones(4096, device="cuda", dtype=torch.float16)
    codes, absmax, _, Y, _ = lib.add_rmsnorm_quantize(X, W, eps=EPS)
    assert torch.equal(Y[0], torch.ones_like(Y[0])) and bool((codes[0] == 127).all())
    x = float(X[1, 0])
    assert abs(float(Y[1, 0]) - x / (x * x + EPS) ** 0.5) <= 2.0 ** -11 * float(Y[1, 0]) + 2.0 ** -25
    assert not Y[2].any() and not codes[2].any() and absmax[2] == 0


@pytest.mark.parametrize("rows,cols", [(1, 16), (3, 4096), (1000, 272), (0, 64)])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_dequantize_rowwise(lib, rows, cols, dtype):
    """Two fp32 roundings (of absmax / 127 and of the product), then half a step of the type."""
    g = torch.Generator(device="cuda").manual_seed(cols)
    codes = torch.randint(-127, 128, (rows, cols), generator=g, device="cuda", dtype=torch.int8)
    absmax = torch.rand(rows, generator=g, device="cuda") * 10
    got = lib.dequantize_rowwise(codes, absmax, dtype=dtype)
    assert got.dtype == dtype and got.shape == codes.shape
    ref = codes.double() * absmax.double()[:, None] / 127
    half = torch.finfo(dtype).eps / 2
    assert bool(((got.double() - ref).abs() <= ref.abs() * (half + 2.0 ** -22) + 2.0 ** -25).all())


def test_norm_feeds_the_linear(lib):
    """Codes, absmax, outlier columns and Y into matmul_codes: what matmul_mixed makes of Y, up to the order of the
    fp32 sum over the outlier columns and so one step of fp16."""
    X, R, W = draw(48, 1024, torch.float16, seed=21)
    weight = (0.02 * torch.randn((512, 1024), device="cuda")).half()
    CB, SCB, _ = lib.quantize_rowwise(weight)
    codes, absmax, bitmap, Y, _ = lib.add_rmsnorm_quantize(X, W, R, eps=EPS, threshold=6.0)
    col, count, n = lib.find_outlier_cols(bitmap, 1024)
    assert n > 0
    got = lib.matmul_codes(codes, absmax, Y, CB, SCB, col, count, W_f16=weight)
    ref = lib.matmul_mixed(Y, CB, SCB, weight, 6.0)
    cols = col[:n].long()
    size = Y[:, cols].float().abs() @ weight[:, cols].float().abs().T
    assert bool(((got.float() - ref.float()).abs() <= 2.0 ** -10 * ref.float().abs() + 2.0 ** -20 * size + 2.0 ** -24).all())
