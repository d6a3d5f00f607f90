"""GPU checks of the GEMM called right behind the kernel that writes its weight operand: it starts while that kernel
runs, and must not load weight tiles before it is complete."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import int8_mixed_precision_rowwise_b200 as m
    return m


def product(A, B):
    """Exact: sums of at most 4096 products of 127 * 127 fit 53 bits."""
    return (A.double() @ B.double().T).to(torch.int32)


@pytest.mark.parametrize("M", [8, 24, 100, 700])
@pytest.mark.parametrize("N,K", [(4096, 1024), (20000, 4096)])
def test_weights_quantized_just_before(lib, M, N, K):
    g = torch.Generator(device="cuda").manual_seed(M)
    CX, SX, _ = lib.quantize_rowwise(torch.randn((M, K), generator=g, device="cuda").half())
    X = torch.zeros((M, K), dtype=torch.float16, device="cuda")
    col, count = torch.zeros(K, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    CB, SCB = torch.zeros((N, K), dtype=torch.int8, device="cuda"), torch.zeros(N, device="cuda")
    for i in range(4):
        W = torch.randn((N, K), generator=g, device="cuda").half()
        CB.fill_(i)
        torch.cuda.synchronize()
        lib.quantize_rowwise(W, 0.0, codes=CB, row_absmax=SCB)
        if i % 2:
            acc = lib.gemm_s8s8s32(CX, CB)
            assert torch.equal(acc, product(CX, CB))
        else:
            Y = lib.matmul_codes(CX, SX, X, CB, SCB, col, count)
            torch.cuda.synchronize()
            assert torch.equal(Y, lib.matmul_codes(CX, SX, X, CB, SCB, col, count))
            want = product(CX, CB).double() * SX.double()[:, None] * SCB.double() / (127 * 127)
            # fp32: the sum's conversion, the scale's and the product's roundings; then half a step of fp16
            assert bool(((Y.double() - want).abs() <= want.abs() * (2.0 ** -11 + 2.0 ** -21) + 2.0 ** -25).all())


@pytest.mark.parametrize("M", [16, 300])
def test_codes_of_the_norm_as_weights(lib, M):
    g = torch.Generator(device="cuda").manual_seed(M)
    A = torch.randint(-127, 128, (M, 4096), generator=g, device="cuda", dtype=torch.int8)
    w = torch.ones(4096, dtype=torch.float16, device="cuda")
    codes = torch.zeros((9000, 4096), dtype=torch.int8, device="cuda")
    for t in (0.0, 4.0):
        x = torch.randn((9000, 4096), generator=g, device="cuda").half()
        codes.zero_()
        torch.cuda.synchronize()
        lib.add_rmsnorm_quantize(x, w, threshold=t, codes=codes)
        acc = lib.gemm_s8s8s32(A, codes)
        assert bool(codes.any()) and torch.equal(acc, product(A, codes))
