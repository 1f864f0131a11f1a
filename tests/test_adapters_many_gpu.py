"""GPU tests of the adapter calls with more than 256 tokens of many adapters: the small
products take them in the adapters' order up to 1024 adapters and in their own beyond,
and the lists are made before them or beside them."""
import pytest

from test_adapters_gpu import adapters, check_both, indices, matrix

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def hqq():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import weight_only_quantization_b200 as m
    return m


@pytest.mark.parametrize("M", [256, 257, 700])
@pytest.mark.parametrize("count", [2, 40, 300, 1024, 1025])
@pytest.mark.parametrize("kind", ["mixed", "runs", "none"])
def test_many_tokens_of_many_adapters(hqq, M, count, kind):
    rows, cols = 136, 256
    q, W = matrix(hqq, rows, cols, 4, 64, seed=count)
    ad = adapters(hqq, count, 8, rows, cols, torch.float16, seed=count)
    check_both(hqq, q, W, ad, M, indices(M, count, kind, count), seed=count + M)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("count", [40, 1025])
def test_many_adapters_of_other_types(hqq, dtype, count):
    """Odd ranks and rows that are not whole 16-byte runs, all tokens on the last
    adapter but a few."""
    rows, cols, M = 77, 160, 500
    q, W = matrix(hqq, rows, cols, 3, 32, seed=count)
    ad = adapters(hqq, count, 13, rows, cols, dtype, seed=count)
    index = torch.full((M,), count - 1, dtype=torch.int32)
    index[::61] = torch.arange(len(index[::61]), dtype=torch.int32)
    check_both(hqq, q, W, ad, M, index, seed=3)
