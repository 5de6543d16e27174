"""The experts' products and the matrix memory through the C entry points, where rows, results, matrices and scratch
lie further than 32 bits from the start of their arrays."""
import pytest
import torch

from laplace_matvec_amd import laplex as lx

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def give_memory_back():
    yield
    torch.cuda.empty_cache()


def ok(status):
    torch.cuda.synchronize()
    assert status == 0, lx.load().laplex_last_error()


def test_many_rows_of_no_sequence(gpu):
    """2^25 rows before the only sequence, 512 heads of one value: 2^31 places of a workgroup's column block."""
    outside, rows, heads = 1 << 25, 64, 512
    n = outside + rows
    one = torch.ones(n, 1, dtype=torch.bfloat16, device=gpu)
    g = torch.zeros(n, heads, dtype=torch.bfloat16, device=gpu)  # 34 GB, and y
    y = torch.ones(n, heads, dtype=torch.bfloat16, device=gpu)
    at = torch.tensor([outside, n], dtype=torch.int32, device=gpu)
    p = lambda t: t.data_ptr()  # noqa: E731
    lib = lx.load()
    assert lib.laplex_attend_workspace(n, 1, heads, 1, 1, 1, 1, 1, 1, 0) == 0
    ok(lib.laplex_attend(n, 1, p(at), heads, 1, 1, 1, 1, 1, 1, 1, 1.0, p(one), 1, p(one), 1, p(one), 1, p(g), heads, None,
                         p(y), heads, None, None, None, 0, torch.cuda.current_stream().cuda_stream))
    assert not y[:outside].any()
    count = torch.arange(1, rows + 1, device=gpu).view(rows, 1).expand(rows, heads)
    assert torch.equal(y[outside:].float(), count.float())
