"""GPU tests of the layer products past the limits of one launch.  Rows that
overlap in memory (row r starts at element r of a buffer) make the operands long
without their bytes.  The values are -1, 0 and 1, as in test_gpu_linear_extents.py:
their sums are exact in any order."""
import pytest

from gpu_helpers import say, torch_mod
from test_gpu_linear_extents import signs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    torch = torch_mod()
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import optimizer_muon_step_amd as mu
    mu._lib.load()
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def sliding(rows, cols, kind, seed):
    """rows x cols, row r the elements r .. of one buffer."""
    return signs((rows + cols,), kind, seed).as_strided((rows, cols), (1, 1))


def test_copies_of_more_blocks_than_a_launch():
    """2^28 + 3 rows of 127 and 5, 64 and 4 GB as they are copied: 2^24 blocks and more."""
    torch = torch_mod()
    import optimizer_muon_step_amd as mu
    m, k, n, step = (1 << 28) + 3, 127, 5, 1 << 23
    x, w, dz = sliding(m, k, "bf16", 1), signs((k, n), "bf16", 2), sliding(m, n, "bf16", 3)
    say("[forward]")
    y = mu.muon_linear(x, w)  # sums of 127: exact in bf16
    for a in range(0, m, step):
        assert torch.equal(y[a:a + step].float(), x[a:a + step].float() @ w.float()), a
    del y
    say("[dw]")
    dw, db = torch.empty(k, n, device="cuda"), torch.empty(n, device="cuda")
    mu.muon_linear_dw(x, dz, dw, dbias=db)
    # random walks of 2^28 steps: about 2^13 on their way, a thousandth of 2^24
    want, want_db = torch.zeros(k, n, dtype=torch.float64, device="cuda"), torch.zeros(n, dtype=torch.float64, device="cuda")
    for a in range(0, m, step):
        grad = dz[a:a + step].float()
        want += (x[a:a + step].float().T @ grad).double()
        want_db += grad.double().sum(0)
    assert torch.equal(dw.double(), want) and torch.equal(db.double(), want_db)


def test_more_tiles_than_a_launch():
    """2^29 + 3 rows of 61 into 8: 64 x 64 tiles, the fastest for such rows, would be 2^32 threads."""
    torch = torch_mod()
    import optimizer_muon_step_amd as mu
    m, k, n, step = (1 << 29) + 3, 61, 8, 1 << 24
    x, w = sliding(m, k, "fp16", 4), signs((k, n), "fp16", 5)
    say("[forward]")
    y = mu.muon_linear(x, w)
    assert y.shape == (m, n)
    for a in range(0, m, step):
        assert torch.equal(y[a:a + step].float(), x[a:a + step].float() @ w.float()), a


@pytest.mark.parametrize("order", ["rows", "columns"])
@pytest.mark.parametrize("m,n", [(1, 20000), (32, 50264), (5, 16392), (1, 50257)])
def test_few_rows_of_many_columns(m, n, order):
    """More tiles than compute units: two to a unit."""
    torch = torch_mod()
    import optimizer_muon_step_amd as mu
    k = 768
    x, w = signs((m, k), "bf16", 6), signs((k, n), "bf16", 7) if order == "rows" else signs((n, k), "bf16", 7).T
    bias = signs((n,), "bf16", 8)
    want = (x.double() @ w.double()).float() + bias.float()
    assert torch.equal(mu.muon_linear(x, w, bias=bias, out_dtype=torch.float32), want)
    assert torch.equal(mu.muon_linear_dx(x, w.T, residual=bias.expand(m, n)), want.bfloat16())
