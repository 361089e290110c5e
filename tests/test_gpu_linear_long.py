"""GPU tests of the layer products over long reductions, in every tile, split
and not: every ring of slices is refilled many times, and every slice has to
arrive.  The bound of a sum of many terms would hide a lost slice, so the values are
-1, 0 and 1 and the results exact: a lost slice of 64 changes nine sums in ten
(tests/test_linear_limits.py), one that is read twice as many.  Which tile each
size takes is checked in tests/native/linear_limits_check.cpp."""
import pytest

from gpu_helpers import say, torch_mod
from linear_helpers import dtype
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


def stored(shape, kind, seed, order):
    return signs(shape, kind, seed) if order == "rows" else signs(shape[::-1], kind, seed).T


# rows, reduction, columns: each tile whole and split; the last ones through registers and through copies
LAYERS = [(8200, 1608, 1400), (1504, 20000, 1504), (4160, 1608, 2304), (2048, 20000, 1032), (2000, 1608, 1104), (520, 20000, 1000),
          (1500, 1608, 1304), (257, 30000, 520), (1000, 2312, 760), (64, 6408, 1600), (130, 1608, 1000), (130, 9000, 200),
          (20, 1608, 16000), (1, 4104, 2304), (700, 1001, 1003), (257, 30001, 513), (4097, 1609, 2311)]


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("order", ["rows", "columns"])
@pytest.mark.parametrize("shape", LAYERS, ids=str)
def test_layers(shape, order, kind):
    torch = torch_mod()
    import optimizer_muon_step_amd as mu
    m, k, n = shape
    say(f"[long] {shape} {order} {kind}")
    x, w, bias = signs((m, k), kind, 1), stored((k, n), kind, 2, order), signs((n,), "fp32", 3)
    want = (x.double() @ w.double()).float()
    assert torch.equal(mu.muon_linear(x, w, out_dtype=torch.float32), want)
    z = torch.empty(m, n, dtype=dtype(kind), device="cuda")
    res = signs((m, n), kind, 4)
    y = mu.muon_linear(x, w, bias=bias, act="relu", preact=z, residual=res)
    want += bias
    # each rounded once, from the exact value
    assert torch.equal(z, want.to(dtype(kind)))
    assert torch.equal(y, (want.clamp(min=0) + res.float()).to(dtype(kind)))
    del want, z, y
    # the same sizes as the gradient of an input
    w = stored((n, k), kind, 5, order)
    want = (x.double() @ w.double().T).float()
    pre = signs((m, n), kind, 6)
    assert torch.equal(mu.muon_linear_dx(x, w, act="relu", preact=pre, residual=res, out_dtype=dtype(kind)),
                       (torch.where(pre > 0, want, 0.0) + res.float()).to(dtype(kind)))
    assert torch.equal(mu.muon_linear_dx(x, w, out_dtype=torch.float32), want)


# reduction, rows and columns of the output as it is stored
GRADS = [(3000, 8200, 1400), (20000, 1400, 2040), (3000, 4160, 2304), (16384, 768, 2304), (4000, 2504, 1304), (3000, 2000, 1104),
         (4000, 1504, 1304), (30000, 520, 264), (2004, 333, 2001), (3001, 131, 300), (20001, 1001, 771)]


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("order", ["rows", "columns"])
@pytest.mark.parametrize("shape", GRADS, ids=str)
def test_grads(shape, order, kind):
    torch = torch_mod()
    import optimizer_muon_step_amd as mu
    m, rows, cols = shape
    k, n = (rows, cols) if order == "rows" else (cols, rows)
    say(f"[long dw] {shape} {order} {kind}")
    x, dz = signs((m, k), kind, 1), signs((m, n), kind, 2)
    want, want_db = x.double().T @ dz.double(), dz.double().sum(0)
    dw = torch.full((rows, cols), float("nan"), device="cuda")
    dw = dw if order == "rows" else dw.T
    db = torch.full((n,), float("nan"), device="cuda")
    mu.muon_linear_dw(x, dz, dw, dbias=db)
    assert torch.equal(dw.double(), want) and torch.equal(db.double(), want_db)
    mu.muon_linear_dw(x, dz, dw, dbias=db, accumulate=True)
    assert torch.equal(dw.double(), 2 * want) and torch.equal(db.double(), 2 * want_db)
    mu.muon_linear_dw(x, dz, dw)
    assert torch.equal(dw.double(), want)
