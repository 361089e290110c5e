"""GPU tests of dropout from a counter (muon_dropout, and the mask in the
products' epilogues) against the oracle: the mask exactly, the values within
the bounds of linear_helpers."""
import numpy as np
import pytest

from gpu_helpers import say, torch_mod
from linear_helpers import U, check, dtype, make, outside_unchanged, slope_bound, stored, values
from oracle import linear_oracle as lo

pytestmark = pytest.mark.gpu
NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    torch = torch_mod()
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import optimizer_muon_step_amd as mu
    mu._lib.load()
    yield
    torch.cuda.synchronize()


def check_dropout(mu, x, p, rng, site=0, act=None, preact=None, residual=None, out=None, out_kind=None):
    seed, step = rng if isinstance(rng, tuple) else (int(v) for v in rng.cpu())
    rows = x.numel() // max(1, x.shape[-1] if x.dim() else 1)
    cols = x.shape[-1] if x.dim() else 1
    xv = values(x).reshape(rows, cols)
    zv = None if preact is None else values(preact).reshape(rows, cols)
    rv = None if residual is None else values(residual).reshape(rows, cols)
    kind = {str(dtype(k)): k for k in ("fp32", "bf16", "fp16")}
    got = mu.muon_dropout(x, p, rng, site=site, act=act, preact=preact, residual=residual, out=out,
                          out_dtype=None if out_kind is None else dtype(out_kind))
    assert got.shape == x.shape
    factor = lo.keep_factor(rows, cols, p, seed, step, site)
    want = lo.through(xv, act, zv, factor, rv)
    v, err = np.abs(xv), 0.0
    if act is not None:
        s = np.abs(lo.slope(zv, act))
        err = v * (slope_bound(zv, act) + U * s)
        v = v * s
    err = factor * (err + 2 * U * (v + err))
    if rv is not None:
        err = err + U * (np.abs(want) + err)
    got_kind = kind[str(got.dtype)]
    check(values(got).reshape(rows, cols), want, stored(err, want, got_kind), f"dropout {tuple(x.shape)}", got_kind)
    if residual is None and act is None:
        assert np.array_equal(values(got).reshape(rows, cols) != 0, (factor != 0) & (xv != 0)), "mask"
    return got


COLS = [1, 2, 7, 8, 9, 15, 16, 31, 64, 100, 768, 1000, 8190, 8192, 8193, 8200, 20001]


@pytest.mark.parametrize("kind", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("cols", COLS)
def test_shapes(cols, kind):
    import optimizer_muon_step_amd as mu
    say(f"[dropout] {cols} {kind}")
    for rows in (1, 3, 130):
        x = make(np.random.default_rng(cols + rows), (rows, cols), kind, fill=NAN)
        check_dropout(mu, x, 0.1, (rows * 2 ** 40 + cols, 2 ** 32 - rows), site=2 ** 32 - 1)


@pytest.mark.parametrize("kind,out", [("fp32", "fp32"), ("bf16", "bf16"), ("fp16", "fp16"), ("bf16", "fp32"), ("fp32", "bf16"),
                                      ("fp16", "fp32"), ("fp16", "bf16")])
@pytest.mark.parametrize("act", [None, "gelu", "relu", "relu2"])
@pytest.mark.parametrize("residual", [False, True])
def test_parts_and_types(kind, out, act, residual):
    import optimizer_muon_step_amd as mu
    rng = np.random.default_rng(31)
    for shape in ((65, 96), (37, 131)):
        x = make(rng, shape, kind)
        pre = make(rng, shape, kind, 2.0) if act else None
        check_dropout(mu, x, 0.4, (7, 1), 3, act, pre, make(rng, shape, out) if residual else None, out_kind=out)
        check_dropout(mu, x, 0.0, (7, 1), 3, act, pre, make(rng, shape, out) if residual else None, out_kind=out)


@pytest.mark.parametrize("p", [0.0, 1e-6, 7.6e-6, 1.6e-5, 0.5, 0.9, 0.99999, 1 - 2.0 ** -24])
def test_probabilities(p):
    import optimizer_muon_step_amd as mu
    x = make(np.random.default_rng(32), (400, 512), "fp32")
    check_dropout(mu, x, p, (2 ** 64 - 1, 2 ** 32 - 1))


def test_the_share_that_is_kept():
    """2^24 elements at p = 0.1: the share kept is within 6 standard deviations,
    and neighbours are kept independently of one another (as their products'
    mean shows, within 6 of its own)."""
    torch = torch_mod()
    import optimizer_muon_step_amd as mu
    x = torch.ones(4096, 4096, dtype=torch.bfloat16, device="cuda")
    t = lo.border(0.1)
    keep, n = 1 - t / 65536, 2.0 ** 24
    k = (mu.muon_dropout(x, 0.1, (1, 1)) != 0).double()
    assert abs(k.mean().item() - keep) < 6 * (keep * (1 - keep) / n) ** 0.5
    others = [k.roll(1, 0), k.roll(1, 1), (mu.muon_dropout(x, 0.1, (1, 2)) != 0).double(),
              (mu.muon_dropout(x, 0.1, (2, 1)) != 0).double(), (mu.muon_dropout(x, 0.1, (1, 1), site=1) != 0).double()]
    for other in others:
        assert abs((k * other).mean().item() - keep * keep) < 6 * (keep ** 2 * (1 - keep ** 2) / n) ** 0.5


def test_layouts():
    torch = torch_mod()
    import optimizer_muon_step_amd as mu
    rng = np.random.default_rng(33)
    for offset, gap in ((0, 3), (1, 0), (5, 11), (8, 64)):
        x = make(rng, (40, 99), "bf16", offset=offset, gap=gap, fill=NAN)
        out = make(rng, (40, 99), "fp32", offset=offset, gap=gap, fill=7.0)
        res = make(rng, (40, 99), "fp32", offset=gap, gap=offset, fill=NAN)
        check_dropout(mu, x, 0.2, (5, 6), residual=res, out=out)
        assert outside_unchanged(out, 7.0)
    x = torch.randn(2, 3, 5, 24, device="cuda")
    flat = check_dropout(mu, x.view(30, 24), 0.3, (9, 9))
    assert torch.equal(check_dropout(mu, x, 0.3, (9, 9)).view(30, 24), flat)
    check_dropout(mu, torch.randn(100_003, device="cuda"), 0.3, (9, 9))     # one row
    check_dropout(mu, torch.randn((), device="cuda"), 0.3, (9, 9))
    check_dropout(mu, torch.randn(24, device="cuda").expand(7, 24), 0.3, (9, 9))
    assert mu.muon_dropout(torch.empty(0, 5, device="cuda"), 0.3, (9, 9)).shape == (0, 5)
    assert mu.muon_dropout(torch.empty(5, 0, device="cuda"), 0.3, (9, 9)).shape == (5, 0)
    y = torch.randn(37, 131, device="cuda")
    want = mu.muon_dropout(y, 0.3, (9, 9))
    assert mu.muon_dropout(y, 0.3, (9, 9), out=y) is y and torch.equal(y, want)


def test_dropped_specials_vanish():
    torch = torch_mod()
    import optimizer_muon_step_amd as mu
    kept = torch.from_numpy(lo.keep_factor(64, 99, 0.5, 3, 4, 5) != 0).cuda()
    for bad in (NAN, float("inf")):
        x = torch.full((64, 99), bad, device="cuda")
        y = mu.muon_dropout(x, 0.5, (3, 4), site=5)
        assert not torch.isfinite(y[kept]).any() and (y[~kept] == 0).all()
        y = mu.muon_dropout(torch.ones_like(x), 0.5, (3, 4), site=5, act="gelu", preact=torch.full_like(x, NAN),
                            residual=torch.ones_like(x))
        assert torch.isnan(y[kept]).all() and (y[~kept] == 1).all()


def test_one_mask_in_every_operator():
    """Forward in the product's epilogue, backward by itself and in the gradient
    product's epilogue: the mask is the same one."""
    torch = torch_mod()
    import optimizer_muon_step_amd as mu
    drop = dict(rng=(77, 5), site=9)
    for n in (136, 131):
        ones, eye = torch.ones(70, n, dtype=torch.bfloat16, device="cuda"), torch.eye(n, dtype=torch.bfloat16, device="cuda")
        want = mu.muon_dropout(ones, 0.3, **drop) != 0
        assert torch.equal(mu.muon_linear(ones, eye, dropout=0.3, **drop) != 0, want)
        assert torch.equal(mu.muon_linear_dx(ones, eye, dropout=0.3, **drop) != 0, want)
        state = torch.tensor([77, 5], dtype=torch.int64, device="cuda")
        assert torch.equal(mu.muon_linear(ones, eye, dropout=0.3, rng=state, site=9) != 0, want)
        assert torch.equal(mu.muon_dropout(ones, 0.3, state, site=9) != 0, want)
    # seeds and steps beyond the signed ranges
    big = torch.tensor([2 ** 63 + 11 - 2 ** 64, 2 ** 32 - 3], dtype=torch.int64, device="cuda")
    x = torch.ones(33, 47, device="cuda")
    assert torch.equal(mu.muon_dropout(x, 0.3, big), mu.muon_dropout(x, 0.3, (2 ** 63 + 11, 2 ** 32 - 3)))


def test_captured_with_a_counter_on_the_gpu():
    """A captured dropout reads its step at every replay."""
    torch = torch_mod()
    import optimizer_muon_step_amd as mu
    x = torch.randn(300, 131, device="cuda")
    state = torch.tensor([123, 0], dtype=torch.int64, device="cuda")
    y = torch.empty_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mu.muon_dropout(x, 0.3, state, site=2, out=y)
        state[1:].add_(1)
    seen = []
    for step in range(4):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, mu.muon_dropout(x, 0.3, (123, step), site=2)), step
        seen.append(y.clone())
    assert not any(torch.equal(a, b) for i, a in enumerate(seen) for b in seen[:i])
