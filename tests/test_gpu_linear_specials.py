"""GPU tests of the layers' products and dropout at special values: activations
and slopes at zeros of either sign, infinities and NaN, in whole tiles and at edges,
against the oracle; subnormal operands; every value of a 16-bit type."""
import numpy as np
import pytest

from gpu_helpers import torch_mod
from linear_helpers import dtype
from oracle import linear_oracle as lo

pytestmark = pytest.mark.gpu
SPECIAL = [0.0, -0.0, float("inf"), -float("inf"), float("nan"), 1.0, -1.0, 2.0 ** -14, -(2.0 ** -14)]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    torch = torch_mod()
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import optimizer_muon_step_amd as mu
    mu._lib.load()
    yield
    torch.cuda.synchronize()


def same(got, want):
    """Equal, NaN where it is NaN."""
    return np.array_equal(got.double().cpu().numpy(), want, equal_nan=True)


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("act", ["relu", "relu2"])
@pytest.mark.parametrize("m,n", [(64, 128), (70, 131), (4160, 2304)])
def test_relu(m, n, act, kind):
    """Exact: the products are of ones and twos, the slopes small."""
    torch = torch_mod()
    import optimizer_muon_step_amd as mu
    z = torch.tensor(SPECIAL, dtype=dtype(kind), device="cuda").repeat(-(-m * n // len(SPECIAL)))[:m * n].view(m, n)
    zv = z.double().cpu().numpy()
    ones, eye = torch.ones(m, 8, dtype=dtype(kind), device="cuda"), torch.zeros(n, 8, dtype=dtype(kind), device="cuda")
    eye[:, 0] = 2.0
    with np.errstate(over="ignore", invalid="ignore"):
        want = 2.0 * lo.slope(zv, act)  # 2^-13 and its like are exact in every type
        p, seed, step, site = 0.5, 99, 3, 4
        factor = lo.keep_factor(m, n, p, seed, step, site)
        dropped = np.where(factor == 0, 0.0, want * 2.0)
    for out in (kind, "fp32"):
        args = dict(act=act, preact=z, out_dtype=dtype(out))
        assert same(mu.muon_linear_dx(ones, eye, **args), want)
        assert same(mu.muon_linear_dx(ones, eye, dropout=p, rng=(seed, step), site=site, **args), dropped)
        twos = torch.full_like(z, 2.0)
        assert same(mu.muon_dropout(twos, 0.0, None, **args), want)
        assert same(mu.muon_dropout(twos, p, (seed, step), site=site, **args), dropped)
    # forward: z comes from the bias
    bias = z[0].clone()
    want = np.broadcast_to(lo.act(bias.double().cpu().numpy(), act), (m, n))
    x, w = torch.zeros(m, 8, dtype=dtype(kind), device="cuda"), torch.zeros(8, n, dtype=dtype(kind), device="cuda")
    assert same(mu.muon_linear(x, w, bias=bias, act=act, out_dtype=torch.float32), want)


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("m,k,n", [(64, 128, 64), (70, 75, 131), (4160, 136, 2304), (1, 4096, 72), (8200, 72, 1400)])
def test_subnormal_operands(m, k, n, kind):
    """Gradients without enough of a loss scale: whole multiples of the type's smallest number, by -1, 0
    and 1 in fp16 and by 2^100 in bf16, whose sums are exact."""
    torch = torch_mod()
    import optimizer_muon_step_amd as mu
    gen = torch.Generator(device="cuda").manual_seed(m)
    whole = lambda *s: torch.randint(-8, 9, s, generator=gen, device="cuda").double()  # noqa: E731
    tiny, big = (2.0 ** -24, 1.0) if kind == "fp16" else (2.0 ** -133, 2.0 ** 100)
    sign = lambda *s: torch.randint(-1, 2, s, generator=gen, device="cuda").double() * big  # noqa: E731
    t = dtype(kind)
    x, w = (whole(m, k) * tiny).to(t), sign(k, n)
    assert bool((x.double() != 0).any()) and x.abs().max().double() == 8 * tiny
    want = x.double() @ w
    for wide in (w.to(t), w.float(), w.T.contiguous().to(t).T):
        assert torch.equal(mu.muon_linear(x, wide, out_dtype=torch.float32).double(), want)
    assert torch.equal(mu.muon_linear_dx(x, w.to(t).T.contiguous(), out_dtype=torch.float32).double(), want)
    if kind == "fp16":  # a subnormal output, and weights that round to subnormals
        res = torch.zeros(m, n, dtype=t, device="cuda")
        assert torch.equal(mu.muon_linear(x, w.to(t), residual=res), want.to(t))
        wide, up = whole(k, n).float() * 2.0 ** -25, sign(m, k).to(t)
        assert torch.equal(mu.muon_linear(up, wide, out_dtype=torch.float32).double(), up.double() @ wide.half().double())
    dz = sign(m, n).to(t)
    dw = torch.empty(k, n, device="cuda")
    mu.muon_linear_dw(x, dz, dw)
    assert torch.equal(dw.double(), x.double().T @ dz.double())


@pytest.mark.parametrize("kind,tiny", [("fp32", 2.0 ** -149), ("bf16", 2.0 ** -133), ("fp16", 2.0 ** -24)])
def test_subnormals_through_dropout(kind, tiny):
    """Twice a subnormal, and a subnormal added to another, are exact."""
    torch = torch_mod()
    import optimizer_muon_step_amd as mu
    for m, n in ((64, 96), (37, 131)):
        v = np.random.default_rng(n).integers(-6, 7, (2, m, n)) * tiny
        x, res = (torch.from_numpy(a).to(dtype(kind)).cuda() for a in v)
        factor = lo.keep_factor(m, n, 0.5, 8, 9, 0)
        assert same(mu.muon_dropout(x, 0.5, (8, 9)), np.where(factor == 0, 0.0, 2 * v[0]))
        assert same(mu.muon_dropout(x, 0.5, (8, 9), residual=res), np.where(factor == 0, 0.0, 2 * v[0]) + v[1])


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("how", ["direct", "registers", "copy"])
def test_every_value(how, kind):
    """All 65536 bit patterns, times 1: the values they stand for, as operands that are read
    where they lie, through registers and through a copy, forward and as a weight's gradient."""
    torch = torch_mod()
    import optimizer_muon_step_amd as mu
    t = dtype(kind)
    every = torch.arange(65536, device="cuda").to(torch.int16).view(t)
    width = 1 if how == "copy" else 8
    x = torch.zeros(65536 * width + 8, dtype=t, device="cuda")[how == "registers":][:65536 * width].view(65536, width)
    x[:, 0] = every
    w = torch.zeros(width, 8, dtype=t, device="cuda")
    w[0] = 1.0
    want = every.double().cpu().numpy()
    for out in (kind, "fp32"):
        y = mu.muon_linear(x, w, out_dtype=dtype(out))
        assert same(y, np.broadcast_to(want[:, None], (65536, 8)))
    # the same values as what is summed, one to a row: x^T of one row of them
    row = x[:, 0].clone().view(1, -1)
    one = torch.ones(1, width, dtype=t, device="cuda")
    dw = torch.empty(65536, width, device="cuda")
    mu.muon_linear_dw(row, one, dw)
    assert same(dw, np.broadcast_to(want[:, None], (65536, width)))
