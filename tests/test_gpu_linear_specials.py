"""GPU tests of activations and their slopes at special values: zeros of either
sign, infinities and NaN, in whole tiles and at edges, against the oracle."""
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
