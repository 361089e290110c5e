"""GPU tests of the layers' products and of dropout at the ends of what they
take: rows so far apart, or so many, that offsets pass 2^31 and 2^32, the widest matrices,
and distances between rows that the kernels read through a copy.

Equal values give equal bits whatever the distances between their rows, so far rows are compared
with near ones, which test_gpu_linear.py compares with the oracle.  At the largest sizes the
values are -1, 0 and 1: their sums stay below 2^24 and are exact in any order."""
import numpy as np
import pytest

from gpu_helpers import say, torch_mod
from linear_helpers import dtype, make
from oracle import linear_oracle as lo

pytestmark = pytest.mark.gpu
FAR = 32768  # elements from row to row


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


def far(t, ld=FAR):
    """A copy of a matrix with rows ld elements apart; what lies between is not set."""
    torch = torch_mod()
    buf = torch.empty(t.shape[0] * ld, dtype=t.dtype, device="cuda")
    view = buf.as_strided(t.shape, (ld, 1))
    view.copy_(t)
    return view


def signs(shape, kind, seed, zeros=0.5):
    """-1, 0 and 1."""
    torch = torch_mod()
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = torch.empty(shape, dtype=dtype(kind), device="cuda").uniform_(-1.0, 1.0, generator=g)
    # rounding to 1 or -1 beyond `zeros`, to 0 within
    return torch.where(t.abs() >= zeros, t.sign(), torch.zeros((), dtype=t.dtype, device="cuda"))


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
def test_far_rows_forward(kind):
    """70001 rows of 64 KB: x, y, z and the residual each reach past 4 GB."""
    torch = torch_mod()
    import optimizer_muon_step_amd as mu
    rng = np.random.default_rng(1)
    x, w, res = make(rng, (70001, 72), kind), make(rng, (72, 88), kind), make(rng, (70001, 88), kind)
    args = dict(act="gelu", dropout=0.1, rng=(5, 6), site=7)
    z = torch.empty_like(res)
    y = mu.muon_linear(x, w, residual=res, preact=z, **args)
    far_y, far_z = far(res), far(res)
    say("[far forward]")
    mu.muon_linear(far(x), w, residual=far(res), preact=far_z, out=far_y, **args)
    assert torch.equal(y, far_y) and torch.equal(z, far_z)
    mu.muon_linear(far(x), w, residual=far_z, out=far_z, **args)
    assert torch.equal(mu.muon_linear(x, w, residual=z, **args), far_z)


def test_far_rows_backward():
    torch = torch_mod()
    import optimizer_muon_step_amd as mu
    rng = np.random.default_rng(2)
    m, k, n = 70001, 80, 64
    x, dz, w = make(rng, (m, k), "bf16"), make(rng, (m, n), "bf16"), make(rng, (k, n), "fp32")
    args = dict(act="relu2", dropout=0.25, rng=(1, 2))
    say("[far dx]")
    far_z = far(x)
    mu.muon_linear_dx(far(dz), w, preact=far_z, out=far_z, **args)
    assert torch.equal(mu.muon_linear_dx(dz, w, preact=x, **args), far_z)
    say("[far dw]")
    dw, far_dw, db, far_db = (torch.empty(s, device="cuda") for s in [(k, n), (k, n), (n,), (n,)])
    mu.muon_linear_dw(x, dz, dw, dbias=db)
    mu.muon_linear_dw(far(x), far(dz), far_dw, dbias=far_db)
    assert torch.equal(dw, far_dw) and torch.equal(db, far_db)


@pytest.mark.parametrize("order", ["rows", "columns"])
def test_far_rows_of_weights(order):
    """A weight of 70001 rows that lie 64 or 128 KB apart, and its gradient."""
    torch = torch_mod()
    import optimizer_muon_step_amd as mu
    rng = np.random.default_rng(3)
    m, rows, cols = 40, 70001, 72
    w = make(rng, (rows, cols), "bf16")
    wide, narrow = make(rng, (m, rows), "bf16"), make(rng, (m, cols), "bf16")
    dw, far_dw = torch.zeros(rows, cols, device="cuda"), far(torch.zeros(rows, cols, device="cuda"))
    far_w = far(w)
    say(f"[far weight] {order}")
    if order == "rows":
        x, dz = wide, narrow
    else:
        x, dz, w, far_w, dw, far_dw = narrow, wide, w.T, far_w.T, dw.T, far_dw.T
    assert torch.equal(mu.muon_linear(x, w), mu.muon_linear(x, far_w))
    assert torch.equal(mu.muon_linear_dx(dz, w), mu.muon_linear_dx(dz, far_w))
    for accumulate in (False, True):
        mu.muon_linear_dw(x, dz, dw, accumulate=accumulate)
        mu.muon_linear_dw(x, dz, far_dw, accumulate=accumulate)
        assert torch.equal(dw, far_dw)


def test_rows_too_far_for_direct_loads():
    """More than 2^22 elements apart: read through registers, or, of a large product, through a copy."""
    torch = torch_mod()
    import optimizer_muon_step_amd as mu
    ld = (1 << 22) + 8
    for m, k, n in ((70, 72, 88), (8192, 768, 3072)):
        x, w, dz = signs((m, k), "bf16", 1), signs((k, n), "bf16", 2), signs((m, n), "bf16", 3)
        far_w = far(w, ld)
        say(f"[too far] {m} {k} {n}")
        assert torch.equal(mu.muon_linear(x, w, out_dtype=torch.float32), mu.muon_linear(x, far_w, out_dtype=torch.float32))
        assert torch.equal(mu.muon_linear_dx(dz, w, out_dtype=torch.float32), mu.muon_linear_dx(dz, far_w, out_dtype=torch.float32))
        del far_w
    m, k, n = 515, 72, 88
    x, w, dz = signs((m, k), "fp16", 4), signs((k, n), "fp16", 5), signs((m, n), "fp16", 6)
    far_x, far_dz = far(x, ld), far(dz, ld)
    assert torch.equal(mu.muon_linear(x, w), mu.muon_linear(far_x, w))
    dw, far_dw = torch.empty(k, n, device="cuda"), far(torch.empty(k, n, device="cuda"), ld)
    mu.muon_linear_dw(x, dz, dw)
    mu.muon_linear_dw(far_x, far_dz, far_dw)
    assert torch.equal(dw, far_dw)


@pytest.mark.parametrize("order", ["rows", "columns"])
def test_widest_inputs(order):
    """2^22 inputs: a reduction as long as they come, and as wide an output of the backward pass."""
    torch = torch_mod()
    import optimizer_muon_step_amd as mu
    m, k, n = 70, 1 << 22, 40
    x, dz = signs((m, k), "bf16", 1), signs((m, n), "bf16", 2)
    w = signs((k, n), "bf16", 3) if order == "rows" else signs((n, k), "bf16", 3).T
    say(f"[widest inputs] {order}")
    want = torch.zeros(m, n, dtype=torch.float32, device="cuda")
    for c in range(0, k, 1 << 19):
        want += x[:, c:c + (1 << 19)].float() @ w[c:c + (1 << 19)].float()
    assert want.abs().max() < 2 ** 24 and want.abs().max() > 100
    assert torch.equal(mu.muon_linear(x, w, out_dtype=torch.float32), want)
    assert torch.equal(mu.muon_linear_dx(dz, w, out_dtype=torch.float32), dz.float() @ w.float().T)
    dw = torch.empty(k, n, device="cuda") if order == "rows" else torch.empty(n, k, device="cuda").T
    mu.muon_linear_dw(x, dz, dw)
    assert torch.equal(dw, x.float().T @ dz.float())


def test_most_rows():
    """2^28 + 3 rows, 4 GB of them."""
    torch = torch_mod()
    import optimizer_muon_step_amd as mu
    m, k, n = (1 << 28) + 3, 8, 8
    x, w, dz = signs((m, k), "bf16", 4), signs((k, n), "bf16", 5), signs((m, n), "bf16", 6)
    say("[most rows]")
    y = mu.muon_linear(x, w)  # sums of 8: exact in bf16
    dw, db = torch.empty(k, n, device="cuda"), torch.empty(n, device="cuda")
    mu.muon_linear_dw(x, dz, dw, dbias=db)
    # random walks of 2^28 steps: about 2^13 on their way, a thousandth of 2^24
    want_dw, want_db = torch.zeros(k, n, dtype=torch.float64, device="cuda"), torch.zeros(n, dtype=torch.float64, device="cuda")
    for a in range(0, m, 1 << 24):
        part, grad = x[a:a + (1 << 24)], dz[a:a + (1 << 24)].double()
        assert torch.equal(y[a:a + (1 << 24)].float(), part.float() @ w.float()), a
        want_db += grad.sum(0)
        want_dw += part.double().T @ grad
    assert torch.equal(dw.double(), want_dw) and torch.equal(db.double(), want_db)


@pytest.mark.parametrize("rows,cols", [(1, (1 << 32) + 21), (2, (1 << 31) + 13)])
def test_dropout_past_32_bits(rows, cols):
    """8 GB in place; the mask is compared around the borders and at the ends."""
    torch = torch_mod()
    import optimizer_muon_step_amd as mu
    seed, step, site, p = 0x1234567890, 11, 3, 0.25
    x = torch.full((rows, cols), 2.0, dtype=torch.bfloat16, device="cuda")
    say(f"[dropout] {rows} x {cols}")
    mu.muon_dropout(x, p, (seed, step), site=site, out=x)
    ends = [0, 1 << 30, 1 << 31, 1 << 32, cols]
    for row in range(rows):
        for end in ends:
            lo_col, hi_col = max(0, end - 4096) // 8 * 8, min(cols, end + 4096)
            if lo_col >= hi_col:
                continue
            groups = np.arange(lo_col // 8, (hi_col + 7) // 8, dtype=np.uint64)
            counter = [groups.astype(np.uint32), np.full(len(groups), row, np.uint32), np.full(len(groups), site, np.uint32),
                       np.full(len(groups), step, np.uint32)]
            words = lo.philox(counter, (seed & 0xffffffff, seed >> 32))
            bits = np.stack([(w >> s) & 0xffff for w in words for s in (0, 16)], axis=-1).reshape(-1)[:hi_col - lo_col]
            want = np.where(bits >= lo.border(p), 2.0 * 65536.0 / (65536.0 - lo.border(p)), 0.0)
            got = x[row, lo_col:hi_col].double().cpu().numpy()
            assert np.array_equal(got != 0, want != 0), (row, end)
            assert np.abs(got - want).max() <= 2.0 * 4 / 3 * 2.0 ** -8, (row, end)
    # every element was visited: 2 is neither 0 nor 8/3
    for a in range(0, cols, 1 << 28):
        part = x[:, a:a + (1 << 28)]
        assert not bool((part == 2.0).any()), a


def test_dropout_on_streams_with_counters():
    """Calls on streams of their own that read their numbers from the GPU, the
    numbers set on the same stream just before."""
    torch = torch_mod()
    import optimizer_muon_step_amd as mu
    x = [torch.randn(3001, 515 + i, device="cuda") for i in range(4)]
    want = [mu.muon_dropout(t, 0.3, (9, i + 1), site=i) for i, t in enumerate(x)]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in x], []
    for i, (t, s) in enumerate(zip(x, streams)):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            state = torch.zeros(2, dtype=torch.int64, device="cuda")
            state[0] = 9
            state[1:].add_(i + 1)
            got.append((mu.muon_dropout(t, 0.3, state, site=i), state))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, (b, _) in zip(want, got))
