"""GPU tests of the layers' products (muon_linear, muon_linear_dx,
muon_linear_dw) against the oracle in fp64, with the bounds of linear_helpers."""
import numpy as np
import pytest

from gpu_helpers import say, torch_mod
from linear_helpers import U, act_bound, check, dtype, make, outside_unchanged, slope_bound, stored, values
from oracle import linear_oracle as lo

pytestmark = pytest.mark.gpu

SHAPES = [(1, 1, 1), (1, 8, 8), (3, 5, 7), (2, 64, 64), (33, 64, 40), (64, 72, 128), (128, 128, 128), (129, 136, 257),
          (130, 200, 1000), (257, 768, 96), (300, 1001, 264), (1000, 264, 520), (5, 2048, 72)]
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


def _weight(w, kind):
    """Values of a weight as the products take it."""
    return values(w.to(dtype(kind)))


def _product_error(a, b):
    return a.shape[1] * 2.0 ** -23 * (np.abs(a) @ np.abs(b))


def check_linear(mu, x, w, kind, out="same", bias=None, act=None, drop=None, residual=None, keep=False, y=None, what=""):
    """One muon_linear call against the oracle.  drop: (p, seed, step, site)."""
    torch = torch_mod()
    out_kind = kind if out == "same" else out
    xv, wv = values(x).reshape(-1, x.shape[-1]), _weight(w, kind)
    rows, cols = xv.shape[0], wv.shape[1]
    res = None if residual is None else values(residual).reshape(rows, cols)
    bv = None if bias is None else values(bias)
    factor = None if drop is None else lo.keep_factor(rows, cols, *drop[:4])
    preact = torch.full((*x.shape[:-1], cols), NAN, dtype=x.dtype, device="cuda") if keep else None
    got = mu.muon_linear(x, w, bias=bias, act=act, residual=residual, preact=preact, out=y, out_dtype=dtype(out_kind),
                         **({} if drop is None else dict(dropout=drop[0], rng=(drop[1], drop[2]), site=drop[3])))
    want, z = lo.linear(xv, wv, bv, act, factor, res)
    err = _product_error(xv, wv)
    if bias is not None:
        err = err + U * (np.abs(z) + err)
    if keep:
        check(values(preact).reshape(rows, cols), z, stored(err, z, kind), what + " preact", kind)
    err = act_bound(z, err, act)
    if factor is not None:
        err = factor * (err + 2 * U * (np.abs(lo.act(z, act)) + err))
    if res is not None:
        err = err + U * (np.abs(want) + err)
    check(values(got).reshape(rows, cols), want, stored(err, want, out_kind), what, out_kind)
    return got


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("order", ["rows", "columns"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_linear_shapes(shape, order, kind):
    import optimizer_muon_step_amd as mu
    m, k, n = shape
    rng = np.random.default_rng(m * 7 + k * 3 + n)
    say(f"[linear] {shape} {order} {kind}")
    x, w = make(rng, (m, k), kind), make(rng, (k, n), kind, 0.1, order=order)
    b = make(rng, (1, n), "fp32")[0]
    check_linear(mu, x, w, kind, what="plain")
    check_linear(mu, x, w, kind, out="fp32", bias=b, act="gelu", keep=True, what="gelu")


LARGE = [(8200, 72, 1400), (4097, 72, 2311), (4160, 136, 2304), (1500, 72, 1304), (2000, 200, 1100), (3000, 72, 264), (1000, 2304, 760)]


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("order", ["rows", "columns"])
@pytest.mark.parametrize("shape", LARGE, ids=str)
def test_large_tiles(shape, order, kind):
    """Shapes that take the large tiles, with ragged ends, in all three products."""
    import optimizer_muon_step_amd as mu
    m, k, n = shape
    rng = np.random.default_rng(m + n)
    say(f"[large tiles] {shape} {order} {kind}")
    x, w = make(rng, (m, k), kind), make(rng, (k, n), kind, 0.1, order=order)
    res = make(rng, (m, n), kind)
    check_linear(mu, x, w, kind, bias=make(rng, (1, n), "fp32")[0], act="gelu", drop=(0.1, 5, 6, 7), residual=res, keep=True)
    check_linear(mu, x, w, kind, out="fp32", act="relu2")
    # the same sizes with the roles of k and m in their places for the backward products
    dz, wt = make(rng, (m, k), kind, 0.1), make(rng, (n, k), kind, 0.1, order=order)
    check_dx(mu, dz, wt, kind, act="gelu", preact=make(rng, (m, n), kind), residual=res)
    x, dz = make(rng, (k, m), kind), make(rng, (k, n), kind, 0.1)
    check_dw(mu, x, dz, make(rng, (m, n), "fp32", order=order), kind, bias=True, add=True)


@pytest.mark.parametrize("act", [None, "gelu", "relu", "relu2"])
@pytest.mark.parametrize("parts", ["", "bias", "residual", "drop", "bias residual drop keep"])
@pytest.mark.parametrize("out", ["same", "fp32"])
@pytest.mark.parametrize("kind,w_kind,shape", [("bf16", "bf16", (70, 96, 136)), ("fp16", "fp32", (131, 75, 259))])
def test_linear_epilogues(act, parts, out, kind, w_kind, shape):
    import optimizer_muon_step_amd as mu
    m, k, n = shape
    rng = np.random.default_rng(5)
    x, w = make(rng, (m, k), kind), make(rng, (k, n), w_kind, 0.2)
    res = make(rng, (m, n), kind if out == "same" else out) if "residual" in parts else None
    bias = make(rng, (1, n), "fp32" if out == "fp32" else kind)[0] if "bias" in parts else None
    check_linear(mu, x, w, kind, out, bias, act, (0.3, 0x123456789ABCDEF0, 77, 5) if "drop" in parts else None, res,
                 "keep" in parts)


# few tiles and a long reduction, which is split, in tiles of each kind
SPLIT = [(1, 4096, 72), (257, 30000, 520), (64, 6400, 1600), (9, 20001, 31), (257, 30000, 513), (130, 9000, 200), (520, 20000, 1000), (2048, 20000, 1032), (1500, 20000, 1500)]


@pytest.mark.parametrize("order", ["rows", "columns"])
@pytest.mark.parametrize("shape", SPLIT, ids=str)
def test_split_reductions(shape, order):
    import optimizer_muon_step_amd as mu
    m, k, n = shape
    rng = np.random.default_rng(m + k * 3 + n)
    say(f"[linear, dx] {shape} {order}")
    x, w = make(rng, (m, k), "bf16"), make(rng, (k, n), "bf16", 0.1, order=order)
    check_linear(mu, x, w, "bf16", bias=make(rng, (1, n), "fp32")[0], act="gelu", drop=(0.2, 1, 2, 3), keep=True)
    dz, w = make(rng, (m, k), "fp16", 0.1), make(rng, (n, k), "fp16", 0.1, order=order)
    check_dx(mu, dz, w, "fp16", out="fp32", residual=make(rng, (m, n), "fp32"))


@pytest.mark.parametrize("act", [None, "gelu", "relu", "relu2"])
@pytest.mark.parametrize("parts", ["", "bias", "residual", "drop", "bias residual drop keep"])
@pytest.mark.parametrize("out", ["same", "fp32"])
@pytest.mark.parametrize("kind,w_kind,shape", [("bf16", "fp32", (33, 2001, 67)), ("fp16", "fp16", (1, 4096, 136))])
def test_split_epilogues(act, parts, out, kind, w_kind, shape):
    """Forward with a bias, dx without one."""
    import optimizer_muon_step_amd as mu
    m, k, n = shape
    rng = np.random.default_rng(7)
    x, w = make(rng, (m, k), kind), make(rng, (k, n), w_kind, 0.1)
    res = make(rng, (m, n), kind if out == "same" else out) if "residual" in parts else None
    bias = make(rng, (1, n), "fp32")[0] if "bias" in parts else None
    drop = (0.3, 0x123456789ABCDEF0, 77, 5) if "drop" in parts else None
    check_linear(mu, x, w, kind, out, bias, act, drop, res, "keep" in parts)
    pre = None if act is None else make(rng, (m, n), kind, 2.0)
    check_dx(mu, x, w.T, kind, out=out, act=act, preact=pre, residual=res, drop=drop)


# read through a copy: rows shorter than 8, or products too large for 64 x 64 tiles
COPIED = [(70, 5, 72), (300, 6, 7), (5000, 1001, 1003), (8200, 771, 1029)]


@pytest.mark.parametrize("order", ["rows", "columns"])
@pytest.mark.parametrize("w_kind", ["bf16", "fp32"])
@pytest.mark.parametrize("shape", COPIED, ids=str)
def test_copied_operands(shape, w_kind, order):
    import optimizer_muon_step_amd as mu
    m, k, n = shape
    rng = np.random.default_rng(m + k * 3 + n)
    say(f"[copied] {shape} {w_kind} {order}")
    x, w = make(rng, (m, k), "bf16", offset=1, fill=NAN), make(rng, (k, n), w_kind, 0.1, order=order, fill=NAN)
    check_linear(mu, x, w, "bf16")
    dz = make(rng, (m, n), "bf16", 0.1, gap=3, fill=NAN)
    check_dx(mu, dz, w, "bf16", residual=make(rng, (m, k), "bf16"))
    check_dw(mu, x, dz, make(rng, (k, n), "fp32", order=order), "bf16", bias=True, add=True)


# read through registers: rows of 8 elements up, that end inside a chunk of 8 or a tile, that lie apart
# or anywhere, fp32 weights, a reduction of one slice to several splits
@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("order", ["rows", "columns"])
@pytest.mark.parametrize("m,k,n,gap,offset", [(1, 9, 8, 1, 1), (5, 8, 9, 0, 3), (64, 127, 65, 0, 0), (65, 128, 63, 1, 0),
                                              (3, 129, 193, 2, 5), (1, 768, 768, 0, 1), (77, 257, 15, 0, 7), (33, 1031, 129, 5, 0),
                                              (9, 10007, 71, 0, 2)])
def test_any_rows(m, k, n, gap, offset, order, kind):
    import optimizer_muon_step_amd as mu
    rng = np.random.default_rng(m + k * 3 + n)
    say(f"[any] {(m, k, n)} {gap} {offset} {order} {kind}")
    x, dz = make(rng, (m, k), kind, 1.0, offset, gap, fill=NAN), make(rng, (m, n), kind, 0.1, offset, gap, fill=NAN)
    for w_kind in (kind, "fp32"):
        w = make(rng, (k, n), w_kind, 0.1, offset, gap, order=order, fill=NAN)
        check_linear(mu, x, w, kind, act="gelu", bias=make(rng, (1, n), "fp32")[0], keep=True)
        check_dx(mu, dz, w, kind, out="fp32")
    dw = make(rng, (k, n), "fp32", offset=offset, gap=gap, order=order, fill=NAN)
    check_dw(mu, x, dz, dw, kind, bias=True)
    assert outside_unchanged(dw, NAN)


def test_split_in_place_and_captured():
    """Two captured calls whose reductions are split, the output the residual, replayed among eager calls."""
    torch = torch_mod()
    import optimizer_muon_step_amd as mu
    rng = np.random.default_rng(8)
    x, w = make(rng, (33, 4100), "bf16"), make(rng, (4100, 4100), "bf16", 0.02)
    y, start = make(rng, (33, 4100), "bf16"), make(rng, (33, 4100), "bf16")
    for _ in range(2):
        mu.muon_linear(x, w, residual=y, out=y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mu.muon_linear(x, w, residual=y, out=y)
        mu.muon_linear(y, w, residual=y, act="relu", preact=(z := torch.empty_like(y)), out=(out := torch.empty_like(y)))
    for _ in range(3):
        y.copy_(start)
        graph.replay()
        torch.cuda.synchronize()
        want = mu.muon_linear(x, w, residual=start)
        want_z = torch.empty_like(y)
        assert torch.equal(out, mu.muon_linear(want, w, residual=want, act="relu", preact=want_z))
        assert torch.equal(y, want) and torch.equal(z, want_z)


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("order", ["rows", "columns"])
@pytest.mark.parametrize("m,k,n,gap,offset", [(40, 72, 88, 56, 0), (130, 72, 200, 8, 0), (129, 136, 136, 64, 8),
                                              (20, 72, 88, 3, 0), (20, 72, 88, 0, 1), (37, 61, 83, 5, 3), (1, 72, 88, 5, 8)])
def test_linear_reads_and_writes_only_its_own(m, k, n, gap, offset, order, kind):
    """Operands inside buffers of NaN: one that got into a sum would show.  Outputs
    inside buffers of a marker."""
    import optimizer_muon_step_amd as mu
    rng = np.random.default_rng(11)
    x = make(rng, (m, k), kind, offset=offset, gap=gap, fill=NAN)
    w = make(rng, (k, n), kind, 0.2, offset=offset, gap=gap, order=order, fill=NAN)
    res = make(rng, (m, n), kind, offset=offset, gap=gap, fill=NAN)
    y = make(rng, (m, n), kind, offset=offset, gap=gap, fill=7.0)
    check_linear(mu, x, w, kind, residual=res, act="relu", y=y)
    assert outside_unchanged(y, 7.0)
    # the gradient of the input, and of the weight in either order
    dz = make(rng, (m, n), kind, offset=offset, gap=gap, fill=NAN)
    pre = make(rng, (m, k), kind, offset=offset, gap=gap, fill=NAN)
    dx = make(rng, (m, k), kind, offset=offset, gap=gap, fill=7.0)
    check_dx(mu, dz, w, kind, act="gelu", preact=pre, y=dx)
    assert outside_unchanged(dx, 7.0)
    dw = make(rng, (k, n), "fp32", offset=offset, gap=gap, order=order, fill=7.0)
    check_dw(mu, x, dz, dw, kind, bias=True)
    assert outside_unchanged(dw, 7.0)


def check_dx(mu, dz, w, kind, out="same", act=None, preact=None, drop=None, residual=None, y=None, what="dx"):
    out_kind = kind if out == "same" else out
    dzv, wv = values(dz).reshape(-1, dz.shape[-1]), _weight(w, kind).T
    rows, cols = dzv.shape[0], wv.shape[1]
    res = None if residual is None else values(residual).reshape(rows, cols)
    zv = None if preact is None else values(preact).reshape(rows, cols)
    factor = None if drop is None else lo.keep_factor(rows, cols, *drop[:4])
    got = mu.muon_linear_dx(dz, w, act=act, preact=preact, residual=residual, out=y, out_dtype=dtype(out_kind),
                            **({} if drop is None else dict(dropout=drop[0], rng=(drop[1], drop[2]), site=drop[3])))
    v = dzv @ wv
    err = _product_error(dzv, wv)
    want = lo.through(v, act, zv, factor, res)
    if act is not None:
        s, es = np.abs(lo.slope(zv, act)), slope_bound(zv, act)
        err = err * (s + es) + np.abs(v) * (es + U * s)
        v = v * lo.slope(zv, act)
    if factor is not None:
        err = factor * (err + 2 * U * (np.abs(v) + err))
    if res is not None:
        err = err + U * (np.abs(want) + err)
    check(values(got).reshape(rows, cols), want, stored(err, want, out_kind), what, out_kind)
    return got


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("order", ["rows", "columns"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_dx_shapes(shape, order, kind):
    import optimizer_muon_step_amd as mu
    m, k, n = shape
    rng = np.random.default_rng(m * 5 + k + n)
    say(f"[dx] {shape} {order} {kind}")
    dz, w = make(rng, (m, n), kind, 0.1), make(rng, (k, n), kind, 0.1, order=order)
    check_dx(mu, dz, w, kind)
    check_dx(mu, dz, w, kind, out="fp32", act="gelu", preact=make(rng, (m, k), kind), residual=make(rng, (m, k), "fp32"))


@pytest.mark.parametrize("act", [None, "gelu", "relu", "relu2"])
@pytest.mark.parametrize("parts", ["", "residual", "drop", "residual drop"])
@pytest.mark.parametrize("kind,w_kind,shape", [("bf16", "fp32", (70, 136, 96)), ("fp16", "fp16", (131, 259, 75))])
def test_dx_epilogues(act, parts, kind, w_kind, shape):
    import optimizer_muon_step_amd as mu
    m, k, n = shape
    rng = np.random.default_rng(6)
    dz, w = make(rng, (m, n), kind), make(rng, (k, n), w_kind, 0.2)
    pre = None if act is None else make(rng, (m, k), kind, 2.0)
    if act is not None:
        pre[0, 0], pre[0, 1], pre[0, 2], pre[0, 3] = 0.0, -0.0, 60000.0, -60000.0
    check_dx(mu, dz, w, kind, act=act, preact=pre, residual=make(rng, (m, k), kind) if "residual" in parts else None,
             drop=(0.25, 99, 3, 1) if "drop" in parts else None)


def check_dw(mu, x, dz, dw, kind, bias=False, add=False, what="dw"):
    torch = torch_mod()
    xv, dzv = values(x).reshape(-1, x.shape[-1]), values(dz).reshape(-1, dz.shape[-1])
    db = torch.from_numpy(np.random.default_rng(3).standard_normal(dz.shape[-1]).astype(np.float32)).cuda() if bias else None
    dw0, db0 = values(dw), None if db is None else values(db)
    mu.muon_linear_dw(x, dz, dw, dbias=db, accumulate=add)
    err = _product_error(xv.T, dzv)
    want = xv.T @ dzv + (dw0 if add else 0)
    check(dw, want, stored(err + (U * np.abs(want) if add else 0), want, "fp32"), what)
    if bias:
        err = (xv.shape[0] + 1) * 2.0 ** -23 * np.abs(dzv).sum(0)
        want = dzv.sum(0) + (db0 if add else 0)
        check(db, want, stored(err + U * np.abs(want), want, "fp32"), "dbias")


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("order", ["rows", "columns"])
@pytest.mark.parametrize("shape", SHAPES + [(4100, 72, 200), (9000, 264, 136), (20000, 8, 8), (3001, 131, 300), (30000, 520, 264), (8200, 1040, 520)], ids=str)
def test_dw_shapes(shape, order, kind):
    """The last ones are long enough for the reduction to be split."""
    import optimizer_muon_step_amd as mu
    m, k, n = shape
    rng = np.random.default_rng(m + k * 3 + n)
    say(f"[dw] {shape} {order} {kind}")
    x, dz = make(rng, (m, k), kind), make(rng, (m, n), kind, 0.1)
    check_dw(mu, x, dz, make(rng, (k, n), "fp32", order=order, fill=NAN), kind)
    check_dw(mu, x, dz, make(rng, (k, n), "fp32", order=order), kind, bias=True, add=True)
    dw = make(rng, (k, n), "fp32", order=order)
    dw.fill_(NAN)  # what it held does not matter
    check_dw(mu, x, dz, dw, kind, bias=True)


def test_no_rows():
    torch = torch_mod()
    import optimizer_muon_step_amd as mu
    x, dz = torch.empty(0, 24, dtype=torch.bfloat16, device="cuda"), torch.empty(0, 40, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(24, 40, dtype=torch.bfloat16, device="cuda")
    assert mu.muon_linear(x, w).shape == (0, 40)
    assert mu.muon_linear_dx(dz, w).shape == (0, 24)
    assert mu.muon_linear(x.view(3, 0, 24), w).shape == (3, 0, 40)
    dw, db = torch.full((24, 40), 3.0, device="cuda"), torch.full((40,), 3.0, device="cuda")
    mu.muon_linear_dw(x, dz, dw, dbias=db, accumulate=True)
    assert (dw == 3).all() and (db == 3).all()
    mu.muon_linear_dw(x, dz, dw, dbias=db)
    assert (dw == 0).all() and (db == 0).all()


def test_leading_dimensions_and_repeated_rows():
    torch = torch_mod()
    import optimizer_muon_step_amd as mu
    rng = np.random.default_rng(21)
    x, w = make(rng, (2 * 3 * 5, 40), "bf16"), make(rng, (40, 56), "bf16")
    flat = check_linear(mu, x, w, "bf16")
    assert torch.equal(mu.muon_linear(x.view(2, 3, 5, 40), w), flat.view(2, 3, 5, 56))
    one = x[0].clone()
    assert torch.equal(mu.muon_linear(one, w), flat[0])
    # the same row over and over (a distance of 0)
    assert torch.equal(mu.muon_linear(one.expand(9, 40), w), flat[0].expand(9, 56))
    res = make(rng, (1, 56), "bf16")
    check_linear(mu, x, w, "bf16", residual=res.expand(30, 56))
    # columns of one buffer: x on the left, y on the right
    buf = torch.zeros(30, 96, dtype=torch.bfloat16, device="cuda")
    buf[:, :40] = x
    mu.muon_linear(buf[:, :40], w, out=buf[:, 40:])
    assert torch.equal(buf[:, 40:], flat) and torch.equal(buf[:, :40], x)


def test_in_place():
    torch = torch_mod()
    import optimizer_muon_step_amd as mu
    rng = np.random.default_rng(22)
    x, w, res = make(rng, (70, 40), "fp16"), make(rng, (40, 131), "fp16"), make(rng, (70, 131), "fp32")
    want = mu.muon_linear(x, w, residual=res, act="relu2")
    got = mu.muon_linear(x, w, residual=res, act="relu2", out=res)
    assert got is res and torch.equal(res, want)
    dz, pre = make(rng, (70, 131), "fp16"), make(rng, (70, 40), "fp16")
    want = mu.muon_linear_dx(dz, w, act="gelu", preact=pre)
    assert mu.muon_linear_dx(dz, w, act="gelu", preact=pre, out=pre) is pre and torch.equal(pre, want)


def test_specials():
    """Infinities and NaN stay in their rows and columns; dropped ones vanish."""
    torch = torch_mod()
    import optimizer_muon_step_amd as mu
    rng = np.random.default_rng(23)
    x, w = make(rng, (40, 72), "bf16"), make(rng, (72, 88), "bf16")
    clean = mu.muon_linear(x, w)
    x2 = x.clone()
    x2[7, 3], x2[9, 70] = NAN, float("inf")
    y = mu.muon_linear(x2, w)
    rest = [r for r in range(40) if r not in (7, 9)]
    assert torch.isnan(y[7]).all() and not torch.isfinite(y[9]).any() and torch.equal(y[rest], clean[rest])
    w2 = w.clone()
    w2[71, 87] = NAN
    y = mu.muon_linear(x, w2)
    assert torch.isnan(y[:, 87]).all() and torch.equal(y[:, :87], clean[:, :87])
    # NaN behind a dropped element, in the product, its slope or the tensor itself
    p, seed, step, site = 0.5, 12345, 6, 7
    kept = torch.from_numpy(lo.keep_factor(40, 88, p, seed, step, site) != 0).cuda()
    bad = torch.full_like(x, NAN)
    y = mu.muon_linear(bad, w, dropout=p, rng=(seed, step), site=site)
    assert torch.isnan(y[kept]).all() and (y[~kept] == 0).all()
    for act in ("gelu", "relu2"):
        dx = mu.muon_linear_dx(x, w.T, act=act, preact=torch.full_like(clean, NAN), dropout=p, rng=(seed, step), site=site)
        assert torch.isnan(dx[kept]).all() and (dx[~kept] == 0).all()
    # activations of infinities
    e = torch.eye(8, dtype=torch.float16, device="cuda")
    z = torch.zeros(8, dtype=torch.float32, device="cuda")
    z[0], z[1], z[2], z[3], z[4] = float("inf"), -1e30, NAN, 1e30, -3e4
    y = mu.muon_linear(torch.zeros_like(e), e, bias=z, act="gelu", out_dtype=torch.float32)[0]
    assert y[0] == float("inf") and y[1] == 0 and torch.isnan(y[2]) and y[3] == 1e30 and y[4] == 0
    y = mu.muon_linear(torch.zeros_like(e), e, bias=z, act="relu", out_dtype=torch.float32)[0]
    assert y[0] == float("inf") and y[1] == 0 and torch.isnan(y[2]) and y[3] == 1e30


def test_same_bits_every_time():
    torch = torch_mod()
    import optimizer_muon_step_amd as mu
    rng = np.random.default_rng(24)
    x, w, dz = make(rng, (5000, 200), "bf16"), make(rng, (200, 300), "bf16"), make(rng, (5000, 300), "bf16")
    first = mu.muon_linear(x, w, act="gelu")
    dw, db = torch.empty(200, 300, device="cuda"), torch.empty(300, device="cuda")
    mu.muon_linear_dw(x, dz, dw, dbias=db)
    for _ in range(10):
        assert torch.equal(mu.muon_linear(x, w, act="gelu"), first)
        dw2, db2 = torch.empty_like(dw), torch.empty_like(db)
        mu.muon_linear_dw(x, dz, dw2, dbias=db2)
        assert torch.equal(dw, dw2) and torch.equal(db, db2)


def test_streams():
    """Calls on streams of their own, made at the same time."""
    torch = torch_mod()
    import optimizer_muon_step_amd as mu
    rng = np.random.default_rng(25)
    cases = [(make(rng, (3000 + 70 * i, 129), "bf16"), make(rng, (129, 257), "fp32"), make(rng, (3000 + 70 * i, 257), "bf16"))
             for i in range(4)]
    want = []
    for x, w, dz in cases:
        dw = torch.empty(129, 257, device="cuda")
        mu.muon_linear_dw(x, dz, dw)
        want.append((mu.muon_linear(x, w), mu.muon_linear_dx(dz, w), dw))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = []
    for (x, w, dz), s in zip(cases, streams):
        dw = torch.empty(129, 257, device="cuda")
        s.wait_stream(torch.cuda.current_stream())
        y = mu.muon_linear(x, w, stream=s)
        dx = mu.muon_linear_dx(dz, w, stream=s)
        mu.muon_linear_dw(x, dz, dw, stream=s)
        got.append((y, dx, dw))
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_versions_and_results():
    torch = torch_mod()
    import optimizer_muon_step_amd as mu
    x, w = torch.ones(4, 8, dtype=torch.bfloat16, device="cuda"), torch.ones(8, 16, dtype=torch.bfloat16, device="cuda")
    y, z = torch.empty(4, 16, dtype=torch.bfloat16, device="cuda"), torch.empty(4, 16, dtype=torch.bfloat16, device="cuda")
    before = (y._version, z._version, x._version)
    assert mu.muon_linear(x, w, out=y, preact=z) is y and (y == 8).all() and (z == 8).all()
    assert y._version > before[0] and z._version > before[1] and x._version == before[2]
    dw, db = torch.zeros(8, 16, device="cuda"), torch.zeros(16, device="cuda")
    before = (dw._version, db._version, z._version)
    assert mu.muon_linear_dw(x, y, dw, dbias=db) is None and (dw == 32).all() and (db == 32).all()
    assert dw._version > before[0] and db._version > before[1]
    assert mu.muon_linear(x, w, residual=torch.ones(4, 16, device="cuda")).dtype == torch.float32
    assert z._version == before[2]


def test_refusals_on_the_gpu():
    torch = torch_mod()
    import optimizer_muon_step_amd as mu
    half = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    x, w, y = half(4, 8), half(8, 16), half(4, 16)
    f32 = torch.zeros
    for match, call in [
            ("x: float32, expected bfloat16 or float16", lambda: mu.muon_linear(x.float(), w)),
            ("w: float16", lambda: mu.muon_linear(x, w.half())),
            ("last dimension of 8, w is 16 x 8", lambda: mu.muon_linear(x, w.T)),
            ("expected a matrix", lambda: mu.muon_linear(x, w[0])),
            ("adjacent elements along one", lambda: mu.muon_linear(x, half(16, 32)[::2, ::2])),
            ("adjacent elements along the last", lambda: mu.muon_linear(half(4, 16)[:, ::2], w)),
            ("evenly spaced", lambda: mu.muon_linear(half(4, 6, 16)[:, :3, :8], w)),
            ("bias", lambda: mu.muon_linear(x, w, bias=half(8))),
            ("bias", lambda: mu.muon_linear(x, w, bias=half(32)[::2])),
            ("bias: float16", lambda: mu.muon_linear(x, w, bias=half(16).half())),
            ("residual: shape", lambda: mu.muon_linear(x, w, residual=half(4, 8))),
            ("residual: bfloat16, expected float32", lambda: mu.muon_linear(x, w, residual=y, out_dtype=torch.float32)),
            ("out: shape", lambda: mu.muon_linear(x, w, out=half(16, 4))),
            ("out: float16", lambda: mu.muon_linear(x, w, out=y.half())),
            ("out: its type", lambda: mu.muon_linear(x, w, out=y, out_dtype=torch.float32)),
            ("preact: float32", lambda: mu.muon_linear(x, w, preact=y.float())),
            ("on the GPU", lambda: mu.muon_linear(x, w.cpu())),
            ("rng: dropout needs", lambda: mu.muon_linear(x, w, dropout=0.5)),
            ("rng: expected", lambda: mu.muon_linear(x, w, dropout=0.5, rng=5)),
            ("rng: expected", lambda: mu.muon_linear(x, w, dropout=0.5, rng=(1, 2, 3))),
            ("rng: expected", lambda: mu.muon_linear(x, w, dropout=0.5, rng=torch.zeros(2, dtype=torch.int64))),
            ("rng: expected", lambda: mu.muon_linear(x, w, dropout=0.5, rng=f32(2, device="cuda"))),
            ("rng: seed", lambda: mu.muon_linear(x, w, dropout=0.5, rng=(-1, 0))),
            ("rng: seed", lambda: mu.muon_linear(x, w, dropout=0.5, rng=(1.5, 0))),
            ("rng: step", lambda: mu.muon_linear(x, w, dropout=0.5, rng=(1, 2 ** 32))),
            ("site", lambda: mu.muon_linear(x, w, dropout=0.5, rng=(1, 2), site=-1)),
            ("dz: last dimension", lambda: mu.muon_linear_dx(x, w)),
            ("dw: expected 8 x 16", lambda: mu.muon_linear_dw(x, y, f32(16, 8, device="cuda"))),
            ("dw: bfloat16", lambda: mu.muon_linear_dw(x, y, w)),
            ("dz: float16", lambda: mu.muon_linear_dw(x, y.half(), w.float())),
            ("dimensions before the last", lambda: mu.muon_linear_dw(x, half(5, 16), w.float())),
            ("dbias", lambda: mu.muon_linear_dw(x, y, w.float(), dbias=f32(8, device="cuda"))),
            ("preact: shape", lambda: mu.muon_dropout(x, 0.5, (1, 2), act="relu", preact=y)),
            ("preact: bfloat16", lambda: mu.muon_dropout(x.float(), 0.5, (1, 2), act="relu", preact=x)),
            ("rng: dropout needs", lambda: mu.muon_dropout(x, 0.5, None)),
            ("hipStreamPerThread", lambda: mu.muon_linear(x, w, stream=2))]:
        with pytest.raises(ValueError, match=match):
            call()
    for match, call in [
            ("overlap", lambda: mu.muon_linear(x, half(8, 8), out=x)),
            ("overlap", lambda: mu.muon_linear(x, w, out=half(1, 16).expand(4, 16))),
            ("dropout = 1", lambda: mu.muon_linear(x, w, dropout=1.0, rng=(1, 2))),
            ("dropout = nan", lambda: mu.muon_dropout(x, float("nan"), (1, 2))),
            ("come together", lambda: mu.muon_linear_dx(y, w, act="gelu")),
            ("come together", lambda: mu.muon_dropout(x, 0.5, (1, 2), preact=x)),
            ("overlaps", lambda: mu.muon_linear(x, w, out=y, preact=y))]:
        with pytest.raises(mu.MuonError, match=match):
            call()
    torch.cuda.synchronize()
