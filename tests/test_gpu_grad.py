"""GPU tests of the global gradient norm and clipping (muon_grad_norm,
muon_grad_clip).

The norm and the factor are one rounding to fp32 of values held in fp64: half
a step, 2^-24 relative, and 1e-12 for the order of the fp64 sum (2^31 terms of
2^-53 each stay below it).  The clipped gradients are the fp32 product with
the record's own factor, rounded once: compared bit for bit."""
import math

import numpy as np
import pytest

from gpu_helpers import say, torch_mod
from oracle import grad_oracle as go

pytestmark = pytest.mark.gpu

HALF_STEP = 2.0 ** -24 * (1 + 1e-6) + 1e-12
KINDS = ("fp32", "bf16", "fp16")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    torch = torch_mod()
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import optimizer_muon_step_amd as mu
    mu._lib.load()
    yield
    torch.cuda.synchronize()


def _dtype(kind):
    torch = torch_mod()
    return {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}[kind]


def _values(t):
    """A tensor's values as fp32 numpy (exact)."""
    return t.detach().float().cpu().numpy()


def _bits(t):
    torch = torch_mod()
    return t.detach().contiguous().view(torch.int32 if t.dtype == torch.float32 else torch.int16).cpu()


def _make(rng, sizes, kinds, offset=0, scale=1.0):
    """Gradients on the GPU, each `offset` elements into a buffer of its own."""
    torch = torch_mod()
    out = []
    for i, n in enumerate(sizes):
        buf = torch.from_numpy((rng.standard_normal(n + offset) * scale).astype(np.float32)).to(_dtype(kinds[i % len(kinds)]))
        out.append(buf.cuda()[offset:])
    return out


def _check_record(record, grads, max_norm=math.inf, scale=1.0):
    norm, factor = go.norm_factor([_values(g) for g in grads], max_norm, scale)
    got = record.cpu().numpy().astype(np.float64)
    assert abs(got[0] - norm) <= HALF_STEP * norm, (got, norm)
    assert abs(got[1] - factor) <= HALF_STEP * factor, (got, factor)
    return got


EDGES = [1, 2, 3, 4, 5, 63, 64, 65, 255, 256, 257, 1023, 1024, 1025, 4095, 4096, 4097, 8191, 8192, 8193, 12289]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("offset", [0, 1, 3])
def test_norm_single_tensor_sizes(kind, offset):
    import optimizer_muon_step_amd as mu
    rng = np.random.default_rng(50 + offset)
    say(f"[norm sizes] {kind} offset {offset}")
    for n in EDGES:
        g = _make(rng, [n], [kind], offset)
        _check_record(mu.muon_grad_norm(g, 0.5), g, 0.5)


@pytest.mark.parametrize("sizes,kinds", [
    ([], KINDS), ([0], KINDS), ([0, 0, 0], KINDS), ([1, 0, 3], KINDS), (EDGES, KINDS), (EDGES, ("bf16",)),
    ([768] * 8, ("fp32",)), ([64] * 251, ("fp32",)), ([64] * 252, ("bf16",)), ([65] * 253, KINDS),
    ([1000 + 37 * k for k in range(600)], KINDS), ([3_000_001], ("fp32",)), ([20_000_003, 7, 9_000_001], KINDS)])
@pytest.mark.parametrize("max_norm,scale", [(math.inf, 1.0), (1.0, 0.125), (1e6, 3.0)])
def test_norm_lists(sizes, kinds, max_norm, scale):
    import optimizer_muon_step_amd as mu
    rng = np.random.default_rng(51)
    say(f"[norm lists] {len(sizes)} tensors, {sum(sizes)} elements")
    g = _make(rng, sizes, kinds)
    _check_record(mu.muon_grad_norm(g, max_norm, scale=scale), g, max_norm, scale)


def test_norm_same_bits_every_time():
    torch = torch_mod()
    import optimizer_muon_step_amd as mu
    g = _make(np.random.default_rng(52), [5_000_001, 3, 70_000] + [333] * 300, KINDS)
    first = mu.muon_grad_norm(g, 1.0)
    for _ in range(20):
        assert torch.equal(_bits(mu.muon_grad_norm(g, 1.0)), _bits(first))


def test_norm_never_takes_partials_of_an_earlier_call():
    """Calls on g and 2 g in turn, without a wait: a partial left from the call
    before would show, since the two norms are exactly a factor of 2 apart."""
    torch = torch_mod()
    import optimizer_muon_step_amd as mu
    for sizes in ([40_000], [300_000, 77], [9_000_001, 3, 400_000], [5000] * 600):
        one = _make(np.random.default_rng(74), sizes, ["fp32"])
        two = [2 * t for t in one]
        want = mu.muon_grad_norm(one)[0].item()
        got = torch.stack([mu.muon_grad_norm(two if k % 2 else one)[0] for k in range(300)])
        assert torch.equal(got.cpu(), torch.tensor([want, 2 * want] * 150)), sizes


def test_norm_counts_a_repeated_tensor_each_time_and_leaves_gradients():
    torch = torch_mod()
    import optimizer_muon_step_amd as mu
    g = torch.full((9,), 2.0, device="cuda")
    keep = g.clone()
    assert mu.muon_grad_norm([g, g, g, g])[0].item() == 12.0
    assert torch.equal(g, keep)


@pytest.mark.parametrize("value,norm,factor", [
    (0.0, 0.0, 1.0), (1e-42, None, 1.0), (2e-30, None, 1.0), (1e30, None, None), (3e38, math.inf, None),
    (math.inf, math.inf, 0.0), (-math.inf, math.inf, 0.0), (math.nan, math.nan, math.nan)])
def test_norm_special_values(value, norm, factor):
    """Squares that leave the fp32 range do not leave the sum's."""
    torch = torch_mod()
    import optimizer_muon_step_amd as mu
    for n, at in ((2, 1), (4097, 4096), (100_000, 50_000)):
        g = torch.zeros(n, device="cuda")
        g[at] = g[0] = value
        got = mu.muon_grad_norm([g], 1.0).cpu().numpy()
        want, want_factor = go.norm_factor([_values(g)], 1.0)
        for x, w in ((got[0], want if norm is None else norm), (got[1], want_factor if factor is None else factor)):
            if math.isfinite(w):
                # a subnormal result is off by half of the subnormals' step
                assert abs(float(x) - w) <= max(HALF_STEP * w, 2.0 ** -150), (value, n, got, w)
            else:
                assert np.array_equal(np.float32(w), x, equal_nan=True), (value, n, got)


@pytest.mark.parametrize("max_norm", [0.0, 1e-30, 5.0, 5.000001, 3e38])
def test_norm_limits(max_norm):
    torch = torch_mod()
    import optimizer_muon_step_amd as mu
    g = [torch.tensor([3.0, 4.0], device="cuda")]
    _check_record(mu.muon_grad_norm(g, max_norm), g, max_norm)


def test_norm_of_dense_layouts():
    torch = torch_mod()
    import optimizer_muon_step_amd as mu
    t = torch.from_numpy(np.random.default_rng(53).standard_normal((40, 30, 20)).astype(np.float32)).cuda()
    for g in (t.permute(2, 0, 1), t.transpose(0, 1), t[3:7]):
        _check_record(mu.muon_grad_norm([g]), [g])
    for bad in (t[:, :10], t[..., ::2], t[:1].expand(5, 30, 20)):
        with pytest.raises(ValueError, match="dense"):
            mu.muon_grad_norm([bad])


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
def test_norm_and_clip_past_32_bit_offsets(kind):
    """More than 2^31 elements (and 2^32 bytes): only the last elements, and
    one in the middle, are not zero."""
    torch = torch_mod()
    import optimizer_muon_step_amd as mu
    n = 2 ** 31 + 4097
    say(f"[large] {kind} {n} elements")
    g = torch.zeros(n, dtype=_dtype(kind), device="cuda")
    g[-1], g[-4096], g[2 ** 30 + 1] = 3.0, 4.0, 12.0
    record = mu.muon_grad_clip([g], 6.5)
    norm, factor = go.norm_factor([np.array([3.0, 4.0, 12.0])], 6.5)
    got = record.cpu().numpy()
    assert abs(got[0] - norm) <= HALF_STEP * norm and abs(got[1] - factor) <= HALF_STEP
    want = go.rounded(go.clipped(np.array([3.0, 4.0, 12.0], np.float32), got[1]), kind)
    assert [g[-1].item(), g[-4096].item(), g[2 ** 30 + 1].item()] == want.tolist()
    assert torch.count_nonzero(g[:-1].view(-1, 4096).amax(1)).item() == 2  # nothing else was written
    del g
    torch.cuda.empty_cache()


@pytest.mark.parametrize("kind_in", KINDS)
@pytest.mark.parametrize("kind_out", KINDS)
@pytest.mark.parametrize("offset", [0, 1])
def test_clip_into_other_tensors(kind_in, kind_out, offset):
    """Every pair of types, sizes around the chunk edges; the elements behind
    each out stay as they were."""
    torch = torch_mod()
    import optimizer_muon_step_amd as mu
    rng = np.random.default_rng(54)
    sizes = EDGES + [0, 100_003]
    g = _make(rng, sizes, [kind_in], offset, 0.3)
    bufs = [torch.full((n + 7 + offset,), -7.0, dtype=_dtype(kind_out), device="cuda") for n in sizes]
    outs = [b[offset + 3:offset + 3 + n] for b, n in zip(bufs, sizes)]
    before = [t.clone() for t in g]
    record = mu.muon_grad_clip(g, 2.0, scale=0.5, outs=outs)
    got = _check_record(record, before, 2.0, 0.5)
    for t, k, o, b, n in zip(g, before, outs, bufs, sizes):
        assert torch.equal(_bits(t), _bits(k))
        want = go.rounded(go.clipped(_values(k), np.float32(got[1])), kind_out)
        assert np.array_equal(_values(o).view(np.uint32), want.view(np.uint32)), (kind_in, kind_out, n)
        assert (b[:offset + 3] == -7.0).all() and (b[offset + 3 + n:] == -7.0).all()


@pytest.mark.parametrize("kind", KINDS)
def test_clip_in_place(kind):
    torch = torch_mod()
    import optimizer_muon_step_amd as mu
    rng = np.random.default_rng(55)
    bufs = _make(rng, [n + 5 for n in EDGES + [300_007]], [kind])
    g = [b[2:-3] for b in bufs]
    before = [b.clone() for b in bufs]
    below = mu.muon_grad_clip(g, 1e9)
    assert below[1].item() == 1.0 and all(torch.equal(_bits(b), _bits(k)) for b, k in zip(bufs, before))
    got = mu.muon_grad_clip(g, 1.0).cpu().numpy()
    assert got[1] < 1.0
    for b, k in zip(bufs, before):
        want = _values(k)
        want[2:-3] = go.rounded(go.clipped(want[2:-3], got[1]), kind)
        assert np.array_equal(_values(b).view(np.uint32), want.view(np.uint32))


@pytest.mark.parametrize("kind_in", KINDS)
@pytest.mark.parametrize("kind_out", KINDS + ("in place",))
@pytest.mark.parametrize("offset", [0, 1, 5])
def test_small_clips(kind_in, kind_out, offset):
    """Calls of one launch: a tensor of each size alone, then lists of up to
    16 chunks, below and above the limit; nothing outside an out is written."""
    torch = torch_mod()
    import optimizer_muon_step_amd as mu
    rng = np.random.default_rng(70)
    chunk = 4096 if kind_in == "fp32" else 8192
    lists = [[n] for n in EDGES] + [[], [0, 3], [chunk] * 16, [chunk * 15 + 1], [1] * 16, [chunk - 1, 2 * chunk + 3, 1, 0, 700]]
    for sizes in lists:
        for limit in (1e9, 0.25):
            bufs = _make(rng, [n + offset + 4 for n in sizes], [kind_in])
            g = [b[offset:-4] for b in bufs]
            before = [b.clone() for b in bufs]
            if kind_out == "in place":
                obufs, outs, kind = bufs, None, kind_in
            else:
                kind = kind_out
                obufs = [torch.full((n + offset + 4,), -7.0, dtype=_dtype(kind), device="cuda") for n in sizes]
                outs = [b[offset:-4] for b in obufs]
            record = mu.muon_grad_clip(g, limit, outs=outs)
            got = _check_record(record, [b[offset:-4] for b in before], limit)
            assert torch.equal(_bits(record), _bits(mu.muon_grad_norm([b[offset:-4] for b in before], limit)))
            for b, k in zip(obufs, before):
                want = _values(k) if outs is None else np.full(b.numel(), -7.0, np.float32)
                want[offset:-4] = go.rounded(go.clipped(_values(k)[offset:-4], np.float32(got[1])), kind)
                assert np.array_equal(_values(b).view(np.uint32), want.view(np.uint32)), (sizes, limit)


def _device_record(grads, max_norm, scale=1.0):
    """The record from sums in fp64 on the device, for lists that are long on the CPU."""
    total = sum(float(piece.double().square().sum()) for g in grads for piece in g.split(1 << 24))
    norm = scale * math.sqrt(total)
    return norm, scale * min(1.0, max_norm / (norm + 1e-6))


@pytest.mark.parametrize("kinds,kinds_out", [(("fp32",), ("bf16",)), (("bf16", "fp16"), ("fp32",)), (KINDS, ("fp16", "fp32", "bf16"))])
def test_clip_into_other_tensors_past_a_whole_group_of_runs(kinds, kinds_out):
    """Enough chunks of 4096 for one group of 8 runs of 64 and a rest that no
    multiple of 8 fills, over tensors that begin and end anywhere in them."""
    torch = torch_mod()
    import optimizer_muon_step_amd as mu
    sizes = [1_500_003, 9, 700_001, 4096, 1_250_077, 40_001, 1, 8191, 333_333]
    items = sum(-(-n // 4096) for n in sizes)
    assert items > 8 * 64 and items % 8 and items % 64
    rng = np.random.default_rng(77)
    g = _make(rng, sizes, kinds, 1)
    bufs = [torch.full((n + 5,), -7.0, dtype=_dtype(kinds_out[i % len(kinds_out)]), device="cuda") for i, n in enumerate(sizes)]
    record = mu.muon_grad_clip(g, 3.0, scale=0.5, outs=[b[2:-3] for b in bufs])
    got = _check_record(record, g, 3.0, 0.5)
    for i, (t, b) in enumerate(zip(g, bufs)):
        want = np.full(b.numel(), -7.0, np.float32)
        want[2:-3] = go.rounded(go.clipped(_values(t), np.float32(got[1])), kinds_out[i % len(kinds_out)])
        assert np.array_equal(_values(b).view(np.uint32), want.view(np.uint32)), i


@pytest.mark.parametrize("sizes,kinds", [
    ([100_000_003, 30_000_001, 5, 12_345_677, 3, 4099], ("bf16", "fp32", "fp16")),  # one launch, kept from inside it
    ([400_001 + 2 * k for k in range(300)], KINDS),                                 # two launches, kept from inside the first
    ([80_000_001, 70_000_003, 11], ("fp32",))])
def test_norm_of_a_list_longer_than_what_is_kept(sizes, kinds):
    """More than 256 MiB under a limit: the front is read one way, the end another."""
    torch = torch_mod()
    import optimizer_muon_step_amd as mu
    say(f"[norm long] {len(sizes)} tensors, {sum(sizes)} elements")
    gen = torch.Generator(device="cuda").manual_seed(78)
    g = [torch.randn(n, generator=gen, device="cuda").to(_dtype(kinds[i % len(kinds)])) for i, n in enumerate(sizes)]
    assert sum(t.numel() * t.element_size() for t in g) > 256 << 20
    for limit, scale in ((2.0, 0.5), (1e9, 1.0)):
        norm, factor = _device_record(g, limit, scale)
        got = mu.muon_grad_norm(g, limit, scale=scale).cpu().numpy().astype(np.float64)
        assert abs(got[0] - norm) <= HALF_STEP * norm and abs(got[1] - factor) <= HALF_STEP * factor, (got, norm, factor)


@pytest.mark.parametrize("kinds", [("fp32",), ("bf16", "fp16")])
def test_long_clip_in_place(kinds):
    """More chunks than an in-place launch has blocks, over several tensors:
    each element is clipped once, and nothing beside them."""
    torch = torch_mod()
    import optimizer_muon_step_amd as mu
    sizes = [40_000_003, 17, 30_000_001, 4097, 5_000_001]
    assert sum(-(-n // 4096) for n in sizes) > 16384
    say(f"[clip long] {kinds} {sum(sizes)} elements")
    gen = torch.Generator(device="cuda").manual_seed(79)
    bufs = [torch.randn(n + 5, generator=gen, device="cuda").to(_dtype(kinds[i % len(kinds)])) for i, n in enumerate(sizes)]
    g = [b[1:-4] for b in bufs]
    before = [b.clone() for b in bufs]
    norm, factor = _device_record(g, 1.0)
    record = mu.muon_grad_clip(g, 1.0)
    got = record.cpu().numpy().astype(np.float64)
    assert abs(got[0] - norm) <= HALF_STEP * norm and abs(got[1] - factor) <= HALF_STEP * factor
    for b, k in zip(bufs, before):
        want = k.clone()
        want[1:-4] = (k[1:-4].float() * record[1]).to(k.dtype)
        assert torch.equal(b.view(torch.int32 if b.element_size() == 4 else torch.int16),
                           want.view(torch.int32 if b.element_size() == 4 else torch.int16))


def test_clip_scale_alone_and_many_tensors():
    """No limit: only the scale; more tensors than one launch's table holds."""
    import optimizer_muon_step_amd as mu
    rng = np.random.default_rng(56)
    g = _make(rng, [100 + 3 * k for k in range(400)], ["fp32"])
    before = [_values(t) for t in g]
    got = mu.muon_grad_clip(g, math.inf, scale=0.25).cpu().numpy()
    assert got[1] == 0.25
    for t, b in zip(g, before):
        assert np.array_equal(_values(t), b * np.float32(0.25))


@pytest.mark.parametrize("value", [math.inf, math.nan])
@pytest.mark.parametrize("max_norm", [1.0, math.inf])
def test_clip_of_gradients_that_are_not_finite(value, max_norm):
    """The formula's values: under a limit inf gives factor 0 (so NaN at the
    infinity, 0 elsewhere); a NaN spreads; without a limit inf stays."""
    torch = torch_mod()
    import optimizer_muon_step_amd as mu
    g = torch.ones(5000, device="cuda")
    g[77] = value
    before = _values(g)
    got = mu.muon_grad_clip([g], max_norm).cpu().numpy()
    norm, factor = go.norm_factor([before], max_norm)
    assert np.array_equal(got, np.array([norm, factor], np.float32), equal_nan=True)
    assert np.array_equal(_values(g), go.clipped(before, got[1]), equal_nan=True)


def test_clip_keeps_memory_order_and_refuses_others():
    torch = torch_mod()
    import optimizer_muon_step_amd as mu
    t = torch.from_numpy(np.random.default_rng(57).standard_normal((30, 50)).astype(np.float32)).cuda()
    out = torch.empty(50, 30, device="cuda").t()
    want = t.t().contiguous().t() * mu.muon_grad_clip([t.t().contiguous().t()], 1.0, outs=[out])[1]
    assert torch.equal(out, want)
    with pytest.raises(ValueError, match="memory order"):
        mu.muon_grad_clip([t], 1.0, outs=[out])
    with pytest.raises(ValueError, match="same length"):
        mu.muon_grad_clip([t], 1.0, outs=[])
    with pytest.raises(mu.MuonError, match="overlaps"):
        mu.muon_grad_clip([t, t], 1.0)
    with pytest.raises(mu.MuonError, match="another type"):
        h = torch.zeros(8, dtype=torch.bfloat16, device="cuda")
        mu.muon_grad_clip([h], 1.0, outs=[h.view(torch.float16)])
    with pytest.raises(mu.MuonError, match="max_norm"):
        mu.muon_grad_clip([t], -1.0)
    with pytest.raises(ValueError, match="record"):
        mu.muon_grad_norm([t], record=torch.zeros(3, device="cuda"))


def test_autograd_notices_a_clip():
    """What a clip writes counts as changed, as after torch's own in-place
    operations: a backward pass through values saved before is refused."""
    torch = torch_mod()
    import optimizer_muon_step_amd as mu
    for n in (300, 200_001):  # one launch and two
        x = torch.full((n,), 2.0, device="cuda", requires_grad=True)
        (grad,) = torch.autograd.grad((x * x * x).sum(), x, create_graph=True)
        loss = (grad * grad).sum()  # saves grad
        version, still = grad._version, x._version
        with pytest.raises(mu.MuonError):
            mu.muon_grad_clip([grad], -1.0)
        assert grad._version == version
        mu.muon_grad_norm([grad])
        assert grad._version == version
        mu.muon_grad_clip([grad], 1.0)
        assert grad._version == version + 1 and x._version == still
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            loss.backward()
        source, out, record = torch.ones(n, device="cuda"), torch.empty(n, device="cuda"), torch.empty(2, device="cuda")
        mu.muon_grad_clip([source], 1.0, outs=[out], record=record)
        assert (source._version, out._version, record._version) == (0, 1, 1)
        mu.muon_grad_norm([source], record=record)
        assert record._version == 2
        with torch.inference_mode():  # tensors without a counter
            quiet = torch.ones(n, device="cuda")
            mu.muon_grad_clip([quiet], 1.0, record=torch.empty(2, device="cuda"))
        assert quiet[0].item() < 1.0


@pytest.mark.parametrize("limit", [0.01, 1e6])
def test_clip_agrees_with_torch_on_a_model(limit):
    """An independent implementation: torch.nn.utils.clip_grad_norm_ in fp64 on
    the CPU, on the gradients of a small model.  Three roundings to fp32 lie
    between them (the norm is not one of them): the factor, the product, and
    the limit's own."""
    torch = torch_mod()
    import optimizer_muon_step_amd as mu
    torch.manual_seed(73)
    model = torch.nn.Sequential(torch.nn.Embedding(50, 24), torch.nn.Linear(24, 72), torch.nn.GELU(),
                                torch.nn.LayerNorm(72), torch.nn.Linear(72, 50)).cuda()
    out = model(torch.randint(0, 50, (8, 16), device="cuda"))
    torch.nn.functional.cross_entropy(out.view(-1, 50), torch.randint(0, 50, (128,), device="cuda")).backward()
    params = list(model.parameters())
    twins = [torch.nn.Parameter(p.detach().double().cpu()) for p in params]
    for p, t in zip(params, twins):
        t.grad = p.grad.double().cpu()
    norm = torch.nn.utils.clip_grad_norm_(twins, limit).item()
    record = mu.muon_grad_clip([p.grad for p in params], limit)
    assert abs(record[0].item() - norm) <= HALF_STEP * norm
    for p, t in zip(params, twins):
        err = (p.grad.double().cpu() - t.grad).abs()
        assert (err <= 3.1 * 2.0 ** -24 * t.grad.abs() + 2.0 ** -149).all()


def test_two_streams_at_once():
    """Calls on two streams overlap: each has a workspace of its own."""
    torch = torch_mod()
    import optimizer_muon_step_amd as mu
    rng = np.random.default_rng(58)
    lists = [_make(rng, [8_000_001, 5, 1000], ["fp32"]), _make(rng, [9_000_003, 77], ["bf16"])]
    want = [mu.muon_grad_norm(g, 1.0).clone() for g in lists]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for k in (0, 1):
            got[k].append(mu.muon_grad_norm(lists[k], 1.0, stream=streams[k]))
    torch.cuda.synchronize()
    for k in (0, 1):
        assert all(torch.equal(_bits(r), _bits(want[k])) for r in got[k])
    # a raw stream handle, and a record handed in
    record = torch.zeros(2, device="cuda")
    torch.cuda.synchronize()
    assert mu.muon_grad_norm(lists[0], 1.0, record=record, stream=streams[1].cuda_stream) is record
    streams[1].synchronize()
    assert torch.equal(_bits(record), _bits(want[0]))


def test_streams_that_are_not_torchs():
    """Streams made elsewhere come and go; no call leaves a workspace behind."""
    import ctypes

    torch = torch_mod()
    import optimizer_muon_step_amd as mu
    hip = mu._lib.load()  # the HIP runtime that the library is linked against
    grads = _make(np.random.default_rng(76), [700_001, 5, 1000], KINDS)
    want = mu.muon_grad_norm(grads, 1.0)
    kept = set(mu._norm_workspaces)
    for _ in range(3):
        handle = ctypes.c_void_p()
        assert hip.hipStreamCreate(ctypes.byref(handle)) == 0
        torch.cuda.synchronize()
        got = [mu.muon_grad_norm(grads, 1.0, stream=handle.value) for _ in range(4)]
        got.append(mu.muon_grad_norm(grads, 1.0, stream=torch.cuda.ExternalStream(handle.value)))
        torch.cuda.synchronize()
        assert all(torch.equal(_bits(r), _bits(want)) for r in got)
        assert hip.hipStreamDestroy(handle) == 0
    assert set(mu._norm_workspaces) == kept
    with pytest.raises(ValueError, match="hipStreamPerThread"):
        mu.muon_grad_clip(grads, 1.0, stream=torch.cuda.ExternalStream(2))
    # a stream of torch's keeps one workspace, by object or by handle
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    for s in (stream, stream.cuda_stream, stream):
        record = mu.muon_grad_norm(grads, 1.0, stream=s)
        stream.synchronize()
        assert torch.equal(_bits(record), _bits(want))
    assert len(set(mu._norm_workspaces) - kept) == 1


def test_two_threads_on_one_stream():
    """Both threads' calls take the stream's one workspace, and several
    launches each: a call's launches stay together."""
    import threading

    torch = torch_mod()
    import optimizer_muon_step_amd as mu
    rng = np.random.default_rng(72)
    lists = [_make(rng, [1000 + k for k in range(600)], ["fp32"]), _make(rng, [700 + 3 * k for k in range(550)], KINDS)]
    want = [mu.muon_grad_norm(g, 1.0) for g in lists]
    got = [[], []]

    def work(k):
        for _ in range(50):
            got[k].append(mu.muon_grad_norm(lists[k], 1.0))

    threads = [threading.Thread(target=work, args=(k,)) for k in (0, 1)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for k in (0, 1):
        assert len(got[k]) == 50 and all(torch.equal(_bits(r), _bits(want[k])) for r in got[k])


def test_a_list_that_another_thread_changes():
    """Tensors of zeros come and go while the calls run: each call takes the
    list as it was at one time, and the norm is the same."""
    import threading

    torch = torch_mod()
    import optimizer_muon_step_amd as mu
    grads = _make(np.random.default_rng(75), [5000, 77, 300_001], ["fp32"])
    want = mu.muon_grad_norm(grads)
    zeros, done = [torch.zeros(3, device="cuda") for _ in range(300)], threading.Event()

    def work():
        while not done.is_set():
            grads.extend(zeros)
            del grads[3:]

    thread = threading.Thread(target=work)
    thread.start()
    try:
        got = [mu.muon_grad_norm(grads) for _ in range(200)]
    finally:
        done.set()
        thread.join()
    # longer lists may take another split of the sum: half a step on either side
    got = torch.stack(got).cpu().numpy().astype(np.float64)[:, 0]
    assert (np.abs(got - want[0].item()) <= 2 * HALF_STEP * want[0].item()).all()


def test_captured_norm_and_clip_without_an_earlier_call():
    """Captured at once, replayed with new gradients and eager work between;
    two graphs replayed in turn."""
    torch = torch_mod()
    import optimizer_muon_step_amd as mu
    rng = np.random.default_rng(59)
    sets = [[_make(rng, sizes, KINDS) for _ in range(4)] for sizes in ([70_001, 33, 4096] * 100, [12345, 2_000_003])]
    graphs, state = [], []
    for fresh in sets:
        g = [t.clone() for t in fresh[0]]
        outs = [torch.empty(t.shape, device="cuda") for t in g]
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            record = mu.muon_grad_clip(g, 1.0, scale=0.5, outs=outs)
        graphs.append(graph)
        state.append((g, outs, record))
    for rep in range(4):
        for fresh, graph, (g, outs, record) in zip(sets, graphs, state):
            for a, b in zip(g, fresh[rep]):
                a.copy_(b)
            graph.replay()
        torch.cuda.synchronize()
        for fresh, (g, outs, record) in zip(sets, state):
            eager_outs = [torch.empty_like(o) for o in outs]
            eager = mu.muon_grad_clip(g, 1.0, scale=0.5, outs=eager_outs)
            torch.cuda.synchronize()
            assert torch.equal(_bits(record), _bits(eager)), rep
            assert all(torch.equal(a, b) for a, b in zip(outs, eager_outs)), rep


def test_captured_norm_clears_its_workspace():
    """The graph's memory is not clear: the graph clears the norm's part of it
    on every replay."""
    torch = torch_mod()
    import optimizer_muon_step_amd as mu
    g = _make(np.random.default_rng(71), [300_001, 5, 40_000], KINDS)
    want = mu.muon_grad_norm(g, 1.0)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        junk = torch.full((8192,), 7.0, dtype=torch.float64, device="cuda")
        del junk  # what is allocated next gets its memory
        record = mu.muon_grad_norm(g, 1.0)
    for _ in range(3):
        record.fill_(-1.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(_bits(record), _bits(want))


def test_timing_families():
    torch = torch_mod()
    import optimizer_muon_step_amd as mu
    g = [torch.ones(100_000, device="cuda")]
    for kernel in (mu.KERNEL_GRAD_NORM, mu.KERNEL_GRAD_CLIP):
        mu.muon_timing_enable(kernel)
        mu.muon_grad_clip(g, 1.0, scale=0.5)
        ms, launches = mu.muon_timing_read()
        mu.muon_timing_enable(-1)
        assert launches == 1 and ms > 0


def test_release_between_norms():
    torch = torch_mod()
    import optimizer_muon_step_amd as mu
    g = [torch.full((4,), 2.0, device="cuda")]
    assert mu.muon_grad_norm(g)[0].item() == 4.0
    mu.muon_release()
    assert mu.muon_grad_norm(g)[0].item() == 4.0
