"""GPU tests of the AdamW and Muon steps on clipped gradients, and of norm,
clip and steps together, as a training loop uses them.

g' is one fp32 product of the gradient and the record's factor, and the steps'
own arithmetic follows on g'.  So every comparison is bit for bit: AdamW with
the CPU oracle fed g', Muon with the library's own unclipped step fed g'."""
import math

import numpy as np
import pytest

from gpu_helpers import COEFFS, bf16_to_np, say, to_gpu, torch_mod
from oracle import adamw_oracle as ao
from oracle import grad_oracle as go

pytestmark = pytest.mark.gpu

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


def _bits_equal(got, want, tag):
    got = np.ascontiguousarray(got.cpu().numpy() if hasattr(got, "cpu") else got, np.float32).view(np.uint32)
    want = np.ascontiguousarray(want, np.float32).view(np.uint32)
    bad = np.flatnonzero(got.ravel() != want.ravel())
    assert bad.size == 0, f"{tag}: {bad.size} of {got.size} differ, first at {bad[:5]}"


SIZES = [1, 3, 4, 5, 63, 4095, 4096, 4097, 8193, 12289, 100_003, (7, 9), (33, 130), 0]


def _adamw_set(rng, sizes, kinds, offset=0):
    torch = torch_mod()

    def dev(a, dtype=torch.float32):
        flat = np.concatenate([np.zeros(offset, np.float32), a.ravel()])
        return torch.from_numpy(flat).to(dtype).cuda()[offset:].view(a.shape)

    out = []
    for i, s in enumerate(sizes):
        p, g, u = (rng.standard_normal(s).astype(np.float32) for _ in range(3))
        v = rng.random(s).astype(np.float32) * np.float32(1e-3)
        out.append(dict(p=p, u=u * np.float32(1e-2), v=v,
                        P=dev(p), G=dev(g, _dtype(kinds[i % len(kinds)])), U=dev(u * np.float32(1e-2)), V=dev(v)))
    return out


def _lists(ts):
    return [[t[k] for t in ts] for k in "PGUV"]


def _adamw_check(ts, factor, lr, betas, eps, wds, step):
    for i, t in enumerate(ts):
        g = go.clipped(t["G"].float().cpu().numpy(), factor)
        p, u, v = ao.adamw_step(t["p"], g, t["u"], t["v"], lr, betas[0], betas[1], eps, wds[i], step)
        for k, want in (("P", p), ("U", u), ("V", v)):
            _bits_equal(t[k], want, f"{k}[{i}]")


@pytest.mark.parametrize("kinds", [("fp32",), ("bf16",), ("fp16",), KINDS])
@pytest.mark.parametrize("offset", [0, 1])
def test_adamw_on_clipped_gradients(kinds, offset):
    import optimizer_muon_step_amd as mu
    ts = _adamw_set(np.random.default_rng(60), SIZES, kinds, offset)
    wds = [0.0 if i % 3 else 0.1 for i in range(len(ts))]
    P, G, U, V = _lists(ts)
    record = mu.muon_grad_norm(G, 5.0, scale=0.5)
    mu.muon_adamw_step(P, G, U, V, 1e-3, (0.9, 0.95), 1e-8, wds, step=7, clip=record)
    factor = record.cpu().numpy()[1]
    assert factor < 0.5
    _adamw_check(ts, factor, 1e-3, (0.9, 0.95), 1e-8, wds, 7)


@pytest.mark.parametrize("count,decays", [(99, 1), (100, 2), (101, 4), (250, 9)])
def test_adamw_many_tensors_and_decays(count, decays):
    """More tensors than one launch's table holds, more decays than it holds."""
    import optimizer_muon_step_amd as mu
    ts = _adamw_set(np.random.default_rng(61), [100 + 7 * k for k in range(count)], KINDS)
    wds = [0.01 * (i % decays) for i in range(count)]
    P, G, U, V = _lists(ts)
    record = mu.muon_grad_norm(G, 1.0)
    mu.muon_adamw_step(P, G, U, V, 1e-3, (0.9, 0.999), 1e-8, wds, step=1, clip=record)
    _adamw_check(ts, record.cpu().numpy()[1], 1e-3, (0.9, 0.999), 1e-8, wds, 1)


@pytest.mark.parametrize("kind", KINDS)
def test_adamw_long_call(kind):
    """A call long enough for the long chunks: equal to the unclipped
    step on gradients multiplied beforehand."""
    torch = torch_mod()
    import optimizer_muon_step_amd as mu
    gen = torch.Generator(device="cuda").manual_seed(69)
    sizes = [2 ** 26 + 4097, 8191, 8192, 8193, 3]
    say(f"[adamw long] {kind}")
    P, U, V, G = ([torch.randn(n, generator=gen, device="cuda") for n in sizes] for _ in "PUVG")
    V = [v.square_() for v in V]
    G = [g.to(_dtype(kind)) for g in G]
    record = mu.muon_grad_norm(G, 100.0)
    Pe, Ue, Ve = ([t.clone() for t in L] for L in (P, U, V))
    wds = [0.1, 0.0, 0.1, 0.3, 0.2]
    mu.muon_adamw_step(P, G, U, V, 1e-3, weight_decay=wds, step=3, clip=record)
    mu.muon_adamw_step(Pe, [g.float() * record[1] for g in G], Ue, Ve, 1e-3, weight_decay=wds, step=3)
    assert all(torch.equal(a, b) for a, b in zip(P + U + V, Pe + Ue + Ve))
    assert record[1].item() < 0.1


def test_adamw_without_a_record():
    """16-bit gradients as they are; fp32 ones under a factor of 1 give the
    plain step's bits."""
    torch = torch_mod()
    import optimizer_muon_step_amd as mu
    ts = _adamw_set(np.random.default_rng(62), SIZES, ("bf16", "fp16"))
    P, G, U, V = _lists(ts)
    mu.muon_adamw_step(P, G, U, V, 1e-3, weight_decay=0.1, step=3)
    _adamw_check(ts, np.float32(1.0), 1e-3, (0.9, 0.999), 1e-8, [0.1] * len(ts), 3)
    ts = _adamw_set(np.random.default_rng(63), SIZES, ("fp32",))
    P, G, U, V = _lists(ts)
    Pe, Ue, Ve = ([t.clone() for t in L] for L in (P, U, V))
    record = mu.muon_grad_norm(G, math.inf)
    mu.muon_adamw_step(P, G, U, V, 1e-3, weight_decay=0.1, step=3, clip=record)
    mu.muon_adamw_step(Pe, G, Ue, Ve, 1e-3, weight_decay=0.1, step=3)
    assert all(torch.equal(a, b) for a, b in zip(P + U + V, Pe + Ue + Ve))


@pytest.mark.parametrize("bad", [math.inf, math.nan])
@pytest.mark.parametrize("max_norm", [1.0, math.inf])
def test_steps_skip_a_norm_that_is_not_finite(bad, max_norm):
    torch = torch_mod()
    import optimizer_muon_step_amd as mu
    rng = np.random.default_rng(64)
    ts = _adamw_set(rng, [5000, 77], ("fp32", "bf16"))
    ts[1]["G"][5] = bad
    W, M = ([to_gpu(rng.standard_normal(s).astype(np.float32)) for s in ((96, 200), (300, 40))] for _ in "WM")
    W[0][0, 0] = -0.0
    Gm = [to_gpu(rng.standard_normal(w.shape).astype(np.float32)) for w in W]
    X = [torch.ones(w.shape, dtype=torch.bfloat16, device="cuda") for w in W]
    P, G, U, V = _lists(ts)
    keep = [t.clone() for t in P + U + V + W + M]
    record = mu.muon_grad_norm(G + Gm, max_norm)
    assert not torch.isfinite(record[0])
    mu.muon_adamw_step(P, G, U, V, 1e-3, weight_decay=0.1, step=3, clip=record)
    mu.muon_step(W, Gm, M, -0.02, 0.95, 5, COEFFS, updates=X, clip=record)
    assert all(torch.equal(a.view(torch.int32), b.view(torch.int32)) for a, b in zip(P + U + V + W + M, keep))
    assert all((x == 0).all() for x in X)


SHAPES = [[(256, 512)], [(96, 200), (300, 40), (1, 7), (5, 1)], [(768, 2304), (768, 768), (2000, 768)],
          [(1500, 2800), (2048, 2048)], [(4200, 1030)]]


@pytest.mark.parametrize("shapes", SHAPES)
@pytest.mark.parametrize("ns_steps", [0, 5])
def test_muon_on_clipped_gradients(shapes, ns_steps):
    """Equal to the unclipped step on gradients multiplied beforehand, bit for bit."""
    torch = torch_mod()
    import optimizer_muon_step_amd as mu
    rng = np.random.default_rng(65)
    say(f"[muon clip] {shapes}")
    W, G, M = ([to_gpu(rng.standard_normal(s).astype(np.float32)) for s in shapes] for _ in "WGM")
    We, Me = [t.clone() for t in W], [t.clone() for t in M]
    X, Xe = ([torch.zeros(s, dtype=torch.bfloat16, device="cuda") for s in shapes] for _ in "ab")
    record = mu.muon_grad_norm(G, 3.0)
    Ge = [g * record[1] for g in G]
    mu.muon_step(W, G, M, 0.02, 0.95, ns_steps, COEFFS, updates=X, clip=record)
    mu.muon_step(We, Ge, Me, 0.02, 0.95, ns_steps, COEFFS, updates=Xe)
    for a, b in zip(W + M + X, We + Me + Xe):
        assert torch.equal(a, b)
    assert bf16_to_np(X[0]).any()


def test_muon_clip_schedule_and_lanes():
    torch = torch_mod()
    import optimizer_muon_step_amd as mu
    rng = np.random.default_rng(66)
    shapes = [(300, 500), (500, 300), (128, 700)]
    sched = [(4.0, -6.0, 3.0), (3.4445, -4.775, 2.0315), (2.0, -1.5, 0.5)]
    W, G, M = ([to_gpu(rng.standard_normal(s).astype(np.float32)) for s in shapes] for _ in "WGM")
    record = mu.muon_grad_norm(G, 3.0)
    Ge = [g * record[1] for g in G]
    states = [([t.clone() for t in W], [t.clone() for t in M]) for _ in range(3)]
    mu.muon_step(states[0][0], Ge, states[0][1], 0.02, 0.95, 3, sched)
    mu.muon_step(states[1][0], G, states[1][1], 0.02, 0.95, 3, sched, clip=record)
    mu.muon_set_lanes(3)
    mu.muon_step(states[2][0], G, states[2][1], 0.02, 0.95, 3, sched, clip=record)
    mu.muon_set_lanes(1)
    for s in states[1:]:
        assert all(torch.equal(a, b) for a, b in zip(s[0] + s[1], states[0][0] + states[0][1]))


def test_step_refusals():
    torch = torch_mod()
    import optimizer_muon_step_amd as mu
    W, G, M = (torch.ones(8, 8, device="cuda") for _ in "WGM")
    record = mu.muon_grad_norm([G])
    with pytest.raises(ValueError, match="record"):
        mu.muon_step([W], [G], [M], clip=record.double())
    with pytest.raises(ValueError, match="record"):
        mu.muon_adamw_step([W], [G], [M], [M.clone()], 1e-3, clip=1.0)
    with pytest.raises(mu.MuonError, match="overlaps"):
        mu.muon_step([W], [G], [M], clip=W.view(-1)[:2])
    with pytest.raises(mu.MuonError, match="overlaps"):
        mu.muon_adamw_step([W], [G], [M], [M.clone()], 1e-3, clip=M.view(-1)[:2])
    with pytest.raises(mu.MuonError, match="ns_steps"):
        mu.muon_step([W], [G], [M], ns_steps=-1, clip=record)
    with pytest.raises(mu.MuonError, match="ns_steps"):
        mu.muon_step([W], [G], [M], ns_steps=10 ** 9, clip=record)
    with pytest.raises(ValueError, match="element counts differ"):
        mu.muon_adamw_step([W], [G[:4]], [M], [M.clone()], 1e-3, clip=record)
    with pytest.raises(ValueError, match="contiguous"):
        mu.muon_adamw_step([W.t()[:, :5]], [G], [M], [M.clone()], 1e-3, clip=record)
    with pytest.raises(ValueError, match="same length"):
        mu.muon_adamw_step([W], [], [M], [M.clone()], 1e-3, clip=record)


def _training_state(rng):
    shapes = [(256, 512), (512, 256), (100, 60)]
    sizes = [768, 4097, 50_257, 3]
    W, M = [to_gpu(rng.standard_normal(s).astype(np.float32)) for s in shapes], [to_gpu(np.zeros(s, np.float32)) for s in shapes]
    P = [to_gpu(rng.standard_normal(n).astype(np.float32)) for n in sizes]
    U, V = ([to_gpu(np.zeros(n, np.float32)) for n in sizes] for _ in "UV")
    return shapes, sizes, W, M, P, U, V


def test_training_loop_fused_equals_clip_in_place():
    """Norm over both parameter sets, Muon and AdamW by its record: the same
    bits as clipping every gradient in place and stepping unclipped."""
    torch = torch_mod()
    import optimizer_muon_step_amd as mu
    rng = np.random.default_rng(67)
    shapes, sizes, W, M, P, U, V = _training_state(rng)
    We, Me, Pe, Ue, Ve = ([t.clone() for t in L] for L in (W, M, P, U, V))
    for step in range(1, 6):
        std = 10.0 ** rng.uniform(-4, 1)  # below the limit on some steps, above it on others
        Gw = [to_gpu((rng.standard_normal(s) * std).astype(np.float32)) for s in shapes]
        Gp = [to_gpu((rng.standard_normal(n) * std).astype(np.float32)) for n in sizes]
        Gc = [t.clone() for t in Gw + Gp]
        record = mu.muon_grad_norm(Gw + Gp, 1.0)
        mu.muon_step(W, Gw, M, 0.02, 0.95, 5, COEFFS, clip=record)
        mu.muon_adamw_step(P, Gp, U, V, 6e-4, (0.9, 0.95), 1e-8, 0.1, step=step, clip=record)
        again = mu.muon_grad_clip(Gc, 1.0)
        assert torch.equal(record, again)
        mu.muon_step(We, Gc[:len(shapes)], Me, 0.02, 0.95, 5, COEFFS)
        mu.muon_adamw_step(Pe, Gc[len(shapes):], Ue, Ve, 6e-4, (0.9, 0.95), 1e-8, 0.1, step=step)
        assert all(torch.equal(a, b) for a, b in zip(W + M + P + U + V, We + Me + Pe + Ue + Ve)), step


def test_training_step_on_16_bit_gradients():
    """muon_step takes fp32 gradients: 16-bit ones are clipped into fp32 first,
    which gives the bits of clipping as the steps read their exact fp32 copies."""
    torch = torch_mod()
    import optimizer_muon_step_amd as mu
    rng = np.random.default_rng(80)
    shapes, sizes, W, M, P, U, V = _training_state(rng)
    We, Me, Pe, Ue, Ve = ([t.clone() for t in L] for L in (W, M, P, U, V))
    k = len(shapes)
    G = [to_gpu(rng.standard_normal(s).astype(np.float32)).to(_dtype(kind))
         for s, kind in zip(shapes + [(n,) for n in sizes], ("bf16", "fp16", "bf16") * 3)]
    record = mu.muon_grad_norm(G, 1.0)
    before = [t.clone() for t in W + M]
    with pytest.raises(ValueError, match=r"grads\[0\]: expected a contiguous float32 tensor"):
        mu.muon_step(W, G[:k], M, clip=record)
    assert all(torch.equal(a, b) for a, b in zip(W + M, before))
    G32 = [torch.empty(t.shape, device="cuda") for t in G]
    mu.muon_grad_clip(G, 1.0, outs=G32)
    mu.muon_step(W, G32[:k], M, lr=0.02)
    mu.muon_adamw_step(P, G32[k:], U, V, 6e-4, step=1)
    mu.muon_step(We, [t.float() for t in G[:k]], Me, lr=0.02, clip=record)
    mu.muon_adamw_step(Pe, G[k:], Ue, Ve, 6e-4, step=1, clip=record)
    assert all(torch.equal(a, b) for a, b in zip(W + M + P + U + V, We + Me + Pe + Ue + Ve))


def test_captured_training_step_replays_like_eager():
    torch = torch_mod()
    import optimizer_muon_step_amd as mu
    rng = np.random.default_rng(68)
    shapes, sizes, W, M, P, U, V = _training_state(rng)
    fresh = [[to_gpu(rng.standard_normal(s).astype(np.float32)) for s in shapes + [(n,) for n in sizes]] for _ in range(5)]
    fresh[3][1][2, 2] = math.nan  # a replay that is skipped
    G = [t.clone() for t in fresh[0]]
    k = len(shapes)

    def step(W, M, P, U, V, G):
        record = mu.muon_grad_norm(G, 1.0)
        mu.muon_step(W, G[:k], M, 0.02, 0.95, 5, COEFFS, clip=record)
        mu.muon_adamw_step(P, G[k:], U, V, 6e-4, (0.9, 0.95), 1e-8, [0.1, 0.0, 0.1, 0.0], step=9, clip=record)
        return record

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(W, M, P, U, V, G)  # the Muon plan of these shapes
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    We, Me, Pe, Ue, Ve = ([t.clone() for t in L] for L in (W, M, P, U, V))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        record = step(W, M, P, U, V, G)
    for rep in range(5):
        for a, b in zip(G, fresh[rep]):
            a.copy_(b)
        graph.replay()
        eager = step(We, Me, Pe, Ue, Ve, [t.clone() for t in G])
        torch.cuda.synchronize()
        assert torch.equal(record.view(torch.int32), eager.view(torch.int32)), rep
        for a, b in zip(W + M + P + U + V, We + Me + Pe + Ue + Ve):
            assert torch.equal(a, b), f"replay {rep} differs from the eager step"
