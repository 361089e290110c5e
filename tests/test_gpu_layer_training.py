"""GPU tests of the layers' products, dropout, clipping and the optimizer steps
together: one MLP block with its residual, forward, backward, and stepped by
muon_step and muon_adamw_step, eagerly and as a captured graph."""
import numpy as np
import pytest

from gpu_helpers import rel_f, say, torch_mod
from linear_helpers import make, values
from oracle import linear_oracle as lo

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


P, SITE1, SITE2 = 0.1, 1, 2


class Block:
    """x + drop(drop(act(x w1 + b1)) w2 + b2), fp32 weights, 16-bit activations."""

    def __init__(self, rng, width, hidden, act, order="rows"):
        torch = torch_mod()
        self.act = act
        self.w1, self.w2 = make(rng, (width, hidden), "fp32", 0.05, order=order), make(rng, (hidden, width), "fp32", 0.05, order=order)
        self.w1, self.w2 = (t.clone(memory_format=torch.preserve_format) for t in (self.w1, self.w2))
        self.b1, self.b2 = make(rng, (1, hidden), "fp32", 0.1)[0].clone(), make(rng, (1, width), "fp32", 0.1)[0].clone()
        self.params = [self.w1, self.w2, self.b1, self.b2]
        self.grads = [torch.zeros_like(p) for p in self.params]

    def forward(self, mu, x, state):
        torch = torch_mod()
        self.z = torch.empty(*x.shape[:-1], self.w1.shape[1], dtype=x.dtype, device="cuda")
        self.h = mu.muon_linear(x, self.w1, self.b1, act=self.act, dropout=P, rng=state, site=SITE1, preact=self.z)
        return mu.muon_linear(self.h, self.w2, self.b2, dropout=P, rng=state, site=SITE2, residual=x)

    def backward(self, mu, x, dy, state, accumulate):
        g1, g2, h1, h2 = self.grads
        self.dz2 = mu.muon_dropout(dy, P, state, site=SITE2)
        mu.muon_linear_dw(self.h, self.dz2, g2, dbias=h2, accumulate=accumulate)
        self.dz1 = mu.muon_linear_dx(self.dz2, self.w2, act=self.act, preact=self.z, dropout=P, rng=state, site=SITE1)
        mu.muon_linear_dw(x, self.dz1, g1, dbias=h1, accumulate=accumulate)
        return mu.muon_linear_dx(self.dz1, self.w1, residual=dy)


def _exact(block, x, dy, kind, seed, step):
    """y and every gradient in fp64 from the weights' 16-bit values, nothing between rounded."""
    torch = torch_mod()
    t = {"bf16": torch.bfloat16, "fp16": torch.float16}[kind]
    xv, dyv = values(x).reshape(-1, x.shape[-1]), values(dy).reshape(-1, x.shape[-1])
    w1, w2 = (values(w.to(t)) for w in (block.w1, block.w2))
    f1 = lo.keep_factor(xv.shape[0], w1.shape[1], P, seed, step, SITE1)
    f2 = lo.keep_factor(xv.shape[0], w2.shape[1], P, seed, step, SITE2)
    h, z = lo.linear(xv, w1, values(block.b1), block.act, f1)
    y, _ = lo.linear(h, w2, values(block.b2), None, f2, xv)
    dz2 = lo.through(dyv, factor=f2)
    dz1 = lo.through(dz2 @ w2.T, block.act, z, f1)
    return y, [xv.T @ dz1, h.T @ dz2, dz1.sum(0), dz2.sum(0)], dyv + dz1 @ w1.T


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("act", ["gelu", "relu2"])
@pytest.mark.parametrize("shape,width,hidden,order", [((4, 96), 64, 256, "rows"), ((3, 77), 50, 203, "columns"), ((1, 1), 24, 40, "rows")])
def test_block_gradients(kind, act, shape, width, hidden, order):
    """Against fp64 without roundings between.  The values stored in 16 bits on
    the way (z, h, dz2, dz1, and the result) are each off by at most half a step,
    relative; what one of them does to a later value is of its own relative size
    times at most 2 (relu2 squares z and its slope is proportional to it; GELU's
    z act'(z) / act(z) and z act''(z) / act'(z) stay near or below 2 where the values are not
    small).  Five roundings, each times 2, bound the relative error of whole
    tensors at 10 half steps."""
    torch = torch_mod()
    import optimizer_muon_step_amd as mu
    rng = np.random.default_rng(sum(shape) + width)
    block = Block(rng, width, hidden, act, order)
    x = make(rng, (shape[0] * shape[1], width), kind).view(*shape, width)
    dy = make(rng, (shape[0] * shape[1], width), kind, 0.5).view(*shape, width)
    state = torch.tensor([41, 7], dtype=torch.int64, device="cuda")
    y = block.forward(mu, x, state)
    dx = block.backward(mu, x, dy, state, accumulate=False)
    want_y, want, want_dx = _exact(block, x, dy, kind, 41, 7)
    bound = 10 * {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}[kind]
    for name, got, ref in [("y", y, want_y), ("dx", dx, want_dx)] + list(zip(("dw1", "dw2", "db1", "db2"), block.grads, want)):
        err = rel_f(values(got).reshape(ref.shape), ref)
        say(f"  {kind} {act} {name}: relF {err:.1e}")
        assert err <= bound, (name, err)


def test_micro_batches_add_up():
    """Two halves of a batch, the second added to the first, against the whole:
    the mask goes by the rows of each call, so without dropout."""
    torch = torch_mod()
    import optimizer_muon_step_amd as mu
    rng = np.random.default_rng(8)
    x, dz = make(rng, (600, 72), "bf16"), make(rng, (600, 136), "bf16")
    whole, halves = torch.empty(72, 136, device="cuda"), torch.empty(72, 136, device="cuda")
    b_whole, b_halves = torch.empty(136, device="cuda"), torch.empty(136, device="cuda")
    mu.muon_linear_dw(x, dz, whole, dbias=b_whole)
    mu.muon_linear_dw(x[:300], dz[:300], halves, dbias=b_halves)
    mu.muon_linear_dw(x[300:], dz[300:], halves, dbias=b_halves, accumulate=True)
    xv, dzv = values(x), values(dz)
    # either is off by at most 600 steps of 2^-23 of the absolute sum
    bound = 2 * 601 * 2.0 ** -23 * (np.abs(xv).T @ np.abs(dzv))
    assert (np.abs(values(whole) - values(halves)) <= bound).all()
    assert (np.abs(values(b_whole) - values(b_halves)) <= 2 * 601 * 2.0 ** -23 * np.abs(dzv).sum(0)).all()


def _train_step(mu, block, x, dy, state, moments, momentum):
    block.forward(mu, x, state)
    block.backward(mu, x, dy, state, accumulate=False)
    record = mu.muon_grad_norm(block.grads, 1.0)
    mu.muon_step(block.params[:2], block.grads[:2], momentum, lr=0.02, clip=record)
    mu.muon_adamw_step(block.params[2:], block.grads[2:], moments[0], moments[1], 1e-3, step=5, clip=record)
    state[1:].add_(1)
    return record


@pytest.mark.parametrize("tokens,width,hidden", [(128, 64, 256), (300, 50, 203)])
def test_captured_training_equals_eager(tokens, width, hidden):
    """A whole step in one graph: weights, gradients and moments after each replay
    are those of eager steps, bit for bit, masks and all; in between the program
    makes eager calls of the same operators on other tensors."""
    torch = torch_mod()
    import optimizer_muon_step_amd as mu

    def setup():
        rng = np.random.default_rng(50)
        block = Block(rng, width, hidden, "gelu")
        x, dy = make(rng, (tokens, width), "bf16"), make(rng, (tokens, width), "bf16", 0.5)
        state = torch.tensor([9, 0], dtype=torch.int64, device="cuda")
        moments = [[torch.zeros_like(b) for b in block.params[2:]] for _ in range(2)]
        return block, x.clone(), dy.clone(), state, moments, [torch.zeros_like(w) for w in block.params[:2]]

    eager, captured = setup(), setup()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _train_step(mu, *captured)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    _train_step(mu, *eager)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        record = _train_step(mu, *captured)
    other = setup()
    for rep in range(4):
        graph.replay()
        want = _train_step(mu, *eager)
        _train_step(mu, *other)
        torch.cuda.synchronize()
        assert torch.equal(record, want)
        for a, b in zip(captured[0].params + captured[0].grads + captured[5] + sum(captured[4], []) + [captured[3]],
                        eager[0].params + eager[0].grads + eager[5] + sum(eager[4], []) + [eager[3]]):
            assert torch.equal(a, b), f"replay {rep}"
    assert int(captured[3][1]) == 5


def test_two_graphs_do_not_share_workspaces():
    """Products that copy operands and split sums, captured twice and replayed at the same time on two streams."""
    torch = torch_mod()
    import optimizer_muon_step_amd as mu
    rng = np.random.default_rng(60)
    sets = [(make(rng, (9000, 67), "bf16"), make(rng, (9000, 131), "bf16"), make(rng, (67, 131), "fp32")) for _ in range(2)]
    graphs, outs, streams = [], [], [torch.cuda.Stream() for _ in sets]
    for x, dz, w in sets:
        g, dw = torch.cuda.CUDAGraph(), torch.empty(67, 131, device="cuda")
        with torch.cuda.graph(g):
            y = mu.muon_linear(x, w)
            dx = mu.muon_linear_dx(dz, w)
            mu.muon_linear_dw(x, dz, dw)
        graphs.append(g)
        outs.append((y, dx, dw))
    for _ in range(5):
        for t in sum(outs, ()):
            t.zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for (x, dz, w), (y, dx, dw) in zip(sets, outs):
            want = torch.empty_like(dw)
            mu.muon_linear_dw(x, dz, want)
            assert torch.equal(y, mu.muon_linear(x, w)) and torch.equal(dx, mu.muon_linear_dx(dz, w)) and torch.equal(dw, want)


def test_timing_families():
    import optimizer_muon_step_amd as mu
    rng = np.random.default_rng(61)
    x, w, dz = make(rng, (64, 7), "bf16"), make(rng, (7, 72), "bf16"), make(rng, (64, 72), "bf16")
    dw = make(rng, (7, 72), "fp32")  # x is copied first
    for kernel, call, launches in ((mu.KERNEL_LINEAR, lambda: mu.muon_linear(x, w), 2),
                                   (mu.KERNEL_LINEAR_DW, lambda: mu.muon_linear_dw(x, dz, dw), 2),
                                   (mu.KERNEL_DROPOUT, lambda: mu.muon_dropout(x, 0.5, (1, 2)), 1)):
        mu.muon_timing_enable(kernel)
        call()
        ms, count = mu.muon_timing_read()
        mu.muon_timing_enable(-1)
        assert count == launches and ms > 0
