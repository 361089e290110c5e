"""GPU test of README's example of the layers' products: it runs, its gradients
are the definition's, and no two micro-batches drop the same places."""
import os
import re

import numpy as np
import pytest

from gpu_helpers import rel_f, torch_mod
from linear_helpers import make, values
from oracle import linear_oracle as lo

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    """The block of README that accumulates the gradients of an MLP."""
    with open(os.path.join(ROOT, "README.md")) as f:
        blocks = re.findall(r"```python\n(.*?)```", f.read(), flags=re.S)
    found = [b for b in blocks if "muon_linear_dw" in b]
    assert len(found) == 1
    return found[0]


def test_micro_batches_of_the_example():
    torch = torch_mod()
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import optimizer_muon_step_amd as mu
    rng = np.random.default_rng(70)
    tokens, width, hidden, seed, step = 96, 64, 256, 1234, 5
    w1, w2 = make(rng, (width, hidden), "fp32", 0.1).clone(), make(rng, (hidden, width), "fp32", 0.1).clone()
    b1, b2 = make(rng, (1, hidden), "fp32", 0.1)[0].clone(), make(rng, (1, width), "fp32", 0.1)[0].clone()
    before = [values(t.bfloat16()) if t.dim() == 2 else values(t) for t in (w1, b1, w2, b2)]
    batches = [tuple(make(rng, (tokens, width), "bf16").clone() for _ in range(3)) for _ in range(3)]  # x, r, dy
    momentum = [torch.zeros_like(w) for w in (w1, w2)]
    dw1, dw2, db1, db2 = (torch.zeros_like(t) for t in (w1, w2, b1, b2))
    grads = (dw1, db1, dw2, db2)
    numbers = []

    class Recorded:
        def __getattr__(self, name):
            def call(*args, **kw):
                if "rng" in kw or name == "muon_dropout":
                    numbers.append((name, kw["rng"] if "rng" in kw else args[2], kw.get("site", 0)))
                return getattr(mu, name)(*args, **kw)
            return call

    names = dict(torch=torch, mu=Recorded(), batches=batches, w1=w1, w2=w2, b1=b1, b2=b2, dw1=dw1, dw2=dw2, db1=db1, db2=db2,
                 momentum=momentum, tokens=tokens, seed=seed, step=step)
    exec(compile(example(), "README.md", "exec"), names)
    torch.cuda.synchronize()
    forward = [n for n in numbers if n[0] == "muon_linear"]
    backward = [n for n in numbers if n[0] == "muon_dropout"]
    assert len(forward) == len(set(forward)) == len(batches), "a mask of its own for every micro-batch"
    assert [n[1:] for n in forward] == [n[1:] for n in backward], "the same mask in both passes"
    # the definition in 64 bits; the values stored in 16 bits on the way are off by half a step each, as in
    # tests/test_gpu_layer_training.py: ten half steps for whole tensors
    want = [0, 0, 0, 0]
    v1, c1, v2, c2 = before
    for (x, r, dy), (_, (s, count), site) in zip(batches, forward):
        f = lo.keep_factor(tokens, width, 0.1, s, count, site)
        h, z = lo.linear(values(x), v1, c1, "gelu")
        dz2 = lo.through(values(dy), factor=f)
        dz1 = lo.through(dz2 @ v2.T, "gelu", z)
        for i, g in enumerate((values(x).T @ dz1, dz1.sum(0), h.T @ dz2, dz2.sum(0))):
            want[i] = want[i] + g
    for got, ref in zip(grads, want):
        assert rel_f(values(got), ref) <= 10 * 2.0 ** -8
    assert not np.array_equal(values(w1.bfloat16()), v1), "the step was made"
