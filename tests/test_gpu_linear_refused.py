"""GPU tests of refused calls of the layer products: a refusal leaves the
device's memory alone."""
import pytest

from gpu_helpers import torch_mod

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


def test_a_refused_call_allocates_no_workspace():
    """Calls that would need a workspace (copies, splits), refused for another reason."""
    torch = torch_mod()
    import optimizer_muon_step_amd as mu
    x, w = torch.zeros(9000, 67, dtype=torch.bfloat16, device="cuda"), torch.zeros(67, 5, dtype=torch.bfloat16, device="cuda")
    z = torch.zeros(9000, 5, dtype=torch.bfloat16, device="cuda")
    long, deep = torch.zeros(64, 6400, dtype=torch.bfloat16, device="cuda"), torch.zeros(6400, 1600, dtype=torch.bfloat16, device="cuda")
    y = torch.zeros(64, 1600, dtype=torch.bfloat16, device="cuda")
    dw = torch.zeros(67, 5, device="cuda")
    for match, call in [("overlaps preact", lambda: mu.muon_linear(x, w, out=z, preact=z)),
                        ("dropout = 1", lambda: mu.muon_linear(x, w, out=z, dropout=1.0, rng=(1, 2))),
                        ("overlaps preact", lambda: mu.muon_linear(long, deep, out=y, preact=y)),
                        ("come together", lambda: mu.muon_linear_dx(z, w, act="gelu", out=x)),
                        ("overlaps dbias", lambda: mu.muon_linear_dw(x, z, dw, dbias=dw.view(-1)[:5]))]:
        torch.cuda.reset_peak_memory_stats()
        before = torch.cuda.memory_allocated()
        with pytest.raises(mu.MuonError, match=match) as refusal:
            call()
        assert refusal.value.code == -1
        assert torch.cuda.max_memory_allocated() == before, match
    # the same sizes, allowed: a workspace
    for call in (lambda: mu.muon_linear(x, w, out=z), lambda: mu.muon_linear(long, deep, out=y), lambda: mu.muon_linear_dw(x, z, dw)):
        torch.cuda.reset_peak_memory_stats()
        before = torch.cuda.memory_allocated()
        call()
        assert torch.cuda.max_memory_allocated() > before and torch.cuda.memory_allocated() == before
    torch.cuda.synchronize()


def test_refusals_do_not_depend_on_the_memory_left():
    """2^28 rows of 127 would be copied to 64 GB: an overlap is what is said, whether they are there or not."""
    torch = torch_mod()
    import optimizer_muon_step_amd as mu
    m = 1 << 28
    x = torch.zeros(m + 127, dtype=torch.bfloat16, device="cuda").as_strided((m, 127), (1, 1))
    w, y = torch.zeros(127, 5, dtype=torch.bfloat16, device="cuda"), torch.empty(m, 5, dtype=torch.bfloat16, device="cuda")
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    with pytest.raises(mu.MuonError, match="y overlaps preact"):
        mu.muon_linear(x, w, out=y, preact=y)
    assert torch.cuda.max_memory_allocated() == before


def test_the_per_thread_stream_is_refused():
    torch = torch_mod()
    import optimizer_muon_step_amd as mu
    x, w = torch.zeros(64, 67, dtype=torch.bfloat16, device="cuda"), torch.zeros(67, 131, dtype=torch.bfloat16, device="cuda")
    y, dw = torch.zeros(64, 131, dtype=torch.bfloat16, device="cuda"), torch.zeros(67, 131, device="cuda")
    per_thread = torch.cuda.ExternalStream(2)
    calls = [lambda **s: mu.muon_linear(x, w, **s), lambda **s: mu.muon_linear_dx(y, w, **s),
             lambda **s: mu.muon_linear_dw(x, y, dw, **s), lambda **s: mu.muon_dropout(x, 0.1, (1, 2), **s)]
    for call in calls:
        with pytest.raises(ValueError, match="hipStreamPerThread"):
            call(stream=per_thread)
        with torch.cuda.stream(per_thread), pytest.raises(ValueError, match="hipStreamPerThread"):
            call()
        call(stream=torch.cuda.Stream())
        call(stream=0)
    torch.cuda.synchronize()
