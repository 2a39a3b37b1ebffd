"""The linear-attention block's operators on another stream than the current one: what a call allocates is not memory that
work waiting on the current stream still writes, and the results are the current stream's."""
import pytest
import torch

from test_gpu_linattn import dev, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible")


def leaves(got):
    for t in got.values() if isinstance(got, dict) else got if isinstance(got, tuple) else (got,):
        if isinstance(t, torch.Tensor):
            yield t


def cases():
    import selective_state_space_41_amd as V
    gen = torch.Generator(device="cuda").manual_seed(1)
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    x, w = rnd(3000, 1024), rnd(1024)
    rstd = torch.rsqrt(x.square().mean(-1) + 1e-5)
    p = make(2, 4, 600, 4, 2, 64, 64, "bf16")
    t = {k: dev(p, k) for k in ("q", "k", "v", "g", "dout", "s0")}
    pos, f, axis = rnd(600, 1), rnd(32).abs(), torch.zeros(32, dtype=torch.int32, device="cuda")
    one = [t[k][:, 0].contiguous() for k in "qkvg"]
    states = [t["s0"].clone(), t["s0"].clone()]  # one for each call, made before it
    return dict(rmsnorm_fwd=lambda **k: V.rmsnorm_fwd(x, w, residual=x, out_dtype=torch.float8_e4m3fn, **k),
                rmsnorm_bwd=lambda **k: V.rmsnorm_bwd(x, x, w, rstd, **k),
                rope_axes=lambda **k: V.rope_axes(t["q"], t["k"], pos, f, axis, **k),
                linattn_fwd=lambda **k: V.linattn_fwd(t["q"], t["k"], t["v"], t["g"], initial_state=t["s0"], **k),
                linattn_bwd=lambda **k: V.linattn_bwd(t["q"], t["k"], t["v"], t["g"], t["dout"], initial_state=t["s0"], **k),
                linattn_step=lambda **k: V.linattn_step(*one, states.pop(), **k))


@pytest.mark.parametrize("name", ["rmsnorm_fwd", "rmsnorm_bwd", "rope_axes", "linattn_fwd", "linattn_bwd", "linattn_step"])
def test_memory_of_the_current_stream(name):
    call = cases()[name]
    want = [t.clone() for t in leaves(call())]
    sizes = [t.numel() * t.element_size() for t in want]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    print(f"[streams] {name}", flush=True)
    # blocks of the outputs' sizes, freed with a write to them still waiting on the current stream
    held = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(2)]
    torch.cuda._sleep(200_000_000)
    for h in held:
        h.fill_(7)
    del held
    got = call(stream=side)
    side.synchronize()
    torch.cuda.synchronize()
    for a, b in zip(want, leaves(got)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_given_tensors_and_prepared_calls():
    import selective_state_space_41_amd as V
    p = make(5, 2, 100, 2, 2, 32, 32, "f32")
    t = {k: dev(p, k) for k in ("q", "k", "v", "g", "s0")}
    want = V.linattn_fwd(t["q"], t["k"], t["v"], t["g"], initial_state=t["s0"])
    side = torch.cuda.Stream()
    out, state = torch.zeros_like(want[0]), t["s0"].clone()
    side.wait_stream(torch.cuda.current_stream())
    got = V.linattn_fwd(t["q"], t["k"], t["v"], t["g"], initial_state=state, final_state=state, out=out, stream=side)
    assert got[0] is out and got[1] is state
    run, out2, last = V.linattn_fwd(t["q"], t["k"], t["v"], t["g"], initial_state=t["s0"], stream=side, prepare=True)
    run()
    torch.cuda.current_stream().wait_stream(side)
    for a, b in ((want[0], out), (want[1], state), (want[0], out2), (want[1], last)):
        assert torch.equal(a, b)
