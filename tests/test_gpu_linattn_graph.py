"""Single tokens of linear attention in a HIP graph: the step, which changes its states in place, captured once and replayed
with new inputs and new slots, eager work of the same operators in between; every replay gives the eager recurrence."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_step_replayed(dtype):
    import selective_state_space_41_amd as V
    gen = torch.Generator(device="cuda").manual_seed(3)
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    B, pool, H, Hk, dk, dv, L = 5, 9, 4, 2, 64, 40, 70
    fixed = dict(q=rnd(B, Hk, dk).to(dtype), k=rnd(B, Hk, dk).to(dtype), v=rnd(B, H, dv).to(dtype), g=-rnd(B, H).abs(),
                 slots=torch.arange(B, dtype=torch.int32, device="cuda"))
    state, out = rnd(pool, H, dk, dv), torch.empty(B, H, dv, dtype=dtype, device="cuda")
    eager = state.clone()
    step = lambda x, s, o=None: V.linattn_step(x["q"], x["k"], x["v"], x["g"], s, slots=x["slots"], out=o)
    long = [rnd(1, L, Hk, dk).to(dtype), rnd(1, L, Hk, dk).to(dtype), rnd(1, L, H, dv).to(dtype), -rnd(1, L, H).abs()]
    want_long = V.linattn_fwd(*long)[0]
    warm = state.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(fixed, warm, out)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(fixed, state, out)
    for turn in range(6):
        for key in ("q", "k", "v"):
            fixed[key].copy_(rnd(*fixed[key].shape).to(dtype))
        fixed["g"].copy_(-rnd(B, H).abs())
        slots = torch.randperm(pool, generator=gen, device="cuda")[:B].to(torch.int32)
        slots[turn % B] = -1 if turn % 2 else pool  # a row without a state
        fixed["slots"].copy_(slots)
        want = step({k: v.clone() for k, v in fixed.items()}, eager)
        print(f"[linattn graph] replay {turn}", flush=True)
        graph.replay()
        assert torch.equal(V.linattn_fwd(*long)[0], want_long)  # eager work beside it
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(state, eager)
