"""Memory of the layer's calls on a stream that is not the current one: an output's block is not taken
from work that is still to run, nor given away before work on it has run."""
from __future__ import annotations

import pytest

import synth
from delta_ref import draw
from gpu_util import make_layer

pytestmark = pytest.mark.gpu

N, B, H = 4096, 2, 4
WAIT = 400_000_000  # clock cycles, some 0.2 s: longer than everything behind it takes


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from rank_state_read_b200 import build
    build.build()


@pytest.fixture()
def layer():
    import torch
    cfg = synth.config(3).replace(B=B, H=H, Hqk=H, G=1, n_dense=1)
    made = make_layer(cfg, synth.layer_rank_table(cfg), synth.basis(cfg), synth.init_state(cfg, range(B)))
    made.norm_weight = torch.ones(cfg.V, device="cuda")
    yield made
    torch.cuda.synchronize()
    made.close()


def calls(layer, seed):
    """Calls that allocate what they return, all of it [N][H][V] fp32."""
    import torch
    V = layer.plan.desc.value_dim
    x = draw(seed, N, B, H, H, V)
    d = {m: torch.from_numpy(x[m]).cuda() for m in ("q", "k", "v", "a", "beta")}
    cu = torch.tensor([0, 1000, N], dtype=torch.int32, device="cuda")
    slot = torch.full((N,), -1, dtype=torch.int32, device="cuda")
    slot[:2] = torch.tensor([1, 0], dtype=torch.int32)
    z, y = torch.randn(N, H, V, device="cuda"), torch.randn(N, H, V, device="cuda")
    own = torch.empty(N, H, V, device="cuda")
    return {
        "prompt": lambda s: layer.prompt(cu, d["q"], d["k"], d["v"], d["a"], d["beta"], stream=s),
        "prompt_gate": lambda s: layer.prompt(cu, d["q"], d["k"], d["v"], d["a"], d["beta"], out=own, gate=z, stream=s),
        "step": lambda s: layer.step(d["q"], d["k"], d["v"], d["a"], d["beta"], slot=slot, stream=s),
        "norm": lambda s: layer.gated_norm(y, z, stream=s),
    }


@pytest.mark.parametrize("raw", [False, True], ids=["stream", "handle"])
@pytest.mark.parametrize("call", ["prompt", "prompt_gate", "step", "norm"])
def test_an_output_does_not_overwrite_what_the_current_stream_still_reads(layer, call, raw):
    import torch
    V = layer.plan.desc.value_dim
    run = calls(layer, 1)[call]
    s, cur = torch.cuda.Stream(), torch.cuda.current_stream()
    read = torch.zeros(N, H, V, device="cuda")
    run(s)  # what the first call loads is loaded
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    t = torch.full((N, H, V), 3.0, device="cuda")
    torch.cuda.synchronize()
    torch.cuda._sleep(WAIT)
    read.copy_(t)      # waits behind the sleep
    del t              # its block is free for the current stream, whose reader has not run
    out = run(s.cuda_stream if raw else s)
    assert not cur.query(), "the sleep was too short to show anything"
    torch.cuda.synchronize()
    assert bool((read == 3.0).all())
    layer.plan.check()
    assert out.shape == (N, H, V)


@pytest.mark.parametrize("raw", [False, True], ids=["stream", "handle"])
@pytest.mark.parametrize("call", ["prompt", "prompt_gate", "step", "norm"])
def test_an_output_outlives_its_readers_on_the_current_stream(layer, call, raw):
    import torch
    first, second = calls(layer, 1)[call], calls(layer, 2)[call]
    s, cur = torch.cuda.Stream(), torch.cuda.current_stream()
    handle = s.cuda_stream if raw else s
    torch.cuda.synchronize()
    out = first(handle)
    torch.cuda.synchronize()
    want, read = out.clone(), torch.zeros_like(out)  # step writes the first two rows
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    torch.cuda._sleep(WAIT)
    read.copy_(out)
    del out
    again = second(handle)
    assert not cur.query(), "the sleep was too short to show anything"
    torch.cuda.synchronize()
    assert torch.equal(read[:2], want[:2]) and not torch.equal(again[:2], want[:2])


def test_the_default_stream_by_its_handle(layer):
    """The handle of the current stream, 0 for the default one, as the stream argument."""
    import torch
    run = calls(layer, 3)["norm"]
    want = run(None)
    got = run(torch.cuda.current_stream().cuda_stream)
    assert torch.equal(got, want)


@pytest.mark.parametrize("call", ["prompt", "prompt_gate", "step", "norm"])
def test_captured_on_a_side_stream(layer, call):
    """A call on a stream that a capture forked: its output belongs to the graph and is what replays give."""
    import torch
    run = calls(layer, 4)[call]
    S0 = layer.S.clone()
    want = run(None)[:2].clone()
    S1 = layer.S.clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()  # the copies are made before the other stream writes the state
    run(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        side.wait_stream(torch.cuda.current_stream())
        out = run(side)
        torch.cuda.current_stream().wait_stream(side)
    for _ in range(2):
        layer.S.copy_(S0)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[:2], want) and torch.equal(layer.S, S1)
    layer.plan.check()
