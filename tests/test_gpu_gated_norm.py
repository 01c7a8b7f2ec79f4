"""The gated norm (sketchssm_gated_norm) against fp64: types, widths from one vector to the widest,
both orders, gates, strides, in place, infinities, refusals; and a layer's calls with it behind them.
"""
from __future__ import annotations

import numpy as np
import pytest

import oracle
import synth
from delta_ref import K, delta_ref, draw, norm_ref, state_tol
from gpu_util import TOL, make_layer, rel_err, to_dev

pytestmark = pytest.mark.gpu

TYPES = ("float32", "bfloat16", "float16")


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from rank_state_read_b200 import build
    build.build()


def tensors(rows, groups, width, xt, t, seed=0, weights=1, scale=1.0):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = (scale * torch.randn(rows, groups, width, generator=g, device="cuda")).to(getattr(torch, xt))
    z = torch.randn(rows, groups, width, generator=g, device="cuda").to(getattr(torch, t))
    w = 1 + 0.2 * torch.randn(*([width] if weights == 1 else [groups, width]), generator=g, device="cuda")
    return x, z, w


def check(out, x, z, w, eps=1e-6, activation="silu", gate_first=False):
    """fp32: the sum of squares takes at most width / 8 + 40 roundings on a term's way (half of them
    in the root), the rest about 12; the stored value is rounded once more."""
    import torch
    host = lambda t: None if t is None else t.double().cpu().numpy()
    ref = norm_ref(host(x), host(z), host(w), eps, activation, gate_first)
    tol = (x.shape[-1] / 16 + 32) * 2.0 ** -24 + (torch.finfo(out.dtype).eps / 2 if out.dtype != torch.float32 else 0)
    tiny = torch.finfo(out.dtype).tiny if out.dtype != torch.float16 else 2.0 ** -25  # fp16 subnormals: half a step
    got = host(out)
    assert np.all(np.abs(got - ref) <= tol * np.abs(ref) + tiny), np.max(np.abs(got - ref) / (np.abs(ref) + tiny))


@pytest.mark.parametrize("xt", TYPES)
@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("gate_first", [False, True])
def test_types_and_orders(xt, t, gate_first):
    import torch
    import rank_state_read_b200 as rs
    for activation in ("silu", "sigmoid"):
        x, z, w = tensors(5, 3, 128, xt, t, weights=3)
        out = torch.empty_like(z)
        rs.sketchssm_gated_norm(x, z, w, out, activation=activation, gate_first=gate_first)
        check(out, x, z, w, 1e-6, activation, gate_first)


@pytest.mark.parametrize("width", [8, 16, 56, 64, 72, 80, 128, 136, 256, 264, 512, 520, 1024, 1280, 2048, 2056, 8192, 8200, 16384])
@pytest.mark.parametrize("rows,groups", [(1, 1), (3, 5), (37, 2)])
def test_widths(width, rows, groups):
    import torch
    import rank_state_read_b200 as rs
    x, z, w = tensors(rows, groups, width, "float32", "bfloat16", seed=1)
    out = torch.full_like(z, 9)
    rs.sketchssm_gated_norm(x, z, w, out, eps=1e-5)
    check(out, x, z, w, 1e-5)


def test_without_a_gate_and_in_place():
    import torch
    import rank_state_read_b200 as rs
    x, z, w = tensors(6, 2, 80, "bfloat16", "bfloat16", seed=2)
    out = torch.empty_like(x)
    rs.sketchssm_gated_norm(x, None, w, out)
    check(out, x, None, w)
    want = torch.empty_like(x)
    rs.sketchssm_gated_norm(x, z, w, want)
    for target in (x, z):
        a, b = x.clone(), z.clone()
        rs.sketchssm_gated_norm(a, b, w, a if target is x else b)
        assert torch.equal(a if target is x else b, want)


def test_strides():
    import torch
    import rank_state_read_b200 as rs
    x, z, w = tensors(9, 3, 80, "float32", "float16", seed=3)
    xw = torch.full((9, 300), float("nan"), device="cuda")
    zw = torch.full((9, 264), float("nan"), device="cuda", dtype=torch.float16)
    ow = torch.full((9, 256), 4.0, device="cuda", dtype=torch.float16)
    xw[:, 4:244], zw[:, 16:256] = x.view(9, -1), z.view(9, -1)
    rs.sketchssm_gated_norm(xw[:, 4:244].view(9, 3, 80), zw[:, 16:256].view(9, 3, 80), w, ow[:, 8:248].view(9, 3, 80), gate_first=True)
    check(ow[:, 8:248].reshape(9, 3, 80), x, z, w, gate_first=True)
    assert bool((ow[:, :8] == 4).all()) and bool((ow[:, 248:] == 4).all())


def test_ends_of_the_range():
    """Zero groups, tiny and huge values, gates of +-infinity; NaN stays in its group."""
    import torch
    import rank_state_read_b200 as rs
    x, z, w = tensors(6, 2, 128, "float32", "float32", seed=4)
    x[0] = 0
    x[1] *= 1e-20
    x[2] *= 1e15
    z[3, 0] = float("-inf")
    z[3, 1] = 1e30
    z[4, 0] = -200.0
    x[5, 1, 7] = float("nan")
    out = torch.empty_like(z)
    rs.sketchssm_gated_norm(x, z, w, out)
    keep = [0, 1, 2]
    check(out[keep], x[keep], z[keep], w)
    check(out[5:, :1], x[5:, :1], z[5:, :1], w)
    assert bool((out[0] == 0).all()) and bool((out[3, 0] == 0).all()) and bool((out[4, 0].abs() < 1e-30).all())
    assert bool(torch.isfinite(out[3, 1]).all()) and bool(torch.isnan(out[5, 1]).all())


def test_refusals():
    import torch
    import rank_state_read_b200 as rs
    x, z, w = tensors(4, 2, 64, "bfloat16", "bfloat16")
    out = torch.full_like(z, 3)

    def refused(status, *args, **kw):
        with pytest.raises(rs.SketchSSMError) as e:
            rs.sketchssm_gated_norm(*args, **kw)
        assert e.value.status == status

    refused(3, x[..., :60].contiguous(), z[..., :60].contiguous(), w[:60].contiguous(), out[..., :60].contiguous())
    refused(1, x, z, w, out, eps=-1.0)
    refused(1, x, z, w, out, eps=float("nan"))
    odd = torch.zeros(4, 132, device="cuda", dtype=torch.bfloat16)
    refused(2, odd[:, :128].view(4, 2, 64), z, w, out)
    big = torch.zeros(1, 1, 16392, device="cuda")
    refused(3, big, big, torch.zeros(16392, device="cuda"), big)
    for args, err in (((x, z.float(), w, out), TypeError), ((x, z[:3], w, out), ValueError), ((x, z, w[:8], out), ValueError),
                      ((x.view(4, 128), z, w, out), TypeError), ((x, z, w.bfloat16(), out), TypeError),
                      ((x, z.transpose(0, 1), w, out), ValueError), ((x.cpu(), z, w, out), ValueError)):
        with pytest.raises(err):
            rs.sketchssm_gated_norm(*args)
    with pytest.raises(ValueError):
        rs.sketchssm_gated_norm(x, z, w, out, activation="relu")
    rs.sketchssm_gated_norm(x[:0], z[:0], w, out[:0])
    torch.cuda.synchronize()
    assert bool((out == 3).all())


def test_prompt_decode_step_and_norm_together():
    """A Gated DeltaNet layer as a server runs it: packed prompts into two of its rows with their
    outputs normed and gated, sketch decodes of all rows, a flush, then single tokens on two rows."""
    import torch
    cfg = synth.config(3).replace(B=3, H=4, Hqk=4, G=1, n_dense=1)
    H, V = cfg.H, cfg.V
    rank, omega = synth.layer_rank_table(cfg), synth.basis(cfg)
    layer = make_layer(cfg, rank, omega, synth.init_state(cfg, range(3)))
    w = np.random.default_rng(5).standard_normal(V).astype(np.float32)
    layer.norm_weight = torch.from_numpy(w).cuda()
    S = layer.S.double().cpu().numpy()
    lens, slot = [70, 9], [2, 0]
    x = draw(6, 79, 3, H, H, V)
    bf = {m: torch.from_numpy(x[m]).cuda().bfloat16() for m in "qkv"}
    gate = torch.randn(79, H, V, device="cuda").bfloat16()
    ab = {m: torch.from_numpy(x[m]).cuda() for m in ("a", "beta")}
    cu = torch.tensor([0, 70, 79], dtype=torch.int32, device="cuda")
    slots = torch.tensor(slot, dtype=torch.int32, device="cuda")
    y = layer._read(layer.prompt(cu, bf["q"], bf["k"], bf["v"], ab["a"], ab["beta"], slots), None, None)
    host = {m: t.double().cpu().numpy() for m, t in bf.items()}
    yr, S, _ = delta_ref([0, 70, 79], slot, host["q"], host["k"], host["v"], x["a"], x["beta"], S)
    top = np.sqrt((S * S).sum(2)).max()
    assert np.abs(layer.S.double().cpu().numpy() - S).max() <= state_tol(70) * top
    assert np.all(np.abs(y.double().cpu().numpy() - yr) <= 2 ** -8 * np.abs(yr) + 2 * state_tol(70) * top)
    out = layer.gated_norm(y, gate)
    check(out, y, gate, layer.norm_weight)

    orc = oracle.OracleLayer(cfg.kind, H=H, Hqk=H, K=K, V=V, W=cfg.W, G=1, rank=rank, omega=omega, S0=S)
    orc.flush(0)
    assert rel_err(layer.Y.cpu().numpy(), orc.Y) <= TOL
    for t in range(cfg.W):
        inp = synth.step_inputs(cfg, t, range(3))
        d = to_dev(inp)
        z = torch.randn(3, H, V, device="cuda")
        got = layer.decode(t, d["q"], d["k"], d["v"], d["a"], d["beta"], gate=z)
        want = orc.decode(t, inp)
        assert rel_err(layer.y.cpu().numpy(), want) <= TOL
        check(got, layer.y, z, layer.norm_weight)
    layer.flush(cfg.W)
    orc.flush(cfg.W)
    x = draw(7, 2, 3, H, H, V)
    d = {m: torch.from_numpy(x[m]).cuda() for m in ("q", "k", "v", "a", "beta")}
    y = layer.step(d["q"], d["k"], d["v"], d["a"], d["beta"], slot=torch.tensor([1, 2], dtype=torch.int32, device="cuda"))
    yr, S, _ = delta_ref([0, 1, 2], [1, 2], x["q"], x["k"], x["v"], x["a"], x["beta"], orc.S)
    assert rel_err(y.cpu().numpy(), yr) <= TOL and rel_err(layer.S.cpu().numpy(), S) <= TOL
    layer.plan.check()
    layer.close()


def test_mamba2_layer_norm_behind_every_read():
    """Mamba-2: the gate first, one norm and one weight a basis group; every kind of read takes it."""
    import torch
    cfg = synth.config(1).replace(B=3)
    layer = make_layer(cfg, synth.layer_rank_table(cfg), synth.basis(cfg), synth.init_state(cfg, range(3)))
    layer.norm_weight = torch.randn(cfg.H * cfg.V, device="cuda")
    layer.flush(0)
    shape = (3, cfg.G, cfg.H * cfg.V // cfg.G)
    d = to_dev(synth.step_inputs(cfg, 0, range(3)))
    z = torch.randn(3, cfg.H, cfg.V, device="cuda").bfloat16()
    zero = torch.zeros(3, dtype=torch.int32, device="cuda")
    for call in (lambda: layer.decode(0, d["q"], d["k"], d["v"], d["a"], gate=z),
                 lambda: layer.dense_decode(0, d["q"], d["k"], d["v"], d["a"], gate=z),
                 lambda: layer.decode_rows(zero, d["q"], d["k"], d["v"], d["a"], gate=z),
                 lambda: layer.standard_step(d["q"], d["k"], d["v"], d["a"], gate=z)):
        out = call()
        assert out.shape == z.shape and out.dtype == z.dtype
        check(out.view(shape), layer.y.view(shape), z.view(shape), layer.norm_weight.view(shape[1:]), gate_first=True)
    layer.norm_weight = None
    with pytest.raises(ValueError):
        layer.decode(0, d["q"], d["k"], d["v"], d["a"], gate=z)
    layer.close()


def test_layer_calls_on_another_stream():
    """The stream by argument: allocations and kernels of both calls belong to it."""
    import torch
    cfg = synth.config(3).replace(B=2, H=4, Hqk=4, G=1, n_dense=1)
    x = draw(8, 40, 2, 4, 4, cfg.V)
    d = {m: torch.from_numpy(x[m]).cuda() for m in ("q", "k", "v", "a", "beta")}
    cu = torch.tensor([0, 25, 40], dtype=torch.int32, device="cuda")
    z = torch.randn(40, 4, cfg.V, device="cuda")
    got = []
    for stream in (None, torch.cuda.Stream()):
        layer = make_layer(cfg, synth.layer_rank_table(cfg), synth.basis(cfg), synth.init_state(cfg, range(2)))
        layer.norm_weight = torch.ones(cfg.V, device="cuda")
        torch.cuda.synchronize()
        out = layer.prompt(cu, d["q"], d["k"], d["v"], d["a"], d["beta"], gate=z, stream=stream)
        torch.cuda.synchronize()
        got.append((out, layer.S, layer.Y))
        layer.plan.check()
    assert all(torch.equal(a, b) for a, b in zip(*got))


@pytest.mark.parametrize("t", ["bfloat16", "float32"])
@pytest.mark.parametrize("activation", ["silu", "sigmoid"])
@pytest.mark.parametrize("gate_first", [False, True])
def test_gates_next_to_nothing(t, activation, gate_first):
    """exp(-z) passes fp32's range at z = -88.7 and its reciprocal leaves the normal numbers at -87.3;
    z / (1 + exp(-z)) is one down to -91.9, and a weight brings results back from below."""
    import torch
    import rank_state_read_b200 as rs
    z = torch.linspace(-91.75, -80, 48, device="cuda").to(getattr(torch, t)).view(1, 6, 8).contiguous()
    x = torch.ones(1, 6, 8, device="cuda", dtype=z.dtype) * (2.0 ** 64 if gate_first else 1.0)
    w = torch.full((8,), 2.0 ** 30, device="cuda")
    out = torch.empty_like(z)
    eps = 1e-38 if gate_first else 1e-6
    rs.sketchssm_gated_norm(x, z, w, out, eps=eps, activation=activation, gate_first=gate_first)
    zz = z.double().cpu().numpy()
    ref = norm_ref(x.double().cpu().numpy(), zz, w.double().cpu().numpy(), eps, activation, gate_first)
    # the exponent z log2(e), up to 133, is off by 2^-17 before it is raised (relative 2^-17.5), or a
    # subnormal gate by half a step of 2^-149 (2^-17.6 of exp(-91.75)); a group's root takes as much on
    # again; then the rounding to the type
    tol = 2.0 ** -16.5 + torch.finfo(z.dtype).eps / 2
    low = 2.0 ** -149 * 2.0 ** 30
    got = out.double().cpu().numpy()
    assert np.all(np.abs(got - ref) <= tol * np.abs(ref) + (low if not gate_first else 0)), got / ref
