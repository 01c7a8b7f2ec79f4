"""The gated delta rule on packed tokens (sketchssm_delta_chunk, sketchssm_delta_step) against the
definition in fp64: types, head layouts, lengths from 0 tokens on and around a chunk, ragged and
empty sequences, slots, strides, decays of 0 and 1, equal keys, padding, bad rows, streams, graphs.
"""
from __future__ import annotations

import numpy as np
import pytest

from delta_ref import K, delta_ref, draw, state_tol

pytestmark = pytest.mark.gpu

DTYPES = ("bfloat16", "float16", "float32")


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from rank_state_read_b200 import build
    build.build()


def make_plan(B, H, Hqk, V, kind="gdn"):
    import rank_state_read_b200 as rs
    return rs.Plan(kind, batch=B, heads=H, qk_heads=Hqk, key_dim=K, value_dim=V, window=16, groups=1,
                   basis_rows=64, rank_cap=64, rank=[rs.DENSE] * H)


def cum(lens):
    return [0] + np.cumsum(lens).tolist()


class Case:
    """Inputs on the GPU in their type, and the same values in fp64 on the host."""

    def __init__(self, lens, B, H, Hqk, V, dtype, *, slot=None, seed=0, unit=True, behind=0, change=None):
        import torch
        self.cu, self.slot = cum(lens), list(range(len(lens))) if slot is None else slot
        n = sum(lens) + behind
        x = draw(seed, n, B, H, Hqk, V, unit)
        if change:
            change(x)
        dt = getattr(torch, dtype)
        self.dev = {m: torch.from_numpy(t).cuda().to(dt if m in "qkv" else torch.float32) for m, t in x.items()}
        self.host = {m: t.double().cpu().numpy() for m, t in self.dev.items()}
        self.dev["y"] = torch.full((n, H, V), 7.0, device="cuda", dtype=dt)
        self.cu_d = torch.tensor(self.cu, dtype=torch.int32, device="cuda")
        self.slot_d = torch.tensor(self.slot, dtype=torch.int32, device="cuda")
        self.longest = max(lens) if lens else 0
        self.eps = torch.finfo(dt).eps / 2 if dtype != "float32" else 0.0
        self.plan = make_plan(B, H, Hqk, V)

    def args(self):
        return [self.dev[m] for m in ("q", "k", "v", "a", "beta", "S", "y")]

    def check(self, normalize=False, scale=1.0, report=None, grow=1.0):
        import torch
        torch.cuda.synchronize()
        h = self.host
        y, S, touched = delta_ref(self.cu, self.slot, h["q"], h["k"], h["v"], h["a"], h["beta"], h["S"], normalize, scale)
        got_y, got_S = self.dev["y"].double().cpu().numpy(), self.dev["S"].double().cpu().numpy()
        assert np.all(got_y[~touched] == 7.0), "rows without a token were written"
        idle = [s for s in range(S.shape[0]) if not any(t == s and self.cu[i + 1] > self.cu[i] for i, t in enumerate(self.slot))]
        assert np.array_equal(got_S[idle], h["S"][idle]), "states without a token were written"
        top = max(np.sqrt((S * S).sum(2)).max(), np.sqrt((h["S"] ** 2).sum(2)).max())
        tol = grow * state_tol(self.longest) * top
        assert np.abs(got_S - S).max() <= tol, ("S", np.abs(got_S - S).max() / top)
        # |q| <= 1 before the scale; one rounding of y
        qn = scale * (1.0 if normalize else np.sqrt((h["q"] ** 2).sum(-1)).max())
        off = np.abs(got_y - y)[touched] - self.eps * np.abs(y[touched])
        assert off.max(initial=0) <= tol * qn * (1 + self.eps), ("y", off.max() / top)


def run_chunk(c, **kw):
    import rank_state_read_b200 as rs
    rs.sketchssm_delta_chunk(c.plan, c.cu_d, *c.args(), slot=c.slot_d, **kw)


LENGTHS = [[1], [5], [63], [64], [65], [128], [200], [1, 0, 64, 17], [0, 0, 3], [130, 1, 63, 129, 2], [0]]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("lens", LENGTHS, ids=str)
def test_chunk_lengths(dtype, lens):
    c = Case(lens, len(lens) + 1, 2, 2, 128, dtype, slot=list(range(len(lens), 0, -1)), seed=1, behind=3)
    run_chunk(c)
    c.plan.check()
    c.check()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("H,Hqk,V", [(1, 1, 128), (6, 2, 80), (4, 1, 16), (3, 3, 144), (2, 1, 256), (5, 5, 96), (4, 2, 112), (1, 1, 16)])
def test_chunk_head_layouts(dtype, H, Hqk, V):
    c = Case([70, 0, 131], 3, H, Hqk, V, dtype, seed=2)
    run_chunk(c, scale=0.25)
    c.check(scale=0.25)


@pytest.mark.parametrize("dtype", DTYPES)
def test_chunk_normalizes_q_and_k(dtype):
    def change(x):
        x["q"][3] = 0  # a zero row stays zero
        x["k"][70] = 0
        x["k"][5] *= 40  # long and short rows
        x["q"][9] *= 2.0 ** -6
    c = Case([100, 33], 2, 4, 2, 128, dtype, unit=False, seed=3, change=change)
    run_chunk(c, normalize_qk=True, scale=K ** -0.5)
    c.check(normalize=True, scale=K ** -0.5)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("what", ["a0", "a1", "beta0", "beta1", "a_tiny", "mixed"])
def test_chunk_gates_at_their_ends(dtype, what):
    """Decays of 0 (all before is forgotten), 1 and next to nothing, betas of 0 and 1."""
    def change(x):
        n = x["a"].shape[0]
        if what == "a0":
            x["a"][::7] = 0
        if what == "a1":
            x["a"][:] = 1
        if what == "beta0":
            x["beta"][:] = 0
        if what == "beta1":
            x["beta"][:] = 1
        if what == "a_tiny":
            x["a"][:] = 1e-30
            x["a"][1::3] = 1e-42  # a subnormal
        if what == "mixed":
            x["a"][: n // 2] = 0
            x["a"][n // 2:] = 1
    c = Case([150, 64], 2, 2, 2, 128, dtype, seed=4, change=change)
    run_chunk(c)
    # without decay the errors of all 150 tokens stay
    c.check(grow=151 / 64 if what in ("a1", "mixed") else 1.0)


@pytest.mark.parametrize("dtype", DTYPES)
def test_chunk_equal_keys(dtype):
    """Every token writes to the same key with beta = 1: the state forgets what it held there, and the
    triangular system of a chunk is the hardest that unit keys make."""
    def change(x):
        x["k"][:] = 0
        x["k"][:, :, 5] = 1
        x["beta"][:] = 1
        x["a"][:] = 1
    c = Case([130], 1, 2, 2, 128, dtype, seed=5, change=change)
    run_chunk(c)
    c.check(grow=131 / 64)


@pytest.mark.parametrize("dtype", DTYPES)
def test_values_of_very_different_size(dtype):
    """Columns and tokens whose values differ by 2^24: each is as exact as its own column."""
    def change(x):
        x["v"][:, :, :40] *= 2.0 ** -12
        x["S"][..., :40] *= 2.0 ** -12
        x["v"][:, :, 40:60] *= 2.0 ** 12
        x["S"][..., 40:60] *= 2.0 ** 12
    c = Case([90], 1, 2, 2, 128, dtype, seed=6, change=change if dtype != "float16" else
             lambda x: (x["v"][:, :, :40].__imul__(2.0 ** -6), x["S"][..., :40].__imul__(2.0 ** -6)))
    run_chunk(c)
    import torch
    torch.cuda.synchronize()
    h = c.host
    _, S, _ = delta_ref(c.cu, c.slot, h["q"], h["k"], h["v"], h["a"], h["beta"], h["S"])
    top = np.sqrt((S * S).sum(2)).max((0, 1))  # per column
    off = np.abs(c.dev["S"].double().cpu().numpy() - S).max((0, 1, 2))
    assert np.all(off <= state_tol(90) * np.maximum(top, np.sqrt((h["S"] ** 2).sum(2)).max((0, 1))))


@pytest.mark.parametrize("dtype", DTYPES)
def test_two_calls_continue_one_another(dtype):
    """A prompt in two pieces leaves what the whole leaves."""
    import rank_state_read_b200 as rs
    c = Case([170], 1, 2, 1, 128, dtype, seed=7)
    q, k, v, a, beta, S, y = c.args()
    for lo, hi in ((0, 83), (83, 170)):
        cu = c.cu_d.new_tensor([0, hi - lo])
        rs.sketchssm_delta_chunk(c.plan, cu, q[lo:hi], k[lo:hi], v[lo:hi], a[lo:hi], beta[lo:hi], S, y[lo:hi])
    c.check()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,H,Hqk,V", [(1, 4, 2, 128), (7, 2, 2, 80), (3, 6, 2, 256), (5, 1, 1, 16)])
def test_step(dtype, rows, H, Hqk, V):
    import rank_state_read_b200 as rs
    slot = [(5 * i + 2) % (rows + 4) if rows + 4 != 5 else i for i in range(rows)]
    assert len(set(slot)) == rows
    if rows > 2:
        slot[1] = -1
    c = Case([1] * rows, rows + 4, H, Hqk, V, dtype, slot=slot, seed=8, unit=False)
    rs.sketchssm_delta_step(c.plan, *c.args(), slot=c.slot_d, normalize_qk=True, scale=0.5)
    c.plan.check()
    c.check(normalize=True, scale=0.5)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("chunk", [True, False])
def test_strided_tensors(dtype, chunk):
    """q, k and v as slices of one projection's output, y into a wider buffer."""
    import torch
    import rank_state_read_b200 as rs
    c = Case([66, 5] if chunk else [1, 1, 1], 3, 4, 2, 80, dtype, seed=9)
    q, k, v, a, beta, S, y = c.args()
    n = q.shape[0]
    fused = torch.cat([q.reshape(n, -1), k.reshape(n, -1), v.reshape(n, -1), torch.full((n, 8), float("nan"), device="cuda", dtype=q.dtype)], 1)
    Q = 2 * K
    q2, k2, v2 = fused[:, :Q].view(n, 2, K), fused[:, Q:2 * Q].view(n, 2, K), fused[:, 2 * Q:2 * Q + 320].view(n, 4, 80)
    wide = torch.full((n, 320 + 16), 3.0, device="cuda", dtype=q.dtype)
    y2 = wide[:, 8:328].view(n, 4, 80) if dtype != "float32" else wide[:, 4:324].view(n, 4, 80)
    if chunk:
        rs.sketchssm_delta_chunk(c.plan, c.cu_d, q2, k2, v2, a, beta, S, y2)
    else:
        rs.sketchssm_delta_step(c.plan, q2, k2, v2, a, beta, S, y2)
    y.copy_(y2)
    c.check()
    lo = 8 if dtype != "float32" else 4
    assert bool((wide[:, :lo] == 3).all()) and bool((wide[:, lo + 320:] == 3).all())


@pytest.mark.parametrize("dtype", DTYPES)
def test_tokens_of_others_do_not_matter(dtype):
    """NaN and infinities in the tokens behind a sequence, in another sequence and in other states
    stay where they are."""
    import torch
    lens = [65, 40, 30]
    c = Case(lens, 4, 2, 2, 128, dtype, seed=10, behind=5)
    for m in "qkv":
        c.dev[m][65:105] = float("nan")
        c.dev[m][135:] = float("inf")
    c.dev["a"][65:105] = float("nan")
    c.dev["beta"][135:] = float("nan")
    c.dev["S"][3] = float("nan")
    before = c.dev["S"][3].clone()
    run_chunk(c)
    torch.cuda.synchronize()
    h = c.host
    y, S, _ = delta_ref(c.cu, c.slot, h["q"], h["k"], h["v"], h["a"], h["beta"], h["S"])
    got = c.dev["S"].double().cpu().numpy()
    top = np.sqrt((S * S).sum(2)).max()
    assert np.abs(got[[0, 2]] - S[[0, 2]]).max() <= state_tol(65) * top
    gy = c.dev["y"].double().cpu().numpy()
    for lo, hi in ((0, 65), (105, 135)):
        off = np.abs(gy[lo:hi] - y[lo:hi]) - c.eps * np.abs(y[lo:hi])
        assert off.max() <= 2 * state_tol(65) * top
    assert np.isnan(got[1]).all() and bool((c.dev["y"][135:] == 7).all())
    assert torch.equal(torch.isnan(c.dev["S"][3]), torch.isnan(before))


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("what", ["slot_high", "slot_twice", "cu_back", "cu_past"])
def test_bad_rows_are_left_alone_and_reported(dtype, what):
    import torch
    import rank_state_read_b200 as rs
    c = Case([20, 70, 10], 3, 2, 2, 128, dtype, seed=11)
    cu, slot = list(c.cu), list(c.slot)
    if what == "slot_high":
        slot[1] = 3
    if what == "slot_twice":
        slot[1] = 0
    if what == "cu_back":
        cu[1], cu[2] = 20, 15   # sequence 1 runs backwards, sequence 2 is 15 .. 100
    if what == "cu_past":
        cu[3] = 101
    bad = 2 if what == "cu_past" else 1
    c.cu_d.copy_(torch.tensor(cu))
    c.slot_d.copy_(torch.tensor(slot))
    S0 = c.dev["S"].clone()
    run_chunk(c)
    with pytest.raises(rs.SketchSSMError) as e:
        c.plan.check()
    assert e.value.status == 1
    c.plan.check()  # reported once
    assert torch.equal(c.dev["S"][bad], S0[bad])
    if what in ("slot_high", "slot_twice"):
        assert bool((c.dev["y"][20:90] == 7).all())
    if what == "cu_past":
        assert bool((c.dev["y"][90:] == 7).all())
    assert not torch.equal(c.dev["S"][0], S0[0])
    # and what the good sequence 0 gives is what it gives alone
    alone = Case([20, 70, 10], 3, 2, 2, 128, dtype, seed=11)
    run_chunk(alone)
    torch.cuda.synchronize()
    assert torch.equal(alone.dev["S"][0], c.dev["S"][0])


def test_step_with_the_same_slot_twice():
    import torch
    import rank_state_read_b200 as rs
    c = Case([1] * 4, 4, 2, 2, 128, "bfloat16", slot=[2, 1, 2, 0], seed=12)
    rs.sketchssm_delta_step(c.plan, *c.args(), slot=c.slot_d)
    with pytest.raises(rs.SketchSSMError):
        c.plan.check()
    torch.cuda.synchronize()
    assert bool((c.dev["y"][2] == 7).all())
    c.slot[2] = -1  # the first row that names it has it
    c.check()


@pytest.mark.parametrize("dtype", DTYPES)
def test_captured_calls_and_another_stream(dtype):
    import torch
    import rank_state_read_b200 as rs
    c = Case([65, 3, 130], 3, 2, 2, 128, dtype, seed=13)
    S0 = c.dev["S"].clone()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(st):
        run_chunk(c)
    rs.sketchssm_delta_chunk(c.plan, c.cu_d, *c.args(), slot=c.slot_d, stream=st)  # the stream by argument
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        run_chunk(c)
    c.dev["S"].copy_(S0)
    c.dev["y"].fill_(7)
    g.replay()
    c.check()
    c.dev["S"].copy_(S0)
    for m in "qkv":  # other values in the same place: nothing is kept from the capture
        c.dev[m].mul_(0.5)
        c.host[m] = c.host[m] * 0.5
    g.replay()
    c.check()


@pytest.mark.parametrize("rows", [5, 160])
def test_captured_steps(rows):
    import torch
    import rank_state_read_b200 as rs
    c = Case([1] * rows, rows, 4, 2, 128, "bfloat16", slot=list(range(rows))[::-1], seed=26)
    S0 = c.dev["S"].clone()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        rs.sketchssm_delta_step(c.plan, *c.args(), slot=c.slot_d)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        rs.sketchssm_delta_step(c.plan, *c.args(), slot=c.slot_d)
    c.dev["S"].copy_(S0)
    c.slot_d[0] = -1  # a row that has left the batch since
    c.slot[0] = -1
    c.dev["y"].fill_(7)
    g.replay()
    c.check()
    c.plan.check()


def test_the_same_call_gives_the_same_bits():
    import torch
    out = []
    for _ in range(2):
        c = Case([300, 64, 77], 3, 4, 2, 128, "bfloat16", seed=14)
        run_chunk(c)
        torch.cuda.synchronize()
        out.append((c.dev["y"], c.dev["S"]))
    assert torch.equal(out[0][0], out[1][0]) and torch.equal(out[0][1], out[1][1])


def test_no_write_outside_the_tensors():
    import torch
    c = Case([65, 1, 64], 3, 3, 1, 80, "bfloat16", seed=15)
    for name in ("S", "y"):
        t = c.dev[name]
        big = torch.full((t.numel() + 128,), 5.0, dtype=t.dtype, device="cuda")
        big[64:-64] = t.reshape(-1)
        c.dev[name] = big[64:-64].view(t.shape)
        setattr(c, name + "_big", big)
    run_chunk(c)
    c.check()
    for big in (c.S_big, c.y_big):
        assert bool((big[:64] == 5).all()) and bool((big[-64:] == 5).all())


def test_refusals():
    import torch
    import rank_state_read_b200 as rs
    c = Case([4, 4], 2, 4, 2, 80, "bfloat16", seed=16)
    q, k, v, a, beta, S, y = c.args()
    before = (S.clone(), y.clone())
    call = lambda plan=c.plan, cu=c.cu_d, args=None, **kw: rs.sketchssm_delta_chunk(plan, cu, *(args or c.args()), **kw)

    def refused(status, **kw):
        with pytest.raises(rs.SketchSSMError) as e:
            call(**kw)
        assert e.value.status == status

    refused(3, plan=make_plan(2, 4, 2, 80, "kda"))
    refused(3, plan=make_plan(2, 4, 2, 80, "mamba2"))
    cu3 = torch.tensor([0, 2, 4, 8], dtype=torch.int32, device="cuda")
    refused(1, cu=cu3)  # three sequences, two states, no slots
    wide = torch.zeros(8, 4 * 80 + 4, device="cuda", dtype=torch.bfloat16)
    refused(2, args=[q, k, wide[:, :320].view(8, 4, 80), a, beta, S, y])   # rows 8 bytes off
    flat = torch.zeros(8 * 320 + 8, device="cuda", dtype=torch.bfloat16)
    refused(2, args=[q, k, flat[4:-4].view(8, 4, 80), a, beta, S, y])      # starts 8 bytes off
    for bad, err in (([q.float(), k, v, a, beta, S, y], TypeError), ([q, k, v, a.double(), beta, S, y], TypeError),
                     ([q, k, v[:, :3], a, beta, S, y], ValueError), ([q, k, v, a[:7], beta, S, y], ValueError),
                     ([q.cpu(), k, v, a, beta, S, y], ValueError), ([q, k, v.transpose(1, 2), a, beta, S, y], ValueError),
                     ([q, k, v, a, beta, S.bfloat16(), y], TypeError), ([q, k, v, a, beta, S, y[:1].expand(8, 4, 80)], ValueError),
                     ([q.double(), k.double(), v.double(), a, beta, S, y.double()], TypeError)):
        with pytest.raises(err):
            call(args=bad)
    with pytest.raises(TypeError):
        call(cu=c.cu_d.long())
    with pytest.raises(ValueError):
        call(slot=c.slot_d[:1])
    torch.cuda.synchronize()
    assert torch.equal(S, before[0]) and torch.equal(y, before[1])


def test_nothing_to_do():
    import torch
    import rank_state_read_b200 as rs
    c = Case([2], 1, 2, 2, 80, "bfloat16", seed=17)
    q, k, v, a, beta, S, y = (t[:0] if m != "S" else t for m, t in zip(("q", "k", "v", "a", "beta", "S", "y"), c.args()))
    S0 = S.clone()
    rs.sketchssm_delta_chunk(c.plan, c.cu_d[:1], *c.args())
    rs.sketchssm_delta_chunk(c.plan, torch.zeros(2, dtype=torch.int32, device="cuda"), q, k, v, a, beta, S, y)
    rs.sketchssm_delta_step(c.plan, q, k, v, a, beta, S, y)
    torch.cuda.synchronize()
    c.plan.check()
    assert torch.equal(S, S0)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("H,Hqk,V", [(4, 2, 128), (6, 2, 80), (4, 4, 256), (5, 1, 144), (4, 1, 16)])
def test_step_of_many_rows(dtype, H, Hqk, V):
    """Enough states that the step streams them (several a CTA): permuted slots, padding and a bad
    slot among them, rows whose states one CTA starts and another ends."""
    import torch
    import rank_state_read_b200 as rs
    rows = 151
    slot = np.random.default_rng(20).permutation(rows + 2)[:rows].tolist()
    slot[7] = slot[8] = slot[150] = -1
    c = Case([1] * rows, rows + 2, H, Hqk, V, dtype, slot=slot, seed=20, unit=False)
    c.slot_d[100] = rows + 2
    rs.sketchssm_delta_step(c.plan, *c.args(), slot=c.slot_d, normalize_qk=True, scale=0.5)
    with pytest.raises(rs.SketchSSMError):
        c.plan.check()
    c.slot[100] = -1
    c.check(normalize=True, scale=0.5)
    again = c.dev["S"].clone(), c.dev["y"].clone()
    c2 = Case([1] * rows, rows + 2, H, Hqk, V, dtype, slot=slot, seed=20, unit=False)
    c2.slot_d[100] = -1
    rs.sketchssm_delta_step(c2.plan, *c2.args(), slot=c2.slot_d, normalize_qk=True, scale=0.5)
    torch.cuda.synchronize()
    c2.plan.check()
    assert torch.equal(again[0], c2.dev["S"]) and torch.equal(again[1], c2.dev["y"])


def test_step_equals_the_framework_s_own_step():
    """fp32, packed, row i on state i: sketchssm_step computes the same."""
    import torch
    import rank_state_read_b200 as rs
    for rows in (3, 160):
        a, b = (Case([1] * rows, rows, 4, 2, 80, "float32", seed=21) for _ in range(2))
        q, k, v, g, beta, S, y = a.args()
        rs.sketchssm_delta_step(a.plan, q, k, v, g, beta, S, y)
        rs.sketchssm_step(b.plan, *b.args())
        torch.cuda.synchronize()
        scale = float(b.dev["S"].abs().max())
        assert float((a.dev["S"] - b.dev["S"]).abs().max()) <= 2 * state_tol(1) * scale * 12
        assert float((a.dev["y"] - b.dev["y"]).abs().max()) <= 2 * state_tol(1) * scale * 12


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
def test_many_sequences_of_mixed_lengths(dtype):
    """More sequences than SMs, from nothing to many chunks, heads and slices dealt out over the CTAs
    in several rounds; padding and a slot named twice among them."""
    import torch
    import rank_state_read_b200 as rs
    g = np.random.default_rng(22)
    lens = [int(x) for x in g.integers(0, 90, 60)] + [0, 300, 1, 64]
    slot = g.permutation(len(lens)).tolist()
    slot[5] = -1
    c = Case(lens, len(lens), 5, 5, 144, dtype, slot=slot, seed=22)
    twin = 40
    assert lens[10] > 0 and lens[twin] > 0
    c.slot_d[twin] = slot[10]
    run_chunk(c)
    with pytest.raises(rs.SketchSSMError):
        c.plan.check()
    c.slot[twin] = -1
    c.check()


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("chunk", [True, False])
def test_short_wait_limit_is_reported_and_outputs_complete(dtype, chunk):
    """With the plan's wait limit at one cycle the CTAs' waits run past it: recorded, and continued for
    the same copies and products, so that the results are those of any other run."""
    import torch
    import rank_state_read_b200 as rs
    rows = 3 if chunk else 160
    lens = [130, 70, 64] if chunk else [1] * rows
    a, b = (Case(lens, rows, 4, 2, 128, dtype, seed=23) for _ in range(2))
    b.plan.set_wait_limit(1)
    for c in (a, b):
        if chunk:
            run_chunk(c)
        else:
            rs.sketchssm_delta_step(c.plan, *c.args())
    torch.cuda.synchronize()
    assert torch.equal(a.dev["S"], b.dev["S"]) and torch.equal(a.dev["y"], b.dev["y"])
    a.plan.check()
    if chunk and dtype == "float32":
        b.plan.check()  # token by token: nothing to wait for
    else:
        # the chain of a chunk certainly waits for its products; a step's copies may have landed
        # before it looks for them, and then there is nothing to record
        try:
            b.plan.check()
            assert not chunk
        except rs.SketchSSMError as e:
            assert e.status == 5
    b.plan.set_wait_limit(2_000_000_000)
    b.check()


def test_two_streams_share_a_plan():
    """Calls on one plan whose rows have different states may overlap: they share nothing but the
    status word."""
    import torch
    import rank_state_read_b200 as rs
    a = Case([130, 200], 4, 4, 2, 128, "bfloat16", slot=[0, 1], seed=24)
    b = Case([90, 260], 4, 4, 2, 128, "bfloat16", slot=[2, 3], seed=24)
    both = a.dev["S"]
    b.dev["S"].copy_(both)
    b.host["S"] = a.host["S"]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(3):
        both.copy_(b.dev["S"])
        torch.cuda.synchronize()
        for c, st in zip((a, b), streams):
            q, k, v, g, beta, _, y = c.args()
            rs.sketchssm_delta_chunk(a.plan, c.cu_d, q, k, v, g, beta, both, y, slot=c.slot_d, stream=st)
        torch.cuda.synchronize()
    a.plan.check()
    for c in (a, b):
        h = c.host
        y, S, _ = delta_ref(c.cu, c.slot, h["q"], h["k"], h["v"], h["a"], h["beta"], h["S"])
        top = np.sqrt((S * S).sum(2)).max()
        got = both.double().cpu().numpy()[c.slot]
        assert np.abs(got - S[c.slot]).max() <= state_tol(c.longest) * top
        off = np.abs(c.dev["y"].double().cpu().numpy() - y) - c.eps * np.abs(y)
        assert off.max() <= 2 * state_tol(c.longest) * top


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
def test_strong_decays_next_to_weak_ones(dtype):
    """Chunks whose decays span more than fp32's exponents beside chunks without decay: the products of
    both are those of the definition, and nothing overflows on the way."""
    def change(x):
        g = np.random.default_rng(25)
        x["a"][:64] = g.choice([1.0, 1e-8, 0.5], (64, x["a"].shape[1]))
        x["a"][64:128] = 1.0
        x["a"][128:192] = g.choice([1.0, 0.0], (64, x["a"].shape[1]), p=[0.9, 0.1])
    c = Case([192 + 30], 1, 3, 1, 128, dtype, seed=25, change=change)
    run_chunk(c)
    c.check(grow=223 / 64)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("slots", ["none", "turned"])
def test_more_sequences_than_one_launch_takes(dtype, slots):
    """Over a thousand sequences: in their own order without slots, and with slots turned round,
    padding and one that a sequence of another launch has named."""
    import rank_state_read_b200 as rs
    g = np.random.default_rng(23)
    lens = [int(x) for x in g.integers(0, 28, 1090)]
    lens[3] = lens[514] = lens[1089] = 70
    n = len(lens)
    assert sum(lens) > 10 * n
    slot = list(range(n)) if slots == "none" else list(range(n - 1, -1, -1))
    if slots == "turned":
        slot[20] = slot[700] = -1
    c = Case(lens, n, 2, 1, 16, dtype, slot=slot, seed=23)
    if slots == "none":
        rs.sketchssm_delta_chunk(c.plan, c.cu_d, *c.args())
        c.plan.check()
    else:
        c.slot_d[1089] = slot[3]
        c.slot_d[1030] = slot[514]
        assert lens[1030] > 0
        run_chunk(c)
        with pytest.raises(rs.SketchSSMError):
            c.plan.check()
        c.slot[1089] = c.slot[1030] = -1
    c.check()


@pytest.mark.parametrize("dtype", DTYPES)
def test_padding_needs_no_bounds(dtype):
    """A padded batch: the bounds behind the last sequence are whatever is there, the slots -1."""
    import torch
    c = Case([70, 40, 1, 1], 4, 2, 2, 128, dtype, slot=[2, 0, -1, -1], seed=24)
    c.cu_d[3:] = torch.tensor([0, 1 << 30], dtype=torch.int32)
    run_chunk(c)
    c.plan.check()
    c.check()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_what_is_not_finite_stays_in_its_sequence(dtype, bad):
    """Many sequences in each CTA, some with values that are not finite: the others give the bits
    that they give without them."""
    import torch
    g = np.random.default_rng(25)
    lens = [int(x) for x in g.integers(30, 150, 90)]
    sick = list(range(1, 90, 4))
    got = []
    for spoil in (False, True):
        c = Case(lens, 90, 5, 5, 144, dtype, seed=25)
        if spoil:
            for i in sick:
                m = ("q", "k", "v", "a", "beta")[i // 4 % 5]
                c.dev[m][c.cu[i] + lens[i] // 2] = bad
            c.dev["S"][sick[0]] = bad
        run_chunk(c)
        c.plan.check()
        got.append((c.dev["y"], c.dev["S"], c))
    c = got[0][2]
    well = [i for i in range(90) if i not in sick]
    rows = torch.cat([torch.arange(c.cu[i], c.cu[i + 1]) for i in well]).cuda()
    assert torch.equal(got[0][0][rows], got[1][0][rows])
    assert torch.equal(got[0][1][well], got[1][1][well])
    # and the outputs of whole chunks of 64 before the value are finite
    for i in sick[1:]:
        first = c.cu[i] + lens[i] // 2 // 64 * 64
        assert bool(torch.isfinite(got[1][0][c.cu[i]:first].float()).all())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n", [41, 63, 64, 65])
def test_sequences_taken_longest_first(dtype, n):
    """Short sequences, many of them of one length or empty, on more CTAs than there are SMs; a slot out
    of range, one named twice, bounds out of order, and padding with any bounds among them."""
    import torch
    import rank_state_read_b200 as rs
    g = np.random.default_rng(26)
    lens = [int(x) for x in g.integers(0, 8, n)]
    lens[2], lens[30], lens[7], lens[33], lens[n - 2], lens[n - 1] = 40, 40, 3, 3, 0, 0
    slot = g.permutation(n).tolist()
    slot[n - 2] = slot[n - 1] = -1
    assert sum(lens) <= 10 * n
    c = Case(lens, n, 5, 5, 144, dtype, slot=slot, seed=26, behind=2)
    c.slot_d[7] = n
    c.slot_d[33] = slot[2]
    c.cu_d[n - 1:] = torch.tensor([-(1 << 31), (1 << 31) - 1], dtype=torch.int32)
    c.cu_d[n - 2] = c.cu[n - 2] + 2**20
    bad_last = c.slot[n - 3]  # its end lies far behind the tokens
    run_chunk(c)
    with pytest.raises(rs.SketchSSMError):
        c.plan.check()
    c.slot[7] = c.slot[33] = c.slot[n - 3] = -1
    assert bad_last >= 0
    c.check()


def test_one_short_sequence_either_way():
    """A single sequence of up to 20 tokens and one of 21 go different ways: the first 20 tokens of both
    have the same outputs, within twice what each may be off."""
    import rank_state_read_b200 as rs
    a = Case([20], 1, 4, 2, 128, "float16", seed=27, behind=1)
    b = Case([21], 1, 4, 2, 128, "float16", seed=27)
    for c in (a, b):
        rs.sketchssm_delta_chunk(c.plan, c.cu_d, *c.args())
        c.check()
    top = float(b.dev["S"].norm(dim=2).max())
    off = (a.dev["y"][:20].double() - b.dev["y"][:20].double()).abs() - 2 * b.eps * a.dev["y"][:20].double().abs()
    assert float(off.max()) <= 4 * state_tol(21) * max(top, 3.0)


def test_threads_with_states_of_different_size():
    """Layers whose states differ in width, stepped from several threads through the C entry: no call
    changes what another's launch needs."""
    import ctypes
    import threading

    import torch
    import rank_state_read_b200 as rs
    lib, td = rs.load(), rs.TokenDesc(1, 0, 1.0, 0, 0, 0, 0)
    cases = [Case([1] * 40, 40, 4, 2, V, "bfloat16", seed=28) for V in (128, 64) * 4]
    streams = [torch.cuda.Stream() for _ in cases]
    bad = []
    start = threading.Barrier(len(cases))
    torch.cuda.synchronize()

    def work(c, st):
        args = [c.plan.handle, ctypes.byref(td), 40, None, *(t.data_ptr() for t in c.args()), st.cuda_stream]
        start.wait()
        for _ in range(5000):
            status = lib.sketchssm_delta_step(*args)
            if status:
                bad.append((status, lib.sketchssm_last_error()))
                return
    threads = [threading.Thread(target=work, args=a) for a in zip(cases, streams)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not bad, bad


@pytest.mark.parametrize("chunk", [True, False])
def test_outputs_that_share_memory_are_refused(chunk):
    import torch
    import rank_state_read_b200 as rs
    n, H = 6, 2
    c = Case([4, 2] if chunk else [1] * n, 2 if chunk else n, H, H, K, "bfloat16", seed=29)
    q, k, v, a, beta, S, y = c.args()
    before = [t.clone() for t in c.args()]

    def call(**kw):
        args = [kw.get(m, t) for m, t in zip(("q", "k", "v", "a", "beta", "S", "y"), c.args())]
        slot = kw.get("slot", c.slot_d)
        if chunk:
            rs.sketchssm_delta_chunk(c.plan, kw.get("cu", c.cu_d), *args, slot=slot)
        else:
            rs.sketchssm_delta_step(c.plan, *args, slot=slot)

    buf = torch.zeros(4 * n * H * K, device="cuda", dtype=torch.bfloat16)
    off = buf[K:K + n * H * K].view(n, H, K)             # the same rows, half a row on
    wide = torch.zeros(n, 4 * H * K, device="cuda", dtype=torch.bfloat16)
    part = lambda lo: wide[:, lo:lo + H * K].view(n, H, K)
    flat = S.view(-1)
    bad = [dict(y=q), dict(y=k), dict(y=v), dict(y=off, v=buf[:n * H * K].view(n, H, K)),
           dict(y=part(K), q=part(2 * K)),                # columns that meet
           dict(y=part(0), k=wide.view(-1)[3 * K:3 * K + n * H * K].view(n, H, K)),  # another stride
           dict(y=flat[:n * H * K // 2].view(torch.bfloat16).view(n, H, K)),
           dict(a=flat[:n * H].view(n, H)), dict(beta=flat[8:8 + n * H].view(n, H)),
           dict(a=buf[:2 * n * H].view(torch.float32).view(n, H), y=buf[:n * H * K].view(n, H, K)),
           dict(slot=flat[:c.slot_d.numel()].view(torch.int32))]
    if chunk:
        bad.append(dict(cu=flat[16:16 + c.cu_d.numel()].view(torch.int32)))
    for kw in bad:
        with pytest.raises(rs.SketchSSMError, match="overlaps") as e:
            call(**kw)
        assert e.value.status == 1, kw.keys()
    torch.cuda.synchronize()
    assert all(torch.equal(t, u) for t, u in zip(c.args(), before))
    # rows of one buffer between one another: q | y | k | v
    for lo, t in ((0, q), (2 * H * K, k), (3 * H * K, v)):
        part(lo).copy_(t)
    call(q=part(0), k=part(2 * H * K), v=part(3 * H * K), y=part(H * K))
    y.copy_(part(H * K))
    c.check()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V", [48, 64])
def test_step_of_many_rows_of_narrow_states(dtype, V):
    """The widest states that many rows take one by one, and the narrowest that are streamed."""
    import rank_state_read_b200 as rs
    rows = 90
    slot = np.random.default_rng(32).permutation(rows + 3)[:rows].tolist()
    slot[3] = slot[89] = -1
    c = Case([1] * rows, rows + 3, 6, 2, V, dtype, slot=slot, seed=32, unit=False)
    c.slot_d[50] = slot[7]
    rs.sketchssm_delta_step(c.plan, *c.args(), slot=c.slot_d, normalize_qk=True, scale=0.5)
    with pytest.raises(rs.SketchSSMError):
        c.plan.check()
    c.slot[50] = -1
    c.check(normalize=True, scale=0.5)
