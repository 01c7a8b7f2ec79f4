"""Host checks of the delta-rule and gated-norm calls that need no GPU: what the C entry points refuse
before they touch a pointer, the descriptors' layout, and the fp64 references against other forms."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest

import rank_state_read_b200 as rs
from delta_ref import delta_ref, draw, norm_ref
from rank_state_read_b200 import build as rbuild


@pytest.fixture(scope="module")
def lib():
    rbuild.build()
    return rs.load()


def test_delta_calls_without_a_plan(lib):
    td = rs.TokenDesc(1, 0, 1.0, 0, 0, 0, 0)
    assert lib.sketchssm_delta_chunk(None, ctypes.byref(td), 1, 4, *([None] * 10)) == 1
    assert lib.sketchssm_delta_step(None, ctypes.byref(td), 1, *([None] * 9)) == 1
    assert b"plan" in lib.sketchssm_last_error()


@pytest.mark.parametrize("over,rows,status", [
    (dict(x_dtype=3), 1, 1), (dict(dtype=-1), 1, 1), (dict(gate=2), 1, 1), (dict(groups=0), 1, 1), (dict(width=0), 1, 1),
    (dict(), -1, 1), (dict(weight_groups=3), 1, 1), (dict(eps=-1e-6), 1, 1), (dict(eps=float("nan")), 1, 1),
    (dict(width=68), 1, 3), (dict(width=16392), 1, 3), (dict(x_stride=120), 2, 1), (dict(z_stride=132), 2, 2),
    (dict(out_stride=1 << 50), 2, 1), (dict(groups=1 << 20), 1 << 12, 3), (dict(), 0, 0), (dict(), 1, 1),
])
def test_gated_norm_refuses_bad_descriptors(lib, over, rows, status):
    d = dict(x_dtype=1, dtype=1, groups=2, width=64, weight_groups=1, gate=0, gate_first=0, eps=1e-6, x_stride=0,
             z_stride=0, out_stride=0)
    d.update(over)
    nd = rs.NormDesc(*[d[f] for f, _ in rs.NormDesc._fields_])
    assert lib.sketchssm_gated_norm(ctypes.byref(nd), rows, None, None, None, None, None) == status
    assert lib.sketchssm_gated_norm(None, rows, None, None, None, None, None) == 1


def test_binding_refuses_host_tensors():
    import torch
    x = torch.zeros(2, 3, 64)
    with pytest.raises(ValueError, match="CUDA"):
        rs.sketchssm_gated_norm(x, x, x[0, 0], x)
    with pytest.raises(TypeError):
        rs.sketchssm_gated_norm(x.numpy(), x, x[0, 0], x)
    with pytest.raises(ValueError, match="activation"):
        rs.sketchssm_gated_norm(x, x, x[0, 0], x, activation="tanh")


def test_delta_reference_against_explicit_matrices():
    """S_t = a (I - beta k k^T) S_{t-1} + beta k v^T with the matrices written out, two heads on one
    q/k head; and the chunk's closed form U = (I + A)^-1 diag(beta) (V - diag(exp G) K S_0)."""
    n, H, V = 9, 2, 16
    x = {m: t.astype(np.float64) for m, t in draw(0, n, 1, H, 1, V).items()}
    y, S, touched = delta_ref([0, n], [0], *(x[m] for m in ("q", "k", "v", "a", "beta", "S")))
    assert touched.all()
    for h in range(H):
        M = x["S"][0, h].copy()
        for t in range(n):
            k, q = x["k"][t, 0], x["q"][t, 0]
            M = x["a"][t, h] * (np.eye(128) - x["beta"][t, h] * np.outer(k, k)) @ M + x["beta"][t, h] * np.outer(k, x["v"][t, h])
            assert np.allclose(y[t, h], M.T @ q, rtol=0, atol=1e-13)
        assert np.allclose(S[0, h], M, rtol=0, atol=1e-13)
        k, q, b, G = x["k"][:, 0], x["q"][:, 0], x["beta"][:, h], np.cumsum(np.log(x["a"][:, h]))
        D = np.exp(G[:, None] - G[None])
        A = np.tril(b[:, None] * D * (k @ k.T), -1)
        U = np.linalg.solve(np.eye(n) + A, b[:, None] * (x["v"][:, h] - np.exp(G)[:, None] * (k @ x["S"][0, h])))
        assert np.allclose(np.exp(G)[:, None] * (q @ x["S"][0, h]) + np.tril(D * (q @ k.T)) @ U, y[:, h], rtol=0, atol=1e-13)
        assert np.allclose(np.exp(G[-1]) * x["S"][0, h] + (np.exp(G[-1] - G)[:, None] * k).T @ U, S[0, h], rtol=0, atol=1e-13)


def test_delta_reference_skips_padding_and_keeps_other_states():
    x = draw(1, 6, 3, 2, 2, 16)
    y, S, touched = delta_ref([0, 2, 4, 4], [1, -1, 0], *(x[m] for m in ("q", "k", "v", "a", "beta", "S")), True, 0.5)
    assert touched.tolist() == [True, True, False, False, False, False] and not y[2:].any()
    assert np.array_equal(S[[0, 2]], x["S"][[0, 2]].astype(np.float64)) and not np.array_equal(S[1], x["S"][1])


def test_norm_reference():
    x, z, w = np.array([[[3.0, 4.0]]]), np.array([[[0.0, 100.0]]]), np.array([2.0, 1.0])
    r = np.sqrt(12.5)
    assert np.allclose(norm_ref(x, z, w, 0.0, "sigmoid", False), [[[3 / r, 4 / r]]])
    assert np.allclose(norm_ref(x, z, w, 0.0, "silu", True), [[[0, np.sqrt(2)]]])
    assert np.allclose(norm_ref(x, None, w, 0.0, "silu", False), [[[6 / r, 4 / r]]])


def test_binding_refuses_counts_past_32_bits():
    import torch
    for n in (2**31, 2**32 + 2):
        x = torch.empty(n, 1, 128, device="meta", dtype=torch.bfloat16)
        few = torch.empty(8, device="meta", dtype=torch.int32)
        with pytest.raises(ValueError, match="more than a call takes"):
            rs.sketchssm_gated_norm(x, x, torch.empty(128, device="meta"), x)
        with pytest.raises(ValueError, match="more than a call takes"):
            rs.sketchssm_delta_step(None, x, x, x, x, x, x, x)
        with pytest.raises(ValueError, match="more than a call takes"):
            rs.sketchssm_delta_chunk(None, few, x, x, x, x, x, x, x)


def test_spans_past_64_bits_are_refused(lib):
    """rows * stride may wrap round 64 bits; what is left then looks like a tensor of one row."""
    text = lambda: lib.sketchssm_last_error().decode()
    fake = ctypes.c_void_p(1 << 40)  # never read: the span is refused before any pointer is looked at
    for stride, rows in ((1 << 36, (1 << 28) + 1), (1 << 36, (1 << 29) + 1), (1 << 36, (1 << 27) + 1), (1 << 35, (1 << 30) + 1),
                         (1 << 36, 0x7FFFFFFF), (1 << 34, 0x7FFFFFFF), (128, 1 << 25)):
        for field in ("x_stride", "z_stride", "out_stride"):
            nd = rs.NormDesc(1, 1, 1, 128, 1, 0, 0, 1e-6, 0, 0, 0)
            setattr(nd, field, stride)
            status = lib.sketchssm_gated_norm(ctypes.byref(nd), rows, fake, fake, fake, fake, None)
            assert status == 1, (stride, rows, field, status)
            large = stride * (rows - 1) > 1 << 46
            assert (f"{field[:-7]} spans" in text()) == large, (stride, rows, text())


def test_gated_norm_refuses_outputs_that_share_memory(lib):
    """Against the bytes written out: out may be x or z, row for row, or lie between their rows."""
    g = np.random.default_rng(3)
    base = 1 << 40

    def taken(at, row, stride, rows):
        return np.concatenate([at + r * stride + np.arange(0, row, 16) for r in range(rows)])

    seen = {True: 0, False: 0}
    for _ in range(4000):
        rows, width = int(g.integers(1, 6)), 8 * int(g.integers(1, 4))
        xt, t = int(g.integers(0, 3)), int(g.integers(0, 3))
        xe, e = (4 if xt == 0 else 2), (4 if t == 0 else 2)
        es = (xe, e, e)
        same = 16 * int(g.integers(width // 4, width // 4 + 8))  # bytes
        strides = [same if g.random() < 0.5 else width * s + 16 * int(g.integers(0, 6)) for s in es]
        at = [base + 16 * int(g.integers(0, 40)) for _ in es]
        if g.random() < 0.3:
            at[2] = at[int(g.integers(0, 2))]
        weight = base + 16 * int(g.integers(0, 60))
        nd = rs.NormDesc(xt, t, 1, width, 1, 0, 0, 1e-6, *(b // s for b, s in zip(strides, es)))
        out = taken(at[2], width * e, strides[2], rows)
        want = np.intersect1d(out, taken(weight, width * 4, 0, 1)).size > 0
        for i in range(2):
            itself = at[i] == at[2] and es[i] == e and (rows == 1 or strides[i] == strides[2])
            want = want or (not itself and np.intersect1d(out, taken(at[i], width * es[i], strides[i], rows)).size > 0)
        p = [ctypes.c_void_p(a) for a in (at[0], at[1], weight, at[2])]
        assert lib.sketchssm_gated_norm(ctypes.byref(nd), rows, *p, None) == 1  # none of them is device memory
        found = "overlaps" in lib.sketchssm_last_error().decode()
        assert found == want, (rows, width, xt, t, strides, at, weight, lib.sketchssm_last_error())
        seen[want] += 1
    assert min(seen.values()) > 500, seen
