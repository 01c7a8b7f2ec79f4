"""How exact the chunked delta rule is: bounds near what its arithmetic gives, so that an operand's low
part that is lost, or decays that are a little off, show."""
from __future__ import annotations

import numpy as np
import pytest

from delta_ref import delta_ref
from test_gpu_delta import Case, run_chunk

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from rank_state_read_b200 import build
    build.build()


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
def test_decays_far_from_a_chunk_s_middle(dtype):
    """The last token of a chunk (beta = 1) takes back what the one before it wrote to the same key: the
    state there is 0, and what is left of it is the error of the decay between the two, which lie 60 to
    95 powers of two from the chunk's middle.

    Relative to a u, what the second token finds: its A is a product of 2^(G_63 - G_31) and 2^(G_31 - G_62)
    (ex2: 2^-22 each) with three roundings of 2^-24; T and R are pairs (2^-23 each, half a step of 2^-22);
    the sum T R is off by 2^-23: 8.5 * 2^-23.  The state's factor of the first token is off by 2^-22, its
    pairs of both by 2^-23 each, and sums and factors of both by 2 * 2^-23 each: 8 * 2^-23.
    """
    import torch
    H, V, n = 32, 16, 64

    def change(x):
        g = np.random.default_rng(30)
        x["k"][:] = 0
        x["k"][np.arange(n), :, np.arange(n) // 2] = 1
        x["q"][:] = x["k"]
        x["v"][:] = np.round(x["v"] * 64) / 64
        x["v"][1::2] = 0
        x["a"][:] = np.linspace(0.13, 0.26, H) * (1 + 0.02 * g.standard_normal((n, H)))
        x["beta"][:] = 1
        x["S"][:] = 0
    c = Case([n], 1, H, 1, V, dtype, seed=30, change=change)
    run_chunk(c)
    c.plan.check()
    torch.cuda.synchronize()
    left = np.abs(c.dev["S"][0, :, 31].double().cpu().numpy()).max(1)
    found = (c.host["a"][63][:, None] * np.abs(c.host["v"][62])).max(1)
    assert np.all(left <= 16.5 * 2.0 ** -23 * found), (left / found).max()


# A chunk's roundings, as they reach the state: sums in fp32 of 16 (K S), 12 (T R) and 8 (the increment)
# accumulations, which the tensor cores cut off, 2^-24 in the mean of each partial sum; the products
# A holds two factors of 2^-22 of a decay, the state's increment one: 12 * 2^-24.  The pairs' 2^-22 and the
# other roundings are spread to both sides, and disappear beside these in a 2-norm over 128 x V values.
# A low part that is left out costs 2^-12 a value: 3e-6 (S, a chunk of 64 tokens) to 2e-4 (R) of the state.
STATE = 48 * 2.0 ** -24


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("lens", [[21], [64], [65], [200], [130, 64, 33]], ids=str)
@pytest.mark.parametrize("decays", ["weak", "half", "strong"])
def test_state_and_outputs_to_their_last_bits(dtype, lens, decays):
    """The state in the 2-norm of each sequence and head; the outputs against the exact ones rounded to
    their type.  Two roundings of values that are apart by d of a step differ in d of the cases, by a step
    each: the sum of squares is then d * step^2, at most STATE * eps * |y|^2, since a step is at most
    eps |y|.  One step of the largest value is allowed beside it, where few values make up the mean."""
    import torch
    H, V = 8, 128

    def change(x):
        g = np.random.default_rng(31)
        if decays == "half":
            x["a"][:] = g.uniform(0.4, 0.6, x["a"].shape)
        if decays == "strong":  # more than 100 powers of two in a chunk
            x["a"][:] = np.exp2(-g.exponential(5.0, x["a"].shape))
    c = Case(lens, len(lens), H, 4, V, dtype, seed=31, change=change)
    run_chunk(c)
    c.plan.check()
    torch.cuda.synchronize()
    h = c.host
    y, S, _ = delta_ref(c.cu, c.slot, h["q"], h["k"], h["v"], h["a"], h["beta"], h["S"])
    got = c.dev["S"].double().cpu().numpy()
    size = lambda t: np.sqrt((t * t).sum((2, 3)))
    off = size(got - S) / size(S)
    assert off.max() <= STATE, off.max()
    eps = torch.finfo(c.dev["y"].dtype).eps
    gy = c.dev["y"].double().cpu().numpy()
    ry = torch.from_numpy(y).to(c.dev["y"].dtype).double().numpy()
    limit = np.sqrt(STATE * eps) * np.linalg.norm(y) + eps * np.abs(y).max()
    assert np.linalg.norm(gy - ry) <= limit, (np.linalg.norm(gy - ry) / np.linalg.norm(y), limit / np.linalg.norm(y))
