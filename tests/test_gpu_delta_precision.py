"""How exact the chunked delta rule is: bounds near what its arithmetic gives, so that an operand's low
part that is lost, or decays that are a little off, show."""
from __future__ import annotations

import numpy as np
import pytest

from delta_ref import K
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
