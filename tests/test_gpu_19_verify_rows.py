"""Draft verification where a row is shared by a whole cluster of CTAs: residuals that are
empty, tokens in each CTA's and each warp's part, two-byte probabilities.  Against the
64-bit reference; every output is a whole number and has to be equal."""
import numpy as np
import pytest
import torch

from _serve_ref import verify
from test_gpu_15_verify import _equal, _inputs, _run

pytestmark = pytest.mark.gpu

WIDE = 2048 * 16 + 5  # tokens of a row that 16 CTAs share, where there are few sequences


@pytest.mark.parametrize("V", [50, 2048, 4100, WIDE, 131075])
@pytest.mark.parametrize("mode", ["replacement", "distinct", "certain"])
def test_a_residual_that_is_empty(V, mode):
    """Two refusals take all of p away: the token comes from p itself, wherever it lies."""
    a, b = V // 2 + 1, V - 2
    p = np.zeros((1, 3, V), np.float32)
    p[0, :, [0, a, b]] = 0.25
    tok, par = np.array([[0, a, b]], np.int32), np.array([[-1, 0, 0]], np.int32)
    q = None if mode == "certain" else np.full((1, 3, V), 0.5, np.float32)
    if q is None:
        p[0, :, 0] = 0.0
    for x in (0.0, 0.3, 0.45, 0.9):
        u = np.array([[x, 0.6, 0.6]], np.float32)
        got, status = _run(p, q, tok, par, u, mode == "replacement")
        _equal(got, verify(p, q, tok, par, u, mode == "replacement"))
        assert got[1][0] == 1 and got[2][0] in (0, a, b) and status == 0


@pytest.mark.parametrize("B,V", [(1, WIDE), (38, WIDE), (70, 4100), (300, 2300), (640, 700)])
@pytest.mark.parametrize("mode", ["distinct", "certain"])
def test_a_token_after_a_refusal_in_every_part(B, V, mode):
    """All drafts are refused, and u_0 walks over the row: the first part of the first warp as often as any."""
    rng = np.random.default_rng(B + V)
    p = rng.random((1, 3, V)).astype(np.float32)
    p = np.repeat(p / p.sum(-1, keepdims=True, dtype=np.float64).astype(np.float32), B, 0)
    q = None if mode == "certain" else np.repeat(rng.permutation(p[0, 0])[None, None], B, 0).repeat(3, 1)
    tok = np.tile(np.array([0, V // 3, V // 5], np.int32), (B, 1))
    par = np.tile(np.array([-1, 0, 0], np.int32), (B, 1))
    if q is not None:
        q[:, 0, tok[0, 1:]] = 0.25
    for k in range(1 if B > 1 else 24):
        u = np.full((B, 3), 0.75, np.float32)
        u[:, 0] = (np.arange(B) + 0.5) / B if B > 1 else (k / 24.0) ** 3
        got, status = _run(p, q, tok, par, u)
        _equal(got, verify(p, q, tok, par, u, False))
        assert (got[1] == 1).all() and status == 0
