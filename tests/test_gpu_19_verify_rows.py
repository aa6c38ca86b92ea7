"""Draft verification where a row is shared by a whole cluster of CTAs: residuals that are
empty, tokens in each CTA's and each warp's part, two-byte probabilities.  Against the
64-bit reference; every output is a whole number and has to be equal."""
import numpy as np
import pytest
import torch

import masked_attention_paged_gb300 as lib
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


@pytest.mark.parametrize("mode", ["replacement", "distinct", "certain"])
@pytest.mark.parametrize("B,T,V,wide", [(1, 6, WIDE, 3), (3, 9, 40001, 4), (30, 4, 2 * 16384, 2), (70, 5, 4097, 3)])
def test_two_byte_probabilities_over_a_cluster(B, T, V, wide, mode):
    p, q, tok, par, u = _inputs(B, T, V, seed=B + V, wide=wide, mode=mode, dtype=torch.bfloat16)
    q = None if mode == "certain" else q
    got, status = _run(p, q, tok, par, u, mode == "replacement", dtype=torch.bfloat16)
    _equal(got, verify(p, q, tok, par, u, mode == "replacement"))
    assert status == 0


@pytest.mark.parametrize("B", [1, 9, 38])
def test_calls_right_behind_one_another(B):
    """Clusters of 16 that are placed while those of the call ahead still run, over trees with and without idle
    sequences between them."""
    p, q, tok, par, u = _inputs(B, 5, WIDE, seed=B, wide=3)
    idle = par.copy()
    idle[::2, 0] = -2
    to = lambda x: torch.from_numpy(x).cuda()  # noqa: E731
    P, Q, K, U, trees, ws = to(p), to(q), to(tok), to(u), [to(par), to(idle)], lib.Workspace(256)
    got = [lib.draft_verify(P, K, trees[i % 2], U, draft_probs=Q, workspace=ws) for i in range(60)]
    want = [verify(p, q, tok, x, u, False) for x in (par, idle)]
    for i, x in enumerate(got):
        _equal([y.cpu().numpy() for y in x], want[i % 2])
    assert ws.status() == 0
