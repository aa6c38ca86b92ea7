"""Draft verification on the GPU against the 64-bit reference: every output is a whole
number and has to be equal."""
import numpy as np
import pytest
import torch

import masked_attention_paged_gb300 as lib
from _serve_ref import verify, verify_one

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _softmax(x):
    e = np.exp(x - x.max(-1, keepdims=True))
    return (e / e.sum(-1, keepdims=True)).astype(np.float32)


def _inputs(B, T, V, seed, wide=3, mode="distinct", sharp=3.0, blur=0.7, short=True, dtype=torch.float32):
    """Trees with tokens drawn at each node from the draft's row."""
    rng = np.random.default_rng(seed)
    z = rng.normal(size=(B, T, V)) * sharp
    p, q = _softmax(z), _softmax(z + blur * rng.normal(size=z.shape))
    if dtype == torch.bfloat16:
        p, q = (torch.from_numpy(x).bfloat16().float().numpy() for x in (p, q))
    par = np.full((B, T), -2, np.int32)
    tok = np.zeros((B, T), np.int32)
    for b in range(B):
        n = T if not short or b % 4 != 2 else max(1, T // 2)
        par[b, 0] = -1
        kids = {}
        for t in range(1, n):
            up = int(rng.integers(max(0, t - 1 - wide), t))
            par[b, t] = up
            gone = kids.setdefault(up, [])
            row = q[b, up].astype(np.float64)
            if mode == "distinct" and len(gone) < V:
                row[gone] = 0.0
            tok[b, t] = rng.choice(V, p=row / row.sum()) if row.sum() > 0 else rng.integers(V)
            gone.append(int(tok[b, t]))
    return p, q, tok, par, rng.random((B, T)).astype(np.float32)


def _run(p, q, tok, par, u, replacement=False, dtype=torch.float32, **kw):
    to = lambda x, t: torch.from_numpy(np.ascontiguousarray(x)).to(DEV, t)  # noqa: E731
    ws = lib.Workspace(256)
    got = lib.draft_verify(to(p, dtype), to(tok, torch.int32), to(par, torch.int32), to(u, torch.float32),
                           draft_probs=None if q is None else to(q, dtype), replacement=replacement, workspace=ws, **kw)
    return [x.cpu().numpy() for x in got], ws.status()


def _equal(got, want):
    for name, a, b in zip(("path", "n_accept", "next_token"), got, want):
        assert np.array_equal(a, b), (name, a, b)


@pytest.mark.parametrize("mode", ["distinct", "replacement", "certain"])
@pytest.mark.parametrize("B,T,V,wide", [(1, 1, 1, 0), (1, 1, 50, 0), (3, 2, 7, 0), (2, 8, 1000, 0), (5, 9, 31, 3),
                                        (4, 25, 4099, 3), (2, 64, 517, 5), (1, 256, 40, 7), (1, 6, 70001, 4),
                                        (33, 12, 333, 4)])
def test_against_the_reference(B, T, V, wide, mode):
    p, q, tok, par, u = _inputs(B, T, V, seed=B + T + V, wide=wide, mode=mode)
    q = None if mode == "certain" else q
    got, status = _run(p, q, tok, par, u, mode == "replacement")
    _equal(got, verify(p, q, tok, par, u, mode == "replacement"))
    assert status == 0


@pytest.mark.parametrize("mode", ["distinct", "certain"])
def test_bf16(mode):
    p, q, tok, par, u = _inputs(6, 17, 3001, seed=4, mode=mode, dtype=torch.bfloat16)
    q = None if mode == "certain" else q
    got, _ = _run(p, q, tok, par, u, dtype=torch.bfloat16)
    _equal(got, verify(p, q, tok, par, u, False))


@pytest.mark.parametrize("V", [1, 5, 33, 1024, 1025, 8193, 131072])
def test_the_next_token_at_the_ends(V):
    """u = 0 draws the first possible token, the largest u the last; zeros are never drawn."""
    rng = np.random.default_rng(V)
    p = rng.random((3, 1, V)).astype(np.float32)
    p[rng.random(p.shape) < 0.4] = 0.0
    p[:, :, V // 2] = 0.5
    one = np.zeros((3, 1), np.int32)
    for x in (0.0, 0.25, 1.0 - 2.0 ** -24):
        u = np.full((3, 1), x, np.float32)
        got, _ = _run(p, None, one, one - 1, u)
        want = verify(p, None, one, one - 1, u, False)
        _equal(got, want)
        assert (np.take_along_axis(p[:, 0], got[2][:, None].astype(np.int64), 1) > 0).all()


def test_a_sure_target_keeps_its_own_chain_alone():
    """Greedy decoding: the target's rows are one at a token."""
    V, T = 97, 6
    want = np.array([5, 90, 1, 2, 3, 40])
    p = np.zeros((2, T, V), np.float32)
    p[:, np.arange(T), want] = 1.0
    tok = np.zeros((2, T), np.int32)
    tok[:, 1:] = want[:-1]
    tok[1, 3] = 4  # the second sequence's third draft is another one
    par = np.tile(np.arange(-1, T - 1, dtype=np.int32), (2, 1))
    u = np.full((2, T), 0.999, np.float32)
    for q in (None, np.full_like(p, 1.0 / V)):
        got, _ = _run(p, q, tok, par, u)
        assert got[1].tolist() == [T, 3] and got[2].tolist() == [40, 1]


def test_what_the_draft_model_knows_exactly_is_taken():
    p, _, tok, par, u = _inputs(4, 10, 100, seed=2, wide=0)
    got, _ = _run(p, p, tok, par, np.minimum(u, np.float32(1 - 2.0 ** -24)))
    assert got[1].tolist() == [(row != -2).sum() for row in par]


def test_nothing_left_of_the_target():
    """q at or above p everywhere: the residual is empty, and the token comes from p."""
    V = 50
    p = np.zeros((1, 3, V), np.float32)
    p[0, :, 7] = p[0, :, 9] = 0.25
    q = np.full((1, 3, V), 0.5, np.float32)
    tok, par = np.array([[0, 3, 4]], np.int32), np.array([[-1, 0, 0]], np.int32)
    for x in (0.1, 0.9):
        u = np.array([[x, 0.5, 0.5]], np.float32)
        for replacement in (True, False):
            got, _ = _run(p, q, tok, par, u, replacement)
            _equal(got, verify(p, q, tok, par, u, replacement))
            assert got[2][0] == (7 if x < 0.5 else 9)


def test_siblings_with_the_same_token():
    V, T = 20, 6
    rng = np.random.default_rng(0)
    p, q = _softmax(rng.normal(size=(8, T, V))), _softmax(rng.normal(size=(8, T, V)))
    tok = np.array([[0, 4, 4, 4, 7, 4]] * 8, np.int32)
    par = np.array([[-1, 0, 0, 0, 0, 0]] * 8, np.int32)
    u = rng.random((8, T)).astype(np.float32)
    for qq, replacement in ((q, True), (q, False), (None, False)):
        got, _ = _run(p, qq, tok, par, u, replacement)
        _equal(got, verify(p, qq, tok, par, u, replacement))


def test_a_draft_row_that_is_used_up():
    """Without replacement, both tokens that the draft model knows are refused: nothing is tested after them."""
    V = 8
    q = np.zeros((1, 4, V), np.float32)
    q[..., 1] = q[..., 2] = 0.5
    p = np.full((1, 4, V), 1e-6, np.float32)
    p[..., 6] = 0.9
    tok, par = np.array([[0, 1, 2, 6]], np.int32), np.array([[-1, 0, 0, 0]], np.int32)
    u = np.array([[0.5, 0.9, 0.9, 0.0]], np.float32)
    got, _ = _run(p, q, tok, par, u)
    _equal(got, verify(p, q, tok, par, u, False))
    assert got[1][0] == 1


def test_idle_sequences_absent_drafts_and_one_tree_for_all():
    p, q, tok, _, u = _inputs(5, 7, 60, seed=9)
    row = np.array([-1, 0, -2, 0, 2, 3, 3], np.int32)  # node 4 follows an absent one
    par = torch.from_numpy(row).to(DEV).expand(5, 7)
    to = lambda x: torch.from_numpy(x).to(DEV)  # noqa: E731
    got = [x.cpu().numpy() for x in lib.draft_verify(to(p), to(tok), par, to(u), draft_probs=to(q))]
    _equal(got, verify(p, q, tok, np.tile(row, (5, 1)), u, False))
    idle = np.tile(row, (5, 1))
    idle[1, 0] = idle[4, 0] = -2
    got, status = _run(p, q, tok, idle, u)
    _equal(got, verify(p, q, tok, idle, u, False))
    assert got[2][1] == -1 and status == 0


def test_bad_parents_and_tokens_are_reported_and_absent():
    p, q, tok, par, u = _inputs(4, 6, 40, seed=5, wide=1, short=False)
    par[0, 3], tok[1, 2], tok[2, 1], par[3, 0] = 3, 40, -1, 0
    tok[0, 0] = 10 ** 6  # node 0's is not looked at
    got, status = _run(p, q, tok, par, u)
    _equal(got, verify(p, q, tok, par, u, False))
    assert status == 5
    _, status = _run(p[:1], q[:1], tok[:1] * 0, np.abs(par[:1]) * 0 - 1, u[:1])
    assert status == 0


def test_rows_without_anything_to_draw():
    p = np.zeros((2, 1, 300), np.float32)
    p[1] = np.nan
    one = np.zeros((2, 1), np.int32)
    got, status = _run(p, None, one, one - 1, np.full((2, 1), 0.5, np.float32))
    assert got[2].tolist() == [-1, -1] and got[1].tolist() == [1, 1] and status == 5


def test_nan_entries_count_as_zero():
    p, q, tok, par, u = _inputs(3, 9, 500, seed=12)
    rng = np.random.default_rng(1)
    p[rng.random(p.shape) < 0.1] = np.nan
    q[rng.random(q.shape) < 0.1] = np.nan
    got, _ = _run(p, q, tok, par, u)
    _equal(got, verify(p, q, tok, par, u, False))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_strided_views(dtype):
    """Rows of a larger logits tensor, at odd places, and tables with wider rows."""
    p, q, tok, par, u = _inputs(3, 8, 1001, seed=21, dtype=dtype)
    to = lambda x, t: torch.from_numpy(x).to(DEV, t)  # noqa: E731

    def wide(x, t, left, right):
        big = torch.full((x.shape[0], x.shape[1] + 2, *x.shape[2:]), 7, device=DEV, dtype=t)
        if x.ndim == 3:
            big = torch.full((x.shape[0], x.shape[1] + 2, x.shape[2] + left + right), 7.0, device=DEV, dtype=t)
            view = big[:, 1:-1, left:left + x.shape[2]]
        else:
            view = big[:, :x.shape[1]]
        view.copy_(to(x, t))
        return view

    got = lib.draft_verify(wide(p, dtype, 3, 2), wide(tok, torch.int32, 0, 0), wide(par, torch.int32, 0, 0),
                           wide(u, torch.float32, 0, 0), draft_probs=wide(q, dtype, 1, 5))
    _equal([x.cpu().numpy() for x in got], verify(p, q, tok, par, u, False))


def test_emitted_tokens_are_distributed_as_the_target():
    """The first token after node 0 over 60000 draws: within five standard deviations of the target's row, whatever
    the draft's was."""
    B, V = 60000, 6
    rng = np.random.default_rng(3)
    p, q = _softmax(rng.normal(size=V)), _softmax(1.5 * rng.normal(size=V))
    for mode in ("replacement", "distinct"):
        if mode == "replacement":
            tok = rng.choice(V, size=(B, 3), p=q / q.sum(dtype=np.float64))
        else:  # the largest of log q + noise, in order
            tok = np.argsort(-(np.log(q) + rng.gumbel(size=(B, V))), axis=1)[:, :3]
        tok = np.concatenate([np.zeros((B, 1), int), tok], 1).astype(np.int32)
        par = np.tile(np.array([-1, 0, 0, 0], np.int32), (B, 1))
        u = rng.random((B, 4)).astype(np.float32)
        P = torch.from_numpy(p).to(DEV).expand(B, 4, V)
        Q = torch.from_numpy(q).to(DEV).expand(B, 4, V)
        to = lambda x: torch.from_numpy(x).to(DEV)  # noqa: E731
        path, n, nxt = [x.cpu().numpy() for x in lib.draft_verify(P, to(tok), to(par), to(u), draft_probs=Q,
                                                                 replacement=mode == "replacement")]
        first = np.where(n == 1, nxt, tok[np.arange(B), np.maximum(path[:, 1], 0)])
        count = np.bincount(first, minlength=V)
        assert (np.abs(count - B * p) <= 5 * np.sqrt(B * p * (1 - p)) + 1).all(), (mode, count, B * p)
        # min(p, q) sums to 0.07 here: one draft in ten is taken, and these as the reference says
        k = 2000
        want = verify(np.tile(p, (k, 4, 1)), np.tile(q, (k, 4, 1)), tok[:k], par[:k], u[:k], mode == "replacement")
        _equal([x[:k] for x in (path, n, nxt)], want)
        assert (n == 2).any() and (n == 1).any()


def test_the_split_of_a_row_does_not_matter():
    """One sequence (a large cluster) and the same among 40 (a small one)."""
    p, q, tok, par, u = _inputs(1, 7, 40000, seed=31)
    rep = lambda x: np.repeat(x, 40, 0)  # noqa: E731
    a, _ = _run(p, q, tok, par, u)
    b, _ = _run(rep(p), rep(q), rep(tok), rep(par), rep(u))
    _equal(b, [rep(x) for x in a])
    _equal([a[0][0], a[1][0], a[2][0]], verify_one(p[0], q[0], tok[0], par[0], u[0], False))


def test_captured_and_on_another_stream():
    p, q, tok, par, u = _inputs(4, 9, 2000, seed=41)
    to = lambda x: torch.from_numpy(x).to(DEV)  # noqa: E731
    args = [to(x) for x in (p, tok, par, u)]
    Q, ws = to(q), lib.Workspace(256)
    want = verify(p, q, tok, par, u, False)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = lib.draft_verify(*args, draft_probs=Q, workspace=ws, stream=s)
    s.synchronize()
    _equal([x.cpu().numpy() for x in got], want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = lib.draft_verify(*args, draft_probs=Q, workspace=ws)
    p2, q2, tok2, par2, u2 = _inputs(4, 9, 2000, seed=42)
    for t, x in zip((*args, Q), (p2, tok2, par2, u2, q2)):
        t.copy_(to(x))
    g.replay()
    torch.cuda.synchronize()
    _equal([x.cpu().numpy() for x in got], verify(p2, q2, tok2, par2, u2, False))
