"""Sessions of the calls together, as a server makes them: an e4m3 cache whose blocks are
reserved, filled, attended to, forked, given back and moved together, and steps of
drafting (reserve, tree attention, verification, acceptance), eager and captured."""
import math

import numpy as np
import pytest
import torch

import masked_attention_paged_gb300 as lib
from _serve_ref import BS, append_f8, attn_f8, verify
from test_gpu_17_f8 import F8, _bf, _compare, _ints

pytestmark = pytest.mark.gpu
DEV = "cuda"


class F8Server:
    """The books of one layer's e4m3 cache, and its reference in numpy."""

    def __init__(self, N, B, width, H, G, D):
        self.H, self.G, self.D, self.N = H, G, D, N
        self.codes = [torch.zeros((N, H, BS, D), dtype=torch.uint8, device=DEV).view(F8) for _ in range(2)]
        self.scales = [torch.full((N, H), math.nan, device=DEV) for _ in range(2)]  # none is written
        self.refs = _ints([0] * N)
        self.table, self.lens = _ints(np.full((B, width), -1)), _ints([-1] * B)
        self.ws = lib.Workspace(max([lib.kv_pool_workspace_size(N, 4 * B)] + [
            lib.paged_attn_f8_workspace_size(B, H * G, H, T, width, BS, D) for T in (1, 9, 17, 30, 33, 40)]))

    def caches(self):
        return [*self.codes, *self.scales]

    def step(self, q, k, v, new):
        """Reserve, append, attend with new[b] tokens a sequence; the reference's state is read back before."""
        n = _ints(new)
        lib.kv_reserve(self.refs, self.table, self.lens, n, workspace=self.ws)
        table, start = self.table.cpu().numpy(), self.lens.cpu().numpy()
        want = [[c.view(torch.uint8).cpu().numpy() for c in self.codes], [s.cpu().numpy() for s in self.scales]]
        for i, x in enumerate((k, v)):
            assert not append_f8(want[0][i], want[1][i], table, start, x.float().cpu().numpy(), new)
        lib.kv_append_f8(*self.caches(), self.table, self.lens, k, v, lens=n, workspace=self.ws)
        got, lse = lib.paged_attn_f8(q, *self.caches(), self.table, self.lens, lens=n, return_lse=True,
                                     workspace=self.ws)
        for i in range(2):
            assert np.array_equal(self.codes[i].view(torch.uint8).cpu().numpy(), want[0][i])
            assert np.array_equal(self.scales[i].cpu().numpy(), want[1][i], equal_nan=True)
        qn, T = q.double().cpu().numpy(), q.shape[2]
        ref = attn_f8(qn, want[0][0], want[1][0], want[0][1], want[1][1], table, start, 1 / math.sqrt(self.D), True, new)
        _compare(got, lse, *ref, qn, want[0], want[1], 1 / math.sqrt(self.D), T * self.G, torch.bfloat16)
        self.lens += torch.where(self.lens >= 0, n, 0)
        assert self.ws.status() == 0
        return got

    def look(self, q):
        """Attention of one query each at the last token."""
        return lib.paged_attn_f8(q, *self.caches(), self.table, self.lens - 1, workspace=self.ws)


@pytest.mark.parametrize("H,G,D", [(2, 4, 128), (3, 1, 64), (1, 16, 128)])
def test_an_e4m3_cache_through_its_life(H, G, D):
    rng = np.random.default_rng(H)
    B, N, width = 5, 26, 8
    s = F8Server(N, B, width, H, G, D)

    def rows(T):
        return _bf((B, H * G, T, D), rng), _bf((B, H, T, D), rng), _bf((B, H, T, D), rng, 20.0)

    # two prompts of a batch of five rows, in chunks; the others idle
    s.lens.copy_(_ints([0, 0, -1, -1, -1]))
    s.step(*rows(40), [40, 23, 40, 40, 40])
    s.step(*rows(17), [0, 17, 0, 0, 0])
    # samples of both go on from their prompts, in rows 2 to 4
    child, cl = s.table[2:], s.lens[2:]
    lib.kv_fork(s.caches(), s.refs, s.table[:2], s.lens[:2], _ints([0, 1, 0]), child, cl, workspace=s.ws)
    assert s.lens.cpu().tolist() == [40, 40, 40, 40, 40] and s.ws.status() == 0
    assert s.refs.sum().item() == 5 * 3 and (s.refs == 3).sum().item() == 2 and (s.refs == 2).sum().item() == 2
    q = _bf((B, H * G, D), rng)
    for _ in range(2):  # every row has its own last block
        s.step(*rows(9), [9, 3, 1, 9, 0])
    # rows 0 and 3 end; what the others see stays through the moves
    lib.kv_free(s.refs, s.table, s.lens, _ints([1, 0, 0, 1, 0]), workspace=s.ws)
    before = s.look(q)
    used = lib.kv_compact(s.caches(), s.refs, s.table, workspace=s.ws)
    left = s.table.cpu().numpy()
    assert used.item() == len(np.unique(left[left >= 0])) == left.max() + 1
    after = s.look(q)
    assert torch.equal(before, after) and s.lens.cpu().tolist() == [-1, 46, 42, -1, 40]
    assert (after[0] == 0).all() and (after[3] == 0).all()
    # the freed rows take new sequences, among the moved blocks
    s.lens.copy_(_ints([0, 46, 42, -1, 40]))
    s.step(*rows(33), [33, 1, 5, 33, 30])
    lib.kv_free(s.refs, s.table, s.lens, workspace=s.ws)
    assert (s.refs == 0).all() and (s.table == -1).all() and (s.lens == -1).all() and s.ws.status() == 0


# --------------------------------------------------------------------------
# drafting
# --------------------------------------------------------------------------
T, H, G, D, V, WIDTH = 7, 2, 2, 64, 500, 6
PARENTS = [[-1, 0, 0, 1, 1, 2, 3], [-1, 0, 1, 2, 3, 4, 5], [-1, 0, 0, 0, 1, 2, -2]]
B = len(PARENTS)


class Drafting:
    def __init__(self, seed=0):
        g = torch.Generator(device=DEV).manual_seed(seed)
        rand = lambda *s: torch.randn(*s, device=DEV, generator=g)
        self.k, self.v = (torch.zeros(24, H, BS, D, device=DEV, dtype=torch.bfloat16) for _ in range(2))
        self.refs, self.table, self.lens = _ints([0] * 24), _ints(np.full((B, WIDTH), -1)), _ints([5, 0, 30])
        self.parents, self.new = _ints(PARENTS), _ints([T] * B)
        self.embed = {x: rand(V, h, D).to(torch.bfloat16) for x, h in (("q", H * G), ("k", H), ("v", H))}
        self.head = rand(H * G * D, V) * 0.3
        self.tokens = _ints(np.zeros((B, T)))
        self.uniforms, self.draft = torch.empty(B, T, device=DEV), torch.empty(B, T, V, device=DEV)
        self.ws = lib.Workspace(max(lib.kv_pool_workspace_size(24, B), lib.draft_verify_workspace_size(B, T, V),
                                    lib.paged_tree_workspace_size(B, H * G, H, T, WIDTH, BS, D)))
        self.path, self.n, self.next = _ints(np.zeros((B, T))), _ints([0] * B), _ints([0] * B)
        self.probs = torch.empty(B, T, V, device=DEV)
        lib.kv_reserve(self.refs, self.table, _ints([0] * B), self.lens, workspace=self.ws)
        for c in (self.k, self.v):
            c.copy_(rand(*c.shape))

    def draw(self, rng):
        """What the draft model does: a distribution a node, and its children drawn without replacement."""
        p = rng.dirichlet(np.full(V, 0.02), (B, T)).astype(np.float32)
        tok = np.zeros((B, T), np.int32)
        for b in range(B):
            tok[b, 0] = self.next[b].item()
            for node in range(T):
                kids = [t for t in range(T) if PARENTS[b][t] == node]
                tok[b, kids] = rng.choice(V, len(kids), replace=False, p=p[b, node].astype(np.float64) / p[b, node].sum(
                    dtype=np.float64)) if kids else 0
        self.tokens.copy_(_ints(tok))
        self.draft.copy_(torch.from_numpy(p))
        self.uniforms.copy_(torch.from_numpy(rng.random((B, T), np.float32)))

    def step(self):
        lib.kv_reserve(self.refs, self.table, self.lens, self.new, workspace=self.ws)
        q, k, v = (self.embed[x][self.tokens.long()].transpose(1, 2) for x in "qkv")
        o = lib.paged_tree_attn(q, self.k, self.v, self.table, self.lens, self.parents, k_new=k, v_new=v,
                                workspace=self.ws)
        logits = o.transpose(1, 2).reshape(B, T, -1).float() @ self.head
        # (half the target is the draft's, so that some drafts are kept)
        self.probs.copy_(0.5 * torch.softmax(logits, -1) + 0.5 * self.draft)
        lib.draft_verify(self.probs, self.tokens, self.parents, self.uniforms, self.draft, path=self.path,
                         n_accept=self.n, next_token=self.next, workspace=self.ws)
        lib.kv_tree_accept(self.k, self.v, self.table, self.lens, self.path, self.n, workspace=self.ws)
        self.lens += self.n

    def state(self):
        return [x.clone() for x in (self.k, self.v, self.refs, self.table, self.lens, self.path, self.n, self.next)]


def test_steps_of_drafting():
    d, rng, kept = Drafting(), np.random.default_rng(3), 0
    said = [[] for _ in range(B)]  # the tokens behind each prompt
    first = d.lens.cpu().tolist()
    for _ in range(5):
        d.draw(rng)
        tokens = d.tokens.cpu().numpy()
        d.step()
        path, n, nxt = verify(d.probs.double().cpu().numpy(), d.draft.double().cpu().numpy(), tokens,
                              np.array(PARENTS), d.uniforms.double().cpu().numpy(), False)
        assert d.path.cpu().tolist() == np.asarray(path).tolist() and d.n.cpu().tolist() == list(n)
        assert d.next.cpu().tolist() == list(nxt) and d.ws.status() == 0
        kept += sum(n) - B
        lens = d.lens.cpu().tolist()
        got = [lib.paged_kv_gather(c, d.table, d.lens, max(lens)) for c in (d.k, d.v)]
        for b in range(B):
            said[b] += [int(tokens[b, t]) for t in path[b][:n[b]]]
            assert lens[b] == first[b] + len(said[b])
            for c, x in zip(got, "kv"):  # their rows, in order, behind the prompt
                assert torch.equal(c[b, :, first[b]:lens[b]], d.embed[x][said[b]].transpose(0, 1))
    assert kept > 0  # (the draws above keep some drafts, and refuse some)
    assert kept < 5 * 12
    have = (d.table >= 0).sum(1).cpu().tolist()  # blocks that were drafted into stay reserved
    assert all(h * BS >= x for h, x in zip(have, d.lens.cpu().tolist())) and d.refs.sum().item() == sum(have)


def test_a_captured_step_of_drafting():
    eager, graph = Drafting(), Drafting()
    for d in (eager, graph):  # warm
        d.draw(np.random.default_rng(8))
    saved = graph.state()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph.step()
    torch.cuda.current_stream().wait_stream(side)
    for x, y in zip((graph.k, graph.v, graph.refs, graph.table, graph.lens, graph.path, graph.n, graph.next), saved):
        x.copy_(y)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        graph.step()
    for i in range(4):
        for d in (eager, graph):
            d.draw(np.random.default_rng(20 + i))
        eager.step()
        g.replay()
        for x, y in zip(eager.state(), graph.state()):
            assert torch.equal(x, y)
    assert eager.ws.status() == 0 and graph.ws.status() == 0


def test_two_pools_on_two_streams():
    """Calls with workspaces and tensors of their own do not meet."""
    servers = [F8Server(40, 3, 8, 2, 2, 64) for _ in range(2)]
    alone = F8Server(40, 3, 8, 2, 2, 64)
    rng = np.random.default_rng(11)
    data = [(_bf((3, 4, 30, 64), rng), _bf((3, 2, 30, 64), rng), _bf((3, 2, 30, 64), rng)) for _ in range(4)]

    def run(s, stream):
        outs = []
        for q, k, v in data:
            n = s.n30
            lib.kv_reserve(s.refs, s.table, s.lens, n, workspace=s.ws, stream=stream)
            lib.kv_append_f8(*s.caches(), s.table, s.lens, k, v, workspace=s.ws, stream=stream)
            outs.append(lib.paged_attn_f8(q, *s.caches(), s.table, s.lens, workspace=s.ws, stream=stream))
            with torch.cuda.stream(stream):
                s.lens += n
        used = lib.kv_compact(s.caches(), s.refs, s.table, workspace=s.ws, stream=stream)
        return outs + [used]

    for s in servers + [alone]:
        s.n30 = _ints([30] * 3)
        s.lens.zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [run(s, st) for s, st in zip(servers, streams)]
    torch.cuda.synchronize()
    want = run(alone, torch.cuda.current_stream())
    torch.cuda.synchronize()
    for got, s in zip(outs, servers):
        for x, y in zip(got, want):
            assert torch.equal(x, y)
        assert torch.equal(s.table, alone.table) and torch.equal(s.refs, alone.refs) and s.ws.status() == 0


@pytest.mark.parametrize("shape", [(3, 4, 64), (3, 4, 1, 64), (3, 4, 9, 64), (3, 4, 40, 128)])
def test_results_made_or_given(shape):
    """The same numbers in tensors of the caller, in those that the call makes, on a stream that is passed, and
    without a workspace."""
    rng = np.random.default_rng(len(shape))
    Bq, Hq, D = shape[0], shape[1], shape[-1]
    n = shape[2] if len(shape) == 4 else 1
    s = F8Server(30, Bq, 6, 2, Hq // 2, D)
    s.lens.copy_(_ints([0, 0, 0]))
    k, v = (_bf((Bq, 2, 50, D), rng) for _ in range(2))
    lib.kv_reserve(s.refs, s.table, s.lens, _ints([50] * 3), workspace=s.ws)
    lib.kv_append_f8(*s.caches(), s.table, s.lens, k, v, workspace=s.ws)
    start = _ints([50 - n, 3, -1])
    q = _bf(shape, rng)
    ws = lib.Workspace(lib.paged_attn_f8_workspace_size(Bq, Hq, 2, n, 6, BS, D))
    args = (q, *s.caches(), s.table, start)
    out, lse = torch.empty_like(q), torch.empty(shape[:-1], device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = [(lib.paged_attn_f8(*args, out=out, lse=lse, workspace=ws), lse)]
    got.append(lib.paged_attn_f8(*args, return_lse=True, workspace=ws))
    got.append((lib.paged_attn_f8(*args, lse=torch.empty_like(lse), workspace=ws), lse))
    got.append(lib.paged_attn_f8(*args, out=torch.empty_like(q), return_lse=True, workspace=ws))
    got.append(lib.paged_attn_f8(*args, return_lse=True))
    got.append((lib.paged_attn_f8(*args, workspace=ws), lse))
    torch.cuda.synchronize()
    got.append(lib.paged_attn_f8(*args, return_lse=True, workspace=ws, stream=side))
    torch.cuda.synchronize()
    assert got[0][0] is out
    for o, l in got:
        assert o.shape == shape and o.dtype == q.dtype and o.is_contiguous() and torch.equal(o, out)
        assert l.shape == shape[:-1] and l.dtype == torch.float32 and torch.equal(l, lse)
    f32 = lib.paged_attn_f8(*args, out=torch.empty(shape, device=DEV), workspace=ws)
    assert f32.dtype == torch.float32 and torch.equal(f32.to(torch.bfloat16), out)
    for bad in (dict(out=torch.empty(shape[1:], device=DEV)), dict(lse=torch.empty(7, device=DEV)),
                dict(lens=_ints([1, 1])), dict(lse=True), dict(lse=True, return_lse=True, stream=side)):
        with pytest.raises(ValueError):
            lib.paged_attn_f8(*args, workspace=ws, **bad)


def test_verified_paths_and_used_blocks_made_or_given():
    d = Drafting()
    d.draw(np.random.default_rng(1))
    d.probs.copy_(d.draft)
    args = (d.probs, d.tokens, d.parents, d.uniforms, d.draft)
    want = lib.draft_verify(*args, path=d.path, n_accept=d.n, next_token=d.next, workspace=d.ws)
    assert want[0] is d.path and want[1] is d.n and want[2] is d.next
    for kw in (dict(workspace=d.ws), dict(), dict(workspace=d.ws, n_accept=_ints([9] * B)),
               dict(workspace=d.ws, path=_ints(np.zeros((B, T))), next_token=_ints([9] * B)),
               dict(workspace=d.ws, stream=torch.cuda.current_stream())):
        got = lib.draft_verify(*args, **kw)
        for x, y in zip(got, want):
            assert x.dtype == torch.int32 and x.shape == y.shape and x.is_contiguous() and torch.equal(x, y)
        for name, x in zip(("path", "n_accept", "next_token"), got):
            assert kw.get(name, x) is x
    for bad in (dict(path=_ints(np.zeros((B, T + 1)))), dict(n_accept=_ints([0])), dict(next_token=d.uniforms[:, 0])):
        with pytest.raises(ValueError):
            lib.draft_verify(*args, workspace=d.ws, **bad)
    q = torch.zeros(B, H * G, T, D, device=DEV, dtype=torch.bfloat16)
    with pytest.raises(ValueError):  # a result that no call makes
        lib.paged_tree_attn(q, d.k, d.v, d.table, d.lens, d.parents, lse=True, workspace=d.ws)
    with pytest.raises(ValueError):
        lib.draft_verify(*args[:4], True, workspace=d.ws)
    used = [lib.kv_compact([d.k, d.v], d.refs, d.table, workspace=w, used=u)
            for w in (d.ws, None) for u in (None, _ints([77]))]
    assert len({u.item() for u in used}) == 1 and all(u.shape == (1,) and u.dtype == torch.int32 for u in used)
