"""GPU tests of the calls together, as a server with a cache budget makes them:
a prompt with rotary positions, a step with a tree of drafts, single tokens,
the weights that each call's rows give to the cached tokens, the eviction, and
on over the shorter cache.  Every step is held against its definition in 64
bits, from the tensors that it was given, with the bounds of that operator's own
tests; a chain of steps as one captured graph gives the eager chain's bits."""
import ctypes
import math
import os
import sys

import pytest
import torch

import masked_attention_paged_gb300 as lib

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from test_gpu_10_rope import _define as rope_define, _freqs, _hold  # noqa: E402
from test_gpu_11_tree import _define as tree_define  # noqa: E402
from test_gpu_12_evict import _define as weights_define, _evict_define  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda"
B, HQ, HKV, T0, T1, KEEP, SINK, RECENT = 3, 8, 2, 70, 9, 48, 4, 16
PARENTS = [-1, 0, 0, 1, 1, 2, 3, -1, 7]
DEPTH = [0, 1, 1, 2, 2, 2, 3, 0, 1]
PATHS = [[0, 1, 3, 6], [7, 8, 0, 0], [0, 2, 5, 0]]
ACCEPT = [4, 2, 3]


def _int(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class _Server:
    def __init__(self, D, seed):
        g = torch.Generator().manual_seed(seed)
        self.D, self.gen = D, g
        mb, db = (T0 + 2 * T1 + 15) // 16, (KEEP + 15) // 16 + 1
        n = B * (mb + db) + 1
        perm = torch.randperm(n, generator=g).to(torch.int32).to(DEV)
        self.bt, self.dt = perm[:B * mb].view(B, mb), perm[B * mb:B * (mb + db)].view(B, db)
        self.kc, self.vc = (torch.zeros(n, HKV, 16, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        self.acc = torch.zeros(n, HKV, 16, device=DEV)
        self.inv, self.fr = _freqs(D // 2)
        size = max(lib.paged_tree_workspace_size(B, HQ, HKV, T1, mb, 16, D),
                   lib.paged_attn_weights_workspace_size(B, HKV, mb), lib.paged_decode_workspace_size(B, HQ, mb, 16, D))
        self.ws = lib.Workspace(size)  # one for every call

    def rand(self, heads, T):
        return torch.randn(B, T, heads, self.D, generator=self.gen).bfloat16().to(DEV).transpose(1, 2)

    def rows(self, cache, table, at):
        """[B, Hkv, n, D] of the slots at [B, n]."""
        blk = torch.gather(table.long(), 1, at // 16)
        return cache[blk, :, at % 16].transpose(1, 2)

    def weigh(self, q, lse, table, start, q_lens=None):
        was = self.acc.clone()
        lib.paged_attn_weights(q, lse, self.kc, table, start, self.acc, q_lens=q_lens, workspace=self.ws)
        four = q.dim() == 4
        ref, tol = weights_define(dict(q=q if four else q[:, :, None], lse=lse if four else lse[:, :, None], kc=self.kc,
                                       bt=table, acc=was, scale=1.0 / math.sqrt(self.D), causal=True, start=start,
                                       q_lens=q_lens))
        assert bool(((self.acc.double() - ref).abs() <= tol).all())

    def token(self, table, start, positions):
        """One token a sequence, as a tree of one: rotated, appended, attended to, weighed."""
        q, k, v = (self.rand(h, 1)[:, :, 0] for h in (HQ, HKV, HKV))
        rq = lib.rope_kv_append(q, k, v, positions, self.fr, self.kc, self.vc, table, start, workspace=self.ws)
        _hold(rq[:, :, None], *rope_define(q[:, :, None], positions[:, None], self.inv, False))
        kept = self.rows(self.kc, table, start.long()[:, None])
        _hold(kept, *rope_define(k[:, :, None], positions[:, None], self.inv, False))
        assert torch.equal(self.rows(self.vc, table, start.long()[:, None])[:, :, 0], v)
        out, lse = lib.paged_tree_attn(rq[:, :, None], self.kc, self.vc, table, start, _int([[-1]] * B),
                                       return_lse=True, workspace=self.ws)
        self.attended(out, lse, rq[:, :, None], kept, v[:, :, None], table, start, [[-1]] * B)
        self.weigh(rq, lse[:, :, 0], table, start)
        dec, dl = lib.paged_decode_attn(rq, self.kc, self.vc, table, start + 1, return_lse=True, workspace=self.ws)
        # the same rows by the decode call: weights rounded to bf16 shift a sum by 2^-8 at most, scores by far less
        assert dec.shape == rq.shape and bool(((dl - lse[:, :, 0]).abs() < 2.0 ** -7).all())

    def attended(self, out, lse, q, k, v, table, start, parents):
        ro, to, rl, tl, _, _ = tree_define(dict(q=q, k_new=k, v_new=v, kc=self.kc, vc=self.vc, bt=table, lens=start,
                                                parents=_int(parents)), 1.0 / math.sqrt(self.D))
        assert bool(((out.double() - ro).abs() <= to + ro.abs() * 2.0 ** -8 + 1e-30).all())
        assert bool(((lse.double() - rl).abs() <= tl).all())


@pytest.mark.parametrize("D", [64, 128])
def test_a_server_with_a_cache_budget(D):
    s = _Server(D, seed=D)
    zero = _int([0] * B)
    # the prompt
    q, k, v = s.rand(HQ, T0), s.rand(HKV, T0), s.rand(HKV, T0)
    pos = torch.arange(T0, dtype=torch.int32, device=DEV).expand(B, T0)
    rq = lib.rope_kv_append(q, k, v, pos, s.fr, s.kc, s.vc, s.bt, zero, workspace=s.ws)
    _hold(rq, *rope_define(q, pos, s.inv, False))
    _hold(s.rows(s.kc, s.bt, pos.long()), *rope_define(k, pos, s.inv, False))
    assert torch.equal(s.rows(s.vc, s.bt, pos.long()), v)
    _, lse = lib.paged_prefill_attn(rq, s.kc, s.vc, s.bt, zero, return_lse=True, workspace=s.ws)
    s.weigh(rq, lse, s.bt, zero)
    # a tree of drafts, of which a path each is accepted
    lens = zero + T0
    q, k, v = s.rand(HQ, T1), s.rand(HKV, T1), s.rand(HKV, T1)
    pos = T0 + _int([DEPTH] * B)
    rq, rk = lib.rope_apply(q, pos, s.fr), lib.rope_apply(k, pos, s.fr)
    out, lse = lib.paged_tree_attn(rq, s.kc, s.vc, s.bt, lens, _int([PARENTS] * B), k_new=rk, v_new=v, return_lse=True,
                                   workspace=s.ws)
    s.attended(out, lse, rq, rk, v, s.bt, lens, [PARENTS] * B)
    path, n = _int(PATHS), _int(ACCEPT)
    lib.kv_tree_accept(s.kc, s.vc, s.bt, lens, path, n, workspace=s.ws)
    for b in range(B):
        at = T0 + torch.arange(ACCEPT[b], device=DEV)
        for cache, new in ((s.kc, rk), (s.vc, v)):
            got = cache[s.bt[b, at // 16].long(), :, at % 16]
            assert torch.equal(got.transpose(0, 1), new[b][:, PATHS[b][:ACCEPT[b]]])
    idx = path.long()[:, None, :].expand(B, HQ, 4)
    s.weigh(torch.gather(rq, 2, idx[..., None].expand(B, HQ, 4, D)), torch.gather(lse, 2, idx).contiguous(), s.bt, lens,
            q_lens=n)
    lens = lens + n
    # single tokens
    for _ in range(2):
        s.token(s.bt, lens, lens)
        lens = lens + 1
    # the eviction, and on at the true positions over the shorter cache
    want = _evict_define(s.kc, s.vc, s.acc, s.bt, lens, s.dt, KEEP, SINK, RECENT)
    new_lens, kept = lib.kv_evict(s.kc, s.vc, s.acc, s.bt, lens, s.dt, KEEP, sink=SINK, recent=RECENT, workspace=s.ws)
    assert torch.equal(new_lens, want[0]) and torch.equal(kept, want[1])
    assert torch.equal(s.kc, want[2]) and torch.equal(s.vc, want[3])
    assert torch.equal(s.acc.view(torch.int32), want[4].view(torch.int32))
    for _ in range(3):
        s.token(s.dt, new_lens, lens)
        lens, new_lens = lens + 1, new_lens + 1
    assert s.ws.status() == 0


def test_the_same_steps_as_one_graph():
    """A draft step, its acceptance, its weights and the eviction, captured once and replayed, against eager calls."""
    s = _Server(128, seed=9)
    lens, n, path, parents = _int([T0, 31, 0]), _int(ACCEPT), _int(PATHS), _int([PARENTS] * B)
    s.kc.copy_(torch.randn(s.kc.shape, generator=s.gen))
    s.vc.copy_(torch.randn(s.vc.shape, generator=s.gen))
    s.acc.copy_(torch.rand(s.acc.shape, generator=s.gen))
    q, k, v = s.rand(HQ, T1), s.rand(HKV, T1), s.rand(HKV, T1)
    pos = lens[:, None] + _int([DEPTH])
    idx = path.long()[:, None, :].expand(B, HQ, 4)
    kept = torch.zeros(B, HKV, 40, dtype=torch.int32, device=DEV)
    new_lens = torch.zeros(B, dtype=torch.int32, device=DEV)

    def step():
        rq, rk = lib.rope_apply(q, pos, s.fr), lib.rope_apply(k, pos, s.fr)
        out, lse = lib.paged_tree_attn(rq, s.kc, s.vc, s.bt, lens, parents, k_new=rk, v_new=v, return_lse=True,
                                       workspace=s.ws)
        lib.kv_tree_accept(s.kc, s.vc, s.bt, lens, path, n, workspace=s.ws)
        lib.paged_attn_weights(torch.gather(rq, 2, idx[..., None].expand(B, HQ, 4, 128)),
                               torch.gather(lse, 2, idx).contiguous(), s.kc, s.bt, lens, s.acc, q_lens=n,
                               workspace=s.ws)
        lib.kv_evict(s.kc, s.vc, s.acc, s.bt, lens + n, s.dt, 40, sink=SINK, recent=RECENT, new_lens=new_lens,
                     kept=kept, workspace=s.ws)
        return rq, out, lse

    start = [x.clone() for x in (s.kc, s.vc, s.acc)]

    def results(got):
        return [x.clone() for x in (*got, s.kc, s.vc, s.acc, new_lens, kept)]

    want = results(step())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(2):
        for x, y in zip((s.kc, s.vc, s.acc), start):
            x.copy_(y)
        graph.replay()
        for x, y in zip(results(got), want):
            assert torch.equal(x, y)
    assert s.ws.status() == 0


def test_another_stream_than_the_current_one():
    """What a call allocates belongs to the stream that it runs on: nothing still queued on the current stream may
    write to it, and it may be called with a raw handle."""
    s = _Server(64, seed=3)
    lens, parents, path, n = _int([T0, 31, 5]), _int([PARENTS] * B), _int(PATHS), _int(ACCEPT)
    s.kc.copy_(torch.randn(s.kc.shape, generator=s.gen))
    s.vc.copy_(torch.randn(s.vc.shape, generator=s.gen))
    q, k, v, pos = s.rand(HQ, T1), s.rand(HKV, T1), s.rand(HKV, T1), _int([DEPTH] * B)
    start = s.kc.clone(), s.vc.clone(), s.acc.clone()
    big = torch.randn(4096, 4096, device=DEV)

    def chain(stream):
        for x, y in zip((s.kc, s.vc, s.acc), start):
            x.copy_(y)
        torch.cuda.synchronize()
        if stream is not None:
            for _ in range(20):
                big @ big  # the current stream stays busy, and fills what it then frees
            for shape in ((B, HQ, T1, 64), (B, HQ, T1), (B, HKV, 40), (B,)):
                torch.full(shape, 7, dtype=torch.int32, device=DEV)
        kw = dict(stream=stream)
        rq, rk = lib.rope_apply(q, pos, s.fr, **kw), lib.rope_apply(k, pos, s.fr, **kw)
        out, lse = lib.paged_tree_attn(rq, s.kc, s.vc, s.bt, lens, parents, k_new=rk, v_new=v, return_lse=True, **kw)
        lib.kv_tree_accept(s.kc, s.vc, s.bt, lens, path, n, **kw)
        lib.paged_attn_weights(rq, lse, s.kc, s.bt, lens, s.acc, q_lens=n, **kw)
        nl, kept = lib.kv_evict(s.kc, s.vc, s.acc, s.bt, lens, s.dt, 40, sink=1, recent=2, **kw)
        torch.cuda.synchronize()
        return [x.clone() for x in (rq, out, lse, s.kc, s.vc, s.acc, nl, kept)]

    want = chain(None)
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        for x, y in zip(chain(stream), want):
            assert torch.equal(x, y)


@pytest.mark.parametrize("D,Hkv", [(128, 2), (64, 1)])
def test_a_captured_decode_step_whose_contexts_grow(D, Hkv):
    """One graph over contexts that gain splits between replays, and lose some again: the eager call's bits."""
    g = torch.Generator().manual_seed(4)
    mb = 400
    bt = torch.randperm(2 * mb, generator=g).to(torch.int32).view(2, mb).to(DEV)
    kc, vc = (torch.randn(2 * mb, Hkv, 16, D, generator=g).bfloat16().to(DEV) for _ in range(2))
    q = torch.randn(2, 4 * Hkv, D, generator=g).bfloat16().to(DEV)
    lens, out = _int([1000, 900]), torch.empty_like(q)
    ws = lib.Workspace(lib.paged_decode_workspace_size(2, 4 * Hkv, mb, 16, D))
    lib.paged_decode_attn(q, kc, vc, bt, lens, out=out, workspace=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lib.paged_decode_attn(q, kc, vc, bt, lens, out=out, workspace=ws)
    for now in ([1000, 900], [2500, 900], [4700, 1100], [6400, 6000], [1500, 6400], [3100, 17]):
        lens.copy_(_int(now))
        want = lib.paged_decode_attn(q, kc, vc, bt, lens)
        for _ in range(3):
            out.zero_()
            graph.replay()
            assert torch.equal(out, want), now
    assert ws.status() == 0


def test_a_compiled_call_passes_what_the_worded_checks_pass(monkeypatch):
    """Each call takes its arguments in one compiled step where they are plainly as documented: the same ones."""
    s = _Server(64, seed=1)
    got, keep = [], []
    bytes_of = lambda p, n: ctypes.string_at(p, n)  # noqa: E731

    def entry(name):
        """A C function of the entry's type that notes its arguments, descriptors by their bytes."""
        res, types = lib._signatures()[name]
        tensors, cache = {"rope_apply": ((0, 8), -1), "rope_kv_append": ((0, 1, 2, 9), 10),
                          "paged_tree_attn": ((0, 1, 2, 11), 3), "kv_tree_accept": ((), 0),
                          "paged_attn_weights": ((0,), 2), "kv_evict": ((), 0)}[name]

        def note(*args):
            seen = list(args)
            for i in (*tensors, cache):
                if i >= 0 and seen[i] is not None:
                    seen[i] = bytes_of(seen[i], ctypes.sizeof(lib.AttnKVCache if i == cache else lib.AttnTensor))
            got.append((name, seen))
            return 0
        keep.append(ctypes.CFUNCTYPE(res, *types)(note))
        return keep[-1]

    names = ("rope_apply", "rope_kv_append", "paged_tree_attn", "kv_tree_accept", "paged_attn_weights", "kv_evict")
    fake = {n: entry(n) for n in names}

    class Recorder:
        def __getattr__(self, name):
            return ctypes.CFUNCTYPE(ctypes.c_int, *lib._signatures()[name][1])(
                ctypes.cast(fake[name], ctypes.c_void_p).value)

    lens, path, n = _int([5, 6, 7]), _int(PATHS), _int(ACCEPT)
    q, k, v, pos = s.rand(HQ, T1), s.rand(HKV, T1), s.rand(HKV, T1), _int([DEPTH] * B)
    out, lse = torch.empty_like(q), torch.empty(B, HQ, T1, device=DEV)
    nl, kept = torch.empty_like(lens), torch.empty(B, HKV, 40, dtype=torch.int32, device=DEV)
    ws = s.ws
    calls = [
        lambda: lib.rope_apply(q, pos, s.fr, interleaved=True, magnitude=1.5, out=out),
        lambda: lib.rope_apply(q[:, :, 0], pos[:, 0], s.fr, inverse=True, out=out[:, :, 0]),
        lambda: lib.rope_kv_append(q, k, v, pos, s.fr, s.kc, s.vc, s.bt, lens, q_out=out, workspace=ws),
        lambda: lib.rope_kv_append(q[:, :, 1], k[:, :, 1], v[:, :, 1], lens, s.fr, s.kc, s.vc, s.bt[:, :2], lens,
                                   q_out=out[:, :, 0]),
        lambda: lib.paged_tree_attn(q, s.kc, s.vc, s.bt, lens, pos, k_new=k, v_new=v, out=out, lse=lse, workspace=ws),
        lambda: lib.paged_tree_attn(q, s.kc, s.vc, s.bt, lens, pos[:1].expand(B, T1), out=out, scale=0.5, workspace=ws),
        lambda: lib.kv_tree_accept(s.kc, s.vc, s.bt, lens, path, n, workspace=ws),
        lambda: lib.paged_attn_weights(q, lse, s.kc, s.bt, lens, s.acc, q_lens=n, causal=False, workspace=ws),
        lambda: lib.paged_attn_weights(q[:, :, 0], lse[:, :, 0].contiguous(), s.kc, s.bt, lens, s.acc, workspace=ws),
        lambda: lib.kv_evict(s.kc, s.vc, s.acc, s.bt, lens, s.dt, 40, sink=1, recent=2, new_lens=nl, kept=kept,
                             workspace=ws),
    ]
    lib.rope_apply(q, pos, s.fr)  # the module is loaded
    assert lib._marshal is not None, "marshal.cpp was not built"
    monkeypatch.setattr(lib, "_entries", {n: ctypes.cast(f, ctypes.c_void_p).value for n, f in fake.items()})
    for call in calls:
        call()
    compiled, got[:] = list(got), []
    assert len(compiled) == len(calls)
    monkeypatch.setattr(lib, "_call", lambda *a: False)
    monkeypatch.setattr(lib, "load", lambda *a, **k: Recorder())
    for call in calls:
        call()
    assert got == compiled
    # what is not plainly as documented goes the other way, and calls nothing
    entry = ctypes.cast(fake["rope_apply"], ctypes.c_void_p).value
    got[:] = []

    def go(fmt, *args, name="rope_apply"):
        return lib._marshal.call(entry, name, fmt, *args)

    for fmt, args in (("x", [q.cpu()]), ("x", [q.half()]), ("x", [q[0]]), ("x", [None]), ("x", [1.0]), ("x", []),
                      ("x", [q, q]), ("yR", [q, pos.long()]), ("yR", [q, pos[:, :3]]), ("yR", [q, pos.t()]),
                      ("xv", [q, lens[:2]]), ("xb", [q, s.bt[:2]]), ("xb", [q, s.bt.t()]), ("xl", [q, lse[:, :, ::2]]),
                      ("xY", [q, q.float()]), ("xX", [q, k]), ("yf", [q, s.fr.int()]), ("yf", [q, s.fr.repeat(4)]),
                      ("c", [s.kc, s.vc[:-1]]), ("c", [s.kc, s.vc.float()]), ("cA", [s.kc, s.vc, s.acc[:-1]]),
                      ("bV", [s.bt[:2], lens]), ("c", [s.kc]), ("=", ["1"]), ("=", [1 << 70]), ("x" * 9, [q] * 9),
                      ("=" * 40, [0] * 40), ("=", [None]), ("W", [lens]), ("W", [ws.tensor[::2]]), ("S", [1.5])):
        assert go(fmt, *args) is None, fmt
    for bad in (lambda: go("?", q), lambda: go("x", q), lambda: go("x", q, name="attn_fwd")):
        with pytest.raises(ValueError):
            bad()
    assert got == []
