"""GPU tests of the tree attention against its definition in 64 bits.

Error bounds.  A score is an fp32 sum of D exact products: off by at most D
2^-23 of the sum of their sizes (an accumulation may truncate), call it e_s
after scaling (in natural-log units), plus 2^-20 for the log2 scaling, the
subtraction and ex2.approx over the range the tests draw (|x| < 8 is off by
2^-21; larger |x| weigh less than e^-8).  Weights go to bf16 before P.V: half a
step, 2^-8 of each.  So out is off by at most (2^-8 + 2 e_s) sum p |v| plus half
a step of its own type, and lse by e_s + 2^-22 |lse|."""
import math

import pytest
import torch

import masked_attention_paged_gb300 as lib

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _tree(T, wide, g):
    par = [-1]
    for t in range(1, T):
        par.append(int(torch.randint(max(-1, t - 1 - wide), t, (1,), generator=g)))
    return par


def _make(lens, T, Hq, Hkv, D, seed, wide=3, gain=1.0, cut=True, extra=0):
    """Caches whose free slots are NaN, a shuffled table, q/k/v, and trees (every third one cut short)."""
    g = _gen(seed)
    B = len(lens)
    mb = max(1, (max(max(lens), 0) + T + 15) // 16 + extra)
    nb = B * mb + 3
    bt = torch.randperm(nb, generator=g)[:B * mb].to(torch.int32).view(B, mb)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    kc, vc = (torch.full((nb, Hkv, 16, D), float("nan"), dtype=torch.bfloat16) for _ in range(2))
    for b, n in enumerate(lens):
        for i in range(max(0, (n + 15) // 16)):
            m = min(16, n - 16 * i)
            kc[bt[b, i], :, :m] = r(Hkv, m, D).bfloat16()
            vc[bt[b, i], :, :m] = r(Hkv, m, D).bfloat16()
    parents = torch.full((B, T), -2, dtype=torch.int32)
    for b in range(B):
        n = T if not cut or b % 3 != 1 else max(1, T // 2)
        parents[b, :n] = torch.tensor(_tree(n, wide, g), dtype=torch.int32)
    s = dict(q=(r(B, T, Hq, D) * gain).bfloat16().transpose(1, 2), k_new=r(B, Hkv, T, D).bfloat16(),
             v_new=r(B, T, Hkv, D).bfloat16().transpose(1, 2), kc=kc, vc=vc, bt=bt, parents=parents,
             lens=torch.tensor(lens, dtype=torch.int32))
    return {k: v.to(DEV) for k, v in s.items()}


def _seen(parents):
    """[T, T] bool: row t sees draft a; all False for absent drafts."""
    T = len(parents)
    see = torch.zeros(T, T, dtype=torch.bool)
    for t in range(T):
        a, path = t, []
        while 0 <= a < T:
            path.append(a)
            up = parents[a]
            if up >= a or up < -1:
                path = []
                break
            a = up
        see[t, path] = True
    return see


def _define(s, scale):
    """out, lse, their bounds before the output's rounding, and the caches after the append."""
    q = s["q"].double()
    B, Hq, T, D = q.shape
    Hkv = s["kc"].shape[1]
    G = Hq // Hkv
    out, tol_o = torch.zeros_like(q), torch.zeros_like(q)
    lse = torch.full((B, Hq, T), -math.inf, dtype=torch.float64, device=DEV)
    tol_l = torch.zeros_like(lse)
    kc, vc = s["kc"].clone(), s["vc"].clone()
    mb = s["bt"].shape[1]
    for b in range(B):
        n = int(s["lens"][b])
        if n < 0 or n + T > mb * 16:
            continue
        see = _seen(s["parents"][b].tolist()).to(DEV)
        there = see.any(1)
        at = torch.arange(n, device=DEV)
        blk = s["bt"][b, at // 16].long()
        for j in torch.nonzero(there).flatten().tolist():
            p = n + j
            kc[s["bt"][b, p // 16].long(), :, p % 16] = s["k_new"][b, :, j]
            vc[s["bt"][b, p // 16].long(), :, p % 16] = s["v_new"][b, :, j]
        for h in range(Hq):
            k = torch.cat([s["kc"][blk, h // G, at % 16], s["k_new"][b, h // G]]).double()
            v = torch.cat([s["vc"][blk, h // G, at % 16], s["v_new"][b, h // G]]).double()
            for t in torch.nonzero(there).flatten().tolist():
                idx = torch.cat([at, n + torch.nonzero(see[t]).flatten()])
                kk, vv = k[idx], v[idx]
                x = kk @ q[b, h, t] * scale
                l = torch.logsumexp(x, 0)
                w = torch.exp(x - l)
                out[b, h, t], lse[b, h, t] = w @ vv, l
                size = float((kk.abs() @ q[b, h, t].abs()).max()) * abs(scale)
                e = D * 2.0 ** -23 * size + 2.0 ** -20
                tol_o[b, h, t] = (2.0 ** -8 + 2 * e) * (w @ vv.abs())
                tol_l[b, h, t] = e + 2.0 ** -22 * abs(float(l))
    return out, tol_o, lse, tol_l, kc, vc


def _bits(t):
    return t.view(torch.int16)


def _run(s, scale=None, out=None, ws=None, **kw):
    B, Hq, T, D = s["q"].shape
    Hkv, mb = s["kc"].shape[1], s["bt"].shape[1]
    ws = ws or lib.Workspace(lib.paged_tree_workspace_size(B, Hq, Hkv, T, mb, 16, D))
    kc, vc = s["kc"].clone(), s["vc"].clone()
    kw = {"k_new": s["k_new"], "v_new": s["v_new"], **kw}
    o, l = lib.paged_tree_attn(s["q"], kc, vc, s["bt"], s["lens"], s["parents"], scale=scale, out=out,
                               return_lse=True, workspace=ws, **kw)
    return o, l, kc, vc, ws.status()


def _check(s, scale=None, out_dtype=torch.bfloat16, status=0):
    D = s["q"].shape[-1]
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    out = torch.full(s["q"].shape, 55.0, dtype=out_dtype, device=DEV)
    o, l, kc, vc, st = _run(s, scale, out)
    assert st == status
    ro, to, rl, tl, ek, ev = _define(s, scale)
    assert torch.equal(torch.isneginf(l), torch.isneginf(rl))
    fin = ~torch.isneginf(rl)
    assert bool(((l.double() - rl).abs()[fin] <= tl[fin]).all()), float(((l.double() - rl).abs()[fin] - tl[fin]).max())
    bound = to + ro.abs() * torch.finfo(out_dtype).eps / 2
    err = (o.double() - ro).abs()
    assert bool((err <= bound * (1 + 1e-9) + 1e-30).all()), float((err - bound).max())
    assert torch.equal(_bits(kc), _bits(ek)) and torch.equal(_bits(vc), _bits(ev))
    return o, l


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T,Hq,Hkv", [(1, 2, 2), (1, 8, 1), (7, 6, 2), (32, 8, 2), (33, 8, 2), (20, 5, 1), (64, 8, 2),
                                      (100, 4, 2), (128, 1, 1), (129, 2, 1), (200, 3, 1), (256, 2, 2), (23, 100, 1)])
def test_tree(T, Hq, Hkv, D):
    """No context, contexts around block and tile ends, one row tile, two, and several pairs of them."""
    _check(_make([0, 1, 15, 130, 256, 301], T, Hq, Hkv, D, seed=T * 7 + D))


@pytest.mark.parametrize("D,T,Hq,Hkv", [(128, 9, 8, 2), (64, 40, 16, 4)])
def test_many_sequences_of_mixed_lengths(D, T, Hq, Hkv):
    """Items that lie inside a CTA's run, and items cut between CTAs, in one call."""
    lens = [(37 * b * b + 11 * b) % 900 for b in range(40)]
    _check(_make(lens, T, Hq, Hkv, D, seed=3))


@pytest.mark.parametrize("D", [64, 128])
def test_one_long_context_is_split_over_every_sm(D):
    _check(_make([30011], 5, 4, 1, D, seed=4))
    _check(_make([20011], 70, 4, 1, D, seed=5))


def test_f32_output_scales_and_peaked_scores():
    s = _make([300, 0, 129], 12, 4, 2, 128, seed=6)
    _check(s, out_dtype=torch.float32)
    _check(s, scale=0.0)
    _check(s, scale=-0.05)
    # queries eight times as large: the running maximum moves by tens of log2 units between tiles
    _check(_make([700, 400], 12, 4, 2, 128, seed=7, gain=8.0))
    _check(_make([700, 400], 40, 8, 2, 64, seed=8, gain=8.0))


@pytest.mark.parametrize("T,Hq", [(20, 4), (70, 4)])
def test_scores_that_keep_rising_over_large_values(T, Hq):
    """Each 128 keys outscore the ones before by up to e^20, and the values are 1e32: no weight may be large enough to
    take a product past float32."""
    s = _make([900, 400], T, Hq, 1, 128, seed=21)
    g = _gen(22)
    for b, n in enumerate((900, 400)):
        at = torch.arange(n, device=DEV)
        blk = s["bt"][b, at // 16].long()
        up = 0.5 * (at // 128).to(torch.bfloat16) + torch.randn(n, generator=g).to(DEV).bfloat16() * 0.1
        s["kc"][blk, 0, at % 16, 0] = up
        s["vc"][blk, 0, at % 16] = (torch.randn(n, 128, generator=g) * 1e32).bfloat16().to(DEV)
    s["q"][..., 0] = 40.0  # a step of 0.5 in the first dim is 20 in the score, at scale 1
    s["v_new"] = s["v_new"] * 1e32
    s["q"][..., 1:] *= 0.05
    o, _ = _check(s, scale=1.0)
    assert bool(torch.isfinite(o).all())


@pytest.mark.parametrize("T", [128, 256])
def test_deep_chains_whole_and_cut(T):
    """Ancestors a hundred levels up; chains that break off at an absent draft, or at one that names itself, which take
    everything below with them; two chains interleaved."""
    s = _make([40, 7, 0, 300, 18], T, 1, 1, 64, seed=23)
    chain = list(range(-1, T - 1))
    par = [list(chain) for _ in range(5)]
    par[1][100] = -2
    par[2][60] = 60
    par[3] = [-1, -1, *range(T - 2)]
    par[4][T - 1], par[4][T // 2] = T - 3, -1
    s["parents"] = torch.tensor(par, dtype=torch.int32, device=DEV)
    _check(s, status=5)
    s["parents"][2, 60] = -1
    _check(s)


def test_a_chain_is_a_causal_chunk():
    """Parents -1, 0, 1, ...: the same cache and, within both calls' rounding, the same rows as paged_prefill_attn."""
    s = _make([77, 512], 50, 8, 2, 128, seed=9, cut=False)
    s["parents"] = torch.arange(-1, 49, dtype=torch.int32, device=DEV).expand(2, 50)
    o, l = _check(s)
    kc, vc = s["kc"].clone(), s["vc"].clone()
    po, pl = lib.paged_prefill_attn(s["q"], kc, vc, s["bt"], s["lens"], k_new=s["k_new"], v_new=s["v_new"],
                                    return_lse=True)
    ro, to, _, tl, ek, _ = _define(s, 1.0 / math.sqrt(128))
    assert torch.equal(_bits(kc), _bits(ek))
    assert bool(((o.double() - po.double()).abs() <= 2 * to + ro.abs() * 2.0 ** -7).all())
    assert bool(((l - pl).abs().double() <= 2 * tl).all())


@pytest.mark.parametrize("T,Hq", [(30, 8), (118, 2), (250, 4)])
def test_drafts_already_cached(T, Hq):
    s = _make([77, 512, 3], T, Hq, 2, 128, seed=10)
    o, l, kc, vc, _ = _run(s)
    s2 = dict(s, kc=kc, vc=vc)
    o2, l2, k2, v2, st = _run(s2, k_new=None, v_new=None)
    assert st == 0 and torch.equal(_bits(k2), _bits(kc)) and torch.equal(_bits(v2), _bits(vc))
    # the drafts' keys start inside a block, so the row's terms are added in another order: each result is within its
    # bound of the definition, the two within twice that of each other
    ro, to, _, tl, _, _ = _define(s, 1.0 / math.sqrt(128))
    there = ~torch.isneginf(l)
    assert torch.equal(torch.isneginf(l2), ~there)
    assert bool(((l2 - l).abs().double()[there] <= 2 * tl[there]).all())
    assert bool(((o2.double() - o.double()).abs() <= 2 * to + ro.abs() * 2.0 ** -7).all())
    o3, l3, _, _, _ = _run(s2, k_new=None, v_new=None)  # the same call again: bit for bit
    assert torch.equal(o3, o2) and torch.equal(l3, l2)


@pytest.mark.parametrize("D,T,Hq", [(128, 24, 4), (64, 150, 4)])
def test_infinities_and_nan_reach_only_those_who_attend(D, T, Hq):
    """A draft whose K or V is not finite changes its own row and its descendants' and no other."""
    s = _make([200, 31], T, Hq, 1, D, seed=11, cut=False)
    clean, lse = _check(s)
    see = [_seen(s["parents"][b].tolist()) for b in range(2)]
    for which, val in (("v_new", float("nan")), ("v_new", float("inf")), ("k_new", float("nan"))):
        bad = T // 2
        z = dict(s, **{which: s[which].clone()})
        z[which][:, :, bad, 5] = val
        o, l, _, _, st = _run(z)
        assert st == 0
        for b in range(2):
            hit = see[b][:, bad].to(DEV)
            assert bool(hit.any()) and not bool(hit.all())
            assert torch.equal(o[b][:, ~hit], clean[b][:, ~hit]) and torch.equal(l[b][:, ~hit], lse[b][:, ~hit])
            if which == "k_new":
                assert bool(torch.isnan(o[b][:, hit]).all()) and bool(torch.isnan(l[b][:, hit]).all())
            else:
                col = o[b][:, hit, 5]
                assert bool((torch.isnan(col) if math.isnan(val) else torch.isposinf(col)).all())
                keep = torch.arange(D, device=DEV) != 5
                assert torch.equal(o[b][:, hit][..., keep], clean[b][:, hit][..., keep])
                assert torch.equal(l[b], lse[b])


def test_idle_absent_and_refused_sequences():
    """Idle (-1), a tree that runs past the table, a parent that comes after its child, children of absent drafts."""
    s = _make([40, -1, 50, 60, 70], 6, 4, 2, 128, seed=12, cut=False)
    s["parents"][0] = torch.tensor([-1, -2, 1, 0, -1, -7], dtype=torch.int32)
    _check(s)
    s["parents"][3] = torch.tensor([-1, 0, 2, 1, 5, 4], dtype=torch.int32)  # 2 -> 2, 4 -> 5
    s["lens"][4] = s["bt"].shape[1] * 16 - 5  # one slot short
    o, l = _check(s, status=5)
    assert bool(torch.isneginf(l[4]).all()) and bool((o[4] == 0).all())


def test_bad_block_ids_are_reported_and_harm_no_other_sequence():
    s = _make([300, 300, 20], 6, 4, 2, 64, seed=13)
    o, l, kc, vc, _ = _run(s)
    z = dict(s, bt=s["bt"].clone())
    z["bt"][0, 3] = z["kc"].shape[0]
    z["bt"][0, 18] = -5
    o2, l2, k2, v2, st = _run(z)
    assert st == 5
    assert torch.equal(o2[1:], o[1:]) and torch.equal(l2[1:], l[1:])


def test_workspace_reuse_streams_and_graphs():
    """One workspace, filled with garbage, through calls of different shapes; two graphs captured over it and replayed
    in turn with other contents; a side stream.  Bit for bit the same rows every time."""
    a, b = _make([700, 90, 400], 11, 8, 2, 128, seed=14), _make([2000], 90, 4, 1, 128, seed=15)
    size = max(lib.paged_tree_workspace_size(x["q"].shape[0], x["q"].shape[1], x["kc"].shape[1], x["q"].shape[2],
                                             x["bt"].shape[1], 16, 128) for x in (a, b))
    ws = lib.Workspace(size)
    ws.tensor[256:].random_(0, 256)
    ref = [_run(x)[:2] for x in (a, b)]
    for x, r in ((a, ref[0]), (b, ref[1]), (a, ref[0])):
        o, l, _, _, st = _run(x, ws=ws)
        assert st == 0 and torch.equal(o, r[0]) and torch.equal(l, r[1])
    calls = []
    for x in (a, b):
        kc, vc, out = x["kc"].clone(), x["vc"].clone(), torch.zeros_like(x["q"])
        lse = torch.zeros(x["q"].shape[:3], device=DEV)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            lib.paged_tree_attn(x["q"], kc, vc, x["bt"], x["lens"], x["parents"], k_new=x["k_new"], v_new=x["v_new"],
                                out=out, lse=lse, workspace=ws)
        calls.append((g, out, lse, kc, vc))  # the graph keeps no tensor alive
    for i in (0, 1, 1, 0, 0):
        g, out, lse = calls[i][:3]
        out.zero_()
        g.replay()
        assert torch.equal(out, ref[i][0]) and torch.equal(lse, ref[i][1])
    a["lens"].sub_(torch.tensor([300, 0, 17], dtype=torch.int32, device=DEV))  # other lengths, other cuts
    want = _run(a)
    calls[0][0].replay()
    assert torch.equal(calls[0][1], want[0]) and torch.equal(calls[0][2], want[1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        o, l, _, _, _ = _run(a, ws=ws)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(o, want[0])


@pytest.mark.parametrize("D,Hkv", [(64, 3), (128, 1)])
def test_accept(D, Hkv):
    """Rows move bit for bit behind the context, across block ends; paths that need no move, none accepted, an idle
    sequence, and paths that are refused."""
    g = _gen(16)
    B, mb = 8, 12
    nb = B * mb
    kc, vc = (torch.randn(nb, Hkv, 16, D, generator=g).bfloat16().to(DEV) for _ in range(2))
    bt = torch.randperm(nb, generator=g).to(torch.int32).view(B, mb).to(DEV)
    ctx = [0, 14, 33, 60, -1, 100, 5, 180]
    long = list(range(3, 150, 1))
    paths = [[0, 1, 2], [1, 4, 7, 30], [], long[:100], [0, 2], [2, 2, 3], [3, 9, -1], [0, 11, 12]]
    n = [len(p) for p in paths]
    n[2] = -3
    path = torch.zeros(B, 120, dtype=torch.int32)
    for b, p in enumerate(paths):
        path[b, :len(p)] = torch.tensor(p, dtype=torch.int32)
    want = []
    for c in (kc, vc):
        e = c.clone()
        for b in (0, 1, 3):
            for i, j in enumerate(paths[b]):
                d, f = ctx[b] + i, ctx[b] + j
                e[bt[b, d // 16].long(), :, d % 16] = c[bt[b, f // 16].long(), :, f % 16]
        want.append(e)
    ws = lib.Workspace(256)
    args = (bt, torch.tensor(ctx, dtype=torch.int32, device=DEV), path.to(DEV), torch.tensor(n, dtype=torch.int32,
                                                                                             device=DEV))
    lib.kv_tree_accept(kc, vc, *args, workspace=ws)
    assert ws.status() == 5  # sequences 5, 6 and 7 (180 + 12 slots are past the table)
    assert torch.equal(kc, want[0]) and torch.equal(vc, want[1])
    ws.reset()
    lib.kv_tree_accept(kc, vc, bt[:5], args[1][:5], args[2][:5], args[3][:5], workspace=ws)
    assert ws.status() == 0
    n[0] = 121  # longer than the path's row
    k2 = kc.clone()
    lib.kv_tree_accept(k2, vc.clone(), bt[:1], args[1][:1], args[2][:1], torch.tensor(n[:1], dtype=torch.int32,
                                                                                     device=DEV), workspace=ws)
    assert ws.status() == 5 and torch.equal(k2, kc)


@pytest.mark.parametrize("before", ["nothing", "memset", "copy", "join"])
def test_accept_captured_after_anything(before):
    """The call may begin a graph, follow work that is no kernel, or wait for two streams: it sees what they wrote."""
    g = _gen(17)
    kc, vc = (torch.randn(12, 2, 16, 64, generator=g).bfloat16().to(DEV) for _ in range(2))
    bt = torch.randperm(12, generator=g).to(torch.int32).view(2, 6).to(DEV)
    ctx, path = torch.tensor([10, 30], dtype=torch.int32), torch.tensor([[0, 2, 5], [1, 4, 0]], dtype=torch.int32)
    n = torch.tensor([3, 2], dtype=torch.int32)
    want = [c.clone() for c in (kc, vc)]
    ws = lib.Workspace(256)
    dev = [x.to(DEV) for x in (ctx, path, n)]
    lib.kv_tree_accept(*want, bt, *dev, workspace=ws)
    spare = dev[0].clone()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    k2, v2 = kc.clone(), vc.clone()
    with torch.cuda.graph(graph):
        if before == "memset":
            dev[0].zero_()
        elif before in ("copy", "join"):
            dev[0].copy_(spare)
        if before == "join":
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                k2.copy_(kc)
            v2.copy_(vc)
            torch.cuda.current_stream().wait_stream(side)
        lib.kv_tree_accept(k2, v2, bt, *dev, workspace=ws)
    if before == "memset":
        ctx.zero_()
        want = [c.clone() for c in (kc, vc)]
        lib.kv_tree_accept(*want, bt, ctx.to(DEV), *dev[1:], workspace=ws)
    for _ in range(3):
        k2.copy_(kc)
        v2.copy_(vc)
        graph.replay()
        assert torch.equal(k2, want[0]) and torch.equal(v2, want[1])
        if before in ("copy", "join"):
            dev[0].random_(0, 20)
    assert ws.status() == 0
