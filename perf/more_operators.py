"""Cases and plain forms of the operators of a decode step over shared pages: which
drafted tokens the target model keeps, pages that are shared, copied, freed and
compacted, and a cache held in 8 bits with one scale per block of tokens and head.

``own`` False: every operator in elementary torch operations (float32; float64 for
sums over a vocabulary), as a program without this library would write it.  ``own``
True: the library's calls.
"""
import math
import random

import torch

own = False

BS = 16  # tokens per cache block
MOST_SCORES = 1 << 29  # query rows times keys of a case
MOST_TOKENS = 1 << 19  # cached tokens of a case
MOST_PROBS = 1 << 28   # probabilities of a case


# --------------------------------------------------------------------------
# the cases
# --------------------------------------------------------------------------
def listed():
    return [
        # one request with a chain of four drafts, a small vocabulary: what a call costs at least
        dict(name="verify_1x5", op="verify", B=1, T=5, V=32000, wide=0, mode="replacement", dtype="float32"),
        # a batch with trees drafted without replacement, some cut short, an odd vocabulary
        dict(name="verify_16x27", op="verify", B=16, T=27, V=100003, wide=4, mode="distinct", dtype="float32"),
        # the decode batch of the repository's benchmark, each request with a tree, a large vocabulary
        dict(name="verify_64x25", op="verify", B=64, T=25, V=131072, wide=3, mode="distinct", dtype="float32"),
        # four answers to one prompt that begin anew, one layer
        dict(name="fork_1to4", op="fork", P=1, C=4, ctx=701, ragged=0, layers=1, Hkv=8, D=128, spare=40, n_new=64),
        # a step of a search over 16 prompts with 64 rows, eight layers: rows are dropped and others doubled
        dict(name="fork_16to64", op="fork", P=16, C=64, ctx=8190, ragged=50, layers=8, Hkv=8, D=128, spare=400,
             n_new=16),
        # a small pool after a few requests have left, one layer
        dict(name="compact_1k", op="compact", B=16, blocks=1021, left=40, layers=1, Hkv=8, D=128),
        # a pool of several GB, half of it left, eight layers
        dict(name="compact_16k", op="compact", B=64, blocks=16384, left=50, layers=8, Hkv=8, D=128),
        # a decode batch's newest tokens
        dict(name="append_64x1", op="append", B=64, T=1, Hkv=8, D=128, ctx=4099, ragged=30, short=0),
        # prompts written in one pass, the chunks of some requests shorter
        dict(name="append_16x1024", op="append", B=16, T=1024, Hkv=8, D=128, ctx=37, ragged=80, short=40),
        # one request decoding alone, head dim 64
        dict(name="attn_1x1", op="attn", B=1, T=1, Hq=16, Hkv=8, D=64, ctx=700, ragged=0, short=0, causal=True),
        # the decode batch of the repository's benchmark
        dict(name="attn_64x1", op="attn", B=64, T=1, Hq=32, Hkv=8, D=128, ctx=8191, ragged=50, short=0, causal=True),
        # two long prompts, each with its next chunk, one of them shorter
        dict(name="attn_2x1024", op="attn", B=2, T=1024, Hq=32, Hkv=8, D=128, ctx=8192, ragged=20, short=30,
             causal=True),
    ]


def _log(rng, lo, hi):
    """An integer of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["verify", "verify", "fork", "compact", "append", "attn", "attn", "attn"])
    D = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    if op == "verify":
        B = _log(rng, 1, 64)
        T = _log(rng, 1, 64)
        V = _log(rng, 1000, min(262144, MOST_PROBS // (B * T)))
        return dict(op=op, B=B, T=T, V=V, wide=rng.randint(0, 5),
                    mode=rng.choice(["replacement", "distinct", "distinct", "sure"]),
                    dtype=rng.choice(["float32", "float32", "bfloat16"]))
    if op == "fork":
        P = _log(rng, 1, 32)
        return dict(op=op, P=P, C=_log(rng, 1, 64), ctx=_log(rng, 1, min(8192, 131072 // P)),
                    ragged=rng.choice([0, 30, 90]), layers=rng.randint(1, 8), Hkv=Hkv, D=D,
                    spare=rng.randint(64, 400), n_new=_log(rng, 1, 64))
    if op == "compact":
        B = _log(rng, 1, 64)
        return dict(op=op, B=B, blocks=_log(rng, 2 * B + 64, 16384), left=rng.choice([0, 20, 50, 90]),
                    layers=rng.randint(1, 8), Hkv=Hkv, D=D)
    if op == "append":
        B = _log(rng, 1, 64)
        return dict(op=op, B=B, T=_log(rng, 1, 16384 // B), Hkv=Hkv, D=D, ctx=rng.randint(0, 5000),
                    ragged=rng.choice([0, 30, 90]), short=rng.choice([0, 0, 40]))
    G = rng.choice([1, 2, 3, 4, 5, 7, 8])
    B = _log(rng, 1, 64)
    T = _log(rng, 1, max(1, min(4096, math.isqrt(MOST_SCORES // (B * Hkv * G)) // 2)))
    ctx = _log(rng, 1, max(1, min(131072, MOST_TOKENS // B, MOST_SCORES // (B * Hkv * G * T) - T)))
    return dict(op=op, B=B, T=T, Hq=Hkv * G, Hkv=Hkv, D=D, ctx=ctx, ragged=rng.choice([0, 30, 90]),
                short=rng.choice([0, 0, 40]), causal=rng.random() < 0.7)


def _lens(n, ctx, ragged):
    """Lengths of n sequences: ctx down to `ragged` percent less."""
    return [ctx - ctx * ragged * ((37 * b + 11) % n) // (100 * n) for b in range(n)]


def _new_lens(case):
    """New tokens of each sequence: all T, or `short` percent fewer for every third one."""
    return [case["T"] if b % 3 != 1 else max(1, case["T"] - case["T"] * case["short"] // 100)
            for b in range(case["B"])]


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _tree(case, seed):
    """Parents [B][T]: node 0 is the token chosen last, the others follow a node up to `wide` places before the
    latest; -2 past the end of trees that are cut short (every fifth)."""
    rng = random.Random(seed)
    T, parents = case["T"], []
    for b in range(case["B"]):
        n = T if b % 5 != 3 else max(1, T // 2)
        par = [-1]
        for t in range(1, n):
            par.append(rng.randint(max(0, t - 1 - case["wide"]), t - 1))
        parents.append(par + [-2] * (T - n))
    return parents


def _prepare_verify(case, seed, g):
    B, T, V = case["B"], case["T"], case["V"]
    dtype = getattr(torch, case["dtype"])
    parents = _tree(case, seed)
    s = dict(case, parents=_ints(parents))
    s["uniforms"] = torch.rand((B, T), generator=g, device="cuda")
    s["p"] = torch.empty((B, T, V), dtype=dtype, device="cuda")
    s["q"] = None if case["mode"] == "sure" else torch.empty((B, T, V), dtype=dtype, device="cuda")
    rank = [[par[:t].count(par[t]) for t in range(T)] for par in parents]  # place among the siblings
    most = 1 + max(r for b in range(B) for t, r in enumerate(rank[b]) if parents[b][t] >= -1)
    drawn = torch.empty((B, T, most), dtype=torch.int64, device="cuda")  # the tokens drawn at each node, in order
    for b in range(B):  # logits as of a model that is sure of some tokens; the draft model sees them blurred
        z = torch.randn((T, V), generator=g, device="cuda").mul_(4.0)
        d = torch.randn((T, V), generator=g, device="cuda").mul_(0.7).add_(z)
        s["p"][b] = torch.softmax(z, dim=-1)
        if s["q"] is not None:
            s["q"][b] = torch.softmax(d, dim=-1)
        if case["mode"] == "replacement":
            for i in range(most):
                drawn[b, :, i] = (d - torch.empty_like(d).exponential_(generator=g).log_()).argmax(dim=-1)
        else:
            if case["mode"] == "distinct":
                d = d - torch.empty_like(d).exponential_(generator=g).log_()
            drawn[b] = d.topk(most, dim=-1).indices
    par, r = s["parents"].long().clamp(min=0), torch.tensor(rank, device="cuda").clamp(max=most - 1)
    at = torch.arange(B, device="cuda")[:, None]
    s["tokens"] = drawn[at, par, r].to(torch.int32)
    return s


def _caches(layers, blocks, Hkv, D, g):
    return [torch.randn((blocks, Hkv, BS, D), generator=g, device="cuda", dtype=torch.bfloat16)
            for _ in range(2 * layers)]


def _prepare_fork(case, seed, g):
    """P prompts in a pool of shuffled blocks; C rows that continue one of them each."""
    P, C = case["P"], case["C"]
    lens = _lens(P, case["ctx"], case["ragged"])
    need = [(n + BS - 1) // BS for n in lens]
    width = max(need) + (case["n_new"] + BS - 1) // BS + 1
    blocks = sum(need) + C * (2 + (case["n_new"] + BS - 1) // BS) + case["spare"]
    order = torch.randperm(blocks, generator=g, device="cuda").to(torch.int32)
    s = dict(case, lens=_ints(lens), refs=torch.zeros(blocks, dtype=torch.int32, device="cuda"))
    s["bt"] = torch.full((P, width), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        s["bt"][b, :n] = order[at:at + n]
        at += n
    s["refs"][order[:at].long()] = 1
    s["src"] = torch.randint(0, P, (C,), generator=g, device="cuda", dtype=torch.int32)
    s["child_bt"] = torch.full((C, width), -1, dtype=torch.int32, device="cuda")
    s["child_lens"] = torch.full((C,), -1, dtype=torch.int32, device="cuda")
    s["n_new"] = torch.full((C,), case["n_new"], dtype=torch.int32, device="cuda")
    s["caches"] = _caches(case["layers"], blocks, case["Hkv"], case["D"], g)
    return s


def _prepare_compact(case, seed, g):
    """A pool that was full of B sequences, of whose blocks `left` percent have been given back; some blocks are
    shared by two sequences."""
    B, N = case["B"], case["blocks"]
    width = N // B
    order = torch.randperm(N, generator=g, device="cuda").to(torch.int32)
    bt = order[:B * width].reshape(B, width).clone()
    bt[torch.rand((B, width), generator=g, device="cuda") < case["left"] / 100.0] = -1
    if B > 1:  # a prompt's first blocks that two sequences have in common
        n = max(1, width // 8)
        bt[1, :n] = bt[0, :n]
    refs = torch.zeros(N + 1, dtype=torch.int32, device="cuda")
    refs.index_add_(0, bt.reshape(-1).long().remainder(N + 1), torch.ones(bt.numel(), dtype=torch.int32,
                                                                          device="cuda"))
    s = dict(case, bt0=bt, refs0=refs[:N].clone())
    s["bt"], s["refs"] = bt.clone(), s["refs0"].clone()
    s["caches"] = _caches(case["layers"], N, case["Hkv"], case["D"], g)
    return s


def _f8_pool(blocks, Hkv, D, g):
    """Codes and scales of a cache that is full of standard normal rows (three of four blocks have the scale that a
    block of 16 rows of 128 such numbers gets, some a larger one)."""
    x = torch.randn((blocks, Hkv, BS, D), generator=g, device="cuda", dtype=torch.bfloat16)
    e = -6 + (torch.rand((blocks, Hkv), generator=g, device="cuda") < 0.25).float()
    scale = torch.exp2(e)
    return (x.float() / scale[:, :, None, None]).clamp_(-448.0, 448.0).to(torch.float8_e4m3fn), scale


def _table(B, each, g):
    n = B * each
    perm = torch.randperm(n + 3, generator=g, device="cuda")[:n]
    return perm.to(torch.int32).reshape(B, each).contiguous(), n + 3


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    if op == "verify":
        return _prepare_verify(case, seed, g)
    if op == "fork":
        return _prepare_fork(case, seed, g)
    if op == "compact":
        return _prepare_compact(case, seed, g)
    B, T, Hkv, D = case["B"], case["T"], case["Hkv"], case["D"]
    s = dict(case)
    lens, new = _lens(B, case["ctx"], case["ragged"]), _new_lens(case)
    s["max_len"] = max(lens) + T
    s["start"], s["n"] = _ints(lens), _ints(new) if case["short"] else None
    s["bt"], blocks = _table(B, (s["max_len"] + BS - 1) // BS, g)
    s["kq"], s["ks"] = _f8_pool(blocks, Hkv, D, g)
    s["vq"], s["vs"] = _f8_pool(blocks, Hkv, D, g)
    if op == "append":  # a projection's output: k and v side by side in one row a token
        kv = torch.randn((B, T, 2 * Hkv, D), generator=g, device="cuda").to(torch.bfloat16)
        s["k_new"], s["v_new"] = (x.transpose(1, 2) for x in kv.split([Hkv, Hkv], dim=2))
    else:
        s["q"] = torch.randn((B, T, case["Hq"], D), generator=g, device="cuda").to(torch.bfloat16).transpose(1, 2)
        s["scale"] = 1.0 / math.sqrt(D)
    return s


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def run(s):
    op = s["op"]
    if op == "compact":  # the pool as the pass finds it (blocks that move leave their bytes where they were)
        s["bt"].copy_(s["bt0"])
        s["refs"].copy_(s["refs0"])
    if own:
        return _run_own(s)
    return {"verify": _plain_verify, "fork": _plain_fork, "compact": _plain_compact, "append": _plain_append,
            "attn": _plain_attn}[op](s)


def _run_own(s):
    import masked_attention_paged_gb300 as lib
    op = s["op"]
    if "ws" not in s:  # a serving program keeps one workspace for its shapes
        nbytes = 256
        if op == "verify":
            nbytes = lib.draft_verify_workspace_size(s["B"], s["T"], s["V"])
        elif op in ("fork", "compact"):
            nbytes = lib.kv_pool_workspace_size(s["refs"].shape[0], s["C"] if op == "fork" else s["B"])
        elif op == "attn":
            nbytes = lib.paged_attn_f8_workspace_size(s["B"], s["Hq"], s["Hkv"], s["T"], s["bt"].shape[1], BS, s["D"])
        s["ws"] = lib.Workspace(nbytes)
    ws = s["ws"]
    if op == "verify":
        return lib.draft_verify(s["p"], s["tokens"], s["parents"], s["uniforms"], draft_probs=s["q"],
                                replacement=s["mode"] == "replacement", workspace=ws)
    if op == "fork":
        lib.kv_free(s["refs"], s["child_bt"], s["child_lens"], workspace=ws)
        lib.kv_fork(s["caches"], s["refs"], s["bt"], s["lens"], s["src"], s["child_bt"], s["child_lens"],
                    workspace=ws)
        lib.kv_reserve(s["refs"], s["child_bt"], s["child_lens"], s["n_new"], workspace=ws)
        return [s["refs"], s["child_bt"], s["child_lens"]] + s["caches"]
    if op == "compact":
        used = lib.kv_compact(s["caches"], s["refs"], s["bt"], workspace=ws)
        return [used, s["refs"], s["bt"]] + s["caches"]
    if op == "append":
        lib.kv_append_f8(s["kq"], s["vq"], s["ks"], s["vs"], s["bt"], s["start"], s["k_new"], s["v_new"],
                         lens=s["n"], workspace=ws)
        return [s["kq"], s["vq"], s["ks"], s["vs"]]
    return lib.paged_attn_f8(s["q"], s["kq"], s["vq"], s["ks"], s["vs"], s["bt"], s["start"], lens=s["n"],
                             causal=s["causal"], scale=s["scale"], return_lse=True, workspace=ws)


# --------------------------------------------------------------------------
# plain forms
# --------------------------------------------------------------------------
def _plain_verify(s):
    """Drafts in index order: a draft is tested when its parent is the node where its sequence stands.  The
    residual after some rejections is max(p - c q, 0), c a sum of scalars.  Float64 throughout: tests and sums decide
    between whole numbers."""
    p, q, u = s["p"], s["q"], s["uniforms"].double()
    B, T, V = p.shape
    parents, tokens = s["parents"].long(), s["tokens"].long()
    rows = torch.arange(B, device="cuda")
    there = parents[:, 0] == -1
    cur = torch.zeros(B, dtype=torch.int64, device="cuda")
    took = torch.zeros((B, T), dtype=torch.bool, device="cuda")
    took[:, 0] = there
    refused = torch.zeros((B, T), dtype=torch.bool, device="cuda")  # at the node where the sequence stands
    one = torch.ones(B, dtype=torch.float64, device="cuda")
    c, mass, left = 0.0 * one, one.clone(), one.clone()

    def residual(c, refused):
        r = p[rows, cur].double()
        if q is not None:
            return (r - c[:, None] * q[rows, cur].double()).clamp_(min=0.0)
        gone = torch.zeros((B, V), dtype=torch.int32, device="cuda").scatter_add_(1, tokens.clamp(0, V - 1),
                                                                                  refused.int())
        return r.masked_fill_(gone > 0, 0.0)

    for t in range(1, T):
        x = tokens[:, t]
        asked = there & (parents[:, t] == cur) & (x >= 0) & (x < V)
        x = x.clamp(0, V - 1)
        px = p[rows, cur, x].double()
        if s["mode"] != "replacement":
            asked &= ~(refused & (tokens == x[:, None])).any(dim=1)
        if q is None:
            yes = u[:, t] * mass < px
            no = asked & ~yes
            mass = torch.where(no, mass - px, mass)
            refused[:, t] = no
        else:
            qx = q[rows, cur, x].double()
            asked &= left > 0
            yes = u[:, t] * qx * mass < (px - c * qx).clamp(min=0.0) * left
            no = asked & ~yes
            c = torch.where(no, c + mass / left, c)
            if s["mode"] != "replacement":
                left = torch.where(no, left - qx, left)
                refused[:, t] = no
            mass = torch.where(no, residual(c, refused).sum(dim=1), mass)
        yes &= asked
        took[:, t] = yes
        cur = torch.where(yes, t, cur)
        refused &= ~yes[:, None]
        c, mass, left = torch.where(yes, 0.0, c), torch.where(yes, 1.0, mass), torch.where(yes, 1.0, left)
    r = residual(c, refused)
    r = torch.where((r.sum(dim=1) > 0)[:, None], r, p[rows, cur].double())
    sums = r.cumsum(dim=1)
    past = sums > (u[:, :1] * sums[:, -1:])
    last = V - 1 - (r > 0).flip(1).int().argmax(dim=1)
    token = torch.where(past.any(dim=1), past.int().argmax(dim=1), last)
    n = took.sum(dim=1)
    at = torch.where(took, took.cumsum(dim=1) - 1, T)
    path = torch.full((B, T + 1), -1, dtype=torch.int32, device="cuda")
    path.scatter_(1, at, torch.arange(T, dtype=torch.int32, device="cuda").expand(B, T))
    return path[:, :T].contiguous(), n.int(), torch.where(there, token, -1).int()


def _free_blocks(refs, n):
    """The n lowest blocks that nobody has."""
    return (refs == 0).nonzero()[:n, 0].to(torch.int32)


def _plain_fork(s):
    refs, bt, lens, src = s["refs"], s["bt"], s["lens"], s["src"].long()
    ct, cl = s["child_bt"], s["child_lens"]
    one = torch.ones(ct.numel(), dtype=torch.int32, device="cuda")
    # the rows of the step before give their blocks back
    have = ct.reshape(-1) >= 0
    refs.index_add_(0, ct.reshape(-1)[have].long(), -one[:int(have.sum())])
    ct.fill_(-1)
    cl.fill_(-1)
    # full blocks are shared, a partial one is copied
    n = lens[src]
    col = torch.arange(bt.shape[1], device="cuda")
    shared = torch.where(col < (n // BS)[:, None], bt[src], -1)
    ct.copy_(shared)
    cl.copy_(n)
    part = (n % BS != 0).nonzero()[:, 0]
    new = _free_blocks(refs, part.numel())
    at = (n // BS)[part].long()
    old = bt[src[part], at].long()
    ct[part, at] = new
    have = shared.reshape(-1) >= 0
    refs.index_add_(0, shared.reshape(-1)[have].long(), one[:int(have.sum())])
    refs[new.long()] = 1
    for c in s["caches"]:
        c[new.long()] = c[old]
    # blocks for the next tokens
    first, end = (n + BS - 1) // BS, (n + s["n_new"] + BS - 1) // BS
    want = (col >= first[:, None]) & (col < end[:, None])
    new = _free_blocks(refs, int(want.sum()))
    ct[want] = new
    refs[new.long()] = 1
    return [refs, ct, cl] + s["caches"]


def _plain_compact(s):
    refs, bt = s["refs"], s["bt"]
    used = refs != 0
    n = used.sum()
    at = torch.arange(refs.shape[0], device="cuda")
    move, hole = (used & (at >= n)).nonzero()[:, 0], (~used & (at < n)).nonzero()[:, 0]
    to = at.clone()
    to[move] = hole
    for c in s["caches"]:
        c[hole] = c[move]
    refs[hole] = refs[move]
    refs[move] = 0
    bt.copy_(torch.where(bt >= 0, to[bt.clamp(min=0).long()].to(torch.int32), bt))
    return [n.to(torch.int32).reshape(1), refs, bt] + s["caches"]


def _window(s, T):
    """The blocks that each sequence's new tokens may touch: ids [B, n], their tokens' positions [B, n * 16], and
    which of those are new, and which older."""
    start = s["start"].long()
    n = s["n"].long() if s["n"] is not None else torch.full_like(start, T)
    blk = start[:, None] // BS + torch.arange((T + BS - 1) // BS + 1, device="cuda")
    ids = torch.gather(s["bt"], 1, blk.clamp(max=s["bt"].shape[1] - 1)).long()
    pos = (blk[:, :, None] * BS + torch.arange(BS, device="cuda")).flatten(1)
    new = (pos >= start[:, None]) & (pos < (start + n)[:, None])
    return ids, pos, new, pos < start[:, None]


def _plain_append(s):
    T = s["T"]
    ids, pos, new, old = _window(s, T)
    B, nb = ids.shape
    for x, code, scale in ((s["k_new"], s["kq"], s["ks"]), (s["v_new"], s["vq"], s["vs"])):
        Hkv, D = x.shape[1], x.shape[3]
        i = (pos - s["start"].long()[:, None]).clamp(0, T - 1)
        rows = torch.gather(x.transpose(1, 2), 1, i[:, :, None, None].expand(B, nb * BS, Hkv, D)).float()
        rows = rows.reshape(B, nb, BS, Hkv, D).transpose(2, 3)  # [B, nb, Hkv, 16, D]
        is_new, is_old = (m.reshape(B, nb, 1, BS, 1) for m in (new, old))
        a = rows.abs().masked_fill_(~is_new, 0.0).amax(dim=(3, 4))
        m, e = torch.frexp(a)  # a = 2 m 2^(e - 1)
        need = torch.where(a > 0, torch.ldexp(torch.ones_like(a), (e - 9 + (m > 0.875).int()).clamp(min=-126)), 0.0)
        before = torch.where(is_old[:, :, :, 0, 0], scale[ids], 0.0)
        sc = torch.maximum(before, need)
        div = torch.where(sc > 0, sc, 1.0)
        fresh = (rows / div[..., None, None]).clamp_(-448.0, 448.0).to(torch.float8_e4m3fn)
        was = code.view(torch.uint8)[ids].view(torch.float8_e4m3fn)
        kept = (was.float() * (before / div)[..., None, None]).clamp_(-448.0, 448.0).to(torch.float8_e4m3fn)
        got = torch.where(is_new, fresh.view(torch.uint8),
                          torch.where(is_old, kept.view(torch.uint8), was.view(torch.uint8)))
        touched = is_new.any(dim=3)[:, :, 0, 0]
        code.view(torch.uint8)[ids[touched]] = got[touched]
        scale[ids[touched]] = sc[touched]
    return [s["kq"], s["vq"], s["ks"], s["vs"]]


def _plain_attn(s):
    q = s["q"]
    B, Hq, T, D = q.shape
    Hkv = s["Hkv"]
    starts, lens = s["start"].tolist(), s["n"].tolist() if s["n"] is not None else [T] * B
    out = torch.zeros((B, Hq, T, D), dtype=q.dtype, device="cuda")
    lse = torch.full((B, Hq, T), -math.inf, device="cuda")
    for b in range(B):
        t, end = lens[b], starts[b] + lens[b]
        ids = s["bt"][b, :(end + BS - 1) // BS].long()
        k = (s["kq"].view(torch.uint8)[ids].view(torch.float8_e4m3fn).float() * s["ks"][ids][:, :, None, None])
        v = (s["vq"].view(torch.uint8)[ids].view(torch.float8_e4m3fn).float() * s["vs"][ids][:, :, None, None])
        k, v = (x.transpose(0, 1).reshape(Hkv, -1, D)[:, :end] for x in (k, v))
        x = (q[b, :, :t].float().reshape(Hkv, -1, D) @ k.transpose(1, 2)).mul_(s["scale"]).view(Hkv, -1, t, end)
        if s["causal"]:
            see = torch.arange(end, device="cuda") <= starts[b] + torch.arange(t, device="cuda")[:, None]
            x.masked_fill_(~see, -math.inf)
        top = x.amax(dim=-1, keepdim=True)
        w = x.sub_(top).exp_()
        total = w.sum(dim=-1, keepdim=True)
        o = (w.view(Hkv, -1, end) @ v).view(Hkv, -1, t, D) / total
        out[b, :, :t] = o.reshape(Hq, t, D).to(q.dtype)
        lse[b, :, :t] = (top + total.log()).reshape(Hq, t)
    return out, lse


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------
def work(case):
    op = case["op"]
    if op == "verify":
        # the rows of the node where a sequence stops, and the drafts' own probabilities
        size = 2 if case["dtype"] == "bfloat16" else 4
        rows = 1 if case["mode"] == "sure" else 2
        B, T, V = case["B"], case["T"], case["V"]
        return {"bytes": B * (V * rows * size + T * (rows * size + 16) + 8), "flops": 4 * B * V}
    if op == "fork":
        row = 2 * case["layers"] * case["Hkv"] * BS * case["D"] * 2  # bytes of a block in all layers
        part = sum(n % BS != 0 for n in _lens(case["P"], case["ctx"], case["ragged"])) / case["P"]
        table = (case["ctx"] + case["n_new"]) // BS + 1
        return {"bytes": case["C"] * (2 * part * row + 3 * 4 * table), "flops": 0}
    if op == "compact":
        row = 2 * case["layers"] * case["Hkv"] * BS * case["D"] * 2
        held = 1.0 - case["left"] / 100.0
        return {"bytes": 2 * case["blocks"] * held * (1.0 - held) * row + 16 * case["blocks"], "flops": 0}
    B, T, Hkv, D = case["B"], case["T"], case["Hkv"], case["D"]
    new = _new_lens(case) if case["short"] else [T] * B
    if op == "append":
        return {"bytes": sum(new) * Hkv * D * 2 * (2 + 1) + B * (T // BS + 1) * Hkv * 2 * 8, "flops": 0}
    lens = _lens(B, case["ctx"], case["ragged"])
    keys = sum(n + t for n, t in zip(lens, new))
    seen = sum(t * n + (t * (t + 1) // 2 if case["causal"] else t * t) for n, t in zip(lens, new))
    return {"bytes": keys * Hkv * (2 * D + 8 / BS) + sum(new) * case["Hq"] * (4 * D + 4),
            "flops": 4 * seen * case["Hq"] * D}


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return {"verify": _exact_verify, "fork": _exact_fork, "compact": _exact_compact, "append": _exact_append,
            "attn": _exact_attn}[case["op"]](s)


def _exact_verify(s):
    """One sequence after the other, the residual rows written out at every rejection."""
    B, T, V = s["p"].shape
    parents, tokens, u = s["parents"].tolist(), s["tokens"].tolist(), s["uniforms"].double().tolist()
    path, count, token = [], [], []
    for b in range(B):
        node, way = 0, [0]
        while True:
            p = s["p"][b, node].double()
            r, q = p / 1.0, None if s["q"] is None else s["q"][b, node].double()
            mass, taken, gone = 1.0, -1, set()
            for t in range(node + 1, T):
                x = tokens[b][t]
                if parents[b][t] != node or (x in gone and s["mode"] != "replacement"):
                    continue
                if q is None:  # the draft is sure of its token: its row is 1 there
                    if u[b][t] < float(r[x]) / mass:
                        taken = t
                        break
                    mass -= float(r[x])
                    r[x] = 0.0
                else:
                    if u[b][t] * float(q[x]) < float(r[x]) / mass:
                        taken = t
                        break
                    r = (r / mass - q).clamp(min=0.0)
                    mass = float(r.sum())
                    if mass == 0.0:
                        break
                    if s["mode"] != "replacement":
                        q = q.clone()
                        rest = 1.0 - float(q[x])
                        if rest <= 0.0:
                            break
                        q[x] = 0.0
                        q = q / rest
                gone.add(x)
            if taken < 0:
                break
            node = taken
            way.append(node)
        if float(r.sum()) <= 0.0:
            r = p
        sums = r.cumsum(dim=0)
        token.append(int((sums <= u[b][0] * sums[-1]).sum().clamp(max=V - 1)))
        path.append(way + [-1] * (T - len(way)))
        count.append(len(way))
    return _ints(path), _ints(count), _ints(token)


def _exact_fork(s):
    """The pool's books kept in Python."""
    refs, bt, lens, src = s["refs"].tolist(), s["bt"].tolist(), s["lens"].tolist(), s["src"].tolist()
    width, copies, table, size = len(bt[0]), [], [], []
    free = [i for i, n in enumerate(refs) if n == 0]
    for j in src:
        n = lens[j]
        row = bt[j][:n // BS]
        for i in row:
            refs[i] += 1
        if n % BS:
            new = free.pop(0)
            refs[new] = 1
            copies.append((bt[j][n // BS], new))
            row = row + [new]
        table.append(row)
        size.append(n)
    for row, n in zip(table, size):
        for _ in range((n + s["n_new"][0].item() + BS - 1) // BS - len(row)):
            new = free.pop(0)
            refs[new] = 1
            row.append(new)
    for old, new in copies:
        for c in s["caches"]:
            c[new] = c[old]
    return [_ints(refs), _ints([r + [-1] * (width - len(r)) for r in table]), _ints(size)] + s["caches"]


def _exact_compact(s):
    refs, bt = s["refs0"].tolist(), s["bt0"].tolist()
    used = [i for i, n in enumerate(refs) if n]
    n = len(used)
    moved = dict(zip([i for i in used if i >= n], [i for i in range(n) if refs[i] == 0]))
    old, new = torch.tensor(list(moved), device="cuda"), torch.tensor(list(moved.values()), device="cuda")
    if moved:
        for c in s["caches"]:
            c[new] = c[old]
    for a, b in moved.items():
        refs[b], refs[a] = refs[a], 0
    return [_ints([n]), _ints(refs), _ints([[moved.get(i, i) for i in row] for row in bt])] + s["caches"]


def _e4m3(x):
    """The nearest numbers of 3 bits after the point and exponents from -6, ties to even, at most 448."""
    m, e = torch.frexp(x)
    step = torch.exp2((e - 1).clamp(min=-6).double() - 3.0)
    return ((x / step).round() * step).clamp(-448.0, 448.0)


def _exact_append(s):
    T, starts = s["T"], s["start"].tolist()
    lens, bt = s["n"].tolist() if s["n"] is not None else [T] * len(starts), s["bt"].tolist()
    out = []
    for x, code, scale in ((s["k_new"], s["kq"], s["ks"]), (s["v_new"], s["vq"], s["vs"])):
        value, scale = code.float(), scale.clone()
        for b, first in enumerate(starts):
            for blk in range(first // BS, (first + lens[b] - 1) // BS + 1):
                lo, hi = max(first, blk * BS), min(first + lens[b], (blk + 1) * BS)
                rows = x[b, :, lo - first:hi - first].double()
                i, a, had = bt[b][blk], rows.abs().amax(dim=(1, 2)), lo - blk * BS
                need = torch.where(a > 0, torch.exp2(torch.ceil(torch.log2(a / 448.0)).clamp(min=-126)), 0.0)
                before = scale[i].double() if had else torch.zeros_like(need)
                sc = torch.maximum(before, need)
                by = torch.where(sc > 0, sc, 1.0)[:, None, None]
                value[i, :, :had] = _e4m3(value[i, :, :had].double() * before[:, None, None] / by).float()
                value[i, :, had:had + hi - lo] = _e4m3(rows / by).float()
                scale[i] = sc.float()
        out.append((value, scale))
    return [out[0][0], out[1][0], out[0][1], out[1][1]]


def _exact_attn(s):
    q = s["q"].double()
    B, Hq, T, D = q.shape
    G = Hq // s["Hkv"]
    out = torch.zeros((B, Hq, T, D), dtype=torch.float64, device="cuda")
    lse = torch.full((B, Hq, T), -math.inf, dtype=torch.float64, device="cuda")
    for b in range(B):
        first = int(s["start"][b])
        t = int(s["n"][b]) if s["n"] is not None else T
        at = torch.arange(first + t, device="cuda")
        blk, slot = s["bt"][b, at // BS].long(), at % BS
        row = torch.arange(t, device="cuda")[:, None]
        hide = at > (first + row if s["causal"] else first + t + 0 * row)
        for g in range(s["Hkv"]):
            k, v = (c.view(torch.uint8)[blk, g, slot].view(torch.float8_e4m3fn).double() * sc[blk, g, None].double()
                    for c, sc in ((s["kq"], s["ks"]), (s["vq"], s["vs"])))
            for h in range(g * G, (g + 1) * G):
                x = (q[b, h, :t] @ k.t() * s["scale"]).masked_fill(hide, -math.inf)
                lse[b, h, :t] = torch.logsumexp(x, dim=1)
                out[b, h, :t] = torch.exp(x - lse[b, h, :t, None]) @ v
    return out, lse
