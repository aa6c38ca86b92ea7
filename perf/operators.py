"""Cases and plain forms of the operators that surround the paged KV cache in a
serving step: rotary positions joined with the append, attention of a tree of
drafted tokens over the cache, and eviction by accumulated attention weight.

``own`` False: every operator in elementary torch operations (float32, angles
in float64), as a program without this library would write it.  ``own`` True:
the library's calls.
"""
import math

import torch

own = False

BS = 16  # tokens per cache block
MOST_SCORES = 1 << 29  # query rows times keys of the largest cases


# --------------------------------------------------------------------------
# the cases
# --------------------------------------------------------------------------
def listed():
    return [
        # one request decoding alone: one new token, what a call costs at least
        dict(name="rope_append_1x1", op="rope_append", B=1, T=1, Hq=32, Hkv=8, D=128, rot=128, inter=False,
             ctx=700, far=700),
        # a decode batch far into a long context, positions past what 32-bit angles hold, half of the head
        # rotated, neighbouring pairs
        dict(name="rope_append_64x1", op="rope_append", B=64, T=1, Hq=32, Hkv=8, D=128, rot=64, inter=True,
             ctx=8176, far=900000),
        # prompts prefilled in one pass: 16 of 1024 tokens
        dict(name="rope_append_16x1024", op="rope_append", B=16, T=1024, Hq=32, Hkv=8, D=128, rot=128,
             inter=False, ctx=0, far=0),
        # the gradient of the rotation, float32 (the transposed rotation), an odd number of tokens
        dict(name="rope_apply_f32_back", op="rope_apply", B=3, T=1031, Hq=16, D=64, rot=48, inter=True, inverse=True,
             dtype="float32", far=5000),
        # one request, a small tree of drafts, short context, head dim 64
        dict(name="tree_1x8", op="tree", B=1, T=8, Hq=16, Hkv=8, D=64, ctx=700, ragged=0, wide=3, accept=3),
        # a batch with trees of 27 drafts, some of them cut short, contexts of mixed lengths
        dict(name="tree_16x27", op="tree", B=16, T=27, Hq=32, Hkv=8, D=128, ctx=4096, ragged=70, wide=4, accept=5),
        # one request over a very long context, 64 drafts: the work has to be split over the context
        dict(name="tree_1x64_long", op="tree", B=1, T=64, Hq=64, Hkv=8, D=128, ctx=131063, ragged=0, wide=4,
             accept=9),
        # the decode batch of the repository's benchmark, each request with a tree of drafts
        dict(name="tree_64x25", op="tree", B=64, T=25, Hq=32, Hkv=8, D=128, ctx=8192, ragged=50, wide=3, accept=4),
        # weights of one decode step, added up after the attention of the same batch
        dict(name="weights_64x1", op="weights", B=64, T=1, Hq=32, Hkv=8, D=128, ctx=8192, ragged=50),
        # weights of a whole prompt, before its cache is cut to a budget
        dict(name="weights_1x4096", op="weights", B=1, T=4096, Hq=32, Hkv=8, D=128, ctx=0, ragged=0),
        # a decode batch that has grown a little past its budget
        dict(name="evict_64x4160", op="evict", B=64, Hkv=8, D=128, ctx=4160, ragged=3, keep=4096, sink=4,
             recent=64),
        # two long prompts cut to a small budget, head dim 64
        dict(name="evict_2x65521", op="evict", B=2, Hkv=8, D=64, ctx=65521, ragged=10, keep=2048, sink=4,
             recent=128),
    ]


def _log(rng, lo, hi):
    """An integer of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["rope_append", "rope_append", "rope_apply", "tree", "tree", "tree", "weights", "weights",
                     "evict"])
    D = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    if op in ("rope_append", "rope_apply"):
        B = _log(rng, 1, 64)
        T = _log(rng, 1, max(1, 16384 // B // 4))
        Hq = Hkv * rng.choice([1, 2, 3, 4])
        rot = rng.choice([D, D // 2, D // 4, 2 * rng.randint(1, D // 2)])
        case = dict(op=op, B=B, T=T, Hq=Hq, D=D, rot=rot, inter=rng.random() < 0.5,
                    far=rng.choice([0, _log(rng, 1000, 1000000)]))
        if op == "rope_apply":
            case.update(inverse=rng.random() < 0.5, dtype=rng.choice(["float32", "bfloat16"]))
        else:
            case.update(Hkv=Hkv, ctx=rng.randint(0, 5000))
        return case
    if op == "tree":
        G = rng.choice([1, 2, 3, 4, 5, 8])
        B = _log(rng, 1, 64)
        ctx = _log(rng, 1, min(65536, 262144 // B))
        T = _log(rng, 1, max(1, min(200, 4096 // (B * G), MOST_SCORES // (B * Hkv * G * ctx))))
        return dict(op=op, B=B, T=T, Hq=Hkv * G, Hkv=Hkv, D=D, ctx=ctx, ragged=rng.choice([0, 30, 90]),
                    wide=rng.randint(1, 5), accept=rng.randint(0, min(T, 12)))
    if op == "weights":
        G = rng.choice([1, 2, 4, 7, 8])
        B = _log(rng, 1, 64)
        T = _log(rng, 1, math.isqrt(MOST_SCORES // (B * Hkv * G)) // 2)
        ctx = _log(rng, 1, max(1, min(32768, 262144 // B, MOST_SCORES // (B * Hkv * G * T) - T)))
        return dict(op=op, B=B, T=T, Hq=Hkv * G, Hkv=Hkv, D=D, ctx=ctx, ragged=rng.choice([0, 30, 90]))
    B = _log(rng, 1, 64)
    ctx = _log(rng, 16, min(65536, 262144 // B))
    keep = _log(rng, 8, min(ctx, 4096))
    return dict(op=op, B=B, Hkv=Hkv, D=D, ctx=ctx, ragged=rng.choice([0, 10, 60]), keep=keep,
                sink=rng.randint(0, min(4, keep // 2)), recent=rng.randint(0, keep // 2))


def _lens(case):
    """Context lengths of the batch: case["ctx"] down to `ragged` percent less."""
    B, ctx, r = case["B"], case["ctx"], case.get("ragged", 0)
    return [ctx - ctx * r * ((37 * b + 11) % B) // (100 * B) for b in range(B)]


def _drafts(case):
    """Drafted tokens of each sequence: all T, every fifth sequence cut short."""
    return [case["T"] if b % 5 != 3 else max(1, case["T"] // 2) for b in range(case["B"])]


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _table(B, blocks_each, g):
    """A block table over a shuffled pool with a few blocks to spare."""
    n = B * blocks_each
    perm = torch.randperm(n + 3, generator=g, device="cuda")[:n]
    return perm.to(torch.int32).reshape(B, blocks_each).contiguous(), n + 3


def _rand(shape, g, dtype=torch.bfloat16):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _pool(blocks, Hkv, D, g):
    # bfloat16 draws directly: caches of a GB would cost two in float32
    return torch.randn((blocks, Hkv, BS, D), generator=g, device="cuda", dtype=torch.bfloat16)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _frequencies(rot):
    """Angles a token: base 10000 over rot dimensions, positions interpolated by 4 (a context four times
    as long), in radians and as 64-bit fractions of a turn."""
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot) / 4.0
    turns = (inv / (2.0 * math.pi) * 2.0 ** 64).to(torch.int64)
    return inv.cuda(), turns.cuda()


def _tree(case, seed):
    """Parents [B, T] of each sequence's drafted tokens (-1: follows the context, -2: no token), and a path of
    `accept` nodes that starts at a root."""
    import random
    rng = random.Random(seed)
    T, parents, paths, taken = case["T"], [], [], []
    for n in _drafts(case):
        par = [-1]
        for t in range(1, n):
            par.append(rng.randint(max(-1, t - 1 - case["wide"]), t - 1))
        node, path = rng.randrange(n), []
        while node >= 0:
            path.append(node)
            node = par[node]
        path = path[::-1][:case["accept"]]
        parents.append(par + [-2] * (T - n))
        taken.append(len(path))
        paths.append(path + [0] * (T - len(path)))
    return _ints(parents), _ints(paths), _ints(taken)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, B, D = case["op"], case["B"], case["D"]
    s = dict(case, B=B)
    if op in ("rope_append", "rope_apply"):
        T, Hq = case["T"], case["Hq"]
        s["inv_freq"], s["freqs"] = _frequencies(case["rot"])
        s["first"] = torch.randint(0, case["far"] + 1, (B, 1), generator=g, device="cuda")
        s["positions"] = (s["first"] + torch.arange(T, device="cuda")).to(torch.int32)
        if op == "rope_apply":
            s["x"] = _rand((B, T, Hq, D), g, getattr(torch, case["dtype"])).transpose(1, 2)
            return s
        Hkv = case["Hkv"]
        # a projection's output: q, k and v side by side in one row a token
        qkv = _rand((B, T, Hq + 2 * Hkv, D), g)
        s["q"], s["k_new"], s["v_new"] = (x.transpose(1, 2) for x in qkv.split([Hq, Hkv, Hkv], dim=2))
        s["bt"], blocks = _table(B, (case["ctx"] + T + BS - 1) // BS, g)
        s["start"] = _ints([case["ctx"]] * B)
        s["k_cache"], s["v_cache"] = _pool(blocks, Hkv, D, g), _pool(blocks, Hkv, D, g)
        return s
    lens = _lens(case)
    Hkv = case["Hkv"]
    s["max_len"] = max(lens)
    s["lens"] = _ints(lens)
    s["scale"] = 1.0 / math.sqrt(D)
    if op == "tree":
        T = case["T"]
        s["bt"], blocks = _table(B, (s["max_len"] + T + BS - 1) // BS, g)
        s["q"] = _rand((B, T, case["Hq"], D), g).transpose(1, 2)
        s["k_new"], s["v_new"] = (_rand((B, T, Hkv, D), g).transpose(1, 2) for _ in range(2))
        s["parents"], s["path"], s["taken"] = _tree(case, seed)
    elif op == "weights":
        T = case["T"]
        s["bt"], blocks = _table(B, (s["max_len"] + T + BS - 1) // BS, g)
        s["q"] = _rand((B, case["Hq"], T, D), g)
        s["acc"] = torch.rand((blocks, Hkv, BS), generator=g, device="cuda")
    else:
        s["bt"], blocks = _table(B, (s["max_len"] + BS - 1) // BS, g)
        new = (case["keep"] + BS - 1) // BS
        s["dst"] = (blocks + torch.arange(B * new, device="cuda")).to(torch.int32).reshape(B, new)
        blocks += B * new
        # weights as they come: a few large ones, most near zero, many of them equal
        s["acc"] = torch.rand((blocks, Hkv, BS), generator=g, device="cuda").pow_(8).mul_(4096).round_().div_(256)
    s["k_cache"] = _pool(blocks, Hkv, D, g)
    if op == "weights":
        s["lse"] = _lse(s)
    else:
        s["v_cache"] = _pool(blocks, Hkv, D, g)
    return s


def _lse(s):
    """The log-sum-exp that the attention of the same rows returned: [B, Hq, T]."""
    B, Hq, T, D = s["q"].shape
    got = torch.empty((B, Hq, T), device="cuda")
    G = Hq // s["Hkv"]
    for b in range(B):
        n = int(s["lens"][b]) + T
        k = _rows(s["k_cache"], s["bt"][b:b + 1], n)[0].float()  # [n, Hkv, D]
        see = torch.arange(n, device="cuda") <= int(s["lens"][b]) + torch.arange(T, device="cuda")[:, None]
        for h in range(s["Hkv"]):
            x = s["q"][b, h * G:(h + 1) * G].float() @ k[:, h].t() * s["scale"]
            got[b, h * G:(h + 1) * G] = torch.logsumexp(x.masked_fill(~see, -math.inf), dim=-1)
    return got


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def run(s):
    if own:
        return _run_own(s)
    return {"rope_append": _plain_rope_append, "rope_apply": _plain_rope_apply, "tree": _plain_tree,
            "weights": _plain_weights, "evict": _plain_evict}[s["op"]](s)


def _run_own(s):
    import masked_attention_paged_gb300 as lib
    op = s["op"]
    if op == "rope_apply":
        return lib.rope_apply(s["x"], s["positions"], s["freqs"], interleaved=s["inter"], inverse=s["inverse"])
    if "ws" not in s:  # a serving program keeps one workspace for its shapes
        nbytes = 256
        if op == "tree":
            nbytes = lib.paged_tree_workspace_size(s["B"], s["Hq"], s["Hkv"], s["T"], s["bt"].shape[1], BS, s["D"])
        elif op == "weights":
            nbytes = lib.paged_attn_weights_workspace_size(s["B"], s["Hkv"], s["bt"].shape[1], BS)
        s["ws"] = lib.Workspace(nbytes)
    if op == "rope_append":
        q = lib.rope_kv_append(s["q"], s["k_new"], s["v_new"], s["positions"], s["freqs"], s["k_cache"], s["v_cache"],
                               s["bt"], s["start"], interleaved=s["inter"], workspace=s["ws"])
        return [q, s["k_cache"], s["v_cache"]]
    if op == "tree":
        out, lse = lib.paged_tree_attn(s["q"], s["k_cache"], s["v_cache"], s["bt"], s["lens"], s["parents"],
                                       k_new=s["k_new"], v_new=s["v_new"], scale=s["scale"], return_lse=True,
                                       workspace=s["ws"])
        lib.kv_tree_accept(s["k_cache"], s["v_cache"], s["bt"], s["lens"], s["path"], s["taken"], workspace=s["ws"])
        return [out, lse, s["k_cache"], s["v_cache"]]
    if op == "weights":
        lib.paged_attn_weights(s["q"], s["lse"], s["k_cache"], s["bt"], s["lens"], s["acc"], scale=s["scale"],
                               workspace=s["ws"])
        return s["acc"]
    new_lens, kept = lib.kv_evict(s["k_cache"], s["v_cache"], s["acc"], s["bt"], s["lens"], s["dst"], s["keep"],
                                  sink=s["sink"], recent=s["recent"], workspace=s["ws"])
    return [new_lens, kept, s["acc"], s["k_cache"], s["v_cache"]]


# --------------------------------------------------------------------------
# plain forms
# --------------------------------------------------------------------------
def _rows(cache, bt, n):
    """Rows [B, n, Hkv, ...] of the first n slots of each sequence of a paged tensor."""
    at = torch.arange(n, device=cache.device)
    return cache[bt[:, at // BS].long(), :, at % BS]


def _put(cache, bt, slot, rows, ok):
    """Row [b, i] of rows [B, n, Hkv, D] to slot[b, i] of its sequence, where ok[b, i]."""
    blk = torch.gather(bt, 1, (slot // BS).clamp(0, bt.shape[1] - 1)).long()
    cache[blk[ok], :, (slot % BS)[ok]] = rows[ok]


def _rotate(x, positions, inv_freq, inter, inverse=False):
    """x [B, H, T, D] rotated by its tokens' positions, in float32."""
    n = inv_freq.numel()
    angle = positions.double()[:, None, :, None] * inv_freq
    c, si = angle.cos().float(), angle.sin().float()
    if inverse:
        si = -si
    x = x.float()
    r, rest = x[..., :2 * n], x[..., 2 * n:]
    a, b = (r[..., 0::2], r[..., 1::2]) if inter else (r[..., :n], r[..., n:])
    u, v = a * c - b * si, a * si + b * c
    r = torch.stack([u, v], dim=-1).flatten(-2) if inter else torch.cat([u, v], dim=-1)
    return torch.cat([r, rest], dim=-1)


def _plain_rope_apply(s):
    return _rotate(s["x"], s["positions"], s["inv_freq"], s["inter"], s["inverse"]).to(s["x"].dtype)


def _plain_rope_append(s):
    q = _rotate(s["q"], s["positions"], s["inv_freq"], s["inter"]).to(s["q"].dtype)
    k = _rotate(s["k_new"], s["positions"], s["inv_freq"], s["inter"]).to(s["k_cache"].dtype)
    slot = s["start"].long()[:, None] + torch.arange(s["T"], device="cuda")
    ok = torch.ones_like(slot, dtype=torch.bool)
    _put(s["k_cache"], s["bt"], slot, k.transpose(1, 2), ok)
    _put(s["v_cache"], s["bt"], slot, s["v_new"].transpose(1, 2), ok)
    return [q, s["k_cache"], s["v_cache"]]


def _plain_tree(s):
    B, Hq, T, D = s["q"].shape
    Hkv, n, lens, parents = s["Hkv"], s["max_len"], s["lens"].long(), s["parents"].long()
    there = parents >= -1
    # see[t, a]: a is t or one of its ancestors; paths double in length at each product
    see = torch.eye(T, device="cuda") + (parents[:, :, None] == torch.arange(T, device="cuda"))
    for _ in range((T - 1).bit_length()):
        see = (see @ see).clamp_(max=1.0)
    see = (see > 0) & there[:, :, None] & there[:, None, :]
    ctx = (torch.arange(n, device="cuda") < lens[:, None])[:, None, :] & there[:, :, None]
    mask = torch.cat([ctx, see], dim=2)[:, None].expand(B, Hq // Hkv, T, n + T).reshape(B, 1, -1, n + T)
    k = torch.cat([_rows(s["k_cache"], s["bt"], n), s["k_new"].transpose(1, 2)], dim=1).float().permute(0, 2, 1, 3)
    v = torch.cat([_rows(s["v_cache"], s["bt"], n), s["v_new"].transpose(1, 2)], dim=1).float().permute(0, 2, 1, 3)
    q = s["q"].float().reshape(B, Hkv, -1, D)
    x = (q @ k.transpose(2, 3)).mul_(s["scale"]).masked_fill_(~mask, -math.inf)
    top = x.amax(dim=-1, keepdim=True)
    p = x.sub_(top.clamp(min=-1e30)).exp_()
    total = p.sum(dim=-1, keepdim=True)
    out = (p @ v) / total.clamp(min=1e-30)
    lse = (total.log() + top).reshape(B, Hq, T)
    slot = lens[:, None] + torch.arange(T, device="cuda")
    _put(s["k_cache"], s["bt"], slot, s["k_new"].transpose(1, 2), there)
    _put(s["v_cache"], s["bt"], slot, s["v_new"].transpose(1, 2), there)
    # the accepted path's rows move up behind the context
    take = s["path"].long()[:, :, None, None].expand(B, T, Hkv, D)
    ok = torch.arange(T, device="cuda") < s["taken"].long()[:, None]
    _put(s["k_cache"], s["bt"], slot, s["k_new"].transpose(1, 2).gather(1, take), ok)
    _put(s["v_cache"], s["bt"], slot, s["v_new"].transpose(1, 2).gather(1, take), ok)
    return [out.reshape(B, Hq, T, D).to(s["q"].dtype), lse, s["k_cache"], s["v_cache"]]


def _plain_weights(s):
    B, Hq, T, D = s["q"].shape
    Hkv, n, lens = s["Hkv"], s["max_len"] + T, s["lens"].long()
    k = _rows(s["k_cache"], s["bt"], n).float().permute(0, 2, 1, 3)
    q = s["q"].float().reshape(B, Hkv, -1, D)
    x = (q @ k.transpose(2, 3)).mul_(s["scale"]).sub_(s["lse"].reshape(B, Hkv, -1, 1)).exp_()
    at = torch.arange(n, device="cuda")
    see = at <= lens[:, None, None] + torch.arange(T, device="cuda")[:, None]  # [B, T, n]
    got = x.reshape(B, Hkv, Hq // Hkv, T, n).masked_fill_(~see[:, None, None], 0.0).sum(dim=(2, 3))
    # tokens before the chunk have a sum already, the chunk's own begin theirs
    slot = at.expand(B, n)
    old = _rows(s["acc"], s["bt"], n).masked_fill_((slot >= lens[:, None])[:, :, None], 0.0)
    _put(s["acc"], s["bt"], slot, old + got.transpose(1, 2), slot < lens[:, None] + T)
    return s["acc"]


def _plain_evict(s):
    n, keep, lens = s["max_len"], s["keep"], s["lens"].long()
    at = torch.arange(max(n, keep), device="cuda")
    there = at < lens[:, None]
    acc = torch.nn.functional.pad(_rows(s["acc"], s["bt"], n), (0, 0, 0, max(0, keep - n)))
    held = (at < s["sink"]) | (at >= lens[:, None] - s["recent"])
    rank = acc.masked_fill(held[:, :, None], math.inf).masked_fill(~there[:, :, None], -math.inf)
    best = torch.sort(rank, dim=1, descending=True, stable=True).indices[:, :keep]
    kept = torch.where(best < lens[:, None, None], best, at.numel()).sort(dim=1).values  # [B, keep, Hkv]
    ok = kept[:, :, :1] < at.numel()
    src = kept.clamp(max=n - 1)
    blk = torch.gather(s["bt"][:, :, None].expand(-1, -1, s["Hkv"]), 1, src // BS).long()
    head = torch.arange(s["Hkv"], device="cuda")
    slot = at[:keep].expand(s["B"], keep)
    for name in ("k_cache", "v_cache", "acc"):
        _put(s[name], s["dst"], slot, s[name][blk, head, src % BS], ok[:, :, 0])
    kept = torch.where(ok, kept, -1).transpose(1, 2).contiguous()
    return [lens.clamp(max=keep).to(torch.int32), kept.to(torch.int32), s["acc"], s["k_cache"], s["v_cache"]]


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------
def work(case):
    op, B, D = case["op"], case["B"], case["D"]
    if op == "rope_apply":
        n = B * case["T"] * case["Hq"] * D
        return {"bytes": 2 * n * (4 if case["dtype"] == "float32" else 2) + 4 * B * case["T"],
                "flops": 3 * B * case["T"] * case["Hq"] * case["rot"]}
    if op == "rope_append":
        n = B * case["T"] * (case["Hq"] + 2 * case["Hkv"]) * D
        return {"bytes": 4 * n + 4 * B * (case["T"] + 1),
                "flops": 3 * B * case["T"] * (case["Hq"] + case["Hkv"]) * case["rot"]}
    Hkv, lens = case["Hkv"], _lens(case)
    if op == "tree":
        T, Hq, drafts = case["T"], case["Hq"], _drafts(case)
        rows = 2 * D * Hkv * 2  # K and V of one token
        nbytes = sum(lens) * rows + 2 * sum(drafts) * rows + B * Hq * T * (4 * D + 4) + 4 * B * T
        nbytes += 2 * B * case["accept"] * rows
        return {"bytes": nbytes, "flops": sum(4 * Hq * n * (c + n // 4 + 1) * D for n, c in zip(drafts, lens))}
    if op == "weights":
        T, Hq = case["T"], case["Hq"]
        keys = sum(lens) + B * T
        return {"bytes": keys * Hkv * (2 * D + 8) + B * Hq * T * (2 * D + 4),
                "flops": sum(2 * Hq * T * (c + (T + 1) / 2) * D for c in lens)}
    kept = sum(min(c, case["keep"]) for c in lens)
    return {"bytes": 4 * Hkv * sum(lens) + kept * Hkv * (2 * 4 * D + 8), "flops": Hkv * sum(lens)}


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return {"rope_append": _exact_rope_append, "rope_apply": _exact_rope_apply, "tree": _exact_tree,
            "weights": _exact_weights, "evict": _exact_evict}[case["op"]](s)


def _exact_turned(x, s, sign):
    """Each pair as a complex number times e^{i angle}."""
    B, H, T, D = x.shape
    n = s["rot"] // 2
    even = torch.arange(n, device="cuda") * (2 if s["inter"] else 1)
    odd = even + (1 if s["inter"] else n)
    x = x.double()
    z = torch.complex(x[..., even], x[..., odd])
    angle = (s["first"] + torch.arange(T, device="cuda")).double()[:, None, :, None] * s["inv_freq"] * sign
    z = z * torch.polar(torch.ones_like(angle), angle)
    y = x.clone()
    y[..., even], y[..., odd] = z.real, z.imag
    return y


def _exact_rope_apply(s):
    return _exact_turned(s["x"], s, -1.0 if s["inverse"] else 1.0)


def _exact_rope_append(s):
    k = _exact_turned(s["k_new"], s, 1.0)
    k_cache, v_cache = s["k_cache"].double(), s["v_cache"].double()
    for i in range(s["T"]):
        at = s["ctx"] + i
        blk = s["bt"][:, at // BS].long()
        k_cache[blk, :, at % BS] = k[:, :, i]
        v_cache[blk, :, at % BS] = s["v_new"][:, :, i].double()
    return [_exact_turned(s["q"], s, 1.0), k_cache, v_cache]


def _exact_tree(s):
    B, Hq, T, D = s["q"].shape
    G = Hq // s["Hkv"]
    out = torch.zeros((B, Hq, T, D), dtype=torch.float64, device="cuda")
    lse = torch.full((B, Hq, T), -math.inf, dtype=torch.float64, device="cuda")
    parents, lens = s["parents"].tolist(), s["lens"].tolist()
    for b in range(B):
        see = torch.zeros((T, T), dtype=torch.bool)
        n = sum(p >= -1 for p in parents[b])
        for t in range(n):
            a = t
            while a >= 0:
                see[t, a] = True
                a = parents[b][a]
        see = see[:n, :n].cuda()
        for h in range(s["Hkv"]):
            kc, vc = (_rows(s[c], s["bt"][b:b + 1], lens[b])[0, :, h].double() for c in ("k_cache", "v_cache"))
            for j in range(h * G, (h + 1) * G):
                q = s["q"][b, j, :n].double() * s["scale"]
                x = torch.cat([q @ kc.t(), (q @ s["k_new"][b, h, :n].double().t()).masked_fill(~see, -math.inf)], dim=1)
                lse[b, j, :n] = torch.logsumexp(x, dim=1)
                p = torch.exp(x - lse[b, j, :n, None])
                out[b, j, :n] = p[:, :lens[b]] @ vc + p[:, lens[b]:] @ s["v_new"][b, h, :n].double()
    return [out, lse, None, None]


def _exact_weights(s):
    B, Hq, T, D = s["q"].shape
    G = Hq // s["Hkv"]
    acc = s["acc"].double()
    lens = s["lens"].tolist()
    for b in range(B):
        n = lens[b] + T
        for h in range(s["Hkv"]):
            k = _rows(s["k_cache"], s["bt"][b:b + 1], n)[0, :, h].double()
            total = torch.zeros(n, dtype=torch.float64, device="cuda")
            for j in range(h * G, (h + 1) * G):
                x = s["q"][b, j].double() @ k.t() * s["scale"] - s["lse"][b, j].double()[:, None]
                total += torch.tril(x.exp(), diagonal=lens[b]).sum(dim=0)
            at = torch.arange(n, device="cuda")
            blk = s["bt"][b, at // BS].long()
            before = torch.where(at < lens[b], acc[blk, h, at % BS], 0.0)
            acc[blk, h, at % BS] = before + total
    return acc


def _exact_evict(s):
    acc = s["acc"].double().cpu().numpy()
    bt, dst, lens = s["bt"].tolist(), s["dst"].tolist(), s["lens"].tolist()
    for b in range(s["B"]):
        n = lens[b]
        for h in range(s["Hkv"]):
            x = [float(v) for blk in bt[b] for v in acc[blk, h]][:n]
            free = range(min(s["sink"], n), max(n - s["recent"], min(s["sink"], n)))
            held = [i for i in range(n) if i not in free]
            order = held + sorted(free, key=lambda i: (-x[i], i))
            for i, j in enumerate(sorted(order[:s["keep"]])):
                acc[dst[b][i // BS], h, i % BS] = x[j]
    return [None, None, torch.from_numpy(acc), None, None]
