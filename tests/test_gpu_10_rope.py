"""GPU tests of the rotary calls against a plain implementation in 64 bits.

The kernel's own error of a pair (a, b) before the last rounding: its sines and
cosines are off by at most 2^-22 (the angle, at most pi / 4 after the quarter
turns are taken off, is rounded once: 2^-24 pi / 4; sincospif itself is within
2 ulp, 2^-23), and the two products and the sum round three times, 2^-24 each:
less than 2^-21 (|a| + |b|) m in all.  The definition's angle position * f in
64 bits is itself off by |position| f 2^-52.  The output's rounding adds half a
step, finfo.eps / 2 of its value."""
import math

import numpy as np
import pytest
import torch

import masked_attention_paged_gb300 as lib

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _freqs(rot, factor=1.0):
    inv = 10000.0 ** (-np.arange(0, rot, 2, dtype=np.float64) / rot) / factor
    got, _ = lib.rope_frequencies(rot, scaling="linear", factor=factor)
    return inv, got


def _define(x, positions, inv, inter, inverse=False, m=1.0):
    """(rotated, error bound before the output's rounding), in 64 bits, x [B, H, T, D]."""
    x = x.double().cpu().numpy()
    n = len(inv)
    pos = positions.cpu().numpy().astype(np.float64)
    ang = pos[:, None, :, None] * inv * (-1.0 if inverse else 1.0)
    c, s = np.cos(ang) * m, np.sin(ang) * m
    y, tol = x.copy(), np.zeros_like(x)
    ia, ib = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if inter else (slice(0, n), slice(n, 2 * n))
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, a * s + b * c
    own = (np.abs(a) + np.abs(b)) * m * (2.0 ** -21 + np.abs(ang) * 2.0 ** -52)
    tol[..., ia] = tol[..., ib] = own
    return y, tol


def _hold(got, ref, tol):
    got64 = got.detach().double().cpu().numpy()
    bound = tol + np.abs(ref) * torch.finfo(got.dtype).eps / 2
    bad = ~(np.abs(got64 - ref) <= bound * (1 + 1e-12))
    assert not bad.any(), (np.argwhere(bad)[:3], got64[bad][:3], ref[bad][:3])


def _rand(shape, seed, dtype):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype).to(DEV)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("B,H,T,D,rot", [(1, 1, 1, 64, 64), (3, 5, 7, 128, 128), (2, 4, 33, 128, 64), (2, 3, 9, 128, 34),
                                         (1, 2, 5, 64, 2), (2, 2, 6, 80, 48), (1, 3, 4, 6, 6), (2, 3, 3, 37, 12),
                                         (1, 1, 3, 512, 512), (2, 40, 700, 64, 32)])
def test_apply(B, H, T, D, rot, inter, dtype):
    inv, fr = _freqs(rot)
    x = _rand((B, H, T, D), 1, dtype)
    pos = torch.randint(0, 5000, (B, T), generator=torch.Generator().manual_seed(2), dtype=torch.int32).to(DEV)
    y, tol = _define(x, pos, inv, inter)
    got = lib.rope_apply(x, pos, fr, interleaved=inter)
    _hold(got, y, tol)
    assert torch.equal(got[..., rot:], x[..., rot:])  # the rest of the head is copied
    # the transposed rotation, a magnitude, and one row of positions for the whole batch
    one = pos[:1].expand(B, T)
    y, tol = _define(x, one, inv, inter, inverse=True, m=1.25)
    _hold(lib.rope_apply(x, one, fr, interleaved=inter, inverse=True, magnitude=1.25), y, tol)
    # in place
    z = x.clone()
    assert lib.rope_apply(z, pos, fr, interleaved=inter, out=z) is z
    assert torch.equal(z, got)


@pytest.mark.parametrize("inter", [False, True])
def test_far_and_negative_positions(inter):
    """Angles of millions of radians: a float32 product would be off by whole turns at 2^31."""
    inv, fr = _freqs(64, factor=4.0)
    pos = torch.tensor([[0, -1, 1 << 20, 1000003, -(1 << 31), (1 << 31) - 1, 131071, -77]], dtype=torch.int32).to(DEV)
    x = _rand((1, 3, 8, 64), 3, torch.float32)
    y, tol = _define(x, pos, inv, inter)
    _hold(lib.rope_apply(x, pos, fr, interleaved=inter), y, tol)


@pytest.mark.parametrize("inter", [False, True])
def test_strided_views_and_odd_alignment(inter):
    """Slices of a packed projection, tokens before heads, and rows that start 2 bytes off a vector."""
    inv, fr = _freqs(64)
    qkv = _rand((2, 9, 12, 64), 4, torch.bfloat16)
    pos = torch.arange(9, dtype=torch.int32, device=DEV).expand(2, 9)
    x = qkv[:, :, 2:7].transpose(1, 2)
    y, tol = _define(x, pos, inv, inter)
    got = lib.rope_apply(x, pos, fr, interleaved=inter)
    _hold(got, y, tol)
    flat = torch.zeros(2 * 9 * 5 * 72 + 1, dtype=torch.bfloat16, device=DEV)
    odd = flat[1:].view(2, 9, 5, 72)[..., 1:65].transpose(1, 2)
    odd.copy_(x)
    out = torch.empty_like(x)
    assert torch.equal(lib.rope_apply(odd, pos, fr, interleaved=inter, out=out), got)
    lib.rope_apply(odd, pos, fr, interleaved=inter, out=odd)
    assert torch.equal(odd, got)
    assert int((flat != 0).sum()) <= 2 * 9 * 5 * 64  # nothing beside the rows was written


def test_gradient_against_the_formula_and_differences():
    inv, fr = _freqs(48)
    B, H, T, D = 2, 3, 11, 64
    x, g, d = (_rand((B, H, T, D), s, torch.float32) for s in (5, 6, 7))
    pos = torch.randint(0, 9000, (B, T), generator=torch.Generator().manual_seed(8), dtype=torch.int32).to(DEV)
    f = lambda z: lib.rope_apply(z, pos, fr, interleaved=True, magnitude=1.5)  # noqa: E731
    back = lib.rope_apply(g, pos, fr, interleaved=True, inverse=True, magnitude=1.5)
    # the formula's: autograd through the rotation in 64 bits
    z = x.double().requires_grad_()
    n = 24
    ang = (pos.double()[:, None, :, None] * torch.from_numpy(inv).to(DEV))
    a, b = z[..., 0:2 * n:2], z[..., 1:2 * n:2]
    c, s = 1.5 * ang.cos(), 1.5 * ang.sin()
    y = torch.cat([torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2), z[..., 2 * n:]], -1)
    y.backward(g.double())
    _, tol = _define(g, pos, inv, True, inverse=True, m=1.5)
    _hold(back, z.grad.cpu().numpy(), tol)
    # differences: the rotation is linear, so the quotient has no error of its own beyond the rounding of
    # f(x + d) and f(x - d): 2^-21 of their sizes each, summed over the products with g
    quot = ((f(x + d) - f(x - d)) / 2).double().mul(g.double()).sum().item()
    want = back.double().mul(d.double()).sum().item()
    slack = 2.0 ** -20 * 2 * 1.5 * ((x.abs() + d.abs()).double().sum() * g.abs().max()).item()
    assert abs(quot - want) <= slack


def _cache(nb, Hkv, D, fill=float("nan")):
    return (torch.full((nb, Hkv, 16, D), fill, dtype=torch.bfloat16, device=DEV) for _ in range(2))


@pytest.mark.parametrize("rot,inter", [(128, False), (64, True), (34, False), (20, True)])
@pytest.mark.parametrize("T,Hq,Hkv", [(1, 8, 2), (1, 6, 6), (21, 12, 4), (300, 4, 1)])
def test_append_is_apply_and_copy(T, Hq, Hkv, rot, inter):
    """Bit for bit rope_apply and kv_append: q, the rotated keys and the values in their slots, nothing else; a NaN
    payload in the values survives."""
    B, D = 3, 128
    _, fr = _freqs(rot)
    q, k, v = (_rand((B, h, T, D), 9 + i, torch.bfloat16) for i, h in enumerate((Hq, Hkv, Hkv)))
    v.view(torch.int16)[0, 0, 0, :3] = torch.tensor([0x7fa5, -0x7f, 0x7f81], dtype=torch.int16)
    pos = torch.randint(0, 100000, (B, T), generator=torch.Generator().manual_seed(3), dtype=torch.int32).to(DEV)
    start = torch.tensor([0, 13, 100], dtype=torch.int32, device=DEV)
    mb = (100 + T + 15) // 16
    bt = torch.randperm(B * mb + 2, generator=torch.Generator().manual_seed(4))[:B * mb].to(torch.int32).view(B, mb).to(DEV)
    kc, vc = _cache(B * mb + 2, Hkv, D)
    ek, ev = kc.clone(), vc.clone()
    ws = lib.Workspace(256)
    qo = lib.rope_kv_append(q, k, v, pos, fr, kc, vc, bt, start, interleaved=inter, workspace=ws)
    assert ws.status() == 0
    assert torch.equal(qo, lib.rope_apply(q, pos, fr, interleaved=inter))
    kr = lib.rope_apply(k, pos, fr, interleaved=inter)
    for i in range(T):
        lib.kv_append(ek, ev, bt, start + i, kr[:, :, i].contiguous(), v[:, :, i].contiguous())
    assert torch.equal(kc.view(torch.int16), ek.view(torch.int16))
    assert torch.equal(vc.view(torch.int16), ev.view(torch.int16))
    if T == 1:  # without the token dimension, q rotated in place
        k2, v2 = _cache(B * mb + 2, Hkv, D)
        q3 = q[:, :, 0].clone()
        assert lib.rope_kv_append(q3, k[:, :, 0], v[:, :, 0], pos[:, 0], fr, k2, v2, bt, start, interleaved=inter,
                                  q_out=q3) is q3
        assert torch.equal(q3, qo[:, :, 0]) and torch.equal(k2.view(torch.int16), kc.view(torch.int16))


@pytest.mark.parametrize("D,rot,inter", [(128, 128, False), (128, 64, True), (64, 32, False), (64, 20, True)])
@pytest.mark.parametrize("T,Hq,Hkv", [(1, 8, 2), (37, 5, 5), (3, 3, 1)])
def test_append_q8_is_apply_and_quantise(T, Hq, Hkv, D, rot, inter):
    B = 2
    _, fr = _freqs(rot)
    q, k, v = (_rand((B, h, T, D), 20 + i, torch.bfloat16) for i, h in enumerate((Hq, Hkv, Hkv)))
    v[1, 0, 0] = 0  # an all-zero row: scale 0, codes 0
    pos = torch.randint(0, 3000, (B, T), generator=torch.Generator().manual_seed(3), dtype=torch.int32).to(DEV)
    start = torch.tensor([15, 2], dtype=torch.int32, device=DEV)
    mb = 4
    bt = torch.randperm(B * mb, generator=torch.Generator().manual_seed(4)).to(torch.int32).view(B, mb).to(DEV)
    codes = lambda: torch.full((B * mb, Hkv, 16, D), 99, dtype=torch.int8, device=DEV)  # noqa: E731
    scale = lambda: torch.full((B * mb, Hkv, 16), -1.0, device=DEV)  # noqa: E731
    got = [codes(), codes(), scale(), scale()]
    ref = [codes(), codes(), scale(), scale()]
    qo = lib.rope_kv_append_q8(q, k, v, pos, fr, *got, bt, start, interleaved=inter)
    assert torch.equal(qo, lib.rope_apply(q, pos, fr, interleaved=inter))
    kr = lib.rope_apply(k, pos, fr, interleaved=inter)
    for i in range(T):
        lib.kv_append_q8(*ref, bt, start + i, kr[:, :, i].contiguous(), v[:, :, i].contiguous())
    for a, b in zip(got, ref):
        assert torch.equal(a, b)


def test_idle_sequences_and_bad_tables():
    """A negative start caches nothing; a start past the table and a bad block id are reported, the rest is written,
    and q is rotated for every sequence."""
    B, T, Hq, Hkv, D = 5, 20, 4, 2, 64
    _, fr = _freqs(64)
    q, k, v = (_rand((B, h, T, D), 30 + i, torch.bfloat16) for i, h in enumerate((Hq, Hkv, Hkv)))
    pos = torch.arange(T, dtype=torch.int32, device=DEV).expand(B, T)
    start = torch.tensor([3, -1, 29, 0, 12], dtype=torch.int32, device=DEV)  # 29 + 20 > 48
    bt = torch.arange(B * 3, dtype=torch.int32, device=DEV).view(B, 3)
    bt[3, 1] = B * 3  # past the cache
    bt[4, 1] = -7
    kc, vc = _cache(B * 3, Hkv, D, fill=7.0)
    ws = lib.Workspace(256)
    qo = lib.rope_kv_append(q, k, v, pos, fr, kc, vc, bt, start, workspace=ws)
    assert ws.status() == 5
    assert torch.equal(qo, lib.rope_apply(q, pos, fr))
    kr = lib.rope_apply(k, pos, fr)
    for c, rows in ((kc, kr), (vc, v)):
        want = torch.full_like(c, 7.0)
        for b, slots in ((0, range(20)), (3, list(range(0, 16)) + list(range(16, 20))), (4, range(20))):
            for i in slots:
                at = int(start[b]) + i
                blk = int(bt[b, at // 16])
                if 0 <= blk < B * 3:
                    want[blk, :, at % 16] = rows[b, :, i]
        assert torch.equal(c, want)


def test_stream_and_graph():
    """The call on a side stream, and captured and replayed with other contents in its buffers."""
    B, T, Hq, Hkv, D = 2, 1, 8, 2, 128
    _, fr = _freqs(128)
    q, k, v = (_rand((B, h, T, D), 40 + i, torch.bfloat16) for i, h in enumerate((Hq, Hkv, Hkv)))
    pos = torch.tensor([[5], [900]], dtype=torch.int32, device=DEV)
    start = torch.tensor([0, 17], dtype=torch.int32, device=DEV)
    bt = torch.arange(4, dtype=torch.int32, device=DEV).view(2, 2)
    kc, vc = _cache(4, Hkv, D, fill=0.0)
    qo, ws = torch.empty_like(q), lib.Workspace(256)
    call = lambda: lib.rope_kv_append(q, k, v, pos, fr, kc, vc, bt, start, q_out=qo, workspace=ws)  # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(qo, lib.rope_apply(q, pos, fr))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    q.mul_(-2.0)
    pos.add_(31)
    start.add_(1)
    g.replay()
    assert torch.equal(qo, lib.rope_apply(q, pos, fr))
    kr = lib.rope_apply(k, pos, fr)
    assert torch.equal(kc[0, :, 1], kr[0, :, 0]) and torch.equal(kc[3, :, 2], kr[1, :, 0])
    assert math.isfinite(float(vc.float().sum()))
