"""Rotary positions without a GPU: the frequencies against their formulas, and
what the calls refuse before anything is launched."""
import ctypes
import math

import pytest
import torch

import masked_attention_paged_gb300 as lib
from test_binding_marshalling import rec  # noqa: F401  (fixture)
from test_boundary import FAKE, INVALID, L, OK, UNSUPPORTED, WORKSPACE, _cache, _cache_q8, _t  # noqa: F401

TURN = 2.0 * math.pi


def _radians(*args, **kw):
    turns, magnitude = lib.rope_frequencies(*args, device="cpu", **kw)
    assert turns.dtype == torch.int64 and turns.min() >= 0
    return (turns.double() / 2.0 ** 64 * TURN).tolist(), magnitude


def _plain(d, base=10000.0):
    return [base ** (-2.0 * i / d) for i in range(d // 2)]


def _near(x, y):
    """pow, the blend, the division by 2 pi and the product above round a few times, 2^-53 each: 64 of them are
    allowed; and a fraction is a whole number of 2^-64 turns, so it is off by half a unit, pi 2^-64 radians."""
    return abs(x - y) <= 64 * 2.0 ** -53 * abs(y) + TURN * 2.0 ** -65


def _close(a, b):
    assert len(a) == len(b)
    for x, y in zip(a, b):
        assert _near(x, y), (x, y)


@pytest.mark.parametrize("d", [2, 6, 64, 96, 128])
def test_plain_linear_and_base(d):
    got, m = _radians(d)
    _close(got, _plain(d))
    assert m == 1.0
    _close(_radians(d, base=500000.0, scaling="linear", factor=8.0)[0], [f / 8.0 for f in _plain(d, 500000.0)])
    if d > 2:
        _close(_radians(d, scaling="base", factor=4.0)[0], _plain(d, 10000.0 * 4.0 ** (d / (d - 2))))


def test_banded_keeps_fast_pairs_and_interpolates_slow_ones():
    d, n, s, low, high = 128, 8192, 8.0, 1.0, 4.0
    got, m = _radians(d, base=500000.0, scaling="banded", factor=s, original_len=n, low=low, high=high)
    assert m == 1.0
    kept = slowed = 0
    for f, g in zip(_plain(d, 500000.0), got):
        wave = TURN / f
        if wave < n / high:
            assert _near(g, f)
            kept += 1
        elif wave > n / low:
            assert _near(g, f / s)
            slowed += 1
        else:
            w = (n / wave - low) / (high - low)
            assert _near(g, (1 - w) * f / s + w * f)
    assert kept > 0 and slowed > 0


def test_ramp_blends_over_the_pair_index_and_scales_the_magnitude():
    d, n, s, low, high = 64, 4096, 16.0, 1.0, 32.0
    got, m = _radians(d, scaling="ramp", factor=s, original_len=n, low=low, high=high)
    assert abs(m - (0.1 * math.log(s) + 1.0)) < 1e-6

    def index(r):
        return d * math.log(n / (r * TURN)) / (2 * math.log(10000.0))
    lo, hi = math.floor(index(high)), math.ceil(index(low))
    assert 0 < lo < hi < d // 2
    for i, (f, g) in enumerate(zip(_plain(d), got)):
        w = 1.0 - min(max((i - lo) / (hi - lo), 0.0), 1.0)
        assert _near(g, f * w + f / s * (1 - w))
    assert _radians(d, scaling="ramp", factor=1.0, original_len=n, low=low, high=high)[1] == 1.0


@pytest.mark.parametrize("kw", [dict(rotary_dim=0), dict(rotary_dim=7), dict(rotary_dim=-2), dict(base=1.0),
                                dict(base=float("inf")), dict(factor=0.5), dict(factor=float("nan")),
                                dict(rotary_dim=2, scaling="base"), dict(scaling="banded", original_len=0),
                                dict(scaling="ramp", original_len=4096, low=4.0, high=4.0),
                                dict(scaling="banded", original_len=4096, low=0.0)])
def test_frequencies_refuse(kw):
    with pytest.raises(lib.LibAttnError, match="INVALID_ARG"):
        lib.rope_frequencies(**{"rotary_dim": 64, "device": "cpu", **kw})
    with pytest.raises(ValueError, match="scaling must be one of"):
        lib.rope_frequencies(64, scaling="other", device="cpu")


def _apply(L, x, out=None, pos=FAKE, ps=40, fr=FAKE, rot=64, inter=0, inv=0, mag=1.0):
    out = out or x
    return L.rope_apply(ctypes.byref(x), pos, ps, fr, rot, inter, inv, mag, ctypes.byref(out), None)


def test_rope_apply_rejects(L):
    x = _t([2, 4, 40, 64])
    assert _apply(L, _t([4, 40, 64])) == INVALID
    assert _apply(L, x, out=_t([2, 4, 41, 64])) == INVALID
    assert _apply(L, x, out=_t([2, 4, 40, 64], 0)) == INVALID
    assert _apply(L, x, rot=66) == INVALID
    assert _apply(L, x, rot=31) == INVALID
    assert _apply(L, x, rot=0) == INVALID
    assert _apply(L, x, inter=2) == INVALID
    assert _apply(L, x, inv=-1) == INVALID
    assert _apply(L, x, mag=float("inf")) == INVALID
    assert _apply(L, x, pos=None) == INVALID
    assert _apply(L, x, pos=FAKE + 2) == INVALID
    assert _apply(L, x, fr=None) == INVALID
    assert _apply(L, x, fr=FAKE + 4) == INVALID
    assert _apply(L, x, ps=39) == INVALID
    assert _apply(L, x, ps=-40) == INVALID
    assert _apply(L, _t([2, 4, 40, 64], data=FAKE + 1)) == INVALID
    assert _apply(L, _t([2, 4, 40, 514]), rot=64) == UNSUPPORTED
    assert _apply(L, _t([2, 4, 0, 64])) == OK and _apply(L, _t([0, 4, 9, 64])) == OK


def test_rope_kv_append_rejects(L):
    def call(q=None, k=None, v=None, qo=None, c=None, pos=FAKE, sp=FAKE, bt=FAKE, bts=10, mb=10, ws=FAKE, rot=128,
             q8=False):
        q = q or _t([2, 32, 5, 128])
        k = k or _t([2, 8, 5, 128])
        fn, c = (L.rope_kv_append_q8, c or _cache_q8()) if q8 else (L.rope_kv_append, c or _cache())
        return fn(ctypes.byref(q), ctypes.byref(k), ctypes.byref(v or k), pos, 5, FAKE, rot, 0, 1.0,
                  ctypes.byref(qo or q), ctypes.byref(c), bt, bts, mb, sp, ws, 256, None)
    for q8 in (False, True):
        assert call(k=_t([2, 4, 5, 128]), q8=q8) == INVALID  # heads differ from the cache
        assert call(k=_t([2, 8, 6, 128]), q8=q8) == INVALID  # tokens differ
        assert call(v=_t([2, 8, 5, 128], 0), q8=q8) == INVALID
        assert call(q=_t([2, 30, 5, 128]), q8=q8) == INVALID  # 30 % 8
        assert call(q=_t([2, 32, 5, 128], 0), q8=q8) == UNSUPPORTED  # f32
        assert call(qo=_t([2, 32, 4, 128]), q8=q8) == INVALID
        assert call(rot=130, q8=q8) == INVALID
        assert call(sp=None, q8=q8) == INVALID
        assert call(bt=None, q8=q8) == INVALID
        assert call(bts=9, q8=q8) == INVALID
        assert call(mb=0, q8=q8) == INVALID
        assert call(ws=None, q8=q8) == WORKSPACE
        assert call(q=_t([2, 32, 0, 128]), k=_t([2, 8, 0, 128]), q8=q8) == OK
    assert call(c=_cache(bs=32)) == UNSUPPORTED
    assert call(rot=40, q8=True) == UNSUPPORTED  # half layout, 20 pairs
    assert call(q=_t([2, 32, 5, 128], data=FAKE + 2), q8=True) == UNSUPPORTED  # rows not 16-byte aligned


def test_binding_checks():
    x = torch.zeros(2, 4, 5, 64, dtype=torch.bfloat16)
    pos, fr = torch.zeros(2, 5, dtype=torch.int32), torch.zeros(32, dtype=torch.int64)
    with pytest.raises(ValueError, match="positions must be int32"):
        lib.rope_apply(x, pos.long(), fr)
    with pytest.raises(ValueError, match=r"positions must be \[2, 5\]"):
        lib.rope_apply(x, pos[:, :4], fr)
    with pytest.raises(ValueError, match="freqs must be contiguous int64"):
        lib.rope_apply(x, pos, fr.float())
    with pytest.raises(ValueError, match="freqs must hold 1 to 32 pairs, got 33"):
        lib.rope_apply(x, pos, torch.zeros(33, dtype=torch.int64))
    with pytest.raises(ValueError, match="out must be"):
        lib.rope_apply(x, pos, fr, out=x[:, :, :4])
    with pytest.raises(ValueError, match="must be on a CUDA device"):
        lib.rope_apply(x, pos, fr)


def test_marshalling(rec):  # noqa: F811
    B, Hq, Hkv, D, T = 2, 8, 2, 128, 3
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    kc, kq, sc = bf(10, Hkv, 16, D), torch.zeros(10, Hkv, 16, D, dtype=torch.int8), torch.zeros(10, Hkv, 16)
    bt, one = torch.zeros(B, 4, dtype=torch.int32), torch.ones(B, dtype=torch.int32)
    pos, fr = torch.zeros(B, T, dtype=torch.int32), torch.zeros(D // 2, dtype=torch.int64)
    lib.rope_apply(bf(B, Hq, T, D), pos, fr, stream=0)
    assert lib.rope_apply(bf(B, Hq, D), pos[:, 0], fr, interleaved=True, inverse=True, stream=0).shape == (B, Hq, D)
    k = bf(B, Hkv, T, D)
    lib.rope_kv_append(bf(B, Hq, T, D), k, k, pos, fr, kc, kc, bt, one, stream=0)
    lib.rope_kv_append(bf(B, Hq, D), k[:, :, 0], k[:, :, 0], pos[:, 0], fr, kc, kc, bt, one, stream=0)
    lib.rope_kv_append_q8(bf(B, Hq, T, D), k, k, pos, fr, kq, kq, sc, sc, bt, one, stream=0)
    assert rec.calls == ["rope_apply", "rope_apply", "rope_kv_append", "rope_kv_append", "rope_kv_append_q8"]
