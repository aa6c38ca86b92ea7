"""The e4m3 cache on the GPU: appended codes and scales bit for bit, attention against the
64-bit reference within the roundings that the call states."""
import math

import numpy as np
import pytest
import torch

import masked_attention_paged_gb300 as lib
from _serve_ref import BS, E4M3, append_f8, attn_f8

pytestmark = pytest.mark.gpu
DEV = "cuda"
F8 = torch.float8_e4m3fn


def _ints(x):
    return torch.tensor(np.asarray(x, np.int32).copy(), device=DEV)


def _table(B, width, N, rng):
    return rng.permutation(N)[:B * width].reshape(B, width).astype(np.int32)


def _codes(x):
    return torch.from_numpy(x).to(DEV).view(F8)


def _bf(shape, rng, size=1.0):
    return (torch.from_numpy(rng.normal(size=shape).astype(np.float32)) * size).to(DEV, torch.bfloat16)


# --------------------------------------------------------------------------
# append
# --------------------------------------------------------------------------
def _append(codes, scales, table, start, rows, lens=None, **kw):
    """GPU and reference on the same state: ((K, V) codes and scales, status) both."""
    g = [_codes(c.copy()) for c in codes] + [torch.from_numpy(s.copy()).to(DEV) for s in scales]
    ws = lib.Workspace(256)
    lib.kv_append_f8(*g, _ints(table), _ints(start), *rows, lens=None if lens is None else _ints(lens), workspace=ws,
                     **kw)
    want_c, want_s, flag = [c.copy() for c in codes], [s.copy() for s in scales], False
    for i in range(2):
        x = rows[i] if rows[i].dim() == 4 else rows[i].unsqueeze(2)
        flag |= append_f8(want_c[i], want_s[i], table, start, x.float().cpu().numpy(), lens)
    for i in range(2):
        assert np.array_equal(g[2 + i].cpu().numpy(), want_s[i], equal_nan=True)
        got = g[i].view(torch.uint8).cpu().numpy()
        nan = np.isnan(E4M3[want_c[i]])
        assert np.array_equal(np.where(nan, 0, got), np.where(nan, 0, want_c[i]))
        assert np.isnan(E4M3[got[nan]]).all()  # of either sign
    assert ws.status() == (5 if flag else 0)
    return want_c, want_s


def _state(N, H, D, rng):
    codes = [rng.integers(0, 127, (N, H, BS, D)).astype(np.uint8) | (rng.integers(0, 2, (N, H, BS, D)) * 128
                                                                    ).astype(np.uint8) for _ in range(2)]
    return codes, [np.ldexp(1.0, rng.integers(-9, -3, (N, H))).astype(np.float32) for _ in range(2)]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B,T,H,start,lens", [
    (1, 1, 1, [0], None), (3, 1, 8, [16, 5, 15], None), (4, 2, 3, [15, 14, 0, 31], None),
    (2, 16, 2, [0, 1], None), (2, 17, 5, [15, 16], None), (3, 100, 4, [3, 0, 29], [100, 0, 41]),
    (5, 18, 2, [-1, 2, 7, 200, 33], [18, 30, -4, 18, 1]),
])
def test_append(D, B, T, H, start, lens):
    rng = np.random.default_rng(T + D)
    width = 13
    table = _table(B, width, B * width + 2, rng)
    codes, scales = _state(B * width + 2, H, D, rng)
    rows = [_bf((B, H, T, D), rng, s) for s in (1.0, 30.0)]
    _append(codes, scales, table, start, rows, lens)


def test_append_token_by_token_as_a_block_grows():
    """Rows of very different sizes into one block: the scale grows, the older codes are rounded again."""
    rng = np.random.default_rng(3)
    codes, scales = _state(4, 2, 64, rng)
    table, size = np.array([[2, 0]], np.int32), [1e-3, 2e-3, 1.0, 0.5, 500.0, 1e4, 1e-2, 0.0, 3e38, 1.0, 7.0] * 2
    for pos, x in enumerate(size[:20]):
        codes, scales = _append(codes, scales, table, [pos], [_bf((1, 2, 1, 64), rng, x) for _ in range(2)])


def test_append_values_at_the_borders():
    """Exactly 448 times a power of two, just above, halves between codes, subnormals of both types, zeros."""
    D, H = 64, 1
    vals = [448.0, 450.0, 447.0, 1.0, 1.0625, 1.1875, 2.0 ** -9, 2.0 ** -10, 3 * 2.0 ** -11, 2.0 ** -130, 2.0 ** -133, 0.0,
            -0.0, 3.3895e38, 1.17e-38, -1.5]
    rows = torch.zeros((len(vals), H, 3, D))
    for b, v in enumerate(vals):
        rows[b, 0, 0, :] = v
        rows[b, 0, 1, :8] = torch.tensor([1.0, 0.0625, 0.1, -3.0, 2.0 ** -8, 5 * 2.0 ** -11, 0.0, 17.0]) * v
    rng = np.random.default_rng(0)
    codes, scales = _state(len(vals), H, D, rng)
    table = np.arange(len(vals), dtype=np.int32)[:, None]
    x = rows.to(DEV, torch.bfloat16)
    _append(codes, scales, table, [0] * len(vals), [x, -x])
    _append(codes, scales, table, [4] * len(vals), [x, -x])


def test_append_infinities_and_nans_do_not_set_the_scale():
    rng = np.random.default_rng(6)
    codes, scales = _state(3, 2, 128, rng)
    rows = [_bf((1, 2, 20, 128), rng) for _ in range(2)]
    rows[0][0, 0, 3, 5] = math.inf
    rows[0][0, 1, 7, :] = -math.inf
    rows[1][0, 0, 1, 9] = math.nan
    rows[1][0, 1, 2:20] = math.nan
    _append(codes, scales, np.array([[1, 2]], np.int32), [5], rows)
    scales[0][1] = np.nan  # the scale of a block that begins anew is not looked at
    _append(codes, scales, np.array([[1, 2]], np.int32), [0], rows)


def test_append_strided_rows_bad_blocks_and_one_token():
    rng = np.random.default_rng(7)
    codes, scales = _state(9, 4, 128, rng)
    qkv = _bf((2, 5, 16, 128), rng).transpose(1, 2)  # a projection's output
    table = np.array([[3, -1, 8], [9, 0, 2]], np.int32)
    _append(codes, scales, table, [14, 30], [qkv[:, 8:12], qkv[:, 12:16]])
    one = _bf((2, 12, 128), rng)
    _append(codes, scales, table, [17, 3], [one[:, 4:8], one[:, 8:12]])


# --------------------------------------------------------------------------
# attention
# --------------------------------------------------------------------------
def _check(q, codes, scales, table, start, scale=None, causal=True, lens=None, dtype=torch.bfloat16, status=0, rows=None,
           **kw):
    B, Hq, T, D = q.shape
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    g = [_codes(c) for c in codes] + [torch.from_numpy(s).to(DEV) for s in scales]
    ws = lib.Workspace(lib.paged_attn_f8_workspace_size(B, Hq, codes[0].shape[1], T, table.shape[1], BS, D))
    out = torch.full(q.shape, 7.0, device=DEV, dtype=dtype)
    got, lse = lib.paged_attn_f8(q, *g, _ints(table), _ints(start), lens=None if lens is None else _ints(lens),
                                 causal=causal, scale=scale, out=out, return_lse=True, workspace=ws, **kw)
    assert ws.status() == status
    qn = q.double().cpu().numpy()
    ref, ref_lse, mag, all_v = attn_f8(qn, codes[0], scales[0], codes[1], scales[1], table, start, scale, causal, lens)
    _compare(got, lse, ref, ref_lse, mag, all_v, qn, codes, scales, scale, T * (Hq // codes[0].shape[1]), dtype)
    return got, lse


def _compare(got, lse, ref, ref_lse, mag, all_v, qn, codes, scales, scale, rows, dtype):
    """A score is off by q's split, 2^-19 of its row's largest element an element (against the largest |K| of a
    dimension), and by D float32 additions; a weight also by its rounding (fp16, with more than 16 rows bf16) and the
    exponential's 2^-21; the output by its type's.  fp16 weights below 2^-14 of the largest are multiples of 2^-24: off
    by 2^-25 at most, next to a sum of 1 or more (the reference maximum is never above the true one)."""
    D = qn.shape[-1]
    with np.errstate(invalid="ignore"):
        kmax = np.nanmax(np.abs(E4M3[codes[0]]) * scales[0][:, :, None, None])
    top = np.abs(qn).max(-1)
    ds = abs(scale) * top * kmax * D * (2.0 ** -19 + 4 * 2.0 ** -24)
    ds = np.minimum(ds, 1.0) + 2.0 ** -22 * np.abs(np.where(np.isfinite(ref_lse), ref_lse, 0.0))
    w = 2 * np.expm1(2 * ds) + (2.0 ** -11 if rows <= 16 else 2.0 ** -8) + 2.0 ** -18
    tol = w[..., None] * mag + np.abs(ref) * (torch.finfo(dtype).eps / 2) + (rows <= 16) * 2.0 ** -25 * all_v + 1e-30
    got, lse = got.double().cpu().numpy(), lse.double().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    assert (np.abs(got - ref)[~np.isnan(ref)] <= tol[~np.isnan(ref)]).all(), np.nanmax(np.abs(got - ref) - tol)
    assert np.array_equal(np.isneginf(lse), np.isneginf(ref_lse)) and np.array_equal(np.isnan(lse), np.isnan(ref_lse))
    fin = np.isfinite(ref_lse)
    assert (np.abs(lse - ref_lse)[fin] <= (ds * 2 + 2.0 ** -18)[fin]).all(), np.abs(lse - ref_lse)[fin].max()


def _cache(N, H, D, rng):
    """Normal rows at scales that differ from block to block, in codes."""
    from _serve_ref import to_e4m3
    codes, scales = [], []
    for _ in range(2):
        s = np.ldexp(1.0, rng.integers(-7, -4, (N, H))).astype(np.float32)
        x = rng.normal(size=(N, H, BS, D)) / s[:, :, None, None]
        codes.append(to_e4m3(x))
        scales.append(s)
    return codes, scales


SHAPES = [  # B, T, Hq, Hkv, D, start, lens
    (1, 1, 1, 1, 128, [0], None),
    (1, 1, 8, 1, 64, [16], None),
    (3, 1, 8, 2, 128, [0, 15, 700], None),
    (2, 1, 16, 2, 64, [1300, 31], None),
    (2, 1, 12, 4, 128, [2047, 2048], None),
    (2, 1, 16, 1, 128, [100, 333], None),     # 16 heads to a KV head
    (2, 1, 5, 1, 64, [64, 65], [1, 0]),
    (2, 2, 8, 2, 128, [17, 0], None),
    (2, 4, 12, 4, 128, [60, 1021], [4, 3]),
    (1, 16, 4, 4, 64, [5], None),
    (2, 5, 14, 2, 128, [129, 15], [5, 2]),    # 35 rows
    (1, 33, 8, 2, 128, [0], None),
    (2, 130, 4, 1, 64, [3, 250], [130, 77]),
    (1, 300, 3, 3, 128, [64], None),
    (3, 7, 32, 1, 128, [-1, 40, 13], None),
    (1, 3, 128, 1, 64, [20], None),           # 128 heads to a KV head
    (1, 257, 2, 1, 128, [700], None),
]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("B,T,Hq,Hkv,D,start,lens", SHAPES)
def test_attention(B, T, Hq, Hkv, D, start, lens, causal):
    rng = np.random.default_rng(B * 1000 + T)
    width = (max(start) + T + BS - 1) // BS + 1
    N = B * width + 1
    codes, scales = _cache(N, Hkv, D, rng)
    table = _table(B, width, N, rng)
    q = _bf((B, T, Hq, D), rng).transpose(1, 2)
    _check(q, codes, scales, table, start, causal=causal, lens=lens, dtype=torch.float32 if T % 2 else torch.bfloat16)


@pytest.mark.parametrize("T", [1, 6, 150])
def test_what_unused_slots_hold_does_not_matter(T):
    """NaN codes in every slot past the context, NaN scales in the blocks past it, and any ids there."""
    rng = np.random.default_rng(T)
    B, Hq, Hkv, D, start = 2, 8, 2, 128, [37, 5]
    width = 20
    codes, scales = _cache(B * width, Hkv, D, rng)
    table = _table(B, width, B * width, rng)
    for b in range(B):
        end = start[b] + T
        for i in range(width):
            lo = max(0, end - i * BS)
            for c, s in zip(codes, scales):
                c[table[b, i], :, min(lo, BS):] = 0x7f
                if lo <= 0:
                    s[table[b, i]] = np.nan
        table[b, -(-end // BS):] = [-1, 10 ** 9][b]
    q = _bf((B, Hq, T, D), rng)
    _check(q, codes, scales, table, start)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T,G", [(3, 2), (4, 4), (40, 2), (200, 1)])
def test_a_nan_reaches_the_rows_that_see_it_alone(T, G, D):
    rng = np.random.default_rng(T * G)
    B, Hkv, start = 2, 2, [30, 7]
    width = (30 + T) // BS + 2
    codes, scales = _cache(B * width, Hkv, D, rng)
    table = _table(B, width, B * width, rng)
    at = lambda b, t: (table[b, t // BS], t % BS)  # noqa: E731
    x, y = at(0, start[0] + T - 1), at(0, start[0] + T // 2)
    codes[1][x[0], 0, x[1], 3] = 0x7f
    codes[1][y[0], 1, y[1], [0, 9, D - 1]] = 0xff
    z = at(1, start[1] + T - 2)
    codes[0][z[0], 1, z[1], 4] = 0x7f  # a key
    q = _bf((B, Hkv * G, T, D), rng)
    _check(q, codes, scales, table, start, dtype=torch.float32)
    w = at(1, 2)
    codes[1][w[0], 1, w[1], 5] = 0x7f  # in the context of all rows
    _check(q, codes, scales, table, start, dtype=torch.float32)


@pytest.mark.parametrize("T", [1, 50])
def test_queries_that_are_not_finite(T):
    rng = np.random.default_rng(1)
    codes, scales = _cache(8, 2, 64, rng)
    q = _bf((1, 4, T, 64), rng)
    q[0, 1, 0, 3] = math.nan
    q[0, 2, 0, 60] = math.nan
    _check(q, codes, scales, np.arange(8, dtype=np.int32)[None], [60])


@pytest.mark.parametrize("T", [1, 40])
@pytest.mark.parametrize("ke,ve", [(-126, 0), (0, -126), (20, 100), (-3, 60), (90, -100)])
def test_scales_of_any_size(T, ke, ve):
    """Blocks of zeros (scale 0), and scales at the ends of their range; q and scale make up for the keys'."""
    rng = np.random.default_rng(T)
    codes, scales = _cache(12, 2, 128, rng)
    scales[0] = np.ldexp(np.float32(1.0), np.full(scales[0].shape, ke)).astype(np.float32)
    scales[1] = np.ldexp(1.0, ve - rng.integers(0, 8, scales[1].shape)).astype(np.float32)
    codes[0][3], scales[0][3], codes[1][4], scales[1][4] = 0, 0, 0, 0
    q = _bf((1, 8, T, 128), rng)
    _check(q, codes, scales, rng.permutation(12).astype(np.int32)[None], [150], scale=2.0 ** (-ke - 9),
           dtype=torch.float32)


@pytest.mark.parametrize("T", [1, 40])
@pytest.mark.parametrize("size,scale", [(1e30, 1e-31), (1e-30, 1e29), (1.0, -0.3), (1.0, 0.0), (60.0, 0.2)])
def test_queries_of_any_size(T, size, scale):
    rng = np.random.default_rng(2)
    codes, scales = _cache(24, 2, 128, rng)
    q = _bf((2, 8, T, 128), rng, size)
    _check(q, codes, scales, rng.permutation(24).astype(np.int32).reshape(2, 12), [150, 19], scale=scale,
           dtype=torch.float32)


def test_a_row_with_elements_of_all_sizes():
    """Elements down to 2^-19 of the row's largest, and one key direction each."""
    D = 128
    q = torch.zeros((1, 1, 1, D))
    q[0, 0, 0] = torch.tensor([(-1) ** d * (1.0 + (d % 5) / 4.0) * 2.0 ** -(d % 22) for d in range(D)])
    rng = np.random.default_rng(0)
    codes, scales = _cache(20, 1, D, rng)
    _check(q.to(DEV, torch.bfloat16), codes, scales, np.arange(20, dtype=np.int32)[None], [310], dtype=torch.float32)


@pytest.mark.parametrize("T", [1, 30])
def test_many_small_weights_next_to_a_large_one(T):
    """A sink with most of the weight, thousands of tokens with 2^-20 of it each, which together matter."""
    rng = np.random.default_rng(4)
    D, N = 64, 600
    codes = [np.zeros((N, 1, BS, D), np.uint8) for _ in range(2)]
    scales = [np.ones((N, 1), np.float32) for _ in range(2)]
    codes[0][0, 0, 0, 0] = 0x38 + 0x20  # 16.0 in the first key
    codes[1][...] = rng.integers(0x30, 0x40, codes[1].shape)
    q = torch.zeros((1, 1, T, D))
    q[..., 0] = 13.86 / 16
    _check(q.to(DEV, torch.bfloat16), codes, scales, np.arange(N, dtype=np.int32)[None], [N * BS - T], scale=1.0,
           dtype=torch.float32)


@pytest.mark.parametrize("T", [1, 20])
def test_positions_past_the_table_and_bad_blocks(T):
    rng = np.random.default_rng(5)
    codes, scales = _cache(20, 2, 128, rng)
    table = rng.permutation(20).astype(np.int32).reshape(4, 5)
    q = _bf((4, 4, T, 128), rng)
    start = [80 - T, 81 - T, -5, 2 ** 31 - 1]
    _check(q, codes, scales, table, start, status=5)
    table[0, 1], table[1, 0] = -1, 20
    _check(q, codes, scales, table, [60, 50, 3, 2], status=5)


def test_outputs_with_strides_and_one_token_rows():
    rng = np.random.default_rng(8)
    codes, scales = _cache(30, 2, 128, rng)
    table = rng.permutation(30).astype(np.int32).reshape(3, 10)
    g = [_codes(c) for c in codes] + [torch.from_numpy(s).to(DEV) for s in scales]
    start = [100, 7, 55]
    for T in (1, 24):
        qkv = _bf((3, T, 12, 128), rng)
        q = qkv[:, :, :8].transpose(1, 2)
        big = torch.full((3, T, 10, 128), 5.0, device=DEV, dtype=torch.bfloat16)
        out = big[:, :, 1:9].transpose(1, 2)
        lib.paged_attn_f8(q, *g, _ints(table), _ints(start), out=out)
        want = lib.paged_attn_f8(q.contiguous(), *g, _ints(table), _ints(start))
        assert torch.equal(out, want) and (big[:, :, 0] == 5).all() and (big[:, :, 9] == 5).all()
        if T == 1:
            rows = lib.paged_attn_f8(q[:, :, 0], *g, _ints(table), _ints(start))
            assert torch.equal(rows, want[:, :, 0])


@pytest.mark.parametrize("T", [1, 3, 40])
def test_captured_replayed_and_on_two_streams(T):
    rng = np.random.default_rng(9)
    B, Hq, Hkv, D, width = 2, 8, 2, 128, 130
    codes, scales = _cache(B * width, Hkv, D, rng)
    g = [_codes(c) for c in codes] + [torch.from_numpy(s).to(DEV) for s in scales]
    table, start = _ints(_table(B, width, B * width, rng)), _ints([1900, 40])
    q = _bf((B, Hq, T, D), rng)
    size = lib.paged_attn_f8_workspace_size(B, Hq, Hkv, T, width, BS, D)
    ws = [lib.Workspace(size) for _ in range(2)]
    ws[1].tensor[256:].random_(0, 256)  # nothing in it counts
    call = lambda i, **kw: lib.paged_attn_f8(q, *g, table, start, return_lse=True, workspace=ws[i], **kw)  # noqa: E731
    want = call(0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call(1)
    for first in (1900, 3, 700, 1900):
        start[0] = first
        want = call(0)
        for _ in range(3):
            graph.replay()
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = [[call(i, stream=s) for _ in range(20)] for i, s in enumerate(streams)]
    torch.cuda.synchronize()
    for o, l in outs[0] + outs[1]:
        assert torch.equal(o, want[0]) and torch.equal(l, want[1])


def test_a_cache_whose_offsets_pass_32_bits():
    """Codes past 4 GB: the last blocks of a large pool."""
    D, H, N = 128, 8, 270000  # 16 KB a block
    kq, vq = (torch.zeros((N, H, BS, D), dtype=torch.uint8, device=DEV).view(F8) for _ in range(2))
    ks, vs = (torch.zeros((N, H), device=DEV) for _ in range(2))
    rng = np.random.default_rng(1)
    far = np.array([[N - 1, 3, N - 7]], np.int32)
    near = np.array([[0, 3, 1]], np.int32)
    for T in (1, 30):
        kn, vn, q = _bf((1, H, T, D), rng), _bf((1, H, T, D), rng), _bf((1, 2 * H, T, D), rng)
        outs = []
        for table in (far, near):
            lib.kv_append_f8(kq, vq, ks, vs, _ints(table), _ints([3]), kn, vn)
            outs.append(lib.paged_attn_f8(q, kq, vq, ks, vs, _ints(table), _ints([3])))
        assert torch.equal(*outs) and outs[0].abs().max() > 0


@pytest.mark.parametrize("T", [1, 64])
def test_it_equals_the_bf16_call_on_the_values(T):
    """Values are exact in bf16, so the bf16 cache's calls see the same numbers."""
    rng = np.random.default_rng(12)
    B, Hq, Hkv, D, width = 3, 8, 2, 128, 40
    codes, scales = _cache(B * width, Hkv, D, rng)
    k, v = ((_codes(c).float() * torch.from_numpy(s).to(DEV)[:, :, None, None]) for c, s in zip(codes, scales))
    kb, vb = k.bfloat16(), v.bfloat16()
    assert torch.equal(kb.float(), k) and torch.equal(vb.float(), v)
    table, start = _ints(_table(B, width, B * width, rng)), [500, 33, 0]
    q = _bf((B, Hq, T, D), rng)
    want, want_lse = lib.paged_prefill_attn(q, kb, vb, table, _ints(start), return_lse=True)
    got, lse = lib.paged_attn_f8(q, *[_codes(c) for c in codes], *[torch.from_numpy(s).to(DEV) for s in scales], table,
                                 _ints(start), return_lse=True)
    # both round weights (bf16 there) and outputs: |v| <= 8
    assert (got.float() - want.float()).abs().max() <= 8 * 2.0 ** -8 + 2 * want.float().abs().max() * 2.0 ** -8
    assert (lse - want_lse).abs().max() <= 1e-4


@pytest.mark.parametrize("T,Hkv,G,D", [(1, 1, 2, 64), (1, 3, 1, 128), (2, 4, 2, 64), (1, 6, 2, 128), (1, 12, 1, 64),
                                       (1, 16, 1, 64), (3, 8, 4, 64), (20, 2, 1, 64), (70, 1, 2, 128)])
def test_many_sequences_most_of_them_idle(T, Hkv, G, D):
    """More of them than a warp looks at in one step, with long gaps: before, between and behind."""
    rng = np.random.default_rng(T * Hkv)
    B, width, N = 175, 8, 90
    codes, scales = _cache(N, Hkv, D, rng)
    table = rng.integers(0, N, (B, width)).astype(np.int32)
    start = rng.integers(0, width * BS - T, B).astype(np.int32)
    lens = rng.integers(0, T + 1, B).astype(np.int32)
    start[rng.random(B) < 0.4] = -1
    start[:35] = -1
    start[80:150] = -1
    lens[85:120] = 0
    lens[-3:] = 0
    _check(_bf((B, Hkv * G, T, D), rng), codes, scales, table, start, lens=lens)
    # one sequence at the end of them all
    start[:-4] = -1
    start[-4], lens[-4] = 100 - T, T
    _check(_bf((B, Hkv * G, T, D), rng), codes, scales, table, start, lens=lens)


@pytest.mark.parametrize("T,Hkv,G,D", [(1, 2, 1, 64), (2, 1, 6, 128), (5, 1, 4, 64)])
def test_a_large_batch_of_short_sequences(T, Hkv, G, D):
    """More items than warps: most runs hold several whole ones."""
    rng = np.random.default_rng(T)
    B, width, N = 2100, 3, 50
    codes, scales = _cache(N, Hkv, D, rng)
    start = rng.integers(-1, width * BS - T + 1, B).astype(np.int32)
    _check(_bf((B, Hkv * G, T, D), rng), codes, scales, rng.integers(0, N, (B, width)).astype(np.int32), start)
