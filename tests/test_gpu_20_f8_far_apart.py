"""The e4m3 cache where numbers are far apart, against the 64-bit reference."""
import math

import numpy as np
import pytest
import torch

import masked_attention_paged_gb300 as lib
from _serve_ref import BS, attn_f8
from test_gpu_17_f8 import _codes, _ints

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _attn(q, codes, scales, table, start, scale):
    g = [_codes(c) for c in codes] + [torch.from_numpy(s).to(DEV) for s in scales]
    B, Hq, T, D = q.shape
    ws = lib.Workspace(lib.paged_attn_f8_workspace_size(B, Hq, codes[0].shape[1], T, table.shape[1], BS, D))
    out = torch.empty(q.shape, device=DEV)
    got, lse = lib.paged_attn_f8(q, *g, _ints(table), _ints(start), scale=scale, out=out, return_lse=True, workspace=ws)
    assert ws.status() == 0
    return got.double().cpu().numpy(), lse.double().cpu().numpy()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T,G", [(1, 1), (2, 8), (30, 1), (60, 4)])
@pytest.mark.parametrize("log2w", [-20, -25.5, -27, -30])
def test_a_long_tail_of_small_weights(log2w, T, G, D):
    """A key of each block has all the weight and a value of zero, the others 2^log2w of it: the output is theirs alone.

    A weight is off by its rounding, 2^-11 (bf16 2^-8, with more than 16 rows) relative or, fp16 below its normal
    numbers, 2^-32 of the largest; the sum that divides is that of all weights relative to the largest.  The rest as in
    _compare of the e4m3 tests: q's split and the additions of a score, the exponential."""
    rng = np.random.default_rng(D)
    N = 64
    codes = [np.zeros((N, 1, BS, D), np.uint8) for _ in range(2)]
    scales = [np.ones((N, 1), np.float32) for _ in range(2)]
    codes[0][:, 0, 0, 0] = 0x58  # 16
    codes[1][:, 0, 1:] = rng.integers(0x30, 0x40, (N, BS - 1, D))
    q = torch.zeros((1, G, T, D))
    q[..., 0] = -log2w * math.log(2.0) / 16
    q = q.to(DEV, torch.bfloat16)
    table, start = rng.permutation(N).astype(np.int32)[None], [N * BS - T]
    got, lse = _attn(q, codes, scales, table, start, 1.0)
    qn = q.double().cpu().numpy()
    ref, ref_lse, mag, all_v = attn_f8(qn, codes[0], scales[0], codes[1], scales[1], table, start, 1.0, True)
    ds = qn[..., 0] * 16 * (2.0 ** -19 + 4 * D * 2.0 ** -24) + 2.0 ** -22 * ref_lse
    w = 2 * np.expm1(2 * ds) + (2.0 ** -11 if T * G <= 16 else 2.0 ** -8) + 2.0 ** -18
    small = 2.0 ** -32 * np.exp(qn[..., 0] * 16 - ref_lse)[..., None] * all_v if T * G <= 16 else 0.0
    tol = w[..., None] * mag + np.abs(ref) * 2.0 ** -24 + small
    assert (np.abs(got - ref) <= tol).all(), (np.abs(got - ref) / np.abs(ref)).max()
    assert (np.abs(lse - ref_lse) <= 2 * ds + 2.0 ** -18).all()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T,G", [(1, 1), (1, 12), (20, 1), (60, 4)])
@pytest.mark.parametrize("nats", [12.0, 30.0, 36.0])
def test_scores_that_outgrow_the_first_keys_before_large_values(nats, T, G, D):
    """Values near 2^100, and keys from 300 on that score `nats` above all others: the weights that the first keys set
    the measure for must not carry the sums past float32's range."""
    rng = np.random.default_rng(T)
    B, Hkv, width = 48, 2, 40
    N = 60
    codes = [np.zeros((N, Hkv, BS, D), np.uint8) for _ in range(2)]
    scales = [np.ones((N, Hkv), np.float32), np.full((N, Hkv), 2.0 ** 92, np.float32)]
    codes[0][N // 2:, :, :, 0] = 0x58  # 16
    codes[1][...] = rng.integers(0x70, 0x7f, codes[1].shape) | (rng.integers(0, 2, codes[1].shape) * 128).astype(np.uint8)
    table = rng.integers(0, N // 2, (B, width)).astype(np.int32)
    table[:, 19:] += N // 2
    q = torch.zeros((B, Hkv * G, T, D))
    q[..., 0] = nats / 16
    q = q.to(DEV, torch.bfloat16)
    start = [width * BS - T - b for b in range(B)]
    got, lse = _attn(q, codes, scales, table, start, 1.0)
    assert np.isfinite(got).all()
    got, lse, qn = got[::6], lse[::6], q[::6].double().cpu().numpy()
    ref, ref_lse, mag, _ = attn_f8(qn, codes[0], scales[0], codes[1], scales[1], table[::6], start[::6], 1.0, True)
    ds = qn[..., 0] * 16 * (2.0 ** -19 + 4 * D * 2.0 ** -24) + 2.0 ** -22 * np.abs(ref_lse)
    w = 2 * np.expm1(2 * ds) + (2.0 ** -11 if T * G <= 16 else 2.0 ** -8) + 2.0 ** -18
    # (a weight below fp16's normal numbers is off by 2^-32 of the largest, of sums of 64 keys and more)
    assert (np.abs(got - ref) <= w[..., None] * mag + np.abs(ref) * 2.0 ** -24 + 2.0 ** -32 * 640 * 448 * 2.0 ** 92).all()
    assert (np.abs(lse - ref_lse) <= 2 * ds + 2.0 ** -18).all()


@pytest.mark.parametrize("D", [64, 128])
def test_a_block_that_begins_with_infinities_alone(D):
    """Scale 0, so their codes stand for 0; when later rows set a scale, code times old scale over new is 0 again (and
    a NaN stays one)."""
    N, H = 2, 2
    codes = [torch.zeros((N, H, BS, D), dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn) for _ in range(2)]
    scales = [torch.full((N, H), 3.0, device=DEV) for _ in range(2)]
    table = _ints([[1, 0]])
    new = torch.zeros((1, H, 3, D), device=DEV, dtype=torch.bfloat16)
    new[0, :, 0, ::2], new[0, :, 1, 1], new[0, :, 1, 2] = math.inf, -math.inf, math.nan
    lib.kv_append_f8(*codes, *scales, table, _ints([0]), new, -new)
    assert (scales[0][1] == 0).all() and (scales[1][1] == 0).all()
    rows = torch.full((1, H, 1, D), 3.0, device=DEV, dtype=torch.bfloat16)
    lib.kv_append_f8(*codes, *scales, table, _ints([3]), rows, rows)
    for c, s in zip(codes, scales):
        x = c[1].float() * s[1][:, None, None]
        want = torch.zeros((H, BS, D), device=DEV)
        want[:, 3] = 3.0
        want[:, 1, 2] = math.nan
        assert torch.equal(s[1], torch.full((H,), 2.0 ** -7, device=DEV))
        assert torch.equal(x.isnan(), want.isnan()) and torch.equal(x.nan_to_num(), want.nan_to_num())
