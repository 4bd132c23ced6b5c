"""GPU parity of the rotary queries and the rotating appends against plain 64-bit forms (needs a B200).

Tolerance of a rotated value y = a (x0 c - x1 s): the angle is off by at most 2^-26 turns (fp32 of its top 32
bits) plus the 2^-33 of their truncation, 2 pi 2^-26 < 2^-23 rad; sine, cosine, the magnitude and the two
products and their sum add at most 2^-22 relative to a (|x0| + |x1|); the result is rounded to bf16 once
(half a step, 2^-8 relative). A normed latent: the fp32 sum of squares, rsqrt and two products are within
2^-20 relative, then one rounding: bf16 2^-8, E4M3 2^-4 relative (half its smallest step 2^-10 absolute below
2^-6), so a stored value differs from the exactly rounded one only next to a border between two.
"""
import numpy as np
import pytest
import torch

import mla_decode_attention_14_b200 as mla
from mla_decode_attention_14_b200 import workloads as W
from tests import plain_serving as plain

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)


ROPES = [dict(interleaved=True), dict(interleaved=False),
         dict(interleaved=True, factor=40.0, original_len=4096, magnitude=1.3688879),
         dict(interleaved=False, factor=4.0, magnitude=1.0), dict(interleaved=False, base=500000.0)]


def freq_of(kw):
    return plain.inv_freq(**{k: v for k, v in kw.items() if k in ("base", "factor", "original_len")})


def bits(shape, seed, scale=1.0):
    b = W.f32_to_bf16_bits(np.random.default_rng(seed).standard_normal(shape, dtype=np.float32) * np.float32(scale))
    return b, W.bf16_bits_to_f32(b).astype(np.float64)


def up(b):
    return torch.from_numpy(b).view(torch.bfloat16).cuda()


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def rotated_close(got, x, pos, kw):
    mag = np.float64(np.float32(kw.get("magnitude", 1.0)))
    ref = plain.rotate(x, pos, freq_of(kw), kw["interleaved"], mag)
    size = np.abs(mag) * (np.abs(x[..., 0::2]) + np.abs(x[..., 1::2]) if kw["interleaved"]
                          else np.abs(x[..., :32]) + np.abs(x[..., 32:]))
    size = np.repeat(size, 2, axis=-1) if kw["interleaved"] else np.concatenate([size, size], axis=-1)
    err = np.abs(got - ref)
    assert np.all(err <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -21 * size), err.max()


@pytest.mark.parametrize("kw", ROPES)
@pytest.mark.parametrize("b,s_q,h", [(1, 1, 1), (1, 1, 16), (3, 2, 5), (7, 1, 128), (2, 9, 24), (40, 4, 17)])
def test_rope_q_rows(b, s_q, h, kw):
    xb, x = bits((b, s_q, h, 192), 1)
    qb, _ = bits((b, s_q, h, 576), 2)
    sl = np.random.default_rng(3).integers(0, 163840, b).astype(np.int32)
    sl[0] = -3  # counts as 0
    q = up(qb)
    got = mla.rope_q(up(xb)[..., 128:], q, mla.rope(**kw), seqlens=torch.from_numpy(sl).cuda())
    assert got.data_ptr() == q.data_ptr() and mla.check_status() == 0
    pos = np.maximum(sl, 0)[:, None] + np.arange(s_q)
    rotated_close(f64(q)[..., 512:], x[..., 128:], pos[..., None], kw)
    assert np.array_equal(q.view(torch.uint16).cpu().numpy()[..., :512], qb[..., :512])  # the latent dims stay


@pytest.mark.parametrize("kw", ROPES[:3])
def test_rope_q_packed_positions_in_place(kw):
    """Packed tokens, any int32 positions (negative and the largest ones among them), x = q[..., 512:]."""
    qb, qf = bits((301, 16, 576), 5)
    pos = np.random.default_rng(6).integers(-2 ** 31, 2 ** 31, 301).astype(np.int32)
    pos[:4] = [0, 1, 2 ** 31 - 1, -2 ** 31]
    q = up(qb)
    mla.rope_q(q[..., 512:], q, mla.rope(**kw), positions=torch.from_numpy(pos).cuda())
    assert mla.check_status() == 0
    x = qf[..., 512:]
    # the plain form's own fp64 angle is off by |p| f 2^-53 or more at these positions: far below the bound
    rotated_close(f64(q)[..., 512:], x, pos[:, None], kw)
    assert np.array_equal(q.view(torch.uint16).cpu().numpy()[..., :512], qb[..., :512])


def cache_case(new, had, fp8, seed, spare=3):
    rng = np.random.default_rng([seed, 9])
    w = [(a + b + 63) // 64 for a, b in zip(new, had)]
    blocks = sum(w) + spare
    perm, off = rng.permutation(blocks).astype(np.int32), 0
    bt = np.full((len(new), max(1, max(w)) + 1), -1, np.int32)
    for i, k in enumerate(w):
        bt[i, :k] = perm[off:off + k]
        off += k
    kv = (rng.integers(0, 256, (blocks, 64, 1, 640)).astype(np.uint8) if fp8 else
          W.f32_to_bf16_bits(rng.standard_normal((blocks, 64, 1, 576), dtype=np.float32)))
    return bt, kv


def e4m3(x):
    """Float64 to the nearest E4M3 value, ties to even, saturated."""
    step = 2.0 ** (np.maximum(np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -30))), -6) - 3)
    return np.clip(np.round(x / step) * step, -448, 448)


def check_cache(kv, before, bt, new, had, x, kw, weight, eps, fp8, kv_scale, pos=None):
    rows, seqpos = [], []
    for b, (n, h) in enumerate(zip(new, had)):
        for t in range(n):
            p = max(h, 0) + t
            rows.append(int(bt[b, p // 64]) * 64 + p % 64)
            seqpos.append(p)
    pos = np.array(seqpos) if pos is None else pos
    mag = np.float64(np.float32(kw.get("magnitude", 1.0)))
    ref = plain.append_values(x, pos, freq_of(kw), kw["interleaved"], mag, weight, eps)
    got = kv.cpu()
    untouched = np.ones(before.shape[0] * 64, bool)
    untouched[rows] = False
    flat = got.view(torch.uint8).reshape(before.shape[0] * 64, -1).numpy()
    assert np.array_equal(flat[untouched], before.view(np.uint8).reshape(flat.shape)[untouched])
    mine = torch.from_numpy(flat[rows].copy())
    if fp8:
        lat = mine[:, :512].view(torch.float8_e4m3fn).float().numpy().astype(np.float64)
        want = ref[:, :512] / np.float64(np.float32(kv_scale))
        # within the rounding of a value that may be 2^-19 off
        slack = np.abs(want) * 2.0 ** -19
        ok = (lat >= e4m3(want - slack)) & (lat <= e4m3(want + slack))
        assert ok.all(), (int((~ok).sum()), lat[~ok][:4], want[~ok][:4])
        rot = mine[:, 512:].contiguous().view(torch.bfloat16)
    else:
        mine = mine.view(torch.bfloat16)
        lat, want = f64(mine[:, :512]), ref[:, :512]
        if weight is None:
            assert np.array_equal(lat, want)
        assert np.all(np.abs(lat - want) <= (2.0 ** -8 + 2.0 ** -19) * np.abs(want))
        rot = mine[:, 512:]
    rotated_close(f64(rot), x[:, 512:], pos, kw)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("kw", ROPES[:3])
@pytest.mark.parametrize("norm", [False, True])
def test_append_uniform(fp8, kw, norm):
    """Tokens that stay in a block, cross into a new one, or start one; strided rows."""
    had, n_new = [5, 62, 64, 130, 0, 63], 3
    new = [n_new] * len(had)
    bt, before = cache_case(new, had, fp8, 1)
    xb, x = bits((len(had), n_new, 640), 2)
    wb, w = bits((512,), 3, 0.5)
    kv = torch.from_numpy(before.copy()).cuda() if fp8 else up(before.copy())
    args = (up(xb)[..., :576], kv, torch.from_numpy(bt).cuda(), torch.tensor(had, dtype=torch.int32).cuda())
    more = dict(norm_weight=up(wb) if norm else None, eps=1e-5)
    if fp8:
        mla.append_kv_rope_fp8(*args, 0.0123, mla.rope(**kw), **more)
    else:
        mla.append_kv_rope(*args, mla.rope(**kw), **more)
    assert mla.check_status() == 0
    check_cache(kv, before, bt, new, had, x[..., :576].reshape(-1, 576), kw, w if norm else None, 1e-5, fp8, 0.0123)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("batch", [1, 2, 33, 1500])
def test_append_packed(fp8, batch):
    """Ragged prompts with empty ones among them, explicit positions, rows behind the last sequence left alone."""
    rng = np.random.default_rng(batch)
    new = [int(v) for v in rng.integers(0, 5 if batch > 100 else 90, batch)]
    new[0], new[-1] = max(new[0], 1), 0 if batch > 1 else max(new[-1], 1)
    had = [int(v) for v in rng.integers(0, 70, batch)]
    bt, before = cache_case(new, had, fp8, 4)
    total = sum(new)
    xb, x = bits((total + 5, 576), 5)
    pos = rng.integers(0, 1 << 20, total + 5).astype(np.int32)
    cu = torch.from_numpy(np.concatenate([[0], np.cumsum(new)]).astype(np.int32)).cuda()
    wb, w = bits((512,), 6)
    kv = torch.from_numpy(before.copy()).cuda() if fp8 else up(before.copy())
    args = (up(xb), kv, torch.from_numpy(bt).cuda(), torch.tensor(had, dtype=torch.int32).cuda())
    more = dict(norm_weight=up(wb), positions=torch.from_numpy(pos).cuda(), cu_new=cu)
    if fp8:
        mla.append_kv_rope_fp8(*args, W.F8_SCALE, mla.rope(**ROPES[1]), **more)
    else:
        mla.append_kv_rope(*args, mla.rope(**ROPES[1]), **more)
    assert mla.check_status() == 0
    check_cache(kv, before, bt, new, had, x[:total], ROPES[1], w, 1e-6, fp8, W.F8_SCALE, pos[:total])
