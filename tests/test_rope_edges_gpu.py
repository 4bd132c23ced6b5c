"""Edges of the rotary kernels on a B200: positions at the ends of int32 against angles reduced in 160-bit integers,
latents of every size and of no numbers.

Tolerance of y = a (x0 c - x1 s), relative to a (|x0| + |x1|): the angle is off by 2^-26 turns (fp32 of its top 32
bits), their truncation (2^-32) and the frequency (2^-32), in all 2 pi (2^-26 + 2^-31) < 2^-23.3 rad; sine and
cosine by an ulp (2^-24); the magnitude, the two products and their sum round by 2^-24 each: 2^-23.3 + 4 * 2^-24 <
2^-21.5. Then one rounding to bf16 (2^-8 of the value; relative to the rounded one, 2^-8 of the bound more).
"""
import numpy as np
import pytest
import torch

import mla_decode_attention_14_b200 as mla
from mla_decode_attention_14_b200 import workloads as W
from tests import exact_rope
from tests.test_rope_gpu import bits, e4m3, f64, up

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)


def rotated_close(got, x, ang, interleaved, mag):
    """got, x float64 [tokens, ..., 64]; ang [tokens][32]."""
    first, second = (slice(0, 64, 2), slice(1, 64, 2)) if interleaved else (slice(0, 32), slice(32, 64))
    a = np.asarray(ang).reshape((len(ang),) + (1,) * (x.ndim - 2) + (32,))
    x0, x1, size = x[..., first], x[..., second], mag * (np.abs(x[..., first]) + np.abs(x[..., second]))
    for part, ref in ((first, mag * (x0 * np.cos(a) - x1 * np.sin(a))), (second, mag * (x0 * np.sin(a) + x1 * np.cos(a)))):
        err = np.abs(got[..., part] - ref)
        assert np.all(err <= 2.0 ** -8 * np.abs(ref) + (1 + 2.0 ** -8) * 2.0 ** -21.5 * size), err.max()


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("kw", [dict(), dict(factor=40.0, original_len=4096), dict(base=500000.0, factor=8.0)])
def test_far_positions(kw, interleaved):
    rng = np.random.default_rng(2)
    pos = np.concatenate([[0, 1, -1, 2 ** 31 - 1, -2 ** 31, 2 ** 30, 10 ** 6],
                          rng.integers(-2 ** 31, 2 ** 31, 90), 2 ** 31 - 1 - rng.integers(0, 1000, 90)]).astype(np.int32)
    mag = float(np.float32(1.3688879))
    rope = mla.rope(interleaved=interleaved, magnitude=mag, **kw)
    qb, qf = bits((len(pos), 5, 576), 5)
    q = up(qb)
    d_pos = torch.from_numpy(pos).cuda()
    mla.rope_q(q[..., 512:], q, rope, positions=d_pos)
    xb, x = bits((len(pos), 576), 6)
    kv = torch.zeros((4, 64, 1, 576), dtype=torch.bfloat16, device="cuda")
    bt = torch.arange(4, dtype=torch.int32, device="cuda")[None]
    mla.append_kv_rope(up(xb)[None], kv, bt, torch.zeros(1, dtype=torch.int32, device="cuda"), rope, positions=d_pos)
    assert mla.check_status() == 0
    ang = exact_rope.angles(pos, **kw)
    rotated_close(f64(q)[..., 512:], qf[..., 512:], ang, interleaved, mag)
    rotated_close(f64(kv).reshape(-1, 576)[:len(pos), 512:], x[:, 512:], ang, interleaved, mag)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("eps", [0.0, 1e-30, 1e-6, 100.0])
def test_norm_of_every_size(fp8, interleaved, eps):
    """Rows of 2^-130 to 2^125, past where an fp32 sum of squares holds them, each beside ordinary ones; a row that one
    value rules. Before the rounding to the cache's type a value is off by an fp32 root and two products, or a
    double and two roundings: under 2^-19, as in tests/test_rope_gpu.py. bf16's own smallest step is 2^-133."""
    exps = np.array([0, -130, -126, -100, -80, -64, -51, -50, -49, -30, -1, 1, 30, 60, 62, 63, 64, 65, 90, 125])
    rng = np.random.default_rng(8)
    x = rng.standard_normal((len(exps) + 2, 576)).astype(np.float32)
    x[:len(exps), :512] = np.clip(x[:len(exps), :512], -3.9, 3.9) * np.ldexp(1.0, exps)[:, None].astype(np.float64)
    x[-2, 17] = 2.0 ** 100
    x[-1, 300] = -2.0 ** 63.5
    xb = W.f32_to_bf16_bits(x)
    xf = W.bf16_bits_to_f32(xb).astype(np.float64)
    wb, w = bits((512,), 9, 0.5)
    n, scale = len(x), 2.0 ** -6
    kv = torch.zeros((1, 64, 1, 640), dtype=torch.uint8, device="cuda") if fp8 else \
        torch.zeros((1, 64, 1, 576), dtype=torch.bfloat16, device="cuda")
    args = (up(xb)[None], kv, torch.zeros((1, 1), dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda"))
    rope, more = mla.rope(interleaved=interleaved), dict(norm_weight=up(wb), eps=eps)
    if fp8:
        mla.append_kv_rope_fp8(*args, scale, rope, **more)
    else:
        mla.append_kv_rope(*args, rope, **more)
    assert mla.check_status() == 0
    want = xf[:, :512] / np.sqrt((xf[:, :512] ** 2).mean(axis=1, keepdims=True) + np.float64(np.float32(eps))) * w
    rows = kv.view(64, -1)[:n]
    if fp8:
        lat = f64(rows[:, :512].contiguous().view(torch.float8_e4m3fn))
        slack = np.abs(want / scale) * 2.0 ** -19
        ok = (lat >= e4m3(want / scale - slack)) & (lat <= e4m3(want / scale + slack))
        rot = f64(rows[:, 512:].contiguous().view(torch.bfloat16))
    else:
        lat = f64(rows[:, :512])
        ok = np.abs(lat - want) <= (2.0 ** -8 + 2.0 ** -19) * np.abs(want) + 2.0 ** -134
        rot = f64(rows[:, 512:])
    assert ok.all(), sorted(set(np.argwhere(~ok)[:, 0].tolist()))
    rotated_close(rot, xf[:, 512:], exact_rope.angles(range(n)), interleaved, 1.0)
    assert not kv.view(64, -1)[n:].any()


@pytest.mark.parametrize("fp8", [False, True])
def test_norm_of_no_numbers(fp8):
    """As the formula has it: a NaN makes the row NaN; an infinity makes itself NaN and the rest 0; a row of zeros is
    0 * rsqrt(eps), NaN for eps = 0. The rows beside them are those of a call without them."""
    rng = np.random.default_rng(3)
    x = rng.standard_normal((6, 576)).astype(np.float32)
    x[1, 5], x[2, 500], x[4, :512] = np.nan, np.inf, 0.0
    xb = W.f32_to_bf16_bits(x)
    xb[1, 5] = W.BF16_NAN
    one = torch.ones(512, dtype=torch.bfloat16, device="cuda")
    at = (torch.zeros((1, 1), dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda"))

    def call(rows, eps):
        kv = torch.zeros((1, 64, 1, 640), dtype=torch.uint8, device="cuda") if fp8 else \
            torch.zeros((1, 64, 1, 576), dtype=torch.bfloat16, device="cuda")
        pos = torch.zeros(len(rows), dtype=torch.int32, device="cuda")
        if fp8:
            mla.append_kv_rope_fp8(up(rows)[None], kv, *at, 1.0, mla.rope(), norm_weight=one, eps=eps, positions=pos)
        else:
            mla.append_kv_rope(up(rows)[None], kv, *at, mla.rope(), norm_weight=one, eps=eps, positions=pos)
        lat = kv.view(64, -1)[:len(rows), :512]
        return (lat.contiguous().view(torch.float8_e4m3fn) if fp8 else lat).float().cpu()

    for eps in (1e-6, 0.0):
        lat = call(xb, eps)
        assert lat[1].isnan().all()
        assert lat[2, 500].isnan() and not lat[2, :500].any() and not lat[2, 501:].any()
        assert lat[4].isnan().all() if eps == 0.0 else not lat[4].any()
        assert torch.equal(lat[[0, 3, 5]], call(xb[[0, 3, 5]].copy(), eps))
    assert mla.check_status() == 0
