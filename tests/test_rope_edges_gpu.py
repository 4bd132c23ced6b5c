"""Edges of the rotary kernels on a B200: positions at the ends of int32 against angles reduced in 160-bit integers.

Tolerance of y = a (x0 c - x1 s), relative to a (|x0| + |x1|): the angle is off by 2^-26 turns (fp32 of its top 32
bits), their truncation (2^-32) and the frequency (2^-32), in all 2 pi (2^-26 + 2^-31) < 2^-23.3 rad; sine and
cosine by an ulp (2^-24); the magnitude, the two products and their sum round by 2^-24 each: 2^-23.3 + 4 * 2^-24 <
2^-21.5. Then one rounding to bf16 (2^-8 of the value; relative to the rounded one, 2^-8 of the bound more).
"""
import numpy as np
import pytest
import torch

import mla_decode_attention_14_b200 as mla
from tests import exact_rope
from tests.test_rope_gpu import bits, f64, up

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
