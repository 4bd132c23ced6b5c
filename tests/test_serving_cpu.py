"""Checks of the shared-prefix decode, the rotary queries and the rotating appends that need no GPU: argument
checks on the host, the sizes a caller plans with, the frequencies, and the plain 64-bit forms themselves."""
import ctypes
import math

import numpy as np
import pytest
import torch

import mla_decode_attention_14_b200 as mla
import oracle
from mla_decode_attention_14_b200 import build as mla_build
from mla_decode_attention_14_b200 import workloads as W
from tests import plain_serving as plain

FAKE = 1 << 20  # a 256-aligned non-null address; never dereferenced (validation fails first)


@pytest.fixture(scope="module")
def L():
    mla_build.build()
    return mla.lib()


# ---------------------------------------------------------------- shared-prefix decode

def _shared(L, **kw):
    a = dict(q=FAKE, kv=FAKE, nblk=10, st=FAKE, sb=2, bt=FAKE, bts=4, sl=FAKE, tm=FAKE, ns=FAKE, P=4, b=2, s_q=1,
             h_q=16, scale=0.1, causal=0, out=FAKE, lse=FAKE, ws=FAKE, wsb=1 << 40)
    a.update(kw)
    return L.mla_decode_shared(a["q"], a["kv"], a["nblk"], a["st"], a["sb"], a["bt"], a["bts"], a["sl"], a["tm"], a["ns"],
                               a["P"], a["b"], a["s_q"], a["h_q"], a["scale"], a["causal"], a["out"], a["lse"], a["ws"],
                               a["wsb"], None)


@pytest.mark.parametrize("bad", [
    dict(q=None), dict(kv=None), dict(st=None), dict(bt=None), dict(sl=None), dict(tm=None), dict(ns=None), dict(out=None),
    dict(lse=None), dict(ws=None), dict(q=FAKE + 8), dict(kv=FAKE + 2), dict(out=FAKE + 8), dict(ws=FAKE + 128),
    dict(st=FAKE + 2), dict(bt=FAKE + 1), dict(b=0), dict(b=65537), dict(s_q=0), dict(h_q=1025), dict(P=0), dict(P=65536),
    dict(nblk=0), dict(nblk=1 << 31), dict(bts=0), dict(sb=-1), dict(sb=(1 << 24) + 1), dict(scale=float("nan")),
    dict(scale=float("inf")), dict(scale=-0.5), dict(causal=2),
])
def test_shared_decode_refuses(L, bad):
    assert _shared(L, **bad) == 1  # MLA_ERR_INVALID_ARG


def test_shared_decode_refuses_a_small_workspace(L):
    need = L.mla_shared_workspace_bytes(2, 1, 16, 2, 4)
    assert _shared(L, wsb=need - 1) == 3  # MLA_ERR_WORKSPACE
    assert _shared(L, wsb=need) in (2, 4)  # every check passed: no B200 here
    assert _shared(L, wsb=need, st=None, sb=0) in (2, 4)  # no prefix needs no table


@pytest.mark.parametrize("bad", [dict(sl=None), dict(tm=None), dict(ns=None), dict(b=0), dict(P=0), dict(C=-1), dict(sb=-1),
                                 dict(sl=FAKE + 2), dict(h_q=0)])
def test_shared_metadata_refuses(L, bad):
    a = dict(sl=FAKE, b=4, s_q=1, h_q=16, sb=2, P=4, C=2, tm=FAKE, ns=FAKE)
    a.update(bad)
    assert L.mla_get_metadata_shared(a["sl"], a["b"], a["s_q"], a["h_q"], a["sb"], a["P"], a["C"], a["tm"], a["ns"], None) == 1


@pytest.mark.parametrize("b,s_q,h_q,sb", [(1, 1, 16, 3), (64, 1, 16, 3), (33, 1, 64, 9), (5, 3, 40, 1), (9, 2, 96, 2),
                                          (7, 1, 128, 4), (3, 2, 128, 4), (6, 1, 16, 0)])
def test_shared_units_and_workspace(L, b, s_q, h_q, sb):
    rows = s_q * h_q
    prefix = math.ceil(b * rows / 128) if sb and rows % 128 else 0
    own = b * math.ceil(rows / 128)
    assert L.mla_shared_units(b, s_q, h_q, sb) == prefix + own
    for P in (1, 74):
        slots = ((prefix + P) * 128 if prefix else 0) + (own + P) * min(rows, 128)
        assert L.mla_shared_workspace_bytes(b, s_q, h_q, sb, P) == (slots * 513 * 4 + 255) // 256 * 256
    assert L.mla_shared_units(0, s_q, h_q, sb) == 0 and L.mla_shared_workspace_bytes(b, s_q, h_q, sb, 0) == 0


def test_plain_shared_decode_is_the_oracle_s_decode():
    """The plain form equals the oracle's paged decode over tables that begin with the shared one."""
    lens = np.array([0, 5, 128, 129, 300], np.int32)
    rng = np.random.default_rng(3)
    table, bt = rng.permutation(12).astype(np.int32), np.full((5, 5), -1, np.int32)
    bt[:, :2], shared = table[:2], table[:2]
    bt[3, 2], bt[4, 2:5] = table[2], table[3:6]
    kv = W.f32_to_bf16_bits(rng.standard_normal((12, 64, 1, 576), dtype=np.float32))
    q = W.f32_to_bf16_bits(rng.standard_normal((5, 2, 4, 576), dtype=np.float32))
    ro, rl = oracle.decode(q, kv, bt, lens, W.SCALE, True)
    f = lambda a: W.bf16_bits_to_f32(a).astype(np.float64)  # noqa: E731
    own = bt.copy()
    own[:, :2] = -1
    o, l, mix, span = plain.decode_shared(f(q), f(kv).reshape(-1, 64, 576), shared, own, lens, W.SCALE, True)
    assert np.allclose(o, ro, rtol=0, atol=1e-12)
    assert np.array_equal(np.isneginf(l), np.isneginf(rl))
    assert np.allclose(np.where(np.isneginf(l), 0, l), np.where(np.isneginf(rl), 0, rl), rtol=0, atol=1e-12)


# ---------------------------------------------------------------- rotary positions

@pytest.mark.parametrize("kw", [dict(), dict(base=500000.0), dict(factor=4.0), dict(factor=40.0, original_len=4096),
                                dict(factor=8.0, original_len=8192, beta_fast=16.0, beta_slow=2.0),
                                dict(factor=2.0, original_len=1)])
def test_rope_frequencies(kw):
    r = mla.rope(**kw)
    f = plain.inv_freq(**kw)
    got = np.array([t / 2.0 ** 64 * 2 * math.pi for t in r.turns])
    # each turn is rounded to 2^-64 and computed in fp64
    assert np.all(np.abs(got - f) <= 1e-14 * f + 2.0 ** -61)
    assert r.magnitude == 1.0 and r.interleaved


@pytest.mark.parametrize("bad", [dict(base=1.0), dict(base=float("inf")), dict(base=float("nan")), dict(factor=0.5),
                                 dict(factor=float("nan")), dict(original_len=-1), dict(beta_slow=0.0),
                                 dict(beta_fast=0.5), dict(magnitude=float("nan")), dict(magnitude=1e39)])
def test_rope_refuses(bad):
    with pytest.raises(mla.MLAError):
        mla.rope(**bad)


def _rope_q(L, rope, **kw):
    a = dict(x=FAKE, ldx=2048, hx=128, y=FAKE, ldy=9216, hy=576, tokens=4, heads=16, pos=None, sl=FAKE, s_q=2)
    a.update(kw)
    return L.mla_rope_q(a["x"], a["ldx"], a["hx"], a["y"], a["ldy"], a["hy"], a["tokens"], a["heads"], a["pos"], a["sl"],
                        a["s_q"], rope, None)


def test_rope_q_refuses(L):
    r = mla.rope().ref
    for bad in (dict(x=None), dict(y=None), dict(sl=None), dict(x=FAKE + 8), dict(y=FAKE + 2), dict(ldx=2044), dict(hx=4),
                dict(ldy=9220), dict(hy=580), dict(ldx=-8), dict(hy=-576), dict(tokens=0), dict(tokens=(1 << 24) + 1),
                dict(heads=0), dict(heads=4097), dict(s_q=0), dict(s_q=3), dict(pos=FAKE + 2), dict(ldx=1 << 41),
                dict(hy=56), dict(ldy=56), dict(hy=0), dict(ldy=16 * 576 - 520)):
        assert _rope_q(L, r, **bad) == 1, bad
    assert _rope_q(L, None) == 1
    assert _rope_q(L, r) in (2, 4)
    assert _rope_q(L, r, hx=0, ldx=0) in (2, 4)               # one row for all
    assert _rope_q(L, r, ldy=64, hy=256) in (2, 4)            # heads outermost
    assert _rope_q(L, r, pos=FAKE, sl=None, s_q=0) in (2, 4)  # positions need neither


# ---------------------------------------------------------------- rotating appends

def _append(L, fp8, rope, **kw):
    a = dict(x=FAKE, ld=576, tokens=6, n=3, cu=None, w=FAKE, eps=1e-6, pos=None, kv=FAKE, nblk=10, scale=0.5, bt=FAKE, bts=4,
             sl=FAKE, b=2)
    a.update(kw)
    head = (a["x"], a["ld"], a["tokens"], a["n"], a["cu"], a["w"], a["eps"], rope, a["pos"], a["kv"], a["nblk"])
    tail = (a["bt"], a["bts"], a["sl"], a["b"], None)
    if fp8:
        return L.mla_append_kv_rope_fp8(*head, a["scale"], *tail)
    return L.mla_append_kv_rope(*head, *tail)


@pytest.mark.parametrize("fp8", [False, True])
def test_append_refuses(L, fp8):
    r = mla.rope().ref
    for bad in (dict(x=None), dict(kv=None), dict(bt=None), dict(sl=None), dict(x=FAKE + 8), dict(kv=FAKE + 8),
                dict(w=FAKE + 8), dict(cu=FAKE + 2), dict(pos=FAKE + 2), dict(bt=FAKE + 2), dict(ld=568), dict(ld=580),
                dict(ld=1 << 33), dict(tokens=-1), dict(tokens=(1 << 30) + 1), dict(n=-1), dict(n=4), dict(tokens=5),
                dict(eps=-1e-6), dict(eps=float("nan")), dict(b=0), dict(b=65537), dict(nblk=0), dict(bts=0)):
        assert _append(L, fp8, r, **bad) == 1, bad
    assert _append(L, fp8, None) == 1
    assert _append(L, fp8, r) in (2, 4)
    assert _append(L, fp8, r, w=None, eps=float("nan")) in (2, 4)  # eps is not used without a norm
    assert _append(L, fp8, r, cu=FAKE, n=-7, tokens=5) in (2, 4)   # nor n_new with cu_new
    if fp8:
        for s in (0.0, -1.0, float("nan"), float("inf"), 1e-45):
            assert _append(L, True, r, scale=s) == 1


def test_binding_refuses_cpu_tensors_and_wrong_shapes():
    bf, i32 = torch.bfloat16, torch.int32
    z = lambda *s, dt=bf: torch.zeros(s, dtype=dt)  # noqa: E731
    r = mla.rope()
    with pytest.raises(ValueError):
        mla.rope_q(z(2, 1, 4, 64), z(2, 1, 4, 576), r, seqlens=z(2, dt=i32))
    with pytest.raises(TypeError):
        mla.rope_q(z(2, 1, 4, 64, dt=torch.float32), z(2, 1, 4, 576), r, seqlens=z(2, dt=i32))
    with pytest.raises(ValueError):
        mla.append_kv_rope(z(2, 1, 576), z(4, 64, 1, 576), z(2, 3, dt=i32), z(2, dt=i32), r)
    with pytest.raises(TypeError):
        mla.append_kv_rope_fp8(z(2, 1, 576, dt=torch.float16), z(4, 64, 1, 640, dt=torch.uint8), z(2, 3, dt=i32), z(2, dt=i32),
                               0.5, r)
    meta = mla.SharedMetadata(z(4, 8, dt=i32), z(4, dt=i32), 4, 2, 16, 1, 0, 2)
    with pytest.raises(ValueError):
        mla.decode_shared(z(2, 1, 16, 576), z(4, 64, 1, 576), z(2, dt=i32), z(2, 3, dt=i32), z(2, dt=i32), 0.1, False, meta)
    with pytest.raises(ValueError):
        mla.get_metadata_shared(z(4, dt=i32), 16, 1, 2, num_parts=4)


def test_rotation_is_a_rotation():
    """The plain form against complex multiplication, and its inverse by the negative position."""
    x = np.random.default_rng(0).standard_normal((7, 64))
    pos, f = np.arange(7) * 1000, plain.inv_freq()
    y = plain.rotate(x, pos, f, True)
    z = (x[:, 0::2] + 1j * x[:, 1::2]) * np.exp(1j * pos[:, None] * f)
    assert np.allclose(y[:, 0::2], z.real) and np.allclose(y[:, 1::2], z.imag)
    assert np.allclose(plain.rotate(y, -pos, f, True), x)
    h = plain.rotate(np.concatenate([x[:, 0::2], x[:, 1::2]], axis=1), pos, f, False)
    assert np.allclose(h[:, :32], y[:, 0::2]) and np.allclose(h[:, 32:], y[:, 1::2])
