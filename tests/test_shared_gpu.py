"""GPU parity of the shared-prefix decode against a plain 64-bit form (needs a B200).

Tolerances, from the roundings it makes: the probabilities are rounded to bf16 for the second product (half
a step: 2^-8 of each term, so 2^-8 sum_j p_j |v_j| in all) and the result to bf16 (2^-8 |out|). A score is
a sum of 576 exact products accumulated in fp32 by 36 steps of the tensor core, each off by at most
2^-22 of the sum of magnitudes (fp32 with truncation): 36 2^-22 < 2^-16 of scale sum_i |q_i k_i|; that moves
lse by as much, and the outputs by twice that times sum_j p_j |v_j|. Exponentials and sums add under 2^-18.
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


def make(batch, h_q, s_q, shared, lens, seed=0, nan_tails=True, own_entries=True):
    """Inputs as numpy arrays: bf16 bits of q and kv, tables, lengths. Rows past every sequence's end are NaN."""
    rng = np.random.default_rng([seed, 77])
    lens = np.asarray(lens, np.int32)
    w = np.maximum((np.maximum(lens, 0) + 63) // 64 - shared, 0)
    blocks = shared + int(w.sum()) + 1
    perm = rng.permutation(blocks).astype(np.int32)
    table, bt, off = perm[:shared].copy(), np.full((batch, shared + max(1, int(w.max()))), -1, np.int32), shared
    kv = W.f32_to_bf16_bits(rng.standard_normal((blocks, 64, 1, 576), dtype=np.float32))
    if nan_tails:
        kv[perm[-1]] = W.BF16_NAN  # a block of nobody
        top = max(0, int(lens.max()))
        if top < 64 * shared:  # the prefix rows that no sequence reaches
            pre = kv[table].reshape(-1, 576)
            pre[top:] = W.BF16_NAN
            kv[table] = pre.reshape(shared, 64, 1, 576)
    for b in range(batch):
        bt[b, shared:shared + w[b]] = perm[off:off + w[b]]
        off += w[b]
        if nan_tails and w[b] and lens[b] % 64:
            kv[bt[b, shared + w[b] - 1], lens[b] % 64:] = W.BF16_NAN
    q = W.f32_to_bf16_bits(rng.standard_normal((batch, s_q, h_q, 576), dtype=np.float32))
    return dict(q=q, kv=kv, table=table, bt=bt, lens=lens)


def device_inputs(inp, dev="cuda"):
    bf = lambda a: torch.from_numpy(a).view(torch.bfloat16).to(dev)  # noqa: E731
    return (bf(inp["q"]), bf(inp["kv"]), torch.from_numpy(inp["table"]).to(dev), torch.from_numpy(inp["bt"]).to(dev),
            torch.from_numpy(inp["lens"]).to(dev))


def reference(inp, scale, causal):
    q = W.bf16_bits_to_f32(inp["q"]).astype(np.float64)
    kv = W.bf16_bits_to_f32(inp["kv"]).astype(np.float64).reshape(-1, 64, 576)
    return plain.decode_shared(q, kv, inp["table"], inp["bt"], inp["lens"], scale, causal)


def check(out, lse, ref):
    ro, rl, mix, span = ref
    o, l = out.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
    ds = 2.0 ** -16 * span[..., None] + 2.0 ** -18
    tol = 2.0 ** -8 * np.abs(ro) + (2.0 ** -8 + 2 * ds) * mix * (1 + 2.0 ** -8)
    bad = ~(np.abs(o - ro) <= tol)
    assert not bad.any(), ("out", int(bad.sum()), np.argwhere(bad)[:4].tolist())
    none = np.isneginf(rl)
    assert np.array_equal(np.isneginf(l), none)
    l, rl = np.where(none, 0, l), np.where(none, 0, rl)
    ltol = ds[..., 0].transpose(0, 2, 1) + 2.0 ** -20 * np.abs(rl)
    assert np.all(np.abs(l - rl) <= ltol), np.abs(l - rl).max()


def run(inp, scale=W.SCALE, causal=False, num_parts=None, **kw):
    q, kv, table, bt, sl = device_inputs(inp)
    meta = mla.get_metadata_shared(sl, q.shape[2], q.shape[1], table.shape[0], num_parts=num_parts)
    out, lse = mla.decode_shared(q, kv, table, bt, sl, scale, causal, meta, **kw)
    assert mla.check_status() == 0
    return out, lse


CASES = [
    # batch, h_q, s_q, shared blocks, lengths, causal, parts
    (1, 16, 1, 1, [65], False, 1),
    (1, 16, 1, 1, [64], False, None),
    (2, 16, 1, 4, [257, 356], False, None),
    (3, 16, 1, 2, [129, 128, 500], False, 2),
    (1, 128, 1, 3, [300], False, 1),
    (3, 128, 1, 3, [193, 700, 192], False, 4),
    (2, 128, 2, 2, [129, 333], True, 3),
    (5, 40, 3, 5, [321, 323, 900, 322, 340], True, 3),
    (9, 96, 2, 3, [200 + 17 * i for i in range(9)], True, 7),
    (33, 8, 1, 7, [449 + i for i in range(33)], False, 5),
    (20, 16, 4, 9, [577 + 3 * i for i in range(20)], True, None),
    (4, 1, 1, 2, [129, 130, 131, 200], False, None),
    (2, 128, 8, 1, [100, 72], True, 2),
    # lengths that end inside the prefix, at its end, or are nothing; all of them short; no prefix at all
    (6, 16, 1, 4, [0, 5, 64, 256, 257, 400], False, 3),
    (6, 16, 2, 4, [0, 1, 2, 130, 255, 300], True, 3),
    (4, 128, 2, 3, [0, 1, 150, 250], True, 2),
    (5, 16, 1, 6, [3, 70, 0, 130, 129], False, 4),
    (3, 128, 1, 6, [3, 70, 0], False, 4),
    (3, 16, 1, 3, [0, 0, 0], False, 2),
    (3, 24, 1, 0, [1, 64, 333], False, 2),
    (2, 128, 1, 0, [0, 777], False, 3),
    (3, 16, 1, 2, [-5, 140, 2], False, 2),
    # a long prefix in many pieces, and more parts than tiles
    (4, 16, 1, 70, [4481, 4500, 4481 + 640, 4480], False, None),
    (2, 64, 1, 33, [2113, 2200], False, 200),
]


@pytest.mark.parametrize("batch,h_q,s_q,shared,lens,causal,parts", CASES)
def test_matches_plain(batch, h_q, s_q, shared, lens, causal, parts):
    inp = make(batch, h_q, s_q, shared, lens)
    check(*run(inp, causal=causal, num_parts=parts), reference(inp, W.SCALE, causal))


@pytest.mark.parametrize("scale", [0.0, 0.3])
def test_scales(scale):
    """Uniform weights, and scores large enough for one key to take all and the maximum to keep moving."""
    inp = make(3, 16, 1, 5, [321, 400, 500], seed=4)
    check(*run(inp, scale=scale, num_parts=2), reference(inp, scale, False))


def test_scale_zero_of_huge_scores():
    """Scores of up to +-2^123 keep uniform weights."""
    inp = make(2, 16, 1, 2, [150, 200], seed=6)
    q, kv = W.bf16_bits_to_f32(inp["q"]), W.bf16_bits_to_f32(inp["kv"])
    q[..., 575] = 2.0 ** 62
    live = np.isfinite(kv[..., 575])
    kv[..., 575] = np.where(live, np.where(kv[..., 575] > 0, 2.0 ** 61, -2.0 ** 61), kv[..., 575])
    inp["q"], inp["kv"] = W.f32_to_bf16_bits(q), W.f32_to_bf16_bits(kv)
    check(*run(inp, scale=0.0, num_parts=2), reference(inp, 0.0, False))


def test_growing_scores_rescale():
    """Keys whose scores grow along the sequence: the running maximum moves in every tile."""
    inp = make(2, 128, 1, 4, [700, 640], seed=5, nan_tails=False)
    kv = W.bf16_bits_to_f32(inp["kv"])
    for b in range(2):
        order = list(inp["table"]) + [int(x) for x in inp["bt"][b, 4:] if x >= 0]
        for k, blk in enumerate(order):
            kv[blk] *= 1.0 + 0.6 * k
    inp["kv"] = W.f32_to_bf16_bits(kv)
    for parts in (1, 3):
        check(*run(inp, scale=0.15, num_parts=parts), reference(inp, 0.15, False))
