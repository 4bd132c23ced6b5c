"""Edges of the shared-prefix decode on a B200: row slices that a tile fills only in part, queries that are no finite
numbers. Tolerances are those of tests/test_shared_gpu.py."""
import numpy as np
import pytest
import torch

from mla_decode_attention_14_b200 import workloads as W
from tests.test_shared_gpu import check, make, reference, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)


@pytest.mark.parametrize("rows", [1, 7, 8, 24, 33, 40, 63, 65, 97, 104, 127, 129, 200])
@pytest.mark.parametrize("shared,parts", [(0, 1), (0, 3), (2, 1), (2, 5)])
def test_partly_filled_row_slices(rows, shared, parts):
    """A warp serves 32 rows: 1 to 31 of them are there in some slice, in outputs written whole and in pieces, several
    sequences (and so several outputs) to a part."""
    inp = make(3, rows, 1, shared, [64 * shared + n for n in (70, 1, 333)], seed=rows)
    check(*run(inp, num_parts=parts), reference(inp, W.SCALE, False))


@pytest.mark.parametrize("h_q,shared", [(16, 3), (128, 3), (24, 0), (128, 0)])
@pytest.mark.parametrize("parts", [1, 2, 7, 40])
@pytest.mark.parametrize("value", ["nan", "inf", "-inf"])
def test_non_finite_queries_show_in_their_rows_alone(h_q, shared, parts, value):
    """A row with a NaN score or a score of +inf is NaN, out and lse, whether its unit is cut or not; without a key it
    is the row of zeros and -inf that it is for any query; no other row changes."""
    lens = [64 * shared + 900, 0, 64 * shared + 333, 64 * shared + 77]
    inp = make(4, h_q, 1, shared, lens, seed=9)
    rows = [(0, 0, 0), (0, 0, h_q - 1), (1, 0, 2), (2, 0, 5), (3, 0, 9)]
    q = W.bf16_bits_to_f32(inp["q"])
    clean = reference(inp, W.SCALE, False)
    for r in rows:
        q[r][100] = float(value)  # keys of either sign there: +inf among the scores of each of these rows
    inp["q"] = W.f32_to_bf16_bits(q)
    out, lse = run(inp, num_parts=parts)
    o, l = out.float().cpu(), lse.cpu()
    for b, t, h in rows:
        if lens[b]:
            assert o[b, t, h].isnan().all() and l[b, h, t].isnan(), (b, h)
            o[b, t, h] = torch.from_numpy(clean[0][b, t, h]).float()
            l[b, h, t] = float(clean[1][b, h, t])
    check(o, l, clean)


@pytest.mark.parametrize("h_q,shared", [(16, 3), (128, 3)])
@pytest.mark.parametrize("parts", [1, 7])
def test_scores_of_minus_infinity_weigh_nothing(h_q, shared, parts):
    """Keys whose dim meets an infinite query with the other sign: the rest of the keys share the weight, and a row
    without any other key is a row without keys."""
    inp = make(2, h_q, 1, shared, [64 * shared + 500, 64 * shared + 130], seed=10, nan_tails=False)
    kv, q = W.bf16_bits_to_f32(inp["kv"]), W.bf16_bits_to_f32(inp["q"])
    kv[..., 575] = 1.0
    inp["kv"] = W.f32_to_bf16_bits(kv)
    ref = reference(inp, W.SCALE, False)
    q[0, 0, 3, 575] = -np.inf  # every score of this row
    inp["q"] = W.f32_to_bf16_bits(q)
    out, lse = run(inp, num_parts=parts)
    assert not out[0, 0, 3].any() and bool(lse[0, 3, 0].isneginf())
    out, lse = out.float().cpu(), lse.cpu()
    out[0, 0, 3], lse[0, 3, 0] = torch.from_numpy(ref[0][0, 0, 3]).float(), float(ref[1][0, 3, 0])
    check(out, lse, ref)
