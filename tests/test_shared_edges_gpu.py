"""Edges of the shared-prefix decode on a B200: row slices that a tile fills only in part. Tolerances are those of
tests/test_shared_gpu.py."""
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
