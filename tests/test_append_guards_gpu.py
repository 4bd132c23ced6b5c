"""The rotating appends on tables and counts that are wrong (a B200): what no valid token addresses stays as it was,
byte for byte, in the cache and in guard blocks on both sides of it, and the valid tokens are written."""
import numpy as np
import pytest
import torch

import mla_decode_attention_14_b200 as mla

pytestmark = pytest.mark.gpu
KV_SCALE = 2.0 ** -6
GUARD = 3  # blocks


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)


def cache(blocks, fp8, seed):
    """A cache with guard blocks on both sides (whole buffer, the cache's view), random bytes that are finite values."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    shape = (blocks + 2 * GUARD, 64, 1, 640 if fp8 else 576)
    if fp8:
        whole = torch.randint(0, 100, shape, generator=g, device="cuda", dtype=torch.uint8)
    else:
        whole = torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)
    return whole, whole[GUARD:GUARD + blocks]


def append(fp8, x, kv, bt, sl, **kw):
    rope = mla.rope(interleaved=False)
    if fp8:
        mla.append_kv_rope_fp8(x, kv, bt, sl, KV_SCALE, rope, **kw)
    else:
        mla.append_kv_rope(x, kv, bt, sl, rope, **kw)


def changed_rows(whole, before):
    """Rows of the cache (negative or past its end: of a guard block) whose bytes are not what they were."""
    a, b = (t.view(torch.uint8).reshape(t.shape[0] * 64, -1) for t in (whole, before))
    return set((torch.nonzero((a != b).any(dim=1)).flatten().cpu() - 64 * GUARD).tolist())


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("bad", ["none", "past", "far", "narrow"])
def test_bad_entries(fp8, packed, bad):
    """Sequence 0's table misses the block of its new tokens; the other two are written all the same."""
    blocks, n = 12, 3
    whole, kv = cache(blocks, fp8, 1)
    had = [64 * 3 + 5, 62, 130]
    bt = torch.arange(blocks, dtype=torch.int32, device="cuda").view(3, 4).contiguous()
    if bad == "narrow":
        bt = bt[:, :3].contiguous()  # entry 3 is not there
    else:
        bt[0, 3] = {"none": -1, "past": blocks, "far": 1 << 29}[bad]
    sl = torch.tensor(had, dtype=torch.int32, device="cuda")
    x = torch.randn((3, n, 576), device="cuda").to(torch.bfloat16)
    before = whole.clone()
    if packed:
        append(fp8, x.view(-1, 576), kv, bt, sl, cu_new=torch.tensor([0, n, 2 * n, 3 * n], dtype=torch.int32, device="cuda"))
    else:
        append(fp8, x, kv, bt, sl)
    assert mla.check_status() == 6  # MLA_ERR_BOUNDS
    assert mla.check_status() == 0
    table = bt.cpu()
    rows = {b: [int(table[b, (had[b] + t) // 64]) * 64 + (had[b] + t) % 64 for t in range(n)] for b in (1, 2)}
    assert changed_rows(whole, before) == set(rows[1] + rows[2])
    for b in (1, 2):  # the latents as mla_append_kv / _fp8 store them: no norm was asked for
        got = kv.view(blocks * 64, -1)[torch.tensor(rows[b], device="cuda")]
        if fp8:
            want = (x[b, :, :512].float() / KV_SCALE).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            assert torch.equal(got[:, :512], want)
        else:
            assert torch.equal(got[:, :512].view(torch.int16), x[b, :, :512].view(torch.int16))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("cu", [[0, 3, 1, 3], [2, 1, 0, 3], [0, 0, 5, 3], [-7, 90, -90, 2], [3, 3, 3, 3], [0, 1 << 30, 2, 3],
                                [-(1 << 31), (1 << 31) - 1, 0, (1 << 31) - 1],
                                # row 0 is token 2^31 of sequence 0: a place past 32 bits, and past its table
                                [-(1 << 31), 1, 2, 3], [-(1 << 31), (1 << 31) - 1, (1 << 31) - 1, (1 << 31) - 1],
                                [2 - (1 << 31), 2, 2, 3]])
def test_broken_counts(fp8, cu):
    """Counts that decrease, overlap or point outside: which token goes where is open, but only rows that some
    sequence's table and length address are written (what the last kept count leaves out is not)."""
    blocks, tokens = 12, 3
    whole, kv = cache(blocks, fp8, 2)
    had = [5, 62, 130]
    bt = torch.full((3, 4), -1, dtype=torch.int32, device="cuda")
    bt[:, :3] = torch.arange(9, dtype=torch.int32, device="cuda").view(3, 3)  # blocks 9 to 11 belong to nobody
    sl = torch.tensor(had, dtype=torch.int32, device="cuda")
    x = torch.randn((tokens, 576), device="cuda").to(torch.bfloat16)
    before = whole.clone()
    append(fp8, x, kv, bt, sl, cu_new=torch.tensor(cu, dtype=torch.int32, device="cuda"))
    assert mla.check_status() in (0, 6)
    # a token's place within its sequence is its row less some count at or below it
    own = [{b * 192 + p for p in range(had[b], 192)} for b in range(3)]
    got = changed_rows(whole, before)
    assert got <= own[0] | own[1] | own[2], sorted(got)
    assert len(got) <= tokens
    if cu == [3, 3, 3, 3]:
        assert not got


@pytest.mark.parametrize("fp8", [False, True])
def test_rows_outside_the_counts_are_left(fp8):
    """Rows before the first count and behind the last are no sequence's."""
    blocks = 6
    whole, kv = cache(blocks, fp8, 3)
    bt = torch.arange(blocks, dtype=torch.int32, device="cuda").view(2, 3).contiguous()
    sl = torch.tensor([63, 0], dtype=torch.int32, device="cuda")
    x = torch.randn((40, 576), device="cuda").to(torch.bfloat16)
    before = whole.clone()
    append(fp8, x, kv, bt, sl, cu_new=torch.tensor([7, 9, 20], dtype=torch.int32, device="cuda"))
    assert mla.check_status() == 0
    assert changed_rows(whole, before) == {63, 64} | {192 + t for t in range(11)}
