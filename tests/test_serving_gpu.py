"""The serving-step operators together and in the ways a program calls them: a whole step against the plain
64-bit forms, CUDA graphs, other streams, repeated and overlapping calls, schedules, bad tables, a cache past
32-bit offsets (needs a B200)."""
import numpy as np
import pytest
import torch

import mla_decode_attention_14_b200 as mla
import oracle
from mla_decode_attention_14_b200 import workloads as W
from tests import plain_serving as plain
from tests.test_shared_gpu import check, device_inputs, make, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)


def f64(bits):
    return W.bf16_bits_to_f32(bits).astype(np.float64)


def up(bits):
    return torch.from_numpy(bits).view(torch.bfloat16).cuda()


# ---------------------------------------------------------------- a step

@pytest.mark.parametrize("h_q,s_q,interleaved", [(16, 1, True), (128, 2, False)])
def test_serving_step(h_q, s_q, interleaved):
    """New tokens normed, rotated and appended, the queries rotated into place, then attention over prefix and own
    blocks: each stage's inputs are what the stage before left on the GPU."""
    shared, lens = 3, [200, 255, 300, 193, 520]
    b = len(lens)
    inp = make(b, h_q, s_q, shared, [n + s_q for n in lens], seed=11, nan_tails=False)
    old = np.array(lens, np.int32)
    rng = np.random.default_rng(12)
    bits = lambda *s: W.f32_to_bf16_bits(rng.standard_normal(s, dtype=np.float32))  # noqa: E731
    xb, wb, pb = bits(b, s_q, 576), bits(512), bits(b, s_q, h_q, 192)
    kw = dict(interleaved=interleaved, factor=4.0, original_len=4096, magnitude=1.125)
    freq = plain.inv_freq(factor=4.0, original_len=4096)
    rope = mla.rope(**kw)
    q, kv, table, bt, sl = device_inputs(inp)
    kv_before = kv.clone()
    full = bt.clone()
    full[:, :shared] = table
    d_old = torch.from_numpy(old).cuda()

    mla.append_kv_rope(up(xb), kv, full, d_old, rope, norm_weight=up(wb), eps=1e-5)
    mla.rope_q(up(pb)[..., 128:], q, rope, seqlens=d_old)
    meta = mla.get_metadata_shared(sl, h_q, s_q, shared)
    out, lse = mla.decode_shared(q, kv, table, bt, sl, W.SCALE, True, meta)
    assert mla.check_status() == 0

    pos = old[:, None] + np.arange(s_q)
    vals = plain.append_values(f64(xb).reshape(-1, 576), pos.reshape(-1), freq, interleaved, 1.125, f64(wb), 1e-5)
    rows = full.cpu().numpy()[np.arange(b)[:, None], pos // 64] * 64 + pos % 64
    got = kv.view(-1, 576)[torch.from_numpy(rows.reshape(-1)).long().cuda()].float().cpu().numpy().astype(np.float64)
    # a value within one bf16 rounding (2^-8); a rotary one is a difference of two terms, which bounds its fp32 error
    assert np.all(np.abs(got - vals) <= 2.0 ** -8 * np.abs(vals) + 2.0 ** -18 * (1 + np.abs(vals)).max())
    rot = plain.rotate(f64(pb)[..., 128:], pos[..., None], freq, interleaved, 1.125)
    gq = q.float().cpu().numpy().astype(np.float64)
    assert np.all(np.abs(gq[..., 512:] - rot) <= 2.0 ** -8 * np.abs(rot) + 2.0 ** -18 * (1 + np.abs(rot)).max())
    same = torch.ones(kv.shape[0] * 64, dtype=torch.bool)
    same[torch.from_numpy(rows.reshape(-1)).long()] = False
    assert torch.equal(kv.view(-1, 576)[same.cuda()].view(torch.int16), kv_before.view(-1, 576)[same.cuda()].view(torch.int16))
    now = dict(inp, q=q.view(torch.uint16).cpu().numpy(), kv=kv.view(torch.uint16).cpu().numpy())
    check(out, lse, reference(now, W.SCALE, True))


def test_append_is_the_plain_append_without_norm_at_position_zero():
    """No norm, no turn (all positions 0, magnitude 1): bit for bit mla_append_kv and mla_append_kv_fp8."""
    rng = np.random.default_rng(5)
    x = up(W.f32_to_bf16_bits(rng.standard_normal((6, 2, 576), dtype=np.float32)))
    bt = torch.arange(12, dtype=torch.int32, device="cuda").view(6, 2)
    sl = torch.tensor([0, 5, 62, 63, 64, 100], dtype=torch.int32, device="cuda")
    pos = torch.zeros((6, 2), dtype=torch.int32, device="cuda")
    for interleaved in (True, False):
        r = mla.rope(interleaved=interleaved)
        a, b = torch.zeros((12, 64, 1, 576), dtype=torch.bfloat16, device="cuda"), torch.zeros((12, 64, 1, 576), dtype=torch.bfloat16, device="cuda")
        mla.append_kv(x, a, bt, sl)
        mla.append_kv_rope(x, b, bt, sl, r, positions=pos)
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))
        a, b = torch.zeros((12, 64, 1, 640), dtype=torch.uint8, device="cuda"), torch.zeros((12, 64, 1, 640), dtype=torch.uint8, device="cuda")
        mla.append_kv_fp8(x, a, bt, sl, 0.0123)
        mla.append_kv_rope_fp8(x, b, bt, sl, 0.0123, r, positions=pos)
        assert torch.equal(a, b)


# ---------------------------------------------------------------- schedules

@pytest.mark.parametrize("seed", range(8))
def test_shared_metadata_is_the_oracle_s_partition(seed):
    rng = np.random.default_rng(seed)
    b, h_q, s_q = int(rng.integers(1, 400)), int(rng.choice([16, 40, 64, 96, 128])), int(rng.choice([1, 2, 3]))
    sb, P, C = int(rng.choice([0, 1, 5, 64])), int(rng.integers(1, 200)), int(rng.integers(0, 6))
    lens = rng.integers(-3, 64 * sb + (50 if seed % 3 == 0 else 3000), size=b).astype(np.int32)
    m = mla.get_metadata_shared(torch.from_numpy(lens).cuda(), h_q, s_q, sb, num_parts=P, fixed_cost=C)
    rows = h_q * s_q
    blocks = lambda n: (max(int(n), 0) + 63) // 64  # noqa: E731
    reach = min(max(0, int(lens.max())), 64 * sb)
    prefix = -(-b * rows // 128) if sb and rows % 128 else 0
    tiles = [-(-blocks(reach) // 2)] * prefix
    for n in lens:
        tiles += [-(-max(0, blocks(n) - (sb if prefix else 0)) // 2)] * -(-rows // 128)
    tm, ns = oracle.metadata(64 * np.array(tiles, np.int32), P, C)
    tm[:, 5] = reach
    assert np.array_equal(m.tile_meta.cpu().numpy(), tm) and np.array_equal(m.num_splits.cpu().numpy(), ns)


def test_metadata_of_another_kind_is_refused():
    inp = make(2, 128, 1, 1, [100, 200])
    q, kv, table, bt, sl = device_inputs(inp)
    shared, plainm = mla.get_metadata_shared(sl, 128, 1, 1), mla.get_metadata(sl, 128, 1)
    with pytest.raises(ValueError):
        mla.decode_shared(q, kv, table, bt, sl, 0.1, False, plainm)
    with pytest.raises(ValueError):
        mla.decode(q, kv, bt, sl, 0.1, False, shared)
    with pytest.raises(ValueError):
        mla.decode_shared(q, kv, table[:0], bt, sl, 0.1, False, shared)
    with pytest.raises(ValueError):
        mla.decode_shared(q[:1], kv, table, bt[:1], sl[:1], 0.1, False, shared)
    for bad in (dict(out=torch.empty((2, 1, 128, 512), device="cuda")), dict(workspace=torch.empty(8, device="cuda")),
                dict(lse=torch.empty((2, 1, 128), device="cuda"))):
        with pytest.raises((ValueError, TypeError)):
            mla.decode_shared(q, kv, table, bt, sl, 0.1, False, shared, **bad)


# ---------------------------------------------------------------- ways of calling

@pytest.mark.parametrize("h_q", [16, 128])
def test_graph_of_a_step_replays_on_new_inputs(h_q):
    inp = make(4, h_q, 1, 2, [130, 200, 140, 400], seed=21)
    q, kv, table, bt, sl = device_inputs(inp)
    x, rope = torch.randn((4, 1, h_q, 64), device="cuda").to(torch.bfloat16), mla.rope(interleaved=False)
    new = torch.randn((4, 1, 576), device="cuda").to(torch.bfloat16)
    full = bt.clone()
    full[:, :2] = table
    before = sl - 1

    def step():
        mla.append_kv_rope(new, kv, full, before, rope)
        mla.rope_q(x, q, rope, seqlens=before)
        meta = mla.get_metadata_shared(sl, h_q, 1, 2, num_parts=5)
        return mla.decode_shared(q, kv, table, bt, sl, W.SCALE, False, meta)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        og, lg = step()
    for k in range(3):
        x.copy_(torch.randn(x.shape, device="cuda"))
        new.copy_(torch.randn(new.shape, device="cuda"))
        graph.replay()
        a, b = og.clone(), lg.clone()
        oe, le = step()
        assert torch.equal(a, oe) and torch.equal(b, le), k
        # another length for a sequence: the plan is part of the graph
        if k == 1:
            sl[3] = 390
            before[3] = 389
    assert mla.check_status() == 0


def test_streams_workspaces_and_repeats():
    """Two calls at once on two streams, each with its own workspace; the same call again gives the same bits,
    whatever the workspace held."""
    inp = make(24, 16, 1, 40, [2561 + 40 * i for i in range(24)], seed=31)
    ref = reference(inp, W.SCALE, False)
    q, kv, table, bt, sl = device_inputs(inp)
    meta = mla.get_metadata_shared(sl, 16, 1, 40)
    o0, l0 = mla.decode_shared(q, kv, table, bt, sl, W.SCALE, False, meta)
    check(o0, l0, ref)
    size = mla.shared_workspace_bytes(24, 1, 16, 40, meta.num_parts)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    w1, w2 = torch.full((size,), 255, dtype=torch.uint8, device="cuda"), torch.full((size,), 127, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        for s, w in ((s1, w1), (s2, w2)):
            out, lse = torch.empty_like(o0), torch.empty_like(l0)
            with torch.cuda.stream(s):
                mla.decode_shared(q, kv, table, bt, sl, W.SCALE, False, meta, out=out, lse=lse, workspace=w)
            got.append((out, lse))
    # and a stream given by hand, not the current one
    out, lse = torch.empty_like(o0), torch.empty_like(l0)
    mla.decode_shared(q, kv, table, bt, sl, W.SCALE, False, meta, out=out, lse=lse, workspace=w1, stream=s1)
    got.append((out, lse))
    torch.cuda.synchronize()
    assert mla.check_status() == 0
    for out, lse in got:
        assert torch.equal(out, o0) and torch.equal(lse, l0)


def test_tensors_made_by_a_call_belong_to_its_stream():
    """Another stream fills whatever memory is free while the calls run: nothing of theirs is."""
    inp = make(24, 16, 1, 40, [2561 + 40 * i for i in range(24)], seed=31)
    q, kv, table, bt, sl = device_inputs(inp)
    meta = mla.get_metadata_shared(sl, 16, 1, 40)
    o0, l0 = mla.decode_shared(q, kv, table, bt, sl, W.SCALE, False, meta)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        m = mla.get_metadata_shared(sl, 16, 1, 40, stream=s)
        got.append(mla.decode_shared(q, kv, table, bt, sl, W.SCALE, False, m, stream=s) + (m,))
        for size in (m.workspace_bytes, 2 * o0.numel(), 4 * l0.numel()):
            torch.full((size,), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    assert mla.check_status() == 0
    for out, lse, m in got:
        assert torch.equal(m.tile_meta, meta.tile_meta) and torch.equal(out, o0) and torch.equal(lse, l0)


def test_repeated_rows_are_refused_by_the_appends():
    """A token broadcast over the batch has rows 0 elements apart: refused, not read as if they were 576 apart."""
    kv = torch.zeros((4, 64, 1, 576), dtype=torch.bfloat16, device="cuda")
    kv8 = torch.zeros((4, 64, 1, 640), dtype=torch.uint8, device="cuda")
    bt, sl = torch.arange(3, dtype=torch.int32, device="cuda")[:, None].contiguous(), torch.zeros(3, dtype=torch.int32, device="cuda")
    cu = torch.arange(4, dtype=torch.int32, device="cuda")
    row, r = torch.ones((1, 1, 576), dtype=torch.bfloat16, device="cuda"), mla.rope()
    for x, c in ((row.expand(3, 1, 576), None), (row[0].expand(3, 576), cu), (row.expand(3, 2, 576), None)):
        with pytest.raises(ValueError):
            mla.append_kv_rope(x, kv, bt, sl, r, cu_new=c)
        with pytest.raises(ValueError):
            mla.append_kv_rope_fp8(x, kv8, bt, sl, 0.5, r, cu_new=c)
    torch.cuda.synchronize()
    assert not kv.any() and not kv8.any()
    mla.append_kv_rope(row, kv, bt[:1], sl[:1], r)  # one token has no distance to the next
    assert torch.equal(kv[0, 0, 0, :512], row[0, 0, :512])


def test_output_on_a_16_byte_boundary():
    inp = make(3, 128, 1, 1, [100, 64, 300], seed=41)
    q, kv, table, bt, sl = device_inputs(inp)
    meta = mla.get_metadata_shared(sl, 128, 1, 1, num_parts=2)
    o0, l0 = mla.decode_shared(q, kv, table, bt, sl, W.SCALE, False, meta)
    flat = torch.empty(o0.numel() + 8, dtype=torch.bfloat16, device="cuda")
    out = flat[8:].view(o0.shape)
    assert out.data_ptr() % 32 == 16
    mla.decode_shared(q, kv, table, bt, sl, W.SCALE, False, meta, out=out)
    assert torch.equal(out, o0)


def test_bad_tables_are_reported_not_read():
    inp = make(3, 16, 1, 2, [200, 260, 190], seed=51)
    q, kv, table, bt, sl = device_inputs(inp)
    meta = mla.get_metadata_shared(sl, 16, 1, 2)
    for which, value in (("own", -1), ("own", 1 << 30), ("shared", kv.shape[0]), ("narrow", 0)):
        t, o = table.clone(), bt.clone()
        if which == "own":
            o[1, 3] = value
        elif which == "shared":
            t[1] = value
        else:
            o = o[:, :4].contiguous()  # sequence 1 needs entry 4
        out, lse = mla.decode_shared(q, kv, t, o, sl, W.SCALE, False, meta)
        assert mla.check_status() == 6, which  # MLA_ERR_BOUNDS
        assert mla.check_status() == 0
    new = torch.zeros((3, 1, 576), dtype=torch.bfloat16, device="cuda")
    before = kv.clone()
    o = bt.clone()
    o[0, 3] = 1 << 29
    mla.append_kv_rope(new, kv, o, sl, mla.rope())
    assert mla.check_status() == 6
    # a broken cu_new (decreasing) reads and writes nothing out of range
    cu = torch.tensor([0, 3, 1, 3], dtype=torch.int32, device="cuda")
    mla.append_kv_rope(new.view(3, 576), before, bt, sl, mla.rope(), cu_new=cu)
    assert mla.check_status() in (0, 6)


def test_stale_schedule_stays_in_bounds():
    """Lengths changed after the schedule was made: values are unspecified, nothing hangs or leaves its buffers."""
    inp = make(6, 16, 1, 2, [200, 260, 190, 500, 300, 129], seed=61)
    q, kv, table, bt, sl = device_inputs(inp)
    meta = mla.get_metadata_shared(sl, 16, 1, 2, num_parts=7)
    for lens in ([128] * 6, [0] * 6, [130, 500, 129, 1, 500, 129]):
        size = mla.shared_workspace_bytes(6, 1, 16, 2, 7)
        ws = torch.full((size + 4096,), 77, dtype=torch.uint8, device="cuda")
        mla.decode_shared(q, kv, table, bt, torch.tensor(lens, dtype=torch.int32, device="cuda"), W.SCALE, False, meta,
                          workspace=ws[:size])
        assert mla.check_status() in (0, 6)
        assert bool((ws[size:] == 77).all())


def test_cache_past_32_bit_offsets():
    """Blocks at the end of a cache of more than 2^32 bytes (and 2^31 elements)."""
    blocks = (1 << 31) // (64 * 576) + 600
    kv = torch.empty((blocks, 64, 1, 576), dtype=torch.bfloat16, device="cuda")
    small = make(3, 16, 1, 2, [200, 150, 320], seed=71)
    q, kv_s, table, bt, sl = device_inputs(small)
    shift = blocks - kv_s.shape[0]
    kv[shift:] = kv_s
    table2 = table + shift
    bt2 = torch.where(bt >= 0, bt + shift, bt)
    meta = mla.get_metadata_shared(sl, 16, 1, 2, num_parts=3)
    o1, l1 = mla.decode_shared(q, kv_s, table, bt, sl, W.SCALE, False, meta)
    o2, l2 = mla.decode_shared(q, kv, table2, bt2, sl, W.SCALE, False, meta)
    assert mla.check_status() == 0
    assert torch.equal(o1, o2) and torch.equal(l1, l2)
    new = torch.randn((3, 1, 576), device="cuda").to(torch.bfloat16)
    at = sl - 1
    full1, full2 = bt.clone(), bt2.clone()
    full1[:, :2], full2[:, :2] = table, table2
    mla.append_kv_rope(new, kv_s, full1, at, mla.rope())
    mla.append_kv_rope(new, kv, full2, at, mla.rope())
    assert mla.check_status() == 0
    assert torch.equal(kv[shift:].view(torch.int16), kv_s.view(torch.int16))


@pytest.mark.parametrize("b,h_q,s_q,shared,lens", [(200, 16, 1, 3, None), (1, 128, 8, 2, [129]), (40, 24, 4, 20, None)])
def test_larger_batches(b, h_q, s_q, shared, lens):
    rng = np.random.default_rng(b)
    lens = lens or [64 * shared + int(v) for v in rng.integers(-20, 200, b)]
    inp = make(b, h_q, s_q, shared, lens, seed=81)
    q, kv, table, bt, sl = device_inputs(inp)
    meta = mla.get_metadata_shared(sl, h_q, s_q, shared)
    out, lse = mla.decode_shared(q, kv, table, bt, sl, W.SCALE, True, meta)
    assert mla.check_status() == 0
    check(out, lse, reference(inp, W.SCALE, True))
