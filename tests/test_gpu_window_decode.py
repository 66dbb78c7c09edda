"""Windowed and block-scaled decode attention on the GPU against the fp64
oracle: every cache type, head layout and block size, windows and sinks that
start and end inside blocks, splits, poisoned unseen rows and freed blocks."""
import numpy as np
import pytest
import torch

import paged_kv_cache_137_gb300 as pkv
from window_cases import Inputs

pytestmark = pytest.mark.gpu

CTX = [0, 1, 15, 16, 17, 31, 32, 33, 63, 64, 65, 100, 257, 700, 1100]


@pytest.fixture(scope="module", autouse=True)
def built():
    pkv.build()
    assert torch.cuda.is_available()


@pytest.fixture(params=["auto", "simt"])
def kernel(request):
    pkv.pkv_set_attention_kernel(request.param)
    yield request.param
    pkv.pkv_set_attention_kernel("auto")


def attend(x, part=0, out=None, ws=None, stream=None):
    out = torch.full_like(x.q_d, float("nan")) if out is None else out
    if ws is None:
        ws = pkv.window_workspace_for(len(x.ctx), x.hq, x.max_blocks, x.desc, x.window, x.sinks, part)
    if x.block_scales is not None:
        pkv.pkv_attention_decode_block_scaled(out, x.q_d, x.k_cache, x.v_cache, x.block_scales, x.tables_d,
                                              x.ctx_d, x.desc, x.scale, x.window, x.sinks, part, ws, stream)
    else:
        pkv.pkv_attention_decode_window(out, x.q_d, x.k_cache, x.v_cache, x.tables_d, x.ctx_d, x.desc, x.window,
                                        x.sinks, x.scale, x.k_scale, x.v_scale, part, ws, stream)
    torch.cuda.synchronize()
    if ws is not None:   # left as it was found: zero counters
        assert int(ws[:len(x.ctx) * x.hkv * 4].count_nonzero()) == 0
    return out


WINDOWS = [(1, 0), (1, 1), (16, 4), (33, 0), (100, 17), (256, 300), (4096, 4)]


@pytest.mark.parametrize("window,sinks", WINDOWS)
@pytest.mark.parametrize("kv,q,d,t", [("bf16", "bf16", 128, 16), ("f16", "f16", 64, 32), ("f16", "f16", 128, 32),
                                      ("bf16", "bf16", 64, 16), ("f32", "f32", 64, 16), ("f32", "f32", 128, 32),
                                      ("e4m3", "bf16", 128, 32), ("e4m3", "f16", 64, 16)])
def test_window(kv, q, d, t, window, sinks, kernel):
    x = Inputs(CTX, hq=6, hkv=2, d=d, t=t, kv=kv, q=q, window=window, sinks=sinks, seed=window)
    for part in (0, 64):
        x.check(attend(x, part))
    assert pkv.pkv_device_status() == 0


@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 2), (50, 3), (300, 20)])
@pytest.mark.parametrize("q,d,t", [("bf16", 128, 16), ("f16", 128, 32), ("bf16", 64, 16), ("f16", 64, 32)])
def test_block_scaled(q, d, t, window, sinks, kernel):
    x = Inputs(CTX, hq=6, hkv=2, d=d, t=t, kv="e4m3", q=q, scales="block", window=window, sinks=sinks, seed=t)
    for part in (0, 64):
        x.check(attend(x, part))


@pytest.mark.parametrize("hq,hkv", [(1, 1), (4, 4), (7, 1), (28, 4), (9, 1), (32, 2), (15, 3)])
@pytest.mark.parametrize("kv,scales", [("bf16", None), ("e4m3", "block"), ("e4m3", "head"), ("f32", None)])
def test_query_groups(hq, hkv, kv, scales, kernel):
    q = "f32" if kv == "f32" else "bf16"
    x = Inputs([5, 130, 600], hq=hq, hkv=hkv, kv=kv, q=q, scales=scales, window=200, sinks=5, seed=hq)
    x.check(attend(x, 64))


def test_block_scales_far_apart(kernel):
    """V scales over 2^72: a block far below its neighbours keeps its bits
    where the weights pick it."""
    x = Inputs([300, 90], hq=4, hkv=2, kv="e4m3", scales="block", seed=8, spread=33, k_gain=6.0)
    x.check(attend(x, 64))


def test_scales_that_are_no_power_of_two(kernel):
    x = Inputs([300, 90], hq=4, hkv=2, kv="e4m3", scales="block", seed=8)
    f = torch.rand(x.block_scales.shape, generator=torch.Generator().manual_seed(1)).add(0.5).cuda()
    x.block_scales.mul_(f)
    for w in (0, 1):
        x.values[w] = x.values[w] * f[:, :, w].double().cpu().numpy()[:, :, None, None]
    x.check(attend(x, 64))


def test_long_contexts_split_many_ways(kernel):
    x = Inputs([9000, 6001], hq=4, hkv=2, kv="bf16", window=5000, sinks=70, seed=11)
    x.check(attend(x))
    x.check(attend(x, 64))
    y = Inputs([9000, 6001], hq=4, hkv=2, kv="e4m3", scales="block", seed=11)
    y.check(attend(y))


@pytest.mark.parametrize("kv,scales", [("bf16", None), ("e4m3", "block")])
def test_no_window_equals_plain_decode(kv, scales):
    """A window over the whole context sees what pkv_attention_decode sees (the
    splits differ, so within rounding), and a scale shared by all blocks is the
    per-tensor scale."""
    x = Inputs([1, 40, 333, 900], hq=8, hkv=2, kv=kv, scales=None, window=0, seed=3)
    if scales:
        x.block_scales = torch.empty((x.nb, x.hkv, 2), device="cuda")
        x.block_scales[..., 0], x.block_scales[..., 1] = x.k_scale, x.v_scale
    else:
        x.window = 1000
    got = attend(x).double()
    ws = pkv.workspace_for(4, x.hq, x.max_blocks, x.desc)
    ref = torch.empty_like(x.q_d)
    pkv.pkv_attention_decode(ref, x.q_d, x.k_cache, x.v_cache, x.tables_d, x.ctx_d, x.desc, x.scale, x.k_scale,
                             x.v_scale, workspace=ws)
    assert (got - ref.double()).abs().max().item() <= 2.0 ** -6


def test_results_do_not_depend_on_the_blocks_or_the_batch():
    """The same sequence in two rows, over different physical blocks, and
    alone: the same bits (split boundaries go by its own length only)."""
    x = Inputs([700, 700, 64], hq=8, hkv=2, kv="bf16", window=300, sinks=4, seed=12)
    owned = x.tables[0] >= 0
    for c in (x.k_cache, x.v_cache):
        c[x.tables[1][owned]] = c[x.tables[0][owned]]
    x.q_d[1] = x.q_d[0]
    out = attend(x, 64)
    assert torch.equal(out[0], out[1])
    alone = torch.empty_like(out[:1])
    ws = pkv.window_workspace_for(1, x.hq, x.max_blocks, x.desc, 300, 4, 64)
    pkv.pkv_attention_decode_window(alone, x.q_d[:1], x.k_cache, x.v_cache, x.tables_d[:1], x.ctx_d[:1], x.desc,
                                    300, 4, x.scale, partition_tokens=64, workspace=ws)
    assert torch.equal(out[:1], alone)


@pytest.mark.parametrize("kv,scales", [("bf16", None), ("e4m3", "block"), ("f32", None)])
def test_bad_tables_and_lengths_give_nan_and_status(kv, scales, kernel):
    q = "f32" if kv == "f32" else "bf16"
    x = Inputs([400, 400, 400, 400], hq=4, hkv=2, kv=kv, q=q, scales=scales, window=200, sinks=4, seed=1)
    pkv.pkv_device_status(clear=True)
    x.tables_d[1, 20] = x.nb
    out = attend(x, 64)
    assert pkv.pkv_device_status(clear=True) == pkv.PKV_DEVICE_BAD_TABLE
    assert torch.isnan(out[1]).all() and not torch.isnan(out[[0, 2, 3]]).any()
    x.ctx_d[2], x.ctx_d[3] = x.max_blocks * x.t + 1, -1
    out = attend(x, 64)
    assert pkv.pkv_device_status(clear=True) == pkv.PKV_DEVICE_BAD_TABLE | pkv.PKV_DEVICE_BAD_LENGTH
    assert torch.isnan(out[1:]).all() and not torch.isnan(out[0]).any()


def test_stage_wait_give_up_sets_status_and_nan_then_recovers():
    x = Inputs([400, 900], hq=4, hkv=2, kv="bf16", window=500, sinks=4, seed=1)
    ws = pkv.window_workspace_for(2, x.hq, x.max_blocks, x.desc, 500, 4, 64)
    pkv.pkv_device_status(clear=True)
    pkv.pkv_set_stage_wait_limit(0)
    try:
        out = attend(x, 64, ws=ws)
    finally:
        pkv.pkv_set_stage_wait_limit(50_000_000)
    assert torch.isnan(out).all()
    assert pkv.pkv_device_status(clear=True) == pkv.PKV_DEVICE_WAIT_TIMEOUT
    x.check(attend(x, 64, ws=ws))


def test_captured_and_replayed_on_another_stream():
    x = Inputs([400, 900, 33], hq=8, hkv=2, kv="e4m3", scales="block", window=500, sinks=4, seed=2)
    want = attend(x, 64)
    ws = pkv.window_workspace_for(3, x.hq, x.max_blocks, x.desc, 500, 4, 64)
    out = torch.full_like(want, float("nan"))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        pkv.pkv_attention_decode_block_scaled(out, x.q_d, x.k_cache, x.v_cache, x.block_scales, x.tables_d, x.ctx_d,
                                              x.desc, x.scale, 500, 4, 64, ws, torch.cuda.current_stream())
    for _ in range(3):
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_infinite_logits_and_values():
    """Keys of -inf logits get no weight; an infinite value a query sees with a
    positive weight is its output."""
    x = Inputs([40], hq=2, hkv=1, d=128, kv="bf16", window=100, seed=4)
    x.q_d.abs_().clamp_(min=0.1)
    blk = int(x.tables[0, 0])
    x.k_cache[blk, 0, :16] = float("-inf")   # a whole chunk without weight
    out = attend(x)
    x.values[0][blk, 0, :16] = -50.0   # far enough below for a weight of 0
    x.q = x.q_d.cpu()
    x.check(out)
    x.v_cache[int(x.tables[0, 2]), 0, 0, 5] = float("inf")
    assert torch.isinf(attend(x)[0, :, 5]).all()


@pytest.mark.parametrize("window,sinks", [(2 ** 31 - 1, 0), (2 ** 31 - 1, 2 ** 31 - 1), (5, 2 ** 31 - 1)])
def test_the_largest_windows_and_sinks(window, sinks, kernel):
    x = Inputs(CTX, hq=4, hkv=2, kv="bf16", window=window, sinks=sinks, seed=6)
    for part in (0, 64):
        x.check(attend(x, part))


def test_two_calls_at_once_and_graphs_that_share_a_workspace():
    """Calls on two streams, each with a workspace of its own; two captured
    calls of one workspace, replayed one after the other."""
    xs = [Inputs([400, 900, 33], hq=8, hkv=2, kv="bf16", window=w, sinks=4, seed=w) for w in (500, 300)]
    want = [attend(x, 64) for x in xs]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    spaces = [pkv.window_workspace_for(3, x.hq, x.max_blocks, x.desc, x.window, 4, 64) for x in xs]
    outs = [torch.full_like(w, float("nan")) for w in want]

    def call(i, ws, stream):
        x = xs[i]
        pkv.pkv_attention_decode_window(outs[i], x.q_d, x.k_cache, x.v_cache, x.tables_d, x.ctx_d, x.desc, x.window,
                                        x.sinks, x.scale, partition_tokens=64, workspace=ws, stream=stream)

    torch.cuda.synchronize()
    for _ in range(5):
        for i in range(2):
            call(i, spaces[i], streams[i])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    shared = max(spaces, key=torch.Tensor.numel)
    graphs = []
    for i in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[i]):
            call(i, shared, None)
    for _ in range(3):
        for o in outs:
            o.fill_(float("nan"))
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


@pytest.mark.parametrize("scales", [None, "block"])
def test_offsets_past_32_bits(scales, kernel):
    """Contexts in the last blocks of a cache of more than 2^32 elements."""
    x = Inputs([40, 33, 100], hq=8, hkv=8, kv="e4m3", scales=scales, window=60, sinks=3, seed=7)
    want = attend(x)
    nb = (1 << 32) // (8 * 16 * 128) + 64
    x.desc = pkv.kv_desc(nb, 8, 128, 16, "e4m3")
    for name in ("k_cache", "v_cache", "block_scales"):
        small = getattr(x, name)
        if small is not None:
            big = torch.zeros((nb,) + small.shape[1:], dtype=small.dtype, device="cuda")
            big[nb - x.nb:] = small
            setattr(x, name, big)
    x.tables_d = torch.where(x.tables_d >= 0, x.tables_d + (nb - x.nb), x.tables_d).int()
    assert torch.equal(attend(x), want)
