"""Windowed and block-scaled prefill attention on the GPU against the fp64
oracle: cache types, head layouts, chunks of one token to several row pairs,
windows and sinks that start and end inside blocks and steps, poisoned unseen
rows, freed blocks."""
import numpy as np
import pytest
import torch

import paged_kv_cache_137_gb300 as pkv
from window_cases import Inputs

pytestmark = pytest.mark.gpu

CTX = [1, 16, 40, 63, 64, 65, 130, 257, 500, 700]
NEW = [1, 1, 40, 10, 64, 33, 128, 1, 300, 200]


@pytest.fixture(scope="module", autouse=True)
def built():
    pkv.build()
    assert torch.cuda.is_available()
    pkv.pkv_device_status(clear=True)


def attend(x, out=None, max_query_len=None, scale=None, stream=None):
    out = torch.full_like(x.q_d, float("nan")) if out is None else out
    scale = x.scale if scale is None else scale
    longest = int(x.n.max()) if max_query_len is None else max_query_len
    if x.block_scales is not None:
        pkv.pkv_attention_prefill_block_scaled(out, x.q_d, x.k_cache, x.v_cache, x.block_scales, x.tables_d, x.ctx_d,
                                               x.start, x.desc, scale, longest, x.window, x.sinks, stream)
    else:
        pkv.pkv_attention_prefill_window(out, x.q_d, x.k_cache, x.v_cache, x.tables_d, x.ctx_d, x.start, x.desc,
                                         x.window, x.sinks, scale, longest, x.k_scale, x.v_scale, stream)
    torch.cuda.synchronize()
    return out


WINDOWS = [(1, 0), (1, 1), (16, 4), (33, 0), (100, 17), (256, 300), (4096, 4)]


@pytest.mark.parametrize("window,sinks", WINDOWS)
@pytest.mark.parametrize("kv,q,d,t", [("bf16", "bf16", 128, 16), ("f16", "f16", 64, 32), ("f16", "f16", 128, 32),
                                      ("bf16", "bf16", 64, 16), ("e4m3", "bf16", 128, 32), ("e4m3", "f16", 128, 16)])
def test_window(kv, q, d, t, window, sinks):
    x = Inputs(CTX, NEW, hq=6, hkv=2, d=d, t=t, kv=kv, q=q, window=window, sinks=sinks, seed=window)
    x.check(attend(x))
    assert pkv.pkv_device_status() == 0


@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 2), (50, 3), (300, 20)])
@pytest.mark.parametrize("q,t", [("bf16", 16), ("f16", 32)])
def test_block_scaled(q, t, window, sinks):
    x = Inputs(CTX, NEW, hq=6, hkv=2, t=t, kv="e4m3", q=q, scales="block", window=window, sinks=sinks, seed=t)
    x.check(attend(x))


@pytest.mark.parametrize("hq,hkv", [(1, 1), (4, 4), (7, 1), (28, 4), (20, 1), (32, 2), (15, 3)])
@pytest.mark.parametrize("kv,scales", [("bf16", None), ("e4m3", "block"), ("e4m3", "head")])
def test_query_groups(hq, hkv, kv, scales):
    x = Inputs([300, 77, 600], [300, 3, 150], hq=hq, hkv=hkv, kv=kv, scales=scales, window=130, sinks=5, seed=hq)
    x.check(attend(x))


@pytest.mark.parametrize("chunk", [1, 2, 18, 19, 36, 37, 73, 74, 400])
def test_chunks_around_a_row_pair(chunk):
    """7 heads a KV head: 128 rows are 18.3 positions, 256 are 36.6."""
    x = Inputs([400, 401], [chunk, chunk], hq=7, hkv=1, kv="bf16", window=90, sinks=20, seed=chunk)
    x.check(attend(x))


def test_block_scales_far_apart():
    x = Inputs([300, 90], [100, 90], hq=4, hkv=2, kv="e4m3", scales="block", seed=8, spread=33, k_gain=3.0)
    x.check(attend(x))


def test_scales_that_are_no_power_of_two():
    x = Inputs([300, 90], [100, 90], hq=4, hkv=2, kv="e4m3", scales="block", seed=8)
    f = torch.rand(x.block_scales.shape, generator=torch.Generator().manual_seed(1)).add(0.5).cuda()
    x.block_scales.mul_(f)
    for w in (0, 1):
        x.values[w] = x.values[w] * f[:, :, w].double().cpu().numpy()[:, :, None, None]
    # scale / R and its product with the value, each rounded to f16
    x.check(attend(x), extra_rounding=2.0 ** -10 * (1 + 2.0 ** -10))


def test_a_scale_that_is_not_positive():
    for scale in (-0.05, 0.0):
        x = Inputs([200, 90], [60, 90], hq=4, hkv=2, kv="bf16", window=100, sinks=3, seed=3)
        x.scale = scale
        x.check(attend(x, scale=scale))


@pytest.mark.parametrize("kv,scales", [("bf16", None), ("e4m3", "block")])
def test_long_prompt(kv, scales):
    x = Inputs([2500], [2500], hq=2, hkv=1, kv=kv, scales=scales, window=0 if scales else 700, sinks=0 if scales else 9,
               seed=5)
    x.check(attend(x))


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_no_window_equals_plain_prefill(kv):
    x = Inputs([40, 333, 900], [40, 100, 300], hq=8, hkv=2, kv=kv, window=0, seed=3)
    x.window = 1000
    got = attend(x).double()
    ref = torch.empty_like(x.q_d)
    pkv.pkv_attention_prefill(ref, x.q_d, x.k_cache, x.v_cache, x.tables_d, x.ctx_d, x.start, x.desc, x.scale,
                              300, x.k_scale, x.v_scale)
    assert (got - ref.double()).abs().max().item() <= 2.0 ** -5


def test_one_token_chunks_equal_decode():
    x = Inputs([400, 33, 1100], hq=8, hkv=2, kv="e4m3", scales="block", window=300, sinks=4, seed=9)
    a = attend(x).double()
    ws = pkv.window_workspace_for(3, 8, x.max_blocks, x.desc, 300, 4)
    b = torch.empty_like(x.q_d)
    pkv.pkv_attention_decode_block_scaled(b, x.q_d, x.k_cache, x.v_cache, x.block_scales, x.tables_d, x.ctx_d, x.desc,
                                          x.scale, 300, 4, workspace=ws)
    x.check(b)
    assert (a - b.double()).abs().max().item() <= 2.0 ** -5 * float(a.abs().max())


def test_bad_tables_and_lengths_give_nan_and_status_and_nothing_else():
    x = Inputs([400, 400, 400, 400, 50], [90, 90, 90, 90, 50], hq=4, hkv=2, kv="bf16", window=200, sinks=4, seed=1)
    x.tables_d[1, 20] = x.nb
    x.ctx_d[2], x.ctx_d[3] = x.max_blocks * x.t + 1, 89
    out = attend(x)
    assert pkv.pkv_device_status(clear=True) == pkv.PKV_DEVICE_BAD_TABLE | pkv.PKV_DEVICE_BAD_LENGTH
    assert torch.isnan(out[180:360]).all() and not torch.isnan(out[:90]).any() and not torch.isnan(out[360:]).any()
    # the queries that do not see the bad block's positions may keep their values; those that do are NaN
    assert torch.isnan(out[90:180]).any()
    # a chunk longer than declared
    y = Inputs([400, 90], [300, 20], hq=4, hkv=2, kv="bf16", window=200, sinks=4, seed=1)
    out = attend(y, max_query_len=64)
    assert pkv.pkv_device_status(clear=True) == pkv.PKV_DEVICE_BAD_LENGTH
    assert torch.isnan(out[:300]).all() and not torch.isnan(out[300:]).any()


def test_rows_outside_the_chunks_are_left_alone():
    x = Inputs([100, 30], [40, 0], hq=4, hkv=2, kv="bf16", window=50, sinks=4, seed=2)
    x.q_d = torch.cat([x.q_d, torch.ones_like(x.q_d[:5])])
    out = torch.full_like(x.q_d, 7.0)
    attend(x, out=out)
    assert (out[40:] == 7).all()
    x.check(out[:40])


def test_captured_and_replayed_on_another_stream():
    x = Inputs([400, 900, 33], [100, 300, 33], hq=8, hkv=2, kv="e4m3", scales="block", window=500, sinks=4, seed=2)
    want = attend(x)
    out = torch.full_like(want, float("nan"))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        pkv.pkv_attention_prefill_block_scaled(out, x.q_d, x.k_cache, x.v_cache, x.block_scales, x.tables_d, x.ctx_d,
                                               x.start, x.desc, x.scale, 300, 500, 4, torch.cuda.current_stream())
    for _ in range(2):
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


@pytest.mark.parametrize("window,sinks", [(2 ** 31 - 1, 0), (2 ** 31 - 1, 2 ** 31 - 1), (5, 2 ** 31 - 1)])
def test_the_largest_windows_sinks_and_chunk_bounds(window, sinks):
    x = Inputs(CTX, NEW, hq=4, hkv=2, kv="bf16", window=window, sinks=sinks, seed=6)
    x.check(attend(x, max_query_len=2 ** 31 - 1))
    assert pkv.pkv_device_status() == 0


@pytest.mark.parametrize("hq", [129, 300, 1024])
def test_many_heads_of_one_kv_head(hq):
    """A position's heads over several tiles, and over several units."""
    x = Inputs([50, 9], [5, 2], hq=hq, hkv=1, d=64, kv="f16", q="f16", window=20, sinks=3, seed=hq)
    x.check(attend(x))


def test_more_heads_than_that_are_refused():
    x = Inputs([5], [2], hq=1025, hkv=1, d=64, kv="f16", q="f16", window=20, seed=1)
    with pytest.raises(pkv.PkvError, match="query heads per KV head"):
        attend(x)


def test_two_calls_at_once():
    xs = [Inputs([400, 900, 33], [100, 300, 33], hq=8, hkv=2, kv="bf16", window=w, sinks=4, seed=w) for w in (500, 90)]
    want = [attend(x) for x in xs]
    outs = [torch.full_like(w, float("nan")) for w in want]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for x, out, st in zip(xs, outs, streams):
            st.wait_stream(torch.cuda.current_stream())
            pkv.pkv_attention_prefill_window(out, x.q_d, x.k_cache, x.v_cache, x.tables_d, x.ctx_d, x.start, x.desc,
                                             x.window, x.sinks, x.scale, 300, stream=st)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))


@pytest.mark.parametrize("scales", [None, "block"])
def test_offsets_past_32_bits(scales):
    """Contexts in the last blocks of a cache of more than 2^32 elements."""
    x = Inputs([40, 33, 100], [40, 2, 70], hq=8, hkv=8, kv="e4m3", scales=scales, window=60, sinks=3, seed=7)
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


@pytest.mark.parametrize("seqs", [3, 40])
def test_a_query_start_out_of_order_sets_the_status(seqs):
    """Few and many sequences: a chunk outside the inputs is not written and says so."""
    x = Inputs([60] * seqs, [10] * seqs, hq=4, hkv=2, kv="bf16", window=50, sinks=4, seed=2)
    x.start[-1] = x.total + 30
    out = torch.full_like(x.q_d, 7.0)
    attend(x, out=out)
    assert pkv.pkv_device_status(clear=True) == pkv.PKV_DEVICE_BAD_LENGTH
    assert (out[-10:] == 7).all() and not (out[:-10] == 7).all(dim=(1, 2)).any()


@pytest.mark.parametrize("seqs", [31, 32, 33, 70])
def test_many_sequences(seqs):
    """The scheduler ranks up to 32 sequences and searches among more."""
    r = np.random.RandomState(seqs)
    ctx = r.randint(1, 200, size=seqs)
    x = Inputs(ctx, [int(r.randint(0, c + 1)) for c in ctx], hq=6, hkv=2, kv="bf16", window=64, sinks=3, seed=seqs)
    x.check(attend(x))
    assert pkv.pkv_device_status() == 0
