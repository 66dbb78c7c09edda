"""pkv_append on the GPU against the oracle, bit for bit: rotated keys and
queries (fp32 arithmetic of one rounding per operation, then one rounding to
the stored type), E4M3 caches with per-tensor, per-head and per-block scales,
strided inputs, chunks that start and end anywhere, and what a call must leave
alone."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import append as OA
from oracle import e4m3

import paged_kv_cache_137_gb300 as pkv

pytestmark = pytest.mark.gpu

TORCH = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BITS = {"f32": torch.int32, "f16": torch.int16, "bf16": torch.int16}


@pytest.fixture(scope="module", autouse=True)
def built():
    pkv.build()
    assert torch.cuda.is_available()


@pytest.fixture(autouse=True)
def clean_status():
    pkv.pkv_device_status(clear=True)
    yield
    pkv.pkv_device_status(clear=True)


class Batch:
    """A pool, tables over scrambled blocks and one chunk per sequence."""

    def __init__(self, ctx, n, *, hq=8, hkv=2, d=128, t=16, src="bf16", kv="bf16", rotary=None, inter=False,
                 seed=0, packed=True):
        r = np.random.RandomState(seed)
        self.ctx, self.n = np.asarray(ctx), np.asarray(n)
        self.hq, self.hkv, self.d, self.t, self.src, self.kv = hq, hkv, d, t, src, kv
        self.rotary, self.inter = d if rotary is None else rotary, inter
        per = -(-np.maximum(self.ctx, 0) // t)
        self.nb = int(per.sum()) + 4
        order = r.permutation(self.nb)
        self.max_blocks = max(1, int(per.max()))
        self.tables = np.full((len(ctx), self.max_blocks), -1, dtype=np.int32)
        at = 0
        for s, k in enumerate(per):
            self.tables[s, :k] = order[at:at + k]
            at += k
        self.desc = pkv.kv_desc(self.nb, hkv, d, t, kv)
        g = torch.Generator().manual_seed(seed)
        self.total = int(self.n.sum())
        rows = [torch.randn((self.total, h, d), generator=g).mul(2.0).to(TORCH[src]) for h in (hq, hkv, hkv)]
        self.q_host, self.k_host, self.v_host = rows
        if packed:
            width = (hq + 2 * hkv) * d
            buf = torch.cat([x.reshape(self.total, -1) for x in rows], dim=1).cuda()
            assert buf.shape[1] == width
            self.q = buf[:, :hq * d].unflatten(1, (hq, d))
            self.k = buf[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d))
            self.v = buf[:, (hq + hkv) * d:].unflatten(1, (hkv, d))
        else:
            self.q, self.k, self.v = (x.cuda() for x in rows)
        self.q_out = torch.full((self.total, hq, d), 7.0, dtype=TORCH[src], device="cuda")
        self.start = torch.from_numpy(np.concatenate([[0], np.cumsum(self.n)]).astype(np.int32)).cuda()
        self.tables_d = torch.from_numpy(self.tables).cuda()
        self.ctx_d = torch.from_numpy(self.ctx.astype(np.int32)).cuda()
        self.table = pkv.rope_table(self.max_blocks * t, self.rotary) if self.rotary else None
        self.rope = pkv.rope(self.table, inter) if self.rotary else None
        # a cache that already holds something everywhere
        shape = self.desc.cache_shape
        if kv == "e4m3":
            self.before = [e4m3.encode(r.randn(*shape) * 40).astype(np.uint8) for _ in range(2)]
            self.k_cache, self.v_cache = (torch.from_numpy(x.copy()).cuda() for x in self.before)
        else:
            held = [torch.randn(shape, generator=g).to(TORCH[kv]) for _ in range(2)]
            self.before = held
            self.k_cache, self.v_cache = (x.cuda() for x in held)

    def positions(self):
        return np.concatenate([np.arange(c - k, c) for c, k in zip(self.ctx, self.n)] or [np.zeros(0)]).astype(int)

    def rotated(self, x):
        """fp32 rows as the call computes them, from the same table."""
        f = x.float().numpy()
        return OA.rotate(f, self.table.cpu().numpy(), self.positions(), self.inter) if self.rotary else f

    def call(self, one=False, **kw):
        a = dict(query_start=None if one else self.start, max_query_len=int(self.n.max()), rope=self.rope,
                 q=self.q, q_out=self.q_out)
        a.update(kw)
        pkv.pkv_append(self.k_cache, self.v_cache, self.k, self.v, self.tables_d, self.ctx_d, self.desc, **a)
        torch.cuda.synchronize()

    def check_q(self):
        want = torch.from_numpy(self.rotated(self.q_host)).to(TORCH[self.src])
        assert torch.equal(self.q_out.cpu().view(BITS[self.src]), want.view(BITS[self.src]))

    def check_values(self):
        """A 16/32-bit cache: the new rows' bits, everything else as it was."""
        for cache, before, rows in ((self.k_cache, self.before[0], self.rotated(self.k_host)),
                                    (self.v_cache, self.before[1], self.v_host.float().numpy())):
            want = before.clone()
            x = torch.from_numpy(np.ascontiguousarray(rows)).to(TORCH[self.kv])
            for i, (s, p) in enumerate(self.places()):
                want[self.tables[s, p // self.t], :, p % self.t] = x[i]
            assert torch.equal(cache.cpu().view(BITS[self.kv]), want.view(BITS[self.kv]))

    def places(self):
        return [(s, p) for s in range(len(self.ctx)) for p in range(self.ctx[s] - self.n[s], self.ctx[s])]


CTX = [1, 15, 16, 17, 31, 32, 33, 64, 100]


@pytest.mark.parametrize("rotary,inter", [(0, False), (16, False), (16, True), (48, False), (64, True)])
@pytest.mark.parametrize("d,t", [(64, 16), (128, 32)])
@pytest.mark.parametrize("src", ["bf16", "f16", "f32"])
def test_values_and_rotation(src, d, t, rotary, inter):
    b = Batch(CTX, np.minimum(CTX, [1, 15, 7, 17, 20, 1, 33, 5, 99]), d=d, t=t, src=src, kv=src, rotary=rotary,
              inter=inter, seed=rotary)
    b.call()
    b.check_q()
    b.check_values()


@pytest.mark.parametrize("packed", [True, False])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (28, 4), (40, 8), (15, 3)])
def test_one_token_each(hq, hkv, packed):
    b = Batch(CTX, [1] * len(CTX), hq=hq, hkv=hkv, inter=False, seed=hq, packed=packed)
    b.call(one=True)
    b.check_q()
    b.check_values()


def test_a_full_rotary_row_and_many_tokens():
    """Enough tokens for the wide form (several rows per thread at a time)."""
    b = Batch([3000, 1301], [3000, 1300], hq=8, hkv=2, seed=3)
    b.call()
    b.check_q()
    b.check_values()


def test_keys_alone_and_queries_in_place():
    b = Batch(CTX, [1] * len(CTX), seed=5)
    b.call(one=True, q=None, q_out=None)
    b.check_values()
    assert (b.q_out == 7).all()
    c = Batch(CTX, [1] * len(CTX), seed=5, packed=False)
    c.call(one=True, q_out=c.q)
    c.q_out = c.q
    c.check_q()


@pytest.mark.parametrize("src", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("heads", [False, True])
def test_tensor_and_head_scales(src, heads):
    b = Batch(CTX, np.minimum(CTX, 20), src=src, kv="e4m3", seed=9)
    inv = np.array([[3.5, 17.0], [1.25, 40.0]], dtype=np.float32)   # K, V by head
    kw = {}
    if heads:
        rows = np.concatenate([1 / inv, inv]).astype(np.float32)
        b.desc = pkv.with_head_scales(b.desc, torch.from_numpy(rows).cuda())
    else:
        inv = np.repeat(inv[:, :1], b.hkv, axis=1)
        kw = dict(k_inv_scale=float(inv[0, 0]), v_inv_scale=float(inv[1, 0]))
    b.call(**kw)
    b.check_q()
    for cache, before, rows, i in ((b.k_cache, b.before[0], b.rotated(b.k_host), inv[0]),
                                   (b.v_cache, b.before[1], b.v_host.float().numpy(), inv[1])):
        want = before.copy()
        x = e4m3.quantize_fp32(rows, i[None, :, None])
        for k, (s, p) in enumerate(b.places()):
            want[b.tables[s, p // b.t], :, p % b.t] = x[k]
        assert np.array_equal(cache.cpu().numpy(), want)


def block_scaled_oracle(b, scales, caches):
    for w, rows in enumerate((b.rotated(b.k_host), b.v_host.float().numpy())):
        OA.append_block_scaled(caches[w], scales, w, rows, b.tables, b.ctx, b.n)


@pytest.mark.parametrize("src", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("d,t", [(64, 16), (64, 32), (128, 16), (128, 32)])
@pytest.mark.parametrize("one", [True, False])
def test_block_scales(src, d, t, one):
    """Fresh blocks, blocks whose scale holds and blocks whose scale grows (by
    much and by little), several tokens and blocks per chunk."""
    n = [1] * len(CTX) if one else np.minimum(CTX, [1, 4, 7, 17, 20, 1, 33, 50, 99])
    b = Batch(CTX, n, src=src, kv="e4m3", d=d, t=t, rotary=d // 2, seed=d + t)
    r = np.random.RandomState(t)
    # 2^-43 .. 2^2 against new values around 2^-7: some grow, some hold
    scales = np.exp2(r.choice([-40, -20, -10, -8, -7, -6, 2], size=(b.nb, b.hkv, 2))).astype(np.float32)
    dev = torch.from_numpy(scales.copy()).cuda()
    caches = [x.copy() for x in b.before]
    block_scaled_oracle(b, scales, caches)
    b.call(one=one, block_scales=dev)
    b.check_q()
    assert np.array_equal(dev.cpu().numpy(), scales)
    assert np.array_equal(b.k_cache.cpu().numpy(), caches[0])
    assert np.array_equal(b.v_cache.cpu().numpy(), caches[1])
    # the same call again: nothing grows, nothing changes
    b.call(one=one, block_scales=dev)
    assert np.array_equal(dev.cpu().numpy(), scales)
    assert np.array_equal(b.k_cache.cpu().numpy(), caches[0])


def test_block_scales_at_the_ends_of_their_range():
    """Zeros, values far below and above the scales' range, infinities and NaN
    among the new rows, and scales never written."""
    b = Batch([20, 20, 20, 20, 20, 20], [4] * 6, hq=2, hkv=2, src="f32", kv="e4m3", rotary=0, seed=1)
    rows = torch.zeros(24, 2, 128)
    for s, x in enumerate([0.0, 1e-20, 3e30, 448.0, 448.001, 1.0]):
        rows[4 * s:4 * s + 4] = x
    rows[21, 0, 3], rows[21, 0, 4], rows[22, 1, 5] = float("inf"), float("-inf"), float("nan")
    b.k_host = b.v_host = rows
    b.k = b.v = rows.cuda()
    scales = np.zeros((b.nb, 2, 2), dtype=np.float32)
    scales[:, 1] = 1.0
    dev = torch.from_numpy(scales.copy()).cuda()
    caches = [x.copy() for x in b.before]
    block_scaled_oracle(b, scales, caches)
    b.call(block_scales=dev, q=None, q_out=None)
    assert np.array_equal(dev.cpu().numpy(), scales)
    assert np.array_equal(b.k_cache.cpu().numpy(), caches[0])
    assert np.array_equal(b.v_cache.cpu().numpy(), caches[1])
    # a scale that is no number counts as never written
    dev[:] = float("nan")
    b.call(block_scales=dev, q=None, q_out=None)
    assert torch.isfinite(dev[b.tables_d[:, 1].long()]).all()


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_invalid_lengths_and_tables_write_nothing_of_theirs(kv):
    b = Batch([40, 40, 40, 40, 40], [3, 3, 3, 3, 3], kv=kv, seed=2)
    scales = torch.ones((b.nb, b.hkv, 2), device="cuda") if kv == "e4m3" else None
    good = [0, 4]
    b.ctx_d[1], b.ctx_d[2] = 2, b.max_blocks * b.t + 1     # shorter than its chunk; past the table
    b.tables_d[3, 2] = b.nb                                # outside the pool
    b.call(block_scales=scales)
    assert pkv.pkv_device_status(clear=True) == pkv.PKV_DEVICE_BAD_LENGTH | pkv.PKV_DEVICE_BAD_TABLE
    nan = torch.isnan(b.q_out.float()).all(dim=(1, 2)).cpu().numpy()
    assert nan.tolist() == [False] * 3 + [True] * 6 + [False] * 6
    for cache, before in ((b.k_cache, b.before[0]), (b.v_cache, b.before[1])):
        same = torch.as_tensor(before).view(torch.uint8).flatten(1).eq(cache.cpu().view(torch.uint8).flatten(1))
        changed = {int(i) for i in torch.nonzero(~same.all(dim=1)).flatten()}
        assert changed <= {int(b.tables[s, 2]) for s in good} and changed
    # a position past the angle table, and a chunk longer than declared
    c = Batch([40, 40], [3, 20], kv=kv, seed=2)
    c.rope = pkv.rope(c.table[:39].contiguous())
    c.call(block_scales=None if scales is None else torch.ones((c.nb, c.hkv, 2), device="cuda"))
    assert pkv.pkv_device_status(clear=True) == pkv.PKV_DEVICE_BAD_LENGTH
    assert torch.isnan(c.q_out.float()).all()
    e = Batch([40, 40], [3, 20], kv=kv, seed=2)
    e.call(max_query_len=4, block_scales=None if scales is None else torch.ones((e.nb, e.hkv, 2), device="cuda"))
    assert pkv.pkv_device_status(clear=True) == pkv.PKV_DEVICE_BAD_LENGTH
    assert torch.isnan(e.q_out[3:].float()).all() and not torch.isnan(e.q_out[:3].float()).any()


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_the_largest_longest_chunk(kv):
    """max_query_len bounds the chunks from above: any larger value, the largest
    of its type as well, gives the same call."""
    a, b = (Batch(CTX, [1, 3, 16, 5, 0, 32, 20, 64, 7], kv=kv, seed=8) for _ in range(2))
    sa, sb = ((torch.ones((x.nb, x.hkv, 2), device="cuda") if kv == "e4m3" else None) for x in (a, b))
    a.call(block_scales=sa)
    b.call(block_scales=sb, max_query_len=2 ** 31 - 1)
    assert pkv.pkv_device_status() == 0
    assert torch.equal(a.q_out, b.q_out) and (sa is None or torch.equal(sa, sb))
    assert torch.equal(a.k_cache.view(torch.uint8), b.k_cache.view(torch.uint8))
    assert torch.equal(a.v_cache.view(torch.uint8), b.v_cache.view(torch.uint8))


def test_rows_outside_the_chunks_are_left_alone():
    """Rows before the first chunk and behind the last, an empty chunk, and an
    empty sequence of a one-token call."""
    b = Batch([20, 30, 9], [5, 0, 4], seed=4)
    extra = 3
    for name in ("q", "k", "v"):
        x = getattr(b, name)
        setattr(b, name, torch.cat([x, torch.full((extra,) + x.shape[1:], 5.0, dtype=x.dtype, device="cuda")]))
    b.q_out = torch.full((b.total + extra, b.hq, b.d), 7.0, dtype=TORCH["bf16"], device="cuda")
    b.call()
    assert (b.q_out[b.total:] == 7).all()
    b.q_out = b.q_out[:b.total]
    b.check_q()
    b.check_values()
    c = Batch([20, 0, 9], [1, 1, 1], seed=4)
    before = [c.k_cache.clone(), c.v_cache.clone()]
    c.call(one=True)
    assert (c.q_out[1] == 0).all() and pkv.pkv_device_status() == 0
    for cache, was, row in ((c.k_cache, before[0], None), (c.v_cache, before[1], c.v)):
        changed = torch.nonzero((cache != was).flatten(1).any(dim=1)).flatten().tolist()
        assert set(changed) == {int(c.tables[0, 1]), int(c.tables[2, 0])}


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_prepared_captured_and_on_another_stream(kv):
    """A prepared call, replayed from a graph on a stream of its own, gives the
    plain call's bytes."""
    a, b = (Batch(CTX, [1] * len(CTX), kv=kv, seed=6) for _ in range(2))
    sa, sb = ((torch.full((x.nb, x.hkv, 2), 2.0 ** -9, device="cuda") if kv == "e4m3" else None) for x in (a, b))
    a.call(one=True, block_scales=sa)
    step = pkv.prepare_append(b.k_cache, b.v_cache, b.k, b.v, b.tables_d, b.ctx_d, b.desc, rope=b.rope, q=b.q,
                              q_out=b.q_out, block_scales=sb)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step(torch.cuda.current_stream())
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(a.q_out, b.q_out)
    assert torch.equal(a.k_cache.view(torch.uint8), b.k_cache.view(torch.uint8))
    assert torch.equal(a.v_cache.view(torch.uint8), b.v_cache.view(torch.uint8))
    assert sa is None or torch.equal(sa, sb)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("start", [[0, 5, 3, 9], [0, 5, 9, 60], [-2, 0, 4, 9]])
def test_a_query_start_out_of_order_sets_the_status(kv, start):
    """Chunks outside the inputs write nothing and say so; nothing else is hurt."""
    b = Batch([20, 30, 19], [5, 4, 0], kv=kv, seed=4)
    b.start = torch.tensor(start, dtype=torch.int32, device="cuda")
    scales = torch.ones((b.nb, b.hkv, 2), device="cuda") if kv == "e4m3" else None
    b.call(block_scales=scales, max_query_len=9)
    assert pkv.pkv_device_status(clear=True) == pkv.PKV_DEVICE_BAD_LENGTH
    whole = [s for s in range(3) if 0 <= start[s] <= start[s + 1] <= b.total]
    for cache, before in ((b.k_cache, b.before[0]), (b.v_cache, b.before[1])):
        same = torch.as_tensor(before).view(torch.uint8).flatten(1).eq(cache.cpu().view(torch.uint8).flatten(1))
        changed = {int(i) for i in torch.nonzero(~same.all(dim=1)).flatten()}
        assert changed <= {int(x) for s in whole for x in b.tables[s] if x >= 0}


def test_a_rope_filled_by_hand():
    a, b = (Batch(CTX, [1] * len(CTX), seed=9) for _ in range(2))
    b.rope = pkv.pkv_rope(b.table.data_ptr(), b.table.shape[0], b.table.shape[1], 0)
    a.call(one=True)
    b.call(one=True)
    assert torch.equal(a.q_out, b.q_out) and torch.equal(a.k_cache, b.k_cache)


def test_two_calls_at_once():
    """Calls on two streams, each on blocks of its own, give what they give one
    after the other."""
    a, b = (Batch(CTX, [1, 3, 16, 5, 0, 32, 20, 64, 7], kv="e4m3", seed=s) for s in (10, 11))
    both = [Batch(CTX, [1, 3, 16, 5, 0, 32, 20, 64, 7], kv="e4m3", seed=s) for s in (10, 11)]
    scales = [torch.full((x.nb, x.hkv, 2), 2.0 ** -9, device="cuda") for x in (a, b, *both)]
    a.call(block_scales=scales[0])
    b.call(block_scales=scales[1])
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for x, sc, st in zip(both, scales[2:], streams):
            st.wait_stream(torch.cuda.current_stream())
            pkv.pkv_append(x.k_cache, x.v_cache, x.k, x.v, x.tables_d, x.ctx_d, x.desc, query_start=x.start,
                           max_query_len=64, rope=x.rope, q=x.q, q_out=x.q_out, block_scales=sc, stream=st)
    torch.cuda.synchronize()
    for x, y, sx, sy in zip((a, b), both, scales[:2], scales[2:]):
        assert torch.equal(x.q_out, y.q_out) and torch.equal(sx, sy)
        assert torch.equal(x.k_cache, y.k_cache) and torch.equal(x.v_cache, y.v_cache)


def test_copied_blocks_take_their_scales_along():
    desc = pkv.kv_desc(40, 3, 64, 16, "e4m3")
    layers = [torch.rand((40, 3, 2), device="cuda") for _ in range(3)]
    want = [x.clone() for x in layers]
    pairs = np.array([[3, 17], [39, 0], [8, 9]], dtype=np.int32)
    for w in want:
        for s, d in pairs:
            w[d] = w[s]
    pkv.pkv_copy_block_scales(layers, pairs, desc)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(layers, want))
    pkv.pkv_copy_block_scales(layers, np.zeros((0, 2), dtype=np.int32), desc)


def test_offsets_past_32_bits():
    """The last blocks of a cache of more than 2^32 elements."""
    nb = (1 << 32) // (8 * 16 * 128) + 64
    desc = pkv.kv_desc(nb, 8, 128, 16, "e4m3")
    cache = torch.zeros(desc.cache_shape, dtype=torch.uint8, device="cuda")
    scales = pkv.empty_block_scales(desc)
    x = torch.ones((2, 8, 128), dtype=torch.bfloat16, device="cuda")
    tables = torch.tensor([[nb - 1], [nb - 2]], dtype=torch.int32, device="cuda")
    ctx = torch.tensor([1, 1], dtype=torch.int32, device="cuda")
    pkv.pkv_append(cache, cache.clone(), x, x, tables, ctx, desc, block_scales=scales)
    torch.cuda.synchronize()
    assert (scales[nb - 2:] == 2.0 ** -8).all() and (scales[:nb - 2] == 0).all()
    byte = int(e4m3.encode(np.array([256.0]))[0])
    assert (cache[nb - 2:, :, 0] == byte).all() and int(cache.count_nonzero()) == 2 * 8 * 128
