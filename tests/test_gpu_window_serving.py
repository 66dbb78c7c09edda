"""The operators together, as a serving loop uses them: a prompt appended in
chunks with rotation and attended by the prefill call, then tokens appended
and decoded, with the allocator's tables, forks and copy-on-write, over a
block-scaled E4M3 cache and over a 16-bit cache whose blocks behind the window
go back to the pool.  The oracle follows every byte of the cache and every
output."""
import numpy as np
import pytest
import torch

from oracle import append as OA
from oracle import e4m3
from oracle import window as OW

import paged_kv_cache_137_gb300 as pkv

pytestmark = pytest.mark.gpu

HQ, HKV, D, T = 8, 2, 128, 16


@pytest.fixture(scope="module", autouse=True)
def built():
    pkv.build()
    assert torch.cuda.is_available()
    pkv.pkv_device_status(clear=True)


class Loop:
    def __init__(self, kv, window, sinks, seed, num_blocks=300):
        self.kv, self.window, self.sinks = kv, window, sinks
        self.pool = pkv.Pool(num_blocks, T, np.random.RandomState(seed).permutation(num_blocks))
        self.desc = pkv.kv_desc(num_blocks, HKV, D, T, kv)
        self.k_cache, self.v_cache = pkv.empty_cache(self.desc, fill_byte=0xFF)
        self.scales = pkv.empty_block_scales(self.desc) if kv == "e4m3" else None
        self.table = pkv.rope_table(2048, D)
        self.rope = pkv.rope(self.table)
        self.gen = torch.Generator().manual_seed(seed)
        shape = self.desc.cache_shape
        self.o_bytes = [np.full(shape, 0xFF, np.uint8) for _ in range(2)]
        self.o_scales = np.zeros(shape[:2] + (2,), np.float32)
        self.o_values = [np.full(shape, np.nan) for _ in range(2)]

    def copies(self, cow):
        if len(cow) == 0:
            return
        pkv.pkv_copy_blocks([self.k_cache], [self.v_cache], cow, self.desc)
        if self.scales is not None:
            pkv.pkv_copy_block_scales([self.scales], cow, self.desc)
        for s, d in cow:
            for x in self.o_bytes + self.o_values + [self.o_scales]:
                x[d] = x[s]

    def step(self, ids, n):
        """Append n[i] tokens to sequence ids[i] and attend from them."""
        for s, k in zip(ids, n):
            _, cow = self.pool.seq_append(s, k)
            self.copies(cow)
        tables, ctx = self.pool.block_tables(ids, 64)
        n = np.asarray(n)
        total = int(n.sum())
        qkv = torch.randn((total, (HQ + 2 * HKV) * D), generator=self.gen).mul(1.5).bfloat16()
        dev = qkv.cuda()
        q, k, v = (dev[:, a * D:b * D].unflatten(1, (b - a, D)) for a, b in ((0, HQ), (HQ, HQ + HKV), (HQ + HKV, HQ + 2 * HKV)))
        one = bool((n == 1).all())
        start = torch.from_numpy(np.concatenate([[0], np.cumsum(n)]).astype(np.int32)).cuda()
        t_d, c_d = torch.from_numpy(tables).cuda(), torch.from_numpy(ctx).cuda()
        q_rot = torch.empty((total, HQ, D), dtype=torch.bfloat16, device="cuda")
        out = torch.empty_like(q_rot)
        pkv.pkv_append(self.k_cache, self.v_cache, k, v, t_d, c_d, self.desc, query_start=None if one else start,
                       max_query_len=int(n.max()), rope=self.rope, q=q, q_out=q_rot, block_scales=self.scales)
        scale = D ** -0.5
        if one:
            ws = pkv.window_workspace_for(len(ids), HQ, 64, self.desc, self.window, self.sinks, 64)
            if self.scales is None:
                pkv.pkv_attention_decode_window(out, q_rot, self.k_cache, self.v_cache, t_d, c_d, self.desc, self.window,
                                                self.sinks, scale, partition_tokens=64, workspace=ws)
            else:
                pkv.pkv_attention_decode_block_scaled(out, q_rot, self.k_cache, self.v_cache, self.scales, t_d, c_d,
                                                      self.desc, scale, self.window, self.sinks, 64, ws)
        elif self.scales is None:
            pkv.pkv_attention_prefill_window(out, q_rot, self.k_cache, self.v_cache, t_d, c_d, start, self.desc,
                                             self.window, self.sinks, scale, int(n.max()))
        else:
            pkv.pkv_attention_prefill_block_scaled(out, q_rot, self.k_cache, self.v_cache, self.scales, t_d, c_d, start,
                                                   self.desc, scale, int(n.max()), self.window, self.sinks)
        torch.cuda.synchronize()
        assert pkv.pkv_device_status() == 0
        self.check(tables, ctx, n, qkv, q_rot, out, scale)

    def check(self, tables, ctx, n, qkv, q_rot, out, scale):
        pos = np.concatenate([np.arange(c - k, c) for c, k in zip(ctx, n)])
        rows = qkv.float().numpy().reshape(len(pos), -1, D)
        table = self.table.cpu().numpy()
        q = torch.from_numpy(OA.rotate(rows[:, :HQ], table, pos, False)).bfloat16()
        assert torch.equal(q_rot.cpu(), q)
        new = [OA.rotate(rows[:, HQ:HQ + HKV], table, pos, False), rows[:, HQ + HKV:]]
        for w, cache in enumerate((self.k_cache, self.v_cache)):
            if self.kv == "e4m3":
                OA.append_block_scaled(self.o_bytes[w], self.o_scales, w, new[w], tables, ctx, n)
                assert np.array_equal(cache.cpu().numpy(), self.o_bytes[w])
                self.o_values[w] = e4m3.decode(self.o_bytes[w]) * self.o_scales[:, :, w, None, None].astype(np.float64)
            else:
                x = torch.from_numpy(np.ascontiguousarray(new[w])).bfloat16().double().numpy()
                OA.append_values(self.o_values[w], x, tables, ctx, n)
                assert np.array_equal(cache.double().cpu().numpy(), self.o_values[w], equal_nan=True)
        if self.kv == "e4m3":
            assert np.array_equal(self.scales.cpu().numpy(), self.o_scales)
        ref, mag, top = OW.paged_attention_window(q.double().numpy(), *self.o_values, tables, ctx, n, scale, self.window,
                                                  self.sinks)
        # roundings of q and P (bf16 products, or f16 ones with q rounded to
        # f16), fp32 sums, the bf16 output; f16 weights below 2^-25
        u = 2.0 ** -8 if self.kv == "bf16" else 2.0 ** -11
        dl = ((0 if self.kv == "bf16" else 2.0 ** -11) + 140 * 2.0 ** -24) * top[:, :, None]
        rel = np.expm1(2 * dl) + u + 1100 * 2.0 ** -24
        bound = 1.01 * rel * mag + 2.0 ** -8 * np.abs(ref) + 1100 * 2.0 ** -25 * 8
        assert (np.abs(out.double().cpu().numpy() - ref) <= bound).all()


@pytest.mark.parametrize("kv,window,sinks", [("e4m3", 0, 0), ("e4m3", 100, 4), ("bf16", 70, 5)])
def test_prompt_forks_and_decode(kv, window, sinks):
    x = Loop(kv, window, sinks, seed=window)
    for s in (1, 2):
        x.pool.seq_create(s)
    x.step([1, 2], [200, 37])          # prompts
    x.step([1, 2], [150, 1])           # a second chunk beside a decode token
    x.pool.seq_fork(1, 3)              # forked inside a block: copy-on-write
    for _ in range(20):
        x.step([1, 2, 3], [1, 1, 1])
    x.pool.seq_free(2)
    x.pool.seq_create(4)
    x.step([4, 1], [90, 3])            # its blocks, reused: stale scales are forgotten
    for _ in range(4):
        x.step([3, 4, 1], [1, 1, 1])
