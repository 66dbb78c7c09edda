"""Inputs and error bounds shared by the windowed and block-scaled attention
tests (decode and prefill)."""
import numpy as np
import torch

from oracle import e4m3
from oracle import window as OW

import paged_kv_cache_137_gb300 as pkv

TORCH = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


class Inputs:
    """A scrambled pool, queries, and what must not matter: NaN bytes behind
    each context's end and in every block nobody owns, freed table entries
    where no query of the call sees the block."""

    def __init__(self, ctx, n=None, *, hq=8, hkv=2, d=128, t=16, kv="bf16", q="bf16", scales=None, window=0,
                 sinks=0, seed=0, spread=6, k_gain=1.0):
        r = np.random.RandomState(seed)
        self.ctx = np.asarray(ctx)
        self.n = np.ones(len(ctx), dtype=int) if n is None else np.asarray(n)
        self.hq, self.hkv, self.d, self.t, self.kv, self.qt = hq, hkv, d, t, kv, q
        self.window, self.sinks, self.scale = window, sinks, d ** -0.5
        per = -(-self.ctx // t)
        self.nb = int(per.sum()) + 5
        order = r.permutation(self.nb)
        self.max_blocks = max(1, int(per.max()))
        self.tables = np.full((len(ctx), self.max_blocks), -1, dtype=np.int32)
        at = 0
        for s, k in enumerate(per):
            self.tables[s, :k] = order[at:at + k]
            at += k
        shape = (self.nb, hkv, t, d)
        vals = [r.randn(*shape) * k_gain, r.randn(*shape)]
        self.head_scales = self.block_scales = None
        self.k_scale = self.v_scale = 1.0
        if kv == "e4m3":
            if scales == "block":
                # power-of-two scales over a wide range
                e = r.randint(-spread, spread + 1, size=(self.nb, hkv, 2))
                sc = np.exp2(e - 7.0)
                sc[..., 0] = np.exp2(-7.0 + r.randint(-1, 2, size=(self.nb, hkv)))
                self.block_scales = torch.from_numpy(sc.astype(np.float32)).cuda()
                k_sc, v_sc = sc[..., 0][:, :, None, None], sc[..., 1][:, :, None, None]
                bits = [e4m3.encode(vals[0] / k_sc), e4m3.encode(vals[1] * 100)]
            elif scales == "head":
                rows = np.exp2(r.uniform(-7, -5, size=(4, hkv))).astype(np.float32)
                self.head_scales = torch.from_numpy(rows).cuda()
                k_sc, v_sc = (rows[i].astype(np.float64)[None, :, None, None] for i in (0, 1))
                bits = [e4m3.encode(vals[0] / k_sc), e4m3.encode(vals[1] / v_sc)]
            else:
                self.k_scale, self.v_scale = float(np.float32(0.013)), float(np.float32(0.007))
                k_sc, v_sc = self.k_scale, self.v_scale
                bits = [e4m3.encode(vals[0] / k_sc), e4m3.encode(vals[1] / v_sc)]
            self.values = [e4m3.decode(bits[0]) * k_sc, e4m3.decode(bits[1]) * v_sc]
            raw = [torch.from_numpy(b.astype(np.uint8)) for b in bits]
        else:
            raw = [torch.from_numpy(x).to(TORCH[kv]) for x in vals]
            self.values = [x.double().numpy() for x in raw]
        # poison what nobody may read
        owned = np.zeros((self.nb, t), dtype=bool)
        freed = self.tables.copy()
        for s, c in enumerate(self.ctx):
            first = int(c - self.n[s])
            w0 = max(0, first + 1 - window) if window else 0
            s0 = sinks if window else 0
            for j in range(per[s]):
                p = np.arange(j * t, min((j + 1) * t, int(c)))
                see = p[(p >= w0) | (p < s0)]
                if len(see) == 0 or self.n[s] == 0:
                    freed[s, j] = -1
                else:
                    owned[self.tables[s, j], see % t] = True
        self.tables_d = torch.from_numpy(freed).cuda()
        for x in raw:
            hide = torch.from_numpy(~owned)[:, None, :, None].expand(shape)
            x.view(torch.uint8).view(*shape, -1)[hide] = 0xFF
        self.k_cache, self.v_cache = (x.cuda() for x in raw)
        if self.block_scales is not None:
            lost = torch.from_numpy(~owned.any(axis=1)).cuda()
            self.block_scales[lost] = float("nan")
        self.total = int(self.n.sum())
        g = torch.Generator().manual_seed(seed)
        self.q = torch.randn((self.total, hq, d), generator=g).to(TORCH[q])
        self.q_d = self.q.cuda()
        self.ctx_d = torch.from_numpy(self.ctx.astype(np.int32)).cuda()
        self.start = torch.from_numpy(np.concatenate([[0], np.cumsum(self.n)]).astype(np.int32)).cuda()
        self.desc = pkv.kv_desc(self.nb, hkv, d, t, kv, self.head_scales)

    def oracle(self):
        return OW.paged_attention_window(self.q.double().numpy(), *self.values, self.tables, self.ctx, self.n,
                                         self.scale, self.window, self.sinks)

    def check(self, got, extra_rounding=0.0):
        """The output against fp64 within a bound derived from the roundings
        the kernels make.  With u(t) = eps(t) / 2 the largest relative rounding
        of type t:
        * q rounded to the MMA's type (exact unless bf16 queries meet f16
          products: u(f16), and an absolute half step below f16's normals), and
          fp32 sums of d products (each sum off by at most d u(f32) of the
          magnitudes), move a logit by at most dl = (u_q + (d + 4) u(f32)) *
          sum |q_d K_d| scale, so a weight by a factor exp(2 dl);
        * P rounded to the MMA's type: u_p of each weight, and fp32 exponents
          and sums over c keys: (c + 16) u(f32);
        * extra_rounding: a further relative rounding of each product;
        all of it relative to sum w |V|; and the output rounded once, u(out).
        fp16 P underflows below 2^-24 of the largest weight: c 2^-25 more."""
        out, mag, top = self.oracle()
        u32, u16 = 2.0 ** -24, 2.0 ** -11
        u_q = u16 if self.kv == "e4m3" and self.qt == "bf16" else 0.0
        u_p = {"f32": 0.0, "bf16": 2.0 ** -8, "f16": u16, "e4m3": u16}[self.kv]
        c = int(self.ctx.max())
        dl = (u_q + extra_rounding + (self.d + 4) * u32) * top[:, :, None]
        rel = np.expm1(2 * dl) + u_p + extra_rounding + (c + 16) * u32
        vmax = np.abs(np.concatenate([v[np.isfinite(v)] for v in (self.values[1],)])).max()
        u_out = {"f32": u32, "bf16": 2.0 ** -8, "f16": u16}[self.qt]
        tiny = c * 2.0 ** -25 * vmax if self.kv in ("f16", "e4m3") else 1e-30
        bound = rel * mag * (1 + 2 * rel) + u_out * (np.abs(out) + rel * mag) + tiny + 2.0 ** -25
        g = got.double().cpu().numpy()
        assert not np.isnan(g).any(), "NaN in the output"
        over = np.abs(g - out) / bound
        assert over.max() <= 1, f"{over.max():.3g} of the bound at {np.unravel_index(over.argmax(), over.shape)}"
