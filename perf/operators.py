"""Cases of the cache append with rotation, of attention over a block-scaled
E4M3 cache and of attention with a sliding window and sinks: inputs, the plain
forms in elementary torch operations, and the calls of the library.

A case names one operator ("op": append, decode or prefill), the cache ("kv":
f32, f16, bf16 or e4m3; "scales": none, tensor or block), the dtype of q, k and
v ("src"), the head layout, the lengths and, for attention, the window (0: the
whole context) and the number of first tokens that stay visible.  The lengths
of a case come from its "lens" seed, so that every pass of a case has the same
work; the values and the physical blocks come from the seed of prepare.
"""
import math
import random

import numpy as np
import torch

own = False

TORCH = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2, "e4m3": 1}
E4M3_MAX = 448.0
MIN_EXP, MAX_EXP = -40, 40    # exponents a block scale may take


def listed():
    return [
        # --- append: one token of each sequence of a decode batch (the
        # smallest launches: latency), 28 query and 4 KV heads
        dict(name="append_step_bf16", op="append", kv="bf16", scales="none", src="bf16", batch=64, hq=28,
             hkv=4, d=128, t=16, lo=256, hi=4096, dist="uniform", new=1, rotary=128, inter=False, lens=11),
        # a chunked prefill's ragged chunks
        dict(name="append_chunk_bf16", op="append", kv="bf16", scales="none", src="bf16", batch=16, hq=28,
             hkv=4, d=128, t=16, lo=1024, hi=4096, dist="uniform", new=512, rotary=128, inter=False, lens=12),
        # a large decode batch into an 8-bit cache with a scale per block and head
        dict(name="append_step_block", op="append", kv="e4m3", scales="block", src="bf16", batch=512, hq=64,
             hkv=8, d=128, t=16, lo=64, hi=8192, dist="log", new=1, rotary=128, inter=False, lens=13),
        # long prompts into the same cache, part of head_dim rotated in
        # adjacent pairs: the largest append
        dict(name="append_prompt_block", op="append", kv="e4m3", scales="block", src="bf16", batch=16, hq=64,
             hkv=8, d=128, t=16, lo=1024, hi=4096, dist="uniform", new=4096, rotary=64, inter=True, lens=14),
        # --- attention over the block-scaled cache: a few short sequences
        # (latency), the large churned batch, and a prefill's chunks
        dict(name="decode_block_small", op="decode", kv="e4m3", scales="block", src="bf16", batch=4, hq=32,
             hkv=8, d=128, t=16, lo=1, hi=128, dist="uniform", window=0, sinks=0, lens=15),
        dict(name="decode_block_churn", op="decode", kv="e4m3", scales="block", src="bf16", batch=512, hq=64,
             hkv=8, d=128, t=16, lo=64, hi=8192, dist="log", window=0, sinks=0, lens=16),
        dict(name="prefill_block_chunk", op="prefill", kv="e4m3", scales="block", src="bf16", batch=16, hq=28,
             hkv=4, d=128, t=16, lo=1024, hi=4096, dist="uniform", new=512, window=0, sinks=0, lens=17),
        # --- a sliding window and sinks: tiny fp32 heads, a decode batch, long
        # contexts with one KV head per query head, chunks, one long prompt
        dict(name="decode_window_f32", op="decode", kv="f32", scales="none", src="f32", batch=4, hq=4, hkv=4,
             d=64, t=16, lo=0, hi=128, dist="uniform", window=33, sinks=2, lens=18),
        dict(name="decode_window_gqa", op="decode", kv="bf16", scales="none", src="bf16", batch=64, hq=28,
             hkv=4, d=128, t=16, lo=256, hi=4096, dist="uniform", window=1024, sinks=4, lens=19),
        dict(name="decode_window_long", op="decode", kv="f16", scales="none", src="f16", batch=8, hq=32,
             hkv=32, d=128, t=32, lo=16384, hi=32768, dist="uniform", window=4096, sinks=4, lens=20),
        dict(name="prefill_window_chunk", op="prefill", kv="bf16", scales="none", src="bf16", batch=16, hq=28,
             hkv=4, d=128, t=16, lo=1024, hi=4096, dist="uniform", new=512, window=1024, sinks=4, lens=21),
        dict(name="prefill_window_prompt", op="prefill", kv="bf16", scales="none", src="bf16", batch=1, hq=32,
             hkv=8, d=128, t=32, lo=8192, hi=8192, dist="uniform", new=8192, window=2048, sinks=4, lens=22),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "append", "decode", "decode", "decode", "prefill", "prefill"])
    hkv = rng.choice([1, 2, 3, 4, 8])
    group = rng.choice([1, 2, 4, 5, 7, 8, 16])
    t = rng.choice([16, 32])
    if op == "append":
        kv = rng.choice(["f32", "f16", "bf16", "e4m3", "e4m3", "e4m3"])
        scales = rng.choice(["tensor", "block", "block"]) if kv == "e4m3" else "none"
        src = rng.choice(["f32", "f16", "bf16"]) if kv == "e4m3" else kv
        d = rng.choice([64, 128])
        hi = _log(rng, 1, 4096)
        new = rng.choice([1, 1, 2, _log(rng, 1, hi), hi])
        batch = max(1, min(_log(rng, 1, 512), 60000 // hi, 400_000_000 // (new * hkv * (group + 2) * d)))
        return dict(op=op, kv=kv, scales=scales, src=src, batch=batch, hq=hkv * group, hkv=hkv, d=d, t=t,
                    lo=max(1, hi // rng.choice([1, 4, 1000])), hi=hi, dist=rng.choice(["uniform", "log"]),
                    new=new, rotary=rng.choice([0, 16, 48, 64, d]),
                    inter=rng.random() < 0.5, lens=rng.randrange(1 << 30))
    window = rng.choice([0, 1, _log(rng, 1, 8192), _log(rng, 1, 8192), _log(rng, 1, 8192)])
    sinks = rng.choice([0, 1, 4, _log(rng, 1, 256)])
    if op == "decode":
        kv = rng.choice(["f32", "f16", "bf16", "e4m3", "e4m3"])
        scales = ("block" if window == 0 else rng.choice(["tensor", "block"])) if kv == "e4m3" else "none"
        if kv != "e4m3" and window == 0:
            window = _log(rng, 1, 8192)
        src = rng.choice(["f16", "bf16"]) if kv == "e4m3" else kv
        hi = _log(rng, 1, 32768)
        batch = max(1, min(_log(rng, 1, 512), 6_000_000 // (hi * hkv)))
        return dict(op=op, kv=kv, scales=scales, src=src, batch=batch, hq=hkv * group, hkv=hkv,
                    d=rng.choice([64, 128]), t=t, lo=hi // rng.choice([1, 3, 40000]), hi=hi,
                    dist="uniform", window=window, sinks=sinks, lens=rng.randrange(1 << 30))
    kv = rng.choice(["f16", "bf16", "e4m3", "e4m3"])
    scales = ("block" if window == 0 else rng.choice(["tensor", "block"])) if kv == "e4m3" else "none"
    if kv != "e4m3" and window == 0:
        window = _log(rng, 1, 8192)
    src = rng.choice(["f16", "bf16"]) if kv == "e4m3" else kv
    hq = hkv * min(group, 8)
    hi = _log(rng, 1, 6000)
    new = rng.choice([1, _log(rng, 1, hi), hi])
    batch = max(1, min(_log(rng, 1, 32), 500_000_000 // (hi * new * hq)))
    return dict(op=op, kv=kv, scales=scales, src=src, batch=batch, hq=hq, hkv=hkv,
                d=128 if kv == "e4m3" else rng.choice([64, 128]), t=t, lo=max(1, hi // rng.choice([1, 3, 10000])),
                hi=hi, dist="uniform", new=new, window=window, sinks=sinks, lens=rng.randrange(1 << 30))


# ------------------------------------------------------------------ lengths
def _lengths(case):
    """(context lengths, new tokens) of the batch, as int64 arrays."""
    r = random.Random(case["lens"])
    lo, hi = case["lo"], case["hi"]
    if case["dist"] == "log":
        ctx = [_log(r, max(lo, 1), hi) for _ in range(case["batch"])]
    else:
        ctx = [r.randint(lo, hi) for _ in range(case["batch"])]
    top = case.get("new", 1)
    if case["op"] == "append" or case["op"] == "prefill":
        # one token each, or chunks of up to `new` tokens, most of them full
        n = [min(c, top if r.random() < 0.6 else r.randint(1, top)) for c in ctx]
    else:
        n = [1] * len(ctx)
    return np.asarray(ctx, dtype=np.int64), np.asarray(n, dtype=np.int64)


def _visible(case, ctx):
    """(first position of the window, sink positions before it) of a query at
    position ctx - 1."""
    if not case["window"]:
        return 0, 0
    w0 = max(0, ctx - case["window"])
    return w0, min(case["sinks"], w0)


def work(case):
    ctx, n = _lengths(case)
    eb, sb = BYTES[case["kv"]], BYTES[case["src"]]
    hq, hkv, d, t = case["hq"], case["hkv"], case["d"], case["t"]
    if case["op"] == "append":
        tok = int(n.sum())
        by = tok * ((hq + 2 * hkv) * d * sb + 2 * hkv * d * eb + hq * d * sb)
        by += min(tok, int(ctx.max())) * case["rotary"] * 4
        blocks = sum(-(-int(c) // t) - (int(c) - int(k)) // t for c, k in zip(ctx, n))
        by += 4 * blocks + 4 * (2 * len(ctx) + 1)
        if case["scales"] == "block":
            by += 16 * blocks * hkv      # K and V scale of each touched block and head, read and written
        return {"bytes": by, "flops": tok * (hq + hkv) * case["rotary"] * 3}
    by, fl = 4 * len(ctx), 0
    for c, k in zip(ctx.tolist(), n.tolist()):
        if c == 0:
            by += hq * d * sb
            continue
        w0, s0 = _visible(case, c - k + 1)       # keys the chunk's first query sees
        keys = c - w0 + s0
        by += 2 * keys * hkv * d * eb + 2 * k * hq * d * sb + 4 * (keys // t)
        if case["scales"] == "block":
            by += 8 * hkv * (-(-keys // t))
        for_rows = np.arange(c - k + 1, c + 1)
        lows = np.maximum(0, for_rows - case["window"]) if case["window"] else np.zeros_like(for_rows)
        seen = for_rows - lows + np.minimum(case["sinks"], lows)
        fl += 4 * int(seen.sum()) * hq * d
    return {"bytes": by, "flops": fl}


# ------------------------------------------------------------------- inputs
def _quantise(x):
    """fp32 -> E4M3 bytes, to nearest even, saturated."""
    return x.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)


def _grow_exponent(amax):
    """The smallest e with amax <= 448 * 2^e, within the range of a block scale."""
    m, e = torch.frexp(amax)
    e = torch.where(amax > 0, e - 9 + (m > 0.875).to(e.dtype), torch.full_like(e, MIN_EXP))
    return e.clamp(MIN_EXP, MAX_EXP)


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(int(seed))
    nprng = np.random.RandomState(int(seed) % (1 << 32))
    ctx, n = _lengths(case)
    b, hq, hkv, d, t = case["batch"], case["hq"], case["hkv"], case["d"], case["t"]
    src = TORCH[case["src"]]

    # a pool handed out in a scrambled order; a few blocks belong to nobody
    per = -(-ctx // t)
    num_blocks = int(per.sum()) + 3
    order = nprng.permutation(num_blocks).astype(np.int32)
    max_blocks = max(1, int(per.max()))
    tables = np.full((b, max_blocks), -1, dtype=np.int32)
    at = np.concatenate([[0], np.cumsum(per)])
    for s in range(b):
        tables[s, :per[s]] = order[at[s]:at[s + 1]]
    st = {"case": case, "ctx_host": ctx, "n_host": n, "num_blocks": num_blocks, "max_blocks": max_blocks,
          "ctx": torch.from_numpy(ctx.astype(np.int32)).to(dev),
          "start": torch.from_numpy(np.concatenate([[0], np.cumsum(n)]).astype(np.int32)).to(dev),
          "total": int(n.sum()), "max_new": int(n.max()), "scale": d ** -0.5,
          "block_scales": None, "k_scale": 1.0, "v_scale": 1.0}

    # the cache: keys with a few strong channels, values around 1, each block
    # at its own magnitude where there is a scale for each
    shape = (num_blocks, hkv, t, d)
    gain_k = torch.ones(d, device=dev)
    gain_k[torch.randint(0, d, (4,), generator=g, device=dev)] = 4.0
    caches, scales = [], []
    for gain in (gain_k, torch.ones(d, device=dev)):
        x = torch.randn(shape, generator=g, device=dev) * gain
        if case["kv"] != "e4m3":
            caches.append(x.to(TORCH[case["kv"]]))
            continue
        if case["scales"] == "block":
            x *= torch.exp2(torch.randn(shape[:2], generator=g, device=dev))[:, :, None, None]
            s = torch.exp2(_grow_exponent(x.abs().amax(dim=(2, 3))).float())
            scales.append(s)
            caches.append(_quantise(x / s[:, :, None, None]))
        else:
            s = float(np.float32(gain.max().item() * 5.0 / E4M3_MAX))
            scales.append(s)
            caches.append(_quantise(x / s))
        del x
    st["k_cache"], st["v_cache"] = caches
    if case["scales"] == "block":
        st["block_scales"] = torch.stack(scales, dim=2).contiguous()
    elif case["scales"] == "tensor":
        st["k_scale"], st["v_scale"] = scales

    if case["op"] == "append":
        # q, k, v as views of one packed projection; the position table
        width = (hq + 2 * hkv) * d
        qkv = torch.randn((st["total"], width), generator=g, device=dev).to(src)
        st["q"] = qkv[:, :hq * d].unflatten(1, (hq, d))
        st["k"] = qkv[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d))
        st["v"] = qkv[:, (hq + hkv) * d:].unflatten(1, (hkv, d))
        st["q_out"] = torch.empty((st["total"], hq, d), dtype=src, device=dev)
        r = case["rotary"]
        if r:
            top = max_blocks * t
            inv = 10000.0 ** (-torch.arange(0, r, 2, dtype=torch.float64, device=dev) / r)
            ang = torch.arange(top, dtype=torch.float64, device=dev)[:, None] * inv
            st["table"] = torch.cat([ang.cos(), ang.sin()], dim=1).float().contiguous()
        # where each token goes, as the allocator's append returns it, and for
        # each touched block the tokens that land in it
        pos = np.concatenate([np.arange(c - k, c) for c, k in zip(ctx, n)])
        row = np.repeat(np.arange(b), n)
        blk = tables[row, pos // t].astype(np.int64)
        st["pos"] = torch.from_numpy(pos).to(dev)
        st["slot_block"] = torch.from_numpy(blk).to(dev)
        st["slot_row"] = torch.from_numpy(pos % t).to(dev)
        new_unit = np.concatenate([[True], (blk[1:] != blk[:-1])])
        first = np.flatnonzero(new_unit)
        count = np.diff(np.concatenate([first, [len(blk)]]))
        st["unit_block"] = torch.from_numpy(blk[first]).to(dev)
        st["unit_token"] = torch.from_numpy(first).to(dev)
        st["unit_row"] = torch.from_numpy(pos[first] % t).to(dev)
        st["unit_count"] = torch.from_numpy(count).to(dev)
    else:
        # what lies behind a sequence's end in its last block was never written
        for c in (st["k_cache"], st["v_cache"]):
            last = [(tables[s, per[s] - 1], ctx[s] % t) for s in range(b) if ctx[s] % t]
            if last:
                ids = torch.tensor([x for x, _ in last], device=dev, dtype=torch.long)
                offs = torch.tensor([y for _, y in last], device=dev)
                stale = torch.arange(t, device=dev)[None, :] >= offs[:, None]
                tail = c[ids].view(torch.uint8).unflatten(-1, (d, -1))
                tail.masked_fill_(stale[:, None, :, None, None], 0xFF)
                c[ids] = tail.flatten(-2).view(c.dtype)
        if case["window"]:
            # blocks that no query of the call sees went back to the pool
            for s in range(b):
                w0, s0 = _visible(case, int(ctx[s] - n[s] + 1))
                tables[s, -(-s0 // t):w0 // t] = -1
        st["q"] = torch.randn((st["total"], hq, d), generator=g, device=dev).to(src)
        st["out"] = torch.empty_like(st["q"])
    st["tables"] = torch.from_numpy(tables).to(dev)

    if own:
        import paged_kv_cache_137_gb300 as pkv
        st["desc"] = pkv.kv_desc(num_blocks, hkv, d, t, case["kv"])
        if case["op"] == "append":
            st["rope"] = pkv.rope(st["table"], interleaved=case["inter"]) if case["rotary"] else None
        if case["op"] == "decode":
            st["workspace"] = pkv.window_workspace_for(b, hq, max_blocks, st["desc"], case["window"],
                                                       case["sinks"])
    return st


# --------------------------------------------------------------- plain forms
def _rotate(st, x):
    """x [tokens, heads, d] in fp32, its first `rotary` elements rotated by the
    token's angles."""
    case = st["case"]
    r = case["rotary"]
    x = x.float()
    if not r:
        return x
    row = st["table"][st["pos"]]
    c, s = row[:, None, :r // 2], row[:, None, r // 2:]
    y = x.clone()
    if case["inter"]:
        x0, x1 = x[..., 0:r:2], x[..., 1:r:2]
        y[..., 0:r:2] = x0 * c - x1 * s
        y[..., 1:r:2] = x0 * s + x1 * c
    else:
        x0, x1 = x[..., :r // 2], x[..., r // 2:r]
        y[..., :r // 2] = x0 * c - x1 * s
        y[..., r // 2:r] = x0 * s + x1 * c
    return y


def _store_blocks(st, cache, which, y):
    """The touched blocks of a block-scaled cache with the new rows y in them."""
    t = st["case"]["t"]
    rows = torch.arange(t, device=y.device)
    rel = rows[None, :] - st["unit_row"][:, None]
    new = (rel >= 0) & (rel < st["unit_count"][:, None])                   # [units, t]
    token = (st["unit_token"][:, None] + rel).clamp(0, y.shape[0] - 1)
    x = y[token].transpose(1, 2)                                           # [units, heads, t, d]
    mag = torch.where(torch.isfinite(x) & new[:, None, :, None], x.abs(), torch.zeros_like(x))
    grown = torch.exp2(_grow_exponent(mag.amax(dim=(2, 3))).float())       # [units, heads]
    before = st["block_scales"][st["unit_block"], :, which]
    fresh = (st["unit_row"] == 0)[:, None]
    scale = torch.where(fresh, grown, torch.maximum(before, grown))
    held = cache[st["unit_block"]]
    old = held.view(torch.float8_e4m3fn).float() * (before / scale)[:, :, None, None]
    keep = (rel < 0)[:, None, :, None] & (scale > before)[:, :, None, None]
    out = torch.where(keep, _quantise(old), held)
    out = torch.where(new[:, None, :, None], _quantise(x * (1.0 / scale)[:, :, None, None]), out)
    cache[st["unit_block"]] = out
    st["block_scales"][st["unit_block"], :, which] = scale


def _append(st):
    case = st["case"]
    k, v, q = _rotate(st, st["k"]), st["v"].float(), _rotate(st, st["q"])
    st["q_out"].copy_(q)
    if case["scales"] == "block":
        _store_blocks(st, st["k_cache"], 0, k)
        _store_blocks(st, st["v_cache"], 1, v)
        return
    for cache, y, s in ((st["k_cache"], k, st["k_scale"]), (st["v_cache"], v, st["v_scale"])):
        rows = _quantise(y * _inverse(s)) if case["kv"] == "e4m3" else y.to(cache.dtype)
        cache[st["slot_block"], :, st["slot_row"]] = rows


def _inverse(scale):
    return float(np.float32(1.0) / np.float32(scale))


def _gather(st, cache, which, pos, seen):
    """fp32 [batch, heads, positions, d] of the cache at pos [batch, positions],
    zero where not seen or where the block went back to the pool."""
    case = st["case"]
    t = case["t"]
    blk = st["tables"].long().gather(1, (pos // t).clamp(0, st["max_blocks"] - 1))
    seen = seen & (blk >= 0)
    blk = blk.clamp(min=0)
    raw = cache[blk, :, pos % t]                                           # [batch, positions, heads, d]
    x = raw.view(torch.float8_e4m3fn).float() if case["kv"] == "e4m3" else raw.float()
    if case["scales"] == "block":
        x = x * st["block_scales"][blk, :, which][..., None]
    elif case["scales"] == "tensor":
        x = x * (st["k_scale"], st["v_scale"])[which]
    return torch.where(seen[:, :, None, None], x, torch.zeros_like(x)).transpose(1, 2)


def _softmax_av(logits, seen, v):
    logits = logits.masked_fill(~seen, -math.inf)
    top = logits.amax(dim=-1, keepdim=True)
    p = torch.exp(logits - torch.where(torch.isfinite(top), top, torch.zeros_like(top)))
    total = p.sum(dim=-1, keepdim=True)
    o = torch.matmul(p, v)
    return torch.where(total > 0, o / total, torch.zeros_like(o))


def _decode(st):
    case = st["case"]
    b, hq, hkv, d = case["batch"], case["hq"], case["hkv"], case["d"]
    ctx = st["ctx"].long()[:, None]
    top = int(st["ctx_host"].max())
    if case["window"] and case["window"] + case["sinks"] < top:
        i = torch.arange(case["window"] + case["sinks"], device=ctx.device)[None, :]
        w0 = (ctx - case["window"]).clamp(min=0)
        sink = i < case["sinks"]
        pos = torch.where(sink, i, w0 + i - case["sinks"])
        seen = torch.where(sink, (i < w0) & (i < ctx), pos < ctx)
    else:
        pos = torch.arange(max(1, top), device=ctx.device)[None, :].expand(b, -1)
        seen = pos < ctx
        if case["window"]:
            seen = seen & ((pos >= ctx - case["window"]) | (pos < case["sinks"]))
    pos = pos.expand(b, -1)
    k = _gather(st, st["k_cache"], 0, pos, seen)
    v = _gather(st, st["v_cache"], 1, pos, seen)
    q = st["q"].float().view(b, hkv, hq // hkv, d)
    logits = torch.matmul(q, k.transpose(2, 3)) * st["scale"]
    o = _softmax_av(logits, seen[:, None, None, :], v)
    st["out"].copy_(o.reshape(b, hq, d))


def _prefill(st):
    case = st["case"]
    b, hq, hkv, d = case["batch"], case["hq"], case["hkv"], case["d"]
    top, most = int(st["ctx_host"].max()), st["max_new"]
    ctx, start = st["ctx"].long(), st["start"].long()
    n = start[1:] - start[:-1]
    i = torch.arange(most, device=ctx.device)[None, :]
    row = (start[:-1, None] + i).clamp(max=st["total"] - 1)
    qpos = (ctx - n)[:, None] + i                                          # [batch, queries]
    pos = torch.arange(top, device=ctx.device)[None, :].expand(b, -1)
    inside = pos < ctx[:, None]
    k = _gather(st, st["k_cache"], 0, pos, inside)
    v = _gather(st, st["v_cache"], 1, pos, inside)
    seen = (pos[:, None, :] <= qpos[:, :, None]) & inside[:, None, :]
    if case["window"]:
        seen = seen & ((pos[:, None, :] > qpos[:, :, None] - case["window"]) | (pos[:, None, :] < case["sinks"]))
    q = st["q"][row].float().view(b, most, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4)
    logits = torch.matmul(q, k[:, :, None].transpose(3, 4)) * st["scale"]  # [batch, hkv, group, queries, keys]
    o = _softmax_av(logits, seen[:, None, None], v[:, :, None])
    o = o.permute(0, 3, 1, 2, 4).reshape(b, most, hq, d)
    tok = torch.arange(st["total"], device=ctx.device)
    seq = torch.searchsorted(start, tok, right=True) - 1
    st["out"].copy_(o[seq, tok - start[seq]])


# ------------------------------------------------------------------- passes
def run(st):
    case = st["case"]
    if own:
        import paged_kv_cache_137_gb300 as pkv
        if case["op"] == "append":
            one = case["new"] == 1
            kinv, vinv = (_inverse(st["k_scale"]), _inverse(st["v_scale"])) if case["scales"] == "tensor" else (1.0, 1.0)
            pkv.pkv_append(st["k_cache"], st["v_cache"], st["k"], st["v"], st["tables"], st["ctx"], st["desc"],
                           query_start=None if one else st["start"], max_query_len=st["max_new"],
                           rope=st["rope"], q=st["q"], q_out=st["q_out"], block_scales=st["block_scales"],
                           k_inv_scale=kinv, v_inv_scale=vinv)
        elif case["op"] == "decode":
            if case["scales"] == "block":
                pkv.pkv_attention_decode_block_scaled(
                    st["out"], st["q"], st["k_cache"], st["v_cache"], st["block_scales"], st["tables"], st["ctx"],
                    st["desc"], st["scale"], window_tokens=case["window"], sink_tokens=case["sinks"],
                    workspace=st["workspace"])
            else:
                pkv.pkv_attention_decode_window(
                    st["out"], st["q"], st["k_cache"], st["v_cache"], st["tables"], st["ctx"], st["desc"],
                    case["window"], case["sinks"], st["scale"], k_scale=st["k_scale"], v_scale=st["v_scale"],
                    workspace=st["workspace"])
        elif case["scales"] == "block":
            pkv.pkv_attention_prefill_block_scaled(
                st["out"], st["q"], st["k_cache"], st["v_cache"], st["block_scales"], st["tables"], st["ctx"],
                st["start"], st["desc"], st["scale"], max_query_len=st["max_new"], window_tokens=case["window"],
                sink_tokens=case["sinks"])
        else:
            pkv.pkv_attention_prefill_window(
                st["out"], st["q"], st["k_cache"], st["v_cache"], st["tables"], st["ctx"], st["start"], st["desc"],
                case["window"], case["sinks"], st["scale"], max_query_len=st["max_new"], k_scale=st["k_scale"],
                v_scale=st["v_scale"])
    elif case["op"] == "append":
        _append(st)
    elif case["op"] == "decode":
        _decode(st)
    else:
        _prefill(st)
    if case["op"] != "append":
        return st["out"]
    # an 8-bit cache's bytes as the values they stand for, next to their scales
    fp8 = case["kv"] == "e4m3"
    out = {"q": st["q_out"],
           "k": st["k_cache"].view(torch.float8_e4m3fn) if fp8 else st["k_cache"],
           "v": st["v_cache"].view(torch.float8_e4m3fn) if fp8 else st["v_cache"]}
    if case["scales"] == "block":
        out["scales"] = st["block_scales"]
    return out


# ------------------------------------------------------- definitions in 64 bits
def _nearest_e4m3(x):
    """x rounded to the nearest E4M3 value, ties to even, in 64 bits."""
    mag = x.abs().clamp(max=E4M3_MAX)
    e = torch.floor(torch.log2(mag.clamp(min=2.0 ** -6)))
    e = torch.where(torch.exp2(e) > mag.clamp(min=2.0 ** -6), e - 1, e)
    step = torch.exp2(e - 3)
    return torch.sign(x) * (torch.round(mag / step) * step).clamp(max=E4M3_MAX)


def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    ctx, n = st["ctx_host"], st["n_host"]
    hq, hkv, d, t = case["hq"], case["hkv"], case["d"], case["t"]
    tables = st["tables"].long()
    at = np.concatenate([[0], np.cumsum(n)])
    if case["op"] == "append":
        if st["k_cache"].numel() > 2_000_000_000:
            return None
        r = case["rotary"]
        keep = {}
        for name in ("q", "k", "v"):
            x = st[name].double()
            if r and name != "v":
                z = x[..., :r].unflatten(-1, (r // 2, 2) if case["inter"] else (2, r // 2))
                z = z if case["inter"] else z.transpose(-1, -2)
                turn = torch.complex(st["table"][:, :r // 2].double(), st["table"][:, r // 2:].double())
                z = torch.view_as_complex(z.contiguous()) * turn[st["pos"]][:, None]
                z = torch.view_as_real(z)
                z = z if case["inter"] else z.transpose(-1, -2)
                x = torch.cat([z.flatten(-2), x[..., r:]], dim=-1)
            keep[name] = x
        out = {"q": keep["q"]}
        scales = None if st["block_scales"] is None else st["block_scales"].double()
        for w, name in enumerate(("k", "v")):
            cache = st[name + "_cache"]
            val = (cache.view(torch.float8_e4m3fn) if case["kv"] == "e4m3" else cache).double()
            for s in range(case["batch"]):
                p0, p1 = int(ctx[s] - n[s]), int(ctx[s])
                for j in range(p0 // t, -(-p1 // t)):
                    a, z = max(p0, j * t), min(p1, (j + 1) * t)
                    blk = tables[s, j]
                    x = keep[name][at[s] + a - p0:at[s] + z - p0].transpose(0, 1)    # [heads, rows, d]
                    if case["scales"] == "block":
                        big = x.abs().amax(dim=(1, 2))
                        e = torch.ceil(torch.log2(big / E4M3_MAX)).clamp(MIN_EXP, MAX_EXP)
                        sc = torch.exp2(e)
                        if a > j * t:
                            was_sc = scales[blk, :, w]
                            sc = torch.maximum(sc, was_sc)
                            old = val[blk, :, :a - j * t]
                            val[blk, :, :a - j * t] = torch.where(
                                (sc > was_sc)[:, None, None], _nearest_e4m3(old * (was_sc / sc)[:, None, None]), old)
                        scales[blk, :, w] = sc
                        x = _nearest_e4m3(x / sc[:, None, None])
                    elif case["scales"] == "tensor":
                        x = _nearest_e4m3(x * _inverse((st["k_scale"], st["v_scale"])[w]))
                    val[blk, :, a - j * t:z - j * t] = x
            out[name] = val
        if scales is not None:
            out["scales"] = scales
        return out

    if sum(float(a) * float(b) for a, b in zip(ctx, n)) * hq * d > 4e12:
        return None
    out = torch.zeros((st["total"], hq, d), dtype=torch.float64, device="cuda")
    for s in range(case["batch"]):
        c, k = int(ctx[s]), int(n[s])
        if c == 0:
            continue
        p = torch.arange(c, device="cuda")
        qp = torch.arange(c - k, c, device="cuda")
        seen = p[None, :] <= qp[:, None]
        if case["window"]:
            seen &= (qp[:, None] - p[None, :] < case["window"]) | (p[None, :] < case["sinks"])
        any_seen = seen.any(dim=0)
        p = p[any_seen]
        seen = seen[:, any_seen]
        blk = tables[s, p // t]
        kv = []
        for w, cache in enumerate((st["k_cache"], st["v_cache"])):
            x = cache[blk, :, p % t]
            x = (x.view(torch.float8_e4m3fn) if case["kv"] == "e4m3" else x).double()
            if case["scales"] == "block":
                x = x * st["block_scales"][blk, :, w].double()[:, :, None]
            elif case["scales"] == "tensor":
                x = x * float(np.float32((st["k_scale"], st["v_scale"])[w]))
            kv.append(x)
        q = st["q"][at[s]:at[s + 1]].double()
        for h in range(hkv):
            heads = slice(h * (hq // hkv), (h + 1) * (hq // hkv))
            logit = torch.einsum("qgd,pd->gqp", q[:, heads], kv[0][:, h]) * st["scale"]
            prob = torch.softmax(logit.masked_fill(~seen[None], -math.inf), dim=-1)
            out[at[s]:at[s + 1], heads] = torch.einsum("gqp,pd->qgd", prob, kv[1][:, h])
    return out
