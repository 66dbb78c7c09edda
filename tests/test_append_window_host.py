"""Refusals of pkv_append and of the windowed and block-scaled attention calls
through the C ABI on the host (no GPU): every call here is refused, or empty,
before anything is launched, so the pointers only have to look right."""
import ctypes

import pytest
import torch

import paged_kv_cache_137_gb300 as pkv

INVALID, UNSUPPORTED = pkv.PKV_ERR_INVALID_ARG, pkv.PKV_ERR_UNSUPPORTED
P = 1 << 20   # an address no refused call follows
F32, F16, BF16, E4M3 = (pkv.DTYPE_OF_NAME[n] for n in ("f32", "f16", "bf16", "e4m3"))


@pytest.fixture(scope="module", autouse=True)
def built():
    pkv.build()
    pkv.lib()


def desc_of(kv="bf16", d=128, t=16, hkv=4, nb=64, heads=0):
    x = pkv.kv_desc(nb, hkv, d, t, kv)
    x.head_scales = heads
    return x


def refused(code, want, message):
    assert code == want, (code, pkv.lib().pkv_last_error())
    assert message in pkv.lib().pkv_last_error().decode(), pkv.lib().pkv_last_error()


# ------------------------------------------------------------------ append
APPEND = dict(k_cache=P, v_cache=P, block_scales=None, k=P, k_stride=512, v=P, v_stride=512, q_out=P, q=P,
              q_stride=1024, num_q_heads=8, src=BF16, tables=P, max_blocks=8, ctx=P, start=P, num_seqs=3, total=5,
              longest=4, rope=None, desc=None, k_inv=1.0, v_inv=1.0, stream=None)


def append(desc=None, rope=None, **kw):
    a = {**APPEND, **kw}
    a["desc"] = ctypes.byref(desc or desc_of())
    a["rope"] = None if rope is None else ctypes.byref(rope)
    return pkv.lib().pkv_append(*a.values())


@pytest.mark.parametrize("kw,code,message", [
    (dict(num_seqs=-1), INVALID, "negative"),
    (dict(total=-1), INVALID, "negative"),
    (dict(longest=-1), INVALID, "negative"),
    (dict(num_q_heads=-4), INVALID, "negative"),
    (dict(max_blocks=-1), INVALID, "negative"),
    (dict(src=E4M3), INVALID, "src_dtype"),
    (dict(src=9), INVALID, "src_dtype"),
    (dict(src=F32), INVALID, "src_dtype == kv_dtype"),
    (dict(block_scales=P), INVALID, "E4M3"),
    (dict(desc=desc_of("e4m3", heads=P), block_scales=P), INVALID, "exclude"),
    (dict(desc=desc_of("e4m3"), block_scales=P + 4), INVALID, "misaligned"),
    (dict(rope=pkv.pkv_rope(P, 64, 24, 0)), UNSUPPORTED, "multiple of 16"),
    (dict(rope=pkv.pkv_rope(P, 64, 144, 0)), UNSUPPORTED, "at most head_dim"),
    (dict(rope=pkv.pkv_rope(P, 64, -16, 0)), INVALID, "negative"),
    (dict(rope=pkv.pkv_rope(P, -1, 16, 0)), INVALID, "negative"),
    (dict(rope=pkv.pkv_rope(None, 64, 16, 0)), INVALID, "cos_sin"),
    (dict(rope=pkv.pkv_rope(P + 8, 64, 16, 0)), INVALID, "cos_sin"),
    (dict(num_q_heads=6), INVALID, "multiple of num_kv_heads"),
    (dict(num_seqs=65536, total=65536), UNSUPPORTED, "65535"),
    (dict(max_blocks=0), INVALID, "max_blocks is 0"),
    (dict(start=None), INVALID, "one token per sequence"),
    (dict(max_blocks=1 << 27), UNSUPPORTED, "2^30"),
    (dict(q=None), INVALID, "q or q_out"),
    (dict(q_out=None), INVALID, "q or q_out"),
    (dict(q_out=P + 2), INVALID, "16-byte"),
    (dict(tables=P + 2), INVALID, "tables misaligned"),
    (dict(ctx=P + 1), INVALID, "tables misaligned"),
    (dict(start=P + 2), INVALID, "tables misaligned"),
    (dict(k_stride=504), INVALID, "stride"),
    (dict(v_stride=516), INVALID, "stride"),
    (dict(k_stride=0), INVALID, "stride"),
    (dict(q_stride=1016), INVALID, "q_stride"),
    (dict(q_stride=1028), INVALID, "q_stride"),
    (dict(q_stride=1536), INVALID, "contiguous"),   # q_out is q
    (dict(desc=desc_of(d=96)), UNSUPPORTED, "head_dim"),
    (dict(desc=desc_of(t=8)), UNSUPPORTED, "block_size"),
] + [({name: None}, INVALID, "NULL") for name in ("k_cache", "v_cache", "k", "v", "tables", "ctx")]
  + [({name: P + 8}, INVALID, "16-byte") for name in ("k_cache", "v_cache", "k", "v", "q")])
def test_append_refuses(kw, code, message):
    refused(append(**kw), code, message)


@pytest.mark.parametrize("kw", [dict(num_seqs=0, total=0), dict(total=0), dict(longest=0)])
def test_an_empty_append_is_nothing(kw):
    assert append(**kw) == pkv.PKV_OK


def test_copied_scales_refuse():
    fn = pkv.lib().pkv_copy_block_scales
    d = desc_of("e4m3")

    def call(ptrs, pairs, desc=d, layers=None, n=None):
        a = (ctypes.c_void_p * max(len(ptrs), 1))(*ptrs)
        p = (ctypes.c_int32 * max(len(pairs), 1))(*pairs)
        return fn(a, len(ptrs) if layers is None else layers, p, len(pairs) // 2 if n is None else n,
                  ctypes.byref(desc), None)

    assert call([], []) == pkv.PKV_OK
    refused(call([P], [0, 1], desc=desc_of()), INVALID, "E4M3")
    refused(call([P], [0, 1], n=-1), INVALID, "negative")
    refused(call([], [0, 1]), INVALID, "num_layers")
    refused(call([P] * 129, [0, 1]), INVALID, "num_layers")
    refused(call([P, None], [0, 1]), INVALID, "NULL or misaligned")
    refused(call([P, P + 4], [0, 1]), INVALID, "NULL or misaligned")
    for pair in ([0, 64], [64, 0], [-1, 0], [0, -1]):
        refused(call([P], pair), INVALID, "block id")
    refused(fn(None, 1, (ctypes.c_int32 * 2)(0, 1), 1, ctypes.byref(d), None), INVALID, "NULL")


# --------------------------------------------------------------- attention
DECODE = dict(out=P, q=P, q_dtype=BF16, k_cache=P, v_cache=P, block_scales=P, tables=P, max_blocks=64, ctx=P,
              num_seqs=3, num_q_heads=8, desc=None, window=100, sinks=4, scale=0.1, k_scale=1.0, v_scale=1.0,
              part=0, ws=P, ws_bytes=1 << 30, stream=None)
PREFILL = dict(out=P, q=P, q_dtype=BF16, k_cache=P, v_cache=P, block_scales=P, tables=P, max_blocks=64, ctx=P,
               start=P, num_seqs=3, total=5, longest=4, num_q_heads=8, desc=None, window=100, sinks=4, scale=0.1,
               k_scale=1.0, v_scale=1.0, stream=None)


def attend(form, block, desc=None, **kw):
    """The four calls by form ("decode", "prefill") and whether block-scaled."""
    a = {**(DECODE if form == "decode" else PREFILL), **kw}
    a["desc"] = ctypes.byref(desc or desc_of("e4m3" if block else "bf16"))
    for name in ("k_scale", "v_scale") if block else ("block_scales",):
        del a[name]
    return getattr(pkv.lib(), f"pkv_attention_{form}_{'block_scaled' if block else 'window'}")(*a.values())


BOTH = [("decode", False), ("decode", True), ("prefill", False), ("prefill", True)]


@pytest.mark.parametrize("form,block", BOTH)
@pytest.mark.parametrize("kw,code,message", [
    (dict(num_seqs=-1), INVALID, "negative"),
    (dict(num_q_heads=0), INVALID, "no query heads"),
    (dict(max_blocks=-1), INVALID, "negative"),
    (dict(num_q_heads=6), INVALID, "multiple of num_kv_heads"),
    (dict(window=-1), INVALID, "window_tokens"),
    (dict(sinks=-1), INVALID, "sink_tokens"),
    (dict(num_seqs=65536), UNSUPPORTED, "65535"),
    (dict(max_blocks=0), INVALID, "max_blocks is 0"),
    (dict(max_blocks=1 << 27), UNSUPPORTED, "2^30"),
    (dict(tables=P + 2), INVALID, "tables misaligned"),
    (dict(ctx=P + 2), INVALID, "tables misaligned"),
    (dict(scale=float("nan")), INVALID, "NaN"),
] + [({name: None}, INVALID, "NULL") for name in ("out", "q", "k_cache", "v_cache", "tables", "ctx")]
  + [({name: P + 8}, INVALID, "16-byte") for name in ("out", "q", "k_cache", "v_cache")])
def test_attention_refuses(form, block, kw, code, message):
    refused(attend(form, block, **kw), code, message)


@pytest.mark.parametrize("form", ["decode", "prefill"])
def test_window_and_block_scales_are_checked(form):
    refused(attend(form, False, window=0), INVALID, "at least 1")
    refused(attend(form, True, desc=desc_of("bf16")), INVALID, "E4M3")
    refused(attend(form, True, desc=desc_of("e4m3", heads=P)), INVALID, "exclude")
    refused(attend(form, True, block_scales=None), INVALID, "block_scales")
    refused(attend(form, True, block_scales=P + 4), INVALID, "block_scales")


def test_decode_refuses():
    for kv, q in (("bf16", F16), ("f16", BF16), ("f32", BF16), ("e4m3", F32), ("e4m3", E4M3)):
        refused(attend("decode", False, desc=desc_of(kv), q_dtype=q), INVALID, "q_dtype")
    refused(attend("decode", False, part=-64), INVALID, "negative")
    refused(attend("decode", False, part=100), INVALID, "multiple of 64")
    refused(attend("decode", False, num_q_heads=4 * 17), UNSUPPORTED, "16 query heads")
    for kw in (dict(ws=None), dict(ws_bytes=100), dict(ws_bytes=0)):
        refused(attend("decode", False, part=64, **kw), INVALID, "workspace")
    refused(attend("decode", False, part=64, ws=P + 128), INVALID, "256-byte")
    pkv.pkv_set_attention_kernel("tc")
    try:
        refused(attend("decode", False, desc=desc_of("f32"), q_dtype=F32), UNSUPPORTED, "tensor-core")
    finally:
        pkv.pkv_set_attention_kernel("auto")


def test_prefill_refuses():
    for kw in (dict(total=-1), dict(longest=-1)):
        refused(attend("prefill", False, **kw), INVALID, "negative")
    refused(attend("prefill", False, start=None), INVALID, "NULL")
    refused(attend("prefill", False, start=P + 2), INVALID, "tables misaligned")
    for kv, q in (("bf16", F16), ("f16", BF16), ("f32", F32), ("e4m3", F32), ("e4m3", E4M3)):
        refused(attend("prefill", False, desc=desc_of(kv), q_dtype=q), UNSUPPORTED, "windowed prefill")
    refused(attend("prefill", False, desc=desc_of(nb=1 << 26, hkv=8)), UNSUPPORTED, "2^31 rows")


@pytest.mark.parametrize("form,block", BOTH)
def test_an_empty_batch_is_nothing(form, block):
    assert attend(form, block, num_seqs=0) == pkv.PKV_OK
    if form == "prefill":
        assert attend(form, block, total=0) == pkv.PKV_OK
        assert attend(form, block, longest=0) == pkv.PKV_OK


def test_workspace_sizes():
    """(sequence, KV head) counters, then m and l, then the partial outputs, of
    each split of the visible span (its chunks of 16: the window's and one, and
    the sinks', and no more than the 64 that a table of 64 blocks of 16 holds);
    nothing where a span is one split or an argument is bad."""
    d = desc_of(hkv=4)
    size = pkv.pkv_window_workspace_bytes

    def up(x):
        return -(-x // 256) * 256

    for window, sinks, part, splits in ((1000, 4, 64, 16), (1000, 0, 64, 16), (64, 0, 64, 2), (0, 0, 64, 16),
                                        (4096, 64, 128, 8), (48, 0, 64, 1)):
        rows = 5 * 8 * splits
        want = 0 if splits == 1 else up(5 * 4 * 4) + 2 * up(rows * 4) + up(rows * 128 * 4)
        assert size(5, 8, 64, d, window, sinks, part) == want, (window, sinks, part)
    for bad in ((0, 8, 64), (5, 0, 64), (5, 6, 64), (5, 8, 0), (5, 8, 1 << 27)):
        assert size(*bad, d, 100, 4, 64) == 0
    assert size(5, 8, 64, d, -1, 4, 64) == size(5, 8, 64, d, 100, -1, 64) == size(5, 8, 64, d, 100, 4, 65) == 0


def test_the_binding_refuses_a_table_on_the_host():
    with pytest.raises(ValueError, match="CUDA"):
        pkv.rope(torch.zeros((8, 16)))
    table = pkv.rope_table(100, 32, device="cpu")
    p = torch.arange(100, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(16, dtype=torch.float64) / 16)
    assert table.shape == (100, 32) and torch.equal(table, torch.cat([p.cos(), p.sin()], dim=1).float())
    assert pkv.rope_table(0, 32, device="cpu").shape == (0, 32)
    assert pkv.empty_block_scales(desc_of("e4m3"), device="cpu").shape == (64, 4, 2)
