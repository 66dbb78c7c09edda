"""Pins of the append and window oracles (CPU): closed forms, brute force and
planted mistakes."""
import math

import numpy as np
import pytest
import torch

from oracle import append as OA
from oracle import e4m3
from oracle import window as OW


def test_rotation_is_the_complex_product():
    r = np.random.RandomState(0)
    x = r.randn(5, 3, 64)
    pos = np.array([0, 1, 7, 100, 4000])
    table = OA.angle_table(4096, 32)
    for inter in (False, True):
        y = OA.rotate(x, table, pos, inter)
        assert np.array_equal(y[..., 32:], x[..., 32:]) and np.allclose(y[0], x[0], atol=0)
        for i in range(16):
            a, b = (2 * i, 2 * i + 1) if inter else (i, i + 16)
            turn = np.exp(1j * pos * 10000.0 ** (-2 * i / 32))[:, None]
            z = (x[..., a] + 1j * x[..., b]) * turn
            assert np.allclose(y[..., a] + 1j * y[..., b], z, atol=1e-12)


def test_rotated_products_depend_on_the_distance_only():
    r = np.random.RandomState(1)
    table = OA.angle_table(300, 64)
    q, k = r.randn(1, 1, 64), r.randn(1, 1, 64)
    dots = [float((OA.rotate(q, table, [p + 37], False) * OA.rotate(k, table, [p], False)).sum())
            for p in (0, 5, 200)]
    assert np.allclose(dots, dots[0], atol=1e-12)
    wrong = (OA.rotate(q, table, [37], False) * OA.rotate(k, table, [5], False)).sum()
    assert abs(wrong - dots[0]) > 1e-6


def test_library_table_matches_the_definition():
    import paged_kv_cache_137_gb300 as pkv
    got = pkv.rope_table(500, 48, 10000.0, device="cpu").numpy()
    assert np.abs(got - OA.angle_table(500, 48)).max() <= 2.0 ** -24


@pytest.mark.parametrize("amax,want", [(448.0, 1.0), (448.001, 2.0), (0.0, 2.0 ** -40), (224.0, 0.5), (1.75, 2.0 ** -8),
                                       (1.7500001, 2.0 ** -7), (1e30, 2.0 ** 40)])
def test_scale_is_the_least_power_of_two(amax, want):
    assert OA.scale_for(float(np.float64(amax))) == want


def test_appending_token_by_token_ends_at_the_same_scales():
    """The scale of a block does not depend on how its tokens were grouped; the
    bytes differ from one append of all by at most one more rounding."""
    r = np.random.RandomState(2)
    x = (r.randn(40, 2, 64) * np.exp2(r.randint(-6, 7, size=(40, 1, 1)))).astype(np.float32)
    tables, shape = [[1, 2, 0]], (3, 2, 16, 64)
    a, sa = np.zeros(shape, np.uint8), np.zeros((3, 2, 2))
    OA.append_block_scaled(a, sa, 0, x, tables, [40], [40])
    b, sb = np.zeros(shape, np.uint8), np.zeros((3, 2, 2))
    for c in range(1, 41):
        OA.append_block_scaled(b, sb, 0, x[c - 1:c], tables, [c], [1])
    assert np.array_equal(sa, sb)
    va, vb = (e4m3.decode(z) * sa[:, :, 0][:, :, None, None] for z in (a, b))
    want = np.zeros(shape)
    OA.append_values(want, x.astype(np.float64), tables, [40], [40])
    # half a step of the normals, or of the subnormals at the block's scale
    for v, k in ((va, 1), (vb, 2)):
        assert (np.abs(v - want) <= k * np.maximum(np.abs(want) * 2.0 ** -4, sa[:, :, 0][:, :, None, None] * 2.0 ** -10)
                * (1 + 2.0 ** -4)).all()


def test_a_reused_block_forgets_its_old_scale():
    cache, scales = np.zeros((1, 1, 16, 64), np.uint8), np.full((1, 1, 2), 64.0)
    OA.append_block_scaled(cache, scales, 0, np.ones((2, 1, 64), np.float32), [[0]], [2], [2])
    assert scales[0, 0, 0] == 2.0 ** -8 and scales[0, 0, 1] == 64.0


def brute(q, k, v, p, window, sinks, scale):
    keys = [i for i in range(p + 1) if not window or i > p - window or i < sinks]
    x = [math.fsum(a * b for a, b in zip(q, k[i])) * scale for i in keys]
    m = max(x)
    w = [math.exp(y - m) for y in x]
    return [math.fsum(w[j] * v[i][d] for j, i in enumerate(keys)) / math.fsum(w) for d in range(len(q))]


@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (5, 2), (16, 20), (40, 1)])
def test_window_attention_by_brute_force(window, sinks):
    r = np.random.RandomState(3)
    ctx, n, t = [23, 9], [6, 9], 16
    k, v = r.randn(4, 2, t, 8), r.randn(4, 2, t, 8)
    tables = [[2, 0], [3]]
    q = r.randn(15, 4, 8)
    out, mag, top = OW.paged_attention_window(q, k, v, tables, ctx, n, 0.3, window, sinks)
    at = 0
    for s in range(2):
        ks = np.stack([k[tables[s][p // t], :, p % t] for p in range(ctx[s])])
        vs = np.stack([v[tables[s][p // t], :, p % t] for p in range(ctx[s])])
        for i in range(n[s]):
            for j in range(4):
                p = ctx[s] - n[s] + i
                want = brute(q[at, j], ks[:, j // 2], vs[:, j // 2], p, window, sinks, 0.3)
                assert np.allclose(out[at, j], want, atol=1e-12)
            at += 1
    assert (mag >= np.abs(out) - 1e-12).all() and (top >= 0).all()


def test_a_window_off_by_one_is_caught():
    r = np.random.RandomState(4)
    k, v, q = r.randn(2, 1, 16, 8), r.randn(2, 1, 16, 8), r.randn(1, 1, 8)
    a = OW.paged_attention_window(q, k, v, [[0, 1]], [30], [1], 1.0, 5, 2)[0]
    b = OW.paged_attention_window(q, k, v, [[0, 1]], [30], [1], 1.0, 6, 2)[0]
    c = OW.paged_attention_window(q, k, v, [[0, 1]], [30], [1], 1.0, 5, 3)[0]
    assert np.abs(a - b).max() > 1e-6 and np.abs(a - c).max() > 1e-6


def test_empty_context_gives_zero():
    z = np.zeros((1, 1, 16, 8))
    out, _, _ = OW.paged_attention_window(np.ones((1, 2, 8)), z, z, [[0]], [0], [1], 1.0, 4, 1)
    assert not out.any()


def test_whole_window_equals_scaled_dot_product_attention():
    r = np.random.RandomState(5)
    k, v, q = r.randn(3, 2, 16, 64), r.randn(3, 2, 16, 64), r.randn(40, 2, 64)
    out, _, _ = OW.paged_attention_window(q, k, v, [[2, 0, 1]], [40], [40], 0.125, 0, 0)
    ks, vs = (np.concatenate([x[b] for b in (2, 0, 1)], axis=1)[:, :40] for x in (k, v))
    ref = torch.nn.functional.scaled_dot_product_attention(
        torch.from_numpy(q).transpose(0, 1), torch.from_numpy(ks), torch.from_numpy(vs), is_causal=True, scale=0.125)
    assert np.allclose(out, ref.transpose(0, 1).numpy(), atol=1e-12)
