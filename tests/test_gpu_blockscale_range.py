"""The block-scale decode where weights and V scales lie far apart: a block that carries the
weight beside one of a much larger scale, a large scale that nothing attends to, a position of
weight without a value. The bar is that of the other decode tests, and 2^-7 of every sequence's
output by itself (these outputs may be far below the others of a batch)."""
import numpy as np
import pytest

import paged_kv_cache_442_b200 as pa
from oracle import fp8_block
from oracle.paged_attention import bf16_bits_to_f64
from tests.gpu_helpers import to_f64
from tests.test_gpu_blockscale import Case, close
from workloads import f32_to_bf16_bits

pytestmark = pytest.mark.gpu


def close_each(c, what):
    got, ref = to_f64(c.gpu()), c.oracle()
    assert np.isfinite(got).all(), what
    for s in range(len(ref)):
        for h in range(ref.shape[1]):
            size = np.linalg.norm(ref[s, h])
            assert np.linalg.norm(got[s, h] - ref[s, h]) <= 2.0 ** -7 * size, (what, s, h)


def attend(c, s, positions, nats):
    """Keys of the positions of sequence s such that every head's score there is `nats` (a
    group's heads get one query)."""
    G = c.q.shape[1] // c.hkv
    q = bf16_bits_to_f64(c.q)
    for g in range(c.hkv):
        q[s, g * G:(g + 1) * G] = q[s, g * G]
        unit = q[s, g * G] / np.linalg.norm(q[s, g * G])
        key = nats / (c.scale * np.linalg.norm(q[s, g * G])) * unit
        for at in positions:
            b = c.tables[s, at // c.bs]
            c.kc[b, at % c.bs, g] = fp8_block.encode(np.clip(key / c.ks[b, g], -448, 448))
    c.q = f32_to_bf16_bits(q.astype(np.float32))


@pytest.mark.parametrize("g", [1, 2, 4, 8, 16])
@pytest.mark.parametrize("octaves", [10, 16, 24])
@pytest.mark.parametrize("peak", [3, 5, 40])   # blocks of 64: in the large scale's tile, in a later one, far behind
def test_the_attended_block_has_a_small_scale(g, octaves, peak):
    c = Case([64 * 44], 2 * g, 2, 64, seed=g + octaves + peak, spread=0.3)
    attend(c, 0, [64 * peak + 7, 64 * peak + 8], 34.0)
    c.vs[c.tables[0, peak]] *= 2.0 ** -octaves
    close_each(c, f"G {g}, 2^-{octaves} in block {peak}")


@pytest.mark.parametrize("octaves", [9, 12, 16, 20, 40])
@pytest.mark.parametrize("ctx,at", [(3000, 0), (3000, 5), (3000, 11), (500, 1), (40000, 100)])
def test_a_large_scale_that_nothing_attends_to(octaves, ctx, at):
    """Its weight times its scale is 2^-10 of the others'."""
    c = Case([ctx], 4, 2, 256, seed=octaves + at)
    rows = range(256 * at, min(ctx, 256 * at + 256))
    attend(c, 0, rows, -(octaves + 10) * np.log(2.0))
    c.vs[c.tables[0, at]] *= 2.0 ** octaves
    close_each(c, f"2^{octaves} in block {at} of {ctx}")


@pytest.mark.parametrize("g", [1, 4, 8, 16])
@pytest.mark.parametrize("ctx", [600, 14000])
@pytest.mark.parametrize("nats", [10.0, 13.0, 15.0, 18.0])
@pytest.mark.parametrize("where", [0, 300])
def test_a_position_of_weight_without_a_value(g, ctx, nats, where):
    """Its values are zero; the others' have a mean of 1 (they would cancel otherwise)."""
    rng = np.random.default_rng(int(nats) + g)
    c = Case([ctx], 2 * g, 2, 64, seed=g, spread=0.0)
    for b in range(-(-ctx // 64)):
        rows = min(64, ctx - 64 * b)
        x = 1.0 + 0.5 * rng.standard_normal((rows, 2, 128))
        c.vc[c.tables[0, b], :rows] = fp8_block.encode(np.clip(x * 96, -448, 448))
    attend(c, 0, [where], nats)
    c.vc[c.tables[0, where // 64], where % 64] = 0
    close_each(c, f"G {g}, {nats} nats over {ctx}")


def test_weights_of_both_bands_come_and_go():
    """Peaked and flat tiles in turn: what a tile left in the second band is cleared."""
    for g in (1, 4, 16):
        c = Case([9000, 2100], 2 * g, 2, 64, seed=g, q_factor=0.5, spread=0.3)
        for s in range(2):
            n = int(c.ctx[s])
            for t in range(1, n // 256, 3):
                attend(c, s, range(256 * t, 256 * t + 200, 3), -9.0)   # far below
            attend(c, s, [n // 2], 9.0)
        close(c.gpu(), c.oracle(), f"G {g}")
        close_each(c, f"G {g}")


@pytest.mark.parametrize("exponent", [-126, -60, 60, 110])
def test_scales_at_the_ends_of_the_range(exponent):
    """Every V scale near 2^exponent: outputs follow, as far as bf16 holds them."""
    c = Case([1200, 70], 8, 2, 64, seed=3, spread=0.2)
    ok = ~np.isnan(c.vs)
    c.vs[ok] = np.ldexp(np.maximum(c.vs[ok] * 96, 1.0), exponent).astype(np.float32)
    got, ref = to_f64(c.gpu()), c.oracle()
    assert np.isfinite(got).all()
    for s in range(2):
        # below bf16's smallest normal number a step is 2^-133
        err = np.abs(got[s] - ref[s]).max()
        assert err <= 2.0 ** -7 * np.abs(ref[s]).max() + 2.0 ** -133
    assert pa.pa_check_device_errors() == 0


@pytest.mark.parametrize("g", [1, 4, 16])
@pytest.mark.parametrize("octaves", [8, 14, 17])
def test_a_query_s_small_elements_beside_a_large_one(g, octaves):
    """One element is 2^octaves above the others and meets keys that are zero there: the scores
    are those of the small ones."""
    c = Case([1500, 300], 2 * g, 2, 64, seed=octaves, spread=0.3)
    q = bf16_bits_to_f64(c.q) * 3.0
    q[..., 17] = 2.0 ** octaves * 3.3
    c.q = f32_to_bf16_bits(q.astype(np.float32))
    c.kc[..., 17] = 0
    close_each(c, f"G {g}, 2^{octaves}")


@pytest.mark.parametrize("exponent", [-130, -100, 60])
def test_queries_of_any_size(exponent):
    """q and the K scales cancel, as far as the scales' range goes."""
    c = Case([900, 70], 8, 2, 64, seed=5, spread=0.2)
    q = np.ldexp(bf16_bits_to_f64(c.q), exponent)
    c.q = f32_to_bf16_bits(q.astype(np.float32))
    ok = ~np.isnan(c.ks)
    c.ks[ok] = np.ldexp(c.ks[ok], min(-exponent, 120))
    close_each(c, f"2^{exponent}")


def test_an_infinite_query_element_stays_in_its_head():
    c = Case([700, 40], 4, 2, 64, seed=6)
    ok = to_f64(c.gpu())
    c.dev[0][0, 1, 5] = float("inf")
    got = to_f64(c.gpu())
    assert np.isnan(got[0, 1]).all()
    got[0, 1] = ok[0, 1]
    assert np.array_equal(got, ok)
