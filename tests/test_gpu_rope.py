"""GPU parity of the rotary positions, alone and with the store into the bf16 pools.

Tolerance of a rotated value: its one rounding to bf16 (half a step, 2^-8 relative) plus the
fp32 error of the turn and the two products: the angle's remainder is below half a turn and
rounded to fp32 (2^-24 of it), sine and cosine are within 2 units in the last place, and two
products and a sum round three times: below 2^-20 (|a| + |b|) amplitude in all.
"""
import numpy as np
import pytest
import torch

import paged_kv_cache_442_b200 as pa
from oracle import rope
from oracle.paged_attention import bf16_bits_to_f64
from tests.gpu_helpers import bf16_dev, i32_dev, to_bits, to_f64
from workloads import f32_to_bf16_bits

pytestmark = pytest.mark.gpu


def rows(rng, t, h, d):
    return f32_to_bf16_bits((rng.standard_normal((t, h, d)) * 10.0 ** rng.uniform(-2, 2, (t, h, 1))).astype(np.float32))


def table(rot, factor=1.0):
    f, amp = pa.pa_rope_inv_freq(rot, scaling="ramp" if factor > 1 else "none", factor=factor,
                                 original_context=4096.0) if rot else ([], 1.0)
    return torch.tensor(f, dtype=torch.float32, device="cuda"), np.array(f, np.float32), amp


def check(got, x, positions, f, inter, amp):
    x = bf16_bits_to_f64(x)
    want = rope.rotate(x, positions, f, inter, amp)
    size = np.abs(x)
    rot = 2 * len(f)
    pair = size.copy()
    if inter:
        pair[..., 0:rot:2] += size[..., 1:rot:2]
        pair[..., 1:rot:2] += size[..., 0:rot:2]
    else:
        h = rot // 2
        pair[..., :h] += size[..., h:rot]
        pair[..., h:rot] += size[..., :h]
    tol = np.where(np.arange(x.shape[-1]) < rot, 2.0 ** -8 * np.abs(want) + 2.0 ** -20 * amp * pair, 0.0)
    assert np.all(np.abs(got - want) <= tol)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("t,h,d,rot", [(1, 1, 128, 128), (5, 3, 64, 64), (7, 16, 128, 64), (33, 5, 128, 16),
                                       (4, 2, 64, 48), (9, 3, 128, 2), (6, 4, 64, 20), (3, 7, 128, 126),
                                       (2, 2, 128, 0), (2500, 2, 64, 32)])
def test_rope_matches_the_formula(t, h, d, rot, inter):
    rng = np.random.default_rng(t + d + rot)
    x = rows(rng, t, h, d)
    positions = rng.integers(-5, 5000, t).astype(np.int32)
    positions[-1] = 2 ** 31 - 1
    positions[0] = 0 if t > 1 else 1000003
    fd, f, amp = table(rot, factor=8.0)
    xd, out = bf16_dev(x), torch.full((t, h, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    pa.pa_rope(out, xd, i32_dev(positions), fd, interleaved=inter, amplitude=amp)
    check(to_f64(out), x, positions, f, inter, amp)
    if positions[0] == 0 and amp == 1.0:
        assert torch.equal(out[0], xd[0])
    # in place
    pa.pa_rope(xd, xd, i32_dev(positions), fd, interleaved=inter, amplitude=amp)
    assert np.array_equal(to_bits(xd), to_bits(out))


def test_a_turn_back_is_the_transpose():
    """The gradient of a rotation is the rotation by -position: <R x, y> = <x, R^T y>."""
    rng = np.random.default_rng(8)
    x, y = rows(rng, 50, 4, 128), rows(rng, 50, 4, 128)
    pos = rng.integers(0, 100000, 50).astype(np.int32)
    fd, _, _ = table(128)
    xd, yd = bf16_dev(x), bf16_dev(y)
    rx, ry = torch.empty_like(xd), torch.empty_like(yd)
    pa.pa_rope(rx, xd, i32_dev(pos), fd)
    pa.pa_rope(ry, yd, i32_dev(-pos), fd)
    a, b = to_f64(rx) * to_f64(yd), to_f64(xd) * to_f64(ry)
    # each rotated value carries half a bf16 step
    bound = 2.0 ** -8 * (np.abs(a).sum((1, 2)) + np.abs(b).sum((1, 2))) * 1.01
    assert np.all(np.abs(a.sum((1, 2)) - b.sum((1, 2))) <= bound)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("t,hq,hkv,d,bs,rot", [(1, 8, 8, 64, 16, 64), (64, 16, 8, 128, 256, 128),
                                               (37, 3, 1, 128, 64, 64), (3001, 4, 2, 64, 32, 32),
                                               (11, 6, 3, 128, 16, 6), (5, 0, 2, 128, 16, 128),
                                               # 2, 4, 4 and 8 tokens a CTA
                                               (901, 28, 2, 128, 64, 128), (903, 2, 1, 128, 64, 96),
                                               (4801, 30, 1, 128, 256, 64), (2503, 4, 2, 128, 64, 16)])
def test_rope_store_equals_rope_then_store(t, hq, hkv, d, bs, rot, inter):
    """From slices of one projection; bit for bit, rows no token names untouched."""
    rng = np.random.default_rng(t + hq)
    nb = -(-t // bs) + 2
    qkv = bf16_dev(rows(rng, t, hq + 2 * hkv, d))
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    slots = rng.permutation(nb * bs)[:t].astype(np.int32)
    if t > 3:
        slots[[1, t // 2]] = -1
    pos = i32_dev(rng.integers(0, 2 ** 22, t))
    fd, _, _ = table(rot)
    kc, vc = (bf16_dev(rows(rng, nb * bs, hkv, d)).view(nb, bs, hkv, d) for _ in range(2))
    kc2, vc2 = kc.clone(), vc.clone()
    q_out = torch.empty((t, hq, d), dtype=torch.bfloat16, device="cuda") if hq else None
    pa.pa_rope_store_kvcache(q_out, q if hq else None, k, v, kc, vc, i32_dev(slots), pos, fd, interleaved=inter)
    rk = torch.empty((t, hkv, d), dtype=torch.bfloat16, device="cuda")
    pa.pa_rope(rk, k, pos, fd, interleaved=inter)
    pa.pa_store_kvcache(rk, v.contiguous(), kc2, vc2, i32_dev(slots))
    assert np.array_equal(to_bits(kc), to_bits(kc2)) and np.array_equal(to_bits(vc), to_bits(vc2))
    if hq:
        rq = torch.empty_like(q_out)
        pa.pa_rope(rq, q, pos, fd, interleaved=inter)
        assert np.array_equal(to_bits(q_out), to_bits(rq))
        # q turned in place inside the projection: k and v beside it unchanged
        keep = qkv[:, hq:].clone()
        pa.pa_rope_store_kvcache(q, q, k, v, kc, vc, i32_dev(slots), pos, fd, interleaved=inter)
        assert np.array_equal(to_bits(q.contiguous()), to_bits(q_out))
        assert np.array_equal(to_bits(qkv[:, hq:].contiguous()), to_bits(keep))


def test_rope_store_bad_slot_is_reported_and_skipped():
    rng = np.random.default_rng(1)
    k, v = bf16_dev(rows(rng, 6, 2, 128)), bf16_dev(rows(rng, 6, 2, 128))
    kc = torch.zeros((4, 16, 2, 128), dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    fd, _, _ = table(128)
    slots = i32_dev(np.array([0, 1, 64, 3, 2 ** 31 - 1, 5]))
    with pytest.raises(pa.PAError) as e:
        pa.pa_rope_store_kvcache(None, None, k, v, kc, vc, slots, i32_dev(np.zeros(6)), fd)
    assert e.value.status == 3
    flat = vc.view(64, 2, 128)
    for t, s in ((0, 0), (1, 1), (3, 3), (5, 5)):
        assert torch.equal(flat[s], v[t])
    assert not flat[[2, 4]].any() and not flat[6:].any()


def test_binding_shape_checks():
    x = torch.zeros(4, 2, 128, dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros(4, dtype=torch.int32, device="cuda")
    f = torch.zeros(64, device="cuda")
    with pytest.raises(ValueError, match="contiguous"):
        pa.pa_rope(x, x.transpose(0, 1), pos, f)
    with pytest.raises(ValueError, match="positions"):
        pa.pa_rope(x, x, pos[:3], f)
    with pytest.raises(ValueError, match="shape"):
        pa.pa_rope(x[:3], x, pos, f)
    with pytest.raises(TypeError, match="inv_freq"):
        pa.pa_rope(x, x, pos, f.double())
    with pytest.raises(pa.PAError):                    # more turned dims than the head has
        pa.pa_rope(x, x, pos, torch.zeros(65, device="cuda"))
    odd = torch.zeros(4 * 260, dtype=torch.bfloat16, device="cuda")
    odd = odd.as_strided((4, 2, 128), (260, 128, 1))
    with pytest.raises(pa.PAError):                    # token stride not a multiple of 8
        pa.pa_rope(x, odd, pos, f)
