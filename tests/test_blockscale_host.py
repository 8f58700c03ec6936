"""Rotary frequencies, refusals of the rotary and block-scale entry points, and pins of their
oracle. No GPU needed."""
import ctypes
import math

import numpy as np
import pytest

import paged_kv_cache_442_b200 as pa
from oracle import fp8, fp8_block, rope
from paged_kv_cache_442_b200 import build as pa_build
from workloads import f32_to_bf16_bits

NULL = ctypes.c_void_p(0)
FAKE = ctypes.c_void_p(1 << 20)  # never dereferenced: validation fails first
ODD = ctypes.c_void_p((1 << 20) + 8)


@pytest.fixture(scope="module")
def lib():
    pa_build.build()
    return pa.load_library()


def desc(nb=16, bs=16, hkv=2, d=128):
    return pa.pa_cache_desc(nb, bs, hkv, d)


def turn(rot=128, inter=0, amp=1.0, freq=1 << 20):
    return pa.pa_rope_desc(freq, rot, inter, amp)


# ------------------------------------------------------------------- frequency tables
@pytest.mark.parametrize("rot,base,scaling,kw", [
    (128, 10000.0, "none", {}), (64, 500000.0, "none", {}), (2, 10000.0, "none", {}),
    (96, 10000.0, "linear", dict(factor=4.0)), (128, 10000.0, "base", dict(factor=8.0)),
    (128, 10000.0, "ramp", dict(factor=16.0, original_context=4096.0)),
    (64, 10000.0, "ramp", dict(factor=2.0, original_context=2048.0, beta_fast=20.0, beta_slow=2.0)),
])
def test_inv_freq_tables(lib, rot, base, scaling, kw):
    got, amp = pa.pa_rope_inv_freq(rot, base, scaling, **kw)
    want, wamp = rope.inv_freq(rot, base, scaling, **kw)
    # both in 64 bits; fp32 holds the result to half a step (2^-24 relative), logs and powers
    # of the two computations differ by far less
    assert np.allclose(got, want, rtol=2.0 ** -23, atol=0.0)
    assert abs(amp - wamp) <= 2.0 ** -23 * wamp


def test_inv_freq_ends_of_the_stretched_tables(lib):
    plain, _ = pa.pa_rope_inv_freq(128)
    by_base, _ = pa.pa_rope_inv_freq(128, scaling="base", factor=8.0)
    assert by_base[0] == plain[0] == 1.0
    assert math.isclose(by_base[-1], plain[-1] / 8.0, rel_tol=1e-6)
    ramp, amp = pa.pa_rope_inv_freq(128, scaling="ramp", factor=8.0, original_context=4096.0)
    assert ramp[0] == plain[0] and math.isclose(ramp[-1], plain[-1] / 8.0, rel_tol=1e-6)
    assert amp > 1.0


@pytest.mark.parametrize("args", [
    dict(rot_dim=0), dict(rot_dim=7), dict(rot_dim=64, base=1.0), dict(rot_dim=64, base=float("nan")),
    dict(rot_dim=64, scaling="linear", factor=0.5), dict(rot_dim=64, scaling="linear", factor=float("inf")),
    dict(rot_dim=2, scaling="base", factor=2.0),
    dict(rot_dim=64, scaling="ramp", factor=2.0),                       # no original context
    dict(rot_dim=64, scaling="ramp", factor=2.0, original_context=4096.0, beta_fast=1.0, beta_slow=1.0),
])
def test_inv_freq_refusals(lib, args):
    with pytest.raises(pa.PAError) as e:
        pa.pa_rope_inv_freq(**args)
    assert e.value.status == 1


def test_inv_freq_unknown_scaling(lib):
    with pytest.raises(ValueError, match="scaling"):
        pa.pa_rope_inv_freq(64, scaling="cubic")


# ------------------------------------------------------------------- refusals
def test_rope_argument_checks(lib):
    def call(out=FAKE, os_=512, x=FAKE, xs=512, t=4, h=4, d=128, pos=FAKE, r=None):
        return lib.pa_rope(out, os_, x, xs, t, h, d, pos, r or turn(), NULL)
    assert call(d=96) == 1
    assert call(t=-1) == 1 and call(h=-1) == 1
    assert call(out=NULL) == 1 and call(x=NULL) == 1 and call(pos=NULL) == 1
    assert call(out=ODD) == 1 and call(x=ODD) == 1
    assert call(os_=504) == 1 and call(xs=504) == 1          # rows overlap
    assert call(xs=516) == 1                                 # not a multiple of 8
    assert call(r=turn(rot=130)) == 1 and call(r=turn(rot=-2)) == 1 and call(r=turn(rot=31)) == 1
    assert call(r=turn(inter=2)) == 1 and call(r=turn(amp=float("inf"))) == 1
    assert call(r=turn(freq=0)) == 1
    assert call(t=0, out=NULL, x=NULL) == 0 and call(h=0, out=NULL, x=NULL) == 0  # no-ops


def test_rope_store_argument_checks(lib):
    def call(qo=FAKE, q=FAKE, qs=512, k=FAKE, ks=256, v=FAKE, kc=FAKE, vc=FAKE, c=None, slots=FAKE,
             t=4, hq=4, pos=FAKE, r=None):
        return lib.pa_rope_store_kvcache(qo, qs, q, qs, k, ks, v, 256, kc, vc, c or desc(), slots, t,
                                         hq, pos, r or turn(), NULL)
    assert call(c=desc(bs=12)) == 1 and call(c=desc(d=96)) == 1
    assert call(t=-1) == 1 and call(hq=-1) == 1
    for bad in (dict(qo=NULL), dict(q=NULL), dict(k=NULL), dict(v=NULL), dict(kc=NULL), dict(vc=NULL),
                dict(slots=NULL), dict(pos=NULL), dict(k=ODD), dict(vc=ODD), dict(ks=248), dict(qs=520 - 4)):
        assert call(**bad) == 1, bad
    assert call(r=turn(rot=192)) == 1
    assert call(t=0, k=NULL) == 0


def test_append_argument_checks(lib):
    def call(qo=NULL, q=NULL, hq=0, k=FAKE, ks=256, v=FAKE, kc=FAKE, vc=FAKE, ksc=FAKE, vsc=FAKE, c=None,
             bt=FAKE, mb=4, cu=FAKE, ctx=FAKE, b=2, t=4, m=2, pos=FAKE, r=None):
        return lib.pa_rope_store_kvcache_fp8_blockscale(
            qo, 512, q, 512, k, ks, v, 256, kc, vc, ksc, vsc, c or desc(), bt, mb, cu, ctx, b, t, m, hq,
            pos, r or turn(), NULL)
    assert call(c=desc(bs=2048)) == 1 and call(b=-1) == 1 and call(t=-1) == 1 and call(m=-1) == 1
    assert call(mb=0) == 1 and call(hq=-1) == 1
    for bad in (dict(k=NULL), dict(v=NULL), dict(kc=NULL), dict(vc=NULL), dict(ksc=NULL), dict(vsc=NULL),
                dict(bt=NULL), dict(cu=NULL), dict(ctx=NULL), dict(pos=NULL), dict(hq=4), dict(k=ODD),
                dict(kc=ODD), dict(vsc=ODD), dict(ks=252)):
        assert call(**bad) == 1, bad
    # pairs that do not fill 16 dims: valid, not implemented in the fused call
    assert call(r=turn(rot=40)) == 2
    for none in (dict(b=0), dict(t=0), dict(m=0)):
        assert call(k=NULL, v=NULL, **none) == 0
    # without a rotation
    st = lib.pa_store_kvcache_fp8_blockscale(NULL, 256, FAKE, 256, FAKE, FAKE, FAKE, FAKE, desc(), FAKE, 4,
                                             FAKE, FAKE, 2, 4, 2, NULL)
    assert st == 1


def test_blockscale_decode_argument_checks(lib):
    need = pa.pa_decode_fp8_blockscale_workspace_size(4, 2)

    def call(out=FAKE, q=FAKE, kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE, c=None, bt=FAKE, mb=4, ctx=FAKE, b=2, hq=4,
             scale=0.1, mc=32, ws=FAKE, wb=need):
        return lib.pa_decode_fp8_blockscale(out, q, kc, vc, ks, vs, c or desc(), bt, mb, ctx, b, hq, scale,
                                            mc, ws, wb, NULL)
    assert call(hq=3) == 1 and call(scale=float("nan")) == 1 and call(mc=65) == 1 and call(b=-1) == 1
    assert call(mb=0) == 1 and call(mc=-1) == 1 and call(c=desc(bs=24)) == 1
    for bad in (dict(out=NULL), dict(q=NULL), dict(kc=NULL), dict(vc=NULL), dict(ks=NULL), dict(vs=NULL),
                dict(bt=NULL), dict(ctx=NULL), dict(ws=NULL), dict(out=ODD), dict(ks=ODD), dict(ws=ODD),
                dict(wb=need - 1)):
        assert call(**bad) == 1, bad
    assert call(c=desc(d=64)) == 2 and call(hq=6) == 2
    assert call(b=0, out=NULL, ws=NULL) == 0
    assert pa.pa_decode_fp8_blockscale_workspace_size(3, 2) == 0
    assert pa.pa_decode_fp8_blockscale_workspace_size(0, 2) == 0


def test_binding_refuses_cpu_tensors():
    import torch
    x = torch.zeros(4, 2, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        pa.pa_rope(x, x, torch.zeros(4, dtype=torch.int32), torch.zeros(64))


# ------------------------------------------------------------------- pins of the oracle
def test_needed_scale_is_the_smallest_power_of_two():
    for top, want in ((448.0, 1.0), (449.0, 2.0), (224.0, 0.5), (1.75, 2.0 ** -8), (1.7578125, 2.0 ** -7),
                      (0.0, 2.0 ** -126), (2.0 ** -140, 2.0 ** -126), (3e38, 2.0 ** 120)):
        assert fp8_block.needed_scale([0.1 * top, -top]) == want
    assert fp8_block.needed_scale([np.inf, -3.0, np.nan]) == fp8_block.needed_scale([3.0])


def test_encode_agrees_with_the_scalar_codec():
    rng = np.random.default_rng(3)
    y = np.concatenate([rng.standard_normal(2000) * 100, rng.standard_normal(500) * 0.01,
                        (np.arange(400) - 200) / 1024.0, [448.0, 464.0, 480.0, -500.0, 0.0, -0.0]])
    assert [fp8.float_to_e4m3(v) for v in y] == list(fp8_block.encode(y))


def test_appending_row_by_row_ends_at_the_scale_of_all_rows():
    rng = np.random.default_rng(4)
    x = f32_to_bf16_bits((rng.standard_normal((16, 2, 64)) * np.exp(rng.uniform(-4, 4, (16, 2, 1)))).astype(np.float32))
    codes = np.full((3, 16, 2, 64), 0x7F, np.uint8)
    scales = np.full((3, 2), 7.0, np.float32)
    tables = np.array([[2]])
    whole = fp8_block.append(codes, scales, x, tables, [0, 16], [16])
    c, s = codes, scales
    for t in range(16):
        c, s = fp8_block.append(c, s, x[t:t + 1], tables, [0, 1], [t + 1])
    assert np.array_equal(s[2], whole[1][2])
    # one rounding of the final grid at most doubles when a code is rounded again as the grid
    # coarsens (1/2 + 1/4 + ... of a step): values within one subnormal step or 2^-4 relative
    a, b = fp8_block.dequantize(c, s)[2], fp8_block.dequantize(*whole)[2]
    step = s[2][None, :, None] * 2.0 ** -9
    assert np.all(np.abs(a - b) <= np.maximum(step, 2.0 ** -3 * np.abs(b)))
    assert np.array_equal(c[:2], codes[:2]) and np.array_equal(s[:2], scales[:2])
