"""A step of the bf16 path as it is used: one projection's q, k and v rotated and stored, then
attended, prefill chunk first and single tokens after it, against the oracle on the rows the
pools hold."""
import numpy as np
import pytest
import torch

import oracle
import paged_kv_cache_442_b200 as pa
from tests.gpu_helpers import assert_close, bf16_dev, i32_dev, to_bits, to_f64
from workloads import f32_to_bf16_bits

pytestmark = pytest.mark.gpu


def test_rotated_prefill_then_decode_steps():
    rng = np.random.default_rng(12)
    hq, hkv, d, bs, B = 8, 2, 128, 64, 3
    freqs, amp = pa.pa_rope_inv_freq(d, scaling="ramp", factor=4.0, original_context=64.0)
    f = torch.tensor(freqs, dtype=torch.float32, device="cuda")
    steps = [np.array([130, 64, 7])] + [np.ones(B, int)] * 3
    width = -(-int(sum(steps).max()) // bs)
    tables = rng.permutation(B * width).reshape(B, width).astype(np.int32)
    kc = torch.full((B * width, bs, hkv, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    vc = kc.clone()
    ctx = np.zeros(B, int)
    scale = d ** -0.5
    for new in steps:
        ctx = ctx + new
        cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        T = int(cu[-1])
        pos = np.concatenate([np.arange(c - n, c) for c, n in zip(ctx, new)])
        seq = np.repeat(np.arange(B), new)
        slots = tables[seq, pos // bs] * bs + pos % bs
        qkv = bf16_dev(f32_to_bf16_bits(rng.standard_normal((T, hq + 2 * hkv, d)).astype(np.float32)))
        q = torch.empty((T, hq, d), dtype=torch.bfloat16, device="cuda")
        pa.pa_rope_store_kvcache(q, qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], kc, vc, i32_dev(slots),
                                 i32_dev(pos), f, amplitude=amp)
        out = torch.empty_like(q)
        hk, hv = to_bits(kc), to_bits(vc)
        if new.max() > 1:
            pa.pa_prefill(out, q, kc, vc, i32_dev(tables), i32_dev(cu), i32_dev(ctx), scale, int(new.max()))
            ref = oracle.prefill(to_bits(q), hk, hv, tables, cu, ctx, scale)
        else:
            ws, P = pa.decode_workspace(B, hq, hkv, d, int(ctx.max()))
            pa.pa_decode(out, q, kc, vc, i32_dev(tables), i32_dev(ctx), scale, int(ctx.max()), P, ws)
            ref = oracle.decode(to_bits(q), hk, hv, tables, ctx, scale)
        assert_close(to_f64(out), ref, f"step of {new}")


def test_calls_captured_and_replayed_on_another_stream():
    """Rotation, append and decode of a step in one graph, replayed for changed inputs."""
    rng = np.random.default_rng(13)
    hq, hkv, d, bs, B = 4, 2, 128, 16, 5
    f = torch.tensor(pa.pa_rope_inv_freq(d)[0], dtype=torch.float32, device="cuda")
    ctx = np.array([1, 33, 700, 16, 90])
    width = -(-int(ctx.max() + 4) // bs)
    tables = i32_dev(rng.permutation(B * width).reshape(B, width))
    codes = [torch.randint(0, 0x7E, (B * width, bs, hkv, d), dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.full((B * width, hkv), 2.0 ** -6, device="cuda") for _ in range(2)]
    cu = i32_dev(np.arange(B + 1))
    ws = pa.decode_fp8_blockscale_workspace(B, hq, hkv)
    qkv = torch.empty((B, hq + 2 * hkv, d), dtype=torch.bfloat16, device="cuda")
    dctx, pos = i32_dev(ctx), i32_dev(ctx - 1)
    q = torch.empty((B, hq, d), dtype=torch.bfloat16, device="cuda")
    out = torch.empty_like(q)

    def step(c, s, q_, out_):
        pa.pa_rope_store_kvcache_fp8_blockscale(q_, qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], *c, *s,
                                                tables, cu, dctx, 1, pos, f)
        pa.pa_decode_fp8_blockscale(out_, q_, *c, *s, tables, dctx, d ** -0.5, int(ctx.max()) + 4, ws)

    pa.pa_set_debug_checks(False)
    try:
        spare = [t.clone() for t in codes], [t.clone() for t in scales]
        qkv.normal_()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step(*spare, q.clone(), out.clone())
        side.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            step(codes, scales, q, out)
        eager = [t.clone() for t in codes], [t.clone() for t in scales]
        eq, eo = torch.empty_like(q), torch.empty_like(out)
        for _ in range(4):
            qkv.normal_()
            torch.cuda.synchronize()
            with torch.cuda.stream(side):
                g.replay()
            side.synchronize()
            step(*eager, eq, eo)
            torch.cuda.synchronize()
            assert torch.equal(out.view(torch.int16), eo.view(torch.int16))
            assert all(torch.equal(a, b) for a, b in zip(codes + scales, eager[0] + eager[1]))
            dctx += 1
            pos += 1
        del g
    finally:
        pa.pa_set_debug_checks(True)
    assert pa.pa_check_device_errors() == 0


def test_tensors_of_another_device_are_refused():
    if torch.cuda.device_count() < 2:
        pytest.skip("one GPU")
    x = torch.zeros(2, 1, 128, dtype=torch.bfloat16, device="cuda:1")
    with pytest.raises(ValueError, match="current device"):
        pa.pa_rope(x, x, torch.zeros(2, dtype=torch.int32, device="cuda:1"), torch.zeros(64, device="cuda:1"))
