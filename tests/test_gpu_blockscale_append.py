"""The append's kernels one by one: which variant a call takes follows from its sizes (one row a
sequence; a warp for few rows of a block; a CTA or a cluster for more; a CTA per 64 positions of
small blocks; counted units for batches of very different lengths)."""
import numpy as np
import pytest

import paged_kv_cache_442_b200 as pa
from oracle import fp8_block
from tests.gpu_helpers import bf16_dev, i32_dev, to_bits
from tests.test_gpu_blockscale import f32_dev, pools_of, same_codes, tables_of, u8_dev
from workloads import f32_to_bf16_bits

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new,seqs,bs", [(3, 40, 64), (8, 20, 256), (12, 300, 64), (16, 300, 32)])
def test_few_rows_whose_blocks_all_grow(new, seqs, bs, d):
    """Every block holds rows whose scale the new ones exceed: all lanes of a warp take part in
    writing the old rows again, with the scale that was there before."""
    rng = np.random.default_rng(new + d)
    hkv, old = 4, bs - new - 3
    ctx = np.full(seqs, old + new)
    tables, nb = tables_of(rng, ctx, bs)
    cu = np.arange(seqs + 1) * new
    x = f32_to_bf16_bits((50.0 * rng.standard_normal((seqs * new, hkv, d))).astype(np.float32))
    codes, _ = pools_of(rng, nb, bs, hkv, d)
    scales = np.ldexp(1.0, rng.integers(-9, -6, (nb, hkv))).astype(np.float32)
    want = fp8_block.append(codes, scales, x, tables, cu, ctx)
    used = tables[:, 0]
    assert (want[1][used] > scales[used]).all()
    args = i32_dev(tables), i32_dev(cu), i32_dev(ctx), new
    k = bf16_dev(x)
    for _ in range(10):
        t = [u8_dev(codes), u8_dev(codes), f32_dev(scales), f32_dev(scales)]
        pa.pa_store_kvcache_fp8_blockscale(k, k, *t, *args)
        for got_c, got_s in ((t[0], t[2]), (t[1], t[3])):
            assert np.array_equal(got_s.cpu().numpy(), want[1]) and same_codes(got_c.cpu().numpy(), want[0])


def test_append_bad_lengths_and_blocks_are_reported_and_skipped():
    rng = np.random.default_rng(2)
    hkv, d, bs = 2, 128, 16
    k = bf16_dev(f32_to_bf16_bits(rng.standard_normal((6, hkv, d)).astype(np.float32)))
    kc, ks = pools_of(rng, 5, bs, hkv, d)
    good = np.array([[1], [2], [3]], np.int32)

    def run(tables, cu, ctx, m=2):
        t = [u8_dev(kc), u8_dev(kc), f32_dev(ks), f32_dev(ks)]
        with pytest.raises(pa.PAError) as e:
            pa.pa_store_kvcache_fp8_blockscale(k, k, *t, i32_dev(tables), i32_dev(np.array(cu)),
                                               i32_dev(np.array(ctx)), m)
        assert e.value.status == 3
        return t[0].cpu().numpy()

    want = fp8_block.append(kc, ks, to_bits(k), good, [0, 2, 4, 6], [2, 2, 2])[0]
    for tables, cu, ctx, skipped in (
            (np.array([[1], [5], [3]], np.int32), [0, 2, 4, 6], [2, 2, 2], 2),     # block past the pool
            (np.array([[1], [-1], [3]], np.int32), [0, 2, 4, 6], [2, 2, 2], 2),
            (good, [0, 2, 4, 6], [2, 1, 2], 2),                                     # more new than context
            (good, [0, 2, 4, 6], [2, 17, 2], 2),                                    # context past the table
            (good, [0, 2, 4, 7], [2, 2, 3], 3)):                                    # past the tokens
        got = run(tables, cu, ctx, 3)
        exp = want.copy()
        exp[skipped] = kc[skipped]
        assert np.array_equal(got, exp)
    got = run(good, [0, 2, 5, 6], [2, 3, 1], 2)                                     # above max_q_len
    assert np.array_equal(got[2], kc[2]) and np.array_equal(got[1], want[1])


KERNELS = [
    # kv heads, head dim, block size, new rows
    (2, 128, 16, [1] * 7),                       # one row a sequence
    (40, 64, 64, [1] * 5),
    (2, 128, 16, [3, 2, 7, 8, 1]),               # warps of up to 8 rows
    (4, 64, 64, [12, 9, 16, 1] * 80),            # of up to 16
    (8, 128, 64, [100, 70, 130]),                # CTAs of 2 heads, half the rows a thread
    (3, 64, 64, [100, 70, 130]),                 # of one
    (8, 128, 64, [100, 70, 130, 90] * 20),       # of 4 heads
    (2, 128, 128, [150, 140, 200, 190] * 80),    # of 2
    (3, 128, 256, [300, 400, 350] * 40),         # of one
    (1, 128, 1024, [1500, 900]),                 # a cluster a block
    (2, 64, 1024, [1400, 1100, 1200]),
    (8, 128, 1024, [1500, 1200] * 10),
    (8, 128, 16, [100, 70, 90]),                 # 64 positions of small blocks
    (8, 64, 32, [900, 700, 1000, 800] * 4),
    (8, 128, 64, [1] * 40 + [600] + [2] * 20),   # counted units
    (3, 128, 1024, [1] * 25 + [900] + [40, 3, 16] * 8),
]


def faulty_calls(new, ctx, cu, tables, bs, nb):
    """(what, cu, ctx, tables, bound, sequence skipped whole or None, table entry skipped or None)"""
    s, last, bound = int(np.argmax(new)), len(new) - 1, max(new)
    yield "a context shorter than its new rows", cu, np.where(np.arange(len(new)) == s, new[s] - 1, ctx), tables, bound, s, None
    yield "a context past the table", cu, np.where(np.arange(len(new)) == s, bs * tables.shape[1] + 1, ctx), tables, bound, s, None
    yield "a negative context", cu, np.where(np.arange(len(new)) == s, -5, ctx), tables, bound, s, None
    over = cu.copy()
    over[-1] += 1
    yield "rows past the tokens", over, np.where(np.arange(len(new)) == last, ctx + 1, ctx), tables, bound, last, None
    falling = cu.copy()
    falling[last] = cu[-1] + 1      # the last sequence ends before it begins, the one before it past the tokens
    yield "falling lengths", falling, ctx, tables, bound, (last - 1, last), None
    if bound > 1:
        yield "more new rows than the bound", cu, ctx, tables, bound - 1, [i for i, n in enumerate(new) if n == bound], None
    for block in sorted({(int(ctx[s]) - 1) // bs, (int(ctx[s]) - new[s]) // bs}):
        for bad in (nb, -1, 2 ** 31 - 1):
            t = tables.copy()
            t[s, block] = bad
            yield f"block {bad}", cu, ctx, t, bound, None, (s, block)


@pytest.mark.parametrize("hkv,d,bs,new", KERNELS)
def test_every_kernel_reports_and_skips_what_does_not_fit(hkv, d, bs, new):
    rng = np.random.default_rng(bs + sum(new))
    ctx = np.array(new) + 5
    tables, nb = tables_of(rng, ctx, bs)
    cu = np.concatenate([[0], np.cumsum(new)])
    k = bf16_dev(f32_to_bf16_bits(rng.standard_normal((int(cu[-1]), hkv, d)).astype(np.float32)))
    kc, ks = pools_of(rng, nb, bs, hkv, d)
    want = fp8_block.append(kc, ks, to_bits(k), tables, cu, ctx)
    dev = u8_dev(kc), f32_dev(ks)
    for what, cu2, ctx2, tables2, bound, skipped, entry in faulty_calls(new, ctx, cu, tables, bs, nb):
        t = [dev[0].clone(), dev[0].clone(), dev[1].clone(), dev[1].clone()]
        with pytest.raises(pa.PAError) as e:
            pa.pa_store_kvcache_fp8_blockscale(k, k, *t, i32_dev(tables2), i32_dev(cu2), i32_dev(ctx2), bound)
        assert e.value.status == 3, what
        codes, scales = want[0].copy(), want[1].copy()
        left = [int(tables[entry])] if entry else [int(b) for s in np.atleast_1d(skipped) for b in tables[s] if b >= 0]
        codes[left], scales[left] = kc[left], ks[left]
        for got_c, got_s in ((t[0], t[2]), (t[1], t[3])):
            assert np.array_equal(got_c.cpu().numpy(), codes), what
            assert np.array_equal(got_s.cpu().numpy(), scales), what


@pytest.mark.parametrize("new", [[1] * 6, [3, 1, 2], [70, 200], [700, 800]])
def test_queries_of_skipped_sequences_are_turned(new):
    """A sequence whose lengths do not fit loses its rows, not its queries."""
    import torch
    rng = np.random.default_rng(sum(new))
    hq, hkv, d, bs, T = 4, 2, 128, 64, sum(new)
    ctx = np.array(new) + 5
    tables, nb = tables_of(rng, ctx, bs)
    cu = np.concatenate([[0], np.cumsum(new)])
    qkv = bf16_dev(f32_to_bf16_bits(rng.standard_normal((T, hq + 2 * hkv, d)).astype(np.float32)))
    kc, ks = pools_of(rng, nb, bs, hkv, d)
    t = [u8_dev(kc), u8_dev(kc), f32_dev(ks), f32_dev(ks)]
    pos, f = i32_dev(np.arange(T)), torch.tensor(pa.pa_rope_inv_freq(d)[0], device="cuda")
    want, got = (torch.empty((T, hq, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    pa.pa_rope(want, qkv[:, :hq], pos, f)
    ctx[1] = 0
    with pytest.raises(pa.PAError) as e:
        pa.pa_rope_store_kvcache_fp8_blockscale(got, qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], *t,
                                                i32_dev(tables), i32_dev(cu), i32_dev(ctx), max(new), pos, f)
    assert e.value.status == 3
    assert np.array_equal(to_bits(got), to_bits(want))
    left = tables[1][tables[1] >= 0]
    assert np.array_equal(t[0].cpu().numpy()[left], kc[left])
