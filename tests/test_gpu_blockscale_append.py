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
