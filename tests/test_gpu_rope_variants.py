"""The rotary store with 1, 2, 4 and 8 tokens a CTA at both head dims: against the formula, and
against the calls made apart (which take other variants)."""
import numpy as np
import pytest
import torch

import paged_kv_cache_442_b200 as pa
import tests.test_gpu_rope as base
from tests.gpu_helpers import bf16_dev, i32_dev, to_f64

pytestmark = pytest.mark.gpu

# tokens, q heads, kv heads, head dim, rotated dims (a card of 148 SMs)
SHAPES = [(592, 6, 1, 64, 64), (592, 6, 1, 128, 96),
          (593, 60, 2, 64, 64), (4736, 52, 6, 64, 32), (700, 28, 2, 128, 128),      # 2
          (593, 24, 4, 64, 48), (4737, 60, 2, 64, 64), (2368, 6, 1, 64, 16), (4737, 28, 2, 128, 64),  # 4
          (2369, 14, 1, 64, 64), (6001, 2, 1, 64, 48), (2371, 6, 1, 128, 112)]      # 8


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("t,hq,hkv,d,rot", SHAPES)
def test_tokens_a_cta(t, hq, hkv, d, rot, inter):
    base.test_rope_store_equals_rope_then_store(t, hq, hkv, d, 64, rot, inter)
    rng = np.random.default_rng(t)
    x = base.rows(rng, t, hq + 2 * hkv, d)
    positions = rng.integers(-1000, 2 ** 24, t).astype(np.int32)
    fd, f, amp = base.table(rot, factor=4.0)
    out = torch.full(x.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
    pa.pa_rope(out, bf16_dev(x), i32_dev(positions), fd, interleaved=inter, amplitude=amp)
    some = rng.permutation(t)[:40]
    some[:8] = np.arange(t - 8, t)
    base.check(to_f64(out)[some], x[some], positions[some], f, inter, amp)
