"""GPU parity of the e4m3 cache with block scales: append (bit for bit against the oracle) and
decode (the decode bar, and 2^-7 over the whole tensor: the output's rounding to bf16 is at
most 2^-8 of a value and the two-term probabilities add at most as much)."""
import numpy as np
import pytest
import torch

import paged_kv_cache_442_b200 as pa
from oracle import fp8_block
from tests.gpu_helpers import assert_close, bf16_dev, i32_dev, to_bits, to_f64
from workloads import f32_to_bf16_bits

pytestmark = pytest.mark.gpu


def u8_dev(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.uint8)).cuda()


def f32_dev(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).cuda()


def tables_of(rng, ctx, bs, spare=2):
    """Shuffled block tables; returns (tables, blocks of the pool)."""
    need = [-(-max(0, int(c)) // bs) for c in ctx]
    nb = sum(need) + spare
    perm = rng.permutation(nb)
    out = np.full((len(ctx), max(1, max(need))), -1, np.int32)
    at = 0
    for s, n in enumerate(need):
        out[s, :n] = perm[at:at + n]
        at += n
    return out, nb


# ------------------------------------------------------------------------------ append
def wild_rows(rng, t, hkv, d):
    """bf16 rows whose sizes vary by row (scales grow as a block fills), with edges."""
    x = rng.standard_normal((t, hkv, d)) * np.exp(rng.uniform(-3, 3, (t, hkv, 1)))
    x = x.astype(np.float32)
    x[0, 0] = 0.0
    if t > 8:
        x[2, 0] = 1e-39                      # bf16 subnormals
        x[3, 0] = 448.0 * 2.0 ** -3          # exactly at a scale's top
        x[4, -1] = 3e38
        x[5, 0, :4] = np.inf
        x[6, 0, 0] = np.nan
        x[7, 0] = np.round(rng.standard_normal(d) * 4) / 4
    return f32_to_bf16_bits(x)


def pools_of(rng, nb, bs, hkv, d):
    codes = rng.integers(0, 256, (nb, bs, hkv, d)).astype(np.uint8)
    codes[(codes & 0x7F) == 0x7F] = 0x33
    scales = np.ldexp(1.0, rng.integers(-8, 3, (nb, hkv))).astype(np.float32)
    return codes, scales


def same_codes(got, want):
    """Equal, where both NaN codes count as one."""
    g, w = got.copy(), want.copy()
    g[(g & 0x7F) == 0x7F] = 0x7F
    w[(w & 0x7F) == 0x7F] = 0x7F
    return np.array_equal(g, w)


@pytest.mark.parametrize("hkv,d,bs,new,old", [
    (8, 128, 256, [1] * 6, [0, 1, 255, 256, 300, 37]),       # decode steps
    (2, 64, 16, [1, 1, 1], [0, 15, 16]),
    (40, 128, 64, [1, 0, 1], [63, 5, 64]),                    # more heads than a pass, one idle
    (96, 128, 16, [1] * 48, list(range(1, 49))),              # scales grow in pass after pass
    (3, 128, 1024, [1, 1], [1023, 1024]),
    (8, 128, 64, [3, 1, 2], [62, 0, 31]),                     # a few rows each
    (2, 128, 16, [40, 0, 16, 7], [0, 5, 8, 9]),               # blocks of 16, one sequence idle
    (1, 128, 32, [33, 64, 95], [31, 0, 1]),
    (3, 128, 64, [61, 130, 1], [3, 63, 64]),
    (2, 128, 256, [600, 256], [10, 0]),                       # whole blocks in registers
    (1, 64, 512, [700], [100]),
    (8, 128, 256, [700, 513, 0, 900], [10, 255, 5, 256]),     # many units per SM
    (4, 128, 64, [3000, 200], [63, 5]),
    (2, 64, 128, [2500, 77], [100, 127]),
    (3, 128, 256, [3000], [1]),
    (2, 128, 1024, [1500, 900], [700, 0]),                    # blocks read twice
    # many units: eight (row, head) pairs a thread, of 2, 4 and 1 heads, a block by one CTA and by several
    (2, 128, 128, [6000, 3000], [5, 127]),
    (4, 64, 128, [5000, 4000, 3000], [1, 64, 120]),
    (2, 64, 256, [6000, 5000, 4000], [0, 9, 255]),
    (8, 128, 1024, [1500, 900, 2000], [1000, 3, 512]),
    (8, 128, 64, [12] * 300, list(range(300))),               # up to sixteen rows a warp
    (4, 64, 16, [16, 9, 0, 3] * 200, list(range(800))),
    (8, 128, 16, [5000, 3000], [3, 16]),                      # several blocks a CTA, of 4, 2 and 1 heads
    (4, 64, 16, [9000, 7000], [15, 1]),
    (2, 128, 32, [6000, 33], [5, 31]),
    (2, 64, 32, [5000], [40]),
    (3, 128, 16, [17, 100, 0, 63, 1], [15, 47, 9, 1, 63]),
    (1, 128, 32, [500, 64], [95, 64]),
    (8, 128, 64, [16, 9, 12, 1], [60, 0, 52, 3]),             # nine to sixteen rows a CTA
    (3, 64, 512, [2000, 3000, 1000, 2500, 1500, 700], [1, 2, 3, 4, 500, 511]),
    # one long chunk beside many short ones
    (8, 128, 16, [1] * 30 + [700] + [2, 0, 17, 5] * 8, list(range(63))),
    (8, 128, 64, [1] * 20 + [33, 17, 16, 0] + [600] + [1] * 20, list(range(40, 85))),
    (3, 128, 1024, [1] * 25 + [900] + [40, 3, 16] * 8, [1000] * 20 + list(range(30))),
    (4, 64, 256, [1] * 40 + [1300, 300] + [1, 2] * 10, list(range(200, 262))),
    (1, 64, 64, [1] * 1100 + [0] * 5 + [300] + [1, 2, 3] * 100, [3] * 1406),   # two windows of sequences
])
def test_append_matches_the_oracle_bit_for_bit(hkv, d, bs, new, old):
    rng = np.random.default_rng(bs + d + sum(new))
    ctx = np.array(new) + np.array(old)
    tables, nb = tables_of(rng, ctx, bs)
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    T = int(cu[-1])
    k, v = wild_rows(rng, T, hkv, d), wild_rows(rng, T, hkv, d)[::-1].copy()
    kc, ks = pools_of(rng, nb, bs, hkv, d)
    vc, vs = pools_of(rng, nb, bs, hkv, d)
    want_k = fp8_block.append(kc, ks, k, tables, cu, ctx)
    want_v = fp8_block.append(vc, vs, v, tables, cu, ctx)
    dk, dv, dks, dvs = u8_dev(kc), u8_dev(vc), f32_dev(ks), f32_dev(vs)
    pa.pa_store_kvcache_fp8_blockscale(bf16_dev(k), bf16_dev(v), dk, dv, dks, dvs, i32_dev(tables),
                                       i32_dev(cu), i32_dev(ctx), max(new))
    assert np.array_equal(dks.cpu().numpy(), want_k[1]) and np.array_equal(dvs.cpu().numpy(), want_v[1])
    assert same_codes(dk.cpu().numpy(), want_k[0])
    assert same_codes(dv.cpu().numpy(), want_v[0])


@pytest.mark.parametrize("inter,rot", [(False, 128), (True, 64), (False, 16), (True, 48), (False, 0)])
@pytest.mark.parametrize("new,bs,steady", [([1, 1, 1], 256, True), ([1, 0, 1, 1], 64, True), ([70, 3], 64, False),
                                           ([70, 3], 64, True), ([300, 129, 1000], 256, True), ([5, 20], 32, True),
                                           ([1024 + 700], 1024, True), ([400], 512, False),
                                           ([1] * 150 + [900] + [20, 1, 2] * 9, 256, True),
                                           ([3] * 200 + [600], 16, True), ([300, 77, 1], 16, True),
                                           ([200, 55], 32, False)])
def test_rope_append_equals_rope_then_append(new, bs, steady, inter, rot):
    """steady: positions follow one another, as a rule; else they are anywhere."""
    rng = np.random.default_rng(rot + bs)
    hq, hkv, d = 4, (1 if bs == 512 else 2), 128
    ctx = np.array(new) + 13
    tables, nb = tables_of(rng, ctx, bs)
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    T = int(cu[-1])
    qkv = bf16_dev(f32_to_bf16_bits(rng.standard_normal((T, hq + 2 * hkv, d)).astype(np.float32)))
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    pos = rng.integers(-2 ** 20, 2 ** 30, T)
    if steady:
        pos = np.concatenate([rng.integers(-300, 10 ** 6) + np.arange(n) for n in new])
    pos = i32_dev(pos)
    f = torch.tensor(pa.pa_rope_inv_freq(rot)[0] if rot else [], dtype=torch.float32, device="cuda")
    kc, ks = pools_of(rng, nb, bs, hkv, d)
    vc, vs = pools_of(rng, nb, bs, hkv, d)
    a = [u8_dev(kc), u8_dev(vc), f32_dev(ks), f32_dev(vs)]
    b = [t.clone() for t in a]
    q_out = torch.empty((T, hq, d), dtype=torch.bfloat16, device="cuda")
    rest = (i32_dev(tables), i32_dev(cu), i32_dev(ctx), max(new))
    pa.pa_rope_store_kvcache_fp8_blockscale(q_out, q, k, v, *a, *rest, pos, f, interleaved=inter, amplitude=1.25)
    rq, rk = torch.empty_like(q_out), torch.empty((T, hkv, d), dtype=torch.bfloat16, device="cuda")
    pa.pa_rope(rq, q, pos, f, interleaved=inter, amplitude=1.25)
    pa.pa_rope(rk, k, pos, f, interleaved=inter, amplitude=1.25)
    pa.pa_store_kvcache_fp8_blockscale(rk, v, *b, *rest)
    assert np.array_equal(to_bits(q_out), to_bits(rq))
    for x, y in zip(a, b):
        assert torch.equal(x, y)


@pytest.mark.parametrize("last", [2 ** 31 - 1, -1, 0])
def test_rope_append_at_the_ends_of_the_positions(last):
    """Positions that run up to the largest int32, to -1 and through 0, over a shared block."""
    rng = np.random.default_rng(7)
    n, bs, hq, hkv, d = 1500, 1024, 2, 1, 128
    tables, nb = tables_of(rng, [n], bs)
    qkv = bf16_dev(f32_to_bf16_bits(rng.standard_normal((n, hq + 2 * hkv, d)).astype(np.float32)))
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    pos = i32_dev(np.arange(last - n + 1, last + 1) if last else np.arange(n) - 700)
    f = torch.tensor(pa.pa_rope_inv_freq(d)[0], dtype=torch.float32, device="cuda")
    a = [torch.zeros((nb, bs, hkv, d), dtype=torch.uint8, device="cuda") for _ in range(2)]
    a += [torch.zeros((nb, hkv), dtype=torch.float32, device="cuda") for _ in range(2)]
    b = [t.clone() for t in a]
    q_out = torch.empty((n, hq, d), dtype=torch.bfloat16, device="cuda")
    rest = (i32_dev(tables), i32_dev(np.array([0, n])), i32_dev(np.array([n])), n)
    pa.pa_rope_store_kvcache_fp8_blockscale(q_out, q, k, v, *a, *rest, pos, f)
    rk = torch.empty((n, hkv, d), dtype=torch.bfloat16, device="cuda")
    pa.pa_rope(rk, k, pos, f)
    pa.pa_store_kvcache_fp8_blockscale(rk, v, *b, *rest)
    for x, y in zip(a, b):
        assert torch.equal(x, y)


@pytest.mark.parametrize("seqs", [0, 2])
def test_rope_append_of_nothing_still_turns_the_queries(seqs):
    """Padding tokens only: no sequence, or none with new rows and 0 as the bound of their count."""
    rng = np.random.default_rng(8)
    qkv = bf16_dev(f32_to_bf16_bits(rng.standard_normal((5, 8, 128)).astype(np.float32)))
    q, k, v = qkv[:, :4], qkv[:, 4:6], qkv[:, 6:]
    kc, ks = pools_of(rng, 3, 16, 2, 128)
    dev = [u8_dev(kc), u8_dev(kc), f32_dev(ks), f32_dev(ks)]
    pos, f = i32_dev(np.arange(5)), torch.tensor(pa.pa_rope_inv_freq(128)[0], device="cuda")
    want, got = (torch.full((5, 4, 128), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    pa.pa_rope(want, q, pos, f)
    lens = i32_dev(np.zeros(seqs)), 0
    tables = i32_dev(np.ones((seqs, 1)))
    pa.pa_rope_store_kvcache_fp8_blockscale(got, q, k, v, *dev, tables, i32_dev(np.zeros(seqs + 1)), *lens, pos, f)
    assert torch.equal(got.view(torch.int16), want.view(torch.int16))
    assert np.array_equal(dev[0].cpu().numpy(), kc) and np.array_equal(dev[2].cpu().numpy(), ks)


@pytest.mark.parametrize("bs", [64, 512])
def test_a_long_append_is_complete_for_what_follows(bs):
    """The queries and the rows of many tokens are two launches that may overlap; what comes
    before and after them in the stream must not. Captured and replayed."""
    rng = np.random.default_rng(bs)
    n, hq, hkv, d = 2600, 16, 4, 128
    tables, nb = tables_of(rng, [n], bs)
    qkv = bf16_dev(f32_to_bf16_bits(rng.standard_normal((n, hq + 2 * hkv, d)).astype(np.float32)))
    work, seen_q = torch.empty_like(qkv), torch.empty((n, hq, d), dtype=torch.bfloat16, device="cuda")
    q_out = torch.empty_like(seen_q)
    pools = [torch.zeros((nb, bs, hkv, d), dtype=torch.uint8, device="cuda") for _ in range(2)]
    pools += [torch.zeros((nb, hkv), dtype=torch.float32, device="cuda") for _ in range(2)]
    seen = [torch.empty_like(t) for t in pools]
    rest = (i32_dev(tables), i32_dev(np.array([0, n])), i32_dev(np.array([n])), n)
    pos, f = i32_dev(np.arange(n)), torch.tensor(pa.pa_rope_inv_freq(d)[0], device="cuda")

    def step():
        work.copy_(qkv)
        pa.pa_rope_store_kvcache_fp8_blockscale(q_out, work[:, :hq], work[:, hq:hq + hkv], work[:, hq + hkv:],
                                                *pools, *rest, pos, f)
        for a, b in zip([seen_q] + seen, [q_out] + pools):
            a.copy_(b)
            b.zero_()
        work.zero_()

    step()
    want = [t.clone() for t in [seen_q] + seen]
    rq = torch.empty_like(q_out)
    pa.pa_rope(rq, qkv[:, :hq], pos, f)
    assert torch.equal(rq.view(torch.int16), want[0].view(torch.int16)) and all(t.any() for t in want)
    pa.pa_set_debug_checks(False)
    try:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            for _ in range(3):
                step()
        for _ in range(10):
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip([seen_q] + seen, want))
        del graph
    finally:
        pa.pa_set_debug_checks(True)
    assert pa.pa_check_device_errors() == 0


@pytest.mark.parametrize("bs", [16, 32])
def test_append_of_small_blocks_skips_a_bad_one(bs):
    rng = np.random.default_rng(13)
    hkv, d, new, old = 2, 128, np.array([100, 70]), 9
    ctx = new + old
    tables, nb = tables_of(rng, ctx, bs)
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    k = wild_rows(rng, int(cu[-1]), hkv, d)
    kc, ks = pools_of(rng, nb, bs, hkv, d)
    codes, scales = fp8_block.append(kc, ks, k, tables, cu, ctx)
    for at, bad in (((0, 2), nb), ((1, 0), -1)):
        t = [u8_dev(kc), u8_dev(kc), f32_dev(ks), f32_dev(ks)]
        broken = tables.copy()
        broken[at] = bad
        with pytest.raises(pa.PAError) as e:
            pa.pa_store_kvcache_fp8_blockscale(bf16_dev(k), bf16_dev(k), *t, i32_dev(broken), i32_dev(cu), i32_dev(ctx), 100)
        assert e.value.status == 3
        want_c, want_s, left = codes.copy(), scales.copy(), int(tables[at])
        want_c[left], want_s[left] = kc[left], ks[left]
        for got_c, got_s in ((t[0], t[2]), (t[1], t[3])):
            assert same_codes(got_c.cpu().numpy(), want_c) and np.array_equal(got_s.cpu().numpy(), want_s)


def test_append_of_a_ragged_batch_reports_what_it_skips():
    rng = np.random.default_rng(12)
    new = np.array([1] * 40 + [600] + [2] * 20)
    hkv, d, bs, n, old = 8, 128, 64, len(new), 5
    ctx = new + old
    tables, nb = tables_of(rng, ctx, bs)
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    k = bf16_dev(f32_to_bf16_bits(rng.standard_normal((int(cu[-1]), hkv, d)).astype(np.float32)))
    kc, ks = pools_of(rng, nb, bs, hkv, d)
    want = fp8_block.append(kc, ks, to_bits(k), tables, cu, ctx)
    skipped, bad_block = (3, 45), 40
    ctx2, tables2 = ctx.copy(), tables.copy()
    ctx2[3], ctx2[45] = 0, bs * tables.shape[1] + 1     # fewer than the new rows; past the table
    tables2[bad_block, 2] = nb                          # one block of the chunk
    t = [u8_dev(kc), u8_dev(kc), f32_dev(ks), f32_dev(ks)]
    with pytest.raises(pa.PAError) as e:
        pa.pa_store_kvcache_fp8_blockscale(k, k, *t, i32_dev(tables2), i32_dev(cu), i32_dev(ctx2), 600)
    assert e.value.status == 3
    codes, scales = want[0].copy(), want[1].copy()
    left = [int(tables[s, 0]) for s in skipped] + [int(tables[bad_block, 2])]
    codes[left], scales[left] = kc[left], ks[left]
    for got_c, got_s in ((t[0], t[2]), (t[1], t[3])):
        assert np.array_equal(got_c.cpu().numpy(), codes) and np.array_equal(got_s.cpu().numpy(), scales)


# ------------------------------------------------------------------------------ decode
class Case:
    """Random codes and scales as pools (every byte of rows past a context is a NaN code)."""

    def __init__(self, ctx, hq, hkv, bs, seed, q_factor=1.0, spread=1.0, widen=0):
        rng = np.random.default_rng(seed)
        self.ctx = np.array(ctx, np.int32)
        self.tables, self.nb = tables_of(rng, np.maximum(self.ctx, 0), bs)
        if widen:
            self.tables = np.pad(self.tables, ((0, 0), (0, widen)), constant_values=-1)
        self.q = f32_to_bf16_bits((q_factor * rng.standard_normal((len(ctx), hq, 128))).astype(np.float32))
        shape = (self.nb, bs, hkv, 128)

        def pool():
            c = np.full(shape, 0x7F, np.uint8)
            s = np.full((self.nb, hkv), np.nan, np.float32)
            for i, n in enumerate(np.maximum(self.ctx, 0)):
                for b in range(-(-int(n) // bs)):
                    rows = min(bs, int(n) - b * bs)
                    x = rng.standard_normal((rows, hkv, 128))
                    c[self.tables[i, b], :rows] = fp8_block.encode(np.clip(x * 96, -448, 448))
                    s[self.tables[i, b]] = np.exp(spread * rng.standard_normal(hkv)) / 96
            return c, s
        (self.kc, self.ks), (self.vc, self.vs) = pool(), pool()
        self.bs, self.hkv, self.scale = bs, hkv, 128 ** -0.5

    def gpu(self, ws=None, max_ctx=None, out=None, stream=None):
        if not hasattr(self, "dev"):
            self.dev = (bf16_dev(self.q), u8_dev(self.kc), u8_dev(self.vc), f32_dev(self.ks), f32_dev(self.vs),
                        i32_dev(self.tables), i32_dev(self.ctx))
        q = self.dev[0]
        out = torch.full_like(q, float("nan")) if out is None else out
        ws = pa.decode_fp8_blockscale_workspace(q.shape[0], q.shape[1], self.hkv) if ws is None else ws
        pa.pa_decode_fp8_blockscale(out, *self.dev, self.scale, int(max(0, self.ctx.max())) if max_ctx is None else max_ctx,
                                    ws, stream=stream)
        return out

    def oracle(self):
        return fp8_block.decode(self.q, self.kc, self.vc, self.ks, self.vs, self.tables, self.ctx, self.scale)


def close(gpu, ref, what=""):
    c = assert_close(to_f64(gpu), ref, what)
    assert c["norm_rel"] <= 2.0 ** -7, (what, c)


@pytest.mark.parametrize("ctx,hq,hkv,bs", [
    ([1], 1, 1, 16), ([5, 0, 256, 257, -3, 31], 4, 2, 16), ([512], 8, 8, 32), ([100, 700, 33], 16, 8, 256),
    ([1000, 1, 2047, 64], 32, 8, 64), ([300, 300], 16, 1, 128), ([700, 129], 32, 2, 16), ([1025, 600], 3, 3, 512),
    ([2500, 1024], 6, 6, 1024), ([9000], 8, 1, 128), ([1, 255, 256, 1023, 5], 2, 2, 1024), ([30000], 1, 1, 32), ([0, 0], 4, 2, 64), ([40] * 70, 4, 4, 16),
    ([20000], 2, 1, 16), ([6001, 17], 16, 4, 256),
])
def test_decode_matches_the_oracle(ctx, hq, hkv, bs):
    c = Case(ctx, hq, hkv, bs, seed=len(ctx) + hq + bs)
    close(c.gpu(), c.oracle(), f"{ctx[:4]} {hq}/{hkv} {bs}")


@pytest.mark.parametrize("ctx,hq,hkv,bs", [
    ([512, 0, 511, 257, 1], 16, 8, 64), ([513, 0, 511, 257, 1], 16, 8, 64),   # each item whole; one split
    ([512] * 36, 8, 4, 128), ([512] * 38, 8, 4, 128),                         # as many items as groups; more
    ([3, 0, 0, 500] * 18, 4, 1, 16), ([0] * 33 + [512, 0, 400], 32, 2, 256),  # beyond a window of 32
])
def test_decode_short_contexts_whole_and_split(ctx, hq, hkv, bs):
    c = Case(ctx, hq, hkv, bs, seed=sum(ctx) + bs)
    close(c.gpu(), c.oracle(), f"{len(ctx)} x {max(ctx)} {hq}/{hkv} {bs}")


@pytest.mark.parametrize("g", [1, 2, 4, 8, 16])
@pytest.mark.parametrize("q_factor,spread", [(8.0, 0.3), (0.0, 2.0), (30.0, 1.0)])
def test_decode_peaked_flat_and_uneven_scales(g, q_factor, spread):
    c = Case([3000, 517, 60], 2 * g, 2, 64, seed=g, q_factor=q_factor, spread=spread)
    close(c.gpu(), c.oracle(), f"G {g} q x{q_factor} spread {spread}")


def test_decode_one_dominant_value_block():
    """A block whose V scale is 2^9 above the others, anywhere in the context."""
    for at in (0, 5, 11):
        c = Case([3000], 4, 2, 256, seed=at)
        c.vs[c.tables[0, at]] *= 512.0
        close(c.gpu(), c.oracle(), f"dominant block {at}")


def test_decode_zero_value_scales():
    c = Case([1500, 700], 4, 2, 64, seed=3)
    c.vs[c.tables[0, :10]] = 0.0          # the first tiles' values are all zero
    c.vs[c.tables[1, :11]] = 0.0          # every value of the second sequence
    out = c.gpu()
    close(out[:1], c.oracle()[:1])
    assert not to_f64(out)[1].any()


def test_decode_is_deterministic_and_reuses_a_workspace():
    c = Case([7000, 100, 4100, 0, 900], 8, 4, 64, seed=9)
    big = Case([300] * 40, 8, 4, 16, seed=10)
    ws = pa.decode_fp8_blockscale_workspace(5, 8, 4)
    ws.view(torch.int32).fill_(-1)
    first, other = c.gpu(ws), big.gpu(ws)
    for _ in range(20):
        assert torch.equal(c.gpu(ws).view(torch.int16), first.view(torch.int16))
        assert torch.equal(big.gpu(ws).view(torch.int16), other.view(torch.int16))
    close(first, c.oracle())


@pytest.mark.parametrize("g", [1, 4, 16])
def test_decode_beside_other_work_keeps_its_bits(g):
    """Another stream's traffic moves the order in which the parts of split items arrive."""
    c = Case([5000, 700, 3300, 40, 2600, 9000] * 4, 4 * g, 4, 64, seed=g)
    ws = pa.decode_fp8_blockscale_workspace(24, 4 * g, 4)
    first = c.gpu(ws)
    junk, side = torch.zeros(32 << 20, device="cuda"), torch.cuda.Stream()
    torch.cuda.synchronize()
    for i in range(30):
        if i % 3:
            with torch.cuda.stream(side):
                junk[:: i % 3 + 1].add_(1.0)
        assert torch.equal(c.gpu(ws).view(torch.int16), first.view(torch.int16))
    torch.cuda.synchronize()


def test_decode_graphs_share_a_workspace():
    """Two captured calls on one workspace, replayed in turn without clearing it."""
    a, b = Case([5000, 40], 8, 2, 64, seed=21), Case([900] * 9, 8, 2, 16, seed=22)
    ws = pa.decode_fp8_blockscale_workspace(9, 8, 2)
    want = [x.gpu(ws) for x in (a, b)]
    outs = [torch.empty_like(w) for w in want]
    pa.pa_set_debug_checks(False)
    try:
        graphs = []
        for x, o in zip((a, b), outs):
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                x.gpu(ws, out=o)
            torch.cuda.current_stream().wait_stream(side)
            torch.cuda.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                x.gpu(ws, out=o)
            graphs.append(g)
        for i in (0, 1, 0, 0, 1, 1, 0):
            outs[i].zero_()
            graphs[i].replay()
            torch.cuda.synchronize()
            assert torch.equal(outs[i].view(torch.int16), want[i].view(torch.int16))
        del graphs
    finally:
        pa.pa_set_debug_checks(True)
    assert pa.pa_check_device_errors() == 0


def test_decode_on_two_streams_with_their_own_workspaces():
    a, b = Case([4000, 300], 8, 2, 64, seed=31), Case([2000] * 6, 16, 2, 32, seed=32)
    want = [a.gpu().clone(), b.gpu().clone()]
    torch.cuda.synchronize()
    pa.pa_set_debug_checks(False)
    try:
        streams = [torch.cuda.Stream() for _ in range(2)]
        ws = [pa.decode_fp8_blockscale_workspace(8, 8, 2), pa.decode_fp8_blockscale_workspace(8, 16, 2)]
        outs = [torch.empty_like(w) for w in want]
        torch.cuda.synchronize()
        for _ in range(5):
            for x, w, o, st in zip((a, b), ws, outs, streams):
                x.gpu(w, out=o, stream=st)
        torch.cuda.synchronize()
    finally:
        pa.pa_set_debug_checks(True)
    for o, w in zip(outs, want):
        assert torch.equal(o.view(torch.int16), w.view(torch.int16))


def test_decode_bad_block_id_and_too_long_a_context_are_reported():
    c = Case([500, 90], 4, 2, 64, seed=4)
    ok = c.gpu()
    c.dev[5][0, 2] = c.nb + 7
    out = torch.zeros_like(ok)
    with pytest.raises(pa.PAError) as e:
        c.gpu(out=out)
    assert e.value.status == 3
    assert torch.equal(out[1], ok[1])          # the other sequence is not touched by it
    d = Case([500, 90], 4, 2, 64, seed=4, widen=3)
    with pytest.raises(pa.PAError) as e:
        d.gpu(max_ctx=400, out=out)
    assert e.value.status == 3
    d.ctx = np.array([400, 90], np.int32)      # clipped to the host's bound
    close(out, d.oracle())


def test_decode_clipped_to_nothing_gives_zeros():
    c = Case([70, 0, 300], 4, 2, 64, seed=5)
    out = torch.full((3, 4, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(pa.PAError) as e:
        c.gpu(max_ctx=0, out=out)
    assert e.value.status == 3
    assert not out.any()


def test_decode_not_a_number_stays_in_its_head():
    """A NaN in one query head reaches that head's output only; NaN and infinite rows past a
    context reach none (every Case has them)."""
    c = Case([700, 40], 4, 2, 64, seed=6)
    ok = c.gpu()
    c.dev[0][0, 1, 5] = float("nan")
    out = c.gpu()
    assert torch.isnan(out[0, 1].float()).all()
    same = torch.ones(2, 4, dtype=torch.bool)
    same[0, 1] = False
    assert torch.equal(out[same.cuda()].view(torch.int16), ok[same.cuda()].view(torch.int16))


def test_decode_wait_that_runs_out_is_reported():
    c = Case([700, 129, 3000, 1], 8, 2, 64, seed=33)
    ws = pa.decode_fp8_blockscale_workspace(4, 8, 2)
    pa.pa_set_wait_limit_ns(1)
    try:
        with pytest.raises(pa.PAError) as e:
            c.gpu(ws)
        assert e.value.status == 5
    finally:
        pa.pa_set_wait_limit_ns(0)
    torch.cuda.synchronize()
    assert pa.pa_check_device_errors() == 0
    close(c.gpu(ws), c.oracle(), "after a timeout")


# --------------------------------------------------------------------- a run of them together
@pytest.mark.parametrize("bs,rot,inter", [(64, 128, False), (16, 64, True)])
def test_prefill_then_decode_steps_over_the_block_scaled_cache(bs, rot, inter):
    """Chunks, then single tokens: rotate and append, decode from the pools. Every step's
    output follows the values the oracle's pools hold."""
    rng = np.random.default_rng(bs)
    hq, hkv, d, B = 8, 2, 128, 3
    f_host, _ = pa.pa_rope_inv_freq(rot, scaling="linear", factor=2.0)
    f = torch.tensor(f_host, dtype=torch.float32, device="cuda")
    steps = [np.array([150, 37, 1]), np.array([30, 0, 80])] + [np.ones(B, int)] * 4
    total = sum(steps)
    tables, nb = tables_of(rng, total, bs)
    kc, ks = pools_of(rng, nb, bs, hkv, d)
    vc, vs = pools_of(rng, nb, bs, hkv, d)
    dev = [u8_dev(kc), u8_dev(vc), f32_dev(ks), f32_dev(vs)]
    ws = pa.decode_fp8_blockscale_workspace(B, hq, hkv)
    ctx = np.zeros(B, int)
    for new in steps:
        ctx = ctx + new
        cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        T = int(cu[-1])
        x = f32_to_bf16_bits((rng.standard_normal((T, hq + 2 * hkv, d)) * np.exp(rng.uniform(-1, 1, (T, 1, 1)))).astype(np.float32))
        qkv = bf16_dev(x)
        pos = np.concatenate([np.arange(c - n, c) for c, n in zip(ctx, new)]).astype(np.int32)
        q_out = torch.empty((T, hq, d), dtype=torch.bfloat16, device="cuda")
        k = qkv[:, hq:hq + hkv]
        pa.pa_rope_store_kvcache_fp8_blockscale(q_out, qkv[:, :hq], k, qkv[:, hq + hkv:], *dev, i32_dev(tables),
                                                i32_dev(cu), i32_dev(ctx), int(new.max()), i32_dev(pos), f,
                                                interleaved=inter)
        rk = torch.empty((T, hkv, d), dtype=torch.bfloat16, device="cuda")
        pa.pa_rope(rk, k, i32_dev(pos), f, interleaved=inter)
        kc, ks = fp8_block.append(kc, ks, to_bits(rk), tables, cu, ctx)
        vc, vs = fp8_block.append(vc, vs, x[:, hq + hkv:], tables, cu, ctx)
        assert np.array_equal(dev[0].cpu().numpy(), kc) and np.array_equal(dev[1].cpu().numpy(), vc)
        if (new > 0).all():
            ends = torch.from_numpy(cu[1:].astype(np.int64) - 1).cuda()
            q = q_out[ends].contiguous()
            out = torch.empty_like(q)
            pa.pa_decode_fp8_blockscale(out, q, *dev, i32_dev(tables), i32_dev(ctx), d ** -0.5, int(ctx.max()), ws)
            close(out, fp8_block.decode(to_bits(q), kc, vc, ks, vs, tables, ctx, d ** -0.5))
