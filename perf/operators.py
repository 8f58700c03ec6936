"""Rotary positions, the block-scaled 8-bit KV cache and the attention that reads it: what is timed.

Three operators of a serving step over a paged KV cache:

  rope_store  rotate this step's queries and keys by their positions and scatter the keys and
              values into the bf16 pools (pa_rope_store_kvcache);
  append8     the same rotation with the keys and values appended to e4m3 pools that hold one
              scale for each (block, kv head) (pa_rope_store_kvcache_fp8_blockscale);
  decode8     attention of one query token per sequence over such pools
              (pa_decode_fp8_blockscale).

`run` computes them with elementary torch operations where `own` is false and calls the library
where it is true. `exact` gives the same outputs in 64 bits.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
MIN_EXP = -126  # the smallest block scale is 2**-126


# ------------------------------------------------------------------------------- cases
def _rope(name, seqs, new, ctx, heads, block, layout, rot, *, ragged=False, far=0, factor=1.0, op="rope_store"):
    return {"name": name, "op": op, "seqs": seqs, "new": new, "ragged": ragged, "ctx": ctx, "q_heads": heads[0],
            "kv_heads": heads[1], "head_dim": heads[2], "block": block, "interleaved": layout == "interleaved",
            "rot_dim": rot, "far": far, "factor": factor}


def _decode(name, seqs, lo, hi, heads, block):
    return {"name": name, "op": "decode8", "seqs": seqs, "ctx_lo": lo, "ctx_hi": hi, "q_heads": heads[0],
            "kv_heads": heads[1], "head_dim": 128, "block": block}


def listed():
    return [
        # a decode step of a small model with four requests: nothing but latency
        _rope("rope tiny step", 4, 1, 512, (8, 8, 64), 16, "interleaved", 64),
        # a decode step of a batch of 64
        _rope("rope decode step", 64, 1, 4096, (16, 8, 128), 256, "half", 128),
        # ragged chunks of requests whose oldest blocks were dropped (positions run far ahead of
        # the rows), half of the head rotated
        _rope("rope ragged far part", 37, 61, 700, (32, 8, 128), 64, "interleaved", 64, ragged=True, far=1_000_003),
        # a chunked prefill step, frequencies stretched for a longer context
        _rope("rope prefill chunk", 32, 512, 2560, (32, 8, 128), 256, "half", 128, factor=4.0),
        # the same steps into the 8-bit cache
        _rope("append8 decode step", 64, 1, 4096, (16, 8, 128), 256, "half", 128, op="append8"),
        _rope("append8 ragged part", 19, 301, 1000, (16, 8, 128), 64, "interleaved", 64, ragged=True, op="append8"),
        _rope("append8 prefill chunk", 32, 512, 2560, (32, 8, 128), 256, "half", 128, factor=4.0, op="append8"),
        # decode attention: a handful of short requests, small blocks
        _decode("decode8 tiny", 4, 1, 512, (8, 8), 16),
        # a batch of 64 with mixed contexts
        _decode("decode8 batch 64", 64, 512, 4096, (16, 8), 256),
        # many requests of very different lengths, a finished (empty) one among them
        _decode("decode8 ragged many", 256, 0, 2047, (32, 8), 64),
        # a few long contexts
        _decode("decode8 long", 8, 32768, 32768, (32, 8), 256),
        # one user, one long odd context, all query heads on one kv head
        _decode("decode8 one user", 1, 100001, 100001, (8, 1), 128),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("rope_store", "append8", "decode8", "decode8"))
    block = rng.choice((16, 32, 64, 128, 256, 512, 1024))
    if op == "decode8":
        kv = rng.choice((1, 2, 3, 4, 8))
        g = rng.choice((1, 2, 4, 8, 16) if kv < 8 else (1, 2, 4))
        hi = _spread(rng, 1, 60000)
        seqs = _spread(rng, 1, max(1, min(300, 2 * 262144 * 8 // kv // hi // 4)))
        lo = rng.choice((0, 1, hi // 3, hi))
        return {"op": op, "seqs": seqs, "ctx_lo": lo, "ctx_hi": hi, "q_heads": kv * g, "kv_heads": kv, "head_dim": 128, "block": block}
    kv = rng.choice((1, 2, 3, 4, 8))
    g = rng.choice((1, 2, 4))
    dim = rng.choice((64, 128, 128))
    new = _spread(rng, 1, 1500)
    seqs = _spread(rng, 1, max(1, min(200, 16000 // new)))
    rot = rng.choice([r for r in (16, 32, 48, 64, 96, 128) if r <= dim])
    return {"op": op, "seqs": seqs, "new": new, "ragged": rng.random() < 0.7, "ctx": new + _spread(rng, 1, 2048), "q_heads": kv * g,
            "kv_heads": kv, "head_dim": dim, "block": block, "interleaved": rng.random() < 0.5, "rot_dim": rot,
            "far": rng.choice((0, 0, _spread(rng, 10, 10_000_000))), "factor": rng.choice((1.0, 1.0, 2.0, 8.0))}


def _context_lens(case):
    """The contexts of a case's sequences, in rising order (a seed only permutes them)."""
    n = case["seqs"]
    if case["op"] == "decode8":
        lo, hi = case["ctx_lo"], case["ctx_hi"]
        return [hi - (hi - lo) * i // max(1, n - 1) for i in range(n)][::-1]
    return [case["ctx"] - (case["ctx"] - case["new"]) * i // max(1, 2 * n) for i in range(n)][::-1]


def _new_lens(case):
    n, new = case["seqs"], case["new"]
    return [1 + (new - 1) * (i + 1) // n if case["ragged"] else new for i in range(n)]


def _ceil_div(a, b):
    return -(-a // b)


# ------------------------------------------------------------------------------- inputs
def _layout(case, seed):
    """Context lengths, new tokens and block tables on shuffled physical blocks, on the host."""
    g = torch.Generator().manual_seed(seed)
    order = torch.randperm(case["seqs"], generator=g)
    ctx = torch.tensor(_context_lens(case), dtype=torch.int64)[order]
    bs = case["block"]
    blocks = (ctx + bs - 1) // bs
    used = int(blocks.sum())
    pool = max(used + 1, math.ceil(1.1 * used))
    width = max(1, int(blocks.max()))
    perm = torch.randperm(pool, generator=g)[:used]
    at = torch.arange(width)[None, :]
    first = (torch.cumsum(blocks, 0) - blocks)[:, None]
    inside = at < blocks[:, None]
    tables = torch.where(inside, torch.cat([perm, perm.new_zeros(1)])[torch.where(inside, first + at, used)], -1)
    return order, ctx, pool, tables


def _values(shape, g, dev):
    return torch.randn(shape, generator=g, device=dev)


def _quantised_pool(blocks, bs, kv, d, g, dev, channels):
    """e4m3 codes (uint8) and block scales of a pool whose blocks and channels differ in size."""
    x = _values((blocks, bs, kv, d), g, dev)
    x *= torch.exp(channels * _values((1, 1, kv, d), g, dev))
    x *= torch.exp(0.5 * _values((blocks, 1, kv, 1), g, dev))
    _, e = torch.frexp(x.abs().amax(dim=(1, 3)) / E4M3_MAX)
    scales = torch.ldexp(torch.ones((), device=dev), e)
    x /= scales[:, None, :, None]
    return x.to(torch.float8_e4m3fn).view(torch.uint8), scales


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    order, ctx, pool, tables = _layout(case, seed)
    bs, hq, kv, d = case["block"], case["q_heads"], case["kv_heads"], case["head_dim"]
    s = {"case": case, "op": case["op"], "bs": bs, "scale": 1.0 / math.sqrt(d), "max_ctx": int(ctx.max()),
         "tables": tables.to(torch.int32).to(dev), "ctx": ctx.to(torch.int32).to(dev)}
    if case["op"] == "decode8":
        s["q"] = _values((case["seqs"], hq, d), g, dev).to(torch.bfloat16)
        s["out"] = torch.empty_like(s["q"])
        s["k_codes"], s["k_scales"] = _quantised_pool(pool, bs, kv, d, g, dev, 0.3)
        s["v_codes"], s["v_scales"] = _quantised_pool(pool, bs, kv, d, g, dev, 0.1)
        return s
    new = torch.tensor(_new_lens(case), dtype=torch.int64)[order]
    new = torch.minimum(new, ctx)
    total = int(new.sum())
    cu = torch.cat([new.new_zeros(1), torch.cumsum(new, 0)])
    seq = torch.repeat_interleave(torch.arange(case["seqs"]), new)
    row = torch.arange(total) - cu[seq] + (ctx - new)[seq]
    slots = tables[seq, row // bs] * bs + row % bs
    half = case["rot_dim"] // 2
    inv = 10000.0 ** (-torch.arange(half, dtype=torch.float64) / half) / case["factor"]
    # one projection's output holds q, k and v of a token side by side
    qkv = _values((total, hq + 2 * kv, d), g, dev).to(torch.bfloat16)
    s |= {"qkv": qkv, "q": qkv[:, :hq], "k": qkv[:, hq:hq + kv], "v": qkv[:, hq + kv:],
          "q_out": torch.empty((total, hq, d), dtype=torch.bfloat16, device=dev),
          "positions": (row + case["far"]).to(torch.int32).to(dev), "slots": slots.to(torch.int32).to(dev),
          "cu": cu.to(torch.int32).to(dev), "max_new": int(new.max()), "inv_freq": inv.to(torch.float32).to(dev),
          "interleaved": case["interleaved"], "amplitude": 1.0 + 0.1 * math.log(case["factor"])}
    if case["op"] == "rope_store":
        s["k_cache"] = _values((pool, bs, kv, d), g, dev).to(torch.bfloat16)
        s["v_cache"] = _values((pool, bs, kv, d), g, dev).to(torch.bfloat16)
    else:
        s["k_codes"], s["k_scales"] = _quantised_pool(pool, bs, kv, d, g, dev, 0.1)
        s["v_codes"], s["v_scales"] = _quantised_pool(pool, bs, kv, d, g, dev, 0.1)
    return s


# ------------------------------------------------------------------------------- plain forms
def _rotate(x, positions, inv_freq, interleaved, amplitude):
    """x [T, H, D] rotated by its tokens' positions: angles in 64 bits, products in 32, rounded to bf16."""
    half = inv_freq.numel()
    angle = positions.double()[:, None] * inv_freq.double()[None, :]
    cos, sin = (amplitude * angle.cos()).float()[:, None, :], (amplitude * angle.sin()).float()[:, None, :]
    r = x[..., :2 * half].float()
    a, b = (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., :half], r[..., half:])
    y = (a * cos - b * sin, b * cos + a * sin)
    y = torch.stack(y, -1).flatten(-2) if interleaved else torch.cat(y, -1)
    return torch.cat([y.to(x.dtype), x[..., 2 * half:]], -1)


def _plain_rope_store(s):
    k = _rotate(s["k"], s["positions"], s["inv_freq"], s["interleaved"], s["amplitude"])
    s["q_out"] = _rotate(s["q"], s["positions"], s["inv_freq"], s["interleaved"], s["amplitude"])
    at = s["slots"].long()
    s["k_cache"].flatten(0, 1)[at] = k
    s["v_cache"].flatten(0, 1)[at] = s["v"]
    return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _power_scale(amax):
    """The smallest power of two (2**-126 at least) whose product with 448 is not below amax."""
    m, e = torch.frexp(amax)  # amax = m 2**e, m in [1/2, 1); 448 = 0.875 * 2**9
    e = torch.where(amax > 0, e - 9 + (m > 0.875), MIN_EXP).clamp(min=MIN_EXP)
    return torch.ldexp(torch.ones_like(amax), e)


def _append(codes, scales, x, slots, bs):
    """Rows x [T, H, D] into their blocks: scales grow to fit, and what a grown block held is requantised."""
    block = slots // bs
    kv = x.shape[1]
    blocks = codes.shape[0]
    inf = slots.new_full((blocks,), bs)
    first = inf.scatter_reduce(0, block, slots % bs, "amin")  # first new row of each block
    amax = scales.new_zeros((blocks, kv)).scatter_reduce(
        0, block[:, None].expand(-1, kv), x.float().abs().amax(-1), "amax")
    need = _power_scale(amax)
    touched = (first < bs)[:, None]
    grown = torch.where(first[:, None] == 0, need, torch.maximum(scales, need))
    now = torch.where(touched, grown, scales)
    again = torch.unique(block)
    old = codes[again].view(torch.float8_e4m3fn).float() * (scales[again] / now[again])[:, None, :, None]
    keep = torch.arange(bs, device=x.device)[None, :] < first[again][:, None]
    codes[again] = torch.where(keep[:, :, None, None], old.to(torch.float8_e4m3fn).view(torch.uint8), codes[again])
    y = (x.float() / now[block][:, :, None]).clamp(-E4M3_MAX, E4M3_MAX)
    codes.flatten(0, 1)[slots] = y.to(torch.float8_e4m3fn).view(torch.uint8)
    scales.copy_(now)


def _codes_and_scales(s):
    """The pools as the values they hold: e4m3 numbers, and the scale of each (block, kv head)."""
    return {"q": s["q_out"], "k_codes": s["k_codes"].view(torch.float8_e4m3fn), "k_scales": s["k_scales"],
            "v_codes": s["v_codes"].view(torch.float8_e4m3fn), "v_scales": s["v_scales"]}


def _plain_append(s):
    k = _rotate(s["k"], s["positions"], s["inv_freq"], s["interleaved"], s["amplitude"])
    s["q_out"] = _rotate(s["q"], s["positions"], s["inv_freq"], s["interleaved"], s["amplitude"])
    at = s["slots"].long()
    _append(s["k_codes"], s["k_scales"], k, at, s["bs"])
    _append(s["v_codes"], s["v_scales"], s["v"], at, s["bs"])
    return _codes_and_scales(s)


def _plain_decode(s):
    q, bs = s["q"], s["bs"]
    seqs, hq, d = q.shape
    kv = s["k_codes"].shape[2]
    n = s["max_ctx"]
    pos = torch.arange(n, device=q.device)
    block = s["tables"].long()[:, pos // bs].clamp(min=0)
    row = block * bs + pos % bs

    def rows(codes, scales):
        x = codes.flatten(0, 1)[row].view(torch.float8_e4m3fn).float()
        return (x * scales[block][..., None]).transpose(1, 2)  # [B, kv, n, d]

    k, v = rows(s["k_codes"], s["k_scales"]), rows(s["v_codes"], s["v_scales"])
    scores = s["scale"] * (q.float().view(seqs, kv, hq // kv, d) @ k.transpose(2, 3))
    seen = (pos[None, :] < s["ctx"][:, None])[:, None, None, :]
    scores = scores.masked_fill(~seen, -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(top > -math.inf, top, 0.0))
    total = p.sum(-1, keepdim=True)
    out = (p @ v) / torch.where(total > 0, total, 1.0)
    return out.reshape(seqs, hq, d).to(torch.bfloat16)


# ------------------------------------------------------------------------------- one pass
def run(state):
    s = state
    if not own:
        if s["op"] == "decode8":
            return _plain_decode(s)
        return _plain_rope_store(s) if s["op"] == "rope_store" else _plain_append(s)
    import paged_kv_cache_442_b200 as pa
    if s["op"] == "rope_store":
        pa.pa_rope_store_kvcache(s["q_out"], s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["slots"], s["positions"],
                                 s["inv_freq"], interleaved=s["interleaved"], amplitude=s["amplitude"])
        return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if s["op"] == "append8":
        pa.pa_rope_store_kvcache_fp8_blockscale(
            s["q_out"], s["q"], s["k"], s["v"], s["k_codes"], s["v_codes"], s["k_scales"], s["v_scales"], s["tables"], s["cu"],
            s["ctx"], s["max_new"], s["positions"], s["inv_freq"], interleaved=s["interleaved"], amplitude=s["amplitude"])
        return _codes_and_scales(s)
    if "workspace" not in s:  # a user's program makes it once for its largest batch
        s["workspace"] = pa.decode_fp8_blockscale_workspace(s["q"].shape[0], s["q"].shape[1], s["k_codes"].shape[2])
    pa.pa_decode_fp8_blockscale(s["out"], s["q"], s["k_codes"], s["v_codes"], s["k_scales"], s["v_scales"], s["tables"],
                                s["ctx"], s["scale"], s["max_ctx"], s["workspace"])
    return s["out"]


# ------------------------------------------------------------------------------- work
def work(case):
    hq, kv, d, bs = case["q_heads"], case["kv_heads"], case["head_dim"], case["block"]
    ctx = _context_lens(case)
    if case["op"] == "decode8":
        rows, blocks = sum(ctx), sum(_ceil_div(c, bs) for c in ctx)
        return {"bytes": 2 * rows * kv * d + blocks * (4 + 8 * kv) + 4 * len(ctx) + 4 * len(ctx) * hq * d, "flops": 4 * rows * hq * d}
    tokens = sum(min(n, c) for n, c in zip(_new_lens(case), ctx))
    stored = 2 if case["op"] == "rope_store" else 1
    per_token = 4 * hq * d + 2 * kv * d * (2 + stored) + 8
    return {"bytes": tokens * per_token + 2 * case["rot_dim"], "flops": tokens * (hq + kv) * case["rot_dim"] * 3}


# ------------------------------------------------------------------------------- 64 bits
def _exact_turn(x, s):
    """Each pair (a, b) as the complex number a + ib, times amplitude e^(i angle)."""
    x = x.double().clone()
    f = s["inv_freq"].double()
    h = f.numel()
    turn = torch.polar(torch.full_like(f[None] * 1.0, s["amplitude"]).expand(x.shape[0], -1).contiguous(),
                       s["positions"].double().outer(f))
    first, second = (slice(0, 2 * h, 2), slice(1, 2 * h, 2)) if s["interleaved"] else (slice(0, h), slice(h, 2 * h))
    z = torch.complex(x[..., first], x[..., second]) * turn[:, None, :]
    x[..., first], x[..., second] = z.real, z.imag
    return x


def _exact_e4m3(y):
    """Nearest e4m3 number, ties to even, in 64 bits: steps of 2**(e-3) at 2**e, of 2**-9 below 2**-6."""
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(y / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _exact_append(codes, scales, x, s):
    """Block by block of each sequence, as the definition reads."""
    bs = s["bs"]
    kv = x.shape[1]
    val = codes.view(torch.float8_e4m3fn).double()
    sc = scales.double()
    cu, ctx, tables = s["cu"].tolist(), s["ctx"].tolist(), s["tables"].tolist()
    for i in range(len(ctx)):
        t, end = cu[i], cu[i + 1]
        p = ctx[i] - (end - t)
        while t < end:
            b, r = tables[i][p // bs], p % bs
            n = min(bs - r, end - t)
            rows = x[t:t + n]
            amax = rows.abs().amax(dim=(0, 2))
            need = torch.exp2(torch.ceil(torch.log2(torch.clamp(amax / E4M3_MAX, min=2.0 ** MIN_EXP))))
            was = sc[b].clone() if r else torch.zeros(kv, dtype=torch.float64, device=x.device)
            sc[b] = torch.maximum(was, need)
            if r:
                val[b, :r] = _exact_e4m3(val[b, :r] * (was / sc[b])[None, :, None])
            val[b, r:r + n] = _exact_e4m3(rows / sc[b][None, :, None])
            t, p = t + n, p + n
    return val, sc


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "decode8":
        q = s["q"].double()
        seqs, hq, d = q.shape
        kv, bs = s["k_codes"].shape[2], s["bs"]
        out = torch.zeros((seqs, hq, d), dtype=torch.float64, device=q.device)
        for i, n in enumerate(s["ctx"].tolist()):
            if n == 0:
                continue
            blocks = s["tables"][i, :_ceil_div(n, bs)].long()
            k = (s["k_codes"][blocks].view(torch.float8_e4m3fn).double() * s["k_scales"][blocks].double()[:, None, :, None]).flatten(0, 1)[:n]
            v = (s["v_codes"][blocks].view(torch.float8_e4m3fn).double() * s["v_scales"][blocks].double()[:, None, :, None]).flatten(0, 1)[:n]
            a = torch.einsum("hgd,nhd->hgn", q[i].view(kv, hq // kv, d), k) * s["scale"]
            out[i] = torch.einsum("hgn,nhd->hgd", torch.softmax(a, -1), v).reshape(hq, d)
        return out
    q, k = _exact_turn(s["q"], s), _exact_turn(s["k"], s)
    if case["op"] == "rope_store":
        kc, vc = s["k_cache"].double(), s["v_cache"].double()
        at = s["slots"].long()
        kc.view(-1, *kc.shape[2:])[at] = k
        vc.view(-1, *vc.shape[2:])[at] = s["v"].double()
        return {"q": q, "k_cache": kc, "v_cache": vc}
    # the cache takes the rotated keys as bf16 holds them
    kval, ksc = _exact_append(s["k_codes"], s["k_scales"], k.to(torch.bfloat16).double(), s)
    vval, vsc = _exact_append(s["v_codes"], s["v_scales"], s["v"].double(), s)
    return {"q": q, "k_codes": kval, "k_scales": ksc, "v_codes": vval, "v_scales": vsc}
