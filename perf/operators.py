"""Cases, plain forms and 64-bit values of the cache and window operators.

Five operators of the decode / prefill path over a paged KV cache:

* ``append``          rotate q and k by their positions, write k and v into a bf16 paged cache
* ``append_q8``       the same into an 8-bit (e4m3) cache with one scale per (page, KV head)
* ``decode_q8``       block-sparse decode attention over an 8-bit cache (e4m3 or int8)
* ``window_decode``   one query token per sequence, sliding window plus sink tokens
* ``window_prefill``  a ragged chunk of query tokens, sliding window plus sink tokens

``own`` selects the plain form (elementary torch operations in 32 bits) or the
library's entry points.
"""
import math
import random

import torch

own = False

D = 128
DEV = "cuda"
E4M3 = torch.float8_e4m3fn


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one sequence decoding one token, one GQA group: the latency of a call
        dict(name="append_b1_g4_decode", op="append", batch=1, q_heads=4, kv_heads=1, block=64,
             past_lo=4095, past_hi=4095, new_lo=1, new_hi=1, rotary=128, interleaved=False, fused=True, kbar=False),
        # a 2 x 16K prompt from one fused projection, pooled keys for the gate on the way
        dict(name="append_b2_h40_prompt16k", op="append", batch=2, q_heads=40, kv_heads=8, block=64,
             past_lo=0, past_hi=0, new_lo=16384, new_hi=16384, rotary=128, interleaved=False, fused=True, kbar=True),
        # a ragged decode batch over an 8-bit cache: scales grow, newest blocks are pooled again
        dict(name="append_q8_b64_h64_decode", op="append_q8", batch=64, q_heads=64, kv_heads=8, block=64,
             past_lo=63, past_hi=4096, new_lo=1, new_hi=1, rotary=128, interleaved=False, fused=True, kbar=True),
        # chunked prefill of a ragged batch, half of each head rotated in pairs, pages of 128
        dict(name="append_q8_b8_h32_chunks", op="append_q8", batch=8, q_heads=32, kv_heads=8, block=128,
             past_lo=0, past_hi=2000, new_lo=77, new_hi=2501, rotary=64, interleaved=True, fused=False, kbar=True),
        # one GQA group, 4K context, a budget of 512 tokens (8 of 64 blocks)
        dict(name="decode_q8_b1_g4_L4k_budget512", op="decode_q8", batch=1, q_heads=4, kv_heads=1, block=64,
             len_lo=4096, len_hi=4096, permille=0, budget=512, cache="e4m3"),
        # 16 sequences of 32K, 90 % sparse (52 of 512 blocks): the decode benchmark's shape
        dict(name="decode_q8_b16_h40_L32k_s90", op="decode_q8", batch=16, q_heads=40, kv_heads=8, block=64,
             len_lo=32768, len_hi=32768, permille=900, budget=0, cache="e4m3"),
        # a ragged batch at 80 %, odd lengths, pages of 128, int8 codes
        dict(name="decode_q8_b64_h64_ragged_s80", op="decode_q8", batch=64, q_heads=64, kv_heads=8, block=128,
             len_lo=4097, len_hi=32749, permille=800, budget=0, cache="int8"),
        # one sequence, one GQA group, a short window: the latency of a call
        dict(name="window_decode_b1_g4_w512", op="window_decode", batch=1, q_heads=4, kv_heads=1, block=64,
             len_lo=4096, len_hi=4096, window=512, sinks=4, cache="bf16"),
        # a ragged decode batch with a 4K window
        dict(name="window_decode_b64_h64_w4k", op="window_decode", batch=64, q_heads=64, kv_heads=8, block=64,
             len_lo=511, len_hi=16384, window=4096, sinks=64, cache="bf16"),
        # a short chunk behind a context: few query rows
        dict(name="window_prefill_b1_g4_chunk77", op="window_prefill", batch=1, q_heads=4, kv_heads=1, block=64,
             past_lo=1000, past_hi=1000, new_lo=77, new_hi=77, window=256, sinks=4),
        # chunked prefill of a ragged batch behind ragged contexts
        dict(name="window_prefill_b4_h32_chunks", op="window_prefill", batch=4, q_heads=32, kv_heads=8, block=128,
             past_lo=0, past_hi=4001, new_lo=129, new_hi=2050, window=1000, sinks=130),
        # an 8K prompt at once
        dict(name="window_prefill_b1_h40_prompt8k", op="window_prefill", batch=1, q_heads=40, kv_heads=8, block=64,
             past_lo=0, past_hi=0, new_lo=8192, new_hi=8192, window=2048, sinks=4),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "append_q8", "decode_q8", "window_decode", "window_prefill"])
    kv = rng.choice([1, 2, 3, 4, 8])
    group = rng.choice([1, 2, 4, 5, 7, 8, 8, 12, 16])
    c = dict(op=op, q_heads=kv * group, kv_heads=kv, block=rng.choice([64, 128]))
    if op in ("append", "append_q8"):
        if rng.random() < 0.5:
            c.update(batch=_log(rng, 1, 128), past_lo=0, past_hi=_log(rng, 64, 4096), new_lo=1, new_hi=1)
        else:
            new = _log(rng, 2, 8192)
            c.update(batch=_log(rng, 1, max(1, min(16, 12288 // new))), past_lo=0, past_hi=_log(rng, 1, 3000),
                     new_lo=max(1, new // rng.choice([1, 2, 5])), new_hi=new)
        rotary = rng.choice([128, 128, 64, 32, 96])
        c.update(rotary=rotary, interleaved=rng.random() < 0.4, fused=rng.random() < 0.5, kbar=rng.random() < 0.6)
    elif op == "decode_q8":
        hi = _log(rng, 1, 32768)
        batch = _log(rng, 1, max(1, min(96, 230000 // (hi * kv // 8 + 1))))
        c.update(batch=batch, len_lo=max(1, hi // rng.choice([1, 2, 9])), len_hi=hi,
                 permille=rng.choice([0, 500, 800, 900, 950]), budget=rng.choice([0, 0, 1024]), cache=rng.choice(["e4m3", "int8"]))
    elif op == "window_decode":
        hi = _log(rng, 1, 16384)
        batch = _log(rng, 1, max(1, min(64, 230000 // (hi * kv // 8 + 1))))
        c.update(batch=batch, len_lo=max(1, hi // rng.choice([1, 2, 9])), len_hi=hi, window=_log(rng, 1, 8192),
                 sinks=rng.choice([0, 1, 4, 16, 100]), cache=rng.choice(["bf16", "e4m3", "int8"]))
    else:
        c["q_heads"] = kv * min(group, 8)
        new = _log(rng, 1, 4096)
        past = _log(rng, 1, 4096) - 1
        batch = _log(rng, 1, max(1, min(8, (1 << 26) // (new * (new + past) * max(1, c["q_heads"] // 8)))))
        c.update(batch=batch, past_lo=past // rng.choice([1, 3]), past_hi=past, new_lo=max(1, new // rng.choice([1, 3])), new_hi=new,
                 window=_log(rng, 1, 4096), sinks=rng.choice([0, 1, 4, 64, 100]))
    return c


def _spread(lo, hi, n):
    """n whole numbers over [lo, hi], both ends among them."""
    return [hi if n == 1 else lo + (hi - lo) * i // (n - 1) for i in range(n)]


def _sizes(case):
    """(past, new) of each sequence, as lists, in the order of size."""
    n = case["batch"]
    if "len_hi" in case:
        lens = _spread(case["len_lo"], case["len_hi"], n)
        return [x - 1 for x in lens], [1] * n
    return _spread(case["past_lo"], case["past_hi"], n), _spread(case["new_hi"], case["new_lo"], n)


def _k_of(case, length):
    nb = -(-length // case["block"])
    if case["budget"]:
        return max(1, min(nb, case["budget"] // case["block"]))
    return max(1, -(-(1000 - case["permille"]) * nb // 1000))


def _visible(length, window, sinks):
    """Tokens that the query at position length - 1 sees."""
    return min(length, window) + min(sinks, max(0, length - window))


def work(case):
    past, new = _sizes(case)
    hq, hkv, bs, op = case["q_heads"], case["kv_heads"], case["block"], case["op"]
    if op in ("append", "append_q8"):
        t = sum(new)
        kv_out = 2 * hkv * D * (2 if op == "append" else 1)
        nbytes = t * (2 * hq * D * 2 + 2 * hkv * D * 2 + kv_out) + 4 * case["rotary"] * len({p + i for p, n in zip(past, new) for i in range(n)})
        if case["kbar"]:
            blocks = sum((p + n - 1) // bs - p // bs + 1 for p, n in zip(past, new))
            nbytes += blocks * hkv * D * 4 + sum(p % bs for p in past) * hkv * D * (2 if op == "append" else 1)
        return {"bytes": nbytes, "flops": t * (hq + hkv) * case["rotary"] * 3}
    if op == "decode_q8":
        toks = sum(min(p + 1, (_k_of(case, p + 1) - 1) * bs + (p % bs + 1)) for p in past) * hkv
        return {"bytes": toks * 2 * D + 4 * toks // bs * 3 + len(past) * hq * D * 4, "flops": 4.0 * D * toks * (hq // hkv)}
    each = {"bf16": 2}.get(case.get("cache", "bf16"), 1)
    if op == "window_decode":
        toks = sum(_visible(p + 1, case["window"], case["sinks"]) for p in past)
        return {"bytes": toks * hkv * 2 * D * each + len(past) * hq * D * 4, "flops": 4.0 * D * hq * toks}
    w, s = case["window"], case["sinks"]
    pairs = sum(_visible(q + 1, w, s) for p, n in zip(past, new) for q in range(p, p + n))
    rows = sum(min(p + n, n - 1 + _visible(p + 1, w, s)) for p, n in zip(past, new))
    return {"bytes": rows * hkv * 2 * D * 2 + sum(new) * hq * D * 4, "flops": 4.0 * D * hq * pairs}


# ------------------------------------------------------------------- inputs
def _rope_table(positions, rotary):
    """[positions][rotary]: cosines, then sines, of position x 10000^(-2i / rotary), worked out in 64 bits."""
    inv = torch.pow(torch.tensor(10000.0, dtype=torch.float64, device=DEV), -torch.arange(0, rotary, 2, dtype=torch.float64, device=DEV) / rotary)
    ang = torch.arange(positions, dtype=torch.float64, device=DEV)[:, None] * inv
    return torch.cat([ang.cos(), ang.sin()], 1).float()


def _least_power(x):
    """The least power of two that is not below x > 0, from its bits; 0 for 0."""
    m, e = torch.frexp(x)
    e = torch.where(m == 0.5, e - 1, e)
    return torch.where(x > 0, ((e + 127) << 23).int().view(torch.float32), 0.0)


def _quantise(x, cache):
    """Codes and scales [P][H] of rows x [P][bs][H][D] in 32 bits: powers of two for e4m3, amax / 127 for int8."""
    amax = x.abs().amax((1, 3))
    if cache == "e4m3":
        scale = _least_power(amax / 448.0)
        return (x / scale.clamp(min=1e-30)[:, None, :, None]).to(E4M3), scale
    scale = amax / 127.0
    return torch.round(x / scale.clamp(min=1e-30)[:, None, :, None]).clamp(-127, 127).to(torch.int8), scale


def _pool(pages, case, cache, gen):
    """A pool of pages: normal rows with a spread of its own per (page, head), in bf16 or in codes and scales."""
    hkv, bs = case["kv_heads"], case["block"]
    dtype = {"bf16": torch.bfloat16, "e4m3": E4M3, "int8": torch.int8}[cache]
    pool = torch.empty((pages, bs, hkv, D), dtype=dtype, device=DEV)
    scale = None if cache == "bf16" else torch.empty((pages, hkv), dtype=torch.float32, device=DEV)
    step = max(1, (1 << 27) // (bs * hkv * D))
    for p in range(0, pages, step):
        n = min(step, pages - p)
        x = torch.randn((n, bs, hkv, D), generator=gen, device=DEV)
        x *= torch.exp(0.3 * torch.randn((n, 1, hkv, 1), generator=gen, device=DEV))
        if cache == "bf16":
            pool[p:p + n] = x
        else:
            codes, scale[p:p + n] = _quantise(x, cache)
            pool[p:p + n].view(torch.uint8).copy_(codes.view(torch.uint8))
    return pool, scale


def prepare(case, seed):
    op, hq, hkv, bs = case["op"], case["q_heads"], case["kv_heads"], case["block"]
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    past, new = _sizes(case)
    order = list(range(len(past)))
    random.Random(seed).shuffle(order)
    past, new = [past[i] for i in order], [new[i] for i in order]
    lens = [p + n for p, n in zip(past, new)]
    nb = [-(-x // bs) for x in lens]
    pages, nbmax, t = sum(nb), max(nb), sum(new)
    perm = torch.randperm(pages, generator=gen, device=DEV).int()
    table = torch.full((len(past), nbmax), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(nb):
        table[b, :n] = perm[at:at + n]
        at += n
    cache = case.get("cache", "e4m3" if op == "append_q8" else "bf16")
    s = dict(case=dict(case), past=torch.tensor(past, device=DEV), new=torch.tensor(new, device=DEV), max_new=max(new), page_table=table,
             seqlens=torch.tensor(lens, dtype=torch.int32, device=DEV), cu=torch.tensor([sum(new[:i]) for i in range(len(new) + 1)], dtype=torch.int32, device=DEV),
             seq_of=torch.repeat_interleave(torch.arange(len(new), device=DEV), torch.tensor(new, device=DEV)), pages=pages, nbmax=nbmax, nb=max(nb), cache=cache)
    s["k_pool"], s["k_scale"] = _pool(pages, case, cache, gen)
    s["v_pool"], s["v_scale"] = _pool(pages, case, cache, gen)
    s["status"] = torch.zeros(1, dtype=torch.int32, device=DEV)
    if op in ("append", "append_q8"):
        rows = torch.randn((t, (hq + 2 * hkv) * D), generator=gen, device=DEV).bfloat16()
        parts = [rows[:, :hq * D], rows[:, hq * D:(hq + hkv) * D], rows[:, (hq + hkv) * D:]]
        s["q"], s["k"], s["v"] = [(x if case["fused"] else x.contiguous()).unflatten(1, (-1, D)) for x in parts]
        s["rope"] = _rope_table(max(lens), case["rotary"])
        s["q_out"] = torch.empty((t, hq, D), dtype=torch.bfloat16, device=DEV)
        s["kbar"] = torch.zeros((len(past), hkv, nbmax, D), device=DEV) if case["kbar"] else None
        tiles = [(b, j) for b in range(len(past)) for j in range(past[b] // bs, (lens[b] - 1) // bs + 1)]
        s["tile_seq"] = torch.tensor([x[0] for x in tiles], device=DEV)
        s["tile_block"] = torch.tensor([x[1] for x in tiles], device=DEV)
    else:
        s["q"] = torch.randn((t, hq, D), generator=gen, device=DEV).bfloat16()
        s["out"] = torch.empty_like(s["q"])
        # one row of lse per query head: by sequence for a decode token, by query token for a chunk
        s["lse"] = torch.empty((t, hq) if op != "window_prefill" else (hq, t), dtype=torch.float32, device=DEV)
    if op == "decode_q8":
        ks = [_k_of(case, x) for x in lens]
        merit = torch.rand((len(past), hkv, nbmax), generator=gen, device=DEV)
        j = torch.arange(nbmax, device=DEV)
        last = torch.tensor(nb, device=DEV)[:, None, None] - 1
        merit = torch.where(j > last, -1.0, torch.where(j == last, 2.0, merit))
        idx = merit.argsort(2, descending=True)[:, :, :max(ks)]
        live = torch.arange(max(ks), device=DEV) < torch.tensor(ks, device=DEV)[:, None, None]
        idx = torch.where(live, idx, nbmax).sort(2).values
        s["idx"] = torch.where(idx < nbmax, idx, -1).int().contiguous()
        s["n_sel"] = torch.tensor(ks, dtype=torch.int32, device=DEV)[:, None].repeat(1, hkv).contiguous()
    if own:
        _handle(s)
    return s


def _handle(s):
    """The dims and argument block that a program over this cache keeps from call to call."""
    from block_sparse_attention_step_b200 import seer
    c = s["case"]
    s["seer"], op = seer, c["op"]
    s["dims"] = seer.make_dims(c["batch"], c["q_heads"], c["kv_heads"], D, c["block"], s["nbmax"], s["pages"])
    if op in ("append", "append_q8"):
        s["args"] = seer.append_args(s["k"], s["v"], s["k_pool"], s["v_pool"], s["page_table"], s["seqlens"], q=s["q"], q_out=s["q_out"], rope=s["rope"],
                                     interleaved=c["interleaved"], cu_tokens=s["cu"], max_new=s["max_new"], k_scale=s["k_scale"], v_scale=s["v_scale"],
                                     kbar=s["kbar"], dev_status=s["status"])
        return
    common = dict(k_scale=s["k_scale"], v_scale=s["v_scale"], softmax_scale=1 / math.sqrt(D), out=s["out"], lse_out=s["lse"], dev_status=s["status"])
    if op == "decode_q8":
        k_max = s["idx"].shape[2]
        splits = seer.seer_sparse_decode_q8_splits(s["dims"], k_max)
        ws = torch.empty(seer.seer_split_workspace_bytes(s["dims"], splits), dtype=torch.uint8, device=DEV)
        s["args"] = seer.sparse_decode_q8_args(s["q"], s["k_pool"], s["v_pool"], s["page_table"], s["seqlens"], s["idx"], s["n_sel"], k_max=k_max,
                                               num_splits=splits, workspace=ws, **common)
    elif op == "window_decode":
        splits = seer.seer_window_decode_splits(s["dims"], c["window"], c["sinks"])
        ws = torch.empty(seer.seer_split_workspace_bytes(s["dims"], splits), dtype=torch.uint8, device=DEV)
        s["args"] = seer.window_decode_args(s["q"], s["k_pool"], s["v_pool"], s["page_table"], s["seqlens"], window=c["window"], sinks=c["sinks"],
                                            num_splits=splits, workspace=ws, **common)
    else:
        s["args"] = seer.window_prefill_args(s["q"], s["k_pool"], s["v_pool"], s["page_table"], s["seqlens"], cu_tokens=s["cu"], max_new=s["max_new"],
                                             window=c["window"], sinks=c["sinks"], softmax_scale=1 / math.sqrt(D), out=s["out"], lse_out=s["lse"],
                                             dev_status=s["status"])


# ---------------------------------------------------------------- one pass
def run(state):
    op = state["case"]["op"]
    if own:
        call = {"append": "seer_append_rope", "append_q8": "seer_append_rope", "decode_q8": "seer_sparse_decode_q8",
                "window_decode": "seer_window_decode", "window_prefill": "seer_window_prefill"}[op]
        getattr(state["seer"], call)(state["dims"], state["args"])
    else:
        {"append": _append, "append_q8": _append_q8, "decode_q8": _decode_q8, "window_decode": _window_decode, "window_prefill": _window_prefill}[op](state)
    if op in ("append", "append_q8"):
        got = {k: state[k] for k in ("q_out", "k_pool", "v_pool", "k_scale", "v_scale", "kbar")}
        return {k: v for k, v in got.items() if v is not None}
    return {"out": state["out"], "lse": state["lse"]}


def _rotate(x, pos, s):
    """x [T][H][D] in 32 bits, its first `rotary` dims turned by the angles of pos [T]."""
    rot = s["case"]["rotary"]
    c, w = s["rope"][pos][:, None, :rot // 2], s["rope"][pos][:, None, rot // 2:]
    y = x.float().clone()
    first, second = (slice(0, rot, 2), slice(1, rot, 2)) if s["case"]["interleaved"] else (slice(0, rot // 2), slice(rot // 2, rot))
    a, b = x[..., first].float(), x[..., second].float()
    y[..., first] = a * c - b * w
    y[..., second] = b * c + a * w
    return y


def _positions(s):
    row = torch.arange(s["seq_of"].numel(), device=DEV)
    return row - s["cu"][s["seq_of"]] + s["past"][s["seq_of"]]


def _tiles(s):
    """Of each (sequence, block) that receives rows: its page, positions [N][bs], which of them are new, old, and the new rows' numbers."""
    bs = s["case"]["block"]
    b, j = s["tile_seq"], s["tile_block"]
    pos = j[:, None] * bs + torch.arange(bs, device=DEV)
    past = s["past"][b][:, None]
    new = (pos >= past) & (pos < s["seqlens"][b][:, None])
    return s["page_table"][b, j].long(), new, pos < past, torch.where(new, s["cu"][b][:, None] + pos - past, 0)


def _append(s):
    pos = _positions(s)
    bs = s["case"]["block"]
    page = s["page_table"][s["seq_of"], pos // bs].long()
    s["q_out"].copy_(_rotate(s["q"], pos, s))
    s["k_pool"][page, pos % bs] = _rotate(s["k"], pos, s).bfloat16()
    s["v_pool"][page, pos % bs] = s["v"]
    if s["kbar"] is not None:
        page, new, old, _ = _tiles(s)
        live = (new | old)[:, :, None, None]
        rows = torch.where(live, s["k_pool"][page].float(), 0.0)
        s["kbar"][s["tile_seq"], :, s["tile_block"]] = rows.sum(1) / live.sum(1)


def _scale_for(amax, old):
    """The scale of a block: that of its rows so far, doubled until the largest value fits, or the least power of two where there is none."""
    return torch.maximum(_least_power(amax / 448.0), old)


def _append_q8(s):
    pos = _positions(s)
    s["q_out"].copy_(_rotate(s["q"], pos, s))
    page, new, old, row = _tiles(s)
    new, old = new[:, :, None, None], old[:, :, None, None]
    for x, pool, scale in ((_rotate(s["k"], pos, s), s["k_pool"], s["k_scale"]), (s["v"].float(), s["v_pool"], s["v_scale"])):
        x = torch.where(new, x[row], 0.0)
        had = torch.where(old.any(1)[:, :, 0], scale[page], 0.0)
        now = _scale_for(x.abs().amax((1, 3)), had)
        inv = torch.where(now > 0, 1.0 / now, 0.0)[:, None, :, None]
        codes = pool.view(torch.uint8)[page].view(E4M3)
        kept = (codes.float() * (had[:, None, :, None] * inv)).to(E4M3)
        codes = torch.where(new, (x * inv).to(E4M3).view(torch.uint8), torch.where(old, kept.view(torch.uint8), codes.view(torch.uint8)))
        pool.view(torch.uint8)[page] = codes
        scale[page] = now
        if pool is s["k_pool"] and s["kbar"] is not None:
            rows = torch.where(new | old, codes.view(E4M3).float(), 0.0) * now[:, None, :, None]
            s["kbar"][s["tile_seq"], :, s["tile_block"]] = rows.sum(1) / (new | old).sum(1)


def _rows(s, pool, scale, page, slot, head):
    """Rows of the pool as 32-bit values: page, slot and head are broadcast indices."""
    if scale is None:
        return pool[page, slot, head].float()
    x = pool.view(torch.uint8)[page, slot, head].view(pool.dtype).float()
    return x * scale[page, head][..., None]


def _attend(s, q, k, v, seen, out, lse):
    """q [..., G, D], k and v [..., N, D], seen [..., 1, N]: out and the natural log of the sum."""
    x = torch.matmul(q, k.transpose(-1, -2)) * (1 / math.sqrt(D))
    x = torch.where(seen, x, float("-inf"))
    top = x.amax(-1, keepdim=True)
    x = torch.exp(x - torch.where(top.isinf(), 0.0, top))
    total = x.sum(-1, keepdim=True)
    out.copy_(torch.matmul(x / total, v).reshape(out.shape))
    lse.copy_((top + torch.log(total)).reshape(lse.shape))


def _decode_q8(s):
    c = s["case"]
    b, hkv, bs, kmax = c["batch"], c["kv_heads"], c["block"], s["idx"].shape[2]
    j = s["idx"].long().clamp(min=0)
    page = torch.gather(s["page_table"].long()[:, None, :].expand(b, hkv, -1), 2, j)[..., None]
    slot, head = torch.arange(bs, device=DEV), torch.arange(hkv, device=DEV)[None, :, None, None]
    pos = j[..., None] * bs + slot
    seen = (s["idx"] >= 0)[..., None] & (pos < s["seqlens"][:, None, None, None])
    k = _rows(s, s["k_pool"], s["k_scale"], page, slot, head).reshape(b, hkv, kmax * bs, D)
    v = _rows(s, s["v_pool"], s["v_scale"], page, slot, head).reshape(b, hkv, kmax * bs, D)
    _attend(s, s["q"].float().view(b, hkv, -1, D), k, v, seen.reshape(b, hkv, 1, kmax * bs), s["out"], s["lse"])


def _window_decode(s):
    c = s["case"]
    b, hkv, bs, w, n = c["batch"], c["kv_heads"], c["block"], c["window"], c["sinks"]
    length = s["seqlens"].long()[:, None]
    w = min(w, s["nb"] * bs)
    pos = torch.cat([torch.arange(n, device=DEV).expand(b, n), length - w + torch.arange(w, device=DEV)], 1)
    first = torch.arange(n + w, device=DEV) < n
    seen = (pos >= 0) & (pos < torch.where(first, (length - w).clamp(min=0), length))
    pos = torch.where(seen, pos, 0)
    page = s["page_table"].long()[torch.arange(b, device=DEV)[:, None], pos // bs][:, None]
    slot, head = (pos % bs)[:, None], torch.arange(hkv, device=DEV)[None, :, None]
    k = _rows(s, s["k_pool"], s["k_scale"], page, slot, head)
    v = _rows(s, s["v_pool"], s["v_scale"], page, slot, head)
    _attend(s, s["q"].float().view(b, hkv, -1, D), k, v, seen[:, None, None, :], s["out"], s["lse"])


def _window_prefill(s):
    c = s["case"]
    b, hkv, bs, w, n, most = c["batch"], c["kv_heads"], c["block"], c["window"], c["sinks"], s["max_new"]
    g = c["q_heads"] // hkv
    key = torch.arange(s["nb"] * bs, device=DEV)
    page = s["page_table"].long().clamp(min=0)[:, key // bs][:, None]
    slot, head = (key % bs)[None, None], torch.arange(hkv, device=DEV)[None, :, None]
    k, v = _rows(s, s["k_pool"], None, page, slot, head), _rows(s, s["v_pool"], None, page, slot, head)
    pos = s["past"][:, None] + torch.arange(most, device=DEV)
    seen = (key <= pos[..., None]) & ((key > pos[..., None] - w) | (key < n))
    at = _positions(s) - s["past"][s["seq_of"]]
    q = torch.zeros((b, most, c["q_heads"], D), device=DEV)
    q[s["seq_of"], at] = s["q"].float()
    q = q.view(b, most, hkv, g, D).permute(0, 2, 3, 1, 4)
    out, lse = torch.empty(q.shape, device=DEV), torch.empty(q.shape[:-1], device=DEV)
    _attend(s, q, k[:, :, None], v[:, :, None], seen[:, None, None], out, lse)
    s["out"].copy_(out.permute(0, 3, 1, 2, 4)[s["seq_of"], at].reshape(s["out"].shape))
    s["lse"].copy_(lse.permute(0, 3, 1, 2)[s["seq_of"], at].reshape(-1, c["q_heads"]).t())


# ------------------------------------------------------- values in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("append", "append_q8"):
        return _exact_append(s, case)
    return _exact_attention(s, case)


def _turned(x, start, s, case):
    """Rows x [n][H][D] of one sequence from position `start`, as complex numbers times their unit ones."""
    rot, y = case["rotary"], x.double().clone()
    turn = s["rope"][start:start + x.shape[0]].double()
    turn = torch.complex(turn[:, :rot // 2], turn[:, rot // 2:])[:, None]
    if case["interleaved"]:
        z = torch.view_as_complex(y[..., :rot].unflatten(-1, (-1, 2)).contiguous()) * turn
        y[..., :rot] = torch.view_as_real(z).flatten(-2)
    else:
        z = torch.complex(y[..., :rot // 2].contiguous(), y[..., rot // 2:rot].contiguous()) * turn
        y[..., :rot] = torch.cat([z.real, z.imag], -1)
    return y


def _exact_append(s, case):
    bs = case["block"]
    q8 = case["op"] == "append_q8"
    got = {"q_out": torch.zeros(s["q_out"].shape, dtype=torch.float64, device=DEV), "k_pool": s["k_pool"].double(), "v_pool": s["v_pool"].double()}
    if q8:
        got["k_scale"], got["v_scale"] = s["k_scale"].double(), s["v_scale"].double()
    if s["kbar"] is not None:
        got["kbar"] = None  # a mean of rows as they are held, in 16 or 8 bits
    cu = s["cu"].tolist()
    for b, (past, new) in enumerate(zip(s["past"].tolist(), s["new"].tolist())):
        rows = slice(cu[b], cu[b] + new)
        got["q_out"][rows] = _turned(s["q"][rows], past, s, case)
        k, v = _turned(s["k"][rows], past, s, case), s["v"][rows].double()
        for j in range(past // bs, (past + new - 1) // bs + 1):
            lo, hi = max(past, j * bs), min(past + new, (j + 1) * bs)
            page = int(s["page_table"][b, j])
            for x, name in ((k, "k"), (v, "v")):
                x = x[lo - past:hi - past]
                if not q8:
                    got[name + "_pool"][page, lo - j * bs:hi - j * bs] = x
                    continue
                had = got[name + "_scale"][page] if lo > j * bs else torch.zeros(case["kv_heads"], dtype=torch.float64, device=DEV)
                top = x.abs().amax((0, 2)) / 448
                need = torch.where(top > 0, torch.exp2(torch.ceil(torch.log2(top))), 0.0)
                now = torch.maximum(need, had)
                got[name + "_pool"][page, :lo - j * bs] *= (had / now)[:, None]
                got[name + "_pool"][page, lo - j * bs:hi - j * bs] = x / now[:, None]
                got[name + "_scale"][page] = now
    return got


def _exact_attention(s, case):
    hq, hkv, bs, op = case["q_heads"], case["kv_heads"], case["block"], case["op"]
    g = hq // hkv
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device=DEV)
    cu, lens = s["cu"].tolist(), s["seqlens"].tolist()
    for b, length in enumerate(lens):
        pages = s["page_table"][b, :-(-length // bs)].long()
        rows = slice(cu[b], cu[b + 1])
        for h in range(hkv):
            kv = []
            for pool, scale in ((s["k_pool"], s["k_scale"]), (s["v_pool"], s["v_scale"])):
                x = pool.view(torch.uint8)[pages].view(pool.dtype)[:, :, h].double()
                kv.append((x * scale[pages, h].double()[:, None, None] if scale is not None else x).flatten(0, 1)[:length])
            t = torch.arange(length, device=DEV)
            at = torch.arange(length - (cu[b + 1] - cu[b]), length, device=DEV)[:, None]
            if op == "decode_q8":
                seen = torch.isin(t // bs, s["idx"][b, h][: int(s["n_sel"][b, h])].long())[None]
            else:
                seen = (t <= at) & ((at - t < case["window"]) | (t < case["sinks"]))
            for i in range(h * g, (h + 1) * g):
                x = (s["q"][rows, i].double() @ kv[0].t()) / math.sqrt(D)
                x = x.masked_fill(~seen, float("-inf"))
                total = torch.logsumexp(x, 1)
                out[rows, i] = torch.exp(x - total[:, None]) @ kv[1]
                if op == "window_prefill":
                    lse[i, rows] = total
                else:
                    lse[rows, i] = total
    return {"out": out, "lse": lse}
