"""The paged-cache operators in a row, as a server runs them: an 8-bit cache
with the gate, the selection and the decode; the rotary append feeding the
bf16 step; two streams with caches of their own."""
import math

import numpy as np
import pytest
import torch

from block_sparse_attention_step_b200 import seer
from oracle import cache_oracle as C
from oracle import seer_oracle as O

import test_gpu_cache_decode as decode
from gpu_util import MARGIN, require_gpu

D = 128
SCALE = 1 / math.sqrt(D)


def rows(T, Hq, Hkv, g):
    x = torch.randn((T, (Hq + 2 * Hkv) * D), generator=g).bfloat16().cuda()
    return [y.unflatten(1, (-1, D)) for y in x.split([Hq * D, Hkv * D, Hkv * D], 1)]


class Server:
    """A ragged batch over one paged cache."""

    def __init__(self, cache, B=3, Hq=8, Hkv=2, bs=64, blocks=16, seed=0):
        self.B, self.Hq, self.Hkv, self.bs, self.cache = B, Hq, Hkv, bs, cache
        self.g = torch.Generator().manual_seed(seed)
        pages = B * blocks + 3
        dtype = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "int8": torch.int8}[cache]
        self.kp, self.vp = [torch.zeros((pages, bs, Hkv, D), device="cuda").to(dtype) for _ in range(2)]
        self.ks = self.vs = None
        if cache != "bf16":
            self.ks, self.vs = [torch.full((pages, Hkv), float("nan"), device="cuda") for _ in range(2)]   # first rows set them
        self.table = torch.randperm(pages, generator=self.g)[:B * blocks].view(B, blocks).int().cuda()
        self.d = seer.make_dims(B, Hq, Hkv, D, bs, blocks, pages)
        self.kbar = torch.zeros((B, Hkv, blocks, D), device="cuda")
        self.rope = seer.seer_rope_table(blocks * bs, 128)
        self.w_gate = (torch.randn((Hkv, D, D), generator=self.g) / math.sqrt(D)).cuda()
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.lens, self.blocks = [0] * B, blocks

    def append(self, new):
        q, k, v = rows(sum(new), self.Hq, self.Hkv, self.g)
        self.lens = [x + n for x, n in zip(self.lens, new)]
        self.seqlens = torch.tensor(self.lens, dtype=torch.int32).cuda()
        cu = torch.tensor([sum(new[:i]) for i in range(self.B + 1)], dtype=torch.int32).cuda()
        self.q = torch.empty((sum(new), self.Hq, D), dtype=torch.bfloat16, device="cuda")
        seer.seer_append_rope(self.d, seer.append_args(k, v, self.kp, self.vp, self.table, self.seqlens, q=q, q_out=self.q, rope=self.rope, cu_tokens=cu,
                                                       max_new=max(new), k_scale=self.ks, v_scale=self.vs, kbar=self.kbar, dev_status=self.status))

    def held(self, b, h):
        """(K, V) [L][D] in fp64 as the cache holds them."""
        L = self.lens[b]
        t = np.arange(L)
        pages = self.table[b].cpu().numpy()[t // self.bs]
        out = []
        for pool, scale in ((self.kp, self.ks), (self.vp, self.vs)):
            if self.cache == "bf16":
                x = pool[:, :, h].double().cpu().numpy()
            else:
                x = pool[:, :, h].contiguous()
                x = C.e4m3_value(x.view(torch.uint8).cpu().numpy()) if self.cache == "e4m3" else x.double().cpu().numpy()
                x = x * scale[:, h].double().cpu().numpy()[:, None, None]
            out.append(x[pages, t % self.bs])
        return out


@pytest.mark.gpu
@pytest.mark.parametrize("cache", ["e4m3", "int8"])
def test_append_gate_select_and_decode_over_an_8_bit_cache(cache):
    require_gpu()
    s = Server(cache)
    s.append([400, 130, 64])
    k_max = 3
    k_per_seq = torch.full((s.B,), k_max, dtype=torch.int32, device="cuda")
    for step in range(3):
        s.append([1, 1, 1])
        scores = torch.empty((s.B, s.Hkv, s.blocks), device="cuda")
        idx = torch.empty((s.B, s.Hkv, k_max), dtype=torch.int32, device="cuda")
        n_sel = torch.empty((s.B, s.Hkv), dtype=torch.int32, device="cuda")
        out, lse = torch.empty((s.B, s.Hq, D), dtype=torch.bfloat16, device="cuda"), torch.empty((s.B, s.Hq), device="cuda")
        seer.seer_gate_scores(s.d, s.q, s.w_gate, s.kbar, s.seqlens, SCALE, scores, s.status)
        seer.seer_block_select(s.d, scores, s.seqlens, k_per_seq, True, k_max, idx, n_sel, s.status)
        splits = seer.seer_sparse_decode_q8_splits(s.d, k_max)
        a = seer.sparse_decode_q8_args(s.q, s.kp, s.vp, s.table, s.seqlens, idx, n_sel, k_scale=s.ks, v_scale=s.vs, k_max=k_max, num_splits=splits,
                                       softmax_scale=SCALE, out=out, lse_out=lse, dev_status=s.status)
        seer.seer_sparse_decode_q8(s.d, a)
        torch.cuda.synchronize()
        assert s.status.item() == 0
        got = out.double().cpu().numpy()
        for b in range(s.B):
            L = s.lens[b]
            for h in range(s.Hkv):
                K, V = s.held(b, h)
                G = s.Hq // s.Hkv
                q = s.q[b, h * G:(h + 1) * G].double().cpu().numpy()
                nb = -(-L // s.bs)
                kbar = np.stack([K[j * s.bs:(j + 1) * s.bs].mean(0) for j in range(nb)])
                # pooled keys: fp32 sums of up to 64 held rows
                assert np.abs(s.kbar[b, h, :nb].double().cpu().numpy() - kbar).max() <= 64 * 2.0 ** -24 * np.abs(K).max() + 2.0 ** -24 * np.abs(kbar).max()
                want_scores = kbar @ (s.w_gate[h].double().cpu().numpy() @ q.mean(0)) * SCALE
                merit = want_scores[:nb - 1]
                order = np.sort(merit)[::-1]
                chosen = idx[b, h, :int(n_sel[b, h])].cpu().tolist()
                if len(order) <= k_max - 1 or order[k_max - 2] - order[k_max - 1] > MARGIN:
                    assert chosen == sorted([nb - 1] + np.argsort(-merit, kind="stable")[:k_max - 1].tolist())
                seen = np.isin(np.arange(L) // s.bs, chosen)
                for i in range(G):
                    want, want_lse = C.softmax_attention(q[i], K, V, seen, SCALE)
                    # weights in f16 (2^-11), out in bf16 (2^-8)
                    w = np.exp(K[seen] @ q[i] * SCALE - want_lse)
                    tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -11 + 1e-4) * (w @ np.abs(V[seen]) + np.abs(want))
                    assert (np.abs(got[b, h * G + i] - want) <= tol).all()


@pytest.mark.gpu
def test_rotary_append_feeds_the_bf16_step():
    """Pooled keys written by the append make the step's result the same bits as its own full pooling."""
    require_gpu()
    s = Server("bf16", seed=3)
    s.append([400, 130, 64])
    s.append([1, 1, 1])
    k_max, splits = 3, 2
    outs = []
    for update, kbar in ((0, s.kbar), (2, torch.zeros_like(s.kbar))):
        ws = torch.empty(seer.seer_step_workspace_bytes(s.d, k_max, splits), dtype=torch.uint8, device="cuda")
        seer.seer_step_workspace_init(s.d, k_max, splits, ws)
        out, lse = torch.empty((s.B, s.Hq, D), dtype=torch.bfloat16, device="cuda"), torch.empty((s.B, s.Hq), device="cuda")
        a = seer.step_args(s.q, s.kp, s.vp, s.table, s.seqlens, s.w_gate, kbar, torch.full((s.B,), k_max, dtype=torch.int32, device="cuda"), update_kbar=update,
                           force_newest=True, k_max=k_max, num_splits=splits, gate_scale=SCALE, softmax_scale=SCALE, workspace=ws, out=out, lse_out=lse,
                           dev_status=s.status)
        seer.seer_decode_step(s.d, a)
        outs.append((out, lse))
    torch.cuda.synchronize()
    assert s.status.item() == 0
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])


@pytest.mark.gpu
def test_calls_that_follow_each_other_at_once():
    """Append and decode of one cache and prefill of another, 40 rounds enqueued without a wait: every call sees what
    the one before it wrote (the launches overlap their starts)."""
    require_gpu()
    s = Server("e4m3", B=2, Hq=8, Hkv=2, seed=5, blocks=8)
    s.append([64, 100])
    base = s.lens
    outs, steps = [], 40
    out = [torch.empty((s.B, s.Hq, D), dtype=torch.bfloat16, device="cuda") for _ in range(steps)]
    args, keep = [], []
    for i in range(steps):
        q, k, v = rows(2, s.Hq, s.Hkv, s.g)
        lens = torch.tensor([x + i + 1 for x in base], dtype=torch.int32).cuda()
        qr = torch.empty((2, s.Hq, D), dtype=torch.bfloat16, device="cuda")
        args.append((seer.append_args(k, v, s.kp, s.vp, s.table, lens, q=q, q_out=qr, rope=s.rope, k_scale=s.ks, v_scale=s.vs, kbar=s.kbar, dev_status=s.status),
                     seer.window_decode_args(qr, s.kp, s.vp, s.table, lens, window=90, sinks=4, num_splits=2, softmax_scale=SCALE, out=out[i], k_scale=s.ks,
                                             v_scale=s.vs, dev_status=s.status)))
        keep.append(qr)
    pools = [x.clone() for x in (s.kp.view(torch.uint8), s.vp.view(torch.uint8), s.ks, s.vs)]
    torch.cuda.synchronize()
    for a, w in args:                                   # at once
        seer.seer_append_rope(s.d, a)
        seer.seer_window_decode(s.d, w)
    torch.cuda.synchronize()
    first = [x.clone() for x in out]
    for x, y in zip((s.kp.view(torch.uint8), s.vp.view(torch.uint8), s.ks, s.vs), pools):
        x.copy_(y)
    for a, w in args:                                   # one by one
        seer.seer_append_rope(s.d, a)
        torch.cuda.synchronize()
        seer.seer_window_decode(s.d, w)
        torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(first, out)) and s.status.item() == 0


@pytest.mark.gpu
def test_two_streams_with_their_own_caches():
    require_gpu()
    servers = [Server("int8", seed=i) for i in (7, 8)]
    for s in servers:
        s.append([300, 70, 1])
    torch.cuda.synchronize()
    outs = []
    for at_once in (True, False):
        got = []
        for s in servers:
            out = torch.zeros((s.B, s.Hq, D), dtype=torch.bfloat16, device="cuda")
            q = s.q[[s.lens[0] - 1, s.lens[0] + s.lens[1] - 1, sum(s.lens) - 1]].contiguous()
            a = seer.window_decode_args(q, s.kp, s.vp, s.table, s.seqlens, window=250, sinks=2, num_splits=4, softmax_scale=SCALE, out=out, k_scale=s.ks, v_scale=s.vs)
            got.append((s, a, out))
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream(), torch.cuda.Stream()] if at_once else [None, None]
        for _ in range(10):
            for (s, a, out), st in zip(got, streams):
                seer.seer_window_decode(s.d, a, st)
        torch.cuda.synchronize()
        outs.append([x[2] for x in got])
    for x, y in zip(*outs):
        assert torch.equal(x, y)


@pytest.mark.gpu
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_append_prefill_and_decode_far_into_a_pool(cache):
    """Pages behind 2^32 elements and rows 2^27 elements apart give the bits of near ones (bf16: append, prefill and
    decode; e4m3: append with pooled keys and decode)."""
    require_gpu()
    T, Hq, Hkv, bs, blocks = 40, 4, 1, 64, 2
    far = (1 << 32) // (bs * Hkv * D) + 5
    g = torch.Generator().manual_seed(21)
    packed = torch.randn((T, (Hq + 2 * Hkv) * D), generator=g).bfloat16().cuda()
    apart = torch.empty((T, 1 << 27), dtype=torch.bfloat16, device="cuda")
    apart[:, :packed.shape[1]] = packed
    dtype = torch.bfloat16 if cache == "bf16" else torch.float8_e4m3fn
    cu, lens = torch.tensor([0, T], dtype=torch.int32).cuda(), torch.tensor([T + 30], dtype=torch.int32).cuda()
    rope = seer.seer_rope_table(bs * blocks, 128)
    got = []
    for pages, table, x in ((4, [1, 2], packed), (far, [far - 1, far - 3], apart[:, :packed.shape[1]])):
        q, k, v = [y.unflatten(1, (-1, D)) for y in x.split([Hq * D, Hkv * D, Hkv * D], 1)]
        kp, vp = [torch.zeros((pages, bs, Hkv, D), dtype=torch.uint8 if cache == "e4m3" else dtype, device="cuda").view(dtype) for _ in range(2)]
        ks = vs = None
        if cache == "e4m3":
            ks, vs = torch.zeros((pages, Hkv), device="cuda"), torch.zeros((pages, Hkv), device="cuda")
        d = seer.make_dims(1, Hq, Hkv, D, bs, blocks, pages)
        tab = torch.tensor([table], dtype=torch.int32).cuda()
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        qr, kbar = torch.empty((T, Hq, D), dtype=torch.bfloat16, device="cuda"), torch.zeros((1, Hkv, blocks, D), device="cuda")
        seer.seer_append_rope(d, seer.append_args(k, v, kp, vp, tab, lens, q=q, q_out=qr, rope=rope, cu_tokens=cu, max_new=T, k_scale=ks, v_scale=vs,
                                                  kbar=kbar if cache == "e4m3" else None, dev_status=status))
        res = [qr, kbar] + [p.view(torch.uint8 if cache == "e4m3" else torch.int16)[table] for p in (kp, vp)]
        if cache == "bf16":
            out, lse = torch.zeros_like(qr), torch.zeros((Hq, T), device="cuda")
            seer.seer_window_prefill(d, seer.window_prefill_args(qr, kp, vp, tab, lens, window=25, sinks=2, softmax_scale=SCALE, out=out, cu_tokens=cu, max_new=T,
                                                                 lse_out=lse, dev_status=status))
            res += [out, lse]
        one = torch.zeros((1, Hq, D), dtype=torch.bfloat16, device="cuda")
        seer.seer_window_decode(d, seer.window_decode_args(qr[-1:].contiguous(), kp, vp, tab, lens, window=60, sinks=1, num_splits=2, softmax_scale=SCALE,
                                                           out=one, k_scale=ks, v_scale=vs, dev_status=status))
        got.append(res + [one, status])
        torch.cuda.synchronize()
        del kp, vp
    for a, b in zip(*got):
        assert torch.equal(a, b)
    assert got[0][-1].item() == 0 and got[0][-2].abs().max() > 0


@pytest.mark.gpu
@pytest.mark.parametrize("cache", ["e4m3", "int8"])
@pytest.mark.parametrize("sizes", [(1e-36,), (1e-30, 1.0), (1e33,), (1.0, 1e-36, 1e30, 0.0), (1e-30, 0.0)])
def test_decodes_read_whatever_scales_the_append_writes(cache, sizes):
    """Values from 1e-36 to 1e33, block by block, through the append and both decodes: out and lse against fp64 over the
    cache as it is held, and nothing flagged."""
    require_gpu()
    Hq, Hkv, bs, blocks, L = 8, 2, 64, 8, 64 * 7 + 5
    g = torch.Generator().manual_seed(31)
    q, k, v = rows(L, Hq, Hkv, g)
    v = (v.float() * torch.tensor([sizes[t // bs % len(sizes)] for t in range(L)], device="cuda")[:, None, None]).bfloat16()
    dtype = torch.float8_e4m3fn if cache == "e4m3" else torch.int8
    kp, vp = [torch.zeros((blocks + 2, bs, Hkv, D), device="cuda").to(dtype) for _ in range(2)]
    ks, vs = [torch.full((blocks + 2, Hkv), float("nan"), device="cuda") for _ in range(2)]
    table = torch.randperm(blocks + 2, generator=g)[:blocks].int()[None]
    d = seer.make_dims(1, Hq, Hkv, D, bs, blocks, blocks + 2)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    seer.seer_append_rope(d, seer.append_args(k, v, kp, vp, table.cuda(), torch.tensor([L], dtype=torch.int32).cuda(),
                                              cu_tokens=torch.tensor([0, L], dtype=torch.int32).cuda(), max_new=L, k_scale=ks, v_scale=vs, dev_status=status))
    torch.cuda.synchronize()
    assert status.item() == 0
    c = {"k": kp.cpu(), "v": vp.cpu(), "ks": ks.cpu(), "vs": vs.cpu(), "cache": cache, "layout": "nhd", "bs": bs, "lens": [L], "Hkv": Hkv, "table": table,
         "nbmax": blocks, "pages": blocks + 2, "nb": [blocks]}
    one = q[-1:].contiguous()
    for splits in (1, 3, 16):
        chosen = [[[0, 1, 2, 5, 7], list(range(blocks))]]
        seen = [[np.isin(np.arange(L) // bs, x) for x in chosen[0]]]
        out, lse = decode.run_list(c, one, chosen, splits)
        decode.check_far(c, one, seen, out, lse, splits)
        out, lse, _ = decode.run_window(c, one, 300, 40, splits)
        decode.check_far(c, one, [[C.window_seen(L - 1, L, 300, 40)] * Hkv], out, lse, splits)


@pytest.mark.gpu
def test_calls_whose_tensors_are_too_small_launch_nothing():
    require_gpu()
    s = Server("bf16", seed=9)
    s.append([70, 3, 64])
    k, v, table = s.kp.clone(), s.vp.clone(), s.table[:, :-1].contiguous()
    q, new_k, new_v = rows(3, s.Hq, s.Hkv, s.g)
    out = torch.full((s.B, s.Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match="page_table"):
        seer.seer_append_rope(s.d, seer.append_args(new_k, new_v, s.kp, s.vp, table, s.seqlens))
    with pytest.raises(ValueError, match="positions"):
        seer.seer_append_rope(s.d, seer.append_args(new_k, new_v, s.kp, s.vp, s.table, s.seqlens, rope=s.rope, positions=s.seqlens[:2]))
    with pytest.raises(ValueError, match="seqlens"):
        seer.seer_window_decode(s.d, seer.window_decode_args(q.contiguous(), s.kp, s.vp, s.table, s.seqlens[:2], window=9, sinks=0, num_splits=1, softmax_scale=SCALE,
                                                             out=out))
    with pytest.raises(ValueError, match="lse_out"):
        seer.seer_window_prefill(s.d, seer.window_prefill_args(q.contiguous(), s.kp, s.vp, s.table, s.seqlens, window=9, sinks=0, softmax_scale=SCALE, out=out,
                                                               lse_out=torch.zeros(2, device="cuda")))
    torch.cuda.synchronize()
    assert torch.equal(k, s.kp) and torch.equal(v, s.vp) and (out == 7).all() and s.status.item() == 0


@pytest.mark.gpu
def test_append_prefill_append_and_decode_without_a_wait():
    """A chunk's append and prefill, single tokens' append and decode, and prefills and decodes one behind the other over
    one bf16 cache, 20 rounds enqueued at once: rotated queries, outputs, lse, pooled keys and pages have the bits that
    they have with a wait after every call.  (The prefill lets its successor start before its own predecessor has ended.)"""
    require_gpu()
    s = Server("bf16", B=2, Hq=8, Hkv=2, seed=15)
    s.append([64, 100])
    lens, calls, held = list(s.lens), [], []

    def empty(*shape, dtype=torch.float32):
        held.append(torch.empty(shape, dtype=dtype, device="cuda"))
        return held[-1]

    for i in range(20):
        for new in ([3 + 5 * (i % 4), 1 + i % 3], [1, 1]):
            T = sum(new)
            lens = [x + n for x, n in zip(lens, new)]
            seqlens = torch.tensor(lens, dtype=torch.int32).cuda()
            cu = torch.tensor([0, new[0], T], dtype=torch.int32).cuda()
            q, k, v = rows(T, s.Hq, s.Hkv, s.g)
            qr = empty(T, s.Hq, D, dtype=torch.bfloat16)
            a = seer.append_args(k, v, s.kp, s.vp, s.table, seqlens, q=q, q_out=qr, rope=s.rope, cu_tokens=cu, max_new=max(new),
                                 kbar=s.kbar if i % 2 else None, dev_status=s.status)
            pre = [seer.window_prefill_args(qr, s.kp, s.vp, s.table, seqlens, cu_tokens=cu, max_new=max(new), window=w, sinks=4, softmax_scale=SCALE,
                                            out=empty(T, s.Hq, D, dtype=torch.bfloat16), lse_out=empty(s.Hq, T), dev_status=s.status) for w in (90, 300)]
            calls.append((seer.seer_append_rope, a))
            if new == [1, 1]:
                w = seer.window_decode_args(qr, s.kp, s.vp, s.table, seqlens, window=90, sinks=4, num_splits=1 + i % 3, softmax_scale=SCALE,
                                            out=empty(2, s.Hq, D, dtype=torch.bfloat16), lse_out=empty(2, s.Hq), dev_status=s.status)
                calls += [(seer.seer_window_decode, w), (seer.seer_window_prefill, pre[0])][:: 1 if i % 2 else -1]
            else:
                calls += [(seer.seer_window_prefill, x) for x in pre[: 1 + i % 2]]
    written = [s.kp, s.vp, s.kbar] + held
    start = [x.clone() for x in written]
    torch.cuda.synchronize()
    for fn, a in calls:                                 # at once
        fn(s.d, a)
    torch.cuda.synchronize()
    first = [x.clone() for x in written]
    for x, y in zip(written, start):
        x.copy_(y)
    for fn, a in calls:                                 # one by one
        fn(s.d, a)
        torch.cuda.synchronize()
    assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(first, written)) and s.status.item() == 0
    assert any(not torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(first, start))
