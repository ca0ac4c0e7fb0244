"""seer_window_prefill against softmax attention in fp64: ragged chunks behind
contexts, head groups, windows and sinks around the tile edges, pages that are
gone, rows that must stay as they were; and the append, prefill and decode
operators in a row over one cache."""
import math

import numpy as np
import pytest
import torch

from block_sparse_attention_step_b200 import seer
from oracle import cache_oracle as C

from gpu_util import require_gpu
from test_gpu_cache_decode import make_cache, on_gpu, poison, values

D = 128
SCALE = 1 / math.sqrt(D)


def run(c, past, new, Hq, window, sinks, seed=0, softmax_scale=SCALE, spread=1.0, drop_pages=False, expect_status=0, with_cu=True):
    B, bs, Hkv = len(past), c["bs"], c["Hkv"]
    g = torch.Generator().manual_seed(seed + 7)
    T = sum(new) + (5 if with_cu else 0)
    q = (torch.randn((T, Hq, D), generator=g) * spread).bfloat16().cuda()
    cu = torch.tensor([sum(new[:i]) for i in range(B + 1)], dtype=torch.int32).cuda()
    table = c["table"].clone()
    if drop_pages:                                       # blocks that no query sees
        for b in range(B):
            for j in range(c["nb"][b]):
                t = np.arange(j * bs, min((j + 1) * bs, past[b] + new[b]))
                if not any(C.window_seen(p, past[b] + new[b], window, sinks)[t].any() for p in range(past[b], past[b] + new[b])):
                    table[b, j] = -1
    d = seer.make_dims(B, Hq, Hkv, D, bs, c["nbmax"], c["pages"])
    if c["layout"] == "hnd":
        d.stride_page, d.stride_head, d.stride_token = Hkv * bs * D, bs * D, D
    out = torch.full((T, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((Hq, T), 7.0, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    a = seer.window_prefill_args(q, on_gpu(c, "k"), on_gpu(c, "v"), table.cuda(), torch.tensor(c["lens"], dtype=torch.int32).cuda(),
                                 cu_tokens=cu if with_cu else None, max_new=max(new + [1]), window=window, sinks=sinks, softmax_scale=softmax_scale, out=out,
                                 lse_out=lse, dev_status=status)
    seer.seer_window_prefill(d, a)
    torch.cuda.synchronize()
    assert status.item() == expect_status
    return q, out, lse, (d, a)


def check(c, past, new, q, out, lse, window, sinks, softmax_scale=SCALE, seqs=None):
    """A weight is rounded to bf16 (2^-8) after its fp32 score (128 half-steps of sum |q k|) and exp2 (2^-21);
    out adds its own bf16 rounding.  Rows of no sequence keep their 7."""
    K, V = values(c, "k"), values(c, "v")
    qd, got, gl = q.double().cpu().numpy(), out.double().cpu().numpy(), lse.double().cpu().numpy()
    Hq, Hkv, bs = q.shape[1], c["Hkv"], c["bs"]
    G, row = Hq // Hkv, 0
    for b in range(len(past)):
        L = past[b] + new[b]
        if seqs is not None and b not in seqs:
            assert (got[row:row + new[b]] == 7).all()
            row += new[b]
            continue
        t = np.arange(L)
        pages = c["table"][b].numpy()[t // bs]
        for h in range(Hkv):
            k, v = K[pages, t % bs, h], V[pages, t % bs, h]
            seen = np.stack([C.window_seen(p, L, window, sinks) for p in range(past[b], L)]) if new[b] else np.zeros((0, L), bool)
            vis = seen.any(0)
            k, v, seen = k[vis], v[vis], seen[:, vis]
            for i in range(h * G, (h + 1) * G):
                x = qd[row:row + new[b], i] @ k.T * softmax_scale
                size = (np.abs(qd[row:row + new[b], i]) @ np.abs(k).T).max(1, initial=0) * softmax_scale
                x = np.where(seen, x, -np.inf)
                top = x.max(1, initial=-np.inf)
                w = np.exp(x - top[:, None])
                total = w.sum(1)
                want = (w @ v) / total[:, None]
                spread = (w @ np.abs(v)) / total[:, None]
                want_lse = top + np.log(total)
                dx = (128 * 2.0 ** -24 * size + 2.0 ** -21)[:, None]
                tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -8 + 2 * dx) * (spread + np.abs(want))
                err = np.abs(got[row:row + new[b], i] - want)
                assert (err <= tol).all(), (b, i, np.argwhere(err > tol)[:5], err.max())
                assert (np.abs(gl[i, row:row + new[b]] - want_lse) <= 2 * dx[:, 0] + 4 * 2.0 ** -24 * np.abs(want_lse)).all(), (b, i)
        row += new[b]
    assert (got[row:] == 7).all() and (gl[:, row:] == 7).all()


def seen_of(c, past, new, window, sinks):
    out = []
    for p, n in zip(past, new):
        s = np.zeros(p + n, dtype=bool)
        for pos in range(p, p + n):
            s |= C.window_seen(pos, p + n, window, sinks)
        out.append([s] * c["Hkv"])
    return out


@pytest.mark.gpu
@pytest.mark.parametrize("G,Hkv", [(1, 2), (2, 1), (3, 2), (4, 1), (5, 2), (7, 1), (8, 2), (16, 1)])
def test_groups(G, Hkv):
    require_gpu()
    past, new = [0, 100, 513], [70, 1, 131]
    c = make_cache([p + n for p, n in zip(past, new)], Hkv, 64, "bf16", seed=G)
    poison(c, seen_of(c, past, new, 90, 5))
    q, out, lse, _ = run(c, past, new, G * Hkv, 90, 5, seed=G)
    check(c, past, new, q, out, lse, 90, 5)


@pytest.mark.gpu
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 3), (64, 0), (127, 128), (128, 129), (129, 1), (1000, 0), (5000, 64), (300, 300), (40, 5000), (2 ** 31 - 1, 2 ** 31 - 1)])
@pytest.mark.parametrize("bs,layout", [(64, "nhd"), (128, "hnd")])
def test_windows_and_sinks(window, sinks, bs, layout):
    require_gpu()
    past, new = [0, 700, 63, 0], [300, 65, 1, 0]
    c = make_cache([p + n for p, n in zip(past, new)], 1, bs, "bf16", layout, seed=(window + sinks) % 1000)
    poison(c, seen_of(c, past, new, window, sinks))
    q, out, lse, _ = run(c, past, new, 4, window, sinks, seed=window % 1000, drop_pages=True)
    check(c, past, new, q, out, lse, window, sinks)


@pytest.mark.gpu
def test_single_tokens_match_the_decode_operator():
    """One token per sequence, with and without offsets; the decode form sees the same tokens."""
    require_gpu()
    lens = [1, 64, 500, 777]
    past, new = [x - 1 for x in lens], [1] * 4
    c = make_cache(lens, 2, 64, "bf16", seed=3)
    for with_cu in (True, False):
        q, out, lse, (d, a) = run(c, past, new, 8, 200, 3, seed=3, with_cu=with_cu)
        check(c, past, new, q, out, lse, 200, 3)
    dec, dlse = torch.empty_like(out), torch.empty((4, 8), device="cuda")
    w = seer.window_decode_args(q, on_gpu(c, "k"), on_gpu(c, "v"), c["table"].cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), window=200, sinks=3,
                                num_splits=2, softmax_scale=SCALE, out=dec, lse_out=dlse)
    seer.seer_window_decode(d, w)
    torch.cuda.synchronize()
    assert (dec.float() - out.float()).abs().max() <= 3 * 2.0 ** -8 * out.float().abs().max()   # two bf16 roundings and bf16 weights
    assert (dlse.t() - lse).abs().max() <= 1e-4


@pytest.mark.gpu
def test_scores_that_climb():
    """Scores that climb by hundreds along the keys: the reference moves and O is rescaled, over many tiles."""
    require_gpu()
    L = 1500
    c = make_cache([L], 1, 64, "bf16", seed=5)
    ramp = torch.linspace(-2, 12, L)
    for t in range(L):
        c["k"][c["table"][0, t // 64], t % 64, 0] = ramp[t].bfloat16() + 0.05 * c["k"][c["table"][0, t // 64], t % 64, 0]
    q, out, lse, (d, a) = run(c, [L - 200], [200], 4, 1400, 10, seed=5)
    check(c, [L - 200], [200], q, out, lse, 1400, 10)
    one = torch.ones_like(q)
    q.copy_(one)
    seer.seer_window_prefill(d, a)
    torch.cuda.synchronize()
    check(c, [L - 200], [200], q, out, lse, 1400, 10)


@pytest.mark.gpu
def test_scales_and_magnitudes():
    require_gpu()
    c = make_cache([400], 1, 128, "bf16", seed=6)
    for scale, spread in ((1.0, 1.0), (1e-3, 1.0), (SCALE, 100.0)):
        q, out, lse, _ = run(c, [150], [250], 2, 333, 0, seed=6, softmax_scale=scale, spread=spread)
        check(c, [150], [250], q, out, lse, 333, 0, scale)


@pytest.mark.gpu
def test_many_sequences_and_repeatability():
    """More sequences than a warp scans at once, many of them empty; the same bits again."""
    require_gpu()
    rng = np.random.default_rng(0)
    new = [int(x) for x in rng.choice([0, 0, 1, 2, 30, 65], 70)]
    past = [int(x) if n else 0 for x, n in zip(rng.integers(0, 200, 70), new)]
    c = make_cache([p + n for p, n in zip(past, new)], 1, 64, "bf16", seed=8)
    q, out, lse, (d, a) = run(c, past, new, 4, 100, 2, seed=8)
    check(c, past, new, q, out, lse, 100, 2)
    first = out.clone()
    for _ in range(3):
        seer.seer_window_prefill(d, a)
        assert torch.equal(first, out)


@pytest.mark.gpu
def test_long_chunk_gives_the_same_bits_every_time():
    """Some 600 CTAs of 20 and more key tiles, 30 times over: no warp's lead over another shows in a result."""
    require_gpu()
    g = torch.Generator(device="cuda").manual_seed(12)
    L, Hq, Hkv, bs = 2048, 20, 4, 64
    kp, vp = [torch.randn((L // bs, bs, Hkv, D), generator=g, device="cuda").bfloat16() for _ in range(2)]
    q = torch.randn((L, Hq, D), generator=g, device="cuda").bfloat16()
    d = seer.make_dims(1, Hq, Hkv, D, bs, L // bs, L // bs)
    out, lse, status = torch.empty_like(q), torch.empty((Hq, L), device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    a = seer.window_prefill_args(q, kp, vp, None, torch.tensor([L], dtype=torch.int32, device="cuda"), cu_tokens=torch.tensor([0, L], dtype=torch.int32, device="cuda"),
                                 max_new=L, window=1300, sinks=4, softmax_scale=SCALE, out=out, lse_out=lse, dev_status=status)
    seer.seer_window_prefill(d, a)
    first, first_lse = out.clone(), lse.clone()
    for _ in range(30):
        out.zero_()
        lse.zero_()
        seer.seer_window_prefill(d, a)
        assert torch.equal(first, out) and torch.equal(first_lse, lse)
    assert status.item() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("window,sinks,bs", [(70, 3, 64), (9, 0, 128), (400, 130, 64)])
def test_odd_values_reach_only_the_queries_that_see_them(window, sinks, bs):
    """NaN and infinities in keys and values of tokens ahead of some queries, behind the window of others, and in a sink."""
    require_gpu()
    past, new, L = 200, 90, 290
    c = make_cache([L], 1, bs, "bf16", seed=window)
    g = torch.Generator().manual_seed(window)
    for t, d, x in ((289, 5, math.nan), (250, 100, math.inf), (215, 3, -math.inf), (201, 64, math.nan), (200 - window + 40, 7, math.inf), (200 - window + 5, 127, math.nan)):
        c["v"][c["table"][0, t // bs], t % bs, 0, d] = x
    c["v"][c["table"][0, 270 // bs], 270 % bs, 0] = math.nan
    c["k"][c["table"][0, 275 // bs], 275 % bs, 0, 3] = math.nan
    q, out, lse, _ = run(c, [past], [new], 5, window, sinks, seed=window)
    K, V = values(c, "k"), values(c, "v")
    t = np.arange(L)
    pages = c["table"][0].numpy()[t // bs]
    k, v = K[pages, t % bs, 0], V[pages, t % bs, 0]
    got, qd, gl = out.double().cpu().numpy(), q.double().cpu().numpy(), lse.double().cpu().numpy()
    for i in range(new):
        seen = C.window_seen(past + i, L, window, sinks)
        for h in range(5):
            with np.errstate(invalid="ignore"):
                want, want_lse = C.softmax_attention(qd[i, h], k, v, seen, SCALE)
            assert np.array_equal(np.isnan(got[i, h]), np.isnan(want)), (i, h)
            assert np.array_equal(np.isposinf(got[i, h]), np.isposinf(want)) and np.array_equal(np.isneginf(got[i, h]), np.isneginf(want))
            fine = np.isfinite(want)
            if fine.any():
                w = np.exp(k[seen] @ qd[i, h] * SCALE - want_lse)
                spread = w @ np.abs(np.where(np.isfinite(v[seen]), v[seen], 0))
                a, b = got[i, h][fine], want[fine]
                assert (np.abs(a - b) <= 2.0 ** -8 * np.abs(b) + (2.0 ** -8 + 1e-4) * (spread[fine] + np.abs(b))).all()
            assert np.isnan(gl[h, i]) == np.isnan(want_lse)


@pytest.mark.gpu
@pytest.mark.parametrize("Hkv", [4, 12, 30, 80])
@pytest.mark.parametrize("window,sinks", [(600, 70), (200, 0)])
def test_keys_shared_by_the_ctas_of_a_cluster(Hkv, window, sinks):
    """Few row tiles: their keys are split over 8, 4 or 2 CTAs; many: one CTA each.  Some pieces hold keys
    that only some rows see, some none at all (the sequence of one token and its neighbours)."""
    require_gpu()
    past, new = [700, 0, 63], [40, 130, 1]
    c = make_cache([p + n for p, n in zip(past, new)], Hkv, 64, "bf16", seed=Hkv)
    poison(c, seen_of(c, past, new, window, sinks))
    q, out, lse, (d, a) = run(c, past, new, Hkv, window, sinks, seed=Hkv, drop_pages=True)
    check(c, past, new, q, out, lse, window, sinks)


@pytest.mark.gpu
@pytest.mark.parametrize("window,sinks,bs", [(70, 3, 64), (9, 0, 128), (400, 130, 64)])
def test_odd_values_in_one_piece_and_in_many(window, sinks, bs):
    """The same keys, values and queries as one KV head (keys split over a cluster) and as 100 of them (one CTA for
    each row tile): NaN and inf in the same places, the rest within both roundings."""
    require_gpu()
    past, new, L = 200, 90, 290
    c = make_cache([L], 1, bs, "bf16", seed=window)
    for t, d, x in ((289, 5, math.nan), (250, 100, math.inf), (215, 3, -math.inf), (200 - window + 40, 7, math.inf), (200 - window + 5, 127, math.nan)):
        c["v"][c["table"][0, t // bs], t % bs, 0, d] = x
    c["v"][c["table"][0, 270 // bs], 270 % bs, 0] = math.nan
    q, few, few_lse, (d, _) = run(c, [past], [new], 5, window, sinks, seed=window)
    H, T = 100, q.shape[0]
    d.num_kv_heads, d.num_q_heads = H, 5 * H
    d.stride_page, d.stride_token, d.stride_head = bs * H * D, H * D, D
    kp, vp = [on_gpu(c, x).repeat(1, 1, H, 1).contiguous() for x in "kv"]
    qq = q.repeat(1, H, 1).contiguous()
    out, lse = torch.empty_like(qq), torch.empty((5 * H, T), device="cuda")
    cu = torch.tensor([0, new], dtype=torch.int32).cuda()
    seer.seer_window_prefill(d, seer.window_prefill_args(qq, kp, vp, c["table"].cuda(), torch.tensor([L], dtype=torch.int32).cuda(), cu_tokens=cu, max_new=new,
                                                         window=window, sinks=sinks, softmax_scale=SCALE, out=out, lse_out=lse))
    a, b = few[:new].float(), out[:new].float()
    for h in range(0, 5 * H, 5):
        x = b[:, h:h + 5]
        assert torch.equal(x.isnan(), a.isnan()) and torch.equal(x.isposinf(), a.isposinf()) and torch.equal(x.isneginf(), a.isneginf())
        assert torch.equal(x, b[:, :5]) or torch.equal(x.nan_to_num(9.0), b[:, :5].nan_to_num(9.0))
    fine = a.isfinite()
    # both round their weights and outputs to bf16: 2 (2^-8 + 2^-8) of the largest value
    assert (a - b[:, :5])[fine].abs().max() <= 4 * 2.0 ** -8 * vp.float()[vp.isfinite()].abs().max()
    assert (few_lse[:, :new] - lse[:5, :new]).abs().max() <= 1e-4


@pytest.mark.gpu
def test_sequences_that_do_not_fit_are_left_out():
    require_gpu()
    past, new = [10, 0, 70], [9, 20, 3]
    c = make_cache([p + n for p, n in zip(past, new)], 1, 64, "bf16", seed=9)
    c["lens"] = [19, 15, 73]                              # sequence 1: 20 new tokens, length 15
    q, out, lse, _ = run(c, past, new, 2, 50, 0, seed=9, expect_status=seer.DEV_BAD_TOKENS)
    got = out.float().cpu()
    assert (got[9:29] == 7).all() and (got[:9] != 7).any() and (got[29:32] != 7).any() and (got[32:] == 7).all()
    c["lens"] = [19, 20, 73]
    c["table"][2, 1] = 10 ** 6
    run(c, past, new, 2, 50, 0, seed=9, expect_status=seer.DEV_BAD_PAGE)


@pytest.mark.gpu
def test_captured_and_replayed_on_new_inputs():
    require_gpu()
    past, new = [30, 200], [80, 33]
    c = make_cache([110, 233], 2, 64, "bf16", seed=10)
    q, out, lse, (d, a) = run(c, past, new, 8, 128, 1, seed=10)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        seer.seer_window_prefill(d, a)
    q.copy_(torch.randn(q.shape, generator=torch.Generator().manual_seed(1)).bfloat16())
    out.fill_(7)
    lse.fill_(7)
    graph.replay()
    torch.cuda.synchronize()
    check(c, past, new, q, out, lse, 128, 1)


@pytest.mark.gpu
def test_prompt_chunk_and_decode_over_one_cache():
    """A prompt, a second chunk and decode tokens of a ragged batch: rotary append, window prefill and window decode
    over one bf16 cache, as a server would run them, against attention over the rotated rows in fp64."""
    require_gpu()
    B, Hq, Hkv, bs, window, sinks = 3, 10, 2, 64, 150, 4
    g = torch.Generator().manual_seed(11)
    rope = seer.seer_rope_table(1024, 128)
    pages = 40
    kp, vp = [torch.full((pages, bs, Hkv, D), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    table = torch.randperm(pages, generator=g)[:B * 12].view(B, 12).int().cuda()
    d = seer.make_dims(B, Hq, Hkv, D, bs, 12, pages)
    lens = [0] * B
    hist = [[[], []] for _ in range(B)]                  # rotated k (as the cache holds it) and v rows
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for new in ([200, 17, 64], [90, 130, 1], [1, 1, 1], [1, 1, 1]):
        T = sum(new)
        rows = torch.randn((T, (Hq + 2 * Hkv) * D), generator=g).bfloat16().cuda()
        q, k, v = [x.unflatten(1, (-1, D)) for x in rows.split([Hq * D, Hkv * D, Hkv * D], 1)]
        cu = torch.tensor([sum(new[:i]) for i in range(B + 1)], dtype=torch.int32).cuda()
        lens = [x + n for x, n in zip(lens, new)]
        seqlens = torch.tensor(lens, dtype=torch.int32).cuda()
        qr, out = torch.empty((T, Hq, D), dtype=torch.bfloat16, device="cuda"), torch.empty((T, Hq, D), dtype=torch.bfloat16, device="cuda")
        seer.seer_append_rope(d, seer.append_args(k, v, kp, vp, table, seqlens, q=q, q_out=qr, rope=rope, cu_tokens=cu, max_new=max(new), dev_status=status))
        if max(new) == 1:
            splits = seer.seer_window_decode_splits(d, window, sinks)
            seer.seer_window_decode(d, seer.window_decode_args(qr, kp, vp, table, seqlens, window=window, sinks=sinks, num_splits=splits, softmax_scale=SCALE,
                                                               out=out, dev_status=status))
        else:
            seer.seer_window_prefill(d, seer.window_prefill_args(qr, kp, vp, table, seqlens, cu_tokens=cu, max_new=max(new), window=window, sinks=sinks,
                                                                 softmax_scale=SCALE, out=out, dev_status=status))
        torch.cuda.synchronize()
        assert status.item() == 0
        got, rp = out.double().cpu().numpy(), rope.double().cpu().numpy()
        qd, kd, vd = [x.double().cpu().numpy() for x in (q, k, v)]
        for b in range(B):
            for i in range(new[b]):
                t, pos = int(cu[b]) + i, lens[b] - new[b] + i
                cs, sn = rp[pos][:64], rp[pos][64:]
                hist[b][0].append(np.stack([C.rotate_row(kd[t, h], cs, sn, 128, False) for h in range(Hkv)]))
                hist[b][1].append(vd[t])
            K, V = np.stack(hist[b][0]), np.stack(hist[b][1])
            for i in range(0, new[b], 7):
                t, pos = int(cu[b]) + i, lens[b] - new[b] + i
                seen = C.window_seen(pos, lens[b], window, sinks)
                for qh in (0, Hq - 1):
                    h = qh // (Hq // Hkv)
                    qrow = C.rotate_row(qd[t, qh], rp[pos][:64], rp[pos][64:], 128, False)
                    want, _ = C.softmax_attention(qrow, K[:, h], V[:, h], seen, SCALE)
                    # q and k rounded to bf16 (each moves a score by 2^-8 sum |q k|, at most, and by its root over 128 dims in the mean), weights and out too
                    size = (np.abs(K[seen][:, h]) @ np.abs(qrow)).max() * SCALE
                    tol = 2 * 2.0 ** -8 * size * np.abs(V[seen][:, h]).max() + 2 * 2.0 ** -8 * np.abs(V[seen][:, h]).max()
                    assert np.abs(got[t, qh] - want).max() <= tol
                    assert np.linalg.norm(got[t, qh] - want) <= 1e-2 * np.linalg.norm(want) + 2.0 ** -8


@pytest.mark.gpu
@pytest.mark.parametrize("with_cu", [True, False])
def test_a_token_for_each_of_many_sequences(with_cu):
    """Many single tokens, some sequences without one, one too long: the others agree with a call of their own."""
    require_gpu()
    B, Hkv, G, bs, nbmax, pages = 150, 2, 4, 64, 5, 40
    g = torch.Generator().manual_seed(3)
    lens = torch.randint(1, nbmax * bs + 1, (B,), generator=g, dtype=torch.int32)
    new = torch.ones(B, dtype=torch.int32)
    new[5::9] = 0
    lens[5::9] = 0
    lens[20] = nbmax * bs + 1
    if not with_cu:
        new[:] = 1
    cu = torch.cat([torch.zeros(1), new.cumsum(0)]).int()
    T = int(cu[-1])
    k, v = [torch.randn((pages, bs, Hkv, D), generator=g).bfloat16().cuda() for _ in range(2)]
    table = torch.randint(0, pages, (B, nbmax), generator=g, dtype=torch.int32)
    q = torch.randn((T, Hkv * G, D), generator=g).bfloat16().cuda()
    out, lse, status = torch.full_like(q, 7), torch.full((Hkv * G, T), 7.0, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    d = seer.make_dims(B, Hkv * G, Hkv, D, bs, nbmax, pages)
    seer.seer_window_prefill(d, seer.window_prefill_args(q, k, v, table.cuda(), lens.cuda(), cu_tokens=cu.cuda() if with_cu else None, max_new=1, window=90, sinks=3,
                                                         softmax_scale=SCALE, out=out, lse_out=lse, dev_status=status))
    assert status.item() == seer.DEV_BAD_TOKENS
    for b in range(B):
        row = int(cu[b])
        if new[b] == 0:
            continue
        if lens[b] in (0, nbmax * bs + 1):
            assert (out[row] == 7).all() and (lse[:, row] == 7).all()
            continue
        o, l = torch.full_like(q[:1], 7), torch.full((Hkv * G, 1), 7.0, device="cuda")
        d1 = seer.make_dims(1, Hkv * G, Hkv, D, bs, nbmax, pages)
        seer.seer_window_prefill(d1, seer.window_prefill_args(q[row:row + 1], k, v, table[b:b + 1].cuda(), lens[b:b + 1].cuda(), window=90, sinks=3, softmax_scale=SCALE,
                                                              out=o, lse_out=l))
        # keys split over another number of CTAs: both round their weights and outputs to bf16
        assert (o[0].float() - out[row].float()).abs().max() <= 4 * 2.0 ** -8 * v.float().abs().max() and (l[:, 0] - lse[:, row]).abs().max() <= 1e-4


@pytest.mark.gpu
@pytest.mark.parametrize("Hkv", [1, 100])
@pytest.mark.parametrize("window,sinks,bs", [(70, 3, 64), (9, 0, 128), (400, 130, 64)])
def test_large_values_that_a_query_does_not_see_weigh_nothing(window, sinks, bs, Hkv):
    """Finite values next to bf16's largest, one dim of each token: where a query sees none of them in a dim, the dim is
    as if they were not there, whatever the key's place in a tile.  One CTA for each row tile, and keys split over a cluster."""
    require_gpu()
    past, new, L = 200, 90, 290
    c = make_cache([L], Hkv, bs, "bf16", seed=window)
    t = np.arange(L)
    pages = c["table"][0].numpy()[t // bs]
    huge = np.zeros((L, D), dtype=bool)
    for lo, first in ((past, 0), (max(0, past - window + 1), 32)):    # ahead of some queries, behind the window of some
        for i in range(min(new, 96)):
            huge[lo + i, first + i % 96] = True
            c["v"][pages[lo + i], (lo + i) % bs, :, first + i % 96] = 3e38 if i % 2 else -3e38
    G = 5
    q, out, lse, _ = run(c, [past], [new], G * Hkv, window, sinks, seed=window)
    K, V = values(c, "k"), values(c, "v")
    qd, got = q.double().cpu().numpy(), out.double().cpu().numpy()
    for h in {0, Hkv // 2, Hkv - 1}:
        k, v = K[pages, t % bs, h], V[pages, t % bs, h]
        for i in range(new):
            seen = C.window_seen(past + i, L, window, sinks)
            clean = ~huge[seen].any(0)
            assert clean.any()
            for qh in range(h * G, (h + 1) * G):
                want, want_lse = C.softmax_attention(qd[i, qh], k, v[:, clean], seen, SCALE)
                w = np.exp(k[seen] @ qd[i, qh] * SCALE - want_lse)
                # weights and out rounded to bf16 (2^-8 each); 1e-4 for scores of this size
                tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -8 + 1e-4) * (w @ np.abs(v[seen][:, clean]) + np.abs(want))
                assert (np.abs(got[i, qh, clean] - want) <= tol).all(), (i, qh, np.abs(got[i, qh, clean] - want).max())


@pytest.mark.gpu
@pytest.mark.parametrize("slot", [0, 1, 2])
@pytest.mark.parametrize("length", [-2 ** 31, -2 ** 31 + 70, -2 ** 31 + 71, -2 ** 31 + 100, -2 ** 31 + 101, -1, 2 ** 31 - 1])
def test_length_of_a_slot_without_new_tokens_does_not_matter(length, slot):
    """Windows of 70 whose difference from the length passes 32 bits: the other sequences' rows have the bits that they
    have beside a slot of length 0, through the append and the prefill."""
    require_gpu()
    past, new = [10, 300, 63], [40, 90, 2]
    past[slot] = new[slot] = 0
    c = make_cache([p + n for p, n in zip(past, new)], 2, 64, "bf16", seed=slot)
    c["k"], c["v"] = [torch.nan_to_num(c[n]) for n in "kv"]
    T, Hq, Hkv = sum(new), 8, 2
    g = torch.Generator().manual_seed(slot)
    q, k, v = [torch.randn((T, h, D), generator=g).bfloat16().cuda() for h in (Hq, Hkv, Hkv)]
    cu = torch.tensor([sum(new[:i]) for i in range(4)], dtype=torch.int32).cuda()
    got = []
    for at in (0, length):
        lens = list(c["lens"])
        lens[slot] = at
        seqlens, table = torch.tensor(lens, dtype=torch.int32).cuda(), c["table"].cuda()
        d = seer.make_dims(3, Hq, Hkv, D, 64, c["nbmax"], c["pages"])
        kp, vp, status = on_gpu(c, "k"), on_gpu(c, "v"), torch.zeros(1, dtype=torch.int32, device="cuda")
        qr, out, lse = torch.empty_like(q), torch.full_like(q, 7), torch.full((Hq, T), 7.0, device="cuda")
        kbar = torch.full((3, Hkv, c["nbmax"], D), 9.0, device="cuda")
        seer.seer_append_rope(d, seer.append_args(k, v, kp, vp, table, seqlens, q=q, q_out=qr, rope=seer.seer_rope_table(512, 128), cu_tokens=cu,
                                                  max_new=max(new), kbar=kbar, dev_status=status))
        seer.seer_window_prefill(d, seer.window_prefill_args(qr, kp, vp, table, seqlens, cu_tokens=cu, max_new=max(new), window=70, sinks=3,
                                                             softmax_scale=SCALE, out=out, lse_out=lse, dev_status=status))
        torch.cuda.synchronize()
        assert status.item() == 0
        got.append((qr, kp, vp, kbar, out, lse))
    assert all(torch.equal(a, b) for a, b in zip(*got)) and (got[1][4] != 7).any((1, 2)).all()


@pytest.mark.gpu
def test_prefills_on_two_streams_at_once():
    """A short chunk (keys split over clusters) on one stream and a long one on another, enqueued 12 times without a wait:
    the bits of calls one by one."""
    require_gpu()
    runs = []
    for seed, (past, new, Hkv) in enumerate((([700, 0], [40, 130], 2), ([100], [1500], 8))):
        c = make_cache([p + n for p, n in zip(past, new)], Hkv, 64, "bf16", seed=seed)
        runs.append(run(c, past, new, 4 * Hkv, 300, 5, seed=seed))
    want = [(out.clone(), lse.clone()) for _, out, lse, _ in runs]
    streams = [torch.cuda.Stream() for _ in runs]
    for _, out, lse, _ in runs:
        out.fill_(7)
        lse.fill_(7)
    torch.cuda.synchronize()
    for _ in range(12):
        for (_, _, _, (d, a)), stream in zip(runs, streams):
            seer.seer_window_prefill(d, a, stream)
    torch.cuda.synchronize()
    assert all(torch.equal(out, o) and torch.equal(lse, l) for (_, out, lse, _), (o, l) in zip(runs, want))
