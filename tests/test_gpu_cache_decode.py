"""seer_sparse_decode_q8 and seer_window_decode against softmax attention in
fp64 over the cache's values: head groups, lengths from none to long, page
sizes, layouts, split counts, scales, and NaN wherever a row does not look."""
import math

import numpy as np
import pytest
import torch

from block_sparse_attention_step_b200 import seer
from oracle import cache_oracle as C

from gpu_util import require_gpu

D = 128
SCALE = 1 / math.sqrt(D)


def make_cache(lens, Hkv, bs, cache, layout="nhd", seed=0, scales="usual"):
    """Pools of random rows behind a random page table; on the host the values
    [pages][bs][Hkv][D] in fp64."""
    g = torch.Generator().manual_seed(seed)
    B = len(lens)
    nb = [-(-x // bs) for x in lens]
    nbmax = max(max(nb), 1) + 1
    pages = sum(nb) + 2
    table = torch.full((B, nbmax), -1, dtype=torch.int32)
    perm, at = torch.randperm(pages, generator=g), 0
    for b in range(B):
        table[b, :nb[b]] = perm[at:at + nb[b]].int()
        at += nb[b]
    out = {"table": table, "nbmax": nbmax, "pages": pages, "nb": nb, "cache": cache, "layout": layout, "bs": bs, "lens": lens, "Hkv": Hkv}
    for n in ("k", "v"):
        x = torch.randn((pages, bs, Hkv, D), generator=g)
        if cache == "bf16":
            out[n], out[n + "s"] = x.bfloat16(), None
            continue
        if scales == "usual":
            s = torch.exp(torch.randn((pages, Hkv), generator=g) * 0.5 - (4.0 if cache == "int8" else 5.0))
        else:                                             # scales far apart, some zero
            s = torch.exp2(torch.randint(-30, 5, (pages, Hkv), generator=g).float())
            s[torch.rand((pages, Hkv), generator=g) < 0.2] = 0.0
        if cache == "e4m3":
            out[n] = (x * 120).clamp(-448, 448).to(torch.float8_e4m3fn)
        else:
            out[n] = (x * 40).round().clamp(-127, 127).to(torch.int8)
        if scales == "usual" and cache == "e4m3":
            s = s / 1.2
        out[n + "s"] = s
    return out


def values(c, n):
    x = c[n]
    if x.dtype == torch.float8_e4m3fn:
        v = C.e4m3_value(x.view(torch.uint8).numpy())
    else:
        v = x.double().numpy()
    return v if c[n + "s"] is None else v * c[n + "s"].double().numpy()[:, None, :, None]


def poison(c, seen):
    """NaN (int8: the largest code) at every token of every page that no row of
    that head sees; seen[b][h]: visible tokens."""
    keep = torch.zeros((c["pages"], c["bs"], c["Hkv"]), dtype=torch.bool)
    for b, per_head in enumerate(seen):
        for h, s in enumerate(per_head):
            t = np.nonzero(s)[0]
            keep[c["table"][b].numpy()[t // c["bs"]], t % c["bs"], h] = True
    for n in ("k", "v"):
        if c["cache"] == "bf16":
            c[n][~keep] = float("nan")
        elif c["cache"] == "e4m3":
            c[n].view(torch.uint8)[~keep] = 0x7F
        else:
            c[n][~keep] = 127


def on_gpu(c, n):
    x = c[n]
    if c["layout"] == "hnd":
        y = x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x
        x = y.transpose(1, 2).contiguous().view(x.dtype)
    return x.cuda()


def dims(c, B, Hq):
    d = seer.make_dims(B, Hq, c["Hkv"], D, c["bs"], c["nbmax"], c["pages"])
    if c["layout"] == "hnd":
        d.stride_page, d.stride_head, d.stride_token = c["Hkv"] * c["bs"] * D, c["bs"] * D, D
    return d


def check(c, q, seen, out, lse, softmax_scale=SCALE):
    """Against fp64, row by row.  A weight's relative error: the fp32 sum of 128 products (128 half-steps of
    sum |q k|), exp2 (2^-21) and its own rounding (f16 2^-11, bf16 hi + lo 2^-17); out adds its bf16 rounding, 2^-8."""
    K, V = values(c, "k"), values(c, "v")
    qd = q.double().cpu().numpy()
    got, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
    G = q.shape[1] // c["Hkv"]
    for b in range(q.shape[0]):
        L = c["lens"][b]
        t = np.arange(L)
        pages = c["table"][b].numpy()[t // c["bs"]]
        for h in range(c["Hkv"]):
            k, v = K[pages, t % c["bs"], h], V[pages, t % c["bs"], h]
            s = seen[b][h]
            for i in range(h * G, (h + 1) * G):
                want, want_lse = C.softmax_attention(qd[b, i], k, v, s, softmax_scale)
                if not s.any():
                    assert (got[b, i] == 0).all() and gl[b, i] == -math.inf
                    continue
                size = (np.abs(k[s]) @ np.abs(qd[b, i])).max() * abs(softmax_scale)
                dx = 128 * 2.0 ** -24 * size + 2.0 ** -21
                w = np.exp((k[s] @ qd[b, i]) * softmax_scale - want_lse)
                spread = w @ np.abs(v[s])
                tol = 2.0 ** -8 * np.abs(want) + ((2.0 ** -17 if c["cache"] == "bf16" else 2.0 ** -11) + 2 * dx) * (spread + np.abs(want))
                assert (np.abs(got[b, i] - want) <= tol).all(), (b, i, np.abs(got[b, i] - want).max(), tol.min())
                assert abs(gl[b, i] - want_lse) <= 2 * dx + 4 * 2.0 ** -24 * abs(want_lse), (b, i, gl[b, i], want_lse)


def run_window(c, q, window, sinks, splits, softmax_scale=SCALE, stream=None):
    B, Hq, _ = q.shape
    d = dims(c, B, Hq)
    ws = torch.empty(max(1, seer.seer_split_workspace_bytes(d, splits)), dtype=torch.uint8, device="cuda")
    out = torch.full((B, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((B, Hq), 7.0, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    a = seer.window_decode_args(q, on_gpu(c, "k"), on_gpu(c, "v"), c["table"].cuda(), torch.tensor(c["lens"], dtype=torch.int32).cuda(),
                                window=window, sinks=sinks, num_splits=splits, softmax_scale=softmax_scale, out=out, lse_out=lse, workspace=ws,
                                k_scale=None if c["ks"] is None else c["ks"].cuda(), v_scale=None if c["vs"] is None else c["vs"].cuda(), dev_status=status)
    seer.seer_window_decode(d, a, stream)
    torch.cuda.synchronize()
    assert status.item() == 0
    return out, lse, (d, a)


def run_list(c, q, chosen, splits, k_max=None, expect_status=0):
    """chosen[b][h]: ascending block lists."""
    B, Hq, _ = q.shape
    k_max = k_max or max(1, max(len(x) for r in chosen for x in r))
    idx = torch.full((B, c["Hkv"], k_max), -1, dtype=torch.int32)
    n_sel = torch.zeros((B, c["Hkv"]), dtype=torch.int32)
    for b in range(B):
        for h in range(c["Hkv"]):
            idx[b, h, :len(chosen[b][h])] = torch.tensor(chosen[b][h], dtype=torch.int32)
            n_sel[b, h] = len(chosen[b][h])
    d = dims(c, B, Hq)
    ws = torch.empty(max(1, seer.seer_split_workspace_bytes(d, splits)), dtype=torch.uint8, device="cuda")
    out = torch.full((B, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((B, Hq), 7.0, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    a = seer.sparse_decode_q8_args(q, on_gpu(c, "k"), on_gpu(c, "v"), c["table"].cuda(), torch.tensor(c["lens"], dtype=torch.int32).cuda(), idx.cuda(),
                                   n_sel.cuda(), k_scale=c["ks"].cuda(), v_scale=c["vs"].cuda(), k_max=k_max, num_splits=splits, softmax_scale=SCALE,
                                   out=out, lse_out=lse, workspace=ws, dev_status=status)
    seer.seer_sparse_decode_q8(d, a)
    torch.cuda.synchronize()
    assert status.item() == expect_status
    return out, lse


def queries(B, Hq, seed, spread=1.0):
    g = torch.Generator().manual_seed(seed + 100)
    return (torch.randn((B, Hq, D), generator=g) * spread).bfloat16().cuda()


def draw_lists(c, seed, share):
    g = np.random.default_rng(seed)
    chosen, seen = [], []
    for b, L in enumerate(c["lens"]):
        nb, row, srow = c["nb"][b], [], []
        for _ in range(c["Hkv"]):
            n = min(nb, max(1, round(share * nb))) if nb else 0
            pick = sorted(g.choice(nb, n, replace=False).tolist()) if n else []
            row.append(pick)
            srow.append(np.isin(np.arange(L) // c["bs"], pick))
        chosen.append(row)
        seen.append(srow)
    return chosen, seen


@pytest.mark.gpu
@pytest.mark.parametrize("cache", ["e4m3", "int8"])
@pytest.mark.parametrize("G", [1, 3, 5, 8, 12, 16])
@pytest.mark.parametrize("bs,layout,splits", [(64, "nhd", 1), (128, "hnd", 3), (64, "hnd", 16), (128, "nhd", 7)])
def test_sparse_decode_q8(cache, G, bs, layout, splits):
    require_gpu()
    c = make_cache([0, 1, 63, 65, 1000], 2, bs, cache, layout, seed=G)
    chosen, seen = draw_lists(c, G, 0.6)
    poison(c, seen)
    q = queries(5, 2 * G, G)
    out, lse = run_list(c, q, chosen, splits)
    check(c, q, seen, out, lse)


@pytest.mark.gpu
@pytest.mark.parametrize("cache", ["e4m3", "int8"])
@pytest.mark.parametrize("splits", [1, 2, 8, 64])
def test_sparse_decode_q8_scales_far_apart(cache, splits):
    """Block scales from 2^-30 to 2^4 and zeros: the weights stay accurate where V's scale is tiny."""
    require_gpu()
    c = make_cache([700, 130], 2, 64, cache, seed=21, scales="wide")
    c["ks"] = torch.full_like(c["ks"], 0.01)
    c["ks"][1::5] = 0.0
    chosen, seen = draw_lists(c, 5, 1.0)
    q = queries(2, 8, 22)
    out, lse = run_list(c, q, chosen, splits)
    check(c, q, seen, out, lse)


@pytest.mark.gpu
def test_sparse_decode_q8_queries_of_any_size():
    require_gpu()
    c = make_cache([300, 64], 2, 64, "e4m3", seed=31)
    chosen, seen = draw_lists(c, 6, 1.0)
    for spread in (1e-20, 1e-3, 30.0):
        q = queries(2, 6, 32, spread)
        out, lse = run_list(c, q, chosen, 2)
        check(c, q, seen, out, lse)
    q = torch.zeros_like(q)
    out, lse = run_list(c, q, chosen, 2)
    check(c, q, seen, out, lse)


@pytest.mark.gpu
def test_sparse_decode_q8_bad_indices_and_pages_are_flagged():
    require_gpu()
    c = make_cache([300], 1, 64, "e4m3", seed=33)
    q = queries(1, 4, 34)
    out, lse = run_list(c, q, [[[1, 3, 5, 2 ** 30]]], 2, expect_status=seer.DEV_BAD_INDEX)   # blocks 0..4 exist
    seen = [[np.isin(np.arange(300) // 64, [1, 3])]]
    check(c, q, seen, out, lse)
    out, lse = run_list(c, q, [[[-5, 1, 3]]], 1, expect_status=seer.DEV_BAD_INDEX)
    check(c, q, seen, out, lse)
    c["table"][0, 3] = c["pages"]
    run_list(c, q, [[[1, 3]]], 1, expect_status=seer.DEV_BAD_PAGE)


@pytest.mark.gpu
def test_nan_that_a_row_sees_reaches_its_output():
    require_gpu()
    c = make_cache([200, 200], 1, 64, "e4m3", seed=35)
    c["k"].view(torch.uint8)[c["table"][0, 1], 3, 0, 5] = 0x7F
    c["v"].view(torch.uint8)[c["table"][1, 1], 3, 0, 5] = 0x7F
    q = queries(2, 4, 36)
    out, lse = run_list(c, q, [[[0, 1, 2]], [[0, 1, 2]]], 2)
    assert torch.isnan(out[0]).all() and torch.isnan(lse[0]).all()
    assert torch.isnan(out[1, :, 5]).all() and torch.isfinite(lse[1]).all() and torch.isfinite(out[1, :, 6:]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("cache", ["bf16", "e4m3", "int8"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (63, 4), (64, 64), (200, 100), (1000, 3), (5000, 0), (17, 5000), (2 ** 31 - 1, 0), (5, 2 ** 31 - 1)])
def test_window_decode(cache, window, sinks):
    require_gpu()
    n = window + sinks
    bs, layout, splits, G = [(64, "nhd", 1, 4), (128, "hnd", 2, 5), (64, "hnd", 8, 8), (128, "nhd", 32, 12)][n % 4]
    lens = [0, 1, 64, 129, 1203]
    c = make_cache(lens, 2, bs, cache, layout, seed=n)
    seen = [[C.window_seen(L - 1, L, window, sinks)] * 2 for L in lens]
    poison(c, seen)
    q = queries(5, 2 * G, n)
    out, lse, _ = run_window(c, q, window, sinks, splits)
    check(c, q, seen, out, lse)


@pytest.mark.gpu
@pytest.mark.parametrize("cache", ["bf16", "int8"])
@pytest.mark.parametrize("G", [1, 2, 7, 9, 16])
def test_window_decode_groups(cache, G):
    require_gpu()
    lens = [777, 90]
    c = make_cache(lens, 3, 64, cache, seed=G)
    seen = [[C.window_seen(L - 1, L, 300, 10)] * 3 for L in lens]
    q = queries(2, 3 * G, G)
    out, lse, _ = run_window(c, q, 300, 10, 4)
    check(c, q, seen, out, lse)


@pytest.mark.gpu
@pytest.mark.parametrize("splits", [6, 8, 24, 64])
def test_long_row_is_split_and_deterministic(splits):
    """One row of 20,000 tokens; the same bits from every call."""
    require_gpu()
    c = make_cache([20000], 1, 64, "e4m3", seed=41)
    seen = [[C.window_seen(19999, 20000, 18000, 130)]]
    q = queries(1, 4, 41)
    out, lse, (d, a) = run_window(c, q, 18000, 130, splits)
    check(c, q, seen, out, lse)
    first = out.clone()
    for _ in range(3):
        out.zero_()
        seer.seer_window_decode(d, a)
        assert torch.equal(out, first)


@pytest.mark.gpu
def test_scores_that_climb_and_a_negative_scale():
    """Scores that climb by hundreds over the sequence (the softmax reference moves again and again)."""
    require_gpu()
    L = 640
    c = make_cache([L], 1, 64, "bf16", seed=43)
    ramp = torch.linspace(0, 40, L)
    for t in range(L):
        c["k"][c["table"][0, t // 64], t % 64, 0] = ramp[t].bfloat16()
    q = torch.ones((1, 2, D)).bfloat16().cuda()
    seen = [[np.ones(L, dtype=bool)]]
    for scale in (SCALE, -SCALE):
        out, lse, _ = run_window(c, q, L, 0, 2, softmax_scale=scale)
        check(c, q, seen, out, lse, scale)


@pytest.mark.gpu
def test_offsets_past_32_bits():
    """Pages whose element offsets pass 2^31 and byte offsets pass 2^32."""
    require_gpu()
    Hkv, bs, pages = 8, 64, 68000                        # 68000 pages x 65536 codes = 4.46e9 bytes per pool
    k = torch.zeros((pages, bs, Hkv, D), dtype=torch.int8, device="cuda")
    v = torch.zeros_like(k)
    g = torch.Generator().manual_seed(5)
    tab = torch.tensor([[67999, 33000, 0, 65537]], dtype=torch.int32)
    kk, vv = [torch.randint(-127, 128, (4, bs, Hkv, D), generator=g, dtype=torch.int8) for _ in range(2)]
    for i, p in enumerate(tab[0].tolist()):
        k[p], v[p] = kk[i].cuda(), vv[i].cuda()
    c = {"k": kk, "v": vv, "ks": torch.full((4, Hkv), 0.02), "vs": torch.full((4, Hkv), 0.03), "cache": "int8", "layout": "nhd", "bs": bs, "lens": [250],
         "Hkv": Hkv, "table": torch.arange(4, dtype=torch.int32)[None]}
    scale = torch.full((pages, Hkv), 0.02, device="cuda")
    d = seer.make_dims(1, 16, Hkv, D, bs, 4, pages)
    q = queries(1, 16, 6)
    out, lse = torch.empty((1, 16, D), dtype=torch.bfloat16, device="cuda"), torch.empty((1, 16), device="cuda")
    a = seer.window_decode_args(q, k, v, tab.cuda(), torch.tensor([250], dtype=torch.int32).cuda(), window=250, sinks=0, num_splits=2, softmax_scale=SCALE,
                                out=out, lse_out=lse, k_scale=scale, v_scale=scale * 1.5)
    seer.seer_window_decode(d, a)
    c["vs"] = (scale[:4] * 1.5).cpu()
    c["ks"] = scale[:4].cpu()
    check(c, q, [[np.ones(250, dtype=bool)] * Hkv], out, lse)


@pytest.mark.gpu
def test_captured_graphs_with_their_own_workspaces_replay_together():
    require_gpu()
    c = make_cache([3000, 2000], 2, 64, "e4m3", seed=51)
    seen = [[C.window_seen(L - 1, L, 2500, 4)] * 2 for L in c["lens"]]
    sides = []
    for i in range(2):
        q = queries(2, 8, 52 + i)
        out, lse, (d, a) = run_window(c, q, 2500, 4, 16)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            seer.seer_window_decode(d, a)
        sides.append((q, out, lse, graph, side))
    for q, out, lse, graph, side in sides:
        out.zero_()
    torch.cuda.synchronize()
    for _ in range(5):
        for q, out, lse, graph, side in sides:
            with torch.cuda.stream(side):
                graph.replay()
    torch.cuda.synchronize()
    for q, out, lse, graph, side in sides:
        check(c, q, seen, out, lse)


@pytest.mark.gpu
@pytest.mark.parametrize("B,G", [(40, 4), (41, 16), (256, 1), (300, 2)])
def test_rows_of_large_ragged_batches_go_where_they_belong(B, G):
    """More CTAs than fit at once go out longest sequence first (to 256 sequences): every row has the bits that it has in
    a small batch.  Lengths repeat, and some are 0."""
    require_gpu()
    Hkv, bs, nbmax, S = 8, 64, 6, 2
    g = torch.Generator().manual_seed(B)
    lens = torch.randint(0, nbmax * bs + 1, (B,), generator=g, dtype=torch.int32)
    lens[::7] = 100
    lens[3::11] = 0
    pages = 64
    k, v = [torch.randint(-127, 128, (pages, bs, Hkv, D), generator=g, dtype=torch.int8).cuda() for _ in range(2)]
    ks, vs = [torch.rand((pages, Hkv), generator=g).cuda() * 0.02 + 0.001 for _ in range(2)]
    table = torch.randint(0, pages, (B, nbmax), generator=g, dtype=torch.int32)
    q = queries(B, Hkv * G, B)
    idx = torch.arange(nbmax, dtype=torch.int32).repeat(B, Hkv, 1).cuda()
    n_sel = ((lens + bs - 1) // bs)[:, None].repeat(1, Hkv).int()
    n_sel[:, 1] = torch.clamp(n_sel[:, 1] - 1, min=0)
    got = []
    for step in (B, 9):
        out, lse, status = torch.full_like(q, 7), torch.full((B, Hkv * G), 7.0, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
        for i in range(0, B, step):
            n = min(step, B - i)
            d = seer.make_dims(n, Hkv * G, Hkv, D, bs, nbmax, pages)
            a = seer.sparse_decode_q8_args(q[i:i + n], k, v, table[i:i + n].cuda(), lens[i:i + n].cuda(), idx[i:i + n], n_sel[i:i + n].cuda(), k_scale=ks,
                                           v_scale=vs, k_max=nbmax, num_splits=S, softmax_scale=SCALE, out=out[i:i + n], lse_out=lse[i:i + n], dev_status=status)
            seer.seer_sparse_decode_q8(d, a)
        torch.cuda.synchronize()
        assert status.item() == 0
        got.append((out, lse))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    empty = (lens == 0).cuda()
    assert (got[0][0][empty] == 0).all() and got[0][1][empty].isneginf().all() and got[0][0][~empty].abs().amax((1, 2)).min() > 0


def block_scales(c, exponents):
    """Sets V's scales of sequence 0's blocks to 2^e (e None: 0, whose codes count as zero)."""
    for j, e in enumerate(exponents):
        page = c["table"][0, j]
        c["vs"][page] = 0.0 if e is None else 2.0 ** e


def check_far(c, q, seen, out, lse, splits, softmax_scale=SCALE):
    """check() where single tokens or blocks take nearly all the weight.  A weight's f16 rounding is relative to the
    largest of w_t vs_t (the running reference is at most that), so below 2^-14 of it a step is 2^-24: 2^-25 of it
    times every token's code is added.  So is 2^-134, half the least step of bf16 numbers.  More than 8 pieces are joined
    with the weights e^(lse_piece - the largest) in fp32, where those below 2^-126 are 0: a piece's out, at most the
    largest value, may go missing with that weight.  Past bf16's largest number, 255 * 2^120, out is an infinity."""
    K, V = values(c, "k"), values(c, "v")
    qd, got, gl = q.double().cpu().numpy(), out.double().cpu().numpy(), lse.double().cpu().numpy()
    G, vs = q.shape[1] // c["Hkv"], c["vs"].double().numpy()
    for b in range(q.shape[0]):
        t = np.arange(c["lens"][b])
        pages = c["table"][b].numpy()[t // c["bs"]]
        for h in range(c["Hkv"]):
            s = seen[b][h]
            k, v, scale = K[pages, t % c["bs"], h][s], V[pages, t % c["bs"], h][s], vs[pages, h][s]
            codes = np.abs(v / np.where(scale > 0, scale, 1.0)[:, None]).sum(0)
            for i in range(h * G, (h + 1) * G):
                want, want_lse = C.softmax_attention(qd[b, i], k, v, np.ones(len(k), dtype=bool), softmax_scale)
                size = (np.abs(k) @ np.abs(qd[b, i])).max() * abs(softmax_scale)
                dx = 128 * 2.0 ** -24 * size + 2.0 ** -21
                w = np.exp((k @ qd[b, i]) * softmax_scale - want_lse)
                tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -11 + 2 * dx) * (w @ np.abs(v) + np.abs(want)) + 2.0 ** -25 * (w * scale).max() * codes + 2.0 ** -134
                tol += 2.0 ** -126 * np.abs(v).max() if splits > 8 else 0.0
                past = (np.abs(want) + tol > 255 * 2.0 ** 120) & (got[b, i] == np.copysign(np.inf, want))
                assert ((np.abs(got[b, i] - want) <= tol) | past).all(), (b, i, np.abs(got[b, i] - want).max(), tol.min())
                assert abs(gl[b, i] - want_lse) <= 2 * dx + 4 * 2.0 ** -24 * abs(want_lse), (b, i, gl[b, i], want_lse)


FAR = [[-118], [110], [-126, -100, -126], [-120, 0, 90, None, -60], [0, -119, 3, -108], [None, -126], [121, -126, 40, -70, None, 0]]


@pytest.mark.gpu
@pytest.mark.parametrize("form", ["list", "window"])
@pytest.mark.parametrize("cache,splits", [("e4m3", 1), ("int8", 3), ("e4m3", 8), ("int8", 16)])
@pytest.mark.parametrize("far", range(len(FAR)))
def test_value_scales_over_the_whole_range(far, cache, splits, form):
    """V scales from the least normal number to the largest that rows can ask for, alone and side by side: out and lse
    are those of the values, also where a block of tiny values takes all the weight."""
    require_gpu()
    L = 64 * 12 - 9
    c = make_cache([L], 2, 64, cache, seed=far)
    block_scales(c, [FAR[far][j % len(FAR[far])] for j in range(12)])
    for heavy in (False, True):
        if heavy:                                        # the first block's keys: some 40 above the others
            page = c["table"][0, 0]
            c["ks"][page] *= 4
        q = queries(1, 12, far, 12.0 if heavy else 1.0)
        seen = [[np.ones(L, dtype=bool)] * 2]
        out, lse = run_list(c, q, [[list(range(12))] * 2], splits) if form == "list" else run_window(c, q, L, 0, splits)[:2]
        check_far(c, q, seen, out, lse, splits)


@pytest.mark.gpu
@pytest.mark.parametrize("cache", ["e4m3", "int8"])
@pytest.mark.parametrize("splits", [1, 4, 16])
def test_zero_block_that_takes_all_the_weight(cache, splits):
    """A block of zero values whose scores lie 60 above the others': out is the others' share, as small as it is."""
    require_gpu()
    L = 64 * 6
    c = make_cache([L], 1, 64, cache, seed=61)
    page = c["table"][0, 2]
    code = 100 if cache == "int8" else 96.0
    c["k"][page] = torch.full(c["k"][page].shape, code).to(c["k"].dtype)
    q = (torch.ones((1, 4, D)) + 0.1 * torch.randn((1, 4, D), generator=torch.Generator().manual_seed(62))).bfloat16().cuda()
    c["ks"][page] = 60 / (code * D * SCALE)
    c["vs"][page] = 0.0
    seen = [[np.ones(L, dtype=bool)]]
    out, lse = run_list(c, q, [[list(range(6))]], splits)
    assert out.abs().max() > 0
    check_far(c, q, seen, out, lse, splits)
