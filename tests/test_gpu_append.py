"""seer_append_rope against its fp64 definition: ragged and single-token
appends to bf16 and 8-bit caches, rotation styles, strides, layouts, growing
scales, pooled keys, and rows that must stay as they were."""
import numpy as np
import pytest
import torch

from block_sparse_attention_step_b200 import seer
from oracle import cache_oracle as C

from gpu_util import require_gpu

D = 128
EPS32 = 2.0 ** -24


def setup_case(B, Hq, Hkv, bs, past, new, cache="bf16", layout="nhd", seed=0, fused=True, spare_pages=2, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    lens = [p + n for p, n in zip(past, new)]
    nb = [max(1, -(-x // bs)) for x in lens]
    nbmax = max(nb) + 1
    pages = sum(nb) + spare_pages
    perm = torch.randperm(pages, generator=g)
    table = torch.full((B, nbmax), -1, dtype=torch.int32)
    at = 0
    for b in range(B):
        table[b, :nb[b]] = perm[at:at + nb[b]].int()
        at += nb[b]
    T = sum(new) + 3                       # three rows behind the last sequence
    rows = torch.randn((T, (Hq + 2 * Hkv) * D), generator=g) * spread
    rows = rows.bfloat16().cuda()
    q, k, v = [x.unflatten(1, (-1, D)) for x in rows.split([Hq * D, Hkv * D, Hkv * D], 1)]
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    shape = (pages, bs, Hkv, D) if layout == "nhd" else (pages, Hkv, bs, D)
    if cache == "bf16":
        kp, vp = [torch.randn(shape, generator=g).bfloat16().cuda() for _ in range(2)]
        ks = vs = None
    elif cache == "e4m3":
        kp, vp = [(torch.randn(shape, generator=g) * 60).clamp(-440, 440).to(torch.float8_e4m3fn).cuda() for _ in range(2)]
        ks, vs = [torch.exp2(torch.randint(-9, -5, (pages, Hkv), generator=g).float()).cuda() for _ in range(2)]
    else:
        kp, vp = [torch.randint(-127, 128, shape, generator=g, dtype=torch.int8).cuda() for _ in range(2)]
        ks, vs = [(torch.rand((pages, Hkv), generator=g) * 0.03 + 0.005).cuda() for _ in range(2)]
    d = seer.make_dims(B, Hq, Hkv, D, bs, nbmax, pages)
    if layout == "hnd":
        d.stride_page, d.stride_head, d.stride_token = Hkv * bs * D, bs * D, D
    cu = torch.tensor([sum(new[:i]) for i in range(B + 1)], dtype=torch.int32).cuda()
    return dict(B=B, Hq=Hq, Hkv=Hkv, bs=bs, past=past, new=new, lens=lens, table=table, T=T, q=q, k=k, v=v, kp=kp, vp=vp, ks=ks, vs=vs,
                dims=d, cu=cu, seqlens=torch.tensor(lens, dtype=torch.int32).cuda(), nbmax=nbmax, layout=layout, cache=cache,
                status=torch.zeros(1, dtype=torch.int32).cuda())


def token_major(pool, layout):
    return pool if layout == "nhd" else pool.transpose(1, 2)


def values(pool, layout):
    """[pages][bs][Hkv][D] fp64 codes or values on the host."""
    x = token_major(pool, layout).contiguous()
    if x.dtype == torch.float8_e4m3fn:
        return C.e4m3_value(x.view(torch.uint8).cpu().numpy())
    return x.double().cpu().numpy()


def f64(t):
    return t.double().cpu().numpy()


def run_and_check(s, rotary=128, interleaved=False, kbar=False, positions=None, use_cu=True, with_q=True, in_place=False, expect_status=0):
    max_pos = max(s["lens"] + [1]) if positions is None else int(positions.max()) + 1
    rope = seer.seer_rope_table(max_pos, rotary) if rotary else None
    q_out = torch.full_like(s["q"], 7.0).contiguous() if with_q else None
    q_in = s["q"].clone()
    if in_place:
        q_out = s["q"]
    kb = torch.full((s["B"], s["Hkv"], s["nbmax"], D), 9.0, device="cuda") if kbar else None
    before = {n: values(s[n], s["layout"]) for n in ("kp", "vp")}
    scales = {n: f64(s[n]) for n in ("ks", "vs")} if s["ks"] is not None else None
    T = s["T"] if use_cu else s["B"]
    a = seer.append_args(s["k"][:T], s["v"][:T], s["kp"], s["vp"], s["table"].cuda(), s["seqlens"], q=s["q"][:T] if with_q else None,
                         q_out=q_out[:T] if with_q else None, rope=rope, interleaved=interleaved, cu_tokens=s["cu"] if use_cu else None,
                         max_new=max(s["new"] + [1]) if use_cu else 1, positions=positions, k_scale=s["ks"], v_scale=s["vs"], kbar=kb, dev_status=s["status"])
    seer.seer_append_rope(s["dims"], a)
    torch.cuda.synchronize()
    assert s["status"].item() == expect_status
    after = {n: values(s[n], s["layout"]) for n in ("kp", "vp")}
    now = {n: f64(s[n]) for n in ("ks", "vs")} if scales is not None else None
    expect = {n: before[n].copy() for n in before}      # what must not change, and what the old codes become
    written = {n: np.zeros(before[n].shape[:3], dtype=bool) for n in before}
    q, k, v = f64(q_in), f64(s["k"]), f64(s["v"])
    qo = f64(q_out) if with_q else None
    q_seen = np.zeros(s["T"], dtype=bool)
    table = s["table"].numpy()
    kb_want = f64(torch.full_like(kb, 9.0)) if kbar else None
    cu = s["cu"].cpu().tolist()
    for b in range(s["B"]):
        if s["new"][b] == 0:
            continue
        rows, cosines = [], []
        for i in range(s["new"][b]):
            t = (cu[b] if use_cu else b) + i
            p = s["past"][b] + i
            rp = p if positions is None else int(positions[t])
            cos, sin = C.rope_angles(rp, rotary) if rotary else (None, None)
            # the library reads fp32 table entries: the reference does too
            if rotary:
                row = rope[rp].double().cpu().numpy()
                assert np.abs(row - np.concatenate([cos, sin])).max() <= 2.0 ** -24   # half a step of values up to 1
                cos, sin = row[:rotary // 2], row[rotary // 2:]
            cosines.append((cos, sin))
            kr = np.stack([C.rotate_row(k[t, h], cos, sin, rotary, interleaved) if rotary else k[t, h] for h in range(s["Hkv"])])
            rows.append((t, p, kr, v[t]))
            q_seen[t] = True
            if with_q:
                for h in range(s["Hq"]):
                    want = C.rotate_row(q[t, h], cos, sin, rotary, interleaved) if rotary else q[t, h]
                    # one bf16 rounding (half a step: 2^-8 of the value), three fp32 roundings of terms up to 2 max|q|
                    tol = 2.0 ** -8 * np.abs(want) + 3 * EPS32 * 2 * np.abs(q[t, h]).max()
                    assert (np.abs(qo[t, h] - want) <= tol).all(), (b, i, h)
        for j in range(s["past"][b] // s["bs"], (s["lens"][b] - 1) // s["bs"] + 1):
            page = table[b, j]
            mine = [(p - j * s["bs"], kr, vr) for _, p, kr, vr in rows if p // s["bs"] == j]
            old_rows = max(0, s["past"][b] - j * s["bs"])
            for name, which, sc in (("kp", 1, "ks"), ("vp", 2, "vs")):
                for h in range(s["Hkv"]):
                    if s["cache"] != "bf16":
                        amax = max(np.abs(np.float32(m[which][h])).max() for m in mine)
                        had = scales[sc][page, h]
                        want = C.block_scale(s["cache"], float(amax), had, old_rows > 0)
                        got = now[sc][page, h]
                        # the same rule on fp32 values: a power of two exactly, or within fp32 rounding of amax / 127
                        assert got == want or (s["cache"] == "int8" and abs(got - want) <= 4 * EPS32 * want), (name, b, j, h, got, want)
                        if old_rows and got != had:
                            r = expect[name][page, :old_rows, h] * (had / got if had else 0.0)
                            if s["cache"] == "int8":
                                r = np.rint(r)
                            else:
                                r = C.e4m3_value(torch.tensor(r).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy())
                            expect[name][page, :old_rows, h] = r
                    for row, *kv in mine:
                        x = kv[which - 1][h]
                        written[name][page, row, h] = True
                        got = after[name][page, row, h]
                        fp32 = 3 * EPS32 * 2 * np.abs(x).max()
                        if s["cache"] == "bf16":
                            assert (np.abs(got - x) <= 2.0 ** -8 * np.abs(x) + fp32).all()
                        else:
                            sc_now = now[sc][page, h]
                            if sc_now == 0:
                                assert (x == 0).all() and (got == 0).all()
                                continue
                            y = x / sc_now
                            half = C.e4m3_half_step(y) if s["cache"] == "e4m3" else 0.5
                            assert (np.abs(got - y) <= half + fp32 / sc_now + 4 * EPS32 * np.abs(y)).all(), (name, b, j, h)
            if kbar:
                n = min(s["bs"], s["lens"][b] - j * s["bs"])
                for h in range(s["Hkv"]):
                    x = after["kp"][page, :n, h] * (now["ks"][page, h] if now else 1.0)
                    kb_want[b, h, j] = x.mean(0)
    for name in before:
        same = ~written[name]
        assert np.array_equal(after[name][same], expect[name][same], equal_nan=True), name
    if with_q and not in_place:
        assert (qo[~q_seen] == 7.0).all()
    if with_q and in_place:
        assert np.array_equal(qo[~q_seen], q[~q_seen])
    if kbar:
        got = f64(kb)
        # sums of up to 128 fp32 values in 24 steps: 24 half-steps of the largest partial sum, n * max / n
        tol = 24 * EPS32 * max(1.0, np.abs(kb_want[kb_want != 9.0]).max() * 16)
        assert np.abs(got - kb_want).max() <= tol
    return kb


CASES = [
    # B, Hq, Hkv, bs, past, new
    (1, 4, 1, 64, [0], [1]),
    (3, 8, 2, 64, [63, 64, 100], [1, 1, 1]),
    (4, 10, 2, 64, [0, 5, 63, 130], [70, 0, 1, 129]),
    (3, 6, 3, 128, [127, 0, 250], [2, 257, 7]),
    (2, 2, 1, 128, [1, 128], [126, 128]),
]


@pytest.mark.gpu
@pytest.mark.parametrize("cache", ["bf16", "e4m3", "int8"])
@pytest.mark.parametrize("case", range(len(CASES)))
@pytest.mark.parametrize("kbar", [False, True])
def test_append_matches_definition(case, cache, kbar):
    require_gpu()
    s = setup_case(*CASES[case], cache=cache, seed=case, layout="hnd" if case % 2 else "nhd", fused=case != 2)
    run_and_check(s, kbar=kbar)


@pytest.mark.gpu
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("rotary,interleaved", [(0, False), (16, False), (16, True), (64, True), (96, False), (128, True)])
def test_rotation_styles(rotary, interleaved, cache):
    require_gpu()
    s = setup_case(2, 4, 2, 64, [10, 0], [9, 70], cache=cache, seed=3)
    run_and_check(s, rotary=rotary, interleaved=interleaved, kbar=cache == "e4m3")


@pytest.mark.gpu
def test_own_positions_and_no_queries():
    require_gpu()
    s = setup_case(2, 4, 2, 64, [10, 0], [9, 20], seed=4)
    pos = torch.randint(0, 5000, (s["T"],), generator=torch.Generator().manual_seed(1)).int().cuda()
    run_and_check(s, positions=pos)
    s = setup_case(2, 4, 2, 64, [10, 0], [9, 20], seed=5)
    run_and_check(s, with_q=False, kbar=True)


@pytest.mark.gpu
@pytest.mark.parametrize("kbar", [False, True])
def test_queries_turned_in_place(kbar):
    require_gpu()
    s = setup_case(2, 4, 2, 64, [10, 0], [9, 20], seed=6)
    run_and_check(s, in_place=True, kbar=kbar)


@pytest.mark.gpu
@pytest.mark.parametrize("cache", ["bf16", "e4m3", "int8"])
def test_one_token_per_sequence_without_offsets(cache):
    require_gpu()
    s = setup_case(4, 8, 2, 64, [0, 64, 127, 3], [1, 1, 1, 1], cache=cache, seed=7)
    run_and_check(s, use_cu=False, kbar=cache != "bf16")


@pytest.mark.gpu
@pytest.mark.parametrize("cache", ["e4m3", "int8"])
def test_scales_double_until_rows_fit_and_zero_blocks(cache):
    """Token by token: growing magnitudes, a block of zero rows, tiny rows."""
    require_gpu()
    s = setup_case(1, 2, 2, 64, [0], [1], cache=cache, seed=8)
    for p in range(12):
        s["past"], s["new"], s["lens"] = [p], [1], [p + 1]
        s["seqlens"].fill_(p + 1)
        g = torch.Generator().manual_seed(p)
        s["k"] = (torch.randn((1, 2, D), generator=g) * 1.9 ** p).bfloat16().cuda()
        s["v"] = (torch.randn((1, 2, D), generator=g) * (0.0 if p < 3 else 1e-30 if p < 5 else 3.0 ** (p - 8))).bfloat16().cuda()
        s["q"], s["T"] = torch.randn((1, 2, D), generator=g).bfloat16().cuda(), 1
        s["cu"] = torch.tensor([0, 1], dtype=torch.int32).cuda()
        run_and_check(s, kbar=True)


@pytest.mark.gpu
def test_int8_regrowth_stays_below_one_step():
    """However often a block's scale doubles, a code stays within half its first step plus one
    half-step per doubling, the steps doubling: together below 1.0 step of the last scale (and
    the first rounding's own half-step, at most half a last step)."""
    require_gpu()
    s = setup_case(1, 1, 1, 64, [0], [1], cache="int8", seed=9)
    rows = []
    for p in range(40):
        g = torch.Generator().manual_seed(p)
        k = (torch.randn((1, 1, D), generator=g) * 1.3 ** p).bfloat16().cuda()
        rows.append(k[0, 0].double().cpu().numpy())
        a = seer.append_args(k, k.clone(), s["kp"], s["vp"], s["table"].cuda(), torch.tensor([p + 1], dtype=torch.int32).cuda(),
                             k_scale=s["ks"], v_scale=s["vs"], dev_status=s["status"])
        seer.seer_append_rope(s["dims"], a)
    torch.cuda.synchronize()
    page = s["table"][0, 0]
    step = float(s["ks"][page, 0])
    got = values(s["kp"], "nhd")[page, :40, 0] * step
    assert np.abs(got - np.stack(rows)).max() <= 1.0 * step
    assert s["status"].item() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("cache", ["e4m3", "int8"])
def test_nonfinite_rows_are_flagged_and_bounded(cache):
    require_gpu()
    s = setup_case(1, 1, 1, 64, [0], [3], cache=cache, seed=10)
    k = torch.ones((3, 1, D)).bfloat16()
    k[1, 0, 5], k[2, 0, 6], k[2, 0, 7] = float("nan"), float("inf"), float("-inf")
    k = k.cuda()
    a = seer.append_args(k, k.clone(), s["kp"], s["vp"], s["table"].cuda(), s["seqlens"], cu_tokens=s["cu"], max_new=3, k_scale=s["ks"], v_scale=s["vs"],
                         dev_status=s["status"])
    seer.seer_append_rope(s["dims"], a)
    torch.cuda.synchronize()
    assert s["status"].item() == seer.DEV_NONFINITE_KV
    top = {"e4m3": 448.0, "int8": 127.0}[cache]
    for pool, scale in ((s["kp"], s["ks"]), (s["vp"], s["vs"])):
        x = values(pool, "nhd")[s["table"][0, 0], :3, 0]
        assert float(scale[s["table"][0, 0], 0]) == C.block_scale(cache, 1.0, 0.0, False)
        assert x[2, 6] == top and x[2, 7] == -top
        assert np.isnan(x[1, 5]) if cache == "e4m3" else x[1, 5] == 0
        x[1, 5] = x[2, 6] = x[2, 7] = x[0, 0]
        assert (x == x[0, 0]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("bs", [64, 128])
@pytest.mark.parametrize("cache", ["e4m3", "int8"])
def test_nonfinite_rows_next_to_zeros_do_not_read_as_zero(cache, bs):
    """Nothing finite but zeros: the scale is 2^-60, not 0, so NaN stays NaN through a decode,
    and a later row finds the scale doubled until it fits."""
    require_gpu()
    s = setup_case(1, 1, 1, bs, [0], [2], cache=cache, seed=13)
    page = s["table"][0, 0]

    def append(rows, length):
        x = rows.cuda()
        a = seer.append_args(x, x.clone(), s["kp"], s["vp"], s["table"].cuda(), torch.tensor([length], dtype=torch.int32).cuda(),
                             cu_tokens=torch.tensor([0, len(rows)], dtype=torch.int32).cuda(), max_new=len(rows),
                             k_scale=s["ks"], v_scale=s["vs"], dev_status=s["status"])
        seer.seer_append_rope(s["dims"], a)
        torch.cuda.synchronize()
        return [values(pool, "nhd")[page, :length, 0] for pool in (s["kp"], s["vp"])]

    first = torch.zeros((2, 1, D)).bfloat16()
    first[0, 0, 3], first[1, 0, 4], first[1, 0, 5] = float("nan"), float("inf"), float("-inf")
    top = {"e4m3": 448.0, "int8": 127.0}[cache]
    for x, scale in zip(append(first, 2), (s["ks"], s["vs"])):
        assert float(scale[page, 0]) == 2.0 ** -60
        assert np.isnan(x[0, 3]) if cache == "e4m3" else x[0, 3] == 0
        assert x[1, 4] == top and x[1, 5] == -top
        x[0, 3] = x[1, 4] = x[1, 5] = 0
        assert (x == 0).all()
    assert s["status"].item() == seer.DEV_NONFINITE_KV
    if cache == "e4m3":
        q = torch.ones((1, 1, D)).bfloat16().cuda()
        out = torch.zeros_like(q)
        w = seer.window_decode_args(q, s["kp"], s["vp"], s["table"].cuda(), torch.tensor([2], dtype=torch.int32).cuda(), out=out, window=2, sinks=0,
                                    softmax_scale=0.1, k_scale=s["ks"], v_scale=s["vs"], num_splits=1)
        seer.seer_window_decode(s["dims"], w)
        assert out.isnan().all()
    for x, scale in zip(append(torch.ones((1, 1, D)).bfloat16(), 3), (s["ks"], s["vs"])):
        step = C.block_scale(cache, 1.0, 2.0 ** -60, True)
        assert float(scale[page, 0]) == step
        assert (x[2] == 1.0 / step).all()


@pytest.mark.gpu
@pytest.mark.parametrize("cache,kbar", [("bf16", False), ("bf16", True), ("e4m3", True)])
def test_sequences_that_do_not_fit_are_left_out(cache, kbar):
    """A sequence shorter than its new tokens, one longer than its table, one with a bad page, rows
    past max_new and positions past the table: flagged, the others appended, nothing else written."""
    require_gpu()
    def fresh():
        return setup_case(3, 4, 2, 64, [10, 0, 70], [9, 20, 3], cache=cache, seed=11)

    def call(s, seqlens, max_new=20, table=None, rope_rows=200):
        before = [values(x, "nhd") for x in (s["kp"], s["vp"])]
        a = seer.append_args(s["k"], s["v"], s["kp"], s["vp"], (s["table"] if table is None else table).cuda(), seqlens.cuda(), q=s["q"],
                             q_out=torch.full_like(s["q"], 7.0).contiguous(), rope=seer.seer_rope_table(rope_rows, 128), cu_tokens=s["cu"], max_new=max_new,
                             k_scale=s["ks"], v_scale=s["vs"], kbar=torch.zeros((3, 2, s["nbmax"], D), device="cuda") if kbar else None, dev_status=s["status"])
        seer.seer_append_rope(s["dims"], a)
        torch.cuda.synchronize()
        after = [values(x, "nhd") for x in (s["kp"], s["vp"])]
        return s["status"].item(), {int(p) for x, y in zip(before, after) for p in np.unique(np.nonzero(x != y)[0])}

    def pages(s, *seqs):
        return {int(s["table"][b, j]) for b in seqs for j in range(s["past"][b] // 64, (s["lens"][b] - 1) // 64 + 1)}

    s = fresh()
    got = call(s, torch.tensor([19, 19, 73], dtype=torch.int32))       # sequence 1: 20 new tokens, length 19
    assert got == (seer.DEV_BAD_TOKENS, pages(s, 0, 2))
    s = fresh()
    got = call(s, torch.tensor([19, 20, s["nbmax"] * 64 + 1], dtype=torch.int32))
    assert got == (seer.DEV_BAD_TOKENS, pages(s, 0, 1))
    s = fresh()
    got = call(s, s["seqlens"].cpu(), max_new=10)                        # sequence 1 has more
    assert got == (seer.DEV_BAD_TOKENS, pages(s, 0, 2))
    s = fresh()
    table = s["table"].clone()
    table[0, 0] = 100000
    got = call(s, s["seqlens"].cpu(), table=table)
    assert got == (seer.DEV_BAD_PAGE, pages(s, 1, 2))
    s = fresh()
    got = call(s, s["seqlens"].cpu(), rope_rows=60)                      # positions 70..72 are past it
    assert got == (seer.DEV_BAD_POSITION, pages(s, 0, 1, 2))
    s = fresh()
    s["cu"] = torch.tensor([0, 9, 5, 32], dtype=torch.int32).cuda()      # falls back, then runs past the rows
    got = call(s, s["seqlens"].cpu())
    assert got == (seer.DEV_BAD_TOKENS, pages(s, 0))


@pytest.mark.gpu
def test_pooled_keys_have_the_bits_of_seer_pool_keys():
    require_gpu()
    s = setup_case(3, 8, 2, 64, [0, 30, 64], [150, 40, 65], seed=12)
    kb = run_and_check(s, kbar=True)
    full = torch.zeros_like(kb)
    seer.seer_pool_keys(s["dims"], s["kp"], s["table"].cuda(), s["seqlens"], 0, full)
    for b in range(3):
        for j in range(s["past"][b] // 64, (s["lens"][b] - 1) // 64 + 1):
            assert torch.equal(kb[b, :, j], full[b, :, j])


@pytest.mark.gpu
def test_empty_call_and_another_stream():
    require_gpu()
    s = setup_case(2, 4, 2, 64, [10, 0], [0, 0], seed=13)
    before = s["kp"].clone()
    a = seer.append_args(s["k"][:0], s["v"][:0], s["kp"], s["vp"], s["table"].cuda(), s["seqlens"], cu_tokens=s["cu"], max_new=1, dev_status=s["status"])
    seer.seer_append_rope(s["dims"], a)
    torch.cuda.synchronize()
    assert torch.equal(before, s["kp"]) and s["status"].item() == 0
    s = setup_case(2, 4, 2, 64, [10, 0], [9, 70], seed=14)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run_and_check(s)


@pytest.mark.gpu
def test_tensors_of_another_device_than_the_current_one_are_refused(monkeypatch):
    require_gpu()
    s = setup_case(1, 2, 1, 64, [0], [3], seed=15)
    a = seer.append_args(s["k"], s["v"], s["kp"], s["vp"], s["table"].cuda(), s["seqlens"], cu_tokens=s["cu"], max_new=3)
    table = torch.full((8, 16), 7.0, device="cuda")
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)         # no second one is needed: nothing is launched
    with pytest.raises(ValueError, match="current device is cuda:1"):
        seer.seer_append_rope(s["dims"], a)
    with pytest.raises(ValueError, match="current device is cuda:1"):
        seer.seer_rope_table(8, 16, table=table)
    monkeypatch.undo()
    assert (table == 7).all()
