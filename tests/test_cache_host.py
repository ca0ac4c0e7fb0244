"""Argument checks of the paged-cache operators (no GPU: every case is refused
on the host before any CUDA work) and the fp64 definitions they are tested
against."""
import ctypes
import math
import os

import numpy as np
import pytest
import torch

from block_sparse_attention_step_b200 import seer
from oracle import cache_oracle as C


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(seer.LIB_PATH):
        from block_sparse_attention_step_b200 import build
        build.build()
    return seer.library()


OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 4
P = 4096  # stands for a 16-byte aligned device pointer; never followed


def dims(**kw):
    d = seer.make_dims(2, 8, 2, 128, 64, 4, 8)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def fill(struct, **kw):
    a = struct()
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def append(**kw):
    base = dict(q=P, k_new=P, v_new=P, q_out=2 * P, cu_tokens=P, rope=P, total_tokens=5, max_new=3, max_position=100, rotary_dim=64, cache_type=0, k_pool=P,
                v_pool=P, seqlens=P)
    base.update(kw)
    return fill(seer.seer_append_args, **base)


@pytest.mark.parametrize("change,code", [
    (dict(k_new=None), INVALID), (dict(v_new=None), INVALID), (dict(seqlens=None), INVALID), (dict(q_out=None), INVALID), (dict(q=None), INVALID),
    (dict(total_tokens=-1), INVALID), (dict(max_new=0), INVALID), (dict(cu_tokens=None), INVALID), (dict(cu_tokens=None, total_tokens=2), INVALID),
    (dict(rope=None), INVALID), (dict(rotary_dim=0), INVALID), (dict(rotary_dim=-16), INVALID), (dict(max_position=0), INVALID), (dict(interleaved=2), INVALID),
    (dict(rotary_dim=24), UNSUPPORTED), (dict(rotary_dim=144), UNSUPPORTED), (dict(cache_type=3), INVALID), (dict(k_pool=None), INVALID), (dict(v_pool=None), INVALID),
    (dict(k_scale=P), INVALID), (dict(cache_type=1), INVALID), (dict(cache_type=2, k_scale=P), INVALID), (dict(k_pool=P + 8), UNSUPPORTED),
    (dict(q=P + 8), UNSUPPORTED), (dict(k_new=P + 2), UNSUPPORTED), (dict(v_new=P + 2), UNSUPPORTED), (dict(q_out=P + 4), UNSUPPORTED), (dict(rope=P + 4), UNSUPPORTED),
    (dict(kbar=P + 4), UNSUPPORTED), (dict(q_stride=1020), INVALID), (dict(k_stride=128), INVALID), (dict(k_stride=260), UNSUPPORTED), (dict(v_stride=-256), INVALID)])
def test_append_refusals(lib, change, code):
    assert lib.seer_append_rope(ctypes.byref(dims()), ctypes.byref(append(**change)), None) == code


def test_append_refuses_strides_an_8_bit_pool_cannot_have(lib):
    a = append(cache_type=1, k_scale=P, v_scale=P)
    assert lib.seer_append_rope(ctypes.byref(dims(stride_head=136)), ctypes.byref(a), None) == UNSUPPORTED
    assert lib.seer_append_rope(ctypes.byref(dims(head_dim=64)), ctypes.byref(a), None) == UNSUPPORTED
    assert lib.seer_append_rope(ctypes.byref(dims()), None, None) == INVALID
    # no rows: nothing to do, whatever the row pointers are
    assert lib.seer_append_rope(ctypes.byref(dims()), ctypes.byref(append(total_tokens=0, q=None, q_out=None, k_new=None, v_new=None)), None) == OK


def attn(**kw):
    base = dict(q=P, cache_type=1, num_splits=2, k_pool=P, v_pool=P, k_scale=P, v_scale=P, seqlens=P, idx=P, n_sel=P, k_max=4, window=10, sinks=2, softmax_scale=0.1,
                out=P)
    base.update(kw)
    return fill(seer.seer_cache_attn_args, **base)


@pytest.mark.parametrize("form", ["seer_sparse_decode_q8", "seer_window_decode"])
@pytest.mark.parametrize("change,code", [
    (dict(q=None), INVALID), (dict(out=None), INVALID), (dict(seqlens=None), INVALID), (dict(k_pool=None), INVALID), (dict(k_scale=None), INVALID),
    (dict(cache_type=7), INVALID), (dict(num_splits=0), INVALID), (dict(num_splits=9), INVALID), (dict(num_splits=20), INVALID), (dict(num_splits=72), INVALID),
    (dict(q=P + 8), UNSUPPORTED), (dict(v_pool=P + 4), UNSUPPORTED), (dict(num_splits=16), WORKSPACE), (dict(num_splits=16, workspace=P, workspace_bytes=100), WORKSPACE),
    (dict(num_splits=16, workspace=P + 128, workspace_bytes=1 << 20), WORKSPACE)])
def test_decode_refusals(lib, form, change, code):
    assert getattr(lib, form)(ctypes.byref(dims()), ctypes.byref(attn(**change)), None) == code


def test_decode_refusals_of_one_form(lib):
    d = dims()
    for change, code in ((dict(idx=None), INVALID), (dict(n_sel=None), INVALID), (dict(k_max=0), INVALID), (dict(k_max=5), INVALID),
                         (dict(cache_type=0, k_scale=None, v_scale=None), UNSUPPORTED)):
        assert lib.seer_sparse_decode_q8(ctypes.byref(d), ctypes.byref(attn(**change)), None) == code
    for change, code in ((dict(window=0), INVALID), (dict(sinks=-1), INVALID), (dict(cache_type=0), INVALID)):
        assert lib.seer_window_decode(ctypes.byref(d), ctypes.byref(attn(**change)), None) == code


@pytest.mark.parametrize("change,code", [
    (dict(seqlens=None), INVALID), (dict(q=None), INVALID), (dict(out=None), INVALID), (dict(window=0), INVALID), (dict(sinks=-1), INVALID), (dict(max_new=0), INVALID),
    (dict(total_tokens=-1), INVALID), (dict(cu_tokens=None), INVALID), (dict(softmax_scale=0.0), INVALID), (dict(softmax_scale=-1.0), INVALID),
    (dict(softmax_scale=math.inf), INVALID), (dict(softmax_scale=math.nan), INVALID), (dict(k_pool=None), INVALID), (dict(v_pool=P + 2), UNSUPPORTED),
    (dict(q=P + 8), UNSUPPORTED), (dict(out=P + 8), UNSUPPORTED), (dict(total_tokens=0, q=None, out=None), OK)])
def test_window_prefill_refusals(lib, change, code):
    base = dict(q=P, k_pool=P, v_pool=P, cu_tokens=P, seqlens=P, total_tokens=5, max_new=3, window=10, sinks=2, softmax_scale=0.1, out=P)
    base.update(change)
    a = fill(seer.seer_window_prefill_args, **base)
    assert lib.seer_window_prefill(ctypes.byref(dims()), ctypes.byref(a), None) == code


def test_rope_table_refusals(lib):
    for args, code in (((0, 64, 1e4, P), INVALID), ((10, 63, 1e4, P), INVALID), ((10, 0, 1e4, P), INVALID), ((10, 64, 0.0, P), INVALID), ((10, 64, 1e4, None), INVALID),
                       ((10, 130, 1e4, P), UNSUPPORTED), ((10, 64, 1e4, P + 2), UNSUPPORTED)):
        assert lib.seer_rope_table(*args, None) == code


def test_split_helpers(lib):
    for batch, kv, k_max in ((1, 1, 1), (1, 1, 8), (1, 1, 4000), (16, 8, 52), (64, 8, 100), (512, 8, 4000)):
        d = seer.make_dims(batch, kv, kv, 128, 64, 4096, 10)
        for s in (seer.seer_sparse_decode_q8_splits(d, k_max), seer.seer_window_decode_splits(d, 64 * k_max, 4)):
            assert 1 <= s <= 64 and (s <= 8 or s % 8 == 0)
            need = seer.seer_split_workspace_bytes(d, s)
            assert (need == 0) == (s <= 8) and need >= (0 if s <= 8 else batch * kv * (s // 8) * 129 * 4)


def test_binding_checks_types_shapes_and_strides():
    cpu = torch.zeros((4, 2, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        seer.append_args(cpu, cpu, cpu, cpu, None, cpu)          # host tensors
    with pytest.raises(TypeError):
        seer.append_args(cpu.float(), cpu, cpu, cpu, None, cpu)


# ---------------------------------------------------------- the definitions
def test_e4m3_values_match_the_conversion_of_torch():
    codes = torch.arange(256, dtype=torch.uint8)
    want = codes.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(C.e4m3_value(codes.numpy()), want, equal_nan=True)
    for x in (0.0, 2.0 ** -9, 0.3, 1.0, 100.0, 447.0):          # half a step is what rounding may move
        y = float(torch.tensor(x).to(torch.float8_e4m3fn).double())
        assert abs(y - x) <= C.e4m3_half_step(x)


def test_rotation_is_complex_multiplication():
    rng = np.random.default_rng(0)
    x = rng.standard_normal(128)
    for rotary in (16, 96, 128):
        cos, sin = C.rope_angles(37, rotary)
        turn = cos + 1j * sin
        y = C.rotate_row(x, cos, sin, rotary, True)
        z = (x[:rotary:2] + 1j * x[1:rotary:2]) * turn
        assert np.allclose(y[:rotary:2] + 1j * y[1:rotary:2], z, atol=1e-14) and np.array_equal(y[rotary:], x[rotary:])
        y = C.rotate_row(x, cos, sin, rotary, False)
        z = (x[:rotary // 2] + 1j * x[rotary // 2:rotary]) * turn
        assert np.allclose(y[:rotary // 2] + 1j * y[rotary // 2:rotary], z, atol=1e-14)


def test_scale_rules_by_hand():
    assert C.block_scale("e4m3", 448.0, 0.0, False) == 1.0 and C.block_scale("e4m3", 448.1, 0.0, False) == 2.0
    assert C.block_scale("e4m3", 0.9, 0.0, False) == 2.0 ** -8 and C.block_scale("e4m3", 0.0, 0.0, False) == 0.0
    assert C.block_scale("int8", 254.0, 0.0, False) == 2.0
    assert C.block_scale("int8", 254.0, 0.5, True) == 2.0 and C.block_scale("int8", 255.0, 0.5, True) == 4.0 and C.block_scale("int8", 1.0, 0.5, True) == 0.5
    assert C.block_scale("int8", 127.0, 0.0, True) == 1.0       # a block of zeros so far


def test_window_by_hand():
    assert C.window_seen(5, 8, 3, 1).tolist() == [True, False, False, True, True, True, False, False]
    assert C.window_seen(1, 4, 9, 0).tolist() == [True, True, False, False]
    assert C.window_seen(3, 4, 1, 2).tolist() == [True, True, False, True]


# ------------------------------------------------- sizes against the dims
class Sized:
    """Stands for a device tensor: what the binding's checks ask of one."""

    is_cuda, device = True, torch.device("cuda", 0)

    def __init__(self, dtype, *shape):
        self.dtype, self.shape = dtype, shape

    def numel(self):
        return math.prod(self.shape)

    def dim(self):
        return len(self.shape)

    def stride(self, i):
        return math.prod(self.shape[i + 1:])

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 16 * id(self)


BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


def fitting(op):
    """Tensors that just fit dims(): B 2, 8 / 2 heads, 4 blocks of 64, 8 pages; 5 rows of new tokens."""
    pool = {"k_pool": Sized(BF, 8, 64, 2, 128), "v_pool": Sized(BF, 8, 64, 2, 128)}
    if op in ("sparse_decode_q8", "append_q8"):
        pool = {"k_pool": Sized(torch.int8, 8, 64, 2, 128), "v_pool": Sized(torch.int8, 8, 64, 2, 128), "k_scale": Sized(F32, 8, 2), "v_scale": Sized(F32, 8, 2)}
    t = {**pool, "page_table": Sized(I32, 2, 4), "seqlens": Sized(I32, 2), "dev_status": Sized(I32, 1)}
    if op.startswith("append"):
        t.update(k_new=Sized(BF, 5, 2, 128), v_new=Sized(BF, 5, 2, 128), q=Sized(BF, 5, 8, 128), q_out=Sized(BF, 5, 8, 128), rope=Sized(F32, 100, 64),
                 cu_tokens=Sized(I32, 3), positions=Sized(I32, 5), kbar=Sized(F32, 2, 2, 4, 128))
        return t, dict(max_new=3)
    if op == "window_prefill":
        t.update(q=Sized(BF, 5, 8, 128), out=Sized(BF, 5, 8, 128), lse_out=Sized(F32, 8, 5), cu_tokens=Sized(I32, 3))
        return t, dict(max_new=3, window=10, sinks=2, softmax_scale=0.1)
    t.update(q=Sized(BF, 2, 8, 128), out=Sized(BF, 2, 8, 128), lse_out=Sized(F32, 2, 8))
    if op == "window_decode":
        return t, dict(window=10, sinks=2, num_splits=1, softmax_scale=0.1)
    t.update(idx=Sized(I32, 2, 2, 3), n_sel=Sized(I32, 2, 2))
    return t, dict(k_max=3, num_splits=1, softmax_scale=0.1)


OPS = ["append", "append_q8", "sparse_decode_q8", "window_decode", "window_prefill"]


def block_of(op, t, more):
    return getattr(seer, op.replace("append_q8", "append") + "_args")(**t, **more)


@pytest.mark.parametrize("op", OPS)
def test_tensors_smaller_than_the_dims_are_refused(lib, op):
    d = dims()
    t, more = fitting(op)
    seer._check_sizes(op, d, block_of(op, t, more))                    # just large enough
    for name in t:
        shape = t[name].shape
        for less in {(shape[0] - 1,) + shape[1:], shape[:-1] + (shape[-1] - 1,)}:
            small = {**t, name: Sized(t[name].dtype, *less)}
            if name == "k_new":
                small["v_new"] = Sized(BF, *less)
            if name in ("q", "q_out") and op.startswith("append"):
                small["q"], small["q_out"] = Sized(BF, *less), Sized(BF, *less)
            rows_are_ours = name in ("q", "k_new") and op in ("append", "append_q8", "window_prefill")
            if name == "rope" or (rows_are_ours and less[0] != shape[0]):
                continue                                               # these say themselves how many rows there are
            with pytest.raises(ValueError):
                seer._check_sizes(op, d, block_of(op, small, more))


@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("change", [dict(batch=5), dict(max_blocks=5), dict(num_pages=9), dict(num_q_heads=10), dict(num_kv_heads=4), dict(block_size=128),
                                    dict(stride_page=64 * 2 * 128 + 16), dict(stride_token=512)])
def test_larger_dims_than_the_tensors_are_refused(lib, op, change):
    t, more = fitting(op)
    a = block_of(op, t, more)
    with pytest.raises(ValueError, match=op):
        seer._check_sizes(op, dims(**change), a)


def test_heads_that_only_add_up_are_refused(lib):
    t, more = fitting("append")
    for name in ("q", "k_new"):
        other = "q_out" if name == "q" else "v_new"
        shape = (10, t[name].shape[1] // 2, 128)
        with pytest.raises(ValueError):
            seer._check_sizes("append", dims(), block_of("append", {**t, name: Sized(BF, *shape), other: Sized(BF, *shape)}, more))
    # tables and outputs made for a larger batch stay allowed
    t, more = fitting("window_decode")
    t.update(page_table=Sized(I32, 5, 4), seqlens=Sized(I32, 5), out=Sized(BF, 5, 8, 128), k_pool=Sized(BF, 9, 64, 2, 128))
    seer._check_sizes("window_decode", dims(), block_of("window_decode", t, more))


def test_a_call_checks_sizes_before_anything_else_and_again_when_something_changed(lib, monkeypatch):
    t, more = fitting("window_decode")
    a, d = block_of("window_decode", t, more), dims()
    calls = []
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(seer, "_lib_handle", type("Lib", (), {"seer_window_decode": staticmethod(lambda *x: calls.append(x) or 0)}))
    for _ in range(2):
        seer.seer_window_decode(d, a, 0)
    assert len(calls) == 2
    d.batch = 5
    with pytest.raises(ValueError, match="seer_window_decode: q has 2048 elements"):
        seer.seer_window_decode(d, a, 0)
    d.batch = 2
    seer.seer_window_decode(d, a, 0)
    a.k_max = 7                                                         # of the other form: asks for no tensor here
    seer.seer_window_decode(d, a, 0)
    assert len(calls) == 4


@pytest.mark.parametrize("op,name,shape", [
    ("append", "page_table", (2, 6)), ("append", "kbar", (2, 2, 5, 128)), ("append_q8", "k_scale", (8, 3)), ("window_decode", "page_table", (2, 5)),
    ("window_decode", "q", (2, 10, 128)), ("window_decode", "out", (2, 8, 256)), ("window_decode", "lse_out", (2, 9)), ("sparse_decode_q8", "idx", (2, 2, 4)),
    ("sparse_decode_q8", "n_sel", (2, 3)), ("window_prefill", "lse_out", (8, 6)), ("window_prefill", "q", (5, 10, 128)), ("window_prefill", "page_table", (2, 8))])
def test_tensors_of_other_inner_extents_are_refused(lib, op, name, shape):
    """Larger, so every read is inside, but rows lie elsewhere; flat ones and a single row are taken as they come."""
    t, more = fitting(op)
    wide = {**t, name: Sized(t[name].dtype, *shape)}
    if name == "q" and op == "window_prefill":
        wide["out"] = wide["q"]
    with pytest.raises(ValueError, match=name):
        seer._check_sizes(op, dims(), block_of(op, wide, more))
    if name != "q" or op == "window_decode":
        seer._check_sizes(op, dims(), block_of(op, {**t, name: Sized(t[name].dtype, math.prod(shape))}, more))
    if name in ("page_table", "lse_out") and op == "window_decode":
        d = dims()
        d.batch = 1
        seer._check_sizes(op, d, block_of(op, wide, more))
