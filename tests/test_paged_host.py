"""Checks of the paged-cache entry points that need no GPU: struct layouts, the rotary plan
against the fp64 reference, and every refusal the host makes before a CUDA call."""
import ctypes
import math
import os
import subprocess

import numpy as np
import pytest

import fourier_basis_attention_b200 as fa
from oracle import paged_oracle as po

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 0x10000  # an aligned address that is never dereferenced


def test_structs_match_header_layout(tmp_path):
    structs = {"fa_paged_shape": fa.fa_paged_shape, "fa_paged_cache": fa.fa_paged_cache,
               "fa_rope_config": fa.fa_rope_config, "fa_rope_plan": fa.fa_rope_plan}
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "fourier_attention.h"', "int main(void) {"]
    want = []
    for name, cls in structs.items():
        lines.append(f'  printf("%zu ", sizeof({name}));')
        want.append(ctypes.sizeof(cls))
        for field, _ in cls._fields_:
            lines.append(f'  printf("%zu ", offsetof({name}, {field}));')
            want.append(getattr(cls, field).offset)
    lines += ["  return 0;", "}"]
    (tmp_path / "layout.c").write_text("\n".join(lines))
    exe = str(tmp_path / "layout")
    subprocess.run(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), str(tmp_path / "layout.c"), "-o", exe],
                   check=True)
    out = subprocess.run([exe], capture_output=True, text=True, check=True).stdout
    assert [int(x) for x in out.split()] == want


@pytest.mark.parametrize("kw", [
    dict(), dict(base=500000.0), dict(scaling="linear", factor=4.0), dict(scaling="ntk", factor=8.0),
    dict(scaling="bands", base=500000.0, factor=8.0, low=1.0, high=4.0, original_len=8192),
    dict(scaling="yarn", factor=16.0, low=1.0, high=32.0, original_len=4096),
    dict(scaling="yarn", factor=2.0, low=1.0, high=32.0, original_len=7)], ids=str)
@pytest.mark.parametrize("rot", [2, 6, 64, 128])
def test_rope_plan_matches_reference(kw, rot):
    plan = fa.fa_rope_init(rot_dim=rot, **kw)
    f, m = po.rope_frequencies(rot, **kw)
    turns = np.array([plan.turns[i] for i in range(rot // 2)], dtype=np.float64) / 2.0 ** 64
    # pow, log and a handful of products in fp64 on both sides; 2^-64 turns of truncation
    assert (np.abs(turns - f / (2 * math.pi)) <= 32 * 2.0 ** -53 * f + 2.0 ** -64).all()
    assert abs(plan.magnitude - m) <= 2.0 ** -24 * m
    assert all(plan.turns[i] == 0 for i in range(rot // 2, 64))
    assert fa.fa_rope_init(rot_dim=rot, magnitude=0.5, **kw).magnitude == 0.5


@pytest.mark.parametrize("kw", [
    dict(rot_dim=0), dict(rot_dim=7), dict(rot_dim=130), dict(rot_dim=-2), dict(base=1.0), dict(base=math.nan),
    dict(base=math.inf), dict(factor=0.5), dict(factor=math.nan), dict(magnitude=-1.0), dict(magnitude=math.inf),
    dict(scaling="other"), dict(scaling="bands"), dict(scaling="bands", original_len=10, low=4.0, high=4.0),
    dict(scaling="yarn", original_len=10, low=0.0), dict(scaling="yarn", original_len=10, high=math.inf)], ids=str)
def test_rope_init_refusals(kw):
    with pytest.raises(fa.FaError) as e:
        fa.fa_rope_init(**kw)
    assert e.value.code == fa.FA_ERR_INVALID


def refused(code, name, *args):
    r = getattr(fa.LIB, name)(*args)
    assert r == code, (r, fa.fa_last_error())
    return fa.fa_last_error()


def rope_args(**kw):
    a = dict(rope=fa.fa_rope_init(), B=2, T=3, H=4, pos=P, x=P, xs=(1536, 512, 128), y=P + 65536,
             ys=(1536, 512, 128), dtype=fa.FA_F32, transpose=0)
    a.update(kw)
    three = lambda s: None if s is None else (ctypes.c_int64 * 3)(*s)  # noqa: E731
    return (a["rope"], a["B"], a["T"], a["H"], a["pos"], a["x"], three(a["xs"]), a["y"], three(a["ys"]),
            a["dtype"], a["transpose"], None)


def edited_plan(**kw):
    plan = fa.fa_rope_init()
    for k, v in kw.items():
        setattr(plan, k, v)
    return plan


@pytest.mark.parametrize("kw,code", [
    (dict(rope=None), 1), (dict(rope=edited_plan(rot_dim=256)), 1), (dict(rope=edited_plan(rot_dim=3)), 1),
    (dict(rope=edited_plan(interleaved=2)), 1), (dict(rope=edited_plan(magnitude=math.nan)), 1),
    (dict(B=-1), 1), (dict(H=-1), 1), (dict(dtype=2), 1), (dict(transpose=2), 1),
    (dict(B=1 << 16, T=1 << 16), 2), (dict(H=1 << 21), 2),
    (dict(pos=None), 1), (dict(pos=P + 2), 1), (dict(x=None), 1), (dict(x=P + 8), 1), (dict(y=P + 4), 1),
    (dict(xs=None), 1), (dict(xs=(1536, 512, 130)), 1), (dict(xs=(-1536, 512, 128)), 1),
    (dict(ys=(1536, 512, 64)), 1), (dict(ys=(0, 512, 128)), 1), (dict(ys=(1536, 384, 128)), 1),
    (dict(ys=(128, 256, 768), dtype=fa.FA_F32, B=3), 1),
    (dict(y=P, ys=(1536, 128, 384)), 1),
    (dict(xs=(1536, 512, 132), dtype=fa.FA_BF16), 1)], ids=str)
def test_rope_refusals(kw, code):
    refused(code, "fa_rope", *rope_args(**kw))


@pytest.mark.parametrize("kw", [dict(B=0), dict(T=0), dict(H=0, x=None, y=None, pos=None)], ids=str)
def test_rope_without_rows_is_a_no_op(kw):
    assert fa.LIB.fa_rope(*rope_args(**kw)) == fa.FA_OK


SHAPE = dict(B=2, Hq=8, Hkv=2, D=128, page_size=16, num_pages=40, max_pages=20, total_q=30, max_q=20, max_kv=320)
CACHE = dict(K=P, V=P, page_table=P, q_start=P, kv_len=P)


def shape_of(**kw):
    return fa.fa_paged_shape(**{**SHAPE, **kw})


def cache_of(**kw):
    return fa.fa_paged_cache(**{**CACHE, **kw})


BAD_SHAPES = [(dict(D=64), 2), (dict(B=-1), 1), (dict(B=65536), 2), (dict(Hkv=0), 1), (dict(Hq=9), 1), (dict(Hq=0), 1),
              (dict(Hq=2048), 2), (dict(page_size=0), 1), (dict(num_pages=0), 1), (dict(max_kv=321), 1),
              (dict(max_kv=-1), 1), (dict(total_q=-1), 1), (dict(max_q=-1), 1), (dict(max_pages=-1), 1),
              (dict(num_pages=1 << 27), 2), (dict(total_q=1 << 28), 2),
              (dict(max_pages=1 << 27, max_kv=1 << 30), 2)]
BAD_CACHES = [dict(K=None), dict(K=P + 8), dict(page_table=None), dict(page_table=P + 2), dict(q_start=None),
              dict(kv_len=None), dict(kv_len=P + 1)]


def append_args(shape=None, cache=None, **kw):
    a = dict(rope=None, pos=None, q=None, qs=0, qo=None, qos=0, k=P, ks=256, v=P, vs=256)
    a.update(kw)
    return (shape if shape is not None else shape_of(), cache if cache is not None else cache_of(), a["rope"],
            a["pos"], a["q"], a["qs"], a["qo"], a["qos"], a["k"], a["ks"], a["v"], a["vs"], None)


def attend_args(shape=None, cache=None, **kw):
    a = dict(q=P, qs=1024, scale=0.0, window=0, out=2 * P, os=1024, lse=P, ws=P, bytes=1 << 40)
    a.update(kw)
    return (shape if shape is not None else shape_of(), cache if cache is not None else cache_of(), a["q"], a["qs"],
            a["scale"], a["window"], a["out"], a["os"], a["lse"], a["ws"], a["bytes"], None)


def weights_args(shape=None, cache=None, **kw):
    a = dict(q=P, qs=1024, scale=0.0, window=0, lse=P, w=P, ld=320)
    a.update(kw)
    return (shape if shape is not None else shape_of(), cache if cache is not None else cache_of(), a["q"], a["qs"],
            a["scale"], a["window"], a["lse"], a["w"], a["ld"], None)


def evict_args(shape=None, cache=None, **kw):
    a = dict(w=P, ld=320, keep=100, sink=4, recent=10, ds=shape_of(max_kv=112, max_pages=7),  # weights: 2 x 2 x 320 floats at P
             dc=cache_of(K=2 * P, V=2 * P, q_start=None, kv_len=None), dw=P + 65536, dld=100, index=P, n=P + 64, ws=None,
             bytes=0)
    a.update(kw)
    return (shape if shape is not None else shape_of(), cache if cache is not None else cache_of(), a["w"], a["ld"],
            a["keep"], a["sink"], a["recent"], a["ds"], a["dc"], a["dw"], a["dld"], a["index"], a["n"], a["ws"],
            a["bytes"], None)


CALLS = {"fa_paged_append": append_args, "fa_paged_attend": attend_args, "fa_paged_weights": weights_args,
         "fa_evict": evict_args}


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("kw,code", BAD_SHAPES, ids=str)
def test_bad_shapes(name, kw, code):
    refused(code, name, *CALLS[name](shape=shape_of(**kw)))


@pytest.mark.parametrize("name", CALLS)
def test_null_structs(name):
    args = CALLS[name]()
    assert "shape is NULL" in refused(1, name, None, *args[1:])
    assert "cache is NULL" in refused(1, name, args[0], None, *args[2:])


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("kw", BAD_CACHES, ids=str)
def test_bad_caches(name, kw):
    if name == "fa_evict" and "q_start" in kw:
        pytest.skip("not read by fa_evict")
    refused(1, name, *CALLS[name](cache=cache_of(**kw)))


@pytest.mark.parametrize("name,kw,code", [
    ("fa_paged_append", dict(k=None), 1), ("fa_paged_append", dict(v=P + 2), 1), ("fa_paged_append", dict(ks=248), 1),
    ("fa_paged_append", dict(vs=260), 1), ("fa_paged_append", dict(q=P, qs=1024, qo=P, qos=1024), 1),
    ("fa_paged_append", dict(pos=P), 1), ("fa_paged_append", dict(rope=fa.fa_rope_init(), q=P, qs=1024), 1),
    ("fa_paged_append", dict(rope=fa.fa_rope_init(), q=P, qs=1024, qo=P, qos=2048), 1),
    ("fa_paged_append", dict(rope=fa.fa_rope_init(), q=P, qs=512, qo=2 * P, qos=1024), 1),
    ("fa_paged_append", dict(rope=fa.fa_rope_init(), pos=P + 1), 1),
    ("fa_paged_append", dict(rope=edited_plan(rot_dim=130)), 1),
    ("fa_paged_attend", dict(q=None), 1), ("fa_paged_attend", dict(out=None), 1), ("fa_paged_attend", dict(qs=1016), 1),
    ("fa_paged_attend", dict(os=1028), 1), ("fa_paged_attend", dict(lse=P + 2), 1),
    ("fa_paged_attend", dict(scale=-1.0), 1), ("fa_paged_attend", dict(scale=math.nan), 1),
    ("fa_paged_attend", dict(scale=math.inf), 1), ("fa_paged_attend", dict(scale=1e-30), 2),
    ("fa_paged_weights", dict(scale=1e30), 2), ("fa_paged_attend", dict(window=-1), 1),
    ("fa_paged_attend", dict(shape=shape_of(page_size=20, max_kv=300)), 2),
    ("fa_paged_weights", dict(q=P + 8), 1), ("fa_paged_weights", dict(lse=None), 1),
    ("fa_paged_weights", dict(w=None), 1), ("fa_paged_weights", dict(ld=319), 1),
    ("fa_paged_weights", dict(window=-5), 1), ("fa_paged_weights", dict(scale=-0.5), 1),
    ("fa_paged_weights", dict(shape=shape_of(page_size=24, max_kv=300)), 2),
    ("fa_evict", dict(w=None), 1), ("fa_evict", dict(ld=319), 1), ("fa_evict", dict(keep=0, sink=0, recent=0), 1),
    ("fa_evict", dict(sink=-1), 1), ("fa_evict", dict(recent=-1), 1), ("fa_evict", dict(sink=60, recent=41), 1),
    ("fa_evict", dict(sink=2 ** 31 - 1, recent=2 ** 31 - 1), 1), ("fa_evict", dict(keep=113, dld=113), 1),
    ("fa_evict", dict(ds=shape_of(B=1)), 1), ("fa_evict", dict(ds=shape_of(Hq=8, Hkv=4)), 1),
    ("fa_evict", dict(ds=shape_of(num_pages=0)), 1), ("fa_evict", dict(dc=cache_of(page_table=None)), 1),
    ("fa_evict", dict(dc=cache_of(V=P + 8)), 1), ("fa_evict", dict(dw=P), 1), ("fa_evict", dict(dld=99), 1),
    ("fa_evict", dict(index=None), 1), ("fa_evict", dict(n=None), 1), ("fa_evict", dict(n=P), 1), ("fa_evict", dict(n=P + 4), 1), ("fa_evict", dict(dw=P + 2400), 1),
    ("fa_paged_attend", dict(out=P), 1)], ids=str)
def test_argument_refusals(name, kw, code):
    refused(code, name, *CALLS[name](**kw))


@pytest.mark.parametrize("kw", [dict(B=0), dict(total_q=0)], ids=str)
@pytest.mark.parametrize("name", ["fa_paged_append", "fa_paged_attend", "fa_paged_weights"])
def test_calls_without_rows_launch_nothing(name, kw):
    assert getattr(fa.LIB, name)(*CALLS[name](shape=shape_of(**kw))) == fa.FA_OK


def test_workspace_sizes_of_refused_shapes_are_zero():
    assert fa.LIB.fa_paged_attend_workspace_size(shape_of(D=64), 0) == 0
    assert fa.LIB.fa_paged_attend_workspace_size(shape_of(), -1) == 0
    assert fa.LIB.fa_paged_attend_workspace_size(None, 0) == 0
    assert fa.LIB.fa_evict_workspace_size(shape_of(), 0) == 0


def test_binding_refuses_host_tensors_types_and_shapes():
    import torch
    K = torch.zeros(4, 2, 16, 128, dtype=torch.bfloat16)
    table = torch.zeros(1, 2, dtype=torch.int32)
    for args in [(K, K, table), (K.float(), K, table), (K[..., :64], K, table), (K, K, table.long()), ([], K, table)]:
        with pytest.raises(fa.FaError) as e:
            fa.PagedCache(*args)
        assert e.value.code == fa.FA_ERR_INVALID
    x = torch.zeros(1, 2, 3, 128)
    pos = torch.zeros(1, 2, dtype=torch.int32)
    for args in [(x, pos, x), (x.half(), pos, x.half()), (x[0], pos, x[0]), (x[..., :64], pos, x[..., :64]),
                 (x, pos, x.bfloat16())]:
        with pytest.raises(fa.FaError) as e:
            fa.fa_rope(fa.fa_rope_init(), *args)
        assert e.value.code == fa.FA_ERR_INVALID


# --------------------------------------------------------------------------- the reference itself

def test_reference_attention_by_hand():
    """Two keys, one hidden: weights by the softmax of two scores; a window of one sees itself."""
    K = np.zeros((1, 1, 16, 128))
    V = np.zeros_like(K)
    K[0, 0, 0, 0], K[0, 0, 1, 0], V[0, 0, 0, 5], V[0, 0, 1, 5] = 1.0, 2.0, 10.0, 20.0
    q = np.zeros((2, 1, 128))
    q[:, 0, 0] = 1.0
    table = np.zeros((1, 1), dtype=int)
    out, _, lse, _, w = po.attend(q, K, V, table, [0, 2], [2], scale=1.0)
    e = math.exp(1.0) / (math.exp(1.0) + math.exp(2.0))
    assert np.isclose(out[0, 0, 5], 10.0) and np.isclose(out[1, 0, 5], 10 * e + 20 * (1 - e))
    assert np.allclose(lse[:, 0], [1.0, math.log(math.exp(1) + math.exp(2))])
    assert np.allclose(w[0, 0], [1 + e, 1 - e])
    out, _, lse, _, w = po.attend(q, K, V, table, [0, 2], [2], window=1, scale=1.0)
    assert np.allclose(out[:, 0, 5], [10.0, 20.0]) and np.allclose(lse[:, 0], [1.0, 2.0])
    out, _, lse, _, _ = po.attend(q, K, V, table, [0, 2], [1], scale=1.0)  # the first token is not cached
    assert out[0, 0].any() == 0 and np.isneginf(lse[0, 0]) and np.isclose(out[1, 0, 5], 10.0)


def test_reference_rope_is_a_rotation():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((2, 3, 128))
    f, m = po.rope_frequencies(96)
    y = po.rope(x, [7, 8], f, m)
    assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1)) and np.array_equal(y[..., 96:], x[..., 96:])
    assert np.allclose(po.rope(y, [7, 8], f, m, transpose=True), x)
    # scores depend on distances alone
    a, b = rng.standard_normal((2, 1, 1, 128))
    s = [(po.rope(a, [p], f, m) * po.rope(b, [p + 5], f, m)).sum() for p in (0, 90)]
    assert np.isclose(*s)


def test_reference_eviction_by_hand():
    w = np.array([[[5, 1, 9, 1, 7, 1, 1, 2]]], dtype=np.float32)
    assert po.evict_index(w, [8], 4, 1, 1)[0, 0].tolist() == [0, 2, 4, 7]
    assert po.evict_index(w, [8], 7, 0, 0)[0, 0].tolist() == [0, 1, 2, 3, 4, 5, 7]
    assert po.evict_index(w, [3], 4, 1, 1)[0, 0].tolist() == [0, 1, 2, -1]
