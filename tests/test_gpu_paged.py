"""GPU parity of the paged-cache operators against the fp64 reference.

Tolerances (u16 = 2^-8, u32 = 2^-24: half steps of bf16 and fp32; A: the largest sum of
|scale q_d k_d| of a row's scores):
- a score is an fp32 sum of 128 exact products, off by at most 129 u32 A; the exponential of it
  and the log-sum-exp are off by that, by the rounding of their argument (at most 4 u32 A) and by
  2 u32 of the approximate exp2; the sums of n terms in fp32 by at most n u32.
- attention rounds each weight to bf16 (u16 of sum p |v|) and the output once (u16 of |o|).
- rotation: cos and sin are off by 2 u32 + pi 2^-26, products and the sum by u32 each.
"""
import ctypes
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import fourier_basis_attention_b200 as fa
from oracle import paged_oracle as po

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
D = 128
U16, U32 = 2.0 ** -8, 2.0 ** -24
BF = torch.bfloat16


def make(seqs, Hq, Hkv, page, seed=0, spare_rows=0, q_scale=1.5, max_q=None, max_kv=None, fill=float("nan")):
    """Pools (every slot no sequence uses holds `fill`), shuffled pages, ragged rows; spare_rows
    rows lie behind the last sequence."""
    gen = torch.Generator().manual_seed(seed)
    qs, kvs = [n for n, _ in seqs], [kv for _, kv in seqs]
    B = len(seqs)
    max_kv = max(kvs) if max_kv is None else max_kv
    max_pages = max(1, -(-max_kv // page))
    need = [-(-kv // page) for kv in kvs]
    pages = sum(need) + 2
    order = torch.randperm(pages, generator=gen).to(torch.int32)
    table = torch.full((B, max_pages), -7, dtype=torch.int32)  # unused entries are out of range
    K = torch.full((pages, Hkv, page, D), fill)
    V = K.clone()
    at = 0
    for b, m in enumerate(need):
        table[b, :m] = order[at:at + m]
        at += m
        for i in range(m):
            n = min(page, kvs[b] - i * page)
            K[table[b, i], :, :n] = torch.randn(Hkv, n, D, generator=gen)
            V[table[b, i], :, :n] = torch.randn(Hkv, n, D, generator=gen) + 0.5
    total = sum(qs) + spare_rows
    q = q_scale * torch.randn(total, Hq, D, generator=gen)
    st = dict(K=K.to(BF).cuda(), V=V.to(BF).cuda(), table=table.cuda(), q=q.to(BF).cuda(),
              q_start=torch.tensor(np.cumsum([0] + qs), dtype=torch.int32).cuda(),
              kv_len=torch.tensor(kvs, dtype=torch.int32).cuda(), used=sum(qs), total=total)
    st["cache"] = fa.PagedCache(st["K"], st["V"], st["table"])
    st["batch"] = fa.PagedBatch(st["cache"], Hq, st["q_start"], st["kv_len"], total_q=total,
                                max_q=max(qs) if max_q is None else max_q, max_kv=max_kv)
    return st


def reference(st, window=0, scale=0.0, q=None):
    n = lambda t: t.cpu().double().numpy()  # noqa: E731
    return po.attend(n(st["q"] if q is None else q), n(st["K"]), n(st["V"]), st["table"].cpu().numpy(),
                     st["q_start"].cpu().numpy(), st["kv_len"].cpu().numpy(), window, scale)


def attend(st, window=0, scale=0.0, lse=True, out=None, q=None, workspace=None):
    batch = st["batch"]
    shape = st["q"].shape
    out = torch.full(shape, 3.0, dtype=BF, device="cuda") if out is None else out
    lse = torch.full(shape[:2], 3.0, dtype=torch.float32, device="cuda") if lse else None
    size = fa.fa_paged_attend_workspace_size(batch, window)
    if workspace is None and size:
        workspace = torch.full((size // 4,), float("nan"), device="cuda")
    fa.fa_paged_attend(batch, st["q"] if q is None else q, out, workspace, lse=lse, window=window,
                       scale=scale)
    return out, lse


def check_attend(st, out, lse, ref):
    o, oa, l, size, w = ref
    n, keys = st["used"], w.shape[2]
    got = out.cpu().double().numpy()
    assert np.array_equal(got[n:], np.full_like(got[n:], 3.0))  # rows behind the last sequence
    p_err = (2 * 133 * U32 * size + (4 + keys) * U32)[..., None]
    tol = (U16 + 2 * p_err) * oa + U16 * np.abs(o) + 1e-30
    bad = ~(np.abs(got - o) <= tol)[:n]
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:3], np.abs(got - o)[:n].max())
    if lse is None:
        return
    got = lse.cpu().double().numpy()
    assert np.array_equal(got[n:], np.full_like(got[n:], 3.0))
    empty = np.isneginf(l)
    assert np.array_equal(np.isneginf(got), empty) and not got[:n][empty[:n]].size or \
        np.isneginf(got[:n][empty[:n]]).all()
    live = ~empty[:n]
    err = np.abs(got[:n][live] - l[:n][live])
    bound = (133 * U32 * size + (8 + keys) * U32 + 4 * U32 * np.abs(np.where(empty, 0, l)))[:n][live]
    assert (err <= bound).all(), (err.max(), bound.min())


CASES = {
    "one_key": ([(1, 1)], 4, 1, 16, 0),
    "tiny_mixed": ([(1, 17), (3, 16), (0, 50), (5, 5), (2, 31)], 4, 2, 16, 0),
    "padded": ([(4, 2), (1, 0), (0, 0), (3, 3), (20, 5)], 8, 2, 16, 0),
    "decode_long_split": ([(1, 3001), (1, 15), (1, 700)], 8, 2, 64, 0),
    "decode_no_sharing": ([(1, 513), (1, 1), (1, 255)], 4, 4, 32, 0),
    "decode_g7": ([(1, 1000), (2, 77), (3, 129)], 7, 1, 48, 0),
    "decode_g5": ([(1, 100), (4, 1029)], 30, 6, 16, 0),
    "decode_g32": ([(1, 600), (2, 90)], 32, 1, 16, 0),
    "chunk": ([(130, 700)], 8, 2, 64, 0),
    "prompt": ([(257, 257)], 4, 1, 128, 0),
    "prompt_pages_80": ([(300, 411), (129, 129)], 4, 4, 80, 0),
    "prompt_page_256": ([(200, 1000)], 2, 1, 256, 0),
    "chunk_long_few_rows": ([(33, 4099)], 4, 1, 16, 0),
    "chunk_g3": ([(100, 350), (1, 900), (65, 65)], 6, 2, 32, 0),
    "window_1": ([(1, 40), (30, 60)], 4, 2, 16, 1),
    "window_5": ([(1, 300), (100, 200), (9, 9)], 4, 1, 16, 5),
    "window_64": ([(300, 900), (1, 2000)], 4, 2, 64, 64),
    "window_700": ([(250, 2100), (1, 2100), (3, 100)], 8, 2, 32, 700),
    "window_wide": ([(50, 90), (1, 33)], 4, 4, 16, 100000),
    "window_int_max": ([(50, 90), (1, 33)], 4, 4, 16, 2 ** 31 - 1),
    "many_short": ([(1 + i % 3, 1 + (37 * i) % 90) for i in range(40)], 4, 2, 16, 0),
    "not_cached": ([(40, 0), (30, 10), (17, 3), (1, 0)], 8, 2, 16, 0),
    "not_cached_window": ([(60, 0), (50, 20), (5, 2)], 8, 2, 16, 7),
    "g100": ([(1, 300), (9, 200)], 100, 1, 16, 0),
    "g128": ([(1, 60), (7, 200), (2, 1100)], 128, 1, 16, 0),
    "g200": ([(1, 100), (3, 40)], 200, 1, 16, 9),
    "many_chunks": ([(5 + i % 40, 60 + (91 * i) % 300) for i in range(70)], 4, 1, 16, 0),
    "many_items": ([(9 + i % 30 if i % 3 else 1, 100 + (91 * i) % 600) for i in range(60)], 16, 4, 16, 0),
    "many_items_window": ([(9 + i % 30 if i % 3 else 1, 100 + (91 * i) % 600) for i in range(60)], 16, 4, 32, 150),
    # more than 1280 keys: two tiles a CTA
    "pair_prompt": ([(1400, 1400)], 4, 1, 128, 0),
    "pair_window": ([(300, 3001), (1, 2100), (257, 1300)], 8, 2, 64, 1300),
    "pair_g3": ([(200, 2000), (90, 90), (1, 1400), (43, 1290)], 6, 2, 16, 0),
    "pair_no_sharing": ([(300, 1500), (129, 129)], 4, 4, 80, 0),
    "pair_not_cached": ([(300, 100), (150, 2000), (20, 10), (70, 0)], 8, 2, 16, 0),
    "pair_many": ([(33 + i % 50, 300 + (211 * i) % 1200) for i in range(45)], 8, 2, 16, 0),
    "one_tile_long": ([(30, 2500), (32, 4000), (5, 1300)], 8, 2, 32, 0),
    "decode_over_4096": ([(1, 9001), (2, 4200), (1, 5)], 8, 2, 64, 0),
    "decode_4096": ([(1, 4096), (1, 1), (2, 513), (0, 9)], 8, 2, 128, 0),
    "decode_4096_window": ([(1, 4096), (3, 700), (1, 1)], 4, 1, 64, 600),
    "decode_window_600": ([(1, 9000), (2, 8111), (1, 5), (2, 602)], 8, 2, 64, 600),
    "decode_window_100": ([(1, 7003), (3, 500), (1, 100), (2, 101)], 4, 1, 16, 100),
    "decode_window_1200": ([(1, 5003), (1, 1201), (1, 9)], 16, 8, 16, 1200),
    "mixed_window": ([(1, 6000), (100, 3000), (2, 1300), (33, 700)], 8, 2, 32, 300),
    "mixed": ([(1, 1800), (140, 900), (1, 3), (260, 1500), (2, 1200)], 16, 4, 64, 0),
}


@pytest.mark.parametrize("name", CASES)
def test_attend(name):
    seqs, Hq, Hkv, page, window = CASES[name]
    st = make(seqs, Hq, Hkv, page, seed=len(name), spare_rows=3)
    out, lse = attend(st, window)
    fa.fa_device_status()
    check_attend(st, out, lse, reference(st, window))


@pytest.mark.parametrize("name", CASES)
def test_weights(name):
    seqs, Hq, Hkv, page, window = CASES[name]
    st = make(seqs, Hq, Hkv, page, seed=len(name) + 1, spare_rows=2)
    _, _, l, size, w = reference(st, window)
    st["V"].fill_(float("nan"))  # the values are not read
    lse = torch.tensor(np.where(np.isnan(l), 0.0, l), dtype=torch.float32, device="cuda")
    B, keys = len(seqs), w.shape[2]
    ld = keys + 5
    acc = torch.rand(B, Hkv, ld, device="cuda")
    before = acc.clone()
    fa.fa_paged_weights(st["batch"], st["q"], lse, acc, window=window)
    first = acc.clone()
    fa.fa_device_status()
    got = (acc.double() - before.double()).cpu().numpy()
    for b, (n, kv) in enumerate(seqs):
        assert torch.equal(acc[b, :, kv:], before[b, :, kv:])
        rows = n * (Hq // Hkv)
        top = np.nanmax(size) if size.size else 0.0
        tol = w[b, :, :kv] * (2 * 137 * U32 * top + (8 + rows) * U32) + 2 * U32 * (1 + w[b, :, :kv]) + rows * 1e-37
        assert (np.abs(got[b, :, :kv] - w[b, :, :kv]) <= tol).all(), b
    acc.copy_(before)
    fa.fa_paged_weights(st["batch"], st["q"], lse, acc, window=window)
    assert torch.equal(acc, first)  # no atomics


@pytest.mark.parametrize("row", [64, 65, 70, 71, 127, 199])
def test_weights_of_a_nan_query(row):
    # one head a KV head: row = token, 256 rows in two blocks; the keys that it sees get NaN
    st = make([(256, 1000)], 2, 2, 32, seed=row)
    st["q"][row, 0] = float("nan")
    _, lse = attend(st)
    acc = torch.zeros(1, 2, 1000, device="cuda")
    fa.fa_paged_weights(st["batch"], st["q"], lse, acc)
    fa.fa_device_status()
    seen = 1000 - 256 + row + 1
    assert torch.isnan(acc[0, 0, :seen]).all()
    assert torch.isfinite(acc[0, 0, seen:]).all() and torch.isfinite(acc[0, 1]).all()


@pytest.mark.parametrize("seqs", [[(1, 900), (1, 3)], [(200, 600)], [(200, 1600)]],
                         ids=["decode", "chunk", "pair"])
@pytest.mark.parametrize("scale", [0.011, 4.0])
def test_attend_scale_and_large_scores(seqs, scale):
    st = make(seqs, 8, 2, 32, seed=5, q_scale=4.0)
    out, lse = attend(st, scale=scale)
    fa.fa_device_status()
    check_attend(st, out, lse, reference(st, scale=float(np.float32(scale))))


@pytest.mark.parametrize("seqs", [[(1, 700), (2, 40)], [(150, 400), (70, 70)], [(150, 1400), (70, 70)]],
                         ids=["decode", "chunk", "pair"])
def test_attend_strides_and_alias_free_rows(seqs):
    """q and out as slices of wider rows; no lse."""
    st = make(seqs, 8, 2, 16, seed=6)
    wide = torch.zeros(st["total"], 13, D, dtype=BF, device="cuda")
    wide[:, 3:11] = st["q"]
    dst = torch.full((st["total"], 11, D), 3.0, dtype=BF, device="cuda")
    out, _ = attend(st, lse=False, q=wide[:, 3:11], out=dst[:, 1:9])
    fa.fa_device_status()
    check_attend(st, out, None, reference(st))
    assert (dst[:, 0] == 3.0).all() and (dst[:, 9:] == 3.0).all()


@pytest.mark.parametrize("seqs,window", [([(1, 3000)], 100), ([(150, 2000)], 333)],
                         ids=["decode", "chunk"])
def test_nan_before_the_window_and_behind_the_end(seqs, window):
    st = make(seqs, 4, 1, 64, seed=7)
    n, kv = seqs[0]
    first = kv - n - window + 1
    for j in range(first):
        pg = st["table"][0, j // 64]
        st["K"][pg, :, j % 64] = float("nan")
        st["V"][pg, :, j % 64] = float("nan")
    out, lse = attend(st, window)
    fa.fa_device_status()
    check_attend(st, out, lse, reference(st, window))


def test_masked_row_and_nan_query():
    """A NaN query spoils its own row and no other."""
    st = make([(40, 100), (1, 50)], 4, 2, 16, seed=8)
    ref = reference(st)
    st["q"][7, 1] = float("nan")
    out, lse = attend(st)
    fa.fa_device_status()
    assert torch.isnan(out[7, 1].float()).all() and torch.isnan(lse[7, 1])
    out[7, 1], lse[7, 1] = torch.tensor(ref[0][7, 1]).to(BF), float(ref[2][7, 1])
    check_attend(st, out, lse, ref)


@pytest.mark.parametrize("seqs", [[(1, 2500), (1, 20)], [(200, 1500), (1, 900)], [(200, 1200), (1, 900)]],
                         ids=["decode", "mixed", "short"])
def test_repeated_calls_give_identical_bits(seqs):
    st = make(seqs, 8, 2, 32, seed=9)
    a = attend(st)
    b = attend(st)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("seqs,window", [([(1, 300), (1, 77)], 0), ([(150, 400), (1, 90)], 0), ([(1, 900)], 50)],
                         ids=["decode", "mixed", "window"])
def test_calls_in_a_row_keep_the_order_of_the_stream(seqs, window):
    """Each call's inputs are written by the kernel before it and overwritten by the one behind it;
    the same calls with waits between them give the same bits."""
    st = make(seqs, 8, 2, 16, seed=12)
    kvs, total, B = [kv for _, kv in seqs], st["total"], len(seqs)
    gen = torch.Generator().manual_seed(3)
    N = 20
    qs, ks = (torch.randn(N, total, h, D, generator=gen).to(BF).cuda() for h in (8, 2))
    rope = fa.fa_rope_init()
    K0, V0 = st["K"].clone(), st["V"].clone()

    def run(wait):
        st["K"].copy_(K0)
        st["V"].copy_(V0)
        q, k = torch.empty_like(qs[0]), torch.empty_like(ks[0])
        lse, out = torch.empty(total, 8, device="cuda"), torch.empty_like(q)
        w = torch.empty(B, 2, max(kvs), device="cuda")
        index, length = torch.empty(B, 2, 40, dtype=torch.int32, device="cuda"), torch.empty(B, dtype=torch.int32, device="cuda")
        dst = fa.PagedCache.dense(*torch.zeros(2, B, 2, 40, D, dtype=BF, device="cuda"))
        ws = torch.empty(fa.fa_paged_attend_workspace_size(st["batch"], window) + 16, dtype=torch.uint8, device="cuda")
        evict_ws = torch.empty(fa.fa_evict_workspace_size(st["batch"], 40) + 16, dtype=torch.uint8, device="cuda")
        kept = []
        torch.cuda.synchronize()
        for i in range(N):
            steps = [lambda: (q.copy_(qs[i]), k.copy_(ks[i]), w.zero_()),
                     lambda: fa.fa_paged_append(st["batch"], k, k, q=q, q_out=q, rope=rope),
                     lambda: fa.fa_paged_attend(st["batch"], q, out, ws, lse=lse, window=window),
                     lambda: fa.fa_paged_weights(st["batch"], q, lse, w, window=window),
                     lambda: fa.fa_evict(st["batch"], w, 40, dst, index, length, evict_ws, sink=2, recent=3),
                     lambda: kept.append([t.clone() for t in (q, out, lse, w, index, dst.K, dst.V)]),
                     lambda: (q.fill_(float("nan")), k.fill_(float("nan")), out.zero_(), lse.zero_(), index.zero_())]
            for step in steps:
                step()
                if wait:
                    torch.cuda.synchronize()
        fa.fa_device_status()
        return kept

    for a, b in zip(run(True), run(False)):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("seqs", [[(1, 300), (1, 77)], [(150, 400), (1, 90)]], ids=["decode", "mixed"])
def test_capture_behind_memsets_copies_and_other_streams(seqs):
    """Calls whose predecessors in a graph are a memset, a copy, or kernels of two streams."""
    st = make(seqs, 8, 2, 16, seed=13)
    total, B, longest = st["total"], len(seqs), max(kv for _, kv in seqs)
    q, host = torch.zeros_like(st["q"]), st["q"].cpu().pin_memory()
    out, other, lse = torch.zeros_like(q), torch.zeros_like(q), torch.zeros(total, 8, device="cuda")
    other_lse = torch.zeros_like(lse)
    w = torch.ones(B, 2, longest, device="cuda")
    size = fa.fa_paged_attend_workspace_size(st["batch"]) + 16
    ws = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(2)]
    main, side = torch.cuda.Stream(), torch.cuda.Stream()

    def step():
        q.copy_(host, non_blocking=True)
        fork = torch.cuda.Event()
        fork.record(main)
        side.wait_event(fork)
        fa.fa_paged_attend(st["batch"], q, out, ws[0], lse=lse)
        with torch.cuda.stream(side):
            fa.fa_paged_attend(st["batch"], q, other, ws[1], lse=other_lse)
            join = torch.cuda.Event()
            join.record(side)
        main.wait_event(join)
        w.zero_()
        fa.fa_paged_weights(st["batch"], q, other_lse, w)
        w.mul_(2.0)
        fa.fa_paged_weights(st["batch"], q, lse, w)

    with torch.cuda.stream(main):
        step()
        torch.cuda.synchronize()
        expect = [t.clone() for t in (out, other, lse, other_lse, w)]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=main):
            step()
        for t in (q, out, other, lse, other_lse, w):
            t.fill_(7.0)
        for _ in range(5):
            graph.replay()
        torch.cuda.synchronize()
    fa.fa_device_status()
    assert torch.equal(expect[0], expect[1])
    for t, e in zip((out, other, lse, other_lse, w), expect):
        assert torch.equal(t, e)
    check_attend(st, out, lse, reference(st))


def test_captured_graph_replays_with_new_lengths():
    """A graph captured at one set of lengths (all sequences short) gives those of another."""
    seqs = [(3, 900), (1, 33), (120, 500)]
    st = make(seqs, 8, 2, 32, seed=10, max_q=200, max_kv=1000)
    real = st["q_start"].clone(), st["kv_len"].clone()
    out = torch.full(st["q"].shape, 3.0, dtype=BF, device="cuda")
    lse = torch.full(st["q"].shape[:2], 3.0, device="cuda")
    ws = torch.empty(max(1, fa.fa_paged_attend_workspace_size(st["batch"])), dtype=torch.uint8, device="cuda")
    acc = torch.zeros(3, 2, 1000, device="cuda")
    go = lambda: (fa.fa_paged_attend(st["batch"], st["q"], out, ws, lse=lse),  # noqa: E731
                  fa.fa_paged_weights(st["batch"], st["q"], lse, acc))
    go()
    st["q_start"].copy_(torch.tensor([0, 1, 2, 3], dtype=torch.int32))
    st["kv_len"].copy_(torch.tensor([5, 1, 9], dtype=torch.int32))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go()
    st["q_start"].copy_(real[0])
    st["kv_len"].copy_(real[1])
    for t in (out, lse):
        t.fill_(3.0)
    acc.zero_()
    graph.replay()
    fa.fa_device_status()
    ref = reference(st)
    check_attend(st, out, lse, ref)
    for b, (n, kv) in enumerate(seqs):
        w = ref[4][b, :, :kv]
        # lse is the kernel's own: its error counts again
        tol = w * (4 * 137 * U32 * np.nanmax(ref[3]) + (16 + 2 * n * 4 + 2 * kv) * U32) + 1e-30
        assert (np.abs(acc[b, :, :kv].double().cpu().numpy() - w) <= tol).all()
        assert not acc[b, :, kv:].any()


def test_two_streams_at_once():
    sts = [make([(1, 2000), (60, 300)], 8, 2, 32, seed=s) for s in (11, 12)]
    streams = [torch.cuda.Stream() for _ in sts]
    res = []
    torch.cuda.synchronize()
    for st, stream in zip(sts, streams):
        with torch.cuda.stream(stream):
            res.append(attend(st))
    torch.cuda.synchronize()
    for st, (out, lse) in zip(sts, res):
        check_attend(st, out, lse, reference(st))


# --------------------------------------------------------------------------- rotary positions

SCALINGS = {
    "plain": dict(),
    "linear": dict(scaling="linear", factor=4.0),
    "ntk": dict(scaling="ntk", factor=8.0),
    "bands": dict(scaling="bands", base=500000.0, factor=8.0, low=1.0, high=4.0, original_len=8192),
    "yarn": dict(scaling="yarn", factor=16.0, low=1.0, high=32.0, original_len=4096),
}


def check_rope(got, x, pos, rot, kw, interleaved, transpose, bf16):
    f, m = po.rope_frequencies(rot, **kw)
    ref = po.rope(x, pos, f, m, interleaved, transpose)
    n = rot // 2
    ia = np.arange(0, rot, 2) if interleaved else np.arange(n)
    ib = ia + 1 if interleaved else ia + n
    size = np.zeros_like(ref)
    size[..., ia] = size[..., ib] = m * (np.abs(x[..., ia]) + np.abs(x[..., ib]))
    # f itself is exact to 2^-52 relative here and in the reference, the phase to 2^-64 turns
    angle = np.pi * 2.0 ** -26 + 2 * 2.0 ** -52 * np.abs(pos).max(initial=0)
    tol = size * (angle + 6 * U32) + (U16 * np.abs(ref) if bf16 else 0.0) + 1e-37
    assert (np.abs(got - ref) <= tol).all(), np.abs(got - ref).max()
    assert np.array_equal(got[..., rot:], x[..., rot:])


@pytest.mark.parametrize("dtype", [BF, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("rot,interleaved", [(128, False), (128, True), (64, False), (48, True),
                                             (2, False), (6, True), (126, False), (32, False)])
@pytest.mark.parametrize("B,T,H,transpose", [(1, 1, 1, False), (2, 37, 5, True), (3, 900, 2, False)])
def test_rope(dtype, rot, interleaved, B, T, H, transpose):
    kw = list(SCALINGS.values())[(rot + T + interleaved) % len(SCALINGS)]
    rng = np.random.default_rng(rot + T)
    x = torch.tensor(rng.standard_normal((B, H, T, D))).to(dtype).cuda().transpose(1, 2)  # head-major
    pos = torch.tensor(rng.integers(-2 ** 31, 2 ** 31, (B, T)), dtype=torch.int32)
    pos[:, ::3] = torch.tensor(rng.integers(0, 5000, tuple(pos[:, ::3].shape)), dtype=torch.int32)
    out = torch.empty(B, T, H, D, dtype=dtype, device="cuda")
    plan = fa.fa_rope_init(rot_dim=rot, interleaved=interleaved, **kw)
    fa.fa_rope(plan, x, pos.cuda(), out, transpose=transpose)
    fa.fa_device_status()
    check_rope(out.cpu().double().numpy(), x.cpu().double().numpy(), pos.numpy(), rot, kw,
               interleaved, transpose, dtype == BF)


@pytest.mark.parametrize("name", SCALINGS)
def test_rope_in_place_and_back(name):
    """In place; then the transposed map takes the positions out (magnitude m: times m^2)."""
    rng = np.random.default_rng(3)
    x = torch.tensor(rng.standard_normal((2, 50, 3, D)), dtype=torch.float32)
    pos = torch.tensor(rng.integers(0, 2000000, (2, 50)), dtype=torch.int32).cuda()
    plan = fa.fa_rope_init(**SCALINGS[name])
    y = x.cuda()
    fa.fa_rope(plan, y, pos, y)
    check_rope(y.cpu().double().numpy(), x.double().numpy(), pos.cpu().numpy(), D, SCALINGS[name],
               False, False, False)
    fa.fa_rope(plan, y, pos, y, transpose=True)
    _, m = po.rope_frequencies(D, **SCALINGS[name])
    size = np.abs(x.numpy()[..., :64]) + np.abs(x.numpy()[..., 64:])
    err = np.abs(y.cpu().double().numpy() - m * m * x.double().numpy())
    # two rotations, each off by (pi 2^-26 + 6 u32) of |a| + |b|, the first's error rotated again
    assert (err <= m * m * np.tile(size, 2) * 4 * (np.pi * 2.0 ** -26 + 6 * U32)).all()


def test_rope_gradient_matches_differences():
    """The map is linear: <w, R(x + h e) - R(x)> / h of the reference equals the transposed
    call's component."""
    rng = np.random.default_rng(4)
    plan = fa.fa_rope_init(rot_dim=96, interleaved=True, **SCALINGS["yarn"])
    f, m = po.rope_frequencies(96, **SCALINGS["yarn"])
    x, w = rng.standard_normal((2, 1, 3, 2, D))
    pos = rng.integers(0, 100000, (1, 3)).astype(np.int32)
    g = torch.tensor(w, dtype=torch.float32, device="cuda")
    out = torch.empty_like(g)
    fa.fa_rope(plan, g, torch.tensor(pos).cuda(), out, transpose=True)
    for t, h, d in [(0, 0, 0), (1, 1, 51), (2, 0, 95), (1, 0, 96), (2, 1, 127)]:
        e = np.zeros_like(x)
        e[0, t, h, d] = 0.5
        diff = (w * (po.rope(x + e, pos, f, m, True) - po.rope(x, pos, f, m, True))).sum() / 0.5
        assert abs(diff - out[0, t, h, d].item()) <= 2.0 ** -20 * np.abs(w).max()


def test_rope_broadcast_and_padded_strides():
    """x repeats one head (stride 0); out rows lie 136 apart."""
    x = torch.randn(1, 9, 1, D, device="cuda").expand(1, 9, 4, D)
    out = torch.full((1, 9, 4, 136), 7.0, device="cuda")
    pos = torch.arange(9, dtype=torch.int32, device="cuda")[None]
    fa.fa_rope(fa.fa_rope_init(), x, pos, out[..., :D])
    check_rope(out[..., :D].cpu().double().numpy(), x.cpu().double().numpy(), pos.cpu().numpy(), D, {},
               False, False, False)
    assert (out[..., D:] == 7.0).all()


# --------------------------------------------------------------------------- page write

@pytest.mark.parametrize("rotate", ["none", "keys", "both", "in_place", "positions"])
@pytest.mark.parametrize("seqs,page,rot,interleaved", [
    ([(1, 1)], 1, 128, False),
    ([(1, 17), (3, 16), (0, 50), (5, 5), (4, 2), (1, 0)], 16, 128, False),
    ([(130, 700), (1, 40), (33, 33)], 48, 64, True),
    ([(9, 100)] * 300, 7, 6, False)], ids=["one", "padded", "ragged", "many"])
def test_append(rotate, seqs, page, rot, interleaved):
    Hq, Hkv = 6, 2
    st = make(seqs, Hq, Hkv, page, seed=13, spare_rows=2, fill=9.0)
    total = st["total"]
    gen = torch.Generator().manual_seed(1)
    qkv = torch.randn(total, Hq + 2 * Hkv, D, generator=gen).to(BF).cuda()
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    kw = SCALINGS["yarn"]
    plan = fa.fa_rope_init(rot_dim=rot, interleaved=interleaved, **kw)
    pos = torch.cat([torch.arange(kv - n, kv) for n, kv in seqs] + [torch.zeros(2)]).to(torch.int32)
    positions = None
    if rotate == "positions":
        pos = torch.randint(0, 10 ** 6, (total,), generator=gen, dtype=torch.int32)
        positions = pos.cuda()
    K0, V0, q0 = st["K"].clone(), st["V"].clone(), q.cpu().double().numpy()
    k0 = k.cpu().double().numpy()
    q_out = torch.full((total, Hq, D), 3.0, dtype=BF, device="cuda")
    if rotate in ("none", "keys"):
        fa.fa_paged_append(st["batch"], k, v, rope=None if rotate == "none" else plan)
    else:
        if rotate == "in_place":
            q_out = q
        fa.fa_paged_append(st["batch"], k, v, q=q, q_out=q_out, rope=plan, positions=positions)
    fa.fa_device_status()
    n = st["used"]
    f, m = po.rope_frequencies(rot, **kw)
    wantK, wantV = K0.cpu(), V0.cpu()
    tag = torch.zeros(wantK.shape[:3], dtype=torch.bool)
    rows = {}
    t = 0
    for b, (nq, kv) in enumerate(seqs):
        for i in range(nq):
            j = kv - nq + i
            if j >= 0:
                pg = int(st["table"][b, j // page])
                wantV[pg, :, j % page] = v[t].cpu()
                tag[pg, :, j % page] = True
                rows[t] = (pg, j % page)
            t += 1
    assert torch.equal(st["V"].cpu(), wantV)
    assert torch.equal(st["K"].cpu()[~tag], wantK[~tag])
    if rows:
        idx = np.array(list(rows))
        pg, sl = np.array(list(rows.values())).T
        got = st["K"].cpu()[pg, :, sl].double().numpy()
        if rotate == "none":
            assert np.array_equal(got, k0[idx])
        else:
            check_rope(got, k0[idx], pos.numpy()[idx], rot, kw, interleaved, False, True)
    if rotate in ("both", "in_place", "positions"):
        got = q_out.cpu().double().numpy()
        check_rope(got[:n], q0[:n], pos.numpy()[:n], rot, kw, interleaved, False, True)
        assert np.array_equal(got[n:], q0[n:] if rotate == "in_place" else np.full_like(got[n:], 3.0))


# --------------------------------------------------------------------------- eviction

def evict(st, w, keep, sink, recent, dst_page, with_weights=True):
    B, Hkv = st["table"].shape[0], st["K"].shape[1]
    pages = -(-keep // dst_page)
    gen = torch.Generator().manual_seed(2)
    dst_table = torch.randperm(B * pages, generator=gen).to(torch.int32).view(B, pages).cuda()
    dK = torch.full((B * pages, Hkv, dst_page, D), 5.0, dtype=BF, device="cuda")
    dV = torch.full_like(dK, 6.0)
    dst = fa.PagedCache(dK, dV, dst_table)
    index = torch.full((B, Hkv, keep), 77, dtype=torch.int32, device="cuda")
    dst_len = torch.full((B,), 77, dtype=torch.int32, device="cuda")
    dw = torch.full((B, Hkv, keep + 3), 8.0, device="cuda") if with_weights else None
    size = fa.fa_evict_workspace_size(st["batch"], keep)
    ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda") if size else None
    fa.fa_evict(st["batch"], w, keep, dst, index, dst_len, ws, sink=sink, recent=recent, dst_weights=dw)
    fa.fa_device_status()
    return dst_table.cpu().numpy(), dK, dV, index, dst_len, dw


def check_evict(st, w, keep, sink, recent, dst_page, with_weights=True):
    table, dK, dV, index, dst_len, dw = evict(st, w, keep, sink, recent, dst_page, with_weights)
    kv = st["kv_len"].cpu().numpy()
    want = po.evict_index(w.cpu().numpy(), kv, keep, sink, recent)
    assert np.array_equal(index.cpu().numpy(), want)
    assert np.array_equal(dst_len.cpu().numpy(), np.minimum(kv, keep))
    src_table, page = st["table"].cpu().numpy(), st["K"].shape[2]
    for pool, dst, empty in ((st["K"], dK, 5.0), (st["V"], dV, 6.0)):
        pool, expect = pool.cpu(), torch.full(dst.shape, empty, dtype=BF)
        for b in range(len(kv)):
            m = min(int(kv[b]), keep)
            i = np.arange(m)
            for g in range(pool.shape[1]):
                j = want[b, g, :m]
                expect[table[b, i // dst_page], g, i % dst_page] = pool[src_table[b, j // page], g, j % page]
        assert torch.equal(dst.cpu(), expect)
    if with_weights:
        ref = torch.full(dw.shape, 8.0)
        for b in range(len(kv)):
            m = min(int(kv[b]), keep)
            for g in range(dw.shape[1]):
                ref[b, g, :m] = w.cpu()[b, g, want[b, g, :m].astype(np.int64)]
        assert torch.equal(dw.cpu().nan_to_num(-1), ref.nan_to_num(-1))


@pytest.mark.parametrize("kvs,page,keep,sink,recent,dst_page", [
    ([1], 16, 1, 0, 0, 16),
    ([40, 0, 7, 33, 8], 16, 8, 2, 3, 5),
    ([5000, 4096, 17], 64, 333, 4, 100, 48),
    ([1025, 1024, 1023], 1, 1024, 0, 0, 1024),
    ([300, 299], 7, 299, 299, 0, 64),
    ([2000, 3], 48, 50, 0, 50, 16),
    ([40000], 128, 5001, 31, 777, 64),
    ([200000, 9], 128, 150, 3, 50, 64)],
    ids=["one", "short", "ragged", "borders", "all_sink", "all_recent", "long", "read_again"])
@pytest.mark.parametrize("kind", ["random", "ties", "special"])
def test_evict(kvs, page, keep, sink, recent, dst_page, kind):
    st = make([(0, kv) for kv in kvs], 4, 2, page, seed=21, fill=0.0)
    B, ld = len(kvs), max(kvs) + 4
    rng = np.random.default_rng(5)
    w = np.exp(2 * rng.standard_normal((B, 2, ld))).astype(np.float32)
    if kind == "ties":
        w = rng.integers(0, 3, (B, 2, ld)).astype(np.float32)
    if kind == "special":
        w = rng.choice(np.array([0.0, -0.0, np.nan, np.inf, -np.inf, 1e-42, -1e-42, 1.0, -2.0],
                                dtype=np.float32), (B, 2, ld))
    check_evict(st, torch.tensor(w).cuda(), keep, sink, recent, dst_page, with_weights=kind != "ties")


def test_first_call_of_a_process_holds_8191_weights():
    """Dynamic and static shared memory together pass 48 KB before the limit was ever raised."""
    code = ("import sys, torch; sys.path.insert(0, %r)\n"
            "import fourier_basis_attention_b200 as fa\n"
            "K = torch.zeros(1, 64, 8192, 128, dtype=torch.bfloat16, device='cuda')\n"
            "src, dst = fa.PagedCache.dense(K, K), fa.PagedCache.dense(K[:, :, :16].clone(), K[:, :, :16].clone())\n"
            "n = torch.tensor([8191], dtype=torch.int32, device='cuda')\n"
            "b = fa.PagedBatch(src, 64, torch.tensor([0, 0], dtype=torch.int32, device='cuda'), n, 0, 0, 8191)\n"
            "w = torch.arange(8192., device='cuda').repeat(1, 64, 1)\n"
            "i = torch.zeros(1, 64, 16, dtype=torch.int32, device='cuda')\n"
            "fa.fa_evict(b, w, 16, dst, i, torch.zeros_like(n))\n"
            "fa.fa_device_status()\n"
            "assert (i.cpu() == torch.arange(8175, 8191)).all()\n") % ROOT
    subprocess.run([sys.executable, "-c", code], check=True, timeout=120)


def test_evict_into_dense_then_compress():
    """The kept tokens land in the dense tensors fa_compress reads; decode over the compressed
    cache with every dim retained equals attention over the kept tokens."""
    B, Hq, Hkv, keep, S, R = 2, 8, 2, 300, 16, 32
    st = make([(5, 1000), (5, 700)], Hq, Hkv, 64, seed=22, fill=0.0)
    out, lse = attend(st)
    acc = torch.zeros(B, Hkv, 1000, device="cuda")
    fa.fa_paged_weights(st["batch"], st["q"], lse, acc)
    K = torch.zeros(B, Hkv, keep, D, dtype=BF, device="cuda")
    V = torch.zeros_like(K)
    dst = fa.PagedCache.dense(K, V)
    index = torch.empty(B, Hkv, keep, dtype=torch.int32, device="cuda")
    dst_len = torch.empty(B, dtype=torch.int32, device="cuda")
    fa.fa_evict(st["batch"], acc, keep, dst, index, dst_len, sink=S, recent=R)
    plan = fa.fa_plan_init(B, Hq, Hkv, keep, S, R, 1, np.zeros((Hkv, D)))
    cache = fa.Cache(plan)
    fa.fa_compress(plan, K, V, fa.basis_table(plan), cache)
    q = st["q"][[4, 9]].contiguous()
    ws = torch.empty(fa.fa_decode_workspace_size(plan), dtype=torch.uint8, device="cuda")
    dec = torch.empty(B, Hq, D, device="cuda")
    fa.fa_decode(plan, q, cache, dec, ws)
    batch = fa.PagedBatch(dst, Hq, torch.arange(B + 1, dtype=torch.int32, device="cuda"), dst_len,
                          total_q=B, max_q=1)
    size = fa.fa_paged_attend_workspace_size(batch)
    again = torch.empty(B, Hq, D, dtype=BF, device="cuda")
    fa.fa_paged_attend(batch, q, again, torch.empty(max(size, 16), dtype=torch.uint8, device="cuda"))
    fa.fa_device_status()
    scale = dec.abs().max().item()
    # both round to bf16 once or twice; fa_decode's own bound is 3e-3 of the largest value
    assert (again.float() - dec).abs().max().item() <= (3e-3 + 2 * U16) * scale


def test_pools_of_more_than_2_31_elements():
    """Pages at both ends of pools of 2.6e9 elements: write, attention, weights, eviction."""
    page, pages = 128, 160000
    K = torch.empty(pages, 1, page, D, dtype=BF, device="cuda")
    V = torch.empty_like(K)
    table = torch.tensor([[pages - 1, 0, pages - 2]], dtype=torch.int32, device="cuda")
    cache = fa.PagedCache(K, V, table)
    n, Hq = 300, 4
    gen = torch.Generator().manual_seed(7)
    k, v, q = (torch.randn(n, h, D, generator=gen).to(BF).cuda() for h in (1, 1, Hq))
    batch = fa.PagedBatch(cache, Hq, torch.tensor([0, n], dtype=torch.int32, device="cuda"),
                          torch.tensor([n], dtype=torch.int32, device="cuda"), total_q=n, max_q=n, max_kv=n)
    fa.fa_paged_append(batch, k, v)
    small = fa.PagedCache(K[[pages - 1, 0, pages - 2]].contiguous(), V[[pages - 1, 0, pages - 2]].contiguous(),
                          torch.tensor([[0, 1, 2]], dtype=torch.int32, device="cuda"))
    rows = small.K[:, 0].reshape(-1, D)
    assert torch.equal(rows[:n], k[:, 0]) and torch.equal(small.V[:, 0].reshape(-1, D)[:n], v[:, 0])
    st = dict(K=small.K, V=small.V, table=small.page_table, q=q, used=n, total=n, batch=batch,
              q_start=batch.q_start, kv_len=batch.kv_len)
    out, lse = attend(st)
    check_attend(st, out, lse, reference(st))
    first = fa.PagedBatch(cache, Hq, torch.tensor([0, 1], dtype=torch.int32, device="cuda"), batch.kv_len,
                          total_q=1, max_q=1, max_kv=n)
    st1 = dict(st, q=q[-1:], used=1, total=1, batch=first, q_start=first.q_start)
    out, lse = attend(st1)
    check_attend(st1, out, lse, reference(st1))
    acc = torch.zeros(1, 1, n, device="cuda")
    fa.fa_paged_weights(first, q[-1:], lse, acc)
    w = reference(st1)[4]
    assert (np.abs(acc.double().cpu().numpy() - w) <= 1e-3 * w + 1e-30).all()
    far = fa.PagedCache(K, V, torch.tensor([[pages - 3]], dtype=torch.int32, device="cuda"))
    index = torch.empty(1, 1, 100, dtype=torch.int32, device="cuda")
    length = torch.empty(1, dtype=torch.int32, device="cuda")
    fa.fa_evict(batch, acc, 100, far, index, length, recent=10)
    fa.fa_device_status()
    assert torch.equal(K[pages - 3, 0, :100], k[index[0, 0].long(), 0])


def test_first_call_of_a_process_is_captured():
    """Nothing of a first call (module load, limits, tensor maps) breaks a capture."""
    code = ("import sys, torch; sys.path.insert(0, %r)\n"
            "import fourier_basis_attention_b200 as fa\n"
            "bf, i32 = torch.bfloat16, torch.int32\n"
            "K = torch.randn(4, 2, 64, 128, device='cuda').to(bf)\n"
            "c = fa.PagedCache(K, K.clone(), torch.arange(4, dtype=i32, device='cuda').view(2, 2))\n"
            "q = torch.randn(41, 8, 128, device='cuda').to(bf)\n"
            "b = fa.PagedBatch(c, 8, torch.tensor([0, 40, 41], dtype=i32, device='cuda'),\n"
            "                  torch.tensor([100, 90], dtype=i32, device='cuda'), 41, 40, 128)\n"
            "out, lse, acc = torch.empty_like(q), torch.empty(41, 8, device='cuda'), torch.zeros(2, 2, 128, device='cuda')\n"
            "ws = torch.empty(max(16, fa.fa_paged_attend_workspace_size(b)), dtype=torch.uint8, device='cuda')\n"
            "d = fa.PagedCache.dense(torch.zeros(2, 2, 32, 128, dtype=bf, device='cuda'), torch.zeros(2, 2, 32, 128, dtype=bf, device='cuda'))\n"
            "i, n = torch.zeros(2, 2, 32, dtype=i32, device='cuda'), torch.zeros(2, dtype=i32, device='cuda')\n"
            "r = fa.fa_rope_init()\n"
            "def go():\n"
            "    fa.fa_paged_append(b, q[:, :2], q[:, 2:4], q=q, q_out=out, rope=r)\n"
            "    fa.fa_rope(r, q[None], pos, q2[None])\n"
            "    fa.fa_paged_attend(b, q, out, ws, lse=lse)\n"
            "    fa.fa_paged_weights(b, q, lse, acc)\n"
            "    fa.fa_evict(b, acc, 32, d, i, n)\n"
            "pos, q2 = torch.zeros(1, 41, dtype=i32, device='cuda'), torch.empty_like(q)\n"
            "torch.cuda.synchronize()\n"
            "g = torch.cuda.CUDAGraph()\n"
            "with torch.cuda.graph(g): go()\n"
            "acc.zero_(); g.replay(); torch.cuda.synchronize(); fa.fa_device_status()\n"
            "a = [t.clone() for t in (out, lse, acc, i, n, q2)]\n"
            "acc.zero_(); go(); fa.fa_device_status()\n"
            "assert all(torch.equal(x, y) for x, y in zip(a, (out, lse, acc, i, n, q2)))\n") % ROOT
    subprocess.run([sys.executable, "-c", code], check=True, timeout=120)


# --------------------------------------------------------------------------- a run of them together

def test_prompt_in_chunks_then_decode():
    """A prompt read in ragged chunks (append + attend + weights), then decode steps: the outputs
    and gathered weights equal one attention over the whole sequence."""
    Hq, Hkv, page, L = 8, 2, 32, 400
    gen = torch.Generator().manual_seed(3)
    qkv = torch.randn(L, Hq + 2 * Hkv, D, generator=gen).to(BF).cuda()
    plan = fa.fa_rope_init(**SCALINGS["bands"])
    pages = -(-L // page)
    K = torch.full((pages, Hkv, page, D), float("nan"), dtype=BF, device="cuda")
    V = K.clone()
    cache = fa.PagedCache(K, V, torch.randperm(pages, generator=gen).to(torch.int32)[None].cuda())
    acc = torch.zeros(1, Hkv, L, device="cuda")
    outs, qrot = [], []
    at = 0
    for n in [100, 1, 130, 33, 129, 1, 1, 1, 1, 1, 1, 1]:
        x = qkv[at:at + n]
        batch = fa.PagedBatch(cache, Hq, torch.tensor([0, n], dtype=torch.int32, device="cuda"),
                              torch.tensor([at + n], dtype=torch.int32, device="cuda"), total_q=n, max_q=n,
                              max_kv=L)
        q = torch.empty(n, Hq, D, dtype=BF, device="cuda")
        out, lse = torch.empty_like(q), torch.empty(n, Hq, device="cuda")
        fa.fa_paged_append(batch, x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], q=x[:, :Hq], q_out=q, rope=plan)
        ws = torch.empty(max(16, fa.fa_paged_attend_workspace_size(batch)), dtype=torch.uint8, device="cuda")
        fa.fa_paged_attend(batch, q, out, ws, lse=lse)
        fa.fa_paged_weights(batch, q, lse, acc)
        outs.append(out)
        qrot.append(q)
        at += n
    assert at == L
    fa.fa_device_status()
    st = dict(K=K, V=V, table=cache.page_table, q=torch.cat(qrot), used=L, total=L,
              q_start=torch.tensor([0, L], dtype=torch.int32), kv_len=torch.tensor([L], dtype=torch.int32))
    ref = reference(st)
    check_attend(st, torch.cat(outs), None, ref)
    tol = ref[4] * (4 * 137 * U32 * ref[3].max() + (16 + 4 * L * 4) * U32) + 1e-30
    assert (np.abs(acc.double().cpu().numpy() - ref[4]) <= tol).all()


# --------------------------------------------------------------------------- entries out of range

def expect_device_error(what):
    with pytest.raises(fa.FaError) as e:
        fa.fa_device_status()
    assert e.value.code == fa.FA_ERR_DEVICE and what in str(e.value)
    fa.fa_device_status()  # cleared


@pytest.mark.parametrize("seqs", [[(1, 900), (1, 40)], [(140, 300), (30, 40)], [(140, 1400), (30, 40)]],
                         ids=["decode", "chunk", "pair"])
@pytest.mark.parametrize("entry", [-1, 2 ** 31 - 1, "one_past"])
def test_bad_page_is_reported_and_spares_the_others(seqs, entry):
    st = make(seqs, 4, 2, 16, seed=31)
    ref = reference(st)
    bad = st["K"].shape[0] if entry == "one_past" else entry
    st["table"][0, 0] = bad
    out, lse = attend(st)
    expect_device_error("page_table")
    n = seqs[0][0]
    out[:n], lse[:n] = torch.tensor(ref[0][:n]).to(BF), torch.tensor(ref[2][:n]).float()
    check_attend(st, out, lse, ref)
    fa.fa_paged_weights(st["batch"], st["q"], lse, torch.zeros(2, 2, max(kv for _, kv in seqs), device="cuda"))
    expect_device_error("page_table")
    K0 = st["K"].clone()
    st["table"][0] = bad
    k = torch.zeros(st["total"], 2, D, dtype=BF, device="cuda")
    fa.fa_paged_append(st["batch"], k, k)
    expect_device_error("page_table")
    del K0
    w = torch.rand(2, 2, max(kv for _, kv in seqs), device="cuda")
    index = torch.empty(2, 2, 20, dtype=torch.int32, device="cuda")
    n = torch.empty(2, dtype=torch.int32, device="cuda")
    dst = fa.PagedCache.dense(torch.zeros(2, 2, 20, D, dtype=BF, device="cuda"),
                              torch.zeros(2, 2, 20, D, dtype=BF, device="cuda"))
    fa.fa_evict(st["batch"], w, 20, dst, index, n)
    expect_device_error("page_table")


@pytest.mark.parametrize("seqs", [[(2, 60), (3, 40), (1, 9)], [(70, 160), (60, 90), (90, 100)],
                                  [(70, 1400), (60, 90), (90, 100)]], ids=["decode", "chunk", "pair"])
@pytest.mark.parametrize("what", ["kv_long", "kv_negative", "q_descends", "q_past_total", "q_many", "q_negative"])
def test_bad_lengths_are_reported(what, seqs):
    st = make(seqs, 4, 2, 16, seed=32)
    total, longest = st["total"], seqs[0][1]
    if what == "kv_long":
        st["kv_len"][1] = longest + 1
    elif what == "kv_negative":
        st["kv_len"][1] = -1
    elif what == "q_descends":
        st["q_start"][1] = total
    elif what == "q_past_total":
        st["q_start"][3] = total + 1
    elif what == "q_negative":
        st["q_start"][1] = -3
    else:
        st["q_start"][1] = 0
        st["q_start"][2] = total
    attend(st)
    expect_device_error("q_start or kv_len")
    k = torch.zeros(total, 2, D, dtype=BF, device="cuda")
    fa.fa_paged_append(st["batch"], k, k)
    expect_device_error("q_start or kv_len")
    fa.fa_paged_weights(st["batch"], st["q"], torch.zeros(total, 4, device="cuda"),
                        torch.zeros(3, 2, longest, device="cuda"))
    expect_device_error("q_start or kv_len")


def test_stream_argument():
    """The calls run on the stream they are given, behind what is queued there."""
    st = make([(1, 900), (60, 300)], 8, 2, 32, seed=40)
    side = torch.cuda.Stream()
    q = torch.zeros_like(st["q"])
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    ws = torch.empty(max(16, fa.fa_paged_attend_workspace_size(st["batch"])), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        q.copy_(st["q"])
    fa.fa_paged_attend(st["batch"], q, out, ws, lse=lse, stream=side)
    fa.fa_device_status(side)
    check_attend(st, out, lse, reference(st))


def test_c_calls_without_rows_do_nothing():
    st = make([(1, 20)], 4, 2, 16, seed=33)
    shape = fa.fa_paged_shape(0, 4, 2, D, 16, st["K"].shape[0], 2, 0, 0, 20)
    cache = fa.fa_paged_cache(st["K"].data_ptr(), st["V"].data_ptr(), None, None, None)
    s, c = ctypes.byref(shape), ctypes.byref(cache)
    assert fa.LIB.fa_paged_attend(s, c, None, 0, 0.0, 0, None, 0, None, None, 0, None) == fa.FA_OK
    assert fa.LIB.fa_paged_weights(s, c, None, 0, 0.0, 0, None, None, 20, None) == fa.FA_OK
    assert fa.LIB.fa_paged_append(s, c, None, None, None, 0, None, 0, None, 0, None, 0, None) == fa.FA_OK
    fa.fa_device_status()
