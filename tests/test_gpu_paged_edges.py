"""GPU tests of paged calls at the borders of what their shapes allow: no new tokens, no cached
tokens, caches of many chunks, rows that share no stride."""
import threading

import numpy as np
import pytest
import torch

import fourier_basis_attention_b200 as fa
import test_gpu_paged as tgp
from test_gpu_paged import BF, D, attend, check_attend, check_rope, make, reference

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Hq,Hkv,max_kv", [(8, 8, 100000), (8, 2, 300), (200, 1, 5000)],
                         ids=["split", "one_chunk", "wide_group"])
def test_batches_of_spare_rows_only(Hq, Hkv, max_kv):
    """max_q = 0: every row lies behind the last sequence and stays as it was, also where the keys
    of a row would be split over CTAs and joined."""
    st = make([(0, 50), (0, 0)], Hq, Hkv, 128, seed=1, spare_rows=3, max_q=0, max_kv=max_kv)
    out, lse = attend(st)
    K = st["K"].clone()
    acc = torch.full((2, Hkv, max_kv), 3.0, device="cuda")
    fa.fa_paged_weights(st["batch"], st["q"], lse, acc)
    k = torch.zeros(3, Hkv, D, dtype=BF, device="cuda")
    fa.fa_paged_append(st["batch"], k, k)
    fa.fa_device_status()
    assert (out == 3.0).all() and (lse == 3.0).all() and (acc == 3.0).all()
    assert torch.equal(K.nan_to_num(9.0), st["K"].nan_to_num(9.0))


def test_new_tokens_without_max_q_are_reported():
    """A sequence with a new token breaks the bound max_q = 0."""
    st = make([(1, 50)], 8, 8, 128, seed=2, max_q=0, max_kv=100000)
    attend(st)
    with pytest.raises(fa.FaError) as e:
        fa.fa_device_status()
    assert e.value.code == fa.FA_ERR_DEVICE and "q_start or kv_len" in str(e.value)


@pytest.mark.parametrize("seqs", [[(2, 0), (1, 0)], [(2, 0), (40, 0), (0, 0)]], ids=["decode", "chunk"])
@pytest.mark.parametrize("window", [0, 7])
def test_batches_without_cached_tokens(seqs, window):
    """max_kv = 0: no row sees a key."""
    st = make(seqs, 8, 2, 16, seed=3, spare_rows=2, max_kv=0)
    out, lse = attend(st, window)
    acc = torch.full((len(seqs), 2, 4), 3.0, device="cuda")
    fa.fa_paged_weights(st["batch"], st["q"], lse, acc, window=window)
    fa.fa_device_status()
    n = st["used"]
    assert (out[:n] == 0.0).all() and torch.isneginf(lse[:n]).all() and (acc == 3.0).all()
    check_attend(st, out, None, reference(st, window))


@pytest.mark.parametrize("dtype", [BF, torch.float32], ids=["bf16", "f32"])
def test_rope_of_a_transposed_column(dtype):
    """The strides of axes of size 1 may be anything: a [1, 1, 1, 128] view has 1 there."""
    x = torch.randn(D, 1, device="cuda").to(dtype).t()[None, None]
    y = torch.zeros(D, 1, dtype=dtype, device="cuda").t()[None, None]
    assert x.stride(2) == 1 and y.stride(2) == 1
    pos = torch.tensor([[77]], dtype=torch.int32, device="cuda")
    fa.fa_rope(fa.fa_rope_init(), x, pos, y)
    fa.fa_device_status()
    check_rope(y.cpu().double().numpy(), x.cpu().double().numpy(), pos.cpu().numpy(), D, {}, False, False,
               dtype == BF)


@pytest.mark.parametrize("row", [0, 1, 6, 7, 14, 63, 70, 127, 134, 255])
def test_weight_of_the_one_row_that_counts_is_exact(row):
    """Scores 0 and a log-sum-exp of 0: the row gives exp(0) = 1 to every key that it sees, whichever
    unit takes the exponential; the others (log-sum-exp 10000) give less than 2^-24."""
    st = make([(256, 1000)], 1, 1, 32, seed=row)
    st["q"].zero_()
    lse = torch.full((256, 1), 10000.0, device="cuda")
    lse[row] = 0.0
    acc = torch.zeros(1, 1, 1000, device="cuda")
    fa.fa_paged_weights(st["batch"], st["q"], lse, acc)
    fa.fa_device_status()
    seen = 1000 - 256 + row + 1
    assert (acc[0, 0, :seen] == 1.0).all() and (acc[0, 0, seen:] < 2.0 ** -24).all()


# caches of more than 12288 keys: above that the keys of 16-row tiles are cut into 48 chunks where
# partial results are merged, and into as many as fill the launch where none are
LONG = {
    "one_head": ([(1, 131077)], 4, 1, 64, 0),
    "one_head_window": ([(1, 40001), (2, 12289)], 4, 1, 16, 4097),
    "two_heads": ([(1, 30011), (3, 20000), (1, 7)], 8, 2, 64, 0),
    "two_heads_window_700": ([(2, 50021), (1, 13001)], 8, 2, 128, 700),
    "tiles": ([(40, 14001), (1, 16400)], 8, 2, 64, 0),
    "tiles_window": ([(40, 20003), (5, 14001), (1, 300)], 8, 2, 64, 4097),
    "wide_group": ([(2, 13007)], 160, 1, 64, 0),
}


@pytest.mark.parametrize("name", LONG)
def test_attend_over_long_caches(name, monkeypatch):
    monkeypatch.setitem(tgp.CASES, name, LONG[name])
    tgp.test_attend(name)


@pytest.mark.parametrize("name", LONG)
def test_weights_over_long_caches(name, monkeypatch):
    monkeypatch.setitem(tgp.CASES, name, LONG[name])
    tgp.test_weights(name)


@pytest.mark.parametrize("seqs,window", [([(4, 2), (1, 0), (20, 5), (2, 9)], 0), ([(40, 0), (30, 10), (1, 3)], 7),
                                         ([(1, 500), (60, 200)], 0)], ids=["few", "window", "all_see"])
def test_rows_without_a_key_and_no_others_have_an_infinite_lse(seqs, window):
    st = make(seqs, 8, 2, 16, seed=4, spare_rows=2)
    out, lse = attend(st, window)
    fa.fa_device_status()
    n, want = st["used"], np.isneginf(reference(st, window)[2])
    got = lse.cpu().numpy()
    assert np.array_equal(np.isneginf(got[:n]), want[:n]) and np.isfinite(got[:n][~want[:n]]).all()
    assert not out.cpu().float().numpy()[:n][want[:n]].any()


# one page a sequence, of any size: a block of keys that starts in it may end in the next head's or
# sequence's page, or behind the pool
DENSE = {
    "tiny": ([(3, 5), (1, 1), (0, 4), (2, 2)], 4, 2, 5, 0),
    "tiles_100": ([(40, 100), (33, 77), (1, 5), (20, 3)], 8, 2, 100, 0),
    "tiles_333_window": ([(200, 333), (1, 300), (17, 129)], 4, 4, 333, 50),
    "pair_1501": ([(300, 1501), (1, 1499), (150, 150)], 8, 2, 1501, 0),
    "decode_5003": ([(1, 5003), (2, 4999), (1, 1)], 8, 2, 5003, 0),
    "decode_777_window": ([(1, 777), (4, 700)], 4, 1, 777, 100),
}
MANY = {
    "sequences": ([(1 + (i % 7 == 3), 1 + (13 * i) % 40) for i in range(2500)], 4, 2, 16, 0),
    "sequences_and_chunks": ([(30 if i % 97 == 5 else i % 3, 1 + (29 * i) % 70) for i in range(1500)], 4, 2, 16, 9),
}


@pytest.mark.parametrize("name", [*DENSE, *MANY])
def test_attend_over_dense_caches_and_many_sequences(name, monkeypatch):
    monkeypatch.setitem(tgp.CASES, name, {**DENSE, **MANY}[name])
    tgp.test_attend(name)


@pytest.mark.parametrize("name", [*DENSE, *MANY])
def test_weights_over_dense_caches_and_many_sequences(name, monkeypatch):
    monkeypatch.setitem(tgp.CASES, name, {**DENSE, **MANY}[name])
    tgp.test_weights(name)


def test_host_threads_at_once():
    """Calls from several host threads, a stream and a workspace each."""
    sts = [make([(1, 2000 + 50 * i), (60, 300)], 8, 2, 32, seed=20 + i) for i in range(4)]
    streams = [torch.cuda.Stream() for _ in sts]
    res = [None] * len(sts)
    torch.cuda.synchronize()

    def work(i):
        with torch.cuda.stream(streams[i]):
            for _ in range(10):
                res[i] = attend(sts[i])

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(sts))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    fa.fa_device_status()
    for st, (out, lse) in zip(sts, res):
        check_attend(st, out, lse, reference(st))
