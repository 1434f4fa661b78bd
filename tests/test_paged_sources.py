"""Rules that the paged kernels' sources keep, checked on their text: what they guard against shows
only where a wait runs out or another compiler schedules the code."""
import os
import re

import numpy as np
import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "fourier_basis_attention_b200", "csrc")
KERNELS = ["fa_paged.cu", "fa_paged_tc.cu"]


def code(name):
    """The source without comments."""
    with open(os.path.join(CSRC, name)) as fh:
        return re.sub(r"//[^\n]*", "", fh.read())


@pytest.mark.parametrize("name", KERNELS)
def test_bounded_waits_answer_for_the_whole_warp(name):
    """Lanes give up a bounded wait one by one; a warp that branches on its own lane's answer
    around a vote or elect.sync can wait for good."""
    assert not re.search(r"\bmbar_wait\s*\(", code(name))
    assert re.search(r"\bwarp_wait\s*\(", code(name))
    helper = re.search(r"bool warp_wait\([^{]*\{(.*?)\n\}", code("fa_paged.cuh"), re.S).group(1)
    assert re.search(r"return __all_sync\(0xFFFFFFFFu, mbar_wait\(", helper)


def test_loads_from_tensor_memory_are_tied_to_their_wait():
    """A plain wait orders memory, not the registers that the load fills: a use of them that touches
    no memory could be scheduled before it."""
    text = code("fa_paged_tc.cu")
    assert not re.search(r"\btmem_ld_wait\s*\(", text)
    body = text[text.index("void attend_tiles("):]
    loaded = set(re.findall(r"\btmem_ld_32x32b_x32\([^;]*?,\s*(\w+(?:\[\d\])?)\);", body))
    waited = re.findall(r"\btmem_ld_wait_for\(([^;]*)\);", body)
    assert loaded and loaded == {name.strip() for names in waited for name in names.split(",")}


@pytest.mark.parametrize("begin,end", [("void attend_tiles(", "paged_tile_kernel("),
                                       ("paged_weights_tile_kernel(", "FA_WATCHDOG_READER")])
def test_copies_in_flight_are_waited_for_whichever_warp_gave_up(begin, end):
    """The producer may be through when another warp's wait runs out: its copies are waited for
    where all warps have met, not where the producer's own wait failed."""
    text = code("fa_paged_tc.cu")
    body = text[text.index(begin):]
    body = body[:body.index(end, len(begin))]
    joined = body.rindex("__syncthreads();")
    drains = [m.start() for m in re.finditer(r"\bdrain_ring<", body)]
    assert len(drains) == 2 and min(drains) > joined
    assert "*abort_flag" in body[joined:min(drains)]


def test_the_chunk_of_a_batch_without_cached_tokens_is_not_zero():
    """The rows kernel divides by it."""
    plan = code("fa_paged.cu")
    plan = plan[plan.index("static cudaError_t attend_plan("):plan.index("cudaError_t paged_attend_workspace(")]
    one = re.search(r"keys <= 256\) \{\s*P->chunk = ([^;]*);", plan).group(1)
    condition, some, none = re.fullmatch(r"(.*) \? (.*) : (.*)", one).groups()
    assert condition == "s.max_kv > 0" and int(none) > 0
    for max_kv in (1, 63, 64, 65, 256):  # C's division of whole numbers
        assert eval(some.replace("s.max_kv", str(max_kv)).replace("/", "//")) >= max_kv


def test_the_polynomial_of_exp2_is_as_near_as_it_says():
    """Its coefficients, highest first: relative error in exact arithmetic at most 9.6e-8, none at
    whole numbers."""
    body = code("fa_paged_tc.cu")
    body = body[body.index("uint64_t exp2_pair("):body.index("float max3(")]
    c = [float(x) for x in re.findall(r"pack2\((\d\.\d{9}e-?\+?\d\d)f, \1f\)", body)]
    assert len(c) == 6 and c[-1] == 1.0
    f = np.linspace(-0.5, 0.5, 1000001)
    assert np.abs(np.polyval(np.float32(c).astype(np.float64), f) / 2.0 ** f - 1).max() <= 9.6e-8
