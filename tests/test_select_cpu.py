"""CPU pins of the block selection, from the source: the order of its cluster's accesses to shared
memory, and the width of what counts to the budget; and of its oracle."""
import os
import re

import numpy as np

from oracle import int8
from paged_kv_cache_147_gb300 import build


def _code(source):
    with open(os.path.join(build.CSRC, source)) as f:
        return re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)


def test_keys_that_other_ctas_copy_are_not_written_before_they_have_read_them():
    # every CTA of a cluster copies the others' keys, arrives at the cluster's barrier when it has, and
    # later marks the chosen ones in its own: the barrier's wait lies between the two
    code = _code("pkv_select.cu")
    copied = code.index("ld_cluster_v4(keys")
    arrived = code.index("cluster_arrive();", copied)
    writes = [m.start() for m in re.finditer(r"\bkeys\[[^;]*?\]\s*=[^=]", code) if m.start() > arrived]
    assert writes
    for at in writes:
        assert "cluster_wait();" in code[arrived:at]
    # and a CTA does not leave while the others may still read its keys
    assert code.index("cluster_wait();", writes[-1]) > writes[-1]


def test_places_up_to_the_budget_are_counted_in_64_bits():
    # a budget may be as large as an int; the loop's step past it may not
    loops = re.findall(r"for \((\w+) \w+ = [^;]*; \w+ < a\.budget;", _code("pkv_select.cu"))
    assert loops == ["int64_t"]


def test_the_oracle_puts_a_nan_scale_first_whatever_the_queries_hold():
    bounds = np.full((10, 1, 2, 128), 128, np.uint8)
    scales = np.ones((10, 1, 2), np.float32)
    scales[[3, 6], 0, 0] = np.nan
    tables = np.arange(10, dtype=np.int32)[None]
    for x in (1, np.nan, np.inf, 0):
        q = np.full((1, 2, 1, 128), x, np.float16)
        got, lens = int8.select(q, scales, bounds, tables, [160], 16, 5, 1, 1)
        assert list(got[0, 0]) == [0, 1, 3, 6, 9] and lens[0] == 80


def test_the_oracle_puts_unknown_blocks_last_whatever_the_queries_hold():
    bounds = np.full((10, 1, 2, 128), 128, np.uint8)
    scales = np.ones((10, 1, 2), np.float32)
    scales[5, 0, 0] = np.nan
    tables = np.arange(10, dtype=np.int32)[None]
    tables[0, [1, 2, 4]] = [-3, 10, 99]
    for x in (1, np.nan, 0):
        q = np.full((1, 1, 1, 128), x, np.float16)
        got, _ = int8.select(q, scales, bounds, tables, [160], 16, 5, 1, 1)
        assert list(got[0, 0]) == [0, 3, 5, 6, 9]
        got, _ = int8.select(q, scales, bounds, tables, [160], 16, 8, 1, 1)
        assert list(got[0, 0]) == [0, -3, 3, 5, 6, 7, 8, 9]
