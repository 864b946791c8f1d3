"""Both ways in which the 8-bit decode merges a split unit give the same bits: by the CTA with the unit's
first part, which waits for the others a bounded time, and, where that runs out (other work holds the
SMs), by the last one to arrive. A build without the time takes the second way (test_gpu_merge_paths.py
does the same for the fp16 cache)."""
import ctypes
import math

import pytest
import torch

from paged_kv_cache_147_gb300 import pkv

from test_gpu_int8 import _case, _dev
from test_gpu_merge_paths import nowait_lib  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _call(lib, out, a, ws, heads=False):
    q, k, v, scales, tables, lens = a
    B, q_len, hq, d = q.shape
    nb, hkv, bs, _ = k.shape
    f = lib.pkv_selected_attn_decode_int8 if heads else lib.pkv_paged_attn_decode_int8
    status = f(pkv._p(out), pkv._p(q), pkv._p(k), pkv._p(v), pkv._p(scales), nb, pkv._p(tables),
               tables.shape[-1], pkv._p(lens), B, q_len, hq, hkv, d, bs, 1 / math.sqrt(128), pkv._p(ws),
               ws.numel() * ws.element_size(), pkv._stream())
    assert status == pkv.OK


# rows from 1 to 32 (every variant), 2 to 64 parts a unit (whole batches of partials and ragged ones),
# units in the even division and in slices of the stream
@pytest.mark.parametrize("rows", [1, 8, 12, 16, 24, 28, 32])
@pytest.mark.parametrize("lens,hkv", [([2000], 1), ([30000], 1), ([20000, 700], 2), ([9000, 0, 4095, 1], 1),
                                      ([5000, 300, 8000, 40, 2500, 7000] * 7, 4)])
def test_merge_without_wait_matches_default_bitwise(nowait_lib, rows, lens, hkv):  # noqa: F811
    q_len = 1 if rows < 12 else rows // 4
    k, v, scales, _, tables, lens, q = _case(lens, 16, rows // q_len * hkv, hkv, q_len, seed=rows + len(lens))
    a = [_dev(x) for x in (q, k, v, scales, tables, lens)]
    by_head = a[:4] + [a[4][:, None].expand(-1, hkv, -1).contiguous(), a[5]]
    for heads, args in ((False, a), (True, by_head)):
        ws = [pkv.make_workspace(q.shape[0], q_len, q.shape[2], hkv) for _ in range(2)]
        ref = torch.empty_like(a[0])
        _call(pkv.load(), ref, args, ws[0], heads)
        for rep in range(4):
            out = torch.full_like(ref, float("nan"))
            _call(nowait_lib, out, args, ws[1], heads)
            torch.cuda.synchronize()
            differ = (out.view(torch.int16) != ref.view(torch.int16)).sum().item()
            assert differ == 0, f"call {rep}: {differ} of {out.numel()} outputs differ"
        assert (ws[1][:lens.size * hkv * 4] == 0).all()     # the arrival counters
    word = ctypes.c_uint(0)
    for lib in (pkv.load(), nowait_lib):
        assert lib.pkv_device_error(ctypes.byref(word), 1, pkv._stream()) == pkv.OK and word.value == 0
