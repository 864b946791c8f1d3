"""GPU parity of the per-head norm with rotation, within the bound the fp64 oracle derives."""
import numpy as np
import pytest
import torch

from oracle import step
from paged_kv_cache_147_gb300 import pkv

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _dev(a):
    return torch.as_tensor(np.ascontiguousarray(a)).to(DEV)


def _weights(rng):
    return (1 + 0.3 * rng.standard_normal((2, 128))).astype(np.float16)


def _check(out, x, w, eps, pos, table):
    keep = pos >= 0
    want, tol = step.norm_rope(x[keep], w, eps, pos[keep], table)
    got = out.cpu().numpy().astype(np.float64)[keep]
    assert (np.abs(got - want) <= tol).all(), np.max(np.abs(got - want) - tol)


@pytest.mark.parametrize("T,hq,hkv", [(1, 12, 2), (1, 1, 1), (3, 5, 3), (64, 12, 2), (37, 64, 8),
                                      (129, 32, 32), (5000, 7, 1)])
@pytest.mark.parametrize("gain", [3.0, 1e-4, 300.0])
def test_matches_oracle(T, hq, hkv, gain):
    rng = np.random.default_rng(T + hq)
    q = (rng.standard_normal((T, hq, 128)) * gain).astype(np.float16)
    k = (rng.standard_normal((T, hkv, 128)) * gain).astype(np.float16)
    w = _weights(rng)
    table = pkv.rope_table(9000).numpy()
    pos = rng.integers(0, 9000, T)
    pos[0] = 8999
    q_out, k_out = pkv.qk_norm_rope(_dev(q), _dev(k), _dev(w[0]), _dev(w[1]), 1e-6, _dev(pos),
                                    _dev(table))
    torch.cuda.synchronize()
    assert pkv.device_error(clear=True) == 0
    _check(q_out, q, w[0], np.float32(1e-6), pos, table)
    _check(k_out, k, w[1], np.float32(1e-6), pos, table)


def test_strided_parts_of_a_packed_projection_and_in_place():
    rng = np.random.default_rng(4)
    T, hq, hkv = 50, 12, 2
    x = rng.standard_normal((T, (hq + 2 * hkv) * 128)).astype(np.float16)
    w, table, pos = _weights(rng), pkv.rope_table(100), rng.integers(0, 100, T)
    xd, wd = _dev(x), [_dev(v) for v in w]
    q, k = xd[:, :hq * 128].view(T, hq, 128), xd[:, hq * 128:(hq + hkv) * 128].view(T, hkv, 128)
    q_out, k_out = pkv.qk_norm_rope(q, k, *wd, 1e-5, _dev(pos), table.to(DEV))
    qc, kc = q.contiguous(), k.contiguous()
    same = pkv.qk_norm_rope(qc, kc, *wd, 1e-5, _dev(pos), table.to(DEV), q_out=qc, k_out=kc)
    assert same[0] is qc and torch.equal(qc, q_out) and torch.equal(kc, k_out)
    _check(q_out, x[:, :hq * 128].reshape(T, hq, 128), w[0], np.float32(1e-5), pos, table.numpy())


def test_padding_rows_stay_and_a_position_past_the_table_is_said():
    rng = np.random.default_rng(6)
    T, hq, hkv = 70, 6, 2
    q = rng.standard_normal((T, hq, 128)).astype(np.float16)
    k = rng.standard_normal((T, hkv, 128)).astype(np.float16)
    w, table, pos = _weights(rng), pkv.rope_table(64), rng.integers(0, 64, T)
    pos[[3, 69]] = -1
    outs = [torch.full((T, h, 128), 9.0, dtype=torch.float16, device=DEV) for h in (hq, hkv)]
    args = [_dev(q), _dev(k), _dev(w[0]), _dev(w[1]), 1e-6]
    pkv.qk_norm_rope(*args, _dev(pos), table.to(DEV), *outs)
    torch.cuda.synchronize()
    assert pkv.device_error(clear=True) == 0
    for o in outs:
        assert (o[[3, 69]] == 9.0).all()
    _check(outs[0], q, w[0], np.float32(1e-6), pos, table.numpy())
    pos[5] = 64
    outs[0].fill_(9.0)
    pkv.qk_norm_rope(*args, _dev(pos), table.to(DEV), *outs)
    torch.cuda.synchronize()
    assert pkv.device_error(clear=True) == pkv.DEVERR_POSITION
    assert (outs[0][5] == 9.0).all()
    pos[5] = -1
    _check(outs[0], q, w[0], np.float32(1e-6), pos, table.numpy())


def test_zero_rows_and_the_largest_values():
    q = np.zeros((2, 1, 128), np.float16)
    q[1] = 65504
    w, table = np.ones((2, 128), np.float16), pkv.rope_table(4)
    q_out, _ = pkv.qk_norm_rope(_dev(q), _dev(q), _dev(w[0]), _dev(w[1]), 0.0 + 1e-6,
                                _dev(np.array([3, 0])), table.to(DEV))
    assert (q_out[0] == 0).all() and (q_out[1] == 1).all()


def test_binding_refuses_what_the_library_cannot_see():
    q = torch.zeros(4, 3, 128, dtype=torch.float16, device=DEV)
    w = torch.zeros(128, dtype=torch.float16, device=DEV)
    pos = torch.zeros(4, dtype=torch.int64, device=DEV)
    cs = torch.zeros(8, 64, 2, device=DEV)
    odd = torch.zeros(4, 3 * 128 + 2, dtype=torch.float16, device=DEV)[:, :384].view(4, 3, 128)
    heads_apart = torch.zeros(4, 3, 256, dtype=torch.float16, device=DEV)[..., :128]
    bad = [(q.float(), q, w, w, pos, cs), (q, q[:3], w, w, pos, cs), (q, q, w[:64], w, pos, cs),
           (q, q, w, w, pos.int(), cs), (q, q, w, w, pos, cs.double()), (q, q, w, w, pos, cs[:, :32]),
           (odd, q, w, w, pos, cs), (heads_apart, q, w, w, pos, cs), (q[..., :64], q, w, w, pos, cs),
           (q, q, w.cpu(), w, pos, cs)]
    for a in bad:
        with pytest.raises(pkv.PkvError) as e:
            pkv.qk_norm_rope(a[0], a[1], a[2], a[3], 1e-6, a[4], a[5])
        assert e.value.status == pkv.EINVAL
    with pytest.raises(pkv.PkvError):
        pkv.qk_norm_rope(q, q, w, w, -1.0, pos, cs)
