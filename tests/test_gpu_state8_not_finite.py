"""What the 8-bit state makes of moments that are not finite, as
include/zero/train.h says it: the block goes to E = 254, under which ordinary
values vanish, and its neighbours stay as they are."""
import numpy as np
import pytest
import torch

import train_ref as R
import zero_sharded_optimizer_step_amd as Z

pytestmark = pytest.mark.gpu


def bits(x):
    return np.array([x], dtype=np.uint32).view(np.float32)[0]


NAN, MINUS_NAN = bits(0x7FC00000), bits(0xFFC00000)


# (m, its code, v, its code): the code None where the value is an ordinary one of its block
@pytest.mark.parametrize("m,cm,v,cv", [(np.float32(np.inf), 127, np.float32(np.inf), 255), (NAN, 127, NAN, 255),
                                       (MINUS_NAN, 255, MINUS_NAN, 0), (np.float32(-np.inf), 255, NAN, 255)])
def test_not_finite(m, cm, v, cv):
    r = np.random.default_rng(3)
    ms, vs = (r.standard_normal((3, 256)).astype(np.float32) * s for s in (1e-4, 1e-3))
    vs = (vs * vs).astype(np.float32)
    ordinary = R.encode(ms.reshape(-1), vs.reshape(-1))
    a, b = ms.copy(), vs.copy()
    a[1, 77], b[1, 78] = m, v
    s8 = torch.empty(3 * 512, dtype=torch.uint8, device="cuda")
    e8 = torch.empty(6, dtype=torch.uint8, device="cuda")
    Z.zero_state8_encode(torch.from_numpy(a.reshape(-1)).cuda(), torch.from_numpy(b.reshape(-1)).cuda(), s8, e8)
    got, exps = s8.cpu().numpy().reshape(3, 2, 256), e8.cpu().numpy().reshape(3, 2)
    for k in (0, 2):
        assert np.array_equal(got[k], ordinary[0].reshape(3, 2, 256)[k])
        assert np.array_equal(exps[k], ordinary[1].reshape(3, 2)[k])
    assert got[1, 0, 77] == cm and got[1, 1, 78] == cv and exps[1, 0] == 254
    others = np.arange(256) != 77
    assert not got[1, 0, others].any()
    if cv:
        assert exps[1, 1] == 254
        others = np.arange(256) != 78
        assert np.array_equal(got[1, 1, others], (b[1, others] > 0).astype(np.uint8))
    # read back: finite, the least second moment 2^94
    mo, vo = (torch.empty(768, device="cuda") for _ in range(2))
    Z.zero_state8_decode(s8, e8, mo, vo)
    assert bool(torch.isfinite(mo).all() and torch.isfinite(vo).all())
    if cv:
        assert bool((vo.view(3, 256)[1, :78] == 2.0**94).all())
