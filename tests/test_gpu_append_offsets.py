"""wenc_kv_append where a sequence's rows are said to end behind the call's: reported, and nothing of that sequence written."""
import numpy as np
import pytest

from test_gpu_kv_append import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("new,pad", [([2, 3, 4], 0), ([1, 0, 5], 2), ([3000, 2, 1500], 0)])
def test_a_sequence_that_ends_behind_the_rows(dtype, new, pad):
    import torch
    from transformer_encoder_gb300 import WencError, kv_append, sync_status
    c = Case(dtype, new, [20, 3, 9], 2, 2, 64, seed=11, pad=pad)
    c.run()
    want_k, want_v = c.kc.clone(), c.vc.clone()
    start = c.kw["seq_start"].clone()
    start[3] = c.rows + 1
    c.kc.fill_(5.0)
    c.vc.fill_(6.0)
    kv_append(c.k, c.v, c.kc, c.vc, torch.from_numpy(c.table).cuda(), torch.tensor(c.lens, dtype=torch.int32, device="cuda"),
              **{**c.kw, "seq_start": start})
    with pytest.raises(WencError, match="offset out of range") as e:
        sync_status()
    assert e.value.status == 1
    third = torch.from_numpy(np.unique(c.table[2][c.table[2] >= 0])).long().cuda()
    want_k[third], want_v[third] = 5.0, 6.0
    assert torch.equal(c.kc, want_k) and torch.equal(c.vc, want_v)
