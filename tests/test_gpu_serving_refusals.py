"""What the serving operators refuse behind their look at the device."""
import pytest

from test_gpu_chunk_attention import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("what", ["q", "out", "kc", "vc", "table", "tlens", "tstart"])
def test_a_workspace_over_another_argument(what):
    """The workspace of a call on the tensor cores lies apart from all else; refused before anything is launched."""
    import torch
    from transformer_encoder_gb300 import WencError
    c = Case("bf16", [1, 200, 3, 40], [100, 300, 20, 60], 4, 2, seed=10, wide=True)
    c.out = torch.full_like(c.q, 7.0)
    want, room = c.run(), torch.zeros(1 << 26, dtype=torch.uint8, device="cuda")
    c.run(out=c.out, workspace=room)
    assert torch.equal(c.out, want)
    t = getattr(c, what)
    inside = room[256:256 + t.numel() * t.element_size()].view(t.dtype).view(t.shape)
    inside.copy_(t)
    setattr(c, what, inside)
    with pytest.raises(WencError, match="apart"):
        c.run(out=c.out, workspace=room)
    assert torch.equal(inside.view(torch.uint8), t.view(torch.uint8))  # (nothing ran)
