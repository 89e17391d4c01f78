"""Every source with a kernel of the decode side has index checks."""
import os

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_decode_kernels_have_index_checks():
    for f in ("prefix_attn.cu", "prefix_tc.cu", "prefix_tc32.cu", "append.cu", "i8.cu"):
        assert "in_bounds(" in open(os.path.join(ROOT, "transformer_encoder_gb300", "csrc", f)).read(), f
