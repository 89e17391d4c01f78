"""The decode-side float64 definitions, pinned by closed forms (no GPU)."""
import numpy as np

from oracle import decode


def test_attention_joins_prefix_and_own_keys_like_one_list():
    import torch
    r = np.random.default_rng(0)
    q = r.standard_normal((2, 3, 4, 64))
    pre = [(r.standard_normal((7, 2, 64)), r.standard_normal((7, 2, 64)))]
    own = [(r.standard_normal((5, 2, 64)), r.standard_normal((5, 2, 64))) for _ in range(2)]
    out, absv, _ = decode.prefix_attention(q, pre, own, [0, 0])
    for s in range(2):
        K = torch.from_numpy(np.concatenate([pre[0][0], own[s][0]])).permute(1, 0, 2).repeat_interleave(2, 0)
        V = torch.from_numpy(np.concatenate([pre[0][1], own[s][1]])).permute(1, 0, 2).repeat_interleave(2, 0)
        mask = torch.arange(12)[None] <= 7 + 5 - 3 + torch.arange(3)[:, None]
        ref = torch.nn.functional.scaled_dot_product_attention(torch.from_numpy(q[s]).permute(1, 0, 2), K, V, attn_mask=mask)
        assert np.abs(out[s] - ref.permute(1, 0, 2).numpy()).max() < 1e-12
    assert (absv >= np.abs(out) - 1e-12).all()


def test_attention_of_nothing_is_zero_and_of_one_key_its_value():
    q = np.ones((2, 2, 1, 64))
    none = (np.zeros((0, 1, 64)), np.zeros((0, 1, 64)))
    one = (np.ones((1, 1, 64)), np.full((1, 1, 64), 3.0))
    out, _, _ = decode.prefix_attention(q, [none], [none, one], [0, 0])
    assert (out[0] == 0).all()
    assert (out[1, 0] == 0).all() and (out[1, 1] == 3.0).all()  # the older token does not see the newer one's key


def test_rotation_keeps_lengths_and_depends_on_distance_alone():
    r = np.random.default_rng(1)
    f = np.array([10000.0 ** (-2.0 * i / 64) for i in range(32)])
    x, y = r.standard_normal((1, 1, 64)), r.standard_normal((1, 1, 64))
    for inter in (False, True):
        turn = lambda v, p: decode.rotate(v, np.array([p]), f, inter)[0]
        assert abs(np.linalg.norm(turn(x, 123)) - np.linalg.norm(x)) < 1e-12
        assert abs((turn(x, 5) * turn(y, 9)).sum() - (turn(x, 105) * turn(y, 109)).sum()) < 1e-9
        assert np.array_equal(turn(x, 0), x)


def test_quantized_rows_come_back_within_half_a_scale():
    r = np.random.default_rng(2)
    x = r.standard_normal((20, 100)).astype(np.float32)
    q, s = decode.quantize_rows(x)
    assert (np.abs(q * s[:, None].astype(np.float64) - x) <= 0.5 * s[:, None] * (1 + 1e-5)).all()
    assert (np.abs(q).max(1) == 127).all()
