"""CPU pins of the attention oracle: checks that do not re-run its own formulas."""

import numpy as np
import torch

from oracle import attention as ref


def test_e4m3_rounding_is_that_of_the_type():
    """Every bf16 value up to 448, against the type's own conversion."""
    x = torch.arange(0, 1 << 16, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).float()
    x = x[torch.isfinite(x) & (x.abs() <= 448)]
    want = x.to(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(ref.to_e4m3(x.double().numpy()), want)


def test_e4m3_values_are_those_of_the_type():
    want = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(ref.e4m3_values(), want)


def test_scale_is_the_least_power_of_two():
    rng = np.random.default_rng(0)
    for x in [np.array([448.0]), np.array([449.0]), np.array([0.0]), np.array([1e-40]),
              *(rng.standard_normal(8) * 10.0 ** rng.integers(-20, 20) for _ in range(50))]:
        s = ref.block_scale(x)
        most = np.abs(x).max()
        assert np.log2(s) == round(np.log2(s)) and most <= 448 * s
        assert s == 2.0 ** -100 or most > 448 * s / 2


def test_one_open_block_is_plain_causal_attention():
    rng = np.random.default_rng(1)
    q, k, v = rng.standard_normal((50, 4, 16)), rng.standard_normal((50, 2, 16)), rng.standard_normal((50, 2, 16))
    got = ref.attention(q, k, v, 0.3)
    for h in range(4):
        s = q[:, h] @ k[:, h // 2].T * 0.3
        s[np.triu_indices(50, 1)] = -np.inf
        want = torch.softmax(torch.from_numpy(s), -1).numpy() @ v[:, h // 2]
        assert np.abs(got[:, h] - want).max() < 1e-12


def test_values_that_8_bits_hold_make_the_rule_plain_attention():
    """K and V whose every value e4m3 holds exactly: the cache loses nothing, so
    any length is plain causal attention."""
    rng = np.random.default_rng(2)
    grid = np.array([-2.0, -1.0, -0.5, 0.0, 0.25, 1.0, 1.75])
    q, k, v = rng.standard_normal((200, 1, 8)), rng.choice(grid, (200, 1, 8)), rng.choice(grid, (200, 1, 8))
    assert np.array_equal(ref.cached(k), k)
    got = ref.attention(q, k, v, 0.5)
    s = q[:, 0] @ k[:, 0].T * 0.5
    s[np.triu_indices(200, 1)] = -np.inf
    assert np.abs(got[:, 0] - torch.softmax(torch.from_numpy(s), -1).numpy() @ v[:, 0]).max() < 1e-12


def test_norm_rope_gradient_against_differences():
    rng = np.random.default_rng(3)
    for inter, rd in ((False, 8), (True, 4)):
        x, w, dy = rng.standard_normal((3, 2, 8)), rng.standard_normal(8), rng.standard_normal((3, 2, 8))
        ang = rng.standard_normal((3, rd // 2))
        args = (np.cos(ang), np.sin(ang), 1e-3, inter)
        dx, dw, _, _ = ref.norm_rope_backward(x, w, *args, dy)
        loss = lambda x_, w_: (ref.norm_rope(x_, w_, *args) * dy).sum()  # noqa: E731
        for at in np.ndindex(x.shape):
            e = np.zeros_like(x)
            e[at] = 1e-6
            assert abs((loss(x + e, w) - loss(x - e, w)) / 2e-6 - dx[at]) < 1e-7
        for j in range(8):
            e = np.zeros_like(w)
            e[j] = 1e-6
            assert abs((loss(x, w + e) - loss(x, w - e)) / 2e-6 - dw[j]) < 1e-7


def test_rotation_keeps_lengths_and_depends_on_position_differences():
    rng = np.random.default_rng(4)
    a, b = rng.standard_normal((1, 1, 8)), rng.standard_normal((1, 1, 8))
    freq = 0.3 ** np.arange(4)[None, :]
    dots = []
    for shift in (0, 5):
        ra = ref.rotate(a, np.cos((3 + shift) * freq), np.sin((3 + shift) * freq), False)
        rb = ref.rotate(b, np.cos((7 + shift) * freq), np.sin((7 + shift) * freq), False)
        assert abs((ra ** 2).sum() - (a ** 2).sum()) < 1e-12
        dots.append((ra * rb).sum())
    assert abs(dots[0] - dots[1]) < 1e-12


def test_pool_hands_out_every_block_once():
    rng = np.random.default_rng(5)
    p = ref.Pool(6, 9, 30)
    for _ in range(200):
        rows = rng.permutation(6)[:3].tolist()
        p.plan(rows, rng.integers(0, 150, 3).tolist())
        if rng.random() < 0.5:
            p.release(rng.permutation(6)[:2].tolist())
        used = [int(x) for x in p.table[p.table >= 0]]
        assert sorted(used + p.free) == list(range(30))
        assert all(p.held[r] * 64 >= p.len[r] for r in range(6))
