"""Pins of the rotary and paged-cache oracle against things other than itself."""

import math

import numpy as np
import pytest
import torch

import oracle
from oracle import seppaged_ref as P


def test_e4m3_values_are_torch_s():
    codes = torch.arange(256, dtype=torch.int32).to(torch.uint8)
    np.testing.assert_array_equal(P.e4m3_values(), codes.view(torch.float8_e4m3fn).double().numpy())


def test_e4m3_rounding_is_torch_s():
    g = torch.Generator().manual_seed(1)
    x = torch.cat([torch.randn(20000, generator=g) * 2.0 ** torch.randint(-12, 8, (20000,), generator=g),
                   torch.tensor([0.0, -0.0, 448.0, -448.0, 2.0 ** -10, 1.5 * 2.0 ** -9, 1.0625, 1.1875])])
    x = x.clamp(-448.0, 448.0)
    np.testing.assert_array_equal(P.e4m3_encode(x.double().numpy()),
                                  x.to(torch.float8_e4m3fn).view(torch.uint8).numpy())
    assert P.e4m3_encode([math.inf, -math.inf, math.nan]).tolist() == [0x7F] * 3


def test_page_scale_worked_examples():
    # 448 = 1.75 * 2^8: a maximum of 3.5 is 448 * 2^-7, anything above needs 2^-6
    assert P.page_scale([3.5, -1.0]) == 2.0 ** -7
    assert P.page_scale([3.5 * (1 + 2.0 ** -40)]) == 2.0 ** -6
    assert P.page_scale([448.0]) == 1.0 and P.page_scale([-449.0]) == 2.0
    assert P.page_scale([0.0, -0.0]) == 0.0
    assert P.page_scale([math.inf, math.nan, 2.0]) == 2.0 ** -7
    assert P.page_scale([1e-40]) == 2.0 ** -100


def test_rope_turn_is_the_rotate_half_oracle():
    rng = np.random.default_rng(2)
    x = rng.standard_normal((5, 3, 64))
    pos = rng.integers(0, 5000, 5)
    freq = 10000.0 ** (-2.0 * np.arange(32) / 64)
    np.testing.assert_allclose(P.rope_turn(x, pos[:, None], freq),
                               oracle.rope_rotate(x, pos[:, None], 10000.0), atol=1e-11)


def test_rope_turn_layouts_part_and_adjoint():
    rng = np.random.default_rng(3)
    x, g = rng.standard_normal((2, 7, 80))
    pos, freq = rng.integers(-50, 50, 7), rng.random(12)
    inter = P.rope_turn(x, pos, freq, 1.3, interleaved=True)
    # interleaved = half layout of the elements taken evens first
    perm = np.concatenate([np.arange(0, 24, 2), np.arange(1, 24, 2)])
    y = x.copy()
    y[:, :24] = x[:, perm]
    half = P.rope_turn(y, pos, freq, 1.3)
    np.testing.assert_allclose(inter[:, perm], half[:, :24], atol=1e-14)
    np.testing.assert_array_equal(inter[:, 24:], x[:, 24:])
    # <R x, g> = <x, R' g>
    back = P.rope_turn(g, pos, freq, 1.3, interleaved=True, inverse=True)
    assert np.sum(inter * g) == pytest.approx(np.sum(x * back), rel=1e-12)


def test_append_in_pieces_is_append_at_once_up_to_rounding():
    rng = np.random.default_rng(4)
    k, v = rng.standard_normal((2, 37, 2, 64)) * 2.0 ** rng.integers(-3, 4, (2, 37, 2, 1))
    sep = rng.random(37) < 0.3
    table = [5, 2, 0, 7]
    freq = 500.0 ** (-2.0 * np.arange(16) / 32)
    one, many = (P.PagedSim(9, 2, 64, 16, freq) for _ in range(2))
    one.append(table, 0, k, v, sep)
    at = 0
    for c in (1, 1, 3, 9, 5, 17, 1):
        many.append(table, at, k[at:at + c], v[at:at + c], sep[at:at + c])
        at += c
    for x in "kv":
        np.testing.assert_array_equal(one.scale[x], many.scale[x])
        a, b = one.rows(x, table, 37), many.rows(x, table, 37)
        # growing scales round numbers in e4m3's subnormals again: one more half step of 2^-9 at most
        step = 2.0 ** -9 * one.scale[x][[table[j // 16] for j in range(37)]][:, :, None]
        assert np.all(np.abs(a - b) <= step)
        np.testing.assert_array_equal(np.abs(a) >= 8 * step, np.abs(b) >= 8 * step)
    np.testing.assert_array_equal(one.flags, many.flags)
    ref = P.rope_turn(k, np.arange(37)[:, None], freq)
    got = one.rows("k", table, 37)
    amax = np.stack([np.abs(ref[16 * i:16 * i + 16]).max((0, 2)) for i in range(3)])[np.arange(37) // 16]
    assert np.all(np.abs(got - ref) <= 2.0 ** -4 * np.abs(ref) + 2.0 ** -10 * (amax / 224.0)[:, :, None])


@pytest.mark.parametrize("a,n", [(4, 8), (0, 1), (2, 0), (0, 100)])
def test_attend_is_the_masked_attention(a, n):
    """The newest tokens' rows equal the rows of the full masked attention (n = 0 has no counterpart
    there: initial tokens and separators only, by hand)."""
    rng = np.random.default_rng(5)
    L, Hq, Hkv, d, c = 21, 4, 2, 64, 6
    q, k, v = (rng.standard_normal((L, h, d)) for h in (Hq, Hkv, Hkv))
    flag = rng.random(L) < 0.2
    o, lse, _ = P.paged_attend(q[-c:], k, v, flag, a, n, 0.125)
    if n > 0:
        ro, rl = oracle.attn_fwd(q[None], k[None], v[None], flag[None].astype(np.uint8), a, n, 0.125)
        np.testing.assert_allclose(o, ro[0, -c:], atol=1e-12)
        np.testing.assert_allclose(lse, rl[0, :, -c:].T, atol=1e-12)
    else:
        keep = [j for j in range(L) if j < a or flag[j]]
        s = torch.from_numpy(q[-1, 0]) @ torch.from_numpy(k[[j for j in keep], 0]).T * 0.125
        want = torch.softmax(s, 0) @ torch.from_numpy(v[keep, 0])
        np.testing.assert_allclose(o[-1, 0], want.numpy(), atol=1e-12)


def test_attend_without_a_key():
    q = np.ones((2, 1, 64))
    o, lse, _ = P.paged_attend(q, np.ones((1, 1, 64)), np.ones((1, 1, 64)), [False], 0, 1, 1.0)
    # two queries, one token: the first query stands at -1
    assert np.all(o[0] == 0.0) and lse[0, 0] == -math.inf and np.allclose(o[1], 1.0)
