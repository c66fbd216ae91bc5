"""The 4-bit and eviction oracle against closed forms, torch and brute force, on the CPU."""
import numpy as np
import pytest
import torch

from oracle import kv4_oracle as K


def test_bf16_up_against_every_neighbour():
    r = np.random.default_rng(1)
    for x in list(r.random(200) * 10.0 ** r.integers(-30, 30, 200)) + [0.0, 1.0, 0.5, 2.0 ** -140]:
        v = K.bf16_up(float(x))
        t = torch.tensor(v, dtype=torch.float64)
        assert v >= x and float(t.to(torch.bfloat16).double()) == v
        below = torch.nextafter(t.to(torch.bfloat16), torch.tensor(-1.0, dtype=torch.bfloat16))
        assert v == 0.0 or float(below.double()) < x


def test_round_trip_error_is_half_a_scale_and_ends_are_kept():
    r = np.random.default_rng(2)
    x = torch.from_numpy(r.normal(size=(40, 128)) * 3 + 1).to(torch.bfloat16).double().numpy()
    y = K.round_trip(x)
    for row, back in zip(x, y):
        for g in (0, 64):
            a, b = row[g:g + 64], back[g:g + 64]
            c, s, m = K.quantise_group(a)
            assert np.abs(a - b).max() <= s / 2 * (1 + 1e-12)
            assert b[a.argmin()] == a.min() and c.min() == 0 and c.max() in (14, 15)
            assert len(np.unique(b)) <= 16


@pytest.mark.parametrize("x", [np.zeros(64), np.full(64, -3.25), np.r_[np.zeros(63), 15.0]])
def test_constant_and_exact_groups(x):
    c, s, m = K.quantise_group(x)
    assert np.array_equal(m + c * s, x)


def test_groups_that_are_not_finite():
    for bad in (np.inf, -np.inf, np.nan):
        c, s, m = K.quantise_group(np.r_[np.ones(63), bad])
        assert np.isnan(m + c * s).all()
    big = float(torch.finfo(torch.bfloat16).max)
    assert np.isnan(K.quantise_group(np.r_[np.full(63, big), -big])[2])


def test_unpack_places_every_nibble():
    page = np.zeros(K.PAGE_BYTES, dtype=np.uint8)
    meta = page[2048:].view(np.uint16).reshape(16, 4, 2)
    meta[:, :, 0] = 0x3f80                       # scale 1, minimum 0
    page[5 * 64 + 4 * (2 * 3 + 1) + 2] = 0x90    # K row 5, word (i 3, group 1), byte 2: nibbles 4, 5
    page[1024 + 15 * 64] = 0x07                  # V row 15, dim 0
    meta[15, 2] = (0x4000, 0xbf80)               # V group 0 of token 15: scale 2, minimum -1
    k, v = K.unpack_pages(page)
    want = np.zeros((16, 128))
    want[5, 64 + 24 + 5] = 9.0
    assert np.array_equal(k, want)
    want = np.zeros((16, 128))
    want[15, :64] = -1.0
    want[15, 0] = 13.0
    assert np.array_equal(v, want)


def test_mass_sums_to_the_heads_and_matches_torch():
    r = np.random.default_rng(3)
    q, k = r.normal(size=(4, 128)), [r.normal(size=(33, 128)) for _ in range(2)]
    m = K.attention_mass(q, k, 0.1, 2)
    assert np.allclose(m.sum(1), 2.0)
    w = torch.softmax(torch.from_numpy(k[1]) @ torch.from_numpy(q[2:].T) * 0.1, 0).sum(1).numpy()
    assert np.allclose(m[1], w)


def test_kept_slots_by_brute_force():
    r = np.random.default_rng(4)
    for _ in range(200):
        n = int(r.integers(1, 12))
        budget = int(r.integers(1, 12))
        sink = int(r.integers(0, budget + 1))
        recent = int(r.integers(0, budget - sink + 1))
        m = r.integers(0, 4, n) / 2.0             # many ties
        got = K.kept_slots(m, n, sink, recent, budget)
        assert len(got) == min(n, budget) and np.all(np.diff(got) > 0)
        if n <= budget:
            continue
        kept = set(got.tolist())
        assert set(range(sink)) <= kept and set(range(n - recent, n)) <= kept
        for a in kept:                            # nothing given up beats anything chosen
            if sink <= a < n - recent:
                for d in set(range(n)) - kept:
                    assert (m[a], -a) > (m[d], -d)
