"""The oracle's paged e4m3 cache against closed forms and the oracle's plain attention."""
import copy

import numpy as np
import pytest

from oracle import fp8
from oracle import model as M
from oracle import paged
from paged_cases import Case


@pytest.mark.parametrize("amax,e", [(448.0, 0), (448.5, 1), (224.0, -1), (0.0, -40), (1e-30, -40),
                                    (3e38, 100), (1.75, -8), (1.7578125, -7)])
def test_exponent_is_the_smallest_that_fits(amax, e):
    assert paged.exponent(amax) == e


@pytest.mark.parametrize("page", [16, 128])
def test_append_rounds_by_at_most_half_a_step(page):
    c = Case([(37, 21), (0, 5), (150, 0)], 2, 2, 64, page, seed=1)
    k, v = c.heads("k"), c.heads("v")
    paged.append(c.cache, c.seqs, k, v)
    for t0, n, c0, pages in c.seqs:
        for name, x in (("k", k), ("v", v)):
            for g in range(2):
                got = paged.keys_of(c.cache, name, pages, g, c0 + n)[c0:]
                want = x[t0:t0 + n, g].astype(np.float64)
                e = c.cache[name + "_exp"][pages, g].astype(int) - 127
                step = 2.0 ** e[(c0 + np.arange(n)) // page] * 2.0 ** -10  # half a subnormal step
                assert np.all(np.abs(got - want) <= np.maximum(np.abs(want) * 2.0 ** -4,
                                                               step[:, None]))


def test_kept_rows_survive_a_growing_scale_exactly_until_they_turn_subnormal():
    c = Case([(1, 15)], 1, 1, 64, 16, seed=2, exp_range=(119, 120))
    before = paged.keys_of(c.cache, "v", c.seqs[0][3], 0, 15)
    v = np.zeros((1, 1, 64), np.float32)
    v[0, 0, 3] = 448.0 * 2.0 ** (119 - 127) * 8  # the scale grows by 2^3
    paged.append(c.cache, c.seqs, v, v)
    after = paged.keys_of(c.cache, "v", c.seqs[0][3], 0, 16)
    assert c.cache["v_exp"][c.seqs[0][3][0], 0] == 122
    normal = np.abs(before) >= 2.0 ** (122 - 127) * 2.0 ** -6
    assert normal.mean() > 0.9
    assert np.array_equal(before[normal], after[:15][normal])
    assert after[15, 3] == v[0, 0, 3]


def test_writing_the_same_rows_again_changes_nothing():
    c = Case([(40, 21)], 2, 1, 64, 32, seed=3)
    k, v = c.heads("k"), c.heads("v")
    paged.append(c.cache, c.seqs, k, v)
    once = copy.deepcopy(c.cache)
    paged.append(c.cache, c.seqs, k, v)
    for name in once:
        assert np.array_equal(once[name], c.cache[name])


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_keeps_norms_and_depends_on_the_distance_only(interleaved):
    rng = np.random.default_rng(4)
    half = 16
    a = np.arange(64)[:, None] * 10000.0 ** (-np.arange(half) / half)
    rope = np.stack([np.cos(a), np.sin(a)], -1).astype(np.float32)
    q, k = rng.standard_normal((2, 1, 1, 64)).astype(np.float32)

    def dot(pq, pk):
        return float(np.sum(paged.rotate(q, rope, np.array([pq]), interleaved).astype(np.float64)
                            * paged.rotate(k, rope, np.array([pk]), interleaved)))

    assert abs(dot(0, 0) - float(np.sum(q.astype(np.float64) * k))) < 1e-6
    assert abs(dot(40, 33) - dot(7, 0)) < 1e-4
    assert abs(dot(40, 33) - dot(0, 7)) > 1e-3  # the direction matters


@pytest.mark.parametrize("causal", [False, True])
def test_attention_equals_the_plain_attention_of_the_decoded_rows(causal):
    c = Case([(7, 30), (12, 0)], 2, 2, 64, 16, seed=5)
    q = c.heads("q").astype(np.float64)
    out, _ = paged.attend(c.cache, c.seqs, q, causal, 0.125)
    for t0, n, c0, pages in c.seqs:
        k = np.stack([paged.keys_of(c.cache, "k", pages, g, c0 + n) for g in range(2)])
        v = np.stack([paged.keys_of(c.cache, "v", pages, g, c0 + n) for g in range(2)])
        want = M.gqa_attention(q[t0:t0 + n], k[:, c0:].transpose(1, 0, 2),
                               v[:, c0:].transpose(1, 0, 2), k[:, :c0], v[:, :c0], causal, 0.125)
        assert np.allclose(out[t0:t0 + n].reshape(n, -1), np.asarray(want).reshape(n, -1),
                           rtol=1e-10, atol=1e-12)


def test_fp8_values_reads_the_nan_code():
    assert np.isnan(paged.fp8_values(np.array([0x7F, 0xFF], np.uint8))).all()
    assert paged.fp8_values(np.array([0x7E], np.uint8))[0] == fp8.MAX
