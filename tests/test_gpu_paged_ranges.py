"""dg_kv_append_e4m3 and dg_paged_attn_e4m3 at the ends of their ranges, against the oracle in 64 bits.

Scores far below zero, rows of zeros, weights far below the largest, page scales
of every size.  Where nothing else is said the bounds are those of
test_gpu_paged.compare.
"""
import numpy as np
import pytest
import torch

import test_gpu_paged as base
from oracle import paged
from paged_cases import Case
from test_gpu_paged import check_append, dg

pytestmark = pytest.mark.gpu

_compare = base.compare


def compare(case, out, z, *args, **kw):
    """base.compare, which takes the largest error with max() and so passes over NaN, for results
    that have to be finite."""
    assert torch.isfinite(out.float()).all(), "results that are not finite"
    assert z is None or torch.isfinite(z).all(), "log-sum-exps that are not finite"
    _compare(case, out, z, *args, **kw)


def check_attention(*args, **kw):
    with pytest.MonkeyPatch.context() as m:
        m.setattr(base, "compare", compare)
        return base.check_attention(*args, **kw)


def test_the_other_files_results_are_finite(monkeypatch):
    """The batches of test_gpu_paged once more (their rows see finite keys and values only)."""
    monkeypatch.setattr(base, "compare", compare)
    for causal in (False, True):
        for hd, page in ((64, 16), (128, 128), (64, 64), (128, 32)):
            base.test_attention_many_rows(hd, page, causal)
            base.test_attention_few_rows(hd, page, causal)
    for hkv, group, n in ((1, 7, 40), (2, 16, 1), (1, 32, 2), (1, 20, 3), (8, 2, 1), (2, 25, 1)):
        base.test_attention_groups(hkv, group, n)
    base.test_attention_long_key_ranges()
    base.test_attention_scales_differ_between_pages()
    base.test_attention_peaked_rows_and_small_weights()
    base.test_attention_options()
    base.test_append_then_attend_as_a_program_does()
    base.test_attention_of_more_sequences_than_fit_at_once(48, 8, 2, 1)
    base.test_append_and_attention_on_two_streams_at_once()


# Ways that the few-row kernel is launched: (lengths, kv heads, group).  One key;
# several tiles by one CTA; a range per CTA of a cluster; ranges that a second
# launch merges; and the 32-row form unsplit and split.
NARROW = {
    "one key": ([(1, 0)], 2, 2),
    "one CTA": ([(1, 300)] * 40, 8, 1),
    "cluster": ([(1, 1000)], 1, 2),
    "merge launch": ([(1, 3000), (1, 2000), (1, 900)], 8, 2),
    "32 rows": ([(1, 700), (1, 90)], 1, 20),
    "32 rows, merge launch": ([(3, 2000)] * 20, 1, 8),
}
WIDE = {"wide": ([(150, 300)], 2, 2), "wide, split": ([(150, 3000)], 1, 1)}


def lowered(kind, nats, keys=None, hd=64, seed=80):
    """A batch whose scores lie `nats` lower (at the positions `keys` only, where given): element 0
    of every query times element 0 of every key."""
    lengths, hkv, group = {**NARROW, **WIDE}[kind]
    case = Case(lengths, hkv, group, hd, 64, seed=seed, exp_range=(121, 122))
    case.q[:, ::hd] = -nats * hd ** 0.5 / 7.0  # against the keys' 448 * 2^(121 - 127) = 7
    for _, n, c, pages in case.seqs:
        live = np.arange(len(pages) * 64).reshape(-1, 64)
        at = live < n + c if keys is None else keys(live, n + c)
        column = case.cache["k"][pages][..., 0]
        column[:] = np.where((live < n + c)[:, None], 0, column)
        column[np.broadcast_to(at[:, None], column.shape) &
               np.broadcast_to((live < n + c)[:, None], column.shape)] = 0x7E
        block = case.cache["k"][pages]
        block[..., 0] = column
        case.cache["k"][pages] = block
    return case


@pytest.mark.parametrize("nats", [64.0, 100.0, 300.0])
@pytest.mark.parametrize("kind", [*NARROW, *WIDE])
def test_scores_far_below_zero(kind, nats):
    check_attention(lowered(kind, nats), True)


@pytest.mark.parametrize("nats", [2.0 ** 22, -2.0 ** 22])
@pytest.mark.parametrize("kind", [*NARROW, *WIDE])
def test_scores_of_millions_stay_finite(kind, nats):
    check_attention(lowered(kind, nats), True)  # (the bounds grow with the scores)


@pytest.mark.parametrize("kind", ["one CTA", "cluster", "merge launch", "32 rows, merge launch", "wide, split"])
@pytest.mark.parametrize("far", ["first", "last"])
def test_some_key_ranges_far_below_the_others(kind, far):
    keys = (lambda p, total: p < total // 2) if far == "first" else (lambda p, total: p >= total // 2)
    check_attention(lowered(kind, 200.0, keys), True)


@pytest.mark.parametrize("kind", ["one key", "one CTA", "cluster"])
def test_scores_below_zero_under_pages_of_zero_values(kind):
    case = lowered(kind, 80.0)
    case.cache["v"][:] = 0
    case.cache["v_exp"][:] = 127 - 40  # as append stores zeros
    out = check_attention(case, True)
    assert (out == 0).all()


def check_sink(kind, bits, quantum, page=64):
    """Key 0 stands `bits` (log2) above every other key and its value is zero: the result is made of
    the small weights alone.  A weight w_j is held to 2^-11 of itself (f16), and to `quantum` of the
    largest; exp2, the fp32 sums and the result's rounding add 2^-12 and 2^-8 relative:
        |error| <= (2^-8 + 2^-10) |out| + quantum w_0 sum_j |v_j|.
    """
    lengths, hkv, group = {**NARROW, **WIDE}[kind]
    case = Case(lengths, hkv, group, 64, page, seed=81, exp_range=(121, 122))
    case.q[:] = 0.0
    case.q[:, ::64] = 4.0
    case.cache["v"] &= 0x7F  # all positive (the NaN codes behind the sequences stay)
    for _, n, c, pages in case.seqs:
        case.cache["k"][pages[0], :, 0] = 0
        block = case.cache["k"][pages]
        block[..., 0] = np.where(block[..., 0] == 0x7F, 0x7F, 0)
        case.cache["k"][pages] = block
        case.cache["k"][pages[0], :, 0, 0] = 0x7E  # 448 * 2^-6 = 7, times 4
        case.cache["v"][pages[0], :, 0] = 0
    d = dg()
    cache, table, starts, lens = case.device()
    out = torch.zeros((case.T, case.hq * 64), dtype=torch.bfloat16, device="cuda")
    z = torch.zeros((case.T, case.hq), device="cuda")
    scale = bits / (28.0 * np.log2(np.e))
    d.paged_attn_e4m3(case.q.cuda(), cache, table, starts, lens, case.max_new, case.max_prefix, out,
                      n_q_heads=case.hq, lse=z, scale=scale, mask=d.MASK_CAUSAL)
    torch.cuda.synchronize()
    d.check_device_errors()
    q = case.heads("q").astype(np.float64)
    want, wz = paged.attend(case.cache, case.seqs, q, True, scale)
    got = out.float().cpu().numpy().astype(np.float64).reshape(want.shape)
    assert np.isfinite(got).all()
    worst = 0.0
    for t0, n, c, pages in case.seqs:
        for g in range(hkv):
            v = paged.keys_of(case.cache, "v", pages, g, c + n)
            hs = slice(g * group, (g + 1) * group)
            w = want[t0:t0 + n, hs]
            tol = (2.0 ** -8 + 2.0 ** -10) * w + quantum * np.abs(v).sum(0)
            worst = max(worst, float((np.abs(got[t0:t0 + n, hs] - w) / tol).max()))
    assert worst <= 1.0, worst
    assert np.abs(z.cpu().numpy() - wz).max() <= 2.0 ** -19 * (1 + np.abs(wz).max())


# the largest weight is held as 2^4 or more, and f16's half step below 2^-14 is 2^-25
@pytest.mark.parametrize("bits", [12.6, 20.3, 24.6])
@pytest.mark.parametrize("kind", [k for k in NARROW if k != "one key"])
def test_small_weights_beside_a_sink_few_rows(kind, bits):
    check_sink(kind, bits, 2.0 ** -29)


# the largest weight is held as 2^7 or more
@pytest.mark.parametrize("bits", [12.6, 20.3, 27.4])
@pytest.mark.parametrize("kind", [*WIDE])
def test_small_weights_beside_a_sink_many_rows(kind, bits):
    check_sink(kind, bits, 2.0 ** -32)


@pytest.mark.parametrize("kind", [*NARROW, *WIDE])
@pytest.mark.parametrize("causal", [False, True])
def test_zero_and_tiny_query_rows(kind, causal):
    """Scores that underflow to zero: the rows are plain means of what they see."""
    lengths, hkv, group = {**NARROW, **WIDE}[kind]
    for k_exp, scale in ((79, None), (60, None), (1, None), (87, 1e-4), (121, 1e-38)):
        case = Case(lengths, hkv, group, 64, 32, seed=82, exp_range=(121, 122))
        case.cache["k_exp"][:] = k_exp
        case.q[::3] = 0.0
        case.q[1::3] *= 2.0 ** -120
        check_attention(case, causal, scale=scale)


@pytest.mark.parametrize("kind", [*NARROW, *WIDE])
@pytest.mark.parametrize("exp", [30, 87, 200, 227, 253, 254])
def test_value_scales_at_the_ends(kind, exp):
    lengths, hkv, group = {**NARROW, **WIDE}[kind]
    case = Case(lengths, hkv, group, 64, 32, seed=83, exp_range=(121, 122))
    small_values(case)
    case.cache["v_exp"][:] = exp
    check_attention(case, True)


@pytest.mark.parametrize("kind", [*NARROW, *WIDE])
@pytest.mark.parametrize("exp", [1, 2])
def test_value_scales_at_the_lower_end(kind, exp):
    """Results of 2^-126 and less: bf16 values lie 2^-133 apart there, so that their rounding is off
    by up to 2^-134 whatever the value, which compare()'s 2^-8 |out| does not hold.  With it:
        |error| <= 2^-134 + 2^-8 |out| + (2^-10 + 2 ds) max|v|   (ds as in base.compare).
    """
    lengths, hkv, group = {**NARROW, **WIDE}[kind]
    case = Case(lengths, hkv, group, 64, 32, seed=83, exp_range=(121, 122))
    small_values(case)
    case.cache["v_exp"][:] = exp
    worst = []

    def compare_small(case, out, z, causal, scale):
        want, wz = paged.attend(case.cache, case.seqs, case.heads("q").astype(np.float64), causal, scale)
        got = out.float().cpu().numpy().astype(np.float64).reshape(want.shape)
        assert np.isfinite(got).all()
        for t0, n, c0, pages in case.seqs:
            for g in range(case.hkv):
                k, v = (paged.keys_of(case.cache, x, pages, g, c0 + n) for x in "kv")
                hs = slice(g * case.group, (g + 1) * case.group)
                q = case.heads("q")[t0:t0 + n, hs].astype(np.float64)
                ds = 2.0 ** -18 * np.abs(q).max(-1) * scale * np.abs(k).sum(1).max()
                w = want[t0:t0 + n, hs]
                tol = 2.0 ** -134 + 2.0 ** -8 * np.abs(w) + ((2.0 ** -10 + 2 * ds) * np.abs(v).max())[..., None]
                worst.append((np.abs(got[t0:t0 + n, hs] - w) / tol).max())
                worst.append((np.abs(z.cpu().numpy()[t0:t0 + n, hs] - wz[t0:t0 + n, hs]) /
                              (ds + 2.0 ** -19 * (1 + np.abs(wz[t0:t0 + n, hs])))).max())

    with pytest.MonkeyPatch.context() as m:
        m.setattr(base, "compare", compare_small)
        base.check_attention(case, True)
    assert np.max(worst) <= 1.0, np.max(worst)


def small_values(case):
    """Value codes of magnitude 1 at most, so that 2^127 times them is finite; NaN ones stay."""
    nan = (case.cache["v"] & 0x7F) == 0x7F
    g = torch.Generator().manual_seed(84)
    x = (torch.randn(case.cache["v"].shape, generator=g) * 0.3).clamp(-1, 1)
    codes = x.to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    case.cache["v"] = np.where(nan, np.uint8(0x7F), codes)


def spread_case(kind, exps, page=16):
    """Page i of a sequence has the value exponent exps[i % len(exps)]."""
    lengths, hkv, group = {**NARROW, **WIDE}[kind]
    case = Case(lengths, hkv, group, 64, page, seed=85, exp_range=(121, 122))
    small_values(case)
    for _, _, _, pages in case.seqs:
        case.cache["v_exp"][pages] = np.resize(exps, len(pages))[:, None]
    return case


@pytest.mark.parametrize("kind", [k for k in (*NARROW, *WIDE) if k != "one key"])
@pytest.mark.parametrize("exps", [(227, 87), (87, 227), (1, 254), (87, 110, 130, 160, 180, 227),
                                  tuple(range(254, 0, -9)), tuple(range(1, 255, 9))])
def test_value_scales_far_apart_keep_the_weights(kind, exps):
    check_attention(spread_case(kind, exps), True)


@pytest.mark.parametrize("kind", [k for k in (*NARROW, *WIDE) if k != "one key"])
def test_value_scales_far_apart_in_blocks_of_pages(kind):
    # whole tiles of small scales before and behind whole tiles of large ones
    check_attention(spread_case(kind, (87,) * 16 + (227,) * 16), True)
    check_attention(spread_case(kind, (227,) * 16 + (87,) * 16), True)
    check_attention(spread_case(kind, (100,) * 8 + (140,) * 8 + (180,) * 8 + (110,) * 8), True)


@pytest.mark.parametrize("kind", [k for k in (*NARROW, *WIDE) if k != "one key"])
@pytest.mark.parametrize("exps", [(70, 99, 102, 60), (70, 72, 75, 71), (60, 90, 120, 121), (40, 41, 43, 46),
                                  (127, 129, 132, 250)])
def test_value_scales_that_rise_in_steps(kind, exps):
    """A tile of each scale in turn: small steps, a large one, a small one behind it."""
    check_attention(spread_case(kind, tuple(np.repeat(exps, 8))), True)
    check_attention(spread_case(kind, tuple(np.repeat(exps, 2)), page=64), True)


@pytest.mark.parametrize("kind", [k for k in (*NARROW, *WIDE) if k != "one key"])
@pytest.mark.parametrize("low", [0, 1])
def test_large_weights_under_small_value_scales(kind, low):
    """The keys of pages with the small scale stand 60 nats above the others (log-sum-exp tells)."""
    case = spread_case(kind, (87, 227) if low == 0 else (227, 87))
    case.q[:] = 0.0
    case.q[:, ::64] = 4.0
    for _, n, c, pages in case.seqs:
        block = case.cache["k"][pages]
        nan = block[..., 0] == 0x7F
        block[..., 0] = 0
        block[low::2, :, :, 0] = 0x7E
        block[..., 0][nan] = 0x7F
        case.cache["k"][pages] = block
    check_attention(case, True, scale=60.0 / 28.0)


def check_equal_values(kind, code, exp, value):
    """Every value is the same, and so is every mean of them, exactly."""
    lengths, hkv, group = {**NARROW, **WIDE}[kind]
    case = Case(lengths, hkv, group, 64, 32, seed=87, exp_range=(121, 122))
    case.cache["v"][:] = code
    case.cache["v_exp"][:] = exp
    out = check_attention(case, True)
    assert (out.double() == value).all()


@pytest.mark.parametrize("kind", [*NARROW, *WIDE])
def test_largest_finite_values(kind):
    check_equal_values(kind, 0x38, 254, 2.0 ** 127)
    check_equal_values(kind, 0xFE, 245, -448 * 2.0 ** 118)


@pytest.mark.parametrize("kind", [*NARROW, *WIDE])
def test_smallest_value_scales(kind):
    check_equal_values(kind, 0x7E, 1, 448 * 2.0 ** -126)
    check_equal_values(kind, 0xFE, 20, -448 * 2.0 ** -107)
    check_equal_values(kind, 0x7E, 63, 448 * 2.0 ** -64)


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("page", [16, 128])
def test_append_keeps_scales_above_its_own_largest(hd, page):
    """Pages of another origin may hold exponents up to 254: kept rows keep their values."""
    for lo, hi in ((226, 232), (240, 255)):
        case = Case([(1, page - 1), (2, 2 * page - 3), (40, page + 1), (page, 5)], 2, 1, hd, page,
                    seed=86, exp_range=(lo, hi))
        case.k *= 2.0 ** 100
        case.v *= 2.0 ** 118
        check_append(case, 0)
