"""dg_kv_append_e4m3 and dg_paged_attn_e4m3 against the oracle's paged cache in 64 bits.

Appending is exact: the rotation's fp32 operations, the scales and the codes
are compared bit for bit.  Attention's bound is that of its roundings:
  the result's bf16 rounding, half a step:                2^-8 |out|;
  a probability's f16 rounding, 2^-11 of each: a weighted mean of values moves
  by at most                                              2^-11 max|v|,
  and as much again for exp2 and the fp32 sums;
  a query element below 2^-10 of its row's largest is off by at most 2^-18 of
  it, a score by ds = 2^-18 max|q| scale max_j sum|k_j|:  lse by ds, and the
  result by 2 ds max|v|.
"""
import numpy as np
import pytest
import torch

from oracle import paged
from paged_cases import Case

pytestmark = pytest.mark.gpu


def dg():
    import canvas_denoising_denoise_b200 as m
    return m


def rope_for(case, rot, base=10000.0):
    n = max(a + b for a, b in case.lengths)
    return None if not rot else dg().rope_table(n, rot, base)


def run_append(case, rot, interleaved=False, dev=None, with_q=True):
    d = dg()
    cache, table, starts, lens = dev or case.device()
    rope = rope_for(case, rot)
    k, v, q = case.k.cuda(), case.v.cuda(), case.q.cuda()
    q_out = torch.full((case.T, case.hq * case.hd), 7.0, dtype=torch.bfloat16, device="cuda")
    if not rot or not with_q:
        q = q_out = None
    d.kv_append_e4m3(k, v, cache, table, starts, lens, case.max_new, rope=rope,
                     interleaved=interleaved, q=q, q_out=q_out)
    torch.cuda.synchronize()
    d.check_device_errors()
    return cache, rope, q_out


def check_append(case, rot, interleaved=False):
    cache, rope, q_out = run_append(case, rot, interleaved)
    want = {n: x.copy() for n, x in case.cache.items()}
    rp = None if rope is None else rope.cpu().numpy()
    paged.append(want, case.seqs, case.heads("k"), case.heads("v"), rp, interleaved)
    for name, got in (("k_exp", cache.k_exp), ("v_exp", cache.v_exp)):
        assert np.array_equal(got.cpu().numpy(), want[name]), name
    for name, got in (("k", cache.k_pages), ("v", cache.v_pages)):
        # untouched rows too: the whole pool
        a, b = paged.fp8_values(got.cpu().numpy()), paged.fp8_values(want[name])
        assert np.array_equal(a, b, equal_nan=True), name
    if q_out is not None:
        got = q_out.float().cpu().numpy().reshape(case.T, case.hq, case.hd)
        ref = np.full_like(got, 7.0)  # rows of no sequence stay as they were
        for t0, n, c0, _ in case.seqs:
            if n:
                r = paged.rotate(case.heads("q")[t0:t0 + n], rp, np.arange(c0, c0 + n), interleaved)
                ref[t0:t0 + n] = torch.from_numpy(r).to(torch.bfloat16).float().numpy()
        assert np.array_equal(got, ref)
    return cache


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_append_pages_and_ragged_lengths(hd, page):
    check_append(Case([(1, 0), (37, 21), (0, 9), (129, 3), (1, 127), (5, 128), (260, 300)], 3, 2,
                      hd, page, seed=page, pad_rows=3, extra_ld=8), hd)


@pytest.mark.parametrize("hd,rot,interleaved", [(128, 16, False), (128, 64, True), (128, 128, True),
                                                (64, 32, False), (64, 48, True), (64, 0, False),
                                                (128, 0, False), (128, 80, False)])
def test_append_rotations(hd, rot, interleaved):
    check_append(Case([(19, 40), (3, 1000)], 2, 5, hd, 32, seed=rot, spread=1.0), rot, interleaved)


@pytest.mark.parametrize("hkv,group", [(1, 1), (1, 16), (5, 3), (16, 2)])
def test_append_head_counts(hkv, group):
    check_append(Case([(33, 15), (2, 31)], hkv, group, 64, 16, seed=hkv), 64)


def test_append_grows_and_keeps_scales():
    # old scales far below and far above what the new rows need
    for lo, hi in ((90, 95), (140, 150)):
        check_append(Case([(1, 15), (2, 29), (40, 17)], 2, 1, 128, 32, seed=lo, exp_range=(lo, hi)), 0)


def test_append_extremes():
    """Zeros, infinities, NaN, values past the scales' range."""
    case = Case([(64, 0), (16, 16)], 2, 1, 64, 16, seed=9)
    case.k[:16] = 0.0
    case.k[16:20, 5] = float("inf")
    case.k[21, 70] = float("-inf")
    case.v[3, 7] = float("nan")
    case.v[32:48] *= 2.0 ** -100
    case.v[48:64] *= 2.0 ** 120
    case.v[64] = float("inf")
    check_append(case, 0)


def test_append_twice_is_append_once_and_canvas_rewrites():
    case = Case([(100, 77), (256, 0)], 2, 2, 128, 64, seed=11)
    dev = case.device()
    first = run_append(case, 128, dev=dev)[0]
    once = [t.clone() for t in (first.k_pages, first.v_pages, first.k_exp, first.v_exp)]
    run_append(case, 128, dev=dev)
    for a, b in zip(once, (first.k_pages, first.v_pages, first.k_exp, first.v_exp)):
        assert torch.equal(a, b)


def test_append_queries_in_place_and_strided():
    d = dg()
    case = Case([(9, 5), (30, 64)], 2, 3, 64, 16, seed=12)
    cache, table, starts, lens = case.device()
    rope = rope_for(case, 64)
    # one projection's output holds q, k and v side by side
    qkv = torch.cat([case.q, case.k, case.v], 1).cuda()
    q, k, v = qkv[:, :384], qkv[:, 384:512], qkv[:, 512:]
    want = run_append(case, 64)
    d.kv_append_e4m3(k, v, cache, table, starts, lens, case.max_new, rope=rope, q=q, q_out=q)
    torch.cuda.synchronize()
    d.check_device_errors()
    assert torch.equal(q, want[2]) and torch.equal(cache.k_pages, want[0].k_pages)
    assert torch.equal(qkv[:, 384:].cpu(), torch.cat([case.k, case.v], 1))


def check_attention(case, causal, scale=None, lse=True, ldo_extra=0, stream=None):
    d = dg()
    cache, table, starts, lens = case.device()
    wide = torch.full((case.T, case.hq * case.hd + ldo_extra), 7.0, dtype=torch.bfloat16,
                      device="cuda")
    out = wide[:, :case.hq * case.hd]
    z = torch.full((case.T, case.hq), 7.0, device="cuda") if lse else None
    d.paged_attn_e4m3(case.q.cuda(), cache, table, starts, lens, case.max_new, case.max_prefix, out,
                      n_q_heads=case.hq, lse=z, scale=scale,
                      mask=d.MASK_CAUSAL if causal else d.MASK_BIDIR)
    torch.cuda.synchronize()
    d.check_device_errors()
    compare(case, out, z, causal, case.hd ** -0.5 if scale is None else scale)
    assert (wide[:, case.hq * case.hd:] == 7.0).all()
    return out


def compare(case, out, z, causal, scale, cache=None, q=None):
    cache = case.cache if cache is None else cache
    q = case.heads("q").astype(np.float64) if q is None else q
    want, wz = paged.attend(cache, case.seqs, q, causal, scale)
    got = out.float().cpu().numpy().astype(np.float64).reshape(want.shape)
    zz = None if z is None else z.cpu().numpy().astype(np.float64)
    inside = np.zeros(case.T, bool)
    worst = 0.0
    for t0, n, c0, pages in case.seqs:
        if not n:
            continue
        inside[t0:t0 + n] = True
        for g in range(case.hkv):
            k = paged.keys_of(cache, "k", pages, g, c0 + n)
            v = paged.keys_of(cache, "v", pages, g, c0 + n)
            hs = slice(g * case.group, (g + 1) * case.group)
            vmax = np.abs(v).max()
            # (rows, heads): what the query split may move a score by
            ds = 2.0 ** -18 * np.abs(q[t0:t0 + n, hs]).max(-1) * scale * np.abs(k).sum(1).max()
            w, o = want[t0:t0 + n, hs], got[t0:t0 + n, hs]
            tol = 2.0 ** -8 * np.abs(w) + ((2.0 ** -10 + 2 * ds) * vmax)[..., None]
            worst = max(worst, float((np.abs(o - w) / tol).max()))
            if zz is not None:
                dz = np.abs(zz[t0:t0 + n, hs] - wz[t0:t0 + n, hs])
                # fp32 scores and sums: a few steps of the largest magnitudes
                ztol = ds + 2.0 ** -19 * (1 + np.abs(wz[t0:t0 + n, hs]))
                worst = max(worst, float((dz / ztol).max()))
    assert worst <= 1.0, worst
    assert (got[~inside] == 7.0).all() and (zz is None or (zz[~inside] == 7.0).all())


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("causal", [False, True])
def test_attention_many_rows(hd, page, causal):
    check_attention(Case([(256, 0), (200, 77), (0, 50), (130, 513), (65, 127)], 2, 2, hd, page,
                         seed=hd + page, pad_rows=2), causal)


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("causal", [False, True])
def test_attention_few_rows(hd, page, causal):
    check_attention(Case([(1, 0), (1, 127), (1, 128), (2, 1000), (0, 9), (1, 3), (5, 126)], 2, 4,
                         hd, page, seed=hd + page + 1, pad_rows=1), causal)


@pytest.mark.parametrize("hkv,group,n", [(1, 1, 1), (3, 1, 300), (1, 7, 40), (2, 16, 1), (1, 32, 2),
                                         (1, 20, 3), (8, 2, 1), (1, 3, 171), (1, 32, 1),
                                         (2, 3, 9), (1, 128, 2), (2, 25, 1)])
def test_attention_groups(hkv, group, n):
    check_attention(Case([(n, 200), (max(1, n - 1), 5)], hkv, group, 128, 32, seed=group), True)
    check_attention(Case([(n, 391)], hkv, group, 64, 16, seed=group), False)


def test_attention_long_key_ranges():
    # splits over keys, and more key tiles than one CTA holds page ids for
    check_attention(Case([(1, 20001)], 1, 2, 64, 16, seed=20), True)
    check_attention(Case([(3, 9000), (1, 40)], 1, 1, 128, 128, seed=21), True)
    check_attention(Case([(140, 5000)], 1, 1, 64, 64, seed=22), False)


def test_attention_scales_differ_between_pages():
    check_attention(Case([(3, 300), (150, 200)], 2, 2, 128, 16, seed=23, exp_range=(112, 125)), True)
    check_attention(Case([(150, 200)], 2, 2, 64, 32, seed=24, exp_range=(112, 125)), False)


def test_attention_peaked_rows_and_small_weights():
    """Scores over a wide range: one key takes most of the weight, thousands share the rest."""
    case = Case([(2, 3000), (130, 2000)], 1, 2, 64, 64, seed=25, spread=0.7)
    case.q *= 4.0
    check_attention(case, True)
    # a sink: key 0 stands 2^10 above the others and its value is zero
    case = Case([(2, 4000), (140, 4000)], 1, 1, 64, 64, seed=26, exp_range=(119, 120))
    case.q[:] = 0.0
    case.q[:, 0] = 4.0
    for _, _, _, pages in case.seqs:
        case.cache["k"][pages, 0, :, 0] = 0
        case.cache["k"][pages[0], 0, 0, 0] = 0x7E  # 448 / 256 * 4 / 8 = 0.875
        case.cache["v"][pages[0], 0, 0, :] = 0
    check_attention(case, True, scale=8.0)


def test_attention_options():
    case = Case([(20, 100), (300, 40)], 2, 2, 64, 32, seed=27, extra_ld=16)
    check_attention(case, True, scale=0.05, lse=False, ldo_extra=24)
    one = check_attention(case, False)
    two = check_attention(case, False)
    assert torch.equal(one, two)


def test_attention_nan_and_infinity_stay_in_their_rows():
    d = dg()
    for n, c0 in ((3, 50), (300, 40)):
        case = Case([(n, c0), (n, c0 + 1)], 1, 2, 64, 16, seed=28)
        clean = check_attention(case, True)
        case.q[1, 3] = float("nan")
        case.q[2, 70] = float("-inf")
        cache, table, starts, lens = case.device()
        out = torch.zeros((case.T, 128), dtype=torch.bfloat16, device="cuda")
        d.paged_attn_e4m3(case.q.cuda(), cache, table, starts, lens, n, c0 + 1, out, n_q_heads=2,
                          mask=d.MASK_CAUSAL)
        assert out[1, :64].isnan().all() and out[2, 64:].isnan().all()
        out[1, :64], out[2, 64:] = clean[1, :64], clean[2, 64:]
        assert torch.equal(out, clean)


def test_append_then_attend_as_a_program_does():
    """A prompt in two causal pieces, a canvas written twice, then single tokens, on one stream."""
    d = dg()
    hkv, group, hd, page = 2, 2, 64, 32
    hq, rot = hkv * group, 64
    plan = [([70, 33], True), ([5, 40], True), ([64, 64], False), ([64, 64], False), ([1, 1], True),
            ([1, 0], True)]
    rope = d.rope_table(512, rot)
    g = torch.Generator().manual_seed(31)
    cache = d.PagedCache.zeros(40, hkv, page, hd)
    ref = {"k": cache.k_pages.cpu().numpy(), "v": cache.v_pages.cpu().numpy(),
           "k_exp": cache.k_exp.cpu().numpy(), "v_exp": cache.v_exp.cpu().numpy()}
    ids = np.random.default_rng(1).permutation(40)[:32].reshape(2, 16).astype(np.int32)
    table = torch.from_numpy(ids).cuda()
    cache_len = torch.zeros(2, dtype=torch.int32, device="cuda")
    have = [0, 0]
    for step, (new, causal) in enumerate(plan):
        T = sum(new)
        qkv = torch.randn((T, (hq + 2 * hkv) * hd), generator=g).to(torch.bfloat16)
        dev = qkv.cuda()
        q, k, v = dev.split([hq * hd, hkv * hd, hkv * hd], 1)
        starts = torch.tensor([0, new[0], T], dtype=torch.int32).cuda()
        turned = torch.empty((T, hq * hd), dtype=torch.bfloat16, device="cuda")
        out = torch.empty((T, hq * hd), dtype=torch.bfloat16, device="cuda")
        z = torch.empty((T, hq), device="cuda")
        d.kv_append_e4m3(k, v, cache, table, starts, cache_len, max(new), rope=rope, q=q,
                         q_out=turned)
        d.paged_attn_e4m3(turned, cache, table, starts, cache_len, max(new), max(have), out,
                          n_q_heads=hq, lse=z, mask=d.MASK_CAUSAL if causal else d.MASK_BIDIR)
        torch.cuda.synchronize()
        d.check_device_errors()
        seqs = [(0, new[0], have[0], ids[0]), (new[0], new[1], have[1], ids[1])]
        hn = qkv.float().numpy().reshape(T, -1, hd)
        rp = rope.cpu().numpy()
        paged.append(ref, seqs, hn[:, hq:hq + hkv], hn[:, hq + hkv:], rp)
        for name, t in (("k", cache.k_pages), ("v", cache.v_pages), ("k_exp", cache.k_exp),
                        ("v_exp", cache.v_exp)):
            assert np.array_equal(t.cpu().numpy(), ref[name]), (step, name)
        rows = type("Rows", (), dict(seqs=seqs, T=T, hkv=hkv, group=group))
        compare(rows, out, z, causal, hd ** -0.5, cache=ref,
                q=turned.float().cpu().numpy().reshape(T, hq, hd).astype(np.float64))
        if step != 2:  # the first canvas stays uncommitted and is written again
            cache_len += torch.tensor(new, dtype=torch.int32).cuda()
            have = [a + b for a, b in zip(have, new)]


def test_graph_replay_and_streams():
    """A captured append + attention follows lengths and inputs that change on the device."""
    d = dg()
    case = Case([(1, 1000), (1, 300)], 2, 2, 128, 64, seed=41)
    cache, table, starts, lens = case.device()
    rope = rope_for(case, 128)
    q, k, v = case.q.cuda(), case.k.cuda(), case.v.cuda()
    lens -= 3
    turned = torch.empty((2, 512), dtype=torch.bfloat16, device="cuda")
    out = torch.empty((2, 512), dtype=torch.bfloat16, device="cuda")

    def step(stream=None):
        d.kv_append_e4m3(k, v, cache, table, starts, lens, 1, rope=rope, q=q, q_out=turned,
                         stream=stream)
        d.paged_attn_e4m3(turned, cache, table, starts, lens, 1, 1000, out, n_q_heads=4,
                          mask=d.MASK_CAUSAL, stream=stream)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    step(side)  # an explicit stream other than the current one
    side.synchronize()
    start = [t.clone() for t in (cache.k_pages, cache.v_pages, cache.k_exp, cache.v_exp)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    got = []
    for i in range(3):
        k.copy_(torch.roll(case.k, i, 1))
        graph.replay()
        got.append(out.clone())
        lens += 1
    torch.cuda.synchronize()
    lens -= 3
    for t, s in zip((cache.k_pages, cache.v_pages, cache.k_exp, cache.v_exp), start):
        t.copy_(s)
    for i in range(3):
        k.copy_(torch.roll(case.k, i, 1))
        step()
        assert torch.equal(out, got[i])
        lens += 1
    torch.cuda.synchronize()
    d.check_device_errors()


@pytest.mark.parametrize("rows", [1, 40])
def test_device_checks_leave_memory_alone(rows):
    """Lengths and page ids that do not fit: reported, and only their own rows left out."""
    d = dg()
    case = Case([(rows, 20), (rows, 40)], 1, 2, 64, 16, seed=43)

    def attempt(change, max_new=rows, max_prefix=40):
        cache, table, starts, lens = case.device()
        change(table, starts, lens)
        before = [t.clone() for t in (cache.k_pages, cache.v_pages, cache.k_exp, cache.v_exp)]
        d.kv_append_e4m3(case.k.cuda(), case.v.cuda(), cache, table, starts, lens, max_new)
        torch.cuda.synchronize()
        with pytest.raises(d.DgError) as e:
            d.check_device_errors()
        assert e.value.status == 7
        out = torch.full((case.T, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        d.paged_attn_e4m3(case.q.cuda(), cache, table, starts, lens, max_new, max_prefix, out,
                          n_q_heads=2)
        torch.cuda.synchronize()
        with pytest.raises(d.DgError) as e:
            d.check_device_errors()
        assert e.value.status == 7
        return cache, before, out

    def same(cache, before, pages):
        for t, s in zip((cache.k_pages, cache.v_pages, cache.k_exp, cache.v_exp), before):
            assert torch.equal(t[pages], s[pages])

    mine = torch.from_numpy(case.seqs[0][3].astype(np.int64)).cuda()
    good = case.seqs[1]

    for bad in (-1, 1 << 20):  # a cached length that is negative, or past the table
        def change(table, starts, lens, bad=bad):
            lens[0] = bad
        cache, before, out = attempt(change)
        same(cache, before, mine)
        assert (out[:rows] == 7.0).all() and not (out[rows:] == 7.0).all()

    def change(table, starts, lens):  # rows past T
        starts[2] = case.T + 1
    cache, before, out = attempt(change)
    same(cache, before, torch.from_numpy(good[3].astype(np.int64)).cuda())
    assert (out[rows:] == 7.0).all()

    for bad in (-3, case.n_pages, 2 ** 31 - 1):  # the page that the new rows start in
        def change(table, starts, lens, bad=bad):
            table[0, 1] = bad
        cache, before, out = attempt(change)
        want = [p for p in range(case.n_pages) if p not in set(mine.tolist()) | set(good[3].tolist())]
        same(cache, before, torch.tensor(want).cuda())
        assert torch.isfinite(out[rows:].float()).all()


def test_more_rows_than_the_bound_are_reported():
    d = dg()
    case = Case([(6, 20), (2, 40)], 1, 2, 64, 16, seed=44)
    cache, table, starts, lens = case.device()
    out = torch.full((case.T, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    d.paged_attn_e4m3(case.q.cuda(), cache, table, starts, lens, 4, 40, out, n_q_heads=2)
    torch.cuda.synchronize()
    with pytest.raises(d.DgError):
        d.check_device_errors()
    assert (out[:6] == 7.0).all() and not (out[6:] == 7.0).all()
    d.paged_attn_e4m3(case.q.cuda(), cache, table, starts, lens, 6, 30, out, n_q_heads=2)
    torch.cuda.synchronize()
    with pytest.raises(d.DgError):  # a prefix past its bound
        d.check_device_errors()


def test_wrapper_refuses():
    d = dg()
    case = Case([(4, 20)], 1, 2, 64, 16, seed=45)
    cache, table, starts, lens = case.device()
    q, k, v = case.q.cuda(), case.k.cuda(), case.v.cuda()
    out = torch.empty_like(q)
    bad = [
        lambda: d.kv_append_e4m3(k.float(), v, cache, table, starts, lens, 4),
        lambda: d.kv_append_e4m3(k, v[:3], cache, table, starts, lens, 4),
        lambda: d.kv_append_e4m3(k, v, cache, table.long(), starts, lens, 4),
        lambda: d.kv_append_e4m3(k, v, cache, table, starts[:1], lens, 4),
        lambda: d.kv_append_e4m3(k.cpu(), v, cache, table, starts, lens, 4),
        lambda: d.paged_attn_e4m3(q, cache, table, starts, lens, 4, 20, out, n_q_heads=3),
        lambda: d.paged_attn_e4m3(q, cache, table, starts, lens, 4, 20, out[:3], n_q_heads=2),
        lambda: d.paged_attn_e4m3(q.half(), cache, table, starts, lens, 4, 20, out, n_q_heads=2),
        lambda: d.paged_attn_e4m3(q, cache, table, starts, lens, 4, 20, out, n_q_heads=2,
                                  lse=torch.empty(4, 3, device="cuda")),
    ]
    for f in bad:
        with pytest.raises(ValueError):
            f()


@pytest.mark.parametrize("B,hkv,group,n", [(48, 8, 2, 1), (24, 8, 2, 40), (300, 1, 2, 1)])
def test_attention_of_more_sequences_than_fit_at_once(B, hkv, group, n):
    """CTAs that outnumber the SMs' slots, over lengths in no order (some sequences idle)."""
    rng = np.random.default_rng(B)
    lengths = [(0 if b % 11 == 5 else n, int(rng.integers(0, 400))) for b in range(B)]
    check_attention(Case(lengths, hkv, group, 64, 32, seed=B), True)


def test_pages_behind_two_gigabytes():
    """Page ids whose codes lie past 2^31 and 2^32 bytes."""
    d = dg()
    case = Case([(3, 130), (40, 100), (1, 500)], 8, 2, 128, 128, seed=51)
    small = case.cache
    far = 33000  # pages of 128 KB: 4.3 GB of codes each for K and V
    shift = far - case.n_pages
    pages = [torch.zeros((far, 8, 128, 128), dtype=torch.uint8, device="cuda") for _ in range(2)]
    exps = [torch.full((far, 8), 127, dtype=torch.uint8, device="cuda") for _ in range(2)]
    for t, name in zip(pages + exps, ("k", "v", "k_exp", "v_exp")):
        t[shift:] = torch.from_numpy(small[name]).cuda()
    cache = d.PagedCache(pages[0], pages[1], exps[0], exps[1])
    table = torch.from_numpy(np.where(case.table >= 0, case.table + shift, -1).astype(np.int32)).cuda()
    starts, lens = torch.from_numpy(case.tok_start).cuda(), torch.from_numpy(case.cache_len).cuda()
    q, k, v = case.q.cuda(), case.k.cuda(), case.v.cuda()
    out = torch.full((case.T, 16 * 128), 7.0, dtype=torch.bfloat16, device="cuda")
    d.kv_append_e4m3(k, v, cache, table, starts, lens, case.max_new)
    d.paged_attn_e4m3(q, cache, table, starts, lens, case.max_new, case.max_prefix, out,
                      n_q_heads=16, mask=d.MASK_CAUSAL)
    torch.cuda.synchronize()
    d.check_device_errors()
    paged.append(small, case.seqs, case.heads("k"), case.heads("v"))
    for t, name in zip(pages + exps, ("k", "v", "k_exp", "v_exp")):
        assert np.array_equal(t[shift:].cpu().numpy() & 0x7F, small[name] & 0x7F), name
        assert int(t[:shift].max()) in (0, 127)
    compare(case, out, None, True, 128 ** -0.5)


def test_two_captured_graphs_do_not_share_scratch():
    """Two graphs captured without a workspace, replayed at the same time on two streams."""
    d = dg()
    cases = [Case([(60, 1500)], 1, 2, 128, 64, seed=61), Case([(1, 5000)], 2, 2, 128, 64, seed=62)]
    runs = []
    for case in cases:
        dev = case.device()
        q = case.q.cuda()
        out = torch.zeros((case.T, case.hq * 128), dtype=torch.bfloat16, device="cuda")

        def call(dev=dev, q=q, out=out, case=case):
            d.paged_attn_e4m3(q, *dev, case.max_new, case.max_prefix, out, n_q_heads=case.hq,
                              mask=d.MASK_CAUSAL)

        call()
        torch.cuda.synchronize()
        want = out.clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        runs.append((graph, out, want, torch.cuda.Stream(), dev, q))
    for _ in range(20):
        for graph, out, _, stream, _, _ in runs:
            out.zero_()
        torch.cuda.synchronize()
        for graph, _, _, stream, _, _ in runs:
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        for _, out, want, _, _, _ in runs:
            assert torch.equal(out, want)
    d.check_device_errors()


def test_nan_codes_reach_the_rows_that_see_them():
    d = dg()
    for n in (2, 300):
        case = Case([(n, 60), (n, 61)], 1, 2, 64, 16, seed=63)
        pages = case.seqs[0][3]
        case.cache["v"][pages[0], 0, 3, 5] = 0x7F  # position 3 of the first sequence, element 5
        cache, table, starts, lens = case.device()
        out = torch.zeros((case.T, 128), dtype=torch.bfloat16, device="cuda")
        d.paged_attn_e4m3(case.q.cuda(), cache, table, starts, lens, n, 61, out, n_q_heads=2,
                          mask=d.MASK_CAUSAL)
        bad = out.float().isnan()
        assert bad[:n, [5, 69]].all() and int(bad.sum()) == 2 * n


def test_append_and_attention_on_two_streams_at_once():
    """Two batches with their own caches, in flight together."""
    d = dg()
    cases = [Case([(64, 300), (200, 17)], 2, 2, 128, 32, seed=71),
             Case([(1, 900)] * 9, 2, 4, 128, 64, seed=72)]
    streams = [torch.cuda.Stream() for _ in cases]
    state = []
    for case in cases:
        dev = case.device()
        state.append((case, dev, case.q.cuda(), case.k.cuda(), case.v.cuda(), rope_for(case, 128),
                      torch.zeros((case.T, case.hq * 128), dtype=torch.bfloat16, device="cuda"),
                      torch.zeros((case.T, case.hq * 128), dtype=torch.bfloat16, device="cuda")))
    torch.cuda.synchronize()
    for _ in range(5):
        for stream, (case, dev, q, k, v, rope, turned, out) in zip(streams, state):
            d.kv_append_e4m3(k, v, *dev, case.max_new, rope=rope, q=q, q_out=turned, stream=stream)
            d.paged_attn_e4m3(turned, *dev, case.max_new, case.max_prefix, out, n_q_heads=case.hq,
                              mask=d.MASK_CAUSAL, stream=stream)
    torch.cuda.synchronize()
    d.check_device_errors()
    for case, dev, q, k, v, rope, turned, out in state:
        paged.append(case.cache, case.seqs, case.heads("k"), case.heads("v"), rope.cpu().numpy())
        compare(case, out, None, True, 128 ** -0.5,
                q=turned.float().cpu().numpy().reshape(case.T, case.hq, 128).astype(np.float64))
