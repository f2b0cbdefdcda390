"""The paged 8-bit KV cache operators as measured cases: plain forms, the library's calls, and the definitions in 64 bits.

Two operators share one cache.  `append` rotates new keys and queries by their
positions and stores the keys and values of a batch's new rows in the pages of
an e4m3 cache; `attend` lets those new rows attend to everything cached.

The cache holds codes [n_pages, Hkv, page, hd] (e4m3) for K and for V, and one
power-of-two scale 2^(exp - 127) for each page and kv head.  Position p of
sequence b lies in row p % page of page page_table[b, p // page].  Sequence b's
new rows are the token rows tok_start[b] .. tok_start[b + 1] - 1 and take the
positions cache_len[b], cache_len[b] + 1, ...
"""
import math

import torch

own = False

E_MIN, E_MAX = -40, 100  # exponents a page's scale may have


def listed():
    return [
        # one generated token of one sequence: the latency of the smallest append
        dict(name="append_token_b1", op="append", batch=1, new=1, prefix=4103, ragged=False,
             hq=16, hkv=8, hd=128, page=64, rot=128, interleaved=False),
        # a decoding batch, small pages, every sequence at another offset in its page
        dict(name="append_token_b64", op="append", batch=64, new=1, prefix=2048, ragged=True,
             hq=32, hkv=8, hd=128, page=16, rot=128, interleaved=False),
        # the 256-token canvases of eight sequences, written again in every denoising step
        dict(name="append_canvas_b8", op="append", batch=8, new=256, prefix=2048, ragged=True,
             hq=16, hkv=8, hd=128, page=64, rot=128, interleaved=False),
        # four long prompts of unequal length
        dict(name="append_prompt_b4", op="append", batch=4, new=4096, prefix=300, ragged=True,
             hq=16, hkv=8, hd=128, page=128, rot=128, interleaved=False),
        # small heads, odd lengths, half of each head rotated in adjacent pairs
        dict(name="append_hd64_b3", op="append", batch=3, new=77, prefix=129, ragged=True,
             hq=4, hkv=2, hd=64, page=32, rot=32, interleaved=True),
        # one generated token of one sequence: the latency of the smallest attention
        dict(name="attend_token_b1", op="attend", batch=1, new=1, prefix=4096, ragged=False,
             hq=16, hkv=8, hd=128, page=64, causal=True),
        # a decoding batch over long and unequal prefixes: the cache's bytes bound it
        dict(name="attend_token_b64", op="attend", batch=64, new=1, prefix=8192, ragged=True,
             hq=32, hkv=8, hd=128, page=64, causal=True),
        # the denoising step's canvas over a 4096-token prompt
        dict(name="attend_canvas_b1", op="attend", batch=1, new=256, prefix=4096, ragged=False,
             hq=16, hkv=8, hd=128, page=64, causal=False),
        # the canvas over a 32768-token prompt: the matrix products bound it
        dict(name="attend_canvas_32k", op="attend", batch=1, new=256, prefix=32768, ragged=False,
             hq=32, hkv=8, hd=128, page=128, causal=False),
        # eight canvases over unequal prefixes in small pages
        dict(name="attend_canvas_b8", op="attend", batch=8, new=256, prefix=4096, ragged=True,
             hq=16, hkv=8, hd=128, page=32, causal=False),
        # a prompt's causal pass behind an earlier turn of odd length
        dict(name="attend_prompt_b1", op="attend", batch=1, new=4096, prefix=1031, ragged=False,
             hq=16, hkv=8, hd=128, page=128, causal=True),
        # small heads, short odd lengths, the smallest pages
        dict(name="attend_hd64_b5", op="attend", batch=5, new=61, prefix=513, ragged=True,
             hq=4, hkv=2, hd=64, page=16, causal=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(("token", "token", "canvas", "prompt"))
    op = rng.choice(("append", "attend", "attend"))
    hd = rng.choice((64, 128, 128))
    hkv, group = rng.choice(((2, 2), (4, 4), (8, 1), (8, 2), (8, 4), (4, 8), (1, 16)))
    page = rng.choice((16, 32, 64, 128))
    if kind == "token":
        batch, new, prefix = _log_int(rng, 1, 48), rng.choice((1, 1, 1, 2, 5)), _log_int(rng, 1, 8000)
    elif kind == "canvas":
        batch, new, prefix = rng.randint(1, 4), rng.randint(200, 256), _log_int(rng, 16, 8000)
    else:
        batch, new, prefix = rng.randint(1, 2), _log_int(rng, 30, 2500), rng.choice((0, _log_int(rng, 1, 2000)))
    case = dict(op=op, batch=batch, new=new, prefix=prefix, ragged=batch > 1 and rng.random() < 0.7,
                hq=hkv * group, hkv=hkv, hd=hd, page=page)
    if op == "append":
        case["rot"] = rng.choice((hd, hd, hd // 2))
        case["interleaved"] = rng.random() < 0.3
    else:
        case["causal"] = kind != "canvas"
    return case


def _lengths(case):
    """New rows and cached rows of each sequence: the case's own, or shares of them from 20 to 100 percent."""
    new, old = [], []
    for b in range(case["batch"]):
        share = 1.0 if not case["ragged"] else 0.2 + 0.8 * ((b * 37 + 63) % 64) / 63
        old.append(int(case["prefix"] * share))
        share = 1.0 if not case["ragged"] else 0.2 + 0.8 * ((b * 23 + 63) % 64) / 63
        new.append(max(1, int(case["new"] * share)))
    return new, old


def work(case):
    new, old = _lengths(case)
    rows, hq, hkv, hd = sum(new), case["hq"], case["hkv"], case["hd"]
    if case["op"] == "append":
        # bf16 in, codes out, for K and V; bf16 in and out for the queries; cos and sin of each row
        nbytes = rows * (2 * hkv * hd * 3 + hq * hd * 4 + case["rot"] * 4)
        return {"bytes": nbytes, "flops": rows * (hq + hkv) * case["rot"] * 3}
    keys = sum(n + c for n, c in zip(new, old))
    if case["causal"]:
        pairs = sum(n * c + n * (n + 1) // 2 for n, c in zip(new, old))
    else:
        pairs = sum(n * (n + c) for n, c in zip(new, old))
    return {"bytes": keys * 2 * hkv * hd + rows * hq * (hd * 4 + 4), "flops": pairs * hq * hd * 4}


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    new, old = _lengths(case)
    b, hq, hkv, hd, page = case["batch"], case["hq"], case["hkv"], case["hd"], case["page"]
    rows = sum(new)
    max_pages = max((n + c + page - 1) // page for n, c in zip(new, old))
    n_pages = b * max_pages + 1
    # pages come from a shared pool in no order
    table = torch.randperm(n_pages, generator=g, device=dev)[:b * max_pages].view(b, max_pages)
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)

    def normal(*size):
        return torch.randn(size, generator=g, device=dev)

    # heads of unequal strength, as trained projections give; one matrix holds q, k and v
    strength = torch.exp(0.5 * normal(hq + 2 * hkv)).repeat_interleave(hd)
    qkv = (normal(rows, (hq + 2 * hkv) * hd) * strength).to(torch.bfloat16)
    # codes in the pages, as an earlier append left them: scaled so that a page's largest is within a factor 2 of 448
    codes = [(normal(n_pages, hkv, page, hd) * 90).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
             for _ in range(2)]
    exps = [torch.randint(127 - 8, 127 - 5, (n_pages, hkv), generator=g, device=dev, dtype=torch.uint8)
            for _ in range(2)]
    s = dict(case=case, rows=rows, max_new=max(new), max_prefix=max(old),
             q=qkv[:, :hq * hd], k=qkv[:, hq * hd:(hq + hkv) * hd], v=qkv[:, (hq + hkv) * hd:],
             k_pages=codes[0], v_pages=codes[1], k_exp=exps[0], v_exp=exps[1],
             page_table=table.to(torch.int32).contiguous(),
             tok_start=torch.tensor(starts, dtype=torch.int32, device=dev),
             cache_len=torch.tensor(old, dtype=torch.int32, device=dev))
    if case["op"] == "append":
        half = case["rot"] // 2
        n_pos = max(n + c for n, c in zip(new, old))
        angle = (torch.arange(n_pos, device=dev, dtype=torch.float64)[:, None]
                 * 10000.0 ** (-torch.arange(half, device=dev, dtype=torch.float64) / half))
        s["rope"] = torch.stack([angle.cos(), angle.sin()], -1).float().contiguous()
        s["q_out"] = torch.zeros(rows, hq * hd, dtype=torch.bfloat16, device=dev)
    else:
        s["out"] = torch.zeros(rows, hq * hd, dtype=torch.bfloat16, device=dev)
        s["lse"] = torch.zeros(rows, hq, dtype=torch.float32, device=dev)
    if own:
        import canvas_denoising_denoise_b200 as dg
        s["cache"] = dg.PagedCache(s["k_pages"], s["v_pages"], s["k_exp"], s["v_exp"])
        s["ws"] = dg.Workspace("cuda")
    return s


def run(s):
    if s["case"]["op"] == "append":
        if own:
            import canvas_denoising_denoise_b200 as dg
            dg.kv_append_e4m3(s["k"], s["v"], s["cache"], s["page_table"], s["tok_start"], s["cache_len"],
                              s["max_new"], rope=s["rope"], interleaved=s["case"]["interleaved"], q=s["q"],
                              q_out=s["q_out"])
        else:
            _plain_append(s)
        f8 = torch.float8_e4m3fn
        return dict(q=s["q_out"], k=s["k_pages"].view(f8), v=s["v_pages"].view(f8), k_exp=s["k_exp"],
                    v_exp=s["v_exp"])
    if own:
        import canvas_denoising_denoise_b200 as dg
        dg.paged_attn_e4m3(s["q"], s["cache"], s["page_table"], s["tok_start"], s["cache_len"], s["max_new"],
                           s["max_prefix"], s["out"], n_q_heads=s["case"]["hq"], lse=s["lse"],
                           mask=dg.MASK_CAUSAL if s["case"]["causal"] else dg.MASK_BIDIR, ws=s["ws"])
    else:
        _plain_attend(s)
    return dict(out=s["out"], lse=s["lse"])


# --------------------------------------------------------------------------
# Plain forms: elementary torch operations in 32 bits, rounded once at the end
# --------------------------------------------------------------------------
def _plain_rotate(x, rope, pos, interleaved):
    """x [rows, heads, hd] fp32 with the first rot dimensions of each head rotated by the angles of its row's position."""
    half = rope.shape[1]
    c, s = rope[pos, None, :, 0], rope[pos, None, :, 1]
    if interleaved:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        turned = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        turned = torch.cat([a * c - b * s, b * c + a * s], -1)
    return torch.cat([turned, x[..., 2 * half:]], -1)


def _plain_exponent(amax):
    """The smallest integer e in [E_MIN, E_MAX] with amax <= 448 * 2^e."""
    m, e = torch.frexp(amax)  # amax = m * 2^e with m in [0.5, 1)
    e = torch.where(m <= 0.875, e - 9, e - 8)
    return torch.where(amax > 0, e, E_MIN).clamp(E_MIN, E_MAX)


def _plain_codes(x):
    return x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def _plain_append(s):
    case, rope = s["case"], s["rope"]
    hq, hkv, hd, page = case["hq"], case["hkv"], case["hd"], case["page"]
    start, length, table = s["tok_start"].long(), s["cache_len"].long(), s["page_table"].long()
    row = torch.arange(s["rows"], device=start.device)
    seq = torch.bucketize(row, start[1:], right=True)
    pos = length[seq] + row - start[seq]
    at, slot = table[seq, pos // page], pos % page
    q = _plain_rotate(s["q"].float().unflatten(-1, (hq, hd)), rope, pos, case["interleaved"])
    s["q_out"].copy_(q.flatten(-2))
    k = _plain_rotate(s["k"].float().unflatten(-1, (hkv, hd)), rope, pos, case["interleaved"])
    # a page that already holds rows of its sequence: those stay, under the larger of the scales
    kept = length % page
    first = table.gather(1, (length // page).clamp(max=table.shape[1] - 1)[:, None])[:, 0]
    grows = (start[1:] > start[:-1]) & (kept > 0)
    _plain_store(k, s["k_pages"], s["k_exp"], at, slot, first, kept, grows)
    _plain_store(s["v"].float().unflatten(-1, (hkv, hd)), s["v_pages"], s["v_exp"], at, slot, first, kept, grows)


def _plain_store(x, pages, exps, at, slot, first, kept, grows):
    before = exps.int() - 127
    amax = torch.zeros(exps.shape, device=x.device)
    peak = torch.where(torch.isfinite(x), x.abs(), 0.0).amax(-1)
    amax = amax.index_reduce(0, at, peak, "amax")
    after = before.clone()
    after[at] = _plain_exponent(amax)[at]
    after[first] = torch.where(grows[:, None], torch.maximum(after[first], before[first]), after[first])
    shift = torch.exp2((before[first] - after[first]).float())[:, :, None, None]
    held = pages[first]
    mask = grows[:, None, None, None] & (torch.arange(held.shape[2], device=x.device)[:, None] < kept[:, None, None, None])
    pages[first] = torch.where(mask, _plain_codes(held.view(torch.float8_e4m3fn).float() * shift), held)
    pages[at, :, slot] = _plain_codes(x * torch.exp2(-after[at].float())[..., None])
    exps.copy_(after + 127)


def _plain_attend(s):
    case = s["case"]
    b, hq, hkv, hd, page = case["batch"], case["hq"], case["hkv"], case["hd"], case["page"]
    start, length, table = s["tok_start"].long(), s["cache_len"].long(), s["page_table"].long()
    new = start[1:] - start[:-1]
    dev = start.device

    def keys(pages, exps):  # [b, hkv, positions, hd]
        x = pages[table].view(torch.float8_e4m3fn).float() * torch.exp2(exps[table].float() - 127)[..., None, None]
        return x.permute(0, 2, 1, 3, 4).reshape(b, hkv, -1, hd)

    k, v = keys(s["k_pages"], s["k_exp"]), keys(s["v_pages"], s["v_exp"])
    p = torch.arange(k.shape[2], device=dev)
    i = torch.arange(s["max_new"], device=dev)
    live = p < (length + new)[:, None]
    v = torch.where(live[:, None, :, None], v, 0.0)
    rows = (start[:-1, None] + i).clamp(max=s["rows"] - 1)
    q = s["q"].float()[rows].view(b, len(i), hkv, hq // hkv, hd).permute(0, 2, 3, 1, 4).reshape(b, hkv, -1, hd)
    seen = live[:, None, :]
    if case["causal"]:
        seen = seen & (p <= (length[:, None] + i)[..., None])
    score = (q @ k.transpose(-1, -2) * hd ** -0.5).unflatten(2, (hq // hkv, len(i)))
    score = torch.where(seen[:, None, None], score, -math.inf)
    top = score.amax(-1, keepdim=True)
    weight = torch.exp(score - top)
    total = weight.sum(-1, keepdim=True)
    out = (weight.flatten(2, 3) @ v).unflatten(2, (hq // hkv, len(i))) / total
    inside = i < new[:, None]
    s["out"][rows[inside]] = out.permute(0, 3, 1, 2, 4).reshape(b, len(i), hq * hd)[inside].to(torch.bfloat16)
    s["lse"][rows[inside]] = (top + total.log()).permute(0, 3, 1, 2, 4).reshape(b, len(i), hq)[inside]


# --------------------------------------------------------------------------
# The definitions in 64 bits, sequence by sequence
# --------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    new, old = _lengths(case)
    return _exact_append(s, new, old) if case["op"] == "append" else _exact_attend(s, new, old)


def _nearest_e4m3(x):
    """float64 values rounded to the nearest e4m3 value, ties to the even one, held below 448."""
    x = x.clamp(-448.0, 448.0)
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(x / step) * step).clamp(-448.0, 448.0)


def _exact_append(s, new, old):
    case = s["case"]
    hq, hkv, hd, page, half = case["hq"], case["hkv"], case["hd"], case["page"], case["rot"] // 2
    rope = s["rope"].double()
    cos, sin = rope[..., 0], rope[..., 1]
    dims = torch.arange(half, device=rope.device)
    first, second = (2 * dims, 2 * dims + 1) if case["interleaved"] else (dims, dims + half)

    def turned(x, c0):
        y = x.clone()
        c, d = cos[c0:c0 + len(x), None], sin[c0:c0 + len(x), None]
        y[..., first] = x[..., first] * c - x[..., second] * d
        y[..., second] = x[..., first] * d + x[..., second] * c
        return y

    codes = {n: s[n + "_pages"].view(torch.float8_e4m3fn).double() for n in "kv"}
    exps = {n: s[n + "_exp"].long() for n in "kv"}
    table, q_out, t = s["page_table"].tolist(), [], 0
    for b, (n, c0) in enumerate(zip(new, old)):
        q_out.append(turned(s["q"][t:t + n].double().view(n, hq, hd), c0).view(n, -1))
        x = {"k": turned(s["k"][t:t + n].double().view(n, hkv, hd), c0), "v": s["v"][t:t + n].double().view(n, hkv, hd)}
        for name in "kv":
            for j in range(c0 // page, (c0 + n - 1) // page + 1):
                pg, lo, hi = table[b][j], max(j * page, c0), min((j + 1) * page, c0 + n)
                part = x[name][lo - c0:hi - c0].transpose(0, 1)  # [hkv, rows, hd]
                m, e = torch.frexp(part.abs().amax((1, 2)) / 448)  # the quotient is m * 2^e with m in [0.5, 1), or 0
                e = torch.where(m == 0, E_MIN, torch.where(m == 0.5, e - 1, e)).clamp(E_MIN, E_MAX).long()
                if lo % page:
                    e0 = exps[name][pg] - 127
                    e = torch.maximum(e, e0)
                    codes[name][pg, :, :lo % page] = _nearest_e4m3(
                        codes[name][pg, :, :lo % page] * torch.exp2((e0 - e).double())[:, None, None])
                codes[name][pg, :, lo % page:lo % page + hi - lo] = _nearest_e4m3(part * torch.exp2(-e.double())[:, None, None])
                exps[name][pg] = e + 127
        t += n
    return dict(q=torch.cat(q_out), k=codes["k"], v=codes["v"], k_exp=None, v_exp=None)


def _exact_attend(s, new, old):
    case = s["case"]
    hq, hkv, hd = case["hq"], case["hkv"], case["hd"]
    out, lse, t = [], [], 0
    for b, (n, c0) in enumerate(zip(new, old)):
        pages = s["page_table"][b].long()
        kv = []
        for name in "kv":
            x = s[name + "_pages"][pages].view(torch.float8_e4m3fn).double()
            x = torch.ldexp(x, (s[name + "_exp"][pages].int() - 127)[:, :, None, None])
            kv.append(x.transpose(0, 1).reshape(hkv, -1, hd)[:, :n + c0])
        q = s["q"][t:t + n].double().view(n, hq, hd)
        o, z = torch.empty(n, hq, hd, dtype=torch.float64, device=q.device), torch.empty(n, hq, dtype=torch.float64, device=q.device)
        for h in range(hq):
            score = q[:, h] @ kv[0][h * hkv // hq].T / math.sqrt(hd)
            if case["causal"]:
                score.masked_fill_(torch.ones(n, n + c0, dtype=torch.bool, device=q.device).triu(c0 + 1), -math.inf)
            z[:, h] = torch.logsumexp(score, 1)
            o[:, h] = torch.exp(score - z[:, h, None]) @ kv[1][h * hkv // hq]
        out.append(o.view(n, -1))
        lse.append(z)
        t += n
    return dict(out=torch.cat(out), lse=torch.cat(lse))
