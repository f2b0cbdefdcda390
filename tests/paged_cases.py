"""Random paged-cache batches for the tests (inputs only; no method arithmetic)."""
import numpy as np
import torch


class Case:
    """A batch of sequences with (new, cached) row counts over shuffled pages.

    Pages hold codes of N(0, 1) values under the exponents of `exp_range`;
    positions behind each sequence hold NaN codes, as does every spare page.
    """

    def __init__(self, lengths, hkv, group, hd, page, seed=0, exp_range=(119, 122), pad_rows=0,
                 extra_ld=0, spread=0.0):
        rng = np.random.default_rng(seed)
        self.lengths, self.hkv, self.group, self.hd, self.page = lengths, hkv, group, hd, page
        self.hq = hkv * group
        B = len(lengths)
        need = [-(-(n + c) // page) for n, c in lengths]
        self.max_pages = max(1, max(need))
        self.n_pages = sum(need) + 3
        perm = rng.permutation(self.n_pages)
        self.table = np.full((B, self.max_pages), -7, np.int32)  # unused entries are no page ids
        self.T = sum(n for n, _ in lengths) + pad_rows
        self.tok_start = np.zeros(B + 1, np.int32)
        self.seqs, at = [], 0
        g = torch.Generator().manual_seed(seed)
        codes = {}
        for name in "kv":
            x = torch.randn((self.n_pages, hkv, page, hd), generator=g) * 90
            codes[name] = x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).numpy().copy()
            codes[name + "_exp"] = rng.integers(*exp_range, size=(self.n_pages, hkv)).astype(np.uint8)
        used = np.zeros(self.n_pages, bool)
        for b, (n, c) in enumerate(lengths):
            ids = perm[at:at + need[b]]
            at += need[b]
            self.table[b, :need[b]] = ids
            used[ids] = True
            self.tok_start[b + 1] = self.tok_start[b] + n
            self.seqs.append((int(self.tok_start[b]), n, c, ids))
            if (n + c) % page:
                for name in "kv":
                    codes[name][ids[-1], :, (n + c) % page:] = 0x7F
        for name in "kv":
            codes[name][~used] = 0x7F
        self.cache = codes
        self.cache_len = np.array([c for _, c in lengths], np.int32)
        self.max_new = max(n for n, _ in lengths)
        self.max_prefix = max(c for _, c in lengths)

        def bf16(cols):
            x = torch.randn((self.T, cols + extra_ld), generator=g)
            if spread:  # heads and elements of unequal size
                x = x * torch.exp(spread * torch.randn(cols + extra_ld, generator=g))
            return x.to(torch.bfloat16)[:, :cols]

        self.q, self.k, self.v = bf16(self.hq * hd), bf16(hkv * hd), bf16(hkv * hd)

    def heads(self, name):
        x = getattr(self, name)
        return x.float().numpy().reshape(self.T, -1, self.hd)

    def device(self):
        """(PagedCache, page_table, tok_start, cache_len) on the GPU, from copies."""
        import canvas_denoising_denoise_b200 as dg
        cache = dg.PagedCache(*[torch.from_numpy(self.cache[n].copy()).cuda()
                                for n in ("k", "v", "k_exp", "v_exp")])
        return (cache, torch.from_numpy(self.table).cuda(), torch.from_numpy(self.tok_start).cuda(),
                torch.from_numpy(self.cache_len).cuda())
