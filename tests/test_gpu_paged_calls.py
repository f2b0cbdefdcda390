"""The paged calls as programs make them: workspaces that grow, streams, odd widths and bounds."""
import numpy as np
import pytest
import torch

import canvas_denoising_denoise_b200 as dg
import test_gpu_paged as base
from paged_cases import Case

pytestmark = pytest.mark.gpu


def attend(case, dev, q, out, z, **kw):
    cache, table, starts, lens = dev
    dg.paged_attn_e4m3(q, cache, table, starts, lens, case.max_new, case.max_prefix, out,
                       n_q_heads=case.hq, lse=z, mask=dg.MASK_CAUSAL, **kw)


def test_a_workspace_grows_and_serves_smaller_calls_on_a_side_stream():
    cases = [Case([(40, 900)], 1, 1, 128, 64, seed=91), Case([(200, 6000)], 2, 2, 128, 64, seed=92),
             Case([(1, 300)], 2, 2, 64, 16, seed=93), Case([(60, 2000), (3, 40)], 2, 2, 64, 32, seed=94)]
    side, ws, sizes = torch.cuda.Stream(), dg.Workspace("cuda"), []
    state = []
    for case in cases:
        state.append((case, case.device(), case.q.cuda(),
                      torch.zeros((case.T, case.hq * case.hd), dtype=torch.bfloat16, device="cuda"),
                      torch.zeros((case.T, case.hq), device="cuda")))
    torch.cuda.synchronize()
    for _ in range(3):
        for case, dev, q, out, z in state:
            attend(case, dev, q, out, z, ws=ws, stream=side)
            sizes.append(ws.buf.numel() if ws.buf is not None else 0)
            # work of the current stream that would take freed memory
            torch.full((sizes[-1] + 1,), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    dg.check_device_errors()
    assert 0 < sizes[0] < sizes[1] == sizes[2] == sizes[-1]
    for case, dev, q, out, z in state:
        assert torch.isfinite(out.float()).all()
        base.compare(case, out, z, True, case.hd ** -0.5)
