"""Attention over the paged cache where the ordinary problems do not reach: queries that the kernel
holds exactly, so that a result is checked to what the weights' rounding leaves (attention_check)."""
import numpy as np
import pytest
import torch

from tests import attention_check as A
import timestep_adaptive_bit_amd as T

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def ctx():
    c = T.Context()
    yield c
    c.close()


def _run(ctx, p, max_q=None, fill=None):
    d = lambda x: torch.from_numpy(np.ascontiguousarray(x)).to(DEV)       # noqa: E731
    cache = T.KVCache(*[d(p["arr"][x]) for x in ("k_codes", "k_scales", "v_codes", "v_scales")],
                      head_dim=p["D"], had_block=p["had"])
    q = d(p["q"]).bfloat16()
    lse = torch.full(q.shape[:2], 7.0, device=DEV)
    out = None if fill is None else torch.full_like(q, fill)
    out = ctx.kv_attention(cache, q, d(np.asarray(p["cu"], np.int32)), d(p["table"]),
                           d(np.asarray(p["lens"], np.int32)), max_q or int(np.diff(p["cu"]).max()), max(p["lens"]),
                           scale=p["scale"], causal=p["causal"], out=out, lse=lse)
    return out.double().cpu().numpy(), lse.double().cpu().numpy()


def _want(p):
    return A.want(p["q"], p["arr"], p["table"], p["lens"], p["cu"], p["scale"], p["causal"], p["D"], p["had"])


@pytest.mark.parametrize("had", [0, 32])
@pytest.mark.parametrize("hq,hk,D", [(4, 1, 64), (2, 2, 128), (8, 2, 40)])
def test_rows_past_max_q_keep_the_mask(ctx, hq, hk, D, had):
    """Only the first max_q rows of a sequence are computed, and each sees what it sees of the whole
    sequence: the causal limit goes by all of the sequence's queries."""
    p = A.problem(D + hq, [70, 9, 200], [40, 20, 90], hq, hk, D, 16, had, k=3)
    out, lse, room, lroom = _want(p)
    for m in (1, 3, 16, 17, 39, 90):
        print("attention max_q", m, "heads", hq, hk, "D", D, "had", had, flush=True)
        got, glse = _run(ctx, p, m, fill=9.0)
        in_seq = np.concatenate([np.arange(n) for n in np.diff(p["cu"])])
        done = in_seq < m
        A.check(got[done], glse[done], (out[done], lse[done], room[done], lroom[done]))
        assert (got[~done] == 9).all() and (glse[~done] == 7).all()
