"""draft_verify on bf16 rows, on rows that are views of wider ones and on shared rows, of
vocabularies that several CTAs of a request divide between them."""

from __future__ import annotations

import numpy as np
import pytest

import tree_ref as ref
from gpu_util import to_dev_i32
from test_gpu_draft_verify import check, gb, inputs, softmax_rows  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("drawn", [True, False])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("S,Tn,V,kind", [(4, 5, 9001, "binary"), (2, 6, 50257, "star"), (3, 4, 131072, "random"),
                                         (100, 3, 20000, "star")])
def test_rows_over_several_ctas(gb, drawn, dtype, S, Tn, V, kind):
    rng = np.random.default_rng(V + drawn)
    p, q = softmax_rows(rng, S, Tn, V)
    # nodes outermost, rows of V + 5 values of which the first two belong to nobody
    views = []
    for x in (p, q):
        wide = torch.full((Tn, S, V + 5), 0.5, dtype=dtype, device="cuda")
        views.append(wide[:, :, 2:V + 2].transpose(0, 1))
        views[-1].copy_(torch.from_numpy(x))
    hp, hq = (v.float().cpu().numpy() for v in views)
    parents, tokens = inputs(rng, S, Tn, V, kind, hp, hq if drawn else None)
    if kind == "star":  # siblings of one node
        parents[:, 1:] = 0
    u = rng.random((S, Tn), dtype=np.float32)
    args = [to_dev_i32(tokens), to_dev_i32(parents), torch.from_numpy(u).cuda()]
    dense = [v.contiguous() for v in views]
    want = [ref.verify_plain(hp[r], hq[r] if drawn else None, tokens[r], parents[r], u[r], Tn) for r in range(S)]
    for vp, vq in (views, dense, (views[0], dense[1])):
        got = [t.cpu().numpy() for t in gb.draft_verify(vp, vq if drawn else None, *args)]
        check(got, want, Tn)
    # one row of the target for the nodes of a request, one of the draft for all
    got = [t.cpu().numpy() for t in gb.draft_verify(
        views[0][:, :1].expand(S, Tn, V), views[1][:1, :1].expand(S, Tn, V) if drawn else None, *args)]
    check(got, [ref.verify_plain(np.broadcast_to(hp[r, :1], (Tn, V)),
                                 np.broadcast_to(hq[0, :1], (Tn, V)) if drawn else None,
                                 tokens[r], parents[r], u[r], Tn) for r in range(S)], Tn)
    assert gb.attn_device_status() == (gb.ATTN_OK, 0)
