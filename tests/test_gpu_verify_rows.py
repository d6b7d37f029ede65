"""Verification of drafted tokens (gwa_verify_draft) over draft rows that are
not there."""
import numpy as np
import pytest
import torch

import group_wise_affine_gb300 as gwa
from test_gpu_verify import pair, to_device, uniform

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    gwa.build()
    gwa.load()
    assert torch.cuda.is_available()


@pytest.mark.parametrize("R_of", [[3, 1, 4], [5], [2] * 90])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("V", [777, 70001])
def test_draft_rows_that_are_not_there(R_of, bf16, V):
    """Row i of draft_logits is not read where i is a sequence's last row, nor
    a row of no sequence on either side: the buffer may end in front of it."""
    if len(R_of) > 10 and V > 1000:
        V = 9001
    rng = np.random.default_rng(V + len(R_of))
    lead, tail = 2, 3
    rows = lead + sum(R_of) + tail
    x, y = pair(rng, rows, V)
    start = (lead + np.concatenate([[0], np.cumsum(R_of)])).astype(np.int32)
    dx, dy = to_device(x, bf16)[0], to_device(y, bf16)[0]
    t = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    ids, st, u, ud = (t(a) for a in (rng.integers(0, V, rows).astype(np.int32), start, uniform(rng, rows), uniform(rng, len(R_of))))
    ids[1:] = dy[:-1].float().argmax(-1).to(torch.int32)
    want = gwa.verify_draft(dx, ids, st, u, ud, draft_logits=dy)
    # rows [lead, the last row of all): what the call says that it reads
    room = torch.full((sum(R_of) - 1, V), float("nan"), dtype=dy.dtype, device="cuda")
    for a, e in zip(start, start[1:]):
        room[a - lead:e - 1 - lead] = dy[a:e - 1]
    token, accepted, prob = (torch.full_like(w, 99) for w in want)
    work = gwa.make_verify_workspace(rows)
    row = V * dy.element_size()
    gwa._check(gwa.load().gwa_verify_draft(
        dx.data_ptr(), gwa.GWA_BF16 if bf16 else gwa.GWA_FP32, rows, V, V, room.data_ptr() - lead * row, V, ids.data_ptr(),
        st.data_ptr(), len(R_of), u.data_ptr(), ud.data_ptr(), None, None, None, None, token.data_ptr(), accepted.data_ptr(),
        prob.data_ptr(), work.data_ptr(), work.numel(), torch.cuda.current_stream().cuda_stream))
    for a, b in zip((token, accepted, prob), want):
        assert torch.equal(a, b)
