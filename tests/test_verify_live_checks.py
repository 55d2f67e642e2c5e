"""Verification of a plan's entries on the CPU: refusals of the C ABI and of the binding, what the loop does with an entry
that was not served."""
import numpy as np
import pytest
import torch

import oracle.pages_ref as ref
from sink_aware_masked_gb300 import _lib, rollout

FAKE = 0x10000  # 16-byte aligned, never dereferenced: every call below fails validation first
OK, INVALID, UNSUPPORTED, ALIGNMENT, WORKSPACE = 0, 1, 2, 3, 4


def test_live_refuses():
    from sink_aware_masked_gb300 import build

    build.build()
    lib, f = _lib.load(), FAKE
    ws = lib.sinkattn_verify_workspace_size(0, 5, 10)

    def call(x=f, xs=10, y=f, ys=10, dtype=0, rows=5, drafts=3, vocab=10, d=f, cu=f, live=f, n=2, u=f, t=f, tokens=f,
             logp=f, acc=f, rej=f, w=f, size=ws):
        return lib.sinkattn_verify_live_tokens(x, xs, y, ys, dtype, rows, drafts, vocab, d, cu, live, n, u, t, tokens, logp,
                                               acc, rej, w, size, None)

    assert call(live=f + 2) == ALIGNMENT and call(dtype=3) == INVALID and call(n=4097) == UNSUPPORTED
    assert call(cu=None) == INVALID and call(size=ws - 1) == WORKSPACE and call(w=f + 8) == ALIGNMENT
    assert call(n=0, x=None, cu=None, live=None, t=None, acc=None, rej=None) == OK


def test_live_binding_refuses():
    x, u, cu = torch.zeros((3, 8)), torch.zeros(3), torch.tensor([0, 2, 3], dtype=torch.int32)
    d = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(TypeError, match="live has dtype"):
        rollout.verify_tokens(x, d, u, cu, live=torch.zeros(2))
    with pytest.raises(ValueError, match="live has shape"):
        rollout.verify_tokens(x, d, u, cu, live=cu)


def test_what_is_not_served_must_not_be_rejected():
    """By the oracle: `rejected` of an entry without a page, fed to the next plan, drops history; 0 keeps it."""
    lens = []
    for rejected in (2, 0):
        c = ref.Pages(2, 2, 2, 1, 16)
        c.plan([0, 1], [0, 0], [16, 14], 30)
        live, cu, places, _ = c.plan([0, 1], [0, 0], [3, 2], 5)  # slot 0 needs a third page
        assert list(live) == [-1, 1] and list(cu) == [0, 3, 5] and list(places) == [-1, -1, -1, 30, 31]
        c.plan([0, 1], [rejected, 0], [0, 0], 0)
        lens.append(int(c.lens[0]))
    assert lens == [14, 16] and np.array_equal(c.owner, [0, 1])
