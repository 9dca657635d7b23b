"""Calls that need 2^32 threads or more, past what a launch counts, are refused as shapes before anything is launched
(no GPU needed; where the check is missing, the launch is what fails)."""
import pytest

from test_ragged_abi import FAKE, B, _call, _shape

import ctypes


@pytest.mark.parametrize("entry", ["rmw_seq", "prefill"])
@pytest.mark.parametrize("kind,beta", [("gdn", FAKE), ("kda", FAKE), ("mamba2", None)])
def test_sequences(entry, kind, beta):
    # a block of 5 waves per sequence and head: 2^23 x 8 x 320 threads
    assert _call(entry, _shape(kind), n_seqs=1 << 23, total=100, max_len=50, beta=beta) == 2


def test_prefill_chunks():
    # the preparation: 2^31 / 32 chunks of 64 heads, 64 threads each
    assert _call("prefill", _shape(H=64), n_seqs=1, total=2 ** 31 - 1, max_len=2 ** 31 - 1, workspace_bytes=1 << 60) == 2


@pytest.mark.parametrize("heads,H,n", [(1, 8, 1 << 26), (8, 8, 1 << 27), (64, 64, 1 << 25)])
def test_gated_norm_tokens(heads, H, n):
    sh = _shape(H=H)
    assert B.lib().sketchssm_gated_norm(ctypes.byref(sh), FAKE, None, None, FAKE, FAKE, H, heads, 2, 1e-5, n, FAKE,
                                       None) == 2


def test_no_workspace_for_what_is_refused():
    W = B.lib().sketchssm_prefill_workspace
    for sh, n, total in ((_shape(), 1 << 23, 100), (_shape(H=64), 1, 2 ** 31 - 1), (_shape(), 1 << 28, 10000)):
        assert W(ctypes.byref(sh), n, total, 2 ** 31 - 1) == 0
    assert W(ctypes.byref(_shape()), 1 << 12, 100000, 100) > 0
