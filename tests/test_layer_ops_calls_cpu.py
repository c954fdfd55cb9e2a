"""Calls of the layer operators that the C entry points or the binding refuse:
workspaces and streams that are not the call's.  No GPU is needed: every refusal
comes before a device call."""
import types

import pytest
import torch

A = [1 << 20 << k for k in range(14)]  # fake pointers, far apart


@pytest.fixture(scope="module")
def capi():
    from nonlinear_rnn_newton_b200 import build
    build.build()
    from nonlinear_rnn_newton_b200 import capi
    return capi


def calls(P):
    """Each operator on small arguments; kw goes to the call."""
    u, rate = torch.zeros(2, 3, 3, 16), torch.zeros(16)
    h, x, r = torch.zeros(2, 3, 16), torch.zeros(4, 32), torch.ones(4)
    q, s = torch.zeros(4, 32).to(torch.float8_e4m3fn), torch.ones(4, 1)
    w, ws = torch.zeros(8, 32).to(torch.float8_e4m3fn), torch.ones(1, 1)
    with_workspace = [
        lambda **kw: P.pararnn_glr_scan(u, rate, **kw),
        lambda **kw: P.pararnn_glr_adjoint(u, rate, None, h, h, **kw),
        lambda **kw: P.pararnn_rms_norm_adjoint(x, x, torch.ones(32), r, **kw),
        lambda **kw: P.pararnn_fp8_project(q, s, w, ws, **kw),
    ]
    others = [
        lambda **kw: P.pararnn_glr_step(torch.zeros(2, 3, 16), rate, **kw),
        lambda **kw: P.pararnn_rms_norm(x, torch.ones(32), **kw),
        lambda **kw: P.pararnn_fp8_quantize(x, **kw),
    ]
    return with_workspace, others


def test_workspace_of_another_device(capi):
    for call in calls(capi)[0]:
        with pytest.raises(ValueError, match="workspace"):
            call(workspace=torch.empty(1 << 16, dtype=torch.uint8, device="meta"))


def test_workspace_with_gaps(capi):
    for call in calls(capi)[0]:
        with pytest.raises(ValueError, match="workspace"):
            call(workspace=torch.empty(2, 1 << 16, dtype=torch.uint8)[:, ::2])


def test_workspace_that_overlaps_an_array(capi):
    """The workspace is written, so it may meet no array of the call."""
    def scan(ws, starts=None):
        return capi.lib.pararnn_glr_scan(A[0], 1, A[1], A[2], starts, A[9], A[3], 8, 2, 16, ws, 1 << 19, None)

    def adjoint(ws):
        return capi.lib.pararnn_glr_adjoint(A[0], 0, A[1], A[2], A[8], A[3], A[4], A[5], A[6], A[7], A[9], 8, 2, 16, ws,
                                            1 << 19, None)

    def norm(ws):
        return capi.lib.pararnn_rms_norm_adjoint(A[0], 1, A[1], 1, A[2], A[3], A[4], A[5], A[6], 4, 32, ws, 1 << 19, None)

    def project(ws):
        return capi.lib.pararnn_fp8_project(A[0], A[1], A[2], A[3], A[4], A[5], 1, 4, 16, 32, ws, 1 << 19, None)

    for call, arrays in ((scan, (0, 1, 2, 3, 9)), (adjoint, range(10)), (norm, range(7)), (project, range(6))):
        for k in arrays:
            assert call(A[k]) == capi.ERR_INVALID_ARG, (call.__name__, k)
            assert "workspace" in capi.last_error()
    assert scan(A[8], starts=A[8]) == capi.ERR_INVALID_ARG
    # beside every array: nothing to refuse (without a GPU the call then fails there;
    # with one it would run on these addresses)
    if not torch.cuda.is_available():
        for call in (scan, adjoint, norm, project):
            assert call(A[12]) == capi.ERR_CUDA, call.__name__


def test_stream_of_another_device(capi):
    """The call would otherwise run on the current stream of the tensors' device."""
    stream = types.SimpleNamespace(device=torch.device("cuda", 1), cuda_stream=0, device_index=1)
    for call in sum(calls(capi), []):
        with pytest.raises(ValueError, match="stream must be one of"):
            call(stream=stream)


def test_failures_cannot_be_asked_for_without_a_device(capi):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    assert capi.lib.pararnn_take_failure(None) == capi.ERR_CUDA
