"""Host-side validation of the scorer's C entry points: every refusal comes
back as a status code before any device call, so it runs without a GPU."""
import ctypes as C
import math
import os
import shutil

import pytest

OK, INVALID, UNSUPPORTED, OVERFLOW = 0, 1, 5, 6


@pytest.fixture(scope="module")
def E():
    if shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"):
        pytest.skip("nvcc not available")
    from entropy_bound_canvas_b200 import build as B
    B.build()
    import entropy_bound_canvas_b200 as E
    return E


def test_structures_match_the_header(E):
    assert C.sizeof(E.ScoreInput) == 56
    assert C.sizeof(E.Policy) == 72
    assert C.sizeof(E.Preference) == 64


def test_init_validates(E):
    lib = E.library()
    h = C.c_void_p()
    assert lib.eb_scorer_init(None, 16, 0) == INVALID
    assert lib.eb_scorer_init(C.byref(h), 0, 0) == INVALID
    assert lib.eb_scorer_init(C.byref(h), -1, 0) == INVALID
    assert lib.eb_scorer_init(C.byref(h), (1 << 24) + 1, 0) == OVERFLOW
    assert not h.value


def test_null_handles_are_refused(E):
    lib = E.library()
    s, p, q = E.ScoreInput(), E.Policy(), E.Preference()
    assert lib.eb_token_logprobs(None, C.byref(s), None, None, None) == INVALID
    assert lib.eb_token_logprobs_backward(None, C.byref(s), None, None, None, 0, None) == INVALID
    assert lib.eb_policy_loss(None, C.byref(s), C.byref(p), None, None, None, None, 0,
                              None) == INVALID
    assert lib.eb_preference_loss(None, C.byref(s), C.byref(q), None, None, None, None, None, 0,
                                  None) == INVALID
    assert lib.eb_lmhead_logprobs(None, None, None, 1, 1, 8, None, None, 1.0, None, None,
                                  None) == INVALID
    assert lib.eb_scorer_status(None, None, 0, None) == INVALID
    assert lib.eb_scorer_set_wait_limit(None, 0) == INVALID
    assert lib.eb_scorer_workspace_bytes(None) == 0
    lib.eb_scorer_destroy(None)
