"""Corners of the training losses, where a call's answer is easily wrong or
refused.  The helpers and tolerances are those of test_losses.py."""

import math

import numpy as np
import pytest
import torch

import loss_reference as ref
import vocab_log_softmax_gb300 as vls
from test_losses import CFG, DEV, DTYPES, INF, _check_distill, _check_policy, _check_preference, _distill_inputs, _gen
from test_losses import _logits, _np, _policy_inputs, _preference_inputs
from vls_compare import assert_grad_close, bitwise_equal, to_f64
from vocab_log_softmax_gb300 import _lib, build
from vocab_log_softmax_gb300 import binding as B

gpu = pytest.mark.gpu
NAN = float("nan")
P = 0x1000   # non-NULL, never dereferenced


# ---------------------------------------------------------------------------
# label smoothing
# ---------------------------------------------------------------------------

@gpu
@pytest.mark.parametrize("kind", ["hinge", "squared"])
def test_label_smoothing_of_the_other_kinds(kind):
    """The hinge and the squared loss have no smoothing: a call that passes one
    (one training configuration for every kind) gets the loss as it is.  A value
    outside [0, 1/2) stays refused."""
    gen = _gen(1)
    x = _logits(7, 515, "bf16", gen)
    ids, offsets, rf, w, margin = _preference_inputs(x, [3, 4], gen)
    want = B.vls_preference_loss(x, ids, offsets, rf, w, margin, kind=kind)
    got = B.vls_preference_loss(x, ids, offsets, rf, w, margin, kind=kind, label_smoothing=0.1)
    for key in want:
        assert bitwise_equal(want[key], got[key]), key
    a = vls.preference_loss(x, ids, offsets, ref_logp=rf, weights=w, margin=margin, kind=kind, label_smoothing=0.1)
    assert bitwise_equal(a[1], want["pair_loss"])
    for wrong in (0.5, -0.1, NAN):
        with pytest.raises(ValueError):
            B.vls_preference_loss(x, ids, offsets, kind=kind, label_smoothing=wrong)


def test_label_smoothing_reaches_the_sigmoid_loss_alone():
    for kind, code in (("sigmoid", 0), ("hinge", 1), ("squared", 2)):
        cfg = B._pref_cfg(kind, True, 0.25, 0.125)
        assert (cfg.kind, cfg.length_average, cfg.beta) == (code, 1, 0.25)
        assert cfg.label_smoothing == (0.125 if kind == "sigmoid" else 0.0)
        assert B._pref_cfg(kind, False, 0.25, 0.5).label_smoothing == 0.5      # for the library to refuse
