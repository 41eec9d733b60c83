"""Fused non-GEMM Transformer-layer operators for GB300 (sm_103a).

The operators -- bias+dropout+residual, bias+ReLU+dropout, LayerNorm and
masked attention softmax, forward and backward -- live in the C-ABI library
``libls_ops.so`` (declared in ``include/ls_ops.h``); :mod:`.ls_ops` binds it.
The vocabulary operators -- linear cross entropy, top-k distillation and the
embedding lookup -- live in ``libls_vocab.so`` (``include/ls_vocab.h``); bound by
:mod:`.ls_vocab`.
"""
from . import ls_ops, ls_vocab  # noqa: F401

__all__ = ["ls_ops", "ls_vocab"]
