"""Calls of the serving operators that the host has to answer: fields that an operator does not use, host-side rules."""
import ctypes as C

import pytest

from sparse_compressed_attention_gb300 import _lib as L
from sparse_compressed_attention_gb300 import build as B


@pytest.fixture(scope="module")
def lib():
    B.build()
    return L.lib()


@pytest.mark.parametrize("field,value", [("seqlen", 0), ("seqlen", 1 << 30), ("overlap", 7), ("idx_heads", 0), ("idx_dim", 0),
                                         ("idx_dim", 32), ("o_groups", 0), ("o_rank", -1), ("rms_eps", -1.0),
                                         ("indexer_fp8", 5)])
def test_tree_attention_reads_its_own_fields_alone(lib, field, value):
    """The documentation names the configuration's fields that the tree attention uses; the others may hold anything."""
    cfg = L.make_config(2, 1, 64, 512, 64, ratio=4, window=128, topk=512)
    setattr(cfg, field, value)
    n = C.c_size_t(0)
    assert lib.v4_tree_workspace_size(C.byref(cfg), 3, C.byref(n)) == L.V4_OK and n.value > 0
    # a call that is refused for what comes behind the configuration
    assert lib.v4_tree_mqa_fwd(C.byref(cfg), None, 16, 16, 256, 1 << 32, None) == L.V4_ERR_INVALID_ARG
    assert "inputs struct" in lib.v4_last_error().decode()


@pytest.mark.parametrize("field,value,status,text", [
    ("batch", 0, 1, "batch"), ("n_heads", 0, 1, "n_heads"), ("head_dim", 500, 1, "head_dim"), ("rope_dim", 520, 1, "rope_dim"),
    ("ratio", -1, 1, "ratio"), ("window", -2, 1, "window"), ("topk", -1, 1, "topk"), ("ratio", 0, 1, "topk"),
    ("dtype", 4, 1, "dtype"), ("path", 3, 1, "path"), ("q_begin", 1, 2, "q_begin"), ("q_begin", -1, 2, "q_begin")])
def test_tree_attention_checks_its_own_fields(lib, field, value, status, text):
    cfg = L.make_config(2, 1, 64, 512, 64, ratio=4, window=128, topk=512)
    setattr(cfg, field, value)
    v = L.v4_tree_inputs()
    assert lib.v4_tree_mqa_fwd(C.byref(cfg), C.byref(v), 16, 16, 256, 1 << 32, None) == status
    assert text in lib.v4_last_error().decode()
