"""Calls at the edge of the multi-token operators' entry points that need no GPU."""
from persistent_moe_decode_cta_gb300 import binding as B


def test_op_status_needs_somewhere_to_write():
    assert B.load_library().mk_op_status(None, None) == B.MK_ERR_INVALID
