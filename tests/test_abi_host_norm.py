"""Host side of the gradient norm's workspace."""


def test_work_holds_a_ticket_and_a_slot_for_each_cta_of_each_launch():
    """A call over no tensor still launches one CTA, which writes a slot of
    eight bytes behind the ticket's sixteen."""
    from block_wise_dynamic_gb300 import build as b

    b.build()
    from block_wise_dynamic_gb300 import _abi

    lib = _abi.load()
    assert lib.bwd_grad_norm_work_bytes(0) >= 16 + 8
    for tensors in (1, 1024, 1025, 5000):
        launches = -(-tensors // 1024)
        assert lib.bwd_grad_norm_work_bytes(tensors) >= 16 + 8 * launches * 152 * 8
    assert lib.bwd_grad_norm_work_bytes(-1) == -1
