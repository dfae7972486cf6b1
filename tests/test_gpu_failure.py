"""The device-side failure path without any fault: the library's bounded wait,
run on a barrier that nothing completes, gives up, records CR_ERR_TIMEOUT in
the workspace status word, and the context keeps working afterwards."""

import ctypes
import time

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_bounded_wait_records_timeout_and_context_survives():
    from w4a8_rotated_quantized_b200 import binding
    import w4a8_rotated_quantized_b200 as cr

    ws = torch.zeros(1 << 12, dtype=torch.uint8, device="cuda")
    t0 = time.time()
    binding.cr_selftest_wait_timeout(ws)
    torch.cuda.synchronize()
    elapsed = time.time() - t0
    st = ctypes.c_int(-1)
    assert binding._lib.cr_read_device_status(binding._ptr(ws), ctypes.byref(st), binding._stream(ws.device)) == 0
    assert st.value == 7  # CR_ERR_TIMEOUT
    assert 1.0 < elapsed < 30.0  # the wait gave up after its limit, not at once and not never
    # the context is intact: a normal call on a fresh workspace runs and reports no error
    X = torch.randn((64, 512), device="cuda").to(torch.bfloat16)
    Xq, s = cr.cr_rotate_quant_act(X)
    torch.cuda.synchronize()
    assert np.isfinite(s.item()) and s.item() > 0


def test_a_wait_that_ran_out_is_found_without_a_workspace():
    """The calls that take their own scratch note a wait that ran out where it can still be asked for."""
    from w4a8_rotated_quantized_b200 import binding
    import w4a8_rotated_quantized_b200 as cr

    X = torch.randn((200, 512), device="cuda").to(torch.bfloat16)
    down = torch.randn((1, 16, 512), device="cuda").to(torch.bfloat16)
    up, scale = torch.randn((1, 16, 256), device="cuda").to(torch.bfloat16), torch.ones(1, device="cuda")
    want = cr.cr_lora_forward(X, down, up, scale)
    cr.cr_ckpt_load(*cr.cr_ckpt_save(X))
    Wq, s = cr.cr_pack_weight(X)
    for M in (3, 600):
        cr.cr_w4a4_grad_input(torch.ones((M, 200), device="cuda", dtype=torch.bfloat16), Wq, s)
    assert cr.cr_read_device_status() == 0
    assert binding._lib.cr_selftest_lost_wait(binding._stream(X.device)) == 0
    got = cr.cr_lora_forward(X, down, up, scale)  # a call afterwards does not hide it
    assert cr.cr_read_device_status() == 7  # CR_ERR_TIMEOUT
    assert cr.cr_read_device_status() == 0  # told once
    assert torch.equal(got, want)


def test_status_is_read_on_another_stream_and_for_a_device():
    import w4a8_rotated_quantized_b200 as cr

    with torch.cuda.stream(torch.cuda.Stream()):
        assert cr.cr_read_device_status() == 0 and cr.cr_read_device_status(torch.device("cuda", 0)) == 0
