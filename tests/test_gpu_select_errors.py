"""A call that the runtime refuses leaves the calls after it alone."""
import ctypes

import pytest
import torch

from test_gpu_select import BF, boxes, fa  # noqa: F401 (fa is a fixture)

pytestmark = pytest.mark.gpu


def test_the_error_of_a_refused_launch_is_not_the_next_calls(fa):  # noqa: F811
    # a stream whose capture was given up takes no launch: the driver says so on the host, and nothing reaches the GPU
    src = fa.create_block_mask(fa.make_mask_rule([("causal",)]), 1, 2, 1, 64 * 10, 1, 64)
    q, box, k = torch.ones(1, 2, 1, 64, dtype=BF, device="cuda"), boxes((1, 1, 10, 2, 64), 1), torch.ones(1, 1, 64, 64, dtype=BF, device="cuda")
    out = fa.select_blocks(src, q, box, 2)
    torch.cuda.synchronize()
    cu, stream, graph = ctypes.CDLL("libcuda.so.1"), ctypes.c_void_p(), ctypes.c_void_p()
    assert cu.cuStreamCreate(ctypes.byref(stream), 1) == 0
    assert cu.cuStreamBeginCapture_v2(stream, 2) == 0              # relaxed: other streams and threads are as ever
    assert cu.cuStreamSynchronize(stream) != 0                     # not permitted in a capture, which ends with it
    refused = fa.load().fa_block_mask_select_blocks(ctypes.byref(src.c), q.data_ptr(), box.data_ptr(), None, 0, 0, 1, 2, 1, 64, 2, 1, 1, out.buf.data_ptr(),
                                                    out.buf.numel(), ctypes.byref(out.c), None, 0, None, stream)
    bounds = torch.empty(1, 1, 1, 2, 64, dtype=BF, device="cuda")
    after = fa.load().fa_key_bounds(k.data_ptr(), bounds.data_ptr(), 1, 1, 64, 64, 64, torch.cuda.current_stream().cuda_stream)
    assert cu.cuStreamEndCapture(stream, ctypes.byref(graph)) != 0
    assert cu.cuStreamDestroy_v2(stream) == 0
    assert refused == fa.ERR_CUDA
    assert after == fa.OK and bool((bounds == 1).all())
