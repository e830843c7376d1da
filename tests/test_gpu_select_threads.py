"""Choices made by two host threads at once."""
import ctypes
import threading

import pytest
import torch

from test_gpu_select import BF, boxes, fa, gen  # noqa: F401 (fa is a fixture)

pytestmark = pytest.mark.gpu


# Rows whose keys need 42 and 148 KB of shared memory a CTA (one query), and 44 and 150 KB (eight rows a CTA)
@pytest.mark.parametrize("Q,short,long", [(1, 9000, 32000), (700, 1180, 4000)])
def test_rows_of_two_lengths_at_once(fa, Q, short, long):  # noqa: F811
    work = []
    for i, n in enumerate((short, long)):
        off = torch.tensor([4 * n - Q], dtype=torch.int32, device="cuda")
        src = fa.create_block_mask(fa.make_mask_rule([("causal",)], q_offset=off), 1, 2, Q, 4 * n, 1, 4, keep=[off])
        q, box = torch.randn(1, 2, Q, 64, generator=gen(i), device="cuda").to(BF), boxes((1, 1, n, 2, 64), i)
        want = fa.select_blocks(src, q, box, 40).tables()["block_class"].clone()
        ws = torch.empty(max(256, fa.select_blocks_workspace_bytes(src, 1, 2, 1, 64)), dtype=torch.uint8, device="cuda")
        out = fa.select_blocks(src, q, box, 40)
        # the C call with its arguments at hand: the interpreter's own work between two calls keeps those of two threads apart
        call = (ctypes.byref(src.c), q.data_ptr(), box.data_ptr(), None, 0, 0, 1, 2, 1, 64, 40, 1, 1, out.buf.data_ptr(), out.buf.numel(), ctypes.byref(out.c),
                ws.data_ptr(), ws.numel(), None)
        work.append((call, out, want, (src, q, box, ws)))
    torch.cuda.synchronize()
    codes, start, select = [], threading.Barrier(2), fa.load().fa_block_mask_select_blocks

    def run(call, stream):
        start.wait()
        codes.append({select(*call, stream) for _ in range(4000 if Q == 1 else 600)})

    streams = [torch.cuda.Stream() for _ in work]
    threads = [threading.Thread(target=run, args=(w[0], s.cuda_stream)) for w, s in zip(work, streams)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert codes == [{fa.OK}, {fa.OK}]
    for _, out, want, _ in work:
        assert torch.equal(out.tables()["block_class"], want)
