"""A kernel that allocates tensor memory frees it before it waits for other thread blocks of its cluster. Read from the sources, as a wait that
never ends can be shown in no other way."""
import glob
import os
import re

from block_sparse_masked_create_gb300 import build as fa_build

WAITS = re.compile(r"cl\.sync\(\)|this_cluster\(\)\.(sync|barrier_wait)\(\)|barrier\.cluster\.(sync|wait)")


def kernels():
    for path in sorted(glob.glob(os.path.join(fa_build.CSRC, "*.cu"))):
        with open(path) as f:
            text = re.sub(r"//[^\n]*", "", f.read())
        for body in text.split("__global__")[1:]:
            if "tmem_alloc(" in body:
                yield os.path.basename(path), body


def test_no_wait_for_other_thread_blocks_while_tensor_memory_is_held():
    seen = 0
    for name, body in kernels():
        held = body[body.index("tmem_alloc("):body.index("tmem_dealloc(")]
        assert not WAITS.search(held), name
        seen += bool(WAITS.search(body))
    assert seen  # the backward over chosen blocks is one that waits
