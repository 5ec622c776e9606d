"""tcgen05.alloc waits, without a limit, for free columns of its SM's tensor
memory.  A CTA launched programmatically that holds columns while it waits for
the previous kernel blocks a CTA of that kernel which has yet to allocate on
the same SM; so a kernel allocates after the wait, unless its shared memory
keeps every other kernel with tensor memory off its SM."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "rope_chain_gb300", "csrc")
ALONE = {"k2_gemm.cu", "k4_qkv_front.cu"}      # 145 KB a CTA and more: of 228, k5_wide<1> takes 116


def test_tensor_memory_is_allocated_after_the_wait():
    seen = 0
    for name in sorted(os.listdir(CSRC)):
        if not name.endswith(".cu") or name in ALONE:
            continue
        text = open(os.path.join(CSRC, name)).read()
        for alloc in re.finditer(r"tcgen05\.alloc", text):
            kernel = text.rindex("__global__", 0, alloc.start())
            assert "pdl_wait();" in text[kernel:alloc.start()], name
            seen += 1
    assert seen >= 1
