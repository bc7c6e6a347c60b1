"""Packed calls of several host threads at once, each on a stream of its own."""
import sys
import threading

import pytest
import torch

from gated_delta_rule_117_b200 import kda

pytestmark = pytest.mark.gpu


def test_block_maps_of_four_threads():
    # every request count needs more shared memory than a kernel has without asking, no two the same
    page, calls, codes, sizes = 4, 5000, {}, (16384, 4200, 9000, 6000)
    fn = kda.load_library().kda_block_map

    def run(R):
        st = torch.cuda.Stream()
        with torch.cuda.stream(st):
            lens = torch.ones(R, dtype=torch.int32, device="cuda")
            free, table = torch.arange(R, dtype=torch.int32, device="cuda"), torch.full((R, 1), -1, dtype=torch.int32, device="cuda")
            cu, slots, used = kda.block_map(lens, None, free, table, page, R)
            args = (lens.data_ptr(), None, free.data_ptr(), R, table.data_ptr(), 1, page, cu.data_ptr(), slots.data_ptr(),
                    used.data_ptr(), R, R, st.cuda_stream)
            codes[R] = [fn(*args) for _ in range(calls)]
            st.synchronize()
            assert torch.equal(table[:, 0], free) and int(used) == R

    interval = sys.getswitchinterval()
    sys.setswitchinterval(1e-5)
    try:
        threads = [threading.Thread(target=run, args=(R,)) for R in sizes]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
    finally:
        sys.setswitchinterval(interval)
    assert {R: sorted(set(codes[R])) for R in sizes} == {R: [0] for R in sizes}
    assert kda.kda_get_device_status() == 0
