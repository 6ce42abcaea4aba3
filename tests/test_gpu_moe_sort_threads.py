"""Sorts called from several host threads at once: each with its own number of
experts, and so its own amount of shared memory."""

import threading

import pytest
import torch

from quantized_linear_gemm_b200 import lq

pytestmark = pytest.mark.gpu


def test_threads_with_different_expert_counts(cuda_device):
    """No call takes shared memory away from another one between its set-up and its launch."""
    sizes = [(1024, torch.int64), (512, torch.int64), (320, torch.int64), (1000, torch.int64), (330, torch.int64)]
    rounds, failed = 20000, []
    start = threading.Barrier(len(sizes))

    def worker(E, dtype):
        try:
            torch.cuda.set_device(0)
            st = torch.cuda.Stream()
            with torch.cuda.stream(st):
                ids = torch.randint(0, E, (8, 8), device="cuda").to(dtype)
                want = torch.argsort(ids.reshape(-1), stable=True)
                st.synchronize()
                start.wait(timeout=60)
                order = torch.empty(64, dtype=torch.int32, device="cuda")
                off = torch.empty(E + 1, dtype=torch.int32, device="cuda")
                slots = torch.empty((8, 8), dtype=torch.int32, device="cuda")
                lq.moe_sort(ids, E, off, order, slots)
                call = lq.lib().lq_moe_sort           # the C call alone: it releases the interpreter's lock
                args = (ids.data_ptr(), 8, 64, E, off.data_ptr(), order.data_ptr(), slots.data_ptr(), st.cuda_stream)
                codes = {call(*args) for _ in range(rounds)}
                st.synchronize()
                if codes != {0}:
                    failed.append((E, codes))
                if not torch.equal(order.long(), want):
                    failed.append((E, "order"))
        except Exception as e:   # noqa: BLE001 - reported by the test's thread
            failed.append((E, repr(e)))

    threads = [threading.Thread(target=worker, args=s) for s in sizes]
    for t in threads:
        t.start()
    for t in threads:
        t.join(timeout=120)
    assert not failed, failed
