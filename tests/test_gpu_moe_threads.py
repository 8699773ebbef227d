"""Sorts of different expert counts from several host threads, each on its own stream with its own
outputs: every call is valid by itself, so none may fail or change another's result."""
import threading

import pytest
import torch

import block_scaled_fp4_04_b200 as fp4
from moe_testutil import router_ids, sort_reference

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
def test_sorts_of_different_expert_counts_from_several_threads(dtype):
    # shared memory beyond 48 KB in every call, of another size in each thread; one cluster of blocks
    # and (the last) two launches
    jobs = [(32768, 1, 1024), (32768, 1, 512), (16384, 2, 400), (40000, 1, 700)]
    start, errors, results = threading.Barrier(len(jobs)), [], [None] * len(jobs)
    wants = [sort_reference(router_ids(t, k, e, e, 0.1), e) for t, k, e in jobs]

    def work(i):
        t, k, e = jobs[i]
        try:
            torch.cuda.set_device(0)
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                ids = router_ids(t, k, e, e, 0.1, dtype).cuda()
                out = [torch.full(s, -77, dtype=torch.int32, device="cuda") for s in ((e + 1,), (t, k), (t, k))]
                n = fp4.fp4_moe_sort_workspace_size(t, k, e)
                ws = torch.empty(max(1, n), dtype=torch.uint8, device="cuda")
            stream.synchronize()
            args = [ids.data_ptr(), ids.element_size(), t, k, e, *(o.data_ptr() for o in out), ws.data_ptr(), n,
                    stream.cuda_stream]
            start.wait()
            for _ in range(3000):
                fp4.fp4_moe_sort(*args)
            stream.synchronize()
            results[i] = [o.cpu() for o in out]
        except Exception as err:  # noqa: BLE001 (any failure of a thread is the test's)
            errors.append(f"{jobs[i]}: {err}")

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(jobs))]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not errors, errors
    for job, got, want in zip(jobs, results, wants):
        for g, w in zip(got, want):
            assert torch.equal(g, w), job
