"""The sort's shared memory: the most experts, and several host threads at once, a handle each."""
import threading

import pytest
import torch

import persistent_tile_scheduled_gb300 as pts

pytestmark = pytest.mark.gpu


def test_sorts_of_different_sizes_in_two_threads():
    """What a kernel may use of shared memory is set per function and device, not per handle: a thread that sorts for
    fewer experts must not lower it between another thread's setting and launch."""
    tokens, calls = 40000, 3000
    failures, start = [], threading.Barrier(2)

    def sorts(experts):
        h = pts.gemm_create(0)
        stream = torch.cuda.Stream()
        gen = torch.Generator().manual_seed(experts)
        ids = torch.randint(0, experts, (tokens, 1), generator=gen, dtype=torch.int32).cuda()
        offsets = torch.zeros(experts + 1, dtype=torch.int32, device="cuda")
        row_of, src_of = (torch.zeros(tokens, dtype=torch.int32, device="cuda") for _ in range(2))
        torch.cuda.synchronize()
        start.wait()
        try:
            for i in range(calls):
                pts.gemm_expert_sort(h, tokens, 1, experts, ids, offsets, row_of, src_of, stream=stream)
                if i % 500 == 499:
                    stream.synchronize()
        except Exception as e:   # noqa: BLE001 (reported by the test's own thread)
            failures.append(f"{experts} experts, call {i}: {e}")
        torch.cuda.synchronize()
        if not failures:
            order = torch.sort(ids.flatten(), stable=True).indices
            if not torch.equal(src_of.long(), order) or not torch.equal(row_of[order].long(), torch.arange(tokens, device="cuda")):
                failures.append(f"{experts} experts: wrong order")
        pts.gemm_destroy(h)

    threads = [threading.Thread(target=sorts, args=(e,)) for e in (1024, 512)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failures, failures


@pytest.mark.parametrize("tokens", [700, 1000, 1024, 1025, 2048, 2049, 33000])
def test_the_most_experts_with_few_and_with_many_assignments(tokens):
    """1024 experts: counts per warp that need more shared memory than a kernel has by default, in both sort kernels."""
    h = pts.gemm_create(0)
    ids = torch.randint(0, 1024, (tokens, 1), generator=torch.Generator().manual_seed(tokens), dtype=torch.int32).cuda()
    offsets = torch.zeros(1025, dtype=torch.int32, device="cuda")
    row_of, src_of = (torch.zeros(tokens, dtype=torch.int32, device="cuda") for _ in range(2))
    pts.gemm_expert_sort(h, tokens, 1, 1024, ids, offsets, row_of, src_of)
    st, dev = pts.gemm_check(h)
    pts.gemm_destroy(h)
    order = torch.sort(ids.flatten(), stable=True).indices
    assert st == 0 and torch.equal(src_of.long(), order)
    assert torch.equal(row_of[order].long(), torch.arange(tokens, device="cuda"))
    assert torch.equal(offsets[1:].long(), torch.bincount(ids.flatten(), minlength=1024).cumsum(0))
