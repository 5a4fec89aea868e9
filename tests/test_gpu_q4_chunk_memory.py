"""What the steps of several rows and behind a prefix keep of the GPU's memory: one
workspace for a device's stream, whatever the number of caches (a model has one for
each of its layers)."""
import numpy as np
import pytest
import torch

import positional_lsh_approximation_gb300 as plsh

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    plsh.build()
    plsh.load()


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def layers(n, pages=300, cap=256):
    order = torch.randperm(pages, device="cuda").to(torch.int32)
    for _ in range(n):
        data = torch.zeros(plsh.q4_cache_bytes(pages, 2, 64, 128), dtype=torch.uint8, device="cuda")
        yield plsh.Q4Cache(data, order[:cap][None].expand(64, -1).contiguous(), 2, 128, 64)


def test_layers_share_a_workspace():
    q = torch.randn(64, 8, 16, 128, device="cuda").bfloat16()
    q1 = q[:, :, :1].contiguous()
    sigma, pos = np.full(8, 100.0), i32(np.arange(64) * 50)
    caches = list(layers(12))
    prefix = caches[0].table[0, :250].contiguous()
    largest = max(plsh.q4_chunk_work_bytes(q, caches[0]), plsh.q4_prefix_work_bytes(q1, caches[0]))
    assert largest > 2 ** 25                             # the tensor cores'
    out, out1 = torch.empty_like(q), torch.empty_like(q1)
    side = torch.cuda.Stream()
    for stream in (torch.cuda.current_stream(), side):
        torch.cuda.synchronize()
        before = torch.cuda.memory_allocated()
        with torch.cuda.stream(stream):
            for c in caches:
                plsh.alibi_exact_chunk_q4(q, c, sigma, pos, out=out)
                plsh.alibi_exact_prefix_decode_q4(q1, c, sigma, pos, prefix, out=out1)
        torch.cuda.synchronize()
        assert torch.cuda.memory_allocated() - before <= largest + 2 ** 21
    plsh.stream_status()


def test_a_small_call_then_a_large_one_on_two_streams():
    """A workspace that grows between calls in flight, on two streams in turn."""
    a, b = layers(2)
    for c in (a, b):
        k, v = torch.randn(2, 64, 2, 32, 128, device="cuda")
        for at in range(0, 3200, 640):
            plsh.q4_cache_write(c, k, v, i32([at] * 64))
    sigma, pos = np.full(8, 100.0), i32(np.arange(64) * 50)
    qs = [torch.randn(64, 8, m, 128, device="cuda").bfloat16() for m in (1, 3, 16, 40)]
    want = [[plsh.alibi_exact_chunk_q4(q, c, sigma, pos, work=torch.empty(plsh.q4_chunk_work_bytes(q, c), dtype=torch.uint8,
                                                                         device="cuda")) for c in (a, b)] for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for q in qs:
        row = []
        for c, st in zip((a, b), streams):
            with torch.cuda.stream(st):
                row.append(plsh.alibi_exact_chunk_q4(q, c, sigma, pos))
        got.append(row)
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert torch.equal(g[0], w[0]) and torch.equal(g[1], w[1])
    plsh.stream_status()


def test_threads_that_share_a_stream_share_its_workspace():
    """Two caches' calls of different sizes from two threads, on one stream: the calls'
    launches stay together, whoever's workspace was there first."""
    import threading
    caches = list(layers(2))
    for c in caches:
        k, v = torch.randn(2, 64, 2, 32, 128, device="cuda")
        for at in range(0, 3200, 320):
            plsh.q4_cache_write(c, k, v, i32([at] * 64))
    sigma, pos = np.full(8, 100.0), i32(np.arange(64) * 50)
    qs = [torch.randn(64, 8, m, 128, device="cuda").bfloat16() for m in (16, 2)]
    want = [plsh.alibi_exact_chunk_q4(q, c, sigma, pos) for q, c in zip(qs, caches)]
    torch.cuda.synchronize()
    side, got, failed = torch.cuda.Stream(), [[], []], []

    def run(i):
        try:
            with torch.cuda.stream(side):
                for _ in range(60):
                    got[i].append(plsh.alibi_exact_chunk_q4(qs[i], caches[i], sigma, pos))
        except Exception as e:                       # noqa: BLE001 (told to the test's own thread)
            failed.append(e)
    threads = [threading.Thread(target=run, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed
    for i in range(2):
        assert len(got[i]) == 60 and all(torch.equal(g, want[i]) for g in got[i])
    plsh.stream_status()
