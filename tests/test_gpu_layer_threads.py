"""GPU test of layer operators that host threads use at the same time, each its own."""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda"


def test_host_threads_with_handles_of_their_own():
    """Threads with a handle and a stream each; the handles share a kernel and need different
    amounts of its shared memory. Calls follow each other as fast as a thread can make them."""
    from combine_route_layout_gb300.build import build
    build()
    from combine_route_layout_gb300 import ep, layer
    T, k, failed, start = 8, 4, [], threading.Barrier(4, timeout=60)

    def work(E):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                op = layer.EpRouterOp(layer.EpRouterConfig(1, T, E, k, score_func="sigmoid"))
                l = torch.randn((1, T, E), device=DEV)
                want = op.forward(l, balance=True)
                got = [torch.empty_like(t) for t in want]
                stream.synchronize()
                w, i, c, ls = (t.data_ptr() for t in got)
                args = (op._handle, l.data_ptr(), None, None, i, w, c, ls, stream.cuda_stream)
                start.wait()
                for n in range(20000):
                    ep.ep_router_forward(*args)
                    if n % 500 == 0:
                        stream.synchronize()
                stream.synchronize()
                assert all(torch.equal(a, b) for a, b in zip(got, want))
                op.sync()
        except Exception as e:               # noqa: BLE001 - told by the main thread
            failed.append(e)

    threads = [threading.Thread(target=work, args=(E,)) for E in (264, 300, 400, 512)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
