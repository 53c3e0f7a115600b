"""Two host threads calling the products on their own streams at the same time: every call
succeeds, every iteration runs to its end, no wait runs out and every result is that of a
single thread."""
import threading

import pytest
import torch

import combine_ep_route_gb300 as ep

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
ITERATIONS = 25


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()


def job(i):
    g = torch.Generator(device="cuda").manual_seed(41 + i)
    E, rows, k, n, act = ((24, 200, 264, 520, "swiglu"), (3, 40, 4104, 136, "none"))[i]
    x = torch.randn(E, rows, k, generator=g, device="cuda").to(BF16)
    w = (torch.randn(E, 2 * n if act == "swiglu" else n, k, generator=g, device="cuda") * k ** -0.5).to(BF16)
    dy = torch.randn(E, rows, n, generator=g, device="cuda").to(BF16)
    counts = torch.randint(0, rows + 1, (E,), generator=g, device="cuda", dtype=torch.int32)
    logits = torch.randn(rows, 64, generator=g, device="cuda")

    def run(status=None):
        out = torch.zeros(E, rows, n, dtype=BF16, device="cuda")
        ep.experts_product(x, w, counts, act=act, out=out, status=status)
        return (out, ep.experts_product_wgrad(dy, x, counts, out_dtype=F32, status=status),
                ep.linear(x[0], w[0], act=act, status=status), *ep.route_topk(logits, 8))
    return run


def test_every_call_of_two_threads_succeeds():
    jobs = [job(i) for i in range(2)]
    want = [run() for run in jobs]
    torch.cuda.synchronize()
    errors, finished, statuses = [], [0, 0], [torch.zeros(1, dtype=torch.int32, device="cuda") for _ in jobs]

    def worker(i):
        try:
            torch.cuda.set_device(0)
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(ITERATIONS):
                    got = jobs[i](statuses[i])
                    s.synchronize()
                    assert all(torch.equal(a, b) for a, b in zip(got, want[i], strict=True)), f"thread {i}"
                    finished[i] += 1
        except BaseException as e:   # reported by the main thread
            errors.append(e)

    threads = [threading.Thread(target=worker, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(timeout=60)
    assert not any(t.is_alive() for t in threads)
    assert not errors, errors
    assert finished == [ITERATIONS] * 2 and [s.item() for s in statuses] == [0, 0]
    ep.check_products()
