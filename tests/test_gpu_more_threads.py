"""Two host threads with the 4-bit products, the balance loss and the gradient norm on streams of their
own at the same time: every result is that of a single thread."""
import threading

import pytest
import torch

import combine_ep_route_gb300 as ep

pytestmark = pytest.mark.gpu
BF16, I32 = torch.bfloat16, torch.int32
ITERATIONS = 25


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()


def job(i):
    g = torch.Generator(device="cuda").manual_seed(51 + i)
    E, rows, k, n, act = ((90, 60, 256, 136, "swiglu"), (3, 12, 4096, 264, "none"))[i]
    x = torch.randn(E, rows, k, generator=g, device="cuda").to(BF16)
    wn = 2 * n if act == "swiglu" else n
    codes = torch.randint(0, 256, (E, wn, k // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = (torch.rand(E, k // 64, wn, generator=g, device="cuda") * k ** -0.5).to(BF16)
    counts = torch.randint(0, rows + 1, (E,), generator=g, device="cuda", dtype=I32)
    logits = torch.randn(4, 300, 128, generator=g, device="cuda")
    ids = logits.topk(4, dim=-1).indices.to(I32)
    d = torch.tensor([1.0, 0.1], device="cuda")
    grads = [torch.randn(m, generator=g, device="cuda") for m in (5, 70001, 300000)]

    def run():
        out = torch.zeros(E, rows, n, dtype=BF16, device="cuda")
        ep.experts_product_w4(x, codes, scales, counts, act=act, out=out)
        losses, load = ep.balance_loss(logits, ids, per_sequence=bool(i))
        to = [torch.empty_like(t) for t in grads]
        return (out, ep.linear_w4(x[0], codes[0], scales[0], act=act), losses, load,
                ep.balance_loss_backward(d, logits, load, 4, per_sequence=bool(i)), ep.clip_grad_norm(grads, 1.0, out=to), *to)
    return run


def test_every_call_of_two_threads_succeeds():
    jobs = [job(i) for i in range(2)]
    want = [run() for run in jobs]
    torch.cuda.synchronize()
    errors, finished = [], [0, 0]

    def worker(i):
        try:
            torch.cuda.set_device(0)
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(ITERATIONS):
                    got = jobs[i]()
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
    assert finished == [ITERATIONS] * 2
    ep.check_products()
