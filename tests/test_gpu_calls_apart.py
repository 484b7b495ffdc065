"""The stateless calls around the step do not wait behind a call that waits for
the device."""
import threading
import time

import pytest

torch = pytest.importorskip("torch")
import matrix_orthogonalizing_optimizer_momentum_amd as mm  # noqa: E402

pytestmark = pytest.mark.gpu


def test_calls_beside_a_synchronizing_one():
    print("[case] calls beside muonh_get_flags", flush=True)
    g = torch.Generator(device="cpu")
    g.manual_seed(1)
    table = torch.randn(300, 128, generator=g).cuda()
    ids = torch.randint(0, 300, (70,), generator=g).cuda()
    x = torch.randn(70, 128, generator=g).bfloat16().cuda()
    w = table.bfloat16()
    mine, busy = torch.cuda.Stream(), torch.cuda.Stream()

    def calls():
        return [*mm.grad_norm([table, x], max_norm=1.0), *mm.clip_grads([x], 1.0, outputs=[torch.empty_like(x)]),
                mm.embedding(table, ids), mm.embedding_grad(ids, x, 300), *mm.cross_entropy(x, w, ids),
                *mm.cross_entropy(x[:30], w, ids[:30], grad=False)[:2]]

    # the library's first calls, and memory for everything below, out of the way
    mm.ns_orthogonalize([x], K=1)
    torch.cuda.synchronize()
    with torch.cuda.stream(mine):
        want = calls()
        calls()
    torch.cuda.synchronize()
    a = torch.randn(8192, 8192, device="cuda")
    b = torch.empty_like(a)
    for _ in range(3):
        torch.mm(a, a, out=b)
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    for _ in range(5):
        torch.mm(a, a, out=b)
    torch.cuda.synchronize()
    per = (time.perf_counter() - t0) / 5
    entered = threading.Event()
    with torch.cuda.stream(busy):
        for _ in range(max(5, int(1.5 / max(per, 1e-4)))):  # about a second and a half
            torch.mm(a, a, out=b)
        done = torch.cuda.Event()
        done.record()

    def waits():
        entered.set()
        mm.get_flags()  # waits for the device

    other = threading.Thread(target=waits)
    other.start()
    entered.wait()
    time.sleep(0.2)
    waiting = other.is_alive()
    with torch.cuda.stream(mine):
        got = calls()
    running = not done.query()
    other.join()
    torch.cuda.synchronize()
    assert waiting, "get_flags returned at once: nothing was shown"
    assert running, "the calls returned after the device was done"
    for p, q in zip(got, want):
        assert torch.equal(p, q)
