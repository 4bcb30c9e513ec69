"""Products from several host threads at once, each on a stream and with operands of
its own: the same results as one after the other (calls hold no state)."""
import threading

import pytest
import torch

import block_scaled_precision_bf16_amd as mx

pytestmark = pytest.mark.gpu


def test_threads():
    gen = torch.Generator(device="cuda").manual_seed(1)

    def job(i):
        """A tiled product with copied rows, a small one, and a matrix-vector product."""
        def codes(r, c):
            return torch.randint(0, 127, (r, c), dtype=torch.uint8, device="cuda", generator=gen)

        def scales(n):
            return torch.randint(117, 127, (n,), dtype=torch.uint8, device="cuda", generator=gen)

        K = 2065 + i
        big = codes(1500, K), scales(1500 * -(-K // 32)), codes(1300, K), scales(1300 * -(-K // 32))
        x = torch.randn(3 + i, 1024, device="cuda", generator=gen).to(torch.bfloat16)
        w = codes(512, 512), torch.full((512, 64), 0x38, dtype=torch.uint8, device="cuda"), torch.ones(1, device="cuda")
        small = codes(40, 256), scales(40 * 8), codes(96, 256), scales(96 * 8)

        def run(stream=None):
            return (mx.mx_matmul(*big, stream=stream), mx.mx_matmul(*big, flags=mx.OUT_F32, stream=stream),
                    mx.mx_matmul(*small, stream=stream), mx.nvfp4_matvec(x, *w, stream=stream))
        return run

    jobs = [job(i) for i in range(4)]
    want = [[y.clone() for y in run()] for run in jobs]
    torch.cuda.synchronize()
    wrong, start = [], threading.Barrier(len(jobs))

    def work(i):
        try:
            stream = torch.cuda.Stream()
            start.wait(timeout=60)
            got = [jobs[i](stream) for _ in range(8)]
            stream.synchronize()
            wrong.extend(i for ys in got for y, w in zip(ys, want[i]) if not torch.equal(y, w))
        except Exception as e:                     # reported by the test's own thread
            wrong.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(jobs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
