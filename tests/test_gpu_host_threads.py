"""Two host threads with a handle each: calls of one kernel with different sizes at the same time."""
import threading

import pytest
import torch

from quantized_weight_dequant_gb300 import qgemv

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from quantized_weight_dequant_gb300.build import build_library
    build_library()


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
def test_draws_from_rows_of_different_lengths(dtype):
    """A row is held in shared memory, of which each length takes its own amount: neither thread's call is refused."""
    errors = []

    def work(V, rows, calls):
        try:
            torch.cuda.set_device(0)
            stream = torch.cuda.Stream()
            g = torch.Generator(device="cuda").manual_seed(V)
            h = qgemv.create(0)
            with torch.cuda.stream(stream):
                x = torch.randn(rows, V, generator=g, device="cuda").to(dtype)
                u = torch.rand(rows, generator=g, device="cuda")
                first, tokens = (torch.empty(rows, dtype=torch.int32, device="cuda") for _ in range(2))
                qgemv.sample(h, qgemv.sample_desc(x, u, first))
                stream.synchronize()
                desc = qgemv.sample_desc(x, u, tokens)
                started.wait()
                for i in range(calls):
                    qgemv.sample(h, desc)
                    if i % 200 == 0:
                        stream.synchronize()
                stream.synchronize()
                assert torch.equal(first, tokens) and qgemv.check_error(h, stream) == qgemv.OK
            h.close()
        except Exception as e:  # noqa: BLE001
            errors.append((V, repr(e)))
            started.abort()

    started = threading.Barrier(2)
    held = 10000 if dtype == torch.bfloat16 else 12000
    threads = [threading.Thread(target=work, args=a) for a in ((300, 2, 6000), (held, 310, 3000))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
