"""GPU AdamW: what changes between steps.  Bit for bit, as in test_gpu_adamw."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from block_scaled_fp4_06_amd import nvfp4 as N  # noqa: E402
from block_scaled_fp4_06_amd import optim  # noqa: E402
from test_gpu_adamw import F32, HYPER, host, say, step32, tensors  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    N.load()
    yield


def test_weight_decay_between_steps():
    say("adamw weight decay changed between steps")
    params = tensors([300, 5000], F32, 1)
    want = [(host(p), np.zeros(p.numel(), np.float32), np.zeros(p.numel(), np.float32)) for p in params]
    opt = optim.AdamW(params, weight_decay=0.1, **HYPER)
    for t, decay in ((1, [0.1, 0.1]), (2, [0.1, 0.0]), (3, [0.4, 0.2]), (4, [0.25, 0.25])):
        if t == 2:
            opt.weight_decay[1] = 0.0
        elif t > 2:
            opt.weight_decay = decay if t == 3 else 0.25
        grads = tensors([300, 5000], F32, 10 + t, 1e-3)
        opt.step(grads)
        for i, (p, g) in enumerate(zip(params, grads)):
            w, m, v = want[i]
            w, m, v, _ = step32(w, host(g), m, v, t, decay[i], **HYPER)
            want[i] = w, m, v
            assert np.array_equal(host(p), w), (t, i)


@pytest.mark.parametrize("given", [False, True])
def test_table_is_kept_for_the_stream_that_reads_it(given):
    """The table's memory is not handed out again while a step on another stream may read it."""
    say("adamw table on another stream, given=%s" % given)
    params, grads = tensors([300, 5000], F32, 1), tensors([300, 5000], F32, 2)
    opt = optim.AdamW(params, **HYPER)
    opt.step(grads)
    torch.cuda.synchronize()
    old, size = opt._table[4].data_ptr(), opt._table[4].numel()
    other = torch.cuda.Stream()
    with torch.cuda.stream(other):
        torch.cuda._sleep(200000000)
        if not given:
            opt.step(grads)
    if given:
        opt.step(grads, stream=other)
    assert opt._table[4].data_ptr() == old
    opt._table = None
    new = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(64)]
    busy = not other.query()
    assert busy and old not in [t.data_ptr() for t in new]
    other.synchronize()
    opt.step(grads)
    torch.cuda.synchronize()
    assert opt.state.step == 3
