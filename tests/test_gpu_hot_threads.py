"""Two problems of very different widths driven by two host threads at once, whose hot rows take
different amounts of shared memory in the same kernels: each must match the oracle as alone."""
import threading

import numpy as np
import pytest
import torch

from tests import gpu_harness as H
from tests.test_gpu_forward_hot import _custom
from tests.test_gpu_streams import _expected

pytestmark = pytest.mark.gpu
tbe = H.tbe


def problem(D, seed):
    # half of every bag hits eight rows, so that the table has hot rows
    rng = np.random.default_rng(seed)
    E, B = [600, 900], 300
    bags = [[list(np.concatenate([rng.integers(0, 8, 50), rng.integers(0, e, 50)]))
             for _ in range(B)] for e in E]
    return _custom(E, [D, D], bags, seed=seed)


def step(r):
    r.reset_state()
    tbe.tbe_preprocess(r.desc, r.indices, r.offsets, r.psw, r.ws)
    tbe.tbe_forward(r.desc, r.weights, r.indices, r.offsets, r.psw, r.out, r.ws,
                    tbe.TBE_F_PREPROCESSED)
    tbe.tbe_backward_rowwise_adagrad(r.desc, r.grad_out, r.indices, r.offsets, r.psw, r.weights,
                                     r.momentum, r.w.lr, r.w.eps, r.ws, tbe.TBE_F_PREPROCESSED)


@pytest.mark.parametrize("widths", [(32, 256), (128, 136)])
def test_two_widths_in_two_threads(widths):
    made = [problem(d, i) for i, d in enumerate(widths)]
    runs, expected = [H.Run(w) for w in made], [_expected(w) for w in made]
    for r in runs:
        r.backward()
        assert sum(len(h) for h in r.hot_set()) > 0
    errors, start = [], threading.Barrier(len(runs))

    def drive(r):
        stream = torch.cuda.Stream()
        start.wait()
        try:
            with torch.cuda.stream(stream):
                for _ in range(100):
                    step(r)
            stream.synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    torch.cuda.synchronize()
    threads = [threading.Thread(target=drive, args=(r,)) for r in runs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for r, (ref, terms, W, m) in zip(runs, expected):
        assert r.status() == 0
        H.assert_forward_close(r.out.cpu().numpy(), ref, terms)
        H.assert_momentum_close(r.momentum.cpu().numpy(), m)
        H.assert_weights_within_ulp(r.weights.cpu().numpy(), W)
