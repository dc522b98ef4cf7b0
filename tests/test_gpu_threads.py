"""Two host threads, each with a context of its own on one device: the calls
of one must not disturb the launches of the other (a kernel's shared-memory
limit belongs to the function, not to a context or a call)."""
from __future__ import annotations

import threading

import pytest

from activation_sparse_decode_sigmoid_gb300 import pi
from activation_sparse_decode_sigmoid_gb300 import workload as W
from tests import _gpu as G

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["f16", "q4"])
@pytest.mark.parametrize("B", [1, 4, 16])
def test_sparse_layers_of_two_sizes(kind, B):
    t = G.torch()
    lib = pi.load_library()
    wdt = W.Q4_0 if kind == "q4" else W.F16
    cfgs = [W.LayerConfig(f"threads_{kind}_{d}", d, 512, r, 1, W.RELU, wdt, W.F16, alpha=0.8, cfg_id=230 + i)
            for i, (d, r) in enumerate(((128, 16), (8192, 512)))]
    ctxs = [G.ctx(max_layers=1, max_batch=B) for _ in cfgs]
    failed = []
    try:
        bufs = []
        for c, cfg in zip(ctxs, cfgs):
            c.load_layer(0, W.make_layer(cfg, 0, 0))
            x = t.from_numpy(W.decode_inputs(cfg, B, 3).copy()).cuda()
            u, alone = t.empty_like(x), t.empty_like(x)
            c._s()
            assert lib.pi_layer_partial(c.handle, 0, x.data_ptr(), B, alone.data_ptr()) == pi.PI_OK
            c.check()
            bufs.append((x, u, alone))

        def work(c, x, u):
            failed.extend(c.handle for _ in range(3000) if lib.pi_layer_partial(c.handle, 0, x.data_ptr(), B, u.data_ptr()))

        threads = [threading.Thread(target=work, args=(c, x, u)) for c, (x, u, _) in zip(ctxs, bufs)]
        for th in threads:
            th.start()
        for th in threads:
            th.join()
        for c in ctxs:
            c.check()
        assert not failed, (len(failed), [pi.pi_last_error(c.handle) for c in ctxs])
        assert all(u.equal(alone) for _, u, alone in bufs)
    finally:
        for c in ctxs:
            c.close()
