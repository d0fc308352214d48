"""The 4-bit products and sampling as a decode step uses them: the norm, the FFN on ternary weights while the copy
is resident and on 4-bit weights while it is not, the head and the draw; eagerly, from a graph, and from threads."""
import threading

import numpy as np
import pytest

from test_q4_gpu import Matrix
from test_sample_gpu import rule

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tq():
    from ternary_weight_dp4a_gb300 import build
    from ternary_weight_dp4a_gb300 import tq as m
    build.build()
    return m


HIDDEN, INTER, VOCAB = 512, 1024, 4001


class Model:
    """One layer and a head.  The ternary copy of the FFN is under the lifecycle policy."""

    def __init__(self, tq):
        import torch
        from _util import ffn_mats
        self.tq = tq
        self.q4 = [Matrix(tq, INTER, HIDDEN, 64, True, 1), Matrix(tq, INTER, HIDDEN, 64, True, 2), Matrix(tq, HIDDEN, INTER, 64, True, 3)]
        self.head = Matrix(tq, VOCAB, HIDDEN, 32, False, 4)
        self.ternary = [m.dev for m in ffn_mats(HIDDEN, INTER, tq.FMT_TERNARY2)]
        self.room = [1 << 40]
        hooks = type("Hooks", (), {"alloc": lambda s, n, p: 0 if n > self.room[0] else 0x1000, "release": lambda s, a, n, p: None,
                                   "free_bytes": lambda s: self.room[0], "build": lambda s, a, n: True})()
        self.copy = tq.CopyLifecycle(sum(m.nbytes for m in self.ternary), 0, hooks)
        self.gamma = torch.ones(HIDDEN, dtype=torch.bfloat16, device="cuda")

    def ffn(self, x):
        tq = self.tq
        if self.copy.copy is not None:
            return tq.ffn_step(*self.ternary, x)
        gate, up, down = (m.dev for m in self.q4)
        return tq.q4_gemv(down, tq.q4_gateup(gate, up, x))

    def step(self, residual, uniform, **settings):
        """residual float32 [m][HIDDEN] -> (normed x, FFN output, logits, ids, probs)."""
        import torch
        tq, m = self.tq, len(residual)
        x = torch.empty((m, HIDDEN), dtype=torch.bfloat16, device="cuda")
        residual, _, _ = tq.add_rmsnorm_rotq(residual, gamma=self.gamma, x_out=x)
        delta = self.ffn(x)
        last = torch.empty_like(x)
        tq.add_rmsnorm_rotq(residual, delta, self.gamma, x_out=last)
        logits = tq.q4_gemv(self.head.dev, last)
        ids, probs = tq.sample(logits, uniform, **settings)
        return x, delta, last, logits, ids, probs


def _settings(m):
    import torch
    return dict(temperature=torch.full((m,), 0.9, device="cuda"), top_k=torch.full((m,), 60, dtype=torch.int32, device="cuda"),
                top_p=torch.full((m,), 0.95, device="cuda"), min_p=torch.full((m,), 0.001, device="cuda"))


def _check_step(model, got, uniform):
    """Each stage against its definition, from what the stage before gave."""
    x, delta, last, logits, ids, probs = got
    want, tol = model.head.product(last)
    assert ((logits.double() - want).abs() <= tol).all()
    host = logits.double().cpu().numpy()
    for r in range(len(host)):
        i, p = rule(host[r], 3.5e38, float(uniform[r]), float(np.float32(0.9)), 60, float(np.float32(0.95)), float(np.float32(0.001)))
        assert ids[r].item() == i and abs(probs[r].item() - p) < 1e-6


@pytest.mark.parametrize("m", [1, 5, 24])
def test_a_step_with_and_without_the_ternary_copy(tq, m):
    import torch
    model = Model(tq)
    residual, uniform = torch.randn((m, HIDDEN), device="cuda"), torch.rand((m,), device="cuda")
    assert model.copy.load() == "resident"
    if m <= 8:
        ternary = model.step(residual, uniform, **_settings(m))
        _check_step(model, ternary, uniform)
        assert torch.equal(ternary[1], tq.ffn_step(*model.ternary, ternary[0]))
    model.room[0] = 10
    assert model.copy.alloc(100) is None and model.copy.state == "released"  # other work's memory: the copy goes
    got = model.step(residual, uniform, **_settings(m))
    _check_step(model, got, uniform)
    gate, up, down = model.q4
    g, tg = gate.product(got[0])
    u, tu = up.product(got[0])
    s = g * g.sigmoid()
    h = tq.q4_gateup(gate.dev, up.dev, got[0])
    tol = 1.1 * tg * (u.abs() + tu) + s.abs() * tu + 2.0 ** -20 * (s * u).abs()
    assert ((h.double() - s * u).abs() <= tol + 2.0 ** -8 * ((s * u).abs() + tol)).all()
    want, tol = down.product(h)
    assert ((got[1].double() - want).abs() <= tol).all()
    model.copy.destroy()


@pytest.mark.parametrize("m", [1, 8, 40])
def test_two_graphs_of_steps_replayed_by_turns(tq, m):
    """Their first calls are captured, and they share everything that the library keeps."""
    import torch
    model = Model(tq)
    inputs = [torch.randn((m, HIDDEN), device="cuda") for _ in range(4)]
    uniform = torch.rand((m,), device="cuda")
    settings = _settings(m)
    held = [inputs[0].clone(), inputs[0].clone()]
    graphs, outs = [], []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(model.step(held[i], uniform, **settings))
        graphs.append(g)
    want = [[t.clone() for t in model.step(x, uniform, **settings)] for x in inputs]
    for turn in range(4):
        for i in range(2):
            held[i].copy_(inputs[(turn + i) % 4])
            graphs[i].replay()
        torch.cuda.synchronize()
        for i in range(2):
            assert all(torch.equal(a, b) for a, b in zip(outs[i], want[(turn + i) % 4]))
    assert tq.q4_read_error_word() == 0


def test_a_padded_batch(tq):
    """Rows of padding, whatever they hold, leave the others as they are."""
    import torch
    model = Model(tq)
    residual, uniform = torch.randn((6, HIDDEN), device="cuda"), torch.rand((6,), device="cuda")
    alone = model.step(residual[:4].contiguous(), uniform[:4].contiguous(), **_settings(4))
    residual[4] = float("nan")
    residual[5] = float("inf")
    got = model.step(residual, uniform, **_settings(6))
    for a, b in zip(got, alone):
        assert torch.equal(a[:4], b)
    assert got[4][4].item() == -1 and got[5][4].item() == 0.0                # no logit of the row is a number


def test_threads_with_streams_of_their_own(tq):
    import torch
    model = Model(tq)
    sizes = [1, 3, 12, 20, 64, 200]
    jobs = []
    for i, m in enumerate(sizes):
        residual, uniform = torch.randn((m, HIDDEN), device="cuda"), torch.rand((m,), device="cuda")
        x = residual.bfloat16()
        logits = torch.randn((m, 20_000), device="cuda")
        want = (tq.q4_gateup(model.q4[0].dev, model.q4[1].dev, x), tq.q4_gemv(model.head.dev, x), *tq.sample(logits, uniform, **_settings(m)))
        jobs.append((m, x, logits, uniform, _settings(m), want, torch.cuda.Stream()))
    torch.cuda.synchronize()
    errors = []

    def work(job):
        try:
            m, x, logits, uniform, settings, want, stream = job
            with torch.cuda.stream(stream):
                for _ in range(30):
                    got = (tq.q4_gateup(model.q4[0].dev, model.q4[1].dev, x), tq.q4_gemv(model.head.dev, x),
                           *tq.sample(logits, uniform, **settings))
            stream.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want)), m
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(j,)) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
