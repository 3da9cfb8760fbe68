"""The training operators together, as the example's softmax step has them: embedding, layer norm and attention, the softmax
cross entropy, the encoder's backward, the gradients' norm and the clipped AdamW step."""
import os
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

import sequence_encoder as S  # noqa: E402

from vocabulary_label_bce_amd import ops  # noqa: E402

pytestmark = pytest.mark.gpu


def _model(dtype, items=700, dim=64, seed=3):
    model = S.Encoder(items, dim=dim, heads=2, kv_heads=1, dtype=dtype, seed=seed)
    (ids, places, cu, _, nxt), lens = S.histories(9, items, 1, 60, seed=seed)
    nxt[::7] = -1  # some rows have no next item
    return model, (ids, places, cu, nxt)


def _plain_adamw(p, g, m, v, t, lr, decay):
    m += 0.1 * (g - m)
    v += 0.001 * (g * g - v)
    p *= 1 - lr * decay
    p -= lr * (m / (1 - 0.9 ** t)) / ((v / (1 - 0.999 ** t)).sqrt() + 1e-8)


@pytest.mark.parametrize("max_norm", [1e-3, 1e3])
def test_steps_against_autograd_and_plain_adamw(max_norm):
    """Three steps in float32: every step's gradients are autograd's through the differentiable calls (the two accumulate
    the table's in different orders: 1e-4 of a tensor's norm), and its parameters a float64 AdamW's on the gradients that
    the step saw, which its first moments tell to 20 u of the larger of the two, u = 2^-24. A move is off by that twice
    over (m and sqrt(v)) and by a rounding of the parameter, u |p| / lr of it at |p| = 1 and lr = 1e-2 (6e-6): 1e-3 of
    its norm holds with room."""
    model, (ids, places, cu, nxt) = _model(torch.float32)
    opt = model.optimizer(lr=1e-2)
    plain = [p.detach().double() for p in opt.params]
    m, v = [torch.zeros_like(p) for p in plain], [torch.zeros_like(p) for p in plain]
    for step in range(1, 4):
        table = model.items.clone().requires_grad_()
        loss = ops.cut_cross_entropy(model.hidden(ops.embedding(ids, table, model.scale), places, cu), table, nxt)
        loss.backward()
        want = [table.grad] + [t.grad for t in model.p.values()]
        norm = torch.stack([g.double().norm() for g in want]).norm()
        for t in model.p.values():
            t.grad = None
        before = [p.detach().double() for p in opt.params]
        had = [x.double() for x in opt.exp_avgs]
        got_loss, got_norm = model.softmax_step(ids, places, cu, nxt, opt, max_norm=max_norm)
        assert abs(got_loss.item() - loss.item()) <= 1e-5 * loss.item()
        assert abs(got_norm.item() - norm.item()) <= 1e-4 * norm.item()
        clip = min(1.0, max_norm / (norm.item() + 1e-6))
        for i, g in enumerate(want):
            g = g.double() * clip
            mine = (opt.exp_avgs[i].double() - 0.9 * had[i]) / 0.1  # the gradient that the step saw
            assert float((mine - g).norm()) <= 1e-4 * float(g.norm()) + 1e-5 * float(had[i].norm())
            # AdamW on the gradients that the step saw: its arithmetic alone
            p = before[i].clone()
            _plain_adamw(p, mine, m[i], v[i], step, 1e-2, opt.weight_decay[i])
            m[i], v[i] = opt.exp_avgs[i].double(), opt.exp_avg_sqs[i].double()
            move = float((p - before[i]).norm())
            assert float((opt.params[i].detach().double() - p).norm()) <= 1e-3 * move
        assert opt.step_count.item() == step


@pytest.mark.parametrize("bits", [32, 8])
def test_bfloat16_runs_are_the_same_run(bits):
    """Two models from one seed go through the same bits: no order of additions changes from run to run."""
    runs = []
    for _ in range(2):
        model, batch = _model(torch.bfloat16)
        opt = model.optimizer(state_bits=bits, master=True)
        losses = [model.softmax_step(*batch, opt)[0] for _ in range(4)]
        runs.append(losses + [p.detach() for p in opt.params])
    assert all(torch.isfinite(x).all() for x in runs[0])
    assert all(torch.equal(a, b) for a, b in zip(*runs))


def test_a_captured_step_trains():
    """A captured step, replayed between eager work, gives what eager steps give: the steps are counted on the device, the
    learning rate is read there."""
    models = [_model(torch.bfloat16) for _ in range(2)]
    opts, rates = [], []
    for model, _ in models:
        rates.append(torch.full((1,), 1e-3, device="cuda"))
        opts.append(model.optimizer(lr=rates[-1], master=True))
    side = torch.cuda.Stream()
    for (model, batch), opt in zip(models, opts):
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            model.softmax_step(*batch, opt)
        torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = models[0][0].softmax_step(*models[0][1], opts[0])
    for k in range(4):
        for r in rates:
            r.fill_(1e-3 / (k + 1))
        graph.replay()
        torch.cuda.synchronize()
        want = models[1][0].softmax_step(*models[1][1], opts[1])
        torch.cuda.synchronize()
        for a, b in zip(out + tuple(opts[0].params), want + tuple(opts[1].params)):
            assert float((a.detach().double() - b.detach().double()).norm()) <= 1e-6 * float(b.detach().double().norm())
    assert opts[0].step_count.item() == 5


@pytest.mark.parametrize("options", [["--loss", "softmax"], ["--loss", "softmax", "--state-bits", "8"]])
def test_the_example_runs(options, monkeypatch, capsys):
    monkeypatch.setattr(sys, "argv", ["sequence_encoder.py", "--users", "8", "--items", "3000", "--steps", "3", *options])
    S.main()
    out = capsys.readouterr().out
    assert "step 2: loss" in out and "token 2" in out and "nan" not in out
