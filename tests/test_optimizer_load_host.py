"""AdamW.load_state_dict either loads a state whole or changes nothing."""
import pytest
import torch

from vocabulary_label_bce_amd import ops


def _optimizer(sizes=(300, 7), kind=torch.bfloat16, **how):
    opt = ops.AdamW([torch.ones(n, dtype=kind) for n in sizes], **how)
    for i, x in enumerate(_tensors(opt)):
        x.copy_(torch.full_like(x, 2 + i, dtype=torch.float32))
    return opt


def _tensors(opt):
    return [x for v in opt.state_dict().values() if v is not None
            for x in ([v] if isinstance(v, torch.Tensor) else [y for y in v if y is not None])]


def _other(opt):
    """opt's state with other values."""
    twice = lambda x: None if x is None else (x.float() * 2).to(x.dtype)
    return {n: v if v is None else twice(v) if isinstance(v, torch.Tensor) else [twice(x) for x in v]
            for n, v in opt.state_dict().items()}


@pytest.mark.parametrize("bits,master", [(32, False), (32, True), (8, False), (8, True)])
def test_a_refused_state_changes_nothing(bits, master):
    opt = _optimizer(state_bits=bits, master=master)
    names = [n for n, v in opt.state_dict().items() if isinstance(v, list)]
    bad = []
    for n in names:
        last = _other(opt)[n][-1]
        for x in (last[:-1], last.double(), None):
            state = _other(opt)
            state[n][-1] = x
            bad.append(state)
        bad += [dict(_other(opt), **{n: _other(opt)[n][:1]}), dict(_other(opt), **{n: None}),
                {k: v for k, v in _other(opt).items() if k != n}]
    before = [x.clone() for x in _tensors(opt)]
    for state in bad:
        with pytest.raises((ValueError, KeyError)):
            opt.load_state_dict(state)
        assert all(torch.equal(a.float(), b.float()) for a, b in zip(before, _tensors(opt)))


@pytest.mark.parametrize("bits,master", [(32, False), (8, True)])
def test_a_state_is_loaded_whole(bits, master):
    opt = _optimizer(state_bits=bits, master=master)
    state = _other(opt)
    opt.load_state_dict(state)
    for n, v in opt.state_dict().items():
        for a, b in zip([v] if isinstance(v, torch.Tensor) else v or [], [state[n]] if isinstance(v, torch.Tensor) else state[n] or []):
            assert torch.equal(a.float(), b.float())
