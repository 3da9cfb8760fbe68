"""Single tokens over more cache than a launch has workgroups for its tiles of 64 keys and query heads.

Tolerances as in test_gpu_attention."""
import math

import pytest
import torch

from vocabulary_label_bce_amd import ops

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt,u", [(torch.bfloat16, 2.0 ** -8), (torch.float32, 2.0 ** -24)])
def test_single_tokens_over_large_caches(dt, u):
    """256 caches of 65,536 rows, 32 heads over 2; they share one array (sequence stride 0), each filled so far."""
    B, S, hq, hk, dh = 256, 65_536, 32, 2, 64
    gen = torch.Generator(device="cuda").manual_seed(3)
    q = torch.randn(B, hq, dh, generator=gen, device="cuda").to(dt)
    kv = torch.randn(2, 1, S, hk, dh, generator=gen, device="cuda").to(dt)
    lens = torch.tensor([S - 251 * b if b % 3 else b // 3 for b in range(B)], dtype=torch.int32).cuda()
    out = ops.cached_attention(q, kv[0].expand(B, S, hk, dh), kv[1].expand(B, S, hk, dh), lens)
    scale, G = 1 / math.sqrt(dh), hq // hk
    unseen = torch.arange(S, device="cuda")[None] >= lens[:, None]
    for h in range(hq):
        K, V, Q = kv[0, 0, :, h // G].double(), kv[1, 0, :, h // G].double(), q[:, h].double()
        z = (Q @ K.T * scale).masked_fill(unseen, -math.inf)
        P = torch.nan_to_num(torch.softmax(z, 1))
        e = (dh + 16) * 2.0 ** -24 * float((Q.abs() @ K.abs().T).max()) * scale + (S + 17) * 2.0 ** -24
        want = P @ V
        bound = 2 * ((u + e) * (P @ V.abs()) + u * want.abs()) + 1e-30
        assert bool(((out[:, h].double() - want).abs() <= bound).all())
    assert not out[0].any()
