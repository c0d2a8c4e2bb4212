"""The square-root bounds see a lost block: the mistakes are made in the 64-bit
forms here, on the CPU."""
import pytest
import torch

import decode_reference as R
import decode_sums as S


@pytest.mark.parametrize("K", [768, 2048, 7168, 16384])
def test_a_lost_block_of_a_product_is_seen(K):
    gen = torch.Generator().manual_seed(K)
    x = torch.randn((4, K), generator=gen).bfloat16()
    w = torch.randn((160, K), generator=gen, dtype=torch.float64) * 0.02
    y, bound = S.product(x, w, torch.float32)
    lost = x.clone()
    lost[:, 320:352] = 0
    off = (lost.double() @ w.T - y).abs()
    assert (off > bound).double().mean() > 0.5
    late = x.float() @ w.float().T                       # a float32 product stays inside
    R.close(late, y, bound)


@pytest.mark.parametrize("n,lost", [(700, 1), (12000, 1), (131072, 4)])
def test_lost_steps_of_an_attention_are_seen(n, lost):
    """One step of 32 positions, or a CTA's four."""
    gen = torch.Generator().manual_seed(n)
    q = torch.randn((4, 64), generator=gen).half()
    k, v = (torch.randn((n, 64), generator=gen) for _ in range(2))
    o, bound = S.attention(q, k, v, 0.125, torch.float16)
    keep = torch.ones(n, dtype=torch.bool)
    keep[n // 2 // 32 * 32:][:32 * lost] = False
    o2, _ = S.attention(q, k[keep], v[keep], 0.125, torch.float16)
    assert ((o2 - o).abs() > bound).any(dim=-1).all()
