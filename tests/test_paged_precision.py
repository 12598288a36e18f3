"""How exact the weights of single tokens are: bf16 caches, one new token per request, weights in two bf16
parts. Keys come in pairs that nearly agree with values of opposite sign, so that a row's output is far
smaller than the sum of its terms and its own rounding hides nothing."""
import math

import pytest
import torch

from paged_common import Batch, cobs


def _pairs(K, V, g):
    """K [.., L, d] and V of an even number of keys: the second of each pair is the first with a little noise,
    and its value the first's negative."""
    L = K.shape[-2] // 2 * 2
    K, V = K[..., :L, :].float(), V[..., :L, :].clone()
    K[..., 1::2, :] = K[..., ::2, :] + 0.02 * torch.randn(K[..., ::2, :].shape, generator=g)
    V[..., 1::2, :] = -V[..., ::2, :]
    return K.to(torch.bfloat16), V


def _tolerance(q, K, V):
    """(o, tolerance) of one row in 64 bits. Scores are float32 sums of d exact products, scaled and raised: p is
    off by ep = (d + 4) 2^-24 max sum |q k| / sqrt(d) + 2^-21. A p in two parts, cut to 8 bits and the rest (below 2^-7 p)
    rounded to 8 bits: 2^-15. Sums over L keys: L 2^-24 in the numerator and the denominator. With A = sum p |v| / sum p the
    quotient is off by A (2^-15 + 2 ep + 2 L 2^-24); it is rounded to bf16 (2^-8 |o|)."""
    q, K, V = q.double(), K.double(), V.double()
    d, L = q.shape[-1], K.shape[0]
    w = torch.softmax(K @ q / math.sqrt(d), dim=0)
    o, A = w @ V, w @ V.abs()
    ep = (d + 4) * 2.0 ** -24 * (K.abs() @ q.abs()).max().item() / math.sqrt(d) + 2.0 ** -21
    return o, 2.0 ** -8 * o.abs() + A * (2.0 ** -15 + 2 * ep + 2 * L * 2.0 ** -24) * (1 + 2.0 ** -8)


def _emulate(q, K, V, parts):
    """The row with p in one bf16 part (rounded) or two (cut, rounded), sums in 64 bits, o rounded to bf16."""
    s = K.double() @ q.double() / math.sqrt(q.shape[-1])
    p = torch.exp(s - s.max()).float()
    if parts == 1:
        used = p.to(torch.bfloat16).double()
    else:
        high = (p.view(torch.int32) & -65536).view(torch.float32)
        used = high.double() + (p - high).to(torch.bfloat16).double()
    return ((used @ V.double()) / p.double().sum()).to(torch.bfloat16).double()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("L", [2, 16, 300])
def test_the_tolerance_tells_one_part_from_two(d, L):
    g = torch.Generator().manual_seed(d + L)
    off = 0
    for _ in range(8):
        q = torch.randn(d, generator=g).to(torch.bfloat16)
        K, V = _pairs(torch.randn((L, d), generator=g).to(torch.bfloat16), torch.randn((L, d), generator=g).to(torch.bfloat16), g)
        o, tol = _tolerance(q, K, V)
        assert ((_emulate(q, K, V, 2) - o).abs() <= tol).all()
        off += ((_emulate(q, K, V, 1) - o).abs() > tol).sum().item()
    assert off > d   # of 8 d outputs


@pytest.mark.gpu
@pytest.mark.parametrize("G,d,page", [(1, 64, 16), (4, 128, 64), (9, 128, 32), (16, 64, 128)])
def test_single_tokens_keep_their_weights(G, d, page):
    C = cobs()
    g = torch.Generator().manual_seed(G)
    lens = [(1, 1), (15, 1), (299, 1), (4095, 1)]
    b = Batch(C, lens, 2 * G, 2, d, page, seed=G)
    for r in range(len(lens)):
        b.K[r], b.V[r] = _pairs(b.K[r], b.V[r], g)
        for j, at in enumerate(b.table[r].tolist()):
            n = min(page, b.K[r].shape[1] - j * page)
            if n > 0:
                b.k_cache[at, :, :n] = b.K[r][:, j * page:j * page + n].to(b.k_cache.device)
                b.v_cache[at, :, :n] = b.V[r][:, j * page:j * page + n].to(b.v_cache.device)
    C.device_error(reset=True)
    b.run()
    assert C.device_error() == 0
    for r in range(len(lens)):
        for a in range(2 * G):
            o, tol = _tolerance(b.Q[r, a].cpu(), b.K[r][a // G], b.V[r][a // G])
            bad = (b.O[r, a].double().cpu() - o).abs() > tol
            assert not bad.any(), (r, a, int(bad.sum()))
