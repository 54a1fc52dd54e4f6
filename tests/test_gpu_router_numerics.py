"""What the router's numbers are made of, on the GPU: probabilities, and sums over many tokens."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from router_mx4_reference import router_reference

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def moe():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import combine_moe_layout_02_amd
    return combine_moe_layout_02_amd


@pytest.mark.parametrize("E", [7, 64, 128, 200, 256, 500, 1000])
def test_the_loss_has_the_weights_probabilities(moe, E):
    """One token routed to expert e alone: loss = E * p_e, which is exact in 64 bits and rounded once, so the
    probability in it has to be, bit for bit, the route weight of e."""
    z = (torch.randn((16, E), generator=torch.Generator().manual_seed(E)) * 2).to(DEV)
    K = min(E, 8)
    r = moe.moe_router(moe.RouterDesc(16, E, K, renorm=False), z, loss=False)
    one = moe.RouterDesc(1, E, 1)
    got = torch.stack([moe.moe_balance_loss(one, z[t:t + 1], r.topk_idx[t, k].reshape(1, 1)).balance_loss
                       for t in range(16) for k in range(K)]).reshape(16, K)
    want = (r.topk_w.double() * E).float()
    assert torch.equal(got, want), f"{int((got != want).sum())} of {got.numel()} differ"


def _capture(f, n):
    f()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(n):
            f()
    return graph


def test_the_loss_of_many_sequences_takes_time_in_proportion(moe):
    """Four times the sequences take about four times as long (3.8 measured; counting the used sequences in every
    workgroup took 9): at most six."""
    graphs = []
    for G in (2048, 8192):
        desc = moe.RouterDesc(16 * G, 256, 2, seq_len=16)
        z = torch.randn((16 * G, 256), device=DEV)
        r = moe.alloc_router(desc, z.device)
        graphs.append(_capture(lambda: moe.moe_router(desc, z, router=r), 4))
    best = [float("inf")] * 2
    for _ in range(8):
        for i, g in enumerate(graphs):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            g.replay()
            b.record()
            torch.cuda.synchronize()
            best[i] = min(best[i], a.elapsed_time(b))
    assert best[1] < 6 * best[0], best


@pytest.mark.parametrize("G,T,E", [(1023, 3, 16), (1024, 1, 16), (1025, 2, 32), (512, 2, 40), (513, 2, 33), (340, 40, 70),
                                   (1000, 130, 8), (1024, 140, 8)])
def test_sequences_that_count_are_counted(moe, G, T, E):
    """On both sides of where a launch of its own counts them; a third of the sequences have no token that counts."""
    rng = np.random.default_rng(G + T)
    z = rng.standard_normal((G * T, E)).astype(np.float32)
    mask = np.repeat(rng.random(G) < 0.67, T) & (rng.random(G * T) < 0.9)
    idx = rng.integers(0, E, (G * T, 2)).astype(np.int32)
    desc = moe.RouterDesc(G * T, E, 2, seq_len=T)
    r = moe.moe_balance_loss(desc, torch.from_numpy(z).to(DEV), torch.from_numpy(idx).to(DEV), torch.from_numpy(mask).to(DEV))
    ref = router_reference(z.astype(np.float64), 2, seq_len=T, mask=mask, given=idx)
    assert np.array_equal(r.expert_count.cpu().numpy(), ref["count"])
    # a coefficient holds the number of sequences and is rounded once
    assert np.all(np.abs(r.balance_coef.cpu().numpy() - ref["coef"]) <= 2.0 ** -23 * ref["coef"])
    # probabilities within 80 units of 2^-24 (test_gpu_router.py), their sums and the loss a few more
    assert abs(float(r.balance_loss) - ref["loss"]) <= 160 * 2.0 ** -24 * ref["loss"]


@pytest.mark.parametrize("E,S", [(3, 1 << 22), (10, 1 << 21), (250, 1 << 20), (300, 1 << 20), (1000, 1 << 19)])
def test_the_loss_of_a_long_sequence(moe, E, S):
    """Equal logits: every probability is 1/E rounded once and the loss is 1 whatever the routing.  Roundings, half a
    unit (2^-24) each: the probability, a wave's sum, a workgroup's, the loss; sums between them are in 64 bits
    (errors below S * 2^-53 = 2^-31).  Sums of all a wave's tokens in fp32 were off by 15 to 99 such halves here."""
    z = torch.zeros((S, E), dtype=torch.bfloat16, device=DEV)
    idx = torch.randint(0, E, (S, 1), generator=torch.Generator().manual_seed(E), dtype=torch.int32).to(DEV)
    r = moe.moe_balance_loss(moe.RouterDesc(S, E, 1), z, idx)
    assert int(r.expert_count.sum()) == S
    assert abs(float(r.balance_loss) - 1.0) <= 4 * 2.0 ** -24 + 2.0 ** -31


def test_the_loss_of_a_long_sequence_of_near_equal_logits(moe):
    """Logits within 0.1 of each other: a probability has the exponential's one unit (2 halves), its argument's
    rounding (0.1), 6 steps of the sum over the wave and their terms' 2.1, and the quotient's 1; then as above 3."""
    S, E = 1 << 20, 50
    z = torch.rand((S, E), generator=torch.Generator().manual_seed(1)).mul_(0.1).to(DEV)
    idx = torch.randint(0, E, (S, 2), generator=torch.Generator().manual_seed(2), dtype=torch.int32).to(DEV)
    r = moe.moe_balance_loss(moe.RouterDesc(S, E, 2), z, idx)
    count = torch.bincount(idx.flatten(), minlength=E).double()
    p = torch.softmax(z.double(), 1).sum(0)
    want = float((E * count / (2.0 * S) * p / S).sum())
    assert abs(float(r.balance_loss) - want) <= (2.1 + 6 + 2.1 + 1 + 3) * 2.0 ** -24 * want
