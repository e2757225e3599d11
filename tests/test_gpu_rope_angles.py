"""The rotation's angle at far positions, for slow and fast frequencies, against
the exact fraction of a turn (integer arithmetic with 80 digits of pi)."""
import math
from fractions import Fraction

import pytest
import torch

import dynamic_block_sparse_dsa_b200 as dsa

import rope_fp8_reference as ref
from test_gpu_rope_fp8 import BF16_HALF, Batch

pytestmark = pytest.mark.gpu

PI = Fraction(int("314159265358979323846264338327950288419716939937510582097494459230781640628620899"), 10 ** 80)


def exact_angles(pos, inv_freq):
    """[positions][pairs] angles in [0, 2 pi), from the exact product reduced to a turn."""
    return torch.tensor([[float(Fraction(p) * Fraction(f) / (2 * PI) % 1) * 2 * math.pi for f in inv_freq.tolist()]
                         for p in pos], dtype=torch.float64)


POSITIONS = [0, 1, -1, 7, 1048575, 1048577, 2 ** 30 + 12345, 2 ** 31 - 1, -2 ** 31, -2 ** 31 + 1]


@pytest.mark.parametrize("top", [1.0, 2 * math.pi, 10.0, 100.5, 1e4, 2.0 ** 20, -3.25])
def test_far_positions(top, cuda_device):
    """Frequencies from `top` down to top / 1e6, positions over the whole int32 range: within
    the slack of an angle that is right to 2^-24 of a turn."""
    b = Batch((len(POSITIONS),), (len(POSITIONS),), 1, 4, seed=90)
    inv = (top * 1e6 ** (-torch.arange(64, dtype=torch.float64) / 63)).float()
    pos = torch.tensor(POSITIONS, dtype=torch.int64)
    _, cache = b.cache16()
    got = dsa.kv_append_rope(cache, b.seqs, None, None, None, None, dsa.Rotary(inv.cuda()), queries=b.queries, q=b.dq,
                             pos_q=pos.int().cuda()[None], dev_err=b.err).cpu().double()
    assert int(b.err) == 0
    ang = exact_angles(POSITIONS, inv)
    c, s = ang.cos()[:, None], ang.sin()[:, None]
    x, y = b.q.double()[..., :64], b.q.double()[..., 64:]
    # 2^-24 of a turn is 3.8e-7 rad; with cos and sin within 2 ulp and the fp32 products below 2^-19 (|x| + |y|)
    slack = (x.abs() + y.abs()) * 2.0 ** -19
    for part, want in ((got[..., :64], x * c - y * s), (got[..., 64:], y * c + x * s)):
        d = (part - want).abs() - want.abs() * BF16_HALF - slack * (1 + BF16_HALF)
        assert float(d.max()) <= 0, (float(d.max()), divmod(int(d.argmax()) % 64, 64), top)


def test_default_positions_of_a_long_context(cuda_device):
    """The same through the cache positions of an append near 2^21 tokens, both appends, one KV head."""
    n, first = 70, (1 << 21) - 40
    blocks = -(-(first + n) // 64)
    table = torch.full((1, blocks), -1, dtype=torch.int32)
    table[0, first // 64:] = torch.arange(blocks - first // 64, dtype=torch.int32)
    g = torch.Generator().manual_seed(91)
    k = torch.randn(n, 1, 128, generator=g).bfloat16()
    inv = (50.0 * 1e5 ** (-torch.arange(64, dtype=torch.float64) / 63)).float()
    ang = exact_angles(range(first, first + n), inv)
    c, s = ang.cos()[:, None], ang.sin()[:, None]
    x, y = k.double()[..., :64], k.double()[..., 64:]
    want = torch.cat([x * c - y * s, y * c + x * s], dim=-1)[:, 0]
    slack = ((x.abs() + y.abs()) * 2.0 ** -19).repeat(1, 1, 2)[:, 0]
    seqs = dsa.SeqBatch(table.cuda(), torch.tensor([first + n], dtype=torch.int32).cuda())
    cu = torch.tensor([0, n], dtype=torch.int32).cuda()
    at = torch.arange(first, first + n)
    page, slot = table[0, at // 64].long(), at % 64
    for fp8 in (False, True):
        pages = int(table.max()) + 1
        kc = torch.zeros((pages, 64), dtype=torch.int8, device="cuda")
        if fp8:
            pools = [torch.zeros((pages, 64, 1, 128), dtype=torch.uint8, device="cuda") for _ in range(2)]
            scales = [torch.zeros((pages, 1, 1), device="cuda") for _ in range(2)]
            dsa.kv_append_fp8(dsa.PagedKVCacheFP8(*pools, kc, *scales), seqs, cu, k.cuda(), k.cuda(), None,
                              dsa.Rotary(inv.cuda()))
            got = ref.stored(pools[0].cpu(), scales[0].cpu())[page, slot, 0]
            step, floor = 2.0 ** -4, float(scales[0].max()) * 2.0 ** -10
        else:
            pools = [torch.zeros((pages, 64, 1, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
            dsa.kv_append_rope(dsa.PagedKVCache(*pools, kc), seqs, cu, k.cuda(), k.cuda(), None, dsa.Rotary(inv.cuda()))
            got = pools[0].cpu().double()[page, slot, 0]
            step, floor = BF16_HALF, 0.0
        d = (got - want).abs() - want.abs() * step - slack * (1 + step) - floor
        assert float(d.max()) <= 0, (fp8, float(d.max()))
