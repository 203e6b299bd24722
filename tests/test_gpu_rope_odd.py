"""Rotary positions of heads with an odd number of channels: the last one has no
neighbour, and what lies behind a head, a token and the tensor stays.

The bounds are test_gpu_rope's.
"""

import numpy as np
import pytest

from oracle import layer_oracle as lo

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import weight_only_int4_quantize_amd as awq  # noqa: E402

from test_gpu_parity import dev, host, say  # noqa: E402
from test_gpu_rope import check, heads  # noqa: E402


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("D,r,hq,hk,T", [(65, 64, 4, 2, 5), (7, 4, 3, 3, 9), (3, 2, 40, 1, 2), (33, 16, 2, 1, 70), (129, 32, 8, 8, 1),
                                         (4095, 64, 1, 1, 2), (4095, 4094, 1, 2, 1)])
def test_odd_heads(D, r, hq, hk, T, layout):
    say("rope odd", layout, D, r)
    rng, q, k = heads([31, D, r], T, hq, hk, D)
    pos = rng.integers(0, 100000, T).astype(np.int32)
    f, _ = lo.rope_frequencies(r)
    rope = awq.Rope(r, layout=layout)
    qo, ko = awq.awq_rope(dev(q), dev(k), rope, dev(pos))
    check(host(qo), q, pos, f, layout)
    check(host(ko), k, pos, f, layout)
    for h, x, want in ((hq, q, qo), (hk, k, ko)):
        wide = torch.full((T + 1, h + 1, D + 3), 9.0, dtype=torch.float16, device="cuda")
        out = wide[:T, :h, :D]
        awq.awq_rope(dev(x), None, rope, dev(pos), out=(out, None))
        assert torch.equal(out, want)
        inside = torch.zeros_like(wide, dtype=torch.bool)
        inside[:T, :h, :D] = True
        assert (wide[~inside] == 9).all()
        out.copy_(dev(x))
        awq.awq_rope(out, None, rope, dev(pos), out=(out, None))     # in place
        assert torch.equal(out, want) and (wide[~inside] == 9).all()
        # by the batch's positions, every token a sequence
        table = torch.zeros(T, 0, dtype=torch.int32, device="cuda")
        s = awq.KVSeqs(table, torch.arange(T + 1, device="cuda", dtype=torch.int32), dev(pos + 1), 1, 100001)
        wide.fill_(9.0)
        awq.awq_rope(dev(x), None, rope, seqs=s, out=(out, None))
        assert torch.equal(out, want) and (wide[~inside] == 9).all()
