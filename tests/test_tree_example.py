"""The example that runs the operators together (examples/tree_decode.py): its
tokens are a greedy decoding of its model, recomputed in fp32 by plain torch
over the whole text at once."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu


def test_tree_decoding_is_greedy():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_verification_42_gb300 import build
    build.build()
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import tree_decode as ex
    m = ex.Target()
    lens = torch.tensor([5, 40, 17, 1], dtype=torch.int32, device="cuda")
    ids = torch.randint(0, m.vocab, (4, 40), dtype=torch.int32, device="cuda",
                        generator=torch.Generator(device="cuda").manual_seed(1))
    texts = ex.decode(ids, lens, 12, m)
    assert all(13 <= len(t) <= 37 for t in texts)
    assert sum(len(t) for t in texts) > 4 * 13  # some drafts were accepted

    def unit(x):
        return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6)

    for b in range(4):
        seq = torch.tensor(ids[b, :int(lens[b])].tolist() + texts[b], device="cuda")
        x, n = m.embed[seq].float(), len(seq)
        for i in range(m.layers):
            q, k, v = (unit(x) @ m.qkv[i].float()).split([m.hq * m.d, m.hkv * m.d, m.hkv * m.d], -1)
            q, k, v = (y.unflatten(-1, (-1, m.d)) for y in (q, k, v))

            def turn(y, w):
                y = unit(y) * w.float()
                c, s = m.cos_sin[:n].unsqueeze(1).chunk(2, -1)
                a, z = y.chunk(2, -1)
                return torch.cat([a * c - z * s, z * c + a * s], -1)

            q, k = turn(q, m.norms[i][0]), turn(k, m.norms[i][1])
            k, v = (y.repeat_interleave(m.hq // m.hkv, 1) for y in (k, v))
            s = torch.einsum("qhd,khd->hqk", q, k) * m.d ** -0.5
            s = s.masked_fill(torch.ones(n, n, device="cuda").triu(1).bool(), float("-inf"))
            x = x + torch.einsum("hqk,khd->qhd", s.softmax(-1), v).reshape(n, -1) @ m.proj[i].float()
        logits = unit(x) @ m.head.float()
        # a hidden state's bf16 roundings (some tens of 2^-9 each, of terms of size 1)
        # move a logit of spread 2 by a few hundredths; 0.2 is far above that and far
        # below the spread
        at = int(lens[b]) - 1
        for j, t in enumerate(texts[b]):
            row = logits[at + j]
            assert float(row.max() - row[t]) < 0.2, (b, j, t, float(row.max() - row[t]))
